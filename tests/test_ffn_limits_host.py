"""Sizes at the ends of their range in the feed-forward calls and their workspace queries, without a GPU."""
import ctypes

import pytest

import mixed_precision_tensor_gb300 as tcg
from test_ffn_host import (E4M3, F32, INV, NSUP, PA, PB, PD, PX, gated, gated_backward, handle,  # noqa: F401
                           norm, norm_backward, packed)

HUGE = (1 << 31, (1 << 61) + 8, 1 << 62, (1 << 63) - 8, (1 << 63) - 1)


@pytest.mark.parametrize("size", HUGE)
def test_products_refuse_huge_sizes(handle, size):  # noqa: F811
    ld = size // 8 * 8
    for kw in (dict(m=size, ldd=ld), dict(n=size), dict(k=size, lda=ld, ldb=ld)):
        assert gated(handle, **kw) in (INV, NSUP)
        assert packed(handle, **kw) in (INV, NSUP)
    for kw in (dict(m=size, lddd=ld, ldz=ld), dict(n=size), dict(k=size, ldw=ld, ldx=ld, lddx=ld, lddw=ld)):
        assert gated_backward(handle, **kw) in (INV, NSUP)
    # where leading dimensions are as large, so that only the size itself is in the way
    top = (1 << 63) - 16
    assert gated(handle, m=1 << 62, ldd=top) == NSUP
    assert packed(handle, m=1 << 62, ldd=top) == NSUP
    assert packed(handle, k=1 << 62, lda=top, ldb=top) == NSUP
    assert packed(handle, m=1 << 62, ldd=top, gate=1) == NSUP
    assert packed(handle, k=(1 << 63) - 1, lda=top, ldb=top) == INV          # ldb < k


@pytest.mark.parametrize("size", HUGE)
def test_workspace_queries_refuse_huge_sizes(handle, size):  # noqa: F811
    bytes_ = ctypes.c_size_t(77)
    lib = tcg.load_library()
    for m, n, k in ((size, 1, 8), (1, size, 8), (1, 1, size), (size, size, size)):
        assert lib.tcg_gemm_gated_workspace_size(handle, m, n, k, bytes_) == NSUP
        assert lib.tcg_gated_backward_workspace_size(handle, m, n, k, 1, 1, bytes_) == NSUP
        for gate in (0, 1):
            assert lib.tcg_gemm_4bit_workspace_size(handle, m, n, k, gate, bytes_) == NSUP
    assert bytes_.value == 77


@pytest.mark.parametrize("ld", [(1 << 61) + 1, (1 << 62) + 2, (1 << 63) - 1])
def test_leading_dimensions_past_the_range_of_bytes(handle, ld):  # noqa: F811
    """No multiple of 16 bytes, though its bytes wrap to one or to none."""
    assert gated(handle, lda=ld) == INV and gated(handle, ldb=ld) == INV
    assert packed(handle, ldb=ld) == INV
    assert packed(handle, dt=F32, ldd=ld) == INV


@pytest.mark.parametrize("kw", [
    dict(S=PD), dict(S=PA, Y=PA), dict(R=PB, S=PB, Y=PB),                       # both outputs in one place
    dict(yt=E4M3, scale=PX, Y=PA), dict(yt=E4M3, scale=PX, R=PB, Y=PB),         # bytes over 16-bit rows
    dict(Y=PA, ldy=72), dict(S=PA, lds=72), dict(R=PB, S=PB, lds=128), dict(R=PB, Y=PB, ldy=72),
])
def test_norm_refuses_places(handle, kw):  # noqa: F811
    """In place only where rows stay where they are."""
    assert norm(handle, **kw) == INV


@pytest.mark.parametrize("kw", [dict(dX=PA, lddx=72), dict(dS=PX, dX=PX, lddx=72), dict(dX=PB, lddx=128)])
def test_norm_backward_refuses_places(handle, kw):  # noqa: F811
    assert norm_backward(handle, **kw) == INV


def test_packed_product_refuses_places(handle):  # noqa: F811
    assert packed(handle, ldd=72, e=tcg.Epilogue(beta=1.0, C=PD, ldc=64)) == INV
