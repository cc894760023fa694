"""The bench's record of DRAM bytes goes with the sources of the kernel that it was taken of."""
import os

import bench
from test_bench_host import _digest, _tree

SOURCES = {"a.cu": '#include "x.h"\n__global__ void my_kernel(int a)\n', "x.h": '#include <cuda.h>\n#include "y.cuh"\n',
           "y.cuh": "// y\n", "b.cu": '#include "x.h"\n// like my_kernel, but another\n', "z.h": "// z\n"}


def test_other_kernels_sources_do_not_count(tmp_path):
    mine = {n: SOURCES[n] for n in ("a.cu", "x.h", "y.cuh")}
    csrc = _tree(tmp_path, SOURCES, [
        f"kernel=my_kernel workload=w source_sha={_digest(mine)} dram_bytes_per_launch=1234"])
    root = str(tmp_path)
    assert bench.kernel_sources("my_kernel", str(csrc)) == sorted(mine)
    assert bench.traffic_record("my_kernel", "w", root) == 1234.0
    for name in ("b.cu", "z.h"):
        (csrc / name).write_text("// changed\n")
    (csrc / "new.cu").write_text("// new\n")
    assert bench.traffic_record("my_kernel", "w", root) == 1234.0
    for name in mine:                                            # its own do
        (csrc / name).write_text(SOURCES[name] + "// changed\n")
        assert bench.traffic_record("my_kernel", "w", root) is None
        (csrc / name).write_text(SOURCES[name])
    assert bench.kernel_sources("no_such_kernel", str(csrc)) == sorted(os.listdir(csrc))


def test_the_gemm_kernels_record_is_of_its_sources():
    csrc = os.path.join(bench.ROOT, "mixed_precision_tensor_gb300", "csrc")
    assert bench.kernel_sources("tcg_gemm_kernel", csrc) == ["tcg_internal.h", "tcg_kernels.cu", "tcg_pipe.cuh",
                                                             "tcg_ptx.cuh"]
