// tcg_lm_norm.cu -- root-mean-square norm of the language-model calls (sm_103a).
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//
// with s kept for the residual stream, y rounded to 16 bits, or to E4M3 with a scale per row:
// scale = max |y| / 448.  max |y| is r max |s w|, so one pass over the registers gives both
// the sum of squares and the maximum, and a row is joined across its threads once.  Gradient:
//
//   g = dy w,  dx = r g - s r^3 mean(g s) + ds,  dw = sum over rows of dy s r
//
// Again one join a row, of (sum s^2, sum g s).  A thread owns the same columns of every row that
// its block takes, so dw stays in registers until the block's last row; the blocks' sums are
// joined in block order by a second kernel: the order depends only on the sizes.
//
// Bound by memory: every element is read once and written once, 16 bytes a thread.  A row's
// elements stay in registers as they were read (V pieces of eight a thread); s, its square and y
// are formed in FP32 from them.  16384 x 4096 in a graph: 81 us with a residual kept (6.6 TB/s, 98% of
// the copy rate), 76 in 8 bits (6.1), 44 without a residual (6.0); backward 102 (5.2), dx alone 93.

#include <cuda_fp8.h>

#include "tcg_lm_math.cuh"

namespace tcg {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100

// A row's threads hold 16 columns each (8 up to 256 columns, 32 beyond 16384): a warp, eight rows to a
// block, for up to 512 columns, a block for more.
constexpr int kNormRows = 8;
struct NormShape {
    int v, threads, rows;                       // pieces a thread, threads a row, rows of a block
};

NormShape norm_shape(int64_t k)
{
    const int64_t pieces = (k + 7) / 8;
    const int v = pieces <= 32 ? 1 : (pieces <= 2048 ? 2 : 4);
    const int threads = static_cast<int>((pieces + 32 * v - 1) / (32 * v) * 32);
    return {v, threads, threads == 32 ? kNormRows : 1};
}

// Eight elements of a row, those from `left` on zero.
__device__ __forceinline__ uint4 load_piece(const uint16_t *p, int left)
{
    if (left >= 8)
        return *reinterpret_cast<const uint4 *>(p);
    uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left)
            u[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <bool BF16>
__device__ __forceinline__ void store_piece(uint16_t *p, int left, const float (&x)[8])
{
    if (left >= 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack16(x[0], x[1], BF16), pack16(x[2], x[3], BF16),
                                                   pack16(x[4], x[5], BF16), pack16(x[6], x[7], BF16));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left)
            p[i] = round16(x[i], BF16);
}

__device__ __forceinline__ void store_piece8(uint8_t *p, int left, const float (&x)[8])
{
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        u[i] = lo | hi << 16;
    }
    if (left >= 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left)
            p[i] = static_cast<uint8_t>(u[i / 4] >> (8 * (i & 3)));
}

// The weights of a piece, zero past the row's end.
template <bool BF16>
__device__ __forceinline__ void load_weight(const void *w, int w_f32, int64_t i, int left, float (&x)[8])
{
    if (!w_f32) {
        unpack16<BF16>(load_piece(static_cast<const uint16_t *>(w) + i, left), x);
        return;
    }
    const float *f = static_cast<const float *>(w) + i;
    if (left >= 8) {
        const float4 a = reinterpret_cast<const float4 *>(f)[0], b = reinterpret_cast<const float4 *>(f)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = j < left ? f[j] : 0.0f;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Sums of a, and sums or maxima of b, over a row's threads (a block, or a warp).  `room` alternates from row to row,
// so that one barrier a row is enough.
template <bool MAX_B, bool ONE>
__device__ __forceinline__ void join_row(float2 (*part)[32], int room, float &a, float &b)
{
    auto both = [&](float oa, float ob) {
        a += oa;
        b = MAX_B ? max_nan(b, ob) : b + ob;
    };
#pragma unroll
    for (int d = 16; d; d >>= 1)
        both(__shfl_xor_sync(0xffffffffu, a, d), __shfl_xor_sync(0xffffffffu, b, d));
    if constexpr (ONE) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
            part[room][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 p = lane < warps ? part[room][lane] : make_float2(0.0f, 0.0f);
        a = p.x;
        b = p.y;
#pragma unroll
        for (int d = 16; d; d >>= 1)
            both(__shfl_xor_sync(0xffffffffu, a, d), __shfl_xor_sync(0xffffffffu, b, d));
    }
}

// ONE: a row has the block to itself.  RES: with a residual.  Without one a thread has the next row on its way while it finishes a row (16384
// x 4096: 54 us without that); with one a row is enough to keep memory busy, and two take registers
// that hold blocks.
template <int V, bool BF16, bool OUT8, bool RES, bool ONE>
__global__ void __launch_bounds__(1024) tcg_norm_kernel(const NormArgs p)
{
    __shared__ float2 part[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int t = ONE ? threadIdx.x : threadIdx.x & 31, per_row = ONE ? blockDim.x : 32;
    const int at_once = ONE ? 1 : kNormRows, mine_of = ONE ? 0 : threadIdx.x >> 5;
    const int64_t step = static_cast<int64_t>(gridDim.x) * at_once;
    const float inv_k = 1.0f / static_cast<float>(p.k);
    uint4 vx[V], vr[V], next[V];
    auto load = [&](const void *base, int64_t ld, int64_t row, uint4 (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            v[i] = load_piece(static_cast<const uint16_t *>(base) + row * ld + c, p.k - c);
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + mine_of;
    if (!RES && row < p.rows)
        load(p.X, p.ldx, row, next);
    int room = 0;
    for (; row < p.rows; row += step, room ^= 1) {
        if constexpr (RES) {
            load(p.X, p.ldx, row, vx);
            load(p.R, p.ldr, row, vr);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                vx[i] = next[i];
            if (row + step < p.rows)
                load(p.X, p.ldx, row + step, next);
        }
        auto sum_of = [&](int i, float (&s)[8]) {
            unpack16<BF16>(vx[i], s);
            if constexpr (RES) {
                float r[8];
                unpack16<BF16>(vr[i], r);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] += r[j];
            }
        };
        float ss = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            float s[8];
            sum_of(i, s);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = fmaf(s[j], s[j], ss);
            if (OUT8) {
                float w[8];
                load_weight<BF16>(p.W, p.w_f32, c, p.k - c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = max_nan(top, fabsf(s[j] * w[j]));
            }
            if (p.S)
                store_piece<BF16>(static_cast<uint16_t *>(p.S) + row * p.lds + c, p.k - c, s);
        }
        join_row<true, ONE>(part, room, ss, top);
        const float r = rsqrtf(fmaf(ss, inv_k, p.eps));
        float inv = 1.0f;
        if (OUT8) {
            const float scale = max_nan(top * r * (1.0f / kE4m3Max), kMinScale);
            inv = 1.0f / scale;
            if (t == 0)
                p.scale[row] = scale;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            float s[8], w[8];
            sum_of(i, s);
            load_weight<BF16>(p.W, p.w_f32, c, p.k - c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = s[j] * r * w[j];
                if (OUT8)
                    s[j] *= inv;
            }
            if (OUT8)
                store_piece8(static_cast<uint8_t *>(p.Y) + row * p.ldy + c, p.k - c, s);
            else
                store_piece<BF16>(static_cast<uint16_t *>(p.Y) + row * p.ldy + c, p.k - c, s);
        }
    }
}

// ONE: a row is a block of its own.  Blocks of up to 256 threads (FEW) are three to an SM, so that a
// thread has registers for its columns of dw and a row of three tensors: 16384 x 4096 takes 102 us so,
// 103 with four blocks of 64 registers and a few values in memory, 185 with more of them there.
constexpr int kFewThreads = 256;
template <int V, bool BF16, bool ONE, bool FEW>
__global__ void __launch_bounds__(FEW ? kFewThreads : 1024, FEW ? 3 : 1)
    tcg_norm_backward_kernel(const NormBackwardArgs p)
{
    extern __shared__ float rows_dw[];          // at the end: dw of each of the block's rows' threads
    __shared__ float2 part[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int t = ONE ? threadIdx.x : threadIdx.x & 31, per_row = ONE ? blockDim.x : 32;
    const int at_once = ONE ? 1 : kNormRows, mine_of = ONE ? 0 : threadIdx.x >> 5;
    const int64_t step = static_cast<int64_t>(gridDim.x) * at_once;
    const float inv_k = 1.0f / static_cast<float>(p.k);
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.0f;
    int room = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + mine_of; row < p.rows; row += step, room ^= 1) {
        uint4 vx[V], vd[V], vs[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            vx[i] = load_piece(static_cast<const uint16_t *>(p.X) + row * p.ldx + c, p.k - c);
            vd[i] = load_piece(static_cast<const uint16_t *>(p.dY) + row * p.lddy + c, p.k - c);
            if (p.dS)
                vs[i] = load_piece(static_cast<const uint16_t *>(p.dS) + row * p.ldds + c, p.k - c);
        }
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            float x[8], d[8], w[8];
            unpack16<BF16>(vx[i], x);
            unpack16<BF16>(vd[i], d);
            load_weight<BF16>(p.W, p.w_f32, c, p.k - c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(x[j], x[j], ss);
                dot = fmaf(d[j] * w[j], x[j], dot);
            }
        }
        join_row<false, ONE>(part, room, ss, dot);
        const float r = rsqrtf(fmaf(ss, inv_k, p.eps));
        const float m = r * r * (dot * inv_k);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * per_row + t) * 8;
            float x[8], d[8], w[8];
            unpack16<BF16>(vx[i], x);
            unpack16<BF16>(vd[i], d);
            load_weight<BF16>(p.W, p.w_f32, c, p.k - c, w);
            if (p.part) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dw[i][j] = fmaf(d[j], x[j] * r, dw[i][j]);
            }
            if (p.dX) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] = r * fmaf(-x[j], m, d[j] * w[j]);
                if (p.dS) {
                    float s[8];
                    unpack16<BF16>(vs[i], s);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        d[j] += s[j];
                }
                store_piece<BF16>(static_cast<uint16_t *>(p.dX) + row * p.lddx + c, p.k - c, d);
            }
        }
    }
    if (!p.part)
        return;
    float *out = p.part + static_cast<int64_t>(blockIdx.x) * p.k, *mine = at_once > 1 ? rows_dw + mine_of * p.k : out;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((i * per_row + t) * 8 + j < p.k)
                mine[(i * per_row + t) * 8 + j] = dw[i][j];
    if (at_once > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < p.k; c += blockDim.x) {
            float s = 0.0f;
            for (int q = 0; q < at_once; ++q)
                s += rows_dw[q * p.k + c];
            out[c] = s;
        }
    }
}

// dw = the blocks' sums, in block order: 32 columns a block, every 32nd of the blocks a warp.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    tcg_norm_join_kernel(const float *__restrict__ part, int blocks, int k, float *__restrict__ dw)
{
    __shared__ float join[kJoinWarps][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < k) {
        for (int b = warp; b < blocks; b += 8 * kJoinWarps) {            // eight loads at a time
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = b + j * kJoinWarps;
                v[j] = at < blocks ? __ldcg(part + static_cast<int64_t>(at) * k + c) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[j];
        }
    }
    join[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < k) {
#pragma unroll
        for (int i = 1; i < kJoinWarps; ++i)
            s += join[i][lane];
        dw[c] = s;
    }
}

template <int V, bool OUT8, bool ONE>
cudaError_t norm_o(const NormArgs &a, const NormShape &n, int grid, cudaStream_t s)
{
    auto fn = a.R ? (a.in_bf16 ? tcg_norm_kernel<V, true, OUT8, true, ONE> : tcg_norm_kernel<V, false, OUT8, true, ONE>)
                  : (a.in_bf16 ? tcg_norm_kernel<V, true, OUT8, false, ONE> : tcg_norm_kernel<V, false, OUT8, false, ONE>);
    return launch_pdl(fn, dim3(grid), dim3(n.threads * n.rows), s, 0, a);
}

template <int V, bool ONE>
cudaError_t norm_v(const NormArgs &a, const NormShape &n, int grid, cudaStream_t s)
{
    return a.out8 ? norm_o<V, true, ONE>(a, n, grid, s) : norm_o<V, false, ONE>(a, n, grid, s);
}

template <int V, bool ONE, bool FEW>
cudaError_t norm_backward_v(const NormBackwardArgs &a, const NormShape &n, int grid, cudaStream_t s)
{
    const size_t smem = a.part && !ONE ? n.rows * a.k * sizeof(float) : 0;            // at most 16 KiB
    return launch_pdl(a.in_bf16 ? tcg_norm_backward_kernel<V, true, ONE, FEW> : tcg_norm_backward_kernel<V, false, ONE, FEW>,
                      dim3(grid), dim3(n.threads * n.rows), s, smem, a);
}

// Blocks that are resident with `threads` an SM.
int norm_grid(const NormShape &n, int64_t rows, int num_sms, int threads)
{
    const int64_t need = rows / n.rows + (rows % n.rows != 0);
    const int64_t most = static_cast<int64_t>(num_sms) * (threads / (n.threads * n.rows));
    return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t s)
{
    const NormShape n = norm_shape(a.k);
    const int grid = norm_grid(n, a.rows, num_sms, 1024);        // of 64 registers
    return n.v == 1 ? norm_v<1, false>(a, n, grid, s)
         : n.v == 4 ? norm_v<4, true>(a, n, grid, s)
         : n.rows > 1 ? norm_v<2, false>(a, n, grid, s) : norm_v<2, true>(a, n, grid, s);
}

int norm_backward_blocks(int64_t rows, int64_t k, int num_sms)
{
    const NormShape n = norm_shape(k);
    return norm_grid(n, rows, num_sms, n.threads > kFewThreads ? 1024 : 3 * kFewThreads);
}

cudaError_t launch_norm_backward(NormBackwardArgs a, float *dw, int num_sms, cudaStream_t s)
{
    const NormShape n = norm_shape(a.k);
    const int blocks = norm_backward_blocks(a.rows, a.k, num_sms);
    if (blocks == 1)                            // nothing to join
        a.part = dw;
    cudaError_t e = cudaSuccess;
    if (blocks > 0)
        e = n.v == 1 ? norm_backward_v<1, false, true>(a, n, blocks, s)
          : n.v == 4 ? norm_backward_v<4, true, false>(a, n, blocks, s)
          : n.rows > 1 ? norm_backward_v<2, false, true>(a, n, blocks, s)
          : n.threads <= kFewThreads ? norm_backward_v<2, true, true>(a, n, blocks, s)
                                     : norm_backward_v<2, true, false>(a, n, blocks, s);
    if (e == cudaSuccess && dw && blocks != 1)  // without rows: zeros
        e = launch_pdl(tcg_norm_join_kernel, dim3((a.k + 31) / 32), dim3(32 * kJoinWarps), s, 0, a.part, blocks,
                       a.k, dw);
    return e;
}

}  // namespace tcg
