// tcg_lm_w4.cu -- products of a few tokens with 4-bit weights (sm_103a).
//
//   z[t][f] = sum over groups of s[f][g] (sum over k of g of (q[f][k] - zero[f][g]) x[t][k])
//
// Bound by memory: half a byte a weight for 2 T operations.  Turning a weight into a number costs
// more instructions than multiplying it, so a warp does that once for eight tokens or more:
// q - 8, exact in 16 bits, is the A operand of mma.m16n8k16, the tokens are its eight columns
// (tcgen05 would want the weights back in shared memory first, and 128 rows of them).  Sums are
// FP32.  A group's sum is scaled in FP32 when it is complete; with zeros, (8 - zero) times the
// group's sum of x, which one more product with a matrix of ones gives, is added.
//
// A warp has 32 rows and streams them 128 elements at a time through a ring of its own
// (asynchronous 16-byte copies; rows 80 bytes apart, so that the words that eight rows' lanes want
// lie in different banks).  Its lane c of a quad takes elements 8 c .. 8 c + 7 of each 32: in a word
// elements j and j + 4 are 16 bits apart, so one mask gives the pair (j, j + 4); x is paired to
// match.  The warps of a block, and the blocks of a cluster, share the elements of the same rows;
// sums are joined through (distributed) shared memory in a fixed order.

#include "tcg_lm_math.cuh"

namespace tcg {

namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Rows = 32;                         // rows of a warp, and of a block
constexpr int kW4K = 128;                           // elements of a stage
constexpr int kW4RowBytes = kW4K / 2 + 16;          // in the ring
constexpr int kW4StageBytes = kW4Rows * kW4RowBytes;
constexpr int kW4Stages = 4;
constexpr int kW4RingBytes = kW4Warps * kW4Stages * kW4StageBytes;
constexpr int kW4Stride = kW4Rows + 4;              // of a token's sums: no bank conflicts

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// q - 8 of the eight elements of a word: pairs (0, 4), (1, 5), (2, 6), (3, 7).  A nibble below an
// exponent of its own is 128 + q in BF16, and in FP16 1024 + q or, four bits up, 1024 + 16 q;
// taking the constant away is exact.
template <bool BF16>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&q)[4])
{
    if constexpr (BF16) {
        const uint32_t off = 0x43084308u;           // 136
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
            const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&off));
            q[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    } else {
        const uint32_t off = 0x64086408u, sixteenth = 0x2C002C00u, off16 = 0xD480D480u;   // 1032, 1/16, -72
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t u = w >> (4 * i);
            const uint32_t lo = (u & 0x000F000Fu) | 0x64006400u, hi = (u & 0x00F000F0u) | 0x64006400u;
            const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), *reinterpret_cast<const __half2 *>(&off));
            const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&hi),
                                      *reinterpret_cast<const __half2 *>(&sixteenth),
                                      *reinterpret_cast<const __half2 *>(&off16));
            q[i] = *reinterpret_cast<const uint32_t *>(&a);
            q[i + 1] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
}

// Row j of a block's 32 in the weights: of a gated product 16 rows of g, then their 16 of u.  Rows
// past the end repeat the last one.
__device__ __forceinline__ int64_t w4_row(const W4Args &p, int64_t tile, int j)
{
    if (!p.gated) {
        const int64_t r = tile * kW4Rows + j;
        return r < p.rows ? r : p.rows - 1;
    }
    const int64_t n = p.rows / 2, f = tile * (kW4Rows / 2) + j % (kW4Rows / 2);
    return (f < n ? f : n - 1) + (j < kW4Rows / 2 ? 0 : n);
}

// A scale or zero as it is stored, and its value.
__device__ __forceinline__ uint32_t load_raw(const void *s, int64_t i, int f32)
{
    return f32 ? static_cast<const uint32_t *>(s)[i] : static_cast<const uint16_t *>(s)[i];
}
template <bool BF16>
__device__ __forceinline__ float raw_value(uint32_t v, int f32)
{
    return f32 || BF16 ? __uint_as_float(f32 ? v : v << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(v)));
}

__device__ __forceinline__ float load_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int NT, bool BF16, bool ZEROS>
__global__ void __launch_bounds__(kW4Warps * 32) tcg_w4_kernel(const W4Args p, int cluster)
{
    extern __shared__ __align__(128) uint8_t ring[];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x % cluster;
    const int64_t tile = blockIdx.x / cluster;
    const int tok0 = blockIdx.y * (8 * NT);
    const int64_t bytes = (p.k + 1) / 2;
    const int units = static_cast<int>((p.k + kW4K - 1) / kW4K);
    const int stride = cluster * kW4Warps, first = rank * kW4Warps + warp;
    const int groups = static_cast<int>((p.k + p.group - 1) / p.group), per = p.group / 32;

    // Copies: lane l brings pieces l % 4 of rows l / 4 + 8 i.
    uint8_t *mine = ring + warp * (kW4Stages * kW4StageBytes);
    const uint8_t *src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        src[i] = p.W + w4_row(p, tile, g + 8 * i) * p.ldw;
    const uint32_t dst0 = smem_u32(mine) + g * kW4RowBytes + c * 16;
    auto produce = [&](int unit, int stage) {
        if (unit < units) {
            const int64_t at = static_cast<int64_t>(unit) * (kW4K / 2) + c * 16, left = bytes - at;
            const int n = left >= 16 ? 16 : (left > 0 ? static_cast<int>(left) : 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 dst0 + stage * kW4StageBytes + i * 8 * kW4RowBytes),
                             "l"(src[i] + (n ? at : 0)), "r"(n)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // x of this lane's column, eight elements of 32.
    auto load_x = [&](int64_t k, int nt) {
        const int t = tok0 + nt * 8 + g;
        const int64_t at = k + 8 * c, left = p.k - at;
        uint32_t u[4] = {0u, 0u, 0u, 0u};
        if (t < p.tokens && left > 0) {
            const uint16_t *x = static_cast<const uint16_t *>(p.X) + t * p.ldx + at;
            if (left >= 8)
                return *reinterpret_cast<const uint4 *>(x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    u[i / 2] |= static_cast<uint32_t>(x[i]) << (16 * (i & 1));
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    int64_t srow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        srow[i] = w4_row(p, tile, g + 8 * i) * groups;

    uint4 xv[4][NT];
    uint32_t sv[4][4], zv[4][4];
    auto load_unit = [&](int unit, int q) {                  // the 32 elements q of a unit
        const int64_t k = static_cast<int64_t>(unit) * kW4K + q * 32;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            xv[q][nt] = load_x(k, nt);
        if ((q & (per - 1)) == per - 1 && unit < units) {    // where a group ends
            const int gi = min(static_cast<int>(k / p.group), groups - 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sv[q][i] = load_raw(p.scales, srow[i] + gi, p.s_f32);
                if (ZEROS)
                    zv[q][i] = load_raw(p.zeros, srow[i] + gi, p.s_f32);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < kW4Stages - 1; ++s)
        produce(first + s * stride, s);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        load_unit(first, q);

    float tot[2][NT][4], acc[2][NT][4], sx[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tot[0][nt][i] = tot[1][nt][i] = 0.0f;
            acc[0][nt][i] = acc[1][nt][i] = 0.0f;
            sx[nt][i] = 0.0f;
        }
    int stage = 0;
    for (int unit = first; unit < units; unit += stride) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kW4Stages - 2) : "memory");
        __syncwarp();                                        // and every lane has read the stage before
        produce(unit + (kW4Stages - 1) * stride, stage == 0 ? kW4Stages - 1 : stage - 1);
        const uint8_t *st = mine + stage * kW4StageBytes + g * kW4RowBytes + c * 4;
        stage = stage + 1 == kW4Stages ? 0 : stage + 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t b[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 x = xv[q][nt];
                b[nt][0] = __byte_perm(x.x, x.z, 0x5410);
                b[nt][1] = __byte_perm(x.x, x.z, 0x7632);
                b[nt][2] = __byte_perm(x.y, x.w, 0x5410);
                b[nt][3] = __byte_perm(x.y, x.w, 0x7632);
            }
            const uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
            const uint32_t ones[4] = {one, one, one, one};
            if (ZEROS) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816<BF16>(sx[nt], ones, b[nt][0], b[nt][1]);
                    mma16816<BF16>(sx[nt], ones, b[nt][2], b[nt][3]);
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t lo[4], hi[4];
                widen<BF16>(*reinterpret_cast<const uint32_t *>(st + (16 * m) * kW4RowBytes + q * 16), lo);
                widen<BF16>(*reinterpret_cast<const uint32_t *>(st + (16 * m + 8) * kW4RowBytes + q * 16), hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816<BF16>(acc[m][nt], a0, b[nt][0], b[nt][1]);
                    mma16816<BF16>(acc[m][nt], a1, b[nt][2], b[nt][3]);
                }
            }
            if ((q & (per - 1)) == per - 1) {                // the group is complete
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float s0 = raw_value<BF16>(sv[q][2 * m], p.s_f32);
                    const float s1 = raw_value<BF16>(sv[q][2 * m + 1], p.s_f32);
                    float z0 = 0.0f, z1 = 0.0f;
                    if (ZEROS) {
                        z0 = 8.0f - raw_value<BF16>(zv[q][2 * m], p.s_f32);
                        z1 = 8.0f - raw_value<BF16>(zv[q][2 * m + 1], p.s_f32);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v = acc[m][nt][i];
                            if (ZEROS)
                                v = fmaf(i < 2 ? z0 : z1, sx[nt][i & 1], v);
                            tot[m][nt][i] = fmaf(i < 2 ? s0 : s1, v, tot[m][nt][i]);
                            acc[m][nt][i] = 0.0f;
                        }
                }
                if (ZEROS) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sx[nt][i] = 0.0f;
                }
            }
            load_unit(unit + stride, q);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    // The warps' sums, [warp][token][row] in the ring, then the block's, [token][row].
    constexpr int kSums = 8 * NT * kW4Stride;
    float *part = reinterpret_cast<float *>(ring);
    float *red = part + kW4Warps * kSums;
    static_assert((kW4Warps + 1) * kSums * 4 <= kW4RingBytes, "the sums fit the ring");
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp * kSums + (nt * 8 + 2 * c + (i & 1)) * kW4Stride + 16 * m + 8 * (i >> 1) + g] = tot[m][nt][i];
    __syncthreads();
    constexpr int kOuts = 8 * NT * kW4Rows;
#pragma unroll
    for (int o = threadIdx.x; o < kOuts; o += kW4Warps * 32) {
        const int at = o / kW4Rows * kW4Stride + o % kW4Rows;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w)
            v += part[w * kSums + at];
        red[at] = v;
    }
    if (cluster > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (rank == 0) {
        auto total = [&](int at) {
            float v = red[at];
            for (int r = 1; r < cluster; ++r)
                v += load_cluster(mapa_shared(smem_u32(red + at), r));
            return v;
        };
        const int rows = p.gated ? kW4Rows / 2 : kW4Rows;
        const int64_t feats = p.gated ? p.rows / 2 : p.rows;
        for (int o = threadIdx.x; o < 8 * NT * rows; o += kW4Warps * 32) {
            const int t = tok0 + o / rows, j = o % rows;
            const int64_t f = tile * rows + j;
            if (t >= p.tokens || f >= feats)
                continue;
            const int at = o / rows * kW4Stride + j;
            float z = total(at);
            if (p.bias)
                z += p.bias_f32 ? static_cast<const float *>(p.bias)[f] : load16(p.bias, f, BF16);
            z = act_of(p.act, z);
            if (p.gated)
                z *= total(at + kW4Rows / 2);
            if (p.C)
                z = fmaf(p.beta, load_out(p.C, t * p.ldc + f, p.out_kind), z);
            store_out(p.D, t * p.ldd + f, p.out_kind, z);
        }
    }
    if (cluster > 1)
        cluster_sync_all();                                  // the others' sums have been read
}

// 32 elements of a row a thread: FP32, rounded once.
template <bool BF16>
__global__ void __launch_bounds__(256) tcg_w4_expand_kernel(const W4Args p, uint16_t *out, int64_t ldo)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t per = (p.k + 31) / 32, total = p.rows * per, groups = (p.k + p.group - 1) / p.group;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int64_t row = i / per, k = (i - row * per) * 32, g = row * groups + k / p.group;
        const uint8_t *w = p.W + row * p.ldw + k / 2;
        const float s = raw_value<BF16>(load_raw(p.scales, g, p.s_f32), p.s_f32);
        const float z = p.zeros ? raw_value<BF16>(load_raw(p.zeros, g, p.s_f32), p.s_f32) : 8.0f;
        uint16_t *o = out + row * ldo + k;
        if (p.k - k >= 32) {
            const uint4 v = *reinterpret_cast<const uint4 *>(w);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = pack16((static_cast<float>(u[j] >> (8 * e) & 15u) - z) * s,
                                  (static_cast<float>(u[j] >> (8 * e + 4) & 15u) - z) * s, BF16);
                reinterpret_cast<uint4 *>(o)[j] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        } else {
            for (int j = 0; j < static_cast<int>(p.k - k); ++j)
                o[j] = round16((static_cast<float>(w[j / 2] >> (4 * (j & 1)) & 15) - z) * s, BF16);
        }
    }
}

template <int NT, bool BF16, bool ZEROS>
cudaError_t launch_nt(const W4Args &a, int cluster, dim3 grid, cudaStream_t s)
{
    auto fn = tcg_w4_kernel<NT, BF16, ZEROS>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4RingBytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kW4Warps * 32);
    cfg.dynamicSmemBytes = kW4RingBytes;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, fn, a, cluster);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_types(const W4Args &a, int cluster, dim3 grid, cudaStream_t s)
{
    if (a.in_bf16)
        return a.zeros ? launch_nt<NT, true, true>(a, cluster, grid, s) : launch_nt<NT, true, false>(a, cluster, grid, s);
    return a.zeros ? launch_nt<NT, false, true>(a, cluster, grid, s) : launch_nt<NT, false, false>(a, cluster, grid, s);
}

}  // namespace

cudaError_t launch_w4(const W4Args &a, int num_sms, cudaStream_t s)
{
    const int64_t tiles = a.gated ? (a.rows / 2 + kW4Rows / 2 - 1) / (kW4Rows / 2) : (a.rows + kW4Rows - 1) / kW4Rows;
    const int64_t units = (a.k + kW4K - 1) / kW4K;
    const int nt = a.tokens <= 8 ? 1 : (a.tokens <= 16 ? 2 : 4);
    const int blocks = (a.tokens + 8 * nt - 1) / (8 * nt);
    // As many blocks to a tile as leave each warp a stage, up to two blocks an SM in all.
    int cluster = 1;
    while (cluster < 8 && units >= 2 * cluster * kW4Warps && tiles * blocks * cluster * 2 <= 2 * num_sms)
        cluster *= 2;
    const dim3 grid(static_cast<unsigned>(tiles * cluster), static_cast<unsigned>(blocks));
    return nt == 1 ? launch_types<1>(a, cluster, grid, s)
         : nt == 2 ? launch_types<2>(a, cluster, grid, s) : launch_types<4>(a, cluster, grid, s);
}

cudaError_t launch_w4_expand(const W4Args &a, void *out, int64_t ldo, int num_sms, cudaStream_t s)
{
    const int64_t blocks = (a.rows * ((a.k + 31) / 32) + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
    return launch_pdl(a.in_bf16 ? tcg_w4_expand_kernel<true> : tcg_w4_expand_kernel<false>, grid, dim3(256), s, 0, a,
                      static_cast<uint16_t *>(out), ldo);
}

}  // namespace tcg
