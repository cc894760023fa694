// tcg_lm_w4.cu -- products of a few tokens with 4-bit weights (sm_103a), and for many tokens the
// weights as operands of tcg_lm.cu.
//
//   z[t][f] = sum over groups of s[f][g] (sum over k of g of (q[f][k] - zero[f][g]) x[t][k])
//
// Half a byte a weight for 2 T operations.  Turning a weight into a number costs more instructions
// than multiplying it, so a warp does that once for eight tokens or more: the weights are the A
// operand of mma.m16n8k16, the tokens its eight columns (tcgen05 would want the weights back in
// shared memory first, and 128 rows of them).  A nibble becomes q - 8 by a mask and a multiply-add, exactly
// (see widen).  With zeros it is q less the nearest whole number c of 0 .. 15; what is left, c - zero times
// the group's sum of x, which one more product with a matrix of ones gives for all rows, comes in when
// the group is complete and meets its scale.  Sums are FP32.
//
// What bounds it at a few tokens is neither memory nor instructions (4 us of them for one token of 4096
// x 16384, 5.8 us for the loads alone) but a chain of waits in each warp -- rings of two to four stages,
// products one after the other, a group's end -- and, in short calls, the first loads and the join: one
// token of 4096 x 16384 takes 11.7 us (3.0 TB/s), of 16384 x 4096 11.6, of 4096 x 4096 5.1; groups of 32
// with zeros 18.0, 19.6 and 7.1.
//
// A warp has 32 or 64 rows and streams them 128 elements at a time through a ring of its own
// (asynchronous 16-byte copies, x beside the weights), on from one tile of rows to the block's next.
// Its lane c of a quad takes elements 8 c .. 8 c + 7 of each 32: in a word elements j and j + 4 are
// 16 bits apart, so one mask gives the pair (j, j + 4); x is paired to match.  The warps of a block
// and the blocks of a cluster take the stages of the same rows in turn; their sums are joined through
// (distributed) shared memory in a fixed order.

#include <type_traits>

#include "tcg_lm_math.cuh"

namespace tcg {

namespace {

constexpr int kW4K = 128;                           // elements of a stage
constexpr int kW4XRow = kW4K * 2;                   // a token of a stage

// Eight columns a product, NT of them; sixteen rows a product, MT of them.  XR: tokens whose x goes
// through the ring.  PER: groups of 32 PER elements.  W: warps of a block.
template <int NT, int MT, int XR, int PER, int W>
struct W4Cfg {
    static constexpr int kRows = 16 * MT;                            // of a warp
    static constexpr int kWBytes = kRows * kW4K / 2;                 // weights of a stage
    static constexpr int kStageBytes = kWBytes + XR * kW4XRow;
    static constexpr int kScales = W * kRows * (4 / PER) * 8;        // a stage's scales and zeros
    static constexpr int kSums = 8 * NT * kRows;                     // floats of a warp, and of what is sent
    static constexpr int kPart = (W + 1) * kSums * 4;
    static constexpr int kRoom = 227 * 1024 - kScales - kPart - 256;
    static constexpr int kFit = kRoom / (W * kStageBytes);
    static constexpr int kStages = kFit < 4 ? kFit : 4;
    static constexpr int kRing = W * kStages * kStageBytes;
    static constexpr int kSmem = kRing + kScales + kPart + 256;
    static_assert(kStages >= 2, "a stage to read and one to fill");
};

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

// d = a b + c, or (first) d = a b.
template <bool BF16>
__device__ __forceinline__ void mma_group(bool first, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (first)
        d[0] = d[1] = d[2] = d[3] = 0.0f;
    mma16816<BF16>(d, a, b0, b1);
}

// Two 16-bit numbers of the type of x, a b + c.
template <bool BF16>
__device__ __forceinline__ uint32_t fma16(uint32_t a, uint32_t b, uint32_t c)
{
    using T = std::conditional_t<BF16, __nv_bfloat162, __half2>;
    const T r = __hfma2(*reinterpret_cast<const T *>(&a), *reinterpret_cast<const T *>(&b),
                        *reinterpret_cast<const T *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The eight elements of a word as A operands: pairs (0, 4), (1, 5), (2, 6), (3, 7) of q - c, times a
// unit.  A 16-bit word 0 .. 255 read as a number is that many times the smallest subnormal one, 2^-133
// in BF16 and 2^-24 in FP16, so a masked nibble is q or 16 q in that measure; one fused multiply-add
// brings it among the normal numbers and takes c away, exactly (to make numbers of short integers by
// masks and exponents is a known method; subnormal ones need no exponent).  (With c left in, a row of weights
// near zero would be the difference of two large sums; with x scaled instead, its range would end early.)
template <bool BF16>
struct W4Unit {
    static constexpr uint32_t kLow = BF16 ? 0x7F007F00u : 0x78007800u;     // 2^127, 2^15: a nibble
    static constexpr uint32_t kHigh = BF16 ? 0x7D007D00u : 0x68006800u;    // 2^123, 2^11: sixteen times it
    static constexpr uint32_t kOne = BF16 ? 0x3C803C80u : 0x18001800u;     // the unit: 2^-6, 2^-9
    static constexpr uint32_t kMinusLow = BF16 ? 0xFF00FF00u : 0xF800F800u;    // -2^127, -2^15
    static constexpr uint32_t kMinusHigh = BF16 ? 0xFD00FD00u : 0xE800E800u;
    static constexpr uint32_t kLess8 = BF16 ? 0xBE00BE00u : 0xA400A400u;   // -8 units
    static constexpr float kInverse = BF16 ? 64.0f : 512.0f;
};
template <bool BF16>
__device__ __forceinline__ void widen(uint32_t w, uint32_t less, uint32_t (&q)[4])
{
    using U = W4Unit<BF16>;
    const uint32_t v = w >> 8;
    q[0] = fma16<BF16>(w & 0x000F000Fu, U::kLow, less);
    q[1] = fma16<BF16>(w & 0x00F000F0u, U::kHigh, less);
    q[2] = fma16<BF16>(v & 0x000F000Fu, U::kLow, less);
    q[3] = fma16<BF16>(v & 0x00F000F0u, U::kHigh, less);
}

// The whole number of 0 .. 15 nearest to a zero (0 for NaN): above 2^23 the numbers are whole.
__device__ __forceinline__ uint32_t nearest_q(float zero, float &c)
{
    const float at = fminf(fmaxf(zero, 0.0f), 15.0f) + 8388608.0f;
    c = at - 8388608.0f;
    return __float_as_uint(at) & 15u;
}

// -c units, c in bits 4 j .. 4 j + 3 of both halves of a word.
template <bool BF16>
__device__ __forceinline__ uint32_t minus_q(uint32_t c, int j)
{
    using U = W4Unit<BF16>;
    const uint32_t v = j & 2 ? c >> 8 : c;
    return j & 1 ? fma16<BF16>(v & 0x00F000F0u, U::kMinusHigh, 0u) : fma16<BF16>(v & 0x000F000Fu, U::kMinusLow, 0u);
}

__device__ __forceinline__ uint4 load_shared16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t *v)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}

// Row j of a tile's `all` in the weights: of a gated product half are rows of g, then their rows of
// u.  Rows past the end repeat the last one.
template <int kRows>
__device__ __forceinline__ int64_t w4_row(const W4Args &p, int64_t tile, int j)
{
    if (!p.gated) {
        const int64_t r = tile * kRows + j;
        return r < p.rows ? r : p.rows - 1;
    }
    const int64_t n = p.rows / 2, f = tile * (kRows / 2) + j % (kRows / 2);
    return (f < n ? f : n - 1) + (j < kRows / 2 ? 0 : n);
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

// A token's row in a warp's sums: two tokens' rows start in banks of their own.
template <int kRows>
__device__ __forceinline__ int sum_at(int token, int row)
{
    return token * kRows + (row ^ ((token >> 1 & 3) * 8));
}

// Bytes of a 16-byte piece that exist, `left` being those from its start on.
__device__ __forceinline__ int piece_bytes(int left) { return max(0, min(left, 16)); }

// N words side by side, aligned to their size.
template <int N>
__device__ __forceinline__ void load_words(const uint32_t *p, uint32_t *v)
{
    if constexpr (N == 4) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else if constexpr (N == 2) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        v[0] = q.x, v[1] = q.y;
    } else {
        v[0] = *p;
    }
}

__device__ __forceinline__ void store_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int NT, int MT, int XR, int PER, int W, bool BF16, bool ZEROS>
__global__ void __launch_bounds__(W * 32, 1) tcg_w4_kernel(const W4Args p, int cluster)
{
    using Cfg = W4Cfg<NT, MT, XR, PER, W>;
    constexpr int S = Cfg::kStages, R = Cfg::kRows, kTokens = 8 * NT, kGroups = 4 / PER;   // groups of a stage
    extern __shared__ __align__(256) uint8_t ring[];
    float *part = reinterpret_cast<float *>(ring + Cfg::kRing + Cfg::kScales), *room = part + W * Cfg::kSums;
    uint8_t *nothing = ring + Cfg::kSmem - 256;              // 256 bytes of zeros: x of no token
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    if (threadIdx.x < 64)
        reinterpret_cast<uint32_t *>(nothing)[threadIdx.x] = 0u;
    __syncthreads();
    const int rank = blockIdx.x % cluster, first_tile = blockIdx.x / cluster, tile_step = gridDim.x / cluster;
    const int tok0 = blockIdx.y * kTokens;
    const int stride = cluster * W, begin = rank * W + warp;
    const int units = p.units, groups = p.groups, tiles = p.tiles;
    const int k = static_cast<int>(p.k), bytes = (k + 1) / 2, whole = k / kW4K;   // stages without an end of the row
    const bool s_f32 = p.s_f32 != 0;
    const int tokens = p.tokens - tok0;                      // of this block, if fewer than kTokens

    const uint32_t mine = smem_u32(ring) + warp * (S * Cfg::kStageBytes);
    float *sc = reinterpret_cast<float *>(ring + Cfg::kRing) + warp * (2 * R * kGroups);   // scales, then zeros
    griddep_wait();

    // Copies: lane l brings piece l % 4 of rows l / 4 + 8 i, at a place in the row that makes eight
    // rows' reads meet different banks; and piece l % 16 of tokens l / 16 + 2 i of x.  The walk: every
    // `stride`-th stage of a tile, then those of the next tile.
    const uint8_t *src[2 * MT];
    const int rows_x = min(tokens, XR) - (lane >> 4);
    const uint16_t *src_x = static_cast<const uint16_t *>(p.X) + (tok0 + (lane >> 4)) * p.ldx + (lane & 15) * 8;
    const uint32_t to_w = mine + g * 64 + (c ^ ((g >> 1) & 3)) * 16;
    const uint32_t to_x = mine + Cfg::kWBytes + (lane >> 4) * kW4XRow + ((lane & 15) ^ ((lane >> 4) << 2)) * 16;
    int ahead = begin, ahead_tile = first_tile;
    uint32_t sp = 0;                                         // bytes of the stage to fill
    auto aim = [&]() {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            src[i] = p.W + w4_row<R>(p, ahead_tile, g + 8 * i) * p.ldw + c * 16;
    };
    if (begin >= units)                                      // nothing for this warp
        ahead_tile = tiles;
    aim();
    auto copy = [&](int from, int n, int from_x, int xn) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to_w + sp + i * 512),
                         "l"(src[i] + from), "r"(n)
                         : "memory");
#pragma unroll
        for (int i = 0; i < XR / 2; ++i)
            if (2 * i < rows_x)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to_x + sp + i * 512),
                             "l"(src_x + 2 * i * p.ldx + from_x), "r"(xn)
                             : "memory");
    };
    auto produce = [&]() {
        if (ahead_tile < tiles) {
            const int at = ahead * (kW4K / 2), kx = ahead * kW4K;
            if (ahead < whole) {
                copy(at, 16, kx, 16);
            } else {                                         // an end of the rows; nothing is read past it
                const int n = piece_bytes(bytes - at - c * 16), xn = piece_bytes((k - kx - (lane & 15) * 8) * 2);
                copy(n ? at : -c * 16, n, xn ? kx : -(lane & 15) * 8, xn);
            }
            ahead += stride;
            if (ahead >= units) {
                ahead = begin;
                ahead_tile += tile_step;
                if (ahead_tile < tiles)
                    aim();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        sp = sp + Cfg::kStageBytes == S * Cfg::kStageBytes ? 0u : sp + Cfg::kStageBytes;
    };

    // The scales and zeros of rows lane and lane + 32 come a stage ahead through registers: a stage's
    // in one load each where rows of them allow it (joined: two 16-bit ones to a register).
    constexpr int kSr = R / 32;
    const int s_bytes = (s_f32 ? 4 : 2) * kGroups;
    const bool joined = groups % kGroups == 0 && reinterpret_cast<uintptr_t>(p.scales) % s_bytes == 0 &&
                        reinterpret_cast<uintptr_t>(p.zeros) % s_bytes == 0;
    uint32_t raw_s[kSr][kGroups] = {}, raw_z[kSr][kGroups] = {};
    int64_t row_s[kSr];
    auto load_group = [&](const void *base, int64_t row, int unit, uint32_t (&v)[kGroups]) {
        if (joined) {
            const int64_t at = row + unit * kGroups;
            if (s_f32)
                load_words<kGroups>(static_cast<const uint32_t *>(base) + at, v);
            else if constexpr (kGroups > 1)
                load_words<kGroups / 2>(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + at), v);
            else
                v[0] = static_cast<const uint16_t *>(base)[at];
            return;
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
            v[j] = load_raw(base, row + min(unit * kGroups + j, groups - 1), s_f32);
    };
    auto group_value = [&](const uint32_t (&v)[kGroups], int j) {
        if (kGroups > 1 && joined && !s_f32)
            return raw_value<BF16>(v[j / 2] >> (16 * (j & 1)) & 0xFFFFu, false);
        return raw_value<BF16>(v[j], s_f32);
    };
    auto load_scales = [&](int t, int unit) {                // of stage `unit` of tile t
        if (unit == begin) {
#pragma unroll
            for (int i = 0; i < kSr; ++i)
                row_s[i] = w4_row<R>(p, t, lane + 32 * i) * groups;
        }
#pragma unroll
        for (int i = 0; i < kSr; ++i) {
            load_group(p.scales, row_s[i], unit, raw_s[i]);
            if (ZEROS)
                load_group(p.zeros, row_s[i], unit, raw_z[i]);
        }
    };

    for (int s = 0; s < S - 1; ++s)
        produce();
    if (begin < units)
        load_scales(first_tile, begin);

    // For zeros: a matrix of ones gives the sums of x.
    using U = W4Unit<BF16>;
    const uint32_t ones[4] = {U::kOne, U::kOne, U::kOne, U::kOne};
    const uint32_t from_w = mine + lane * 64 + ((lane >> 1) & 3) * 16;
    const uint32_t from_x = mine + Cfg::kWBytes + g * kW4XRow + (g & 1) * 64 + c * 16;
    uint32_t stage = 0;                                      // bytes of the stage to read
    const int here = min(tokens, kTokens), each = kTokens / cluster;     // cluster: a power of two up to 8
    const int rows = p.gated ? R / 2 : R;
    const int64_t feats = p.gated ? p.rows / 2 : p.rows;
    // Bias and residual of an output; those of a thread's first one are loaded before the tile's stages.
    auto extras = [&](int tile, int o, float &bias, float &more) {
        const int t = o / rows, j = o - t * rows, tt = t * cluster + rank;
        const int64_t f = static_cast<int64_t>(tile) * rows + j;
        bias = more = 0.0f;
        if (o >= each * rows || tt >= here || f >= feats)
            return false;
        if (p.bias)
            bias = p.bias_f32 ? static_cast<const float *>(p.bias)[f] : load16(p.bias, f, BF16);
        if (p.C)
            more = load_out(p.C, (tok0 + tt) * p.ldc + f, p.out_kind);
        return true;
    };
    for (int tile = first_tile; tile < tiles; tile += tile_step) {
        float bias, more;
        bool wanted = extras(tile, threadIdx.x, bias, more);
        float tot[MT][NT][4], acc[MT][NT][4], off[NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tot[i][nt][j] = 0.0f;
        for (int unit = begin; unit < units; unit += stride) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();                                        // and every lane has read the stage before
            produce();
            const uint32_t st = from_w + stage;
            uint32_t stx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                stx[nt] = nt * 8 + g < tokens ? from_x + stage + nt * 8 * kW4XRow : smem_u32(nothing);
            stage = stage + Cfg::kStageBytes == S * Cfg::kStageBytes ? 0u : stage + Cfg::kStageBytes;
#pragma unroll
            for (int i = 0; i < kSr; ++i)
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
                    sc[(lane + 32 * i) * kGroups + j] = group_value(raw_s[i], j) * U::kInverse;
            [[maybe_unused]] uint32_t less[2 * MT];              // rows g + 8 i: their c of each group, four bits apart
            if constexpr (ZEROS) {
                uint32_t c_of[kSr];
#pragma unroll
                for (int i = 0; i < kSr; ++i) {
                    c_of[i] = 0u;
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        const float zero = group_value(raw_z[i], j);
                        float whole;
                        c_of[i] |= nearest_q(zero, whole) << (4 * j);
                        sc[(R + lane + 32 * i) * kGroups + j] = whole - zero;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
                    less[i] = __shfl_sync(0xffffffffu, c_of[i / 4], g + 8 * (i & 3)) * 0x10001u;
            }
            __syncwarp();
            if (unit + stride < units)
                load_scales(tile, unit + stride);
            else if (tile + tile_step < tiles)
                load_scales(tile + tile_step, begin);
            uint32_t w[2][2 * MT];                               // rows g + 8 i, of this and the next 32 elements
            uint4 x[2][NT];
            auto fetch = [&](int q) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    x[q & 1][nt] = load_shared16(stx[nt] ^ (q * 64));
#pragma unroll
                for (int i = 0; i < MT; i += 2)
                    ldmatrix4((st + i * 1024) ^ (q * 16), &w[q & 1][2 * i]);
            };
            fetch(0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool first = q % PER == 0;                 // of its group
                if (PER == 1)                                    // a group at a time: more of them want too many registers
                    __syncwarp();
                if (q < 3)
                    fetch(q + 1);
                uint32_t b[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 v = x[q & 1][nt];
                    b[nt][0] = __byte_perm(v.x, v.z, 0x5410);
                    b[nt][1] = __byte_perm(v.x, v.z, 0x7632);
                    b[nt][2] = __byte_perm(v.y, v.w, 0x5410);
                    b[nt][3] = __byte_perm(v.y, v.w, 0x7632);
                    if constexpr (ZEROS) {
                        mma_group<BF16>(first, off[nt], ones, b[nt][0], b[nt][1]);
                        mma_group<BF16>(false, off[nt], ones, b[nt][2], b[nt][3]);
                    }
                }
                uint32_t minus[2 * MT];                          // -c units
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
                    minus[i] = ZEROS ? minus_q<BF16>(less[i], q / PER) : U::kLess8;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t lo[4], hi[4];
                    widen<BF16>(w[q & 1][2 * i], minus[2 * i], lo);
                    widen<BF16>(w[q & 1][2 * i + 1], minus[2 * i + 1], hi);
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_group<BF16>(first, acc[i][nt], a0, b[nt][0], b[nt][1]);
                        mma_group<BF16>(false, acc[i][nt], a1, b[nt][2], b[nt][3]);
                    }
                }
                if (q % PER == PER - 1) {                        // the group is complete
                    const float *at_s = sc + g * kGroups + q / PER;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const float s0 = at_s[16 * i * kGroups], s1 = at_s[(16 * i + 8) * kGroups];
                        if constexpr (ZEROS) {                   // none where zeros are whole: 0 times infinity is no part
                            const float z0 = at_s[(R + 16 * i) * kGroups], z1 = at_s[(R + 16 * i + 8) * kGroups];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float z = j < 2 ? z0 : z1;
                                    if (z != 0.0f)
                                        acc[i][nt][j] = fmaf(z, off[nt][j & 1], acc[i][nt][j]);
                                }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tot[i][nt][j] = fmaf(j < 2 ? s0 : s1, acc[i][nt][j], tot[i][nt][j]);
                    }
                }
            }
        }

        // The warps' sums, [warp][token][row].  A thread adds those of a token and row over the warps; in a
        // cluster it sends them to the block that finishes the token: the tokens go round the cluster,
        // and a block has room for each sender's.
        __syncthreads();                                         // the last tile is finished,
        if (cluster > 1)
            cluster_arrive();                                    // as far as this block goes
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[warp * Cfg::kSums + sum_at<R>(nt * 8 + 2 * c + (j & 1), 16 * i + 8 * (j >> 1) + g)] =
                        tot[i][nt][j];
        __syncthreads();
        auto block_sum = [&](int t, int j) {
            const int at = sum_at<R>(t, j);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                v += part[w * Cfg::kSums + at];
            return v;
        };
        if (cluster > 1) {
            cluster_wait();
            for (int o = threadIdx.x; o < here * R; o += W * 32) {
                const int t = o / R, j = o % R;
                store_cluster(mapa_shared(smem_u32(room + (rank * each + t / cluster) * R + j), t % cluster), block_sum(t, j));
            }
            cluster_sync_all();
        }
        for (int o = threadIdx.x; o < each * rows; o += W * 32) {
            if (o >= W * 32)
                wanted = extras(tile, o, bias, more);
            if (!wanted)
                continue;
            const int t = o / rows, j = o - t * rows;
            const int64_t f = static_cast<int64_t>(tile) * rows + j, tok = tok0 + t * cluster + rank;
            float z = 0.0f, u = 0.0f;
            if (cluster > 1) {
                for (int r = 0; r < cluster; ++r) {
                    z += room[(r * each + t) * R + j];
                    if (p.gated)
                        u += room[(r * each + t) * R + j + R / 2];
                }
            } else {
                z = block_sum(t, j);
                if (p.gated)
                    u = block_sum(t, j + R / 2);
            }
            z = act_of(p.act, z + bias);
            if (p.gated)
                z *= u;
            if (p.C)
                z = fmaf(p.beta, more, z);
            store_out(p.D, tok * p.ldd + f, p.out_kind, z);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The weights as operands of the product of many tokens: q - c as above, the scales and what is left of
// the zeros beside them for its epilogue.  Nothing is rounded: weights times scales would be, to the 8
// or 11 bits of x's type (2-norm error 0.0019 to 0.0024 of the result in BF16, the output's own rounding
// being 0.0017), and where scales are small or large would leave its range.  Eight elements of a row a thread,
// so that a warp writes 512 bytes side by side, and kExpandRows rows at a time, their loads before the first
// store.  What lies past a row's end is not read by the product.
constexpr int kExpandRows = 4;
template <bool BF16>
__global__ void __launch_bounds__(256)
    tcg_w4_expand_kernel(const W4Args p, uint16_t *__restrict__ out, int64_t ldo, float *__restrict__ scale,
                         float *__restrict__ rest, int64_t ld_t)
{
    using U = W4Unit<BF16>;
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x * 256 + threadIdx.x, k = static_cast<int>(p.k), left = k - i * 8;
    if (left <= 0)
        return;
    const int groups = (k + p.group - 1) / p.group;
    const int g = i >> (p.group == 32 ? 2 : (p.group == 64 ? 3 : 4));
    const bool first = i * 8 == g * p.group;                 // of its group
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kExpandRows; row0 < p.rows;
         row0 += static_cast<int64_t>(gridDim.y) * kExpandRows) {
        uint32_t u[kExpandRows], s[kExpandRows], z[kExpandRows];
#pragma unroll
        for (int r = 0; r < kExpandRows; ++r) {
            const int64_t row = row0 + r < p.rows ? row0 + r : p.rows - 1;
            const uint8_t *w = p.W + row * p.ldw + i * 4;
            u[r] = 0u;
            if (left >= 7) {                                 // four bytes of the row
                u[r] = *reinterpret_cast<const uint32_t *>(w);
            } else {
                for (int j = 0; 2 * j < left; ++j)
                    u[r] |= static_cast<uint32_t>(w[j]) << (8 * j);
            }
            s[r] = first ? load_raw(p.scales, row * groups + g, p.s_f32) : 0u;
            z[r] = p.zeros ? load_raw(p.zeros, row * groups + g, p.s_f32) : 0u;
        }
        float sc[kExpandRows], rs[kExpandRows];
#pragma unroll
        for (int r = 0; r < kExpandRows; ++r) {
            const float zero = p.zeros ? raw_value<BF16>(z[r], p.s_f32) : 8.0f;
            float c;
            const uint32_t whole = nearest_q(zero, c);
            sc[r] = raw_value<BF16>(s[r], p.s_f32) * U::kInverse;
            rs[r] = (c - zero) * (1.0f / U::kInverse);
            if (row0 + r >= p.rows)
                continue;
            uint32_t q[4];
            widen<BF16>(u[r], minus_q<BF16>(whole * 0x10001u, 0), q);
            *reinterpret_cast<uint4 *>(out + (row0 + r) * ldo + i * 8) =          // ldo: a multiple of 8
                make_uint4(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                           __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
        }
        if (first) {
            *reinterpret_cast<float4 *>(scale + g * ld_t + row0) = make_float4(sc[0], sc[1], sc[2], sc[3]);
            if (p.zeros)
                *reinterpret_cast<float4 *>(rest + g * ld_t + row0) = make_float4(rs[0], rs[1], rs[2], rs[3]);
        }
    }
}

// Eight elements of a token a thread; a group is 4, 8 or 16 lanes of a warp.
template <bool BF16>
__global__ void __launch_bounds__(256) tcg_w4_sums_kernel(const W4Args p, float *__restrict__ out, int64_t ld)
{
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x * 256 + threadIdx.x, left = static_cast<int>(p.k) - i * 8, lanes = p.group / 8;
    for (int64_t t = blockIdx.y; t < p.tokens; t += gridDim.y) {
        const uint16_t *x = static_cast<const uint16_t *>(p.X) + t * p.ldx + i * 8;
        float v[8];
        if (left >= 8) {
            unpack16<BF16>(*reinterpret_cast<const uint4 *>(x), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = j < left ? load16(x, j, BF16) : 0.0f;
        }
        float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        for (int d = lanes / 2; d; d >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, d);
        if (left > 0 && i % lanes == 0)
            out[i / lanes * ld + t] = s;
    }
}

template <int NT, int MT, int XR, int PER, int W, bool BF16, bool ZEROS>
cudaError_t launch_one(W4Args a, int num_sms, cudaStream_t s)
{
    using Cfg = W4Cfg<NT, MT, XR, PER, W>;
    auto fn = tcg_w4_kernel<NT, MT, XR, PER, W, BF16, ZEROS>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess)
        return e;
    const int rows = a.gated ? Cfg::kRows / 2 : Cfg::kRows;
    a.tiles = static_cast<int>(((a.gated ? a.rows / 2 : a.rows) + rows - 1) / rows);
    a.units = static_cast<int>((a.k + kW4K - 1) / kW4K);
    a.groups = static_cast<int>((a.k + a.group - 1) / a.group);
    const int blocks = (a.tokens + 8 * NT - 1) / (8 * NT), most = num_sms / blocks;
    // As many blocks to a tile as are resident together and leave each warp a stage.
    int cluster = 1;
    while (cluster < 8 && a.units > cluster * W && a.tiles * cluster * 2 <= most)
        cluster *= 2;
    const int wide = a.tiles < most / cluster ? a.tiles : most / cluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(wide * cluster), blocks);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = Cfg::kSmem;
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

template <int NT, int MT, int XR, int W, bool BF16, bool ZEROS>
cudaError_t launch_group(const W4Args &a, int num_sms, cudaStream_t s)
{
    return a.group == 32 ? launch_one<NT, MT, XR, 1, W, BF16, ZEROS>(a, num_sms, s)
         : a.group == 64 ? launch_one<NT, MT, XR, 2, W, BF16, ZEROS>(a, num_sms, s)
                         : launch_one<NT, MT, XR, 4, W, BF16, ZEROS>(a, num_sms, s);
}

template <int NT, int MT, int XR, int W>
cudaError_t launch_types(const W4Args &a, int num_sms, cudaStream_t s)
{
    if (a.in_bf16)
        return a.zeros ? launch_group<NT, MT, XR, W, true, true>(a, num_sms, s)
                       : launch_group<NT, MT, XR, W, true, false>(a, num_sms, s);
    return a.zeros ? launch_group<NT, MT, XR, W, false, true>(a, num_sms, s)
                   : launch_group<NT, MT, XR, W, false, false>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_w4(const W4Args &a, int num_sms, cudaStream_t s)
{
    // Up to eight tokens, 64 rows a warp where that leaves tiles for half of the SMs: what a stage costs
    // besides its weights is shared by more of them (one token, us in a graph, 32 / 64 rows: 4096 x 4096
    // 5.1 / 5.9, 8192 x 4096 8.1 / 7.3, 16384 x 4096 13.3 / 11.6; eight tokens 6.0 / 6.6, 10.3 / 7.9,
    // 16.9 / 12.9).  Rooms for two tokens' x leave those sixteen warps, for eight tokens' twelve (one
    // token of 16384 x 4096: 11.6 and 11.8 us).
    if (a.tokens <= 8 && a.rows >= 32 * num_sms)
        return a.tokens <= 2 ? launch_types<1, 4, 2, 16>(a, num_sms, s) : launch_types<1, 4, 8, 12>(a, num_sms, s);
    // More: sixteen tokens a pass (32 of them with eight warps take longer, 32 tokens of 16384 x 4096
    // 39.5 us for 32.2, and 33 tokens of 4096 x 4096 18.4 for 15.0).
    return a.tokens <= 8 ? launch_types<1, 2, 8, 16>(a, num_sms, s) : launch_types<2, 2, 16, 12>(a, num_sms, s);
}

cudaError_t launch_w4_expand(const W4Args &a, void *out, int64_t ldo, float *scale, float *rest, int64_t ld_t,
                             int num_sms, cudaStream_t s)
{
    const int64_t across = ((a.k + 7) / 8 + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    const int64_t down = (most + across - 1) / across, need = (a.rows + kExpandRows - 1) / kExpandRows;
    const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(need < down ? need : down));
    return launch_pdl(a.in_bf16 ? tcg_w4_expand_kernel<true> : tcg_w4_expand_kernel<false>, grid, dim3(256), s, 0, a,
                      static_cast<uint16_t *>(out), ldo, scale, rest, ld_t);
}

cudaError_t launch_w4_sums(const W4Args &a, float *out, int64_t ld, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>(((a.k + 7) / 8 + 255) / 256),
                    static_cast<unsigned>(a.tokens < 4096 ? a.tokens : 4096));
    return launch_pdl(a.in_bf16 ? tcg_w4_sums_kernel<true> : tcg_w4_sums_kernel<false>, grid, dim3(256), s, 0, a, out, ld);
}

}  // namespace tcg
