// tcg_lm.cu -- device code of the language-model products (sm_103a).
//
// tcg_lm_kernel is a persistent, warp-specialised tensor-core product over CTA pairs
// (tcgen05, cta_group::2; 256 x BN tiles, M = 256 accumulator rows, N = BN columns):
//
//   warp 0 (one lane)   TMA producer into a ring of 128-byte-swizzled stages (64 K elements
//                       of 128 rows of A and BN / 2 rows of B per CTA)
//   warp 1 (one lane)   tcgen05.mma into as many TMEM accumulators as fit
//   warps 2-9           epilogue: TMEM -> registers -> memory, one accumulator row a thread
//
// The epilogues (LmEpi):
//   kEpiNarrow     features on the rows, tokens on the columns: few tokens against a weight
//                  matrix that streams by once
//   kEpiWide       tokens on the rows, features on the columns: a thread holds 32 adjacent
//                  features of a token, so bias, residual, pre-activation and output move in
//                  16-byte pieces
//   kEpiXentStats  logits X W^T that never leave the chip: per row and tile part the maximum
//                  m and sum exp(logit - m), and the target's logit (tokens on the rows)
//   kEpiXentNarrow the same for few tokens (tokens on the columns)
//   kEpiXentGrad   dloss (exp(logit - lse) - [target]), scaled, rounded to 16 bits
//
// What bounds it.  A 64-element block of K costs an SM 32 KiB of operands at tile 256 x 256,
// loaded at 64 bytes a cycle in the 512 cycles that the tensor core takes for it; with both
// at work shared memory is nearly full (written and read at 64 bytes a cycle each of 128),
// so the epilogue's own traffic through it adds to short-K tiles (K = 512: loads alone 36,
// with the product 43, with the epilogue 55 us for 1024 tiles).  From K = 4096 on it hides
// behind the product and the power limit bounds (16384 x 4096 x 4096 BF16, GELU,
// pre-activation kept: 305 us in a graph of a few calls, 1.80 PFLOP/s; 356 us a call, 1.54, one
// after the other for seconds).
//
// Every wait is bounded as in tcg_kernels.cu: a wait that runs out sets a bit in the
// device error word, every role stops and the kernel returns.

#include "tcg_lm_math.cuh"
#include "tcg_pipe.cuh"

namespace tcg {

namespace {

// How the tiles of a call are spread over the pairs (see LmWalk).
struct LmPlan {
    int tiles;          // tiles of the groups
    int whole;          // tiles [0, whole) go whole, round robin; the rest are cut along K
    int share;          // K blocks of the cut tiles per pair
    int splits;         // pairs per cut tile, ranges alike for all of them; 0: laid end to end
    int null_tiles[2];  // tiles of the columns (rows) before the first and after the last group
};

struct LmCtl {
    uint64_t full[kLmMaxStages];
    uint64_t empty[kLmMaxStages];
    uint64_t acc_full[kLmMaxAccs];
    uint64_t acc_empty[kLmMaxAccs];
    uint64_t drain;
    uint32_t tmem_base;
    volatile int abort_flag;
    volatile int last_arrival[4];
    LmPlan plan;
    int cum[kLmMaxGroups + 1];              // tiles before each group of a grouped call
};
constexpr int kLmCtlBytes = 2 * 1024;
static_assert(sizeof(LmCtl) <= kLmCtlBytes, "control area too small");
constexpr int kLmSmemBytes = kLmDataBytes + kLmCtlBytes + 1024;   // + alignment slack

// ------------------------------------------------------------------------------- units
// The tokens of no group: before the first (which = 0) and after the last (1).
__device__ __forceinline__ void null_range(const LmArgs &p, int which, int &begin, int &end)
{
    const int64_t o = p.offsets[which ? p.groups : 0], c = p.tokens;
    const int at = static_cast<int>(o < 0 ? 0 : (o > c ? c : o));
    begin = which ? at : 0;
    end = which ? p.tokens : at;
}

struct LmUnit {
    int g;                  // group; -1: tokens of no group, which come out zero
    int row0, row_end;      // accumulator rows: first, and end of what may be written
    int col0, col_end;      // accumulator columns
    int kb0, kb1;           // K blocks
    int tok0, toks;         // K ragged: first token, tokens
    int slot;               // partial-sum slot of a cut tile's piece; -1: the whole tile
    int first_pair, pieces; // of a cut tile
    int counter;
};

// A role's walk over the units of its pair c of P.  Tiles 0 .. whole - 1 go whole, tile t to
// pair t mod P.  The tiles after them, fewer than P, would keep only some pairs busy: where
// that costs more than joining partial sums, their K blocks are laid end to end and every
// pair takes `share` of them -- a piece of one tile, or the end of one and the start of the
// next (and whole tiles between).  (Where the operands are larger than L2 and shared by
// tiles, every cut tile instead gets the same number of pairs and the same K ranges, so that
// tiles read the same blocks at the same time.)  A pair has at most one piece that starts
// inside a tile (slot 2 c) and one that starts a tile without ending it (slot 2 c + 1).
template <bool WIDE, int BN, bool RK>
struct LmWalk {
    int c, P;
    int t, null_i;
    uint32_t pos;                                   // next block of the cut tiles; ~0: not begun
    int group = 0, at = -1, begin = 0, end = 0;     // group of tile t; whose range is loaded

    __device__ __forceinline__ LmWalk(int pair, int pairs) : c(pair), P(pairs), t(pair),
                                                             null_i(pair), pos(~0u) {}

    __device__ __forceinline__ bool next(const LmArgs &p, const LmCtl *ctl, LmUnit &w)
    {
        const LmPlan &pl = ctl->plan;
        w.slot = -1;
        w.tok0 = w.toks = 0;
        w.kb0 = 0;
        w.kb1 = p.num_k_blocks;
        if (t < pl.whole) {
            locate(p, ctl, t, w);
            t += P;
            return true;
        }
        const int cut = pl.tiles - pl.whole;
        if (cut > 0) {
            const uint32_t nkb = static_cast<uint32_t>(p.num_k_blocks);
            const uint32_t share = static_cast<uint32_t>(pl.share), me = static_cast<uint32_t>(c);
            if (pl.splits) {
                const uint32_t r = me / pl.splits, piece = me - r * pl.splits;
                if (pos == ~0u && r < static_cast<uint32_t>(cut)) {
                    pos = 0;
                    w.kb0 = static_cast<int>(piece * share);
                    w.kb1 = static_cast<int>(min(nkb, (piece + 1) * share));
                    w.slot = 2 * c + (piece == 0 ? 1 : 0);
                    w.first_pair = static_cast<int>(r * pl.splits);
                    w.pieces = pl.splits;
                    w.counter = static_cast<int>(r);
                    locate(p, ctl, pl.whole + static_cast<int>(r), w);
                    return true;
                }
            } else {
                const uint32_t work = static_cast<uint32_t>(cut) * nkb;
                const uint32_t stop = min((me + 1) * share, work);
                if (pos == ~0u)
                    pos = min(me * share, work);
                if (pos < stop) {
                    const uint32_t r = pos / nkb, r0 = r * nkb;
                    w.kb0 = static_cast<int>(pos - r0);
                    w.kb1 = static_cast<int>(min(nkb, stop - r0));
                    pos = r0 + static_cast<uint32_t>(w.kb1);
                    if (w.kb1 - w.kb0 < p.num_k_blocks) {
                        w.slot = 2 * c + (w.kb0 == 0 ? 1 : 0);
                        w.first_pair = static_cast<int>(r0 / share);
                        w.pieces = static_cast<int>((r0 + nkb - 1) / share) - w.first_pair + 1;
                        w.counter = static_cast<int>(r);
                    }
                    locate(p, ctl, pl.whole + static_cast<int>(r), w);
                    return true;
                }
            }
        }
        const int nulls = pl.null_tiles[0] + pl.null_tiles[1];
        if (null_i < nulls) {
            const int which = null_i >= pl.null_tiles[0] ? 1 : 0;
            int b, e;
            null_range(p, which, b, e);
            w.g = -1;
            w.kb1 = 0;
            place(p, null_i - (which ? pl.null_tiles[0] : 0), b, e, w);
            null_i += P;
            return true;
        }
        return false;
    }

    __device__ __forceinline__ void locate(const LmArgs &p, const LmCtl *ctl, int tile, LmUnit &w)
    {
        if constexpr (RK) {
            const int per = p.num_row_tiles * p.num_col_tiles;
            w.g = tile / per;
            if (w.g != at) {
                group_range(p.offsets, p.tokens, w.g, begin, end);
                at = w.g;
            }
            w.tok0 = begin;
            w.toks = end - begin;
            w.kb1 = (w.toks + 63) >> 6;
            place(p, tile - w.g * per, 0, p.rows, w);
            return;
        }
        if (p.offsets) {
            while (tile >= ctl->cum[group + 1])
                ++group;
            if (group != at) {
                group_range(p.offsets, p.tokens, group, begin, end);
                at = group;
            }
            w.g = group;
            place(p, tile - ctl->cum[group], begin, end, w);
        } else {
            w.g = 0;
            place(p, tile, 0, p.tokens, w);
        }
    }

    // Tile t of the grid whose ragged side is the tokens b .. e - 1; group_m tile rows are
    // walked together.
    static __device__ __forceinline__ void place(const LmArgs &p, int t, int b, int e, LmUnit &w)
    {
        const int rts = WIDE && !RK ? (e - b + 255) >> 8 : p.num_row_tiles;
        const int cts = WIDE ? p.num_col_tiles : (e - b + BN - 1) / BN;
        const int span = p.group_m * cts;
        const int first = t / span * p.group_m;
        const int gsize = min(rts - first, p.group_m);
        const int in = t % span;
        const int rt = first + in % gsize, ct = in / gsize;
        if constexpr (WIDE) {
            w.row0 = b + rt * 256;
            w.row_end = e;
            w.col0 = ct * BN;
            w.col_end = p.cols;
        } else {
            w.row0 = rt * 256;
            w.row_end = p.rows;
            w.col0 = b + ct * BN;
            w.col_end = e;
        }
    }
};

// Tiles of a range of tokens.
template <bool WIDE, int BN>
__device__ __forceinline__ int tiles_of_range(const LmArgs &p, int b, int e)
{
    return WIDE ? ((e - b + 255) >> 8) * p.num_col_tiles : (e - b + BN - 1) / BN * p.num_row_tiles;
}

// The call's plan, by one warp.
template <bool WIDE, int BN, bool RK>
__device__ __forceinline__ void make_plan(const LmArgs &p, LmCtl *ctl, int lane, int pairs)
{
    int tiles = 0;
    int nulls[2] = {0, 0};
    if (RK) {
        tiles = p.groups * p.num_row_tiles * p.num_col_tiles;
    } else if (!p.offsets) {
        tiles = tiles_of_range<WIDE, BN>(p, 0, p.tokens);
    } else {
        if (lane == 0)
            ctl->cum[0] = 0;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            int n = 0;
            if (g0 + lane < p.groups) {
                int b, e;
                group_range(p.offsets, p.tokens, g0 + lane, b, e);
                n = tiles_of_range<WIDE, BN>(p, b, e);
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d)
                    n += up;
            }
            if (g0 + lane < p.groups)
                ctl->cum[g0 + lane + 1] = tiles + n;
            tiles += __shfl_sync(0xffffffffu, n, 31);
        }
        for (int i = 0; i < 2; ++i) {
            int b, e;
            null_range(p, i, b, e);
            nulls[i] = tiles_of_range<WIDE, BN>(p, b, e);
        }
    }
    if (lane == 0) {
        LmPlan pl;
        pl.tiles = pl.whole = tiles;
        pl.share = 1;
        pl.splits = 0;
        pl.null_tiles[0] = nulls[0];
        pl.null_tiles[1] = nulls[1];
        const int rest = tiles % pairs;
        if (!RK && p.part && rest > 0) {
            const uint32_t nkb = static_cast<uint32_t>(p.num_k_blocks);
            int splits = 0;
            int share = max(static_cast<int>((rest * nkb + pairs - 1) / pairs), p.min_share);
            // One piece of one tile for each pair, where that leaves few pairs idle (1500 x 1000
            // outputs over K = 8192: 37 -> 30 us), or tokens are on the columns: HBM bounds those
            // loads, and fewer pairs can ask for them as fast (9 tokens, 4096 x 4096: 13.7 -> 12.1
            // us; 100 tokens 21.9 -> 17.7).
            const int busy = pairs / rest * rest;
            if (p.align_splits || (WIDE ? 20 * busy >= 17 * pairs : busy > rest)) {
                share = max(static_cast<int>((nkb + pairs / rest - 1) / (pairs / rest)), p.min_share);
                splits = static_cast<int>((nkb + share - 1) / share);
            }
            if (p.num_k_blocks - share >= p.split_gain) {
                pl.whole = tiles - rest;
                pl.share = share;
                pl.splits = splits;
            }
        }
        ctl->plan = pl;
    }
}

// ------------------------------------------------------------------------- the epilogues
template <int N>
__device__ __forceinline__ void apply_act(int act, float (&x)[N])
{
    auto all = [&](auto f) {
#pragma unroll
        for (int j = 0; j < N; j += 2)
            split2(f(f2(x[j], x[j + 1])), x[j], x[j + 1]);
    };
    switch (act) {
    case kActRelu: all([](F2 v) { return act_fn<kActRelu>(v); }); break;
    case kActGelu: all([](F2 v) { return act_fn<kActGelu>(v); }); break;
    case kActGeluTanh: all([](F2 v) { return act_fn<kActGeluTanh>(v); }); break;
    case kActSilu: all([](F2 v) { return act_fn<kActSilu>(v); }); break;
    default: break;
    }
}

// One feature (row) of kCols tokens from `col` on: each store of a warp is a 64- or 128-byte
// run of one token's features.
template <int OUT, int kCols>
__device__ __forceinline__ void finish_narrow(const LmArgs &p, float (&z)[kCols], const LmUnit &w,
                                              int row, int col, float alpha, float bias)
{
    const int ncol = w.col_end - col;
    if (row >= p.rows || ncol <= 0)
        return;
    const int64_t dbase = static_cast<int64_t>(col) * p.ldd + row;
    uint16_t *zp = static_cast<uint16_t *>(p.Z) + static_cast<int64_t>(col) * p.ldz + row;
    if (w.g < 0) {                             // tokens of no group
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol) {
                store_as<OUT>(p.D, dbase + j * p.ldd, 0.0f);
                if (p.Z)
                    zp[j * p.ldz] = 0;
            }
        return;
    }
    const F2 a = f2(alpha), b = f2(bias);
#pragma unroll
    for (int j = 0; j < kCols; j += 2)
        split2(fma2(a, f2(z[j], z[j + 1]), b), z[j], z[j + 1]);
    if (p.Z) {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol)
                zp[j * p.ldz] = round16(z[j], p.in_bf16);
    }
    apply_act(p.act, z);
    if (p.C) {
        const int64_t cbase = static_cast<int64_t>(col) * p.ldc + row;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol)
                z[j] = fmaf(p.beta, load_as<OUT>(p.C, cbase + j * p.ldc), z[j]);
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        if (j < ncol)
            store_as<OUT>(p.D, dbase + j * p.ldd, z[j]);
}

// A warp's rows (tokens, one per lane in registers) go to and from memory through the warp's
// staging area, 64 bytes of each row at a time (32 16-bit or 16 FP32 features), so that
// memory is accessed in runs of 64 bytes: a lane's own row would go in 16-byte pieces of 32
// different lines per instruction (16384 x 4096 x 1024 BF16: 97 us a call so, 90 us through
// the staging area).  The 16-byte pieces of a row are permuted by row, so that neither side
// has bank conflicts.
__device__ __forceinline__ uint4 *stage_piece(uint8_t *stage, int row, int piece)
{
    return reinterpret_cast<uint4 *>(stage) + row * 4 + (piece ^ ((row >> 1) & 3));
}

// kN = 32 16-bit or 16 FP32 values of this lane's row.
template <int OUT, int kN>
__device__ __forceinline__ void stage_put(uint8_t *stage, int lane, const float *x)
{
    static_assert(kN == (OUT == kOutF32 ? 16 : 32), "64 bytes");
    constexpr bool b = OUT == kOutBF16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (OUT == kOutF32)
            *stage_piece(stage, lane, j) =
                make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                           __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
        else
            *stage_piece(stage, lane, j) =
                make_uint4(pack16(x[8 * j], x[8 * j + 1], b), pack16(x[8 * j + 2], x[8 * j + 3], b),
                           pack16(x[8 * j + 4], x[8 * j + 5], b), pack16(x[8 * j + 6], x[8 * j + 7], b));
    }
}

// A warp's block of a row-major matrix, 32 rows x 64 bytes: `at` is this lane's first piece
// (row lane / 4, piece lane % 4), `step` the bytes to its next one, 8 rows on.
template <int ES>
struct WarpBlock {
    static constexpr int kElems = 16 / ES;
    uint8_t *at;
    int64_t step;

    __device__ __forceinline__ WarpBlock(const void *base, int64_t ld, int64_t row0, int64_t col, int lane)
    {
        at = static_cast<uint8_t *>(const_cast<void *>(base)) +
             ((row0 + lane / 4) * ld + col + lane % 4 * kElems) * ES;
        step = 8 * ld * ES;
    }
};

// The staged block to memory: its first nrow rows and ncol columns.
template <int ES>
__device__ __forceinline__ void stage_flush(uint8_t *stage, int lane, WarpBlock<ES> m, int nrow, int ncol)
{
    using M = WarpBlock<ES>;
    const int row = lane / 4, piece = lane % 4;
    if (nrow >= 32 && ncol >= 4 * M::kElems) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint4 *>(m.at) = *stage_piece(stage, i * 8 + row, piece);
            m.at += m.step;
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i, m.at += m.step) {
        if (i * 8 + row >= nrow)
            break;
        const uint8_t *v = reinterpret_cast<const uint8_t *>(stage_piece(stage, i * 8 + row, piece));
        const int n = ncol - piece * M::kElems;
        if (n >= M::kElems) {
            *reinterpret_cast<uint4 *>(m.at) = *reinterpret_cast<const uint4 *>(v);
        } else {
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                if constexpr (ES == 4)
                    reinterpret_cast<uint32_t *>(m.at)[j] = reinterpret_cast<const uint32_t *>(v)[j];
                else
                    reinterpret_cast<uint16_t *>(m.at)[j] = reinterpret_cast<const uint16_t *>(v)[j];
            }
        }
    }
}

// A block from memory to the staging area, whole (asynchronously; stage_filled waits) or in
// part (what lies outside stays as it was).
template <int ES>
__device__ __forceinline__ void stage_fill(uint8_t *stage, int lane, WarpBlock<ES> m, int nrow, int ncol)
{
    using M = WarpBlock<ES>;
    const int row = lane / 4, piece = lane % 4;
    if (nrow >= 32 && ncol >= 4 * M::kElems) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(stage_piece(stage, i * 8 + row, piece))),
                         "l"(m.at)
                         : "memory");
            m.at += m.step;
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i, m.at += m.step) {
        if (i * 8 + row >= nrow)
            break;
        uint8_t *v = reinterpret_cast<uint8_t *>(stage_piece(stage, i * 8 + row, piece));
        const int n = ncol - piece * M::kElems;
#pragma unroll 1
        for (int j = 0; j < n && j < M::kElems; ++j) {
            if constexpr (ES == 4)
                reinterpret_cast<uint32_t *>(v)[j] = reinterpret_cast<const uint32_t *>(m.at)[j];
            else
                reinterpret_cast<uint16_t *>(v)[j] = reinterpret_cast<const uint16_t *>(m.at)[j];
        }
    }
}
__device__ __forceinline__ void stage_filled()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// x = beta * (this lane's staged row) + x.
template <int OUT, int kN>
__device__ __forceinline__ void stage_add(uint8_t *stage, int lane, float beta, float *x)
{
    const F2 s = f2(beta);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = *stage_piece(stage, lane, j);
        constexpr int kE = kN / 4;
        float r[8];
        if constexpr (OUT == kOutF32) {
            r[0] = __uint_as_float(v.x);
            r[1] = __uint_as_float(v.y);
            r[2] = __uint_as_float(v.z);
            r[3] = __uint_as_float(v.w);
        } else {
            unpack16<OUT == kOutBF16>(v, r);
        }
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
            float *y = x + kE * j + i;
            split2(fma2(s, f2(r[i], r[i + 1]), f2(y[0], y[1])), y[0], y[1]);
        }
    }
}

// z = alpha v + bias for the 32 features from entry i of the bias on (the first n of them),
// the same for every lane: a lane loads one entry, all read them back from the staging area.
__device__ __forceinline__ void scale_bias(const LmArgs &p, float alpha, int64_t i, int n, uint8_t *stage,
                                           int lane, const uint32_t (&v)[32], float (&z)[32])
{
    const F2 a = f2(alpha);
    if (!p.bias) {
#pragma unroll
        for (int j = 0; j < 32; j += 2)
            split2(a * f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), z[j], z[j + 1]);
        return;
    }
    float b = 0.0f;
    if (lane < n)
        b = p.bias_f32 ? static_cast<const float *>(p.bias)[i + lane] : load16(p.bias, i + lane, p.in_bf16);
    reinterpret_cast<float *>(stage)[lane] = b;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float4 q = reinterpret_cast<const float4 *>(stage)[j / 4];
        split2(fma2(a, f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2(q.x, q.y)), z[j], z[j + 1]);
        split2(fma2(a, f2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f2(q.z, q.w)), z[j + 2],
               z[j + 3]);
    }
    __syncwarp();
}

// A warp's 32 tokens (from row0; this lane's pre-activations in z) x 32 features from `col`
// on; the whole warp calls it, with a block that is not empty.
template <int OUT>
__device__ __forceinline__ void finish_wide(const LmArgs &p, float (&z)[32], const LmUnit &w, int row0,
                                            int col, uint8_t *stage, int lane)
{
    constexpr int ES = OUT == kOutF32 ? 4 : 2, kN = 64 / ES;
    const int nrow = w.row_end - row0, ncol = w.col_end - col;
    if (w.g < 0) {                             // tokens of no group
#pragma unroll
        for (int j = 0; j < 32; ++j)
            z[j] = 0.0f;
    }
    if (p.Z) {
        if (p.in_bf16)
            stage_put<kOutBF16, 32>(stage, lane, z);
        else
            stage_put<kOutF16, 32>(stage, lane, z);
        __syncwarp();
        stage_flush<2>(stage, lane, WarpBlock<2>(p.Z, p.ldz, row0, col, lane), nrow, ncol);
        __syncwarp();
    }
    const bool add = p.C && w.g >= 0;
    if (add)                                   // on its way during the activation
        stage_fill<ES>(stage, lane, WarpBlock<ES>(p.C, p.ldc, row0, col, lane), nrow, ncol);
    if (w.g >= 0)
        apply_act(p.act, z);
    uint8_t *d = static_cast<uint8_t *>(p.D) + (p.ragged_k ? w.g * p.strideD * ES : 0);
#pragma unroll
    for (int h = 0; h < 32; h += kN) {
        if (h > 0 && ncol <= h)
            break;
        if (add) {
            if (h > 0)
                stage_fill<ES>(stage, lane, WarpBlock<ES>(p.C, p.ldc, row0, col + h, lane), nrow, ncol - h);
            stage_filled();
            stage_add<OUT, kN>(stage, lane, p.beta, z + h);
            __syncwarp();
        }
        stage_put<OUT, kN>(stage, lane, z + h);
        __syncwarp();
        stage_flush<ES>(stage, lane, WarpBlock<ES>(d, p.ldd, row0, col + h, lane), nrow, ncol - h);
        __syncwarp();
    }
}

// Wait for this thread's TMEM loads; v is not to be touched before.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(v[i]));
}

// ---------------------------------------------------------------------------- the kernel
__host__ __device__ constexpr bool lm_wide(int epi)
{
    return epi == kEpiWide || epi == kEpiXentStats || epi == kEpiXentGrad;
}

template <int EPI, int OUT, int BN, bool RK>
__global__ void __launch_bounds__(LmCfg<BN, lm_wide(EPI)>::kThreadsLm, 1)
    tcg_lm_kernel(const __grid_constant__ LmMaps maps, const LmArgs p)
{
    constexpr bool WIDE = lm_wide(EPI);
    using Cfg = LmCfg<BN, WIDE>;
    constexpr int kStages = Cfg::kStages;
    constexpr int kAccBufs = Cfg::kAccBufs;
    constexpr int kBRows = Cfg::kBRows;
    // The tensor core adds each product of 16 K elements to its FP32 accumulator with
    // truncation, an error that grows with K and always toward zero (with K = 4096 and 1.5
    // standard deviations of logits it moved the loss by 2e-6 of itself).  Where results
    // are FP32 statistics, or the accumulators few, K goes in segments of 512: each starts a
    // new accumulator, and the epilogue adds the segments in registers, rounding to nearest.
    // The gradient of the logits is among them: it takes a certain row's exp(logit - lse) from
    // one, so its logits have to be those of the statistics (in one piece, K = 4096 and a logit
    // of 40 left -6e-4 where nothing should be).
    constexpr bool SEG = EPI != kEpiWide && !(EPI == kEpiNarrow && BN == 256);
    // Narrow tiles of 256 tokens: a group's last tile is multiplied at the width it has, in
    // steps of 32 tokens (tensor time follows N), so that a group of any size wastes 16
    // tokens of work on average.
    constexpr bool FIT = EPI == kEpiNarrow && BN == 256;
    auto width = [](const LmUnit &w) {
        return FIT ? min(BN, (w.col_end - w.col0 + 31) & ~31) : BN;
    };
    constexpr int kSegBlocks = SEG ? 8 : 1 << 30;
    using Walk = LmWalk<WIDE, BN, RK>;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw_u32);
    const uint32_t a_smem = base;
    const uint32_t b_smem = base + kStages * Cfg::kAStage;
    LmCtl *ctl = reinterpret_cast<LmCtl *>(base_ptr + kLmDataBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x / 2;
    const int pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < kAccBufs; ++a) {
            mbar_init(smem_u32(&ctl->acc_full[a]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[a]), Cfg::kEpi * 2);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_mbar_init();
        if (!RK && p.num_k_blocks > 0) {
            tma_prefetch_map(&maps.A);
            tma_prefetch_map(&maps.B);
        }
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    if (threadIdx.x == 0)
        griddep_launch_dependents();
    // The plan of a grouped call reads its offsets, which the kernel before may have written;
    // others wait for that kernel only when their roles begin, the plan made and the first
    // unit found.
    if (p.offsets)
        griddep_wait();
    if (warp == 2)
        make_plan<WIDE, BN, RK>(p, ctl, lane, pairs);
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;

    constexpr uint32_t kKmma = 16;
    constexpr int kMmasPerStage = 4;
    constexpr int kKRow = 64;                                 // K elements per stage
    constexpr uint32_t kChunkBytes = kKRow * kRowBytes;       // 64 M/N elements of the stage
    auto layout = [&](int mode, uint32_t &lbo, uint32_t &sbo, uint32_t *off) {
        sbo = 8 * kRowBytes;
        lbo = mode == kK ? 16u : kChunkBytes;
#pragma unroll
        for (int j = 0; j < kMmasPerStage; ++j)
            off[j] = (mode == kK ? j * 32u : j * kKmma * kRowBytes) >> 4;
    };
    uint32_t issued_mask = 0, issued_parity = 0;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ producer
            Walk walk(pair, pairs);
            LmUnit w;
            int stage = 0;
            uint32_t phase = 0;
            bool skip_once = p.fault_inject != 0 && leader;
            bool ok = true;
            const CUtensorMap *map_a = &maps.A, *map_b = &maps.B;
            int maps_of = -1;
            bool more = walk.next(p, ctl, w);
            if (!p.offsets)
                griddep_wait();
            for (; ok && more; more = walk.next(p, ctl, w)) {
                const int m0 = w.row0 + static_cast<int>(rank) * kBM;
                const int n0 = w.col0 + static_cast<int>(rank) * (width(w) / 2);
                const int za = WIDE ? 0 : w.g, zb = WIDE && !RK ? w.g : 0;
                // maps that end with the group; without tokens there are none
                if (RK && w.kb0 < w.kb1 && w.g != maps_of) {
                    maps_of = w.g;
                    map_a = p.group_maps + 2 * w.g;
                    map_b = map_a + 1;
                    fence_tensormap_acquire(map_a);
                    fence_tensormap_acquire(map_b);
                }
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    const uint32_t fb_local = smem_u32(&ctl->full[stage]);
                    const uint32_t fb = mapa_shared(fb_local, 0);
                    if (!wait_bounded<2>(smem_u32(&ctl->empty[stage]), phase ^ 1u, ctl, p,
                                         kErrProducer)) {
                        ok = false;
                        break;
                    }
                    if (skip_once) {
                        skip_once = false;      // test hook: this stage is never filled
                    } else {
                        if (leader) {
                            mbar_arrive_expect_tx(fb_local, Cfg::kStageBytes * 2);
                            issued_mask |= 1u << stage;
                            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                        }
                        const uint32_t sa = a_smem + stage * Cfg::kAStage;
                        const uint32_t sb = b_smem + stage * Cfg::kBStage;
                        const int k0 = (RK ? w.tok0 : 0) + kb * kKRow;
                        auto load = [&](uint32_t dst, const CUtensorMap *map, int mode, int rows,
                                        int row0, int z) {
                            if (mode == kK)
                                tma_load_3d_pair(dst, map, fb, k0, row0, z);
                            else if (mode == kMN4)
                                tma_load_4d_pair(dst, map, fb, 0, k0, row0 / 64, z);
                            else
                                for (int h = 0; h < rows / 64; ++h)
                                    tma_load_3d_pair(dst + h * kChunkBytes, map, fb, row0 + h * 64,
                                                     k0, z);
                        };
                        load(sa, map_a, p.a_mode, kBM, m0, za);
                        load(sb, map_b, p.b_mode, kBRows, n0, zb);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ----------------------------------------------------------- MMA issue
            uint32_t a_lbo, a_sbo, b_lbo, b_sbo, a_off[kMmasPerStage], b_off[kMmasPerStage];
            layout(p.a_mode, a_lbo, a_sbo, a_off);
            layout(p.b_mode, b_lbo, b_sbo, b_off);
            const uint64_t a_desc0 = smem_desc_sw128(a_smem, a_lbo, a_sbo);
            const uint64_t b_desc0 = smem_desc_sw128(b_smem, b_lbo, b_sbo);
            Walk walk(pair, pairs);
            LmUnit w, next_w;
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            bool ok = true;
            bool more = walk.next(p, ctl, w);
            if (!p.offsets)
                griddep_wait();                            // so that no wait below includes the kernel before
            while (ok && more) {
                bool looked = false;                       // the next unit is known
                int kb = w.kb0;
                do {                                       // one accumulator per segment
                    const int acc = it % kAccBufs;
                    const uint32_t acc_phase = (it / kAccBufs) & 1;
                    ++it;
                    if (!wait_bounded<2>(smem_u32(&ctl->acc_empty[acc]), acc_phase ^ 1u, ctl, p,
                                         kErrMmaAcc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                    const uint32_t idesc = FIT ? (p.idesc & ~(0x3Fu << 17)) |
                                                     (static_cast<uint32_t>(width(w) >> 3) << 17)
                                               : p.idesc;
                    const int first = kb, stop = SEG ? min(kb + kSegBlocks, w.kb1) : w.kb1;
                    for (; kb < stop; ++kb) {
                        if (!wait_bounded<2>(smem_u32(&ctl->full[stage]), phase, ctl, p, kErrMmaFull)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad_s = a_desc0 + ((static_cast<uint32_t>(stage) * Cfg::kAStage) >> 4);
                        const uint64_t bd_s = b_desc0 + ((static_cast<uint32_t>(stage) * Cfg::kBStage) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kMmasPerStage; ++kk)
                            mma_f16_pair(d_tmem, ad_s + a_off[kk], bd_s + b_off[kk], idesc,
                                         (kb > first || kk > 0) ? 1u : 0u);
                        mma_commit_pair_mc(smem_u32(&ctl->empty[stage]), 0x3);
                        if (!looked) {                     // while the tensor core is busy
                            more = walk.next(p, ctl, next_w);
                            looked = true;
                        }
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok)
                        break;
                    mma_commit_pair_mc(smem_u32(&ctl->acc_full[acc]), 0x3);
                } while (kb < w.kb1);
                if (!looked)
                    more = walk.next(p, ctl, next_w);
                w = next_w;
            }
            mma_commit_pair(smem_u32(&ctl->drain));
            wait_bounded<2>(smem_u32(&ctl->drain), 0, ctl, p, kErrDrain, false);
        }
    } else {
        // -------------------------------------------------------------- epilogue
        // Parts of 4 warps; part h owns columns [h kPart, (h + 1) kPart) of each tile for the
        // CTA's 128 rows (warp w reads TMEM lane quarter w % 4).
        constexpr int kParts = Cfg::kParts;
        constexpr int kPart = BN / kParts;
        const int q = warp & 3;
        const int part = (warp - 2) >> 2;
        const bool part_leader = (warp == 2 + 4 * part) && lane == 0;
        const uint32_t bar_id = 1u + static_cast<uint32_t>(part);
        const int rl = q * 32 + lane;
        const uint32_t tmem_part = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(part * kPart);
        if (!p.offsets)
            griddep_wait();
        const float alpha = p.alpha * (p.alpha_dev ? *p.alpha_dev : 1.0f);
        uint8_t *stage = base_ptr + kLmDataBytes - Cfg::kEpi * kLmStageBytes + (warp - 2) * kLmStageBytes;
        Walk walk(pair, pairs);
        LmUnit w{};
        int it = 0;

        // The next accumulator, once it is complete; false: stop.
        auto acquire = [&]() {
            const int acc = it % kAccBufs;
            const bool ok = wait_bounded<2>(smem_u32(&ctl->acc_full[acc]), (it / kAccBufs) & 1, ctl, p,
                                            kErrEpilogue);
            const bool stop = named_barrier_or(bar_id, 128, !ok || ctl->abort_flag);
            tc_fence_after();
            return !stop;
        };
        // This warp has read the accumulator: report to the MMA CTA, go on to the next.
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctl->acc_empty[it % kAccBufs]), 0));
            ++it;
        };
        // A cut tile's piece is stored: whoever stores the last one of a tile part adds them
        // all, in K order whatever the timing, and finishes the tile.  One thread's fence,
        // after the barrier, orders the stores of all.
        auto arrive = [&]() {
            named_barrier_sync(bar_id, 128);
            if (part_leader) {
                uint32_t *cnt = p.cnt + (w.counter * 2 + static_cast<int>(rank)) * kParts + part;
                fence_acq_rel_gpu();
                const bool last = atomicAdd(cnt, 1u) == static_cast<uint32_t>(w.pieces - 1);
                if (last)
                    *cnt = 0u;                             // every piece has arrived
                ctl->last_arrival[part] = last;
                fence_acq_rel_gpu();
            }
            named_barrier_sync(bar_id, 128);
            const bool last = ctl->last_arrival[part] != 0;
            named_barrier_sync(bar_id, 128);               // the flag is free again
            return last;
        };
        auto slot_ptr = [&](int slot) {
            return p.part + ((static_cast<int64_t>(slot) * 2 + rank) * kParts + part) * (kPart * kBM);
        };
        auto piece_slot = [&](int i) { return 2 * (w.first_pair + i) + (i == 0 ? 1 : 0); };

        while (walk.next(p, ctl, w)) {
            const int row = w.row0 + static_cast<int>(rank) * kBM + rl;
            const int col_part = w.col0 + part * kPart;
            const bool cut = w.slot >= 0;
            const bool empty_k = w.kb0 >= w.kb1;
            const int segments = SEG ? (w.kb1 - w.kb0 + kSegBlocks - 1) / kSegBlocks : 1;
            if constexpr (FIT) {
                // --------------------------- tokens on the columns, many: the parts take
                // every second 32 of them
                float bias = 0.0f;
                if (p.bias && row < p.rows && w.g >= 0) {
                    const int64_t i = static_cast<int64_t>(w.g) * p.rows + row;
                    bias = p.bias_f32 ? static_cast<const float *>(p.bias)[i]
                                      : load16(p.bias, i, p.in_bf16);
                }
                if (!acquire())
                    break;
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                       static_cast<uint32_t>(it % kAccBufs * BN);
                const int chunks = width(w) / 32;
                uint32_t v[32];
                __syncwarp();
                if (part < chunks)
                    tmem_ld_32x32b_x32(taddr + 32 * part, v);
                else
                    release();
#pragma unroll 1
                for (int c = part; c < chunks; c += kParts) {
                    float z[32];
                    tmem_ld_done(v);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        z[j] = empty_k ? 0.0f : __uint_as_float(v[j]);
                    __syncwarp();
                    if (c + kParts < chunks)
                        tmem_ld_32x32b_x32(taddr + 32 * (c + kParts), v);
                    else
                        release();
                    finish_narrow<OUT, 32>(p, z, w, row, w.col0 + c * 32, alpha, bias);
                }
            } else if constexpr (EPI == kEpiNarrow || EPI == kEpiXentNarrow) {
                // ------------------------------------------------ tokens on the columns
                constexpr int kCols = kPart < 32 ? kPart : 32;
                float sum[kPart];
#pragma unroll
                for (int j = 0; j < kPart; ++j)
                    sum[j] = 0.0f;
                float bias = 0.0f;
                if (EPI == kEpiNarrow && p.bias && row < p.rows && w.g >= 0) {
                    const int64_t i = static_cast<int64_t>(w.g) * p.rows + row;
                    bias = p.bias_f32 ? static_cast<const float *>(p.bias)[i]
                                      : load16(p.bias, i, p.in_bf16);
                }
                bool stop = false;
                int seg = 0;
                do {
                    if (!acquire()) {
                        stop = true;
                        break;
                    }
                    uint32_t v[kPart];
                    const uint32_t taddr = tmem_part + static_cast<uint32_t>(it % kAccBufs * BN);
                    if constexpr (kPart == 16) {
                        tmem_ld_32x32b_x16(taddr, v);
                    } else {
#pragma unroll
                        for (int c = 0; c < kPart; c += 32)
                            tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t (*)[32]>(v + c));
                    }
                    tmem_ld_done(v);
                    release();
                    if (!empty_k) {
#pragma unroll
                        for (int j = 0; j < kPart; ++j)
                            sum[j] += __uint_as_float(v[j]);
                    }
                } while (++seg < segments);
                if (stop)
                    break;
                const int ncol = w.col_end - col_part;
                if (cut) {
                    // 16 columns at a time, whether all hold tokens or not: loads that each
                    // ask for themselves wait for each other (100 tokens, 4096 x 4096: 27 us)
                    float *sl = slot_ptr(w.slot) + rl;     // [column][row]
#pragma unroll
                    for (int c = 0; c < kPart; c += 16)
                        if (c < ncol) {
#pragma unroll
                            for (int j = c; j < c + 16; ++j)
                                __stcg(sl + j * kBM, sum[j]);
                        }
                    if (!arrive())
                        continue;
#pragma unroll
                    for (int c = 0; c < kPart; c += 16) {
                        if (c >= ncol)
                            break;
#pragma unroll
                        for (int j = c; j < c + 16; ++j)
                            sum[j] = 0.0f;
#pragma unroll 4
                        for (int i = 0; i < w.pieces; ++i) {
                            const float *s = slot_ptr(piece_slot(i)) + rl + c * kBM;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                sum[c + j] += __ldcg(s + j * kBM);
                        }
                    }
                }
                if constexpr (EPI == kEpiNarrow) {
#pragma unroll
                    for (int c = 0; c < kPart; c += kCols)
                        finish_narrow<OUT>(p, *reinterpret_cast<float (*)[kCols]>(sum + c), w, row,
                                           col_part + c, alpha, bias);
                } else {
                    // a warp's 32 vocabulary entries, one token (column) after the other
                    const int slot = (w.row0 >> 8) * 8 + static_cast<int>(rank) * 4 + q;
#pragma unroll
                    for (int j = 0; j < kPart; ++j) {
                        if (j >= ncol)
                            break;
                        const int tok = col_part + j;
                        const int64_t t = p.targets[tok];
                        const float v = row < p.rows ? sum[j] : -INFINITY;
                        if (t == row && t != p.ignore && row < p.rows)
                            p.target_logit[tok] = v;
                        float mx = v;
#pragma unroll
                        for (int d = 16; d; d >>= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        float s = exp_from(v, exp_base(mx));
#pragma unroll
                        for (int d = 16; d; d >>= 1)
                            s += __shfl_xor_sync(0xffffffffu, s, d);
                        if (lane == 0)
                            p.stats[static_cast<int64_t>(slot) * p.tokens + tok] = make_float2(mx, s);
                    }
                }
            } else if constexpr (EPI == kEpiWide) {
                // --------------------------------------------------- tokens on the rows
                constexpr int kChunks = kPart / 32;
                if (!acquire())
                    break;
                const uint32_t taddr = tmem_part + static_cast<uint32_t>(it % kAccBufs * BN);
                float *sl = cut ? slot_ptr(w.slot) + rl : nullptr;       // [column][row]
                uint32_t v[32];
                __syncwarp();
                tmem_ld_32x32b_x32(taddr, v);
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    const int col = col_part + c * 32;
                    const bool inside = row - lane < w.row_end && col < w.col_end;
                    float z[32];
                    tmem_ld_done(v);
                    if (empty_k) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = 0u;
                    }
                    if (cut) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            __stcg(sl + (c * 32 + j) * kBM, __uint_as_float(v[j]));
                    } else if (inside) {
                        scale_bias(p, alpha, static_cast<int64_t>(w.g) * p.cols + col, w.g < 0 ? 0 : w.col_end - col,
                                   stage, lane, v, z);
                    }
                    __syncwarp();
                    if (c + 1 < kChunks)               // on its way while this chunk is finished
                        tmem_ld_32x32b_x32(taddr + 32 * (c + 1), v);
                    else
                        release();
                    if (!cut && inside)
                        finish_wide<OUT>(p, z, w, row - lane, col, stage, lane);
                }
                if (cut && arrive() && row - lane < w.row_end) {
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c) {
                        const int col = col_part + c * 32;
                        if (col >= w.col_end)
                            break;
                        float z[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            z[j] = 0.0f;
#pragma unroll 2
                        for (int i = 0; i < w.pieces; ++i) {
                            const float *q = slot_ptr(piece_slot(i)) + c * 32 * kBM + rl;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                z[j] += __ldcg(q + j * kBM);
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(z[j]);
                        scale_bias(p, alpha, static_cast<int64_t>(w.g) * p.cols + col, w.col_end - col, stage,
                                   lane, v, z);
                        finish_wide<OUT>(p, z, w, row - lane, col, stage, lane);
                    }
                }
            } else {
                // ------------------------------------ cross entropy, tokens on the rows
                const bool row_ok = row < p.rows;
                float row_lse = 0.0f, row_g = 0.0f;
                int target = -1;                           // column of the row's target
                if (row_ok) {
                    const int64_t t = p.targets[row];
                    const bool counts = t != p.ignore && t >= 0 && t < p.vocab;
                    if (counts && t >= p.col0 && t - p.col0 < p.cols)
                        target = static_cast<int>(t - p.col0);
                    if constexpr (EPI == kEpiXentGrad) {
                        row_lse = p.lse[row];
                        row_g = counts ? p.dloss[row] * (p.gscale ? *p.gscale : 1.0f) : 0.0f;
                    }
                }
                // the logits of the row, segment after segment
                float sum[kPart];
#pragma unroll
                for (int j = 0; j < kPart; ++j)
                    sum[j] = 0.0f;
                bool stop = false;
                for (int seg = 0; seg < segments; ++seg) {
                    if (!acquire()) {
                        stop = true;
                        break;
                    }
                    const uint32_t taddr = tmem_part + static_cast<uint32_t>(it % kAccBufs * BN);
                    uint32_t va[16], vb[16];
                    tmem_ld_32x32b_x16(taddr, va);
#pragma unroll
                    for (int c = 0; c < kPart; c += 32) {
                        tmem_ld_done(va);
                        tmem_ld_32x32b_x16(taddr + c + 16, vb);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[c + j] += __uint_as_float(va[j]);
                        tmem_ld_done(vb);
                        if (c + 32 < kPart)
                            tmem_ld_32x32b_x16(taddr + c + 32, va);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[c + 16 + j] += __uint_as_float(vb[j]);
                    }
                    release();
                }
                if (stop)
                    break;
                if constexpr (EPI == kEpiXentStats) {
                    const int ncol = w.col_end - col_part;
                    if (ncol < kPart) {
#pragma unroll
                        for (int j = 0; j < kPart; ++j)
                            if (j >= ncol)
                                sum[j] = -INFINITY;
                    }
                    if (target >= col_part && target < col_part + kPart) {
                        float tl = 0.0f;
#pragma unroll
                        for (int j = 0; j < kPart; ++j)    // by predicate: the sums stay in registers
                            asm("{\n\t.reg .pred q;\n\tsetp.eq.s32 q, %1, %2;\n\t"
                                "@q mov.f32 %0, %3;\n\t}"
                                : "+f"(tl)
                                : "r"(target - col_part), "r"(j), "f"(sum[j]));
                        p.target_logit[row] = tl;
                    }
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kPart; ++j)
                        mx = fmaxf(mx, sum[j]);
                    const F2 less = f2(-exp_base(mx));
                    float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < kPart; j += 2) {
                        float e0, e1;
                        split2(exp_from(f2(sum[j], sum[j + 1]), less), e0, e1);
                        add[j & 3] += e0;
                        add[(j & 3) + 1] += e1;
                    }
                    if (row_ok)
                        p.stats[static_cast<int64_t>(w.col0 / BN * kParts + part) * p.tokens + row] =
                            make_float2(mx, (add[0] + add[1]) + (add[2] + add[3]));
                } else {
#pragma unroll
                    for (int c = 0; c < kPart; c += 32) {
                        const int col = col_part + c;
                        if (col >= w.col_end || row - lane >= w.row_end)
                            break;
                        float *g = sum + c;
                        const F2 less = f2(-row_lse), scale = f2(row_g);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            split2(exp_from(f2(g[j], g[j + 1]), less), g[j], g[j + 1]);
                        if (target >= col && target < col + 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                g[j] -= target == col + j ? 1.0f : 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            split2(f2(g[j], g[j + 1]) * scale, g[j], g[j + 1]);
                        if (row_g == 0.0f) {             // whatever the logits hold
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                g[j] = 0.0f;
                        }
                        __syncwarp();
                        if (p.in_bf16)
                            stage_put<kOutBF16, 32>(stage, lane, g);
                        else
                            stage_put<kOutF16, 32>(stage, lane, g);
                        __syncwarp();
                        stage_flush<2>(stage, lane, WarpBlock<2>(p.D, p.ldd, row - lane, col, lane),
                                       w.row_end - (row - lane), w.col_end - col);
                    }
                    __syncwarp();
                }
            }
        }
    }

    tc_fence_before();
    cluster_sync_all();
    if (ctl->abort_flag && warp == 0 && lane == 0) {
        // Aborted: let every load already issued land before the CTA leaves.
        if (leader)
            for (int s = 0; s < kStages; ++s)
                if (issued_mask & (1u << s))
                    wait_bounded<2>(smem_u32(&ctl->full[s]), (issued_parity >> s) & 1u, ctl, p,
                                    kErrDrain, false);
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000ull) {
        }
    }
    cluster_sync_all();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

typedef void (*LmKernelFn)(const LmMaps, const LmArgs);

template <int OUT>
LmKernelFn linear_fn(int epi, int bn, bool rk)
{
    if (rk)
        return tcg_lm_kernel<kEpiWide, OUT, 256, true>;
    if (epi == kEpiNarrow)
        return bn == 32 ? tcg_lm_kernel<kEpiNarrow, OUT, 32, false>
             : bn == 64 ? tcg_lm_kernel<kEpiNarrow, OUT, 64, false>
             : bn == 128 ? tcg_lm_kernel<kEpiNarrow, OUT, 128, false>
                         : tcg_lm_kernel<kEpiNarrow, OUT, 256, false>;
    return bn == 64 ? tcg_lm_kernel<kEpiWide, OUT, 64, false>
         : bn == 128 ? tcg_lm_kernel<kEpiWide, OUT, 128, false>
                     : tcg_lm_kernel<kEpiWide, OUT, 256, false>;
}

LmKernelFn lm_fn(int epi, int out_kind, int bn, bool rk)
{
    if (epi == kEpiXentStats)
        return tcg_lm_kernel<kEpiXentStats, kOutF32, 256, false>;
    if (epi == kEpiXentNarrow)
        return tcg_lm_kernel<kEpiXentNarrow, kOutF32, 32, false>;
    if (epi == kEpiXentGrad)
        return tcg_lm_kernel<kEpiXentGrad, kOutF16, 256, false>;
    return out_kind == kOutF32 ? linear_fn<kOutF32>(epi, bn, rk)
         : out_kind == kOutF16 ? linear_fn<kOutF16>(epi, bn, rk) : linear_fn<kOutBF16>(epi, bn, rk);
}

// ------------------------------------------------------------------- smaller kernels
// One block per 32 rows; lane = row, the warps share the slots and join through shared
// memory.  Adds the slots' sums relative to the row's maximum.
constexpr int kCombineWarps = 16;
__global__ void __launch_bounds__(32 * kCombineWarps)
    tcg_xent_combine_kernel(const float2 *__restrict__ stats, int slots, int rows,
                            const float *__restrict__ target_logit,
                            const int64_t *__restrict__ targets, int64_t vocab, int64_t ignore,
                            float *__restrict__ loss, float *__restrict__ lse)
{
    __shared__ float2 part[kCombineWarps][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + lane;
    float2 acc = make_float2(-INFINITY, 0.0f);
    if (row < rows) {
#pragma unroll 4
        for (int s = w; s < slots; s += kCombineWarps)
            acc = join_stats(acc, __ldcg(stats + static_cast<int64_t>(s) * rows + row));
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w == 0 && row < rows) {
        for (int i = 1; i < kCombineWarps; ++i)
            acc = join_stats(acc, part[i][lane]);
        const float l = acc.x + logf(acc.y);
        const int64_t t = targets[row];
        const bool counts = t != ignore && t >= 0 && t < vocab;
        lse[row] = l;
        loss[row] = counts ? l - target_logit[row] : 0.0f;
    }
}

// One block for up to kScaleRows rows.  More blocks leave their maxima behind the result, and the
// last of them to arrive joins them: a maximum is the same in any order.
constexpr int kScaleRows = 4096, kScaleBlocks = 32;
__global__ void __launch_bounds__(1024)
    tcg_xent_scale_kernel(const float *__restrict__ dloss, const int64_t *__restrict__ targets,
                          int rows, int64_t vocab, int64_t ignore, float *scale, uint32_t *cnt)
{
    __shared__ float part[32];
    griddep_launch_dependents();
    griddep_wait();
    float m = 0.0f;
#pragma unroll 4
    for (int64_t i = blockIdx.x * 1024ll + threadIdx.x; i < rows; i += gridDim.x * 1024ll) {
        const int64_t t = targets[i];
        const float d = fabsf(dloss[i]);
        m = t != ignore && t >= 0 && t < vocab ? fmaxf(m, d) : m;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 32; ++i)
            m = fmaxf(m, part[i]);
        if (gridDim.x > 1) {
            __stcg(scale + 2 + blockIdx.x, m);
            fence_acq_rel_gpu();
            if (atomicAdd(cnt, 1u) != gridDim.x - 1)
                return;
            *cnt = 0u;                         // every block has arrived
            fence_acq_rel_gpu();
            for (int i = 0; i < static_cast<int>(gridDim.x); ++i)
                m = fmaxf(m, __ldcg(scale + 2 + i));
        }
        float f = 1.0f;
        int e = 0;
        if (m > 0.0f && m < INFINITY) {
            f = frexpf(m, &e);                 // m = f 2^e, 1/2 <= f < 1
            e = 14 - e;
            e = e > 100 ? 100 : e;
        }
        scale[0] = ldexpf(1.0f / f, e);
        scale[1] = ldexpf(f, -e);
    }
}

template <int OUT>
__global__ void __launch_bounds__(256)
    tcg_round_out_kernel(const float *__restrict__ in, int64_t ldi, int rows, int cols,
                         const float *__restrict__ scale, uint16_t *__restrict__ out, int64_t ldo)
{
    griddep_launch_dependents();
    griddep_wait();
    const float s = scale ? *scale : 1.0f;
    const int r4 = (rows + 3) / 4;
    const int64_t total = static_cast<int64_t>(r4) * cols;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int c = static_cast<int>(i / r4);
        const int r = static_cast<int>(i - static_cast<int64_t>(c) * r4) * 4;
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(in + c * ldi + r));
        const float x[4] = {v.x, v.y, v.z, v.w};
        uint16_t *o = out + c * ldo + r;
        uint16_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            y[j] = round16(s * x[j], OUT == kOutBF16);
        if (r + 3 < rows)
            *reinterpret_cast<uint2 *>(o) = make_uint2(y[0] | static_cast<uint32_t>(y[1]) << 16,
                                                       y[2] | static_cast<uint32_t>(y[3]) << 16);
        else
            for (int j = 0; j < 4; ++j)
                if (r + j < rows)
                    o[j] = y[j];
    }
}

// One warp per group copies the two maps and sets their token extent (dimension 1 of either
// layout) to the group's end.  An empty group's maps are never used; extents are at least 1.
__global__ void __launch_bounds__(128)
    tcg_group_maps_kernel(const __grid_constant__ LmMaps maps, const int64_t *__restrict__ offsets,
                          int groups, int tokens, CUtensorMap *out)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, g = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (g >= groups)
        return;
    static_assert(sizeof(CUtensorMap) == 128, "32 words");
    int b, e;
    group_range(offsets, tokens, g, b, e);
    for (int x = 0; x < 2; ++x)
        reinterpret_cast<uint32_t *>(out + 2 * g + x)[lane] =
            reinterpret_cast<const uint32_t *>(x ? &maps.B : &maps.A)[lane];
    __syncwarp();
    if (lane < 2)
        tensormap_set_dim<1>(out + 2 * g + lane, static_cast<uint32_t>(e > 0 ? e : 1));
    fence_tensormap_release();
}

// dZ = dD act'(Z) (column-major m x cols; dZ may be left out), and for each group the sum
// of its columns of dZ before rounding.  Bound by memory: dD and Z are read once and dZ is
// written once, 16 bytes a thread.  Block (x, y): rows 256 x .. + 255 of the y-th `chunk`
// columns; a warp takes a column at a time, the eight warps every eighth column.  The
// columns of a block fall into segments, one per group that meets it; a segment's sums go
// to slot y + g of `part` -- (y, g) steps through a monotone path, so slots are distinct
// and there are chunks + groups of them -- and tcg_bias_join_kernel adds a group's
// segments in order.  Columns of no group get zeros.
template <int ACT, bool BF16>
__global__ void __launch_bounds__(256)
    tcg_epi_backward_kernel(int m, int cols, int groups, const int64_t *__restrict__ offsets,
                            const uint16_t *dD, int64_t lddd, const uint16_t *Z, int64_t ldz,
                            uint16_t *dZ, int64_t lddz, float *__restrict__ part, int chunk)
{
    __shared__ float join[8][256 + 8];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * 256 + lane * 8;
    const int left = m - row;                         // rows of this thread (8, or fewer at the end)
    const int c0 = blockIdx.y * chunk, c1 = min(c0 + chunk, cols);

    auto load8 = [&](const uint16_t *src) {
        if (left >= 8)
            return *reinterpret_cast<const uint4 *>(src);
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left)
                u[i / 2] |= static_cast<uint32_t>(src[i]) << (16 * (i & 1));
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    auto store8 = [&](uint16_t *dst, const float (&v)[8]) {
        if (left >= 8) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = pack16(v[2 * i], v[2 * i + 1], BF16);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    dst[i] = round16(v[i], BF16);
        }
    };
    auto clear = [&](int from, int to) {
        const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (dZ && left > 0)
            for (int c = from + w; c < to; c += 8)
                store8(dZ + static_cast<int64_t>(c) * lddz + row, zero);
    };

    int g = 0, at = c0;
    if (offsets) {                                    // first group that ends past c0
        int hi = groups;
        while (g < hi) {
            const int mid = (g + hi) >> 1;
            if (offsets[mid + 1] > c0)
                hi = mid;
            else
                g = mid + 1;
        }
    }
    for (; at < c1 && g < groups; ++g) {
        int b, e;
        group_range(offsets, cols, g, b, e);
        b = max(b, at);
        e = min(e, c1);
        if (b >= c1)
            break;
        clear(at, b);
        at = b;
        if (e <= b)
            continue;
        float sum[8] = {};
        if (left > 0) {
            // Four columns at a time, all their loads before the first store (dZ may be dD, so
            // the compiler would not move a load up past a store).
            for (int c = b + w; c < e; c += 32) {
                uint4 rd[4], rz[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t col = c + 8 * k;
                    if (col < e) {
                        rd[k] = load8(dD + col * lddd + row);
                        if constexpr (ACT != kActNone)
                            rz[k] = load8(Z + col * ldz + row);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t col = c + 8 * k;
                    if (col >= e)
                        break;
                    float d[8];
                    unpack16<BF16>(rd[k], d);
                    if constexpr (ACT != kActNone) {
                        float z[8];
                        unpack16<BF16>(rz[k], z);
#pragma unroll
                        for (int i = 0; i < 8; i += 2)
                            split2(f2(d[i], d[i + 1]) * act_slope<ACT>(f2(z[i], z[i + 1])), d[i], d[i + 1]);
                    }
                    if (dZ)
                        store8(dZ + col * lddz + row, d);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[i] += d[i];
                }
            }
        }
        at = e;
        if (part) {
            __syncthreads();                          // the previous segment has been added
#pragma unroll
            for (int i = 0; i < 8; ++i)
                join[w][lane * 8 + i] = sum[i];
            __syncthreads();
            const int r = blockIdx.x * 256 + threadIdx.x;
            if (r < m) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s += join[i][threadIdx.x];
                part[(static_cast<int64_t>(blockIdx.y) + g) * m + r] = s;
            }
        }
    }
    clear(at, c1);
}

// dbias of group blockIdx.y: its segments in column order, the four warps of 64 rows taking
// a quarter of them each.
__global__ void __launch_bounds__(256)
    tcg_bias_join_kernel(const float *__restrict__ part, int m, int cols, int groups,
                         const int64_t *__restrict__ offsets, int chunk, float *__restrict__ dbias)
{
    __shared__ float join[4][64];
    griddep_launch_dependents();
    griddep_wait();
    const int g = blockIdx.y, lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int row = blockIdx.x * 64 + lane;
    int b, e;
    group_range(offsets, cols, g, b, e);
    const int y0 = b / chunk, y1 = e > b ? (e - 1) / chunk + 1 : y0;
    const int a0 = y0 + (y1 - y0) * q / 4, a1 = y0 + (y1 - y0) * (q + 1) / 4;
    float s = 0.0f;
    if (row < m) {
#pragma unroll 8
        for (int y = a0; y < a1; ++y)
            s += part[(static_cast<int64_t>(y) + g) * m + row];
    }
    join[q][lane] = s;
    __syncthreads();
    if (q == 0 && row < m)
        dbias[static_cast<int64_t>(g) * m + row] = ((s + join[1][lane]) + join[2][lane]) + join[3][lane];
}

}  // namespace

cudaError_t launch_lm(const LmMaps &maps, const LmArgs &a, int epi, int out_kind, int bn, int grid,
                      cudaStream_t s)
{
    const LmKernelFn fn = lm_fn(epi, out_kind, bn, a.ragged_k != 0);
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kLmSmemBytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(LmCfg<256, true>::kThreadsLm, 1, 1);   // the same for every kind
    cfg.dynamicSmemBytes = kLmSmemBytes;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, fn, maps, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int lm_max_resident_ctas(int num_sms)
{
    const LmKernelFn fn = tcg_lm_kernel<kEpiXentStats, kOutF32, 256, false>;
    if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kLmSmemBytes) != cudaSuccess)
        return num_sms / 2 * 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(num_sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(LmCfg<256, true>::kThreadsLm, 1, 1);
    cfg.dynamicSmemBytes = kLmSmemBytes;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) != cudaSuccess || clusters < 1) {
        cudaGetLastError();
        return num_sms / 2 * 2;
    }
    return clusters * 2;
}

cudaError_t launch_group_maps(const LmMaps &maps, const int64_t *offsets, int groups, int tokens,
                              CUtensorMap *out, cudaStream_t s)
{
    return launch_pdl(tcg_group_maps_kernel, dim3((groups + 3) / 4), dim3(128), s, 0, maps, offsets,
                      groups, tokens, out);
}

cudaError_t launch_xent_combine(const float2 *stats, int slots, int rows, const float *target_logit,
                                const int64_t *targets, int64_t vocab, int64_t ignore, float *loss,
                                float *lse, cudaStream_t s)
{
    return launch_pdl(tcg_xent_combine_kernel, dim3((rows + 31) / 32), dim3(32 * kCombineWarps), s, 0,
                      stats, slots, rows, target_logit, targets, vocab, ignore, loss, lse);
}

cudaError_t launch_xent_scale(const float *dloss, const int64_t *targets, int rows, int64_t vocab,
                              int64_t ignore, float *scale, uint32_t *cnt, cudaStream_t s)
{
    const int blocks = (rows + kScaleRows - 1) / kScaleRows;
    return launch_pdl(tcg_xent_scale_kernel, dim3(blocks < kScaleBlocks ? blocks : kScaleBlocks), dim3(1024), s,
                      0, dloss, targets, rows, vocab, ignore, scale, cnt);
}

cudaError_t launch_round_out(const float *in, int64_t ldi, int rows, int cols, const float *scale,
                             void *out, int64_t ldo, int out_kind, int grid, cudaStream_t s)
{
    return launch_pdl(out_kind == kOutBF16 ? tcg_round_out_kernel<kOutBF16>
                                           : tcg_round_out_kernel<kOutF16>,
                      dim3(grid), dim3(256), s, 0, in, ldi, rows, cols, scale,
                      static_cast<uint16_t *>(out), ldo);
}

template <int ACT>
static cudaError_t epi_backward(int bf16, dim3 grid, cudaStream_t s, int m, int cols, int groups,
                                const int64_t *offsets, const void *dD, int64_t lddd, const void *Z,
                                int64_t ldz, void *dZ, int64_t lddz, float *part, int chunk)
{
    return launch_pdl(bf16 ? tcg_epi_backward_kernel<ACT, true> : tcg_epi_backward_kernel<ACT, false>,
                      grid, dim3(256), s, 0, m, cols, groups, offsets, static_cast<const uint16_t *>(dD),
                      lddd, static_cast<const uint16_t *>(Z), ldz, static_cast<uint16_t *>(dZ), lddz,
                      part, chunk);
}

cudaError_t launch_epi_backward(int act, int bf16, int m, int cols, int groups,
                                const int64_t *offsets, const void *dD, int64_t lddd, const void *Z,
                                int64_t ldz, void *dZ, int64_t lddz, float *dbias, float *part,
                                int chunk, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (cols > 0) {
        const dim3 grid((m + 255) / 256, (cols + chunk - 1) / chunk);
        auto fn = act == kActRelu ? epi_backward<kActRelu>
                : act == kActGelu ? epi_backward<kActGelu>
                : act == kActGeluTanh ? epi_backward<kActGeluTanh>
                : act == kActSilu ? epi_backward<kActSilu> : epi_backward<kActNone>;
        e = fn(bf16, grid, s, m, cols, groups, offsets, dD, lddd, Z, ldz, dZ, lddz,
               dbias ? part : nullptr, chunk);
    }
    if (e == cudaSuccess && dbias)
        e = launch_pdl(tcg_bias_join_kernel, dim3((m + 63) / 64, groups), dim3(256), s, 0,
                       const_cast<const float *>(part), m, cols, groups, offsets, chunk, dbias);
    return e;
}

}  // namespace tcg
