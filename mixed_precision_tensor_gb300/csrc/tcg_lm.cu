// tcg_lm.cu -- device code of the language-model products (sm_103a).
//
// tcg_lm_kernel is a persistent, warp-specialised tensor-core product over CTA pairs
// (tcgen05, cta_group::2), column-major like the rest of the library:
//
//   kEpiLinear     D_g = act(alpha op(A_g) op(B_g) + bias_g) + beta C_g   for every group g
//   kEpiXentStats  logits L = X W^T in tiles that never leave the chip: per row and tile
//                  half the maximum m and s = sum exp(L - m), and the target's logit
//   kEpiXentGrad   G = dloss (exp(L - lse) - [target]), rounded to 16 bits
//
//   warp 0 (one lane)   TMA producer into a ring of 128-byte-swizzled stages (64 K elements
//                       of 128 rows of A and BN / 2 rows of B per CTA)
//   warp 1 (one lane)   tcgen05.mma, M = 256, N = BN, into TMEM accumulators (up to four)
//   warps 2-9           epilogue: TMEM -> registers -> memory
//
// Every wait is bounded as in tcg_kernels.cu: a wait that runs out sets a bit in the
// device error word, every role stops and the kernel returns.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tcg_lm.h"
#include "tcg_pipe.cuh"

namespace tcg {

namespace {

struct LmCtl {
    uint64_t full[kLmMaxStages];
    uint64_t empty[kLmMaxStages];
    uint64_t acc_full[4];
    uint64_t acc_empty[4];
    uint64_t drain;
    uint32_t tmem_base;
    volatile int abort_flag;
    volatile int last_arrival[2];
    int cum[kLmMaxGroups + 3];    // units before slot s (see lm_slots)
};
constexpr int kLmCtlBytes = 2048;
static_assert(sizeof(LmCtl) <= kLmCtlBytes, "control area too small");
constexpr int kLmSmemBytes = kDataBytes + kLmCtlBytes + 1024;   // + alignment slack

// ------------------------------------------------------------------------- activations
// exp2 and the reciprocal run on the special-function unit (ex2.approx, fast division,
// relative error about 2^-22), below the rounding of every output type but FP32, where
// they are of its own size.
//
// GELU: x Phi(x) = max(x, 0) - |x| erfc(|x| / sqrt 2) / 2, with erfc(a) = (a1 t + ... +
// a5 t^5) exp(-a^2), t = 1 / (1 + p a): Abramowitz & Stegun 7.1.26, |error| <= 1.5e-7.
__device__ __forceinline__ float half_erfc(float ax, float &gauss)
{
    const float a = fminf(ax, 20.0f) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, a, 1.0f));
    gauss = __expf(-a * a);
    float q = fmaf(t, 1.061405429f, -1.453152027f);
    q = fmaf(t, q, 1.421413741f);
    q = fmaf(t, q, -0.284496736f);
    q = fmaf(t, q, 0.254829592f);
    return 0.5f * q * t * gauss;
}

template <int ACT>
__device__ __forceinline__ float act_fn(float x)
{
    if constexpr (ACT == kActRelu) {
        return x < 0.0f ? 0.0f : x;
    } else if constexpr (ACT == kActGelu) {
        float g;
        const float ax = fabsf(x), h = half_erfc(ax, g);
        return (x > 0.0f ? x : 0.0f * x) - fminf(ax, 20.0f) * h;
    } else if constexpr (ACT == kActGeluTanh) {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
        const float u2 = -1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.0f);
        return __fdividef(x, 1.0f + __expf(u2));
    } else if constexpr (ACT == kActSilu) {
        return __fdividef(x, 1.0f + __expf(-x));
    } else {
        return x;
    }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float x)
{
    if constexpr (ACT == kActRelu) {
        return x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
    } else if constexpr (ACT == kActGelu) {
        float g;
        const float h = half_erfc(fabsf(x), g);
        return (x > 0.0f ? 1.0f - h : h) + x * (0.39894228040143268f * g);
    } else if constexpr (ACT == kActGeluTanh) {
        const float x2 = x * x;
        const float u2 = -1.5957691216057308f * x * fmaf(0.044715f, x2, 1.0f);
        const float s = __fdividef(1.0f, 1.0f + __expf(u2));
        return s + x * s * (1.0f - s) * 1.5957691216057308f * fmaf(3.0f * 0.044715f, x2, 1.0f);
    } else if constexpr (ACT == kActSilu) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-x));
        return s * fmaf(x, 1.0f - s, 1.0f);
    } else {
        return 1.0f;
    }
}

__device__ __forceinline__ float load16(const void *p, int64_t i, int bf16)
{
    const uint16_t u = static_cast<const uint16_t *>(p)[i];
    return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                : __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ uint16_t round16(float v, int bf16)
{
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

template <int OUT>
__device__ __forceinline__ float load_as(const void *p, int64_t i)
{
    if constexpr (OUT == kOutF32)
        return static_cast<const float *>(p)[i];
    else
        return load16(p, i, OUT == kOutBF16);
}

template <int OUT>
__device__ __forceinline__ void store_as(void *p, int64_t i, float v)
{
    if constexpr (OUT == kOutF32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = round16(v, OUT == kOutBF16);
}

// ------------------------------------------------------------------------------- units
// Range of group g, clamped into the `cols` rows that exist whatever the offsets say.
__device__ __forceinline__ void group_range(const LmArgs &p, int g, int &begin, int &end)
{
    if (!p.offsets) {
        begin = 0;
        end = p.cols;
        return;
    }
    const int64_t b = p.offsets[g], e = p.offsets[g + 1], c = p.cols;
    begin = static_cast<int>(b < 0 ? 0 : (b > c ? c : b));
    end = static_cast<int>(e < begin ? begin : (e > c ? c : e));
}

// Slots of an N-ragged grouped call: slot 0 holds the columns before the first group,
// slots 1 .. groups the groups, slot groups + 1 the columns after the last one.  The
// first and last slots' columns belong to no group and come out zero.
__device__ __forceinline__ void slot_range(const LmArgs &p, int s, int &begin, int &end)
{
    if (s >= 1 && s <= p.groups) {
        group_range(p, s - 1, begin, end);
        return;
    }
    const int64_t o = p.offsets[s == 0 ? 0 : p.groups], c = p.cols;
    const int at = static_cast<int>(o < 0 ? 0 : (o > c ? c : o));
    begin = s == 0 ? 0 : at;
    end = s == 0 ? at : p.cols;
}

struct LmUnit {
    int g;              // group (matrix of A; bias; of D for K-ragged calls); -1: no group
    int mt;             // tile row
    int col0, col_end;  // first column of the tile, end of the columns it may write
    int kb0, kb1, ks;   // K blocks and split index
    int tok0, toks;     // K ragged: first token, tokens
    int tile;           // index of the tile (split counters)
};

// A role's walk over its pair's units: unit u -> LmUnit, u increasing.
template <int BN, bool RK>
struct LmWalk {
    int slot = 0;
    int begin = 0, end = 0, at = -1;     // slot whose range is loaded

    __device__ __forceinline__ LmUnit unit(const LmArgs &p, const int *cum, int u)
    {
        LmUnit w;
        w.tok0 = w.toks = 0;
        if constexpr (RK) {
            const int per = p.num_m_tiles * p.num_n_tiles;
            const int g = u / per;
            if (g != at) {
                group_range(p, g, begin, end);
                at = g;
            }
            int nt;
            tile(p, u - g * per, p.num_n_tiles, w.mt, nt);
            w.g = g;
            w.col0 = nt * BN;
            w.col_end = p.n;
            w.tok0 = begin;
            w.toks = end - begin;
            w.kb0 = 0;
            w.kb1 = (w.toks + 63) >> 6;
            w.ks = 0;
            w.tile = u;
            return w;
        }
        int r = u, nts = p.num_n_tiles;
        w.g = 0;
        if (p.offsets) {
            while (u >= cum[slot + 1])
                ++slot;
            if (slot != at) {
                slot_range(p, slot, begin, end);
                at = slot;
            }
            r = u - cum[slot];
            nts = (end - begin + BN - 1) / BN;
            w.g = slot >= 1 && slot <= p.groups ? slot - 1 : -1;
        } else {
            end = p.cols;
        }
        const int t = r / p.k_splits;
        w.ks = r - t * p.k_splits;
        w.tile = u / p.k_splits;
        int nt;
        tile(p, t, nts, w.mt, nt);
        w.col0 = begin + nt * BN;
        w.col_end = end;
        w.kb0 = w.g < 0 ? 0 : w.ks * p.kb_per_split;
        w.kb1 = w.g < 0 ? 0 : min(w.kb0 + p.kb_per_split, p.num_k_blocks);
        return w;
    }

    // Tile t of a num_m_tiles x nts grid, group_m tile rows walked together.
    static __device__ __forceinline__ void tile(const LmArgs &p, int t, int nts, int &mt, int &nt)
    {
        const int span = p.group_m * nts;
        const int first = t / span * p.group_m;
        const int gsize = min(p.num_m_tiles - first, p.group_m);
        const int in = t % span;
        mt = first + in % gsize;
        nt = in / gsize;
    }
};

template <bool RK>
__device__ __forceinline__ int lm_total_units(const LmArgs &p, const int *cum)
{
    if constexpr (RK)
        return p.groups * p.num_m_tiles * p.num_n_tiles;
    return p.offsets ? cum[p.groups + 2] : p.num_m_tiles * p.num_n_tiles * p.k_splits;
}

// ------------------------------------------------------------------------- the epilogues
// act(alpha v + bias) + beta C for one row and kCols columns from `col`, stored to D (and
// the value before act to Z).  Columns at and past col_end are another group's.
template <int OUT, int ACT, int kCols>
__device__ __forceinline__ void finish_act(const LmArgs &p, const float (&z)[kCols], int row, int col,
                                           int ncol, int64_t dbase)
{
    float r[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        r[j] = act_fn<ACT>(z[j]);
    if (p.C) {
        const int64_t cbase = static_cast<int64_t>(col) * p.ldc + row;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol)
                r[j] = fmaf(p.beta, load_as<OUT>(p.C, cbase + j * p.ldc), r[j]);
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        if (j < ncol)
            store_as<OUT>(p.D, dbase + j * p.ldd, r[j]);
}

template <int OUT, int kCols>
__device__ __forceinline__ void finish_linear(const LmArgs &p, float (&z)[kCols], const LmUnit &w,
                                              int row, int col, float alpha, float bias)
{
    const int ncol = w.col_end - col;
    if (row >= p.m || ncol <= 0)
        return;
    const int64_t dbase = (p.ragged_k ? w.g * p.strideD : 0) + static_cast<int64_t>(col) * p.ldd + row;
    if (w.g < 0) {                             // columns of no group
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol) {
                store_as<OUT>(p.D, dbase + j * p.ldd, 0.0f);
                if (p.Z)
                    static_cast<uint16_t *>(p.Z)[(static_cast<int64_t>(col) + j) * p.ldz + row] = 0;
            }
        return;
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        z[j] = fmaf(alpha, z[j], bias);
    if (p.Z) {
        uint16_t *zp = static_cast<uint16_t *>(p.Z) + static_cast<int64_t>(col) * p.ldz + row;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j < ncol)
                zp[j * p.ldz] = round16(z[j], p.in_bf16);
    }
    switch (p.act) {
    case kActRelu: finish_act<OUT, kActRelu>(p, z, row, col, ncol, dbase); break;
    case kActGelu: finish_act<OUT, kActGelu>(p, z, row, col, ncol, dbase); break;
    case kActGeluTanh: finish_act<OUT, kActGeluTanh>(p, z, row, col, ncol, dbase); break;
    case kActSilu: finish_act<OUT, kActSilu>(p, z, row, col, ncol, dbase); break;
    default: finish_act<OUT, kActNone>(p, z, row, col, ncol, dbase); break;
    }
}

constexpr float kLog2e = 1.4426950408889634f;
// 2^x on the special-function unit, results below 2^-126 flushed to zero (they vanish
// beside the row's largest term, 1)
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------- the kernel
template <int EPI, int OUT, int BN, bool RK>
__global__ void __launch_bounds__(kThreads, 1)
    tcg_lm_kernel(const __grid_constant__ LmMaps maps, const LmArgs p)
{
    using Cfg = LmCfg<BN>;
    constexpr int kStages = Cfg::kStages;
    constexpr int kAccBufs = Cfg::kAccBufs;
    constexpr int kBRows = Cfg::kBRows;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw_u32);
    const uint32_t a_smem = base;
    const uint32_t b_smem = base + kStages * Cfg::kAStage;
    LmCtl *ctl = reinterpret_cast<LmCtl *>(base_ptr + kDataBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster_id = blockIdx.x / 2;
    const int num_clusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < kAccBufs; ++a) {
            mbar_init(smem_u32(&ctl->acc_full[a]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[a]), kEpiWarps * 2);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_mbar_init();
        if (RK ? p.cols > 0 : p.num_k_blocks > 0) {
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
    griddep_wait();
    // Units before each slot of a grouped call, by one warp.
    if (!RK && p.offsets && warp == 2) {
        int sum = 0;
        if (lane == 0)
            ctl->cum[0] = 0;
        for (int s0 = 0; s0 < p.groups + 2; s0 += 32) {
            const int s = s0 + lane;
            int units = 0;
            if (s < p.groups + 2) {
                int b, e;
                slot_range(p, s, b, e);
                units = (e - b + BN - 1) / BN * p.num_m_tiles * p.k_splits;
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, units, d);
                if (lane >= d)
                    units += up;
            }
            if (s < p.groups + 2)
                ctl->cum[s + 1] = sum + units;
            sum += __shfl_sync(0xffffffffu, units, 31);
        }
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const int total = lm_total_units<RK>(p, ctl->cum);

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
            LmWalk<BN, RK> walk;
            int stage = 0;
            uint32_t phase = 0;
            bool skip_once = p.fault_inject != 0 && leader;
            bool ok = true;
            for (int u = cluster_id; ok && u < total; u += num_clusters) {
                const LmUnit w = walk.unit(p, ctl->cum, u);
                const int m0 = w.mt * 2 * kBM + static_cast<int>(rank) * kBM;
                const int n0 = w.col0 + static_cast<int>(rank) * kBRows;
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
                        const int left = w.toks - kb * kKRow;     // K ragged: tokens from k0
                        if (RK && left < kKRow) {
                            // The group's last tokens, then zeros (token index past the end) up
                            // to the stage's 64: boxes of 16, 4 and 1 tokens, each a run of
                            // 128-byte rows of the stage.
                            auto tail = [&](uint32_t dst, const CUtensorMap *map, int rows, int row0) {
                                for (int h = 0; h < rows / 64; ++h) {
                                    uint32_t d = dst + h * kChunkBytes;
                                    auto run = [&](int tok, int step, int count, int from) {
                                        // `count` tokens from stage row `from` on
                                        int at = from;
                                        const int stop = from + count;
                                        while (at < stop) {
                                            const int b = (at % 16 == 0 && stop - at >= 16) ? 0
                                                        : (at % 4 == 0 && stop - at >= 4) ? 1 : 2;
                                            tma_load_3d_pair(d + at * kRowBytes, map + b, fb,
                                                             row0 + h * 64,
                                                             tok + step * (at - from), 0);
                                            at += 16 >> (2 * b);
                                        }
                                    };
                                    run(k0, 1, left, 0);
                                    run(p.cols, 0, kKRow - left, left);
                                }
                            };
                            tail(sa, maps.A_tail, kBM, m0);
                            tail(sb, maps.B_tail, kBRows, n0);
                        } else {
                            load(sa, &maps.A, p.a_mode, kBM, m0, RK ? 0 : w.g);
                            load(sb, &maps.B, p.b_mode, kBRows, n0, 0);
                        }
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
            LmWalk<BN, RK> walk;
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            bool ok = true;
            for (int u = cluster_id; ok && u < total; u += num_clusters, ++it) {
                const LmUnit w = walk.unit(p, ctl->cum, u);
                const int acc = it % kAccBufs;
                const uint32_t acc_phase = (it / kAccBufs) & 1;
                if (!wait_bounded<2>(smem_u32(&ctl->acc_empty[acc]), acc_phase ^ 1u, ctl, p,
                                     kErrMmaAcc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_bounded<2>(smem_u32(&ctl->full[stage]), phase, ctl, p, kErrMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad_s = a_desc0 + ((static_cast<uint32_t>(stage) * Cfg::kAStage) >> 4);
                    const uint64_t bd_s = b_desc0 + ((static_cast<uint32_t>(stage) * Cfg::kBStage) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kMmasPerStage; ++kk)
                        mma_f16_pair(d_tmem, ad_s + a_off[kk], bd_s + b_off[kk], p.idesc,
                                     (kb > w.kb0 || kk > 0) ? 1u : 0u);
                    mma_commit_pair_mc(smem_u32(&ctl->empty[stage]), 0x3);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                mma_commit_pair_mc(smem_u32(&ctl->acc_full[acc]), 0x3);
            }
            mma_commit_pair(smem_u32(&ctl->drain));
            wait_bounded<2>(smem_u32(&ctl->drain), 0, ctl, p, kErrDrain, false);
        }
    } else {
        // -------------------------------------------------------------- epilogue
        // Two halves of 4 warps; half h owns columns [h BN/2, (h + 1) BN/2) of each tile
        // for the CTA's 128 rows (warp w reads TMEM lane quarter w % 4).
        constexpr int kHalf = BN / 2;
        constexpr int kCols = kHalf < 32 ? kHalf : 32;
        constexpr int kChunks = kHalf / kCols;
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        const bool half_leader = (warp == 2 + 4 * half) && lane == 0;
        const uint32_t bar_id = 1u + static_cast<uint32_t>(half);
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const int rl = q * 32 + lane;
        const float alpha = p.alpha * (p.alpha_dev ? *p.alpha_dev : 1.0f);
        LmWalk<BN, RK> walk;
        int it = 0;
        for (int u = cluster_id; u < total; u += num_clusters, ++it) {
            const int acc = it % kAccBufs;
            const uint32_t acc_phase = (it / kAccBufs) & 1;
            const LmUnit w = walk.unit(p, ctl->cum, u);
            const int row = w.mt * 2 * kBM + static_cast<int>(rank) * kBM + rl;
            const bool row_ok = row < p.m;
            // Row data of the tile, loaded while the accumulator fills.
            float bias = 0.0f;
            float row_lse2 = 0.0f, row_g = 0.0f;
            int target = -1;                               // column of the row's target
            if constexpr (EPI == kEpiLinear) {
                if (p.bias && row_ok && w.g >= 0) {
                    const int64_t i = static_cast<int64_t>(w.g) * p.m + row;
                    bias = p.bias_f32 ? static_cast<const float *>(p.bias)[i]
                                      : load16(p.bias, i, p.in_bf16);
                }
            } else if (row_ok) {
                const int64_t t = p.targets[row];
                const bool counts = t != p.ignore && t >= 0 && t < p.vocab;
                if (counts && t >= p.col0 && t - p.col0 < p.cols)
                    target = static_cast<int>(t - p.col0);
                if constexpr (EPI == kEpiXentGrad) {
                    row_lse2 = p.lse[row] * kLog2e;
                    row_g = counts ? p.dloss[row] * (p.gscale ? *p.gscale : 1.0f) : 0.0f;
                }
            }
            const bool ok = wait_bounded<2>(smem_u32(&ctl->acc_full[acc]), acc_phase, ctl, p,
                                            kErrEpilogue);
            if (named_barrier_or(bar_id, 128, !ok || ctl->abort_flag))
                break;
            tc_fence_after();
            const bool empty_k = w.kb0 >= w.kb1;
            const int col_half = w.col0 + half * kHalf;
            const bool split = EPI == kEpiLinear && !RK && p.k_splits > 1 && w.g >= 0;
            float *slices = nullptr;
            if (split)
                slices = p.part + ((static_cast<int64_t>(w.tile) * 2 + rank) * 2 + half) *
                                      p.k_splits * (kHalf * kBM) + rl;
            float smax = -INFINITY, ssum = 0.0f;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                __syncwarp();
                const uint32_t taddr = tmem_base + lane_off +
                                       static_cast<uint32_t>(acc * BN + half * kHalf + c * kCols);
                uint32_t v[kCols];
                if constexpr (kCols == 16)
                    tmem_ld_32x32b_x16(taddr, v);
                else
                    tmem_ld_32x32b_x32(taddr, v);
                tmem_ld_wait();
                if (c == kChunks - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->acc_empty[acc]), 0));
                }
                const int col = col_half + c * kCols;
                const int ncol = w.col_end - col;
                float x[kCols];
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    x[j] = empty_k ? 0.0f : __uint_as_float(v[j]);
                if constexpr (EPI == kEpiLinear) {
                    if (split) {
                        float *sl = slices + (static_cast<int64_t>(w.ks) * kHalf + c * kCols) * kBM;
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (j < ncol)
                                __stcg(sl + j * kBM, x[j]);
                    } else {
                        finish_linear<OUT>(p, x, w, row, col, alpha, bias);
                    }
                } else if constexpr (EPI == kEpiXentStats) {
                    if (ncol <= 0)
                        continue;
                    if (ncol < kCols) {
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (j >= ncol)
                                x[j] = -INFINITY;
                    }
                    if (target >= col && target < col + kCols) {
                        float tl = 0.0f;
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (target - col == j)
                                tl = x[j];
                        p.target_logit[row] = tl;
                    }
                    float mx = smax;
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        mx = fmaxf(mx, x[j]);
                    // a maximum of -inf (nothing but -inf so far) subtracts as zero
                    const float sub = mx == -INFINITY ? 0.0f : mx * kLog2e;
                    float add = 0.0f;
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        add += exp2_fast(fmaf(x[j], kLog2e, -sub));
                    ssum = ssum * exp2_fast(fmaf(smax, kLog2e, -sub)) + add;
                    smax = mx;
                } else {
                    if (ncol <= 0 || !row_ok)
                        continue;
                    uint32_t packed[kCols / 2];
#pragma unroll
                    for (int j = 0; j < kCols; j += 2) {
                        float g[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float pr = exp2_fast(fmaf(x[j + i], kLog2e, -row_lse2));
                            g[i] = row_g == 0.0f ? 0.0f
                                                 : row_g * (target == col + j + i ? pr - 1.0f : pr);
                        }
                        packed[j / 2] = static_cast<uint32_t>(round16(g[0], p.in_bf16)) |
                                        static_cast<uint32_t>(round16(g[1], p.in_bf16)) << 16;
                    }
                    uint16_t *gp = static_cast<uint16_t *>(p.D) + static_cast<int64_t>(row) * p.ldd + col;
                    if (ncol >= kCols) {
#pragma unroll
                        for (int j = 0; j < kCols / 8; ++j)
                            *reinterpret_cast<uint4 *>(gp + 8 * j) =
                                make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2],
                                           packed[4 * j + 3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (j < ncol)
                                gp[j] = static_cast<uint16_t>(packed[j / 2] >> (16 * (j & 1)));
                    }
                }
            }
            if constexpr (EPI == kEpiXentStats) {
                if (row_ok)
                    p.stats[static_cast<int64_t>(w.col0 / BN * 2 + half) * p.m + row] =
                        make_float2(smax, ssum);
            }
            if constexpr (EPI == kEpiLinear) {
                if (split) {
                    // Whoever stores the last of a tile half's partial sums adds them, in
                    // range order, and finishes the tile: the order never depends on timing.
                    __threadfence();
                    named_barrier_sync(bar_id, 128);
                    if (half_leader) {
                        uint32_t *cnt = p.cnt + (w.tile * 2 + static_cast<int>(rank)) * 2 + half;
                        const bool last = atomicAdd(cnt, 1u) == static_cast<uint32_t>(p.k_splits - 1);
                        if (last)
                            *cnt = 0u;                     // every range has arrived
                        ctl->last_arrival[half] = last;
                        __threadfence();
                    }
                    named_barrier_sync(bar_id, 128);
                    if (ctl->last_arrival[half]) {
                        __threadfence();
#pragma unroll 1
                        for (int c = 0; c < kChunks; ++c) {
                            const int col = col_half + c * kCols;
                            const int ncol = w.col_end - col;
                            if (ncol <= 0)
                                break;
                            float x[kCols];
#pragma unroll
                            for (int j = 0; j < kCols; ++j)
                                x[j] = 0.0f;
                            for (int s = 0; s < p.k_splits; ++s) {
                                const float *sl = slices +
                                    (static_cast<int64_t>(s) * kHalf + c * kCols) * kBM;
#pragma unroll
                                for (int j = 0; j < kCols; ++j)
                                    if (j < ncol)
                                        x[j] += __ldcg(sl + j * kBM);
                            }
                            finish_linear<OUT>(p, x, w, row, col, alpha, bias);
                        }
                    }
                    named_barrier_sync(bar_id, 128);       // last_arrival is free again
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
LmKernelFn linear_fn(int bn, bool rk)
{
    if (rk)
        return tcg_lm_kernel<kEpiLinear, OUT, 256, true>;
    switch (bn) {
    case 32: return tcg_lm_kernel<kEpiLinear, OUT, 32, false>;
    case 64: return tcg_lm_kernel<kEpiLinear, OUT, 64, false>;
    case 128: return tcg_lm_kernel<kEpiLinear, OUT, 128, false>;
    default: return tcg_lm_kernel<kEpiLinear, OUT, 256, false>;
    }
}

LmKernelFn lm_fn(int epi, int out_kind, int bn, bool rk)
{
    if (epi == kEpiXentStats)
        return tcg_lm_kernel<kEpiXentStats, kOutF32, 256, false>;
    if (epi == kEpiXentGrad)
        return tcg_lm_kernel<kEpiXentGrad, kOutF16, 256, false>;
    return out_kind == kOutF32 ? linear_fn<kOutF32>(bn, rk)
         : out_kind == kOutF16 ? linear_fn<kOutF16>(bn, rk) : linear_fn<kOutBF16>(bn, rk);
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
    auto join = [](float2 a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        const float sub = m == -INFINITY ? 0.0f : m * kLog2e;
        return make_float2(m, a.y * exp2_fast(fmaf(a.x, kLog2e, -sub)) +
                                  b.y * exp2_fast(fmaf(b.x, kLog2e, -sub)));
    };
    float2 acc = make_float2(-INFINITY, 0.0f);
    if (row < rows) {
#pragma unroll 4
        for (int s = w; s < slots; s += kCombineWarps)
            acc = join(acc, __ldcg(stats + static_cast<int64_t>(s) * rows + row));
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w == 0 && row < rows) {
        for (int i = 1; i < kCombineWarps; ++i)
            acc = join(acc, part[i][lane]);
        const float l = acc.x + logf(acc.y);
        const int64_t t = targets[row];
        const bool counts = t != ignore && t >= 0 && t < vocab;
        lse[row] = l;
        loss[row] = counts ? l - target_logit[row] : 0.0f;
    }
}

__global__ void __launch_bounds__(1024)
    tcg_xent_scale_kernel(const float *__restrict__ dloss, const int64_t *__restrict__ targets,
                          int rows, int64_t vocab, int64_t ignore, float *scale)
{
    __shared__ float part[32];
    griddep_launch_dependents();
    griddep_wait();
    float m = 0.0f;
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
        const int64_t t = targets[i];
        if (t != ignore && t >= 0 && t < vocab)
            m = fmaxf(m, fabsf(dloss[i]));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i)
            m = fmaxf(m, part[i]);
        int e = 0;
        if (m > 0.0f && m < INFINITY) {
            frexpf(m, &e);                     // m = f 2^e, 1/2 <= f < 1
            e = 14 - e;
            e = e > 100 ? 100 : e;
        }
        scale[0] = ldexpf(1.0f, e);
        scale[1] = ldexpf(1.0f, -e);
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
    LmArgs p;
    p.offsets = offsets;
    p.cols = cols;
    p.groups = groups;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * 256 + lane * 8;
    const int left = m - row;                         // rows of this thread (8, or fewer at the end)
    const int c0 = blockIdx.y * chunk, c1 = min(c0 + chunk, cols);

    auto load8 = [&](const uint16_t *src, float (&v)[8]) {
        if (left >= 8) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) {
                    v[2 * i] = __uint_as_float(u[i] << 16);
                    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = i < left ? load16(src, i, BF16) : 0.0f;
        }
    };
    auto store8 = [&](uint16_t *dst, const float (&v)[8]) {
        if (left >= 8) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = static_cast<uint32_t>(round16(v[2 * i], BF16)) |
                       static_cast<uint32_t>(round16(v[2 * i + 1], BF16)) << 16;
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
        group_range(p, g, b, e);
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
#pragma unroll 4
            for (int c = b + w; c < e; c += 8) {
                float d[8];
                load8(dD + static_cast<int64_t>(c) * lddd + row, d);
                if constexpr (ACT != kActNone) {
                    float z[8];
                    load8(Z + static_cast<int64_t>(c) * ldz + row, z);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] *= act_slope<ACT>(z[i]);
                }
                if (dZ)
                    store8(dZ + static_cast<int64_t>(c) * lddz + row, d);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[i] += d[i];
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
    LmArgs p;
    p.offsets = offsets;
    p.cols = cols;
    p.groups = groups;
    const int g = blockIdx.y, lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int row = blockIdx.x * 64 + lane;
    int b, e;
    group_range(p, g, b, e);
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

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
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
    cfg.blockDim = dim3(kThreads, 1, 1);
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
    cfg.blockDim = dim3(kThreads, 1, 1);
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

cudaError_t launch_xent_combine(const float2 *stats, int slots, int rows, const float *target_logit,
                                const int64_t *targets, int64_t vocab, int64_t ignore, float *loss,
                                float *lse, cudaStream_t s)
{
    return launch_pdl(tcg_xent_combine_kernel, dim3((rows + 31) / 32), dim3(32 * kCombineWarps), s,
                      stats, slots, rows, target_logit, targets, vocab, ignore, loss, lse);
}

cudaError_t launch_xent_scale(const float *dloss, const int64_t *targets, int rows, int64_t vocab,
                              int64_t ignore, float *scale, cudaStream_t s)
{
    return launch_pdl(tcg_xent_scale_kernel, dim3(1), dim3(1024), s, dloss, targets, rows, vocab,
                      ignore, scale);
}

cudaError_t launch_round_out(const float *in, int64_t ldi, int rows, int cols, const float *scale,
                             void *out, int64_t ldo, int out_kind, int grid, cudaStream_t s)
{
    return launch_pdl(out_kind == kOutBF16 ? tcg_round_out_kernel<kOutBF16>
                                           : tcg_round_out_kernel<kOutF16>,
                      dim3(grid), dim3(256), s, in, ldi, rows, cols, scale,
                      static_cast<uint16_t *>(out), ldo);
}

template <int ACT>
static cudaError_t epi_backward(int bf16, dim3 grid, cudaStream_t s, int m, int cols, int groups,
                                const int64_t *offsets, const void *dD, int64_t lddd, const void *Z,
                                int64_t ldz, void *dZ, int64_t lddz, float *part, int chunk)
{
    return launch_pdl(bf16 ? tcg_epi_backward_kernel<ACT, true> : tcg_epi_backward_kernel<ACT, false>,
                      grid, dim3(256), s, m, cols, groups, offsets, static_cast<const uint16_t *>(dD),
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
        e = launch_pdl(tcg_bias_join_kernel, dim3((m + 63) / 64, groups), dim3(256), s,
                       const_cast<const float *>(part), m, cols, groups, offsets, chunk, dbias);
    return e;
}

}  // namespace tcg
