// tcg_lm_few.cu -- the language-model products for a few tokens (sm_103a).
//
// With one to four tokens a product is a pass over the weights: 2 T operations for every two
// bytes, bound by memory alone.  The tensor kernel (tcg_lm.cu) pays there for TMEM, whole
// 256-row tiles and the join of tiles cut along K, so these calls run on the FP32 units: a
// persistent block per SM whose sixteen warps work alone.  A warp takes R weight rows
// (features) at a time and streams them through a ring of its own in shared memory: 512 K
// elements of each row a stage, brought by one bulk copy per row, the copies of the next
// rows already under way while these are multiplied (packed FP32 multiply-adds, two K
// elements each).  X stays in the SM's cache.  No barrier between warps, no partial sums in
// memory.
//
// Measured on GB300, one token against 16384 x 16384 BF16 weights: 84 us (6.4 TB/s, 94% of the
// copy bandwidth).  What it took: sixteen warps of three stages (eight of four or six: 104
// and 96 us, each waiting for its own chain of steps; twenty-four of two: 106 us), and X
// loaded a stage ahead (8 rows over 64 experts, where X does not stay cached: 38 -> 25 us).
// X through the ring instead made every SM read the same lines of L2 at once (four tokens:
// 169 us).  The tensor kernel: 12.1 us for 4096 x 4096 where this takes 9.0 (7.6 where the
// weights are still in L2).  Times in a graph.

#include "tcg_lm_math.cuh"

namespace tcg {

namespace {

constexpr int kFewWarps = 16;
constexpr int kFewK = 512;                          // K elements of a stage
constexpr int kFewRowBytes = kFewK * 2;
constexpr int kFewRingBytes = 12 * 1024;            // per warp; the rest of the SM's 228 KiB caches X
constexpr int kFewMaxStages = 12;
constexpr uint64_t kFewDrainNs = 100000000ull;      // longest wait for a copy after a wait ran out

struct FewCtl {
    uint64_t full[kFewWarps][kFewMaxStages];
    int group_of[kLmFewRows];                       // grouped: the group of each row of X, or -1
    int lead[kLmFewRows];                           // rows at which a warp's tokens may start
    int leads;
    float2 stat[kFewWarps][4];
};

template <int R>
struct FewCfg {
    static constexpr int kStageBytes = R * kFewRowBytes;
    static constexpr int kFit = kFewRingBytes / kStageBytes;
    static constexpr int kStages = kFit < kFewMaxStages ? kFit : kFewMaxStages;
    static constexpr int kSmemBytes = kFewWarps * kStages * kStageBytes;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void unpack2(const uint4 &v, F2 (&x)[4])
{
    float f[8];
    unpack16<BF16>(v, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = f2(f[2 * i], f[2 * i + 1]);
}

__device__ __forceinline__ float act_of(int act, float x)
{
    float y, unused;
    F2 v = f2(x, 0.0f);
    switch (act) {
    case kActRelu: v = act_fn<kActRelu>(v); break;
    case kActGelu: v = act_fn<kActGelu>(v); break;
    case kActGeluTanh: v = act_fn<kActGeluTanh>(v); break;
    case kActSilu: v = act_fn<kActSilu>(v); break;
    default: break;
    }
    split2(v, y, unused);
    return y;
}

__device__ __forceinline__ float load_out(const void *p, int64_t i, int kind)
{
    return kind == kOutF32 ? static_cast<const float *>(p)[i] : load16(p, i, kind == kOutBF16);
}

__device__ __forceinline__ void store_out(void *p, int64_t i, int kind, float v)
{
    if (kind == kOutF32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = round16(v, kind == kOutBF16);
}

// What a warp does with task i of its walk: rows f0 .. f0 + R - 1 of group g, tokens t0 ..
// t0 + nt - 1.
struct FewTask {
    int64_t f0;
    int g, t0, nt;
};

template <int TT, int R, bool BF16>
__global__ void __launch_bounds__(kFewWarps * 32, 1)
    tcg_few_kernel(const LmFewArgs p)
{
    using Cfg = FewCfg<R>;
    constexpr int S = Cfg::kStages;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ FewCtl ctl;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(smem_u32(&ctl.full[warp][s]), 1);
        fence_mbar_init();
    }
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();

    // Grouped: the group of every row, then the rows at which work starts: the first of its
    // group and every TT-th after it (rows of no group on their own).
    if (p.offsets) {
        for (int r = threadIdx.x; r < p.tokens; r += kFewWarps * 32)
            ctl.group_of[r] = -1;
        __syncthreads();
        for (int g = threadIdx.x; g < p.groups; g += kFewWarps * 32) {
            int b, e;
            group_range(p.offsets, p.tokens, g, b, e);
            for (int r = b; r < e; ++r)
                ctl.group_of[r] = g;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int n = 0, run = 0;
            for (int r = 0; r < p.tokens; ++r) {
                const int g = ctl.group_of[r];
                run = r > 0 && g >= 0 && g == ctl.group_of[r - 1] ? run + 1 : 0;
                if (run % TT == 0)
                    ctl.lead[n++] = r;
            }
            ctl.leads = n;
        }
        __syncthreads();
    }
    const int64_t quads = (p.feats + R - 1) / R;
    const int64_t tasks = quads * (p.offsets ? ctl.leads : 1);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kFewWarps;
    const int64_t mine = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;   // SMs before warps
    auto task = [&](int64_t i) {
        FewTask w{i * R, 0, 0, p.tokens};
        if (p.offsets) {
            const int64_t l = i / quads;
            w.f0 = (i - l * quads) * R;
            w.t0 = ctl.lead[l];
            w.g = ctl.group_of[w.t0];
            w.nt = 1;
            while (w.g >= 0 && w.nt < TT && w.t0 + w.nt < p.tokens && ctl.group_of[w.t0 + w.nt] == w.g)
                ++w.nt;
        }
        return w;
    };

    uint8_t *my_ring = ring + warp * (S * Cfg::kStageBytes);
    const uint32_t my_ring_u32 = smem_u32(my_ring);
    const int64_t K = p.k, K8 = K & ~static_cast<int64_t>(7);   // the rest of K: see below
    // The producer's place in the walk: chunk at kp of task ip, into stage sp.
    int64_t ip = mine, kp = 0;
    int sp = 0;
    uint32_t filling = 0;                           // stages being filled or not yet read
    bool skip_once = p.fault_inject != 0 && blockIdx.x == 0 && warp == 0;
    FewTask wp{};
    bool have = false;
    auto produce = [&]() {                          // one more chunk, if there is one
        if (K8 == 0)
            return;
        while (!have) {                             // next task that has something to load
            if (ip >= tasks)
                return;
            wp = task(ip);
            have = wp.g >= 0;
            if (!have)
                ip += stride;
        }
        const uint32_t bytes = static_cast<uint32_t>((K8 - kp < kFewK ? K8 - kp : kFewK) * 2);
        const uint32_t bar = smem_u32(&ctl.full[warp][sp]);
        if (skip_once) {
            skip_once = false;                      // test hook: this stage is never filled
        } else {
            if (lane == 0)
                mbar_arrive_expect_tx(bar, bytes * R);
            __syncwarp();
            if (lane < R) {                         // rows past the end repeat the last one
                const int64_t f = wp.f0 + lane < p.feats ? wp.f0 + lane : p.feats - 1;
                bulk_load(my_ring_u32 + sp * Cfg::kStageBytes + lane * kFewRowBytes,
                          static_cast<const uint16_t *>(p.W) + wp.g * p.strideW + f * p.ldw + kp, bytes, bar);
            }
            filling |= 1u << sp;
        }
        sp = sp + 1 == S ? 0 : sp + 1;
        kp += kFewK;
        if (kp >= K8) {
            kp = 0;
            ip += stride;
            have = false;
        }
    };
    for (int s = 0; s < S; ++s)
        produce();

    int sc = 0;
    uint32_t parity = 0;
    bool ok = true;
    float run_m[TT], run_s[TT];                     // cross entropy: maximum and sum so far
    int64_t target[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        run_m[t] = -INFINITY;
        run_s[t] = 0.0f;
        target[t] = -1;
        if (p.targets && t < p.tokens) {
            const int64_t v = p.targets[t];
            target[t] = v == p.ignore ? -1 : v;
        }
    }
    for (int64_t i = mine; ok && i < tasks; i += stride) {
        const FewTask w = task(i);
        F2 acc[R][TT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
                acc[r][t] = f2(0.0f);
        // X comes through the SM's cache: for one or two tokens a stage ahead of its use, for
        // four by halves of the stage, for the registers.
        constexpr int kHalves = TT <= 2 ? 2 : 1;
        uint4 xv[kHalves][TT];
        auto load_x = [&](int64_t k, int h, uint4 (&v)[TT]) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (t < w.nt && k + (h * 32 + lane) * 8 < K8)
                    v[t] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) +
                                                            (w.t0 + t) * p.ldx + k +
                                                            (h * 32 + lane) * 8);
        };
        if (w.g >= 0) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
                load_x(0, h, xv[h]);
        }
        for (int64_t k0 = 0; w.g >= 0 && k0 < K8; k0 += kFewK) {
            const uint32_t bar = smem_u32(&ctl.full[warp][sc]);
            const int pieces = static_cast<int>((K8 - k0 < kFewK ? K8 - k0 : kFewK) / 8);
            if (!mbar_try_wait(bar, parity)) {
                const uint64_t begun = globaltimer_ns();
                while (!mbar_try_wait(bar, parity))
                    if (globaltimer_ns() - begun > p.wait_limit_ns) {
                        atomicOr(p.err, kErrEpilogue);
                        ok = false;
                        break;
                    }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            const uint8_t *st = my_ring + sc * Cfg::kStageBytes + lane * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h >= kHalves)
                    load_x(k0, h, xv[0]);
                if (h * 32 + lane < pieces) {
                    F2 wf[R][4];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        unpack2<BF16>(*reinterpret_cast<const uint4 *>(st + r * kFewRowBytes + h * 512),
                                      wf[r]);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if (t < w.nt) {
                            F2 xf[4];
                            unpack2<BF16>(xv[h < kHalves ? h : 0][t], xf);
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    acc[r][t] = fma2(wf[r][j], xf[j], acc[r][t]);
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
                load_x(k0 + kFewK, h, xv[h]);
            __syncwarp();                           // the stage has been read by every lane
            filling &= ~(1u << sc);
            if (++sc == S) {
                sc = 0;
                parity ^= 1u;
            }
            produce();
        }
        if (!ok)
            break;
        float sum[R][TT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                float a, b;
                split2(acc[r][t], a, b);
                a += b;
                // the last K mod 8 elements, a lane each: no copy reads past a row's end
                if (w.g >= 0 && t < w.nt && K8 + lane < K) {
                    const int64_t f = w.f0 + r < p.feats ? w.f0 + r : p.feats - 1;
                    a = fmaf(load16(p.W, w.g * p.strideW + f * p.ldw + K8 + lane, BF16),
                             load16(p.X, (w.t0 + t) * p.ldx + K8 + lane, BF16), a);
                }
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    a += __shfl_xor_sync(0xffffffffu, a, d);
                sum[r][t] = a;
            }
        if (p.stats) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (t < p.tokens) {
                    float mx = run_m[t], v[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        v[r] = w.f0 + r < p.feats ? sum[r][t] : -INFINITY;
                        mx = fmaxf(mx, v[r]);
                        if (lane == 0 && w.f0 + r == target[t] && w.f0 + r < p.feats)
                            p.target_logit[t] = v[r];
                    }
                    const float base = exp_base(mx);
                    float e = 0.0f;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        e += exp_from(v[r], base);
                    run_s[t] = fmaf(run_s[t], exp_from(run_m[t], base), e);
                    run_m[t] = mx;
                }
            }
            continue;
        }
        float v = 0.0f;                             // lane r + R t finishes row r of token t
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (lane == r + R * t)
                    v = sum[r][t];
        const int64_t f = w.f0 + lane % R, tok = w.t0 + lane / R;
        if (lane < R * w.nt && f < p.feats) {
            float out = 0.0f, z = 0.0f;
            if (w.g >= 0) {
                const int64_t bi = static_cast<int64_t>(w.g) * p.feats + f;
                const float bias = !p.bias ? 0.0f
                                 : p.bias_f32 ? static_cast<const float *>(p.bias)[bi]
                                              : load16(p.bias, bi, BF16);
                z = fmaf(p.alpha, v, bias);
                out = act_of(p.act, z);
                if (p.C)
                    out = fmaf(p.beta, load_out(p.C, tok * p.ldc + f, p.out_kind), out);
            }
            if (p.Z)
                static_cast<uint16_t *>(p.Z)[tok * p.ldz + f] = round16(z, BF16);
            store_out(p.D, tok * p.ldd + f, p.out_kind, out);
        }
    }
    if (!ok) {                                      // the copies under way land before the block leaves
        const uint64_t begun = globaltimer_ns();
        for (int i = 0; i < S; ++i) {
            const uint32_t bar = smem_u32(&ctl.full[warp][sc]);
            while ((filling >> sc & 1u) && !mbar_try_wait(bar, parity) &&
                   globaltimer_ns() - begun <= kFewDrainNs) {
            }
            if (++sc == S) {
                sc = 0;
                parity ^= 1u;
            }
        }
    }
    if (p.stats) {
        if (lane == 0) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                ctl.stat[warp][t] = make_float2(run_m[t], run_s[t]);
        }
        __syncthreads();
        if (threadIdx.x < p.tokens) {
            float2 a = ctl.stat[0][threadIdx.x];
            for (int k = 1; k < kFewWarps; ++k)
                a = join_stats(a, ctl.stat[k][threadIdx.x]);
            p.stats[static_cast<int64_t>(blockIdx.x) * p.tokens + threadIdx.x] = a;
        }
    }
}

template <int TT, int R, bool BF16>
cudaError_t launch_one(const LmFewArgs &a, int grid, cudaStream_t s)
{
    using Cfg = FewCfg<R>;
    auto fn = tcg_few_kernel<TT, R, BF16>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(fn, dim3(grid), dim3(kFewWarps * 32), s, Cfg::kSmemBytes, a);
}

template <int TT>
cudaError_t launch_tt(const LmFewArgs &a, int rows, int grid, cudaStream_t s)
{
    if (rows == 1)
        return a.in_bf16 ? launch_one<TT, 1, true>(a, grid, s) : launch_one<TT, 1, false>(a, grid, s);
    return a.in_bf16 ? launch_one<TT, 4, true>(a, grid, s) : launch_one<TT, 4, false>(a, grid, s);
}

}  // namespace

cudaError_t launch_few(const LmFewArgs &a, int num_sms, cudaStream_t s)
{
    // Four rows a warp read X a quarter as often; one row where four would leave the SMs
    // unevenly filled.
    const int lists = a.offsets ? (a.tokens < a.groups ? a.tokens : a.groups) : 1;
    const int rows = (a.feats + 3) / 4 * lists >= 4 * static_cast<int64_t>(num_sms) ? 4 : 1;
    const int64_t tasks = (a.feats + rows - 1) / rows * (a.offsets ? a.tokens : 1);
    const int grid = a.stats || tasks >= num_sms ? num_sms : static_cast<int>(tasks);
    const int tt = a.offsets && a.tokens > 2 ? 2 : a.tokens;
    return tt <= 1 ? launch_tt<1>(a, rows, grid, s)
         : tt <= 2 ? launch_tt<2>(a, rows, grid, s) : launch_tt<4>(a, rows, grid, s);
}

}  // namespace tcg
