// tcg_lm.h -- definitions shared by the host runtime (tcg_lm_api.cu) and the kernels
// (tcg_lm.cu) of the language-model products: products with a bias, activation and
// residual in their epilogue, products grouped by expert, and the cross entropy of a
// linear head.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tcg_internal.h"

namespace tcg {

constexpr int kLmMaxGroups = 384;      // experts of one grouped call (a table in shared memory)
constexpr int kLmCounters = 4096;      // split counters of a handle
constexpr int kLmMaxStages = 10;
constexpr int kLmMaxSplits = 16;

// What the epilogue of the product kernel does with an accumulator.
enum LmEpi {
    kEpiLinear = 0,    // act(alpha acc + bias) + beta C, optionally the pre-activation Z
    kEpiXentStats = 1, // per-row maximum and sum of exponentials, and the target's logit
    kEpiXentGrad = 2   // (exp(logit - lse) - [target]) * upstream gradient, 16-bit
};

enum LmAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// Column-major products over CTA pairs, 256 x BN tiles.  Three kinds of units:
//   N ragged (ragged_k = 0): D = op(A_g) op(B), the columns of D (tokens) in `groups`
//     ranges offsets[g] .. offsets[g + 1] - 1 of B's and D's columns, each with its own A_g;
//     groups = 1 and offsets = nullptr: one product over all `cols` columns.
//   K ragged (ragged_k = 1): D_g = A[:, range] B[:, range]^T, one m x n matrix per group,
//     the K index (tokens) in the groups' ranges of the `cols` tokens.
struct LmArgs {
    int m;                     // rows of D
    int cols;                  // N ragged: columns of D; K ragged: tokens
    int n;                     // K ragged: columns of D
    int ragged_k;
    int groups;
    const int64_t *offsets;    // device, groups + 1 entries; nullptr: one group of everything
    int num_m_tiles, num_n_tiles;   // num_n_tiles: of a dense call, or of each K-ragged matrix
    int num_k_blocks;          // N ragged
    int k_splits, kb_per_split;     // K ranges per tile (N ragged), joined by the last arrival
    int group_m;
    int a_mode, b_mode;        // OperandMode
    uint32_t idesc;
    int in_bf16;               // the 16-bit input type: BF16 or FP16 (Z, 16-bit bias)

    float alpha;
    const float *alpha_dev;    // multiplies alpha when not null
    void *D;
    int64_t ldd, strideD;      // strideD: between the matrices of a K-ragged call
    const void *bias;          // m entries per group; nullptr: none
    int bias_f32;
    const void *C;             // residual, type of D; nullptr: none
    int64_t ldc;
    float beta;
    void *Z;                   // pre-activation, input type; nullptr: not kept
    int64_t ldz;
    int act;                   // LmAct
    float *part;               // K-split partial sums
    uint32_t *cnt;             // K-split arrival counters, zero before and after a call

    // cross entropy: rows are tokens (m), columns vocabulary entries (cols)
    const int64_t *targets;
    int64_t ignore;
    int64_t vocab;             // targets outside [0, vocab) do not count, like `ignore`
    int col0;                  // vocabulary index of column 0 (gradient pieces)
    float2 *stats;             // [2 n-tile + half][row]: maximum, sum
    float *target_logit;
    const float *lse, *dloss;
    const float *gscale;       // power of two that dloss is multiplied by; nullptr: 1

    uint32_t *err;
    unsigned long long wait_limit_ns;
    int fault_inject;
};

template <int BN>
struct LmCfg {
    static constexpr int kBRows = BN / 2;                    // B rows per CTA of the pair
    static constexpr int kAStage = kABytes;                  // 16 KiB
    static constexpr int kBStage = kBRows * kRowBytes;
    static constexpr int kStageBytes = kAStage + kBStage;
    static constexpr int kFit = kDataBytes / kStageBytes;
    static constexpr int kStages = kFit < kLmMaxStages ? kFit : kLmMaxStages;
    static constexpr int kAccBufs = kTmemCols / BN < 4 ? kTmemCols / BN : 4;
};

// Number of elements of the split workspace: a slice of 128 x BN per (tile, CTA, range).
inline size_t lm_part_bytes(int64_t tiles, int bn, int splits)
{
    return static_cast<size_t>(tiles) * 2 * kBM * bn * splits * sizeof(float);
}

// K-ragged calls load the last tokens of a group with boxes of 16, 4 and 1 tokens, and
// the rest of the stage from past the last token, which TMA fills with zeros.
struct LmMaps {
    CUtensorMap A, B;
    CUtensorMap A_tail[3], B_tail[3];      // boxes of 16, 4, 1 tokens (K ragged only)
};

// Launchers (tcg_lm.cu).  out_kind: type of D.  bn: 32, 64, 128 or 256 (kEpiXent*: 256).
cudaError_t launch_lm(const LmMaps &maps, const LmArgs &a, int epi, int out_kind, int bn,
                      int grid, cudaStream_t s);
int lm_max_resident_ctas(int num_sms);

// loss and log-sum-exp of each row from the slots of kEpiXentStats.
cudaError_t launch_xent_combine(const float2 *stats, int slots, int rows, const float *target_logit,
                                const int64_t *targets, int64_t vocab, int64_t ignore, float *loss,
                                float *lse, cudaStream_t s);
// scale[0] = 2^e with 2^13 < max |dloss| 2^e <= 2^14 over the rows that count (1 where there is
// no such e), scale[1] = 1 / scale[0].
cudaError_t launch_xent_scale(const float *dloss, const int64_t *targets, int rows, int64_t vocab,
                              int64_t ignore, float *scale, cudaStream_t s);
// out[j][i] = scale * in[j][i], rounded to the 16-bit type.
cudaError_t launch_round_out(const float *in, int64_t ldi, int rows, int cols, const float *scale,
                             void *out, int64_t ldo, int out_kind, int grid, cudaStream_t s);
// dZ = dD * act'(Z) and per-group sums of its rows; see tcg_epi_backward_kernel.  part:
// (ceil(cols / chunk) + groups) * m floats.
cudaError_t launch_epi_backward(int act, int bf16, int m, int cols, int groups,
                                const int64_t *offsets, const void *dD, int64_t lddd, const void *Z,
                                int64_t ldz, void *dZ, int64_t lddz, float *dbias, float *part,
                                int chunk, cudaStream_t s);

}  // namespace tcg
