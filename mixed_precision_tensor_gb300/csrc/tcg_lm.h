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
constexpr int kLmCounters = 1024;      // split counters of a handle: 4 per cut tile, one tile per pair at most;
constexpr int kScaleCounter = 1023;    // and one of the cross entropy's scale
constexpr int kLmMaxStages = 12;
constexpr int kLmMaxAccs = 16;
// Shared memory: the operand ring, and (tokens on the rows) 2 KiB of staging per epilogue
// warp, through which a warp's 32 rows leave and arrive in runs of 64 bytes.
constexpr int kLmDataBytes = 224 * 1024;
constexpr int kLmStageBytes = 2 * 1024;

// What the epilogue of the product kernel does with an accumulator (see tcg_lm.cu).
enum LmEpi {
    kEpiNarrow = 0,     // act(alpha acc + bias) + beta C; features x tokens
    kEpiWide = 1,       // the same; tokens x features
    kEpiXentStats = 2,  // per-row maximum and sum of exponentials, and the target's logit
    kEpiXentNarrow = 3, // the same; vocabulary x tokens
    kEpiXentGrad = 4,   // (exp(logit - lse) - [target]) * upstream gradient, 16-bit
    kEpiGatedNarrow = 5, // act(g) u of two products of the same tokens; features x tokens
    kEpiGatedWide = 6,  // the same; tokens x features
    kEpiGroupNarrow = 7, // kEpiNarrow and kEpiGatedNarrow with a scale per feature and group of K
    kEpiGroupGated = 8
};

// A gated product's tile holds both halves of its features: in the wide kind BN / 2 columns of
// g, then those of u (each CTA of the pair loads the rows of one half); in the narrow kind 16
// rows of g, then the 16 of u, four times a CTA (a warp of the epilogue has both).
__host__ __device__ constexpr bool lm_gated(int epi) {
    return epi == kEpiGatedNarrow || epi == kEpiGatedWide || epi == kEpiGroupGated;
}
__host__ __device__ constexpr bool lm_group(int epi) { return epi == kEpiGroupNarrow || epi == kEpiGroupGated; }

enum LmAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// An accumulator (rows x cols) = A (rows, K) times B (cols, K), in 256 x BN tiles.  One side
// of it is the tokens: the columns in the narrow kinds, the rows in the wide ones, where D
// and its companions are addressed as [token * ld + feature] either way.
//   Dense or grouped: the tokens fall into `groups` ranges offsets[g] .. offsets[g + 1] - 1,
//     each with its own matrix of the other operand; offsets = nullptr: one range of all.
//   K ragged (wide only): one rows x cols matrix per group, summed over the group's tokens;
//     D is addressed as [group * strideD + row * ldd + col].
struct LmArgs {
    int rows, cols, tokens;
    int ragged_k;
    int groups;
    const int64_t *offsets;    // device, groups + 1 entries; nullptr: one group of everything
    int num_row_tiles, num_col_tiles;   // of the sides that are not ragged
    int num_k_blocks;          // 64 K elements each
    const CUtensorMap *group_maps;      // K ragged: see launch_group_maps
    int min_share, split_gain; // K splitting: fewest blocks per pair, least saving in blocks
    int align_splits;          // cut tiles in the same K ranges (LmWalk)
    int group_m;
    int a_mode, b_mode;        // OperandMode
    uint32_t idesc;
    int in_bf16;               // the 16-bit input type: BF16 or FP16 (Z, 16-bit bias)

    float alpha;
    const float *alpha_dev;    // multiplies alpha when not null
    void *D;
    int64_t ldd, strideD;      // strideD: between the matrices of a K-ragged call
    const void *bias;          // one entry per feature, per group; nullptr: none
    int bias_f32;
    const void *C;             // residual, type of D; nullptr: none
    int64_t ldc;
    float beta;
    void *Z;                   // pre-activation, input type; nullptr: not kept
    int64_t ldz;
    int act;                   // LmAct
    float *part;               // partial sums of cut tiles; nullptr: never cut
    uint32_t *cnt;             // their arrival counters, zero before and after a call

    // scales per group of K: the product is the sum over the groups of
    // group_scale (the group's product + group_rest times the group's sum of x)
    int group_mmas;            // K elements of a group / 16
    int k_groups;
    const float *group_scale;  // [group][row of W], group_ld apart
    const float *group_rest;   // the same; nullptr: none
    int64_t group_ld;
    const float *group_sum;    // [group][token], sum_ld apart (whole tiles of tokens)
    int64_t sum_ld;

    // cross entropy: the features are vocabulary entries
    const int64_t *targets;
    int64_t ignore;
    int64_t vocab;             // targets outside [0, vocab) do not count, like `ignore`
    int col0;                  // vocabulary index of feature 0 (gradient pieces)
    float2 *stats;             // [slot][token]: maximum, sum
    float *target_logit;
    const float *lse, *dloss;
    const float *gscale;       // what dloss is multiplied by; nullptr: 1

    uint32_t *err;
    unsigned long long wait_limit_ns;
    int fault_inject;
};

template <int BN, bool WIDE>
struct LmCfg {
    // Epilogue warps.  Two per SM sub-partition, with registers for 32 columns under way and
    // 32 in hand each; four with half the registers were slower (16 weight gradients of
    // 2048 x 2048 over 512 tokens each: 82 against 58 us).
    static constexpr int kEpi = 8;
    static constexpr int kParts = kEpi / 4;                  // column ranges of a tile
    static constexpr int kThreadsLm = 64 + 32 * kEpi;
    static constexpr int kRingBytes = kLmDataBytes - (WIDE ? kEpi * kLmStageBytes : 0);
    static constexpr int kBRows = BN / 2;                    // B rows per CTA of the pair
    static constexpr int kAStage = kABytes;                  // 16 KiB
    static constexpr int kBStage = kBRows * kRowBytes;
    static constexpr int kStageBytes = kAStage + kBStage;
    static constexpr int kFit = kRingBytes / kStageBytes;
    // wide 256, 128, 64: 6, 8, 10; narrow 256, 128, 64, 32: 7, 9, 11, 12
    static constexpr int kStages = kFit < kLmMaxStages ? kFit : kLmMaxStages;
    // All of TMEM.  The epilogue falls behind where a pair has pieces of two tiles: the fence
    // that reports the first waits for the loads under way too, 12 us while the second streams
    // in (23 tokens, K = 16384; four accumulators 31.1 us a call, sixteen 30.8).
    static constexpr int kAccBufs = kTmemCols / BN;
};

// Bytes of the partial sums: two 256 x BN slots per pair.
inline size_t lm_part_bytes(int pairs, int bn)
{
    return static_cast<size_t>(pairs) * 2 * 2 * kBM * bn * sizeof(float);
}

// Slots of the cross entropy's statistics: per tile part (wide) or 32 vocabulary entries (narrow).
inline int64_t lm_stat_slots(int64_t vocab, bool narrow)
{
    return (vocab + 255) / 256 * (narrow ? 8 : LmCfg<256, true>::kParts);
}

struct LmMaps {
    CUtensorMap A, B;
};

// K-ragged calls: maps of A and B for each group (2 g and 2 g + 1 of `out`) whose token extent
// ends with the group, so that TMA fills the rest of the group's last block with zeros.
cudaError_t launch_group_maps(const LmMaps &maps, const int64_t *offsets, int groups, int tokens,
                              CUtensorMap *out, cudaStream_t s);

// Launchers (tcg_lm.cu).  out_kind: type of D.  bn: 32, 64, 128 or 256 (kEpiNarrow), 64, 128 or 256
// (kEpiWide), 32, 64 or 128 (kEpiGatedNarrow), 128 or 256 (kEpiGatedWide), 64, 128 or 192
// (kEpiGroupNarrow, kEpiGroupGated), 256 (K ragged, kEpiXentStats, kEpiXentGrad), 32 (kEpiXentNarrow).
cudaError_t launch_lm(const LmMaps &maps, const LmArgs &a, int epi, int out_kind, int bn,
                      int grid, cudaStream_t s);
int lm_max_resident_ctas(int num_sms);

// The products for a few tokens (tcg_lm_few.cu): D[token][feature], weights K-contiguous.
struct LmFewArgs {
    int64_t feats, k;
    int tokens;                // dense and cross entropy: at most kLmFewTokens
    int groups;
    const int64_t *offsets;    // device; nullptr: dense
    const void *W;
    int64_t ldw, strideW;
    const void *X;
    int64_t ldx;
    int in_bf16, out_kind;
    float alpha;
    void *D;
    int64_t ldd;
    const void *bias;
    int bias_f32;
    const void *C;
    int64_t ldc;
    float beta;
    void *Z;
    int64_t ldz;
    int act;
    int gated;                 // W: feats rows of g, then those of u; Z likewise
    const int64_t *targets;    // cross entropy
    int64_t ignore;
    float2 *stats;             // [block][token], one block per SM; nullptr: linear
    float *target_logit;
    uint32_t *err;
    unsigned long long wait_limit_ns;
    int fault_inject;
};
constexpr int kLmFewTokens = 4;        // dense, cross entropy
constexpr int kLmFewRows = 64;         // grouped: rows of all experts
cudaError_t launch_few(const LmFewArgs &a, int num_sms, cudaStream_t s);

// loss and log-sum-exp of each row from the slots of kEpiXentStats.
cudaError_t launch_xent_combine(const float2 *stats, int slots, int rows, const float *target_logit,
                                const int64_t *targets, int64_t vocab, int64_t ignore, float *loss,
                                float *lse, cudaStream_t s);
// scale[0] = 2^14 / max |dloss| over the rows that count (at most 2^101; 1 where there is no
// such quotient), scale[1] = 1 / scale[0]; 32 words after them are scratch.  cnt: a counter that
// is zero before and after.
cudaError_t launch_xent_scale(const float *dloss, const int64_t *targets, int rows, int64_t vocab,
                              int64_t ignore, float *scale, uint32_t *cnt, cudaStream_t s);
// out[j][i] = scale * in[j][i], rounded to the 16-bit type.
cudaError_t launch_round_out(const float *in, int64_t ldi, int rows, int cols, const float *scale,
                             void *out, int64_t ldo, int out_kind, int grid, cudaStream_t s);
// dZ = [dD u act'(g) | dD act(g)] of rows Z = [g | u], n features each.
cudaError_t launch_gate_backward(int act, int bf16, int tokens, int64_t n, const void *dD, int64_t lddd,
                                 const void *Z, int64_t ldz, void *dZ, int64_t lddz, int num_sms,
                                 cudaStream_t s);

// Root-mean-square norm (tcg_lm_norm.cu), row-major.
constexpr int64_t kNormMaxK = 32768;   // a row stays in the registers of a block
struct NormArgs {
    int64_t rows;
    int k;
    const void *X;
    int64_t ldx;
    const void *R;             // residual; nullptr: none
    int64_t ldr;
    void *S;                   // X + R, rounded; nullptr: not kept
    int64_t lds;
    const void *W;
    int w_f32, in_bf16, out8;
    float eps;
    void *Y;                   // 16-bit, or (out8) E4M3 with `scale`
    int64_t ldy;
    float *scale;
};
cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t s);
struct NormBackwardArgs {
    int64_t rows;
    int k;
    const void *dY;
    int64_t lddy;
    const void *X;
    int64_t ldx;
    const void *dS;            // added to dX; nullptr: none
    int64_t ldds;
    const void *W;
    int w_f32, in_bf16;
    float eps;
    void *dX;                  // nullptr: not wanted
    int64_t lddx;
    float *part;               // norm_backward_blocks x k; nullptr: dW is not wanted
};
int norm_backward_blocks(int64_t rows, int64_t k, int num_sms);
cudaError_t launch_norm_backward(NormBackwardArgs a, float *dw, int num_sms, cudaStream_t s);

// Products with 4-bit weights of a few tokens (tcg_lm_w4.cu), row-major: element 2 j of a row in the low half of
// byte j; w = (q - zero) scale per group of `group` elements of a row.
struct W4Args {
    int64_t rows;              // of W: the features, or twice those of a gated product
    int64_t k;
    int tokens, group;
    const uint8_t *W;
    int64_t ldw;               // bytes
    const void *scales, *zeros;   // rows x ceil(k / group); zeros nullptr: 8
    int s_f32;                 // their type: FP32, or that of X
    const void *X;
    int64_t ldx;
    int in_bf16, out_kind;
    void *D;
    int64_t ldd;
    const void *bias;
    int bias_f32;
    const void *C;
    int64_t ldc;
    float beta;
    int act, gated;
    int tiles, units, groups;  // row tiles, stages and groups of a row, by launch_w4
};
cudaError_t launch_w4(const W4Args &a, int num_sms, cudaStream_t s);
// For the product of many tokens: the weights as the type of X without their scales, q less the whole
// number nearest to the zero (exact, in a unit of 2^-6 or 2^-9), ldo elements apart; and for each group of
// K [group][row], ld_t apart (a multiple of four), the scale over that unit and, with zeros, what is left
// of the zero.
cudaError_t launch_w4_expand(const W4Args &a, void *out, int64_t ldo, float *scale, float *rest, int64_t ld_t,
                             int num_sms, cudaStream_t s);
// Each group's sum of X, [group][token].
cudaError_t launch_w4_sums(const W4Args &a, float *out, int64_t ld, cudaStream_t s);

// dZ = dD * act'(Z) and per-group sums of its rows; see tcg_epi_backward_kernel.  part:
// (ceil(cols / chunk) + groups) * m floats.
cudaError_t launch_epi_backward(int act, int bf16, int m, int cols, int groups,
                                const int64_t *offsets, const void *dD, int64_t lddd, const void *Z,
                                int64_t ldz, void *dZ, int64_t lddz, float *dbias, float *part,
                                int chunk, cudaStream_t s);

}  // namespace tcg
