// tcg_lm_api.cu -- host runtime and C ABI of the language-model products (declared in
// include/tcg.h): products with a bias, activation and residual in their epilogue, gated
// products, products grouped by expert, products with 4-bit weights, the cross entropy of a
// linear head, and the norm between them.
//
// Every call checks its arguments on the host, binds the handle, checks that its pointers
// are device memory, and queues kernels of tcg_lm.cu on the handle's stream.

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "tcg_host.h"

using namespace tcg;

namespace {

constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1024;   // 32-bit tile and TMA coordinates
constexpr int64_t kMaxK = int64_t(1) << 30;                 // 32-bit block counts of cut tiles

int out_kind_of(tcgDataType_t t)
{
    return t == TCG_R_32F ? kOutF32 : (t == TCG_R_16F ? kOutF16 : kOutBF16);
}

bool is_16bit(int t) { return t == TCG_R_16F || t == TCG_R_16BF; }

bool bad_ld(int64_t ld, int64_t rows, int es)
{
    return ld < (rows > 1 ? rows : 1) || ld % (16 / es);
}

int pairs_of(tcgContext *h)
{
    if (h->max_ctas[0] == 0)
        h->max_ctas[0] = lm_max_resident_ctas(h->num_sms);
    return h->max_ctas[0] / 2;
}

// One product: D[token][feature] = epilogue(X[token] . W_g[feature]), or (ragged_k) one
// matrix per group, D_g[row][col] = sum over the group's tokens of X[token][row] W[token][col].
struct Product {
    int64_t tokens = 0, feats = 0, k = 0;
    int64_t rows = 0;                       // K ragged: X's extent; W's is feats
    bool x_kmajor = true, w_kmajor = true;
    const void *X = nullptr, *W = nullptr;
    int64_t ldx = 0, ldw = 0, strideW = 0;
    tcgDataType_t in = TCG_R_16BF, out = TCG_R_16BF;
    int64_t groups = 1;
    const int64_t *offsets = nullptr;
    bool ragged_k = false;
    float alpha = 1.0f;
    const float *alpha_dev = nullptr;
    void *D = nullptr;
    int64_t ldd = 0, strideD = 0;
    tcgEpilogue_t epi = {};
    int lm_epi = -1;                        // kEpiXent*, or chosen by shape_of
    bool gated = false;                     // W holds feats rows of g, then those of u
    bool grouped_k = false;                 // scales per group of K (kEpiGroup*)
    int64_t w_rows() const { return gated ? 2 * feats : feats; }
};

// How a product runs: epilogue kind, tile width, whether tiles may be cut along K, pairs.
struct Shape {
    int epi, bn, share, gain, grid;
    int64_t tiles;                          // at most (a grouped call's depend on its offsets)
    bool cut, align;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool is_narrow(int epi)
{
    return epi == kEpiNarrow || epi == kEpiXentNarrow || epi == kEpiGatedNarrow || lm_group(epi);
}

// The most tiles a call can have.
int64_t max_tiles(const Product &p, int epi, int bn)
{
    const bool narrow = is_narrow(epi);
    if (p.ragged_k)
        return p.groups * ceil_div(p.rows, 256) * ceil_div(p.feats, bn);
    const int side = narrow ? bn : 256;
    int64_t along = ceil_div(p.tokens, side);
    if (p.offsets)                          // one more for each range that is not empty
        along = p.tokens / side + (p.groups + 2 < p.tokens ? p.groups + 2 : p.tokens);
    return along * ceil_div(p.feats, (narrow ? 256 : bn) / (p.gated ? 2 : 1));
}

// Saving in K blocks that pays for joining partial sums of a 256 x bn tile.
int gain_of(int bn) { return bn * 24 / 256 < 8 ? 8 : bn * 24 / 256; }
// Fewest K blocks of a cut tile per pair.  Whoever joins a tile's pieces reads bn / 2 KiB of
// each into its SM, and an SM loads 16 + bn / 16 KiB for a K block, both at L2's rate: the
// sum of nkb / pieces blocks and as many pieces is least at pieces^2 = nkb (32 / bn + 1 / 8).
constexpr int kMinShare = 4;
int min_share(int64_t nkb, int bn)
{
    const int s = static_cast<int>(std::ceil(std::sqrt(static_cast<double>(nkb) / (32.0 / bn + 0.125))));
    return s > kMinShare ? s : kMinShare;
}

// KiB that the busiest SM loads for `tiles` 256 x bn tiles, a last wave that fills less than
// half of the pairs cut into one piece for each.
double load_kib(int64_t tiles, int64_t nkb, int bn, int64_t pairs)
{
    const int64_t rest = tiles % pairs;
    const double block = 16.0 + bn / 16.0;
    const int64_t most = rest ? std::min(pairs / rest, nkb / min_share(nkb, bn)) : 1;
    double kib = static_cast<double>(tiles / pairs) * static_cast<double>(nkb) * block;
    if (rest)
        kib += static_cast<double>(most > 1 ? ceil_div(nkb, most) : nkb) * block +
               (most > 1 ? static_cast<double>(most) * bn / 2 : 0.0);
    return kib;
}

Shape shape_of(tcgContext *h, const Product &p)
{
    Shape s;
    const int64_t P = pairs_of(h), nkb = ceil_div(p.k, 64);
    // The tile width with the least predicted time, in the time of a K block at the first width:
    // `cost` of it at the others.
    auto best_of = [&](std::initializer_list<int> widths, auto cost_of, int least = 0) {
        int found = *widths.begin();
        double best = 1e300;
        for (int bn : widths) {
            if (bn < least)
                break;
            const double cost = cost_of(bn);
            const int64_t tiles = max_tiles(p, s.epi, bn), rest = tiles % P;
            int64_t share = ceil_div(rest * nkb, P);
            share = share < min_share(nkb, bn) ? min_share(nkb, bn) : share;
            double t = static_cast<double>(tiles / P) * static_cast<double>(nkb);
            if (rest)
                t += nkb - share >= gain_of(bn) ? static_cast<double>(share) + gain_of(bn) / cost
                                                : static_cast<double>(nkb);
            t = t * cost + 12.0 * bn / 256;
            if (t < best) {
                best = t;
                found = bn;
            }
        }
        return found;
    };
    if (p.ragged_k) {
        s.epi = kEpiWide;
        s.bn = 256;
    } else if (p.lm_epi >= 0) {
        s.epi = p.lm_epi;
        s.bn = p.lm_epi == kEpiXentNarrow ? 32 : 256;
    } else if (p.grouped_k) {
        s.epi = p.gated ? kEpiGroupGated : kEpiGroupNarrow;
        // Whole waves take 0.40, 0.28 and 0.22 us for a block of each tile at groups of 128, cut tiles
        // of the narrower widths more than that; by these costs (4096 x 4096, us at 192, 128, 64
        // columns): 333 tokens 31 32 33, 512 40 27 40, 4096 127 128 196; 16384 x 4096: 333 tokens 80 90 111.
        s.bn = best_of({192, 128, 64}, [](int bn) { return bn == 192 ? 1.0 : (bn == 128 ? 0.8 : 0.68); });
    } else {
        const int64_t per = p.offsets ? p.tokens / p.groups : p.tokens;
        const int narrow_bn = per <= 32 ? 32 : (per <= 64 ? 64 : 128);
        // Tokens on the columns, tiles cut along K.  Of few features, 64 wide tiles of tokens on
        // the rows can be the lesser load (100 tokens, 512 x 8192: 20 us with tokens on the
        // columns, 14 us so; 4096 x 4096: 17.6 and 21.6).  Experts: few rows each, or so few
        // tiles that four pairs share one (4 experts of 1024 x 4096, 50 rows each: 16 us so, 23 us
        // by the rule below; 2 of 4096 x 4096, 120 rows, two pairs to a tile: 25 to 31 and 25 to 26).
        const bool scarce = 4 * p.groups * ceil_div(p.feats, 256) <= P;
        // A gated tile holds both halves of its features; its wide kind starts at 128 columns.
        const int64_t wn = p.w_rows();
        const int least = p.gated || !p.w_kmajor ? 128 : 64;
        if (p.x_kmajor && per <= (p.offsets && !scarce ? 16 : 128) &&
            (p.offsets || !p.w_kmajor || load_kib(ceil_div(wn, 256), nkb, narrow_bn, P) <=
                                             load_kib(ceil_div(wn, least), nkb, least, P))) {
            s.epi = p.gated ? kEpiGatedNarrow : kEpiNarrow;
            s.bn = narrow_bn;
        } else if (p.offsets && p.x_kmajor && per < 1024) {
            // Groups' last tiles at the width that they have.  Narrower tiles read a group's
            // weights once for each of them (8 experts of 4096 x 4096, 62 rows each: 64 wide
            // 64 us, 256 wide 52 us; with a skewed router 69 and 53).  Tokens on the rows instead
            // (below) cost a 256-row tile for every group's end, and pay once tiles are many
            // (us in a graph, on the columns / on the rows; out features x in):
            //   rows   8 of 4096 x 2048   dx of these   32 of 2048 x 2048   64 of 2048 x 4096, skewed
            //    128      33 / 34           29 / 31          59 / 61              197 / 208
            //    512      55 / 52           50 / 48          95 / 91              386 / 417
            //   1024      91 / 83           89 / 92         181 / 167             663 / 682
            //   1536     135 / 125         136 / 130        288 / 248
            //   4096     358 / 307         342 / 312
            s.epi = kEpiNarrow;
            s.bn = 256;
        } else {
            // Tokens on the rows.  A block costs the 16 KiB of A and bn / 16 KiB of B that an
            // SM loads for it, at 64 bytes a cycle: 512, 384 or 320 cycles.
            s.epi = p.gated ? kEpiGatedWide : kEpiWide;
            s.bn = best_of({256, 128, 64}, [](int bn) { return bn == 256 ? 1.0 : (bn == 128 ? 0.75 : 0.625); }, least);
        }
    }
    s.tiles = max_tiles(p, s.epi, s.bn);
    s.share = min_share(nkb, s.bn);
    s.gain = gain_of(s.bn);
    const bool wide = s.epi == kEpiWide || s.epi == kEpiGatedWide;
    const bool linear = is_narrow(s.epi) || wide;
    s.cut = linear && !p.ragged_k && !(s.epi == kEpiNarrow && s.bn == 256) && nkb - s.share >= s.gain &&
            (p.offsets || s.tiles % P != 0) && h->split_k != 1;
    // Tiles share operands along both sides, and the operands exceed half of L2 (129 MB): K
    // ranges alike for all cut tiles (1000 x 1024 outputs over K = 50021: 109 -> 84 us).
    const int64_t x_tiles = ceil_div(p.tokens, wide ? 256 : s.bn);
    const int64_t w_tiles = ceil_div(p.w_rows(), wide ? s.bn : 256);
    s.align = !p.offsets && x_tiles > 1 && w_tiles > 1 && (p.tokens + p.w_rows()) * p.k > (int64_t(32) << 20);
    int64_t pairs = s.tiles;
    if (s.cut && s.tiles < P)
        pairs = s.tiles * nkb / s.share > pairs ? s.tiles * nkb / s.share : pairs;
    s.grid = 2 * static_cast<int>(pairs < P ? pairs : P);
    return s;
}

bool few(const Product &p);
bool few_tokens(int64_t tokens, int64_t feats, int64_t k);

size_t product_ws(tcgContext *h, const Product &p)
{
    if (p.ragged_k)
        return static_cast<size_t>(p.groups) * 2 * sizeof(CUtensorMap);
    if (few(p))
        return 0;
    const Shape s = shape_of(h, p);
    return s.cut ? lm_part_bytes(s.grid / 2, s.bn) : 0;
}

// Queue one product.  ws: workspace of at least product_ws bytes.
tcgStatus_t queue(tcgContext *h, const Product &p, void *ws, LmArgs a = LmArgs{})
{
    LmMaps maps;
    std::memset(&maps, 0, sizeof maps);
    const Shape s = shape_of(h, p);
    if (s.tiles > INT32_MAX)
        return TCG_STATUS_NOT_SUPPORTED;
    const bool narrow = is_narrow(s.epi);
    // accumulator rows and columns
    const int64_t x_ext = p.ragged_k ? p.rows : p.tokens;
    a.rows = static_cast<int>(narrow ? p.feats : x_ext);
    a.cols = static_cast<int>(narrow ? x_ext : p.feats);
    a.tokens = static_cast<int>(p.tokens);
    a.ragged_k = p.ragged_k;
    a.groups = static_cast<int>(p.groups);
    a.offsets = p.offsets;
    const int half = p.gated ? 2 : 1;       // of a tile's features: see lm_gated
    a.num_row_tiles = static_cast<int>(ceil_div(a.rows, narrow ? 256 / half : 256));
    a.num_col_tiles = static_cast<int>(ceil_div(a.cols, narrow ? s.bn : s.bn / half));
    a.num_k_blocks = static_cast<int>(ceil_div(p.k, 64));
    a.min_share = s.share;
    a.split_gain = s.gain;
    a.align_splits = s.align;
    // never more than there are: group_m column tiles x row tiles then fit 32 bits, as all tiles do
    a.group_m = std::min(h->group_m > 0 ? h->group_m : 8, a.num_row_tiles);
    a.in_bf16 = p.in == TCG_R_16BF;
    const bool a_kmajor = narrow ? p.w_kmajor : p.x_kmajor;
    const bool b_kmajor = narrow ? p.x_kmajor : p.w_kmajor;
    a.idesc = (1u << 4) | (static_cast<uint32_t>(a.in_bf16) << 7) |
              (static_cast<uint32_t>(a.in_bf16) << 10) | ((a_kmajor ? 0u : 1u) << 15) |
              ((b_kmajor ? 0u : 1u) << 16) | (static_cast<uint32_t>(s.bn >> 3) << 17) |
              (static_cast<uint32_t>((2 * kBM) >> 4) << 24);
    a.alpha = p.alpha;
    a.alpha_dev = p.alpha_dev;
    a.D = p.D;
    a.ldd = p.ldd;
    a.strideD = p.strideD;
    a.bias = p.epi.bias;
    a.bias_f32 = p.epi.bias_type == TCG_R_32F;
    a.C = p.epi.beta != 0.0f ? p.epi.C : nullptr;
    a.ldc = p.epi.ldc;
    a.beta = p.epi.beta;
    a.Z = p.epi.Z;
    a.ldz = p.epi.ldz;
    a.act = p.epi.activation;
    a.part = s.cut ? static_cast<float *>(ws) : nullptr;
    a.cnt = h->d_cnt;
    a.err = h->d_err;
    a.wait_limit_ns = h->wait_limit_ns;
    a.fault_inject = h->fault_inject;

    // Operands (none where nothing is summed).  A K-ragged call's are both token-major.
    tcgStatus_t st;
    const int64_t kx = p.ragged_k ? p.tokens : p.k;
    if (kx > 0) {
        bool bc;
        st = operand_map(h, p.X, p.in, p.x_kmajor, x_ext, kx, p.ldx, 0, 1, narrow ? s.bn / 2 : kBM,
                         64, &bc, narrow ? &a.b_mode : &a.a_mode, narrow ? &maps.B : &maps.A);
        if (st != TCG_STATUS_SUCCESS)
            return st;
        if (p.gated && narrow) {            // {k, feature, g or u}: 16 features of each a box
            const uint64_t dims[3] = {static_cast<uint64_t>(kx), static_cast<uint64_t>(p.feats), 2};
            const uint64_t str[2] = {static_cast<uint64_t>(p.ldw) * 2, static_cast<uint64_t>(p.feats * p.ldw) * 2};
            const uint32_t box[3] = {64, 16, 2};
            a.a_mode = kK;
            st = get_map(h, p.W, p.in, 3, dims, str, box, &maps.A);
        } else {
            st = operand_map(h, p.W, p.in, p.w_kmajor, p.feats, kx, p.ldw, p.gated ? p.feats * p.ldw : p.strideW,
                             p.gated ? 2 : (p.ragged_k || !p.offsets ? 1 : p.groups), narrow ? kBM : s.bn / 2, 64,
                             &bc, narrow ? &a.a_mode : &a.b_mode, narrow ? &maps.A : &maps.B);
        }
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    if (p.ragged_k && kx > 0) {
        a.group_maps = static_cast<CUtensorMap *>(ws);
        const cudaError_t e = launch_group_maps(maps, p.offsets, a.groups, a.tokens,
                                                static_cast<CUtensorMap *>(ws), h->stream);
        h->launches += 1;
        if (e != cudaSuccess) {
            cudaGetLastError();
            return TCG_STATUS_EXECUTION_FAILED;
        }
    }
    const cudaError_t e = launch_lm(maps, a, s.epi, out_kind_of(p.out), s.bn, s.grid, h->stream);
    h->launches += 1;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

// Few enough tokens that one pass over the weights is faster than tiles: one, two of a K that
// stays in an SM's cache (k = 8192: 16.5 us, by tiles 17.5; 16384: 31.5 and 27.7), or up to four
// where the weights are few and a call's start counts (1024 x 1024: 4.3 and 6.8 us; 4096 x 4096:
// 12.6 and 12.2; 11008 x 4096: 29.9 and 22.7).
bool few_tokens(int64_t tokens, int64_t feats, int64_t k)
{
    return tokens == 1 || (tokens == 2 && k <= 8192) ||
           (tokens <= kLmFewTokens && tokens * k <= 32768 && feats * k <= (int64_t(1) << 23));
}

// Whether a product runs as a pass over the weights (tcg_lm_few.cu): K-contiguous operands
// and at most four tokens, or, grouped, rows that are few for the number of experts.
bool few(const Product &p)
{
    if (p.ragged_k || !p.x_kmajor || !p.w_kmajor || p.k == 0 || p.lm_epi >= 0 || p.alpha_dev || p.grouped_k)
        return false;
    if (!p.offsets)
        return few_tokens(p.tokens, p.w_rows(), p.k);
    // 64 experts of 2048 x 2048: 16 rows 26 us so, 31 us by tiles; 30 rows 40 and 41; 60 rows 60
    // and 60.
    return p.tokens <= kLmFewRows && (p.tokens <= 4 || 2 * p.tokens <= p.groups);
}

tcgStatus_t queue_few(tcgContext *h, const Product &p)
{
    LmFewArgs a;
    std::memset(&a, 0, sizeof a);
    a.feats = p.feats;
    a.k = p.k;
    a.tokens = static_cast<int>(p.tokens);
    a.groups = static_cast<int>(p.groups);
    a.offsets = p.offsets;
    a.W = p.W;
    a.ldw = p.ldw;
    a.strideW = p.strideW;
    a.X = p.X;
    a.ldx = p.ldx;
    a.in_bf16 = p.in == TCG_R_16BF;
    a.out_kind = out_kind_of(p.out);
    a.alpha = p.alpha;
    a.D = p.D;
    a.ldd = p.ldd;
    a.bias = p.epi.bias;
    a.bias_f32 = p.epi.bias_type == TCG_R_32F;
    a.C = p.epi.beta != 0.0f ? p.epi.C : nullptr;
    a.ldc = p.epi.ldc;
    a.beta = p.epi.beta;
    a.Z = p.epi.Z;
    a.ldz = p.epi.ldz;
    a.act = p.epi.activation;
    a.gated = p.gated;
    a.err = h->d_err;
    a.wait_limit_ns = h->wait_limit_ns;
    a.fault_inject = h->fault_inject;
    const cudaError_t e = launch_few(a, h->num_sms, h->stream);
    h->launches += 1;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t check_epilogue(const tcgEpilogue_t &e, int64_t m, int64_t n, tcgDataType_t in,
                           tcgDataType_t out)
{
    if (e.activation < TCG_ACT_NONE || e.activation > TCG_ACT_SILU)
        return TCG_STATUS_INVALID_VALUE;
    if (e.bias) {
        if (!valid_type(e.bias_type))
            return TCG_STATUS_INVALID_VALUE;
        if (e.bias_type != TCG_R_32F && e.bias_type != in)
            return TCG_STATUS_NOT_SUPPORTED;
        if (reinterpret_cast<uintptr_t>(e.bias) % elem_size(e.bias_type))
            return TCG_STATUS_INVALID_VALUE;
    }
    if (e.beta != 0.0f && ((!e.C && m > 0 && n > 0) || !aligned16(e.C) ||
                           bad_ld(e.ldc, m, elem_size(out))))
        return TCG_STATUS_INVALID_VALUE;
    if (e.Z && (!aligned16(e.Z) || bad_ld(e.ldz, m, 2)))
        return TCG_STATUS_INVALID_VALUE;
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t check_types(tcgDataType_t in, tcgDataType_t out)
{
    if (!valid_type(in) || !valid_type(out))
        return TCG_STATUS_INVALID_VALUE;
    if (!is_16bit(in) || (out != in && out != TCG_R_32F))
        return TCG_STATUS_NOT_SUPPORTED;
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t check_groups(int64_t groups, const int64_t *offsets)
{
    if (groups < 1 || !offsets || reinterpret_cast<uintptr_t>(offsets) % 8)
        return TCG_STATUS_INVALID_VALUE;
    return groups > kLmMaxGroups ? TCG_STATUS_NOT_SUPPORTED : TCG_STATUS_SUCCESS;
}

tcgStatus_t check_device(tcgContext *h, std::initializer_list<const void *> ptrs)
{
    return device_ptrs_ok(h->device, ptrs.begin(), static_cast<int>(ptrs.size()));
}

// The product behind tcg_gemm_epilogue and tcg_gemm_grouped.
tcgStatus_t run_product(tcgContext *h, Product &p, const tcgEpilogue_t *e)
{
    if (e)
        p.epi = *e;
    tcgStatus_t st = check_types(p.in, p.out);
    if (st == TCG_STATUS_SUCCESS)
        st = check_epilogue(p.epi, p.feats, p.tokens, p.in, p.out);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (p.feats < 0 || p.tokens < 0 || p.k < 0)
        return TCG_STATUS_INVALID_VALUE;
    if (bad_ld(p.ldw, p.w_kmajor ? p.k : p.feats, 2) || bad_ld(p.ldx, p.x_kmajor ? p.k : p.tokens, 2) ||
        bad_ld(p.ldd, p.feats, elem_size(p.out)))
        return TCG_STATUS_INVALID_VALUE;
    if (p.offsets && ((p.groups > 1 && p.strideW <= 0) || (p.strideW * 2) % 16))
        return TCG_STATUS_INVALID_VALUE;
    if (p.feats > kMaxExtent || p.tokens > kMaxExtent || p.k > kMaxK)
        return TCG_STATUS_NOT_SUPPORTED;
    if (p.feats == 0 || p.tokens == 0)
        return TCG_STATUS_SUCCESS;
    if (!p.D || !aligned16(p.D) ||
        (p.k > 0 && (!p.W || !p.X || !aligned16(p.W) || !aligned16(p.X))))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {p.D, p.k > 0 ? p.W : nullptr, p.k > 0 ? p.X : nullptr, p.offsets,
                              p.epi.bias, p.epi.beta != 0.0f ? p.epi.C : nullptr, p.epi.Z});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    if (few(p))
        return queue_few(h, p);
    void *ws = nullptr;
    const size_t need = product_ws(h, p);
    if (need) {
        st = acquire_ws(h, need, &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    return queue(h, p, ws);
}

// ----------------------------------------------------------------------- cross entropy
size_t pad256(size_t b) { return (b + 255) / 256 * 256; }

// Few rows go on the accumulator's columns (kEpiXentNarrow).
constexpr int64_t kXentNarrowRows = 32;

// Workspace of the forward pass: (maximum, sum) slots for every row, the target logits, and
// the partial sums of cut tiles.
int64_t xent_slots(tcgContext *h, int64_t rows, int64_t vocab, int64_t k)
{
    if (few_tokens(rows, vocab, k))        // blocks of tcg_lm_few.cu
        return h->num_sms;
    return lm_stat_slots(vocab, rows <= kXentNarrowRows);
}
size_t xent_stats_bytes(tcgContext *h, int64_t rows, int64_t vocab, int64_t k)
{
    return pad256(static_cast<size_t>(xent_slots(h, rows, vocab, k) * rows) * sizeof(float2));
}

// Vocabulary entries whose gradient is held at a time, a multiple of 256: 256 MiB of it.
constexpr int64_t kGradPieceBytes = int64_t(256) << 20;
int64_t xent_piece(int64_t rows, int64_t vocab)
{
    int64_t w = kGradPieceBytes / (2 * rows) / 256 * 256;
    w = w < 256 ? 256 : w;
    const int64_t all = (vocab + 255) / 256 * 256;
    return w < all ? w : all;
}

struct XentBackwardPlan {
    int64_t piece, pieces;
    size_t grad_bytes, acc_bytes, scale_bytes, split_bytes, total;
};

Product xent_dx(int64_t rows, int64_t k, int64_t width, int64_t piece, tcgDataType_t in, bool one)
{
    Product p;                              // dX[row][feature] = G[row] . W[:, feature]
    p.tokens = rows;
    p.feats = k;
    p.k = width;
    p.w_kmajor = false;
    p.ldx = piece;
    p.in = in;
    p.out = one ? in : TCG_R_32F;
    return p;
}

Product xent_dw(int64_t rows, int64_t k, int64_t width, int64_t piece, tcgDataType_t in)
{
    Product p;                              // dW[entry][feature] = G[:, entry] . X[:, feature]
    p.tokens = width;
    p.feats = k;
    p.k = rows;
    p.x_kmajor = p.w_kmajor = false;
    p.ldx = piece;
    p.in = p.out = in;
    return p;
}

XentBackwardPlan xent_plan(tcgContext *h, int64_t rows, int64_t vocab, int64_t k, tcgDataType_t in)
{
    XentBackwardPlan pl;
    pl.piece = xent_piece(rows, vocab);
    pl.pieces = (vocab + pl.piece - 1) / pl.piece;
    pl.grad_bytes = pad256(static_cast<size_t>(rows * pl.piece) * 2);
    pl.acc_bytes = pl.pieces > 1 ? pad256(static_cast<size_t>(rows * ((k + 3) / 4 * 4)) * 4) : 0;
    pl.scale_bytes = 256;
    pl.split_bytes = 0;
    for (int last = 0; last < 2; ++last) {
        const int64_t w = last ? vocab - (pl.pieces - 1) * pl.piece : (pl.pieces > 1 ? pl.piece : 0);
        if (w <= 0)
            continue;
        const size_t a = product_ws(h, xent_dx(rows, k, w, pl.piece, in, pl.pieces == 1));
        const size_t b = product_ws(h, xent_dw(rows, k, w, pl.piece, in));
        const size_t c = a > b ? a : b;
        pl.split_bytes = c > pl.split_bytes ? c : pl.split_bytes;
    }
    pl.split_bytes = pad256(pl.split_bytes);
    pl.total = pl.grad_bytes + pl.acc_bytes + pl.scale_bytes + pl.split_bytes;
    return pl;
}

struct Xent {
    int64_t rows, vocab, k;
    const void *X; int64_t ldx;
    const void *W; int64_t ldw;
    tcgDataType_t in;
    const int64_t *targets;
    int64_t ignore;
};

tcgStatus_t check_xent(const Xent &x)
{
    if (!valid_type(x.in))
        return TCG_STATUS_INVALID_VALUE;
    if (!is_16bit(x.in))
        return TCG_STATUS_NOT_SUPPORTED;
    if (x.rows < 0 || x.vocab < 1 || x.k < 1)
        return TCG_STATUS_INVALID_VALUE;
    if (bad_ld(x.ldx, x.k, 2) || bad_ld(x.ldw, x.k, 2))
        return TCG_STATUS_INVALID_VALUE;
    if (x.rows > kMaxExtent || x.vocab > kMaxExtent || x.k > kMaxK)
        return TCG_STATUS_NOT_SUPPORTED;
    if (x.rows == 0)
        return TCG_STATUS_SUCCESS;
    if (!x.X || !x.W || !x.targets || !aligned16(x.X) || !aligned16(x.W) ||
        reinterpret_cast<uintptr_t>(x.targets) % 8)
        return TCG_STATUS_INVALID_VALUE;
    return TCG_STATUS_SUCCESS;
}

Product xent_logits(const Xent &x, int64_t col0, int64_t width, int epi)
{
    Product p;
    p.tokens = x.rows;
    p.feats = width;
    p.k = x.k;
    p.X = x.X;
    p.ldx = x.ldx;
    p.W = static_cast<const uint16_t *>(x.W) + col0 * x.ldw;
    p.ldw = x.ldw;
    p.in = x.in;
    p.lm_epi = epi;
    return p;
}

// The forward pass's product and its workspace.
Product xent_forward_product(const Xent &x)
{
    return xent_logits(x, 0, x.vocab, x.rows <= kXentNarrowRows ? kEpiXentNarrow : kEpiXentStats);
}

size_t xent_forward_bytes(tcgContext *h, const Xent &x)
{
    return xent_stats_bytes(h, x.rows, x.vocab, x.k) + pad256(static_cast<size_t>(x.rows) * 4) +
           (few_tokens(x.rows, x.vocab, x.k) ? 0 : product_ws(h, xent_forward_product(x)));
}

// Columns per block of the epilogue's gradient: about 16 blocks of 256 rows per SM (a few at a
// time), 32 to 256 columns each, 32 of them under way at a time.
int64_t gradient_chunk(tcgContext *h, int64_t m, int64_t n)
{
    int64_t chunk = n * ceil_div(m, 256) / (16 * static_cast<int64_t>(h->num_sms)) / 32 * 32;
    chunk = chunk < 32 ? 32 : (chunk > 256 ? 256 : chunk);
    while (ceil_div(n, chunk) > 65535)                   // the grid's second dimension
        chunk *= 2;
    return chunk;
}

size_t gradient_part_bytes(tcgContext *h, int64_t m, int64_t n, int64_t groups)
{
    return static_cast<size_t>(ceil_div(n, gradient_chunk(h, m, n)) + groups) * static_cast<size_t>(m) * 4;
}

// Arguments of an epilogue's gradient, shared with the whole backward pass.
struct Gradient {
    int act;
    int64_t m, n, groups;
    const int64_t *offsets;
    const void *dD; int64_t lddd;
    const void *Z; int64_t ldz;
    tcgDataType_t type;
    void *dZ; int64_t lddz;
    float *dbias;
};

tcgStatus_t check_gradient(const Gradient &g)
{
    if (g.act < TCG_ACT_NONE || g.act > TCG_ACT_SILU || !valid_type(g.type))
        return TCG_STATUS_INVALID_VALUE;
    if (!is_16bit(g.type))
        return TCG_STATUS_NOT_SUPPORTED;
    if (g.offsets) {
        const tcgStatus_t st = check_groups(g.groups, g.offsets);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    } else if (g.groups != 1) {
        return TCG_STATUS_INVALID_VALUE;
    }
    const bool need_z = g.act != TCG_ACT_NONE;
    if (g.m < 0 || g.n < 0 || bad_ld(g.lddd, g.m, 2) || (need_z && bad_ld(g.ldz, g.m, 2)) ||
        (g.dZ && bad_ld(g.lddz, g.m, 2)))
        return TCG_STATUS_INVALID_VALUE;
    if (g.m > kMaxK || g.n > kMaxK)
        return TCG_STATUS_NOT_SUPPORTED;
    if (g.m > 0 && g.n > 0 &&
        (!g.dD || !aligned16(g.dD) || (need_z && (!g.Z || !aligned16(g.Z))) || !aligned16(g.dZ)))
        return TCG_STATUS_INVALID_VALUE;
    return reinterpret_cast<uintptr_t>(g.dbias) % 4 ? TCG_STATUS_INVALID_VALUE : TCG_STATUS_SUCCESS;
}

tcgStatus_t queue_gradient(tcgContext *h, const Gradient &g, void *part)
{
    const cudaError_t e = launch_epi_backward(
        g.act, g.type == TCG_R_16BF, static_cast<int>(g.m), static_cast<int>(g.n),
        static_cast<int>(g.groups), g.offsets, g.dD, g.lddd, g.act != TCG_ACT_NONE ? g.Z : nullptr, g.ldz,
        g.n > 0 ? g.dZ : nullptr, g.lddz, g.dbias, static_cast<float *>(part),
        static_cast<int>(gradient_chunk(h, g.m, g.n)), h->stream);
    h->launches += g.dbias ? 2 : 1;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

// The two products of a layer's backward pass, without their pointers.
Product layer_dx(int64_t m, int64_t n, int64_t k, int64_t groups, const int64_t *offsets, tcgDataType_t type)
{
    Product p;                              // dX[token][j] = sum over i of dZ[token][i] W[i][j]
    p.tokens = n;
    p.feats = k;
    p.k = m;
    p.w_kmajor = false;
    p.in = p.out = type;
    p.groups = groups;
    p.offsets = offsets;
    return p;
}

Product layer_dw(int64_t m, int64_t n, int64_t k, int64_t groups, const int64_t *offsets, tcgDataType_t type)
{
    Product p;                              // dW[i][j] = sum over tokens of dZ[token][i] X[token][j]
    p.feats = k;
    p.x_kmajor = p.w_kmajor = false;
    p.in = p.out = type;
    if (offsets) {
        p.ragged_k = true;
        p.rows = m;
        p.tokens = n;
        p.groups = groups;
        p.offsets = offsets;
    } else {
        p.tokens = m;
        p.k = n;
    }
    return p;
}

// The workspace of a layer's backward pass: dZ (where it is not dD), the partial sums of dbias,
// and what the products need.
struct LayerPlan {
    int64_t lddz;
    size_t dz_bytes, part_bytes, total;
};

LayerPlan layer_plan(tcgContext *h, bool act, int64_t m, int64_t n, int64_t k, int64_t groups,
                     const int64_t *offsets, bool dx, bool dw, bool dbias)
{
    LayerPlan pl;
    pl.lddz = (m + 7) / 8 * 8;
    pl.dz_bytes = act && (dx || dw) ? pad256(static_cast<size_t>(n) * pl.lddz * 2) : 0;
    pl.part_bytes = dbias && m > 0 ? pad256(gradient_part_bytes(h, m, n, groups)) : 0;
    const size_t x = dx && n > 0 && k > 0
                         ? product_ws(h, layer_dx(m, n, k, groups, offsets, TCG_R_16BF)) : 0;
    const size_t w = dw && m > 0 && k > 0
                         ? product_ws(h, layer_dw(m, n, k, groups, offsets, TCG_R_16BF)) : 0;
    pl.total = pl.dz_bytes + pl.part_bytes + (x > w ? x : w);
    return pl;
}

// The product behind tcg_gemm_gated, without its pointers.
Product gated_product(int64_t m, int64_t n, int64_t k, tcgDataType_t in, tcgDataType_t out)
{
    Product p;
    p.feats = m;
    p.tokens = n;
    p.k = k;
    p.gated = true;
    p.in = in;
    p.out = out;
    return p;
}

tcgStatus_t check_gate(int act, int64_t m, int64_t n, int64_t k)
{
    if (act < TCG_ACT_NONE || act > TCG_ACT_SILU || m < 0 || n < 0 || k < 0)
        return TCG_STATUS_INVALID_VALUE;
    return m > kMaxExtent / 2 || n > kMaxExtent || k > kMaxK ? TCG_STATUS_NOT_SUPPORTED : TCG_STATUS_SUCCESS;
}

// The workspace of a gated backward pass: dZ, and what the products need.
struct GatedPlan {
    int64_t lddz;
    size_t dz_bytes, total;
};

GatedPlan gated_plan(tcgContext *h, int64_t m, int64_t n, int64_t k, bool dx, bool dw)
{
    GatedPlan pl;
    pl.lddz = (2 * m + 7) / 8 * 8;
    pl.dz_bytes = m > 0 ? pad256(static_cast<size_t>(n) * pl.lddz * 2) : 0;
    const size_t x = dx && n > 0 && k > 0 ? product_ws(h, layer_dx(2 * m, n, k, 1, nullptr, TCG_R_16BF)) : 0;
    const size_t w = dw && m > 0 && k > 0 ? product_ws(h, layer_dw(2 * m, n, k, 1, nullptr, TCG_R_16BF)) : 0;
    pl.total = pl.dz_bytes + (x > w ? x : w);
    return pl;
}

// ---------------------------------------------------------------------------- norm
tcgStatus_t check_norm(int64_t rows, int64_t k, const void *W, tcgDataType_t w_type, float eps, tcgDataType_t type)
{
    if (!valid_type(type) || !valid_type(w_type) || rows < 0 || k < 1 || !(eps >= 0.0f))
        return TCG_STATUS_INVALID_VALUE;
    if (!is_16bit(type) || (w_type != type && w_type != TCG_R_32F) || k > kNormMaxK)
        return TCG_STATUS_NOT_SUPPORTED;
    if (rows > 0 && (!W || !aligned16(W)))
        return TCG_STATUS_INVALID_VALUE;
    return TCG_STATUS_SUCCESS;
}

bool bad_rows(const void *p, int64_t ld, int64_t cols, int es) { return !aligned16(p) || bad_ld(ld, cols, es); }

// An output in the place of an input, but with rows elsewhere: it would meet rows not read yet.
bool bad_place(const void *out, int64_t ldo, const void *in, int64_t ldi, int64_t rows)
{
    return out && out == in && ldo != ldi && rows > 1;
}

// --------------------------------------------------------------------- 4-bit weights
// Whether the packed weights are read as they are, once for every 16 tokens, or expanded to 16 bits
// for the product of many tokens (us in a graph, groups of 128, as they are / expanded):
//                 tokens   32            48            64            128
//    1024 x  1024          3.5 / 9.6     3.4 / 9.5     3.5 / 10.3    5.6 / 10.5
//    4096 x  4096         10.8 / 18.1   15.1 / 18.2   19.3 / 18.9   32.2 / 23.3
//   16384 x  4096         32.2 / 61.9   49.4 / 62.5   62.3 / 63.5    118 / 59.4
//    4096 x 16384         30.0 / 61.2   43.6 / 61.6   57.2 / 62.2   98.2 / 67.3
// Gated products (2 x 512 x 1024, 2 x 2048 x 4096, 2 x 8192 x 4096 and 2 x 2048 x 16384):
//    64 tokens   3.3 / 10.5   19.3 / 19.3   62.1 / 65.2   57.1 / 65.0
//   128          5.4 / 11.1   32.1 / 24.4    118 / 61.4   98.2 / 69.6
//   256          9.4 / 11.2   66.4 / 26.6    246 / 79.8    207 / 82.7
// Their limit of 128 tokens, which callers rely on for needing no workspace, is from a time when
// expanded weights cost twice as much.
bool w4_packed(int64_t tokens, int64_t rows, int64_t k, bool gated)
{
    if (gated)
        return tokens <= 128 || (tokens <= 256 && rows * k <= (int64_t(1) << 21));
    return tokens <= 48 || (tokens <= 64 && rows * k <= (int64_t(1) << 24)) ||
           (tokens <= 128 && rows * k <= (int64_t(1) << 21));
}

// The product of the expanded weights, without its pointers, and its workspace: the weights, their
// scales and what is left of their zeros, the sums of X, what the product needs.  Room for the smallest groups.
struct W4Plan {
    Product p;
    int64_t ld_t, ld_sum;                   // between the groups' scales; sums
    size_t w_bytes, t_bytes, sum_bytes, total;
};

W4Plan w4_plan(tcgContext *h, int64_t m, int64_t n, int64_t k, bool gated)
{
    W4Plan pl;
    const int64_t rows = gated ? 2 * m : m, groups = ceil_div(k, 32);
    pl.p.feats = m;
    pl.p.tokens = n;
    pl.p.k = k;
    pl.p.gated = gated;
    pl.p.grouped_k = true;
    pl.p.ldw = (k + 7) / 8 * 8;
    pl.ld_t = (rows + 3) / 4 * 4;
    pl.ld_sum = ceil_div(n, 64) * 64 + 192;          // whole tiles of any width
    pl.w_bytes = pad256(static_cast<size_t>(rows) * pl.p.ldw * 2);
    pl.t_bytes = pad256(static_cast<size_t>(groups) * pl.ld_t * sizeof(float));
    pl.sum_bytes = static_cast<size_t>(groups) * pl.ld_sum * sizeof(float);
    pl.total = pl.w_bytes + 2 * pl.t_bytes + pl.sum_bytes + product_ws(h, pl.p);
    return pl;
}

}  // namespace

extern "C" {

tcgStatus_t tcg_gemm_epilogue(tcgHandle_t h, tcgOp_t transa, tcgOp_t transb, int64_t m, int64_t n,
                              int64_t k, float alpha, const void *A, int64_t lda, const void *B,
                              int64_t ldb, tcgDataType_t ABtype, void *D, tcgDataType_t Dtype,
                              int64_t ldd, const tcgEpilogue_t *epilogue)
{
    if (!h || (transa != TCG_OP_N && transa != TCG_OP_T) || (transb != TCG_OP_N && transb != TCG_OP_T))
        return TCG_STATUS_INVALID_VALUE;
    Product p;
    p.feats = m;
    p.tokens = n;
    p.k = k;
    p.w_kmajor = transa == TCG_OP_T;
    p.x_kmajor = transb == TCG_OP_N;
    p.W = A;
    p.ldw = lda;
    p.X = B;
    p.ldx = ldb;
    p.in = ABtype;
    p.out = Dtype;
    p.alpha = alpha;
    p.D = D;
    p.ldd = ldd;
    return run_product(h, p, epilogue);
}

tcgStatus_t tcg_gemm_grouped(tcgHandle_t h, tcgOp_t transa, int64_t m, int64_t n, int64_t k,
                             int64_t groups, const int64_t *offsets, float alpha, const void *A,
                             int64_t lda, int64_t strideA, const void *B, int64_t ldb,
                             tcgDataType_t ABtype, void *D, tcgDataType_t Dtype, int64_t ldd,
                             const tcgEpilogue_t *epilogue)
{
    if (!h || (transa != TCG_OP_N && transa != TCG_OP_T))
        return TCG_STATUS_INVALID_VALUE;
    const tcgStatus_t st = check_groups(groups, offsets);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    Product p;
    p.feats = m;
    p.tokens = n;
    p.k = k;
    p.w_kmajor = transa == TCG_OP_T;
    p.W = A;
    p.ldw = lda;
    p.strideW = strideA;
    p.X = B;
    p.ldx = ldb;
    p.in = ABtype;
    p.out = Dtype;
    p.groups = groups;
    p.offsets = offsets;
    p.alpha = alpha;
    p.D = D;
    p.ldd = ldd;
    return run_product(h, p, epilogue);
}

tcgStatus_t tcg_gemm_epilogue_workspace_size(tcgHandle_t h, tcgOp_t transa, tcgOp_t transb,
                                             int64_t m, int64_t n, int64_t k, int64_t groups,
                                             size_t *bytes)
{
    if (!h || !bytes || (transa != TCG_OP_N && transa != TCG_OP_T) ||
        (transb != TCG_OP_N && transb != TCG_OP_T) || m < 0 || n < 0 || k < 0 || groups < 0 ||
        groups > kLmMaxGroups)
        return TCG_STATUS_INVALID_VALUE;
    *bytes = 0;
    if (m == 0 || n == 0)
        return TCG_STATUS_SUCCESS;
    const tcgStatus_t st = bind_device(h);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    static const int64_t some = 0;
    Product p;
    p.feats = m;
    p.tokens = n;
    p.k = k;
    p.w_kmajor = transa == TCG_OP_T;
    p.x_kmajor = transb == TCG_OP_N;
    if (groups > 0) {
        p.groups = groups;
        p.offsets = &some;                  // grouped: only whether it is set matters here
    }
    *bytes = product_ws(h, p);
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_gemm_grouped_k(tcgHandle_t h, int64_t m, int64_t n, int64_t k, int64_t groups,
                               const int64_t *offsets, float alpha, const void *A, int64_t lda,
                               const void *B, int64_t ldb, tcgDataType_t ABtype, void *D,
                               tcgDataType_t Dtype, int64_t ldd, int64_t strideD)
{
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_groups(groups, offsets);
    if (st == TCG_STATUS_SUCCESS)
        st = check_types(ABtype, Dtype);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (m < 0 || n < 0 || k < 0)
        return TCG_STATUS_INVALID_VALUE;
    if (bad_ld(lda, m, 2) || bad_ld(ldb, n, 2) || bad_ld(ldd, m, elem_size(Dtype)) || strideD < 0 ||
        (strideD * elem_size(Dtype)) % 16 || (groups > 1 && strideD < (n > 0 ? (n - 1) * ldd + m : 0)))
        return TCG_STATUS_INVALID_VALUE;
    if (m > kMaxExtent || n > kMaxExtent || k > kMaxExtent)
        return TCG_STATUS_NOT_SUPPORTED;
    if (m == 0 || n == 0)
        return TCG_STATUS_SUCCESS;
    if (!D || !aligned16(D) || (k > 0 && (!A || !B || !aligned16(A) || !aligned16(B))))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {D, k > 0 ? A : nullptr, k > 0 ? B : nullptr, offsets});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    Product p;
    p.feats = m;
    p.rows = n;
    p.tokens = k;
    p.ragged_k = true;
    p.x_kmajor = p.w_kmajor = false;
    p.X = B;
    p.W = A;
    p.ldx = ldb;
    p.ldw = lda;
    p.in = ABtype;
    p.out = Dtype;
    p.groups = groups;
    p.offsets = offsets;
    p.alpha = alpha;
    p.D = D;
    p.ldd = ldd;
    p.strideD = strideD;
    void *ws = nullptr;
    st = acquire_ws(h, product_ws(h, p), &ws);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    return queue(h, p, ws);
}

tcgStatus_t tcg_epilogue_backward(tcgHandle_t h, tcgActivation_t activation, int64_t m, int64_t n,
                                  int64_t groups, const int64_t *offsets, const void *dD,
                                  int64_t lddd, const void *Z, int64_t ldz, tcgDataType_t type,
                                  void *dZ, int64_t lddz, float *dbias)
{
    const Gradient g{activation, m, n, groups, offsets, dD, lddd, Z, ldz, type, dZ, lddz, dbias};
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_gradient(g);
    if (st != TCG_STATUS_SUCCESS || m == 0 || (!dZ && !dbias))
        return st;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {n > 0 ? dD : nullptr, n > 0 && activation != TCG_ACT_NONE ? Z : nullptr,
                              n > 0 ? dZ : nullptr, dbias, offsets});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    void *ws = nullptr;
    if (dbias) {
        st = acquire_ws(h, gradient_part_bytes(h, m, n, groups), &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    return queue_gradient(h, g, ws);
}

tcgStatus_t tcg_linear_backward(tcgHandle_t h, tcgActivation_t activation, int64_t m, int64_t n,
                                int64_t k, int64_t groups, const int64_t *offsets, const void *dD,
                                int64_t lddd, const void *Z, int64_t ldz, const void *W, int64_t ldw,
                                int64_t strideW, const void *X, int64_t ldx, tcgDataType_t type, void *dX,
                                int64_t lddx, void *dW, int64_t lddw, int64_t stridedW, float *dbias)
{
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    Gradient g{activation, m, n, groups, offsets, dD, lddd, Z, ldz, type, nullptr, 0, dbias};
    tcgStatus_t st = check_gradient(g);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (k < 0 || k > kMaxK)
        return k < 0 ? TCG_STATUS_INVALID_VALUE : TCG_STATUS_NOT_SUPPORTED;
    if ((dX && (bad_ld(ldw, k, 2) || bad_ld(lddx, k, 2) || !aligned16(W) || !aligned16(dX))) ||
        (dW && (bad_ld(ldx, k, 2) || bad_ld(lddw, k, 2) || !aligned16(X) || !aligned16(dW))))
        return TCG_STATUS_INVALID_VALUE;
    if (offsets && ((dX && ((groups > 1 && strideW <= 0) || (strideW * 2) % 16)) ||
                    (dW && ((groups > 1 && stridedW < (m > 0 ? (m - 1) * lddw + k : 0)) ||
                            (stridedW * 2) % 16))))
        return TCG_STATUS_INVALID_VALUE;
    const bool sums = m > 0 && n > 0 && k > 0;
    if (sums && ((dX && !W) || (dW && !X)))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {n > 0 && m > 0 ? dD : nullptr,
                              n > 0 && m > 0 && activation != TCG_ACT_NONE ? Z : nullptr,
                              sums && dX ? W : nullptr, sums && dW ? X : nullptr,
                              n > 0 && k > 0 ? dX : nullptr, m > 0 && k > 0 ? dW : nullptr,
                              m > 0 ? dbias : nullptr, offsets});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    const LayerPlan pl = layer_plan(h, activation != TCG_ACT_NONE, m, n, k, groups, offsets, dX, dW, dbias);
    void *ws = nullptr;
    if (pl.total) {
        st = acquire_ws(h, pl.total, &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    uint8_t *at = static_cast<uint8_t *>(ws);
    const void *dz = dD;
    int64_t lddz = lddd;
    if (pl.dz_bytes) {
        dz = g.dZ = at;
        lddz = g.lddz = pl.lddz;
    }
    if (pl.dz_bytes || pl.part_bytes) {
        st = queue_gradient(h, g, at + pl.dz_bytes);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    void *tail = at + pl.dz_bytes + pl.part_bytes;
    if (dX && n > 0 && k > 0) {
        Product p = layer_dx(m, n, k, groups, offsets, type);
        p.X = dz;
        p.ldx = lddz;
        p.W = W;
        p.ldw = ldw;
        p.strideW = strideW;
        p.D = dX;
        p.ldd = lddx;
        st = queue(h, p, tail);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    if (dW && m > 0 && k > 0) {
        Product p = layer_dw(m, n, k, groups, offsets, type);
        p.X = dz;
        p.ldx = lddz;
        p.W = X;
        p.ldw = ldx;
        p.D = dW;
        p.ldd = lddw;
        p.strideD = stridedW;
        st = queue(h, p, tail);
    }
    return st;
}

tcgStatus_t tcg_linear_backward_workspace_size(tcgHandle_t h, tcgActivation_t activation, int64_t m,
                                               int64_t n, int64_t k, int64_t groups, int with_dX,
                                               int with_dW, int with_dbias, size_t *bytes)
{
    if (!h || !bytes || activation < TCG_ACT_NONE || activation > TCG_ACT_SILU || m < 0 || n < 0 || k < 0 ||
        groups < 0 || groups > kLmMaxGroups)
        return TCG_STATUS_INVALID_VALUE;
    const tcgStatus_t st = bind_device(h);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    static const int64_t some = 0;          // grouped: only whether offsets are set matters here
    *bytes = layer_plan(h, activation != TCG_ACT_NONE, m, n, k, groups > 0 ? groups : 1,
                        groups > 0 ? &some : nullptr, with_dX, with_dW, with_dbias).total;
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_xent_workspace_size(tcgHandle_t h, int64_t rows, int64_t vocab, int64_t k,
                                    tcgDataType_t type, int backward, size_t *bytes)
{
    if (!h || !bytes || rows < 0 || vocab < 1 || k < 1 || !is_16bit(type))
        return TCG_STATUS_INVALID_VALUE;
    *bytes = 0;
    if (rows == 0)
        return TCG_STATUS_SUCCESS;
    const tcgStatus_t st = bind_device(h);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    const Xent x{rows, vocab, k, nullptr, k, nullptr, k, type, nullptr, -1};
    *bytes = backward ? xent_plan(h, rows, vocab, k, type).total : xent_forward_bytes(h, x);
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_xent_forward(tcgHandle_t h, int64_t rows, int64_t vocab, int64_t k, const void *X,
                             int64_t ldx, const void *W, int64_t ldw, tcgDataType_t type,
                             const int64_t *targets, int64_t ignore_index, float *loss, float *lse)
{
    const Xent x{rows, vocab, k, X, ldx, W, ldw, type, targets, ignore_index};
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_xent(x);
    if (st != TCG_STATUS_SUCCESS || rows == 0)
        return st;
    if (!loss || !lse || reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {X, W, targets, loss, lse});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    void *ws = nullptr;
    const size_t stats_bytes = xent_stats_bytes(h, rows, vocab, k);
    st = acquire_ws(h, xent_forward_bytes(h, x), &ws);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    LmArgs a{};
    a.targets = targets;
    a.ignore = ignore_index;
    a.vocab = vocab;
    a.stats = static_cast<float2 *>(ws);
    a.target_logit = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + stats_bytes);
    if (few_tokens(rows, vocab, k)) {
        LmFewArgs f;
        std::memset(&f, 0, sizeof f);
        f.feats = vocab;
        f.k = k;
        f.tokens = static_cast<int>(rows);
        f.W = W;
        f.ldw = ldw;
        f.X = X;
        f.ldx = ldx;
        f.in_bf16 = type == TCG_R_16BF;
        f.targets = targets;
        f.ignore = ignore_index;
        f.stats = a.stats;
        f.target_logit = a.target_logit;
        f.err = h->d_err;
        f.wait_limit_ns = h->wait_limit_ns;
        f.fault_inject = h->fault_inject;
        if (launch_few(f, h->num_sms, h->stream) != cudaSuccess) {
            cudaGetLastError();
            return TCG_STATUS_EXECUTION_FAILED;
        }
        h->launches += 1;
    } else {
        st = queue(h, xent_forward_product(x),
                   static_cast<uint8_t *>(ws) + stats_bytes + pad256(static_cast<size_t>(rows) * 4), a);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    const cudaError_t e = launch_xent_combine(a.stats, static_cast<int>(xent_slots(h, rows, vocab, k)),
                                              static_cast<int>(rows), a.target_logit, targets, vocab,
                                              ignore_index, loss, lse, h->stream);
    h->launches += 1;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_xent_backward(tcgHandle_t h, int64_t rows, int64_t vocab, int64_t k, const void *X,
                              int64_t ldx, const void *W, int64_t ldw, tcgDataType_t type,
                              const int64_t *targets, int64_t ignore_index, const float *lse,
                              const float *dloss, void *dX, int64_t lddx, void *dW, int64_t lddw)
{
    const Xent x{rows, vocab, k, X, ldx, W, ldw, type, targets, ignore_index};
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_xent(x);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if ((dX && (!aligned16(dX) || bad_ld(lddx, k, 2))) || (dW && (!aligned16(dW) || bad_ld(lddw, k, 2))))
        return TCG_STATUS_INVALID_VALUE;
    if (rows > 0 && (!lse || !dloss || reinterpret_cast<uintptr_t>(lse) % 4 ||
                     reinterpret_cast<uintptr_t>(dloss) % 4))
        return TCG_STATUS_INVALID_VALUE;
    if ((rows == 0 && !dW) || (!dX && !dW))
        return TCG_STATUS_SUCCESS;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = rows > 0 ? check_device(h, {X, W, targets, lse, dloss, dX, dW}) : check_device(h, {dW});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    if (rows == 0) {                                       // no rows: dW is zero
        Product p = xent_dw(0, k, vocab, vocab, type);
        p.ldw = ldx;
        p.D = dW;
        p.ldd = lddw;
        return queue(h, p, nullptr);
    }
    const XentBackwardPlan pl = xent_plan(h, rows, vocab, k, type);
    void *ws = nullptr;
    st = acquire_ws(h, pl.total, &ws);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    uint8_t *at = static_cast<uint8_t *>(ws);
    void *G = at;
    float *acc = reinterpret_cast<float *>(at + pl.grad_bytes);
    float *scale = reinterpret_cast<float *>(at + pl.grad_bytes + pl.acc_bytes);
    void *split_ws = at + pl.grad_bytes + pl.acc_bytes + pl.scale_bytes;
    const int64_t ldacc = (k + 3) / 4 * 4;
    // The gradient of the logits is held in 16 bits times 2^14 / max |dloss|.  FP16 needs the
    // range.  Both types need the factor: with one dloss for all rows, a mean, every row's target
    // entry is near -dloss and would be rounded by the same part of itself, up to 2^-8 (2^-11 in
    // FP16), against all other entries; scaled, it is near a power of two and keeps its bits.
    cudaError_t e = launch_xent_scale(dloss, targets, static_cast<int>(rows), vocab, ignore_index, scale,
                                      h->d_cnt + kScaleCounter, h->stream);
    h->launches += 1;
    for (int64_t i = 0; e == cudaSuccess && i < pl.pieces; ++i) {
        const int64_t c0 = i * pl.piece, width = vocab - c0 < pl.piece ? vocab - c0 : pl.piece;
        LmArgs a{};
        a.targets = targets;
        a.ignore = ignore_index;
        a.vocab = vocab;
        a.col0 = static_cast<int>(c0);
        a.lse = lse;
        a.dloss = dloss;
        a.gscale = scale;
        Product g = xent_logits(x, c0, width, kEpiXentGrad);
        g.D = G;
        g.ldd = pl.piece;
        st = queue(h, g, nullptr, a);
        if (st != TCG_STATUS_SUCCESS)
            return st;
        if (dX) {
            Product p = xent_dx(rows, k, width, pl.piece, type, pl.pieces == 1);
            p.W = static_cast<const uint16_t *>(W) + c0 * ldw;
            p.ldw = ldw;
            p.X = G;
            if (pl.pieces == 1) {
                p.D = dX;
                p.ldd = lddx;
                p.alpha_dev = scale + 1;
            } else {
                p.D = acc;
                p.ldd = ldacc;
                p.epi.C = acc;
                p.epi.ldc = ldacc;
                p.epi.beta = i > 0 ? 1.0f : 0.0f;
            }
            st = queue(h, p, split_ws);
            if (st != TCG_STATUS_SUCCESS)
                return st;
        }
        if (dW) {
            Product p = xent_dw(rows, k, width, pl.piece, type);
            p.W = X;
            p.ldw = ldx;
            p.X = G;
            p.D = static_cast<uint16_t *>(dW) + c0 * lddw;
            p.ldd = lddw;
            p.alpha_dev = scale + 1;
            st = queue(h, p, split_ws);
            if (st != TCG_STATUS_SUCCESS)
                return st;
        }
    }
    if (e == cudaSuccess && dX && pl.pieces > 1) {
        const int64_t work = (k + 3) / 4 * rows;
        const int64_t cap = static_cast<int64_t>(h->num_sms) * 8;
        const int64_t blocks = (work + 255) / 256;
        e = launch_round_out(acc, ldacc, static_cast<int>(k), static_cast<int>(rows),
                             scale + 1, dX, lddx, out_kind_of(type),
                             static_cast<int>(blocks < cap ? blocks : cap), h->stream);
        h->launches += 1;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_gemm_gated(tcgHandle_t h, tcgActivation_t activation, int64_t m, int64_t n, int64_t k,
                           const void *A, int64_t lda, const void *B, int64_t ldb, tcgDataType_t ABtype,
                           void *D, tcgDataType_t Dtype, int64_t ldd, void *Z, int64_t ldz)
{
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_gate(activation, m, n, k);
    if (st == TCG_STATUS_SUCCESS)
        st = check_types(ABtype, Dtype);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (bad_ld(lda, k, 2) || bad_ld(ldb, k, 2) || bad_ld(ldd, m, elem_size(Dtype)) ||
        (Z && (!aligned16(Z) || bad_ld(ldz, 2 * m, 2))))
        return TCG_STATUS_INVALID_VALUE;
    if (m == 0 || n == 0)
        return TCG_STATUS_SUCCESS;
    if (!D || !aligned16(D) || (k > 0 && (!A || !B || !aligned16(A) || !aligned16(B))))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {D, k > 0 ? A : nullptr, k > 0 ? B : nullptr, Z});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    Product p = gated_product(m, n, k, ABtype, Dtype);
    p.W = A;
    p.ldw = lda;
    p.X = B;
    p.ldx = ldb;
    p.D = D;
    p.ldd = ldd;
    p.epi.activation = activation;
    p.epi.Z = Z;
    p.epi.ldz = ldz;
    if (few(p))
        return queue_few(h, p);
    void *ws = nullptr;
    const size_t need = product_ws(h, p);
    if (need) {
        st = acquire_ws(h, need, &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    return queue(h, p, ws);
}

tcgStatus_t tcg_gemm_gated_workspace_size(tcgHandle_t h, int64_t m, int64_t n, int64_t k, size_t *bytes)
{
    if (!h || !bytes)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_gate(TCG_ACT_NONE, m, n, k);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    *bytes = 0;
    if (m == 0 || n == 0)
        return TCG_STATUS_SUCCESS;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        *bytes = product_ws(h, gated_product(m, n, k, TCG_R_16BF, TCG_R_16BF));
    return st;
}

tcgStatus_t tcg_gated_backward(tcgHandle_t h, tcgActivation_t activation, int64_t m, int64_t n, int64_t k,
                               const void *dD, int64_t lddd, const void *Z, int64_t ldz, const void *W,
                               int64_t ldw, const void *X, int64_t ldx, tcgDataType_t type, void *dX,
                               int64_t lddx, void *dW, int64_t lddw)
{
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_gate(activation, m, n, k);
    if (st == TCG_STATUS_SUCCESS)
        st = check_types(type, type);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (bad_rows(dD, lddd, m, 2) || bad_rows(Z, ldz, 2 * m, 2) ||
        (dX && (bad_rows(W, ldw, k, 2) || bad_rows(dX, lddx, k, 2))) ||
        (dW && (bad_rows(X, ldx, k, 2) || bad_rows(dW, lddw, k, 2))))
        return TCG_STATUS_INVALID_VALUE;
    const bool sums = m > 0 && n > 0;
    if ((sums && (!dD || !Z)) || (sums && k > 0 && ((dX && !W) || (dW && !X))))
        return TCG_STATUS_INVALID_VALUE;
    const bool dx = dX && n > 0 && k > 0, dw = dW && m > 0 && k > 0;
    if (!dx && !dw)
        return TCG_STATUS_SUCCESS;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {sums ? dD : nullptr, sums ? Z : nullptr, sums && dx ? W : nullptr,
                              sums && dw ? X : nullptr, dx ? dX : nullptr, dw ? dW : nullptr});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    const GatedPlan pl = gated_plan(h, m, n, k, dx, dw);
    void *ws = nullptr;
    if (pl.total) {
        st = acquire_ws(h, pl.total, &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    void *tail = static_cast<uint8_t *>(ws) + pl.dz_bytes;
    if (sums) {
        const cudaError_t e = launch_gate_backward(activation, type == TCG_R_16BF, static_cast<int>(n), m, dD, lddd,
                                                   Z, ldz, ws, pl.lddz, h->num_sms, h->stream);
        h->launches += 1;
        if (e != cudaSuccess) {
            cudaGetLastError();
            return TCG_STATUS_EXECUTION_FAILED;
        }
    }
    if (dx) {
        Product p = layer_dx(2 * m, n, k, 1, nullptr, type);
        p.X = ws;
        p.ldx = pl.lddz;
        p.W = W;
        p.ldw = ldw;
        p.D = dX;
        p.ldd = lddx;
        st = queue(h, p, tail);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    if (dw) {
        Product p = layer_dw(2 * m, n, k, 1, nullptr, type);
        p.X = ws;
        p.ldx = pl.lddz;
        p.W = X;
        p.ldw = ldx;
        p.D = dW;
        p.ldd = lddw;
        st = queue(h, p, tail);
    }
    return st;
}

tcgStatus_t tcg_gated_backward_workspace_size(tcgHandle_t h, int64_t m, int64_t n, int64_t k, int with_dX,
                                              int with_dW, size_t *bytes)
{
    if (!h || !bytes)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_gate(TCG_ACT_NONE, m, n, k);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        *bytes = gated_plan(h, m, n, k, with_dX, with_dW).total;
    return st;
}

tcgStatus_t tcg_rms_norm(tcgHandle_t h, int64_t rows, int64_t k, const void *X, int64_t ldx, const void *R,
                         int64_t ldr, void *S, int64_t lds, const void *W, tcgDataType_t Wtype, float eps,
                         tcgDataType_t type, void *Y, tcgDataType_t Ytype, int64_t ldy, float *scale)
{
    if (!h || !valid_type(Ytype))
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_norm(rows, k, W, Wtype, eps, type);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    const bool out8 = Ytype == TCG_R_8F_E4M3;
    if (!out8 && Ytype != type)
        return TCG_STATUS_NOT_SUPPORTED;
    if (bad_ld(ldx, k, 2) || (R && bad_rows(R, ldr, k, 2)) || (S && bad_rows(S, lds, k, 2)) ||
        bad_ld(ldy, k, elem_size(Ytype)))
        return TCG_STATUS_INVALID_VALUE;
    if (rows == 0)
        return TCG_STATUS_SUCCESS;
    if (!X || !Y || !aligned16(X) || !aligned16(Y) ||
        (out8 && (!scale || reinterpret_cast<uintptr_t>(scale) % 4)))
        return TCG_STATUS_INVALID_VALUE;
    if (S == Y || (out8 && (Y == X || Y == R)) || bad_place(S, lds, X, ldx, rows) || bad_place(S, lds, R, ldr, rows) ||
        bad_place(Y, ldy, X, ldx, rows) || bad_place(Y, ldy, R, ldr, rows))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {X, R, S, W, Y, out8 ? scale : nullptr});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    NormArgs a{};
    a.rows = rows;
    a.k = static_cast<int>(k);
    a.X = X;
    a.ldx = ldx;
    a.R = R;
    a.ldr = ldr;
    a.S = S;
    a.lds = lds;
    a.W = W;
    a.w_f32 = Wtype == TCG_R_32F;
    a.in_bf16 = type == TCG_R_16BF;
    a.out8 = out8;
    a.eps = eps;
    a.Y = Y;
    a.ldy = ldy;
    a.scale = scale;
    const cudaError_t e = launch_norm(a, h->num_sms, h->stream);
    h->launches += 1;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_rms_norm_backward(tcgHandle_t h, int64_t rows, int64_t k, const void *dY, int64_t lddy,
                                  const void *X, int64_t ldx, const void *dS, int64_t ldds, const void *W,
                                  tcgDataType_t Wtype, float eps, tcgDataType_t type, void *dX, int64_t lddx,
                                  float *dW)
{
    if (!h)
        return TCG_STATUS_INVALID_VALUE;
    tcgStatus_t st = check_norm(rows, k, W, Wtype, eps, type);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (bad_ld(lddy, k, 2) || bad_ld(ldx, k, 2) || (dS && bad_rows(dS, ldds, k, 2)) ||
        (dX && bad_rows(dX, lddx, k, 2)) || reinterpret_cast<uintptr_t>(dW) % 4)
        return TCG_STATUS_INVALID_VALUE;
    if (rows > 0 && (!dY || !X || !aligned16(dY) || !aligned16(X)))
        return TCG_STATUS_INVALID_VALUE;
    if (bad_place(dX, lddx, dY, lddy, rows) || bad_place(dX, lddx, dS, ldds, rows) || bad_place(dX, lddx, X, ldx, rows))
        return TCG_STATUS_INVALID_VALUE;
    if (!dW && (!dX || rows == 0))
        return TCG_STATUS_SUCCESS;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = rows > 0 ? check_device(h, {dY, X, dS, W, dX, dW}) : check_device(h, {dW});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    NormBackwardArgs a{};
    a.rows = rows;
    a.k = static_cast<int>(k);
    a.dY = dY;
    a.lddy = lddy;
    a.X = X;
    a.ldx = ldx;
    a.dS = dS;
    a.ldds = ldds;
    a.W = W;
    a.w_f32 = Wtype == TCG_R_32F;
    a.in_bf16 = type == TCG_R_16BF;
    a.eps = eps;
    a.dX = dX;
    a.lddx = lddx;
    const int blocks = norm_backward_blocks(rows, k, h->num_sms);
    if (dW && blocks > 1) {
        void *ws = nullptr;
        st = acquire_ws(h, static_cast<size_t>(blocks) * k * sizeof(float), &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
        a.part = static_cast<float *>(ws);
    }
    const cudaError_t e = launch_norm_backward(a, dW, h->num_sms, h->stream);
    h->launches += (rows > 0) + (dW && blocks != 1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TCG_STATUS_EXECUTION_FAILED;
    }
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_rms_norm_backward_workspace_size(tcgHandle_t h, int64_t rows, int64_t k, size_t *bytes)
{
    if (!h || !bytes || rows < 0 || k < 1)
        return TCG_STATUS_INVALID_VALUE;
    if (k > kNormMaxK)
        return TCG_STATUS_NOT_SUPPORTED;
    const tcgStatus_t st = bind_device(h);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    const int blocks = norm_backward_blocks(rows, k, h->num_sms);
    *bytes = blocks > 1 ? static_cast<size_t>(blocks) * k * sizeof(float) : 0;
    return TCG_STATUS_SUCCESS;
}

tcgStatus_t tcg_gemm_4bit(tcgHandle_t h, int64_t m, int64_t n, int64_t k, int64_t group, const void *A,
                          int64_t lda, const void *scales, const void *zeros, tcgDataType_t Stype, const void *B,
                          int64_t ldb, tcgDataType_t Btype, void *D, tcgDataType_t Dtype, int64_t ldd, int gated,
                          const tcgEpilogue_t *epilogue)
{
    if (!h || !valid_type(Stype))
        return TCG_STATUS_INVALID_VALUE;
    tcgEpilogue_t epi = {};
    if (epilogue)
        epi = *epilogue;
    tcgStatus_t st = check_types(Btype, Dtype);
    if (st == TCG_STATUS_SUCCESS)
        st = check_epilogue(epi, m, n, Btype, Dtype);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    if (m < 0 || n < 0 || k < 0 || lda < k / 2 + k % 2 || lda < 1 || lda % 16 || bad_ld(ldb, k, 2) ||
        bad_ld(ldd, m, elem_size(Dtype)))
        return TCG_STATUS_INVALID_VALUE;
    if ((group != 32 && group != 64 && group != 128) || (Stype != TCG_R_32F && Stype != Btype) || epi.Z ||
        (gated && (epi.bias || epi.beta != 0.0f)) || m > kMaxExtent / 2 || n > kMaxExtent || k > kMaxK / 2)
        return TCG_STATUS_NOT_SUPPORTED;
    if (m == 0 || n == 0)
        return TCG_STATUS_SUCCESS;
    const uintptr_t es = elem_size(Stype);
    if (!D || !aligned16(D) ||
        (k > 0 && (!A || !B || !scales || !aligned16(A) || !aligned16(B) ||
                   reinterpret_cast<uintptr_t>(scales) % es || reinterpret_cast<uintptr_t>(zeros) % es)))
        return TCG_STATUS_INVALID_VALUE;
    if (epi.beta != 0.0f && bad_place(D, ldd, epi.C, epi.ldc, n))
        return TCG_STATUS_INVALID_VALUE;
    st = bind_device(h);
    if (st == TCG_STATUS_SUCCESS)
        st = check_device(h, {D, k > 0 ? A : nullptr, k > 0 ? B : nullptr, k > 0 ? scales : nullptr,
                              k > 0 ? zeros : nullptr, epi.bias, epi.beta != 0.0f ? epi.C : nullptr});
    if (st != TCG_STATUS_SUCCESS)
        return st;
    h->used = true;
    W4Args a{};
    a.rows = gated ? 2 * m : m;
    a.k = k;
    a.tokens = static_cast<int>(n);
    a.group = static_cast<int>(group);
    a.W = static_cast<const uint8_t *>(A);
    a.ldw = lda;
    a.scales = scales;
    a.zeros = zeros;
    a.s_f32 = Stype == TCG_R_32F;
    a.X = B;
    a.ldx = ldb;
    a.in_bf16 = Btype == TCG_R_16BF;
    a.out_kind = out_kind_of(Dtype);
    a.D = D;
    a.ldd = ldd;
    a.bias = epi.bias;
    a.bias_f32 = epi.bias_type == TCG_R_32F;
    a.C = epi.beta != 0.0f ? epi.C : nullptr;
    a.ldc = epi.ldc;
    a.beta = epi.beta;
    a.act = epi.activation;
    a.gated = gated != 0;
    if (w4_packed(n, a.rows, k, a.gated)) {
        const cudaError_t e = launch_w4(a, h->num_sms, h->stream);
        h->launches += 1;
        if (e != cudaSuccess) {
            cudaGetLastError();
            return TCG_STATUS_EXECUTION_FAILED;
        }
        return TCG_STATUS_SUCCESS;
    }
    W4Plan pl = w4_plan(h, m, n, k, gated != 0);
    void *ws = nullptr;
    if (pl.total) {
        st = acquire_ws(h, pl.total, &ws);
        if (st != TCG_STATUS_SUCCESS)
            return st;
    }
    uint8_t *at = static_cast<uint8_t *>(ws);
    Product &p = pl.p;
    p.in = Btype;
    p.out = Dtype;
    p.W = ws;
    p.X = B;
    p.ldx = ldb;
    p.D = D;
    p.ldd = ldd;
    p.epi = epi;
    LmArgs more{};
    float *scale = reinterpret_cast<float *>(at + pl.w_bytes), *rest = scale + pl.t_bytes / sizeof(float);
    float *sums = rest + pl.t_bytes / sizeof(float);
    more.group_mmas = static_cast<int>(group / 16);
    more.k_groups = static_cast<int>(ceil_div(k, group));
    more.group_scale = scale;
    more.group_rest = zeros ? rest : nullptr;
    more.group_ld = pl.ld_t;
    more.group_sum = sums;
    more.sum_ld = pl.ld_sum;
    if (k > 0) {
        cudaError_t e = launch_w4_expand(a, ws, p.ldw, scale, rest, pl.ld_t, h->num_sms, h->stream);
        if (e == cudaSuccess && zeros)
            e = launch_w4_sums(a, sums, pl.ld_sum, h->stream);
        h->launches += zeros ? 2 : 1;
        if (e != cudaSuccess) {
            cudaGetLastError();
            return TCG_STATUS_EXECUTION_FAILED;
        }
    }
    return queue(h, p, at + pl.w_bytes + 2 * pl.t_bytes + pl.sum_bytes, more);
}

tcgStatus_t tcg_gemm_4bit_workspace_size(tcgHandle_t h, int64_t m, int64_t n, int64_t k, int gated, size_t *bytes)
{
    if (!h || !bytes || m < 0 || n < 0 || k < 0)
        return TCG_STATUS_INVALID_VALUE;
    if (m > kMaxExtent / 2 || n > kMaxExtent || k > kMaxK / 2)
        return TCG_STATUS_NOT_SUPPORTED;
    *bytes = 0;
    if (m == 0 || n == 0 || w4_packed(n, gated ? 2 * m : m, k, gated))
        return TCG_STATUS_SUCCESS;
    const tcgStatus_t st = bind_device(h);
    if (st != TCG_STATUS_SUCCESS)
        return st;
    *bytes = w4_plan(h, m, n, k, gated != 0).total;
    return TCG_STATUS_SUCCESS;
}

}  // extern "C"
