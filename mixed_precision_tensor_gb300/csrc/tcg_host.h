// tcg_host.h -- the handle and the host helpers shared by the library's host sources
// (tcg_api.cu, which defines them, and tcg_lm_api.cu).
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tcg.h"
#include "tcg_internal.h"
#include "tcg_lm.h"

namespace tcg {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
constexpr int kMapCacheSize = 32;
constexpr int kPtrCacheSize = 16;

// Device words of a handle: the error word's line, then the split counters.
constexpr int kErrAreaWords = 64;
constexpr size_t kErrAreaBytes = sizeof(uint32_t) * (kErrAreaWords + kLmCounters);

struct MapKey {
    const void *ptr;
    int dtype;
    int rank;
    int swizzle;
    uint64_t dims[5];
    uint64_t strides[4];
    uint32_t box[5];
    bool operator==(const MapKey &o) const { return std::memcmp(this, &o, sizeof(MapKey)) == 0; }
};

constexpr int kHostChunks = 16;     // chunks of a host-buffer call (events per handle)
constexpr int kHostPanels = 4;      // chunks of the panel / batch-group split

struct MapEntry {
    MapKey key;
    CUtensorMap map;
    bool valid;
};

// A workspace that a newer one has replaced, still in use by a captured graph.
struct KeptBlock {
    void *ptr;
    KeptBlock *next;
};

}  // namespace tcg

struct tcgContext {
    int device = -1;
    int num_sms = 0;
    cudaStream_t stream = nullptr;
    uint32_t *d_err = nullptr;
    uint32_t *d_cnt = nullptr;             // split counters (tcg_lm.h), zero between calls
    unsigned long long *d_clk = nullptr;   // clock probe counters (tcg_set_clock_probe)
    bool clk_on = false;
    void *ws_user = nullptr;
    size_t ws_user_bytes = 0;
    void *ws_own = nullptr;
    size_t ws_own_bytes = 0;
    bool ws_captured = false;              // a captured call has been given ws_own
    tcg::KeptBlock *ws_kept = nullptr;
    unsigned long long wait_limit_ns = tcg::kDefaultWaitNs;
    int fault_inject = 0;
    uint64_t launches = 0;
    uint32_t last_err_bits = 0;
    int cta_group = 2;
    int group_m = 0;           // 0: choose per problem
    int split_k = 0;           // 0: choose per problem, 1: never split, >= 2: that many ranges
    int tile_n = 0;            // 0: choose per problem, or kBN / kBNNarrow
    int tf32_round = 0;        // TF32 rounding: 0 choose, 1 pre-pass kernels, 2 in the GEMM
    // Host-buffer calls: device copies of A, B, C (grown on demand) and two copy streams.
    void *stage_buf[3] = {nullptr, nullptr, nullptr};
    size_t stage_bytes[3] = {0, 0, 0};
    cudaStream_t h2d = nullptr, d2h = nullptr;
    cudaEvent_t ev_in[tcg::kHostChunks] = {}, ev_out[tcg::kHostChunks] = {};
    int max_ctas[3] = {0, 0, 0};
    bool used = false;
    tcg::EncodeTiledFn encode = nullptr;
    tcg::MapEntry cache[tcg::kMapCacheSize];
    int cache_next = 0;
    const void *ptr_ok[tcg::kPtrCacheSize] = {};   // pointers already found to be device memory
    int ptr_next = 0;
};

namespace tcg {

// Binds the handle to the current device on its first call (capability check, error word).
tcgStatus_t bind_device(tcgContext *h);
// SUCCESS if the pointers (null ones aside) are device memory of device dev.
tcgStatus_t device_ptrs_ok(int dev, const void *const *ptrs, int n);
// Tensor map of rank 3 or 4 with zero fill out of range, from the handle's cache of maps.
tcgStatus_t get_map(tcgContext *h, const void *ptr, tcgDataType_t t, int rank,
                    const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
                    CUtensorMap *out, bool swizzle = true);
// Map for one operand as the kernels load it (see OperandMode).
tcgStatus_t operand_map(tcgContext *h, const void *ptr, tcgDataType_t t, bool kmajor,
                        int64_t rows, int64_t k, int64_t ld, int64_t stride, int64_t batch,
                        int box_rows, int k_row, bool *bcast, int *mode, CUtensorMap *out);
// The caller's workspace, or the handle's own grown to `need` bytes.
tcgStatus_t acquire_ws(tcgContext *h, size_t need, void **ws);
int elem_size(tcgDataType_t t);
bool valid_type(int t);
bool aligned16(const void *p);

}  // namespace tcg
