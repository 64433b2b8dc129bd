// subset.h -- internal interface of the decode operators that read a part of
// the cache, or share it between sequences (stream_decode.cu, row_tiles.cu), and
// of eviction (evict.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace pa {

constexpr int kMaxWindowRows = 1 << 20;  // query rows of a windowed multi-token call

enum CacheKind { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheE4m3Block = 2 };

// A unit of the row-tile kernel that was cut between CTAs: query rows r0 ..
// r0 + nr - 1 of sequence s and KV head kvh, row r0 + i seeing tokens before
// base + i, in `pieces` pieces from the CTA on in whose range it begins.
struct alignas(16) CutUnit {
    int s, kvh, r0, nr, base, pieces, pad[2];
};

// Attention of query rows over the tokens a row sees:
//   its sequence's prefix (pt / plen: the prefix blocks of its group), then
//   its own tokens t < lim with t < sinks or t >= lim - window.
struct SubsetArgs {
    const uint16_t *q;            // [rows][Hq][D] bf16
    uint16_t *out;                // [rows][Hq][D] bf16
    const void *kc, *vc;          // the caches, in the layout of `kind`
    const float *k_scale, *v_scale;
    const int32_t *bt, *ctx;      // [nseq][MBS], [nseq]
    const int32_t *cu_q;          // [nseq + 1] query-row offsets; null: one row per sequence
    const int32_t *pt, *plen;     // [ngroups][PMBS], [ngroups] prefixes; null: none
    const int32_t *cu_g;          // [ngroups + 1] sequence offsets of the groups
    float *weights;               // [NB][Hkv][16]: accumulated attention weights; null: none
    int64_t NB;
    int MBS, PMBS, nseq, ngroups, rows, Hq, Hkv, G;
    int window, sinks;            // window: INT_MAX when everything before lim is seen
    float scale_log2;             // softmax scale * log2(e)
    // workspace
    int32_t *status;              // status word
    int32_t *counters;            // [workers] arrivals at what begins in a worker's range and leaves it (zero between calls)
    float *part;                  // [2 * workers] pieces of segments cut between workers: O, m, l
    float *slots;                 // [2 * CTAs] pieces of row-tile units cut between CTAs
    float *rowres, *rowml;        // prefixes: [rows][Hq][D] O and [rows][Hq][2] m, l of units that were not cut
    CutUnit *cuts;                // row tiles over windows: [CTAs] the cut unit that begins in each range
    int4 *desc;                   // prefixes: [rows][Hkv] first CTA, pieces, row tile, first row in it
    int pgrid;                    // prefixes: CTAs of the row-tile kernel
    float *ownres, *ownml;        // prefixes beside the row tiles: [rows][Hq][D] O and [rows][Hq][2] m, l of the own tokens (else null)
    float *lse;                   // weights: [nseq][Hq] log2 of the normaliser
    float *logits;                // weights: [nseq][Hkv][MBS][G][16] logits (log2 domain)
    uint64_t wait_ns;             // limit of every bounded wait
    bool fused_add;               // weights: added by the streaming kernel itself
    int stop_item;                // failure tests: a warp's copies stop at this item (else INT_MAX)
    int min_items;                // row tiles: tiles of a CTA's range at least
};

// What was done per (device, kernel). Allocates nothing and throws nothing: it runs below C entry points. Beyond
// its devices and kernels nothing is noted, and the caller does it again.
struct DoneOnce {
    static constexpr int kDevices = 64, kKernels = 128;
    std::atomic<const void *> at[kDevices][kKernels];

    // the slot that holds the kernel, or the free one to note it in (else null)
    std::atomic<const void *> *find(int dev, const void *kernel, bool &done) noexcept {
        done = false;
        if (dev < 0 || dev >= kDevices) return nullptr;
        const unsigned h = unsigned(reinterpret_cast<uintptr_t>(kernel) >> 4) * 2654435761u >> 25;
        for (unsigned i = 0; i < kKernels; ++i) {
            std::atomic<const void *> &s = at[dev][(h + i) % kKernels];
            const void *k = s.load(std::memory_order_acquire);
            done = k == kernel;
            if (done || !k) return &s;
        }
        return nullptr;
    }
    // a slot that another thread took first is left to it: the kernel is noted at its next call
    static void note(std::atomic<const void *> *slot, const void *kernel) noexcept {
        const void *none = nullptr;
        if (slot) slot->compare_exchange_strong(none, kernel, std::memory_order_acq_rel);
    }
};

// A kernel's limit of dynamic shared memory, set once per device.
inline cudaError_t smem_once(const void *kernel, size_t bytes) noexcept {
    static DoneOnce once;
    int dev = 0;
    bool done;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<const void *> *slot = once.find(dev, kernel, done);
    if (done) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) DoneOnce::note(slot, kernel);
    return e;
}

// one query row per sequence, window and sinks, or (weights set) the dense
// decode that adds up the attention weights, or (pt set) prefix and own tokens,
// with ownres the own ones only; tk, tv: tensor maps of the caches
size_t stream_workers(int sms);
size_t stream_part_floats(int sms, int head_dim);
cudaError_t launch_stream_decode(const CUtensorMap &tk, const CUtensorMap &tv, const SubsetArgs &a, int head_dim,
                                 CacheKind kind, int sms, cudaStream_t stream);

// query rows of any number per sequence over window and sinks, or (pt set) the
// rows of groups of sequences over their prefixes (bf16 cache), left in slots / rowres / desc;
// tq: tensor map of the queries
constexpr int kRowTile = 128;  // rows (query row, head) of a row tile
size_t row_tiles_slot_floats(int head_dim);
cudaError_t launch_row_tiles(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq, const SubsetArgs &a,
                             int head_dim, CacheKind kind, int sms, cudaStream_t stream);

// rows of own part and prefix parts joined, written out
cudaError_t launch_prefix_join(const SubsetArgs &a, int head_dim, cudaStream_t stream);

struct EvictArgs {
    int32_t *kept, *new_lens;     // [B][Hkv][budget], [B]
    uint16_t *kc, *vc;            // [NB][16][Hkv][D] bf16
    float *weights;               // [NB][Hkv][16]
    const int32_t *bt, *ctx, *dst;  // [B][MBS], [B], [B][DMBS]
    int64_t NB;
    int MBS, DMBS, B, Hkv, budget, recent;
};

cudaError_t launch_evict(const EvictArgs &a, int head_dim, int sms, cudaStream_t stream);
cudaError_t launch_reset_weights(float *weights, const int64_t *slots, int64_t T, int Hkv, int64_t NB,
                                 cudaStream_t stream);

}  // namespace pa
