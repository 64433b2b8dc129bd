// evict.cu -- eviction from the cache by accumulated attention weight, and the
// reset of the weights of newly written slots.
//
// For every (sequence, KV head) of n = ctx tokens and a budget: the `recent`
// newest tokens are kept, and of the others the budget - recent with the
// largest weights (ties to the lower position, weights compared in IEEE
// totalOrder); all of them when n <= budget. The kept tokens' K and V rows
// and weights are copied, in ascending order of position, to the sequence's
// destination blocks: token i of the result goes to position i.
#include "common.cuh"
#include "kernels.h"
#include "subset.h"

namespace pa {
namespace {

constexpr int kSelThreads = 1024, kHistCopies = 8;
constexpr int kKeysCap = 48 * 1024;  // keys held in shared memory; longer rows read them again

// one CTA per (sequence, KV head): the kept positions
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int cap) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ int hist[kHistCopies * 256];
    __shared__ int red[2 * kSelThreads / 32 + 3];
    const int b = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv, tid = threadIdx.x;
    pdl_trigger();  // the copy waits for this kernel's end before it reads anything
    pdl_wait();
    const int ctx = min(max(__ldg(a.ctx + b), 0), a.MBS * kBlockSize);
    int32_t *kept = a.kept + int64_t(blockIdx.x) * a.budget;
    if (kvh == 0 && tid == 0) a.new_lens[b] = min(ctx, a.budget);
    if (ctx <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < ctx ? i : -1;
        return;
    }
    const int recent = min(a.recent, a.budget), n = ctx - recent, top = a.budget - recent;
    for (int i = tid; i < recent; i += kSelThreads) kept[top + i] = n + i;
    if (top == 0) return;
    const int32_t *bt = a.bt + int64_t(b) * a.MBS;
    auto load = [&](int j) -> uint32_t {
        const int phys = __ldg(bt + j / kBlockSize);
        if (phys < 0 || phys >= a.NB) return 0u;  // no such block: below every weight
        return f32_order_key(__ldcg(a.weights + (int64_t(phys) * a.Hkv + kvh) * kBlockSize + j % kBlockSize));
    };
    const bool cached = n <= cap;
    if (cached) {
        // four tokens of a block per load, U loads (and their table entries) in flight per thread
        constexpr int U = 4;
        const int nq = (n + 3) / 4;
        for (int q0 = tid; q0 < nq; q0 += U * kSelThreads) {
            int phys[U];
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kSelThreads;
                phys[u] = q < nq ? __ldg(bt + q / (kBlockSize / 4)) : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kSelThreads;
                if (phys[u] >= a.NB) phys[u] = -1;
                if (phys[u] >= 0)
                    v[u] = __ldcg(reinterpret_cast<const float4 *>(
                                      a.weights + (int64_t(phys[u]) * a.Hkv + kvh) * kBlockSize) + q % (kBlockSize / 4));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kSelThreads;
                if (q >= nq) continue;
                const bool in = phys[u] >= 0;
                *reinterpret_cast<uint4 *>(keys + 4 * q) =
                    make_uint4(in ? f32_order_key(v[u].x) : 0u, in ? f32_order_key(v[u].y) : 0u,
                               in ? f32_order_key(v[u].z) : 0u, in ? f32_order_key(v[u].w) : 0u);
            }
        }
        __syncthreads();
    }
    auto key_of = [&](int j) -> uint32_t { return cached ? keys[j] : load(j); };
    uint32_t thr;
    int keq;
    cta_topk_threshold<kSelThreads, kHistCopies>(key_of, n, top, hist, red, thr, keq);
    cta_topk_emit<kSelThreads>(key_of, n, thr, keq, red, [&](int r, int j) { kept[r] = j; });
}

// The copy: a warp per `chunk` (8 or 32) kept tokens of a (sequence, KV head). Bound by HBM:
// every kept row is read and written once. A lane finds one token's rows; then
// the warp moves the tokens one after the other, K and V side by side (D = 128:
// 16 lanes of 16 bytes each; D = 64: two tokens at once), kMove loads per lane
// in flight.
// No early launch of the next kernel: it may read new_lens before it waits.
constexpr int kMove = 8;

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a, int chunk) {
    constexpr int LR = D / 8;         // lanes per row
    constexpr int TP = 32 / (2 * LR); // tokens at once
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int per = (a.budget + chunk - 1) / chunk;  // warps per (sequence, KV head)
    const int64_t warp = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t seg = warp / per;
    if (seg >= int64_t(a.B) * a.Hkv) return;
    const int i0 = int(warp - seg * per) * chunk, kvh = int(seg % a.Hkv), b = int(seg / a.Hkv);
    const int i = i0 + lane;
    const int j = lane < chunk && i < a.budget ? __ldcg(a.kept + seg * a.budget + i) : -1;
    // this lane's token: its row in the cache, before and after; -1: not copied
    int64_t from = -1, to = -1;
    if (j >= 0) {
        const int src = __ldg(a.bt + int64_t(b) * a.MBS + j / kBlockSize);
        const int dst = __ldg(a.dst + int64_t(b) * a.DMBS + i / kBlockSize);
        if (src >= 0 && src < a.NB && dst >= 0 && dst < a.NB) {
            from = (int64_t(src) * kBlockSize + j % kBlockSize) * a.Hkv + kvh;
            to = (int64_t(dst) * kBlockSize + i % kBlockSize) * a.Hkv + kvh;
            a.weights[(int64_t(dst) * a.Hkv + kvh) * kBlockSize + i % kBlockSize] =
                __ldcg(a.weights + (int64_t(src) * a.Hkv + kvh) * kBlockSize + j % kBlockSize);
        }
    }
    if (!__any_sync(0xffffffffu, from >= 0)) return;
    const int half = lane / LR % 2, e = lane % LR;
    uint4 *cache = reinterpret_cast<uint4 *>(half ? a.vc : a.kc) + e;
#pragma unroll 1
    for (int t0 = 0; t0 < chunk; t0 += kMove * TP) {
        uint4 v[kMove];
        int64_t y[kMove];
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            const int t = t0 + u * TP + lane / (2 * LR);
            const int64_t x = __shfl_sync(0xffffffffu, from, t);
            y[u] = __shfl_sync(0xffffffffu, to, t);
            if (x >= 0) v[u] = __ldcs(cache + x * LR);
        }
#pragma unroll
        for (int u = 0; u < kMove; ++u)
            if (y[u] >= 0) __stcs(cache + y[u] * LR, v[u]);
    }
}

__global__ void __launch_bounds__(256) reset_weights_kernel(float *weights, const int64_t *slots, int64_t T, int Hkv,
                                                            int64_t NB) {
    pdl_wait();
    const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (at >= T * Hkv) return;
    const int64_t slot = __ldg(slots + at / Hkv);
    if (slot < 0 || slot >= NB * kBlockSize) return;
    weights[(slot / kBlockSize * Hkv + at % Hkv) * kBlockSize + slot % kBlockSize] = 0.f;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int head_dim, cudaStream_t stream) {
    const int64_t longest = int64_t(a.MBS) * kBlockSize;  // a multiple of four
    const int cap = longest < kKeysCap ? int(longest) : kKeysCap;
    const size_t smem = size_t(cap) * 4;
    cudaError_t e = smem_once(reinterpret_cast<const void *>(evict_select_kernel), size_t(kKeysCap) * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_select_kernel, dim3(a.B * a.Hkv), dim3(kSelThreads), smem, stream, a, cap);
    if (e != cudaSuccess) return e;
    // 32 tokens per warp read kept in whole lines; where that leaves SMs without work (fewer than about
    // 8 warps each), 8 tokens per warp: one sequence of 1024 kept tokens 13.5 -> 11 us, select included
    const int64_t segs = int64_t(a.B) * a.Hkv;
    const int chunk = segs * ((a.budget + 31) / 32) < 1216 ? 8 : 32;
    const int64_t warps = segs * ((a.budget + chunk - 1) / chunk);
    const dim3 grid(unsigned((warps + 7) / 8));
    return head_dim == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(256), 0, stream, a, chunk)
                           : launch_pdl(evict_move_kernel<64>, grid, dim3(256), 0, stream, a, chunk);
}

cudaError_t launch_reset_weights(float *weights, const int64_t *slots, int64_t T, int Hkv, int64_t NB,
                                 cudaStream_t stream) {
    const int64_t n = T * Hkv;
    return launch_pdl(reset_weights_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, stream, weights, slots, T,
                      Hkv, NB);
}

}  // namespace pa
