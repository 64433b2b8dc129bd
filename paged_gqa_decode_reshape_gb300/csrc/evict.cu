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

constexpr int kSelThreads = 512, kHistCopies = 8;
constexpr int kKeysCap = 48 * 1024;  // keys held in shared memory; longer rows read them again

// one CTA per (sequence, KV head): the kept positions
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int cap) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kHistCopies * 256];
    __shared__ int red[2 * kSelThreads / 32 + 3];
    const int b = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv, tid = threadIdx.x;
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
        for (int j = tid; j < n; j += kSelThreads) keys[j] = load(j);
        __syncthreads();
    }
    auto key_of = [&](int j) -> uint32_t { return cached ? keys[j] : load(j); };
    uint32_t thr;
    int keq;
    cta_topk_threshold<kSelThreads, kHistCopies>(key_of, n, top, hist, red, thr, keq);
    cta_topk_emit<kSelThreads>(key_of, n, thr, keq, red, [&](int r, int j) { kept[r] = j; });
}

// one warp per kept token and KV head: its K and V rows and its weight
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t at = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t total = int64_t(a.B) * a.Hkv * a.budget;
    if (at >= total) return;
    const int i = int(at % a.budget), kvh = int(at / a.budget % a.Hkv), b = int(at / a.budget / a.Hkv);
    const int j = __ldcg(a.kept + at);
    if (j < 0) return;
    const int src = __ldg(a.bt + int64_t(b) * a.MBS + j / kBlockSize);
    const int dst = __ldg(a.dst + int64_t(b) * a.DMBS + i / kBlockSize);
    if (src < 0 || src >= a.NB || dst < 0 || dst >= a.NB) return;
    const int64_t x = ((int64_t(src) * kBlockSize + j % kBlockSize) * a.Hkv + kvh) * D;
    const int64_t y = ((int64_t(dst) * kBlockSize + i % kBlockSize) * a.Hkv + kvh) * D;
    for (int e = lane; e < D / 4; e += 32) {
        const int d = 8 * (e % (D / 8));
        uint16_t *c = e < D / 8 ? a.kc : a.vc;
        *reinterpret_cast<uint4 *>(c + y + d) = *reinterpret_cast<const uint4 *>(c + x + d);
    }
    if (lane == 0)
        a.weights[(int64_t(dst) * a.Hkv + kvh) * kBlockSize + i % kBlockSize] =
            a.weights[(int64_t(src) * a.Hkv + kvh) * kBlockSize + j % kBlockSize];
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
    const int64_t longest = int64_t(a.MBS) * kBlockSize;
    const int cap = longest < kKeysCap ? int(longest) : kKeysCap;
    const size_t smem = size_t(cap) * 4;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kKeysCap * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_select_kernel, dim3(a.B * a.Hkv), dim3(kSelThreads), smem, stream, a, cap);
    if (e != cudaSuccess) return e;
    const int64_t warps = int64_t(a.B) * a.Hkv * a.budget;
    const dim3 grid(unsigned((warps + 7) / 8));
    return head_dim == 128 ? launch_pdl(evict_move_kernel<128>, grid, dim3(256), 0, stream, a)
                           : launch_pdl(evict_move_kernel<64>, grid, dim3(256), 0, stream, a);
}

cudaError_t launch_reset_weights(float *weights, const int64_t *slots, int64_t T, int Hkv, int64_t NB,
                                 cudaStream_t stream) {
    const int64_t n = T * Hkv;
    return launch_pdl(reset_weights_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, stream, weights, slots, T,
                      Hkv, NB);
}

}  // namespace pa
