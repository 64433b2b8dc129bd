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

constexpr int kSelThreads = 1024;
constexpr int kBins = 2 * kSelThreads;  // of a selection pass
constexpr int kCand = 256;              // keys ranked against one another at the end
// From this many SMs per (sequence, KV head) on, one launch in which every CTA
// selects and copies a share; below, a CTA selects for all and a second launch
// copies. One sequence of 1500 tokens, 1024 kept: 6.5 us in one launch, 6.8 in two
// (and 2 us of the host); 9 of 2000, 512 kept: 8.5 and 9.6; 9 of 8192, 4096 kept:
// 37.5 and 37.8; 16 of those, two CTAs each: 62.7 and 59.4 (4 KV heads of 128: the
// copy wants more warps than two CTAs of 1024 threads per head have).
constexpr int kMinParts = 4;
constexpr int kKeysCap = 48 * 1024;  // keys held in shared memory; longer rows read them again

struct SelectScratch {
    int hist[kBins];
    uint4 cand[kCand / 4];
    int red[2 * kSelThreads / 32 + 4];
};

// The k-th largest of n keys (n > k >= 1), keys4(j) the four from j on (j a multiple
// of 4), in totalOrder: thr, and keq, how many keys equal to it belong to the k
// (every key above it does). lo, hi: the least and the largest key that this
// thread has seen. A pass sorts the keys of lo .. hi into 2048 bins of equal width
// and goes on with the bin that holds the k-th; once that has at most kCand keys
// they are ranked against one another: one or two passes are the usual case. (Fixed
// digits of 8 bits took four, and weights, which lie within a few octaves, met in
// few bins of the first: 8.2 us for 8.7K keys.)
template <typename Keys4>
__device__ __forceinline__ void kth_largest(Keys4 keys4, int n, int k, uint32_t lo, uint32_t hi, SelectScratch &sm,
                                            uint32_t &thr, int &keq) {
    constexpr int NW = kSelThreads / 32;
    static_assert(NW == 32, "one lane per warp");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *red = sm.red;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        red[warp] = int(lo);
        red[NW + warp] = int(hi);
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, uint32_t(red[lane]));
    hi = __reduce_max_sync(0xffffffffu, uint32_t(red[NW + lane]));
    while (true) {
        thr = hi;
        keq = k;
        if (lo == hi) return;  // every key left equal: the k lowest positions
        const int sh = max(21 - __clz(hi - lo), 0);  // (hi - lo) >> sh < kBins
        sm.hist[tid] = 0;
        sm.hist[tid + kSelThreads] = 0;
        if (tid == 0) red[2 * NW + 3] = 0;
        __syncthreads();
        for (int j = 4 * tid; j < n; j += 4 * kSelThreads) {
            const uint4 u = keys4(j);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < n && v[e] - lo <= hi - lo) atomicAdd(&sm.hist[(v[e] - lo) >> sh], 1);
        }
        __syncthreads();
        // two bins per thread, descending
        const int c0 = sm.hist[kBins - 1 - 2 * tid], c1 = sm.hist[kBins - 2 - 2 * tid];
        int incl = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) red[warp] = incl;
        __syncthreads();
        incl += __reduce_add_sync(0xffffffffu, lane < warp ? red[lane] : 0);
        const int above = incl - c0 - c1;  // keys in higher bins
        if (above < k && k <= incl) {
            const bool first = k <= above + c0;
            red[2 * NW] = kBins - 1 - 2 * tid - (first ? 0 : 1);
            red[2 * NW + 1] = first ? above : above + c0;
            red[2 * NW + 2] = first ? c0 : c1;
        }
        __syncthreads();
        const int m = red[2 * NW + 2];
        k -= red[2 * NW + 1];
        lo += uint32_t(red[2 * NW]) << sh;
        if (hi - lo >= 1u << sh) hi = lo + ((1u << sh) - 1u);
        if (m == k && lo != 0u) {  // the whole bin
            thr = lo - 1u;
            keq = 0;
            return;
        }
        if (m <= kCand) {
            uint32_t *cand = reinterpret_cast<uint32_t *>(sm.cand);
            if (tid < 4 && m + tid < kCand) cand[m + tid] = 0u;  // read as part of the last four: below or equal to all
            for (int j = 4 * tid; j < n; j += 4 * kSelThreads) {
                const uint4 u = keys4(j);
                const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < n && v[e] - lo <= hi - lo) cand[atomicAdd(&red[2 * NW + 3], 1)] = v[e];
            }
            __syncthreads();
            if (tid < m) {
                const uint32_t c = cand[tid];
                int gt = 0, ge = 0;
                for (int i = 0; i < (m + 3) / 4; ++i) {
                    const uint4 o = sm.cand[i];
                    gt += (o.x > c) + (o.y > c) + (o.z > c) + (o.w > c);
                    ge += (o.x >= c) + (o.y >= c) + (o.z >= c) + (o.w >= c);
                }
                if (c == 0u) ge = m;  // not the padding
                if (gt < k && k <= ge) {
                    red[2 * NW] = int(c);
                    red[2 * NW + 1] = k - gt;
                }
            }
            __syncthreads();
            thr = uint32_t(red[2 * NW]);
            keq = red[2 * NW + 1];
            return;
        }
    }
}

// The selection for a threshold, ascending: emit(r, j) for the r-th selected
// position j. Warps own consecutive ranges, a lane four keys at a time (a lane per
// key, with ballots, took 3.4 us for 8.7K keys).
template <typename Keys4, typename Emit>
__device__ __forceinline__ void emit_selected(Keys4 keys4, int n, uint32_t thr, int keq, SelectScratch &sm, Emit emit) {
    constexpr int NW = kSelThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = ((n + 127) / 128 + NW - 1) / NW, j0 = warp * rows * 128, j1 = min(n, j0 + rows * 128);
    int *red = sm.red;
    int gt = 0, eq = 0;
    for (int j = j0 + 4 * lane; j < j1; j += 128) {
        const uint4 u = keys4(j);
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            gt += j + e < j1 && v[e] > thr;
            eq += j + e < j1 && v[e] == thr;
        }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    __syncthreads();  // red is free
    if (lane == 0) {
        red[warp] = gt;
        red[NW + warp] = eq;
    }
    __syncthreads();
    // taken before this warp's range: those above thr, and of those equal to it the first keq
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane] : 0);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? red[NW + lane] : 0);
    for (int j = j0; j < j1; j += 128) {
        const int jj = j + 4 * lane;
        const uint4 u = jj < j1 ? keys4(jj) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
        uint32_t g = 0, q = 0;  // bits of this lane's keys above and at the threshold
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            g |= uint32_t(jj + e < j1 && v[e] > thr) << e;
            q |= uint32_t(jj + e < j1 && v[e] == thr) << e;
        }
        const int mine = __popc(g) | __popc(q) << 16;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        int gb = gt + ((incl - mine) & 0xffff), qb = eq + ((incl - mine) >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool ge = (g >> e) & 1u, qe = (q >> e) & 1u;
            if (ge || (qe && qb < keq)) emit(gb + min(qb, keq), jj + e);
            gb += ge;
            qb += qe;
        }
        gt += all & 0xffff;
        eq += all >> 16;
    }
}

// The kept positions of segment (b, kvh) with ranks r0 <= r < r1, by a whole CTA.
__device__ __forceinline__ void select_kept(const EvictArgs &a, int b, int kvh, int cap, int r0, int r1) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelectScratch sm;
    const int tid = threadIdx.x;
    const int ctx = min(max(__ldg(a.ctx + b), 0), a.MBS * kBlockSize);
    int32_t *kept = a.kept + (int64_t(b) * a.Hkv + kvh) * a.budget;
    if (kvh == 0 && r0 == 0 && tid == 0) a.new_lens[b] = min(ctx, a.budget);
    if (ctx <= a.budget) {
        for (int i = r0 + tid; i < r1; i += kSelThreads) kept[i] = i < ctx ? i : -1;
        return;
    }
    const int recent = min(a.recent, a.budget), n = ctx - recent, top = a.budget - recent;
    for (int i = max(r0 - top, 0) + tid; top + i < r1; i += kSelThreads) kept[top + i] = n + i;
    if (top <= r0) return;
    const int32_t *bt = a.bt + int64_t(b) * a.MBS;
    auto load = [&](int j) -> uint32_t {
        const int phys = __ldg(bt + j / kBlockSize);
        if (phys < 0 || phys >= a.NB) return 0u;  // no such block: below every weight
        return f32_order_key(__ldcg(a.weights + (int64_t(phys) * a.Hkv + kvh) * kBlockSize + j % kBlockSize));
    };
    const bool cached = n <= cap;
    uint32_t lo = 0xffffffffu, hi = 0u;  // of this thread's keys
    auto seen = [&](uint32_t u) {
        lo = min(lo, u);
        hi = max(hi, u);
    };
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
                const uint4 k4 = make_uint4(in ? f32_order_key(v[u].x) : 0u, in ? f32_order_key(v[u].y) : 0u,
                                            in ? f32_order_key(v[u].z) : 0u, in ? f32_order_key(v[u].w) : 0u);
                *reinterpret_cast<uint4 *>(keys + 4 * q) = k4;
                seen(k4.x);
                if (4 * q + 1 < n) seen(k4.y);
                if (4 * q + 2 < n) seen(k4.z);
                if (4 * q + 3 < n) seen(k4.w);
            }
        }
    } else {
        for (int j = tid; j < n; j += kSelThreads) seen(load(j));
    }
    __syncthreads();
    auto keys4 = [&](int j) -> uint4 {
        if (cached) return *reinterpret_cast<const uint4 *>(keys + j);
        return make_uint4(load(j), j + 1 < n ? load(j + 1) : 0u, j + 2 < n ? load(j + 2) : 0u,
                          j + 3 < n ? load(j + 3) : 0u);
    };
    uint32_t thr;
    int keq;
    kth_largest(keys4, n, top, lo, hi, sm, thr, keq);
    emit_selected(keys4, n, thr, keq, sm, [&](int r, int j) {
        if (r >= r0 && r < r1) kept[r] = j;
    });
}

// one CTA per segment: the kept positions
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int cap) {
    pdl_trigger();  // the copy waits for this kernel's end before it reads anything
    pdl_wait();
    select_kept(a, blockIdx.x / a.Hkv, blockIdx.x % a.Hkv, cap, 0, a.budget);
}

// The copy, by a warp: kept tokens i0 .. i0 + CHUNK - 1 (below end) of segment
// (b, kvh). A lane finds one token's rows; then the warp moves them with K and V
// side by side (16 lanes of 16 bytes each, or 8 and two tokens), kMove loads per
// lane in flight.
constexpr int kMove = 8;
template <int D>
constexpr int kMoveChunk = kMove * 16 / (D / 8);  // tokens per warp and turn

template <int D>
__device__ __forceinline__ void move_kept(const EvictArgs &a, int b, int kvh, int i0, int end) {
    constexpr int LR = D / 8;          // lanes per row
    constexpr int TP = 32 / (2 * LR);  // tokens at once
    constexpr int CHUNK = kMove * TP;
    static_assert(CHUNK == kMoveChunk<D>, "");
    const int lane = threadIdx.x & 31, i = i0 + lane;
    const int j = lane < CHUNK && i < end ? __ldcg(a.kept + (int64_t(b) * a.Hkv + kvh) * a.budget + i) : -1;
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
    uint4 v[kMove];
    int64_t y[kMove];
#pragma unroll
    for (int u = 0; u < kMove; ++u) {
        const int t = u * TP + lane / (2 * LR);
        const int64_t x = __shfl_sync(0xffffffffu, from, t);
        y[u] = __shfl_sync(0xffffffffu, to, t);
        if (x >= 0) v[u] = __ldcs(cache + x * LR);
    }
#pragma unroll
    for (int u = 0; u < kMove; ++u)
        if (y[u] >= 0) __stcs(cache + y[u] * LR, v[u]);
}

// Many segments: a warp per chunk. Bound by HBM: every kept row is read and
// written once (263 MB in 47 us, 5.6 TB/s, at 16 sequences of 4096 kept tokens;
// warps of 32 tokens, with fewer CTAs to spread over the SMs, took 2 us longer).
// No early launch of the next kernel: it may read new_lens before it waits.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
    pdl_wait();
    const int per = (a.budget + kMoveChunk<D> - 1) / kMoveChunk<D>;  // warps per segment
    const int64_t warp = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t seg = warp / per;
    if (seg >= int64_t(a.B) * a.Hkv) return;
    move_kept<D>(a, int(seg / a.Hkv), int(seg % a.Hkv), int(warp - seg * per) * kMoveChunk<D>, a.budget);
}

// Few segments: `parts` CTAs per segment, each of which selects (the same, all of
// them at once) and copies its share of the kept tokens.
template <int D>
__global__ void __launch_bounds__(kSelThreads) evict_parts_kernel(const EvictArgs a, int cap, int parts) {
    pdl_wait();
    const int seg = blockIdx.x / parts, part = blockIdx.x % parts, b = seg / a.Hkv, kvh = seg % a.Hkv;
    const int share = ((a.budget + parts - 1) / parts + kMoveChunk<D> - 1) / kMoveChunk<D> * kMoveChunk<D>;
    const int r0 = int(min(int64_t(part) * share, int64_t(a.budget))), r1 = min(r0 + share, a.budget);
    if (r0 >= r1) return;  // fewer chunks than parts (part 0 has some: it writes the length)
    select_kept(a, b, kvh, cap, r0, r1);
    __syncthreads();
    for (int i = r0 + int(threadIdx.x >> 5) * kMoveChunk<D>; i < r1; i += kSelThreads / 32 * kMoveChunk<D>)
        move_kept<D>(a, b, kvh, i, r1);
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

cudaError_t launch_evict(const EvictArgs &a, int head_dim, int sms, cudaStream_t stream) {
    const int64_t longest = int64_t(a.MBS) * kBlockSize;  // a multiple of four
    const int cap = longest < kKeysCap ? int(longest) : kKeysCap;
    const size_t smem = size_t(cap) * 4;
    const int64_t segs = int64_t(a.B) * a.Hkv;
    if (segs * kMinParts <= sms) {
        const auto kernel = head_dim == 128 ? evict_parts_kernel<128> : evict_parts_kernel<64>;
        const cudaError_t e = smem_once(reinterpret_cast<const void *>(kernel), size_t(kKeysCap) * 4);
        if (e != cudaSuccess) return e;
        const int parts = int(sms / segs);
        return launch_pdl(kernel, dim3(unsigned(segs * parts)), dim3(kSelThreads), smem, stream, a, cap, parts);
    }
    cudaError_t e = smem_once(reinterpret_cast<const void *>(evict_select_kernel), size_t(kKeysCap) * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_select_kernel, dim3(unsigned(segs)), dim3(kSelThreads), smem, stream, a, cap);
    if (e != cudaSuccess) return e;
    const int chunk = head_dim == 128 ? kMoveChunk<128> : kMoveChunk<64>;  // kept tokens per warp
    const int64_t warps = segs * ((a.budget + chunk - 1) / chunk);
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
