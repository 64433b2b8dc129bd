// step_plan.cu -- a step's block tables, row offsets, positions and slots built on
// the GPU from request lengths and a stack of free blocks, and blocks given back
// to that stack (sm_103a).
//
// With c = tokens cached and q = tokens to come of sequence b, MBS * BS >= c + q and
// the rows up to its end at most T: its new blocks are numbers rank_b ..
// rank_b + need_b - 1 of the call, need_b = ceil((c + q) / BS) - ceil(c / BS),
// rank_b = sum of the needs before it; block number r is
// free_blocks[num_free - 1 - r]. A sequence whose numbers pass num_free gets none.
//
// Bound by latency: the bytes are few, their reads depend on each other (lengths, prefix sums over the batch, free blocks,
// tables, slots). So one CTA with the sequences in its registers: 16 sequences of a token each 4.1 us, 256 with 9 prompts
// among them 7.0, 64 prompts of 517 to 16000 rows 11.8 (its rows by a second launch). Releases by one CTA or a cluster: the
// rejected tokens of 128 sequences 4.8 us, 81000 blocks of 512 sequences 8.6.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "step.h"
#include "subset.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = kMaxBatch / kPlanThreads;  // sequences of a thread at most
constexpr int kFewBlocks = 4;                       // new blocks of a sequence that its thread writes itself

// A value that the same call may write in its place (context_lens by new_lens, *num_free by *new_free), read exactly
// once and here: a read-only load (__ldg) may only be of what nobody writes while the kernel runs, and the compiler
// may move or repeat it behind the write.
__device__ __forceinline__ int32_t load_once(const int32_t *p) {
    int32_t v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Inclusive prefix sums of two values over the CTA's 1024 threads, the sums of all in `u` and `v`.
struct Pair {
    int64_t u, v;
};
__device__ __forceinline__ Pair cta_scan(Pair x, Pair *sh, Pair &total) {  // sh: 32
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](Pair &y) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, y.u, o), v = __shfl_up_sync(0xffffffffu, y.v, o);
            if (lane >= o) {
                y.u += u;
                y.v += v;
            }
        }
    };
    scan(x);
    __syncthreads();  // sh may still be read from the last scan
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    Pair w = sh[lane];  // by every warp for itself
    scan(w);
    total.u = __shfl_sync(0xffffffffu, w.u, 31);
    total.v = __shfl_sync(0xffffffffu, w.v, 31);
    const int64_t u = __shfl_sync(0xffffffffu, w.u, (warp - 1) & 31), v = __shfl_sync(0xffffffffu, w.v, (warp - 1) & 31);
    if (warp) {
        x.u += u;
        x.v += v;
    }
    return x;
}

// Thread-block clusters: this CTA's rank, their number, a barrier of them all (what was written before it is
// seen after it), and a word of another CTA's shared memory.
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int64_t cluster_read(const int64_t *p, unsigned rank) {
    uint32_t at;
    int64_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}

// Position and slot of the rows r0, r0 + step, ...: cu [B + 1], pos0 [B] the position of a sequence's
// first row, ok [B]: it has its slots. Tables are read past L1: this kernel may have written them.
template <typename Pos0, typename Ok>
__device__ __forceinline__ void write_rows(const PlanArgs &a, const int32_t *cu, Pos0 pos0, Ok ok, int r0, int step) {
    const int rows = cu[a.B];
    for (int r = r0; r < a.T; r += step) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (r < rows) {
            int lo = 0, hi = a.B;  // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= r) lo = mid; else hi = mid;
            }
            pos = pos0(lo) + (r - cu[lo]);
            if (ok(lo)) {
                const int phys = __ldcg(a.bt + int64_t(lo) * a.MBS + pos / kBlockSize);
                if (phys >= 0 && phys < a.NB) slot = int64_t(phys) * kBlockSize + pos % kBlockSize;
            }
        }
        a.pos[r] = pos;
        a.slots[r] = slot;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, bool rows_too) {
    extern __shared__ int32_t plan_sh[];
    int32_t *cu = plan_sh, *pos0 = cu + a.B + 1, *rank_of = pos0 + a.B, *count_of = rank_of + a.B;  // [B + 1], [B] each
    __shared__ Pair scan[32];
    __shared__ int most;
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, lim = a.MBS * kBlockSize;
    const int nf = int(min(max(int64_t(load_once(a.num_free)), int64_t(0)), a.F));
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
    int c[kPlanPer], q[kPlanPer], need[kPlanPer];
    bool fits[kPlanPer];
    Pair sum = {0, 0}, total;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const bool in = i < per && b0 + i < a.B;
        c[i] = in ? min(max(load_once(a.ctx + b0 + i), 0), lim) : 0;
        q[i] = in ? max(__ldg(a.q + b0 + i), 0) : 0;
        fits[i] = int64_t(c[i]) + q[i] <= lim;
        need[i] = fits[i] ? (c[i] + q[i] + kBlockSize - 1) / kBlockSize - (c[i] + kBlockSize - 1) / kBlockSize : 0;
        sum.u += q[i];
        sum.v += need[i];
    }
    if (tid == 0) {
        cu[0] = a.cu[0] = 0;
        most = 0;
    }
    const Pair own = sum;
    Pair upto = cta_scan(sum, scan, total);
    int64_t end = upto.u - own.u, rank = upto.v - own.v;
    if (total.u > a.T) {  // the sequences whose rows end past the last one need no blocks: their ranks once more
        int64_t e = end;
        sum.v = 0;
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            e += q[i];
            fits[i] = fits[i] && e <= a.T;
            if (!fits[i]) need[i] = 0;
            sum.v += need[i];
        }
        const int64_t n = sum.v;
        rank = cta_scan(sum, scan, total).v - n;
    }
    int taken = 0;  // blocks up to this thread's last sequence that gets its own
    bool many = false;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = b0 + i, n = need[i], have = (c[i] + kBlockSize - 1) / kBlockSize;
        const bool in = i < per && b < a.B, ok = fits[i] && (n == 0 || rank + n <= nf);
        if (in) {
            end += q[i];
            if (ok && n > 0) taken = int(rank) + n;
            if (ok && n <= kFewBlocks)
                for (int j = 0; j < n; ++j)
                    a.bt[int64_t(b) * a.MBS + have + j] = __ldg(a.free_blocks + nf - 1 - int(rank) - j);
            pos0[b] = ok ? c[i] : ~c[i];  // negative: no slots
            cu[b + 1] = int(min(end, int64_t(a.T)));
            a.granted[b] = ok ? q[i] : 0;
            a.new_lens[b] = c[i] + (ok ? q[i] : 0);
            a.cu[b + 1] = cu[b + 1];
        }
        if (in) {  // many blocks are written by a warp
            const bool lots = ok && n > kFewBlocks;
            many |= lots;
            rank_of[b] = lots ? int(rank) : -1;
            count_of[b] = n;
        }
        rank += n;
    }
    // ranks ascend, so those that get their blocks come first: the highest taken is the sum of all
    if (taken) atomicMax(&most, taken);
    if (__syncthreads_or(many)) {
        for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {
            const int r = rank_of[b];
            if (r < 0) continue;
            int32_t *row = a.bt + int64_t(b) * a.MBS + (pos0[b] + kBlockSize - 1) / kBlockSize;
            for (int j = lane; j < count_of[b]; j += 32) row[j] = __ldg(a.free_blocks + nf - 1 - r - j);
        }
        __syncthreads();
    }
    if (tid == 0) *a.new_free = nf - most;
    if (rows_too)
        write_rows(a, cu, [&](int b) { return pos0[b] < 0 ? ~pos0[b] : pos0[b]; }, [&](int b) { return pos0[b] >= 0; },
                   tid, kPlanThreads);
}

// Positions and slots of many rows, from what plan_kernel wrote.
constexpr int kRowThreads = 1024;

__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(const PlanArgs a) {
    __shared__ int32_t cu[kMaxBatch + 1];
    pdl_wait();
    for (int i = threadIdx.x; i <= a.B; i += kRowThreads) cu[i] = __ldcg(a.cu + i);
    __syncthreads();
    // a sequence without its slots has none granted; its length is then that of before
    write_rows(a, cu, [&](int b) { return __ldcg(a.new_lens + b) - __ldcg(a.granted + b); },
               [&](int b) { return __ldcg(a.granted + b) > 0; }, blockIdx.x * kRowThreads + threadIdx.x,
               gridDim.x * kRowThreads);
}

// Blocks ceil(keep / BS) .. ceil(ctx / BS) - 1 of every sequence, in order, to the stack, by a cluster of CTAs: a warp
// per sequence looks whether all of them are in the pool, and where that holds for every sequence their places are the
// prefix sums of the lengths, and every warp copies. Otherwise the first CTA goes through the list once more, 1024
// entries at a time, each behind those before it that are in the pool. (81000 blocks of 512 sequences: 8.6 us; that list by
// one CTA for all calls 107.)
__global__ void __launch_bounds__(kPlanThreads) release_kernel(const ReleaseArgs a) {
    extern __shared__ int64_t upto[];  // [B + 1] blocks that go up to each sequence
    int32_t *from = reinterpret_cast<int32_t *>(upto + a.B + 1);  // [B]
    __shared__ Pair scan[32];
    __shared__ int64_t odd;  // an entry that this CTA saw is not in the pool
    const int rank = int(cluster_rank()), ctas = int(cluster_size());
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, lim = a.MBS * kBlockSize;
    const int nf = int(min(max(int64_t(load_once(a.num_free)), int64_t(0)), a.F));
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
    int c[kPlanPer], k[kPlanPer];
    Pair sum = {0, 0}, all;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const bool in = i < per && b0 + i < a.B;
        c[i] = in ? min(max(load_once(a.ctx + b0 + i), 0), lim) : 0;
        k[i] = in ? min(max(__ldg(a.keep + b0 + i), 0), c[i]) : 0;
        sum.u += (c[i] + kBlockSize - 1) / kBlockSize - (k[i] + kBlockSize - 1) / kBlockSize;
    }
    int64_t end = cta_scan(sum, scan, all).u - sum.u;
    const int64_t total = all.u;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        if (i < per && b0 + i < a.B) {
            from[b0 + i] = (k[i] + kBlockSize - 1) / kBlockSize;
            end += (c[i] + kBlockSize - 1) / kBlockSize - from[b0 + i];
            upto[b0 + i + 1] = end;
        }
    }
    if (tid == 0) {
        upto[0] = 0;
        odd = 0;
    }
    __syncthreads();
    constexpr int U = 8;  // entries of a lane in flight
    // every (warp of the cluster)-th sequence: its entries, U at a time, to fn(entries, how many are the sequence's, first)
    auto sequences = [&](auto &&fn) {
        for (int b = rank * (kPlanThreads / 32) + (tid >> 5); b < a.B; b += ctas * (kPlanThreads / 32)) {
            const int n = int(upto[b + 1] - upto[b]);
            const int32_t *row = a.bt + int64_t(b) * a.MBS + from[b];
            for (int j0 = 0; j0 < n; j0 += 32 * U) {
                int p[U];
#pragma unroll
                for (int e = 0; e < U; ++e) p[e] = j0 + 32 * e + lane < n ? __ldg(row + j0 + 32 * e + lane) : 0;
                fn(p, n - j0, nf + upto[b] + j0);
            }
        }
    };
    bool bad = false;
    sequences([&](const int (&p)[U], int, int64_t) {
#pragma unroll
        for (int e = 0; e < U; ++e) bad |= p[e] < 0 || p[e] >= a.NB;
    });
    if (__syncthreads_or(bad) && tid == 0) odd = 1;
    cluster_sync();  // every CTA has read its lengths and the count, too: new_lens and new_free may be the same places
    for (int r = 0; r < ctas; ++r) bad |= cluster_read(&odd, r) != 0;
    bad = __syncthreads_or(bad);
    cluster_sync();  // no CTA is gone while another reads its word
    int64_t to = nf + total;
    if (!bad) {
        sequences([&](const int (&p)[U], int n, int64_t at) {
#pragma unroll
            for (int e = 0; e < U; ++e)
                if (32 * e + lane < n && at + 32 * e + lane < a.F) a.free_blocks[at + 32 * e + lane] = p[e];
        });
    } else if (rank == 0) {
        to = nf;
        for (int64_t i0 = 0; i0 < total; i0 += kPlanThreads) {
            const int64_t i = i0 + tid;
            int p = -1;
            if (i < total) {
                int lo = 0, hi = a.B;  // upto[lo] <= i < upto[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (upto[mid] <= i) lo = mid; else hi = mid;
                }
                p = __ldg(a.bt + int64_t(lo) * a.MBS + from[lo] + int(i - upto[lo]));
            }
            const bool in = p >= 0 && p < a.NB;
            const int64_t put = to + cta_scan(Pair{in, 0}, scan, all).u - 1;
            if (in && put < a.F) a.free_blocks[put] = p;
            to += all.u;
        }
    }
    if (rank != 0) return;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i)
        if (i < per && b0 + i < a.B) a.new_lens[b0 + i] = k[i];
    if (tid == 0) *a.new_free = int(min(to, a.F));
}

}  // namespace

// Neither kernel lets the next one start early: what they write (lengths, tables, row
// offsets) is what the attention calls read before they wait for their predecessor.
//
// Up to kRowsHere rows are written by the planning CTA itself, else by a second launch, which costs the host 2.5 us. Here and
// by a second launch (GPU time): 2031 rows of 250 sequences 5.2 and 6.3 us, 2546 of 256 with 9 prompts 7.0 and 6.3, 3256 of 256
// 4.8 and 5.5.
constexpr int kRowsHere = 4 * kPlanThreads;

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t stream) {
    const bool rows_too = a.T <= kRowsHere;
    const size_t smem = (4 * size_t(a.B) + 1) * 4;
    cudaError_t e = smem_once(reinterpret_cast<const void *>(plan_kernel), (4 * size_t(kMaxBatch) + 1) * 4);
    if (e == cudaSuccess) e = launch_soon(plan_kernel, dim3(1), dim3(kPlanThreads), smem, stream, 1, a, rows_too);
    if (e != cudaSuccess || rows_too) return e;
    const int grid = (a.T + kRowThreads - 1) / kRowThreads;
    return launch_soon(plan_rows_kernel, dim3(unsigned(grid)), dim3(kRowThreads), 0, stream, 1, a);
}

// A warp per sequence: one CTA has 32.
constexpr int kOneCtaSequences = 64;
constexpr unsigned kReleaseCtas = 8;

cudaError_t launch_release(const ReleaseArgs &a, cudaStream_t stream) {
    const cudaError_t e = smem_once(reinterpret_cast<const void *>(release_kernel), 12 * size_t(kMaxBatch) + 8);
    if (e != cudaSuccess) return e;
    const unsigned ctas = a.B <= kOneCtaSequences ? 1 : kReleaseCtas;
    return launch_soon(release_kernel, dim3(ctas), dim3(kPlanThreads), 12 * size_t(a.B) + 8, stream, ctas, a);
}

}  // namespace pa
