// step_plan.cu -- a step's block tables, row offsets, positions and slots built on
// the GPU from request lengths and a stack of free blocks, and blocks given back
// to that stack (sm_103a).
//
// With c = tokens cached and q = tokens to come of sequence b, MBS * BS >= c + q and
// the rows up to its end at most T: its new blocks are numbers rank_b ..
// rank_b + need_b - 1 of the call, need_b = ceil((c + q) / BS) - ceil(c / BS),
// rank_b = sum of the needs before it; block number r is
// free_blocks[num_free - 1 - r]. A sequence whose numbers pass num_free gets none.
#include "common.cuh"
#include "kernels.h"
#include "step.h"
#include "subset.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = kMaxBatch / kPlanThreads;  // sequences of a thread at most

// Inclusive prefix sums over the CTA; `total` gets the sum. sh: 33 words.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *sh, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // sh may still be read from the last scan
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t w = lane < warps ? sh[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        sh[lane] = w;
    }
    __syncthreads();
    total = sh[warps - 1];
    return v + (warp ? sh[warp - 1] : 0);
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
    int32_t *cu = plan_sh, *rank_of = cu + a.B + 1, *pos0 = rank_of + a.B + 1;  // [B + 1], [B + 1], [B]
    __shared__ int64_t scan[33];
    __shared__ unsigned long long most;
    pdl_wait();
    const int tid = threadIdx.x, lim = a.MBS * kBlockSize;
    const int nf = int(min(max(int64_t(__ldg(a.num_free)), int64_t(0)), a.F));
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
    int c[kPlanPer], q[kPlanPer], need[kPlanPer];
    int64_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const bool in = i < per && b0 + i < a.B;
        c[i] = in ? min(max(__ldg(a.ctx + b0 + i), 0), lim) : 0;
        q[i] = in ? max(__ldg(a.q + b0 + i), 0) : 0;
        sum += q[i];
    }
    int64_t end = cta_scan(sum, scan, total) - sum;
    int64_t needs = 0;
    bool fits[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        end += q[i];
        fits[i] = int64_t(c[i]) + q[i] <= lim && end <= a.T;
        need[i] = fits[i] ? (c[i] + q[i] + kBlockSize - 1) / kBlockSize - (c[i] + kBlockSize - 1) / kBlockSize : 0;
        needs += need[i];
        if (i < per && b0 + i < a.B) cu[b0 + i + 1] = int(min(end, int64_t(a.T)));
    }
    if (tid == 0) {
        cu[0] = 0;
        most = 0;
    }
    int64_t rank = cta_scan(needs, scan, total) - needs;
    int64_t taken = 0;  // blocks up to this thread's last sequence that gets its own
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        if (i < per && b0 + i < a.B) {
            const int b = b0 + i;
            const bool ok = fits[i] && (need[i] == 0 || rank + need[i] <= nf);
            const int got = ok ? q[i] : 0;
            if (ok && need[i] > 0) taken = rank + need[i];
            pos0[b] = ok ? c[i] : ~c[i];  // negative: no slots
            rank_of[b + 1] = int(min(rank + need[i], int64_t(nf) + 1));
            a.granted[b] = got;
            a.new_lens[b] = c[i] + got;
            a.cu[b + 1] = cu[b + 1];
        }
        rank += need[i];
    }
    // ranks ascend, so those that get their blocks come first: the highest taken is the sum of all
    if (taken) atomicMax(&most, (unsigned long long)taken);
    if (tid == 0) a.cu[0] = rank_of[0] = 0;
    __syncthreads();
    if (tid == 0) *a.new_free = nf - int(most);
    // new blocks, a warp per sequence
    for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {
        const int r = rank_of[b], n = min(rank_of[b + 1], int(most)) - r, p = pos0[b];
        int32_t *row = a.bt + int64_t(b) * a.MBS + (p + kBlockSize - 1) / kBlockSize;  // n > 0: p >= 0
        for (int j = tid & 31; j < n; j += 32) row[j] = __ldg(a.free_blocks + nf - 1 - r - j);
    }
    __syncthreads();
    if (rows_too)
        write_rows(a, cu, [&](int b) { return pos0[b] < 0 ? ~pos0[b] : pos0[b]; }, [&](int b) { return pos0[b] >= 0; },
                   tid, kPlanThreads);
}

// Positions and slots of many rows, from what plan_kernel wrote.
constexpr int kRowThreads = 256;

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

// Blocks ceil(keep / BS) .. ceil(ctx / BS) - 1 of every sequence, in order, to the stack.
__global__ void __launch_bounds__(kPlanThreads) release_kernel(const ReleaseArgs a) {
    extern __shared__ int64_t upto[];  // [B + 1] blocks that go up to each sequence
    int32_t *from = reinterpret_cast<int32_t *>(upto + a.B + 1);  // [B]
    __shared__ int64_t scan[33];
    pdl_wait();
    const int tid = threadIdx.x, lim = a.MBS * kBlockSize;
    const int nf = int(min(max(int64_t(__ldg(a.num_free)), int64_t(0)), a.F));
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
    int c[kPlanPer], k[kPlanPer];
    int64_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const bool in = i < per && b0 + i < a.B;
        c[i] = in ? min(max(__ldg(a.ctx + b0 + i), 0), lim) : 0;
        k[i] = in ? min(max(__ldg(a.keep + b0 + i), 0), c[i]) : 0;
        sum += (c[i] + kBlockSize - 1) / kBlockSize - (k[i] + kBlockSize - 1) / kBlockSize;
    }
    int64_t end = cta_scan(sum, scan, total) - sum;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        if (i < per && b0 + i < a.B) {
            from[b0 + i] = (k[i] + kBlockSize - 1) / kBlockSize;
            end += (c[i] + kBlockSize - 1) / kBlockSize - from[b0 + i];
            upto[b0 + i + 1] = end;
            a.new_lens[b0 + i] = k[i];
        }
    }
    if (tid == 0) upto[0] = 0;
    __syncthreads();
    int64_t at = nf;  // where the next block goes
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
        int64_t n;
        const int64_t to = at + cta_scan(in ? 1 : 0, scan, n) - 1;
        if (in && to < a.F) a.free_blocks[to] = p;
        at += n;
    }
    if (tid == 0) *a.new_free = int(min(at, a.F));
}

}  // namespace

// Neither kernel lets the next one start early: what they write (lengths, tables, row
// offsets) is what the attention calls read before they wait for their predecessor.
cudaError_t launch_plan(const PlanArgs &a, cudaStream_t stream) {
    const bool rows_too = a.T <= 4 * kPlanThreads;
    const size_t smem = (3 * size_t(a.B) + 2) * 4;
    cudaError_t e = smem_once(reinterpret_cast<const void *>(plan_kernel), (3 * size_t(kMaxBatch) + 2) * 4);
    if (e == cudaSuccess) e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), smem, stream, a, rows_too);
    if (e != cudaSuccess || rows_too) return e;
    const int grid = (a.T + 4 * kRowThreads - 1) / (4 * kRowThreads);
    return launch_pdl(plan_rows_kernel, dim3(unsigned(grid)), dim3(kRowThreads), 0, stream, a);
}

cudaError_t launch_release(const ReleaseArgs &a, cudaStream_t stream) {
    const cudaError_t e = smem_once(reinterpret_cast<const void *>(release_kernel), 12 * size_t(kMaxBatch) + 8);
    if (e != cudaSuccess) return e;
    return launch_pdl(release_kernel, dim3(1), dim3(kPlanThreads), 12 * size_t(a.B) + 8, stream, a);
}

}  // namespace pa
