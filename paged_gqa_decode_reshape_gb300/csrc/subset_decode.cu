// subset_decode.cu -- attention of several query rows per sequence over a
// window and sinks, and over a shared prefix and a sequence's own tokens.
//
// For a query row of sequence b, KV head g and the query heads h of its group
// (z in the log2 domain, z = scale * log2(e) * q_h . K_t):
//   out_h = sum_t 2^(z_t - m) V_t / sum_t 2^(z_t - m),   m = max_t z_t
// over the tokens the row sees. One pass with the running maximum and sum;
// the states of a CTA's warps are merged at the end.
//
// The plain form: one CTA per (query row, KV head), one warp per token, a lane
// per D / 32 dims, everything in fp32.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "subset.h"

namespace pa {
namespace {

constexpr int kWarps = 8;

// what a row sees: prefix tokens [0, np), own tokens [0, s1) and [lo, lim)
struct Seen {
    int seq, group, np, s1, lo, lim;
    __device__ int count() const { return np + s1 + max(lim - lo, 0); }
};

__device__ __forceinline__ Seen row_seen(const SubsetArgs &a, int row) {
    Seen s;
    s.seq = row;
    s.group = -1;
    s.np = 0;
    int back = 0;  // rows of the sequence after this one
    if (a.cu_q) {
        int lo = 0, hi = a.nseq;  // last sequence with cu_q <= row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu_q + mid) <= row) lo = mid; else hi = mid;
        }
        const int c0 = __ldg(a.cu_q + lo), c1 = __ldg(a.cu_q + lo + 1);
        s.seq = (row >= c0 && row < c1) ? lo : -1;
        back = c1 - 1 - row;
    }
    if (s.seq < 0) return s;
    const int ctx = min(max(__ldg(a.ctx + s.seq), 0), a.MBS * kBlockSize);
    s.lim = max(ctx - back, 0);
    s.s1 = min(a.sinks, s.lim);
    s.lo = max(s.s1, a.window >= s.lim ? 0 : s.lim - a.window);
    if (a.pt) {
        int lo = 0, hi = a.ngroups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu_g + mid) <= row) lo = mid; else hi = mid;
        }
        if (row >= __ldg(a.cu_g + lo) && row < __ldg(a.cu_g + lo + 1)) {
            s.group = lo;
            s.np = min(max(__ldg(a.plen + lo), 0), a.PMBS * kBlockSize);
        }
    }
    return s;
}

// physical block of the i-th token the row sees, or -1, and the token's offset in it
__device__ __forceinline__ int64_t block_of(const SubsetArgs &a, const Seen &s, int i, int &off) {
    int phys;
    if (i < s.np) {
        off = i % kBlockSize;
        phys = __ldg(a.pt + int64_t(s.group) * a.PMBS + i / kBlockSize);
    } else {
        i -= s.np;
        const int t = i < s.s1 ? i : i - s.s1 + s.lo;
        off = t % kBlockSize;
        phys = __ldg(a.bt + int64_t(s.seq) * a.MBS + t / kBlockSize);
    }
    return phys >= 0 && phys < a.NB ? phys : -1;
}

template <int D, int V>
__device__ __forceinline__ void load_row(const void *cache, int Hkv, int64_t blk, int off, int kvh, int lane,
                                         float (&x)[V]) {
    const int64_t e = ((blk * kBlockSize + off) * Hkv + kvh) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(uint32_t(static_cast<const uint16_t *>(cache)[e + i]) << 16);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) subset_decode_kernel(const SubsetArgs a) {
    constexpr int V = D / 32;
    __shared__ float sm_acc[kWarps][kMaxGroup][D];
    __shared__ float sm_m[kWarps][kMaxGroup], sm_l[kWarps][kMaxGroup];
    const int row = blockIdx.x, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const Seen s = row_seen(a, row);
    if (s.seq < 0) return;
    const int n = s.count();
    float q[kMaxGroup][V], acc[kMaxGroup][V], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            acc[h][i] = 0.f;
            q[h][i] = h < a.G ? __uint_as_float(uint32_t(a.q[(int64_t(row) * a.Hq + kvh * a.G + h) * D + lane * V + i]) << 16)
                              : 0.f;
        }
    }
    auto logits = [&](int64_t blk, int off, float (&z)[kMaxGroup]) {
        float k[V];
        load_row<D>(a.kc, a.Hkv, blk, off, kvh, lane, k);
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) d = fmaf(q[h][i], k[i], d);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            z[h] = d * a.scale_log2;
        }
    };
    for (int i = warp; i < n; i += kWarps) {
        int off;
        const int64_t blk = block_of(a, s, i, off);
        if (blk < 0) continue;
        float z[kMaxGroup], v[V];
        logits(blk, off, z);
        load_row<D>(a.vc, a.Hkv, blk, off, kvh, lane, v);
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h) {
            const float mn = fmaxf(m[h], z[h]);
            const float al = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn), p = exp2f(z[h] - mn);
            l[h] = l[h] * al + p;
            m[h] = mn;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[h][j] = acc[h][j] * al + p * v[j];
        }
    }
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
#pragma unroll
        for (int j = 0; j < V; ++j) sm_acc[warp][h][lane * V + j] = acc[h][j];
        if (lane == 0) {
            sm_m[warp][h] = m[h];
            sm_l[warp][h] = l[h];
        }
    }
    __syncthreads();
    if (warp < a.G) {
        const int h = warp;
        float Mh = -INFINITY, Lh = 0.f;
        for (int w = 0; w < kWarps; ++w) Mh = fmaxf(Mh, sm_m[w][h]);
        for (int w = 0; w < kWarps; ++w)
            if (sm_m[w][h] != -INFINITY) Lh += sm_l[w][h] * exp2f(sm_m[w][h] - Mh);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float o = 0.f;
            for (int w = 0; w < kWarps; ++w)
                if (sm_m[w][h] != -INFINITY) o += sm_acc[w][h][lane * V + j] * exp2f(sm_m[w][h] - Mh);
            a.out[(int64_t(row) * a.Hq + kvh * a.G + h) * D + lane * V + j] =
                __bfloat16_as_ushort(__float2bfloat16_rn(Lh > 0.f ? o / Lh : 0.f));
        }
    }
}

}  // namespace

cudaError_t launch_subset_decode(const SubsetArgs &a, int head_dim, cudaStream_t stream) {
    const dim3 grid(a.rows, a.Hkv), block(kWarps * 32);
    return head_dim == 128 ? launch_pdl(subset_decode_kernel<128>, grid, block, 0, stream, a)
                           : launch_pdl(subset_decode_kernel<64>, grid, block, 0, stream, a);
}

}  // namespace pa
