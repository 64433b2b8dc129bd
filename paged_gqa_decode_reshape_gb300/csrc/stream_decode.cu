// stream_decode.cu -- one-query-row decode over a part of the cache (sm_103a):
// the sliding window with sinks, the dense decode that also stores its logits
// (for the accumulated weights), short prefixes with the own tokens behind them,
// few query rows per sequence each for itself, and the own tokens of a sequence whose prefix is attended to separately.
//
// For KV head g of sequence b and the query heads h of its group, over the
// tokens t the row sees (z_t = scale * log2(e) * q_h . K_t):
//   out_h = sum_t 2^(z_t - m) V_t / sum_t 2^(z_t - m),   m = max_t z_t.
//
// Bound: every visible K/V byte is read once, at about 2 G flops per byte, so
// HBM bandwidth bounds long calls and latency short ones. Measured (28 / 4 heads
// of 128, all tokens seen): 500 sequences of 2000 tokens 316 us = 6.5 TB/s, 8-bit
// cache 158 us = 6.5 TB/s (161 with a scale per block); 16 of 4096 25.2 us = 5.3 TB/s, of which about 5 us are
// the launch, the lengths, the table and the first copies one after another, and
// the last merges; one of 256 tokens 4.6 us.
//
//  * Work list. A (sequence, KV head) is a segment with one item per two 16-token
//    blocks that hold a visible token (sink blocks, then window blocks; at
//    least one item, so that every output row is written).
//    Up to one segment per SM: every CTA takes one piece of one segment, all
//    pieces at most L items, L the smallest for which the pieces fit the
//    grid. Its warps take the piece's items in turn and merge once.
//    More segments: every warp is a worker of its own. The segments are laid
//    end to end, each with kEndCost empty items after it for what its end
//    costs, and cut into equal ranges, one per warp; no warp waits for
//    another, so many short sequences load the SMs as evenly as a few long.
//  * Each warp is its own producer: its items are copied by TMA (a box per K or V
//    block, 64 dims after 64 dims, 128-byte swizzle; E4M3: a K box and the
//    contiguous V tile) into its private ring of R stages, which only this warp
//    fills and empties.
//  * Math as mma.sync m16n8k16 on S^T = K Q^T and O^T += V^T P^T: tokens (then
//    dims) are the 16 rows, the up to 8 heads of the group the 8 columns, so
//    a K/V byte serves the whole group. tcgen05's smallest M of 64 would be
//    filled, but its results come back through TMEM to warps that would
//    wait for them; at 2 G flops per byte the tensor pipes are nearly idle.
//  * An item (32 tokens) is one copy, one wait and one softmax step. A 16-bit
//    mask per block says which tokens are seen; the V rows of the others (they
//    may hold NaN) are zeroed in the stage, which only edge blocks need.
//  * A segment cut between workers leaves (O, m, l) per piece in the workspace,
//    and the worker that completes its arrival counter merges them (a CTA:
//    each warp every NW-th piece, then the warps), in an order that does not
//    depend on who is last.
//  * Accumulated weights (LOGITS): the logits go to the workspace on the way, and
//    once the normaliser is known p_t = 2^(z_t - lse) is added to the weights, by
//    the CTA that has it or by a second launch. The normaliser sums the fp32 p_t.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "subset.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kPreCap = 512;   // entries of the items-per-sequence prefix in shared memory
// Items that the end of a segment costs a warp (its merge and the next one's query). 128 sequences of 33 to 20011
// tokens in a window of 2048, 8-bit: 2 items 36.7 us, none 45.2, 4 items 35.2; 128 of 1 to 2049 own tokens beside
// their prefixes: 37.0, 46.0 and 39.1.
constexpr int kEndCost = 2;
// Items of a CTA's piece at least, where there are as many; while no segment has
// more than twice that, all stay whole. A cut costs about 1.7 us at the end, an item less per warp
// saves 0.85 us: 16 sequences of 500 tokens take 8.4 us in pieces of 6 and more, 6.5
// whole; one of 2048 tokens 7.5 us in pieces of 12 items, 9.3 of 24, 7.2 of 6; one of
// 8192 tokens 10.4 us, of 24 10.6, of 6 11.0 (28 / 4 heads of 128).
constexpr int kMinPiece = 12;
// Accumulated weights, one piece per CTA: the CTA that has a segment's rows adds
// its weights while the table has at most this many blocks per segment of the
// call; longer ones are added by a launch of their own over the whole grid. One
// CTA's addition takes 0.75 us per 1024 tokens, the launch 3 us or more and 1.6 us
// of the host: one sequence of 2048 tokens 9.8 us fused, 10.3 separate; of 8192
// tokens 16.8 and 13.6; 16 sequences of 8192 tokens 55.0 and 56.5.
constexpr int kFusedAddBlocks = 64;

#ifndef PA_STREAM_WARPS_F8
#define PA_STREAM_WARPS_F8 8
#endif
#ifndef PA_STREAM_STAGES_F8
#define PA_STREAM_STAGES_F8 2
#endif
constexpr int kMaxStreamWarps = 12;

template <int D, CacheKind KIND>
struct StreamCfg {
    static constexpr bool F8 = KIND != kCacheBf16;
    static_assert(!F8 || D == 128, "the E4M3 cache path is for head_dim 128");
    // Warps x stages of 16 KB (bf16) or 8 KB fill the shared memory that the math's latency leaves room for.
    // bf16, 16 sequences of 4096 tokens: 6 x 2 25.4 us, 5 x 2 25.6, 4 x 3 25.9, 3 x 4 28.3 (of 500 tokens 6.3, 7.4,
    // 6.8, 8.7). 8-bit, 128 of 2048: 8 x 2 50.4 us, 10 x 2 53.4 (168 registers, and more pieces to merge), 9 x 2 54.1,
    // 7 x 2 51.4, 5 x 4 63.6 (16 of 4096: 16.7, 17.3, 18.4, 18.8, 22.4).
    static constexpr int NW = F8 ? PA_STREAM_WARPS_F8 : 6;  // warps
    static_assert(NW <= kMaxStreamWarps, "pieces and counters of the workspace");
    static constexpr int KT = kBlockSize * D * (F8 ? 1 : 2);  // bytes of a K (or V) tile of one block
    static constexpr int BLK = 2 * KT;                    // K and V of a block
    static constexpr int STAGE = 2 * BLK;                 // an item: two blocks
    static constexpr int R = F8 ? PA_STREAM_STAGES_F8 : (D == 128 ? 2 : 4);  // stages per warp
    static constexpr int RING = R * STAGE;                // bytes in flight per warp
    static constexpr int NKK = D / 16;
    static constexpr int HALF = kBlockSize * 128;         // bytes of one 64-dim half tile (bf16)
    static constexpr int ROW = D + 4;                     // floats per head row of a warp's state (conflict-free)
    static constexpr int SCR = 8 * ROW;
    static constexpr int PART = 8 * D + 16;               // floats per partial: O[8][D], m[8], l[8]
    static constexpr int THREADS = NW * 32;
    static constexpr size_t off_bars = size_t(NW) * RING;
    static constexpr size_t off_scr = off_bars + size_t(NW) * R * 8;
    static constexpr size_t off_ml = off_scr + size_t(NW) * SCR * 4;
    static constexpr size_t off_flag = off_ml + size_t(NW) * 16 * 4;
    static constexpr size_t off_lse = off_flag + 16;
    static constexpr size_t off_pre = off_lse + kMaxGroup * 4;
    static_assert(off_scr % 16 == 0 && off_ml % 16 == 0 && off_pre % 8 == 0, "vector accesses");
    static constexpr size_t SMEM = 1024 + off_pre + (kPreCap + 1) * 8;
};

// what the streaming kernel is run for
enum StreamMode { kPlain, kLogits, kPrefixed, kRows };

// a sequence's visible tokens [0, s1) and [lo, lim), as items; kPrefixed: the s1
// tokens of its group's prefix (group pg, -1: none), then its own [0, lim);
// kRows: what query row b of a call with several per sequence sees (its sequence
// is pg, -1: none; a.cu_g and a.ngroups are the sequences' row offsets)
struct Span {
    int lim, s1, lo, nb1, jw, nb, n;  // nb1 sink blocks, then blocks jw, jw + 1, ...; nb blocks, n items (at least one)
    int pg;
    __device__ int block(int e) const { return e < nb1 ? e : e - nb1 + jw; }  // logical block of list entry e
};

template <StreamMode MODE>
__device__ __forceinline__ Span span_of(const SubsetArgs &a, int b) {
    Span s;
    s.pg = -1;
    int after = 0;  // kRows: rows of the sequence behind this one
    if constexpr (MODE == kPrefixed || MODE == kRows) {
        int lo = 0, hi = a.ngroups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu_g + mid) <= b) lo = mid; else hi = mid;
        }
        const int end = __ldg(a.cu_g + lo + 1);
        if (b >= __ldg(a.cu_g + lo) && b < end) s.pg = lo;
        after = min(end, a.rows) - 1 - b;
    }
    const int seq = MODE == kRows ? s.pg : b;
    s.lim = seq < 0 ? 0 : max(min(max(__ldg(a.ctx + seq), 0), a.MBS * kBlockSize) - (MODE == kRows ? after : 0), 0);
    if constexpr (MODE == kPrefixed) {
        s.s1 = s.pg < 0 ? 0 : min(max(__ldg(a.plen + s.pg), 0), a.PMBS * kBlockSize);
        s.lo = s.jw = 0;
        s.nb1 = (s.s1 + kBlockSize - 1) / kBlockSize;
    } else {
        s.s1 = min(a.sinks, s.lim);
        s.lo = max(s.s1, a.window >= s.lim ? 0 : s.lim - a.window);
        s.nb1 = (s.s1 + kBlockSize - 1) / kBlockSize;
        s.jw = max(s.lo / kBlockSize, s.nb1);
    }
    s.nb = s.nb1 + max((s.lim + kBlockSize - 1) / kBlockSize - s.jw, 0);
    s.n = max((s.nb + 1) / 2, 1);
    return s;
}

// bits of the offsets t - t0 of tokens t in [a, b)
__device__ __forceinline__ uint32_t bits_between(int a, int b, int t0) {
    const int x = min(max(a - t0, 0), 16), y = min(max(b - t0, 0), 16);
    return y > x ? ((1u << y) - 1u) & ~((1u << x) - 1u) : 0u;
}

// (M, Ls, O) += another part
__device__ __forceinline__ void fold(float &M, float &Ls, float4 &O, float m, float l, float4 v) {
    const float Mn = fmaxf(M, m);
    const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn), w = m == -INFINITY ? 0.f : fast_exp2(m - Mn);
    M = Mn;
    Ls = Ls * f + l * w;
    O = make_float4(O.x * f + v.x * w, O.y * f + v.y * w, O.z * f + v.z * w, O.w * f + v.w * w);
}

// The pieces i0, i0 + by, ... < n of a segment, piece i at slot_of(i), merged by a
// warp: every head's values of two pieces in flight. A lane has the (head,
// four dims) numbers lane + 32 t.
template <int D, typename SlotOf>
__device__ __forceinline__ void merge_pieces(SlotOf slot_of, int G, int i0, int n, int by, float (&M)[D / 16],
                                             float (&Ls)[D / 16], float4 (&O)[D / 16]) {
    constexpr int NT = D / 16;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        M[t] = -INFINITY;
        Ls[t] = 0.f;
        O[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 2
    for (int i = i0; i < n; i += by) {
        const float *ps = slot_of(i);
        float m[NT], l[NT];
        float4 v[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int idx = lane + 32 * t, h = min(idx / (D / 4), G - 1);
            m[t] = __ldcg(ps + 8 * D + h);
            l[t] = __ldcg(ps + 8 * D + 8 + h);
            v[t] = __ldcg(reinterpret_cast<const float4 *>(ps + h * D) + idx % (D / 4));
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) fold(M[t], Ls[t], O[t], m[t], l[t], v[t]);
    }
}

// Accumulated weights: p_t = 2^(z_t - lse) summed over the group, added to the
// cache's weights for the tokens t < lim of one segment; ls: the heads' lse
// (infinite: no head). Four tokens of a block per turn, their logits of every
// head in flight (they come from L2, mostly), U turns at a time.
constexpr int kAddThreads = 256;

template <int U>
__device__ __forceinline__ void add_weights(const SubsetArgs &a, int b, int kvh, int lim, const float (&ls)[kMaxGroup],
                                            int i0, int step) {
    constexpr int QB = kBlockSize / 4;  // turns per block
    const int nq = (lim + 3) / 4;
    const int32_t *bt = a.bt + int64_t(b) * a.MBS;
    const float *seg = a.logits + (int64_t(b) * a.Hkv + kvh) * a.MBS * (a.G * kBlockSize);
    for (; i0 < nq; i0 += U * step) {
        int phys[U];
        float4 z[U][kMaxGroup];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * step, nq - 1), j = i / QB;
            phys[u] = __ldg(bt + j);
            const float *p = seg + int64_t(j) * (a.G * kBlockSize) + 4 * (i % QB);
#pragma unroll
            for (int h = 0; h < kMaxGroup; ++h)
                z[u][h] = h < a.G ? __ldcg(reinterpret_cast<const float4 *>(p + h * kBlockSize))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            if (i >= nq || phys[u] < 0 || int64_t(phys[u]) >= a.NB) continue;
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int h = 0; h < kMaxGroup; ++h) {  // 0 for h >= G, and for unseen tokens (logit -inf)
                w.x += fast_exp2(z[u][h].x - ls[h]);
                w.y += fast_exp2(z[u][h].y - ls[h]);
                w.z += fast_exp2(z[u][h].z - ls[h]);
                w.w += fast_exp2(z[u][h].w - ls[h]);
            }
            // tokens past the context get nothing (their weights may hold anything); a block of one sequence
            // gets one addition: the same bits every time
            float *dst = a.weights + (int64_t(phys[u]) * a.Hkv + kvh) * kBlockSize + 4 * (i % QB);
            const int left = lim - 4 * i;
            if (left >= 4) {
                atomicAdd(reinterpret_cast<float4 *>(dst), w);
            } else {
                atomicAdd(dst, w.x);
                if (left > 1) atomicAdd(dst + 1, w.y);
                if (left > 2) atomicAdd(dst + 2, w.z);
            }
        }
    }
}

template <int D, CacheKind KIND, StreamMode MODE>
__global__ void __launch_bounds__(StreamCfg<D, KIND>::THREADS, 1)
    stream_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const SubsetArgs a) {
    using C = StreamCfg<D, KIND>;
    constexpr int NW = C::NW, R = C::R, NKK = C::NKK, BS = kBlockSize;
    constexpr bool F8 = C::F8, PSC = KIND == kCacheE4m3Block, LOGITS = MODE == kLogits;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *bp = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = a.Hkv, G = a.G;
    float *scr = reinterpret_cast<float *>(bp + C::off_scr);
    float *sm_ml = reinterpret_cast<float *>(bp + C::off_ml);  // [NW][16]: m[8], l[8]
    volatile int *flag = reinterpret_cast<volatile int *>(bp + C::off_flag);
    float *sm_lse = reinterpret_cast<float *>(bp + C::off_lse);
    int64_t *pre = reinterpret_cast<int64_t *>(bp + C::off_pre);
    const uint32_t ring = base + uint32_t(warp) * C::RING;
    const uint32_t bars = base + uint32_t(C::off_bars) + uint32_t(warp) * R * 8;

    pdl_trigger();
    if (tid == 0) {
        prefetch_tensormap(&tm_k);
        if (!F8) prefetch_tensormap(&tm_v);
    }
    if (lane == 0) {
        for (int s = 0; s < R; ++s) mbar_init(bars + s * 8, 1);
        fence_barrier_init();
    }
    // ---- what this warp works on: items [first, last) in steps of `step`, of one segment
    // (item numbers in it) or of the concatenated segments (positions)
    const bool one = int64_t(a.nseq) * Hkv <= gridDim.x;  // a piece of one segment per CTA
    int64_t first, last, L = 1;
    int np = 0, str = 1;
    int b = 0, kvh = 0, piece = 0, npieces = 1, w0 = 0;  // one: the segment, this CTA's piece, the segment's first CTA
    Span sp;
    if (one) {
        int *cnt = reinterpret_cast<int *>(pre);  // items, then pieces per sequence and their prefix
        int *found = reinterpret_cast<int *>(sm_ml);
        int nmax = 0;
        for (int i = tid; i < a.nseq; i += C::THREADS) cnt[i + 1] = span_of<MODE>(a, i).n;
        __syncthreads();
        int64_t sum = 0;
        for (int i = lane; i < a.nseq; i += 32) {
            sum += cnt[i + 1];
            nmax = max(nmax, cnt[i + 1]);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            nmax = max(nmax, __shfl_xor_sync(0xffffffffu, nmax, o));
        }
        // smallest piece size for which Hkv * sum ceil(n / size) <= CTAs, by NW warps at a time
        int lo = nmax > 2 * kMinPiece ? int(min(max((sum * Hkv + gridDim.x - 1) / gridDim.x, int64_t(kMinPiece)), int64_t(nmax)))
                                      : nmax;
        int hi = nmax;  // always fits: one piece per segment
        while (lo < hi) {
            const int at = min(lo + int((int64_t(hi) - lo) * warp / NW), hi);
            int c = 0;
            for (int i = lane; i < a.nseq; i += 32) c += (cnt[i + 1] + at - 1) / at;
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) found[warp] = int64_t(c) * Hkv <= gridDim.x ? at : -1;
            __syncthreads();
            int nlo = lo + 1, nhi = hi;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const int f = found[w], fat = min(lo + int((int64_t(hi) - lo) * w / NW), hi);
                if (f < 0) nlo = max(nlo, fat + 1);
                else nhi = min(nhi, f);
            }
            __syncthreads();
            if (nhi == lo) nlo = lo;
            lo = min(nlo, nhi);
            hi = nhi;
        }
        if (warp == 0) {
            int carry = 0;
            for (int i0 = 0; i0 < a.nseq; i0 += 32) {
                int v = i0 + lane < a.nseq ? (cnt[i0 + lane + 1] + hi - 1) / hi : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += u;
                }
                if (i0 + lane < a.nseq) cnt[i0 + lane + 1] = carry + v;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) cnt[0] = 0;
        }
        __syncthreads();
        if (int(blockIdx.x) >= Hkv * cnt[a.nseq]) return;  // whole CTA: nothing to do
        int x = 0, y = a.nseq;
        while (y - x > 1) {
            const int mid = (x + y) >> 1;
            if (Hkv * cnt[mid] <= int(blockIdx.x)) x = mid; else y = mid;
        }
        b = x;
        npieces = cnt[b + 1] - cnt[b];
        const int rem = int(blockIdx.x) - Hkv * cnt[b];
        kvh = rem / npieces;
        piece = rem - kvh * npieces;
        w0 = int(blockIdx.x) - piece;
        sp = span_of<MODE>(a, b);
        first = int64_t(sp.n) * piece / npieces + warp;
        last = int64_t(sp.n) * (piece + 1) / npieces;
    } else {
        // items (and end costs) of groups of `str` sequences, and their prefix sums
        str = (a.nseq + kPreCap - 1) / kPreCap;
        np = (a.nseq + str - 1) / str;
        for (int i = tid; i < np; i += C::THREADS) {
            int64_t n = 0;
            for (int j = i * str; j < min((i + 1) * str, a.nseq); ++j) n += span_of<MODE>(a, j).n + kEndCost;
            pre[i + 1] = n;
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
        if (warp == 0) {
            int64_t carry = 0;
            for (int i0 = 0; i0 < np; i0 += 32) {
                int64_t v = i0 + lane < np ? pre[i0 + lane + 1] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += u;
                }
                if (i0 + lane < np) pre[i0 + lane + 1] = carry + v;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
        }
        __syncthreads();
        const int64_t total = int64_t(Hkv) * pre[np];
        const int workers = int(gridDim.x) * NW, me = warp * int(gridDim.x) + int(blockIdx.x);
        L = (total + workers - 1) / workers;
        first = me * L;
        last = min(total, first + L);
        if (first >= last) return;  // nothing to do (no barrier of the whole CTA follows)
    }
    const int step_ = one ? NW : 1;

    // the sequence of position p, and p's offset inside its items
    auto locate = [&](int64_t p, Span &s, int64_t &rem) -> int {
        int lo = 0, hi = np;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (int64_t(Hkv) * pre[mid] <= p) lo = mid; else hi = mid;
        }
        int q = lo * str;
        rem = p - int64_t(Hkv) * pre[lo];
        s = span_of<MODE>(a, q);
        while (rem >= int64_t(Hkv) * (s.n + kEndCost) && q + 1 < a.nseq) {
            rem -= int64_t(Hkv) * (s.n + kEndCost);
            s = span_of<MODE>(a, ++q);
        }
        return q;
    };

    // ---- a window of 32 of this warp's items, one per lane
    struct Win {
        int p0, p1;       // physical blocks, or -1: nothing to read
        uint32_t mask;    // their token masks
        int head;         // KV head
        int j;            // first logical block (LOGITS: the second is the next one)
        float4 sc;        // K and V scales of the blocks (per-block scales)
    };
    const int kn = last > first ? int((last - first + step_ - 1) / step_) : 0;  // this warp's items
    auto resolve = [&](int k0) -> Win {
        Win w{-1, -1, 0u, 0, 0, make_float4(0.f, 0.f, 0.f, 0.f)};
        const int k = k0 + lane;
        if (k >= kn) return w;
        const int64_t p = first + int64_t(step_) * k;
        Span s = sp;
        int q = b, e = 2 * int(p);
        w.head = kvh;
        if (!one) {
            int64_t rem;
            q = locate(p, s, rem);
            w.head = int(rem / (s.n + kEndCost));
            e = 2 * int(rem - int64_t(w.head) * (s.n + kEndCost));
        }
        // physical block and token mask of list entry e
        auto entry = [&](int e, int &phys, uint32_t &mask) {
            const int j = s.block(e), t = j * BS;
            if (MODE == kPrefixed && e < s.nb1) {
                phys = __ldg(a.pt + int64_t(s.pg) * a.PMBS + e);
                mask = bits_between(0, s.s1, t);
            } else {
                phys = e < s.nb ? __ldg(a.bt + int64_t(MODE == kRows ? s.pg : q) * a.MBS + j) : -1;
                mask = (MODE == kPrefixed ? 0u : bits_between(0, s.s1, t)) | bits_between(s.lo, s.lim, t);
            }
        };
        int ph0, ph1;
        uint32_t m0, m1;
        entry(e, ph0, m0);
        entry(e + 1, ph1, m1);
        w.j = s.block(e);
        if (ph0 >= 0 && int64_t(ph0) < a.NB) {
            w.p0 = ph0;
            w.mask = m0;
        }
        if (ph1 >= 0 && int64_t(ph1) < a.NB) {
            w.p1 = ph1;
            w.mask |= m1 << 16;
        }
        return w;
    };
    auto scales = [&](Win &w) {
        if constexpr (PSC) {
            const int64_t i0 = int64_t(max(w.p0, 0)) * Hkv + w.head, i1 = int64_t(max(w.p1, 0)) * Hkv + w.head;
            w.sc = make_float4(__ldg(a.k_scale + i0), __ldg(a.v_scale + i0), __ldg(a.k_scale + i1), __ldg(a.v_scale + i1));
        }
    };
    // beside the row-tile kernel: what came before that is complete already, and nothing of its
    // results is read here
    if (!a.ownres) pdl_wait();
    Win cur = resolve(0), nxt = resolve(32);
    scales(cur);
    scales(nxt);
    int wbase = 0;        // first item of cur
    uint32_t armed = 0;   // bit s: parity of the fills of stage s so far
    uint32_t phase = 0;   // bit s: parity of the fill of stage s that is waited for next
    bool dead = false;    // a wait gave up: no further copies or waits
    const uint64_t policy = l2_policy_evict_first();
    // start the copy of item i (i < kn, in cur or nxt) into its stage
    auto issue = [&](int i) {
        const bool c = i < wbase + 32;
        const int p0 = __shfl_sync(0xffffffffu, c ? cur.p0 : nxt.p0, i & 31);
        const int p1 = __shfl_sync(0xffffffffu, c ? cur.p1 : nxt.p1, i & 31);
        const int head = __shfl_sync(0xffffffffu, c ? cur.head : nxt.head, i & 31);
        if ((p0 < 0 && p1 < 0) || dead || i >= a.stop_item) return;
        const uint32_t st = uint32_t(i) % R;
        armed ^= 1u << st;
        const uint32_t fb = bars + st * 8;
        if (lane == 0) mbar_arrive_expect_tx(fb, (p0 >= 0 ? C::BLK : 0) + (p1 >= 0 ? C::BLK : 0));
        __syncwarp();
        // one lane per copy: K and V of the first block, K and V of the second
        const int phys = lane >> 1 ? p1 : p0, part = lane & 1;
        if (lane < 4 && phys >= 0) {
            const uint32_t dst = ring + st * C::STAGE + (lane >> 1) * C::BLK + part * C::KT;
            if constexpr (!F8)
                tma_load_5d(dst, part ? &tm_v : &tm_k, fb, 0, 0, 0, head, phys, policy);
            else if (part)
                bulk_load_1d(dst, static_cast<const uint8_t *>(a.vc) + (int64_t(phys) * Hkv + head) * C::KT, C::KT, fb,
                             policy);
            else
                tma_load_4d(dst, &tm_k, fb, 0, head, 0, phys, policy);
        }
    };

    const int g = lane >> 2, q4 = lane & 3;
    float scale_log2 = a.scale_log2, vref = 0.f;  // as in the dense decode: acc holds O / vref (E4M3)
    uint32_t qb[NKK][2];
    uint2 qn[NKK];  // the next segment's query, on its way
    float acc[NKK][4], m0, m1, l0, l1;
    auto fetch_q = [&](int b, int kvh) {
        const uint32_t *row = reinterpret_cast<const uint32_t *>(a.q + (int64_t(b) * a.Hq + kvh * G + (g < G ? g : 0)) * D);
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
            if constexpr (F8) qn[kk] = __ldg(reinterpret_cast<const uint2 *>(row + 8 * kk + 2 * q4));
            else qn[kk] = make_uint2(__ldg(row + 8 * kk + q4), __ldg(row + 8 * kk + 4 + q4));
        }
    };
    auto begin_segment = [&](int kvh) {
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
            const uint2 v = g < G ? qn[kk] : make_uint2(0u, 0u);
            qb[kk][0] = F8 ? pack_f16x2(bf16_lo(v.x), bf16_hi(v.x)) : v.x;
            qb[kk][1] = F8 ? pack_f16x2(bf16_lo(v.y), bf16_hi(v.y)) : v.y;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[kk][e] = 0.f;
        }
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        if constexpr (KIND == kCacheE4m3) {
            scale_log2 = a.scale_log2 * __ldg(a.k_scale + kvh);
            vref = __ldg(a.v_scale + kvh);
        }
        if constexpr (PSC) vref = 0.f;
    };
    // S^T = K Q^T for the 16 tokens of a staged block
    auto qk = [&](uint32_t kb, float (&sc)[4]) {
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        const int rk = (lane & 7) + (((lane >> 3) & 1) << 3);
        if constexpr (F8) {
            // four codes per lane and 16-byte chunk: k = 2 q4 + e stands for dim 4 q4 + e, k = 2 q4 + 8 + e
            // for dim 4 q4 + 2 + e (the query fragments are in the same order)
#pragma unroll
            for (int c2 = 0; c2 < NKK / 2; ++c2) {
                const int ch = 2 * c2 + (lane >> 4);
                uint32_t r0, r1, r2, r3, l0_, h0_, l1_, h1_, l2_, h2_, l3_, h3_;
                ldsm_x4(kb + rk * 128 + ((ch ^ (lane & 7)) << 4), r0, r1, r2, r3);
                e4m3x4_to_f16x2x2(r0, l0_, h0_);
                e4m3x4_to_f16x2x2(r1, l1_, h1_);
                e4m3x4_to_f16x2x2(r2, l2_, h2_);
                e4m3x4_to_f16x2x2(r3, l3_, h3_);
                mma_f16(sa, l0_, l1_, h0_, h1_, qb[2 * c2][0], qb[2 * c2][1]);
                mma_f16(sb, l2_, l3_, h2_, h3_, qb[2 * c2 + 1][0], qb[2 * c2 + 1][1]);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < NKK; ++kk) {
                const int ch = ((kk & 3) << 1) + (lane >> 4);
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kb + (kk >> 2) * C::HALF + rk * 128 + ((ch ^ (lane & 7)) << 4), a0, a1, a2, a3);
                if (kk & 1) mma_bf16(sb, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
                else mma_bf16(sa, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] = sa[e] + sb[e];
    };
    // zero the staged V rows of the tokens not in mask
    auto hide = [&](uint32_t vb, uint32_t mask) {
        uint8_t *v = bp + (vb - base);
        if constexpr (F8) {  // a row of 16 tokens per dim: word w holds tokens 2w, 2w + 1, 2w + 8, 2w + 9
            uint32_t keep[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t t = mask >> (2 * w);
                keep[w] = (t & 1u ? 0xffu : 0u) | (t & 2u ? 0xff00u : 0u) | (t & 0x100u ? 0xff0000u : 0u) |
                          (t & 0x200u ? 0xff000000u : 0u);
            }
            for (int d = lane; d < D; d += 32) {
                uint4 *r = reinterpret_cast<uint4 *>(v + d * 16);
                const uint4 x = *r;
                *r = make_uint4(x.x & keep[0], x.y & keep[1], x.z & keep[2], x.w & keep[3]);
            }
        } else {
            for (int i = lane; i < BS * D / 8; i += 32)
                if (!((mask >> (i / 8 % BS)) & 1u))
                    *reinterpret_cast<uint4 *>(v + (i / (8 * BS)) * C::HALF + (i % (8 * BS)) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();  // the stage is filled again by a copy
        __syncwarp();
    };
    // O^T += V^T P^T for a staged block
    auto pv = [&](uint32_t vb, uint32_t p01, uint32_t p23) {
        const uint32_t pb0 = movmatrix_trans(p01), pb1 = movmatrix_trans(p23);
        if constexpr (F8) {
#pragma unroll
            for (int c2 = 0; c2 < NKK / 2; ++c2) {
                uint32_t r0, r1, r2, r3, a0, a1, a2, a3, b0, b1, b2, b3;
                ldsm_x4(vb + (32 * c2 + lane) * 16, r0, r1, r2, r3);
                e4m3x4_to_f16x2x2(r0, a0, a2);
                e4m3x4_to_f16x2x2(r1, a1, a3);
                e4m3x4_to_f16x2x2(r2, b0, b2);
                e4m3x4_to_f16x2x2(r3, b1, b3);
                mma_f16(acc[2 * c2], a0, a1, a2, a3, pb0, pb1);
                mma_f16(acc[2 * c2 + 1], b0, b1, b2, b3, pb0, pb1);
            }
        } else {
            const int rv = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int mt = 0; mt < NKK; ++mt) {
                const int ch = ((mt & 3) << 1) + ((lane >> 3) & 1);
                uint32_t a0, a1, a2, a3;
                ldsm_x4_trans(vb + (mt >> 2) * C::HALF + rv * 128 + ((ch ^ (lane & 7)) << 4), a0, a1, a2, a3);
                mma_bf16(acc[mt], a0, a1, a2, a3, pb0, pb1);
            }
        }
    };
    // one online-softmax step over the item's two staged blocks (mask 0: none);
    // ca, cb: their K and V scales (per-block scales)
    auto step = [&](uint32_t s0a, uint32_t ma, float2 ca, uint32_t mb, float2 cb, float *la, float *lb) {
        const uint32_t s1a = s0a + C::BLK;
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
        if (ma) qk(s0a, s0);
        if (mb) qk(s1a, s1);
        float sla = scale_log2, slb = scale_log2, vr = 1.f, ra = 1.f, rb = 1.f;
        if constexpr (PSC) {
            // acc is in units of vref, the largest V scale so far; a block's P
            // enters times its scale over vref (powers of two: exact down to
            // the f16 subnormals)
            sla *= ca.x;
            slb *= cb.x;
            float vnew = vref;
            if (ma) vnew = fmaxf(vnew, ca.y);
            if (mb) vnew = fmaxf(vnew, cb.y);
            // a block never written has scale 0 and holds zeros
            const float rv = vnew > 0.f ? rcp_pow2(vnew) : 0.f;
            vr = vref * rv;
            if (vref == vnew) vr = 1.f;
            vref = vnew;
            ra = ca.y * rv;
            rb = cb.y * rv;
        }
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = e < 2 ? g : g + 8;
            x[e] = (ma >> t) & 1u ? s0[e] * sla : -INFINITY;
            y[e] = (mb >> t) & 1u ? s1[e] * slb : -INFINITY;
        }
        if constexpr (LOGITS) {  // [G][16] per block: heads 2 q4, 2 q4 + 1 of tokens g, g + 8
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int h = 2 * q4 + (e & 1), t = e < 2 ? g : g + 8;
                if (h < G && ma) __stcg(la + h * BS + t, x[e]);
                if (h < G && mb) __stcg(lb + h * BS + t, y[e]);
            }
        }
        float bm0 = fmaxf(fmaxf(x[0], x[2]), fmaxf(y[0], y[2]));
        float bm1 = fmaxf(fmaxf(x[1], x[3]), fmaxf(y[1], y[3]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            bm0 = fmaxf(bm0, __shfl_xor_sync(0xffffffffu, bm0, o));
            bm1 = fmaxf(bm1, __shfl_xor_sync(0xffffffffu, bm1, o));
        }
        const float mn0 = fmaxf(m0, bm0), mn1 = fmaxf(m1, bm1);
        const float r0 = mn0 == -INFINITY ? 0.f : mn0, r1 = mn1 == -INFINITY ? 0.f : mn1;
        const bool grow = mn0 != m0 || mn1 != m1;
        float al0 = fast_exp2(m0 - r0), al1 = fast_exp2(m1 - r1);
        m0 = mn0;
        m1 = mn1;
        float p[4], q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = fast_exp2(x[e] - (e & 1 ? r1 : r0));
            q[e] = fast_exp2(y[e] - (e & 1 ? r1 : r0));
        }
        // P meets V as bf16 (f16 with E4M3 values): off by at most 2^-8 (2^-11) of each weight, as in the dense decode
        auto pk = [](float lo, float hi) { return F8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi); };
        const uint32_t p01 = pk(p[0], p[1]), p23 = pk(p[2], p[3]), q01 = pk(q[0], q[1]), q23 = pk(q[2], q[3]);
        if constexpr (!LOGITS) {
            // the normaliser sums the values that meet V, so a constant V comes out exactly
            auto lo = [](uint32_t v) { return F8 ? f16_lo(v) : bf16_lo(v); };
            auto hi = [](uint32_t v) { return F8 ? f16_hi(v) : bf16_hi(v); };
            p[0] = lo(p01), p[1] = hi(p01), p[2] = lo(p23), p[3] = hi(p23);
            q[0] = lo(q01), q[1] = hi(q01), q[2] = lo(q23), q[3] = hi(q23);
        }  // LOGITS: the weights are fp32, so is their normaliser
        l0 = l0 * al0 + ((p[0] + p[2]) + (q[0] + q[2]));
        l1 = l1 * al1 + ((p[1] + p[3]) + (q[1] + q[3]));
        if (PSC) {
            al0 *= vr;
            al1 *= vr;
        }
        if (__any_sync(0xffffffffu, grow) || (PSC && vr != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < NKK; ++mt) {
                acc[mt][0] *= al0;
                acc[mt][1] *= al1;
                acc[mt][2] *= al0;
                acc[mt][3] *= al1;
            }
        }
        if (ma) {
            if (ma != 0xffffu) hide(s0a + C::KT, ma);
            pv(s0a + C::KT, PSC ? scale_f16x2(p01, ra) : p01, PSC ? scale_f16x2(p23, ra) : p23);
        }
        if (mb) {
            if (mb != 0xffffu) hide(s1a + C::KT, mb);
            pv(s1a + C::KT, PSC ? scale_f16x2(q01, rb) : q01, PSC ? scale_f16x2(q23, rb) : q23);
        }
    };

    // the finished row: O relative to the maximum M with normaliser Ls, head h, dims d .. d + 3
    auto emit = [&](int b, int kvh, int h, int d, float M, float Ls, float4 O) {
        if (a.ownres) {  // the own part of a row with a prefix
            const int64_t r = int64_t(b) * a.Hq + kvh * G + h;
            __stcg(reinterpret_cast<float4 *>(a.ownres + r * D + d), O);
            if (d == 0) __stcg(reinterpret_cast<float2 *>(a.ownml) + r, make_float2(M, Ls));
            return;
        }
        // rows of no sequence stay as they are
        if (MODE == kRows && (b < __ldg(a.cu_g) || b >= __ldg(a.cu_g + a.ngroups))) return;
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
        const int64_t row = int64_t(b) * a.Hq + kvh * G + h;
        *reinterpret_cast<uint2 *>(a.out + row * D + d) =
            make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
        // a row without tokens: every weight 2^(z - inf) = 0 (it has none)
        if (LOGITS && d == 0) {
            const float lse = Ls == 0.f ? INFINITY : M + log2f(Ls);
            if (a.fused_add) sm_lse[h] = lse;
            else a.lse[row] = lse;
        }
    };

    auto wait_item = [&](int k) {
        const uint32_t st = uint32_t(k) % R;
        if (!dead && !mbar_wait_bounded(bars + st * 8, (phase >> st) & 1u, a.wait_ns)) {
            dead = true;
            if (lane == 0) atomicOr(a.status, kStatusTimeout);
        }
        dead = __any_sync(0xffffffffu, dead);
        phase ^= 1u << st;
    };

    int issued = min(kn, R);
    for (int i = 0; i < issued; ++i) issue(i);
    int k = 0;
    // item k is in cur; the items up to k + R are in cur or nxt
    auto shift_windows = [&]() {
        if (k < wbase + 32) return;
        cur = nxt;
        wbase += 32;
        nxt = resolve(wbase + 32);
        scales(nxt);
    };
    // the items k < k1 of segment (cb, ckvh)
    auto stream = [&](int k1, int cb, int ckvh) {
        while (k < k1) {
            shift_windows();
            const uint32_t mask = __shfl_sync(0xffffffffu, cur.mask, k & 31);
            const uint32_t ma = mask & 0xffffu, mb = mask >> 16;
            float2 ca{0.f, 0.f}, cbk{0.f, 0.f};
            if constexpr (PSC) {
                ca = make_float2(__shfl_sync(0xffffffffu, cur.sc.x, k & 31), __shfl_sync(0xffffffffu, cur.sc.y, k & 31));
                cbk = make_float2(__shfl_sync(0xffffffffu, cur.sc.z, k & 31), __shfl_sync(0xffffffffu, cur.sc.w, k & 31));
            }
            float *la = nullptr, *lb = nullptr;
            if constexpr (LOGITS) {
                const int j = __shfl_sync(0xffffffffu, cur.j, k & 31);
                la = a.logits + ((int64_t(cb) * Hkv + ckvh) * a.MBS + j) * (G * BS);
                lb = la + G * BS;
            }
            if (mask) {
                wait_item(k);
                if (!dead) step(ring + uint32_t(k % R) * C::STAGE, ma, ca, mb, cbk, la, lb);
                __syncwarp();  // every lane has read the stage
            }
            ++k;
            if (issued < kn && issued < k + R) issue(issued++);
        }
    };
    // this warp's state into its shared-memory slot
    auto deposit = [&]() {
        l0 += __shfl_xor_sync(0xffffffffu, l0, 4);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 8);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 16);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 4);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 8);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 16);
        float *my = scr + warp * C::SCR;
        const float un = F8 ? vref : 1.f;
#pragma unroll
        for (int mt = 0; mt < NKK; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                my[(2 * q4 + (e & 1)) * C::ROW + 16 * mt + g + (e < 2 ? 0 : 8)] = acc[mt][e] * un;
        if (g == 0) {
            sm_ml[warp * 16 + 2 * q4] = m0;
            sm_ml[warp * 16 + 2 * q4 + 1] = m1;
            sm_ml[warp * 16 + 8 + 2 * q4] = l0;
            sm_ml[warp * 16 + 8 + 2 * q4 + 1] = l1;
        }
    };
    auto put_piece = [&](float *ps, int h, int d, float M, float Ls, float4 O) {
        __stcg(reinterpret_cast<float4 *>(ps + h * D + d), O);
        if (d == 0) {
            __stcg(ps + 8 * D + h, M);
            __stcg(ps + 8 * D + 8 + h, Ls);
        }
    };
    constexpr int NT = D / 16;  // (head, four dims) per lane of a warp
    const int tasks = G * (D / 4);

    if (one) {
        // ---- one piece per CTA: stream it, merge the warps' states once
        fetch_q(b, kvh);
        begin_segment(kvh);
        stream(kn, b, kvh);
        deposit();
        __syncthreads();
        // the warps' states joined: the row, or this CTA's piece of it
        float *slot = a.part + int64_t(blockIdx.x) * C::PART;
        auto join_warps = [&](bool row) {
            for (int idx = tid; idx < tasks; idx += C::THREADS) {
                const int h = idx / (D / 4), d = 4 * (idx % (D / 4));
                float M = -INFINITY, Ls = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    fold(M, Ls, O, sm_ml[w * 16 + h], sm_ml[w * 16 + 8 + h],
                         *reinterpret_cast<const float4 *>(scr + w * C::SCR + h * C::ROW + d));
                if (row) emit(b, kvh, h, d, M, Ls, O);
                else put_piece(slot, h, d, M, Ls, O);
            }
        };
        join_warps(npieces == 1);
        if (npieces > 1) {
            __syncthreads();  // the CTA's piece, published by the release below
            if (tid == 0) *flag = atomic_add_acq_rel_gpu(a.counters + w0, 1) == npieces - 1;
            __syncthreads();
            if (*flag) {
                // every warp takes each NW-th piece, so that many pieces cost few rounds of loads
                float M[NT], Ls[NT];
                float4 O[NT];
                merge_pieces<D>([&](int i) { return a.part + int64_t(w0 + i) * C::PART; }, G, warp, npieces, NW, M, Ls, O);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int idx = lane + 32 * t, h = idx / (D / 4), d = 4 * (idx % (D / 4));
                    if (idx >= tasks) continue;
                    *reinterpret_cast<float4 *>(scr + warp * C::SCR + h * C::ROW + d) = O[t];
                    if (d == 0) {
                        sm_ml[warp * 16 + h] = M[t];
                        sm_ml[warp * 16 + 8 + h] = Ls[t];
                    }
                }
                __syncthreads();
                join_warps(true);
                if (tid == 0) a.counters[w0] = 0;
            }
        }
        if (LOGITS && a.fused_add && (npieces == 1 || *flag)) {
            // the CTA that has the rows has their normalisers; every logit of the segment is published
            __syncthreads();
            float ls[kMaxGroup];
#pragma unroll
            for (int h = 0; h < kMaxGroup; ++h) ls[h] = h < G ? sm_lse[h] : INFINITY;
            add_weights<2>(a, b, kvh, sp.lim, ls, tid, C::THREADS);
        }
    } else {
        // ---- the segments of this warp's range
        int64_t rem;
        b = locate(first, sp, rem);
        kvh = int(rem / (sp.n + kEndCost));
        int64_t s0 = first - (rem - int64_t(kvh) * (sp.n + kEndCost));  // position of the segment's first item
        fetch_q(b, kvh);
        const int64_t me = first / L;
        while (true) {
            const int64_t e0 = s0 + sp.n, end = e0 + kEndCost;
            const int k1 = int(min(e0, last) - first);  // items before the segment's end; none: only its end cost is here
            const int cb = b, ckvh = kvh;
            const int64_t cs0 = s0;
            begin_segment(kvh);
            const bool more = end < last;
            if (more) {  // the next segment, and its query
                s0 = end;
                if (++kvh == Hkv) {
                    kvh = 0;
                    sp = span_of<MODE>(a, ++b);
                }
                fetch_q(b, kvh);
            }
            if (k1 > 0) {
                stream(k1, cb, ckvh);
                deposit();
                __syncwarp();
                const int64_t c0 = cs0 / L;
                const int n = int((e0 - 1) / L - c0) + 1;  // the workers that hold a piece
                // worker c's slot: 2 c + 1 for the segment that begins in its range, 2 c for one that began before
                auto slot_of = [&](int i) { return a.part + (2 * (c0 + i) + (i == 0)) * C::PART; };
                float *slot = slot_of(int(me - c0));
                const float *my = scr + warp * C::SCR;
                for (int idx = lane; idx < tasks; idx += 32) {
                    const int h = idx / (D / 4), d = 4 * (idx % (D / 4));
                    const float M = sm_ml[warp * 16 + h], Ls = sm_ml[warp * 16 + 8 + h];
                    const float4 O = *reinterpret_cast<const float4 *>(my + h * C::ROW + d);
                    if (n == 1) emit(cb, ckvh, h, d, M, Ls, O);
                    else put_piece(slot, h, d, M, Ls, O);
                }
                __syncwarp();
                if (n > 1) {
                    int done = 0;
                    if (lane == 0) done = atomic_add_acq_rel_gpu(a.counters + c0, 1) == n - 1;
                    done = __shfl_sync(0xffffffffu, done, 0);
                    __syncwarp();  // every lane's reads of the pieces follow lane 0's acquire
                    if (done) {
                        float M[NT], Ls[NT];
                        float4 O[NT];
                        merge_pieces<D>(slot_of, G, 0, n, 1, M, Ls, O);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int idx = lane + 32 * t;
                            if (idx < tasks) emit(cb, ckvh, idx / (D / 4), 4 * (idx % (D / 4)), M[t], Ls[t], O[t]);
                        }
                        if (lane == 0) a.counters[c0] = 0;
                    }
                }
            }
            // the end cost's empty items: nothing to wait for, but the next copies start one by one here too,
            // while their entries are in the windows
            while (k < kn && first + k < min(end, last)) {
                shift_windows();
                ++k;
                if (issued < kn && issued < k + R) issue(issued++);
            }
            if (!more) break;
        }
    }
    // after a wait that gave up: no copy may land in memory of a CTA that is gone
    if (dead && lane == 0)
        for (int st = 0; st < R; ++st) mbar_wait_bounded(bars + st * 8, ((armed >> st) & 1u) ^ 1u, a.wait_ns);
    // beside the row-tile kernel: this one is complete when that is, so that the next need wait for one only
    if (a.ownres && blockIdx.x == 0) pdl_wait();
}

// Segments longer than the fused addition is for: a thread per four tokens over the whole grid.
__global__ void __launch_bounds__(kAddThreads) weights_add_kernel(const SubsetArgs a) {
    pdl_trigger();
    const int seg = blockIdx.x, b = seg / a.Hkv, kvh = seg % a.Hkv;
    const int lim = min(max(__ldg(a.ctx + b), 0), a.MBS * kBlockSize);
    pdl_wait();
    float ls[kMaxGroup];
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) ls[h] = h < a.G ? __ldcg(a.lse + int64_t(b) * a.Hq + kvh * a.G + h) : INFINITY;
    add_weights<1>(a, b, kvh, lim, ls, blockIdx.y * kAddThreads + threadIdx.x, gridDim.y * kAddThreads);
}

template <int D, CacheKind KIND, StreamMode MODE>
cudaError_t launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const SubsetArgs &a, int grid,
                     cudaStream_t stream) {
    using C = StreamCfg<D, KIND>;
    const auto kernel = stream_decode_kernel<D, KIND, MODE>;
    const cudaError_t e = smem_once(reinterpret_cast<const void *>(kernel), C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tk, tv, a);
}

}  // namespace

size_t stream_workers(int sms) { return size_t(sms) * kMaxStreamWarps; }
size_t stream_part_floats(int sms, int head_dim) { return 2 * stream_workers(sms) * (size_t(8) * head_dim + 16); }

// ---- rows with a prefix: the own part and the prefix's parts, a warp per row.
// Bound by latency: where the parts are, then the parts, eight in flight; about
// 4 us of a call.
template <int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const SubsetArgs a) {
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    pdl_wait();
    if (r >= int64_t(a.rows) * a.Hq) return;
    constexpr int V = D / 32;  // dims per lane
    const int b = int(r / a.Hq), hq = int(r - int64_t(b) * a.Hq), kvh = hq / a.G, h = hq - kvh * a.G;
    auto load = [&](const float *p, float (&v)[V]) {
        if constexpr (V == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(p) + lane);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(p) + lane);
            v[0] = x.x, v[1] = x.y;
        }
    };
    const int4 at = __ldcg(a.desc + int64_t(b) * a.Hkv + kvh);
    const float2 own = __ldcg(reinterpret_cast<const float2 *>(a.ownml) + r);
    float O[V], M = own.x, Ls = own.y;
    load(a.ownres + r * D, O);
    // in bounds also for row offsets that were not ascending
    const int first = min(max(at.x, 0), a.pgrid - 1), n = min(max(at.y, 0), a.pgrid - first);
    const int prow = min(max(at.w, 0), 128 - a.G) + h;
    auto fold = [&](float m, float l, const float (&v)[V]) {
        const float Mn = fmaxf(M, m);
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn), w = m == -INFINITY ? 0.f : fast_exp2(m - Mn);
        M = Mn;
        Ls = Ls * f + l * w;
#pragma unroll
        for (int i = 0; i < V; ++i) O[i] = O[i] * f + v[i] * w;
    };
    if (n == 1) {
        float v[V];
        load(a.rowres + r * D, v);
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.rowml) + r);
        fold(ml.x, ml.y, v);
    } else {
        constexpr int U = 8;  // pieces in flight
        for (int i0 = 0; i0 < n; i0 += U) {
            float v[U][V], m[U], l[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = min(i0 + u, n - 1);
                const float *ps = a.slots + (2 * int64_t(first + i) + (i == 0)) * (2 * 128 * (D + 2)) +
                                  (at.z & 1) * (128 * (D + 2));
                load(ps + prow * D, v[u]);
                m[u] = __ldcg(ps + 128 * D + prow);
                l[u] = __ldcg(ps + 128 * (D + 1) + prow);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < n) fold(m[u], l[u], v[u]);
        }
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + r * D) + lane * (V / 2);
#pragma unroll
    for (int i = 0; i < V; i += 2) out[i / 2] = pack_bf16x2(O[i] * inv, O[i + 1] * inv);
}

cudaError_t launch_prefix_join(const SubsetArgs &a, int head_dim, cudaStream_t stream) {
    const dim3 grid(unsigned((int64_t(a.rows) * a.Hq + 7) / 8));
    return head_dim == 128 ? launch_pdl(prefix_join_kernel<128>, grid, dim3(256), 0, stream, a)
                           : launch_pdl(prefix_join_kernel<64>, grid, dim3(256), 0, stream, a);
}

cudaError_t launch_stream_decode(const CUtensorMap &tk, const CUtensorMap &tv, const SubsetArgs &a, int head_dim,
                                 CacheKind kind, int sms, cudaStream_t stream) {
    if (a.weights) {
        SubsetArgs f = a;
        f.fused_add = int64_t(a.nseq) * a.Hkv <= sms && a.MBS <= kFusedAddBlocks * a.nseq * a.Hkv;
        cudaError_t e = head_dim == 128 ? launch_t<128, kCacheBf16, kLogits>(tk, tv, f, sms, stream)
                                        : launch_t<64, kCacheBf16, kLogits>(tk, tv, f, sms, stream);
        if (e != cudaSuccess || f.fused_add) return e;
        const int per = kAddThreads / (kBlockSize / 4);  // blocks a CTA takes per turn
        const int x = (a.MBS + per - 1) / per;
        return launch_pdl(weights_add_kernel, dim3(a.nseq * a.Hkv, x < 16 ? x : 16), dim3(kAddThreads), 0, stream, a);
    }
    if (a.cu_q) {
        SubsetArgs f = a;
        f.nseq = a.rows;
        f.ngroups = a.nseq;
        f.cu_g = a.cu_q;
        return head_dim == 128 ? launch_t<128, kCacheBf16, kRows>(tk, tv, f, sms, stream)
                               : launch_t<64, kCacheBf16, kRows>(tk, tv, f, sms, stream);
    }
    if (a.pt && !a.ownres)
        return head_dim == 128 ? launch_t<128, kCacheBf16, kPrefixed>(tk, tv, a, sms, stream)
                               : launch_t<64, kCacheBf16, kPrefixed>(tk, tv, a, sms, stream);
    if (kind == kCacheE4m3) return launch_t<128, kCacheE4m3, kPlain>(tk, tv, a, sms, stream);
    if (kind == kCacheE4m3Block) return launch_t<128, kCacheE4m3Block, kPlain>(tk, tv, a, sms, stream);
    return head_dim == 128 ? launch_t<128, kCacheBf16, kPlain>(tk, tv, a, sms, stream)
                           : launch_t<64, kCacheBf16, kPlain>(tk, tv, a, sms, stream);
}

}  // namespace pa
