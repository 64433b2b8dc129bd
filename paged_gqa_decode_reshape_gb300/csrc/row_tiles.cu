// row_tiles.cu -- attention of many query rows over the same cached tokens on
// the fifth-generation tensor cores (sm_103a): query rows of one sequence over
// its window and sinks (speculative tokens, prefill chunks), and the rows of a
// group of sequences over their shared prefix.
//
// With rows r = (query row, head of the KV head's group), tokens t, z = scale *
// log2(e) * Q K^T:  O_r = sum_t 2^(z_rt - m_r) V_t,  l_r = sum_t 2^(z_rt - m_r),
// out = O / l, one pass with a running m.
//
// Bound: 4 D flops per (row, token) against 4 D bytes per token and KV head:
// with R rows sharing the tokens R flops per byte, so a call is bound by HBM
// below a few hundred rows and by the products above. Measured (28 / 4 heads of
// 128, windows of 4096): 3 prompt chunks of 517 to 2048 rows 250 us = 1.24 PFLOP/s,
// 66 % of what a large library product reaches; 32 sequences of 1 to 6 rows 53 us
// = 3.7 TB/s. What holds the products back (the same call with parts left out):
// without any softmax 203 us, without its exponentials, maxima and sums 226, with
// a quarter of the K/V copies 229. S = Q K^T out of shared memory moves 128 bytes
// per clock, all there is, next to the copies' 64 KB per step; one row tile's
// chain (S, softmax, P V) is hidden by one other row tile only, since S, P and O of
// two fill the tensor memory.
//
//  * A unit is up to 2 x 128 rows of one KV head: two row tiles of RQ =
//    128 / G query rows x G heads, over the union of the blocks they see, in
//    tiles of 128 tokens (8 blocks). Units are concatenated, tile by tile, and
//    cut into equal ranges, one per CTA of a persistent grid: any mix of
//    lengths loads the SMs evenly.
//  * Roles: two producer warps copy K and V tiles by TMA (128-byte swizzle; a K
//    box is 16 tokens of 64 dims, a V box 16 tokens of all dims) into two
//    128-token buffers each, and each unit's queries (a box per row tile and 64
//    dims: RQ rows of G heads); one
//    warp issues the matrix products (a second one, one per row tile, made both
//    fall into step: 322 against 267 us); each row tile has four softmax warps,
//    one thread per row, with its logits S (128 columns, overwritten by the
//    bf16 probabilities P) and its output O (D columns) in tensor memory: 2 x
//    256 of 512 columns. While one row tile's warps work on their softmax the
//    tensor core runs P V and the next Q K^T of the other.
//  * O is rescaled in tensor memory only when a row's maximum has grown by more
//    than 2^8 since the last time: until then probabilities up to 2^8 are exact
//    multiples, bf16 keeps its 8 bits at any magnitude, and l is fp32 (rescaling
//    at every new maximum: 274 against 248 us). P is rounded to bf16 for the product
//    (by at most 2^-8 of a weight); l sums it before that: the sum of rounded values took 277
//    us and gave an error of 2.2e-3 against 2.3e-3 of a row's norm.
//  * Masks: a 16-bit mask per block and row on the tiles at an edge, none
//    inside. V rows no row of the unit sees are zeroed in shared memory. A
//    token that only other rows of the tile see meets them as 0 * V, which
//    is not 0 if V is not finite: a row whose result is not finite, in a unit with
//    such a token, is computed again, over its own tokens only, at the CTA's end.
//  * Units cut between CTAs leave (O, m, l) per row and piece in the workspace;
//    the CTA that completes the count merges them, in piece order, or a join
//    kernel does (for prefixes, with the own tokens' part).
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "subset.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kPreCap = 128;     // entries of the work prefix in shared memory
constexpr int kTileTok = 128;    // tokens per tile
constexpr int kTileBlk = kTileTok / kBlockSize;
constexpr int kStages = 2;       // K tiles, and V tiles, in flight
constexpr int kInfo = 8;         // tile descriptions in flight
constexpr int kWarpsRT = 12;     // 2 x 4 softmax, K producer, products, V producer, one that fills the warpgroup
constexpr float kGrow = 8.f;     // log2 growth of a maximum that rescales O
// Tiles of a CTA's range at least: a piece costs more to merge than a second tile takes. 4 rows on 700 tokens: 1 tile
// 21.5 us, 2 15.8, 3 15.6, 4 19.3; 8 sequences behind a shared prefix of 2001: 15.9, 16.2, 20.1, 18.9.
constexpr int kMinTiles = 2;

// One unit of work, the same in every role.
struct Unit {
    int s, kvh, u;         // sequence (or group), KV head, index of the 2 RQ-row unit
    int r0, nr;            // first query row, query rows (<= 2 RQ)
    int lim0, lim1;        // tokens before which the first and the last row see
    int nb, nb1, jw;       // blocks: nb1 sink blocks, then jw, jw + 1, ...
    int n;                 // tiles (at least one)
};

// What the end of a CTA has to know about rows that came out not finite.
struct After {
    int64_t s0;     // the CTA's first unit, the position of its first tile,
    Unit x;
    int nu;         // and the units per KV head of its sequence
    int odd;        // a row is not finite
    int merged[2];  // cut units merged here, by row tile: kMergedBefore, kMergedHere
    int pad;
};
constexpr int kMergedBefore = 1;  // the unit that began before the CTA's range
constexpr int kMergedHere = 2;    // the unit that begins in it
static_assert(sizeof(After) % 8 == 0, "the prefix sums behind it");

template <int D>
struct RowCfg {
    static constexpr int HV = D / 64;                      // 64-dim halves
    static constexpr int HALF = kTileTok * 128;            // bytes of 64 dims of a tile
    static constexpr int TILE = HV * HALF;                 // a K, V or Q tile
    static constexpr int BLK = kBlockSize * 128;           // a block's 64 dims
    static constexpr size_t off_ring = 2 * size_t(TILE);   // after the two Q tiles
    static constexpr size_t off_stage = off_ring + 2 * size_t(kStages) * TILE;  // 32 rows of 128 bytes per softmax warp
    static constexpr size_t off_bars = off_stage + 8 * 4096;
    static constexpr size_t off_info = off_bars + 224;
    static constexpr size_t off_misc = off_info + 2 * kInfo * 4;
    static constexpr size_t off_after = off_misc + 32;
    static constexpr size_t off_pre = off_after + sizeof(After);
    static constexpr size_t SMEM = 1024 + off_pre + (kPreCap + 1) * 8;
    static constexpr int SLOT = 2 * 128 * (D + 2);         // floats of a piece: per row tile O[128][D], m[128], l[128]
};

template <bool PREFIX>
struct Work {
    const SubsetArgs &a;
    const int RQ;
    __device__ Work(const SubsetArgs &a_) : a(a_), RQ(kTileTok / a_.G) {}
    __device__ int count() const { return PREFIX ? a.ngroups : a.nseq; }
    __device__ void rows(int s, int &r0, int &nr) const {
        const int32_t *cu = PREFIX ? a.cu_g : a.cu_q;
        r0 = min(max(__ldg(cu + s), 0), a.rows);
        nr = min(max(__ldg(cu + s + 1), r0), a.rows) - r0;
    }
    __device__ int units(int s) const {
        int r0, nr;
        rows(s, r0, nr);
        return (nr + 2 * RQ - 1) / (2 * RQ);
    }
    // tokens before which row i (of n) of sequence s sees
    __device__ int limit(int s, int i, int n) const {
        if (PREFIX) return min(max(__ldg(a.plen + s), 0), a.PMBS * kBlockSize);
        return max(min(max(__ldg(a.ctx + s), 0), a.MBS * kBlockSize) - (n - 1 - i), 0);
    }
    __device__ int sinks() const { return PREFIX ? 0 : a.sinks; }
    __device__ int lower(int lim) const {  // first token of the window
        return PREFIX || a.window >= lim ? 0 : lim - a.window;
    }
    __device__ Unit unit(int s, int kvh, int u) const {
        Unit x;
        int n;
        x.s = s;
        x.kvh = kvh;
        x.u = u;
        rows(s, x.r0, n);
        const int i0 = u * 2 * RQ;
        x.nr = max(min(n - i0, 2 * RQ), 0);
        x.lim0 = limit(s, i0, n);
        x.lim1 = limit(s, i0 + x.nr - 1, n);
        x.r0 += i0;
        x.nb1 = (min(sinks(), x.lim1) + kBlockSize - 1) / kBlockSize;
        x.jw = max(lower(x.lim0) / kBlockSize, x.nb1);
        x.nb = x.nb1 + max((x.lim1 + kBlockSize - 1) / kBlockSize - x.jw, 0);
        x.n = max((x.nb + kTileBlk - 1) / kTileBlk, 1);
        return x;
    }
    // tiles of one KV head of sequence s, by a whole warp
    __device__ int64_t tiles(int s) const {
        const int nu = units(s);
        int64_t t = 0;
        for (int u = threadIdx.x & 31; u < nu; u += 32) t += unit(s, 0, u).n;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        return t;
    }
};

// Head h of query row r of sequence s again, over the tokens before lim that it
// sees and nothing else, by a warp in fp32: for rows that other rows' tokens may have
// reached. 32 tokens at a time, a lane per token for its logit, D / 32 dims for V.
template <int D>
__device__ __forceinline__ void redo_row(const SubsetArgs &a, int s, int kvh, int r, int h, int lim) {
    constexpr int V = D / 32, BS = kBlockSize;
    const int lane = threadIdx.x & 31, s1 = min(a.sinks, lim), lo = max(s1, a.window >= lim ? 0 : lim - a.window);
    const int cnt = s1 + max(lim - lo, 0);
    const int64_t ro = (int64_t(r) * a.Hq + kvh * a.G + h) * D;
    const uint4 *q = reinterpret_cast<const uint4 *>(a.q + ro);
    float acc[V], M = -INFINITY, Ls = 0.f;  // Ls: of this lane's tokens
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < cnt; k0 += 32) {
        const int k = min(k0 + lane, cnt - 1), t = k < s1 ? k : k - s1 + lo;
        const int phys = __ldg(a.bt + int64_t(s) * a.MBS + t / BS);
        const bool in = k0 + lane < cnt && phys >= 0 && int64_t(phys) < a.NB;
        const int64_t off = ((int64_t(in ? phys : 0) * BS + t % BS) * a.Hkv + kvh) * D;  // not in: of any row
        const uint4 *kr = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.kc) + off);
        float z = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 x = __ldg(kr + c), y = __ldg(q + c);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) z = fmaf(bf16_hi(ys[e]), bf16_hi(xs[e]), fmaf(bf16_lo(ys[e]), bf16_lo(xs[e]), z));
        }
        z = in ? z * a.scale_log2 : -INFINITY;
        float Mn = z;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
        Mn = fmaxf(M, Mn);
        // a logit of -inf has weight 0, also while no other has come
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn), p = fast_exp2(z - (Mn == -INFINITY ? 0.f : Mn));
        M = Mn;
        Ls = Ls * f + p;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= f;
        const unsigned ins = __ballot_sync(0xffffffffu, in);
#pragma unroll 8
        for (int u = 0; u < 32; ++u) {
            const float pu = __shfl_sync(0xffffffffu, p, u);
            const int64_t at = __shfl_sync(0xffffffffu, off, u) + lane * V;
            const uint32_t *vr = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(a.vc) + at);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const uint32_t v = __ldg(vr + e / 2);
                if ((ins >> u) & 1u) {
                    acc[e] += pu * bf16_lo(v);
                    acc[e + 1] += pu * bf16_hi(v);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
#pragma unroll
    for (int e = 0; e < V; ++e)
        a.out[ro + lane * V + e] =
            __bfloat16_as_ushort(__float2bfloat16_rn(Ls > 0.f ? acc[e] / Ls : Ls != Ls ? Ls : 0.f));
}

// Does a unit whose first row sees tokens before lim0 and whose last one before lim1
// hold a token that its row with the limit lim does not see, with a V row that is
// not finite? By a warp; there are at most a few hundred such tokens, at the ends of
// the window and of the sinks. Without one, a row that is not finite owes it to a
// token it sees itself.
template <int D>
__device__ __forceinline__ bool reached_by_others(const SubsetArgs &a, int s, int kvh, int lim0, int lim1, int lim) {
    constexpr int LR = D / 8, TP = 32 / LR, U = 4, BS = kBlockSize;  // lanes per row, rows at once
    const int lane = threadIdx.x & 31;
    auto lower = [&](int lim) { return a.window >= lim ? 0 : lim - a.window; };
    const int l0 = lower(lim0), l1 = lower(lim1), lo = lower(lim), nb1 = (min(a.sinks, lim1) + BS - 1) / BS;
    bool bad = false;
    auto scan = [&](int from, int to) {
#pragma unroll 1
        for (int t0 = from + lane / LR; t0 - lane / LR < to; t0 += TP * U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * TP;
                const int phys = t < to && !(t >= lo && t < lim) ? __ldg(a.bt + int64_t(s) * a.MBS + t / BS) : -1;
                if (phys < 0 || int64_t(phys) >= a.NB) continue;
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(a.vc) +
                                      ((int64_t(phys) * BS + t % BS) * a.Hkv + kvh) * LR + lane % LR);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    bad = bad || (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
            }
        }
    };
    scan(min(a.sinks, lim), min(nb1 * BS, lim1));
    scan(max(l0 / BS, nb1) * BS, l1);
    scan(lim0, lim1);
    return __any_sync(0xffffffffu, bad);
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kWarpsRT * 32, 1)
    row_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const SubsetArgs a) {
    using C = RowCfg<D>;
    constexpr int BS = kBlockSize, HV = C::HV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *bp = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int Hkv = a.Hkv, G = a.G;
    const Work<PREFIX> work(a);
    const int RQ = work.RQ;
    const uint32_t ring = base + uint32_t(C::off_ring);
    const uint32_t full = base + uint32_t(C::off_bars), empty = full + kStages * 8;
    const uint32_t q_full = empty + kStages * 8, q_empty = q_full + 16, s_full = q_empty + 16;
    const uint32_t p_ready = s_full + 16, o_full = p_ready + 32, drained = o_full + 16, piece_bar = drained + 8, last_bar = piece_bar + 16;
    const uint32_t ml_bar = last_bar + 16;
    volatile int *info = reinterpret_cast<volatile int *>(bp + C::off_info);
    volatile int *vfix = info + kInfo;  // V rows to zero: see the producers
    volatile int *misc = reinterpret_cast<volatile int *>(bp + C::off_misc);  // [0] tensor memory, [1] gave up, [2 + w] queries,
                                                                          // [4 + w] completes the count, [6], [7] steps begun
    int64_t *pre = reinterpret_cast<int64_t *>(bp + C::off_pre);

    if (!PREFIX) pdl_trigger();
    if (tid == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 2);  // K's producer and V's
            mbar_init(empty + 8 * i, 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(q_full + 8 * w, 1);
            mbar_init(q_empty + 8 * w, 1);
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_ready + 16 * w, 128);
            mbar_init(p_ready + 16 * w + 8, 128);
            mbar_init(o_full + 8 * w, 1);
            mbar_init(piece_bar + 8 * w, 4);
            mbar_init(last_bar + 8 * w, 1);
            mbar_init(ml_bar + 8 * w, 4);
        }
        mbar_init(drained, 1);
        fence_barrier_init();
        misc[1] = 0;
        pre[0] = 0;
    }
    // ---- tiles per KV head of groups of `str` sequences, and their prefix sums
    const int ns = work.count(), str = (ns + kPreCap - 1) / kPreCap, np = (ns + str - 1) / str;
    // by a thread where sequences have a unit or two, so that many are looked up at once, else by a warp
    for (int i = tid; i < np; i += kWarpsRT * 32) {
        int64_t t = 0;
        for (int s = i * str; t >= 0 && s < min((i + 1) * str, ns); ++s) {
            const int nu = work.units(s);
            for (int u = 0; u < min(nu, 2); ++u) t += work.unit(s, 0, u).n;
            if (nu > 2) t = -1;
        }
        pre[i + 1] = t;
    }
    __syncthreads();
    for (int i = warp; i < np; i += kWarpsRT) {
        if (pre[i + 1] >= 0) continue;
        int64_t t = 0;
        for (int s = i * str; s < min((i + 1) * str, ns); ++s) t += work.tiles(s);
        if (lane == 0) pre[i + 1] = t;
    }
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
    if (PREFIX) {
        // the kernel for the own tokens runs beside this one: it may start once
        // what came before this kernel is complete
        pdl_wait();
        pdl_trigger();
    }
    if constexpr (PREFIX) {  // sequences of no group have no prefix part
        for (int b = blockIdx.x * (kWarpsRT * 32) + tid; b < a.rows; b += gridDim.x * (kWarpsRT * 32)) {
            int lo = 0, hi = a.ngroups;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(a.cu_g + mid) <= b) lo = mid; else hi = mid;
            }
            if (b < __ldg(a.cu_g + lo) || b >= __ldg(a.cu_g + lo + 1))
                for (int h = 0; h < Hkv; ++h) a.desc[int64_t(b) * Hkv + h] = make_int4(0, 0, 0, 0);
        }
    }
    const int64_t total = int64_t(Hkv) * pre[np];
    const int64_t L = max((total + gridDim.x - 1) / gridDim.x, int64_t(a.min_items));
    const int64_t pos0 = int64_t(blockIdx.x) * L, pos1 = min(total, pos0 + L);
    if (pos0 >= pos1) {  // whole CTA: nothing to do
        // a call without any rows still ends after what came before it, which later kernels may need
        if constexpr (!PREFIX) {
            pdl_wait();
            if (a.cuts && tid == 0) a.cuts[blockIdx.x].pieces = 0;
        }
        return;
    }

    if (warp == 9) tmem_alloc(smem_u32(const_cast<int *>(misc)), 512);
    // ---- the first unit, by every warp
    Unit x;
    int64_t s0;  // global position of its first tile
    int nu;      // units per KV head of its sequence
    {
        int lo = 0, hi = np;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (int64_t(Hkv) * pre[mid] <= pos0) lo = mid; else hi = mid;
        }
        int s = lo * str;
        int64_t rem = pos0 - int64_t(Hkv) * pre[lo], t = str == 1 ? pre[lo + 1] - pre[lo] : work.tiles(s);
        while (rem >= int64_t(Hkv) * t && s + 1 < ns) {
            rem -= int64_t(Hkv) * t;
            t = work.tiles(++s);
        }
        const int kvh = int(rem / t);
        rem -= int64_t(kvh) * t;
        nu = work.units(s);
        int u = 0;
        for (int u0 = 0; u0 < nu; u0 += 32) {  // 32 units at a time
            const int n = u0 + lane < nu ? work.unit(s, kvh, u0 + lane).n : 0;
            int64_t e = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, e, o);
                if (lane >= o) e += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, n > 0 && e > rem);
            if (past) {
                const int at = __ffs(past) - 1;
                u = u0 + at;
                rem -= __shfl_sync(0xffffffffu, e - n, at);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, e, 31);
        }
        x = work.unit(s, kvh, u);
        s0 = pos0 - rem;
    }
    After &after = *reinterpret_cast<After *>(bp + C::off_after);
    if (!PREFIX && tid == 0) {
        after.s0 = s0;
        after.x = x;
        after.nu = nu;
        after.odd = after.merged[0] = after.merged[1] = 0;
    }
    auto next_unit = [&]() {
        s0 += x.n;
        int s = x.s, kvh = x.kvh, u = x.u + 1;
        if (u == nu) {
            u = 0;
            if (++kvh == Hkv) {
                kvh = 0;
                do nu = work.units(++s);
                while (nu == 0 && s + 1 < ns);  // positions are left, so there is one
            }
        }
        x = work.unit(s, kvh, u);
    };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(misc[0]);
    if (!PREFIX) pdl_wait();
    auto give_up = [&]() {
        if (lane == 0) {
            misc[1] = 1;
            atomicOr(a.status, kStatusTimeout);
        }
    };
    // wait unless the CTA gave up; false: it has
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u))) return true;
        const bool ok = !misc[1] && mbar_wait_bounded(bar, parity & 1u, a.wait_ns);
        if (__all_sync(0xffffffffu, ok)) return true;
        give_up();
        return false;
    };

    // registers: the 168 per thread of the launch, 224 + 224 + 56 over its three warpgroups
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8 || warp == 10) {
        // =========================================== producers: K and queries, V
        // step i of the CTA reads K of its tile i and V of its tile i - 1, in buffer pair i % 2
        const bool is_k = warp == 8;
        const int32_t *table = PREFIX ? a.pt : a.bt;
        const int mbs = PREFIX ? a.PMBS : a.MBS;
        const uint64_t policy = l2_policy_normal();  // other units of the KV head read the same blocks
        const uint32_t buf = ring + (is_k ? 0 : kStages * C::TILE);
        uint32_t i = 0;           // the next step
        uint32_t nq[2] = {0, 0};  // query tiles so far
        bool ok = true;
        auto next_step = [&]() -> bool {  // step i's buffers are free
            return (i < kStages || wait(empty + 8 * (i % kStages), i / kStages + 1)) && int(i) < a.stop_item;
        };
        if (!is_k) {  // no V in the first step
            if (lane == 0) mbar_arrive(full);
            i = 1;
        }
        for (int64_t p = pos0; ok && p < pos1;) {
            const int t0 = int(p - s0), t1 = int(min(pos1 - s0, int64_t(x.n)));
            // table entries of 32 list entries (4 tiles), one per lane, one window ahead
            auto entry = [&](int e) -> int {
                if (e >= x.nb) return -1;
                return __ldg(table + int64_t(x.s) * mbs + (e < x.nb1 ? e : e - x.nb1 + x.jw));
            };
            int cur = entry(t0 * kTileBlk + lane), nxt = entry(t0 * kTileBlk + 32 + lane), at = t0;
            for (int t = t0; t < t1; ++t, ++i) {
                if (t == at + 4) {
                    at = t;
                    cur = nxt;
                    nxt = entry(t * kTileBlk + 32 + lane);
                }
                // bit b: block b of the tile is in the pool
                const unsigned blocks = (__ballot_sync(0xffffffffu, cur >= 0 && int64_t(cur) < a.NB) >>
                                         ((t - at) * kTileBlk)) & 0xffu;
                if (!(ok = next_step())) break;
                const uint32_t st = i % kStages, bar = full + 8 * st;
                if (lane == 0) {
                    if (is_k) {
                        info[i % kInfo] = int(blocks);
                    } else {
                        // V rows nobody sees: absent blocks, and what lies past the last row's limit
                        const int tail = x.lim1 % BS, lb = x.nb - 1 - t * kTileBlk;  // lb: the unit's last block
                        const bool cut = tail && lb >= 0 && lb < kTileBlk;
                        vfix[i % kInfo] = blocks == 0xffu && !cut ? 0 : int(blocks | 0x100u | (cut ? (lb << 12 | tail << 16) : 0));
                    }
                    const uint32_t bytes = uint32_t(__popc(blocks)) * C::BLK * HV;
                    if (bytes) mbar_arrive_expect_tx(bar, bytes);
                    else mbar_arrive(bar);
                }
                __syncwarp();
                for (int b = 0; b < kTileBlk; ++b) {
                    const int ph = __shfl_sync(0xffffffffu, cur, (t - at) * kTileBlk + b);
                    if (!((blocks >> b) & 1u) || !tc_elect()) continue;
                    if (is_k) {
#pragma unroll
                        for (int hf = 0; hf < HV; ++hf)
                            tma_load_4d(buf + st * C::TILE + hf * C::HALF + b * C::BLK, &tm_k, bar, hf * 64, x.kvh, 0, ph,
                                        policy);
                    } else {
                        tma_load_5d(buf + st * C::TILE + b * C::BLK * HV, &tm_v, bar, 0, 0, 0, x.kvh, ph, policy);
                    }
                }
                __syncwarp();
                if (is_k && t == t0) {
                    // the unit's queries: rows (query row, head) are consecutive; rows past the
                    // unit's are read too and dropped at the end
                    for (int w = 0; ok && w < (x.nr > RQ ? 2 : 1); ++w) {
                        if (nq[w] > 0) ok = wait(q_empty + 8 * w, nq[w] + 1);
                        if (!ok) break;
                        ++nq[w];
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full + 8 * w, uint32_t(RQ * G * D * 2));
                            for (int f = 0; f < HV; ++f)
                                tma_load_3d(base + w * C::TILE + f * C::HALF, &tm_q, q_full + 8 * w, f * 64,
                                            x.kvh * G, x.r0 + w * RQ, policy);
                        }
                        __syncwarp();
                    }
                }
            }
            p = s0 + t1;
            if (ok && p < pos1) next_unit();
        }
        if (ok && is_k) {  // no K in the last step
            if (next_step() && lane == 0) mbar_arrive(full + 8 * (i % kStages));
        }
        if (lane == 0) {  // what was started, for an end after giving up
            misc[is_k ? 6 : 7] = int(i);
            if (is_k) {
                misc[2] = int(nq[0]);
                misc[3] = int(nq[1]);
            }
        }
    } else if (warp == 9) {
        // ====================================================== matrix products
        constexpr uint32_t id_s = tc_idesc(128, 128, false), id_o = tc_idesc(128, D, true);
        // the same value in every lane, known as such: the products take uniform operands
        auto uniform = [](uint32_t v) -> uint32_t { return __shfl_sync(0xffffffffu, v, 0); };
        const uint32_t td = uniform(tmem), qd = uniform(tc_desc_lo(base, 16)), kd = uniform(tc_desc_lo(ring, 16));
        // V block-major: 16 tokens of 64 dims, then the next 64
        const uint32_t vd = uniform(tc_desc_lo(ring + kStages * C::TILE, C::BLK));
        // S_w = Q_w K^T
        auto qk = [&](int w, uint32_t st) {
            const uint32_t q = qd + w * (C::TILE >> 4), k = uniform(kd + st * (C::TILE >> 4));
            if (tc_elect()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk / 4) * C::HALF + (kk % 4) * 32) >> 4;
                    tc_mma_ss(td + 256 * w, q + o, kTcDescHi, k + o, kTcDescHi, id_s, kk > 0);
                }
                tc_commit(s_full + 8 * w);
            }
        };
        // O_w (+)= P_w V, half hf of the tokens
        auto pv = [&](int w, uint32_t st, bool more, int hf) {
            const uint32_t v = uniform(vd + st * (C::TILE >> 4));
            more = uniform(more);
            if (tc_elect()) {
#pragma unroll
                for (int k = 0; k < kTileTok / 32; ++k) {
                    const int kk = hf * (kTileTok / 32) + k;
                    tc_mma_ts(td + 256 * w + 128, td + 256 * w + 8 * kk, v + (kk * C::BLK * HV >> 4), kTcDescHi, id_o,
                              more || kk > 0);
                }
            }
        };
        uint32_t i = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;  // step; phases of q_full and p_ready
        bool two = false, more = false;  // the tile before: two row tiles; not the first of its piece
        // one step: P V of the tile before, Q K^T of this one; q0: the first tile of a piece, cur:
        // there is a tile, cur2: with two row tiles, qlast: the last of its piece
        auto step = [&](bool q0, bool cur, bool cur2, bool qlast) -> bool {
            const uint32_t st = i % kStages;
            if (!wait(full + 8 * st, i / kStages)) return false;
            if (i > 0) {
                const int fix = vfix[i % kInfo];
                if (fix) {
                    uint8_t *v = bp + C::off_ring + (kStages + st) * C::TILE;
                    const int lb = (fix >> 12) & 15, tail = fix >> 16;
                    for (int b = 0; b < kTileBlk; ++b) {
                        const int from = !((fix >> b) & 1) ? 0 : tail && b == lb ? tail : BS;  // first row to zero
                        for (int idx = from * 8 + lane; idx < BS * 8; idx += 32)
#pragma unroll
                            for (int hf = 0; hf < HV; ++hf)
                                *reinterpret_cast<uint4 *>(v + (b * HV + hf) * C::BLK + idx * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (i > 0 && (w == 0 || two)) {
                    uint32_t &n = w ? np1 : np0;
                    if (!wait(p_ready + 16 * w, n)) return false;
                    tc_fence_after();
                    pv(w, st, more, 0);
                    if (!wait(p_ready + 16 * w + 8, n++)) return false;
                    tc_fence_after();
                    pv(w, st, true, 1);
                    if (q0 && tc_elect()) tc_commit(o_full + 8 * w);
                }
                if (cur && (w == 0 || cur2)) {
                    if (q0 && !wait(q_full + 8 * w, w ? nq1++ : nq0++)) return false;
                    tc_fence_after();
                    qk(w, st);
                    if (qlast && tc_elect()) tc_commit(q_empty + 8 * w);
                }
            }
            if (tc_elect()) tc_commit(empty + 8 * st);
            ++i;
            return true;
        };
        bool ok = true;
        for (int64_t p = pos0; ok && p < pos1;) {
            const int t0 = int(p - s0), t1 = int(min(pos1 - s0, int64_t(x.n)));
            const bool cur2 = x.nr > RQ;
            for (int t = t0; t < t1; ++t) {
                if (!(ok = step(t == t0, true, cur2, t == t1 - 1))) break;
                two = cur2;
                more = t > t0;
            }
            p = s0 + t1;
            if (ok && p < pos1) next_unit();
        }
        if (ok) ok = step(true, false, false, false);
        if (!ok) {
            // gave up: the products in flight end before the memory they use goes
            if (tc_elect()) tc_commit(drained);
            __syncwarp();
            mbar_wait_bounded(drained, 0, a.wait_ns);
        }
    }
    } else {
        // ============================================================= softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lane_base = uint32_t(warp & 3) << 21;  // this warp's 32 of the 128 lanes
        const uint32_t ts = tmem + lane_base + 256 * w, to = ts + 128;
        const int i = row / G, h = row - i * G;
        uint32_t ph = 0, tile_no = 0, units = 0, merges = 0, pubs = 0;
        if (!PREFIX && a.cuts && tid == 0) a.cuts[blockIdx.x].pieces = 0;  // no unit is cut so far
        bool ok = true;
        for (int64_t p = pos0; ok && p < pos1;) {
            const int t0 = int(p - s0), t1 = int(min(pos1 - s0, int64_t(x.n)));
            const int ir = w * RQ + i;  // query row of the unit
            const bool act = i < RQ && ir < x.nr;
            if (w == 0 || x.nr > RQ) {
                // row ir of the unit sees tokens before base + ir (PREFIX: all rows before lim1)
                int base = 0;
                if (!PREFIX) {
                    int rr, nn;
                    work.rows(x.s, rr, nn);
                    base = min(max(__ldg(a.ctx + x.s), 0), a.MBS * BS) - (nn - 1 - (x.r0 - rr));
                }
                const int lim = !act ? 0 : PREFIX ? x.lim1 : max(base + ir, 0);
                const int S1 = min(work.sinks(), lim), lo = max(S1, work.lower(lim));
                float m = -INFINITY, l = 0.f;
                for (int t = t0; t < t1; ++t) {
                    if (!(ok = wait(s_full + 8 * w, ph++))) break;
                    tc_fence_after();
                    const int blocks = info[(tile_no + (t - t0)) % kInfo];
                    const int e0 = t * kTileBlk;
                    auto tok = [&](int e) { return (e < x.nb1 ? e : e - x.nb1 + x.jw) * BS; };
                    const int ta = tok(e0);
                    const bool joined = e0 >= x.nb1 || e0 + kTileBlk <= x.nb1 || x.jw == x.nb1;
                    const bool inside = blocks == 0xff && joined &&
                                        (ta + kTileTok <= S1 || (ta >= lo && ta + kTileTok <= lim));
                    const bool masked = !__all_sync(0xffffffffu, inside || !act);
                    float s[kTileTok];
                    auto load = [&](int c) { tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s[32 * c])); };
                    auto mask = [&](int b) {  // unseen tokens of block b
                        const int tb = tok(e0 + b);
                        auto bits = [&](int from, int to) -> uint32_t {
                            const int y0 = min(max(from - tb, 0), 16), y1 = min(max(to - tb, 0), 16);
                            return y1 > y0 ? ((1u << y1) - 1u) & ~((1u << y0) - 1u) : 0u;
                        };
                        const uint32_t mk = (blocks >> b) & 1 ? bits(0, S1) | bits(lo, lim) : 0u;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (!((mk >> c) & 1u)) s[16 * b + c] = -INFINITY;
                    };
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    // the maximum of one half while the other is on its way
                    load(0);
                    load(1);
                    tc_wait_ld();
                    load(2);
                    load(3);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        if (hf == 1) tc_wait_ld();
                        if (masked) {
#pragma unroll
                            for (int b = 0; b < kTileBlk / 2; ++b) mask(hf * (kTileBlk / 2) + b);
                        }
#pragma unroll
                        for (int c = 64 * hf; c < 64 * hf + 64; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + 2 * e], s[c + 2 * e + 1]);
                    }
                    const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2;
                    const bool grow = mt > m + kGrow || (m == -INFINITY && mt > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? (m == -INFINITY ? 0.f : fast_exp2(m - mt)) : 1.f;
                        if (grow) m = mt;
                        l *= f;
                        if (t > t0) {  // P V of the tile before is complete: S of this one was issued after it
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(to + 16 * c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(to + 16 * c, o);
                            }
                        }
                    }
                    const float mr = m == -INFINITY ? 0.f : m;
                    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mr2 = make_float2(-mr, -mr);
                    float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const int k = 64 * hf + 2 * e;
                            const float2 za = fma2(make_float2(s[k], s[k + 1]), sc2, mr2);
                            const float2 zb = fma2(make_float2(s[k + 2], s[k + 3]), sc2, mr2);
                            const float2 pa = make_float2(fast_exp2(za.x), fast_exp2(za.y));
                            const float2 pb = make_float2(fast_exp2(zb.x), fast_exp2(zb.y));
                            la = add2(la, pa);
                            lb = add2(lb, pb);
                            pk[e] = pack_bf16x2(pa.x, pa.y);
                            pk[e + 1] = pack_bf16x2(pb.x, pb.y);
                        }
                        // P V begins with the first half's tokens
                        tmem_st32(ts + 32 * hf, pk);
                        tc_wait_st();
                        tc_fence_before();
                        mbar_arrive(p_ready + 16 * w + 8 * hf);
                    }
                    l += (la.x + la.y) + (lb.x + lb.y);
                }
                // ---- the end of the unit, or of this CTA's piece of it
                const bool whole = t0 == 0 && t1 == x.n;
                const int c0 = int(s0 / L), npieces = int((s0 + x.n - 1) / L) - c0 + 1, mine = int(blockIdx.x) - c0;
                if (!(ok = wait(o_full + 8 * w, units++))) break;
                tc_fence_after();
                const int64_t orow = int64_t(x.r0 + ir) * a.Hq + x.kvh * G + h;
                auto piece_of = [&](int k) {
                    return a.slots + (2 * int64_t(c0 + k) + (k == 0)) * C::SLOT + w * (C::SLOT / 2);
                };
                const unsigned acts = __ballot_sync(0xffffffffu, act);
                uint8_t *stage = bp + C::off_stage + warp * 4096;
                const int sj = lane & 7, sr = lane >> 3;
                // 32 rows of 128 bytes, one per lane, to global memory: eight lanes per row
                auto store_rows = [&](const uint4 (&v)[8], auto row_at) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = v[j];
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = 4 * k + sr;
                        const uint4 y = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((sj ^ (r & 7)) << 4));
                        const int64_t ro = __shfl_sync(0xffffffffu, orow, r);
                        if ((acts >> r) & 1u) __stcg(reinterpret_cast<uint4 *>(row_at(r, ro)) + sj, y);
                    }
                };
                // this CTA's O columns 32 c .. 32 c + 31; a row that saw no token has 0, whatever the products held
                auto own = [&](int c, float (&v)[32]) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32(to + 32 * c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = l == 0.f ? 0.f : __uint_as_float(o[e]);
                };
                // the O of a piece, with m and l per row; PREFIX: of a whole unit too, by row
                auto publish = [&]() {
                    float *ps = piece_of(mine);
#pragma unroll 1  // code that runs once per unit: what has to be fetched first costs more than a loop
                    for (int c = 0; c < D / 32; ++c) {
                        float v[32];
                        own(c, v);
                        uint4 y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                                              __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
                        store_rows(y, [&](int r, int64_t ro) {
                            return (PREFIX && whole ? a.rowres + ro * D : ps + ((warp & 3) * 32 + r) * D) + 32 * c;
                        });
                    }
                    if (act) {
                        if (PREFIX && whole) {
                            __stcg(reinterpret_cast<float2 *>(a.rowml) + orow, make_float2(m, l));
                        } else {
                            __stcg(ps + 128 * D + row, m);
                            __stcg(ps + 128 * (D + 1) + row, l);
                        }
                    }
                };
                if constexpr (PREFIX) {
                    publish();
                    if (act && h == 0 && t0 == 0)  // where this row's parts are
                        a.desc[int64_t(x.r0 + ir) * Hkv + x.kvh] = make_int4(c0, npieces, w, row);
                } else {
                    if (whole) {
                        const float iv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
                        bool fine = true;
#pragma unroll 1
                        for (int c2 = 0; c2 < HV; ++c2) {
                            uint4 y[8];
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float v[32];
                                own(2 * c2 + q, v);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    v[e] *= iv;
                                    fine = fine && fabsf(v[e]) <= 3.4028234e38f;
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[4 * q + e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]),
                                                              pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                                              pack_bf16x2(v[8 * e + 4], v[8 * e + 5]),
                                                              pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
                            }
                            store_rows(y, [&](int, int64_t ro) { return a.out + ro * D + 64 * c2; });
                        }
                        if (act && !fine) after.odd = 1;
                    } else {
                        publish();
                        if (a.cuts) {  // the join kernel merges
                            if (tid == 0 && t0 == 0)
                                a.cuts[blockIdx.x] = CutUnit{x.s, x.kvh, x.r0, x.nr, base, npieces, {}};
                        } else {
                            // the row tile's four warps publish their part; the piece that completes the count merges
                            __syncwarp();
                            if (lane == 0) mbar_arrive(piece_bar + 8 * w);
                            if ((warp & 3) == 0) {
                                if (!(ok = wait(piece_bar + 8 * w, pubs))) break;
                                if (lane == 0) {
                                    misc[4 + w] = atomic_add_acq_rel_gpu(a.counters + 2 * c0 + w, 1) == npieces - 1;
                                    mbar_arrive(last_bar + 8 * w);
                                }
                            }
                            if (!(ok = wait(last_bar + 8 * w, pubs++))) break;
                            if (misc[4 + w]) {
                                if (row == 0) {
                                    a.counters[2 * c0 + w] = 0;
                                    after.merged[w] |= t0 == 0 ? kMergedHere : kMergedBefore;
                                }
                                // The pieces' common maximum and sum, a row per thread; then the rows, each by a warp with
                                // its columns side by side, RB rows of KB pieces in flight: bound by the latency of L2
                                // loads (2 x 8: 52.9 us for 32 sequences of 1 to 6 rows, 3 x 8 53.3, 4 x 4 53.6; with
                                // rows kept to their thread, a piece at a time, 55.8).
                                float2 *ml = reinterpret_cast<float2 *>(bp + C::off_stage + 4 * w * 4096);  // [128] M, 1 / l
                                if (act) {
                                    constexpr int KW = 8;
                                    float M = -INFINITY, Ls = 0.f;
                                    for (int k = 0; k < npieces; k += KW) {
                                        float mk[KW], lk[KW];
#pragma unroll
                                        for (int e = 0; e < KW; ++e) {
                                            const float *ps = piece_of(min(k + e, npieces - 1)) + 128 * D + row;
                                            mk[e] = __ldcg(ps);
                                            lk[e] = __ldcg(ps + 128);
                                        }
#pragma unroll
                                        for (int e = 0; e < KW; ++e) {
                                            if (k + e >= npieces) break;
                                            const float Mn = fmaxf(M, mk[e]);
                                            const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
                                            Ls = Ls * f + (mk[e] == -INFINITY ? lk[e] : lk[e] * fast_exp2(mk[e] - Mn));
                                            M = Mn;
                                        }
                                    }
                                    ml[row] = make_float2(M == -INFINITY ? 0.f : M, Ls == 0.f ? 0.f : 1.f / Ls);
                                }
                                __syncwarp();
                                if (lane == 0) mbar_arrive(ml_bar + 8 * w);
                                if (!(ok = wait(ml_bar + 8 * w, merges++))) break;
                                constexpr int V = D / 32, RB = 8, KB = 2;
                                const int rows = min(x.nr - w * RQ, RQ) * G;
#pragma unroll 1
                                for (int g0 = warp & 3; g0 < rows; g0 += 4 * RB) {
                                    float acc[RB][V];
                                    float2 mr[RB];
#pragma unroll
                                    for (int u = 0; u < RB; ++u) {
                                        mr[u] = ml[min(g0 + 4 * u, rows - 1)];
#pragma unroll
                                        for (int e = 0; e < V; ++e) acc[u][e] = 0.f;
                                    }
#pragma unroll 1
                                    for (int k = 0; k < npieces; k += KB) {
                                        float o[KB][RB][V], mk[KB][RB];
#pragma unroll
                                        for (int kk = 0; kk < KB; ++kk) {
                                            const float *ps = piece_of(min(k + kk, npieces - 1));
#pragma unroll
                                            for (int u = 0; u < RB; ++u) {
                                                const int r = min(g0 + 4 * u, rows - 1);
                                                mk[kk][u] = __ldcg(ps + 128 * D + r);
                                                if constexpr (V == 4) {
                                                    const float4 z = __ldcg(reinterpret_cast<const float4 *>(ps + r * D) + lane);
                                                    o[kk][u][0] = z.x, o[kk][u][1] = z.y, o[kk][u][2] = z.z, o[kk][u][3] = z.w;
                                                } else {
                                                    const float2 z = __ldcg(reinterpret_cast<const float2 *>(ps + r * D) + lane);
                                                    o[kk][u][0] = z.x, o[kk][u][1] = z.y;
                                                }
                                            }
                                        }
#pragma unroll
                                        for (int kk = 0; kk < KB; ++kk) {
                                            if (k + kk >= npieces) break;
#pragma unroll
                                            for (int u = 0; u < RB; ++u) {
                                                const float f = fast_exp2(mk[kk][u] - mr[u].x) * mr[u].y;
#pragma unroll
                                                for (int e = 0; e < V; ++e) acc[u][e] += f * o[kk][u][e];
                                            }
                                        }
                                    }
#pragma unroll
                                    for (int u = 0; u < RB; ++u) {
                                        const int r = g0 + 4 * u;
                                        if (r >= rows) break;
                                        bool fine = true;
#pragma unroll
                                        for (int e = 0; e < V; ++e) fine = fine && fabsf(acc[u][e]) <= 3.4028234e38f;
                                        if (!fine) after.odd = 1;
                                        uint32_t *dst = reinterpret_cast<uint32_t *>(
                                            a.out + (int64_t(x.r0 + w * RQ + r / G) * a.Hq + x.kvh * G + r % G) * D) + lane * (V / 2);
                                        if constexpr (V == 4)
                                            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[u][0], acc[u][1]),
                                                                                         pack_bf16x2(acc[u][2], acc[u][3]));
                                        else
                                            *dst = pack_bf16x2(acc[u][0], acc[u][1]);
                                    }
                                }
                                __syncwarp();
                            }
                        }
                    }
                }
            }
            tile_no += uint32_t(t1 - t0);
            p = s0 + t1;
            if (p < pos1) next_unit();
        }
    }
    // ---- every role is done: the tensor memory goes back
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
    if (misc[1] && warp == 8) {
        // the CTA gave up: nothing that was started may land after it is gone (otherwise the products have
        // waited for every copy)
        const int steps = max(misc[6], misc[7]);
        for (int i = max(steps - kStages, 0); i < steps; ++i)
            mbar_wait_bounded(full + 8 * (i % kStages), uint32_t(i / kStages) & 1u, a.wait_ns);
        for (int w = 0; w < 2; ++w)
            if (misc[2 + w] > 0) mbar_wait_bounded(q_full + 8 * w, uint32_t(misc[2 + w] - 1) & 1u, a.wait_ns);
    }
    // ---- the rows written here that are not finite, a warp per row, over their own tokens. Only now: this may take
    // long (5 ms of a warp for a row of 40000 tokens), and nothing waits for these warps any more.
    if constexpr (!PREFIX) {
        if (after.odd == 0 || misc[1]) return;
        if (warp >= 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");  // the launch's share for every warp again
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 168;");
        s0 = after.s0;
        x = after.x;
        nu = after.nu;
#pragma unroll 1
        for (int64_t p = pos0; p < pos1;) {
            const int t0 = int(p - s0), t1 = int(min(pos1 - s0, int64_t(x.n)));
#pragma unroll 1
            for (int r = warp; r < x.nr * G; r += kWarpsRT) {
                const int ir = r / G;
                const bool written = (t0 == 0 && t1 == x.n) ||
                                     (after.merged[ir >= RQ] & (t0 == 0 ? kMergedHere : kMergedBefore));
                if (!written) continue;
                const uint32_t *o = reinterpret_cast<const uint32_t *>(
                    a.out + (int64_t(x.r0 + ir) * a.Hq + x.kvh * G + r % G) * D) + lane * (D / 64);
                bool fine = true;
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    const uint32_t v = __ldcg(o + e);
                    fine = fine && (v & 0x7f80u) != 0x7f80u && (v & 0x7f800000u) != 0x7f800000u;
                }
                if (__all_sync(0xffffffffu, fine)) continue;
                int rr, nn;
                work.rows(x.s, rr, nn);
                const int lim = work.limit(x.s, x.r0 + ir - rr, nn);
                if (reached_by_others<D>(a, x.s, x.kvh, x.lim0, x.lim1, lim))
                    redo_row<D>(a, x.s, x.kvh, x.r0 + ir, r % G, lim);
            }
            p = s0 + t1;
            if (p < pos1) next_unit();
        }
    }
}

// The rows of the units that were cut between CTAs: the unit that begins in CTA
// blockIdx.x's range and leaves it, if there is one; a warp per row (RB of them at
// a time), its columns side by side, KB pieces in flight. Bound by latency. For
// calls with fewer units than half the CTAs, whose units have several pieces each:
// one CTA would read them all. Merged by the last piece's CTA and by this kernel
// (which costs 1.6 us of the host as well), on 4000 tokens: 8 sequences of 5 rows
// 32.9 and 28.8 us, 2 of 64 rows 40.8 and 26.8; with 128 units on 152 CTAs, 32
// sequences of 2 rows on 3000 tokens, 49.1 and 54.5.
template <int D>
__global__ void __launch_bounds__(256) cut_join_kernel(const SubsetArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int V = D / 32, RB = 4, KB = 4, SLOT = RowCfg<D>::SLOT;
    const int4 *rec = reinterpret_cast<const int4 *>(a.cuts + blockIdx.x);
    const int4 c0 = __ldcg(rec), c1 = __ldcg(rec + 1);
    const CutUnit u{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, {}};
    if (u.pieces < 2) return;
    const int lane = threadIdx.x & 31, step = int(gridDim.y) * 8;
    const int G = a.G, RQ = kTileTok / G, rows = u.nr * G, np = u.pieces;
    auto slot = [&](int k) { return a.slots + (2 * int64_t(blockIdx.x + k) + (k == 0)) * SLOT; };
    for (int g0 = int(blockIdx.y) * 8 + int(threadIdx.x >> 5); g0 < rows; g0 += RB * step) {
        int at[RB];  // the row's place in its row tile, -1: none; floats of the row tiles before
        int before[RB];
        float acc[RB][V], M[RB], L[RB], o[KB][RB][V];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int g = g0 + i * step, w = g >= RQ * G;
            at[i] = g < rows ? g - w * RQ * G : -1;
            before[i] = w * (SLOT / 2);
            M[i] = -INFINITY;
            L[i] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[i][e] = 0.f;
        }
        auto load = [&](int k) {  // pieces k ...
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int i = 0; i < RB; ++i) {
#pragma unroll
                    for (int e = 0; e < V; ++e) o[j][i][e] = 0.f;
                    if (k + j >= np || at[i] < 0) continue;
                    const float *ps = slot(k + j) + before[i] + at[i] * D;
                    if constexpr (V == 4) {
                        const float4 z = __ldcg(reinterpret_cast<const float4 *>(ps) + lane);
                        o[j][i][0] = z.x, o[j][i][1] = z.y, o[j][i][2] = z.z, o[j][i][3] = z.w;
                    } else {
                        const float2 z = __ldcg(reinterpret_cast<const float2 *>(ps) + lane);
                        o[j][i][0] = z.x, o[j][i][1] = z.y;
                    }
                }
        };
        for (int k0 = 0; k0 < np; k0 += 32) {
            load(k0);
            float m[RB], l[RB], f[RB];  // of piece k0 + lane
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const bool in = k0 + lane < np && at[i] >= 0;
                const float *ps = slot(in ? k0 + lane : 0) + before[i] + 128 * D + max(at[i], 0);
                m[i] = in ? __ldcg(ps) : -INFINITY;
                l[i] = in ? __ldcg(ps + 128) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                float mx = m[i];
#pragma unroll
                for (int s = 16; s >= 1; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float Mn = fmaxf(M[i], mx), old = M[i] == -INFINITY ? 0.f : fast_exp2(M[i] - Mn);
                f[i] = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - Mn);
                float sum = m[i] == -INFINITY ? l[i] : l[i] * f[i];
#pragma unroll
                for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
                L[i] = L[i] * old + sum;
                M[i] = Mn;
#pragma unroll
                for (int e = 0; e < V; ++e) acc[i][e] *= old;
            }
            for (int k = k0; k < min(k0 + 32, np); k += KB) {
                if (k > k0) load(k);
#pragma unroll
                for (int j = 0; j < KB; ++j)
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const float w = __shfl_sync(0xffffffffu, f[i], (k - k0 + j) & 31);  // 0 past the last piece
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[i][e] += w * o[j][i][e];
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            if (at[i] < 0) break;
            const float iv = L[i] == 0.f ? 0.f : 1.f / L[i];  // NaN stays NaN
            bool fine = true;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                acc[i][e] *= iv;
                fine = fine && fabsf(acc[i][e]) <= 3.4028234e38f;
            }
            const int g = g0 + i * step, ir = g / G, h = g - ir * G;
            if (!__all_sync(0xffffffffu, fine) &&
                reached_by_others<D>(a, u.s, u.kvh, max(u.base, 0), max(u.base + u.nr - 1, 0), max(u.base + ir, 0))) {
                redo_row<D>(a, u.s, u.kvh, u.r0 + ir, h, max(u.base + ir, 0));
                continue;
            }
            uint32_t *out = reinterpret_cast<uint32_t *>(a.out + (int64_t(u.r0 + ir) * a.Hq + u.kvh * G + h) * D) +
                            lane * (V / 2);
#pragma unroll
            for (int e = 0; e < V; e += 2) out[e / 2] = pack_bf16x2(acc[i][e], acc[i][e + 1]);
        }
    }
}

template <int D, bool PREFIX>
cudaError_t launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq, const SubsetArgs &a,
                     int grid, cudaStream_t stream) {
    const auto kernel = row_tiles_kernel<D, PREFIX>;
    const cudaError_t e = smem_once(reinterpret_cast<const void *>(kernel), RowCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const cudaError_t f = launch_pdl(kernel, dim3(grid), dim3(kWarpsRT * 32), RowCfg<D>::SMEM, stream, tk, tv, tq, a);
    if (PREFIX || f != cudaSuccess || !a.cuts) return f;
    // 32 rows per slice, by the average unit
    const int rows = std::min(2 * (kTileTok / a.G), (a.rows + a.nseq - 1) / a.nseq) * a.G;
    return launch_pdl(cut_join_kernel<D>, dim3(grid, (rows + 31) / 32), dim3(256), 0, stream, a);
}

}  // namespace

size_t row_tiles_slot_floats(int head_dim) { return size_t(2) * 128 * (head_dim + 2); }

cudaError_t launch_row_tiles(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq,
                             const SubsetArgs &args, int head_dim, int sms, cudaStream_t stream) {
    SubsetArgs a = args;
    a.min_items = kMinTiles;
    const int per_unit = 2 * (kTileTok / a.G);  // query rows
    if (int64_t(a.Hkv) * std::max(a.nseq, (a.rows + per_unit - 1) / per_unit) * 2 > sms) a.cuts = nullptr;
    const int grid = a.pt ? a.pgrid : sms;
    if (a.pt) return head_dim == 128 ? launch_t<128, true>(tk, tv, tq, a, grid, stream) : launch_t<64, true>(tk, tv, tq, a, grid, stream);
    return head_dim == 128 ? launch_t<128, false>(tk, tv, tq, a, grid, stream) : launch_t<64, false>(tk, tv, tq, a, grid, stream);
}

}  // namespace pa
