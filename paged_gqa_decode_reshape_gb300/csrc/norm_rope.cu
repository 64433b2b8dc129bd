// norm_rope.cu -- queries and keys on their way from the projection to the
// attention (sm_103a): the norm of every head, the rotation by position, and the
// write of K and V into the paged cache, in one pass.
//
// Per head x of q (weights w_q) and k (w_k):
//   y_d = x_d / sqrt(mean_d x_d^2 + eps) * w_d          (without weights: y = x)
//   y'_i = y_i cos - y_j sin,   y'_j = y_j cos + y_i sin
// for the R / 2 pairs (i, j) = (i, i + R / 2), interleaved (2 i, 2 i + 1), with cosine
// and sine i of the table's row positions[axis_i][t]; the dims from R on stay. All
// in fp32, rounded once to bf16 or (keys and values of an 8-bit cache) to the E4M3
// code of the value over its head's scale.
//
// Bound by HBM: a head is read and written once, 8 D flops for 4 D bytes. Measured (28 / 4 heads of 128): 8191 tokens
// (156 MB) 28.0 us = 5.6 TB/s, 82 % of the measured copy rate; one token 1.8 us, 128 tokens over the 8-bit cache 3.0:
// a launch and two dependent reads (position, angles).
//
//  * D / 16 lanes per head, each with two chunks of 8 dims whose rotation stays
//    in the lane (chunks c and c + R / 16; the unrotated ones two by two): 16-byte
//    loads and stores, the norm's sum over 3 (D = 64: 2) shuffles, no other exchange.
//  * A step is 4 (D = 64: 8) heads of a token, 1 KB, all queries, keys or values. Weights and
//    angles meet once per token and kind: x' = (x A + y B) f with A = w cos, B = -w sin.
//  * Small calls: a warp per step, its loads issued before the token's position is known.
//  * Many tokens: a range of steps per warp (the ring, below).
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "step.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 2;  // per CTA of small calls

// The E4M3 code of fl32(x / scale), nearest with ties to even, saturated; one NaN code.
__device__ __forceinline__ uint32_t encode2(float x, float y, float scale) {
    const float a = __fdiv_rn(x, scale), b = __fdiv_rn(y, scale);
    uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    if (a != a) pair = (pair & 0xff00u) | 0x7fu;
    if (b != b) pair = (pair & 0x00ffu) | 0x7f00u;
    return pair & 0xffffu;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float2 (&x)[4]) {
    x[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
    x[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
    x[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z));
    x[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ uint2 encode8(const float2 (&x)[4], float scale) {
    return make_uint2(encode2(x[0].x, x[0].y, scale) | encode2(x[1].x, x[1].y, scale) << 16,
                      encode2(x[2].x, x[2].y, scale) | encode2(x[3].x, x[3].y, scale) << 16);
}

// V of n tokens from row t on, in slots `slot`, ... of one 8-bit block, for a half of KV head h's dims, by a warp: two neighbouring
// dims per lane, all tokens on their way at once; a block's 16 tokens are one store per dim.
__device__ __forceinline__ void write_v8(const RopeArgs &a, int64_t t, int64_t slot, int n, int h, int half) {
    constexpr int D = 128, BS = kBlockSize;
    const int o = int(slot % BS), d = half * 64 + 2 * int(threadIdx.x & 31);
    uint32_t x[BS];
#pragma unroll
    for (int i = 0; i < BS; ++i)
        x[i] = i < n ? __ldg(reinterpret_cast<const uint32_t *>(a.v + (t + i) * a.vs + h * D + d)) : 0u;
    const float scale = __ldg(a.v_scale + h);
    uint8_t *dst = static_cast<uint8_t *>(a.vc) + (slot / BS * a.Hkv + h) * int64_t(D * BS) + d * BS;
    if (n == BS) {
        uint32_t lo[4], hi[4];  // word w: tokens 2 w, 2 w + 1, 2 w + 8, 2 w + 9
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            lo[w] = encode2(bf16_lo(x[2 * w]), bf16_lo(x[2 * w + 1]), scale) |
                    encode2(bf16_lo(x[2 * w + 8]), bf16_lo(x[2 * w + 9]), scale) << 16;
            hi[w] = encode2(bf16_hi(x[2 * w]), bf16_hi(x[2 * w + 1]), scale) |
                    encode2(bf16_hi(x[2 * w + 8]), bf16_hi(x[2 * w + 9]), scale) << 16;
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(dst + BS) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < BS - 1; ++i) {
        if (i >= n) break;
        const int k = o + i, at = 4 * ((k & 7) >> 1) + 2 * (k >> 3) + (k & 1);
        const uint32_t code = encode2(bf16_lo(x[i]), bf16_hi(x[i]), scale);
        dst[at] = uint8_t(code & 0xffu);
        dst[BS + at] = uint8_t(code >> 8);
    }
}

// V of the rows t .. t + 31 for a half of KV head h's dims, by a warp: rows whose slots follow each other in a block go together, by the
// first of them (n_rows 1: of row t, if it is such a first one). A run may go on behind the 32.
template <int LONE>
__device__ __forceinline__ void write_v8_runs(const RopeArgs &a, int64_t t, int n_rows, int h, int half) {
    constexpr int BS = kBlockSize;
    const int lane = threadIdx.x & 31;
    auto slot_at = [&](int64_t r) -> int64_t {
        const int64_t s = r >= 0 && r < a.T ? __ldg(a.slots + r) : -1;
        return s < a.NB * BS ? s : -1;
    };
    // lane l: of rows t + l and t + 31 + l (the first 15 rows behind), and of the row before
    const int64_t s0 = slot_at(t + lane), s1 = lane > 0 && lane < BS ? slot_at(t + 31 + lane) : -1, before = slot_at(t - 1);
    int64_t prev = __shfl_up_sync(0xffffffffu, s0, 1), up = __shfl_up_sync(0xffffffffu, s1, 1);
    if (lane == 0) prev = before;
    const int64_t last = __shfl_sync(0xffffffffu, s0, 31);
    if (lane == 1) up = last;
    // bit l: row t + l, t + 31 + l goes on where the row before it is, in the same block
    const uint32_t on0 = __ballot_sync(0xffffffffu, s0 >= 0 && s0 % BS > 0 && prev == s0 - 1);
    const uint32_t on1 = __ballot_sync(0xffffffffu, s1 >= 0 && s1 % BS > 0 && up == s1 - 1);
    const uint64_t on = on0 | uint64_t(on1 >> 1) << 32;
    uint32_t first = __ballot_sync(0xffffffffu, s0 >= 0 && lane < n_rows) & ~on0, lone = first & ~uint32_t(on >> 1);
    for (first &= ~lone; first; first &= first - 1) {
        const int l = __ffs(first) - 1;
        const int n = __ffsll(int64_t(~(on >> (l + 1))));
        write_v8(a, t + l, __shfl_sync(0xffffffffu, s0, l), n, h, half);
    }
    // rows that are alone in their run: LONE of them on their way at once
    const int d = half * 64 + 2 * lane;
    const float scale = __ldg(a.v_scale + h);
#pragma unroll 1
    while (lone) {
        uint32_t x[LONE];
        const uint32_t these = lone;
#pragma unroll
        for (int i = 0; i < LONE; ++i) {
            const int l = __ffs(lone) - 1;
            x[i] = lone ? __ldg(reinterpret_cast<const uint32_t *>(a.v + (t + l) * a.vs + h * 128 + d)) : 0u;
            lone &= lone - 1;
        }
        uint32_t rest = these;
#pragma unroll
        for (int i = 0; i < LONE; ++i) {
            if (!rest) break;
            const int64_t slot = __shfl_sync(0xffffffffu, s0, __ffs(rest) - 1);
            const int o = int(slot % BS);
            uint8_t *dst = static_cast<uint8_t *>(a.vc) + (slot / BS * a.Hkv + h) * int64_t(128 * BS) + d * BS +
                           4 * ((o & 7) >> 1) + 2 * (o >> 3) + (o & 1);
            const uint32_t code = encode2(bf16_lo(x[i]), bf16_hi(x[i]), scale);
            dst[0] = uint8_t(code & 0xffu);
            dst[BS] = uint8_t(code >> 8);
            rest &= rest - 1;
        }
    }
}

// What a lane has of a step: of head lane / LPH the chunks c0 and c1 of 8 dims, which are rotated against each other (INTER:
// within themselves) where turns, by its 8 frequencies from f0 on; o0 and o1 are the chunks' elements in the step.
template <int D, bool INTER>
struct Lane {
    static constexpr int LPH = D / 16, HPS = 32 / LPH;  // lanes per head, heads per step
    bool turns;
    int c0, c1, f0, o0, o1;
    __device__ __forceinline__ Lane(int R) {
        const int lane = threadIdx.x & 31, sub = lane % LPH, rc = R / 16;  // rc: pairs of chunks
        turns = sub < rc;
        c0 = turns ? (INTER ? 2 * sub : sub) : 2 * rc + 2 * (sub - rc);
        c1 = turns && !INTER ? sub + rc : c0 + 1;
        f0 = INTER ? 8 * sub : 8 * c0;
        o0 = lane / LPH * D + c0 * 8;
        o1 = lane / LPH * D + c1 * 8;
    }
};

// A token's steps: queries, then keys, then (bf16 cache) values
struct Steps {
    int q, qk, all;
    template <int HPS, RopeCache CACHE>
    __host__ __device__ static Steps of(int Hq, int Hkv) {
        const int q = (Hq + HPS - 1) / HPS, k = (Hkv + HPS - 1) / HPS;
        return {q, q + k, q + k + (CACHE == kRopeBf16 ? k : 0)};
    }
    __device__ __forceinline__ int kind(int step) const { return step < q ? 0 : step < qk ? 1 : 2; }
    __device__ __forceinline__ int within(int step) const { return step < q ? step : step < qk ? step - q : step - qk; }
};

// The norm's weights of a lane's chunks: ones without a norm.
struct Weights {
    uint4 w0, w1;
    template <int D, bool INTER>
    __device__ __forceinline__ Weights(const uint16_t *w, const Lane<D, INTER> &me) {
        w0 = w1 = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        if (w) {
            w0 = __ldg(reinterpret_cast<const uint4 *>(w) + me.c0);
            w1 = __ldg(reinterpret_cast<const uint4 *>(w) + me.c1);
        }
    }
};

// Weights and angles of a lane's dims: x' = x A + u B and y' = y C + z E, with x of chunk c0, y of chunk c1, u = y and z = x
// (INTER: the other of the pair). Each product of a weight and a cosine or sine is rounded once more in fp32.
struct Turn {
    float2 A[4], B[4], C[4], E[4];
    template <int D, bool INTER>
    __device__ __forceinline__ void set(const Weights &w, const Lane<D, INTER> &me, const float (&c)[8], const float (&s)[8]) {
        unpack8(w.w0, A);
        unpack8(w.w1, C);
        if (!me.turns) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = A[i], w1 = C[i];
            if (INTER) {
                A[i] = make_float2(v.x * c[i], v.y * c[i]);
                B[i] = make_float2(-(v.y * s[i]), v.x * s[i]);
                C[i] = make_float2(w1.x * c[4 + i], w1.y * c[4 + i]);
                E[i] = make_float2(-(w1.y * s[4 + i]), w1.x * s[4 + i]);
            } else {
                A[i] = make_float2(v.x * c[2 * i], v.y * c[2 * i + 1]);
                B[i] = make_float2(-(w1.x * s[2 * i]), -(w1.y * s[2 * i + 1]));
                C[i] = make_float2(w1.x * c[2 * i], w1.y * c[2 * i + 1]);
                E[i] = make_float2(v.x * s[2 * i], v.y * s[2 * i + 1]);
            }
        }
    }
};

// Step `at` of a kind of token t: norm, rotation and stores of what the lane has loaded. A warp calls it together.
template <int D, bool INTER, RopeCache CACHE>
__device__ __forceinline__ void finish_step(const RopeArgs &a, int64_t t, int kind, int at, int64_t slot, const Lane<D, INTER> &me,
                                            const Turn &turn, const uint4 &r0, const uint4 &r1) {
    using L = Lane<D, INTER>;
    const bool in = at * L::HPS + int(threadIdx.x & 31) / L::LPH < (kind == 0 ? a.Hq : a.Hkv);
    const int64_t step = int64_t(at) * (L::HPS * D);  // first element of the row
    auto put = [&](uint16_t *row, const uint4 &lo, const uint4 &hi) {
        *reinterpret_cast<uint4 *>(row + step + me.o0) = lo;
        *reinterpret_cast<uint4 *>(row + step + me.o1) = hi;
    };
    if (CACHE == kRopeBf16 && kind == 2) {  // values, as they are
        if (in && slot >= 0) put(static_cast<uint16_t *>(a.vc) + slot * a.Hkv * D, r0, r1);
        return;
    }
    float2 x[4], y[4];
    unpack8(r0, x);
    unpack8(r1, y);
    float f = 1.f;
    if (kind == 0 ? a.qw : a.kw) {
        float2 m2 = mul2(x[0], x[0]), n2 = mul2(y[0], y[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            m2 = fma2(x[i], x[i], m2);
            n2 = fma2(y[i], y[i], n2);
        }
        m2 = add2(m2, n2);
        float m = m2.x + m2.y;
#pragma unroll
        for (int o = L::LPH / 2; o >= 1; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        f = rsqrtf(fmaf(m, 1.f / D, a.eps));
    }
    const float2 ff = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p = mul2(x[i], ff), q = mul2(y[i], ff);
        const float2 u = INTER ? make_float2(p.y, p.x) : q, z = INTER ? make_float2(q.y, q.x) : p;
        p = mul2(p, turn.A[i]);
        q = mul2(q, turn.C[i]);
        x[i] = me.turns ? fma2(u, turn.B[i], p) : p;
        y[i] = me.turns ? fma2(z, turn.E[i], q) : q;
    }
    if (!in) return;
    const uint4 lo = pack8(x), hi = pack8(y);
    if (kind == 0) {
        put(a.qo + t * a.qos, lo, hi);
        return;
    }
    if (a.ko) put(a.ko + t * a.kos, lo, hi);
    if (CACHE == kRopeNone || slot < 0) return;
    if (CACHE == kRopeBf16) {
        put(static_cast<uint16_t *>(a.kc) + slot * a.Hkv * D, lo, hi);
    } else {
        const float scale = __ldg(a.k_scale + at * L::HPS + int(threadIdx.x & 31) / L::LPH);
        uint8_t *row = static_cast<uint8_t *>(a.kc) + slot * a.Hkv * D + step;
        *reinterpret_cast<uint2 *>(row + me.o0) = encode8(x, scale);
        *reinterpret_cast<uint2 *>(row + me.o1) = encode8(y, scale);
    }
}

__device__ __forceinline__ const uint16_t *row_of(const RopeArgs &a, int64_t t, int kind) {
    return kind == 0 ? a.q + t * a.qs : kind == 1 ? a.k + t * a.ks : a.v + t * a.vs;
}

// ---- small calls: a warp per step; the 8-bit V after a token's steps, a warp per token and half a KV head
template <int D, bool INTER, RopeCache CACHE>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeArgs a) {
    using L = Lane<D, INTER>;
    constexpr int BS = kBlockSize;
    pdl_trigger();
    pdl_wait();
    const Steps steps = Steps::of<L::HPS, CACHE>(a.Hq, a.Hkv);
    const int all = steps.all + (CACHE == kRopeE4m3 ? 2 * a.Hkv : 0);
    const int64_t w = int64_t(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5), t = w / all;
    const int part = int(w - t * all);
    if (t >= a.T) return;
    if (CACHE == kRopeE4m3 && part >= steps.all) {
        write_v8_runs<1>(a, t, 1, (part - steps.all) >> 1, (part - steps.all) & 1);
        return;
    }
    const L me(a.R);
    const int lane = threadIdx.x & 31, half = a.R / 2, kind = steps.kind(part), at = steps.within(part);
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (at * L::HPS + lane / L::LPH < (kind == 0 ? a.Hq : a.Hkv)) {
        const uint16_t *src = row_of(a, t, kind) + at * (L::HPS * D);
        r0 = __ldcg(reinterpret_cast<const uint4 *>(src + me.o0));
        r1 = __ldcg(reinterpret_cast<const uint4 *>(src + me.o1));
    }
    int64_t slot = -1;
    if (CACHE != kRopeNone && kind > 0) {
        slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= a.NB * BS) slot = -1;
    }
    Turn turn;
    if (kind < 2) {
        float cs[8], sn[8];
        int pos = 0;  // on axis lane % 4
        uint32_t axes = 0;  // of the lane's frequencies, two bits each
        if (a.axis) {
            pos = __ldg(a.pos + min(lane & 3, a.naxes - 1) * a.T + t);
            if (me.turns) {
                int ax[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ax[i] = __ldg(a.axis + me.f0 + i);
#pragma unroll
                for (int i = 0; i < 8; ++i) axes |= uint32_t(min(max(ax[i], 0), a.naxes - 1)) << (2 * i);
            }
        } else {
            pos = __ldg(a.pos + t);
        }
        auto row = [&](int i) -> const float * {  // of frequency f0 + i
            const int p = __shfl_sync(0xffffffffu, pos, (axes >> (2 * i)) & 3u);
            return a.table + min(max(int64_t(p), int64_t(0)), a.P - 1) * a.R + me.f0;
        };
        // four frequencies at once where every lane's are of one axis
        const uint32_t rest = axes & 0xffu, more = axes >> 8;
        if (__all_sync(0xffffffffu, rest == (rest & 3u) * 0x55u && more == (more & 3u) * 0x55u)) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float *from = row(i) + i;
                if (!me.turns) continue;
                const float4 x = __ldg(reinterpret_cast<const float4 *>(from)), y = __ldg(reinterpret_cast<const float4 *>(from + half));
                cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
                sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *from = row(i) + i;
                cs[i] = me.turns ? __ldg(from) : 0.f, sn[i] = me.turns ? __ldg(from + half) : 0.f;
            }
        }
        turn.set(Weights(kind == 0 ? a.qw : a.kw, me), me, cs, sn);
    }
    finish_step<D, INTER, CACHE>(a, t, kind, at, slot, me, turn, r0, r1);
}

// ---- many tokens: a warp per range of steps, kRingStages of them on their way in shared memory
//
// The heads come by asynchronous copies that hold no registers, 8 KB per warp and 128 KB per SM in flight, angles and
// slot of a token beside the first of its steps, its position a token ahead. The 8-bit V is for warps of its own. What is left
// is issue: two thirds of the slots (8191 tokens 28.0 us; the weights read again at every token 28.7, with that 12 warps 30.8,
// 20 warps of 6 stages, whose registers spill, 35.4; three steps per warp, each loading its own to registers, 33.4).
constexpr int kRingWarps = 16, kRingStages = 8;
// E4M3: warps of a CTA for V, beside the others: 8191 tokens (148 MB) 33.4 us = 4.4 TB/s, 65 % of the measured copy rate (one
// after the other in every warp 38.2)
constexpr int kRingV8Warps = 4;
// Warps of the small form from which on the ring takes over. Ring and small, 28 / 4 heads of 128: 300 tokens 3.3 and 3.0 us,
// 400 3.5 and 3.4, 500 3.5 and 4.2, 1000 4.7 and 6.5; 8-bit 400 5.5 and 4.9, 600 5.0 and 6.3, 1000 6.1 and 9.5, 1000 of as many
// sequences 6.5 and 9.8.
constexpr int64_t kRingFrom = 4096, kRingFromE4m3 = 8192;

struct RingCfg {
    static constexpr int STEP = 1024;              // bytes of a step's heads
    static constexpr int SIDE = 128 * 4 + 16;      // cosines and sines, slot
    static constexpr int WARP = kRingStages * STEP + (kRingStages + 1) * SIDE;
    static constexpr size_t SMEM = size_t(kRingWarps) * WARP;
    static_assert(kRingStages <= 8, "4 lanes per token of the first steps");
    static_assert(WARP % 16 == 0 && SMEM <= 227 * 1024, "aligned copies, an SM's shared memory");
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int D, bool INTER, RopeCache CACHE>
__global__ void __launch_bounds__(kRingWarps * 32, 1) norm_rope_ring_kernel(const RopeArgs a) {
    using C = RingCfg;
    using L = Lane<D, INTER>;
    constexpr int BS = kBlockSize;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.R / 2;
    const uint8_t *const mem = ring_smem + warp * C::WARP;
    const uint32_t ring = smem_u32(mem), sides = ring + kRingStages * C::STEP;
    const L me(a.R);
    const Steps steps = Steps::of<L::HPS, CACHE>(a.Hq, a.Hkv);
    constexpr int VW = CACHE == kRopeE4m3 ? kRingV8Warps : 0, RW = kRingWarps - VW;
    const int64_t total = a.T * steps.all, W = int64_t(gridDim.x) * RW, w = int64_t(blockIdx.x) * RW + warp;
    const int64_t i0 = total / W * w + min(w, total % W), i1 = i0 + total / W + (w < total % W);
    pdl_trigger();
    pdl_wait();
    if (CACHE == kRopeE4m3 && warp >= RW) {  // 16 rows of half a KV head at a time
        const int64_t n = (a.T + 15) / 16 * 2 * a.Hkv;
#pragma unroll 1
        for (int64_t u = int64_t(blockIdx.x) * VW + warp - RW; u < n; u += int64_t(gridDim.x) * VW) {
            const int part = int(u % (2 * a.Hkv));
            write_v8_runs<8>(a, u / (2 * a.Hkv) * 16, 16, part >> 1, part & 1);
        }
        return;
    }
    // the copies' side: the next step, its token, and that token's place among the warp's
    int64_t ct = i0 / steps.all;
    int left = int(i1 - i0), cstep = int(i0 - ct * steps.all), cside = 0, cstage = 0;
    // axes of frequencies lane and lane + 32; by four, of the lane's four floats of a row, where all fours are of one axis each
    int ax0 = 0, ax1 = 0;
    bool by_four = true;
    if (a.axis) {
        if (lane < half) ax0 = min(max(__ldg(a.axis + lane), 0), a.naxes - 1);
        if (lane + 32 < half) ax1 = min(max(__ldg(a.axis + lane + 32), 0), a.naxes - 1);
        const int f0 = __shfl_sync(0xffffffffu, ax0, lane & ~3), f1 = __shfl_sync(0xffffffffu, ax1, lane & ~3);
        by_four = __all_sync(0xffffffffu, ax0 == f0 && ax1 == f1);
        if (by_four) {
            const int f = lane * 4 < a.R ? lane * 4 % half : 0;
            const int b0 = __shfl_sync(0xffffffffu, ax0, f & 31), b1 = __shfl_sync(0xffffffffu, ax1, f & 31);
            ax0 = f < 32 ? b0 : b1;
        }
    }
    auto position = [&](int64_t t) -> int {  // with axes: on axis lane % 4
        return t < a.T ? __ldg(a.pos + (a.axis ? min(lane & 3, a.naxes - 1) * a.T : 0) + t) : 0;
    };
    // positions of the first kRingStages tokens, 4 lanes each, later of the next token (the first 4 lanes)
    int pos = position(ct + (lane >> 2));
    auto copy_side = [&](int64_t t, int side, int j) {  // j: the token's lanes of pos
        const uint32_t to = sides + side * C::SIDE;
        auto from = [&](int p) { return a.table + min(max(int64_t(p), int64_t(0)), a.P - 1) * a.R; };
        if (by_four) {
            const int p = __shfl_sync(0xffffffffu, pos, 4 * j + ax0);
            if (lane * 4 < a.R) copy_async<16>(to + lane * 16, from(p) + lane * 4);
        } else {
            const int p0 = __shfl_sync(0xffffffffu, pos, 4 * j + ax0), p1 = __shfl_sync(0xffffffffu, pos, 4 * j + ax1);
            if (lane < half) {
                copy_async<4>(to + lane * 4, from(p0) + lane);
                copy_async<4>(to + (half + lane) * 4, from(p0) + half + lane);
            }
            if (lane + 32 < half) {
                copy_async<4>(to + (lane + 32) * 4, from(p1) + lane + 32);
                copy_async<4>(to + (half + lane + 32) * 4, from(p1) + half + lane + 32);
            }
        }
        if (CACHE != kRopeNone && lane == 0) copy_async<8>(to + 512, a.slots + t);
    };
    auto copy_heads = [&]() {  // of the next step
        const int kind = steps.kind(cstep), first = steps.within(cstep) * (L::HPS * D) + lane * 8;
        const int end = (kind == 0 ? a.Hq : a.Hkv) * D;
        const uint16_t *src = row_of(a, ct, kind) + first;
        const uint32_t to = ring + cstage * C::STEP + lane * 16;
        if (first < end) copy_async<16>(to, src);
        if (first + 256 < end) copy_async<16>(to + 512, src + 256);
        --left;
        cstage = cstage + 1 < kRingStages ? cstage + 1 : 0;
        if (++cstep == steps.all) {
            cstep = 0;
            ++ct;
            cside = cside + 1 <= kRingStages ? cside + 1 : 0;
        }
    };
    int64_t t = ct;
    int step = cstep, side = 0, stage = 0;
    // the first steps' heads, before anything waits for a position
    for (int s = 0; s < kRingStages && left > 0; ++s) copy_heads();
    if (i0 < i1) {
#pragma unroll 1
        for (int64_t u = t; u < ct || (u == ct && cstep > 0); ++u) copy_side(u, int(u - t), int(u - t));
        pos = position(ct + (cstep > 0));
    }
    copy_commit();
#pragma unroll 1
    for (int s = 1; s < kRingStages; ++s) copy_commit();
    const Weights wq(a.qw, me), wk(a.kw, me);
    Turn turn;
    bool known = false;  // turn is of this token and kind
    int64_t slot = -1;
#pragma unroll 1
    for (int64_t n = i1 - i0; n > 0; --n) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRingStages - 1) : "memory");
        __syncwarp();
        const uint16_t *at = reinterpret_cast<const uint16_t *>(mem + stage * C::STEP);
        const uint4 r0 = *reinterpret_cast<const uint4 *>(at + me.o0), r1 = *reinterpret_cast<const uint4 *>(at + me.o1);
        const int kind = steps.kind(step);
        if (!known) {
            const uint8_t *sd = mem + kRingStages * C::STEP + side * C::SIDE;
            if (CACHE != kRopeNone) {
                slot = *reinterpret_cast<const int64_t *>(sd + 512);
                if (slot < 0 || slot >= a.NB * BS) slot = -1;
            }
            if (kind < 2) {
                float cs[8], sn[8];
                if (me.turns) {
                    const float *f = reinterpret_cast<const float *>(sd) + me.f0;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(f + e), y = *reinterpret_cast<const float4 *>(f + half + e);
                        cs[e] = x.x, cs[e + 1] = x.y, cs[e + 2] = x.z, cs[e + 3] = x.w;
                        sn[e] = y.x, sn[e + 1] = y.y, sn[e + 2] = y.z, sn[e + 3] = y.w;
                    }
                }
                turn.set(kind == 0 ? wq : wk, me, cs, sn);
            }
            known = true;
        }
        __syncwarp();  // the stage has been read
        if (left > 0) {
            const bool fresh = cstep == 0;
            const int64_t u = ct;
            const int place = cside;
            copy_heads();
            if (fresh) {
                copy_side(u, place, 0);
                pos = position(u + 1);
            }
        }
        copy_commit();
        finish_step<D, INTER, CACHE>(a, t, kind, steps.within(step), slot, me, turn, r0, r1);
        stage = stage + 1 < kRingStages ? stage + 1 : 0;
        ++step;
        if (step == steps.q || step == steps.qk) known = false;
        if (step == steps.all) {
            known = false;
            step = 0;
            ++t;
            side = side + 1 <= kRingStages ? side + 1 : 0;
        }
    }
}

template <int D, bool INTER, RopeCache CACHE>
cudaError_t launch_t(const RopeArgs &a, int sms, cudaStream_t stream) {
    const int64_t warps = a.T * (Steps::of<Lane<D, INTER>::HPS, CACHE>(a.Hq, a.Hkv).all + (CACHE == kRopeE4m3 ? 2 * a.Hkv : 0));
    if (warps >= (CACHE == kRopeE4m3 ? kRingFromE4m3 : kRingFrom)) {
        const auto kernel = norm_rope_ring_kernel<D, INTER, CACHE>;
        const cudaError_t e = smem_once(reinterpret_cast<const void *>(kernel), RingCfg::SMEM);
        return e != cudaSuccess ? e : launch_soon(kernel, dim3(sms), dim3(kRingWarps * 32), RingCfg::SMEM, stream, 1, a);
    }
    return launch_soon(norm_rope_kernel<D, INTER, CACHE>, dim3(unsigned((warps + kRopeWarps - 1) / kRopeWarps)), dim3(kRopeWarps * 32),
                       0, stream, 1, a);
}

template <int D, bool INTER>
cudaError_t launch_c(const RopeArgs &a, RopeCache cache, int sms, cudaStream_t stream) {
    if (cache == kRopeNone) return launch_t<D, INTER, kRopeNone>(a, sms, stream);
    if (cache == kRopeBf16) return launch_t<D, INTER, kRopeBf16>(a, sms, stream);
    if constexpr (D == 128) return launch_t<D, INTER, kRopeE4m3>(a, sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs &a, int head_dim, bool interleaved, RopeCache cache, int sms, cudaStream_t stream) {
    if (head_dim == 128) return interleaved ? launch_c<128, true>(a, cache, sms, stream) : launch_c<128, false>(a, cache, sms, stream);
    return interleaved ? launch_c<64, true>(a, cache, sms, stream) : launch_c<64, false>(a, cache, sms, stream);
}

}  // namespace pa
