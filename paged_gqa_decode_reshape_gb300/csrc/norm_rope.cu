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
// Bound by HBM: a head is read and written once, 8 D flops for 4 D bytes.
//
//  * D / 16 lanes per head, each with two chunks of 8 dims whose rotation stays
//    in the lane (chunks c and c + R / 16; the unrotated ones two by two): 16-byte
//    loads and stores, the norm's sum over 3 (D = 64: 2) shuffles, no other exchange.
//  * A warp has the heads of one token, 4 (D = 64: 8) per step, and reads the
//    angles once for all its steps.
#include "common.cuh"
#include "kernels.h"
#include "step.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 2;  // per CTA
constexpr int kRopeSteps = 3;  // steps of heads of a warp

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

// V of the tokens of one 8-bit block that start with row t, for one KV head, by a warp:
// a row that continues the row before it in the same block leaves it to that one.
// Two neighbouring dims per lane and half; a block's 16 tokens are one store per dim.
__device__ __forceinline__ void write_v8(const RopeArgs &a, int64_t t, int h) {
    constexpr int D = 128, BS = kBlockSize;
    const int lane = threadIdx.x & 31;
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= a.NB * BS) return;
    const int o = int(slot % BS);
    const int64_t p = slot / BS;
    if (o > 0 && t > 0 && __ldg(a.slots + t - 1) == slot - 1) return;
    // rows t + 1 ... that follow in the block
    const bool next = lane > 0 && lane < BS - o && t + lane < a.T && __ldg(a.slots + t + lane) == slot + lane;
    const int n = __ffs(~(__ballot_sync(0xffffffffu, next) | 1u)) - 1;
    const float scale = __ldg(a.v_scale + h);
    uint8_t *dst = static_cast<uint8_t *>(a.vc) + (p * a.Hkv + h) * int64_t(D * BS);
    const uint16_t *src = a.v + t * a.vs + h * D;
    if (n == BS) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int d = half * 64 + 2 * lane;
            uint32_t x[BS];
#pragma unroll
            for (int i = 0; i < BS; ++i) x[i] = __ldg(reinterpret_cast<const uint32_t *>(src + i * a.vs + d));
            uint32_t lo[4], hi[4];  // word w: tokens 2 w, 2 w + 1, 2 w + 8, 2 w + 9
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                lo[w] = encode2(bf16_lo(x[2 * w]), bf16_lo(x[2 * w + 1]), scale) |
                        encode2(bf16_lo(x[2 * w + 8]), bf16_lo(x[2 * w + 9]), scale) << 16;
                hi[w] = encode2(bf16_hi(x[2 * w]), bf16_hi(x[2 * w + 1]), scale) |
                        encode2(bf16_hi(x[2 * w + 8]), bf16_hi(x[2 * w + 9]), scale) << 16;
            }
            *reinterpret_cast<uint4 *>(dst + d * BS) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint4 *>(dst + d * BS + BS) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
        return;
    }
    for (int i = 0; i < n; ++i) {
        const int at = 4 * (((o + i) & 7) >> 1) + 2 * ((o + i) >> 3) + ((o + i) & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int d = half * 64 + 2 * lane;
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t *>(src + i * a.vs + d));
            const uint32_t code = encode2(bf16_lo(x), bf16_hi(x), scale);
            dst[d * BS + at] = uint8_t(code & 0xffu);
            dst[d * BS + BS + at] = uint8_t(code >> 8);
        }
    }
}

// One warp: heads first .. first + NS * HPS - 1 (before `heads`) of token t, HPS at a time. Heads 0 .. Hq - 1 are the
// queries, then the keys, then (bf16 cache) the values. All of them are on their way before the position is asked for.
template <int D, bool INTER, RopeCache CACHE, int NS>
__device__ __forceinline__ void rope_heads(const RopeArgs &a, int64_t t, int first, int heads) {
    constexpr int LPH = D / 16, HPS = 32 / LPH, BS = kBlockSize;  // lanes per head, heads per step
    const int lane = threadIdx.x & 31, sub = lane % LPH, half = a.R / 2, rc = a.R / 16;  // rc: pairs of chunks
    // this lane's chunks of 8 dims
    const bool turns = sub < rc;
    const int c0 = turns ? (INTER ? 2 * sub : sub) : 2 * rc + 2 * (sub - rc);
    const int c1 = turns && !INTER ? sub + rc : c0 + 1;
    const uint16_t *const q = a.q + t * a.qs, *const k = a.k + t * a.ks - a.Hq * D,
                   *const v = a.v + t * a.vs - (a.Hq + a.Hkv) * D;  // head hh at hh * D
    uint4 r0[NS], r1[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int hh = first + s * HPS + lane / LPH;
        const uint16_t *src = (hh < a.Hq ? q : CACHE != kRopeBf16 || hh < a.Hq + a.Hkv ? k : v) + hh * D;
        r0[s] = r1[s] = make_uint4(0, 0, 0, 0);
        if (hh < heads) {
            r0[s] = __ldcg(reinterpret_cast<const uint4 *>(src) + c0);
            r1[s] = __ldcg(reinterpret_cast<const uint4 *>(src) + c1);
        }
    }
    int64_t slot = -1;
    if (CACHE != kRopeNone) {
        slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= a.NB * BS) slot = -1;
    }
    float2 cs[4], sn[4];
    const int f0 = INTER ? 8 * sub : 8 * c0;  // 8 frequencies: of pairs with chunk c1, or of both chunks
    int pos = 0;  // on axis lane % 4
    uint32_t axes = 0;  // of the lane's frequencies, two bits each
    if (a.axis) {
        pos = __ldg(a.pos + min(lane & 3, a.naxes - 1) * a.T + t);
        if (turns) {
            int ax[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ax[i] = __ldg(a.axis + f0 + i);
#pragma unroll
            for (int i = 0; i < 8; ++i) axes |= uint32_t(min(max(ax[i], 0), a.naxes - 1)) << (2 * i);
        }
    } else {
        pos = __ldg(a.pos + t);
    }
    auto row = [&](int i) -> const float * {  // of frequency f0 + i
        const int p = __shfl_sync(0xffffffffu, pos, (axes >> (2 * i)) & 3u);
        return a.table + min(max(int64_t(p), int64_t(0)), a.P - 1) * a.R + f0;
    };
    // four frequencies at once where every lane's are of one axis
    const uint32_t rest = axes & 0xffu, more = axes >> 8;
    if (__all_sync(0xffffffffu, rest == (rest & 3u) * 0x55u && more == (more & 3u) * 0x55u)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *from = row(4 * i) + 4 * i;
            if (!turns) continue;
            const float4 x = __ldg(reinterpret_cast<const float4 *>(from)), y = __ldg(reinterpret_cast<const float4 *>(from + half));
            cs[2 * i] = make_float2(x.x, x.y), cs[2 * i + 1] = make_float2(x.z, x.w);
            sn[2 * i] = make_float2(y.x, y.y), sn[2 * i + 1] = make_float2(y.z, y.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float *from = row(i) + i;
            const float c = turns ? __ldg(from) : 0.f, s = turns ? __ldg(from + half) : 0.f;
            if (i & 1) cs[i / 2].y = c, sn[i / 2].y = s;
            else cs[i / 2].x = c, sn[i / 2].x = s;
        }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int hh = first + s * HPS + lane / LPH;
        const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + a.Hkv;
        const int h = is_q ? hh : is_k ? hh - a.Hq : hh - a.Hq - a.Hkv;
        float2 x[4], y[4];
        unpack8(r0[s], x);
        unpack8(r1[s], y);
        const uint16_t *w = is_q ? a.qw : a.kw;
        if (a.qw || a.kw) {
            float2 m2 = mul2(x[0], x[0]), n2 = mul2(y[0], y[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                m2 = fma2(x[i], x[i], m2);
                n2 = fma2(y[i], y[i], n2);
            }
            float m = (m2.x + m2.y) + (n2.x + n2.y);
#pragma unroll
            for (int o = LPH / 2; o >= 1; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
            if (w) {
                const float f = rsqrtf(fmaf(m, 1.f / D, a.eps));
                float2 w0[4], w1[4];
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c0), w0);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c1), w1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = mul2(mul2(x[i], make_float2(f, f)), w0[i]);
                    y[i] = mul2(mul2(y[i], make_float2(f, f)), w1[i]);
                }
            }
        }
        if (INTER) {
            if (turns) {
                auto turn = [](float2 &p, float c, float s) { p = make_float2(p.x * c - p.y * s, p.y * c + p.x * s); };
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    turn(x[2 * i], cs[i].x, sn[i].x);
                    turn(x[2 * i + 1], cs[i].y, sn[i].y);
                    turn(y[2 * i], cs[2 + i].x, sn[2 + i].x);
                    turn(y[2 * i + 1], cs[2 + i].y, sn[2 + i].y);
                }
            }
        } else if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = x[i];
                x[i] = fma2(p, cs[i], mul2(y[i], make_float2(-sn[i].x, -sn[i].y)));
                y[i] = fma2(y[i], cs[i], mul2(p, sn[i]));
            }
        }
        if (hh >= heads) continue;
        if (CACHE == kRopeBf16 && !is_q && !is_k) {  // a value, as it is
            if (slot < 0) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.vc) + (slot * a.Hkv + h) * D);
            dst[c0] = r0[s];
            dst[c1] = r1[s];
            continue;
        }
        const uint4 lo = pack8(x), hi = pack8(y);
        if (is_q || a.ko) {
            uint4 *dst = reinterpret_cast<uint4 *>((is_q ? a.qo + t * a.qos : a.ko + t * a.kos) + h * D);
            dst[c0] = lo;
            dst[c1] = hi;
        }
        if (CACHE == kRopeNone || is_q || slot < 0) continue;
        if (CACHE == kRopeBf16) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.kc) + (slot * a.Hkv + h) * D);
            dst[c0] = lo;
            dst[c1] = hi;
        } else {
            const float scale = __ldg(a.k_scale + h);
            uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.kc) + (slot * a.Hkv + h) * D);
            dst[c0] = encode8(x, scale);
            dst[c1] = encode8(y, scale);
        }
    }
}

// parts: warps of a token, NS steps of heads each; the 8-bit V after them, a warp per token and KV head
template <int D, bool INTER, RopeCache CACHE, int NS>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeArgs a, int parts) {
    pdl_trigger();
    pdl_wait();
    const int heads = a.Hq + a.Hkv + (CACHE == kRopeBf16 ? a.Hkv : 0);
    const int all = parts + (CACHE == kRopeE4m3 ? a.Hkv : 0);
    const int64_t w = int64_t(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int64_t t = w / all;
    const int part = int(w - t * all);
    if (t >= a.T) return;
    if (CACHE == kRopeE4m3 && part >= parts) {
        write_v8(a, t, part - parts);
        return;
    }
    rope_heads<D, INTER, CACHE, NS>(a, t, part * NS * (512 / D), heads);
}

template <int D, bool INTER, RopeCache CACHE, int NS>
cudaError_t launch_n(const RopeArgs &a, cudaStream_t stream) {
    constexpr int per = NS * (512 / D);
    const int heads = a.Hq + a.Hkv + (CACHE == kRopeBf16 ? a.Hkv : 0), parts = (heads + per - 1) / per;
    const int64_t warps = a.T * (parts + (CACHE == kRopeE4m3 ? a.Hkv : 0));
    return launch_pdl(norm_rope_kernel<D, INTER, CACHE, NS>, dim3(unsigned((warps + kRopeWarps - 1) / kRopeWarps)),
                      dim3(kRopeWarps * 32), 0, stream, a, parts);
}

template <int D, bool INTER, RopeCache CACHE>
cudaError_t launch_t(const RopeArgs &a, cudaStream_t stream) {
    const int steps = (a.Hq + 2 * a.Hkv + 512 / D - 1) / (512 / D);
    return a.T * steps < 4096 ? launch_n<D, INTER, CACHE, 1>(a, stream) : launch_n<D, INTER, CACHE, kRopeSteps>(a, stream);
}

template <int D, bool INTER>
cudaError_t launch_c(const RopeArgs &a, RopeCache cache, cudaStream_t stream) {
    if (cache == kRopeNone) return launch_t<D, INTER, kRopeNone>(a, stream);
    if (cache == kRopeBf16) return launch_t<D, INTER, kRopeBf16>(a, stream);
    if constexpr (D == 128) return launch_t<D, INTER, kRopeE4m3>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs &a, int head_dim, bool interleaved, RopeCache cache, cudaStream_t stream) {
    if (head_dim == 128) return interleaved ? launch_c<128, true>(a, cache, stream) : launch_c<128, false>(a, cache, stream);
    return interleaved ? launch_c<64, true>(a, cache, stream) : launch_c<64, false>(a, cache, stream);
}

}  // namespace pa
