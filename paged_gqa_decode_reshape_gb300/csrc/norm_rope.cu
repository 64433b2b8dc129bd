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

namespace pa {
namespace {

constexpr int kRopeWarps = 4;  // per CTA

// The E4M3 code of fl32(x / scale), nearest with ties to even, saturated; one NaN code.
__device__ __forceinline__ uint32_t encode2(float x, float y, float scale) {
    const float a = __fdiv_rn(x, scale), b = __fdiv_rn(y, scale);
    uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    if (a != a) pair = (pair & 0xff00u) | 0x7fu;
    if (b != b) pair = (pair & 0x00ffu) | 0x7f00u;
    return pair & 0xffffu;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
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

// One warp: heads [first, last) of token t. Heads 0 .. Hq - 1 are the queries, then the
// keys, then (bf16 cache) the values.
template <int D, bool INTER, RopeCache CACHE>
__device__ __forceinline__ void rope_heads(const RopeArgs &a, int64_t t, int first, int last) {
    constexpr int LPH = D / 16, HPS = 32 / LPH, BS = kBlockSize;  // lanes per head, heads per step
    const int lane = threadIdx.x & 31, sub = lane % LPH, half = a.R / 2, rc = a.R / 16;  // rc: pairs of chunks
    // this lane's chunks of 8 dims
    const bool turns = sub < rc;
    const int c0 = turns ? (INTER ? 2 * sub : sub) : 2 * rc + 2 * (sub - rc);
    const int c1 = turns && !INTER ? sub + rc : c0 + 1;
    float cs[8], sn[8];
    if (turns) {
        const int f0 = INTER ? 8 * sub : 8 * c0;  // 8 frequencies: of pairs with chunk c1, or of both chunks
        if (a.axis == nullptr) {
            const int64_t row = min(max(int64_t(__ldg(a.pos + t)), int64_t(0)), a.P - 1);
            const float4 *at = reinterpret_cast<const float4 *>(a.table + row * a.R + f0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = __ldg(at + i), y = __ldg(at + i + half / 4);
                cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ax = min(max(__ldg(a.axis + f0 + i), 0), a.naxes - 1);
                const int64_t row = min(max(int64_t(__ldg(a.pos + ax * a.T + t)), int64_t(0)), a.P - 1);
                cs[i] = __ldg(a.table + row * a.R + f0 + i);
                sn[i] = __ldg(a.table + row * a.R + half + f0 + i);
            }
        }
    }
    int64_t slot = -1;
    if (CACHE != kRopeNone) {
        slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= a.NB * BS) slot = -1;
    }
#pragma unroll 3
    for (int h0 = first; h0 < last; h0 += HPS) {
        const int hh = h0 + lane / LPH;
        const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + a.Hkv;
        const int h = is_q ? hh : is_k ? hh - a.Hq : hh - a.Hq - a.Hkv;
        // a key or value without a place is not read
        const bool in = hh < last && (is_q || (is_k && a.ko) || slot >= 0);
        const uint16_t *src = (is_q ? a.q + t * a.qs : is_k ? a.k + t * a.ks : a.v + t * a.vs) + h * D;
        uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
        if (in) {
            r0 = __ldcg(reinterpret_cast<const uint4 *>(src) + c0);
            r1 = __ldcg(reinterpret_cast<const uint4 *>(src) + c1);
        }
        const bool is_v = CACHE == kRopeBf16 && !is_q && !is_k;
        float x[8], y[8];
        unpack8(r0, x);
        unpack8(r1, y);
        const uint16_t *w = is_q ? a.qw : a.kw;
        if (a.qw || a.kw) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
#pragma unroll
            for (int o = LPH / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (w) {
                const float f = __frsqrt_rn(fmaf(s, 1.f / D, a.eps));
                float w0[8], w1[8];
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c0), w0);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c1), w1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = x[i] * f * w0[i];
                    y[i] = y[i] * f * w1[i];
                }
            }
        }
        if (turns) {
            if (INTER) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = x[2 * i], q = x[2 * i + 1], u = y[2 * i], v = y[2 * i + 1];
                    x[2 * i] = p * cs[i] - q * sn[i];
                    x[2 * i + 1] = q * cs[i] + p * sn[i];
                    y[2 * i] = u * cs[4 + i] - v * sn[4 + i];
                    y[2 * i + 1] = v * cs[4 + i] + u * sn[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = x[i], q = y[i];
                    x[i] = p * cs[i] - q * sn[i];
                    y[i] = q * cs[i] + p * sn[i];
                }
            }
        }
        if (!in) continue;
        if (is_v) {  // as it is
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.vc) + (slot * a.Hkv + h) * D);
            dst[c0] = r0;
            dst[c1] = r1;
            continue;
        }
        if (is_q || a.ko) {
            uint4 *dst = reinterpret_cast<uint4 *>(is_q ? a.qo + t * a.qos + h * D : a.ko + t * a.kos + h * D);
            dst[c0] = pack8(x);
            dst[c1] = pack8(y);
        }
        if (CACHE == kRopeNone || !is_k || slot < 0) continue;
        if (CACHE == kRopeBf16) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.kc) + (slot * a.Hkv + h) * D);
            dst[c0] = pack8(x);
            dst[c1] = pack8(y);
        } else {
            const float scale = __ldg(a.k_scale + h);
            uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.kc) + (slot * a.Hkv + h) * D);
            dst[c0] = make_uint2(encode2(x[0], x[1], scale) | encode2(x[2], x[3], scale) << 16,
                                 encode2(x[4], x[5], scale) | encode2(x[6], x[7], scale) << 16);
            dst[c1] = make_uint2(encode2(y[0], y[1], scale) | encode2(y[2], y[3], scale) << 16,
                                 encode2(y[4], y[5], scale) | encode2(y[6], y[7], scale) << 16);
        }
    }
}

// per: heads of a warp (a multiple of a step's); parts: warps of a token; the 8-bit V after them,
// a warp per token and KV head
template <int D, bool INTER, RopeCache CACHE>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeArgs a, int per, int parts) {
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
    rope_heads<D, INTER, CACHE>(a, t, part * per, min((part + 1) * per, heads));
}

template <int D, bool INTER, RopeCache CACHE>
cudaError_t launch_t(const RopeArgs &a, cudaStream_t stream) {
    constexpr int step = 32 / (D / 16);
    const int heads = a.Hq + a.Hkv + (CACHE == kRopeBf16 ? a.Hkv : 0);
    const int steps = (heads + step - 1) / step;
    const int per = (a.T * steps < 4096 ? 1 : 3) * step;
    const int parts = (heads + per - 1) / per;
    const int64_t warps = a.T * (parts + (CACHE == kRopeE4m3 ? a.Hkv : 0));
    return launch_pdl(norm_rope_kernel<D, INTER, CACHE>, dim3(unsigned((warps + kRopeWarps - 1) / kRopeWarps)),
                      dim3(kRopeWarps * 32), 0, stream, a, per, parts);
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
