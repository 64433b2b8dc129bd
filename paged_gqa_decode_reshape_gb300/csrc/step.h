// step.h -- internal interface of what a serving step does around its attention
// (step_plan.cu: block tables and slots from request lengths; norm_rope.cu: norm
// and rotation of queries and keys with the cache write).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct PlanArgs {
    int32_t *bt;                   // [B][MBS]
    const int32_t *ctx, *q;        // [B] tokens cached, tokens to come
    const int32_t *free_blocks;    // [F], the first *num_free are free
    const int32_t *num_free;       // [1]
    int32_t *new_lens, *new_free;  // [B], [1]; may be ctx and num_free
    int32_t *granted, *cu, *pos;   // [B], [B + 1], [T]
    int64_t *slots;                // [T]
    int64_t NB, F;
    int MBS, B, T;
};

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t stream);

struct ReleaseArgs {
    const int32_t *bt;             // [B][MBS]
    const int32_t *ctx, *keep;     // [B] tokens cached, tokens to keep
    int32_t *free_blocks;          // [F]
    const int32_t *num_free;       // [1]
    int32_t *new_lens, *new_free;  // [B], [1]; may be ctx and num_free
    int64_t NB, F;
    int MBS, B;
};

cudaError_t launch_release(const ReleaseArgs &a, cudaStream_t stream);

struct RopeArgs {
    const uint16_t *q, *k, *v;     // rows of heads; v: null without a cache
    uint16_t *qo, *ko;             // ko: null when the rotated keys go to the cache alone
    int64_t qs, ks, vs, qos, kos;  // elements from one row to the next
    const uint16_t *qw, *kw;       // [D] norm weights; null: no norm
    const float *table;            // [P][R] cosines, then sines
    const int32_t *pos;            // [axes][T]
    const int32_t *axis;           // [R / 2] axis of each frequency; null: axis 0
    void *kc, *vc;                 // caches; null: none
    const float *k_scale, *v_scale;  // [Hkv], 8-bit caches
    const int64_t *slots;          // [T]
    int64_t T, P, NB;
    int Hq, Hkv, R, naxes;
    float eps;
};

enum RopeCache { kRopeNone = 0, kRopeBf16 = 1, kRopeE4m3 = 2 };

cudaError_t launch_norm_rope(const RopeArgs &a, int head_dim, bool interleaved, RopeCache cache, int sms, cudaStream_t stream);

}  // namespace pa
