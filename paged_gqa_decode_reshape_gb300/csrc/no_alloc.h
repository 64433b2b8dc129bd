// no_alloc.h -- internal interface of the dense decode in a scratch buffer of
// fixed size (no_alloc.cu): the buffer holds as many arrival counters as the
// call has, right behind the status word, and the caller clears both.
#pragma once

#include "../../include/paged_decode.h"

namespace pa {

// bytes of scratch, 0 for an invalid or unsupported shape
size_t no_alloc_bytes(int B, int Hq, int Hkv, int D);
int decode_no_alloc(pa_bf16 *out, const pa_bf16 *query, const pa_bf16 *key_cache, const pa_bf16 *value_cache,
                    const int32_t *block_tables, int MBS, const int32_t *context_lens, int B, int Hq, int Hkv, int D,
                    int BS, int64_t NB, float scale, void *scratch, size_t scratch_bytes, void *stream);

}  // namespace pa
