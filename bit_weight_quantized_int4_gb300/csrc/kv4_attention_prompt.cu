// kv4_attention_prompt.cu -- attention of many query rows per key/value head over the paged 4-bit cache.
#include "attention_prompt.cuh"

namespace q4lin {

cudaError_t kv4_attention_prompt_launch(const q4lin_kv4_cache_t& cache, const q4lin_attention_t& a,
                                        int64_t rows_min, const LaunchCtx& c) {
    return prompt_launch<4>(cache, a, rows_min, c);
}

}  // namespace q4lin
