// attention_prompt.cu -- attention of many query rows per key/value head over the paged 8-bit cache.
#include "attention_prompt.cuh"

namespace q4lin {

bool attention_prompt_eligible(const q4lin_kv_cache_t& cache) { return cache.head_dim <= 128; }

cudaError_t attention_prompt_launch(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a,
                                    int64_t rows_min, const LaunchCtx& c) {
    return prompt_launch<8>(cache, a, rows_min, c);
}

}  // namespace q4lin
