// Attention over the paged latent cache on the tensor cores (tc_paged.cu): bf16 at the DeepSeek-V3 sizes.
#pragma once

#include "paged.cuh"

namespace mla {

// Scratch bytes: the tokens' plan and the partials of the tokens that cross the pairs' ranges.
size_t tc_paged_attention_bytes(int64_t total_q);

// o_lat [T, 128, 512] bf16 and lse [T, 128] of the new tokens over all their rows (blocks == nullptr) or the
// rows of their listed blocks.
cudaError_t tc_paged_attention(const PagedView& v, const void* q_abs, const void* q_rope, const int32_t* blocks,
                               int32_t top_k, float scale, void* o_lat, float* lse, void* ws, int num_sms, uint32_t* err,
                               cudaStream_t st);

// Whether mla_test_arm_paged_stall armed this launch; the next one is not.
bool take_paged_stall();

// Scores [T, max_pages] fp32 (at the start of ws) of the blocks that each new token sees, for the tokens with more than
// top_k of them; ws: tc_select_bytes().
size_t tc_select_bytes(int64_t total_q, int64_t max_pages);
cudaError_t tc_select_scores(const PagedView& v, const void* q_abs, const void* q_rope, const void* summaries,
                             int32_t top_k, void* ws, int num_sms, uint32_t* err, cudaStream_t st);

}  // namespace mla
