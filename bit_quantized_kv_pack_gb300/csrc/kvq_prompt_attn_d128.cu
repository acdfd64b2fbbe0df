// kvq_prompt_attn_d128.cu -- attention over prompts, head_dim 128 (kvq_prompt_attn.cuh).
#include "kvq_prompt_attn.cuh"

namespace kvq {

cudaError_t launch_prompt_attn_d128(const PromptAttnArgs& a, int grid, cudaStream_t st) {
  return prompt::launch<128>(a, grid, st);
}

}  // namespace kvq
