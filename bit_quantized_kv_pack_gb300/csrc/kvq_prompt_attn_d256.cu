// kvq_prompt_attn_d256.cu -- attention over prompts, head_dim 256 (kvq_prompt_attn.cuh).
#include "kvq_prompt_attn.cuh"

namespace kvq {

cudaError_t launch_prompt_attn_d256(const PromptAttnArgs& a, int grid, cudaStream_t st) {
  return prompt::launch<256>(a, grid, st);
}

}  // namespace kvq
