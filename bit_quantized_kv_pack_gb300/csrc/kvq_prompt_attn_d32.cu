// kvq_prompt_attn_d32.cu -- attention over prompts, head_dim 32 (kvq_prompt_attn.cuh).
#include "kvq_prompt_attn.cuh"

namespace kvq {

cudaError_t launch_prompt_attn_d32(const PromptAttnArgs& a, int grid, cudaStream_t st) {
  return prompt::launch<32>(a, grid, st);
}

}  // namespace kvq
