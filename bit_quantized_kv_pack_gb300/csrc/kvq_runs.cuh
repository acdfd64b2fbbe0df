// kvq_runs.cuh -- what the calls on runs of several tokens share: their launches, a
// sequence's run and its lengths.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

cudaError_t launch_append_chunk(const Dims& s, const kvq_cache_view& v, const kvq_append_args& args,
                                cudaStream_t st);
cudaError_t launch_read_tokens(const Dims& s, const kvq_cache_view& v, const int32_t* first, int count,
                               void* k_out, void* v_out, uint32_t flags, cudaStream_t st);

// Attention of runs (kvq_chunk_attn.cuh).
size_t chunk_workspace_bytes(const Dims& s, int num_q_heads, int sm_count);
cudaError_t launch_chunk_attention(const Dims& s, const kvq_cache_view& v, const __half* q, int Hq,
                                   const int32_t* cu, int total, int max_len, void* out,
                                   void* workspace, bool causal, uint32_t flags, cudaStream_t st);

// The run of sequence b: rows [c0, c0 + n) of the token-major arrays; n < 0 for
// entries of cu_seqlens that break the rule (the sequence is skipped).
struct Run {
  int c0, n;
};
__device__ __forceinline__ Run run_of(const int32_t* cu, int b, int total, int max_len) {
  const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
  Run r;
  r.c0 = c0;
  r.n = (c0 >= 0 && c1 >= c0 && c1 <= total && c1 - c0 <= max_len) ? c1 - c0 : -1;
  return r;
}

// A sequence's lengths, held to the layout's bounds so that no index leaves it.
struct SeqLens {
  int ns, npk, nres, head;
};
__device__ __forceinline__ SeqLens seq_lens_of(const int32_t* sink_len, const int32_t* packed_len,
                                               const int32_t* res_len, const int32_t* res_head, int b,
                                               int Ns, int cap, int Nr) {
  SeqLens s;
  s.ns = Ns > 0 ? min(max(sink_len[b], 0), Ns) : 0;
  s.npk = min(max(packed_len[b], 0), cap);
  s.nres = min(max(res_len[b], 0), Nr);
  s.head = Nr > 0 ? min(max(res_head[b], 0), Nr - 1) : 0;
  return s;
}

}  // namespace kvq
