// kvq_chunk_attn.cu -- attention of runs of several tokens: the workspace and the
// dispatch on head_dim (the kernel is kvq_chunk_attn.cuh).
#include "kvq_chunk_attn.cuh"

namespace kvq {
namespace {

struct Layout {
  size_t ml, o, total;
};
Layout layout_of(int d, int grid) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t rows = (size_t)2 * grid * chunk_rows(d);
  Layout l;
  l.ml = up((size_t)grid * 64);  // heads first
  l.o = up(l.ml + rows * sizeof(float2));
  l.total = l.o + rows * d * sizeof(float);
  return l;
}

}  // namespace

// Two pieces of units to each block (its first and its last), whatever the lengths.
size_t chunk_workspace_bytes(const Dims& s, int num_q_heads, int sm_count) {
  (void)num_q_heads;
  return layout_of(s.d, sm_count < 256 ? sm_count : 256).total;
}

cudaError_t launch_chunk_attention(const Dims& s, const kvq_cache_view& v, const __half* q, int Hq,
                                   const int32_t* cu, int total, int max_len, void* out,
                                   void* workspace, bool causal, uint32_t flags, cudaStream_t st) {
  const int sms = device_sm_count();
  const int grid = sms < 256 ? sms : 256;  // one block per SM
  const Layout l = layout_of(s.d, grid);
  char* ws = static_cast<char*>(workspace);
  ChunkAttnArgs a;
  a.codes[0] = v.k_codes;
  a.codes[1] = v.v_codes;
  a.params[0] = v.k_params;
  a.params[1] = v.v_params;
  a.res[0] = reinterpret_cast<const __half*>(v.k_res);
  a.res[1] = reinterpret_cast<const __half*>(v.v_res);
  a.sink[0] = reinterpret_cast<const __half*>(v.k_sink);
  a.sink[1] = reinterpret_cast<const __half*>(v.v_sink);
  a.rm = row_map(s, v.block_table);
  a.packed_len = v.packed_len;
  a.res_len = v.res_len;
  a.res_head = v.res_head;
  a.sink_len = v.sink_len;
  a.err_word = v.err_word;
  a.q = q;
  a.out = out;
  a.cu = cu;
  a.heads = reinterpret_cast<int4*>(ws);
  a.ml_part = reinterpret_cast<float2*>(ws + l.ml);
  a.o_part = reinterpret_cast<float4*>(ws + l.o);
  a.B = s.B;
  a.Hkv = s.Hkv;
  a.Hq = Hq;
  a.gq = Hq / s.Hkv;
  // gq_mul = ceil(2^(31 + k) / gq) with 2^k >= gq: exact for rows below 2^31
  int k = 0;
  while ((1 << k) < a.gq) ++k;
  a.gq_shift = 31 + k;
  a.gq_mul = (uint32_t)(((1ull << a.gq_shift) + a.gq - 1) / a.gq);
  a.cap = s.cap;
  a.Nr = s.Nr;
  a.Ns = s.Ns;
  a.total = total;
  a.max_len = max_len;
  a.causal = causal;
  a.out_f32 = (flags & KVQ_OUT_F32) ? 1 : 0;
  const uint32_t fault_us = testing_wait_fault_us();
  a.wait_limit_us = fault_us ? fault_us : 1000000u;
  a.fault = fault_us ? 1 : 0;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)s.d));
  if (s.d == 32) return launch_chunk_attn_d32(a, s.bits, grid, st);
  if (s.d == 64) return launch_chunk_attn_d64(a, s.bits, grid, st);
  if (s.d == 128) return launch_chunk_attn_d128(a, s.bits, grid, st);
  return launch_chunk_attn_d256(a, s.bits, grid, st);
}

}  // namespace kvq
