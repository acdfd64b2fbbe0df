// kvq_chunk_attn.cu -- attention of runs of several tokens over the low-bit cache.
//
// One warp per (row of a run, query head): the row's visible tokens one after the
// other, the scores' running maximum and sum and the output in fp32.  Lane l holds
// element l of every group of 32.
#include <math.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

struct ChunkAttnArgs {
  const uint8_t* codes[2];
  const uint32_t* params[2];
  const __half* res[2];
  const __half* sink[2];
  RowMap rm;
  const int32_t* packed_len;
  const int32_t* res_len;
  const int32_t* res_head;
  const int32_t* sink_len;
  uint32_t* err_word;
  const __half* q;
  void* out;
  const int32_t* cu;
  int B, Hkv, Hq, d, Ng, row_bytes, bits, cap, Nr, Ns, total, max_len, causal, out_f32;
  float scale_log2;
};

constexpr int kMaxGroups = 8;

__device__ __forceinline__ void load_row(const ChunkAttnArgs& a, int w, int b, int h, int t,
                                         const SeqLens& s, int lane, float (&x)[kMaxGroups], bool& ok) {
  const int64_t bh = (int64_t)b * a.Hkv + h;
  ok = true;
  if (t >= s.ns && t < s.ns + s.npk) {
    const int64_t row = a.rm.row(b, h, t - s.ns);
    ok = row >= 0;
    for (int g = 0; g < a.Ng; ++g) {
      if (!ok) break;
      const uint8_t* p = a.codes[w] + row * a.row_bytes + g * 4 * a.bits;
      const int bit = lane * a.bits;
      uint32_t v = p[bit >> 3];
      if ((bit & 7) + a.bits > 8) v |= (uint32_t)p[(bit >> 3) + 1] << 8;
      const float code = (float)((v >> (bit & 7)) & ((1u << a.bits) - 1u));
      const uint32_t prm = a.params[w][row * a.Ng + g];
      x[g] = __half2float(__ushort_as_half((unsigned short)(prm >> 16))) +
             code * __half2float(__ushort_as_half((unsigned short)(prm & 0xffffu)));
    }
    return;
  }
  const __half* p = t < s.ns ? a.sink[w] + (bh * a.Ns + t) * a.d
                             : a.res[w] + (bh * a.Nr + (t - s.ns - s.npk + s.head) % a.Nr) * a.d;
  for (int g = 0; g < a.Ng; ++g) x[g] = __half2float(p[g * 32 + lane]);
}

__global__ void __launch_bounds__(128) chunk_attention_kernel(ChunkAttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / a.Hq), hq = (int)(unit % a.Hq);
  if (t >= a.total) return;
  int b = 0;
  while (b + 1 < a.B && a.cu[b + 1] <= t) ++b;
  const Run run = run_of(a.cu, b, a.total, a.max_len);
  if (run.n < 0 && lane == 0) set_error(a.err_word, KVQ_ERRBIT_BADLEN);
  if (run.n <= 0 || t < run.c0 || t - run.c0 >= run.n) return;
  const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
  const int n = s.ns + s.npk + s.nres;
  const int seen = a.causal ? n - run.n + (t - run.c0) + 1 : n;
  const int h = hq / (a.Hq / a.Hkv);
  float q[kMaxGroups], o[kMaxGroups], x[kMaxGroups];
  for (int g = 0; g < a.Ng; ++g) {
    q[g] = __half2float(a.q[((int64_t)t * a.Hq + hq) * a.d + g * 32 + lane]) * a.scale_log2;
    o[g] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  bool any = false;
  for (int j = 0; j < seen; ++j) {
    bool ok;
    load_row(a, 0, b, h, j, s, lane, x, ok);
    if (!ok) {
      if (lane == 0) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
      continue;
    }
    any = true;
    float sc = 0.0f;
    for (int g = 0; g < a.Ng; ++g) sc += q[g] * x[g];
    for (int k = 16; k > 0; k >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, k);
    const float m2 = fmaxf(m, sc);
    const float f = exp2f(m - m2), p = exp2f(sc - m2);
    load_row(a, 1, b, h, j, s, lane, x, ok);
    for (int g = 0; g < a.Ng; ++g) o[g] = o[g] * f + p * x[g];
    l = l * f + p;
    m = m2;
  }
  if (!any && lane == 0) set_error(a.err_word, KVQ_ERRBIT_EMPTY);
  const float inv = any ? 1.0f / l : 0.0f;
  for (int g = 0; g < a.Ng; ++g) {
    const int64_t at = ((int64_t)t * a.Hq + hq) * a.d + g * 32 + lane;
    if (a.out_f32)
      static_cast<float*>(a.out)[at] = o[g] * inv;
    else
      static_cast<__half*>(a.out)[at] = __float2half_rn(o[g] * inv);
  }
}

}  // namespace

size_t chunk_workspace_bytes(const Dims&, int, int) { return 256; }

cudaError_t launch_chunk_attention(const Dims& s, const kvq_cache_view& v, const __half* q, int Hq,
                                   const int32_t* cu, int total, int max_len, void* out,
                                   void* workspace, bool causal, uint32_t flags, cudaStream_t st) {
  (void)workspace;
  if (total == 0) return cudaSuccess;
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
  a.B = s.B;
  a.Hkv = s.Hkv;
  a.Hq = Hq;
  a.d = s.d;
  a.Ng = s.Ng;
  a.row_bytes = s.row_bytes;
  a.bits = s.bits;
  a.cap = s.cap;
  a.Nr = s.Nr;
  a.Ns = s.Ns;
  a.total = total;
  a.max_len = max_len;
  a.causal = causal;
  a.out_f32 = (flags & KVQ_OUT_F32) ? 1 : 0;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)s.d));
  const int64_t units = (int64_t)total * Hq;
  chunk_attention_kernel<<<(unsigned)((units + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
