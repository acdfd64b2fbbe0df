// kvq_rotate.cu -- rotary positions with several axes, of queries and keys.
//
// Pair i of row t at (c, s) = rope[positions[axis(i)][t]][i]:
//   y_a = x_a c - x_b s,  y_b = x_b c + x_a s   (fp32, each operation rounded; once to fp16)
//
// Mapping.  A lane holds 8 values (16 bytes) of a head, a head is d / 8 neighbouring lanes,
// a warp takes 256 / d rows.  Its cosines and sines stay in registers while it goes through
// heads (queries, then keys), four of them loaded at a time; few rows share the heads out
// over several warps instead.  The partner values (rotary_dim / 2 away) come by shuffles.
// The axis of each pair (2 bits) comes with the launch, and a lane whose pairs have one axis
// reads its row of the table in 16-byte pieces.
//
// Bound by memory: 34169 tokens (6 prompts) of 32 + 8 heads of 128 take 107 us, 96 % of the
// measured copy rate; 14314 of 16 + 16 heads of 64 18.9, 92 % (eight heads in flight and 16
// warps an SM 21.2; two heads 21.1, and 116 for the first).  16 tokens take 2.4 us, which
// is the launch and two dependent loads (eight heads 3.2).
#include "kvq_around.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;  // heads in flight

struct RotateArgs {
  const __half* x[2];  // queries, keys
  __half* y[2];
  int64_t st[2], sh[2], yt[2], yh[2];
  const float2* rope;
  const int32_t* positions;
  uint32_t* err_word;
  uint64_t axis[4];  // 2 bits of each pair
  int Hq, heads, per, d, total, rows, rd, interleaved;  // per: heads of a warp
};

// The 8 values x of the formulas; partner: the 8 values rd / 2 away.
__device__ __forceinline__ uint4 rotate8(const uint4& own, const uint4& partner, const float2 (&cs)[8],
                                         bool interleaved, bool second) {
  const __half2* xh = reinterpret_cast<const __half2*>(&own);
  const __half2* ph = reinterpret_cast<const __half2*>(&partner);
  uint4 r;
  __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(xh[i]);
    float y0, y1;
    if (interleaved) {
      const float c = cs[i].x, s = cs[i].y;
      y0 = __fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s));
      y1 = __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s));
    } else {
      const float2 p = __half22float2(ph[i]);
      const float a0 = __fmul_rn(x.x, cs[2 * i].x), b0 = __fmul_rn(p.x, cs[2 * i].y);
      const float a1 = __fmul_rn(x.y, cs[2 * i + 1].x), b1 = __fmul_rn(p.y, cs[2 * i + 1].y);
      y0 = second ? __fadd_rn(a0, b0) : __fsub_rn(a0, b0);
      y1 = second ? __fadd_rn(a1, b1) : __fsub_rn(a1, b1);
    }
    h[i] = __floats2half2_rn(y0, y1);
  }
  return r;
}

__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
  wait_for_previous();
  const int lane = threadIdx.x & 31, lpr = a.d >> 3;
  const int64_t t = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (32 / lpr) + lane / lpr;
  const bool live = t < a.total;
  const int e = (lane & (lpr - 1)) * 8, half = a.rd >> 1;
  const bool rot = live && e < a.rd, second = !a.interleaved && e >= half;

  float2 cs[8];
  if (rot) {
    const int p0 = a.interleaved ? e >> 1 : second ? e - half : e;  // the lane's first pair
    const int n = a.interleaved ? 4 : 8;
    const uint32_t axes = (uint32_t)(a.axis[p0 >> 5] >> (2 * (p0 & 31))) & (a.interleaved ? 0xffu : 0xffffu);
    auto row = [&](int axis) -> const float2* {
      int pos = a.positions[(int64_t)axis * a.total + t];
      if (pos < 0 || pos >= a.rows) {
        set_error(a.err_word, KVQ_ERRBIT_BADPOS);
        pos = pos < 0 ? 0 : a.rows - 1;
      }
      return a.rope + (int64_t)pos * half + p0;
    };
    if (axes == (axes & 3u) * (a.interleaved ? 0x55u : 0x5555u)) {
      const float4* src = reinterpret_cast<const float4*>(row(axes & 3u));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (2 * i >= n) break;
        const float4 f = src[i];
        cs[2 * i] = make_float2(f.x, f.y);
        cs[2 * i + 1] = make_float2(f.z, f.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) cs[i] = row((axes >> (2 * i)) & 3u)[i];
    }
  }
  const int partner = lane + (second ? -(half >> 3) : half >> 3);

  const int h_end = min(a.heads, (int)(blockIdx.y + 1) * a.per);
  for (int h0 = blockIdx.y * a.per; h0 < h_end; h0 += kHeads) {
    uint4 own[kHeads];
    // plain loads: with rows rotated in place the same lane writes these bytes below
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u, w = h >= a.Hq;
      own[u] = make_uint4(0, 0, 0, 0);
      if (live && h < h_end)
        own[u] = *reinterpret_cast<const uint4*>(a.x[w] + t * a.st[w] + (int64_t)(h - (w ? a.Hq : 0)) * a.sh[w] + e);
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u, w = h >= a.Hq;
      if (h >= h_end) break;  // warp-uniform
      uint4 p = own[u];
      if (!a.interleaved) {
        p.x = __shfl_sync(0xffffffffu, own[u].x, partner);
        p.y = __shfl_sync(0xffffffffu, own[u].y, partner);
        p.z = __shfl_sync(0xffffffffu, own[u].z, partner);
        p.w = __shfl_sync(0xffffffffu, own[u].w, partner);
      }
      if (live)
        *reinterpret_cast<uint4*>(a.y[w] + t * a.yt[w] + (int64_t)(h - (w ? a.Hq : 0)) * a.yh[w] + e) =
            rot ? rotate8(own[u], p, cs, a.interleaved, second) : own[u];
    }
  }
}

}  // namespace

cudaError_t launch_rotate(const kvq_rotate_args& args, cudaStream_t st) {
  RotateArgs a = {};
  a.x[0] = static_cast<const __half*>(args.q);
  a.x[1] = static_cast<const __half*>(args.k);
  a.y[0] = static_cast<__half*>(args.q_out);
  a.y[1] = static_cast<__half*>(args.k_out);
  a.st[0] = args.q_stride_token, a.sh[0] = args.q_stride_head;
  a.st[1] = args.k_stride_token, a.sh[1] = args.k_stride_head;
  a.yt[0] = args.q_out_stride_token, a.yh[0] = args.q_out_stride_head;
  a.yt[1] = args.k_out_stride_token, a.yh[1] = args.k_out_stride_head;
  a.rope = reinterpret_cast<const float2*>(args.rope);
  a.positions = args.positions;
  a.err_word = args.err_word;
  if (args.pair_axis)
    for (int i = 0; i < args.rotary_dim / 2; ++i) a.axis[i / 32] |= (uint64_t)args.pair_axis[i] << (2 * (i % 32));
  a.Hq = args.q ? args.num_q_heads : 0;
  a.heads = a.Hq + (args.k ? args.num_kv_heads : 0);
  a.d = args.head_dim;
  a.total = args.total;
  a.rows = args.rope_rows;
  a.rd = args.rotary_dim;
  a.interleaved = args.interleaved;
  if (a.total == 0 || a.heads == 0) return cudaSuccess;
  const int rows = 256 / a.d * (kThreads / 32);  // of a block
  const int64_t blocks = ((int64_t)a.total + rows - 1) / rows;
  // a warp goes through all heads where there are blocks enough for 128 warps on each SM
  // (14314 tokens of 16 + 16 heads of 64: for 16 warps 24.7 us, 32 20.6, 64 18.3, 128 18.9;
  // 34169 of 32 + 8 heads of 128: 108.4 for any fewer, 107.2)
  const int64_t want = (32 * (int64_t)device_sm_count() + blocks - 1) / blocks;
  const int batches = (a.heads + kHeads - 1) / kHeads;
  const int ny = (int)(want < batches ? want : batches);
  a.per = (batches + ny - 1) / ny * kHeads;
  return launch_overlapped(rotate_kernel, dim3((unsigned)blocks, (a.heads + a.per - 1) / a.per), kThreads, 0, st, a);
}

}  // namespace kvq
