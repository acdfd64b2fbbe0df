// kvq_chunk.cu -- runs of several tokens: the append with the position rotation,
// and tokens read back as values.
//
// Append.  A run of T tokens joins a window of `nres` tokens in a ring of Nr slots;
// in order they are the line C_0 .. C_{nres+T-1}, and as many single appends would
// leave the last Nr of it in the ring and the P = nres + T - Nr before them as
// codes.  C_j always sits in ring slot (head + j) % Nr, so each new token has one
// place: C_j with j < P is packed straight from the input, the others go to their
// slot, where the window token they displace (C_{j % Nr}, if j >= Nr) is packed
// first, by the same thread: no slot is read by one thread and written by another.
//
// Mapping.  A lane holds 8 values of a row (16 bytes), a row is d / 8 neighbouring
// lanes of one warp, a quad of lanes is one quantization group.  A warp takes
// 256 / d tokens and a group of heads of one kind (keys, values or queries), four
// rows' loads in flight at a time, so that a token's cosines and sines are loaded
// once for the heads of a group.  The rotation's partner elements (rotary_dim / 2
// away) are a second load of the same row, which L1 answers.  Bytes bound it.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kRows = 4;  // rows in flight per lane

struct ChunkAppendArgs {
  const __half* x[3];  // keys, values, queries: element j of head h of row t at x + t * st + h * sh + j
  int64_t st[3], sh[3];
  __half* q_out;  // [total][Hq][d]
  const int32_t* cu;
  const int32_t* positions;
  const float2* rope;  // [rope_rows][rd / 2]
  uint8_t* codes[2];
  uint32_t* params[2];
  __half* res[2];
  uint8_t* modes[2];
  RowMap rm;
  int32_t* packed_len;
  int32_t* res_len;
  int32_t* res_head;
  const int32_t* sink_len;
  uint32_t* err_word;
  int B, Hkv, Hq, d, Ng, row_bytes, cap, Nr, Ns;
  int total, max_len, rope_rows, rd, interleaved;
  int hpg;         // heads per group
  int gkv, gq;     // groups of KV heads and of query heads
};

// How a sequence's run enters the cache: tokens taken and tokens packed.
struct Plan {
  int taken, packed;
};
__device__ __forceinline__ Plan plan_of(const SeqLens& s, int n, int cap, int Nr) {
  Plan p;
  const int64_t room = (int64_t)cap - s.npk + (Nr - s.nres);  // >= 0: lengths are held to their bounds
  p.taken = (int)min((int64_t)n, room);
  p.packed = max(0, s.nres + p.taken - Nr);
  return p;
}

__device__ __forceinline__ SeqLens lens_of(const ChunkAppendArgs& a, int b) {
  return seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
}

// The last sequence whose first row is <= t, by a 32-way search of the warp
// (t is warp-uniform; with entries out of order it still ends, at some sequence).
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, i < hi && __ldg(cu + i) <= t);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// R1 for the 8 values of a lane at element e < rd; partner: the 8 values rd / 2 away.
__device__ __forceinline__ uint4 rotate8(const uint4& own, const uint4& partner, const float2 (&cs)[8],
                                         int interleaved, bool second) {
  float x[8], y[8];
  unpack8_f16(own, x);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = cs[i].x, s = cs[i].y;
      y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], c), __fmul_rn(x[2 * i + 1], s));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], c), __fmul_rn(x[2 * i], s));
    }
  } else {
    float p[8];
    unpack8_f16(partner, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xc = __fmul_rn(x[i], cs[i].x), ps = __fmul_rn(p[i], cs[i].y);
      y[i] = second ? __fadd_rn(xc, ps) : __fsub_rn(xc, ps);
    }
  }
  uint4 r;
  __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
  return r;
}

// One warp's unit: the lane's row t of sequence b (live: the lane has one) and
// head group `grp`.  All lanes of the warp take part.
template <int BITS, bool HYB>
__device__ __forceinline__ void append_unit(const ChunkAppendArgs& a, int t, int b, bool live, int grp) {
  const int lane = threadIdx.x & 31;
  const int lpr = a.d >> 3;              // lanes per row
  const int e = (lane & (lpr - 1)) * 8;  // first element of the lane
  const int kind = grp < a.gkv ? 0 : grp < 2 * a.gkv ? 1 : 2;
  const int h0 = (grp - (kind == 0 ? 0 : kind == 1 ? a.gkv : 2 * a.gkv)) * a.hpg;
  const int nh = min(a.hpg, (kind == 2 ? a.Hq : a.Hkv) - h0);

  Run run = {0, -1};
  SeqLens s = {0, 0, 0, 0};
  if (live) {
    run = run_of(a.cu, b, a.total, a.max_len);
    live = run.n > 0 && t >= run.c0 && t - run.c0 < run.n;
    if (live) s = lens_of(a, b);
  }
  const Plan plan = plan_of(s, max(run.n, 0), a.cap, a.Nr);
  const int i = t - run.c0;
  const int j = s.nres + i;  // place in the line
  const bool taken = live && kind != 2 && i < plan.taken;
  const bool direct = taken && j < plan.packed;             // packed straight from the input
  const bool ring = taken && !direct;                       // goes to a window slot
  const bool oust = ring && a.Nr > 0 && j >= a.Nr && j % max(a.Nr, 1) < s.nres;  // a window token leaves it
  const int slot = a.Nr > 0 ? (int)(((int64_t)s.head + j) % a.Nr) : 0;
  const int pack_at = s.npk + (direct ? j : j % max(a.Nr, 1));
  const bool packs = direct || oust;
  const bool any_pack = __any_sync(0xffffffffu, packs);

  // the position's cosines and sines
  float2 cs[8];
  const bool rot = live && kind != 1 && e < a.rd;
  const int half = a.rd >> 1;
  const bool second = !a.interleaved && e >= half;
  if (rot) {
    int pos = a.positions ? __ldg(a.positions + t) : s.ns + s.npk + s.nres + i;
    if (pos < 0 || pos >= a.rope_rows) {
      set_error(a.err_word, KVQ_ERRBIT_BADPOS);
      pos = min(max(pos, 0), a.rope_rows - 1);
    }
    const float2* src = a.rope + (int64_t)pos * half + (a.interleaved ? e / 2 : second ? e - half : e);
    const float4* src4 = reinterpret_cast<const float4*>(src);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (a.interleaved && u >= 2) break;
      const float4 f = __ldg(src4 + u);
      cs[2 * u] = make_float2(f.x, f.y);
      cs[2 * u + 1] = make_float2(f.z, f.w);
    }
  }
  const __half* src = a.x[kind] + (int64_t)t * a.st[kind] + (int64_t)h0 * a.sh[kind] + e;
  const int away = second ? -half : half;
  const int64_t row = packs ? a.rm.row(b, 0, pack_at) : -1;  // of KV head 0
  const int64_t row_step = a.rm.paged ? kPage : a.cap;       // to the next head's row
  if (packs && row < 0) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
  const int w = kind & 1;

  for (int r0 = 0; r0 < nh; r0 += kRows) {
    uint4 own[kRows], other[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      own[u] = other[u] = make_uint4(0, 0, 0, 0);
      if (live && r0 + u < nh) {
        // plain loads: with q rotated in place these rows are written below
        const __half* p = src + (int64_t)(r0 + u) * a.sh[kind];
        own[u] = *reinterpret_cast<const uint4*>(p);
        if (rot && !a.interleaved) {
          other[u] = *reinterpret_cast<const uint4*>(p + away);
        } else if (oust && kind == 1) {
          other[u] = *reinterpret_cast<const uint4*>(
              a.res[1] + (((int64_t)b * a.Hkv + h0 + r0 + u) * a.Nr + slot) * a.d + e);
        }
      }
    }
    __syncwarp();  // every lane has read its rows before any is written
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (r0 + u >= nh) break;  // warp-uniform
      const int h = h0 + r0 + u;
      const uint4 x = rot ? rotate8(own[u], other[u], cs, a.interleaved, second) : own[u];
      if (kind == 2) {
        if (live) *reinterpret_cast<uint4*>(a.q_out + ((int64_t)t * a.Hq + h) * a.d + e) = x;
        continue;
      }
      __half* slot_row = a.res[w] + (((int64_t)b * a.Hkv + h) * a.Nr + slot) * a.d + e;
      if (any_pack) {
        uint4 y = x;
        if (oust) y = kind == 1 ? other[u] : *reinterpret_cast<const uint4*>(slot_row);
        uint32_t prm, asym = 1;
        const uint32_t packed = quantize_quad<BITS>(y, prm, HYB, &asym);
        const uint32_t modes = HYB ? __ballot_sync(0xffffffffu, (lane & 3) == 0 && asym) : 0u;
        const bool ok = packs && row >= 0;
        const int64_t hr = row + (int64_t)h * row_step;
        store_group_codes<BITS>(ok ? a.codes[w] + hr * a.row_bytes + (e >> 5) * (4 * BITS) : nullptr,
                                packed, lane & 3, ok);
        if (ok && (lane & 3) == 0) a.params[w][hr * a.Ng + (e >> 5)] = prm;
        if (HYB && ok && e == 0) a.modes[w][hr] = mode_byte(modes, lane >> 2, a.Ng);
      }
      if (ring) *reinterpret_cast<uint4*>(slot_row) = x;
    }
  }
}

// The counters as the run leaves them, and the errors of the sequence.
__device__ __forceinline__ void finish_seq(const ChunkAppendArgs& a, int b) {
  const Run run = run_of(a.cu, b, a.total, a.max_len);
  if (run.n < 0) {
    set_error(a.err_word, KVQ_ERRBIT_BADLEN);
    return;
  }
  const SeqLens s = lens_of(a, b);
  const Plan p = plan_of(s, run.n, a.cap, a.Nr);
  if (p.taken < run.n) set_error(a.err_word, KVQ_ERRBIT_CAPACITY);
  if (p.taken == 0) return;
  a.packed_len[b] = s.npk + p.packed;
  a.res_len[b] = s.nres + p.taken - p.packed;
  if (a.Nr > 0) a.res_head[b] = (int)(((int64_t)s.head + p.packed) % a.Nr);
}

// Short runs: one block per sequence, which also moves its counters.
template <int BITS, bool HYB>
__global__ void __launch_bounds__(1024) append_run_kernel(ChunkAppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int b = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int tpw = 256 / a.d;  // tokens per warp
  const Run run = run_of(a.cu, b, a.total, a.max_len);
  const int groups = 2 * a.gkv + a.gq;
  const int64_t units = (int64_t)((max(run.n, 0) + tpw - 1) / tpw) * groups;
  for (int64_t u = threadIdx.x >> 5; u < units; u += blockDim.x >> 5) {
    const int i = (int)(u / groups) * tpw + lane / (a.d >> 3);
    append_unit<BITS, HYB>(a, run.c0 + i, b, i < run.n, (int)(u % groups));
  }
  __syncthreads();
  if (threadIdx.x == 0) finish_seq(a, b);
}

// Long runs: the rows of all runs in one line.
template <int BITS, bool HYB>
__global__ void __launch_bounds__(kAppendThreads) append_rows_kernel(ChunkAppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int tpw = 256 / a.d;
  const int groups = 2 * a.gkv + a.gq;
  const int64_t u = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t t0 = (u / groups) * tpw;
  if (t0 >= a.total) return;  // warp-uniform
  int b = find_seq(a.cu, a.B, (int)t0);
  const int64_t t = t0 + lane / (a.d >> 3);
  const bool live = t < a.total;
  if (live)
    while (b + 1 < a.B && __ldg(a.cu + b + 1) <= t) ++b;
  append_unit<BITS, HYB>(a, (int)(live ? t : t0), b, live, (int)(u % groups));
}

__global__ void append_finish_kernel(ChunkAppendArgs a) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < a.B) finish_seq(a, b);
}

// ------------------------------------------------------------------- read ---

constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;  // pieces of 8 values per thread, one grid stride apart

struct ReadArgs {
  const uint8_t* codes[2];
  const uint32_t* params[2];
  const __half* res[2];
  const __half* sink[2];
  void* out[2];
  RowMap rm;
  const int32_t* first;
  const int32_t* packed_len;
  const int32_t* res_len;
  const int32_t* res_head;
  const int32_t* sink_len;
  uint32_t* err_word;
  int Hkv, d, Ng, row_bytes, cap, Nr, Ns, count, lpr_shift;
};

// Codes 8q .. 8q + 7 of a group (its first byte at grp), packed in 8 * BITS bits.
template <int BITS>
__device__ __forceinline__ uint32_t load_codes8(const uint8_t* grp, int q) {
  if (BITS == 4) return __ldg(reinterpret_cast<const uint32_t*>(grp) + q);
  if (BITS == 2) return __ldg(reinterpret_cast<const uint16_t*>(grp) + q);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(grp);  // bytes 3q .. 3q + 2 of 12
  const int i = (3 * q) >> 2;
  return __funnelshift_r(__ldg(w + i), __ldg(w + min(i + 1, 2)), 8 * ((3 * q) & 3)) & 0xffffffu;
}

// A quad of lanes per group: each lane turns 8 codes into 8 values, so that the
// quad's stores are the group's contiguous 64 (or 128) bytes.  Output bytes bound it.
template <int BITS, bool F32>
__global__ void __launch_bounds__(kReadThreads) read_tokens_kernel(ReadArgs a) {
  const int bh = blockIdx.y, w = blockIdx.z;
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
  const int first = a.first ? __ldg(a.first + b) : 0;
  if (first < 0 && blockIdx.x == 0 && w == 0 && h == 0 && threadIdx.x == 0)
    set_error(a.err_word, KVQ_ERRBIT_BADLEN);
  const int64_t n = first < 0 ? 0 : (int64_t)s.ns + s.npk + s.nres;
  const int64_t pieces = (int64_t)a.count << a.lpr_shift;
  const int64_t p0 = (int64_t)blockIdx.x * (kReadThreads * kReadRows) + threadIdx.x;
  const __half* sink = a.sink[w] + (int64_t)bh * a.Ns * a.d;
  const __half* res = a.res[w] + (int64_t)bh * a.Nr * a.d;

  uint4 raw[kReadRows];      // fp16 tokens: the values; packed ones: codes and params
  int kind[kReadRows];       // 0 zero, 1 fp16, 2 packed
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int64_t p = p0 + u * kReadThreads;
    const int64_t t = max(first, 0) + (p >> a.lpr_shift);  // a negative first has n = 0
    const int e = (int)(p & ((1 << a.lpr_shift) - 1)) * 8;
    kind[u] = 0;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (p >= pieces || t >= n) continue;
    if (t < s.ns) {
      kind[u] = 1;
      raw[u] = __ldg(reinterpret_cast<const uint4*>(sink + t * a.d + e));
    } else if (t < s.ns + s.npk) {
      const int64_t row = a.rm.row(b, h, (int)(t - s.ns));
      if (row < 0) {
        set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
        continue;
      }
      kind[u] = 2;
      raw[u].x = load_codes8<BITS>(a.codes[w] + row * a.row_bytes + (e >> 5) * (4 * BITS), (e >> 3) & 3);
      raw[u].y = __ldg(a.params[w] + row * a.Ng + (e >> 5));
    } else {
      kind[u] = 1;
      const int64_t j = (t - s.ns - s.npk + s.head) % a.Nr;
      raw[u] = __ldg(reinterpret_cast<const uint4*>(res + j * a.d + e));
    }
  }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int64_t p = p0 + u * kReadThreads;
    if (p >= pieces) break;
    const int64_t at = ((int64_t)bh << a.lpr_shift) * a.count + p;  // pieces of 8 values
    float x[8];
    if (kind[u] == 2) {
      const float sc = __half2float(__ushort_as_half((unsigned short)(raw[u].y & 0xffffu)));
      const float mn = __half2float(__ushort_as_half((unsigned short)(raw[u].y >> 16)));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = __fadd_rn(mn, __fmul_rn((float)((raw[u].x >> (BITS * j)) & ((1u << BITS) - 1u)), sc));
    }
    if (F32) {
      if (kind[u] != 2) unpack8_f16(raw[u], x);
      float4* dst = reinterpret_cast<float4*>(a.out[w]) + 2 * at;
      dst[0] = make_float4(x[0], x[1], x[2], x[3]);
      dst[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint4 r = raw[u];
      if (kind[u] == 2) {
        __half2* hh = reinterpret_cast<__half2*>(&r);
#pragma unroll
        for (int j = 0; j < 4; ++j) hh[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      }
      reinterpret_cast<uint4*>(a.out[w])[at] = r;
    }
  }
}

template <int BITS, bool HYB>
cudaError_t launch_append_bits(const ChunkAppendArgs& a, bool by_seq, int threads, cudaStream_t st) {
  if (by_seq) {
    append_run_kernel<BITS, HYB><<<a.B, threads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int tpw = 256 / a.d;
  const int64_t warps = (((int64_t)a.total + tpw - 1) / tpw) * (2 * a.gkv + a.gq);
  const int64_t blocks = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
  append_rows_kernel<BITS, HYB><<<(unsigned)blocks, kAppendThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  append_finish_kernel<<<(a.B + 127) / 128, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_chunk(const Dims& s, const kvq_cache_view& v, const kvq_append_args& A,
                                cudaStream_t st) {
  ChunkAppendArgs a;
  a.x[0] = static_cast<const __half*>(A.k);
  a.x[1] = static_cast<const __half*>(A.v);
  a.x[2] = static_cast<const __half*>(A.q);
  a.st[0] = a.st[1] = A.kv_stride_token;
  a.sh[0] = a.sh[1] = A.kv_stride_head;
  a.st[2] = A.q_stride_token;
  a.sh[2] = A.q_stride_head;
  a.q_out = static_cast<__half*>(A.q_out);
  a.cu = A.cu_seqlens;
  a.positions = A.positions;
  a.rope = reinterpret_cast<const float2*>(A.rope);
  a.codes[0] = v.k_codes;
  a.codes[1] = v.v_codes;
  a.params[0] = v.k_params;
  a.params[1] = v.v_params;
  a.res[0] = reinterpret_cast<__half*>(v.k_res);
  a.res[1] = reinterpret_cast<__half*>(v.v_res);
  a.modes[0] = v.k_mode;
  a.modes[1] = v.v_mode;
  a.rm = row_map(s, v.block_table);
  a.packed_len = v.packed_len;
  a.res_len = v.res_len;
  a.res_head = v.res_head;
  a.sink_len = v.sink_len;
  a.err_word = v.err_word;
  a.B = s.B;
  a.Hkv = s.Hkv;
  a.Hq = A.q ? A.num_q_heads : 0;
  a.d = s.d;
  a.Ng = s.Ng;
  a.row_bytes = s.row_bytes;
  a.cap = s.cap;
  a.Nr = s.Nr;
  a.Ns = s.Ns;
  a.total = A.total;
  a.max_len = A.max_len;
  a.rope_rows = A.rope_rows;
  a.rd = A.rotary_dim;
  a.interleaved = A.interleaved;
  // A block per sequence saves the second launch; it is the shorter way while
  // one block's warps take at most a few units each.
  const int tpw = 256 / s.d;
  const int64_t len = A.max_len < A.total ? A.max_len : A.total;
  const int64_t tiles = (len + tpw - 1) / tpw;
  auto groups = [&](int hpg) {
    a.hpg = hpg;
    a.gkv = (a.Hkv + hpg - 1) / hpg;
    a.gq = (a.Hq + hpg - 1) / hpg;
    return 2 * a.gkv + a.gq;
  };
  const int64_t units = tiles * groups(4);
  const bool by_seq = units <= 128;
  int threads = 0;
  if (by_seq)
    threads = 32 * (int)(units < 1 ? 1 : units < 32 ? units : 32);
  else
    groups(8);
  if (s.bits == 4)
    return s.hybrid ? launch_append_bits<4, true>(a, by_seq, threads, st)
                    : launch_append_bits<4, false>(a, by_seq, threads, st);
  if (s.bits == 3)
    return s.hybrid ? launch_append_bits<3, true>(a, by_seq, threads, st)
                    : launch_append_bits<3, false>(a, by_seq, threads, st);
  return s.hybrid ? launch_append_bits<2, true>(a, by_seq, threads, st)
                  : launch_append_bits<2, false>(a, by_seq, threads, st);
}

cudaError_t launch_read_tokens(const Dims& s, const kvq_cache_view& v, const int32_t* first, int count,
                               void* k_out, void* v_out, uint32_t flags, cudaStream_t st) {
  if (count == 0) return cudaSuccess;
  ReadArgs a;
  a.codes[0] = v.k_codes;
  a.codes[1] = v.v_codes;
  a.params[0] = v.k_params;
  a.params[1] = v.v_params;
  a.res[0] = reinterpret_cast<const __half*>(v.k_res);
  a.res[1] = reinterpret_cast<const __half*>(v.v_res);
  a.sink[0] = reinterpret_cast<const __half*>(v.k_sink);
  a.sink[1] = reinterpret_cast<const __half*>(v.v_sink);
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.rm = row_map(s, v.block_table);
  a.first = first;
  a.packed_len = v.packed_len;
  a.res_len = v.res_len;
  a.res_head = v.res_head;
  a.sink_len = v.sink_len;
  a.err_word = v.err_word;
  a.Hkv = s.Hkv;
  a.d = s.d;
  a.Ng = s.Ng;
  a.row_bytes = s.row_bytes;
  a.cap = s.cap;
  a.Nr = s.Nr;
  a.Ns = s.Ns;
  a.count = count;
  a.lpr_shift = __builtin_ctz((unsigned)s.d / 8);
  const int64_t pieces = (int64_t)count << a.lpr_shift;
  const int64_t per = kReadThreads * kReadRows;
  const dim3 grid((unsigned)((pieces + per - 1) / per), (unsigned)(s.B * s.Hkv), 2);
  const bool f32 = (flags & KVQ_OUT_F32) != 0;
  if (s.bits == 4)
    f32 ? read_tokens_kernel<4, true><<<grid, kReadThreads, 0, st>>>(a)
        : read_tokens_kernel<4, false><<<grid, kReadThreads, 0, st>>>(a);
  else if (s.bits == 3)
    f32 ? read_tokens_kernel<3, true><<<grid, kReadThreads, 0, st>>>(a)
        : read_tokens_kernel<3, false><<<grid, kReadThreads, 0, st>>>(a);
  else
    f32 ? read_tokens_kernel<2, true><<<grid, kReadThreads, 0, st>>>(a)
        : read_tokens_kernel<2, false><<<grid, kReadThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
