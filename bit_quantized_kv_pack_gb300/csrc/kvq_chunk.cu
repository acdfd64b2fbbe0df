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
// 256 / d tokens and up to four heads of one kind (keys, values or queries), whose
// rows are loaded together before anything about the sequence is known; the warps
// of a block share their tokens, so that cosines and sines come from L1 after the
// first.  The rotation's partner values (rotary_dim / 2 away) are in a lane of the
// same row and come by shuffles.  Long runs are bound by instructions (70 % of the issue
// slots at a third of the warps): four prompts of 501 to 4096 tokens, 32 / 8 heads, INT2,
// take 55 us for 211 MB read and written.  The four lanes of a group each work out its
// scale; the prefill's pack, with a lane to a group, does not and reaches 0.7 of the
// copy rate.
#include "kvq_ptx.cuh"
#include "kvq_runs.cuh"

namespace kvq {
namespace {

constexpr int kRunThreads = 384;  // at most
constexpr int kRowThreads = 128;  // small: a block lives as long as its slowest warp (a packing one)
constexpr int kHeads = 4;         // heads of a unit: rows in flight per lane

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
  int gkv, groups;  // head groups of the keys (as many of the values), and of all
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
// (t is warp-uniform; with entries out of order it ends at some sequence).
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

// The sequence that append_rows_kernel gives row t to, t of the warp's rows from t0 on.
// With entries in order it is the one that has the row.
__device__ __forceinline__ int seq_of_row(const ChunkAppendArgs& a, int64_t t0, int64_t t, bool live) {
  int b = find_seq(a.cu, a.B, (int)t0);
  if (live)
    while (b + 1 < a.B && __ldg(a.cu + b + 1) <= t) ++b;
  return b;
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

// A unit's head group: its kind (0 keys, 1 values, 2 queries), first head and heads.
struct Group {
  int kind, h0, nh;
};
__device__ __forceinline__ Group group_of(const ChunkAppendArgs& a, int grp) {
  Group g;
  g.kind = grp < a.gkv ? 0 : grp < 2 * a.gkv ? 1 : 2;
  g.h0 = (grp - g.kind * a.gkv) * kHeads;
  g.nh = min(kHeads, (g.kind == 2 ? a.Hq : a.Hkv) - g.h0);
  return g;
}

// The lane's piece of row t of the group's heads.  Plain loads: with q rotated in
// place the same lane writes these bytes below.
__device__ __forceinline__ void load_rows(const ChunkAppendArgs& a, const Group& g, int t, bool there,
                                          uint4 (&own)[kHeads]) {
  const int e = (threadIdx.x & ((a.d >> 3) - 1)) * 8;
  const __half* src = a.x[g.kind] + (int64_t)t * a.st[g.kind] + (int64_t)g.h0 * a.sh[g.kind] + e;
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    own[u] = make_uint4(0, 0, 0, 0);
    if (there && u < g.nh) own[u] = *reinterpret_cast<const uint4*>(src + u * a.sh[g.kind]);
  }
}

// One warp's unit: the lane's row t of sequence b (live: the lane has one) and
// head group g, its values in `own`.  All lanes of the warp take part.
template <int BITS, bool HYB>
__device__ __forceinline__ void append_unit(const ChunkAppendArgs& a, const Group& g, int t, int b, bool live,
                                            const uint4 (&own)[kHeads]) {
  const int lane = threadIdx.x & 31;
  const int e = (lane & ((a.d >> 3) - 1)) * 8;  // first element of the lane
  const int kind = g.kind;

  Run run = {0, -1};
  SeqLens s = {0, 0, 0, 0};
  if (live) {
    run = run_of(a.cu, b, a.total, a.max_len);
    live = run.n > 0 && t >= run.c0 && t - run.c0 < run.n;
    if (live) s = lens_of(a, b);
  }
  const int i = t - run.c0;

  // the position's cosines and sines
  float2 cs[8];
  const bool rot = live && kind != 1 && e < a.rd;
  const int half = a.rd >> 1;
  const bool second = !a.interleaved && e >= half;
  if (rot) {
    // (what the sequence holds may pass 2^31 with its sink and window)
    int64_t pos = a.positions ? __ldg(a.positions + t) : (int64_t)s.npk + (s.ns + s.nres) + i;
    if (pos < 0 || pos >= a.rope_rows) {
      set_error(a.err_word, KVQ_ERRBIT_BADPOS);
      pos = pos < 0 ? 0 : a.rope_rows - 1;
    }
    const float2* src = a.rope + pos * half + (a.interleaved ? e / 2 : second ? e - half : e);
    const float4* src4 = reinterpret_cast<const float4*>(src);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (a.interleaved && u >= 2) break;
      const float4 f = __ldg(src4 + u);
      cs[2 * u] = make_float2(f.x, f.y);
      cs[2 * u + 1] = make_float2(f.z, f.w);
    }
  }
  const int partner = lane + (second ? -(half >> 3) : half >> 3);
  auto rotated = [&](const uint4& x) {
    uint4 y = x;
    if (a.rd > 0 && kind != 1 && !a.interleaved) {
      y.x = __shfl_sync(0xffffffffu, x.x, partner);
      y.y = __shfl_sync(0xffffffffu, x.y, partner);
      y.z = __shfl_sync(0xffffffffu, x.z, partner);
      y.w = __shfl_sync(0xffffffffu, x.w, partner);
    }
    return rot ? rotate8(x, y, cs, a.interleaved, second) : x;
  };

  if (kind == 2) {
    __half* dst = a.q_out + ((int64_t)t * a.Hq + g.h0) * a.d + e;
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      if (u >= g.nh) break;  // warp-uniform
      const uint4 x = rotated(own[u]);
      if (live) *reinterpret_cast<uint4*>(dst + u * a.d) = x;
    }
    return;
  }

  const Plan plan = plan_of(s, max(run.n, 0), a.cap, a.Nr);
  const int j = s.nres + i;  // place in the line
  const bool taken = live && i < plan.taken;
  const bool direct = taken && j < plan.packed;  // packed straight from the input
  const bool ring = taken && !direct;            // goes to a window slot
  int lap = j, slot = 0;
  if (ring) {
    lap = j % a.Nr;  // ring: the window has slots
    slot = (int)(((int64_t)s.head + j) % a.Nr);
  }
  const bool oust = ring && j >= a.Nr && lap < s.nres;  // a window token leaves the slot
  const bool packs = direct || oust;
  const bool any_pack = __any_sync(0xffffffffu, packs);
  const bool any_oust = __any_sync(0xffffffffu, oust);
  const int64_t row = packs ? a.rm.row(b, 0, s.npk + lap) : -1;  // of KV head 0
  const int64_t row_step = a.rm.paged ? kPage : a.cap;           // to the next head's row
  if (packs && row < 0) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
  const bool ok = packs && row >= 0;
  const int w = kind & 1;
  __half* slot_row = a.res[w] + (((int64_t)b * a.Hkv + g.h0) * a.Nr + slot) * a.d + e;
  const int64_t slot_step = (int64_t)a.Nr * a.d;
  uint4 old[kHeads];
  if (any_oust) {  // warp-uniform
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (oust && u < g.nh) old[u] = *reinterpret_cast<const uint4*>(slot_row + u * slot_step);
  }
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    if (u >= g.nh) break;  // warp-uniform
    const uint4 x = rotated(own[u]);
    if (any_pack) {
      uint32_t prm, asym = 1;
      const uint32_t packed = quantize_quad<BITS>(oust ? old[u] : x, prm, HYB, &asym);
      const uint32_t modes = HYB ? __ballot_sync(0xffffffffu, (lane & 3) == 0 && asym) : 0u;
      const int64_t hr = row + (int64_t)(g.h0 + u) * row_step;
      store_group_codes<BITS>(ok ? a.codes[w] + hr * a.row_bytes + (e >> 5) * (4 * BITS) : nullptr, packed,
                              lane & 3, ok);
      if (ok && (lane & 3) == 0) a.params[w][hr * a.Ng + (e >> 5)] = prm;
      if (HYB && ok && e == 0) a.modes[w][hr] = mode_byte(modes, lane >> 2, a.Ng);
    }
    if (ring) *reinterpret_cast<uint4*>(slot_row + u * slot_step) = x;
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

// The shortest runs: one block per sequence, a warp for each unit, which also moves the
// counters once all have read them.
template <int BITS, bool HYB>
__global__ void __launch_bounds__(kRunThreads) append_run_kernel(ChunkAppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int b = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int tpw = 256 / a.d;  // tokens per warp
  const Run run = run_of(a.cu, b, a.total, a.max_len);
  const int u = threadIdx.x >> 5;
  if (u < (max(run.n, 0) + tpw - 1) / tpw * a.groups) {
    const Group g = group_of(a, u % a.groups);
    const int i = u / a.groups * tpw + lane / (a.d >> 3);
    uint4 own[kHeads];
    load_rows(a, g, run.c0 + i, i < run.n, own);
    append_unit<BITS, HYB>(a, g, run.c0 + i, b, i < run.n, own);
  }
  __syncthreads();
  if (threadIdx.x == 0) finish_seq(a, b);
}

// Other runs: the rows of all of them in one line, a block for 256 / d rows.
template <int BITS, bool HYB>
__global__ void __launch_bounds__(kRowThreads, 6) append_rows_kernel(ChunkAppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const int grp = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (grp >= a.groups) return;  // warp-uniform
  const int64_t t0 = (int64_t)blockIdx.x * (256 / a.d);
  const int64_t t = t0 + lane / (a.d >> 3);
  const bool live = t < a.total;
  const Group g = group_of(a, grp);
  uint4 own[kHeads];
  load_rows(a, g, (int)(live ? t : t0), live, own);
  const int b = seq_of_row(a, t0, t, live);
  append_unit<BITS, HYB>(a, g, (int)(live ? t : t0), b, live, own);
}

// Where entries are out of order (a broken one spoils the two sequences beside it), a row
// that sequence b has may have been given to another: those rows of b, before its counters
// move.  Each has its own place in the line, so when they come makes no difference.
template <int BITS, bool HYB>
__device__ __noinline__ void append_late_rows(const ChunkAppendArgs& a, int b) {
  const Run run = run_of(a.cu, b, a.total, a.max_len);
  if (run.n <= 0) return;
  const int lane = threadIdx.x & 31, tpw = 256 / a.d;
  for (int64_t t0 = run.c0 / tpw * tpw; t0 < (int64_t)run.c0 + run.n; t0 += tpw) {
    const int64_t t = t0 + lane / (a.d >> 3);
    const bool there = t >= run.c0 && t < (int64_t)run.c0 + run.n;
    const bool late = seq_of_row(a, t0, t, there) != b && there;
    if (!__any_sync(0xffffffffu, late)) continue;
    for (int grp = threadIdx.x >> 5; grp < a.groups; grp += blockDim.x >> 5) {
      const Group g = group_of(a, grp);
      uint4 own[kHeads];
      load_rows(a, g, (int)(late ? t : t0), late, own);
      append_unit<BITS, HYB>(a, g, (int)(late ? t : t0), b, late, own);
    }
  }
}

// (on its way while the rows are worked on: reads the entries, then waits for the rows)
template <int BITS, bool HYB>
__global__ void __launch_bounds__(kRowThreads) append_finish_kernel(const __grid_constant__ ChunkAppendArgs a) {
  const int b0 = blockIdx.x * kRowThreads;
  bool falls = false;
  for (int i = threadIdx.x; i < a.B; i += kRowThreads) falls |= __ldg(a.cu + i) > __ldg(a.cu + i + 1);
  falls = __syncthreads_or(falls);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (falls) {
    for (int b = b0; b < min(a.B, b0 + kRowThreads); ++b) append_late_rows<BITS, HYB>(a, b);
    __syncthreads();
  }
  const int b = b0 + threadIdx.x;
  if (b < a.B) finish_seq(a, b);
}

// ------------------------------------------------------------------- read ---

constexpr int kReadThreads = 256;
constexpr int kReadRows = 8;  // pieces of 8 values per thread, one block's width apart, at most

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
  int rows;  // pieces per thread
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

// Eight codes (load_codes8) as values min + code * scale; the product is exact in
// fp32, so the fused form rounds as the sum does.
template <int BITS>
__device__ __forceinline__ void values8(uint32_t codes, uint32_t prm, float (&x)[8]) {
  const float sc = __half2float(__ushort_as_half((unsigned short)(prm & 0xffffu)));
  const float mn = __half2float(__ushort_as_half((unsigned short)(prm >> 16)));
  // codes 0-3 in the low half word, 4-7 in the high one
  const uint32_t y = BITS == 4   ? codes
                     : BITS == 3 ? (codes & 0xfffu) | ((codes & 0xfff000u) << 4)
                                 : (codes & 0xffu) | ((codes & 0xff00u) << 8);
  constexpr uint32_t m = (1u << BITS) - 1u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // the bits in the mantissa of 1024, less 1024
    const uint32_t c = ptx::hadd2_u32(ptx::and_or(y >> (BITS * k), m << 16 | m, 0x64006400u), 0xe400e400u);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c));
    x[k] = __fmaf_rn(f.x, sc, mn);
    x[k + 4] = __fmaf_rn(f.y, sc, mn);
  }
}

template <bool F32>
__device__ __forceinline__ void store_piece(void* out, int64_t at, const float (&x)[8]) {
  if (F32) {
    float4* dst = static_cast<float4*>(out) + 2 * at;
    dst[0] = make_float4(x[0], x[1], x[2], x[3]);
    dst[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 r;
    __half2* hh = reinterpret_cast<__half2*>(&r);
#pragma unroll
    for (int j = 0; j < 4; ++j) hh[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
    static_cast<uint4*>(out)[at] = r;
  }
}

// A quad of lanes per group: each lane turns 8 codes into 8 values, so that the
// quad's stores are the group's contiguous 64 (or 128) bytes.  Output bytes bound
// it.  A block whose tokens are all packed has the loads of all its pieces in
// flight together; the others go piece by piece.  32768 tokens of 8 heads at
// head_dim 128, INT4 to fp16, take 34 us (5.2 TB/s; 70 % of the issue slots).
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
  const int64_t block0 = (int64_t)blockIdx.x * (kReadThreads * a.rows);
  const int64_t p0 = block0 + threadIdx.x;
  const int64_t at = ((int64_t)bh << a.lpr_shift) * a.count + p0;  // pieces of 8 values
  const int e = (int)(p0 & ((1 << a.lpr_shift) - 1)) * 8;          // the same in all the thread's pieces
  const int64_t t0 = max(first, 0) + (p0 >> a.lpr_shift);          // a negative first has n = 0
  const int tstep = kReadThreads >> a.lpr_shift;
  const uint8_t* codes = a.codes[w] + (e >> 5) * (4 * BITS);
  const uint32_t* params = a.params[w] + (e >> 5);

  const int64_t tb = max(first, 0) + (block0 >> a.lpr_shift);
  if (a.rows == kReadRows && tb >= s.ns && tb + kReadRows * tstep <= min(n, (int64_t)s.ns + s.npk) &&
      block0 + kReadRows * kReadThreads <= pieces) {
    int64_t row[kReadRows];
    uint32_t c[kReadRows], prm[kReadRows];
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) row[u] = a.rm.row(b, h, (int)(t0 - s.ns) + u * tstep);
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      c[u] = prm[u] = 0;
      if (row[u] >= 0) {
        c[u] = load_codes8<BITS>(codes + row[u] * a.row_bytes, (e >> 3) & 3);
        prm[u] = __ldg(params + row[u] * a.Ng);
      }
    }
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      if (row[u] < 0) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
      float x[8];
      values8<BITS>(c[u], prm[u], x);
      store_piece<F32>(a.out[w], at + u * kReadThreads, x);
    }
    return;
  }

  const __half* sink = a.sink[w] + (int64_t)bh * a.Ns * a.d + e;
  const __half* res = a.res[w] + (int64_t)bh * a.Nr * a.d + e;
#pragma unroll 1
  for (int u = 0; u < a.rows; ++u) {
    if (p0 + u * kReadThreads >= pieces) break;
    const int64_t t = t0 + u * tstep;
    float x[8] = {};
    if (t < n) {
      if (t >= s.ns && t < s.ns + s.npk) {
        const int64_t row = a.rm.row(b, h, (int)(t - s.ns));
        if (row < 0)
          set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
        else
          values8<BITS>(load_codes8<BITS>(codes + row * a.row_bytes, (e >> 3) & 3), __ldg(params + row * a.Ng), x);
      } else {
        const __half* src = t < s.ns ? sink + t * a.d : res + (t - s.ns - s.npk + s.head) % a.Nr * a.d;
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(src));
        if (!F32) {  // as they are, whatever they hold
          static_cast<uint4*>(a.out[w])[at + u * kReadThreads] = raw;
          continue;
        }
        unpack8_f16(raw, x);
      }
    }
    store_piece<F32>(a.out[w], at + u * kReadThreads, x);
  }
}

// threads: of a block per sequence, or 0.
template <int BITS, bool HYB>
cudaError_t launch_append_bits(const ChunkAppendArgs& a, int threads, cudaStream_t st) {
  if (threads > 0) {
    append_run_kernel<BITS, HYB><<<a.B, threads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int per = 256 / a.d;
  constexpr int kWarps = kRowThreads / 32;
  const dim3 grid((unsigned)((a.total + per - 1) / per), (unsigned)((a.groups + kWarps - 1) / kWarps));
  append_rows_kernel<BITS, HYB><<<grid, kRowThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.B + kRowThreads - 1) / kRowThreads));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_finish_kernel<BITS, HYB>, a);
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
  a.gkv = (a.Hkv + kHeads - 1) / kHeads;
  a.groups = 2 * a.gkv + (a.Hq + kHeads - 1) / kHeads;
  // A block per sequence saves the second launch while each unit has a warp of it: one
  // token of 32 / 8 heads at head_dim 128 takes 5.6 us in place of 5.9, for each of 64
  // sequences 6.3 in place of 7.2.  Clusters of blocks were slower for longer runs (8
  // tokens of 64 sequences 13.0 against 8.5 us).
  const int tpw = 256 / s.d;
  const int64_t len = A.max_len < A.total ? A.max_len : A.total;
  const int64_t units = (len + tpw - 1) / tpw * a.groups;
  const int threads = units > kRunThreads / 32 ? 0 : units < 1 ? 32 : 32 * (int)units;
  if (s.bits == 4)
    return s.hybrid ? launch_append_bits<4, true>(a, threads, st)
                    : launch_append_bits<4, false>(a, threads, st);
  if (s.bits == 3)
    return s.hybrid ? launch_append_bits<3, true>(a, threads, st)
                    : launch_append_bits<3, false>(a, threads, st);
  return s.hybrid ? launch_append_bits<2, true>(a, threads, st)
                  : launch_append_bits<2, false>(a, threads, st);
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
  // few pieces: spread over the SMs, one to a thread, before threads take several
  auto blocks = [&](int rows) { return (pieces + kReadThreads * rows - 1) / (kReadThreads * rows); };
  a.rows = kReadRows;
  while (a.rows > 1 && blocks(a.rows) * s.B * s.Hkv * 2 < 4 * device_sm_count()) a.rows /= 2;
  const bool f32 = (flags & KVQ_OUT_F32) != 0;
  auto kernel = s.bits == 4   ? (f32 ? read_tokens_kernel<4, true> : read_tokens_kernel<4, false>)
                : s.bits == 3 ? (f32 ? read_tokens_kernel<3, true> : read_tokens_kernel<3, false>)
                              : (f32 ? read_tokens_kernel<2, true> : read_tokens_kernel<2, false>);
  kernel<<<dim3((unsigned)blocks(a.rows), (unsigned)(s.B * s.Hkv), 2), kReadThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
