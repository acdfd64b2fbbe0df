// kvq_beam.cu -- beam search's selection over beams and vocabulary.
//
// score(w, t) = s_w + x_wt - log sum_u exp(x_wu); the n best of each batch entry, equal
// ones in the order of beams.  Within a row the order is that of (x, t), so a row's n
// largest logits are all that can be selected of it.
//
// Pass 1, a block for a piece of a row: the piece stays in registers (NV 16-byte vectors
// a thread, loaded at once), which gives its maximum M, sum exp(x - M), and its n
// largest (x, t).  For these a bound comes first: of each thread's largest value each warp
// gives its four largest, and the n-th largest of those is at most the n-th largest of
// the piece.  With ordinary logits a few dozen values pass; each counts those before it,
// and that is its place in the result.  Where many pass (equal logits, rows that are
// masked) the bound is made again with the tokens' order in it.
// Keys are 64 bits: the logit in an order of whole numbers, then the token, inverted, so
// that of equal logits the lower token is the larger key.
// Pass 2, a block for a batch entry: the pieces' sums become the rows' log-normalisers, a
// warp merges some pieces of a row, and each lane works out its entry's score (equal ones of a
// beam keep the order of their logits: a score far from zero has no bits for them).  A bound that
// n scores and not many more are at or above is found bit by bit (a barrier that counts for
// each), and those count what is before them.
//
// Bound: the first pass by what a block does one after the other (loads, bound, sum, what
// passes; three blocks an SM), the second by its chain of merges and barriers.  16 x 8 rows of
// 128256 fp32 logits take 19 us (their bytes alone 10 at the copy rate; pieces of 8 vectors,
// four blocks an SM, 2 % more); 4 rows of 32000 take 5.9, 20 x 16 of 1002 with 32 proposals 11.5
// (four bounds of each warp, whether it has tokens or not, took 1.6 times as long).
#include "kvq_around.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kJoinThreads = 1024;
constexpr int kMaxN = 32;   // a list is a lane each
constexpr int kFew = 256;   // values that are ranked by counting

struct BeamArgs {
  const void* x;
  const float* scores;
  const uint8_t* finished;
  int64_t stride;
  uint64_t* keys;  // [rows][pieces][n]
  float2* ms;      // [rows][pieces]: maximum, sum
  int32_t* parent;
  int32_t* token;
  float* score;
  uint32_t* err_word;
  int W, V, n, end, pieces;
};

// Order of whole numbers that is the order of floats (-0 and 0 alike); 0 is no number's.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t token) {
  return (uint64_t)ordered(v) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) { return a < b ? a : b; }

// A bitonic sequence of the warp's lanes, largest first.
__device__ __forceinline__ uint64_t merge_down(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
    k = (lane & o) ? min64(k, other) : max64(k, other);
  }
  return k;
}
// The warp's keys, largest first.
__device__ __forceinline__ uint64_t sort_down(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size < 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
      k = ((lane & o) == 0) == ((lane & size) == 0) ? max64(k, other) : min64(k, other);
    }
  return merge_down(k);
}
// The 32 largest of two lists, both largest first.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
  return merge_down(max64(a, __shfl_sync(0xffffffffu, b, 31 - (threadIdx.x & 31))));
}

// The lists of the block's warps merged into warp 0's (lists: shared, 32 keys for each).
template <int WARPS>
__device__ __forceinline__ uint64_t merge_warps(uint64_t k, uint64_t (*lists)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = WARPS / 2; o > 0; o >>= 1) {
    if (warp >= o && warp < 2 * o) lists[warp][lane] = k;
    __syncthreads();
    if (warp < o) k = merge_lists(k, lists[warp + o][lane]);
  }
  return k;
}

template <typename T>
struct Vec;
template <>
struct Vec<__half> {
  static constexpr int E = 8;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __half2float(__ushort_as_half((unsigned short)(e & 1 ? w >> 16 : w)));
  }
  static __device__ __forceinline__ uint32_t bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
};

// Tokens t0 .. of a row as a vector; places outside the row hold -inf.
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T* row, uint32_t t0, uint32_t V) {
  constexpr int E = Vec<T>::E;
  uint32_t b[E];
#pragma unroll
  for (int e = 0; e < E; ++e) b[e] = Vec<T>::bits(t0 + e < V ? (float)row[t0 + e] : -INFINITY);
  if constexpr (E == 8)
    return make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
  else
    return make_uint4(b[0], b[1], b[2], b[3]);
}

// The vector that starts `bytes` (below 16) into the two vectors a, b.
__device__ __forceinline__ uint4 from_two(const uint4& a, const uint4& b, int bytes) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
  const int s = (bytes & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                    __funnelshift_r(w[3], w[4], s));
}

// A thread's vectors of a row: tokens t0 + j * kThreads * E ..  What a thread has goes by
// the token alone, not by where the row starts: rows of equal logits have equal sums to
// the last bit, and their tokens stay equal.  Rows that do not start on 16 bytes (odd
// vocabularies) read two neighbouring vectors for each, four at a time.
template <typename T, int NV>
__device__ __forceinline__ void load_vecs(uint4 (&v)[NV], const T* row, uint32_t t0, uint32_t V) {
  constexpr uint32_t E = Vec<T>::E, STEP = kThreads * E;
  const int skip = (int)((uintptr_t)row & 15);
  if (skip == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(row + t0);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t t = t0 + j * STEP;
      if (t + E <= V)
        v[j] = src[j * kThreads];
      else
        v[j] = load_edge(row, t, V);
    }
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + t0) - skip);
#pragma unroll
  for (int g = 0; g < NV; g += 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = t0 + (uint32_t)(g + u) * STEP + 2 * E <= V;  // both vectors end in the row
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (in) a[u] = src[(g + u) * kThreads], b[u] = src[(g + u) * kThreads + 1];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t t = t0 + (uint32_t)(g + u) * STEP;
      v[g + u] = from_two(a[u], b[u], skip);
      if (t + 2 * E > V) v[g + u] = load_edge(row, t, V);
    }
  }
}

// The block's values with the n largest keys, largest first, in warp 0's lanes: the bound
// is made of whole keys.  Each thread gives the key that no value of its largest's vector
// is below; only the n threads that give the largest have values that pass.
template <typename T, int NV>
__device__ __noinline__ uint64_t select_many(const T* row, uint32_t first, uint32_t V, int n, uint64_t (*lists)[32],
                                             uint64_t* passed, int* count) {
  constexpr uint32_t E = Vec<T>::E, WARPS = kThreads / 32, kMost = kMaxN * NV * E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4 v[NV];  // (again: the caller's stay in its registers)
  load_vecs(v, row, first, V);
  uint64_t key = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t t0 = first + j * (kThreads * E);
    if (t0 >= V) break;
    float mx = Vec<T>::get(v[j], 0);
#pragma unroll
    for (int e = 1; e < E; ++e) mx = fmaxf(mx, Vec<T>::get(v[j], e));
    if (key == 0 || ordered(mx) > (uint32_t)(key >> 32)) key = key_of(mx, min(t0 + E, V) - 1);
  }
  key = merge_warps<WARPS>(sort_down(key), lists);
  if (warp == 0 && lane == n - 1) lists[0][0] = key;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  const uint64_t least = lists[0][0];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t t0 = first + j * (kThreads * E);
    if (t0 >= V) break;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t k = key_of(Vec<T>::get(v[j], e), t0 + e);
      if (t0 + e < V && k >= least) {
        const uint32_t at = atomicAdd(count, 1);
        if (at < kMost) passed[at] = k;
      }
    }
  }
  __syncthreads();
  const int c = min(*count, (int)kMost);
  uint64_t k = 0;
  for (int i = warp * 32; i < c; i += kThreads) k = merge_lists(k, sort_down(i + lane < c ? passed[i + lane] : 0));
  return merge_warps<WARPS>(k, lists);
}

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 3) beam_piece_kernel(const __grid_constant__ BeamArgs a) {
  constexpr uint32_t E = Vec<T>::E;
  constexpr int WARPS = kThreads / 32;
  __shared__ uint64_t lists[WARPS][32];
  __shared__ __align__(16) uint64_t passed[kMaxN * NV * E];  // (at least kFew)
  __shared__ __align__(16) uint32_t tops[32];
  __shared__ uint32_t top[WARPS];
  __shared__ float part[WARPS];
  __shared__ int count;
  wait_for_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int piece = blockIdx.x, r = blockIdx.y;
  if (a.finished && a.finished[r]) return;  // (the second pass does not look at such a row)
  const T* row = static_cast<const T*>(a.x) + (int64_t)r * a.stride;
  const uint32_t first = (uint32_t)piece * (kThreads * NV * E) + tid * E, V = a.V;
  uint64_t* out = a.keys + ((int64_t)r * a.pieces + piece) * a.n;

  uint4 v[NV];  // (places outside the row hold -inf)
  load_vecs(v, row, first, V);
  if (tid == 0) count = 0;

  // the thread's largest, and of those the warp's four largest (more, where the row's end
  // leaves warps without tokens: 32 in all).  Their last five bits are a number of their
  // own, so that no two are equal: the bound is made of the others
  float best = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) best = fmaxf(best, Vec<T>::get(v[j], e));
  uint32_t left = first < V ? ordered(best) : 0;
  const uint32_t behind = V - (first - tid * E);  // tokens from the piece's first on
  const int share = behind >= kThreads * E ? 0 : __ffs(WARPS) - 1 - (31 - __clz((behind + 32 * E - 1) / (32 * E)));
  const int mine_tops = (32 / WARPS) << share;
  if (lane == 0) top[warp] = 0;
#pragma unroll 4
  for (int i = 0; i < mine_tops; ++i) {
    const uint32_t x = __reduce_max_sync(0xffffffffu, left);
    if (lane == 0 && warp * mine_tops + i < 32) tops[warp * mine_tops + i] = (x & ~31u) | (warp * mine_tops + i);
    if (lane == 0 && i == 0) top[warp] = x;
    if (lane == __ffs(__ballot_sync(0xffffffffu, left == x)) - 1) left = 0;
  }
  __syncthreads();
  // the n-th largest of the 32 (0: there are not so many values), and the largest
  const uint32_t mine = tops[lane];
  int above = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(tops + i);
    above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
  }
  const uint32_t least =
      __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, above == a.n - 1)) - 1) & ~31u;
  const float m = unordered(__reduce_max_sync(0xffffffffu, top[lane % WARPS]));

  // sum exp(x - M): differences first, so that the largest terms' exponents are exact
  const float off = m == -INFINITY ? 0.0f : m;
  const uint64_t off2 = pack_f32x2(off, off), log2e2 = pack_f32x2(1.4426950408889634f, 1.4426950408889634f);
  uint64_t sum2 = 0;  // (two zeros)
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const uint64_t x =
          mul_f32x2(sub_f32x2(pack_f32x2(Vec<T>::get(v[j], e), Vec<T>::get(v[j], e + 1)), off2), log2e2);
      sum2 = add_f32x2(sum2, pack_f32x2(ptx::ex2_ftz(__uint_as_float(lo_bits(x))),
                                        ptx::ex2_ftz(__uint_as_float(hi_bits(x)))));
    }
  float sum = __uint_as_float(lo_bits(sum2)) + __uint_as_float(hi_bits(sum2));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[warp] = sum;

  // what passes the bound: vectors first, whose values are then read again
  const float least_v = least < 0x00800000u ? -INFINITY : unordered(least);  // (below the lowest finite one)
  uint32_t vecs = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float mx = Vec<T>::get(v[j], 0);
#pragma unroll
    for (int e = 1; e < E; ++e) mx = fmaxf(mx, Vec<T>::get(v[j], e));
    vecs |= mx >= least_v ? 1u << j : 0u;
  }
  while (vecs) {
    const uint32_t t0 = first + (__ffs(vecs) - 1) * (kThreads * E);
    vecs &= vecs - 1;
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) {
      const float x = t0 + e < V ? (float)row[t0 + e] : -INFINITY;
      if (x >= least_v && t0 + e < V) {
        const int at = atomicAdd(&count, 1);
        if (at < kFew) passed[at] = key_of(x, t0 + e);
      }
    }
  }
  __syncthreads();
  const int c = count;
  if (c <= kFew) {
    if (tid < max(c, a.n)) {
      const uint64_t k = tid < c ? passed[tid] : 0;
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < c; ++i) place += passed[i] > k;
      if (tid >= c) place = tid;  // (a piece of fewer than n tokens: no token)
      if (place < a.n) out[place] = k;
    }
  } else {
    const uint64_t k = select_many<T, NV>(row, first, V, a.n, lists, passed, &count);
    if (warp == 0 && lane < a.n) out[lane] = k;
  }
  if (tid == 0) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) s += part[i];
    a.ms[(int64_t)r * a.pieces + piece] = make_float2(m, s);
  }
}

// Scores are two fp32 parts, hi + lo with |lo| at most half a step of hi (the chip has few
// units for doubles).  The sum of two numbers so:
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// ... of 53 bits, as a double has: what lies below is not told apart (tokens masked by the
// type's lowest value come in order, whatever their beams' scores)
__device__ __forceinline__ Two of_53_bits(Two v) {
  const int e = (int)(__float_as_uint(v.hi) & 0x7f800000u) - (29 << 23);
  if (e > 0) {
    const float c = 1.5f * __int_as_float(e);
    v.lo = __fsub_rn(__fadd_rn(v.lo, c), c);
  }
  return v;
}
__device__ __forceinline__ uint64_t ordered(const Two& v) { return (uint64_t)ordered(v.hi) << 32 | ordered(v.lo); }

// m + log s, 0 < s.  The exponent of s apart, so that the logarithm is rounded near zero.
__device__ __forceinline__ Two log_norm(float m, float s) {
  int e = 0;
  const float f = frexpf(s, &e);
  // log 2 as a part of few bits, whose product with e is exact, and the rest (Cody, Waite)
  const float hi = 0.693359375f, lo = -2.12194440e-4f;
  const Two a = two_sum(m, __fmul_rn((float)e, hi));
  const Two b = two_sum(a.hi, __fadd_rn(logf(f), __fmul_rn((float)e, lo)));
  return two_sum(b.hi, __fadd_rn(a.lo, b.lo));
}

__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int WARPS = kJoinThreads / 32;
  constexpr int AHEAD = 4;     // lists in flight
  constexpr int kEnough = 64;  // entries that are ranked by counting
  __shared__ __align__(16) uint64_t passed[kJoinThreads];
  __shared__ __align__(16) int2 passed_at[kJoinThreads];  // place (beam * V + token), logit in order
  __shared__ int count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // warp i has row i % W and, of its pieces, every (WARPS / W)-th
  const int per = WARPS / a.W;
  const int w = warp % a.W, part = warp / a.W;
  const int64_t r = (int64_t)blockIdx.x * a.W + w;
  if (tid == 0) count = 0;
  wait_for_previous();
  const float base = a.scores[r];
  const bool done = a.finished && a.finished[r];
  const bool read = part < per && !done;
  const float2 sums = read && lane < a.pieces ? __ldcg(a.ms + r * a.pieces + lane) : make_float2(-INFINITY, 0.0f);

  uint64_t k = 0;
  if (read && base > -INFINITY && base < INFINITY) {
    const uint64_t* src = a.keys + r * a.pieces * a.n + lane;
    for (int i = part; i < a.pieces; i += per * AHEAD) {
      uint64_t x[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int at = i + u * per;
        x[u] = at < a.pieces && lane < a.n ? __ldcg(src + (int64_t)at * a.n) : 0;
      }
      if (i == part) k = x[0];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if ((u > 0 || i > part) && __shfl_sync(0xffffffffu, x[u], 0) > __shfl_sync(0xffffffffu, k, a.n - 1))
          k = merge_lists(k, x[u]);
    }
  }

  // the row's normaliser
  Two norm = {0.0f, 0.0f};
  bool bad = !(base < INFINITY);  // +inf or NaN
  if (read) {
    float m = sums.x;
    for (int i = lane + 32; i < a.pieces; i += 32) m = fmaxf(m, __ldcg(a.ms + r * a.pieces + i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.0f;
    for (int i = lane; i < a.pieces; i += 32) {
      const float2 x = i == lane ? sums : __ldcg(a.ms + r * a.pieces + i);
      // a piece without a maximum has a sum of 0, or NaN
      s += x.x == -INFINITY ? x.y : x.y * ptx::ex2_ftz((x.x - m) * 1.4426950408889634f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    bad = bad || !(m < INFINITY) || s != s;
    norm.hi = -INFINITY;
    if (s > 0.0f) norm = log_norm(m, s);
  }
  if (bad && part == 0 && lane == 0) set_error(a.err_word, KVQ_ERRBIT_BADSCORE);

  // the lane's proposal
  const uint64_t silent = ordered(Two{-INFINITY, 0.0f});
  uint64_t score = 0;  // none, behind all others
  int at = 0x7fffffff;
  uint32_t logit = 0;  // in order; tokens that are not proposed have none
  if (part < per) {
    if (bad || done || base == -INFINITY || norm.hi == -INFINITY) {
      // proposes its end alone, or nothing: the row's first tokens follow at -inf
      if (part == 0 && lane < min(a.n, a.V)) {
        const bool ends = done && !bad && base > -INFINITY;
        score = ends && lane == 0 ? ordered(Two{base, 0.0f}) : silent;
        at = w * a.V + (!ends ? lane : lane == 0 ? a.end : lane - (lane <= a.end));
      }
    } else if (k != 0) {
      logit = (uint32_t)(k >> 32);
      const float x = unordered(logit);
      const Two d = two_sum(x, -norm.hi);
      const Two b = two_sum(base, d.hi);
      // (below fp32's range: -inf)
      score = x == -INFINITY || !(b.hi > -INFINITY) ? silent : ordered(of_53_bits(two_sum(b.hi, b.lo + (d.lo - norm.lo))));
      at = w * a.V + (int)~(uint32_t)k;
    }
  }
  // the scores' upper half that n entries, and few more, are not below, bit by bit
  const uint32_t top = (uint32_t)(score >> 32);
  uint32_t least = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const int c = __syncthreads_count(top >= (least | 1u << bit));
    if (c >= a.n) least |= 1u << bit;
    if (c >= a.n && c <= kEnough) break;
  }
  if (top >= least && score != 0) {
    const int i = atomicAdd(&count, 1);
    passed[i] = score;
    passed_at[i] = make_int2(at, (int)logit);
  }
  __syncthreads();
  const int c = count;
  if (tid < c) {
    const uint64_t s = passed[tid];
    const int mine = passed_at[tid].x, beam = mine / a.V;
    const uint32_t own = (uint32_t)passed_at[tid].y;
    // of equal scores the first beam's, of a beam's the largest logit's, then the first token's
    int place = 0;
#pragma unroll 4
    for (int i = 0; i < c; ++i) {
      const int2 o = passed_at[i];
      const bool larger = (uint32_t)(o.x - beam * a.V) < (uint32_t)a.V && (uint32_t)o.y != own
                              ? (uint32_t)o.y > own
                              : o.x < mine;
      place += passed[i] > s || (passed[i] == s && larger);
    }
    if (place < a.n) {
      const int64_t to = (int64_t)blockIdx.x * a.n + place;
      a.parent[to] = blockIdx.x * a.W + beam;
      a.token[to] = mine - beam * a.V;
      a.score[to] = unordered((uint32_t)(s >> 32));
    }
  }
}

// Vectors of a thread: as many as registers hold, or a third of that where the larger
// pieces would leave SMs without a block (two on each).
int vectors(int64_t rows, int vocab, bool f32) {
  const int64_t big = (int64_t)kThreads * 12 * (f32 ? 4 : 8);
  return rows * ((vocab + big - 1) / big) >= 2 * device_sm_count() ? 12 : 4;
}
int pieces_of(int vocab, int nv, bool f32) {
  const int64_t size = (int64_t)kThreads * nv * (f32 ? 4 : 8);
  return (int)(((int64_t)vocab + size - 1) / size);
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// For either type of logits and either size of piece.
size_t beam_workspace_bytes(int batch, int beams, int vocab, int n) {
  const size_t lists = (size_t)batch * beams * pieces_of(vocab, 4, true);
  return up(lists * n * sizeof(uint64_t)) + up(lists * sizeof(float2));
}

cudaError_t launch_beam_select(const kvq_beam_args& args, cudaStream_t st) {
  const bool f32 = args.flags & KVQ_LOGITS_F32;
  const int64_t rows = (int64_t)args.batch * args.beams;
  const int nv = vectors(rows, args.vocab, f32);
  BeamArgs a;
  a.x = args.logits;
  a.scores = args.scores;
  a.finished = args.finished;
  a.stride = args.stride_row;
  a.parent = args.parent;
  a.token = args.token;
  a.score = args.score;
  a.err_word = args.err_word;
  a.W = args.beams;
  a.V = args.vocab;
  a.n = args.n;
  a.end = args.end_token;
  a.pieces = pieces_of(args.vocab, nv, f32);
  a.keys = static_cast<uint64_t*>(args.workspace);
  a.ms = reinterpret_cast<float2*>(static_cast<char*>(args.workspace) +
                                   up((size_t)rows * a.pieces * a.n * sizeof(uint64_t)));
  const dim3 grid(a.pieces, (unsigned)rows);
  cudaError_t e;
  if (f32)
    e = nv == 12 ? launch_overlapped(beam_piece_kernel<float, 12>, grid, kThreads, 0, st, a)
                 : launch_overlapped(beam_piece_kernel<float, 4>, grid, kThreads, 0, st, a);
  else
    e = nv == 12 ? launch_overlapped(beam_piece_kernel<__half, 12>, grid, kThreads, 0, st, a)
                 : launch_overlapped(beam_piece_kernel<__half, 4>, grid, kThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_overlapped(beam_join_kernel, dim3(args.batch), kJoinThreads, 0, st, a);
}

}  // namespace kvq
