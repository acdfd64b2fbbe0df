// kvq_beam.cu -- beam search's selection over beams and vocabulary.
//
// score(w, t) = s_w + x_wt - log sum_u exp(x_wu); the n best of each batch entry, equal
// ones in the order of (w, t).  Within a row the order is that of (x, t), so a row's n
// largest logits are all that can be selected of it.
//
// Pass 1, a block for a piece of a row: the piece stays in registers (kNV 16-byte vectors
// a thread, loaded at once), which gives its maximum M, sum exp(x - M), and its n
// largest (x, t).  For these a bound comes first: each thread's largest, and the n-th
// largest of those; all that can be in the result is at or above it, in n threads at
// most.  With ordinary logits a few more than n values pass, and one warp sorts them.
// Keys are 64 bits: the logit in an order of whole numbers, then the token, inverted, so
// that of equal logits the lower token is the larger key.
// Pass 2, a block for a batch entry: the pieces' sums become the rows' log-normalisers (64
// bits), a warp merges some pieces of a row, then the warps' lists are merged by the
// scores in 64 bits.
//
// Bound: memory for large batches (the logits are read once), the two launches and the
// chain of merges for a few rows.
#include "kvq_around.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kJoinThreads = 1024;
constexpr int kMaxN = 32;  // a list is a lane each

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
__device__ __forceinline__ uint4 load_edge(const T* row, int64_t t0, int V) {
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
__device__ __forceinline__ void load_vecs(uint4 (&v)[NV], const T* row, int64_t t0, int V) {
  constexpr int E = Vec<T>::E, STEP = kThreads * E;
  const int skip = (int)((uintptr_t)row & 15);
  if (skip == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t t = t0 + j * STEP;
      v[j] = make_uint4(0, 0, 0, 0);
      if (t + E <= V)
        v[j] = __ldg(reinterpret_cast<const uint4*>(row + t));
      else if (t < V)
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
      const bool in = t0 + (g + u) * STEP + 2 * E <= V;  // both vectors end in the row
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (in) a[u] = __ldg(src + (g + u) * kThreads), b[u] = __ldg(src + (g + u) * kThreads + 1);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t t = t0 + (g + u) * STEP;
      v[g + u] = from_two(a[u], b[u], skip);
      if (t + 2 * E > V && t < V) v[g + u] = load_edge(row, t, V);
    }
  }
}

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 2) beam_piece_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int E = Vec<T>::E;
  constexpr int WARPS = kThreads / 32;
  constexpr int kMost = kMaxN * NV * E;  // values that can pass the bound
  __shared__ uint64_t lists[WARPS][32];
  __shared__ uint64_t passed[kMost];
  __shared__ uint64_t bound;
  __shared__ float part[WARPS];
  __shared__ int count;
  wait_for_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int piece = blockIdx.x, r = blockIdx.y;
  if (a.finished && a.finished[r]) return;  // (the second pass does not look at such a row)
  const T* row = static_cast<const T*>(a.x) + (int64_t)r * a.stride;
  const int64_t first = (int64_t)piece * (kThreads * NV * E) + tid * E;

  uint4 v[NV];
  load_vecs(v, row, first, a.V);
  if (tid == 0) count = 0;

  // the thread's largest, and the key that no value of that vector with it is below
  float best = -INFINITY;
  uint64_t key = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t t0 = first + (int64_t)j * (kThreads * E);
    if (t0 >= a.V) break;
    float mx = Vec<T>::get(v[j], 0);
#pragma unroll
    for (int e = 1; e < E; ++e) mx = fmaxf(mx, Vec<T>::get(v[j], e));
    if (key == 0 || mx > best) {
      best = fmaxf(mx, best);
      key = key_of(best, (uint32_t)min(t0 + E, (int64_t)a.V) - 1);
    }
  }
  float m = best;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) part[warp] = m;
  key = merge_warps<WARPS>(sort_down(key), lists);  // (its barriers are part's and count's too)
#pragma unroll
  for (int i = 0; i < WARPS; ++i) m = fmaxf(m, part[i]);
  if (warp == 0 && lane == a.n - 1) bound = key;

  // sum exp(x - M): differences first, so that the largest terms' exponents are exact
  float sum = 0.0f, sum2 = 0.0f;
  const float off = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (first + (int64_t)j * (kThreads * E) >= a.V) break;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      sum += exp2f((Vec<T>::get(v[j], e) - off) * 1.4426950408889634f);
      sum2 += exp2f((Vec<T>::get(v[j], e + 1) - off) * 1.4426950408889634f);
    }
  }
  sum += sum2;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();  // part has been read, bound is there
  if (lane == 0) part[warp] = sum;

  // what passes the bound
  const uint64_t least = bound;
  const float least_v = unordered((uint32_t)(least >> 32));
  if (least == 0 || best >= least_v) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t t0 = first + (int64_t)j * (kThreads * E);
      if (t0 >= a.V) break;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = Vec<T>::get(v[j], e);
        if (least != 0 && !(x >= least_v)) continue;
        const int64_t t = t0 + e;
        const uint64_t k = key_of(x, (uint32_t)t);
        if (t < a.V && k >= least) {
          const int at = atomicAdd(&count, 1);
          if (at < kMost) passed[at] = k;
        }
      }
    }
  }
  __syncthreads();
  const int c = min(count, kMost);
  uint64_t k = 0;
  if (c <= 32) {
    if (warp == 0) k = sort_down(lane < c ? passed[lane] : 0);
  } else {
    for (int i = warp * 32; i < c; i += kThreads) k = merge_lists(k, sort_down(i + lane < c ? passed[i + lane] : 0));
    k = merge_warps<WARPS>(k, lists);
  }
  const int64_t at = (int64_t)r * a.pieces + piece;
  if (warp == 0 && lane < a.n) a.keys[at * a.n + lane] = k;
  if (tid == 0) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) s += part[i];
    a.ms[at] = make_float2(m, s);
  }
}

// A proposal: its score and its place w * V + t, larger in the order of the result.
struct Prop {
  double s;
  int at;
};
__device__ __forceinline__ bool before(const Prop& a, const Prop& b) {
  return a.s > b.s || (a.s == b.s && a.at < b.at);
}
__device__ __forceinline__ Prop shfl(const Prop& p, int src) {
  return {__shfl_sync(0xffffffffu, p.s, src), __shfl_sync(0xffffffffu, p.at, src)};
}
__device__ __forceinline__ Prop merge_props(const Prop& a, const Prop& b) {
  const int lane = threadIdx.x & 31;
  const Prop r = shfl(b, 31 - lane);
  Prop p = before(a, r) ? a : r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Prop q = shfl(p, lane ^ o);
    if (before(p, q) == ((lane & o) != 0)) p = q;
  }
  return p;
}

__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int WARPS = kJoinThreads / 32;
  __shared__ double list_s[WARPS][32];
  __shared__ int list_at[WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warp i has row i % W and, of its pieces, every (WARPS / W)-th
  const int per = WARPS / a.W;
  const int w = warp % a.W, part = warp / a.W;
  const int64_t r = (int64_t)blockIdx.x * a.W + w;
  wait_for_previous();
  Prop p = {-INFINITY, 0x7fffffff};
  if (part < per) {
    const float base = __ldg(a.scores + r);
    const bool done = a.finished && __ldg(a.finished + r);
    // the row's normaliser
    double norm = 0.0;
    bool bad = !(base < INFINITY);  // +inf or NaN
    if (!done) {
      float m = -INFINITY;
      for (int i = lane; i < a.pieces; i += 32) m = fmaxf(m, __ldcg(a.ms + r * a.pieces + i).x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double s = 0.0;
      for (int i = lane; i < a.pieces; i += 32) {
        const float2 x = __ldcg(a.ms + r * a.pieces + i);
        // a piece without a maximum has a sum of 0, or NaN
        s += x.x == -INFINITY ? (double)x.y : (double)x.y * exp((double)x.x - (double)m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      bad = bad || !(m < INFINITY) || s != s;
      norm = (double)m + log(s);
    }
    if (bad && part == 0 && lane == 0) set_error(a.err_word, KVQ_ERRBIT_BADSCORE);
    if (bad || done || base == -INFINITY || norm == -INFINITY) {
      // proposes its end alone, or nothing: the row's first tokens follow at -inf
      if (part == 0 && lane < min(a.n, a.V)) {
        const bool ends = done && !bad;
        const int t = !ends ? lane : lane == 0 ? a.end : lane - (lane <= a.end);
        p.s = ends && lane == 0 ? (double)base : -INFINITY;
        p.at = w * a.V + t;
      }
    } else {
      uint64_t k = 0;
      for (int i = part; i < a.pieces; i += per) {
        const uint64_t x = lane < a.n ? __ldcg(a.keys + (r * a.pieces + i) * a.n + lane) : 0;
        if (__shfl_sync(0xffffffffu, x, 0) > __shfl_sync(0xffffffffu, k, a.n - 1)) k = merge_lists(k, x);
      }
      if (k != 0) {
        p.s = (double)base + ((double)unordered((uint32_t)(k >> 32)) - norm);
        p.at = w * a.V + (int)~(uint32_t)k;
      }
    }
  }
#pragma unroll
  for (int o = WARPS / 2; o > 0; o >>= 1) {
    if (warp >= o && warp < 2 * o) list_s[warp][lane] = p.s, list_at[warp][lane] = p.at;
    __syncthreads();
    if (warp < o) p = merge_props(p, {list_s[warp + o][lane], list_at[warp + o][lane]});
  }
  if (warp == 0 && lane < a.n) {
    const int64_t at = (int64_t)blockIdx.x * a.n + lane;
    const int beam = p.at / a.V;
    a.parent[at] = blockIdx.x * a.W + beam;
    a.token[at] = p.at - beam * a.V;
    a.score[at] = (float)p.s;
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
