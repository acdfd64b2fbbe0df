// kvq_reorder.cu -- sequences copied from one cache to another by an index.
//
// All that a destination sequence gets is cut into runs for one warp each: of one array
// kind and KV head the packed rows of some tokens (codes, params, modes), some slots of the
// window, some rows of the sink; and one run for counters and block table.  The runs of
// all sequences lie in one line (lengths are read on the device), warps take them in turn.
// A warp has all its loads of a run, up to 5 KB, in flight before it stores.  Only live
// bytes are read or written.
//
// Bound by memory: every live byte is read once and written once.  4 sequences of 32768
// tokens, 8 heads, INT4: 56 us, 89 % of the measured copy rate (loads through the cache and
// streaming stores; plain stores 59, loads past the first cache 57; read-only loads 55.5, but
// the kernel before may be writing).  32 sequences with shared pages: 8.1 us, of which the
// lengths' dependent loads and the launch are 4.
#include "kvq_runs.cuh"

#include "kvq_around.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 3;         // of an SM
constexpr int kCodeBytes = 4096;  // of a run, at most

struct Arrays {
  uint8_t* codes[2];
  uint8_t* params[2];
  uint8_t* modes[2];
  uint8_t* res[2];
  uint8_t* sink[2];
  int32_t* table;
  int32_t *packed_len, *res_len, *res_head, *sink_len;
  int B, cap, npages;
};

struct ReorderArgs {
  Arrays s, d;
  const int32_t* index;
  uint32_t* err_word;
  int Hkv, rb, pb, fb;  // bytes of a row: codes, params, fp16
  int Nr, Ns, paged, share, hybrid;
  int chunk;            // tokens of a run of packed rows
  int slots;            // rows of a run of fp16 ones
};

// The warp's 16-byte words of a run into registers, and from there.
template <int N>
__device__ __forceinline__ void load(uint4 (&v)[N], const uint8_t* src, int bytes) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if ((i * 32 + lane) * 16 < bytes) v[i] = reinterpret_cast<const uint4*>(src)[i * 32 + lane];
  }
}
template <int N>
__device__ __forceinline__ void store(const uint4 (&v)[N], uint8_t* dst, int bytes) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((i * 32 + lane) * 16 < bytes) __stcs(reinterpret_cast<uint4*>(dst) + i * 32 + lane, v[i]);
}
// Rows that start anywhere (heads of 32 or 64 with odd capacities), and mode bytes: words
// where both sides and the length allow (four loads in flight), else bytes.
__device__ __forceinline__ void copy_any(uint8_t* dst, const uint8_t* src, int bytes) {
  const int lane = threadIdx.x & 31;
  if ((((uint32_t)(uintptr_t)dst | (uint32_t)(uintptr_t)src | (uint32_t)bytes) & 3) == 0) {
    const int n = bytes / 4;
    for (int i = lane; i < n; i += 128) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = i + 32 * u < n ? reinterpret_cast<const uint32_t*>(src)[i + 32 * u] : 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + 32 * u < n) reinterpret_cast<uint32_t*>(dst)[i + 32 * u] = v[u];
    }
  } else {
#pragma unroll 1
    for (int i = lane; i < bytes; i += 32) dst[i] = src[i];
  }
}

// What destination sequence i gets: from sequence a of the source; a < 0: nothing.
struct Plan {
  int a;
  SeqLens len;
  int t0;                          // first packed token that moves
  int chunks, rings, sinks, runs;  // runs of each kind for one array and head; of the sequence
};

__device__ __forceinline__ Plan plan_of(const ReorderArgs& g, int i, bool report) {
  Plan p;
  p.runs = 0;
  p.a = g.index[i];
  if (p.a < 0 || p.a >= g.s.B) {
    if (report) set_error(g.err_word, KVQ_ERRBIT_BADINDEX);
    p.a = -1;
    return p;
  }
  p.len = seq_lens_of(g.s.sink_len, g.s.packed_len, g.s.res_len, g.s.res_head, p.a, g.Ns, g.s.cap, g.Nr);
  if (p.len.npk > g.d.cap) {
    if (report) set_error(g.err_word, KVQ_ERRBIT_CAPACITY);
    p.a = -1;
    return p;
  }
  p.t0 = g.share ? p.len.npk / kPage * kPage : 0;
  p.chunks = (p.len.npk - p.t0 + g.chunk - 1) / g.chunk;
  p.rings = p.len.nres > 0 ? (g.Nr + g.slots - 1) / g.slots : 0;
  p.sinks = (p.len.ns + g.slots - 1) / g.slots;
  p.runs = 1 + 2 * g.Hkv * (p.chunks + p.rings + p.sinks);
  return p;
}

__device__ __forceinline__ void packed_run(const ReorderArgs& g, const Plan& p, int i, int w, int h, int c) {
  const int lane = threadIdx.x & 31;
  const int t = p.t0 + c * g.chunk, rows = min(g.chunk, p.len.npk - t);
  int64_t from, to;
  if (g.paged) {  // a run is a page of one head
    const int ps = g.s.table[(int64_t)p.a * (g.s.cap / kPage) + t / kPage];
    const int pd = g.d.table[(int64_t)i * (g.d.cap / kPage) + t / kPage];
    if (ps < 0 || ps >= g.s.npages || pd < 0 || pd >= g.d.npages) {
      if (lane == 0) set_error(g.err_word, KVQ_ERRBIT_BADPAGE);
      return;
    }
    from = ((int64_t)ps * g.Hkv + h) * kPage;
    to = ((int64_t)pd * g.Hkv + h) * kPage;
  } else {
    from = ((int64_t)p.a * g.Hkv + h) * g.s.cap + t;
    to = ((int64_t)i * g.Hkv + h) * g.d.cap + t;
  }
  const uint8_t* cs = g.s.codes[w] + from * g.rb;
  const uint8_t* ps = g.s.params[w] + from * g.pb;
  uint8_t* cd = g.d.codes[w] + to * g.rb;
  uint8_t* pd = g.d.params[w] + to * g.pb;
  const int nc = rows * g.rb, np = rows * g.pb;
  const uint32_t any = (uint32_t)(uintptr_t)cs | (uint32_t)(uintptr_t)cd | (uint32_t)nc |
                       (uint32_t)(uintptr_t)ps | (uint32_t)(uintptr_t)pd | (uint32_t)np;
  if ((any & 15) == 0) {
    uint4 vc[kCodeBytes / 512], vp[kCodeBytes / 1024];
    load(vc, cs, nc);
    load(vp, ps, np);
    store(vc, cd, nc);
    store(vp, pd, np);
  } else {
    copy_any(cd, cs, nc);
    copy_any(pd, ps, np);
  }
  if (g.hybrid) copy_any(g.d.modes[w] + to, g.s.modes[w] + from, rows);
}

__device__ __forceinline__ void copy_run(const ReorderArgs& g, const Plan& p, int i, int x) {
  const int lane = threadIdx.x & 31;
  if (x == 0) {
    if (lane == 0) {
      g.d.packed_len[i] = p.len.npk;
      g.d.res_len[i] = p.len.nres;
      g.d.res_head[i] = p.len.head;
      if (g.Ns > 0) g.d.sink_len[i] = p.len.ns;
    }
    if (g.share)
      for (int j = lane; j < p.t0 / kPage; j += 32)
        g.d.table[(int64_t)i * (g.d.cap / kPage) + j] = g.s.table[(int64_t)p.a * (g.s.cap / kPage) + j];
    return;
  }
  x -= 1;
  const int of = p.chunks + p.rings + p.sinks;
  const int wh = x / of, w = wh & 1, h = wh >> 1;
  x -= wh * of;
  if (x < p.chunks) {
    packed_run(g, p, i, w, h, x);
    return;
  }
  x -= p.chunks;
  uint4 v[kCodeBytes / 512];
  const int shift = __ffs(g.fb / 16) - 1;  // a row is 2^shift words
  const bool ring = x < p.rings;
  const int n = ring ? g.Nr : g.Ns;
  const int r0 = (ring ? x : x - p.rings) * g.slots;
  const int64_t from = (((int64_t)p.a * g.Hkv + h) * n + r0) * g.fb;
  const int64_t to = (((int64_t)i * g.Hkv + h) * n + r0) * g.fb;
  const uint8_t* src = (ring ? g.s.res : g.s.sink)[w] + from;
  uint8_t* dst = (ring ? g.d.res : g.d.sink)[w] + to;
  // rows that are live: of the ring nres slots from its head on, of the sink the first ns
  auto live = [&](int at) {
    const int row = r0 + (at >> shift);
    if (row >= n) return false;
    if (!ring) return row < p.len.ns;
    const int age = row - p.len.head;
    return (age < 0 ? age + n : age) < p.len.nres;
  };
#pragma unroll
  for (int j = 0; j < kCodeBytes / 512; ++j) {
    const int at = j * 32 + lane;
    v[j] = make_uint4(0, 0, 0, 0);
    if (live(at)) v[j] = reinterpret_cast<const uint4*>(src)[at];
  }
#pragma unroll
  for (int j = 0; j < kCodeBytes / 512; ++j) {
    const int at = j * 32 + lane;
    if (live(at)) __stcs(reinterpret_cast<uint4*>(dst) + at, v[j]);
  }
}

__global__ void __launch_bounds__(kThreads, kBlocks) reorder_kernel(const __grid_constant__ ReorderArgs g) {
  __shared__ int64_t ends[kThreads];  // runs of 256 sequences, summed up
  __shared__ int64_t sums[kThreads / 32];
  wait_for_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // neighbouring runs go to different blocks: those of one sequence are of one length
  int64_t x = (int64_t)warp * gridDim.x + blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  int64_t base = 0;
  for (int b0 = 0; b0 < g.d.B; b0 += kThreads) {
    const int mine = b0 + tid;
    int64_t scan = mine < g.d.B ? plan_of(g, mine, blockIdx.x == 0).runs : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    __syncthreads();  // the last 256 have been read
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    for (int i = 0; i < warp; ++i) scan += sums[i];
    ends[tid] = base + scan;
    __syncthreads();
    const int64_t end = ends[kThreads - 1];
    int at = -1;
    Plan p;
    for (; x < end; x += step) {  // (x is the warp's)
      int lo = 0;
#pragma unroll
      for (int o = kThreads / 2; o > 0; o >>= 1)
        if (ends[lo + o - 1] <= x) lo += o;
      if (lo != at) p = plan_of(g, b0 + lo, false);
      at = lo;
      copy_run(g, p, b0 + lo, (int)(x - (lo > 0 ? ends[lo - 1] : base)));
    }
    base = end;
  }
}

Arrays arrays_of(const Dims& s, const kvq_cache_view& v) {
  Arrays a;
  a.codes[0] = v.k_codes, a.codes[1] = v.v_codes;
  a.params[0] = reinterpret_cast<uint8_t*>(v.k_params), a.params[1] = reinterpret_cast<uint8_t*>(v.v_params);
  a.modes[0] = v.k_mode, a.modes[1] = v.v_mode;
  a.res[0] = reinterpret_cast<uint8_t*>(v.k_res), a.res[1] = reinterpret_cast<uint8_t*>(v.v_res);
  a.sink[0] = reinterpret_cast<uint8_t*>(v.k_sink), a.sink[1] = reinterpret_cast<uint8_t*>(v.v_sink);
  a.table = v.block_table;
  a.packed_len = v.packed_len, a.res_len = v.res_len, a.res_head = v.res_head, a.sink_len = v.sink_len;
  a.B = s.B, a.cap = s.cap, a.npages = s.npages;
  return a;
}

}  // namespace

cudaError_t launch_reorder(const Dims& d, const kvq_cache_view& dv, const Dims& s, const kvq_cache_view& sv,
                           const int32_t* index, bool share, cudaStream_t st) {
  ReorderArgs g;
  g.s = arrays_of(s, sv);
  g.d = arrays_of(d, dv);
  g.index = index;
  g.err_word = dv.err_word;
  g.Hkv = d.Hkv;
  g.rb = d.row_bytes;
  g.pb = d.Ng * 4;
  g.fb = d.d * 2;
  g.Nr = d.Nr;
  g.Ns = d.Ns;
  g.paged = d.page != 0;
  g.share = share;
  g.hybrid = d.hybrid;
  // whole pages where there are pages, as many rows as the loads in flight hold otherwise
  // (a group's 4 bytes of params go with 8 to 16 of codes)
  g.chunk = g.paged ? kPage : kCodeBytes / g.rb;
  g.slots = kCodeBytes / g.fb;
  // no more warps than there can be runs, and as many blocks as an SM has room for
  const int64_t packed = share ? 1 : ((int64_t)(d.cap < s.cap ? d.cap : s.cap) + g.chunk - 1) / g.chunk;
  const int64_t each = packed + (d.Nr + g.slots - 1) / g.slots + (d.Ns + g.slots - 1) / g.slots;
  const int64_t runs = d.B * (1 + 2 * (int64_t)d.Hkv * each);
  const int64_t blocks = (runs + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = kBlocks * (int64_t)device_sm_count();
  return launch_overlapped(reorder_kernel, dim3((unsigned)(blocks < most ? blocks : most)), kThreads, 0, st, g);
}

}  // namespace kvq
