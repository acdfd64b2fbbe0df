// kvq_chunk_attn.cuh -- attention of runs of several tokens over the low-bit cache on
// the fifth-generation tensor cores.
//
// The mathematics.  The query rows of one (sequence, KV head) are its run's tokens times
// the gq heads that share the KV head, row = token * gq + head: one pass over K and V
// serves them all.  For a tile of tokens S = Q K^T, P = exp2(S c - m c) with the row's
// reference maximum m, O += P V, l += sum P; c = log2(e) / sqrt(d).  m follows the
// running maximum lazily: it moves (and O, l are rescaled) only when the maximum has
// passed it by 2^8, so weights stay below 256 and the sums lose nothing in fp32.
// Roundings: the dequantized keys and values min + code * scale are rounded to fp16 once
// (operands of the MMA), the weights P to fp16 once; scores, m, l and O are fp32.  P and l
// carry a factor 2^7, which O / l and every join of parts cancel: P reaches 2^15, near
// the top of fp16's range, so that weights keep 11 bits down to 2^-21 of the reference
// and lose at most 2^-32 of it below (a long tail under one dominant token).
//
// A block (one per SM, persistent) has 24 warps:
//   0-15   softmax: S from TMEM, P back to TMEM (it takes S's place and is the A operand
//          of the second MMA), the epilogue.  Four groups of four warps: two for each of
//          the block's two accumulators (lanes 0 and 1), each with half of the tile's
//          tokens and half of O's columns, a thread per query row.
//   16-19  dequantize: raw rows in a ring become fp16 in registers and go to shared memory
//          in the MMA's 128-byte swizzle, K as the K-major and V as the MN-major B operand.
//          Up to head_dim 64 each thread also copies its rows (cp.async, no barrier).
//   20     issues the MMAs; 21 works out the segments; 22 copies the raw rows from head_dim
//          128 on (bulk copies: the dequantizing warps spent a quarter of their time on the
//          addresses, 2048 x 32768 tokens of INT2 1039 -> 1002 us, 1024 x 16384 of INT4
//          593 -> 557 us without).
// The MMA warp's lanes all go the same way and one is elected for each batch, so that the
// descriptors are in uniform registers: a lone thread moved each of them there per MMA and
// was the bound (1002 -> 819 us and 557 -> 457 us).  Eight dequantizing warps, keys and
// values apart, made runs of few rows 3-6 % faster and the long ones 6-7 % slower (72
// registers a thread at launch in place of 80).
//
// What bounds it now: the chain S -> softmax -> P -> PV -> next S of each accumulator, with
// the other's MMAs under it, and shared memory: for a shared tile (128 tokens, 256 rows,
// head_dim 128) the MMAs read 192 KB and the dequantizing warps write 64 KB, by count
// about the 2048 cycles that the MMAs themselves take.  2048 x 32768 tokens of INT2 (32
// heads on 8, head_dim 128) take 805 to 855 us by the box, 65 to 69 % of the bf16 rate
// that a library product reaches.  Calls of few rows are bound by the warps that
// dequantize, and the smallest by the way to the first tile (7 us) and the join (5 us).
//
// A unit of work is (sequence, block of query rows, KV head).  With more than 128 rows in
// the block the two lanes are its two halves and share each tile; with fewer they take
// alternate tiles of the same rows and are joined at the end, so that the softmax of one
// tile runs under the MMAs of the next either way.  head_dim 256 has room for one lane.
//
// Balance.  All units' tiles lie in one line, and each of the G blocks takes an equal
// piece of it (the line is cut by cost, so a unit may be cut, into two pieces or, with
// few units, into many).  Pieces of a unit write (O, m, l), with alternating lanes each
// lane its own, and a second kernel joins them in a fixed order: results do not depend
// on timing.
//
// Storage order.  Codes come out of a word in pairs (k, k + 4) (INT4, INT3) or (k, k + 8)
// (INT2).  Instead of sorting them, Q's and the fp16 tokens' elements are put in the same
// order along d, and the output's are put back at the very end.
#pragma once

#include <math.h>

#include <atomic>

#include "kvq_ptx.cuh"
#include "kvq_runs.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

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
  const __half* q;  // [total][Hq][d]
  void* out;        // [total][Hq][d]
  const int32_t* cu;
  int4* heads;        // [G][4]: the Seg of the unit that block g begins and does not end (b < 0: none)
  float2* ml_part;    // [2 G][QB] {m, l}
  float4* o_part;     // [2 G][QB][d / 4]
  int B, Hkv, Hq, gq, cap, Nr, Ns, total, max_len, causal, out_f32;
  uint32_t gq_mul, gq_shift;  // row / gq = row * gq_mul >> gq_shift for rows below 2^31
  uint32_t wait_limit_us;
  int fault;  // testing hook: 1 makes the scores' barriers wait for an arrival that never comes
  float scale_log2;
};

cudaError_t launch_chunk_attn_d32(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d64(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d128(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d256(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);

// Query rows of a block (all its lanes).
__host__ __device__ constexpr int chunk_rows(int d) { return d == 256 ? 128 : 256; }

namespace chunk {

constexpr int kThreads = 768;
constexpr float kWeightBits = 7.0f;  // log2 of the weights' factor
constexpr int kDeqThreads = 128;
// What the line of tiles is cut by, in half microseconds (head_dim 128): a tile of 128
// tokens that the lanes share, one lane's own, a unit's begin and end.  Fitted to blocks'
// times a shared tile takes 2.0 us, an own one 1.1 to 1.4, a unit 3 with few rows and 9
// with many.  The unit's 5 us is between the two: dearer units (20, with 8 for a tile of
// fp16 tokens) made the 40-head case 6 % faster and a batch of drafts 9 % slower.  A cost
// for each kind of unit, and fits at other head_dims (where these serve too), are untried.
constexpr int kCostShared = 4, kCostOwn = 3, kCostUnit = 10;

template <int D, int BITS>
struct Cfg {
  static constexpr int LANES = D == 256 ? 1 : 2;    // accumulators
  static constexpr int QB = chunk_rows(D);
  static constexpr int TN = D == 256 ? 64 : 128;    // tokens of a tile
  static constexpr int G = D / 32;                  // groups of a row
  static constexpr int PW = D < 64 ? D : 64;        // elements of a panel's row
  static constexpr int RB = PW * 2;                 // bytes of it
  static constexpr int SWZ = RB == 128 ? 2 : 4;
  static constexpr int QP = 128 * RB;               // bytes of a panel of Q
  static constexpr int KP = TN * RB;                // of a panel of K or V
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int KBYTES = TN * D * 2;
  static constexpr int ST = D <= 64 ? 4 : 2;        // K and V stages
  static constexpr int HC = TN / 2;                 // a softmax group's columns of S
  static constexpr int HD = D / 2;                  // ... and of O
  static constexpr int TPR = TN == 64 ? 2 : 1;      // dequantizing threads of a row
  static constexpr int GPT = G / TPR;               // groups of each
  static constexpr int CB = 4 * BITS;               // code bytes of a group
  static constexpr int TB = GPT * CB;               // code bytes of a thread, contiguous
  static constexpr int UN = (TB + 15) / 16;         // 16-byte units of them in the ring
  static constexpr int PB = GPT * 4;                // param bytes of a thread
  static constexpr int RAWB = kDeqThreads * (UN * 16 + PB);
  // rows that bulk copies can move (multiples of 16 bytes wherever they start)
  static constexpr bool BULK = D >= 128;
  static constexpr int RAWN = D == 256 ? 2 : D == 128 ? 3 : 6;  // half tiles of the ring
  static constexpr int SMW = 8 * LANES;             // softmax warps
  // TMEM columns
  static constexpr int S0 = 0;
  static constexpr int O0 = 256;
  static constexpr int OSTEP = D;
  // shared memory
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + LANES * QBYTES;
  static constexpr int OFF_V = OFF_K + ST * KBYTES;
  static constexpr int OFF_RAW = OFF_V + ST * KBYTES;
  // where lane 1's accumulator passes to lane 0: 16 columns of 128 rows of each half.  Lane
  // 1's Q (but for its first KiB) is free then, and large enough from head_dim 128 on
  static constexpr int STAGE = 2 * 16 * 128 * 4;
  static constexpr int OFF_STAGE = D >= 128 ? OFF_Q + (LANES - 1) * QBYTES + 1024 : OFF_RAW + RAWN * RAWB;
  static constexpr int OFF_POISON = OFF_RAW + RAWN * RAWB + (D >= 128 ? 0 : STAGE);  // int [3][D]
  static constexpr int OFF_MAX = OFF_POISON + 3 * D * 4;        // float [LANES][2][128]
  static constexpr int OFF_BAR = OFF_MAX + LANES * 1024;
  static constexpr int OFF_SEG = OFF_BAR + 512;                 // Seg [kSegs]
  static constexpr int SMEM = OFF_SEG + 512;
};

// A segment: the block's tiles [lo, hi) of the unit (sequence b, KV head h, query block
// qb).  One warp works the segments out, the others read them from a ring.
constexpr int kSegs = 8;
struct alignas(16) Seg {
  int b, h, qb, lo;
  int hi, npt, nt, alt;     // packed tiles and all tiles of the unit; alt: the lanes take alternate tiles
  int c0, n, ns, npk;       // the run, and the sequence's lengths
  int nres, head, last_b, pad;  // last_b: of a unit that the block begins, the block that ends it; b < 0: the end
};

// Barriers (8 bytes each from OFF_BAR) and words behind them.
enum { B_QFULL = 0, B_SFULL = 2, B_PREADY = 4, B_ODONE = 6, B_PAIR = 8, B_DRAIN = 9, B_KFULL = 10,
       B_KEMPTY = 14, B_VFULL = 18, B_VEMPTY = 22, B_SEGFULL = 26, B_SEGEMPTY = 34, B_MAX = 42, B_RAWFULL = 50,
       B_RAWEMPTY = 53, B_COUNT = 56 };
enum { W_TMEM = 112, W_ABORT = 113, W_PFLAG = 114, W_EPI = 115, W_STARTB = 116, W_STARTQ = 117,
       W_BASE = 118 /* int64 */, W_PAGES = 120 /* a ring slot's pages that are there */ };

__device__ __forceinline__ uint32_t lds(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int4 lds_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ldsf(uint32_t addr) { return __uint_as_float(lds(addr)); }
__device__ __forceinline__ void stsf(uint32_t addr, float v) { sts(addr, __float_as_uint(v)); }
__device__ __forceinline__ uint32_t timer_lo() {  // nanoseconds, modulo 2^32
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}

// Bounded waits (at most a second: the timer's 32 bits do): all give up when one has.
// Few registers: most waits stand between registers full of scores.
struct Waits {
  const ChunkAttnArgs& a;
  uint32_t bars;  // shared address of the barriers and words

  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // (volatile in PTX too: a plain load may be taken out of a loop that polls)
  __device__ __forceinline__ uint32_t word(int i) const {
    uint32_t v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(bars + 4 * i) : "memory");
    return v;
  }
  __device__ __forceinline__ void set_word(int i, uint32_t v) const {
    asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(bars + 4 * i), "r"(v) : "memory");
  }
  __device__ __forceinline__ bool late(uint32_t t0) const {
    if (word(W_ABORT)) return true;
    if (timer_lo() - t0 <= a.wait_limit_us * 1000u) return false;
    set_word(W_ABORT, 1);
    return true;
  }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    const uint32_t b = bar(i);
    if (ptx::mbar_try_wait(b, parity)) return true;
    const uint32_t t0 = timer_lo();
#pragma unroll 1
    for (uint32_t k = 1; !ptx::mbar_try_wait(b, parity); ++k)
      if ((k & 63u) == 0 && late(t0)) return false;
    return true;
  }
  // a whole warp waits; the same answer for all its lanes
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(i, parity));
  }
  __device__ __forceinline__ void arrive_warp(int i) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar(i));
  }
};

__device__ __forceinline__ int token_of(const ChunkAttnArgs& a, int row) {
  return (int)(((uint64_t)(uint32_t)row * a.gq_mul) >> a.gq_shift);
}

// Tokens that token `tok` of a run of n sees, of the packed ones and of the fp16 ones
// (sink, then window): prefixes of both.
__device__ __forceinline__ int seen_of(const ChunkAttnArgs& a, int n, int held, int tok) {
  return a.causal ? max(0, held - n + tok + 1) : held;
}
__device__ __forceinline__ int seen_packed(int ns, int npk, int lim) { return min(max(lim - ns, 0), npk); }
__device__ __forceinline__ int seen_f16(int ns, int npk, int lim) {
  return min(lim, ns) + max(lim - ns - npk, 0);
}

// Where a block is in the line of tiles: the unit (b, qb, h), whose first tile starts
// at `base`, and the block's tiles [lo, hi) of it.
template <int D, int BITS>
struct Walk {
  using C = Cfg<D, BITS>;
  int b, qb, h;
  int64_t base, x0, x1;
  Run run;
  SeqLens s;
  int npt, nt, w;  // packed tiles, all tiles, cost of a tile
  int lo, hi;

  static __device__ __forceinline__ int blocks(const ChunkAttnArgs& a, const Run& run) {
    return run.n > 0 ? (run.n * a.gq + C::QB - 1) / C::QB : 0;
  }
  // Tiles of query block qb (at least one: an empty one writes the zeros of rows that
  // see nothing) and the cost of each.
  static __device__ __forceinline__ void tiles(const ChunkAttnArgs& a, const Run& run, const SeqLens& s,
                                               int qb, int& npt, int& nt, int& w) {
    const int rows = run.n * a.gq;
    const int last = min(rows, (qb + 1) * C::QB) - 1;
    const int lim = seen_of(a, run.n, s.ns + s.npk + s.nres, token_of(a, last));
    npt = (seen_packed(s.ns, s.npk, lim) + C::TN - 1) / C::TN;
    nt = max(1, npt + (seen_f16(s.ns, s.npk, lim) + C::TN - 1) / C::TN);
    w = C::LANES == 2 && last - qb * C::QB >= 128 ? kCostShared : kCostOwn;
  }
  static __device__ __forceinline__ int64_t unit_cost(int nt, int w) { return (int64_t)nt * w + kCostUnit; }
  static __device__ __forceinline__ int64_t seq_cost(const ChunkAttnArgs& a, int b) {
    const Run run = run_of(a.cu, b, a.total, a.max_len);
    const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
    const int nq = blocks(a, run);
    int64_t c = 0;
    for (int qb = 0; qb < nq; ++qb) {
      int npt, nt, w;
      tiles(a, run, s, qb, npt, nt, w);
      c += unit_cost(nt, w);
    }
    return c * a.Hkv;
  }

  __device__ __forceinline__ void load_seq(const ChunkAttnArgs& a) {
    run = run_of(a.cu, b, a.total, a.max_len);
    s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
  }
  __device__ __forceinline__ void range() {
    // tile k starts at base + kCostUnit + k w and is the block's if that is in [x0, x1)
    lo = count_below(x0 - base - kCostUnit);
    hi = count_below(x1 - base - kCostUnit);
  }
  // tiles of the unit that start before e
  __device__ __forceinline__ int count_below(int64_t e) const {
    if (e <= 0) return 0;
    if (e >= (int64_t)nt * w) return nt;
    return (int)(((uint32_t)e + w - 1) / (uint32_t)w);  // (a unit's cost is below 2^31)
  }
  __device__ __forceinline__ void start(const ChunkAttnArgs& a, int b_, int qb_, int64_t base_, int64_t x0_,
                                        int64_t x1_) {
    b = b_;
    qb = qb_;
    x0 = x0_;
    x1 = x1_;
    load_seq(a);
    tiles(a, run, s, qb, npt, nt, w);
    const int64_t unit = unit_cost(nt, w);
    h = (int)((x0 - base_) / unit);
    base = base_ + h * unit;
    range();
  }
  __device__ __forceinline__ bool more(const ChunkAttnArgs& a) const { return b < a.B && base < x1; }
  __device__ __forceinline__ void next(const ChunkAttnArgs& a) {
    base += unit_cost(nt, w);
    if (++h == a.Hkv) {
      h = 0;
      if (++qb >= blocks(a, run)) {
        qb = 0;
        if (base >= x1) {  // nothing of the block's is left
          b = a.B;
          return;
        }
        do {
          if (++b >= a.B) return;
          load_seq(a);
        } while (run.n <= 0);
      }
      tiles(a, run, s, qb, npt, nt, w);
    }
    range();
  }
};

// The warp that works out the segments.
template <int D, int BITS>
__device__ __forceinline__ void walk_role(const ChunkAttnArgs& a, const Waits& wt, Seg* ring, int b, int qb,
                                          int64_t base, int64_t x0, int64_t x1, int64_t W, int64_t G) {
  Walk<D, BITS> k;
  k.start(a, b, qb, base, x0, x1);
  for (uint32_t i = 0;; k.next(a)) {
    const bool more = k.more(a);
    if (more && k.lo >= k.hi) continue;  // the unit's begin is the block's, no tile of it
    const int at = i % kSegs;
    if (!wt.wait(B_SEGEMPTY + at, ((i / kSegs) & 1) ^ 1)) return;
    Seg s;
    s.b = -1;
    if (more) {
      s.b = k.b, s.h = k.h, s.qb = k.qb, s.lo = k.lo, s.hi = k.hi, s.npt = k.npt, s.nt = k.nt;
      s.alt = Cfg<D, BITS>::LANES == 2 && k.w == kCostOwn;
      s.c0 = k.run.c0, s.n = k.run.n, s.ns = k.s.ns, s.npk = k.s.npk, s.nres = k.s.nres, s.head = k.s.head;
      s.last_b = 0;
      if (k.lo == 0 && k.hi < k.nt)  // block c has the starts from floor(c W / G) on
        s.last_b = (int)(((k.base + kCostUnit + (int64_t)(k.nt - 1) * k.w + 1) * G - 1) / W);
    }
    ring[at] = s;
    ptx::mbar_arrive(wt.bar(B_SEGFULL + at));
    if (!more) return;
    ++i;
  }
}

// A reader's place in the ring.
struct SegReader {
  uint32_t i = 0;
  __device__ __forceinline__ bool wait(const Waits& wt) const {
    return wt.wait(B_SEGFULL + i % kSegs, (i / kSegs) & 1);
  }
  __device__ __forceinline__ const Seg& get(const Seg* ring) const { return ring[i % kSegs]; }
};

// ------------------------------------------------------------- storage order ---

// Two neighbouring 16-byte pieces (16 elements) put in storage order.
template <int BITS>
__device__ __forceinline__ void to_storage(uint4& a, uint4& b) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (BITS == 2) {
    a = make_uint4(ptx::prmt(x[0], x[4], 0x5410), ptx::prmt(x[0], x[4], 0x7632),
                   ptx::prmt(x[1], x[5], 0x5410), ptx::prmt(x[1], x[5], 0x7632));
    b = make_uint4(ptx::prmt(x[2], x[6], 0x5410), ptx::prmt(x[2], x[6], 0x7632),
                   ptx::prmt(x[3], x[7], 0x5410), ptx::prmt(x[3], x[7], 0x7632));
  } else {
    a = make_uint4(ptx::prmt(x[0], x[2], 0x5410), ptx::prmt(x[0], x[2], 0x7632),
                   ptx::prmt(x[1], x[3], 0x5410), ptx::prmt(x[1], x[3], 0x7632));
    b = make_uint4(ptx::prmt(x[4], x[6], 0x5410), ptx::prmt(x[4], x[6], 0x7632),
                   ptx::prmt(x[5], x[7], 0x5410), ptx::prmt(x[5], x[7], 0x7632));
  }
}
// The storage place of element e of 16.
template <int BITS>
__host__ __device__ constexpr int place(int e) {
  return BITS == 2 ? ((e & 7) >> 2) * 8 + 2 * (e & 3) + (e >> 3) : (e & 8) + 2 * (e & 3) + ((e >> 2) & 1);
}

// Byte offset of 16-byte piece `c` (of a panel's row) of row r in a swizzled tile.
template <int RB>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return RB == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4))
                   : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ bool f16_nonfinite(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

// --------------------------------------------------------------- dequantize ---

// Eight codes, four pairs at fixed bit places of x, as four exact fp16 pairs: the
// bits are put in the mantissa of 1024 (as 2^s code) and 1024 is taken off again.
template <int BITS>
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&f)[4]) {
  constexpr uint32_t M = 0x64006400u;
  constexpr uint32_t m0 = BITS == 4 ? 0x000f000fu : BITS == 3 ? 0x00070007u : 0x00030003u;
  constexpr uint32_t m1 = m0 << BITS;
  const uint32_t y = BITS == 2 ? x : x >> (2 * BITS);
  // 1 / 2^BITS and -1024 / 2^BITS as fp16 pairs
  constexpr uint32_t i1 = BITS == 4 ? 0x2c002c00u : BITS == 3 ? 0x30003000u : 0x34003400u;
  constexpr uint32_t o1 = BITS == 4 ? 0xd400d400u : BITS == 3 ? 0xd800d800u : 0xdc00dc00u;
  f[0] = ptx::hadd2_u32(ptx::and_or(x, m0, M), 0xe400e400u);
  f[1] = ptx::hfma2_u32(ptx::and_or(x, m1, M), i1, o1);
  if (BITS == 2) {
    f[2] = ptx::hfma2_u32(ptx::and_or(x, 0x00300030u, M), 0x2c002c00u, 0xd400d400u);  // / 16
    f[3] = ptx::hfma2_u32(ptx::and_or(x, 0x00c000c0u, M), 0x24002400u, 0xcc00cc00u);  // / 64
  } else {
    f[2] = ptx::hadd2_u32(ptx::and_or(y, m0, M), 0xe400e400u);
    f[3] = ptx::hfma2_u32(ptx::and_or(y, m1, M), i1, o1);
  }
}

// The four 8-code words of group g, from a thread's raw words.
template <int BITS>
__device__ __forceinline__ void code_words(const uint32_t* raw, int g, uint32_t (&x)[4]) {
  if (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = raw[4 * g + i];
  } else if (BITS == 2) {
    x[0] = raw[2 * g], x[1] = raw[2 * g] >> 8, x[2] = raw[2 * g + 1], x[3] = raw[2 * g + 1] >> 8;
  } else {
    const uint32_t* w = raw + 3 * g;
    const uint32_t v[4] = {w[0], __funnelshift_r(w[0], w[1], 24), __funnelshift_r(w[1], w[2], 16), w[2] >> 8};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (v[i] & 0xfffu) | ((v[i] & 0xfff000u) << 4);
  }
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// What the dequantizing warps share.  Thread dt has row dt of a tile (head_dim 256: half
// of row dt / 2): its codes are contiguous, and 8 neighbouring lanes store the same piece
// of 8 rows, which the swizzle puts into 8 different banks' groups.
template <int D, int BITS>
struct Deq {
  using C = Cfg<D, BITS>;
  const ChunkAttnArgs& a;
  const Waits& wt;
  uint32_t smem;  // base of the block's shared memory
  int* poison;
  const Seg* ring;
  int dt;         // thread of the warps that dequantize
  uint32_t seg;   // segments of the block so far

  // Values that fp16 does not hold as finite ones take no part in the MMA: a weight of
  // zero would make them NaN in rows that do not see the token.  The first token of the
  // segment with +inf, -inf or NaN in a column is noted, and the epilogue gives the rows
  // that see it what the sum would be.  (Rare: one thread per element.)
  __device__ __forceinline__ bool note(int col, int token, uint32_t h) {
    // the notes of earlier segments have been read before this one's are made
    const uint32_t t0 = timer_lo();
    while (wt.word(W_EPI) < seg * C::SMW)
      if (wt.late(t0)) return false;
    const int kind = (h & 0x3ffu) ? 2 : (h & 0x8000u) ? 1 : 0;
    atomicMin(poison + kind * D + col, token);
    wt.set_word(W_PFLAG, 1);
    return true;
  }

  // The cursor of the copies: a half tile of a segment.
  struct Cursor {
    SegReader at;
    int tile = -1, w = 0, hi = 0, npt = 0, npk = 0, b = 0;
    int64_t row0 = 0;  // contiguous: row of the head's token 0; paged: h * 32
  };

  // The thread's raw row of a half tile (keys, then values) into ring slot `slot`; a row
  // that is not there becomes zero codes with zero params, which stand for zeros.
  __device__ __forceinline__ void fetch(const Cursor& c, int slot) {
    const uint32_t dc = smem + C::OFF_RAW + slot * C::RAWB + dt * 16;
    const uint32_t dp = smem + C::OFF_RAW + slot * C::RAWB + kDeqThreads * C::UN * 16 + dt * C::PB;
    const int p = c.tile * C::TN + dt / C::TPR;
    bool there = p < c.npk;
    int64_t row = c.row0 + p;
    if (a.rm.paged && there) {
      const int pg = a.rm.page_of(c.b, p / kPage);
      there = pg >= 0 && pg < a.rm.npages;
      if (!there) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
      row = (int64_t)pg * a.Hkv * kPage + c.row0 + p % kPage;
    }
    if (there) {
      const uint8_t* src = a.codes[c.w] + row * (C::G * C::CB) + (dt % C::TPR) * C::TB;
      constexpr int N = C::TB % 16 == 0 ? 16 : C::TB % 8 == 0 ? 8 : 4;
#pragma unroll
      for (int i = 0; i < C::TB / N; ++i)
        cp_async<N>(dc + (i * N / 16) * (kDeqThreads * 16) + i * N % 16, src + i * N);
      cp_async<C::PB>(dp, a.params[c.w] + row * C::G + (dt % C::TPR) * C::GPT);
    } else {
#pragma unroll
      for (int i = 0; i < C::UN; ++i) st_shared_v4(dc + i * (kDeqThreads * 16), make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int i = 0; i < C::GPT; ++i) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dp + 4 * i), "r"(0) : "memory");
    }
  }

  // Shared address of the thread's row in a tile at dst, with the row's swizzle in its
  // low bits: piece c of panel p is at (this ^ (c << 4)) + p * KP.
  __device__ __forceinline__ uint32_t row_addr(uint32_t dst) const {
    const int r = dt / C::TPR;
    return dst + (dt % C::TPR) * (C::GPT / 2) * C::KP + r * C::RB + ((C::RB == 128 ? r & 7 : (r >> 1) & 3) << 4);
  }
  __device__ __forceinline__ int column(int g, int c) const { return ((dt % C::TPR) * C::GPT + g) * 32 + c * 8; }

  // A fetched half tile as fp16 at `dst`.  first: logical place of the tile's first token;
  // there: the thread's row is one (BULK: others hold what the ring held).
  __device__ __forceinline__ bool packed_tile(int first, int w, int slot, uint32_t dst, bool there) {
    constexpr uint32_t kQmax2 = BITS == 4 ? 0x4b804b80u : BITS == 3 ? 0x47004700u : 0x42004200u;  // 15, 7, 3
    // With rows of codes as they are in memory, lanes take their groups in different
    // orders (by pieces of 16 bytes), so that the banks are all in use.
    const int rot = !C::BULK || BITS == 3 ? 0 : BITS == 4 ? (dt >> 1) & 3 : (dt >> 2) & 1;
    auto group = [&](int g) {
      return BITS == 4 ? (g + rot) & (C::GPT - 1) : BITS == 2 ? g ^ (rot << 1) : g;
    };
    const uint32_t dc = smem + C::OFF_RAW + slot * C::RAWB + dt * (C::BULK ? C::TB : 16);
    const uint32_t dp = smem + C::OFF_RAW + slot * C::RAWB + kDeqThreads * C::UN * 16 + dt * C::PB;
    uint32_t raw[C::UN * 4], prm[C::GPT];
#pragma unroll
    for (int i = 0; i < C::UN; ++i) {
      const uint4 v = ld_shared_v4(dc + (!C::BULK    ? i * (kDeqThreads * 16)
                                         : BITS == 4 ? group(i) * 16
                                         : BITS == 2 ? (i ^ rot) * 16
                                                     : i * 16));
      raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < C::GPT; ++i) {
      const uint32_t x = lds(dp + 4 * group(i));
      prm[i] = there ? x : 0;  // whatever the codes, zeros
    }
    if (C::BULK) wt.arrive_warp(B_RAWEMPTY + slot);
    const uint32_t at = row_addr(dst);
    auto piece = [&](int g, int c) { return (at ^ (((g & 1) * 4 + c) << 4)) + (g / 2) * C::KP; };
    uint32_t rare = 0;
#pragma unroll
    for (int i = 0; i < C::GPT; ++i) {
      const int g = group(i);
      const uint32_t s2 = ptx::prmt(prm[i], prm[i], 0x1010), m2 = ptx::prmt(prm[i], prm[i], 0x3232);
      // the group's largest value; only where it is not finite can any value be so
      if (f16_nonfinite(ptx::hfma2_u32(kQmax2, s2, m2))) rare |= 1u << i;
      uint32_t x[4];
      code_words<BITS>(raw, i, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[4];
        codes_f16<BITS>(x[c], y);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = ptx::hfma2_u32(y[j], s2, m2);
        st_shared_v4(piece(g, c), make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
    if (rare == 0) return true;
    // what is not finite among the stored values: past fp16's largest value by the
    // scale's rounding, or meant (params that are not finite)
#pragma unroll 1
    for (int e = 0; e < 32 * C::GPT; ++e) {
      if (!((rare >> (e >> 5)) & 1u)) continue;
      const int g = group(e >> 5);
      uint32_t pg = prm[0];
#pragma unroll
      for (int i = 1; i < C::GPT; ++i)
        if ((e >> 5) == i) pg = prm[i];
      const uint32_t ea = piece(g, (e >> 3) & 3) + 2 * (e & 7);
      unsigned short hv;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hv) : "r"(ea) : "memory");
      if (!f16_nonfinite(hv)) continue;
      if (!f16_nonfinite(pg) && !f16_nonfinite(pg >> 16))
        hv = (hv & 0x8000u) | 0x7bffu;
      else if (w == 0)
        continue;
      else if (note(column(g, 0) + (e & 31), first + dt / C::TPR, hv))
        hv = 0;
      else
        return false;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(ea), "h"(hv) : "memory");
    }
    return true;
  }

  __device__ __forceinline__ int ring_slot(int j) const { return j < a.Nr ? j : j - a.Nr; }  // j < 2 Nr

  // A half tile of fp16 tokens (sink, then window): rows f0 .. of their line.
  __device__ __forceinline__ bool f16_tile(const Seg& k, int f0, int w, uint32_t dst) {
    const int64_t bh = (int64_t)k.b * a.Hkv + k.h;
    const int f = f0 + dt / C::TPR, n = k.ns + k.nres;
    const __half* src = a.q;  // (not read)
    if (f < k.ns)
      src = a.sink[w] + (bh * a.Ns + f) * D;
    else if (f < n)
      src = a.res[w] + (bh * a.Nr + ring_slot(k.head + f - k.ns)) * D;
    if (f < n) src += column(0, 0);
    const uint32_t at = row_addr(dst);
#pragma unroll
    for (int i = 0; i < 4 * C::GPT; ++i)
      ptx::cp_async_16((at ^ ((i & 7) << 4)) + (i / 8) * C::KP, src + (f < n ? i * 8 : 0), f < n ? 16 : 0);
    ptx::cp_async_wait_all();
    const int token = f < k.ns ? f : f + k.npk;
#pragma unroll 2
    for (int i = 0; i < 4 * C::GPT; i += 2) {  // 16 elements
      const uint32_t p0 = (at ^ ((i & 7) << 4)) + (i / 8) * C::KP, p1 = (at ^ (((i & 7) + 1) << 4)) + (i / 8) * C::KP;
      uint4 u[2] = {ld_shared_v4(p0), ld_shared_v4(p1)};
      to_storage<BITS>(u[0], u[1]);
      st_shared_v4(p0, u[0]);
      st_shared_v4(p1, u[1]);
      if (w == 0) continue;
      const uint32_t* y = reinterpret_cast<const uint32_t*>(u);
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) bad |= f16_nonfinite(y[j]) || f16_nonfinite(y[j] >> 16);
      if (!bad) continue;
#pragma unroll 1
      for (int j = 0; j < 16; ++j) {
        const uint32_t ea = (j < 8 ? p0 : p1) + 2 * (j & 7);
        unsigned short hv;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hv) : "r"(ea) : "memory");
        if (!f16_nonfinite(hv)) continue;
        if (!note(column(0, i) + j, token, hv)) return false;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(ea), "h"((unsigned short)0) : "memory");
      }
    }
    return true;
  }

  __device__ __forceinline__ void run() {
    SegReader k;
    Cursor c;
    bool ok = true, more = true;
    // the next half tile of the line into its ring slot
    auto fetch_next = [&](int slot) {
      if (more && c.tile < 0) {
        ok = ok && __all_sync(0xffffffffu, c.at.wait(wt));
        const Seg& s = c.at.get(ring);
        more = ok && s.b >= 0;
        if (more) {
          c.tile = s.lo, c.hi = s.hi, c.npt = s.npt, c.npk = s.npk, c.b = s.b;
          c.row0 = a.rm.paged ? (int64_t)s.h * kPage : ((int64_t)s.b * a.Hkv + s.h) * a.cap;
        }
      }
      if (more) {
        if (c.tile < c.npt) fetch(c, slot);
        c.w ^= 1;
        if (c.w == 0 && ++c.tile == c.hi) {
          ++c.at.i;
          c.tile = -1;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t kv = 0;     // tiles so far
    int slot = 0;
    uint32_t phase = 0;  // of the slot (BULK)
    // RAWN - 1 half tiles ahead: a free slot is filled before the oldest is taken
    if constexpr (!C::BULK) {
#pragma unroll 1
      for (int i = 0; i < C::RAWN - 1; ++i) fetch_next(i);
    }
    for (; ok; ++k.i, ++seg) {
      ok = ok && __all_sync(0xffffffffu, k.wait(wt));
      if (!ok) break;
      const Seg& s = k.get(ring);
      if (s.b < 0) break;
      const int lo = s.lo, hi = s.hi, npt = s.npt, ns = s.ns, npk = s.npk;
      for (int h = 2 * lo; h < 2 * hi; ++h) {
        if constexpr (!C::BULK) fetch_next(slot == 0 ? C::RAWN - 1 : slot - 1);
        const int t = h >> 1, w = h & 1;
        const int stage = kv % C::ST;
        const uint32_t dst = smem + (w ? C::OFF_V : C::OFF_K) + stage * C::KBYTES;
        ok = ok && wt.wait_warp((w ? B_VEMPTY : B_KEMPTY) + stage, ((kv / C::ST) & 1) ^ 1);
        if (!ok) break;
        if (t < npt) {
          bool there = true;
          if constexpr (C::BULK) {
            ok = wt.wait_warp(B_RAWFULL + slot, phase);
            if (!ok) break;
            const int row = dt / C::TPR;
            there = t * C::TN + row < npk && ((wt.word(W_PAGES + slot) >> (row / kPage)) & 1u);
          } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::RAWN - 1) : "memory");
          }
          ok = packed_tile(ns + t * C::TN, w, slot, dst, there);
        } else {
          ok = f16_tile(s, (t - npt) * C::TN, w, dst);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::fence_proxy_async_shared();
        wt.arrive_warp((w ? B_VFULL : B_KFULL) + stage);
        if (!C::BULK || t < npt) {  // (BULK: slots are of packed half tiles alone)
          if (++slot == C::RAWN) slot = 0, phase ^= 1;
        }
        kv += w;
      }
      wt.arrive_warp(B_SEGEMPTY + k.i % kSegs);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// The warp that copies packed rows into the ring (BULK): of each 32 rows of a half tile
// (a page, where there are pages) one lane copies the codes and another the params.
template <int D, int BITS>
__device__ __forceinline__ void fetch_role(const ChunkAttnArgs& a, const Waits& wt, uint32_t smem, const Seg* ring) {
  using C = Cfg<D, BITS>;
  constexpr int NP = C::TN / kPage;
  const int lane = threadIdx.x & 31, j = lane % NP;
  const bool codes = lane < NP;
  const uint32_t row_bytes = codes ? C::G * C::CB : C::G * 4;
  const uint32_t to = smem + C::OFF_RAW + (codes ? 0 : kDeqThreads * C::UN * 16) + j * kPage * row_bytes;
  SegReader k;
  int slot = 0;
  uint32_t n = 0;  // half tiles copied
  bool ok = true;
  for (; ok && (ok = __all_sync(0xffffffffu, k.wait(wt))); ++k.i) {
    const Seg& s = k.get(ring);
    if (s.b < 0) break;
    const int hi = min(s.hi, s.npt), rows = s.npk - j * kPage;  // (of the sequence, from the lane's on)
    const int64_t row0 = a.rm.paged ? (int64_t)s.h * kPage : ((int64_t)s.b * a.Hkv + s.h) * a.cap + j * kPage;
    const int* table = a.rm.block_table + (int64_t)s.b * (a.cap / kPage) + j;
    auto page_of = [&](int t) { return a.rm.paged && t < hi && t * C::TN < rows ? table[t * NP] : 0; };
    int next = page_of(s.lo);
    for (int t = s.lo; ok && t < hi; ++t) {
      const int page = next;
      next = page_of(t + 1);
      bool there = t * C::TN < rows;
      if (there && (page < 0 || page >= a.rm.npages) && a.rm.paged) {
        there = false;
        set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
      }
      const uint32_t pages = __ballot_sync(0xffffffffu, there);  // (lanes from NP on say the same again)
      const uint32_t bytes = there && lane < 2 * NP ? min(kPage, rows - t * C::TN) * row_bytes : 0;
      const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
      const int64_t row = row0 + (a.rm.paged ? (int64_t)page * a.Hkv * kPage : (int64_t)t * C::TN);
#pragma unroll 1
      for (int w = 0; w < 2; ++w, ++n) {
        ok = wt.wait_warp(B_RAWEMPTY + slot, ((n / C::RAWN) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          wt.set_word(W_PAGES + slot, pages);
          ptx::mbar_arrive_expect_tx(wt.bar(B_RAWFULL + slot), all);
        }
        __syncwarp();
        const void* of = codes ? static_cast<const void*>(a.codes[w]) : a.params[w];
        if (bytes)
          ptx::bulk_load(to + slot * C::RAWB, static_cast<const char*>(of) + row * row_bytes, bytes,
                         wt.bar(B_RAWFULL + slot));
        if (++slot == C::RAWN) slot = 0;
      }
    }
    wt.arrive_warp(B_SEGEMPTY + k.i % kSegs);
  }
  // copies still in flight when the block gives up land before its shared memory goes
  const uint32_t t0 = timer_lo();
  for (uint32_t i = n > C::RAWN ? n - C::RAWN : 0; i < n; ++i)
    while (!ptx::mbar_try_wait(wt.bar(B_RAWFULL + i % C::RAWN), (i / C::RAWN) & 1))
      if (timer_lo() - t0 > 1000000000u) return;
}

// ---------------------------------------------------------------------- MMA ---

// The warp that issues the MMAs: all its lanes go the same way, so that descriptors and
// addresses stay in the warp's uniform registers, and one of them issues.
template <int D, int BITS>
__device__ __forceinline__ void mma_role(const ChunkAttnArgs& a, const Waits& wt, uint32_t smem, uint32_t tmem,
                                         const Seg* ring) {
  using C = Cfg<D, BITS>;
  constexpr uint32_t kIdescQK = tc5::instr_desc(128, C::TN, false);
  constexpr uint32_t kIdescPV = tc5::instr_desc(128, D, true);
  SegReader k;
  uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};  // phases of the lanes' barriers
  uint32_t kv = 0;                          // tiles so far
  bool ok = true;
  auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  for (;; ++k.i) {
    if (!all(k.wait(wt)) || uniform(k.get(ring).b) < 0) break;
    const bool alt = uniform(k.get(ring).alt);
    const int n = uniform(k.get(ring).hi - k.get(ring).lo);
    wt.arrive_warp(B_SEGEMPTY + k.i % kSegs);
    const int U = C::LANES == 2 && !alt ? 2 * n : n;
    ok = wt.wait_warp(B_QFULL, qn[0]++ & 1);
    if (ok && C::LANES == 2 && !alt) ok = wt.wait_warp(B_QFULL + 1, qn[1]++ & 1);
    if (!ok) break;
    auto tile = [&](int u) { return C::LANES == 2 && !alt ? u >> 1 : u; };
    auto lane_of = [&](int u) { return C::LANES == 2 ? u & 1 : 0; };
    // the step's tile is read by no later step
    auto releases = [&](int u) { return C::LANES == 1 || alt || (u & 1); };
    auto qk = [&](int u) -> bool {
      const uint32_t t = kv + tile(u);
      const int stage = t % C::ST, lane = lane_of(u);
      if ((C::LANES == 1 || alt || lane == 0) && !wt.wait_warp(B_KFULL + stage, (t / C::ST) & 1)) return false;
      tc5::fence_after();
      const uint64_t qd = tc5::smem_desc(smem + C::OFF_Q + (alt ? 0 : lane * C::QBYTES), 16, 8 * C::RB, C::SWZ);
      const uint64_t kd = tc5::smem_desc(smem + C::OFF_K + stage * C::KBYTES, 16, 8 * C::RB, C::SWZ);
      if (tc5::elect()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          constexpr int PW = C::PW;
          const int panel = j * 16 / PW, in = (j * 16 % PW) * 2;
          tc5::mma_ss(tmem + C::S0 + lane * C::TN, qd + ((panel * C::QP + in) >> 4), kd + ((panel * C::KP + in) >> 4),
                      kIdescQK, j > 0);
        }
        tc5::commit(wt.bar(B_SFULL + lane));
        if (releases(u)) tc5::commit(wt.bar(B_KEMPTY + stage));
      }
      __syncwarp();
      return true;
    };
    for (int u = 0; ok && u < C::LANES && u < U; ++u) ok = qk(u);
    for (int u = 0; ok && u < U; ++u) {
      const uint32_t t = kv + tile(u);
      const int stage = t % C::ST, lane = lane_of(u);
      ok = wt.wait_warp(B_PREADY + lane, pn[lane]++ & 1);
      if (ok && (C::LANES == 1 || alt || lane == 0)) ok = wt.wait_warp(B_VFULL + stage, (t / C::ST) & 1);
      if (!ok) break;
      tc5::fence_after();
      const uint64_t vd = tc5::smem_desc(smem + C::OFF_V + stage * C::KBYTES, C::KP, 8 * C::RB, C::SWZ);
      const bool acc = u >= C::LANES;  // the lane's first tile of the segment starts O
      if (tc5::elect()) {
#pragma unroll
        for (int j = 0; j < C::TN / 16; ++j) {
          // P of each half of the tokens lies at the start of that half of S
          const int col = j * 16 / C::HC * C::HC + (j * 16 % C::HC) / 2;
          tc5::mma_ts(tmem + C::O0 + lane * C::OSTEP, tmem + C::S0 + lane * C::TN + col,
                      vd + ((j * 16 * C::RB) >> 4), kIdescPV, acc || j > 0);
        }
        if (releases(u)) tc5::commit(wt.bar(B_VEMPTY + stage));
        if (u + C::LANES >= U) tc5::commit(wt.bar(B_ODONE + lane));
      }
      __syncwarp();
      // after PV(u) in the tensor cores' order: S may take P's place
      if (u + C::LANES < U) ok = qk(u + C::LANES);
    }
    if (!ok) break;
    kv += n;
  }
  // nothing of this thread's is in flight when TMEM is freed
  if (tc5::elect()) tc5::commit(wt.bar(B_DRAIN));
  __syncwarp();
  wt.wait_warp(B_DRAIN, 0);
}

// ------------------------------------------------------------------ softmax ---

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <int D, int BITS>
struct Soft {
  using C = Cfg<D, BITS>;
  const ChunkAttnArgs& a;
  const Waits& wt;
  const uint32_t smem, tmem;  // tmem: with the warp's lanes
  uint32_t phases;            // parity bits of the barriers that the thread waits on
  uint32_t at_seg, seg;       // place in the ring of segments, segments so far

  enum { P_S = 0, P_O = 1, P_PAIR = 2, P_MAX = 3, P_STARTED = 4 };

  // Accumulator, half of its columns, and row: by the thread.
  static __device__ __forceinline__ int lane() { return threadIdx.x >> 8; }
  static __device__ __forceinline__ int half() { return (threadIdx.x >> 7) & 1; }
  static __device__ __forceinline__ int r() { return threadIdx.x & 127; }

  __device__ __forceinline__ bool wait(int bar, int bit) {
    const bool ok = wt.wait_warp(bar, (phases >> bit) & 1);
    phases ^= 1u << bit;
    return ok;
  }
  __device__ __forceinline__ bool pair_sync() {
    wt.arrive_warp(B_PAIR);
    return wait(B_PAIR, P_PAIR);
  }
  // with the warp that has the same rows and the other half of the columns
  __device__ __forceinline__ bool row_sync() {
    const int b = B_MAX + lane() * 4 + (r() >> 5);
    wt.arrive_warp(b);
    return wait(b, P_MAX);
  }
  __device__ __forceinline__ uint32_t xmax() const { return smem + C::OFF_MAX + lane() * 1024; }

  // The current segment, read field by field.
  struct Ref {
    uint32_t at;
#define KVQ_SEG_FIELD(name) \
  __device__ __forceinline__ int name() const { return (int)lds(at + (uint32_t)offsetof(Seg, name)); }
    KVQ_SEG_FIELD(b)
    KVQ_SEG_FIELD(h)
    KVQ_SEG_FIELD(qb)
    KVQ_SEG_FIELD(lo)
    KVQ_SEG_FIELD(hi)
    KVQ_SEG_FIELD(npt)
    KVQ_SEG_FIELD(nt)
    KVQ_SEG_FIELD(alt)
    KVQ_SEG_FIELD(c0)
    KVQ_SEG_FIELD(n)
    KVQ_SEG_FIELD(ns)
    KVQ_SEG_FIELD(npk)
    KVQ_SEG_FIELD(nres)
#undef KVQ_SEG_FIELD
  };
  __device__ __forceinline__ Ref ref() const { return {smem + C::OFF_SEG + (at_seg % kSegs) * (uint32_t)sizeof(Seg)}; }
  __device__ __forceinline__ bool wait_seg() const {
    return wt.wait_warp(B_SEGFULL + at_seg % kSegs, (at_seg / kSegs) & 1);
  }

  __device__ __forceinline__ int block_rows(const Ref& k) const { return min(k.n() * a.gq - k.qb() * C::QB, C::QB); }
  __device__ __forceinline__ int block_row(const Ref& k) const { return (k.alt() ? 0 : lane() * 128) + r(); }
  // Where query row `row` of the block is, in q and in the output.
  __device__ __forceinline__ int64_t row_at(const Ref& k, int row) const {
    const int R = k.qb() * C::QB + row;
    const int tok = token_of(a, R);
    return ((int64_t)(k.c0() + tok) * a.Hq + k.h() * a.gq + (R - tok * a.gq)) * D;
  }

  // The lane's 128 rows of Q, in storage order and swizzled.
  __device__ __forceinline__ void load_q() {
    const Ref k = ref();
    if (k.alt() && lane() == 1) return;
    constexpr int LPR = D / 16;    // threads of a row, 32 bytes each
    constexpr int RPI = 32 / LPR;  // rows of a warp at a time
    const int w = half() * 4 + (r() >> 5), l = r() & 31;  // a warp loads 16 rows
    const int rows = block_rows(k) - lane() * 128;
    const uint32_t base = smem + C::OFF_Q + lane() * C::QBYTES;
#pragma unroll 2
    for (int i = 0; i < 16 / RPI; ++i) {
      const int row = w * 16 + i * RPI + l / LPR, c = (l % LPR) * 2;  // c: 16-byte piece of the row
      uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
      if (row < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + row_at(k, lane() * 128 + row)) + c;
        u0 = src[0];
        u1 = src[1];
      }
      to_storage<BITS>(u0, u1);
      const uint32_t at = base + (c * 8 / C::PW) * C::QP;
      const int cc = c % (C::PW / 8);
      st_shared_v4(at + swizzled<C::RB>(row, cc), u0);
      st_shared_v4(at + swizzled<C::RB>(row, cc + 1), u1);
    }
    ptx::fence_proxy_async_shared();
    wt.arrive_warp(B_QFULL + lane());
  }

  // Hides what the row does not see of 32 tokens (a page: `bad` all of them); the largest
  // score that is left.
  static __device__ __forceinline__ float mask(float (&s)[32], int visible, uint32_t bad) {
    // a bit for each token (bits become predicates several at a time)
    const uint32_t seen = bad || visible <= 0 ? 0u : visible >= 32 ? ~0u : (1u << visible) - 1u;
    float x = -INFINITY, y = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      s[j] = (seen >> j) & 1u ? s[j] : -INFINITY;
      s[j + 1] = (seen >> (j + 1)) & 1u ? s[j + 1] : -INFINITY;
      x = fmaxf(x, s[j]);
      y = fmaxf(y, s[j + 1]);
    }
    return fmaxf(x, y);
  }

  // One tile: the weights of the group's half of S's row into TMEM, m (the same in both
  // groups) and l (each group's own) brought up to date.  visible: columns of the half
  // that the row sees (a prefix); bad: pages of it left out.
  __device__ __forceinline__ bool tile(int visible, uint32_t bad, float& m, float& l) {
    const uint32_t sa = tmem + C::S0 + lane() * C::TN + half() * C::HC;
    // 32 scores at a time, read again after the maximum is known: 64 at once and what
    // else lives do not fit the registers, and the small L1 beside the tiles makes a
    // spilled register a trip to L2
    float s[32];
    const bool masked = __any_sync(0xffffffffu, visible < C::HC) || bad;
    float mine = -INFINITY;
#pragma unroll
    for (int h = C::HC - 32; h >= 0; h -= 32) {
      float mx;
      tc5::ld32_max(sa + h, reinterpret_cast<uint32_t*>(s), mx);
      tc5::wait_ld();
      tc5::pin32(reinterpret_cast<uint32_t*>(s));
      asm volatile("" : "+f"(mx));
      if (masked) mx = mask(s, visible - h, (bad >> (h / 32)) & 1u);
      mine = fmaxf(mine, mx);
    }
    // the row's maximum: of this half and of the other group's
    stsf(xmax() + half() * 512 + r() * 4, mine);
    if (!row_sync()) return false;
    const float mn = fmaxf(m, fmaxf(mine, ldsf(xmax() + (half() ^ 1) * 512 + r() * 4)));
    const bool moves = (mn - m) * a.scale_log2 > 8.0f;
    if (__any_sync(0xffffffffu, moves)) {
      const float f = moves ? ptx::ex2_ftz((m - mn) * a.scale_log2) : 1.0f;
      if (moves) m = mn;
      l *= f;
      if (phases & (1u << P_STARTED)) {
        const uint32_t oa = tmem + C::O0 + lane() * C::OSTEP + half() * C::HD;
#pragma unroll 1
        for (int i = 0; i < C::HD; i += 8) {
          uint32_t o[8];
          tc5::ld8(oa + i, o);
          tc5::wait_ld();
          tc5::pin8(o);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tc5::st8(oa + i, o);
        }
      }
    }
    const float off = m == -INFINITY ? 0.0f : fmaf(-m, a.scale_log2, kWeightBits);
    const uint64_t c2 = pack_f32x2(a.scale_log2, a.scale_log2), off2 = pack_f32x2(off, off);
    uint64_t sum2 = pack_f32x2(l, 0.0f);
#pragma unroll
    for (int h = 0; h < C::HC; h += 32) {
      if (h > 0) {
        tc5::ld32(sa + h, reinterpret_cast<uint32_t*>(s));
        tc5::wait_ld();
        tc5::pin32(reinterpret_cast<uint32_t*>(s));
        if (masked) mask(s, visible - h, (bad >> (h / 32)) & 1u);
      }
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t x = fma_f32x2(pack_f32x2(s[i], s[i + 1]), c2, off2);
        const float e0 = ptx::ex2_ftz(__uint_as_float(lo_bits(x)));
        const float e1 = ptx::ex2_ftz(__uint_as_float(hi_bits(x)));
        sum2 = add_f32x2(sum2, pack_f32x2(e0, e1));
        p[i / 2] = ptx::pack_h2(e0, e1);
      }
      tc5::st16(sa + h / 2, p);
    }
    l = __uint_as_float(lo_bits(sum2)) + __uint_as_float(hi_bits(sum2));
    tc5::wait_st();
    return true;
  }

  // What the notes say of the group's columns of the row: it sees `lim` tokens; written over the
  // thread's own earlier stores, to the output (whole) or to the piece's O in `slot`.  A row
  // whose sum is NaN (inv; a seen key may be) stays NaN; the join sees to that for pieces.
  __device__ __forceinline__ void notes(int lim, bool whole, float inv, int64_t at, int slot, int row) const {
    const uint32_t pn = smem + C::OFF_POISON;
#pragma unroll 1
    for (int c = half() * C::HD; c < (half() + 1) * C::HD; ++c) {
      const bool up = (int)lds(pn + 4 * c) < lim, down = (int)lds(pn + 4 * (D + c)) < lim,
                 nan = (int)lds(pn + 4 * (2 * D + c)) < lim;
      if (!(up || down || nan)) continue;
      const float v = nan || (up && down) || inv != inv ? NAN : up ? INFINITY : -INFINITY;
      if (!whole) {
        __stcg(reinterpret_cast<float*>(a.o_part) + ((int64_t)slot * C::QB + row) * D + c, v);
        continue;
      }
      int e = 0;  // the element that is stored at this column
      while (place<BITS>(e) != (c & 15)) ++e;
      e += c & ~15;
      if (a.out_f32)
        static_cast<float*>(a.out)[at + e] = v;
      else
        static_cast<__half*>(a.out)[at + e] = __float2half(v);
    }
  }

  // 16 columns in storage order, times f, to the output's elements at `at`.
  __device__ __forceinline__ void store16(const float* o, float f, int64_t at) const {
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = o[place<BITS>(e)] * f;
    if (a.out_f32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + at);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        dst[e] = make_uint4(ptx::pack_h2(y[8 * e], y[8 * e + 1]), ptx::pack_h2(y[8 * e + 2], y[8 * e + 3]),
                            ptx::pack_h2(y[8 * e + 4], y[8 * e + 5]), ptx::pack_h2(y[8 * e + 6], y[8 * e + 7]));
    }
  }
  __device__ __forceinline__ float inverse(float l) const {
    if (l == 0.0f) set_error(a.err_word, KVQ_ERRBIT_EMPTY);  // nothing seen
    return l == 0.0f ? 0.0f : 1.0f / l;
  }

  // The tiles of a segment: m and l of the row's columns.
  __device__ __forceinline__ bool tiles(float& m, float& l) {
    m = -INFINITY;
    l = 0.0f;
    phases &= ~(1u << P_STARTED);
    // packed tiles, then fp16 ones: t and its end, and the tokens that the row sees from t on
#pragma unroll 1
    for (int f16 = 0; f16 < 2; ++f16) {
      int t, end, visible;
      bool live;
      {
        const Ref k = ref();
        const int row = block_row(k), rows = block_rows(k), npt = k.npt(), alt = k.alt();
        t = k.lo() + (alt ? lane() : 0);
        // (the lane's first tile that is not packed)
        if (f16 && t < npt) t += alt ? (npt - t + 1) & ~1 : npt - t;
        end = f16 ? k.hi() : min(k.hi(), npt);
        live = (row & ~31) < rows;
        visible = 1 << 30;  // rows that are not there need no mask
        if (row < rows) {
          const int ns = k.ns(), npk = k.npk();
          const int lim = seen_of(a, k.n(), ns + npk + k.nres(), token_of(a, k.qb() * C::QB + row));
          visible = (f16 ? seen_f16(ns, npk, lim) + npt * C::TN : seen_packed(ns, npk, lim)) - t * C::TN;
          visible -= half() * C::HC;
        }
      }
#pragma unroll 1
      while (t < end) {
        uint32_t bad = 0;
        if (a.rm.paged && !f16) {
          const Ref k = ref();
          const int j = (t * C::TN + half() * C::HC) / kPage + (r() & 31);
          bool out = false;
          if ((r() & 31) < C::HC / kPage && j * kPage < k.npk()) {
            const int pg = a.rm.page_of(k.b(), j);
            out = pg < 0 || pg >= a.rm.npages;
          }
          bad = __ballot_sync(0xffffffffu, out);
        }
        if (!wait(B_SFULL + lane(), P_S)) return false;
        tc5::fence_after();
        if (live && !tile(visible, bad, m, l)) return false;
        tc5::fence_before();
        wt.arrive_warp(B_PREADY + lane());
        phases |= 1u << P_STARTED;
        const int step = ref().alt() ? 2 : 1;
        t += step;
        if (visible < (1 << 29)) visible -= step * C::TN;
      }
    }
    return true;
  }

  __device__ __forceinline__ bool run(int block) {
    if (!wait_seg()) return false;
    if (ref().b() < 0) return true;
    load_q();
    while (true) {
      float m, l;
      if (!tiles(m, l)) return false;
      const bool any = (phases >> P_STARTED) & 1;
      if (any && !wait(B_ODONE + lane(), P_O)) return false;
      tc5::fence_after();

      const Ref k = ref();
      const bool alt = k.alt();
      const int row = block_row(k), rows = block_rows(k);
      const bool live = (row & ~31) < rows;
      const bool whole = k.lo() == 0 && k.hi() == k.nt();
      // With alternating lanes, lane 1's accumulator of a whole unit goes through shared
      // memory (its Q) to lane 0, 16 columns of each half at a time, with its rows' m and l.
      const bool pass = alt && whole && k.hi() - k.lo() > 1;
      // no MMA reads Q any more (with alternating lanes once the other lane is done too): the
      // next segment's, under this one's epilogue
      if (alt && !pair_sync()) return false;
      ++at_seg;
      if (!wait_seg()) return false;
      const bool more = ref().b() >= 0;
      if (more && !pass) load_q();
      // l of both groups.  The next segment's Q may be there already, and its first maximum
      // goes where l is: the partner says when it has read (waited for below).
      if (live) {
        stsf(xmax() + half() * 512 + r() * 4, l);
        if (!row_sync()) return false;
        l += ldsf(xmax() + (half() ^ 1) * 512 + r() * 4);
        wt.arrive_warp(B_MAX + lane() * 4 + (r() >> 5));
      }
      const bool noted = wt.word(W_PFLAG) != 0;
      const int slot = 2 * block + (k.lo() == 0);
      float inv = 0.0f;
      int64_t at = 0;
      float f0 = 1.0f, f1 = 0.0f;
      if (pass) {
        const uint32_t x1 = smem + C::OFF_Q + (C::LANES - 1) * C::QBYTES + r() * 4;
        if (lane() == 1 && half() == 0 && live) {
          stsf(x1, m);
          stsf(x1 + 512, l);
        }
        if (!pair_sync()) return false;
        if (lane() == 0) {
          const float m1 = ldsf(x1), l1 = ldsf(x1 + 512), mm = fmaxf(m, m1);
          // a lane that saw nothing has weight zero (NaN scores stay NaN through l)
          f0 = m == -INFINITY ? 0.0f : ptx::ex2_ftz((m - mm) * a.scale_log2);
          f1 = m1 == -INFINITY ? 0.0f : ptx::ex2_ftz((m1 - mm) * a.scale_log2);
          if (l != l) f0 = l;
          if (l1 != l1) f1 = l1;
          l = l * f0 + l1 * f1;
          m = mm;
        }
      }
      const bool mine = row < rows && !(alt && whole && lane() == 1);
      const int prow = lane() * 128 + r();  // row in a piece
      if (mine) {
        at = row_at(k, row);
        if (whole)
          inv = inverse(l);
        else if (half() == 0)
          __stcg(a.ml_part + (int64_t)slot * C::QB + prow, make_float2(m, l));
      }
#pragma unroll 1
      for (int c0 = 0; c0 < C::HD; c0 += 16) {
        float o[16];
        if (live && any) {
          tc5::ld16(tmem + C::O0 + lane() * C::OSTEP + half() * C::HD + c0, reinterpret_cast<uint32_t*>(o));
          tc5::wait_ld();
          tc5::pin16(reinterpret_cast<uint32_t*>(o));
        }
        if (pass) {
          const uint32_t st = smem + C::OFF_STAGE + half() * (16 * 128 * 4) + r() * 4;
          if (lane() == 1 && live) {
#pragma unroll
            for (int j = 0; j < 16; ++j) stsf(st + j * 512, o[j]);
          }
          if (!pair_sync()) return false;
          if (lane() == 0 && live) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = o[j] * f0 + ldsf(st + j * 512) * f1;
          }
          if (!pair_sync()) return false;
        }
        const int col = half() * C::HD + c0;
        if (mine && whole) {
          store16(o, inv, at + col);
        } else if (mine) {
          float4* dst = a.o_part + ((int64_t)slot * C::QB + prow) * (D / 4) + col / 4;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            __stcg(dst + j, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        }
        __syncwarp();
      }
      if (noted) {
        if (mine) {
          const int lim = seen_of(a, k.n(), k.ns() + k.npk() + k.nres(), token_of(a, k.qb() * C::QB + row));
          notes(lim, whole, inv, at, slot, prow);
        }
        // the notes have been read: clean them
        if (!pair_sync()) return false;
        for (int i = threadIdx.x; i < 3 * D; i += C::SMW * 32) sts(smem + C::OFF_POISON + 4 * i, 0x7fffffff);
        if (threadIdx.x == 0) wt.set_word(W_PFLAG, 0);
        if (!pair_sync()) return false;
      }
      if (live && !wait(B_MAX + lane() * 4 + (r() >> 5), P_MAX)) return false;  // (as a rule long since)
      tc5::fence_before();
      __threadfence_block();
      __syncwarp();
      if ((r() & 31) == 0)
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(wt.bars + 4 * W_EPI) : "memory");

      if (!whole && k.lo() == 0 && threadIdx.x < 4) a.heads[block * 4 + threadIdx.x] = lds_v4(k.at + 16 * threadIdx.x);
      wt.arrive_warp(B_SEGEMPTY + (at_seg - 1) % kSegs);
      if (!more) return true;
      // (the last read of what passed through Q was followed by a barrier of all)
      if (pass) load_q();
    }
  }
};

// ------------------------------------------------------------------- kernel ---

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkAttnArgs a) {
  using C = Cfg<D, BITS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw;
  const uint32_t smem = ptx::smem_u32(base);
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(base + C::OFF_BAR);
  volatile int64_t* wide = reinterpret_cast<volatile int64_t*>(base + C::OFF_BAR);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lid = tid & 31;
  // nothing is read or written before the kernel before this one is done
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) a.heads[blockIdx.x * 4].x = -1;  // (a later head is this thread's store too)
  if (smem & 1023u) {  // the swizzles count on it (a block without static shared memory has it)
    if (tid == 0) set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
    return;
  }

  // The line of tiles: each thread sums up some sequences, then the block scans.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, tid * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    if (blockIdx.x == 0 && run_of(a.cu, b, a.total, a.max_len).n < 0) set_error(a.err_word, KVQ_ERRBIT_BADLEN);
    mine += Walk<D, BITS>::seq_cost(a, b);
  }
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lid >= o) scan += v;
  }
  volatile int64_t* scans = reinterpret_cast<volatile int64_t*>(base + C::OFF_SEG);  // (the ring is not in use yet)
  if (lid == 31) scans[warp] = scan;
  __syncthreads();
  int64_t before = 0, W = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    const int64_t v = scans[i];
    if (i < warp) before += v;
    W += v;
  }
  // at least two shared tiles, or nearly three of the lanes' own, to a block
  const int64_t G = max((int64_t)1, min((int64_t)gridDim.x, W / (2 * kCostShared)));
  if (W == 0 || (int64_t)blockIdx.x >= G) return;
  const int64_t x0 = (int64_t)blockIdx.x * W / G, x1 = ((int64_t)blockIdx.x + 1) * W / G;
  before += scan - mine;
  if (warp == 20) {
    tc5::alloc(smem + C::OFF_BAR + 4 * W_TMEM, 512);
  } else if (warp == 21) {
    for (int i = lid; i < B_COUNT; i += 32) {
      int n = 1;  // arrivals of a phase
      if (i == B_QFULL || i == B_QFULL + 1 || i == B_PREADY || i == B_PREADY + 1) n = 8;
      if (i == B_SFULL || i == B_SFULL + 1) n = 1 + a.fault;
      if (i >= B_MAX && i < B_MAX + 8) n = 2;
      if (i >= B_SEGEMPTY && i < B_SEGEMPTY + kSegs) n = C::SMW + 4 + 1 + C::BULK;
      if (i >= B_RAWEMPTY && i < B_RAWEMPTY + 3) n = 4;
      if (i == B_PAIR) n = C::SMW;
      if ((i >= B_KFULL && i < B_KFULL + 4) || (i >= B_VFULL && i < B_VFULL + 4)) n = 4;
      ptx::mbar_init(smem + C::OFF_BAR + 8 * i, n);
    }
    if (lid == 0) words[W_ABORT] = words[W_PFLAG] = words[W_EPI] = 0;
    ptx::fence_mbar_init();
  }
  int* poison = reinterpret_cast<int*>(base + C::OFF_POISON);
  for (int i = tid; i < 3 * D; i += kThreads) poison[i] = 0x7fffffff;
  // The warp whose sequences hold x0 finds the sequence, then the query block, 32 at a time.
  const uint32_t holds = __ballot_sync(0xffffffffu, before <= x0 && x0 < before + mine);
  if (holds) {
    int b = b_lo;
    if (before <= x0 && x0 < before + mine) {
      for (; b < b_hi; ++b) {
        const int64_t c = b_hi - b_lo == 1 ? mine : Walk<D, BITS>::seq_cost(a, b);
        if (x0 < before + c) break;
        before += c;
      }
    }
    const int src = __ffs(holds) - 1;
    b = __shfl_sync(0xffffffffu, b, src);
    int64_t at = __shfl_sync(0xffffffffu, before, src);
    const Run run = run_of(a.cu, b, a.total, a.max_len);
    const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
    const int nq = Walk<D, BITS>::blocks(a, run);
    for (int q0 = 0; q0 < nq; q0 += 32) {
      int64_t c = 0;
      if (q0 + lid < nq) {
        int npt, nt, w;
        Walk<D, BITS>::tiles(a, run, s, q0 + lid, npt, nt, w);
        c = Walk<D, BITS>::unit_cost(nt, w) * a.Hkv;
      }
      int64_t sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lid >= o) sum += v;
      }
      const bool here = at + sum - c <= x0 && x0 < at + sum;
      if (here) {
        words[W_STARTB] = b;
        words[W_STARTQ] = q0 + lid;
        wide[W_BASE / 2] = at + sum - c;
      }
      if (__any_sync(0xffffffffu, here)) break;
      at += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[W_TMEM], 0);
  const Waits wt = {a, smem + C::OFF_BAR};
  Seg* ring = reinterpret_cast<Seg*>(base + C::OFF_SEG);
  const int sb = words[W_STARTB], sq = words[W_STARTQ];
  const int64_t sbase = wide[W_BASE / 2];

  // Registers: 80 a thread at launch (61440 in all) = 512 x 88 + 128 x 88 + 128 x 40.
  if (warp < 16) {
    tc5::regs_inc<88>();
    if (warp < C::SMW) {
      Soft<D, BITS> soft = {a, wt, smem, tmem + ((uint32_t)(warp & 3) << 21), 0, 0, 0};
      soft.run(blockIdx.x);
    }
  } else if (warp < 20) {
    tc5::regs_inc<88>();
    Deq<D, BITS> deq = {a, wt, smem, poison, ring, tid - 512, 0};
    deq.run();
  } else {
    tc5::regs_dec<40>();
    if (warp == 20) mma_role<D, BITS>(a, wt, smem, tmem, ring);
    if (tid == 21 * 32) walk_role<D, BITS>(a, wt, ring, sb, sq, sbase, x0, x1, W, G);
    if constexpr (C::BULK)
      if (warp == 22) fetch_role<D, BITS>(a, wt, smem, ring);
    __syncwarp();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (tid == 0 && words[W_ABORT]) set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
  if (warp == 20) tc5::dealloc(tmem, 512);
}

// The pieces of the units that were cut.  All their rows lie in one line; a row is a
// group of D / 4 lanes (head_dim 128 and 256: a warp), which reads its pieces four at a
// time, maxima, sums and values together, and has two rows in flight.  With fewer rows
// than blocks a block has a row, whose pieces its groups share.  The order is fixed.
// Latency bounds it: before the first piece there are only the ends of the units.
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 3;   // of an SM
constexpr int kMaxBlocks = 256;  // of the kernel above

// A part's weight against the row's maximum: never zero, so that an infinite value that a
// part has from the notes stays one (0 x inf is NaN); finite parts of 2^-126 are nothing.
__device__ __forceinline__ float part_weight(float below, float scale_log2) {
  return fmaxf(ptx::ex2_ftz(below * scale_log2), 1.17549435e-38f);
}

template <int D>
struct Joined {
  static constexpr int LPR = D >= 128 ? 32 : D / 4;  // lanes of a row
  static constexpr int V = D / 4 / LPR;              // float4 of a lane
  static constexpr int P = 4 / V;                    // pieces at a time
  float m = -INFINITY, l = 0.0f;
  float4 o[V];

  __device__ __forceinline__ Joined() {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  // Where piece s of row `row` of block `head`'s unit is (alt: pieces and lanes in turn).
  static __device__ __forceinline__ int64_t piece(int head, int alt, int row, int s) {
    const int p = head + (alt ? s >> 1 : s);
    return (2 * (int64_t)p + (p == head)) * chunk_rows(D) + row + (alt ? (s & 1) * 128 : 0);
  }
  struct Loads {
    float2 ml[P];
    float4 x[P][V];
  };
  static __device__ __forceinline__ void load(const ChunkAttnArgs& a, Loads& in, int head, int alt, int row,
                                              int subs, int s, int stride) {
    const int col = threadIdx.x % LPR;
#pragma unroll
    for (int i = 0; i < P; ++i, s += stride) {
      in.ml[i] = make_float2(-INFINITY, 0.0f);
      if (s < subs) {
        const int64_t at = piece(head, alt, row, s);
        in.ml[i] = __ldcg(a.ml_part + at);
#pragma unroll
        for (int v = 0; v < V; ++v) in.x[i][v] = __ldcg(a.o_part + at * (D / 4) + col + v * LPR);
      }
    }
  }
  __device__ __forceinline__ void scale(float f) {
    l *= f;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v].x *= f, o[v].y *= f, o[v].z *= f, o[v].w *= f;
  }
  // (a piece that saw nothing may have written no values)
  __device__ __forceinline__ void add(const Loads& in, float scale_log2) {
    float mm = m;
#pragma unroll
    for (int i = 0; i < P; ++i) mm = fmaxf(mm, in.ml[i].x);
    if (m != -INFINITY) scale(part_weight(m - mm, scale_log2));
    m = mm;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (in.ml[i].x == -INFINITY && in.ml[i].y == 0.0f) continue;
      // a sum without a maximum is NaN, and stays so
      const float f = in.ml[i].x == -INFINITY ? in.ml[i].y : part_weight(in.ml[i].x - mm, scale_log2);
      l += in.ml[i].y * f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v].x += in.x[i][v].x * f;
        o[v].y += in.x[i][v].y * f;
        o[v].z += in.x[i][v].z * f;
        o[v].w += in.x[i][v].w * f;
      }
    }
  }
};

template <int D, int BITS>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) chunk_join_kernel(const ChunkAttnArgs a, int blocks) {
  using J = Joined<D>;
  constexpr int QB = chunk_rows(D);
  constexpr int LPR = J::LPR, V = J::V;
  constexpr int kGroups = kJoinThreads / LPR;  // rows of a block at a time
  __shared__ int ends[kMaxBlocks];             // rows of the units that blocks 0 .. i began
  __shared__ int sums[kJoinThreads / 32];
  __shared__ Seg heads[kMaxBlocks];            // ... and those units
  __shared__ float2 part_ml[kGroups];          // a block's row: the groups' parts of it
  __shared__ float part[kGroups][D + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  {
    int rows = 0;
    if (tid < blocks) {
      int4* to = reinterpret_cast<int4*>(heads + tid);
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = __ldcg(a.heads + tid * 4 + i);
      const Seg& k = heads[tid];
      if (k.b >= 0) rows = min(k.n * a.gq - k.qb * QB, QB);
    }
    int sum = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    for (int i = 0; i < warp; ++i) sum += sums[i];
    ends[tid] = sum;
    __syncthreads();
  }
  const int total = ends[kJoinThreads - 1];
  // the unit of the line's row `it`: the first block with ends > it; rows before it
  auto head_of = [&](int it, int& row) {
    int head = 0;
#pragma unroll
    for (int o = kMaxBlocks / 2; o > 0; o >>= 1)
      if (ends[head + o - 1] <= it) head += o;
    row = it - (head > 0 ? ends[head - 1] : 0);
    return head;
  };
  auto subs_of = [&](int head) { return (heads[head].last_b - head + 1) << (heads[head].alt ? 1 : 0); };
  auto place = [&](int head, int row) {
    const Seg& k = heads[head];
    const int R = k.qb * QB + row;
    const int tok = token_of(a, R);
    return ((int64_t)(k.c0 + tok) * a.Hq + k.h * a.gq + (R - tok * a.gq)) * D;
  };
  auto store = [&](int64_t at, int c, float y) {  // to the element that is stored at column c
    const int c16 = c & 15;
    const int el = (c & ~15) + (BITS == 2 ? (c16 & 1) * 8 + (c16 >> 3) * 4 + ((c16 & 7) >> 1)
                                          : (c16 & 8) + ((c16 & 7) >> 1) + 4 * (c16 & 1));
    if (a.out_f32)
      static_cast<float*>(a.out)[at + el] = y;
    else
      static_cast<__half*>(a.out)[at + el] = __float2half_rn(y);
  };
  auto inverse = [&](float l, bool first) {
    if (l == 0.0f && first) set_error(a.err_word, KVQ_ERRBIT_EMPTY);
    return l == 0.0f ? 0.0f : 1.0f / l;
  };

  const int group = tid / LPR, col = tid % LPR;
  if (total <= (int)gridDim.x) {  // a block to a row
    const int it = blockIdx.x;
    if (it >= total) return;
    int row;
    const int head = head_of(it, row), alt = heads[head].alt, subs = subs_of(head);
    J j;
    for (int s = group; s < subs; s += J::P * kGroups) {
      typename J::Loads in;
      J::load(a, in, head, alt, row, subs, s, kGroups);
      j.add(in, a.scale_log2);
    }
    if (col == 0) part_ml[group] = make_float2(j.m, j.l);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float* to = &part[group][4 * (col + v * LPR)];
      to[0] = j.o[v].x, to[1] = j.o[v].y, to[2] = j.o[v].z, to[3] = j.o[v].w;
    }
    __syncthreads();
    const int64_t at = place(head, row);
    for (int c = tid; c < D; c += kJoinThreads) {
      float m = -INFINITY, l = 0.0f, y = 0.0f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) m = fmaxf(m, part_ml[g].x);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float2 ml = part_ml[g];
        if (ml.x == -INFINITY && ml.y == 0.0f) continue;
        const float f = ml.x == -INFINITY ? ml.y : part_weight(ml.x - m, a.scale_log2);
        l += ml.y * f;
        y += part[g][c] * f;
      }
      store(at, c, y * inverse(l, c == 0));
    }
    return;
  }
  constexpr int K = 2;  // rows in flight
  const int step = gridDim.x * kGroups;
  for (int it = blockIdx.x * kGroups + group; it < total; it += K * step) {
    int row[K], head[K], alt[K], subs[K];
    J j[K];
    int most = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const bool there = it + u * step < total;
      head[u] = head_of(there ? it + u * step : it, row[u]);
      alt[u] = heads[head[u]].alt;
      subs[u] = there ? subs_of(head[u]) : 0;
      most = max(most, subs[u]);
    }
    for (int s = 0; s < most; s += J::P) {
      typename J::Loads in[K];
#pragma unroll
      for (int u = 0; u < K; ++u) J::load(a, in[u], head[u], alt[u], row[u], subs[u], s, 1);
#pragma unroll
      for (int u = 0; u < K; ++u) j[u].add(in[u], a.scale_log2);
    }
#pragma unroll
    for (int u = 0; u < K; ++u) {
      if (subs[u] == 0) continue;
      const float inv = inverse(j[u].l, col == 0);
      const int64_t at = place(head[u], row[u]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y[4] = {j[u].o[v].x, j[u].o[v].y, j[u].o[v].z, j[u].o[v].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) store(at, 4 * (col + v * LPR) + i, y[i] * inv);
      }
    }
  }
}

// The kernels' attributes, once per device.
template <int D, int BITS>
cudaError_t ensure_attrs() {
  auto kernel = chunk_attn_kernel<D, BITS>;
  auto join = chunk_join_kernel<D, BITS>;
  static std::atomic<uint64_t> done{0};  // bit i: set on device i
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
  // the warps' shares (setmaxnreg) come out of what the block is launched with
  if (at.numRegs != 80) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, BITS>::SMEM);
  if (e != cudaSuccess) return e;
  // the same split of L1 and shared memory: an SM that changes it drains first
  e = cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int D, int BITS>
cudaError_t launch(const ChunkAttnArgs& a, int grid, cudaStream_t st) {
  static_assert(Cfg<D, BITS>::SMEM <= 227 * 1024, "shared memory of a block");
  if (grid > kMaxBlocks) return cudaErrorInvalidConfiguration;
  cudaError_t e = ensure_attrs<D, BITS>();
  if (e != cudaSuccess) return e;
  // each may be launched while the kernel before it ends, and waits for it
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = Cfg<D, BITS>::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, chunk_attn_kernel<D, BITS>, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3(kJoinBlocks * grid);
  cfg.blockDim = kJoinThreads;
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, BITS>, a, grid);
}

template <int D>
cudaError_t launch_bits(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st) {
  if (bits == 4) return launch<D, 4>(a, grid, st);
  if (bits == 3) return launch<D, 3>(a, grid, st);
  return launch<D, 2>(a, grid, st);
}

}  // namespace chunk
}  // namespace kvq
