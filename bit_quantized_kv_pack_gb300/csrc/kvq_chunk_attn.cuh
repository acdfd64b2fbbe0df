// kvq_chunk_attn.cuh -- attention of runs of several tokens over the low-bit cache on
// the fifth-generation tensor cores.
//
// The mathematics.  The query rows of one (sequence, KV head) are its run's tokens times
// the gq heads that share the KV head, row = token * gq + head: one pass over K and V
// serves them all.  For a tile of 64 tokens S = Q K^T, P = exp2(S c - m c) with the row's
// reference maximum m, O += P V, l += sum P; c = log2(e) / sqrt(d).  m follows the
// running maximum lazily: it moves (and O, l are rescaled) only when the maximum has
// passed it by 2^8, so weights stay below 256 and the sums lose nothing in fp32.
// Roundings: the dequantized keys and values min + code * scale are rounded to fp16 once
// (operands of the MMA), the weights P to fp16 once; scores, m, l and O are fp32.
//
// A block (one per SM, persistent) has 28 warps:
//   0-15   softmax: S from TMEM, P back to TMEM (it takes S's place and is the A operand
//          of the second MMA), the epilogue.  Four groups of four warps: two for each of
//          the block's two accumulators (lanes 0 and 1), which take its tiles in turns; a
//          thread per query row.
//   16-23  dequantize, four warps the keys and four the values: a piece of a row of codes
//          comes by cp.async into a ring that is private to its thread (no barrier),
//          becomes fp16 in registers and goes to shared memory in the MMA's swizzle, K as
//          the K-major and V as the MN-major B operand.
//   24, 25 issue the MMAs, one thread for each lane; 26 works out the segments.
// What the shape answers to (head_dim 128): a tile's chain S -> P -> PV -> next S takes
// longer than its MMAs, so each lane has two S buffers and the next S is made while the
// softmax works on this one.  TMEM (2 lanes x 2 x 64 columns of S, 2 x 128 of O) then
// holds tiles of 64 tokens; their QK^T runs at 0.6 of the rate of 128 (measured 861
// against 520 cycles for 128 x 128 x 128), which the overlap outweighs.  An MMA takes its
// issuer about 55 cycles and a commit 85 (measured), hence a thread for each lane.
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

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"
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
  float4* o_part;     // [2 G][d / 4][QB]
  int B, Hkv, Hq, gq, cap, Nr, Ns, total, max_len, causal, out_f32;
  uint32_t gq_mul, gq_shift;  // row / gq = row * gq_mul >> gq_shift for rows below 2^31
  uint32_t wait_limit_us;
  int fault;  // testing hook: one barrier of block 0 waits for an arrival that never comes
  float scale_log2;
};

cudaError_t launch_chunk_attn_d32(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d64(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d128(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);
cudaError_t launch_chunk_attn_d256(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st);

// Query rows of a block (all its lanes).
__host__ __device__ constexpr int chunk_rows(int d) { return d == 256 ? 128 : 256; }

namespace chunk {

constexpr int kThreads = 896;
constexpr int kDeqThreads = 128;  // of the keys, and of the values
constexpr int kTile = 64;         // tokens of a tile
constexpr int kSegs = 8;          // ring of segments

template <int D, int BITS>
struct Cfg {
  static constexpr int LANES = D == 256 ? 1 : 2;    // accumulators
  static constexpr int QB = chunk_rows(D);
  static constexpr int TN = kTile;
  static constexpr int G = D / 32;                  // groups of a row
  static constexpr int PW = D < 64 ? D : 64;        // elements of a panel's row
  static constexpr int RB = PW * 2;                 // bytes of it
  static constexpr int SWZ = RB == 128 ? 2 : 4;
  static constexpr int QP = 128 * RB;               // bytes of a panel of Q
  static constexpr int KP = TN * RB;                // of a panel of K or V
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int KBYTES = TN * D * 2;
  static constexpr int ST = D == 256 ? 2 : 4;       // K and V stages
  static constexpr int HD = D / 2;                  // a softmax group's columns of O
  static constexpr int TPR = D == 256 ? 2 : 1;      // dequantizing threads of a row
  static constexpr int NP = 2 / TPR;                // tiles that four dequantizing warps work on at a time
  static constexpr int GPT = G / TPR;               // groups of a thread
  static constexpr int CB = 4 * BITS;               // code bytes of a group
  static constexpr int TB = GPT * CB;               // code bytes of a thread, contiguous
  static constexpr int UN = (TB + 15) / 16;         // 16-byte units of them in the ring
  static constexpr int PB = GPT * 4;                // param bytes of a thread
  static constexpr int RAWB = kDeqThreads * (UN * 16 + PB);
  static constexpr int RAWN = D >= 128 ? 1 : 3;     // rows of the thread's ring
  static_assert(RAWN * NP < kSegs - 1, "the cursor of the copies stays within the ring of segments");
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
  // 1's Q (but for its first 2 KiB) is free then, and large enough from head_dim 128 on
  static constexpr int STAGE = 2 * 16 * 128 * 4;
  static constexpr int OFF_STAGE = D >= 128 ? OFF_Q + (LANES - 1) * QBYTES + 2048 : OFF_RAW + 2 * RAWN * RAWB;
  static constexpr int OFF_MAX = OFF_RAW + 2 * RAWN * RAWB + (D >= 128 ? 0 : STAGE);  // float [LANES][2][128]
  static_assert(OFF_MAX % 1024 == 0, "a thread finds the other group's value by one bit of the address");
  static constexpr int OFF_POISON = OFF_MAX + LANES * 1024;     // int [3][D]
  static constexpr int OFF_BAR = OFF_POISON + 3 * D * 4;
  static constexpr int OFF_SEG = OFF_BAR + 640;                 // Seg [kSegs]
  static constexpr int SMEM = OFF_SEG + 512;
};

// A segment: the block's tiles [lo, hi) of the unit (sequence b, KV head h, query block
// qb).  One warp works the segments out, the others read them from a ring.
struct alignas(16) Seg {
  int b, h, qb, lo;
  int hi, npt, nt, alt;     // packed tiles and all tiles of the unit; alt: the lanes take alternate tiles
  int c0, n, ns, npk;       // the run, and the sequence's lengths
  int nres, head, first_b, last_b;  // blocks that hold the unit's first and last tile; b < 0: the end
};

// Barriers (8 bytes each from OFF_BAR) and words behind them.
// Of two: of each lane (PVLAST: all PV of a segment but the last); S and P: of each lane
// and S buffer; REF: of each lane, 32 rows and S buffer; EMPTY: of each stage and lane.
// Every phase of a barrier is waited on by whoever waits there at all: parities count.
enum { B_QFULL = 0, B_ODONE = 2, B_PVLAST = 4, B_DRAIN = 6, B_SFULL = 8, B_PREADY = 12, B_REF = 16,
       B_KFULL = 32, B_VFULL = 36, B_KEMPTY = 40, B_VEMPTY = 48, B_SEGFULL = 56, B_SEGEMPTY = 64, B_PAIR = 72,
       B_COUNT = 73 };
enum { W_TMEM = 146, W_ABORT = 147, W_PFLAG = 148, W_EPI = 149, W_STARTB = 151,
       W_STARTQ = 152, W_BASE = 154 /* int64 [2] */ };

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
    set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
    return true;
  }
  __device__ __forceinline__ bool wait_at(uint32_t b, uint32_t parity) const {
    if (ptx::mbar_try_wait(b, parity)) return true;
    const uint32_t t0 = timer_lo();
#pragma unroll 1
    for (uint32_t k = 1; !ptx::mbar_try_wait(b, parity); ++k)
      if ((k & 63u) == 0 && late(t0)) return false;
    return true;
  }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const { return wait_at(bar(i), parity); }
  // a whole warp waits; the same answer for all its lanes
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
    return wait_warp_at(bar(i), parity);
  }
  __device__ __forceinline__ bool wait_warp_at(uint32_t b, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait_at(b, parity));
  }
  __device__ __forceinline__ void arrive_warp(int i) const { arrive_warp_at(bar(i)); }
  static __device__ __forceinline__ void arrive_warp_at(uint32_t b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(b);
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
  int npt, nt, w;  // packed tiles, all tiles, cost of a tile (1 or 2)
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
    w = C::LANES == 2 && last - qb * C::QB >= 128 ? 2 : 1;
  }
  static __device__ __forceinline__ int64_t seq_cost(const ChunkAttnArgs& a, int b) {
    const Run run = run_of(a.cu, b, a.total, a.max_len);
    const int nq = blocks(a, run);
    if (nq == 0) return 0;
    const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
    int64_t c = 0;
    for (int qb = 0; qb < nq; ++qb) {
      int npt, nt, w;
      tiles(a, run, s, qb, npt, nt, w);
      c += (int64_t)nt * w;
    }
    return c * a.Hkv;
  }

  __device__ __forceinline__ void load_seq(const ChunkAttnArgs& a) {
    run = run_of(a.cu, b, a.total, a.max_len);
    s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
  }
  __device__ __forceinline__ void range() {
    // tile k starts at base + k w and is the block's if that is in [x0, x1)
    lo = x0 <= base ? 0 : (int)((x0 - base + w - 1) >> (w - 1));
    const int64_t e = x1 - base + w - 1;
    hi = e <= 0 ? 0 : (int)min((int64_t)nt, e >> (w - 1));
  }
  __device__ __forceinline__ void start(const ChunkAttnArgs& a, int b_, int qb_, int64_t base_, int64_t x0_,
                                        int64_t x1_) {
    b = b_;
    qb = qb_;
    x0 = x0_;
    x1 = x1_;
    load_seq(a);
    tiles(a, run, s, qb, npt, nt, w);
    const int64_t unit = (int64_t)nt * w;
    h = (int)((x0 - base_) / unit);
    base = base_ + h * unit;
    range();
    if (lo >= hi) next(a);
  }
  __device__ __forceinline__ bool valid(const ChunkAttnArgs& a) const { return b < a.B && base < x1; }
  __device__ __forceinline__ void next(const ChunkAttnArgs& a) {
    base += (int64_t)nt * w;
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
  for (uint32_t i = 0;; ++i) {
    const int at = i % kSegs;
    if (!wt.wait(B_SEGEMPTY + at, ((i / kSegs) & 1) ^ 1)) return;
    Seg s;
    s.b = -1;
    if (k.valid(a)) {
      s.b = k.b, s.h = k.h, s.qb = k.qb, s.lo = k.lo, s.hi = k.hi, s.npt = k.npt, s.nt = k.nt;
      s.alt = Cfg<D, BITS>::LANES == 2 && k.w == 1;
      s.c0 = k.run.c0, s.n = k.run.n, s.ns = k.s.ns, s.npk = k.s.npk, s.nres = k.s.nres, s.head = k.s.head;
      s.first_b = s.last_b = 0;
      if (k.lo > 0 || k.hi < k.nt) {
        // block c has the starts from floor(c W / G) on
        const int64_t end = k.base + (int64_t)(k.nt - 1) * k.w;
        s.first_b = (int)(((k.base + 1) * G - 1) / W);
        s.last_b = (int)(((end + 1) * G - 1) / W);
      }
    }
    ring[at] = s;
    ptx::mbar_arrive(wt.bar(B_SEGFULL + at));
    if (s.b < 0) return;
    k.next(a);
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

// What four dequantizing warps share, those of the keys (w 0) or of the values (1).  Two
// warps have a tile, a row to a thread (head_dim 256: four warps, half a row), and the two
// pairs take the tiles in turns.  A thread's codes are contiguous, and 8 neighbouring
// lanes store the same piece of 8 rows, which the swizzle puts into 8 different groups of
// banks.  The raw row goes to registers before its turn, and the next one is on its way
// while this one is worked on.
template <int D, int BITS>
struct Deq {
  using C = Cfg<D, BITS>;
  const ChunkAttnArgs& a;
  const Waits& wt;
  uint32_t smem;  // base of the block's shared memory
  int* poison;
  const Seg* ring;
  int w;
  int dt;         // thread of the four warps
  uint32_t seg;   // segments of the block so far

  __device__ __forceinline__ int row() const { return dt % kTile; }
  __device__ __forceinline__ int part() const { return C::TPR == 2 ? dt / kTile : 0; }
  __device__ __forceinline__ int pair() const { return C::NP == 2 ? dt / kTile : 0; }

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

  // The cursor of the copies: a tile of a segment.
  struct Cursor {
    SegReader seg;
    int tile = 0, hi = 0, npt = 0;
    bool open = false;         // seg has been looked at
    int left = 0;              // packed tokens from the thread's row of the tile on
    int64_t at = 0;            // contiguous: that row; paged: row of the head in a page
    const int32_t* pages = nullptr;  // paged: the entry of the thread's row
    int page = 0;              // ... and what it says, read a tile ahead
  };

  __device__ __forceinline__ uint32_t raw_codes(int slot) const {
    return smem + C::OFF_RAW + (w * C::RAWN + slot) * C::RAWB + dt * 16;
  }
  __device__ __forceinline__ uint32_t raw_params(int slot) const {
    return smem + C::OFF_RAW + (w * C::RAWN + slot) * C::RAWB + kDeqThreads * C::UN * 16 + dt * C::PB;
  }

  // The thread's raw piece of a tile into ring slot `slot`; a row that is not there
  // becomes zero codes with zero params, which stand for zeros.
  __device__ __forceinline__ void fetch(Cursor& c, int slot) {
    const uint32_t dc = raw_codes(slot), dp = raw_params(slot);
    bool there = c.left > 0;
    int64_t at = c.at;
    if (a.rm.paged && there) {
      there = c.page >= 0 && c.page < a.rm.npages;
      if (!there) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
      at += (int64_t)c.page * a.Hkv * kPage;
    }
    if (there) {
      const uint8_t* src = a.codes[w] + at * (C::G * C::CB) + part() * C::TB;
      constexpr int N = C::TB % 16 == 0 ? 16 : C::TB % 8 == 0 ? 8 : 4;
#pragma unroll
      for (int i = 0; i < C::TB / N; ++i)
        cp_async<N>(dc + (i * N / 16) * (kDeqThreads * 16) + i * N % 16, src + i * N);
      cp_async<C::PB>(dp, a.params[w] + at * C::G + part() * C::GPT);
    } else {
#pragma unroll
      for (int i = 0; i < C::UN; ++i) st_shared_v4(dc + i * (kDeqThreads * 16), make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int i = 0; i < C::GPT; ++i) sts(dp + 4 * i, 0);
    }
    // on to the pair's next tile; contiguous rows further on are called into L2
    c.left -= C::NP * C::TN;
    if (a.rm.paged) {
      c.pages += C::NP * C::TN / kPage;
      if (c.left > 0) c.page = __ldg(c.pages);
    } else {
      c.at += C::NP * C::TN;
      if (c.left > C::TN * C::NP) {
        const int64_t far = c.at + C::NP * C::TN;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.codes[w] + far * (C::G * C::CB) + part() * C::TB));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.params[w] + far * C::G));
      }
    }
  }

  // Shared address of the thread's row in a tile at dst, with the row's swizzle in its
  // low bits: piece c of the thread's panel p is at (this ^ (c << 4)) + p * KP.
  __device__ __forceinline__ uint32_t row_addr(uint32_t dst) const {
    const int r = row();
    return dst + part() * (C::GPT / 2) * C::KP + r * C::RB + ((C::RB == 128 ? r & 7 : (r >> 1) & 3) << 4);
  }
  __device__ __forceinline__ int column(int g, int c) const { return (part() * C::GPT + g) * 32 + c * 8; }

  // The thread's raw row in registers.
  struct Raw {
    uint32_t code[C::UN * 4], prm[C::GPT];
  };
  __device__ __forceinline__ void take(Raw& x, int slot) const {
    const uint32_t dc = raw_codes(slot), dp = raw_params(slot);
#pragma unroll
    for (int i = 0; i < C::UN; ++i) {
      const uint4 v = ld_shared_v4(dc + i * (kDeqThreads * 16));
      x.code[4 * i] = v.x, x.code[4 * i + 1] = v.y, x.code[4 * i + 2] = v.z, x.code[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < C::GPT; ++i) x.prm[i] = lds(dp + 4 * i);
  }

  // A raw row as fp16 at `dst`.  token: its logical place.
  __device__ __forceinline__ bool packed_row(const Raw& x, int token, uint32_t dst) {
    constexpr uint32_t kQmax2 = BITS == 4 ? 0x4b804b80u : BITS == 3 ? 0x47004700u : 0x42004200u;  // 15, 7, 3
    const uint32_t at = row_addr(dst);
    uint32_t rare = 0;
#pragma unroll
    for (int g = 0; g < C::GPT; ++g) {
      const uint32_t s2 = ptx::prmt(x.prm[g], x.prm[g], 0x1010), m2 = ptx::prmt(x.prm[g], x.prm[g], 0x3232);
      // the group's largest value; only where it is not finite can any value be so
      if (f16_nonfinite(ptx::hfma2_u32(kQmax2, s2, m2))) rare |= 1u << g;
      uint32_t c8[4];
      code_words<BITS>(x.code, g, c8);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[4];
        codes_f16<BITS>(c8[c], y);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = ptx::hfma2_u32(y[j], s2, m2);
        st_shared_v4((at ^ (((g & 1) * 4 + c) << 4)) + (g / 2) * C::KP, make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
    if (rare == 0) return true;
    // what is not finite among the stored values: past fp16's largest value by the
    // scale's rounding, or meant (params that are not finite)
#pragma unroll 1
    for (int e = 0; e < 32 * C::GPT; ++e) {
      const int g = e >> 5;
      if (!((rare >> g) & 1u)) continue;
      uint32_t pg = x.prm[0];
#pragma unroll
      for (int i = 1; i < C::GPT; ++i) pg = g == i ? x.prm[i] : pg;
      const uint32_t ea = (at ^ (((g & 1) * 4 + ((e >> 3) & 3)) << 4)) + (g / 2) * C::KP + 2 * (e & 7);
      unsigned short hv;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hv) : "r"(ea) : "memory");
      if (!f16_nonfinite(hv)) continue;
      if (!f16_nonfinite(pg) && !f16_nonfinite(pg >> 16))
        hv = (hv & 0x8000u) | 0x7bffu;
      else if (w == 0)
        continue;
      else if (note(column(g, 0) + (e & 31), token, hv))
        hv = 0;
      else
        return false;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(ea), "h"(hv) : "memory");
    }
    return true;
  }

  __device__ __forceinline__ int ring_slot(int j) const { return j < a.Nr ? j : j - a.Nr; }  // j < 2 Nr

  // A tile of fp16 tokens (sink, then window): rows f0 .. of their line.
  __device__ __forceinline__ bool f16_tile(const Seg& k, int f0, uint32_t dst) {
    const int64_t bh = (int64_t)k.b * a.Hkv + k.h;
    const int f = f0 + row(), n = k.ns + k.nres;
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
    c.tile = pair();
    bool ok = true, more = true;
    // The pair's next tile into ring slot `slot`.  c.tile is its place in segment c.seg, or
    // past that segment's end by as many tiles as there are to skip in the next.
    auto fetch_next = [&](int slot) {
      while (more && c.tile >= c.hi) {
        if (c.open) ++c.seg.i;
        c.open = true;
        ok = ok && __all_sync(0xffffffffu, c.seg.wait(wt));
        const Seg& s = c.seg.get(ring);
        more = ok && s.b >= 0;
        if (!more) break;
        c.tile += s.lo - c.hi, c.hi = s.hi, c.npt = s.npt;
        const int p = c.tile * C::TN + row();
        c.left = s.npk - p;
        if (a.rm.paged) {
          c.at = (int64_t)s.h * kPage + p % kPage;
          c.pages = a.rm.block_table + (int64_t)s.b * (a.cap / kPage) + p / kPage;
          if (c.left > 0) c.page = __ldg(c.pages);
        } else {
          c.at = ((int64_t)s.b * a.Hkv + s.h) * a.cap + p;
        }
      }
      if (more) {
        if (c.tile < c.npt) fetch(c, slot);
        c.tile += C::NP;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t kv = 0;             // tiles so far
    uint32_t used = 0, par = 0;  // by stage and lane: the lane has the stage; parity of its release
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < C::RAWN; ++i) fetch_next(i);
    for (; ok; ++k.i, ++seg) {
      ok = ok && __all_sync(0xffffffffu, k.wait(wt));
      if (!ok) break;
      const Seg& s = k.get(ring);
      if (s.b < 0) break;
      const int lo = s.lo, hi = s.hi, npt = s.npt, ns = s.ns, alt = s.alt;
      for (int t = lo + (C::NP == 2 ? (pair() ^ kv) & 1 : 0); t < hi; t += C::NP) {
        const uint32_t x = kv + (t - lo);
        const int stage = x % C::ST;
        const uint32_t dst = smem + (w ? C::OFF_V : C::OFF_K) + stage * C::KBYTES;
        Raw raw;
        if (t < npt) {
          asm volatile("cp.async.wait_group %0;" ::"n"(C::RAWN - 1) : "memory");
          take(raw, slot);
        }
        fetch_next(slot);
        if (++slot == C::RAWN) slot = 0;
        // the lanes that had the stage before have read it
#pragma unroll
        for (int l = 0; l < C::LANES; ++l) {
          const int bit = 2 * stage + l;
          if (ok && ((used >> bit) & 1u)) {
            ok = wt.wait_warp((w ? B_VEMPTY : B_KEMPTY) + bit, (par >> bit) & 1u);
            par ^= 1u << bit;
          }
        }
        if (!ok) break;
        used &= ~(3u << (2 * stage));
        used |= (alt ? 1u << ((t - lo) & 1) : C::LANES == 2 ? 3u : 1u) << (2 * stage);
        ok = t < npt ? packed_row(raw, ns + t * C::TN + row(), dst) : f16_tile(s, (t - npt) * C::TN, dst);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::fence_proxy_async_shared();
        wt.arrive_warp((w ? B_VFULL : B_KFULL) + stage);
      }
      kv += hi - lo;
      wt.arrive_warp(B_SEGEMPTY + k.i % kSegs);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// ---------------------------------------------------------------------- MMA ---

template <int D, int BITS>
__device__ __forceinline__ void mma_role(const ChunkAttnArgs& a, const Waits& wt, uint32_t smem, uint32_t tmem,
                                         const Seg* ring, int lane) {
  using C = Cfg<D, BITS>;
  constexpr uint32_t kIdescQK = tc5::instr_desc(128, C::TN, false);
  constexpr uint32_t kIdescPV = tc5::instr_desc(128, D, true);
  const uint32_t s_at = tmem + C::S0 + lane * 2 * C::TN, o_at = tmem + C::O0 + lane * C::OSTEP;
  const uint64_t kd0 = tc5::smem_desc(smem + C::OFF_K, 16, 8 * C::RB, C::SWZ);
  const uint64_t vd0 = tc5::smem_desc(smem + C::OFF_V, C::KP, 8 * C::RB, C::SWZ);
  SegReader k;
  uint32_t qn = 0;           // phases of the lane's barrier of Q
  uint32_t nqk = 0, npv = 0; // the lane's QK^T and PV so far: S buffers take turns
  uint32_t kv = 0;           // tiles so far
  bool ok = true;
  for (;; ++k.i) {
    if (!k.wait(wt) || k.get(ring).b < 0) break;
    const bool alt = k.get(ring).alt;
    const int n = k.get(ring).hi - k.get(ring).lo;
    ptx::mbar_arrive(wt.bar(B_SEGEMPTY + k.i % kSegs));
    // the lane's tiles: all, or every second one (with Q of lane 0)
    const int step = alt ? 2 : 1, t0 = alt ? lane : 0;
    // (the barrier of lane 1 completes in the segments that have tiles for it, and is
    // waited on in just these: no phase is passed over)
    if (t0 < n) ok = wt.wait(B_QFULL + lane, qn++ & 1);
    const uint64_t qd =
        tc5::smem_desc(smem + C::OFF_Q + (alt ? 0 : lane * C::QBYTES), 16, 8 * C::RB, C::SWZ);
    // tile x of the line (of all the block's segments) is in stage x % ST
    auto qk = [&](uint32_t x) {
      const uint32_t buf = nqk & 1;
      const uint64_t kd = kd0 + (x % C::ST) * (C::KBYTES >> 4);
      const uint32_t to = s_at + buf * C::TN;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        constexpr int PW = C::PW;
        const int panel = j * 16 / PW, in = (j * 16 % PW) * 2;
        tc5::mma_ss(to, qd + ((panel * C::QP + in) >> 4), kd + ((panel * C::KP + in) >> 4), kIdescQK, j > 0);
      }
      tc5::commit(wt.bar(B_SFULL + 2 * lane) + 8 * buf);
      tc5::commit(wt.bar(B_KEMPTY + lane) + 16 * (x % C::ST));
      ++nqk;
    };
    const uint32_t end = kv + n;
    for (uint32_t x = kv + t0; ok && x < end && x < kv + t0 + 2 * step; x += step) {
      ok = wt.wait_at(wt.bar(B_KFULL) + 8 * (x % C::ST), (x / C::ST) & 1);
      if (!ok) break;
      tc5::fence_after();
      qk(x);
    }
#pragma unroll 1
    for (uint32_t x = kv + t0; ok && x < end; x += step) {
      // V and P of this tile, and K of the one whose S comes after: asked for at once (the
      // tensor cores idle while this thread waits)
      const uint32_t y = x + 2 * step, buf = npv & 1;
      const uint32_t vb = wt.bar(B_VFULL) + 8 * (x % C::ST), kb = wt.bar(B_KFULL) + 8 * (y % C::ST),
                     pb = wt.bar(B_PREADY + 2 * lane) + 8 * buf;
      const uint32_t vp = (x / C::ST) & 1, kp = (y / C::ST) & 1, pp = (npv >> 1) & 1;
      const bool more = y < end;
      const bool v_ok = ptx::mbar_try_wait(vb, vp), k_ok = !more || ptx::mbar_try_wait(kb, kp),
                 p_ok = ptx::mbar_try_wait(pb, pp);
      if (!(v_ok && k_ok && p_ok))
        ok = wt.wait_at(vb, vp) && (!more || wt.wait_at(kb, kp)) && wt.wait_at(pb, pp);
      if (!ok) break;
      tc5::fence_after();
      const uint64_t vd = vd0 + (x % C::ST) * (C::KBYTES >> 4);
      const uint32_t from = s_at + buf * C::TN;
      // the lane's first tile of the segment starts O
      tc5::mma_ts(o_at, from, vd, kIdescPV, x != kv + t0);
#pragma unroll
      for (int j = 1; j < C::TN / 16; ++j)
        tc5::mma_ts(o_at, from + j * 8, vd + ((j * 16 * C::RB) >> 4), kIdescPV, true);
      // into the buffer of this tile's P: after PV in the tensor cores' order
      if (more)
        qk(y);
      else
        tc5::commit(wt.bar((x + step < end ? B_PVLAST : B_ODONE) + lane));
      tc5::commit(wt.bar(B_VEMPTY + lane) + 16 * (x % C::ST));
      ++npv;
    }
    if (!ok) break;
    kv += n;
  }
  // nothing of this thread's is in flight when TMEM is freed
  tc5::commit(wt.bar(B_DRAIN + lane));
  wt.wait(B_DRAIN + lane, 0);
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
  const uint32_t tid;
  const uint32_t s_tm;        // TMEM: the group's S buffer
  const uint32_t ref_at;      // shared: the thread's reference maximum (^ 512: the other group's)
  uint32_t at_seg;            // place in the ring of segments
  uint32_t nt;                // tiles of the lane so far: its two groups take turns

  enum { P_O = 1, P_PAIR = 2, P_LAST = 3 };

  // Accumulator, group (and half of O's columns), and row: by the thread.
  __device__ __forceinline__ int lane() const { return tid >> 8; }
  __device__ __forceinline__ int half() const { return (tid >> 7) & 1; }
  __device__ __forceinline__ int r() const { return tid & 127; }

  __device__ __forceinline__ bool wait(int bar, int bit) {
    const bool ok = wt.wait_warp(bar, (phases >> bit) & 1);
    phases ^= 1u << bit;
    return ok;
  }
  __device__ __forceinline__ bool pair_sync() {
    wt.arrive_warp(B_PAIR);
    return wait(B_PAIR, P_PAIR);
  }
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
    KVQ_SEG_FIELD(first_b)
    KVQ_SEG_FIELD(last_b)
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
        u0 = __ldg(src);
        u1 = __ldg(src + 1);
      }
      to_storage<BITS>(u0, u1);
      const uint32_t at = base + (c * 8 / C::PW) * C::QP;
      const int cc = c % (C::PW / 8);
      st_shared_v4(at + swizzled<C::RB>(row, cc), u0);
      st_shared_v4(at + swizzled<C::RB>(row, cc + 1), u1);
    }
    ptx::fence_proxy_async_shared();
    wt.arrive_warp(B_QFULL + lane());
    // with alternating lanes the rows are lane 1's too, if there is a tile for it
    if (k.alt() && k.hi() - k.lo() > 1) wt.arrive_warp(B_QFULL + 1);
  }

  // The weights of 16 scores (the visible ones) against the reference (off = -m c), two to a
  // register, and their sum on top of `sum`.
  __device__ __forceinline__ void weights(float (&s)[16], uint32_t (&p)[8], uint64_t c2, uint64_t off2,
                                          uint64_t& sum, bool masked, int visible) const {
    if (masked) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = j < visible ? s[j] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const uint64_t x = fma_f32x2(pack_f32x2(s[i], s[i + 1]), c2, off2);
      const float e0 = ptx::ex2_ftz(__uint_as_float(lo_bits(x))), e1 = ptx::ex2_ftz(__uint_as_float(hi_bits(x)));
      sum = add_f32x2(sum, pack_f32x2(e0, e1));
      p[i / 2] = ptx::pack_h2(e0, e1);
    }
  }

  // One tile, the lane's n-th: P in S's place, m and l brought up to date.  visible:
  // tokens of the tile that the row sees (a prefix); bad: pages (halves) left out.
  // S is read twice, for its maximum and for the weights: 64 scores at once do not fit the
  // registers, and beside the tiles L1 is so small that a spilled register is a trip to
  // L2.  The reference is the lane's: the group that has tile n takes it over from the
  // other, which had n - 1, and passes it on before it works out its weights.
  __device__ __forceinline__ bool tile(int visible, uint32_t bad, bool first, bool last, float& m, float& l) {
    const bool masked = __any_sync(0xffffffffu, visible < C::TN) || bad;
    float mt = -INFINITY;
#pragma unroll
    for (int h = 0; h < C::TN; h += 32) {
      float s[32], mx;
      tc5::ld32_max(s_tm + h, reinterpret_cast<uint32_t*>(s), mx);
      tc5::wait_ld();
      tc5::pin32(reinterpret_cast<uint32_t*>(s));
      asm volatile("" : "+f"(mx));
      if (masked) {
        const int v = (bad >> (h / 32)) & 1u ? 0 : visible - h;
        mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) mx = fmaxf(mx, j < v ? s[j] : -INFINITY);
      }
      mt = fmaxf(mt, mx);
    }
    const uint32_t bar = wt.bar(B_REF) + (lane() * 4 + (r() >> 5)) * 16;
    float was = -INFINITY;  // the lane's reference
    if (!first) {
      if (!wt.wait_warp_at(bar + 8 * (half() ^ 1), ((nt - 1) >> 1) & 1)) return false;
      was = ldsf(ref_at ^ 512);
    }
    const bool moves = (mt - was) * a.scale_log2 > 8.0f;
    const float mn = moves ? mt : was;
    stsf(ref_at, mn);
    wt.arrive_warp_at(bar + 8 * half());
    if (__any_sync(0xffffffffu, moves) && !first) {
      const float f = moves ? ptx::ex2_ftz((was - mn) * a.scale_log2) : 1.0f;
      // O is still when the last tile's PV is done (the next tile's S is made after it) and
      // this one's P is not there
      if (!(last ? wt.wait_warp(B_PVLAST + lane(), (phases >> P_LAST) & 1)
                 : wt.wait_warp_at(wt.bar(B_SFULL) + 16 * lane() + 8 * (half() ^ 1), ((nt + 1) >> 1) & 1)))
        return false;
      tc5::fence_after();
      const uint32_t oa = tmem + C::O0 + lane() * C::OSTEP;
#pragma unroll 1
      for (int i = 0; i < D; i += 16) {
        uint32_t o[16];
        tc5::ld16(oa + i, o);
        tc5::wait_ld();
        tc5::pin16(o);
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tc5::st16(oa + i, o);
      }
    }
    if (m != mn) l *= ptx::ex2_ftz((m - mn) * a.scale_log2);  // (m below mn)
    m = mn;
    const float off = m == -INFINITY ? 0.0f : -m * a.scale_log2;
    const uint64_t c2 = pack_f32x2(a.scale_log2, a.scale_log2), off2 = pack_f32x2(off, off);
    uint64_t sum = pack_f32x2(l, 0.0f);
    float s[2][16];
    tc5::ld16(s_tm, reinterpret_cast<uint32_t*>(s[0]));
#pragma unroll
    for (int h = 0; h < C::TN; h += 16) {
      float (&now)[16] = s[(h / 16) & 1];
      uint32_t p[8];
      tc5::wait_ld();
      tc5::pin16(reinterpret_cast<uint32_t*>(now));
      if (h + 16 < C::TN) tc5::ld16(s_tm + h + 16, reinterpret_cast<uint32_t*>(s[(h / 16 + 1) & 1]));
      weights(now, p, c2, off2, sum, masked, (bad >> (h / 32)) & 1u ? 0 : visible - h);
      // P's columns lie below those of the scores that are still to be read
      tc5::st8(s_tm + h / 2, p);
    }
    l = __uint_as_float(lo_bits(sum)) + __uint_as_float(hi_bits(sum));
    tc5::wait_st();
    return true;
  }

  // What the notes say of the group's columns of the row: it sees `lim` tokens; written over the
  // thread's own earlier stores, to the output (whole) or to the piece's O in `slot`.
  __device__ __forceinline__ void notes(int lim, bool whole, int64_t at, int slot, int row) const {
    const uint32_t pn = smem + C::OFF_POISON;
#pragma unroll 1
    for (int c = half() * C::HD; c < (half() + 1) * C::HD; ++c) {
      const bool up = (int)lds(pn + 4 * c) < lim, down = (int)lds(pn + 4 * (D + c)) < lim,
                 nan = (int)lds(pn + 4 * (2 * D + c)) < lim;
      if (!(up || down || nan)) continue;
      const float v = nan || (up && down) ? NAN : up ? INFINITY : -INFINITY;
      if (!whole) {
        float4* dst = a.o_part + ((int64_t)slot * (D / 4) + c / 4) * C::QB + row;
        __stcg(reinterpret_cast<float*>(dst) + (c & 3), v);
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

  // The group's tiles of a segment: the reference m of the last of them and l.
  __device__ __forceinline__ bool tiles(float& m, float& l, bool& any) {
    m = -INFINITY;
    l = 0.0f;
    int t, end, npt, step, row;
    bool live, mine;
    {
      const Ref k = ref();
      row = block_row(k);
      live = (row & ~31) < block_rows(k);
      mine = row < block_rows(k);
      step = k.alt() ? 2 : 1;
      t = k.lo() + (k.alt() ? lane() : 0);
      end = k.hi();
      npt = k.npt();
    }
    any = t < end;
    const int t0 = t;
    const uint32_t nt0 = nt;
    if ((nt & 1) != (uint32_t)half()) t += step, ++nt;
    int visible = 0, left = 0;  // tokens that the row sees from t on; tiles to go with it
#pragma unroll 1
    for (; t < end; t += 2 * step, nt += 2) {
      if (--left < 0) {
        // the first packed tile, then the first fp16 one
        const Ref k = ref();
        const bool f16 = t >= npt;
        left = ((f16 ? end : min(npt, end)) - t - 1) / (2 * step);
        visible = 1 << 30;  // rows that are not there need no mask
        if (mine) {
          const int ns = k.ns(), npk = k.npk();
          const int lim = seen_of(a, k.n(), ns + npk + k.nres(), token_of(a, k.qb() * C::QB + row));
          visible = (f16 ? seen_f16(ns, npk, lim) + npt * C::TN : seen_packed(ns, npk, lim)) - t * C::TN;
        }
      } else if (mine) {
        visible -= 2 * step * C::TN;
      }
      uint32_t bad = 0;
      if (a.rm.paged && t < npt) {
        const Ref k = ref();
        const int j = t * (C::TN / kPage) + (r() & 1);
        bool out = false;
        if ((r() & 31) < C::TN / kPage && j * kPage < k.npk()) {
          const int pg = a.rm.page_of(k.b(), j);
          out = pg < 0 || pg >= a.rm.npages;
        }
        bad = __ballot_sync(0xffffffffu, out);
      }
      const uint32_t bar = wt.bar(B_SFULL) + 16 * lane() + 8 * half();
      if (!wt.wait_warp_at(bar, (nt >> 1) & 1)) return false;
      tc5::fence_after();
      if (live) {
        if (!tile(visible, bad, t == t0, t + step >= end, m, l)) return false;
      } else {
        wt.arrive_warp_at(wt.bar(B_REF) + (lane() * 4 + (r() >> 5)) * 16 + 8 * half());
      }
      tc5::fence_before();
      wt.arrive_warp_at(bar + 8 * (B_PREADY - B_SFULL));
    }
    const int n = any ? (end - t0 + step - 1) / step : 0;
    nt = nt0 + n;
    if (n > 1) phases ^= 1u << P_LAST;
    return true;
  }

  __device__ __forceinline__ bool run(int block) {
    if (!wait_seg()) return false;
    if (ref().b() < 0) return true;
    load_q();
    while (true) {
      float m, l;
      bool any;
      if (!tiles(m, l, any)) return false;
      if (any && !wait(B_ODONE + lane(), P_O)) return false;
      tc5::fence_after();

      const Ref k = ref();
      const bool alt = k.alt();
      const int row = block_row(k), rows = block_rows(k);
      const bool live = (row & ~31) < rows;
      // m and l of both groups; l through the first KiB of the lane's Q, which no MMA reads
      // once both lanes are done.  The lane's reference is the later one, the larger.
      const uint32_t xl = smem + C::OFF_Q + lane() * C::QBYTES + r() * 4;
      if (!pair_sync()) return false;
      stsf(ref_at, m);
      stsf(xl + half() * 512, l);
      if (!pair_sync()) return false;
      {
        const float mo = ldsf(ref_at ^ 512), lo = ldsf(xl + (half() ^ 1) * 512), mm = fmaxf(m, mo);
        const float fa = m == mm ? 1.0f : ptx::ex2_ftz((m - mm) * a.scale_log2);
        const float fb = mo == mm ? 1.0f : ptx::ex2_ftz((mo - mm) * a.scale_log2);
        l = l * fa + lo * fb;
        m = mm;
      }
      const bool noted = wt.word(W_PFLAG) != 0;
      const bool whole = k.lo() == 0 && k.hi() == k.nt();
      const int slot = 2 * block + (k.lo() == 0);
      float inv = 0.0f;
      int64_t at = 0;
      // With alternating lanes, lane 1's accumulator of a whole unit goes through shared
      // memory to lane 0, 16 columns of each half at a time, with its rows' m and l.
      const bool pass = alt && whole && k.hi() - k.lo() > 1;
      float f0 = 1.0f, f1 = 0.0f;
      if (pass) {
        const uint32_t x1 = smem + C::OFF_Q + (C::LANES - 1) * C::QBYTES + 1024 + r() * 4;
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
          float4* dst = a.o_part + ((int64_t)slot * (D / 4) + col / 4) * C::QB + prow;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            __stcg(dst + j * C::QB, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        }
        __syncwarp();
      }
      if (noted) {
        if (mine) {
          const int lim = seen_of(a, k.n(), k.ns() + k.npk() + k.nres(), token_of(a, k.qb() * C::QB + row));
          notes(lim, whole, at, slot, prow);
        }
        // the notes have been read: clean them
        if (!pair_sync()) return false;
        for (int i = tid; i < 3 * D; i += C::SMW * 32) sts(smem + C::OFF_POISON + 4 * i, 0x7fffffff);
        if (tid == 0) wt.set_word(W_PFLAG, 0);
        if (!pair_sync()) return false;
      }
      tc5::fence_before();
      __threadfence_block();
      __syncwarp();
      if ((r() & 31) == 0)
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(wt.bars + 4 * W_EPI) : "memory");

      if (!whole && k.lo() == 0 && tid < 4) a.heads[block * 4 + tid] = lds_v4(k.at + 16 * tid);
      wt.arrive_warp(B_SEGEMPTY + at_seg % kSegs);
      ++at_seg;
      if (!wait_seg()) return false;
      if (ref().b() < 0) return true;
      // Q goes where l and the accumulator passed: after all have read them
      if (!pair_sync()) return false;
      load_q();
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
  if (smem & 1023u) {  // the swizzles count on it (a block without static shared memory has it)
    set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
    return;
  }
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(base + C::OFF_BAR);
  volatile int64_t* wide = reinterpret_cast<volatile int64_t*>(base + C::OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lid = tid & 31;
  if (tid == 0) a.heads[blockIdx.x * 4].x = -1;  // (a later head is this thread's store too)
  asm volatile("griddepcontrol.launch_dependents;");

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
  // at least four units of cost (two tiles of each lane) to a block
  const int64_t G = max((int64_t)1, min((int64_t)gridDim.x, W / 4));
  if (W == 0 || (int64_t)blockIdx.x >= G) return;
  const int64_t x0 = (int64_t)blockIdx.x * W / G, x1 = ((int64_t)blockIdx.x + 1) * W / G;
  before += scan - mine;
  if (before <= x0 && x0 < before + mine) {
    for (int b = b_lo; b < b_hi; ++b) {
      const int64_t c = Walk<D, BITS>::seq_cost(a, b);
      if (x0 < before + c) {
        words[W_STARTB] = b;
        wide[W_BASE / 2] = before;
        break;
      }
      before += c;
    }
  }
  if (tid == 0) {
    auto init = [&](int i, uint32_t n) { ptx::mbar_init(smem + C::OFF_BAR + 8 * i, n); };
    for (int i = 0; i < 2; ++i) {
      init(B_QFULL + i, 8);
      init(B_ODONE + i, 1);
      init(B_PVLAST + i, 1);
      init(B_DRAIN + i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      init(B_SFULL + i, 1 + (a.fault && blockIdx.x == 0 ? 1 : 0));
      init(B_PREADY + i, 4);
      init(B_KFULL + i, 2 * C::TPR);
      init(B_VFULL + i, 2 * C::TPR);
    }
    for (int i = 0; i < 8; ++i) {
      init(B_KEMPTY + i, 1);
      init(B_VEMPTY + i, 1);
    }
    for (int i = 0; i < 16; ++i) init(B_REF + i, 1);
    for (int i = 0; i < kSegs; ++i) {
      init(B_SEGFULL + i, 1);
      init(B_SEGEMPTY + i, C::SMW + 8 + C::LANES);
    }
    init(B_PAIR, C::SMW);
    words[W_ABORT] = 0;
    words[W_PFLAG] = words[W_EPI] = 0;
    ptx::fence_mbar_init();
  }
  int* poison = reinterpret_cast<int*>(base + C::OFF_POISON);
  for (int i = tid; i < 3 * D; i += kThreads) poison[i] = 0x7fffffff;
  __syncthreads();
  if (warp == 0) {
    // the query block that holds x0, 32 at a time
    const int b = words[W_STARTB];
    const Run run = run_of(a.cu, b, a.total, a.max_len);
    const SeqLens s = seq_lens_of(a.sink_len, a.packed_len, a.res_len, a.res_head, b, a.Ns, a.cap, a.Nr);
    const int nq = Walk<D, BITS>::blocks(a, run);
    int64_t at = wide[W_BASE / 2];
    for (int q0 = 0; q0 < nq; q0 += 32) {
      int64_t c = 0;
      if (q0 + lid < nq) {
        int npt, nt, w;
        Walk<D, BITS>::tiles(a, run, s, q0 + lid, npt, nt, w);
        c = (int64_t)nt * w * a.Hkv;
      }
      int64_t sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lid >= o) sum += v;
      }
      const bool here = at + sum - c <= x0 && x0 < at + sum;
      if (here) {
        words[W_STARTQ] = q0 + lid;
        wide[W_BASE / 2 + 1] = at + sum - c;
      }
      if (__any_sync(0xffffffffu, here)) break;
      at += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  if (warp == 24) tc5::alloc(smem + C::OFF_BAR + 4 * W_TMEM, 512);
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = words[W_TMEM];
  const Waits wt = {a, smem + C::OFF_BAR};
  Seg* ring = reinterpret_cast<Seg*>(base + C::OFF_SEG);
  const int sb = words[W_STARTB], sq = words[W_STARTQ];
  const int64_t sbase = wide[W_BASE / 2 + 1];

  if (warp < 16) {
    tc5::regs_inc<80>();
    if (warp < C::SMW) {
      const uint32_t tm = tmem + ((uint32_t)(warp & 3) << 21);
      Soft<D, BITS> soft = {a, wt, smem, tm, 0, (uint32_t)tid,
                            tm + C::S0 + (tid >> 7) * C::TN,
                            smem + C::OFF_MAX + tid * 4, 0, 0};
      soft.run(blockIdx.x);
    }
  } else if (warp < 24) {
    tc5::regs_dec<64>();
    const int w = (warp - 16) / 4;
    Deq<D, BITS> deq = {a, wt, smem, poison, ring, w, (tid - 512) % kDeqThreads, 0};
    deq.run();
  } else {
    tc5::regs_dec<56>();
    if (lid == 0 && warp - 24 < C::LANES) mma_role<D, BITS>(a, wt, smem, tmem, ring, warp - 24);
    if (tid == 26 * 32) walk_role<D, BITS>(a, wt, ring, sb, sq, sbase, x0, x1, W, G);
    __syncwarp();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (warp == 24) tc5::dealloc(tmem, 512);
}

// The pieces of the units that were cut, in the order of the tiles.  A block looks at the
// unit that block x of the other kernel began; a warp has 16 columns of a row: eight
// lanes' worth of pieces at a time, four columns to a lane.
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 8;

template <int D, int BITS>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const ChunkAttnArgs a) {
  constexpr int QB = chunk_rows(D);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  union {
    int4 v[4];
    Seg s;
  } u;
  u.v[0] = __ldcg(a.heads + blockIdx.x * 4);
  if (u.v[0].x < 0) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) u.v[i] = __ldcg(a.heads + blockIdx.x * 4 + i);
  const Seg& k = u.s;
  const int rows = min(k.n * a.gq - k.qb * QB, QB), lane = threadIdx.x & 31, e = lane & 3;
  const int subs = (k.last_b - k.first_b + 1) << (k.alt ? 1 : 0);  // pieces, or both lanes' of each
  const int warps = kJoinBlocks * kJoinThreads / 32;
  for (int it = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); it < rows * (D / 16); it += warps) {
    const int row = it / (D / 16), cg = it % (D / 16);
    auto ml_at = [&](int s, int64_t& slot, int& prow) {
      const int p = k.first_b + (k.alt ? s >> 1 : s);
      slot = 2 * (int64_t)p + (p == k.first_b);
      prow = row + (k.alt ? (s & 1) * 128 : 0);
      return __ldcg(a.ml_part + slot * QB + prow);
    };
    int64_t slot;
    int prow;
    float m = -INFINITY;
    for (int s = lane >> 2; s < subs; s += 8) m = fmaxf(m, ml_at(s, slot, prow).x);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = lane >> 2; s < subs; s += 8) {
      const float2 ml = ml_at(s, slot, prow);
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // saw nothing (and may have written nothing)
      const float f = ml.x == -INFINITY ? ml.y : ptx::ex2_ftz((ml.x - m) * a.scale_log2);
      const float4 v = __ldcg(a.o_part + (slot * (D / 4) + cg * 4 + e) * QB + prow);
      l += ml.y * f;
      o.x += v.x * f;
      o.y += v.y * f;
      o.z += v.z * f;
      o.w += v.w * f;
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, x);
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    if (lane >= 4) continue;
    if (l == 0.0f) set_error(a.err_word, KVQ_ERRBIT_EMPTY);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int R = k.qb * QB + row;
    const int tok = token_of(a, R);
    const int64_t at = ((int64_t)(k.c0 + tok) * a.Hq + k.h * a.gq + (R - tok * a.gq)) * D + cg * 16;
    const float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = 4 * e + j;  // the element that is stored at this column
      const int el = BITS == 2 ? (c & 1) * 8 + (c >> 3) * 4 + ((c & 7) >> 1) : (c & 8) + ((c & 7) >> 1) + 4 * (c & 1);
      if (a.out_f32)
        static_cast<float*>(a.out)[at + el] = y[j];
      else
        static_cast<__half*>(a.out)[at + el] = __float2half_rn(y[j]);
    }
  }
}

template <int D, int BITS>
cudaError_t launch(const ChunkAttnArgs& a, int grid, cudaStream_t st) {
  static_assert(Cfg<D, BITS>::SMEM <= 227 * 1024, "shared memory of a block");
  auto kernel = chunk_attn_kernel<D, BITS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, BITS>::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, Cfg<D, BITS>::SMEM, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, kJoinBlocks);
  cfg.blockDim = kJoinThreads;
  cfg.stream = st;
  cudaLaunchAttribute at[1];  // its blocks may come as the others leave; they wait for all of them
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, BITS>, a);
}

template <int D>
cudaError_t launch_bits(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st) {
  if (bits == 4) return launch<D, 4>(a, grid, st);
  if (bits == 3) return launch<D, 3>(a, grid, st);
  return launch<D, 2>(a, grid, st);
}

}  // namespace chunk
}  // namespace kvq
