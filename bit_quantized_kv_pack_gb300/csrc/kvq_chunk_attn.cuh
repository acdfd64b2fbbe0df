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
// (operands of the MMA), the weights P to fp16 once; scores, m, l and O are fp32.
//
// A block (one per SM, persistent) has 16 warps:
//   0-7   softmax: one thread per query row, S from TMEM, P back to TMEM (it takes S's
//         place and is the A operand of the second MMA), the epilogue.  Two groups of
//         four warps, one for each of the block's two accumulators (lanes 0 and 1).
//   8-11  dequantize: codes come by cp.async into a ring that is private to each thread
//         (no barrier), become fp16 in registers and go to shared memory in the MMA's
//         128-byte swizzle, K as the K-major and V as the MN-major B operand.
//   12    issues the MMAs.
// A unit of work is (sequence, block of query rows, KV head).  With more than 128 rows in
// the block the two lanes are its two halves and share each tile; with fewer they take
// alternate tiles of the same rows and are joined at the end, so that the softmax of one
// tile runs under the MMAs of the next either way.  head_dim 256 has room for one lane.
//
// Balance.  All units' tiles lie in one line, and each of the G blocks takes an equal
// piece of it (the line is cut by cost, so a unit may be cut, into two pieces or, with
// few units, into many).  Pieces of a unit write (O, m, l) and the last to arrive joins
// them in the order of the tiles: results do not depend on timing.
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
  uint32_t* tickets;  // [G], zero between calls
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

constexpr int kThreads = 512;
constexpr int kDeqThreads = 128;

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
  static constexpr int GPT = TN * G / kDeqThreads;  // groups per dequantizing thread and half tile
  static constexpr int CB = 4 * BITS;               // code bytes of a group
  static constexpr int RAWB = kDeqThreads * GPT * (CB + 4);
  static constexpr int RAWN = D == 256 ? 2 : D == 128 ? 3 : 6;
  static constexpr int SMT = 128 * LANES;           // softmax threads
  // TMEM columns
  static constexpr int S0 = 0;
  static constexpr int O0 = 256;
  static constexpr int OSTEP = D < 32 ? 32 : D;
  // shared memory
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + LANES * QBYTES;
  static constexpr int OFF_V = OFF_K + ST * KBYTES;
  static constexpr int OFF_RAW = OFF_V + ST * KBYTES;
  // where lane 1's accumulator passes to lane 0: 32 columns, m and l of 128 rows.  Lane 1's
  // Q is free then, and large enough from head_dim 128 on
  static constexpr int STAGE = 34 * 128 * 4;
  static constexpr int OFF_STAGE = D >= 128 ? OFF_Q + (LANES - 1) * QBYTES : OFF_RAW + RAWN * RAWB;
  static constexpr int OFF_POISON = OFF_RAW + RAWN * RAWB + (D >= 128 ? 0 : STAGE);  // int [2][3][D]
  static constexpr int OFF_BAR = OFF_POISON + 2 * 3 * D * 4;
  static constexpr int OFF_SEG = OFF_BAR + 512;                 // Seg [kSegs]
  static constexpr int SMEM = OFF_SEG + 512 + 1024;             // slack to align the base
};

// A segment: the block's tiles [lo, hi) of the unit (sequence b, KV head h, query block
// qb).  One warp works the segments out, the others read them from a ring.
constexpr int kSegs = 8;
struct alignas(16) Seg {
  int b, h, qb, lo;
  int hi, npt, nt, alt;     // packed tiles and all tiles of the unit; alt: the lanes take alternate tiles
  int c0, n, ns, npk;       // the run, and the sequence's lengths
  int nres, head, first_b, last_b;  // blocks that hold the unit's first and last tile; b < 0: the end
};

// Barriers (8 bytes each from OFF_BAR) and words behind them.
enum { B_QFULL = 0, B_SFULL = 2, B_PREADY = 4, B_ODONE = 6, B_EPI = 8, B_PAIR = 10, B_DRAIN = 11,
       B_KFULL = 12, B_KEMPTY = 16, B_VFULL = 20, B_VEMPTY = 24, B_SEGFULL = 28, B_SEGEMPTY = 36, B_COUNT = 44 };
enum { W_TMEM = 88, W_ABORT = 89, W_PFLAG = 90 /* [2] */, W_TICKET = 92, W_STARTB = 93, W_STARTQ = 94,
       W_BASE = 96 /* int64 [2] */ };

// Bounded waits: all give up when one has.
__device__ __forceinline__ bool wait_on(uint32_t b, uint32_t parity, volatile uint32_t* words, uint32_t* err_word,
                                     uint32_t limit_us) {
  const uint64_t t0 = ptx::global_timer_ns();
  for (uint32_t k = 1;; ++k) {
    if (ptx::mbar_try_wait(b, parity)) return true;
    if ((k & 63u) == 0) {
      if (words[W_ABORT]) return false;
      if (ptx::global_timer_ns() - t0 > (uint64_t)limit_us * 1000u) {
        words[W_ABORT] = 1;
        set_error(err_word, KVQ_ERRBIT_TIMEOUT);
        return false;
      }
    }
  }
}
struct Waits {
  uint32_t bars;             // shared address of the barriers
  volatile uint32_t* words;  // the same as words
  uint32_t* err_word;
  uint32_t limit_us;

  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    return ptx::mbar_try_wait(bar(i), parity) || wait_on(bar(i), parity, words, err_word, limit_us);
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

// The four 8-code words of a group in raw code memory.
template <int BITS>
__device__ __forceinline__ void code_words(uint32_t addr, uint32_t (&x)[4]) {
  if (BITS == 4) {
    const uint4 v = ld_shared_v4(addr);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if (BITS == 2) {
    uint32_t w0, w1;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(addr) : "memory");
    x[0] = w0, x[1] = w0 >> 8, x[2] = w1, x[3] = w1 >> 8;
  } else {
    uint32_t w[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i) : "memory");
    const uint32_t v[4] = {w[0], __funnelshift_r(w[0], w[1], 24), __funnelshift_r(w[1], w[2], 16), w[2] >> 8};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (v[i] & 0xfffu) | ((v[i] & 0xfff000u) << 4);
  }
}

// What the dequantizing warps share.
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

  // Values of the fp16 format that are not finite take no part in the MMA: a weight of
  // zero would make them NaN in rows that do not see the token.  The first token of
  // the segment with +inf, -inf or NaN in a column is noted, and the epilogue gives
  // the rows that see it what the sum would be.  (Rare: one thread per element.)
  __device__ __forceinline__ bool note(int col, int token, uint32_t h) {
    // the notes of the segment before last are read before this one's are made
    if (seg >= 2 && !wt.wait(B_EPI + (seg & 1), ((seg >> 1) - 1) & 1)) return false;
    const int kind = (h & 0x3ffu) ? 2 : (h & 0x8000u) ? 1 : 0;
    atomicMin(poison + ((seg & 1) * 3 + kind) * D + col, token);
    wt.words[W_PFLAG + (seg & 1)] = 1;
    return true;
  }

  // The cursor of the copies: a half tile of a segment.
  struct Cursor {
    SegReader at;
    int tile = -1, w = 0, hi = 0, npt = 0, npk = 0, b = 0;
    int64_t row0 = 0;  // contiguous: row of the head's token 0; paged: h * 32
  };

  // Raw copies of a half tile (keys, then values) into ring slot `slot`; rows that are
  // not there become zero codes with zero params, which stand for zeros.  A head's groups
  // lie one behind the other, so group gi of the tile is gi groups from its first.
  __device__ __forceinline__ void fetch(const Cursor& c, int slot) {
    const uint32_t dc = smem + C::OFF_RAW + slot * C::RAWB + dt * C::CB;
    const uint32_t dp = smem + C::OFF_RAW + slot * C::RAWB + kDeqThreads * C::GPT * C::CB + dt * 4;
    const uint8_t* codes = a.codes[c.w];
    const uint32_t* params = a.params[c.w];
    const int left = c.npk - c.tile * C::TN;  // rows of the tile that there are
    int64_t at = (c.row0 + c.tile * C::TN) * C::G + dt;
#pragma unroll
    for (int i = 0; i < C::GPT; ++i) {
      const int r = (i * kDeqThreads + dt) / C::G;
      bool there = r < left;
      int64_t from = at + i * kDeqThreads;
      if (a.rm.paged && there) {
        const int p = c.tile * C::TN + r;
        const int pg = a.rm.page_of(c.b, p / kPage);
        there = pg >= 0 && pg < a.rm.npages;
        if (!there) set_error(a.err_word, KVQ_ERRBIT_BADPAGE);
        from = ((int64_t)pg * a.Hkv * kPage + c.row0 + p % kPage) * C::G + dt % C::G;
      }
      const uint32_t d0 = dc + i * kDeqThreads * C::CB, d1 = dp + i * kDeqThreads * 4;
      if (there) {
        const uint8_t* src = codes + from * C::CB;
        if (BITS == 4) {
          ptx::cp_async_16(d0, src, 16);
        } else if (BITS == 2) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d0), "l"(src) : "memory");
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d0 + 4 * j), "l"(src + 4 * j)
                         : "memory");
        }
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d1), "l"(params + from) : "memory");
      } else {
#pragma unroll
        for (int j = 0; j < C::CB / 4; ++j)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(d0 + 4 * j), "r"(0) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(d1), "r"(0) : "memory");
      }
    }
  }

  // The pieces of one group with a value that is not finite in fp16, at `at` + pieces
  // c0 ^ 0..3 (x: their code words, in the order of the pieces; col: the group's first
  // column, xr: the order).
  __device__ __forceinline__ bool rare_group(const uint32_t* x, uint32_t prm, int w, uint32_t at, uint32_t c0, int col,
                                          int xr, int token) {
    const uint32_t s2 = ptx::prmt(prm, prm, 0x1010), m2 = ptx::prmt(prm, prm, 0x3232);
    const bool finite = !f16_nonfinite(prm) && !f16_nonfinite(prm >> 16);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t y[4];
      codes_f16<BITS>(x[c], y);
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t v = ptx::hfma2_u32(y[j], s2, m2);
#pragma unroll 1
        for (int sh = 0; sh < 32; sh += 16) {
          const uint32_t hv = (v >> sh) & 0xffffu;
          if (!f16_nonfinite(hv)) continue;
          uint32_t to = hv;
          if (finite) {
            to = (hv & 0x8000u) | 0x7bffu;  // past fp16's largest value by the scale's rounding
          } else if (w == 1) {
            if (!note(col + (c ^ xr) * 8 + 2 * j + sh / 16, token, hv)) return false;
            to = 0;
          }
          v = (v & ~(0xffffu << sh)) | (to << sh);
        }
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + ((c0 ^ c) << 4) + 4 * j), "r"(v) : "memory");
      }
    }
    return true;
  }

  // A fetched half tile as fp16 at `dst`.
  __device__ __forceinline__ bool packed_tile(const Seg& k, int tile, int w, int slot, uint32_t dst) {
    const uint32_t raw = smem + C::OFF_RAW + slot * C::RAWB;
    constexpr uint32_t kQmax2 = BITS == 4 ? 0x4b804b80u : BITS == 3 ? 0x47004700u : 0x42004200u;  // 15, 7, 3
#pragma unroll 2
    for (int i = 0; i < C::GPT; ++i) {
      const int gi = i * kDeqThreads + dt;
      const int r = gi / C::G, g = gi % C::G;
      const int panel = g / 2;
      uint32_t x[4], prm;
      code_words<BITS>(raw + gi * C::CB, x);
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(prm) : "r"(raw + kDeqThreads * C::GPT * C::CB + gi * 4) : "memory");
      const uint32_t s2 = ptx::prmt(prm, prm, 0x1010), m2 = ptx::prmt(prm, prm, 0x3232);
      // the lanes of a store phase take different pieces first, so that they differ in
      // banks: two panels of a row lie a multiple of 128 bytes apart
      const int xr = D == 256 ? panel : D == 128 ? 2 * panel : 0;
      if (D >= 128 && (xr & 2)) {
        const uint32_t t0 = x[0], t1 = x[1];
        x[0] = x[2], x[1] = x[3], x[2] = t0, x[3] = t1;
      }
      if (D == 256 && (xr & 1)) {
        const uint32_t t0 = x[0], t2 = x[2];
        x[0] = x[1], x[2] = x[3], x[1] = t0, x[3] = t2;
      }
      const uint32_t at = dst + panel * C::KP + r * C::RB;
      const uint32_t c0 = C::RB == 128 ? (((g & 1) * 4) ^ xr ^ (r & 7)) : ((r >> 1) & 3);
      // the group's largest value; only where it is not finite can any value be so
      if (f16_nonfinite(ptx::hfma2_u32(kQmax2, s2, m2))) {
        const uint32_t xs[4] = {x[0], x[1], x[2], x[3]};
        if (!rare_group(xs, prm, w, at, c0, panel * 64 + (g & 1) * 32, xr, k.ns + tile * C::TN + r)) return false;
        continue;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t f[4], y[4];
        codes_f16<BITS>(x[c], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = ptx::hfma2_u32(f[j], s2, m2);
        st_shared_v4(at + ((c0 ^ c) << 4), make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
    return true;
  }

  // The 16 stored elements at p0 and p1, of columns col ..: what is not finite becomes
  // zero and is noted.
  __device__ __forceinline__ bool rare_pieces(uint32_t p0, uint32_t p1, int col, int token) {
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      const uint32_t at = (j < 8 ? p0 : p1) + 2 * (j & 7);
      unsigned short hv;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hv) : "r"(at) : "memory");
      if (!f16_nonfinite(hv)) continue;
      if (!note(col + j, token, hv)) return false;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)0) : "memory");
    }
    return true;
  }

  __device__ __forceinline__ int ring_slot(int j) const { return j < a.Nr ? j : j - a.Nr; }  // j < 2 Nr

  // A half tile of fp16 tokens (sink, then window): rows f0 .. of their line.
  __device__ __forceinline__ bool f16_tile(const Seg& k, int f0, int w, uint32_t dst) {
    const int64_t bh = (int64_t)k.b * a.Hkv + k.h;
    const int n = k.ns + k.nres;
#pragma unroll 1
    for (int i = 0; i < C::GPT; ++i) {
      const int gi = i * kDeqThreads + dt;
      const int r = gi / C::G, g = gi % C::G, f = f0 + r;
      const __half* src = a.q;  // (not read)
      if (f < k.ns)
        src = a.sink[w] + (bh * a.Ns + f) * D + g * 32;
      else if (f < n)
        src = a.res[w] + (bh * a.Nr + ring_slot(k.head + f - k.ns)) * D + g * 32;
      const uint32_t at = dst + (g / 2) * C::KP;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        ptx::cp_async_16(at + swizzled<C::RB>(r, (g & 1) * 4 + c), src + (f < n ? c * 8 : 0), f < n ? 16 : 0);
    }
    ptx::cp_async_wait_all();
#pragma unroll 1
    for (int i = 0; i < C::GPT; ++i) {
      const int gi = i * kDeqThreads + dt;
      const int r = gi / C::G, g = gi % C::G, f = f0 + r;
      const uint32_t at = dst + (g / 2) * C::KP;
#pragma unroll
      for (int c = 0; c < 4; c += 2) {  // (16 elements)
        const uint32_t p0 = at + swizzled<C::RB>(r, (g & 1) * 4 + c), p1 = at + swizzled<C::RB>(r, (g & 1) * 4 + c + 1);
        uint4 u[2] = {ld_shared_v4(p0), ld_shared_v4(p1)};
        to_storage<BITS>(u[0], u[1]);
        st_shared_v4(p0, u[0]);
        st_shared_v4(p1, u[1]);
        if (w == 1) {
          const uint32_t* y = reinterpret_cast<const uint32_t*>(u);
          bool bad = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) bad |= f16_nonfinite(y[j]) || f16_nonfinite(y[j] >> 16);
          if (bad && !rare_pieces(p0, p1, (g / 2) * 64 + (g & 1) * 32 + c * 8, f < k.ns ? f : f + k.npk))
            return false;
        }
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
    uint32_t kv = 0;  // tiles so far
    int slot = 0;
    // RAWN - 1 half tiles ahead: a free slot is filled before the oldest is taken
#pragma unroll 1
    for (int i = 0; i < C::RAWN - 1; ++i) fetch_next(i);
    for (; ok; ++k.i, ++seg) {
      ok = ok && __all_sync(0xffffffffu, k.wait(wt));
      if (!ok) break;
      const Seg& s = k.get(ring);
      if (s.b < 0) break;
      const int lo = s.lo, hi = s.hi, npt = s.npt;
      for (int h = 2 * lo; h < 2 * hi; ++h) {
        fetch_next(slot == 0 ? C::RAWN - 1 : slot - 1);
        const int t = h >> 1, w = h & 1;
        const int stage = kv % C::ST;
        const uint32_t dst = smem + (w ? C::OFF_V : C::OFF_K) + stage * C::KBYTES;
        ok = ok && wt.wait_warp((w ? B_VEMPTY : B_KEMPTY) + stage, ((kv / C::ST) & 1) ^ 1);
        if (!ok) break;
        if (t < npt) {
          asm volatile("cp.async.wait_group %0;" ::"n"(C::RAWN - 1) : "memory");
          ok = packed_tile(s, t, w, slot, dst);
        } else {
          ok = f16_tile(s, (t - npt) * C::TN, w, dst);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::fence_proxy_async_shared();
        wt.arrive_warp((w ? B_VFULL : B_KFULL) + stage);
        if (++slot == C::RAWN) slot = 0;
        kv += w;
      }
      wt.arrive_warp(B_SEGEMPTY + k.i % kSegs);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// ---------------------------------------------------------------------- MMA ---

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
  for (;; ++k.i) {
    if (!k.wait(wt) || k.get(ring).b < 0) break;
    const bool alt = k.get(ring).alt;
    const int n = k.get(ring).hi - k.get(ring).lo;
    ptx::mbar_arrive(wt.bar(B_SEGEMPTY + k.i % kSegs));
    const int U = C::LANES == 2 && !alt ? 2 * n : n;
    ok = wt.wait(B_QFULL, qn[0]++ & 1);
    if (ok && C::LANES == 2 && !alt) ok = wt.wait(B_QFULL + 1, qn[1]++ & 1);
    if (!ok) break;
    auto tile = [&](int u) { return C::LANES == 2 && !alt ? u >> 1 : u; };
    auto lane_of = [&](int u) { return C::LANES == 2 ? u & 1 : 0; };
    // the step's tile is read by no later step
    auto releases = [&](int u) { return C::LANES == 1 || alt || (u & 1); };
    auto qk = [&](int u) -> bool {
      const uint32_t t = kv + tile(u);
      const int stage = t % C::ST, lane = lane_of(u);
      if ((C::LANES == 1 || alt || lane == 0) && !wt.wait(B_KFULL + stage, (t / C::ST) & 1)) return false;
      tc5::fence_after();
      const uint32_t q = smem + C::OFF_Q + (alt ? 0 : lane * C::QBYTES);
      const uint32_t kb = smem + C::OFF_K + stage * C::KBYTES;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int panel = j * 16 / C::PW, in = (j * 16 % C::PW) * 2;
        tc5::mma_ss(tmem + C::S0 + lane * C::TN, tc5::smem_desc(q + panel * C::QP + in, 16, 8 * C::RB, C::SWZ),
                    tc5::smem_desc(kb + panel * C::KP + in, 16, 8 * C::RB, C::SWZ), kIdescQK, j > 0);
      }
      tc5::commit(wt.bar(B_SFULL + lane));
      if (releases(u)) tc5::commit(wt.bar(B_KEMPTY + stage));
      return true;
    };
    for (int u = 0; ok && u < C::LANES && u < U; ++u) ok = qk(u);
    for (int u = 0; ok && u < U; ++u) {
      const uint32_t t = kv + tile(u);
      const int stage = t % C::ST, lane = lane_of(u);
      ok = wt.wait(B_PREADY + lane, pn[lane]++ & 1);
      if (ok && (C::LANES == 1 || alt || lane == 0)) ok = wt.wait(B_VFULL + stage, (t / C::ST) & 1);
      if (!ok) break;
      tc5::fence_after();
      const uint32_t vb = smem + C::OFF_V + stage * C::KBYTES;
      const bool acc = u >= C::LANES;  // the lane's first tile of the segment starts O
#pragma unroll
      for (int j = 0; j < C::TN / 16; ++j)
        tc5::mma_ts(tmem + C::O0 + lane * C::OSTEP, tmem + C::S0 + lane * C::TN + j * 8,
                    tc5::smem_desc(vb + j * 16 * C::RB, C::KP, 8 * C::RB, C::SWZ), kIdescPV, acc || j > 0);
      if (releases(u)) tc5::commit(wt.bar(B_VEMPTY + stage));
      if (u + C::LANES < U)
        ok = qk(u + C::LANES);  // after PV(u) in the tensor cores' order: S may take P's place
      else
        tc5::commit(wt.bar(B_ODONE + lane));
    }
    if (!ok) break;
    kv += n;
  }
  // nothing of this thread's is in flight when TMEM is freed
  tc5::commit(wt.bar(B_DRAIN));
  wt.wait(B_DRAIN, 0);
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
  uint32_t smem, tmem;  // tmem: with the warp's lanes
  int* poison;
  float* stage;         // [column][row]
  const Seg* ring;
  int lane, r;          // accumulator, row in it
  uint32_t sn, on, pairn, seg;

  __device__ __forceinline__ bool pair_sync() {
    wt.arrive_warp(B_PAIR);
    return wt.wait_warp(B_PAIR, pairn++ & 1);
  }

  // The lane's 128 rows of Q, in storage order and swizzled.
  __device__ __forceinline__ int block_rows(const Seg& k) const { return min(k.n * a.gq - k.qb * C::QB, C::QB); }
  __device__ __forceinline__ void load_q(const Seg& k) {
    if (k.alt && lane == 1) return;
    constexpr int LPR = D / 16;    // threads of a row, 32 bytes each
    constexpr int RPI = 32 / LPR;  // rows of a warp at a time
    const int w = r >> 5, l = r & 31;
    const int rows = block_rows(k);
    const int rb = k.qb * C::QB + lane * 128;
    const uint32_t base = smem + C::OFF_Q + lane * C::QBYTES;
#pragma unroll 4
    for (int i = 0; i < 32 / RPI; ++i) {
      const int row = w * 32 + i * RPI + l / LPR, c = (l % LPR) * 2;  // c: 16-byte piece of the row
      uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
      if (lane * 128 + row < rows) {
        const int R = rb + row;
        const int tok = token_of(a, R), g = R - tok * a.gq;
        const uint4* src = reinterpret_cast<const uint4*>(
                               a.q + ((int64_t)(k.c0 + tok) * a.Hq + k.h * a.gq + g) * D) + c;
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
    wt.arrive_warp(B_QFULL + lane);
  }

  // One tile: the weights of S's row into TMEM, m and l brought up to date.
  // visible: tokens of the tile that the row sees (a prefix); bad: pages left out.
  __device__ __forceinline__ void tile(int visible, uint32_t bad, bool has_o, float& m, float& l) {
    const uint32_t sa = tmem + C::S0 + lane * C::TN;
    float s[C::TN];
    float mx[4];
#pragma unroll
    for (int i = 0; i < C::TN; i += 32) tc5::ld32_max(sa + i, reinterpret_cast<uint32_t*>(s + i), mx[i / 32]);
    tc5::wait_ld();
#pragma unroll
    for (int i = 0; i < C::TN; i += 32) {
      tc5::pin32(reinterpret_cast<uint32_t*>(s + i));
      asm volatile("" : "+f"(mx[i / 32]));
    }
    if (__any_sync(0xffffffffu, visible < C::TN) || bad) {
#pragma unroll
      for (int i = 0; i < C::TN; i += kPage) {
        const int v = (bad >> (i / kPage)) & 1u ? 0 : visible - i;
        float x = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPage; ++j) {
          s[i + j] = j < v ? s[i + j] : -INFINITY;
          x = fmaxf(x, s[i + j]);
        }
        mx[i / 32] = x;
      }
    }
    const float mt = C::TN == 128 ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) : fmaxf(mx[0], mx[1]);
    const float c = a.scale_log2;
    const float mn = fmaxf(m, mt);
    const bool moves = (mn - m) * c > 8.0f;
    if (__any_sync(0xffffffffu, moves)) {
      const float f = moves ? ptx::ex2_ftz((m - mn) * c) : 1.0f;
      if (moves) m = mn;
      l *= f;
      if (has_o) {
#pragma unroll 1
        for (int i = 0; i < D; i += 16) {
          uint32_t o[16];
          tc5::ld16(tmem + C::O0 + lane * C::OSTEP + i, o);
          tc5::wait_ld();
          tc5::pin16(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tc5::st16(tmem + C::O0 + lane * C::OSTEP + i, o);
        }
      }
    }
    const float off = m == -INFINITY ? 0.0f : -m * c;
    const uint64_t c2 = pack_f32x2(c, c), off2 = pack_f32x2(off, off);
    uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < C::TN; h += 32) {
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t x = fma_f32x2(pack_f32x2(s[h + i], s[h + i + 1]), c2, off2);
        const float e0 = ptx::ex2_ftz(__uint_as_float(lo_bits(x)));
        const float e1 = ptx::ex2_ftz(__uint_as_float(hi_bits(x)));
        sum2[(i / 2) & 3] = add_f32x2(sum2[(i / 2) & 3], pack_f32x2(e0, e1));
        p[i / 2] = ptx::pack_h2(e0, e1);
      }
      tc5::st16(sa + h / 2, p);
    }
    const uint64_t t2 = add_f32x2(add_f32x2(sum2[0], sum2[1]), add_f32x2(sum2[2], sum2[3]));
    l += __uint_as_float(lo_bits(t2)) + __uint_as_float(hi_bits(t2));
    tc5::wait_st();
  }

  // What the notes say of the row's outputs: the row sees `lim` tokens; written over the
  // thread's own earlier stores, to the output (whole) or to the piece's O in `slot`.
  __device__ __forceinline__ void notes(int lim, bool whole, int64_t at, int slot, int row) const {
    const int* pn = poison + (seg & 1) * 3 * D;
#pragma unroll 1
    for (int c = 0; c < D; ++c) {
      const bool up = pn[c] < lim, down = pn[D + c] < lim, nan = pn[2 * D + c] < lim;
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
  __device__ __forceinline__ int64_t out_at(const Seg& k, int row) const {
    const int R = k.qb * C::QB + row;
    const int tok = token_of(a, R);
    return ((int64_t)(k.c0 + tok) * a.Hq + k.h * a.gq + (R - tok * a.gq)) * D;
  }

  __device__ __forceinline__ float inverse(float l) const {
    if (l == 0.0f) set_error(a.err_word, KVQ_ERRBIT_EMPTY);  // nothing seen
    return l == 0.0f ? 0.0f : 1.0f / l;
  }

  // The pieces of a cut unit, from their (O, m, l) in global memory: 16 columns of a row
  // at a time, all softmax threads.  first .. last: the blocks that hold the pieces.
  __device__ __forceinline__ void join(const Seg& k) const {
    const int rows = block_rows(k), first = k.first_b, last = k.last_b;
    const int tid = lane * 128 + r;
    const float c = a.scale_log2;
    for (int it = tid; it < rows * (D / 16); it += C::SMT) {
      const int cg = it / rows, row = it - cg * rows;
      float m = -INFINITY;
#pragma unroll 4
      for (int p = first; p <= last; ++p)
        m = fmaxf(m, __ldcg(a.ml_part + (int64_t)(2 * p + (p == first)) * C::QB + row).x);
      float l = 0.0f, o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = 0.0f;
#pragma unroll 2
      for (int p = first; p <= last; ++p) {
        const int64_t slot = 2 * p + (p == first);
        const float2 ml = __ldcg(a.ml_part + slot * C::QB + row);
        const float f = ml.x == -INFINITY ? (ml.y != ml.y ? NAN : 0.0f) : ptx::ex2_ftz((ml.x - m) * c);
        l += ml.y * f;
        const float4* src = a.o_part + (slot * (D / 4) + cg * 4) * C::QB + row;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = __ldcg(src + e * C::QB);
          o[4 * e] += v.x * f;
          o[4 * e + 1] += v.y * f;
          o[4 * e + 2] += v.z * f;
          o[4 * e + 3] += v.w * f;
        }
      }
      store16(o, inverse(l), out_at(k, row) + cg * 16);
    }
  }

  __device__ __forceinline__ bool run(int block) {
    SegReader at_seg;
    if (!__all_sync(0xffffffffu, at_seg.wait(wt))) return false;
    if (at_seg.get(ring).b < 0) return true;
    load_q(at_seg.get(ring));
    while (true) {
      const Seg& k = at_seg.get(ring);
      const bool alt = k.alt;
      const int row = (alt ? 0 : lane * 128) + r;  // of the block
      const int rows = block_rows(k);
      const bool warp_live = (row & ~31) < rows;
      int lim = 0;
      if (row < rows) lim = seen_of(a, k.n, k.ns + k.npk + k.nres, token_of(a, k.qb * C::QB + row));
      const int plim = seen_packed(k.ns, k.npk, lim), flim = seen_f16(k.ns, k.npk, lim);
      const int npt = k.npt, hi = k.hi;
      float m = -INFINITY, l = 0.0f;
      const int step = alt ? 2 : 1, t0 = k.lo + (alt ? lane : 0);
      for (int t = t0; t < hi; t += step) {
        const bool packed = t < npt;
        const int visible = packed ? plim - t * C::TN : flim - (t - npt) * C::TN;
        uint32_t bad = 0;
        if (a.rm.paged && packed) {
          const int j = t * (C::TN / kPage) + (r & 31);
          bool out = false;
          if ((r & 31) < C::TN / kPage && j * kPage < k.npk) {
            const int pg = a.rm.page_of(k.b, j);
            out = pg < 0 || pg >= a.rm.npages;
          }
          bad = __ballot_sync(0xffffffffu, out);
        }
        if (!wt.wait_warp(B_SFULL + lane, sn++ & 1)) return false;
        tc5::fence_after();
        if (warp_live) tile(visible, bad, t > t0, m, l);
        tc5::fence_before();
        wt.arrive_warp(B_PREADY + lane);
      }
      const bool any = t0 < hi;
      if (any && !wt.wait_warp(B_ODONE + lane, on++ & 1)) return false;
      tc5::fence_after();

      SegReader after = at_seg;
      ++after.i;
      if (!__all_sync(0xffffffffu, after.wait(wt))) return false;
      const bool more = after.get(ring).b >= 0;
      if (more && !alt) load_q(after.get(ring));  // under the epilogue

      // with alternating lanes the other's tiles may still be on their way
      if (alt && !pair_sync()) return false;
      const bool noted = wt.words[W_PFLAG + (seg & 1)] != 0;
      const bool whole = k.lo == 0 && k.hi == k.nt;
      const int slot = 2 * block + (k.lo == 0);
      const uint32_t oa = tmem + C::O0 + lane * C::OSTEP;
      float inv = 0.0f;
      int64_t at = 0;
      // With alternating lanes, lane 1's accumulator goes through shared memory to lane
      // 0, 32 columns at a time, with its rows' m and l.
      const bool pass = alt && k.hi - k.lo > 1;
      float* xm = stage + 32 * 128;
      float f0 = 1.0f, f1 = 0.0f;
      if (pass) {
        if (lane == 1 && warp_live) {
          xm[r] = m;
          xm[128 + r] = l;
        }
        if (!pair_sync()) return false;
        const float m1 = xm[r], l1 = xm[128 + r], mm = fmaxf(m, m1), c = a.scale_log2;
        if (lane == 0) {
          // a lane that saw nothing has weight zero (NaN scores stay NaN through l)
          f0 = m == -INFINITY ? 0.0f : ptx::ex2_ftz((m - mm) * c);
          f1 = m1 == -INFINITY ? 0.0f : ptx::ex2_ftz((m1 - mm) * c);
          if (l != l) f0 = l;
          if (l1 != l1) f1 = l1;
          l = l * f0 + l1 * f1;
          m = mm;
        }
      }
      const bool mine = row < rows && !(alt && lane == 1);
      if (mine) {
        at = out_at(k, row);
        if (whole)
          inv = inverse(l);
        else
          __stcg(a.ml_part + (int64_t)slot * C::QB + row, make_float2(m, l));
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        if (warp_live && any) {
          tc5::ld32(oa + c0, reinterpret_cast<uint32_t*>(o));
          tc5::wait_ld();
          tc5::pin32(reinterpret_cast<uint32_t*>(o));
        }
        if (pass) {
          if (lane == 1 && warp_live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) stage[j * 128 + r] = o[j];
          }
          if (!pair_sync()) return false;
          if (lane == 0 && warp_live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = o[j] * f0 + stage[j * 128 + r] * f1;
          }
          if (!pair_sync()) return false;
        }
        if (mine && whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 16) store16(o + j, inv, at + c0 + j);
        } else if (mine) {
          float4* dst = a.o_part + ((int64_t)slot * (D / 4) + c0 / 4) * C::QB + row;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            __stcg(dst + j * C::QB, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
        }
        __syncwarp();
      }
      if (noted && mine) notes(lim, whole, at, slot, row);
      // the notes have been read: clean them for the segment after next
      if (noted) {
        if (!pair_sync()) return false;
        for (int i = lane * 128 + r; i < 3 * D; i += C::SMT) poison[(seg & 1) * 3 * D + i] = 0x7fffffff;
        if (lane * 128 + r == 0) wt.words[W_PFLAG + (seg & 1)] = 0;
        if (!pair_sync()) return false;
      }
      tc5::fence_before();
      wt.arrive_warp(B_EPI + (seg & 1));
      ++seg;

      if (!whole) {
        __threadfence();
        if (!pair_sync()) return false;
        if (lane * 128 + r == 0) wt.words[W_TICKET] = atomicAdd(a.tickets + k.first_b, 1u);
        if (!pair_sync()) return false;
        if (wt.words[W_TICKET] == (uint32_t)(k.last_b - k.first_b)) {
          __threadfence();
          join(k);
          if (lane * 128 + r == 0) a.tickets[k.first_b] = 0;
        }
      }
      wt.arrive_warp(B_SEGEMPTY + at_seg.i % kSegs);
      if (!more) return true;
      at_seg = after;
      // with alternating lanes: Q goes where the accumulator passed, after all have read it
      if (alt) load_q(at_seg.get(ring));
    }
  }
};

// ------------------------------------------------------------------- kernel ---

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkAttnArgs a) {
  using C = Cfg<D, BITS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t smem = ptx::smem_u32(base);
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(base + C::OFF_BAR);
  volatile int64_t* wide = reinterpret_cast<volatile int64_t*>(base + C::OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lid = tid & 31;

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
      init(B_QFULL + i, 4);
      init(B_SFULL + i, 1 + (a.fault && blockIdx.x == 0 ? 1 : 0));
      init(B_PREADY + i, 4);
      init(B_ODONE + i, 1);
      init(B_EPI + i, 4 * C::LANES);
    }
    for (int i = 0; i < kSegs; ++i) {
      init(B_SEGFULL + i, 1);
      init(B_SEGEMPTY + i, 4 * C::LANES + 4 + 1);
    }
    init(B_PAIR, 4 * C::LANES);
    init(B_DRAIN, 1);
    for (int i = 0; i < C::ST; ++i) {
      init(B_KFULL + i, 4);
      init(B_KEMPTY + i, 1);
      init(B_VFULL + i, 4);
      init(B_VEMPTY + i, 1);
    }
    words[W_ABORT] = 0;
    words[W_PFLAG] = words[W_PFLAG + 1] = 0;
    ptx::fence_mbar_init();
  }
  int* poison = reinterpret_cast<int*>(base + C::OFF_POISON);
  for (int i = tid; i < 2 * 3 * D; i += kThreads) poison[i] = 0x7fffffff;
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
  if (warp == 12) tc5::alloc(smem + C::OFF_BAR + 4 * W_TMEM, 512);
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = words[W_TMEM];
  const Waits wt = {smem + C::OFF_BAR, words, a.err_word, a.wait_limit_us};
  Seg* ring = reinterpret_cast<Seg*>(base + C::OFF_SEG);
  const int sb = words[W_STARTB], sq = words[W_STARTQ];
  const int64_t sbase = wide[W_BASE / 2 + 1];

  // Registers: 128 a thread at launch (65536 in all) = 256 x 184 + 128 x 96 + 128 x 48.
  if (warp < 8) {
    tc5::regs_inc<184>();
    if (warp < 4 * C::LANES) {
      Soft<D, BITS> soft = {a, wt, smem, tmem + ((uint32_t)(warp & 3) << 21), poison,
                            reinterpret_cast<float*>(base + C::OFF_STAGE), ring,
                            warp >> 2, tid & 127, 0, 0, 0, 0};
      soft.run(blockIdx.x);
    }
  } else if (warp < 12) {
    tc5::regs_dec<96>();
    Deq<D, BITS> deq = {a, wt, smem, poison, ring, tid - 256, 0};
    deq.run();
  } else {
    tc5::regs_dec<48>();
    if (tid == 12 * 32) mma_role<D, BITS>(a, wt, smem, tmem, ring);
    if (tid == 13 * 32) walk_role<D, BITS>(a, wt, ring, sb, sq, sbase, x0, x1, W, G);
    __syncwarp();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (warp == 12) tc5::dealloc(tmem, 512);
}

template <int D, int BITS>
cudaError_t launch(const ChunkAttnArgs& a, int grid, cudaStream_t st) {
  static_assert(Cfg<D, BITS>::SMEM <= 227 * 1024, "shared memory of a block");
  auto kernel = chunk_attn_kernel<D, BITS>;
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, kernel);
  if (e != cudaSuccess) return e;
  // the warps' shares (setmaxnreg) come out of what the block is launched with
  if (at.numRegs != 65536 / kThreads) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, BITS>::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, Cfg<D, BITS>::SMEM, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_bits(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st) {
  if (bits == 4) return launch<D, 4>(a, grid, st);
  if (bits == 3) return launch<D, 3>(a, grid, st);
  return launch<D, 2>(a, grid, st);
}

}  // namespace chunk
}  // namespace kvq
