// kvq_prompt_attn.cuh -- causal attention over whole prompts in full precision, on the
// fifth-generation tensor cores.
//
// The mathematics.  The query rows of a block are T = 128 / gq tokens times the gq heads
// that share a KV head, row = token * gq + head, twice (two lanes): one pass over K and V
// serves them all.  For a tile of TN tokens S = Q K^T, P = exp2(S c - m c) with the row's
// reference maximum m, O += P V, l += sum P; c = log2(e) / sqrt(d).  m follows the running
// maximum lazily: it moves (and O, l are rescaled) only when the maximum has passed it by
// 2^8.  Roundings: the weights P to fp16 once (they and l carry a factor 2^7, which O / l
// cancels, so that they keep 11 bits down to 2^-21 of the reference and lose at most 2^-32
// of it below), the output once; scores, m, l and O are fp32.  For fp32 output the weights
// are two fp16 parts, P and what its rounding left, each times V; and as the tensor cores'
// sums are cut off, not rounded (2^-23 of O a step, all towards zero: 6e-5 over 16384 tokens
// of values of one sign), every kSegment tokens O goes to the output's fp32 sums.
//
// A block (one per SM, persistent) has 12 warps:
//   0-7   softmax: a thread per query row, four warps for each of the two accumulators
//         (lanes): S from TMEM, P back to TMEM in S's place as the A operand of the second
//         MMA, the epilogue.
//   8     issues the MMAs: the lanes' steps in turn, so that the softmax of one runs under
//         the MMAs of the other.
//   9     loads Q, K and V (TMA tiles, 128-byte swizzle).  A slot of the ring has what a batch
//         of MMAs takes, a tile's values and a later tile's keys, under one barrier.
//   10    looks at values that some row of the block does not see (the tiles at the
//         diagonal): a weight of zero would turn an infinite one into NaN.  With fp32 output
//         at those of all tiles: of the weights' second parts about half are negative.
//   11    works out the units.
// head_dim 256 has room for one lane, tiles of 64 tokens, and the scores of two: the next
// tile's are there when a tile's weights are done (4096 tokens of 32 heads on 8: 265 -> 220
// us).  Two smaller tiles of scores in place of one made head_dim 128
// 33 % slower (Q is read from shared memory for each) and 64 up to 70 %.
//
// Bound: at head_dim 128 the tensor cores take 2048 cycles for a tile of both lanes, and a
// lane's own chain about 2600: softmax 1120 (loads from TMEM to the first exponential 280,
// exponentials and weights 750), the MMA warp's waits, two batches of MMAs.  At head_dim 64
// the MMAs of both lanes take 1024 and the chain 2120, of which the MMA warp issues for 420:
// two chains are too few to fill the tensor cores (27 % with fp32 output) or the exponentials
// (17 %).
// 16384 tokens of 32 heads on 8: 1360 us (1.62 PFLOP/s, 1270 between others of its kind);
// 16 prompts of 115 to 2048 tokens: 176 us.
//
// Where there cannot be more units than SMs, a unit is T tokens, and its two lanes have the
// same rows: every second tile is lane 1's, and the lanes' sums meet in the epilogue, each
// lane's warps storing half of the columns.  That halves the longest unit, which is what
// such a call takes (4096 tokens of 8 heads on 2, head_dim 128: 49 -> 30 us; 10836 tokens
// of 3 heads on 1: 120 -> 70); with more units K and V are loaded twice for nothing (4096
// tokens of 16 heads on 4: 50 -> 58 us).
//
// A unit of work is (sequence, KV head, block of 2 T tokens).  Units lie in one line,
// sequence after sequence, the longest first within each.  The grid has a block for each;
// those that run take over the next of those that do not yet (cluster launch control), when
// they load the last tiles of the unit before, so that the loads go on from unit to unit
// and SMs are done at about the same time (units dealt out in turn made 16 prompts of
// 17 to 2048 tokens 10 % slower and 8 of 100 to 1500 at head_dim 64 26 %).
#pragma once

#include <cuda.h>
#include <math.h>

#include <atomic>

#include "kvq_around.cuh"
#include "kvq_ptx.cuh"
#include "kvq_runs.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

struct PromptAttnArgs {
  CUtensorMap mq, mk, mv;  // {element, head of the group, token, KV head}; {element, token, KV head}
  const int32_t* cu;
  uint32_t* err_word;
  void* out;  // [total][Hq][d]
  int B, Hkv, gq, T, total, max_len, out_f32;
  int shared;       // 1: the lanes have the same rows
  uint32_t gq_mul;  // row / gq = row * gq_mul >> 16 for rows below 128
  uint32_t wait_limit_us;
  int fault;  // testing hook: 1 makes the scores' barriers wait for an arrival that never comes
  float scale_log2;
};

cudaError_t launch_prompt_attn_d32(const PromptAttnArgs& a, int grid, cudaStream_t st);
cudaError_t launch_prompt_attn_d64(const PromptAttnArgs& a, int grid, cudaStream_t st);
cudaError_t launch_prompt_attn_d128(const PromptAttnArgs& a, int grid, cudaStream_t st);
cudaError_t launch_prompt_attn_d256(const PromptAttnArgs& a, int grid, cudaStream_t st);

// The kernel's shapes: lanes of a block, tokens of a tile, elements of a tile's row in
// shared memory (a panel; 128 bytes, or 64 at head_dim 32).
__host__ __device__ constexpr int prompt_lanes(int d) { return d == 256 ? 1 : 2; }
__host__ __device__ constexpr int prompt_tile(int d) { return d == 256 ? 64 : 128; }
__host__ __device__ constexpr int prompt_panel(int d) { return d < 64 ? d : 64; }

namespace prompt {

constexpr int kThreads = 384;
constexpr float kWeightBits = 7.0f;  // log2 of the weights' factor
constexpr int kMaxStages = 4;
constexpr int kSegment = 2048;       // tokens whose values the tensor cores add up for fp32 output (a power of two)

template <int D>
struct Cfg {
  static constexpr int LANES = prompt_lanes(D);
  static constexpr int TN = prompt_tile(D);
  static constexpr int NB = D == 256 ? 2 : 1;  // tiles of scores that a lane has room for
  static constexpr int PW = prompt_panel(D);
  static constexpr int NP = D / PW;
  static constexpr int RB = PW * 2;  // bytes of a panel's row
  static constexpr int SWZ = RB == 128 ? 2 : 4;
  static constexpr int QP = 128 * RB;  // bytes of a panel of Q
  static constexpr int KP = TN * RB;   // of a panel of K or V
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int KBYTES = TN * D * 2;
  static constexpr int ST = D >= 128 ? 2 : 4;  // slots of the ring, values and keys each
  static constexpr int SMW = 4 * LANES;        // softmax warps
  // TMEM columns
  static constexpr int S0 = 0;
  static constexpr int O0 = 256;
  // shared memory
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = OFF_Q + LANES * QBYTES;
  static constexpr int OFF_OUT = OFF_KV + ST * 2 * KBYTES;  // 4 KiB of each softmax warp
  static constexpr int OFF_NOTES = OFF_OUT + SMW * 4096;  // int [3][D]
  static constexpr int OFF_BAR = OFF_NOTES + 3 * D * 4;
  static constexpr int OFF_UNIT = OFF_BAR + 512;  // Unit, and the answer of the launch control
  // (more than half an SM's, so that a block has the tensor memory to itself)
  static constexpr int SMEM = OFF_UNIT + 48 > 117 * 1024 ? OFF_UNIT + 48 : 117 * 1024;
};

// Sequence rows [c0, c0 + n), KV head h, first token t0 of the block; tiles of each lane
// (lane 1's are 0 or not fewer; shared rows: every second one, lane 0 begins), and all that
// are loaded; no: 1, 2, .. in the block's order, 0: the end.
struct alignas(16) Unit {
  int c0, n, h, t0;
  int tiles0, tiles1, no, tiles;
};

// Barriers (8 bytes each from OFF_BAR) and words behind them.
enum { B_QFULL = 0, B_QEMPTY = 2, B_SFULL = 4, B_PREADY = 8, B_ODONE = 12, B_DRAIN = 16, B_UFULL = 17,
       B_UEMPTY = 18, B_NEXT = 19, B_JOIN = 20, B_KVFULL = 21, B_KVEMPTY = B_KVFULL + kMaxStages, B_VOK = B_KVEMPTY + kMaxStages, B_COUNT = B_VOK + kMaxStages };
enum { W_TMEM = 96, W_ABORT = 97, W_NOTED = 98 /* the unit that the notes are of */, W_EPI = 99 };
static_assert(B_COUNT * 2 <= W_TMEM, "words behind the barriers");

__device__ __forceinline__ uint32_t lds(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t timer_lo() {  // nanoseconds, modulo 2^32
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// 3D and 4D tile loads, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Bounded waits (at most a second): all give up when one has.
struct Waits {
  uint32_t bars;  // shared address of the barriers and words
  uint32_t limit_us;

  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  __device__ __forceinline__ uint32_t word(int i) const { return lds(bars + 4 * i); }
  __device__ __forceinline__ void set_word(int i, uint32_t v) const { sts(bars + 4 * i, v); }
  __device__ __forceinline__ bool late(uint32_t t0) const {
    if (word(W_ABORT)) return true;
    if (timer_lo() - t0 <= limit_us * 1000u) return false;
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
  __device__ __forceinline__ bool test(int i, uint32_t parity) const {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(bar(i)), "r"(parity)
                 : "memory");
    return ok != 0;
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

// A role's place in the line of units (all of a warp).
struct UnitReader {
  const Waits& wt;
  const Unit* unit;
  uint32_t i = 0;
  // the next unit; no == 0 at the end of the line or when a wait gave up
  __device__ __forceinline__ Unit next() {
    Unit u;
    u.no = 0;
    if (wt.wait_warp(B_UFULL, i & 1)) u = *unit;
    ++i;
    return u;
  }
  __device__ __forceinline__ void release() { wt.arrive_warp(B_UEMPTY); }
};

// -------------------------------------------------------------------- units ---

// Asks for a block of the grid that has not begun; the answer goes to `to` (16 bytes),
// which counts on `bar`.  One thread.
__device__ __forceinline__ void ask_next(uint32_t to, uint32_t bar) {
  ptx::mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
      "r"(bar)
      : "memory");
}
// The answer: that block's index, which is the asker's now, or -1 (all have begun).
__device__ __forceinline__ int next_block(uint32_t at) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n ld.shared.b128 h, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}"
      : "=r"(ok), "=r"(x)
      : "r"(at)
      : "memory");
  // (read before the next answer is written)
  ptx::fence_proxy_async_shared();
  return ok ? (int)x : -1;
}

// The line of units as a warp sees it: a window of 32 sequences goes along it.
struct UnitLine {
  const int32_t* cu;
  int B, total, max_len, Hkv, step;  // step: tokens of a unit
  int b0;                            // the window's first sequence
  int64_t base, scan;                // units before the window; of its sequences up to the lane's
  Run run;

  __device__ __forceinline__ void begin() {
    b0 = 0;
    base = 0;
    window();
  }
  __device__ __forceinline__ void window() {
    const int lane = threadIdx.x & 31;
    run = {0, 0};
    if (b0 + lane < B) run = run_of(cu, b0 + lane, total, max_len);
    scan = run.n > 0 ? (int64_t)((run.n + step - 1) / step) * Hkv : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
  }
  // The window goes to the one that has unit u; false: there are not so many.  Units mostly
  // come in rising order, but nothing says that the blocks a block takes over do.
  __device__ __forceinline__ bool find(int u) {
    if (u < base) begin();
    while (b0 < B) {
      const int64_t all = __shfl_sync(0xffffffffu, scan, 31);
      if (u < base + all) return true;
      base += all;
      b0 += 32;
      window();
    }
    return false;
  }
  // Whether the lane's sequence is the one that has unit u of the window (all lanes ask).
  __device__ __forceinline__ bool has(int u) const {
    const uint32_t at = __ballot_sync(0xffffffffu, u < base + scan);
    return (int)(threadIdx.x & 31) == __ffs(at) - 1;
  }
  // Its head and first token, by that lane: the sequence's last block first, heads within blocks.
  __device__ __forceinline__ void place(int u, int& h, int& t0) const {
    const int r = (int)(base + scan - 1 - u);  // units after it in the sequence
    h = Hkv - 1 - r % Hkv;
    t0 = r / Hkv * step;
  }
};

// The warp that works out the units.
template <int D, bool SHARED>
__device__ __forceinline__ void unit_role(const PromptAttnArgs& a, const Waits& wt, uint32_t smem, Unit* unit) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  UnitLine line;
  line.cu = a.cu;
  line.B = a.B, line.total = a.total, line.max_len = a.max_len, line.Hkv = a.Hkv;
  line.step = (SHARED ? 1 : C::LANES) * a.T;
  line.begin();
  const uint32_t answer = smem + C::OFF_UNIT + sizeof(Unit);
  int u = blockIdx.x;
  bool own = true;
  uint32_t asked = 0;
  for (uint32_t i = 0;; ++i) {
    // the roles have the last unit, and the loads of it are on their way
    if (i > 0 && !wt.wait_warp(B_UEMPTY, (i - 1) & 1)) return;
    while (true) {
      if (!own) {
        if (lane == 0) ask_next(answer, wt.bar(B_NEXT));
        __syncwarp();
        if (!wt.wait_warp(B_NEXT, asked & 1)) {
          // (the block gives up: the answer lands before its shared memory goes)
          for (const uint32_t t0 = timer_lo(); !ptx::mbar_try_wait(wt.bar(B_NEXT), asked & 1);)
            if (timer_lo() - t0 > 1000000000u) break;
          return;
        }
        ++asked;
        u = next_block(answer);
        __syncwarp();
      }
      own = false;
      if (u < 0) break;
      // each block of the grid, and each that is taken over, looks at one sequence's entries
      if (lane == 0 && u < a.B && run_of(a.cu, u, a.total, a.max_len).n < 0)
        set_error(a.err_word, KVQ_ERRBIT_BADLEN);
      if (line.find(u)) break;
      // the grid may have more blocks than there are units: the rest are taken over here
    }
    const bool more = u >= 0;
    // the lane of the sequence that has unit u
    const bool has = line.has(u);
    if (more ? has : lane == 0) {
      Unit s;
      s.no = 0;
      if (more) {
        s.c0 = line.run.c0, s.n = line.run.n;
        line.place(u, s.h, s.t0);
        auto tiles = [&](int l) {
          const int first = s.t0 + l * a.T;
          return first < s.n ? (min(first + a.T, s.n) + C::TN - 1) / C::TN : 0;
        };
        s.tiles0 = tiles(0);
        s.tiles1 = C::LANES == 2 && !SHARED ? tiles(1) : 0;
        s.tiles = max(s.tiles0, s.tiles1);
        if (SHARED) s.tiles1 = s.tiles / 2, s.tiles0 = s.tiles - s.tiles1;
        s.no = i + 1;
      }
      *unit = s;
      ptx::mbar_arrive(wt.bar(B_UFULL));
    }
    __syncwarp();
    if (!more) return;
  }
}

// -------------------------------------------------------------------- loads ---

template <int D, bool SHARED>
__device__ __forceinline__ void load_role(const PromptAttnArgs& a, const Waits& wt, uint32_t smem, const Unit* unit) {
  using C = Cfg<D>;
  const bool one = (threadIdx.x & 31) == 0;
  if (one) {
    ptx::prefetch_tensormap(&a.mq);
    ptx::prefetch_tensormap(&a.mk);
    ptx::prefetch_tensormap(&a.mv);
  }
  UnitReader units = {wt, unit};
  uint32_t item = 0, qn[2] = {0, 0};  // slots so far, units of each lane
  bool ok = true;
  while (ok) {
    const Unit u = units.next();
    if (u.no == 0) break;
    // values of tile tv (keys: its keys) and keys of tile tk into the next slot (none: -1)
    auto fill = [&](int tv, int tk, bool keys) {
      const int slot = item % C::ST;
      ok = ok && wt.wait_warp(B_KVEMPTY + slot, ((item / C::ST) & 1) ^ 1);
      if (!ok) return;
      if (one) {
        ptx::mbar_arrive_expect_tx(wt.bar(B_KVFULL + slot), ((tv >= 0) + (tk >= 0)) * C::KBYTES);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int t = w ? tk : tv;
          if (t < 0) continue;
#pragma unroll
          for (int p = 0; p < C::NP; ++p)
            tma_load(smem + C::OFF_KV + (2 * slot + w) * C::KBYTES + p * C::KP, w || keys ? &a.mk : &a.mv, p * C::PW,
                     u.c0 + t * C::TN, u.h, wt.bar(B_KVFULL + slot));
        }
      }
      ++item;
    };
    constexpr int ahead = C::NB * (SHARED ? 2 : 1);  // (in the order in which the MMAs take them)
    static_assert(ahead <= 2, "a unit's first keys have one slot");
    fill(ahead == 2 && u.tiles > 1 ? 1 : -1, 0, true);
#pragma unroll
    for (int l = 0; l < C::LANES; ++l) {
      if ((l ? u.tiles1 : u.tiles0) == 0 || (l && SHARED)) continue;
      ok = ok && wt.wait_warp(B_QEMPTY + l, (qn[l] & 1) ^ 1);
      if (!ok) break;
      if (one) {
        ptx::mbar_arrive_expect_tx(wt.bar(B_QFULL + l), a.T * a.gq * D * 2);
#pragma unroll
        for (int p = 0; p < C::NP; ++p)
          tma_load(smem + C::OFF_Q + l * C::QBYTES + p * C::QP, &a.mq, p * C::PW, 0, u.c0 + u.t0 + l * a.T, u.h,
                   wt.bar(B_QFULL + l));
      }
      ++qn[l];
    }
    for (int t = 0; ok && t < u.tiles; ++t) fill(t, t + ahead < u.tiles ? t + ahead : -1, false);
    units.release();
  }
  // copies still in flight when the block gives up land before its shared memory goes
  const uint32_t t0 = timer_lo();
  auto landed = [&](int bar, uint32_t parity) {
    while (!ptx::mbar_try_wait(wt.bar(bar), parity))
      if (timer_lo() - t0 > 1000000000u) return;
  };
  for (uint32_t i = item > C::ST ? item - C::ST : 0; i < item; ++i) landed(B_KVFULL + i % C::ST, (i / C::ST) & 1);
  for (int l = 0; l < C::LANES; ++l)
    if (qn[l] > 0) landed(B_QFULL + l, (qn[l] - 1) & 1);
}

// ------------------------------------------------------------- values' check ---

// The first tile that the MMAs of its values wait for the check of: all before it are seen
// whole by every row of the block.  TWO: the notes of those have to be complete when either
// lane's sums are, so the last tile of each lane is waited for in any case (a block of one
// row, at a tile's end, sees all of it).
template <int D, bool TWO, bool SHARED>
__device__ __forceinline__ int checked_from(int t0, int tiles0, int tiles) {
  const int first = (t0 + 1) / Cfg<D>::TN;  // the block's first row sees tokens up to t0
  return TWO ? min(first, (SHARED ? tiles : tiles0) - 1) : first;
}

// Values that are not finite, at tokens that some row of the block does not see (tokens of
// the next sequence among them): zeros take their place in the tile, and the first
// token with +inf, -inf or NaN in a column is noted; the epilogue gives the rows that see
// it what the sum would be.  In tiles that all rows see whole the MMA does that itself,
// unless the weights have two parts (TWO): the second, what the first's rounding left, is
// negative or zero as often as not, and either makes NaN of an infinite value.  So those of
// all tiles are noted then, and what is in O does not count (8 prompts of 245 to 1500 tokens,
// 16 heads of 64: 53.7 -> 54.8 us).
// The warp sees every fill of the ring (a parity alone does not tell a fill from the one
// before the last), and a stage is free when it and the MMAs are done with it.
template <int D, bool TWO, bool SHARED>
__device__ __forceinline__ void check_role(const PromptAttnArgs& a, const Waits& wt, uint32_t smem, const Unit* unit) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  UnitReader units = {wt, unit};
  uint32_t item = 0, before = 0;  // slots so far; earlier units' epilogues, a warp each
  while (true) {
    const Unit u = units.next();
    units.release();
    if (u.no == 0) return;
    bool clean = false;  // the notes are this unit's
    const int checked = checked_from<D, TWO, SHARED>(u.t0, u.tiles0, u.tiles);
    for (int t = -1; t < u.tiles; ++t, ++item) {  // (keys alone first)
      const int stage = item % C::ST;
      if (!wt.wait_warp(B_KVFULL + stage, (item / C::ST) & 1)) return;
      const bool waited = t >= checked;  // by the MMAs, which may read the others by now
      if (t < 0 || (!TWO && !waited)) {
        wt.arrive_warp(B_KVEMPTY + stage);
        continue;
      }
      const uint32_t tile = smem + C::OFF_KV + 2 * stage * C::KBYTES;
      const int r0 = TWO ? 0 : max(0, u.t0 + 1 - t * C::TN);  // rows before it are seen by all
      bool any = false;
#pragma unroll 1
      for (int p = 0; p < C::NP; ++p)
#pragma unroll 4
        for (int at = r0 * C::RB + lane * 16; at < C::KP; at += 512) {
          const uint4 v = lds_v4(tile + p * C::KP + at);
          // an exponent of ones carries into the bit above it
          const uint32_t m = 0x7c007c00u, c = 0x04000400u;
          any |= ((((v.x & m) + c) | ((v.y & m) + c) | ((v.z & m) + c) | ((v.w & m) + c)) & 0x80008000u) != 0;
        }
      if (__any_sync(0xffffffffu, any)) {
        if (!clean) {  // earlier notes have been read
          const uint32_t t0 = timer_lo();
          while (wt.word(W_EPI) < before)
            if (wt.late(t0)) break;
          if (__any_sync(0xffffffffu, wt.word(W_ABORT) != 0)) return;
          for (int i = lane; i < 3 * D; i += 32) sts(smem + C::OFF_NOTES + 4 * i, 0x7fffffffu);
          __syncwarp();
          __threadfence_block();  // (an epilogue of this unit that needs no note may look already)
          wt.set_word(W_NOTED, u.no);
          clean = true;
        }
#pragma unroll 1
        for (int i = r0 * D + lane; i < C::TN * D; i += 32) {
          const int r = i / D, col = i % D, in = (col % C::PW) * 2;
          const uint32_t x = (uint32_t)(C::RB == 128 ? r & 7 : (r >> 1) & 3) << 4;
          const uint32_t at = tile + (col / C::PW) * C::KP + r * C::RB + (in ^ x);
          unsigned short hv;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hv) : "r"(at) : "memory");
          if ((hv & 0x7c00u) != 0x7c00u) continue;
          if (waited) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)0) : "memory");
          const int token = t * C::TN + r, kind = (hv & 0x3ffu) ? 2 : (hv & 0x8000u) ? 1 : 0;
          if (token < u.n)
            asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(smem + C::OFF_NOTES + 4 * (kind * D + col)), "r"(token)
                         : "memory");
        }
        __threadfence_block();
        ptx::fence_proxy_async_shared();
      }
      if (waited) wt.arrive_warp(B_VOK + stage);
      wt.arrive_warp(B_KVEMPTY + stage);
    }
    before += (u.tiles0 > 0 ? 4 : 0) + (u.tiles1 > 0 ? 4 : 0);
  }
}

// ---------------------------------------------------------------------- MMA ---

// All lanes of the warp go the same way, so that descriptors and addresses stay in its
// uniform registers, and one of them issues.  An MMA is taken up when the one before it is
// nearly done, so what the warp does between two batches is added to the time (a wait is
// 120 cycles of it even when it is over): there is one for a slot, looked at while the
// MMAs before it run, and one for a lane's weights (16 prompts 182 -> 176 us, 16384 tokens
// 1395 -> 1355).
//
// A batch is tile k's values and tile k + NB's scores, which go where tile k's were.  Its end
// is a phase of SFULL's barrier k % NB: those scores are there, and values up to tile k's are
// in O.  Where the lane has no tile k + NB in the unit it is one of ODONE's instead, which
// nothing comes after before the softmax has seen it.
template <int D, bool TWO, bool SHARED>
__device__ __forceinline__ void mma_role(const Waits& wt, uint32_t smem, uint32_t tmem, const Unit* ring) {
  using C = Cfg<D>;
  constexpr int NB = C::NB;
  constexpr uint32_t kIdescQK = tc5::instr_desc(128, C::TN, false);
  constexpr uint32_t kIdescPV = tc5::instr_desc(128, D, true);
  UnitReader units = {wt, ring};
  constexpr int seg = TWO ? kSegment / C::TN - 1 : 0x7fffffff;  // (k & seg) == 0: O begins
  uint32_t qn = 0, pn = 0;     // phase bits of the lanes' barriers
  uint32_t vok = 0;            // and of the stages'
  // the place in the ring
  int slot = 0;
  uint32_t phase = 0;
  constexpr int ahead = NB * (SHARED ? 2 : 1);
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  auto next = [&] {
    if (++slot == C::ST) slot = 0, phase ^= 1;
  };
  // (an address has 14 bits of a descriptor, and no sum passes them)
  const uint64_t qd0 = tc5::smem_desc(smem + C::OFF_Q, 16, 8 * C::RB, C::SWZ);
  const uint64_t kd0 = tc5::smem_desc(smem + C::OFF_KV, 16, 8 * C::RB, C::SWZ);
  const uint64_t vd0 = tc5::smem_desc(smem + C::OFF_KV, C::KP, 8 * C::RB, C::SWZ);
  auto qk = [&](int l, int b, int half) {  // by one thread
    const uint64_t qd = qd0 + (SHARED ? 0 : l) * (C::QBYTES >> 4);
    const uint64_t kd = kd0 + (uint32_t)((2 * slot + half) * (C::KBYTES >> 4));
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const int panel = j * 16 / C::PW, in = (j * 16 % C::PW) * 2;
      tc5::mma_ss(tmem + C::S0 + (l * NB + b) * C::TN, qd + ((panel * C::QP + in) >> 4),
                  kd + ((panel * C::KP + in) >> 4), kIdescQK, j > 0);
    }
  };
  auto pv = [&](int l, int b, uint64_t vd, bool begun) {
    const uint32_t p = tmem + C::S0 + (l * NB + b) * C::TN;
#pragma unroll
    for (int j = 0; j < C::TN / 16; ++j)
      tc5::mma_ts(tmem + C::O0 + l * D, p + j * 8, vd + ((j * 16 * C::RB) >> 4), kIdescPV, begun || j > 0);
    if (TWO) {  // the weights' second parts
#pragma unroll
      for (int j = 0; j < C::TN / 16; ++j)
        tc5::mma_ts(tmem + C::O0 + l * D, p + C::TN / 2 + j * 8, vd + ((j * 16 * C::RB) >> 4), kIdescPV, true);
    }
  };
  bool ok = true;
  while (ok) {
    const Unit u = units.next();
    units.release();
    if (uniform(u.no) == 0) break;
    const int n0 = uniform(u.tiles0), n1 = C::LANES == 2 ? uniform(u.tiles1) : 0;
    const int nt = uniform(u.tiles), checked = checked_from<D, TWO, SHARED>(uniform(u.t0), n0, nt);
    auto tiles = [&](int l) { return l ? n1 : n0; };
    // a lane's scores k, of keys in a half of the slot; its Q is free when they are the last
    auto scores = [&](int l, int k, int half) {
      qk(l, k % NB, half);
      tc5::commit(wt.bar(B_SFULL + l * NB + k % NB));
      if (SHARED ? 2 * k + l + 1 == nt : k + 1 == tiles(l)) tc5::commit(wt.bar(B_QEMPTY + (SHARED ? 0 : l)));
    };
    // the unit's first scores
    ok = wt.wait_warp(B_KVFULL + slot, phase);
    const int first = min(ahead, nt);
    for (int t = 0; ok && t < first; ++t) {
#pragma unroll
      for (int l = 0; l < C::LANES; ++l) {
        if (!ok || (SHARED ? (t & 1) != l : t >= tiles(l))) continue;
        const int k = SHARED ? t >> 1 : t;
        if (SHARED ? t == 0 : k == 0) {
          ok = wt.wait_warp(B_QFULL + l, (qn >> l) & 1);
          qn ^= 1u << l;
        }
        tc5::fence_after();
        if (ok && tc5::elect()) {
          scores(l, k, 1 - t);
          if (t + 1 == first && (SHARED || l == (t < n1))) tc5::commit(wt.bar(B_KVEMPTY + slot));
        }
        __syncwarp();
      }
    }
    next();
    bool filled = false;  // the slot is known to be
    for (int t = 0; ok && t < nt; ++t) {
      ok = filled || wt.wait_warp(B_KVFULL + slot, phase);
      filled = false;
      if (ok && t >= checked) {
        ok = wt.wait_warp(B_VOK + slot, (vok >> slot) & 1);
        vok ^= 1u << slot;
      }
      const uint64_t vd = vd0 + (uint32_t)(2 * slot * (C::KBYTES >> 4));
      const int slot1 = slot + 1 == C::ST ? 0 : slot + 1;
#pragma unroll
      for (int l = 0; l < C::LANES; ++l) {
        if (!ok || (SHARED ? (t & 1) != l : t >= tiles(l))) continue;
        const int k = SHARED ? t >> 1 : t, b = k % NB, i = l * NB + b;
        ok = wt.wait_warp(B_PREADY + i, (pn >> i) & 1);
        pn ^= 1u << i;
        if (!ok) continue;
        tc5::fence_after();
        if (tc5::elect()) pv(l, b, vd, (k & seg) > 0);
        __syncwarp();
        // (while those run)
        const bool last = SHARED || l == (t < n1);  // of the slot
        if (last) filled = __all_sync(0xffffffffu, wt.test(B_KVFULL + slot1, phase ^ (slot1 == 0)));
        if (tc5::elect()) {
          if (k + NB < tiles(l))
            scores(l, k + NB, 1);  // after this step in the tensor cores' order: S may take P's place
          else
            tc5::commit(wt.bar(B_ODONE + i));
          if (last) tc5::commit(wt.bar(B_KVEMPTY + slot));
        }
        __syncwarp();
      }
      next();
    }
  }
  // nothing of this thread's is in flight when TMEM is freed
  if (tc5::elect()) tc5::commit(wt.bar(B_DRAIN));
  __syncwarp();
  wt.wait_warp(B_DRAIN, 0);
}

// ------------------------------------------------------------------ softmax ---

template <int D, bool F32, bool SHARED>
struct Soft {
  using C = Cfg<D>;
  const PromptAttnArgs& a;
  const Waits& wt;
  const uint32_t smem, tmem;  // tmem: with the warp's lanes
  uint32_t sn = 0, on = 0, jn = 0;  // phase bits of the scores, of the finished sums and of the join

  static __device__ __forceinline__ int lane() { return threadIdx.x >> 7; }
  static __device__ __forceinline__ int r() { return threadIdx.x & 127; }

  // Hides what the row does not see of 32 tokens; the largest score that is left.
  static __device__ __forceinline__ float mask(float* s, int visible) {
    const uint32_t seen = visible <= 0 ? 0u : visible >= 32 ? ~0u : (1u << visible) - 1u;
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

  // The row's weights of a tile into TMEM, and their sum.  F32: what the rounding to fp16
  // leaves goes beside them.
  static __device__ __forceinline__ void weights(uint32_t sa, const float* s, uint64_t c2, uint64_t off2,
                                                 uint64_t& sum2) {
#pragma unroll
    for (int h = 0; h < C::TN; h += 32) {
      uint32_t p[16], q[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t x = fma_f32x2(pack_f32x2(s[h + i], s[h + i + 1]), c2, off2);
        const float e0 = ptx::ex2_ftz(__uint_as_float(lo_bits(x)));
        const float e1 = ptx::ex2_ftz(__uint_as_float(hi_bits(x)));
        sum2 = add_f32x2(sum2, pack_f32x2(e0, e1));
        p[i / 2] = ptx::pack_h2(e0, e1);
        if (F32) {
          const float2 f = __half22float2(ptx::u32_as_h2(p[i / 2]));
          q[i / 2] = ptx::pack_h2(e0 - f.x, e1 - f.y);
        }
      }
      tc5::st16(sa + h / 2, p);
      if (F32) tc5::st16(sa + C::TN / 2 + h / 2, q);
    }
  }

  // Waits for the scores at b.
  __device__ __forceinline__ bool scored(int b) {
    const bool ok = wt.wait_warp(B_SFULL + lane() * C::NB + b, (sn >> b) & 1);
    sn ^= 1u << b;
    tc5::fence_after();
    return ok;
  }
  // Waits until the tile whose weights were at b is in O; more: scores take their place.
  __device__ __forceinline__ bool summed(int b, bool more) const {
    const bool ok = more ? wt.wait_warp(B_SFULL + lane() * C::NB + b, (sn >> b) & 1)
                         : wt.wait_warp(B_ODONE + lane() * C::NB + b, (on >> b) & 1);
    tc5::fence_after();
    return ok;
  }

  // One tile: the row's weights into TMEM, m and l brought up to date.  visible: tokens of
  // the tile that the row sees (a prefix).  b: its place; more: the unit has a tile after it.
  __device__ __forceinline__ bool tile(int b, bool more, int visible, bool started, float& m, float& l) const {
    const uint32_t sa = tmem + C::S0 + (lane() * C::NB + b) * C::TN;
    float s[C::TN], mx[C::TN / 32];
#pragma unroll
    for (int i = 0; i < C::TN / 32; ++i) tc5::ld32_max(sa + 32 * i, reinterpret_cast<uint32_t*>(s + 32 * i), mx[i]);
    tc5::wait_ld();
#pragma unroll
    for (int i = 0; i < C::TN / 32; ++i) {
      tc5::pin32(reinterpret_cast<uint32_t*>(s + 32 * i));
      asm volatile("" : "+f"(mx[i]));
    }
    if (__any_sync(0xffffffffu, visible < C::TN)) {
#pragma unroll
      for (int i = 0; i < C::TN / 32; ++i) mx[i] = mask(s + 32 * i, visible - 32 * i);
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < C::TN / 32; ++i) mn = fmaxf(mn, mx[i]);
    const bool moves = (mn - m) * a.scale_log2 > 8.0f;
    if (__any_sync(0xffffffffu, moves)) {
      const float f = moves ? ptx::ex2_ftz((m - mn) * a.scale_log2) : 1.0f;
      if (moves) m = mn;
      l *= f;
      if (started) {
        if (C::NB > 1 && !summed(b ^ 1, more)) return false;
        const uint32_t oa = tmem + C::O0 + lane() * D;
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
    }
    const float off = m == -INFINITY ? 0.0f : fmaf(-m, a.scale_log2, kWeightBits);
    const uint64_t c2 = pack_f32x2(a.scale_log2, a.scale_log2), off2 = pack_f32x2(off, off);
    uint64_t sum2 = pack_f32x2(l, 0.0f);
    weights(sa, s, c2, off2, sum2);
    l = __uint_as_float(lo_bits(sum2)) + __uint_as_float(hi_bits(sum2));
    tc5::wait_st();
    return true;
  }

  // The warp's rows of O, times f, to the output.  A thread has a row: its 16-byte pieces go
  // through shared memory (swizzled: no two of a row's or a column's share a bank), so that
  // the warp's stores are whole 128-byte lines.  (A row to a thread, 32 lines a store, took
  // 2.9 us a unit at head_dim 128, as long as two tiles.)  F32, g > 0: added to g times what
  // is there (of the row, by the same thread).  joint: f times lane 0's O, and f1 times lane
  // 1's unless that is 0; the lanes' warps do the rounds in turn.
  __device__ __forceinline__ void store_rows(const Unit& u, float f, float g, bool joint, float f1, bool both) const {
    constexpr int BYTES = F32 ? 4 : 2;
    constexpr int COLS = D * BYTES < 128 ? D : 128 / BYTES;  // of a round
    constexpr int PPR = COLS * BYTES / 16;                   // pieces of a row
    const int lid = threadIdx.x & 31, heads = a.Hkv * a.gq;
    const uint32_t st = smem + C::OFF_OUT + (threadIdx.x >> 5) * 4096;
    auto at = [&](int row, int piece) { return st + row * (PPR * 16) + ((piece ^ (row & (PPR - 1))) << 4); };
    // the lane's first token, and how many it has
    const int t0 = u.t0 + (joint ? 0 : lane() * a.T), tokens = min(a.T, u.n - t0);
    char* const base = static_cast<char*>(a.out) + (((int64_t)u.c0 + t0) * heads + u.h * a.gq) * (D * BYTES);
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += COLS) {
      if (SHARED && joint && (c0 / COLS & 1) != lane()) continue;
#pragma unroll
      for (int c = 0; c < COLS; c += 32) {
        float o[32];
        tc5::ld32(tmem + C::O0 + (joint ? 0 : lane() * D) + c0 + c, reinterpret_cast<uint32_t*>(o));
        tc5::wait_ld();
        tc5::pin32(reinterpret_cast<uint32_t*>(o));
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= f;
        if (SHARED && both) {
          float p[32];
          tc5::ld32(tmem + C::O0 + D + c0 + c, reinterpret_cast<uint32_t*>(p));
          tc5::wait_ld();
          tc5::pin32(reinterpret_cast<uint32_t*>(p));
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(p[i], f1, o[i]);
        }
#pragma unroll
        for (int i = 0; i < 32 * BYTES / 16; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = F32 ? __float_as_uint(o[(4 * i + k) & 31])
                       : ptx::pack_h2(o[(8 * i + 2 * k) & 31], o[(8 * i + 2 * k + 1) & 31]);
          sts_v4(at(lid, c * BYTES / 16 + i), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      __syncwarp();
      uint4 v[PPR];
#pragma unroll
      for (int i = 0; i < PPR; ++i) v[i] = lds_v4(at(i * (32 / PPR) + lid / PPR, lid % PPR));
#pragma unroll
      for (int i = 0; i < PPR; ++i) {
        const uint32_t row = (r() & ~31) + i * (32 / PPR) + lid / PPR, in = (row * a.gq_mul) >> 16;
        uint4* to = reinterpret_cast<uint4*>(base + (uint64_t)(in * heads + (row - in * a.gq)) * (D * BYTES) +
                                             c0 * BYTES + lid % PPR * 16);
        if (F32) {
          const float gr = __shfl_sync(0xffffffffu, g, i * (32 / PPR) + lid / PPR);
          if ((int)in < tokens && gr > 0.0f) {
            const uint4 was = *to;
            v[i].x = __float_as_uint(fmaf(__uint_as_float(was.x), gr, __uint_as_float(v[i].x)));
            v[i].y = __float_as_uint(fmaf(__uint_as_float(was.y), gr, __uint_as_float(v[i].y)));
            v[i].z = __float_as_uint(fmaf(__uint_as_float(was.z), gr, __uint_as_float(v[i].z)));
            v[i].w = __float_as_uint(fmaf(__uint_as_float(was.w), gr, __uint_as_float(v[i].w)));
          }
        }
        if ((int)in < tokens) *to = v[i];
      }
      __syncwarp();
    }
  }

  // What the notes say of the row's columns, over what the warp has stored.  A row whose sum
  // is NaN stays NaN.
  __device__ __forceinline__ void notes(int lim, float inv, int64_t at) const {
    const uint32_t n = smem + C::OFF_NOTES;
#pragma unroll 1
    for (int c = 0; c < D; ++c) {
      const bool up = (int)lds(n + 4 * c) < lim, down = (int)lds(n + 4 * (D + c)) < lim,
                 nan = (int)lds(n + 4 * (2 * D + c)) < lim;
      if (!(up || down || nan)) continue;
      float v = nan || (up && down) || inv != inv ? NAN : up ? INFINITY : -INFINITY;
      if (!F32) {
        // (with an infinite value of the other sign in a tile that all rows see, or NaN there)
        const float o = __half2float(static_cast<__half*>(a.out)[at + c]);
        if (o != o || (isinf(o) && o != v)) v = NAN;
      }
      if (F32)
        static_cast<float*>(a.out)[at + c] = v;
      else
        static_cast<__half*>(a.out)[at + c] = __float2half(v);
    }
  }

  // All the softmax warps of the block, for lanes that share their rows.
  __device__ __forceinline__ bool together() {
    tc5::fence_before();
    wt.arrive_warp(B_JOIN);
    const bool ok = wt.wait_warp(B_JOIN, jn++ & 1);
    tc5::fence_after();
    return ok;
  }

  __device__ __forceinline__ void run(const Unit* unit) {
    UnitReader units = {wt, unit};
    while (true) {
      const Unit u = units.next();
      units.release();
      if (u.no == 0) return;
      const int n = lane() ? u.tiles1 : u.tiles0;
      if (n == 0) continue;
      const bool joint = SHARED && u.tiles1 > 0;  // both lanes have sums of the rows
      const int in = (int)(((uint32_t)r() * a.gq_mul) >> 16), tok = u.t0 + (SHARED ? 0 : lane() * a.T) + in;
      const bool live = in < a.T && tok < u.n;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // (rows that are not there need no mask)
      int visible = live ? tok + 1 - (SHARED ? lane() * C::TN : 0) : 1 << 30;
      constexpr int seg = F32 ? kSegment / C::TN - 1 : 0x7fffffff;
      float m = -INFINITY, l = 0.0f, m_out = 0.0f;
      bool begun = false;  // the output has sums, at the reference m_out
      // what sums at a reference weigh at one that is not below it: never zero, so that an
      // infinite one stays so
      auto weight = [&](float from, float to) {
        return from == to ? 1.0f : fmaxf(ptx::ex2_ftz((from - to) * a.scale_log2), 1.17549435e-38f);
      };
      // the sums so far to the output; both: lane 1's are not there already
      auto store = [&](bool last, bool both) {
        float top = m, f0 = 1.0f, f1 = 0.0f, sum = l;
        if (joint) {
          const uint32_t at = smem + C::OFF_OUT + (threadIdx.x & 31) * 8;
          sts(at + (threadIdx.x >> 5) * 4096, __float_as_uint(m));
          sts(at + (threadIdx.x >> 5) * 4096 + 4, __float_as_uint(l));
          if (!together()) return false;
          const uint32_t of = at + ((threadIdx.x >> 5) ^ 4) * 4096;
          const float om = __uint_as_float(lds(of)), ol = __uint_as_float(lds(of + 4));
          if (!together()) return false;  // (rows go where these were)
          top = fmaxf(m, om);
          f0 = weight(lane() ? om : m, top), f1 = weight(lane() ? m : om, top);
          sum = fmaf(lane() ? ol : l, f0, (lane() ? l : ol) * f1);
        }
        const float inv = last ? 1.0f / sum : 1.0f;  // (of scores that are all -inf: NaN, as of NaN ones)
        if (warp_live)
          store_rows(u, f0 * inv, F32 && begun ? weight(m_out, top) * inv : 0.0f, joint, f1 * inv, joint && both);
        if (joint && !together()) return false;
        m_out = top;
        begun = true;
        if (last && warp_live && wt.word(W_NOTED) == (uint32_t)u.no && live && !(joint && lane()))
          notes(tok + 1, inv, (((int64_t)u.c0 + tok) * a.Hkv * a.gq + u.h * a.gq + (r() - in * a.gq)) * D);
        return true;
      };
      const int end = joint ? u.tiles0 : n;
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        const int b = t % C::NB;
        if (!scored(b)) return;
        if (warp_live && !tile(b, t + 1 < n, visible, (t & seg) > 0, m, l)) return;
        tc5::fence_before();
        wt.arrive_warp(B_PREADY + lane() * C::NB + b);
        if (live) visible -= SHARED ? 2 * C::TN : C::TN;
        if (((t + 1) & seg) == 0 && t + 1 < end) {
          if (!summed(b, t + C::NB < n) || !store(false, true)) return;
          tc5::fence_before();
        }
      }
      for (int t = max(0, n - C::NB); t < n; ++t) {
        if (!summed(t % C::NB, false)) return;
        on ^= 1u << t % C::NB;
      }
      // lane 1's sums may have gone with a segment of lane 0's
      const bool rest = (u.tiles1 & seg) != 0 || u.tiles1 == u.tiles0;
      if (!store(true, rest)) return;
      tc5::fence_before();
      __threadfence_block();
      __syncwarp();
      if ((r() & 31) == 0) asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(wt.bars + 4 * W_EPI) : "memory");
    }
  }
};

// ------------------------------------------------------------------- kernel ---

template <int D, bool F32, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = ptx::smem_u32(smem_raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lid = tid & 31;
  const Waits wt = {smem + C::OFF_BAR, a.wait_limit_us};
  Unit* unit = reinterpret_cast<Unit*>(smem_raw + C::OFF_UNIT);
  if (smem & 1023u) {  // the swizzles count on it (a block without static shared memory has it)
    if (tid == 0) set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
    return;
  }
  if (warp == 8) {
    tc5::alloc(smem + C::OFF_BAR + 4 * W_TMEM, 512);
  } else if (warp == 9) {
    for (int i = lid; i < B_COUNT; i += 32) {
      int n = 1;  // arrivals of a phase
      if (i >= B_PREADY && i < B_PREADY + 4) n = 4;
      if (i >= B_SFULL && i < B_SFULL + 4) n = 1 + a.fault;
      if (i == B_UEMPTY) n = C::SMW + 3;
      if (i == B_JOIN) n = C::SMW;
      if (i >= B_KVEMPTY && i < B_KVEMPTY + kMaxStages) n = 2;
      ptx::mbar_init(smem + C::OFF_BAR + 8 * i, n);
    }
    if (lid == 0) {
      wt.set_word(W_ABORT, 0);
      wt.set_word(W_NOTED, 0);
      wt.set_word(W_EPI, 0);
    }
    ptx::fence_mbar_init();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, wt.word(W_TMEM), 0);
  wait_for_previous();

  // Registers: 168 a thread at launch (64512 in all) = 256 x 208 + 128 x 88.
  if (warp < 8) {
    tc5::regs_inc<208>();
    if (warp < C::SMW) {
      Soft<D, F32, SHARED> soft = {a, wt, smem, tmem + ((uint32_t)(warp & 3) << 21)};
      soft.run(unit);
    }
  } else {
    tc5::regs_dec<88>();
    if (warp == 8) mma_role<D, F32, SHARED>(wt, smem, tmem, unit);
    if (warp == 9) load_role<D, SHARED>(a, wt, smem, unit);
    if (warp == 10) check_role<D, F32, SHARED>(a, wt, smem, unit);
    if (warp == 11) unit_role<D, SHARED>(a, wt, smem, unit);
    __syncwarp();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (tid == 0 && wt.word(W_ABORT)) set_error(a.err_word, KVQ_ERRBIT_TIMEOUT);
  if (warp == 8) tc5::dealloc(tmem, 512);
}

template <int D, bool F32, bool SHARED>
cudaError_t launch_as(const PromptAttnArgs& a, int grid, cudaStream_t st) {
  static_assert(Cfg<D>::SMEM <= 227 * 1024, "shared memory of a block");
  auto kernel = prompt_attn_kernel<D, F32, SHARED>;
  // the kernel's attributes, once per device
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
    // the warps' shares (setmaxnreg) come out of what the block is launched with
    if (at.numRegs != 168) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_overlapped(kernel, dim3(grid), kThreads, Cfg<D>::SMEM, st, a);
}

template <int D>
cudaError_t launch(const PromptAttnArgs& a, int grid, cudaStream_t st) {
  if constexpr (Cfg<D>::LANES == 2)
    if (a.shared) return a.out_f32 ? launch_as<D, true, true>(a, grid, st) : launch_as<D, false, true>(a, grid, st);
  return a.out_f32 ? launch_as<D, true, false>(a, grid, st) : launch_as<D, false, false>(a, grid, st);
}

}  // namespace prompt
}  // namespace kvq
