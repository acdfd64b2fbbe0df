/*
 * kvq.h -- C ABI of the low-bit KV-cache library (libkvq.so).
 *
 * Attention over a key/value cache whose older tokens are stored as asymmetric
 * uniform INT4, INT3 or INT2 codes and whose most recent Nr tokens stay fp16 (and,
 * optionally, whose first tokens stay fp16 as an attention-sink window): single-token
 * decode, and runs of several tokens.
 *
 * Sources the operations follow (web pages on low-bit KV-cache decoding):
 *   - "Tensor Core accelerated low-bit KV cache decoding" (BitDecoding page),
 *     section 2.1: scale = (max - min) / (2^b - 1), code = round((K - min) / scale).
 *   - same page, section 2.2: residual partition, K_pack = KV[:L-Nr] quantized,
 *     K_res = KV[L-Nr:] kept fp16.
 *   - same page, section 2.3: GQA query regrouping, one KV read serves gq query heads.
 *   - same page, section 3.1: per-thread min/max, warp shuffle reduction, pack in registers.
 *   - same page, section 5.1: cache pointers aligned to 128 bytes.
 *   - "KV cache quantization InnerQ" page, section 2.1: groups of G = 32 along the
 *     inner (head_dim) dimension, one row shares its group parameters.
 *   - same page, section 2.2: hybrid mode, each group quantized symmetrically or
 *     asymmetrically, whichever reconstructs it better, with a 1-bit mode mask.
 *   - same page, section 2.3: recent-token window; a new token enters the window and,
 *     when the window is full, its oldest token is quantized into the main cache.
 *     Also the attention-sink window: the first tokens stay in full precision, set
 *     at prefill and fixed afterwards.
 *   - same page, section 3.1: dequantized value = scale * q + zero.
 *   - same page, section 3.2: 32 consecutive head_dim values packed together.
 *   - TurboQuant 3-bit article, section 3.1: eight 3-bit codes in 24 bits; section
 *     6.1: a paged cache of 32-token blocks.
 * The calls on runs of several tokens (kvq_append_chunk, kvq_chunk_attention,
 * kvq_cross_attention, kvq_read_tokens) and those around the cache (kvq_rotate,
 * kvq_prompt_attention, kvq_beam_select, kvq_reorder) are this library's additions.
 *
 * ---------------------------------------------------------------------------
 * Notation
 *   B   batch (sequences)             Hkv  KV heads        Hq  query heads (Hq % Hkv == 0)
 *   gq  = Hq / Hkv                    d    head_dim (multiple of 32, 32..256)
 *   G   = 32 group size along d       Ng   = d / 32 groups per token and head
 *   b   bits per code, 2, 3 or 4      Nr   fp16 residual window length (0..1024)
 *   cap packed-token capacity per (sequence, KV head)
 *   S   fp16 attention-sink window length (0..256)
 *   P   page size of a paged cache (0: contiguous, 32: paged), NP pages in its pool
 *
 * ---------------------------------------------------------------------------
 * Memory layout (all arrays are plain device memory owned by the caller; K and V
 * each have their own four arrays with identical shapes)
 *
 *   codes    uint8  [B][Hkv][cap][d*b/8]
 *            One token row holds d codes as a little-endian bit string: element
 *            e (0 <= e < d) occupies bits [e*b, e*b + b) of the row, so group g
 *            is the contiguous bytes [g*4*b, (g+1)*4*b): 16 bytes for INT4, 12 for
 *            INT3, 8 for INT2.
 *            INT4 byte k = c[2k] | c[2k+1] << 4.
 *            INT3: eight codes per 3 bytes, a code may straddle two bytes.
 *            INT2 byte k = c[4k] | c[4k+1] << 2 | c[4k+2] << 4 | c[4k+3] << 6.
 *            Paged caches (P = 32): codes, params and mode bytes live in a pool of
 *            NP pages, codes uint8 [NP][Hkv][32][d*b/8] (params, mode likewise); packed
 *            token t of sequence b, KV head h is row t % 32 of head h in page
 *            block_table[b][t / 32].  cap must be a multiple of 32.
 *   params   uint32 [B][Hkv][cap][Ng]
 *            One half2 per group: low 16 bits = scale (fp16), high 16 bits =
 *            min (fp16).  Dequantized value x^ = min + code * scale.
 *   residual fp16   [B][Hkv][Nr][d]
 *            Ring of the most recent tokens, kept in full precision.
 *   sink     fp16   [B][Hkv][S][d]
 *            The first sink_len[b] tokens of sequence b, kept in full precision.
 *   mode     uint8  [B][Hkv][cap]   (hybrid caches only)
 *            Bit g of a packed row's byte = mode of its group g: 1 asymmetric,
 *            0 symmetric.  Both modes dequantize as min + code * scale, so
 *            decode does not read it.
 *   block_table int32 [B][cap / 32]   (paged caches only): page of each 32 packed tokens.
 *   packed_len, res_len, res_head, sink_len   int32 [B]   (device)
 *            Per sequence: packed tokens, residual tokens, ring slot of the oldest
 *            residual token, sink tokens.  Sequence b attends over
 *            sink_len[b] + packed_len[b] + res_len[b] tokens.
 *   err_word uint32 (device, sticky bit set, see KVQ_ERRBIT_*)
 *
 * Every device pointer must be 16-byte aligned (KVQ_ERR_MISALIGNED otherwise);
 * 128-byte alignment is recommended.
 *
 * ---------------------------------------------------------------------------
 * Quantization rule, per (sequence, head, token, group) with fp16 inputs x_0..x_31
 *   Q1  mn = min_j x_j, mx = max_j x_j
 *   Q2  scale_f = ((float)mx - (float)mn) / (float)(2^b - 1)   fp32, round-to-nearest-even divide
 *   Q3  scale_h = fp16_rne(scale_f) (subnormals kept); min_h = fp16(mn + 0.0f) (-0 stored as +0)
 *   Q4  s = (float)scale_h; code_j = 0 if s == 0, else
 *       clamp(rint(((float)x_j - (float)mn) / s), 0, 2^b - 1)   fp32 subtract and divide,
 *       rint = round half to even
 *   Q5  pack as in the layout above
 * Hybrid caches (desc.hybrid = 1) replace Q1-Q4 per group by H1-H3:
 *   H1  symmetric candidate: a = max_j |x_j|, h = 2^(b-1), scale_s = fp16_rne(a / (h - 1))
 *       (fp32 divide), s = (float)scale_s, t_j = clamp(rint(x_j / s), -(h-1), h-1)
 *       (fp32 divide; 0 if s == 0), code = t_j + h, min_s = fp16(-h * s + 0.0f).
 *   H2  error of a candidate (fp32, each operation rounded, no fused multiply-add):
 *       e_j = x_j - (min + (float)code_j * scale); S_q = sum of e_j^2 over
 *       j = 8q .. 8q+7 in index order; E = (S_0 + S_1) + (S_2 + S_3).
 *   H3  the symmetric candidate is stored when min_s is finite and E_s < E_a; otherwise
 *       the asymmetric one (Q1-Q4).  Mode bit 0 = symmetric, 1 = asymmetric.
 *   Q6  with ns = min(S, L) and nr = min(Nr, L - ns): tokens [0, ns) are copied to the
 *       sink, tokens [ns, L - nr) are packed into slots [0, L - ns - nr), the last nr
 *       are copied to the residual ring in order, res_head = 0.
 *
 * Decode: O[b][hq] = softmax(q[b][hq] . K^T / sqrt(d)) V over the sink tokens, the
 * dequantized packed tokens and the residual tokens of KV head hq / gq, returned as fp16.
 *
 * ---------------------------------------------------------------------------
 * Conventions
 *   Ownership: the caller owns all memory and the stream.  The library allocates
 *     nothing and never synchronizes, except kvq_read_error and kvq_read_device_error.
 *   Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   Errors: argument errors return synchronously and launch nothing.  A failed
 *     launch returns KVQ_ERR_CUDA.  Data-dependent errors (capacity overflow, an
 *     empty sequence, a bounded wait that ran out) set bits in *err_word on the
 *     device; kvq_read_error reads and clears them.
 */
#ifndef KVQ_H_
#define KVQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1, /* a bad shape, a NULL pointer, a size mismatch */
  KVQ_ERR_UNSUPPORTED = 2, /* a valid but unsupported configuration (bits, d, gq) */
  KVQ_ERR_MISALIGNED = 3,  /* a device pointer that is not 16-byte aligned */
  KVQ_ERR_CAPACITY = 4,    /* a sequence does not fit in the packed capacity */
  KVQ_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed */
  KVQ_ERR_TIMEOUT = 6,     /* a bounded device-side wait ran out */
  KVQ_ERR_EMPTY = 7        /* decode over a sequence with no tokens */
} kvq_status;

/* Bits of *err_word (sticky until kvq_read_error clears them). */
#define KVQ_ERRBIT_CAPACITY 0x1u /* pack or append would pass cap; the token was dropped */
#define KVQ_ERRBIT_EMPTY 0x2u    /* decode saw a sequence with no tokens; output zeroed */
#define KVQ_ERRBIT_TIMEOUT 0x4u  /* a bounded wait gave up; that CTA wrote nothing */
#define KVQ_ERRBIT_BADLEN 0x8u   /* seq_lens[b] < 0 or > Lmax; that sequence was skipped */
#define KVQ_ERRBIT_BADPAGE 0x10u /* a block-table page outside [0, NP): pack/append wrote nothing
                                   there; decode output of that sequence is undefined */
#define KVQ_ERRBIT_BADPOS 0x20u  /* a position outside the rotation table; the nearest row was used */
#define KVQ_ERRBIT_BADINDEX 0x40u /* kvq_reorder: an index outside the source; that sequence was skipped */
#define KVQ_ERRBIT_BADSCORE 0x80u /* kvq_beam_select: NaN or +inf in a beam's logits or score; the beam
                                    proposed nothing */

/* Static description of one layer's cache.  group must be 32.  Every field is
 * significant: zero-initialise the struct (sink = 0 keeps no sink window). */
typedef struct {
  int32_t batch;        /* B   >= 1 */
  int32_t num_kv_heads; /* Hkv >= 1 */
  int32_t head_dim;     /* d: multiple of 32, 32..256 */
  int32_t bits;         /* b: 2, 3 or 4 */
  int32_t group;        /* G: 32 */
  int32_t capacity;     /* packed tokens per (sequence, KV head), >= 0 */
  int32_t residual;     /* Nr: 0..1024 */
  int32_t sink;         /* S: 0..256, first tokens kept fp16 (attention-sink window) */
  int32_t hybrid;       /* 0: asymmetric groups; 1: hybrid sym/asym groups with a mode mask */
  int32_t page_size;    /* P: 0 (contiguous) or 32 (paged) */
  int32_t num_pages;    /* NP: pages in the pool of a paged cache (ignored when P == 0) */
} kvq_cache_desc;

/* Device pointers of one layer's cache (layout above).  k_res/v_res may be NULL
 * when residual == 0, k_sink/v_sink/sink_len when sink == 0, k_mode/v_mode when
 * hybrid == 0. */
typedef struct {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint32_t* k_params;
  uint32_t* v_params;
  uint16_t* k_res; /* fp16 bits */
  uint16_t* v_res;
  int32_t* packed_len;
  int32_t* res_len;
  int32_t* res_head;
  uint32_t* err_word;
  uint16_t* k_sink; /* fp16 bits */
  uint16_t* v_sink;
  int32_t* sink_len;
  uint8_t* k_mode; /* mode bytes [B][Hkv][cap] */
  uint8_t* v_mode;
  int32_t* block_table; /* [B][cap / 32], paged caches only */
} kvq_cache_view;

/* Which array kvq_cache_bytes sizes (each of K and V has one of each). */
#define KVQ_ARRAY_CODES 0
#define KVQ_ARRAY_PARAMS 1
#define KVQ_ARRAY_RESIDUAL 2
#define KVQ_ARRAY_SINK 3
#define KVQ_ARRAY_MODE 4

/* Bytes of one array of the layout (for K or for V; allocate twice).  For a
 * paged cache the codes, params and mode arrays are sized for the page pool.
 * Returns 0 for an invalid desc or `which`. */
size_t kvq_cache_bytes(const kvq_cache_desc* desc, int which);

/* Bytes of scratch kvq_decode_attention and kvq_decode_step need for num_q_heads
 * query heads on the current device.  Returns 0 for an invalid desc. */
size_t kvq_decode_workspace_bytes(const kvq_cache_desc* desc, int32_t num_q_heads);

/* Quantize and pack a prefill (Q1-Q6; BitDecoding page section 2.1 for the rule,
 * section 2.2 for the residual split, section 3.1 for the warp-shuffle kernel;
 * InnerQ page section 2.1 for the grouping along head_dim).
 *   k, v      fp16 device [B][Hkv][Lmax][d], row-major.
 *   seq_lens  int32 device [B], 0 <= seq_lens[b] <= Lmax.
 *   Lmax      host int, >= 0.
 * For each sequence b with L = seq_lens[b], split as in Q6: the first min(S, L)
 * tokens are copied to the sink (InnerQ page section 2.3), the next ones become
 * codes and params in slots [0, ...), the last min(Nr, ...) are copied to the
 * residual ring; packed_len[b], res_len[b], res_head[b] = 0 and (S > 0)
 * sink_len[b] are written.  A hybrid cache quantizes by H1-H3 (InnerQ page
 * section 2.2) and writes each packed row's mode byte.
 * A sequence with more than cap packed tokens sets KVQ_ERRBIT_CAPACITY and stores
 * only the first cap (packed_len[b] = cap).  Asynchronous on `stream`. */
kvq_status kvq_quantize_pack(const kvq_cache_desc* desc, const kvq_cache_view* view,
                             const void* k, const void* v, const int32_t* seq_lens,
                             int32_t Lmax, void* stream);

/* kvq_quantize_pack reading K and V in the layout the prefill produced them, in
 * the same single pass (the quantizer reads each group straight from the
 * producer's memory; nothing is transposed or copied first).  Same rule,
 * split, outputs, errors and asynchrony as kvq_quantize_pack; only the input
 * addressing differs:
 *   element j of head_dim of token t, KV head h, sequence b of k (and of v) is
 *   k[b * stride_b + h * stride_h + t * stride_t + j]   (fp16, strides in elements),
 *   read for t < seq_lens[b] <= Lmax.
 * Head-major [B][Hkv][Lmax][d]: (Hkv*Lmax*d, Lmax*d, d) (kvq_quantize_pack).
 * Token-major [B][L][Hkv][d]: (L*Hkv*d, d, Hkv*d).
 * A fused QKV projection output [B][L][(Hq + 2*Hkv)*d] (queries, then keys, then
 * values of each token): k = base + Hq*d, v = base + (Hq + Hkv)*d, strides
 * (L*W, d, W) with W = (Hq + 2*Hkv)*d.
 * The strides must be non-negative multiples of 8 (KVQ_ERR_MISALIGNED
 * otherwise), k and v 16-byte aligned. */
kvq_status kvq_quantize_pack_strided(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                     const void* k, const void* v, const int32_t* seq_lens,
                                     int32_t Lmax, int64_t stride_b, int64_t stride_h,
                                     int64_t stride_t, void* stream);

/* Append one decode token per sequence (InnerQ page section 2.3, sliding recent
 * window).
 *   k_new, v_new  fp16 device [B][Hkv][d].
 * Per sequence: if res_len == Nr, the oldest residual token (ring slot res_head)
 * is quantized by Q1-Q5 into packed slot packed_len (which then grows by one)
 * and the new token takes its ring slot (res_head advances); otherwise the new
 * token goes to slot (res_head + res_len) % Nr and res_len grows.  With Nr == 0
 * the new token is packed directly (a hybrid cache by H1-H3, with its mode
 * byte).  The sink is never written: it stays as the
 * prefill left it.  A full packed cache sets KVQ_ERRBIT_CAPACITY and leaves that
 * sequence unchanged.  Asynchronous. */
kvq_status kvq_append(const kvq_cache_desc* desc, const kvq_cache_view* view,
                      const void* k_new, const void* v_new, void* stream);

/* Output element type of the decode calls (their `flags`): fp16 by default,
 * fp32 with KVQ_OUT_F32.  Both are rounded once from the fp32 result; fp16
 * rounding alone moves an output of magnitude 4 or more by up to 2^-9 * |O|. */
#define KVQ_OUT_F32 2u

/* Decode attention (BitDecoding page sections 2.2-2.3; InnerQ page section 3.1).
 *   q          fp16 device [B][Hq][d]; query head hq uses KV head hq / (Hq / Hkv).
 *   out        device [B][Hq][d], fp16 (or fp32 with KVQ_OUT_F32):
 *              softmax(q K^T / sqrt(d)) V over the sink, the packed tokens
 *              (dequantized as min + code * scale) and the residual.
 *   workspace  device scratch of ws_bytes >= kvq_decode_workspace_bytes(desc, Hq),
 *              16-byte aligned, zeroed before its first use.  Each completed call
 *              leaves it ready for the next call with the same batch, KV heads,
 *              head_dim and Hq (its counters and accumulators back at zero), so
 *              it is zeroed once, not per call; zero it again before a call with
 *              another shape and after a call that reported KVQ_ERR_TIMEOUT.
 *              One workspace serves one call at a time.
 *   flags      0 or KVQ_OUT_F32; other bits return KVQ_ERR_INVALID_ARG.
 * A sequence with no tokens gets a zero output and sets KVQ_ERRBIT_EMPTY.
 * Asynchronous; lengths are read on the device. */
kvq_status kvq_decode_attention(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                const void* q, int32_t num_q_heads, void* out,
                                void* workspace, size_t ws_bytes, uint32_t flags, void* stream);

/* One decode step of the serving loop: kvq_append(k_new, v_new) and then
 * kvq_decode_attention(q) over the cache as it is after the append (InnerQ page
 * section 2.3 for the window, BitDecoding page sections 2.2-2.3 for the
 * attention; fusing the two is this library's addition).
 *   q, out, workspace, ws_bytes, num_q_heads  as for kvq_decode_attention (the
 *              workspace size from kvq_decode_workspace_bytes covers this call).
 *   k_new, v_new  fp16 device [B][Hkv][d], as for kvq_append.
 * The cache bytes, counters and error bits afterwards are exactly those of the
 * two calls; the output equals the two calls' within rounding (the token packed
 * by this step is attended in fp32 from its codes rather than on the tensor
 * cores).  With head_dim 128 and at most 4 query heads per KV head this is one
 * kernel launch: the packed splits read only rows written before the step, the
 * split of each head that takes its fp16 rows (a split of its own, or in a
 * grid of several waves the last packed split) does the append's writes and
 * attends over the new and the packed token, and the counters move when the
 * last head of a sequence finishes.  Other shapes launch the append and the decode kernels in turn.  A
 * sequence whose packed cache is full is left unchanged, sets
 * KVQ_ERRBIT_CAPACITY and is attended as it was.
 *   flags      0, or KVQ_STEP_EARLY_CACHE_READ: the caller states that the
 *              kernel enqueued on `stream` just before this call does not write
 *              this cache (any array of its view, counters included) -- in a serving loop
 *              it computes q, k_new and v_new, and the cache was last written by
 *              this layer's previous step.  What earlier kernels wrote is seen (a
 *              kvq_reorder into this cache two kernels before, say; one just before
 *              rules the flag out).  The step (launched as a programmatic
 *              dependent of that kernel) then reads the counters and cuts its
 *              ranges before it waits for that kernel, and starts its copies the
 *              moment the wait returns; q, k_new and v_new are read, and anything
 *              is written, only after the wait.
 *              Without the flag nothing is read before the wait.  KVQ_OUT_F32
 *              may be or'ed in (fp32 out).  Other bits return KVQ_ERR_INVALID_ARG.
 * Asynchronous. */
#define KVQ_STEP_EARLY_CACHE_READ 1u
kvq_status kvq_decode_step(const kvq_cache_desc* desc, const kvq_cache_view* view,
                           const void* q, int32_t num_q_heads, const void* k_new,
                           const void* v_new, void* out, void* workspace, size_t ws_bytes,
                           uint32_t flags, void* stream);

/* Bytes of device staging kvq_decode_step_host needs: the packed input
 * [q | k_new | v_new] (fp16, in that order, no padding) and, at the next
 * 256-byte boundary, out (room for an fp32 out).  Returns 0 for an invalid desc
 * or head count. */
size_t kvq_step_io_bytes(const kvq_cache_desc* desc, int32_t num_q_heads);

/* kvq_decode_step with its inputs and output in host memory (no passage of the
 * pages corresponds to it; it is this library's serving-loop entry point).
 *   in_host    host [q (B*Hq*d) | k_new (B*Hkv*d) | v_new (B*Hkv*d)] fp16, the
 *              layouts of kvq_decode_step, contiguous in that order.
 *   out_host   host [B][Hq][d], fp16 (fp32 with KVQ_OUT_F32 in flags).
 *   dev_io     device staging of dev_io_bytes >= kvq_step_io_bytes(desc, Hq),
 *              256-byte aligned, owned by the caller.
 * Enqueues on `stream`: one host-to-device copy of the input block, the step
 * (as kvq_decode_step with the same workspace and flags, less
 * KVQ_STEP_EARLY_CACHE_READ: the step follows the copy, so there is nothing to
 * overlap), and one device-to-host copy of out.  Asynchronous when the host
 * buffers are pinned (page-locked), in which case they must stay valid until
 * the stream reaches the copies; with pageable memory the copies are
 * synchronous.  Argument errors return before anything is enqueued.
 *   flags | KVQ_STEP_HOST_MAPPED: in_host and out_host are page-locked host
 *              memory the device addresses with the same pointer (cudaHostAlloc,
 *              or registered with mapping; checked with cudaPointerGetAttributes,
 *              KVQ_ERR_INVALID_ARG otherwise).  No copy is enqueued: the step
 *              kernel reads the input block and writes out in place over the
 *              host link (NVLink-C2C on Grace hosts), dev_io is unused (may be
 *              NULL), and KVQ_STEP_EARLY_CACHE_READ keeps its meaning (the
 *              kernel before this call is the one it overlaps).  The buffers
 *              must stay valid until the step completes. */
#define KVQ_STEP_HOST_MAPPED 4u
kvq_status kvq_decode_step_host(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                const void* in_host, int32_t num_q_heads, void* out_host,
                                void* dev_io, size_t dev_io_bytes, void* workspace,
                                size_t ws_bytes, uint32_t flags, void* stream);

/* Size of the device scratch array behind kvq_decode_attention_noalloc (8 MiB). */
#define KVQ_NOALLOC_SCRATCH_BYTES (8u << 20)

/* Decode attention without any caller-provided scratch, for callers that cannot
 * allocate device memory when they decode (a runtime that forbids cudaMalloc in
 * its serving loop, an allocator the caller does not own, memory fixed at start
 * up).  No passage of the pages corresponds to this call; it is an addition of
 * this library.
 * Same arguments (flags included), output and error bits as
 * kvq_decode_attention, minus the workspace: the split partials go to one static device array of
 * KVQ_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until the
 * process exits.  Returns KVQ_ERR_UNSUPPORTED when the decode would need more
 * than that (kvq_decode_workspace_bytes(desc, num_q_heads) > the maximum) and
 * KVQ_ERR_INVALID_ARG for an invalid description or head count.  Allocates
 * nothing.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call before
 * any stream capture.  All calls share the array and it keeps the last call's
 * contents (its counters back at zero).  The first call on a device, a call whose
 * cache shape or head count differs from the previous call's there, and the
 * first call after kvq_read_error reported KVQ_ERR_TIMEOUT first clear the
 * array's counters and accumulators with cudaMemsetAsync on `stream`, so that
 * clear is ordered before the decode on the caller's own stream.  Calls whose
 * kernels overlap on the GPU race: keep them on one stream or order the
 * streams. */
kvq_status kvq_decode_attention_noalloc(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                        const void* q, int32_t num_q_heads, void* out,
                                        uint32_t flags, void* stream);

/* ---------------------------------------------------------------------------
 * Runs of several tokens.  The calls below take, for each sequence, a run of
 * consecutive tokens: the drafts of a speculative step, a piece of a prompt, a
 * decoder's prompt over encoder states.  Runs are ragged and concatenated:
 *   cu_seqlens  int32 device [B + 1], nondecreasing, cu_seqlens[0] >= 0; the run of
 *               sequence b is rows [cu_seqlens[b], cu_seqlens[b + 1]) of the
 *               token-major inputs and outputs.  A run may be empty.
 *   total       rows those arrays have (cu_seqlens[B] <= total).  Rows of no
 *               run are not written and have no part in any result.
 *   max_len     host upper bound of the run lengths, >= 0.
 * A sequence whose entries are not 0 <= cu[b] <= cu[b+1] <= total with at most
 * max_len tokens is skipped and sets KVQ_ERRBIT_BADLEN; the others are served.  A row
 * that two of them have (entries out of order) counts for both; its output is either's
 * (queries rotated in place: undefined). */

/* Arguments of kvq_append_chunk; zero-initialise the struct. */
typedef struct {
  const void* k;           /* fp16 device: element j of head h of row t at */
  const void* v;           /*   t * kv_stride_token + h * kv_stride_head + j */
  int64_t kv_stride_token; /* in elements, non-negative multiples of 8 */
  int64_t kv_stride_head;
  const void* q;           /* fp16 device queries to rotate, or NULL */
  void* q_out;             /* fp16 device [total][Hq][d]; may be q itself when q is
                              contiguous, and overlaps no input otherwise */
  int64_t q_stride_token;
  int64_t q_stride_head;
  int32_t num_q_heads;     /* Hq (read only with q) */
  const int32_t* cu_seqlens;
  int32_t total;
  int32_t max_len;
  const float* rope;       /* fp32 device [rope_rows][rotary_dim / 2][2]: cos, sin of each
                              position and pair; NULL when rotary_dim == 0 */
  int32_t rope_rows;
  int32_t rotary_dim;      /* leading elements of a head that are rotated: a multiple of 16,
                              0..head_dim (0: keys and queries are taken as they are) */
  int32_t interleaved;     /* pairs: 0 (i, i + rotary_dim / 2), 1 (2i, 2i + 1) */
  const int32_t* positions; /* int32 device [total], or NULL: token i of a run is at the
                              number of tokens its sequence held before the call + i */
} kvq_append_args;

/* Append a run of tokens to each sequence, rotating keys and queries to their
 * positions on the way.
 *   R1  a pair (a, b) at table entry (c, s) becomes fp16_rne(a*c - b*s) and
 *       fp16_rne(b*c + a*s): fp32 products and one fp32 sum or difference, each
 *       rounded to nearest even (no fused multiply-add).  Elements from
 *       rotary_dim on, and values, are unchanged.
 *   R2  the rotated keys and the values enter the cache exactly as successive
 *       kvq_append calls of one token each would leave it: cache bytes, ring
 *       slots, counters and KVQ_ERRBIT_CAPACITY (tokens that no longer fit are
 *       dropped).  The sink is never written.
 *   R3  with q, q_out[t] is row t's queries rotated to the same position; rows of
 *       dropped tokens included.
 * A position outside [0, rope_rows) sets KVQ_ERRBIT_BADPOS and uses the nearest
 * row.  One launch for the shortest runs (a block per sequence), two otherwise (the
 * counters move in the second).  Asynchronous; needs no workspace. */
kvq_status kvq_append_chunk(const kvq_cache_desc* desc, const kvq_cache_view* view,
                            const kvq_append_args* args, void* stream);

/* Bytes of scratch kvq_chunk_attention and kvq_cross_attention need for
 * num_q_heads query heads on the current device (any run lengths).  Returns 0
 * for an invalid desc or head count. */
size_t kvq_chunk_workspace_bytes(const kvq_cache_desc* desc, int32_t num_q_heads);

/* Causal attention of each sequence's newest tokens over its cache: the run of
 * sequence b is its last T_b tokens (appended before the call), and token i of
 * it attends over the first N_b - T_b + i + 1 of the sequence's N_b = sink_len +
 * packed_len + res_len tokens, in the form in which the cache holds them.
 *   q          fp16 device [total][Hq][d], 16-byte aligned (rotated, where positions are).
 *   out        device [total][Hq][d], fp16 (fp32 with KVQ_OUT_F32 in flags), rounded
 *              once from the fp32 result; overlaps no input.
 *   workspace  device scratch of ws_bytes >= kvq_chunk_workspace_bytes(desc, Hq),
 *              16-byte aligned; whatever it holds, each call writes what it reads.
 *              One workspace serves one call at a time.
 *   flags      0 or KVQ_OUT_F32; other bits return KVQ_ERR_INVALID_ARG.
 * A row with no token to attend over gets zeros and sets KVQ_ERRBIT_EMPTY.
 * Keys, values and weights are rounded to fp16 once each (operands of the tensor
 * cores; weights below 2^-21 of a row's largest by at most 2^-32 of that), scores and
 * sums are fp32; results do not depend on timing.  A value past
 * fp16's range by the rounding of its scale counts as fp16's largest.
 * Tokens a row does not attend over have no part in its output, whatever they
 * hold.  Tokens in a page outside the pool are left out (KVQ_ERRBIT_BADPAGE).
 * With one token for every sequence kvq_decode_attention is the faster call at
 * head_dim 128 with at most 4 query heads per KV head (16 sequences of 4096 tokens, 32
 * heads on 8, INT4: 40 against 66 us; one of 32768: 21 against 44) and this one for most
 * other shapes (head_dim 64, 16 sequences of 1500 tokens, 16 heads: 50 against 95 us).
 * Asynchronous; lengths are read on the device. */
kvq_status kvq_chunk_attention(const kvq_cache_desc* desc, const kvq_cache_view* view,
                               const void* q, int32_t num_q_heads, const int32_t* cu_seqlens,
                               int32_t total, int32_t max_len, void* out, void* workspace,
                               size_t ws_bytes, uint32_t flags, void* stream);

/* kvq_chunk_attention without the mask: every row of sequence b's run attends
 * over all N_b cached tokens (cross attention of decoder tokens to an encoder's
 * states, packed by kvq_quantize_pack; run and cache lengths are unrelated). */
kvq_status kvq_cross_attention(const kvq_cache_desc* desc, const kvq_cache_view* view,
                               const void* q, int32_t num_q_heads, const int32_t* cu_seqlens,
                               int32_t total, int32_t max_len, void* out, void* workspace,
                               size_t ws_bytes, uint32_t flags, void* stream);

/* Read tokens back as the values they stand for.
 *   first      int32 device [B]: first token of each sequence, in the order sink,
 *              packed, residual (oldest first); NULL reads from token 0.
 *   count      tokens per sequence, >= 0.
 *   k_out, v_out  device [B][Hkv][count][d] (the layout kvq_quantize_pack takes), fp16,
 *              or fp32 with KVQ_OUT_F32 in flags; row j of sequence b is token
 *              first[b] + j.  Packed values are min + code * scale in fp32, rounded
 *              once to the output type; sink and residual values are exact.
 * Rows past a sequence's end are zero.  A negative first[b] sets
 * KVQ_ERRBIT_BADLEN and gives that sequence zero rows; a page outside the pool
 * sets KVQ_ERRBIT_BADPAGE and gives its tokens zero rows.  Asynchronous. */
kvq_status kvq_read_tokens(const kvq_cache_desc* desc, const kvq_cache_view* view,
                           const int32_t* first, int32_t count, void* k_out, void* v_out,
                           uint32_t flags, void* stream);

/* ---------------------------------------------------------------------------
 * Around the cache: a generation from prompts of text and images, with beams.
 *   prompt   kvq_rotate (queries and keys to their positions), kvq_prompt_attention (their
 *            attention in full precision), kvq_quantize_pack_strided (keys and values into
 *            the cache; all three read and write the columns of a fused projection's
 *            output in place), kvq_reorder (one cached prompt to all its beams)
 *   token    kvq_rotate, kvq_decode_step, kvq_beam_select, kvq_reorder
 * Where a call takes an err_word (a cache's, or any zeroed device word) and it is NULL, its
 * bits go to a word that the library keeps for the current device: kvq_read_device_error. */

/* Arguments of kvq_rotate; zero-initialise the struct. */
typedef struct {
  const void* q;           /* fp16 device: element j of head h of row t at */
  const void* k;           /*   t * stride_token + h * stride_head + j; q or k may be NULL */
  void* q_out;             /* fp16 device, by strides of its own; may be q itself with the */
  void* k_out;             /*   same strides, and overlaps no input otherwise */
  int64_t q_stride_token;  /* in elements, non-negative multiples of 8 */
  int64_t q_stride_head;
  int64_t k_stride_token;
  int64_t k_stride_head;
  int64_t q_out_stride_token; /* (positive where there is more than one row or head) */
  int64_t q_out_stride_head;
  int64_t k_out_stride_token;
  int64_t k_out_stride_head;
  int32_t num_q_heads;     /* (read only with q) */
  int32_t num_kv_heads;    /* (read only with k) */
  int32_t head_dim;        /* 32, 64, 128 or 256 */
  int32_t total;           /* rows */
  const float* rope;       /* fp32 device [rope_rows][rotary_dim / 2][2]: cos, sin */
  int32_t rope_rows;
  int32_t rotary_dim;      /* leading elements that are rotated: a multiple of 16, 16..head_dim */
  int32_t interleaved;     /* pairs: 0 (i, i + rotary_dim / 2), 1 (2i, 2i + 1) */
  int32_t axes;            /* 1..4 */
  const int32_t* positions; /* int32 device [axes][total] */
  const uint8_t* pair_axis; /* HOST [rotary_dim / 2]: the axis of each pair (NULL: axis 0);
                               read during the call */
  uint32_t* err_word;      /* device, or NULL: the device's own word */
} kvq_rotate_args;

/* Rotate queries and keys to positions on several axes (time, height and width of the
 * patches of images and video; text has the same position on each).  Pair i of row t is
 * rotated by R1 (kvq_append_chunk's rule, with the same roundings) at
 * rope[positions[pair_axis[i]][t]][i]; elements from rotary_dim on are copied.  With one
 * axis the result is the append's, bit for bit: keys rotated here enter the cache by
 * kvq_quantize_pack_strided, kvq_append or kvq_append_chunk without a table.
 * A position outside [0, rope_rows) sets KVQ_ERRBIT_BADPOS and uses the nearest row.
 * Asynchronous. */
kvq_status kvq_rotate(const kvq_rotate_args* args, void* stream);

/* Arguments of kvq_prompt_attention; zero-initialise the struct. */
typedef struct {
  const void* q;           /* fp16 device: element j of head h of row t at */
  const void* k;           /*   t * stride_token + h * stride_head + j */
  const void* v;
  int64_t q_stride_token;  /* in elements, positive multiples of 8 (where there is more than */
  int64_t q_stride_head;   /*   one row or head), below 2^32 */
  int64_t k_stride_token;
  int64_t k_stride_head;
  int64_t v_stride_token;
  int64_t v_stride_head;
  int32_t num_q_heads;     /* Hq, at most 128 Hkv */
  int32_t num_kv_heads;    /* Hkv */
  int32_t head_dim;        /* 32, 64, 128 or 256 */
  int32_t batch;           /* B, at most 2^20 */
  const int32_t* cu_seqlens; /* as for the calls on runs: prompt b is rows */
  int32_t total;           /*   [cu_seqlens[b], cu_seqlens[b + 1]) of q, k, v and out (at most 2^30) */
  int32_t max_len;
  void* out;               /* device [total][Hq][d], fp16 (fp32 with KVQ_OUT_F32); overlaps no input */
  uint32_t flags;          /* 0 or KVQ_OUT_F32 */
  uint32_t* err_word;      /* device, or NULL: the device's own word */
} kvq_prompt_args;

/* Causal attention over whole prompts in full precision (before the cache is packed):
 * row i of a prompt attends over its rows 0..i, query head hq over KV head hq / (Hq / Hkv):
 *   out[i] = sum_j softmax_j(q[i] . k[j] / sqrt(d)) v[j],  j <= i.
 * Weights are rounded to fp16 once (operands of the tensor cores; weights below 2^-21 of a
 * row's largest by at most 2^-32 of that), with KVQ_OUT_F32 they are two fp16 parts (22 bits);
 * scores and sums are fp32, the output is rounded once.  The tensor cores cut their sums off
 * (2^-23 a step of 16 tokens, towards zero): fp32 output is within 2.3e-5 of the sums of
 * values of one sign and about 1e-6 of others, whatever the length.  Results do not depend
 * on timing; the order of a row's sums goes by how many blocks of rows there can be (total,
 * batch and heads), so that a prompt may differ in its last bits from the same one in
 * another batch.  Tokens a row does not attend over, other prompts' among them, have no part in
 * its output, whatever they hold.  An infinite value that it attends over makes its element of the
 * output infinite, or NaN beside one of the other sign or NaN (with fp16 output also where the
 * value's weight rounds to zero, below 2^-32 of the largest).  Entries of cu_seqlens that break the rule set
 * KVQ_ERRBIT_BADLEN (where they let prompts overlap, some may stay unwritten).
 * The waits inside are bounded, by a second of wall time each (a GPU that is held up for that long
 * counts too): KVQ_ERRBIT_TIMEOUT says that one ran out, and rows of the output are then wrong.
 * Asynchronous; lengths are read on the device. */
kvq_status kvq_prompt_attention(const kvq_prompt_args* args, void* stream);

/* Arguments of kvq_beam_select; zero-initialise the struct. */
typedef struct {
  const void* logits;      /* device: token t of row r at r * stride_row + t, rows at any place;
                              fp16, or fp32 with KVQ_LOGITS_F32.  Row b * beams + w is beam w
                              of batch entry b */
  int64_t stride_row;      /* in elements, >= vocab */
  const float* scores;     /* fp32 device [batch * beams]: the beams' sums of log-probabilities */
  const uint8_t* finished; /* device [batch * beams], non-zero: the beam is complete; or NULL */
  int32_t batch;           /* at most 65535 rows in all */
  int32_t beams;           /* W, 1..32 */
  int32_t vocab;           /* V, W V < 2^31 - 1 */
  int32_t n;               /* selected per batch entry: 1..32, at most W V */
  int32_t end_token;       /* what a complete beam goes on with, 0..V-1 (read only with finished) */
  uint32_t flags;          /* 0 or KVQ_LOGITS_F32 */
  int32_t* parent;         /* device [batch][n]: row of the beam (an index for kvq_reorder); the */
                           /*   outputs overlap no input and not each other */
  int32_t* token;          /* device [batch][n] */
  float* score;            /* device [batch][n] */
  void* workspace;         /* device, 16-byte aligned, ws_bytes >= kvq_beam_workspace_bytes;
                              whatever it holds, each call writes what it reads; one call at a time */
  size_t ws_bytes;
  uint32_t* err_word;      /* device, or NULL: the device's own word */
} kvq_beam_args;

#define KVQ_LOGITS_F32 1u

/* Bytes of scratch kvq_beam_select needs (0 for invalid arguments). */
size_t kvq_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t n);

/* Beam search's selection.  Beam w proposes token t with the score
 *   scores[w] + x[t] - log sum_u exp(x[u]),   x its logits;
 * a complete beam proposes end_token alone, at scores[w].  For each batch entry the n
 * best proposals, best first; those of one beam in the order of their logits, equal logits in
 * that of their tokens, and equal scores of two beams in the order of the beams.  (Where a score
 * is so far from zero that its last bit is more than the logits differ by, as at the type's
 * lowest value, the logits still decide within a beam.)  What is not proposed
 * (logits of -inf, other tokens of complete beams, beams with a score of -inf) counts as a
 * score of -inf, so n entries always come back.
 * A beam with a NaN or +inf among its logits, or as its score, proposes nothing and sets
 * KVQ_ERRBIT_BADSCORE (a complete beam's logits are not looked at).
 * The sums of exponentials are fp32 (within 2^-20 of the whole) and so are their logarithms:
 * a beam's normaliser, the same for all that it proposes, is within 2^-19, and proposals of two
 * beams that are nearer to each other than twice that may come in either order.  Scores are
 * compared as pairs of fp32 numbers, cut to 53 bits; they are rounded to fp32 once, and one
 * below fp32's range is -inf.  Beams of equal logits and scores have equal scores to the
 * last bit; results do not depend on timing.  Asynchronous. */
kvq_status kvq_beam_select(const kvq_beam_args* args, void* stream);

/* Copy sequences from one cache to another: sequence i of `dst` becomes sequence index[i]
 * of `src` (beams after a selection, a prompt to its beams, a batch to a larger cache).
 *   index      int32 device [dst_desc.batch]; entries may repeat.
 * The caches have the same heads, head_dim, bits, residual, sink, hybrid and page_size;
 * batch, capacity and pages may differ.  Only live bytes move: packed rows (codes, params,
 * modes), the window's tokens (in the same ring slots), the sink's, the counters.
 * Other bytes of dst stay as they are.  dst's arrays are not src's (the pools of two
 * paged caches may be one, with pages of their own in each table); paged, dst's table
 * has pages for the tokens that it gets.
 *   flags      0, or KVQ_REORDER_SHARE_PAGES (paged caches over one pool): full pages do
 *              not move; dst's table entries for them become the source's.  The page
 *              that is being filled is copied to the page in dst's own table, so that
 *              each sequence appends to a page of its own.  With two tables that take
 *              turns, each with own pages for the tokens to come, a page is never
 *              written again once it is full.
 * An index outside src sets KVQ_ERRBIT_BADINDEX, more packed tokens than dst's capacity
 * KVQ_ERRBIT_CAPACITY; such a sequence stays as it was.  A page outside the pool sets
 * KVQ_ERRBIT_BADPAGE and its tokens are not copied.  (Bits go to dst's err_word.)
 * Asynchronous; lengths and indices are read on the device. */
#define KVQ_REORDER_SHARE_PAGES 1u
kvq_status kvq_reorder(const kvq_cache_desc* dst_desc, const kvq_cache_view* dst,
                       const kvq_cache_desc* src_desc, const kvq_cache_view* src,
                       const int32_t* index, uint32_t flags, void* stream);

/* Synchronize `stream`, copy *err_word to *word_out (may be NULL), clear it, and
 * return KVQ_OK if it was 0, else the status of its lowest set bit. */
kvq_status kvq_read_error(const kvq_cache_view* view, uint32_t* word_out, void* stream);

/* The same for the bits of calls on the current device, of any stream, that were given no
 * err_word: what they set before `stream` gets here (and, of other streams, perhaps later). */
kvq_status kvq_read_device_error(uint32_t* word_out, void* stream);

/* Static text for a status code. */
const char* kvq_status_string(kvq_status status);

/* Library version as 10000 * major + 100 * minor + patch. */
int32_t kvq_version(void); /* 160: two-part weights in the tensor-core MMAs, MMA rounding hook
                              (and, under the same number, the calls on runs and BADPOS,
                              then the calls around the cache, BADINDEX and BADSCORE);
                              150: timeout testing hook, cached tensor maps; 140: paged caches;
                              130: 3-bit; 120: hybrid; 110: sink, fp32 out */

/* Testing hook, for checking the bounded-wait error path without faulting the
 * GPU (no passage of the pages corresponds to it).  With limit_us > 0, every
 * later tensor-core decode call (kvq_decode_attention, kvq_decode_step with
 * head_dim 128 and at most 4 query heads per KV head, and the calls built on
 * them) arms the barrier of the first tile of split 0 of (sequence 0, KV head 0)
 * for 16 bytes more than that tile's copies deliver, and gives every bounded
 * wait a limit of limit_us microseconds instead of one second.  All copies still
 * complete, so nothing is in flight when that CTA gives up: it sets
 * KVQ_ERRBIT_TIMEOUT, contributes nothing to its head's output (which is then
 * wrong for that head) and returns; the call's other results are unaffected.
 * kvq_chunk_attention, kvq_cross_attention and kvq_prompt_attention give the barriers of their scores an
 * arrival that never comes: every block gives up, with nothing in flight, and the
 * output is wrong.
 * limit_us = 0 (the default) restores normal behaviour.  Process-wide; not for
 * production use. */
void kvq_testing_wait_fault(uint32_t limit_us);

/* Testing hook (no passage of the pages corresponds to it): exhaustive checks,
 * on the current device, of the quantizer's fast arithmetic against the IEEE
 * operations it replaces.  div_mismatches[2i], [2i + 1] (i = 0, 1, 2 for the
 * divisors 2^b - 1 = 15, 7, 3): how many non-negative finite floats d give a
 * quotient d / (2^b - 1) other than the IEEE divide's, in all and in the
 * quantizer's domain (0 and the differences of fp16 values, 2^-24 .. 131008);
 * rcp_worst_rel: the largest relative error of the reciprocal used for the codes,
 * over every positive finite fp16 scale.  Synchronous (legacy default stream). */
kvq_status kvq_testing_check_arithmetic(uint64_t* div_mismatches, double* rcp_worst_rel);

/* Testing hook (no passage of the pages corresponds to it): how the tensor
 * cores round the f16 -> f32 MMA that the decode kernel's contractions use.
 * Runs eight fixed cases of one mma.sync m16n8k16, each C = c0 plus one product
 * `big` and fifteen products `small` (small in units of the float spacing at 1,
 * 2^-23): (c0, big, small) = (0, 1, 1/2), (0, 1, 1/4), (0, 1, 1/8),
 * (0, 1, 1/16), (1, 0, 1/2), (1, 0, 1/4), (0, 1, -1/2), (0, 1, -1/4), and
 * writes the first n (<= 8) results to the host array out.  Synchronous (legacy
 * default stream).  KVQ_ERR_INVALID_ARG for a null out or n outside 0..8. */
kvq_status kvq_testing_mma_rounding(float* out, int32_t n);

/* Testing hook (no passage of the pages corresponds to it): where kvq_prompt_attention
 * finds its units of work, on the current device.  A unit is a KV head of `tokens` tokens
 * of a prompt; they lie in one line, prompt after prompt (cu_seqlens, batch, total and
 * max_len as there), the last tokens first, heads within them.  For unit order[i] >= 0,
 * in any order, units[4 i ..] gets the prompt's first row and length, the head and the
 * first token, or -1, 0, 0, 0 where there are fewer.  cu_seqlens, order [n] and units (16-byte
 * aligned) are device arrays.  Synchronous (legacy default stream). */
kvq_status kvq_testing_prompt_units(const int32_t* cu_seqlens, int32_t batch, int32_t total, int32_t max_len,
                                    int32_t heads, int32_t tokens, const int32_t* order, int32_t n,
                                    int32_t* units);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H_ */
