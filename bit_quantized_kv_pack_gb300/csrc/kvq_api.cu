// kvq_api.cu -- the C ABI of libkvq.so: argument checks, launch, status codes.
// Every entry point validates on the host and launches nothing on an error.
#include <string.h>

#include <atomic>
#include <mutex>

#include "kvq_around.cuh"
#include "kvq_runs.cuh"

namespace {

using kvq::Dims;

// A device's word for the errors of calls that are given none, and where it is read through.
__device__ uint32_t g_err_word;
__device__ uint32_t g_err_taken;

__global__ void take_errors_kernel() { g_err_taken = atomicExch(&g_err_word, 0u); }

// The word of the current device (a symbol's address, looked up once for each).
kvq_status device_err_word(uint32_t** word) {
  static std::atomic<uint32_t*> words[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  uint32_t* w = dev < 64 ? words[dev].load(std::memory_order_acquire) : nullptr;
  if (!w) {
    if (cudaGetSymbolAddress(reinterpret_cast<void**>(&w), g_err_word) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ERR_CUDA;
    }
    if (dev < 64) words[dev].store(w, std::memory_order_release);
  }
  *word = w;
  return KVQ_OK;
}

// An error word's status: that of its lowest set bit.
kvq_status status_of(uint32_t w) {
  if (w & KVQ_ERRBIT_CAPACITY) return KVQ_ERR_CAPACITY;
  if (w & KVQ_ERRBIT_EMPTY) return KVQ_ERR_EMPTY;
  if (w & KVQ_ERRBIT_TIMEOUT) return KVQ_ERR_TIMEOUT;
  if (w & (KVQ_ERRBIT_BADLEN | KVQ_ERRBIT_BADPAGE | KVQ_ERRBIT_BADPOS | KVQ_ERRBIT_BADINDEX |
           KVQ_ERRBIT_BADSCORE))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

kvq_status check_desc(const kvq_cache_desc* D) {
  if (!D) return KVQ_ERR_INVALID_ARG;
  if (D->batch < 1 || D->num_kv_heads < 1 || D->capacity < 0 || D->residual < 0 ||
      D->group != kvq::kGroup || D->head_dim < 32 || D->head_dim % 32 != 0)
    return KVQ_ERR_INVALID_ARG;
  if (D->bits < 2 || D->bits > 4) return KVQ_ERR_UNSUPPORTED;
  if (D->head_dim != 32 && D->head_dim != 64 && D->head_dim != 128 && D->head_dim != 256)
    return KVQ_ERR_UNSUPPORTED;
  if (D->sink < 0 || (D->hybrid != 0 && D->hybrid != 1)) return KVQ_ERR_INVALID_ARG;
  if (D->page_size != 0 && D->page_size != kvq::kPage) return KVQ_ERR_UNSUPPORTED;
  if (D->page_size && (D->capacity % kvq::kPage != 0 || D->num_pages < 0 ||
                       (D->capacity > 0 && D->num_pages < 1)))
    return KVQ_ERR_INVALID_ARG;
  if (D->residual > 1024 || D->sink > 256) return KVQ_ERR_UNSUPPORTED;
  if ((int64_t)D->batch * D->num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq_status check_view(const kvq_cache_desc& D, const kvq_cache_view* v) {
  if (!v) return KVQ_ERR_INVALID_ARG;
  if (!v->packed_len || !v->res_len || !v->res_head || !v->err_word) return KVQ_ERR_INVALID_ARG;
  if (D.capacity > 0 && (!v->k_codes || !v->v_codes || !v->k_params || !v->v_params))
    return KVQ_ERR_INVALID_ARG;
  if (D.residual > 0 && (!v->k_res || !v->v_res)) return KVQ_ERR_INVALID_ARG;
  if (D.sink > 0 && (!v->k_sink || !v->v_sink || !v->sink_len)) return KVQ_ERR_INVALID_ARG;
  if (D.hybrid && D.capacity > 0 && (!v->k_mode || !v->v_mode)) return KVQ_ERR_INVALID_ARG;
  if (D.page_size && D.capacity > 0 && !v->block_table) return KVQ_ERR_INVALID_ARG;
  const void* a16[] = {v->k_codes, v->v_codes, v->k_params, v->v_params, v->k_res,
                       v->v_res,   v->k_sink,   v->v_sink,   v->k_mode,   v->v_mode};
  for (const void* p : a16)
    if (!aligned(p, 16)) return KVQ_ERR_MISALIGNED;
  const void* a4[] = {v->packed_len, v->res_len, v->res_head, v->err_word, v->sink_len,
                      v->block_table};
  for (const void* p : a4)
    if (!aligned(p, 4)) return KVQ_ERR_MISALIGNED;
  return KVQ_OK;
}

kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

constexpr uint32_t kStepFlags = KVQ_STEP_EARLY_CACHE_READ | KVQ_OUT_F32;

// A page-locked host buffer the device addresses with the same pointer (the
// allocation registered with the driver, mapped, and the device pointer equal).
bool host_mapped(const void* p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeHost && at.devicePointer == p && at.hostPointer == p;
}

}  // namespace

extern "C" {

size_t kvq_cache_bytes(const kvq_cache_desc* desc, int which) {
  if (check_desc(desc) != KVQ_OK) return 0;
  const Dims s = kvq::dims_of(*desc);
  const size_t rows = (size_t)s.B * s.Hkv;
  // packed rows: every (sequence, head, slot), or every (page, head, slot) of the pool
  const size_t prow = s.page ? (size_t)s.npages * s.Hkv * s.page : rows * (size_t)s.cap;
  switch (which) {
    case KVQ_ARRAY_CODES: return prow * s.row_bytes;
    case KVQ_ARRAY_PARAMS: return prow * s.Ng * sizeof(uint32_t);
    case KVQ_ARRAY_RESIDUAL: return rows * (size_t)s.Nr * s.d * sizeof(uint16_t);
    case KVQ_ARRAY_SINK: return rows * (size_t)s.Ns * s.d * sizeof(uint16_t);
    case KVQ_ARRAY_MODE: return s.hybrid ? prow : 0;
    default: return 0;
  }
}

size_t kvq_decode_workspace_bytes(const kvq_cache_desc* desc, int32_t num_q_heads) {
  if (check_desc(desc) != KVQ_OK || num_q_heads < 1 || num_q_heads % desc->num_kv_heads) return 0;
  // the fused step's plan has at least as many splits; tickets sit at fixed offsets
  return kvq::plan_decode(*desc, num_q_heads, kvq::device_sm_count(), true).ws_total;
}

kvq_status kvq_quantize_pack_strided(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                     const void* k, const void* v, const int32_t* seq_lens,
                                     int32_t Lmax, int64_t stride_b, int64_t stride_h,
                                     int64_t stride_t, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (Lmax < 0 || !seq_lens || (Lmax > 0 && (!k || !v))) return KVQ_ERR_INVALID_ARG;
  if (stride_b < 0 || stride_h < 0 || stride_t < 0) return KVQ_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seq_lens, 4)) return KVQ_ERR_MISALIGNED;
  // every 8-value piece a lane loads must start on a 16-byte boundary
  if (stride_b % 8 || stride_h % 8 || stride_t % 8) return KVQ_ERR_MISALIGNED;
  const Dims s = kvq::dims_of(*desc);
  const int64_t strides[3] = {stride_b, stride_h, stride_t};
  return from_cuda(kvq::launch_quantize_pack(s, *view, static_cast<const __half*>(k),
                                             static_cast<const __half*>(v), seq_lens, Lmax, strides,
                                             static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_quantize_pack(const kvq_cache_desc* desc, const kvq_cache_view* view,
                             const void* k, const void* v, const int32_t* seq_lens,
                             int32_t Lmax, void* stream) {
  if (check_desc(desc) != KVQ_OK) return check_desc(desc);
  const int64_t d = desc->head_dim;
  return kvq_quantize_pack_strided(desc, view, k, v, seq_lens, Lmax,
                                   (int64_t)desc->num_kv_heads * Lmax * d, (int64_t)Lmax * d, d,
                                   stream);
}

kvq_status kvq_append(const kvq_cache_desc* desc, const kvq_cache_view* view, const void* k_new,
                      const void* v_new, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!k_new || !v_new) return KVQ_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return KVQ_ERR_MISALIGNED;
  const Dims s = kvq::dims_of(*desc);
  return from_cuda(kvq::launch_append(s, *view, static_cast<const __half*>(k_new),
                                      static_cast<const __half*>(v_new),
                                      static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_decode_attention(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                const void* q, int32_t num_q_heads, void* out, void* workspace,
                                size_t ws_bytes, uint32_t flags, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!q || !out || !workspace || num_q_heads < 1 || num_q_heads % desc->num_kv_heads ||
      (flags & ~(uint32_t)KVQ_OUT_F32))
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return KVQ_ERR_MISALIGNED;
  if ((int64_t)desc->batch * num_q_heads > 2147483647LL) return KVQ_ERR_UNSUPPORTED;
  const kvq::DecodePlan p = kvq::plan_decode(*desc, num_q_heads, kvq::device_sm_count());
  if ((int64_t)desc->num_kv_heads * p.nqb > 65535) return KVQ_ERR_UNSUPPORTED;
  if (ws_bytes < p.ws_total) return KVQ_ERR_INVALID_ARG;
  const Dims s = kvq::dims_of(*desc);
  return from_cuda(kvq::launch_decode(s, p, *view, static_cast<const __half*>(q), num_q_heads, out,
                                      workspace, static_cast<cudaStream_t>(stream), nullptr,
                                      nullptr, flags));
}

kvq_status kvq_decode_step(const kvq_cache_desc* desc, const kvq_cache_view* view, const void* q,
                           int32_t num_q_heads, const void* k_new, const void* v_new, void* out,
                           void* workspace, size_t ws_bytes, uint32_t flags, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!q || !out || !workspace || !k_new || !v_new || num_q_heads < 1 ||
      num_q_heads % desc->num_kv_heads || (flags & ~kStepFlags))
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(k_new, 16) ||
      !aligned(v_new, 16))
    return KVQ_ERR_MISALIGNED;
  if ((int64_t)desc->batch * num_q_heads > 2147483647LL) return KVQ_ERR_UNSUPPORTED;
  const kvq::DecodePlan p = kvq::plan_decode(*desc, num_q_heads, kvq::device_sm_count(), true);
  if ((int64_t)desc->num_kv_heads * p.nqb > 65535) return KVQ_ERR_UNSUPPORTED;
  if (ws_bytes < p.ws_total) return KVQ_ERR_INVALID_ARG;
  const Dims s = kvq::dims_of(*desc);
  return from_cuda(kvq::launch_decode(s, p, *view, static_cast<const __half*>(q), num_q_heads, out,
                                      workspace, static_cast<cudaStream_t>(stream),
                                      static_cast<const __half*>(k_new),
                                      static_cast<const __half*>(v_new), flags));
}

namespace {
struct StepIo {
  size_t q, kv, in_bytes, out_off, total;
};
// Byte layout of the packed step input [q | k_new | v_new] and of the device
// staging area (the input, then out at a 256-byte boundary).
StepIo step_io(const kvq_cache_desc& D, int32_t num_q_heads) {
  StepIo io;
  io.q = (size_t)D.batch * num_q_heads * D.head_dim * sizeof(uint16_t);
  io.kv = (size_t)D.batch * D.num_kv_heads * D.head_dim * sizeof(uint16_t);
  io.in_bytes = io.q + 2 * io.kv;
  io.out_off = (io.in_bytes + 255) & ~(size_t)255;
  io.total = io.out_off + 2 * io.q;  // room for an fp32 out
  return io;
}
}  // namespace

size_t kvq_step_io_bytes(const kvq_cache_desc* desc, int32_t num_q_heads) {
  if (check_desc(desc) != KVQ_OK || num_q_heads < 1 || num_q_heads % desc->num_kv_heads) return 0;
  return step_io(*desc, num_q_heads).total;
}

kvq_status kvq_decode_step_host(const kvq_cache_desc* desc, const kvq_cache_view* view,
                                const void* in_host, int32_t num_q_heads, void* out_host,
                                void* dev_io, size_t dev_io_bytes, void* workspace,
                                size_t ws_bytes, uint32_t flags, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if (flags & KVQ_STEP_HOST_MAPPED) {
    // the step reads the input block and writes out in place, over the host link
    if (!in_host || !out_host || num_q_heads < 1 || num_q_heads % desc->num_kv_heads)
      return KVQ_ERR_INVALID_ARG;
    if (!host_mapped(in_host) || !host_mapped(out_host)) return KVQ_ERR_INVALID_ARG;
    const StepIo io = step_io(*desc, num_q_heads);
    const char* in = static_cast<const char*>(in_host);
    return kvq_decode_step(desc, view, in, num_q_heads, in + io.q, in + io.q + io.kv, out_host,
                           workspace, ws_bytes, flags & ~(uint32_t)KVQ_STEP_HOST_MAPPED, stream);
  }
  if (!in_host || !out_host || !dev_io || num_q_heads < 1 || num_q_heads % desc->num_kv_heads)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(dev_io, 256)) return KVQ_ERR_MISALIGNED;
  const StepIo io = step_io(*desc, num_q_heads);
  if (dev_io_bytes < io.total) return KVQ_ERR_INVALID_ARG;
  char* d = static_cast<char*>(dev_io);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // every argument the step itself checks is checked before anything is enqueued
  const kvq::DecodePlan p = kvq::plan_decode(*desc, num_q_heads, kvq::device_sm_count(), true);
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!workspace || ws_bytes < p.ws_total || (flags & ~kStepFlags)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return KVQ_ERR_MISALIGNED;
  if (cudaMemcpyAsync(d, in_host, io.in_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return KVQ_ERR_CUDA;
  // the step follows this call's own copy, not a kernel: an early cache read
  // would have nothing to overlap
  st = kvq_decode_step(desc, view, d, num_q_heads, d + io.q, d + io.q + io.kv, d + io.out_off,
                       workspace, ws_bytes, flags & ~(uint32_t)KVQ_STEP_EARLY_CACHE_READ, stream);
  if (st != KVQ_OK) return st;
  const size_t out_bytes = (flags & KVQ_OUT_F32) ? 2 * io.q : io.q;
  if (cudaMemcpyAsync(out_host, d + io.out_off, out_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}

kvq_status kvq_append_chunk(const kvq_cache_desc* desc, const kvq_cache_view* view,
                            const kvq_append_args* args, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!args || !args->cu_seqlens || args->total < 0 || args->max_len < 0) return KVQ_ERR_INVALID_ARG;
  const kvq_append_args& A = *args;
  if (A.total > 0 && (!A.k || !A.v)) return KVQ_ERR_INVALID_ARG;
  if (A.kv_stride_token < 0 || A.kv_stride_head < 0) return KVQ_ERR_INVALID_ARG;
  if (A.q && (!A.q_out || A.num_q_heads < 1 || A.num_q_heads % desc->num_kv_heads ||
              A.q_stride_token < 0 || A.q_stride_head < 0))
    return KVQ_ERR_INVALID_ARG;
  if (A.rotary_dim < 0 || A.rotary_dim > desc->head_dim || (A.interleaved != 0 && A.interleaved != 1))
    return KVQ_ERR_INVALID_ARG;
  if (A.rotary_dim % 16) return KVQ_ERR_UNSUPPORTED;
  if (A.rotary_dim > 0 && (!A.rope || A.rope_rows < 1)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(A.k, 16) || !aligned(A.v, 16) || !aligned(A.q, 16) || !aligned(A.q_out, 16) ||
      !aligned(A.rope, 16) || !aligned(A.cu_seqlens, 4) || !aligned(A.positions, 4))
    return KVQ_ERR_MISALIGNED;
  // every 8-value piece a lane loads must start on a 16-byte boundary
  if (A.kv_stride_token % 8 || A.kv_stride_head % 8) return KVQ_ERR_MISALIGNED;
  if (A.q && (A.q_stride_token % 8 || A.q_stride_head % 8)) return KVQ_ERR_MISALIGNED;
  const Dims s = kvq::dims_of(*desc);
  return from_cuda(kvq::launch_append_chunk(s, *view, A, static_cast<cudaStream_t>(stream)));
}

size_t kvq_chunk_workspace_bytes(const kvq_cache_desc* desc, int32_t num_q_heads) {
  if (check_desc(desc) != KVQ_OK || num_q_heads < 1 || num_q_heads % desc->num_kv_heads) return 0;
  return kvq::chunk_workspace_bytes(kvq::dims_of(*desc), num_q_heads, kvq::device_sm_count());
}

namespace {
kvq_status attend_runs(const kvq_cache_desc* desc, const kvq_cache_view* view, const void* q,
                       int32_t num_q_heads, const int32_t* cu_seqlens, int32_t total, int32_t max_len,
                       void* out, void* workspace, size_t ws_bytes, uint32_t flags, bool causal,
                       void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (!cu_seqlens || total < 0 || max_len < 0 || !workspace || num_q_heads < 1 ||
      num_q_heads % desc->num_kv_heads || (flags & ~(uint32_t)KVQ_OUT_F32))
    return KVQ_ERR_INVALID_ARG;
  if (total > 0 && (!q || !out)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(cu_seqlens, 4))
    return KVQ_ERR_MISALIGNED;
  const Dims s = kvq::dims_of(*desc);
  // rows of one KV head and tokens of one sequence are counted in 32 bits
  const int64_t gq = num_q_heads / desc->num_kv_heads;
  if ((int64_t)(max_len < total ? max_len : total) * gq > (1LL << 30) ||
      (int64_t)s.cap + s.Nr + s.Ns > (1LL << 28))
    return KVQ_ERR_UNSUPPORTED;
  if (ws_bytes < kvq::chunk_workspace_bytes(s, num_q_heads, kvq::device_sm_count()))
    return KVQ_ERR_INVALID_ARG;
  return from_cuda(kvq::launch_chunk_attention(
      s, *view, static_cast<const __half*>(q), num_q_heads, cu_seqlens, total, max_len, out, workspace,
      causal, flags, static_cast<cudaStream_t>(stream)));
}
}  // namespace

kvq_status kvq_chunk_attention(const kvq_cache_desc* desc, const kvq_cache_view* view, const void* q,
                               int32_t num_q_heads, const int32_t* cu_seqlens, int32_t total,
                               int32_t max_len, void* out, void* workspace, size_t ws_bytes,
                               uint32_t flags, void* stream) {
  return attend_runs(desc, view, q, num_q_heads, cu_seqlens, total, max_len, out, workspace, ws_bytes,
                     flags, true, stream);
}

kvq_status kvq_cross_attention(const kvq_cache_desc* desc, const kvq_cache_view* view, const void* q,
                               int32_t num_q_heads, const int32_t* cu_seqlens, int32_t total,
                               int32_t max_len, void* out, void* workspace, size_t ws_bytes,
                               uint32_t flags, void* stream) {
  return attend_runs(desc, view, q, num_q_heads, cu_seqlens, total, max_len, out, workspace, ws_bytes,
                     flags, false, stream);
}

kvq_status kvq_read_tokens(const kvq_cache_desc* desc, const kvq_cache_view* view,
                           const int32_t* first, int32_t count, void* k_out, void* v_out,
                           uint32_t flags, void* stream) {
  kvq_status st = check_desc(desc);
  if (st != KVQ_OK) return st;
  if ((st = check_view(*desc, view)) != KVQ_OK) return st;
  if (count < 0 || (flags & ~(uint32_t)KVQ_OUT_F32)) return KVQ_ERR_INVALID_ARG;
  if (count > 0 && (!k_out || !v_out)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(first, 4)) return KVQ_ERR_MISALIGNED;
  const Dims s = kvq::dims_of(*desc);
  return from_cuda(kvq::launch_read_tokens(s, *view, first, count, k_out, v_out, flags,
                                           static_cast<cudaStream_t>(stream)));
}

namespace {
// One tensor of kvq_rotate: its heads, strides and places.
kvq_status check_rows(const void* x, const void* y, int32_t total, int32_t heads, int64_t st, int64_t sh,
                      int64_t yt, int64_t yh) {
  if (!y || heads < 1 || st < 0 || sh < 0 || yt < 0 || yh < 0) return KVQ_ERR_INVALID_ARG;
  if ((total > 1 && yt == 0) || (heads > 1 && yh == 0)) return KVQ_ERR_INVALID_ARG;  // one place for many rows
  if (x == y && (st != yt || sh != yh)) return KVQ_ERR_INVALID_ARG;  // in place: the same rows
  // every 8-value piece a lane moves must start on a 16-byte boundary
  if (!aligned(x, 16) || !aligned(y, 16) || st % 8 || sh % 8 || yt % 8 || yh % 8) return KVQ_ERR_MISALIGNED;
  return heads > 65535 ? KVQ_ERR_UNSUPPORTED : KVQ_OK;
}
bool head_dim_ok(int32_t d) { return d == 32 || d == 64 || d == 128 || d == 256; }
}  // namespace

kvq_status kvq_rotate(const kvq_rotate_args* args, void* stream) {
  if (!args) return KVQ_ERR_INVALID_ARG;
  kvq_rotate_args A = *args;
  if (A.total < 0 || A.head_dim < 32 || A.head_dim % 32 || (!A.q && !A.k && A.total > 0)) return KVQ_ERR_INVALID_ARG;
  if (!head_dim_ok(A.head_dim)) return KVQ_ERR_UNSUPPORTED;
  if (A.rotary_dim < 1 || A.rotary_dim > A.head_dim || (A.interleaved != 0 && A.interleaved != 1))
    return KVQ_ERR_INVALID_ARG;
  if (A.rotary_dim % 16 || A.axes > 4) return KVQ_ERR_UNSUPPORTED;
  if (A.axes < 1 || !A.rope || A.rope_rows < 1 || (A.total > 0 && !A.positions)) return KVQ_ERR_INVALID_ARG;
  if (A.pair_axis)
    for (int i = 0; i < A.rotary_dim / 2; ++i)
      if (A.pair_axis[i] >= A.axes) return KVQ_ERR_INVALID_ARG;
  kvq_status st;
  if (A.q && (st = check_rows(A.q, A.q_out, A.total, A.num_q_heads, A.q_stride_token, A.q_stride_head,
                              A.q_out_stride_token, A.q_out_stride_head)) != KVQ_OK)
    return st;
  if (A.k && (st = check_rows(A.k, A.k_out, A.total, A.num_kv_heads, A.k_stride_token, A.k_stride_head,
                              A.k_out_stride_token, A.k_out_stride_head)) != KVQ_OK)
    return st;
  if (!aligned(A.rope, 16) || !aligned(A.positions, 4) || !aligned(A.err_word, 4)) return KVQ_ERR_MISALIGNED;
  if (!A.err_word && A.total > 0 && (st = device_err_word(&A.err_word)) != KVQ_OK) return st;
  return from_cuda(kvq::launch_rotate(A, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_prompt_attention(const kvq_prompt_args* args, void* stream) {
  if (!args) return KVQ_ERR_INVALID_ARG;
  kvq_prompt_args A = *args;
  if (A.total < 0 || A.max_len < 0 || A.batch < 1 || !A.cu_seqlens || A.num_kv_heads < 1 || A.num_q_heads < 1 ||
      A.num_q_heads % A.num_kv_heads || A.head_dim < 32 || A.head_dim % 32 || (A.flags & ~(uint32_t)KVQ_OUT_F32))
    return KVQ_ERR_INVALID_ARG;
  if (A.total > 0 && (!A.q || !A.k || !A.v || !A.out)) return KVQ_ERR_INVALID_ARG;
  if (!head_dim_ok(A.head_dim) || A.num_q_heads / A.num_kv_heads > 128 || A.total > (1 << 30) || A.batch > (1 << 20))
    return KVQ_ERR_UNSUPPORTED;
  const int64_t strides[6] = {A.q_stride_token, A.k_stride_token, A.v_stride_token,
                              A.q_stride_head,  A.k_stride_head,  A.v_stride_head};
  for (int i = 0; i < 6; ++i) {
    const int32_t entries = i < 3 ? A.total : i == 3 ? A.num_q_heads : A.num_kv_heads;
    if (strides[i] < 0) return KVQ_ERR_INVALID_ARG;
    if (strides[i] % 8) return KVQ_ERR_MISALIGNED;  // rows start on 16-byte boundaries
    if (entries > 1 && (strides[i] == 0 || strides[i] >= (1LL << 39) / 128)) return KVQ_ERR_UNSUPPORTED;
  }
  if (!aligned(A.q, 16) || !aligned(A.k, 16) || !aligned(A.v, 16) || !aligned(A.out, 16) ||
      !aligned(A.cu_seqlens, 4) || !aligned(A.err_word, 4))
    return KVQ_ERR_MISALIGNED;
  const kvq_status st = A.err_word || A.total == 0 ? KVQ_OK : device_err_word(&A.err_word);
  if (st != KVQ_OK) return st;
  return from_cuda(kvq::launch_prompt_attention(A, static_cast<cudaStream_t>(stream)));
}

namespace {
kvq_status check_beams(int32_t batch, int32_t beams, int32_t vocab, int32_t n) {
  if (batch < 1 || beams < 1 || vocab < 1 || n < 1 || (int64_t)beams * vocab < n) return KVQ_ERR_INVALID_ARG;
  // a selection is a lane each, a proposal's place has 32 bits
  if (beams > 32 || n > 32 || (int64_t)batch * beams > 65535 || (int64_t)beams * vocab > 2147483646LL)
    return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}
}  // namespace

size_t kvq_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t n) {
  return check_beams(batch, beams, vocab, n) == KVQ_OK ? kvq::beam_workspace_bytes(batch, beams, vocab, n) : 0;
}

kvq_status kvq_beam_select(const kvq_beam_args* args, void* stream) {
  if (!args) return KVQ_ERR_INVALID_ARG;
  kvq_beam_args A = *args;
  kvq_status st = check_beams(A.batch, A.beams, A.vocab, A.n);
  if (st != KVQ_OK) return st;
  if (!A.logits || !A.scores || !A.parent || !A.token || !A.score || !A.workspace ||
      (A.flags & ~(uint32_t)KVQ_LOGITS_F32) || A.stride_row < A.vocab)
    return KVQ_ERR_INVALID_ARG;
  if (A.finished && (A.end_token < 0 || A.end_token >= A.vocab)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(A.logits, A.flags & KVQ_LOGITS_F32 ? 4 : 2) || !aligned(A.workspace, 16) || !aligned(A.scores, 4) || !aligned(A.parent, 4) ||
      !aligned(A.token, 4) || !aligned(A.score, 4) || !aligned(A.err_word, 4))
    return KVQ_ERR_MISALIGNED;
  if (A.ws_bytes < kvq::beam_workspace_bytes(A.batch, A.beams, A.vocab, A.n)) return KVQ_ERR_INVALID_ARG;
  if (!A.err_word && (st = device_err_word(&A.err_word)) != KVQ_OK) return st;
  return from_cuda(kvq::launch_beam_select(A, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_reorder(const kvq_cache_desc* dst_desc, const kvq_cache_view* dst,
                       const kvq_cache_desc* src_desc, const kvq_cache_view* src, const int32_t* index,
                       uint32_t flags, void* stream) {
  kvq_status st;
  if ((st = check_desc(dst_desc)) != KVQ_OK || (st = check_desc(src_desc)) != KVQ_OK) return st;
  if ((st = check_view(*dst_desc, dst)) != KVQ_OK || (st = check_view(*src_desc, src)) != KVQ_OK) return st;
  const kvq_cache_desc &d = *dst_desc, &s = *src_desc;
  if (!index || (flags & ~(uint32_t)KVQ_REORDER_SHARE_PAGES) || d.num_kv_heads != s.num_kv_heads ||
      d.head_dim != s.head_dim || d.bits != s.bits || d.residual != s.residual || d.sink != s.sink ||
      d.hybrid != s.hybrid || d.page_size != s.page_size)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(index, 4)) return KVQ_ERR_MISALIGNED;
  auto same = [](const void* a, const void* b) { return a && a == b; };
  const bool share = flags & KVQ_REORDER_SHARE_PAGES, both = d.capacity > 0 && s.capacity > 0;
  // one sequence's bytes would be another's before they are read
  if (same(dst->packed_len, src->packed_len) || same(dst->res_len, src->res_len) ||
      same(dst->res_head, src->res_head) ||
      (d.sink && (same(dst->sink_len, src->sink_len) || same(dst->k_sink, src->k_sink) ||
                  same(dst->v_sink, src->v_sink))) ||
      (d.residual && (same(dst->k_res, src->k_res) || same(dst->v_res, src->v_res))) ||
      (d.page_size && both && same(dst->block_table, src->block_table)))
    return KVQ_ERR_INVALID_ARG;
  if (!d.page_size && both &&
      (same(dst->k_codes, src->k_codes) || same(dst->v_codes, src->v_codes) ||
       same(dst->k_params, src->k_params) || same(dst->v_params, src->v_params) ||
       (d.hybrid && (same(dst->k_mode, src->k_mode) || same(dst->v_mode, src->v_mode)))))
    return KVQ_ERR_INVALID_ARG;
  if (share && (!d.page_size || d.num_pages != s.num_pages || dst->k_codes != src->k_codes ||
                dst->v_codes != src->v_codes || dst->k_params != src->k_params ||
                dst->v_params != src->v_params ||
                (d.hybrid && (dst->k_mode != src->k_mode || dst->v_mode != src->v_mode))))
    return KVQ_ERR_INVALID_ARG;  // there is no one pool
  return from_cuda(kvq::launch_reorder(kvq::dims_of(d), *dst, kvq::dims_of(s), *src, index, share,
                                       static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_read_error(const kvq_cache_view* view, uint32_t* word_out, void* stream) {
  if (!view || !view->err_word) return KVQ_ERR_INVALID_ARG;
  if (!aligned(view->err_word, 4)) return KVQ_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t w = 0;
  cudaError_t e = cudaMemcpyAsync(&w, view->err_word, sizeof(w), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(view->err_word, 0, sizeof(uint32_t), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  if (word_out) *word_out = w;
  if (w & KVQ_ERRBIT_TIMEOUT) kvq::noalloc_forget_layout();
  return status_of(w);
}

kvq_status kvq_read_device_error(uint32_t* word_out, void* stream) {
  static std::mutex one;  // reads through one place
  std::lock_guard<std::mutex> lock(one);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t w = 0;
  // (exchanged: calls on other streams may be setting bits)
  take_errors_kernel<<<1, 1, 0, st>>>();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&w, g_err_taken, sizeof(w), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  if (word_out) *word_out = w;
  return status_of(w);
}

const char* kvq_status_string(kvq_status status) {
  switch (status) {
    case KVQ_OK: return "ok";
    case KVQ_ERR_INVALID_ARG: return "invalid argument";
    case KVQ_ERR_UNSUPPORTED: return "unsupported configuration";
    case KVQ_ERR_MISALIGNED: return "misaligned pointer";
    case KVQ_ERR_CAPACITY: return "packed capacity exceeded";
    case KVQ_ERR_CUDA: return "CUDA error";
    case KVQ_ERR_TIMEOUT: return "device wait timed out";
    case KVQ_ERR_EMPTY: return "sequence with no tokens";
    default: return "unknown status";
  }
}

int32_t kvq_version(void) { return 160; }

void kvq_testing_wait_fault(uint32_t limit_us) { kvq::set_testing_wait_fault_us(limit_us); }

}  // extern "C"
