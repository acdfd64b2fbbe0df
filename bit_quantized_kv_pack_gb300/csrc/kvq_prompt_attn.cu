// kvq_prompt_attn.cu -- attention over prompts: tensor maps and the dispatch on head_dim
// (the kernel is kvq_prompt_attn.cuh).
#include "kvq_prompt_attn.cuh"

#include <mutex>

namespace kvq {
namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's cuTensorMapEncodeTiled, looked up once per process.
EncodeFn encode_fn() {
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// fp16 values, the first dimension contiguous, the others `stride` elements apart; what a
// box has outside is zero.
bool encode(CUtensorMap* map, const void* base, int rank, const uint64_t* extent, const int64_t* stride,
            const uint32_t* box, int head_dim) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4], strides[3];
  cuuint32_t boxes[4], steps[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) dims[i] = extent[i], boxes[i] = box[i];
  // (a dimension of one entry may come with any stride, 0 too)
  for (int i = 1; i < rank; ++i) strides[i - 1] = extent[i] > 1 ? (cuuint64_t)stride[i] * 2 : 16;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(base), dims, strides, boxes, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            head_dim < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Units order[0 .. n) of the line to `units` (kvq_testing_prompt_units), by one warp.
__global__ void units_kernel(prompt::UnitLine line, const int32_t* order, int n, int4* units) {
  line.begin();
  for (int i = 0; i < n; ++i) {
    const bool found = line.find(order[i]), has = line.has(order[i]);
    if (!found) {
      if (threadIdx.x == 0) units[i] = make_int4(-1, 0, 0, 0);
    } else if (has) {
      int h, t0;
      line.place(order[i], h, t0);
      units[i] = make_int4(line.run.c0, line.run.n, h, t0);
    }
  }
}

}  // namespace

cudaError_t launch_prompt_attention(const kvq_prompt_args& A, cudaStream_t st) {
  if (A.total == 0) return cudaSuccess;
  PromptAttnArgs a;
  const int d = A.head_dim;
  a.gq = A.num_q_heads / A.num_kv_heads;
  a.T = 128 / a.gq;
  a.gq_mul = (uint32_t)(65536 / a.gq + (65536 % a.gq != 0));
  const uint64_t rows = (uint64_t)A.total, heads = (uint64_t)A.num_kv_heads;
  const uint32_t panel = prompt_panel(d), tile = prompt_tile(d);
  const uint64_t qe[4] = {(uint64_t)d, (uint64_t)a.gq, rows, heads}, ke[3] = {(uint64_t)d, rows, heads};
  const int64_t qs[4] = {1, A.q_stride_head, A.q_stride_token, A.q_stride_head * a.gq};
  const int64_t ks[3] = {1, A.k_stride_token, A.k_stride_head}, vs[3] = {1, A.v_stride_token, A.v_stride_head};
  const uint32_t qb[4] = {panel, (uint32_t)a.gq, (uint32_t)a.T, 1}, kb[3] = {panel, tile, 1};
  if (!encode(&a.mq, A.q, 4, qe, qs, qb, d) || !encode(&a.mk, A.k, 3, ke, ks, kb, d) ||
      !encode(&a.mv, A.v, 3, ke, vs, kb, d))
    return cudaErrorInvalidValue;
  a.cu = A.cu_seqlens;
  a.err_word = A.err_word;
  a.out = A.out;
  a.B = A.batch;
  a.Hkv = A.num_kv_heads;
  a.total = A.total;
  a.max_len = A.max_len;
  a.out_f32 = (A.flags & KVQ_OUT_F32) ? 1 : 0;
  const uint32_t fault_us = testing_wait_fault_us();
  a.wait_limit_us = fault_us ? fault_us : 1000000u;
  a.fault = fault_us ? 1 : 0;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d));
  // as many blocks as there can be units
  const int64_t tokens = (int64_t)prompt_lanes(d) * a.T;
  int64_t units = (A.total / tokens + A.batch) * (int64_t)heads;
  a.shared = prompt_lanes(d) == 2 && units <= device_sm_count();
  if (a.shared) units = (A.total / a.T + A.batch) * (int64_t)heads;
  if (units > 2147483647) return cudaErrorInvalidValue;
  const int grid = (int)units;
  if (d == 32) return launch_prompt_attn_d32(a, grid, st);
  if (d == 64) return launch_prompt_attn_d64(a, grid, st);
  if (d == 128) return launch_prompt_attn_d128(a, grid, st);
  return launch_prompt_attn_d256(a, grid, st);
}

}  // namespace kvq

extern "C" kvq_status kvq_testing_prompt_units(const int32_t* cu_seqlens, int32_t batch, int32_t total, int32_t max_len,
                                               int32_t heads, int32_t tokens, const int32_t* order, int32_t n,
                                               int32_t* units) {
  if (!cu_seqlens || batch < 1 || total < 0 || max_len < 0 || heads < 1 || tokens < 1 || !order || n < 1 || !units ||
      reinterpret_cast<uintptr_t>(units) % 16)
    return KVQ_ERR_INVALID_ARG;
  kvq::prompt::UnitLine line = {};
  line.cu = cu_seqlens;
  line.B = batch, line.total = total, line.max_len = max_len, line.Hkv = heads, line.step = tokens;
  kvq::units_kernel<<<1, 32>>>(line, order, n, reinterpret_cast<int4*>(units));
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
