// kps_min_p.cu — the sampling step with the min-p stage, over the kernels of kps_sampler.cuh
// compiled with it.
#define KPS_MIN_P 1
#include "kps_sampler.cuh"

extern "C" kps_status kps_sample_min_p(const void* logits, kps_dtype dt, int64_t B, int64_t V, const int32_t* top_k,
                                       const float* top_p, const float* min_p, const float* temperature,
                                       const int32_t* seen_indptr, const int32_t* seen_ids, const float* penalty,
                                       const kps_step_opts* opts, float eps, int need_logits, int64_t* out_idx,
                                       float* out_filtered, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
  const kps::NvtxRange range("kps_sample_min_p");
  if (B > 0 && (!min_p || (reinterpret_cast<uintptr_t>(min_p) & 3u) != 0)) return KPS_ERR_INVALID_ARG;
  return step_impl(logits, dt, B, V, top_k, top_p, min_p, temperature, seen_indptr, seen_ids, penalty, opts, eps,
                   need_logits, out_idx, out_filtered, workspace, workspace_bytes, stream);
}
