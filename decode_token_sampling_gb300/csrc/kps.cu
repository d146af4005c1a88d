// kps.cu — the C ABI of the decode-step sampler without min-p, over the kernels of kps_sampler.cuh.
#define KPS_MIN_P 0
#include "kps_sampler.cuh"

namespace kps {
LastCall& last_call() {
  static thread_local LastCall c = {};
  return c;
}
}  // namespace kps

// ------------------------------------------------------------------------------------------
// C ABI
// ------------------------------------------------------------------------------------------
extern "C" {

size_t kps_workspace_size(int64_t B, int64_t V, kps_dtype dt) {
  if (B < 0 || V < 1 || (dt != KPS_F32 && dt != KPS_BF16)) return 0;
  if (V <= kps::kRKeepAllV) return kps::kWorkspaceMin;
  const int64_t rows = B < kps::kMaxPreRows ? B : kps::kMaxPreRows;
  return kps::kWorkspaceMin + static_cast<size_t>(rows) * kps::kPRecBytes;
}

int64_t kps_max_vocab(kps_dtype dt) {
  if (dt != KPS_F32 && dt != KPS_BF16) return 0;
  const int optin = kps::device_smem_optin();
  if (optin <= 0) return 0;
  const bool bf = dt == KPS_BF16;
  if ((bf ? kps::prepare_kernel<true>() : kps::prepare_kernel<false>()) != cudaSuccess) return 0;
  // the largest chunk (a multiple of 8) whose layout fits one CTA: binary search over its
  // eighths, keeping a chunk that fits in lo
  int lo = 0, hi = kps::kMaxChunk / 8;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (kps::make_layout(mid * 8, bf).total <= static_cast<size_t>(optin)) lo = mid; else hi = mid - 1;
  }
  if (lo == 0) return 0;
  const int nc = lo * 8;
  const size_t smem = kps::make_layout(nc, bf).total;
  // times the widest cluster the device runs with that much shared memory per CTA
  for (int cs = 16; cs >= 1; cs /= 2) {
    const bool fits = bf ? kps::cluster_fits<true>(cs, smem) : kps::cluster_fits<false>(cs, smem);
    if (fits) return static_cast<int64_t>(nc) * cs;
  }
  return 0;
}

const char* kps_status_string(kps_status s) {
  switch (s) {
    case KPS_OK: return "ok";
    case KPS_ERR_INVALID_ARG: return "invalid argument";
    case KPS_ERR_UNSUPPORTED: return "unsupported size";
    case KPS_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case KPS_ERR_CUDA: return "CUDA error";
    case KPS_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

kps_status kps_query_launch(int64_t B, int64_t V, kps_dtype dt, int* cluster_size, int64_t* chunk_elems,
                            size_t* smem_bytes) {
  if (V < 1 || V > INT32_MAX || B < 0 || (dt != KPS_F32 && dt != KPS_BF16)) return KPS_ERR_INVALID_ARG;
  kps::LaunchCfg cfg;
  const kps_status st = dt == KPS_BF16 ? kps::choose_launch<true>(B, V, &cfg) : kps::choose_launch<false>(B, V, &cfg);
  if (st != KPS_OK) return st;
  if (cluster_size) *cluster_size = cfg.cs;
  if (chunk_elems) *chunk_elems = cfg.nc;
  if (smem_bytes) *smem_bytes = cfg.smem;
  return KPS_OK;
}

kps_status kps_sample(const void* logits, kps_dtype dt, int64_t B, int64_t V, const int32_t* top_k,
                      const float* top_p, const float* temperature, const int32_t* seen_indptr,
                      const int32_t* seen_ids, const float* penalty, const float* q, float eps, int need_logits,
                      int64_t* out_idx, float* out_filtered, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
  const kps::NvtxRange range("kps_sample");
  return sample_impl(logits, dt, B, V, top_k, top_p, temperature, seen_indptr, seen_ids, penalty, q, eps,
                     need_logits, out_idx, out_filtered, workspace, workspace_bytes, stream, 0, 0ull, 0ull);
}

kps_status kps_sample_seeded(const void* logits, kps_dtype dt, int64_t B, int64_t V, const int32_t* top_k,
                             const float* top_p, const float* temperature, const int32_t* seen_indptr,
                             const int32_t* seen_ids, const float* penalty, unsigned long long seed,
                             unsigned long long step, float eps, int need_logits, int64_t* out_idx,
                             float* out_filtered, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const kps::NvtxRange range("kps_sample_seeded");
  return sample_impl(logits, dt, B, V, top_k, top_p, temperature, seen_indptr, seen_ids, penalty, nullptr, eps,
                     need_logits, out_idx, out_filtered, workspace, workspace_bytes, stream, 1, seed, step);
}

kps_status kps_sample_step(const void* logits, kps_dtype dt, int64_t B, int64_t V, const int32_t* top_k,
                           const float* top_p, const float* temperature, const int32_t* seen_indptr,
                           const int32_t* seen_ids, const float* penalty, const kps_step_opts* opts, float eps,
                           int need_logits, int64_t* out_idx, float* out_filtered, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  const kps::NvtxRange range("kps_sample_step");
  return step_impl(logits, dt, B, V, top_k, top_p, nullptr, temperature, seen_indptr, seen_ids, penalty, opts, eps,
                   need_logits, out_idx, out_filtered, workspace, workspace_bytes, stream);
}

int kps_last_kernel(void) { return kps::last_call().kernel; }

int kps_last_launch_count(void) { return kps::last_call().launches; }

int kps_last_cluster_size(void) { return kps::last_call().cluster; }

kps_status kps_last_device_status(void* workspace, cudaStream_t stream, int* out) {
  if (!workspace || !out) return KPS_ERR_INVALID_ARG;
  int h = 0;
  if (cudaMemcpyAsync(&h, workspace, sizeof(int), cudaMemcpyDeviceToHost, stream) != cudaSuccess) return KPS_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return KPS_ERR_CUDA;
  if (cudaMemsetAsync(workspace, 0, sizeof(int), stream) != cudaSuccess) return KPS_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return KPS_ERR_CUDA;
  *out = h;
  return KPS_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// No-allocation entry point: the scratch lives in a fixed device array.
// ------------------------------------------------------------------------------------------
namespace kps {
constexpr size_t kNoallocScratchBytes = 4096;
// File-scope scratch for kps_sample_noalloc.  In host code this name is only a
// stand-in for the symbol: its device address comes from cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoallocScratchBytes];

// Device address of g_noalloc_scratch on the current device, looked up once per
// device with that device current.  Returns nullptr on failure.
static void* noalloc_scratch_address() {
  static std::mutex mu;
  static void* addr[kMaxDevices] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) {
      (void)cudaGetLastError();
      return nullptr;
    }
    addr[dev] = p;
  }
  return addr[dev];
}
}  // namespace kps

extern "C" kps_status kps_sample_noalloc(const void* logits, kps_dtype dt, int64_t B, int64_t V,
                                         const int32_t* top_k, const float* top_p, const float* temperature,
                                         const int32_t* seen_indptr, const int32_t* seen_ids,
                                         const float* penalty, const float* q, float eps, int need_logits,
                                         int64_t* out_idx, float* out_filtered, cudaStream_t stream) {
  const kps::NvtxRange range("kps_sample_noalloc");
  // every argument is checked before the shared array is touched: a rejected call queues nothing
  {
    const kps_status st = check_args(dt, B, V, eps, logits, top_k, top_p, temperature, out_idx, need_logits, out_filtered);
    if (st != KPS_OK || B == 0) return st;
  }
  const size_t need = kps::kWorkspaceMin;  // the status word; no room for pre-pass records
  void* scratch = kps::noalloc_scratch_address();
  if (!scratch) return KPS_ERR_CUDA;
  // the shared array keeps the previous call's status word: clear it on this stream first
  if (cudaMemsetAsync(scratch, 0, need, stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  return kps_sample(logits, dt, B, V, top_k, top_p, temperature, seen_indptr, seen_ids, penalty, q, eps,
                    need_logits, out_idx, out_filtered, scratch, need, stream);
}
