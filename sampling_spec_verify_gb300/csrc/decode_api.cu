// Host side of the decoding step around the verify: attention over the paged
// cache, the cache's tables and commits, the sampling rules.  Argument checks,
// launch shapes and launches; no entry point allocates device memory or
// synchronises the stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "adjust.cuh"
#include "attend.cuh"
#include "cache.cuh"
#include "spec_verify.h"

namespace ssv {
cudaError_t count_launch(cudaError_t e);  // spec_api.cu
}

namespace {

using ssv::count_launch;

constexpr int kMaxDevices = 64;
constexpr long long kMaxStride = 1ll << 39;

spec_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Streaming multiprocessors of the current device; 0 on failure.
int device_sms(int* id = nullptr) {
  static int sms[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::call_once(once[dev], [dev]() { cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev); });
  if (id) *id = dev;
  return sms[dev];
}

// Strides of 16-bit tensors in 16-byte steps.
bool strides_ok(const long long* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] <= 0 || s[i] % 8 || s[i] >= kMaxStride) return false;
  return true;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  if (B < 0 || T < 1 || T > 1024 || Hkv < 1 || Hq < 1 || Hq % Hkv || D < 8 || D > 256 || D % 8) return 0;
  return 256;
}

spec_status_t spec_tree_attention(const spec_attention_t* args, uint32_t* dev_status, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_attention_t& A = *args;
  if (A.B < 0 || A.T < 1 || A.rows < 0 || A.Hkv < 1 || A.Hq < 1 || A.Hq % A.Hkv || A.D < 1 || A.pages < 0 ||
      A.page_size < 1 || A.table_width < 0 || (A.dtype != SPEC_BF16 && A.dtype != SPEC_F16) || !std::isfinite(A.scale))
    return SPEC_ERR_INVALID_ARG;
  if (!A.row_offsets && (long long)A.B * A.T != A.rows) return SPEC_ERR_INVALID_ARG;
  if (A.D > 256 || A.D % 8 || A.page_size % 8 || A.T > 1024) return SPEC_ERR_UNSUPPORTED;
  if (A.B == 0 || A.rows == 0) return SPEC_OK;
  if (!A.q || !A.k_new || !A.v_new || !A.out || !A.context_lens) return SPEC_ERR_INVALID_ARG;
  if (A.table_width > 0 && (!A.block_table || A.table_stride < A.table_width)) return SPEC_ERR_INVALID_ARG;
  if (A.pages > 0 && (!A.k_cache || !A.v_cache)) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {A.q, A.k_new, A.v_new, A.k_cache, A.v_cache, (const void*)A.out})
    if (!aligned(p, 16)) return SPEC_ERR_INVALID_ARG;
  if (!strides_ok(A.q_stride, 2) || !strides_ok(A.k_new_stride, 2) || !strides_ok(A.v_new_stride, 2) ||
      (A.pages > 0 && (!strides_ok(A.k_stride, 3) || !strides_ok(A.v_stride, 3))))
    return SPEC_ERR_INVALID_ARG;
  if (workspace_bytes < spec_tree_attention_workspace_bytes(A.B, A.T, A.Hq, A.Hkv, A.D) || !workspace)
    return SPEC_ERR_INVALID_ARG;
  if (A.B > 65535 || A.Hq > 65535) return SPEC_ERR_UNSUPPORTED;
  ssv::AttendParams P = {A, dev_status};
  const dim3 grid((unsigned)((A.T + 3) / 4), (unsigned)A.B, (unsigned)A.Hq);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (A.dtype == SPEC_BF16)
    ssv::attend_plain_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(P);
  else
    ssv::attend_plain_kernel<__half><<<grid, 128, 0, st>>>(P);
  return from_cuda(count_launch(cudaGetLastError()));
}

spec_status_t spec_plan_cache(const int32_t* context_lens, const int32_t* new_lens, const int32_t* block_table,
                              const int32_t* free_pages, const int32_t* free_count, int B, int T, int table_width,
                              int capacity, int page_size, int32_t* out_table, int32_t* out_free, int32_t* out_count,
                              int32_t* out_lens, int32_t* slots, uint32_t* dev_status, void* stream) {
  if (B < 0 || T < 0 || table_width < 1 || capacity < 0 || page_size < 1) return SPEC_ERR_INVALID_ARG;
  if ((long long)B * table_width > 0x7FFFFFFFll || (long long)B * (T > 0 ? T : 1) > 0x7FFFFFFFll ||
      (long long)table_width * page_size > 0x7FFFFFFFll)
    return SPEC_ERR_UNSUPPORTED;
  if (!free_count || !out_count || free_count == out_count) return SPEC_ERR_INVALID_ARG;
  if (capacity > 0 && (!free_pages || !out_free)) return SPEC_ERR_INVALID_ARG;
  if (B > 0 && (!context_lens || !new_lens || !block_table || !out_table || !out_lens || (T > 0 && !slots)))
    return SPEC_ERR_INVALID_ARG;
  const size_t table = (size_t)B * table_width * 4, stack = (size_t)capacity * 4, lens = (size_t)B * 4;
  const size_t map = (size_t)B * T * 4;
  if ((out_table != block_table && overlap(out_table, table, block_table, table)) ||
      (out_free != free_pages && overlap(out_free, stack, free_pages, stack)))
    return SPEC_ERR_INVALID_ARG;
  // nothing that is read may be written, but for table and stack in place
  const struct { const void* p; size_t n; } in[] = {{context_lens, lens}, {new_lens, lens}, {free_count, 4},
                                                    {block_table, table}, {free_pages, stack}},
      out[] = {{out_lens, lens}, {out_count, 4}, {slots, map}, {out_table, table}, {out_free, stack}};
  for (int i = 0; i < 5; ++i)
    for (int o = 0; o < 5; ++o)
      if (!(i == o && i >= 3) && in[i].n && out[o].n && overlap(in[i].p, in[i].n, out[o].p, out[o].n))
        return SPEC_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (!sms) return SPEC_ERR_CUDA;
  ssv::PlanParams P = {context_lens, new_lens, block_table, free_pages, free_count, out_table, out_free, out_count,
                       out_lens, slots, dev_status, B, T, table_width, capacity, page_size, 1};
  P.per = (B + 4 * sms - 1) / (4 * sms);
  if (P.per < 1) P.per = 1;
  int grid = (B + P.per - 1) / P.per;
  if (out_free != free_pages) {
    const int copiers = (int)((capacity + 4095ll) / 4096);
    if (grid < copiers) grid = copiers < 4 * sms ? copiers : 4 * sms;
  }
  if (grid < 1) grid = 1;
  ssv::plan_kernel<<<grid, ssv::kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return from_cuda(count_launch(cudaGetLastError()));
}

spec_status_t spec_commit_cache(const spec_commit_t* args, uint32_t* dev_status, void* stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_commit_t& A = *args;
  if (A.layers < 0 || A.B < 0 || A.T < 1 || A.rows < 0 || A.S < 0 || A.Hkv < 1 || A.D < 1 || A.pages < 0 ||
      A.page_size < 1 || (A.dtype != SPEC_BF16 && A.dtype != SPEC_F16))
    return SPEC_ERR_INVALID_ARG;
  if (!A.row_offsets && (long long)A.B * A.T != A.rows) return SPEC_ERR_INVALID_ARG;
  if (A.D % 8 || (long long)A.pages * A.page_size > 0x7FFFFFFFll || (long long)A.Hkv * A.D > 0x7FFFFFFFll)
    return SPEC_ERR_UNSUPPORTED;
  if (A.layers == 0 || A.B == 0 || A.S == 0 || A.rows == 0) return SPEC_OK;
  if (!A.k_new || !A.v_new || !A.slots) return SPEC_ERR_INVALID_ARG;
  if (A.pages > 0 && (!A.k_cache || !A.v_cache)) return SPEC_ERR_INVALID_ARG;
  if (A.path && A.S > 1 && A.path_stride < A.S - 1) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {A.k_new, A.v_new, (const void*)A.k_cache, (const void*)A.v_cache})
    if (!aligned(p, 16)) return SPEC_ERR_INVALID_ARG;
  if (!strides_ok(A.k_new_stride, 3) || !strides_ok(A.v_new_stride, 3) ||
      (A.pages > 0 && (!strides_ok(A.k_stride, 4) || !strides_ok(A.v_stride, 4))))
    return SPEC_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (!sms) return SPEC_ERR_CUDA;
  ssv::CommitParams P = {A, dev_status};
  const long long blocks = ((long long)A.layers * A.B * A.S + 7) / 8;
  const int grid = blocks < 8ll * sms ? (int)blocks : 8 * sms;
  ssv::commit_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return from_cuda(count_launch(cudaGetLastError()));
}

spec_status_t spec_adjust_logits(const spec_adjust_t* args, uint32_t* dev_status, void* stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_adjust_t& A = *args;
  if (A.B < 0 || A.T < 1 || A.rows < 0 || A.V < 1 || A.history_width < 0 || A.biases < 0 ||
      (A.dtype != SPEC_BF16 && A.dtype != SPEC_F32))
    return SPEC_ERR_INVALID_ARG;
  if (!A.row_offsets && (long long)A.B * A.T != A.rows) return SPEC_ERR_INVALID_ARG;
  if (A.T > ssv::kAdjustMaxRows || A.biases > ssv::kAdjustMaxBiases || A.history_width > ssv::kAdjustMaxHistory ||
      A.V > (1 << 24) || A.B > 65535)
    return SPEC_ERR_UNSUPPORTED;
  if (A.B == 0 || A.rows == 0) return SPEC_OK;
  if (!A.logits || !A.out || !A.tokens || !A.history_lens || (A.history_width > 0 && !A.history) ||
      (A.biases > 0 && (!A.bias_ids || !A.bias)))
    return SPEC_ERR_INVALID_ARG;
  const int es = A.dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(A.logits, es) || !aligned(A.out, es)) return SPEC_ERR_INVALID_ARG;
  const size_t bytes = (size_t)A.rows * A.V * es;
  if (A.out != A.logits && overlap(A.out, bytes, A.logits, bytes)) return SPEC_ERR_INVALID_ARG;
  int dev = 0;
  const int sms = device_sms(&dev);
  if (!sms) return SPEC_ERR_CUDA;
  int parts = (A.V + ssv::kAdjustMaxSlice - 1) / ssv::kAdjustMaxSlice;
  while ((long long)A.B * parts < 2ll * sms && A.V / parts > 4096) ++parts;
  ssv::AdjustParams P = {A, dev_status, ((A.V + parts - 1) / parts + 63) / 64 * 64};
  const size_t smem = ssv::adjust_smem(P.slice, A.biases, A.T);
  static std::once_flag once[2][kMaxDevices];
  static cudaError_t made[2][kMaxDevices];
  const int which = A.dtype == SPEC_BF16;
  std::call_once(once[which][dev], [which, dev]() {
    const int most = (int)ssv::adjust_smem(ssv::kAdjustMaxSlice, ssv::kAdjustMaxBiases, ssv::kAdjustMaxRows);
    made[which][dev] =
        which ? cudaFuncSetAttribute(ssv::adjust_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)
              : cudaFuncSetAttribute(ssv::adjust_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (made[which][dev] != cudaSuccess) return SPEC_ERR_CUDA;
  const dim3 grid((unsigned)((A.V + P.slice - 1) / P.slice), (unsigned)A.B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (which)
    ssv::adjust_kernel<__nv_bfloat16><<<grid, ssv::kAdjustThreads, smem, st>>>(P);
  else
    ssv::adjust_kernel<float><<<grid, ssv::kAdjustThreads, smem, st>>>(P);
  return from_cuda(count_launch(cudaGetLastError()));
}

}  // extern "C"
