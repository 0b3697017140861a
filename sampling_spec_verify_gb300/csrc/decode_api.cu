// Host side of the decoding step around the verify: attention over the paged
// cache, the cache's tables and commits, the sampling rules.  Argument checks,
// launch shapes and launches; no entry point allocates device memory or
// synchronises the stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

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

// ---- attention ---------------------------------------------------------------------

constexpr int kMaxPassRows = 1024;
constexpr int kMaxCtas = 152;  // of the attention, one an SM

struct AttendPlan {
  int dp, mt, tok, slot_rows;
  float* part;
  float4* stat;
  ssv::AttendSplit* split;
  size_t bytes;
};
// Rows of 128 query rows and two such tiles a CTA where a request's pass may have
// more of them (one tile: the cache would be read again for the second).  A head
// beyond 128 fills the tensor memory with one tile.  T, the most rows of a request, decides for
// the whole batch, whose lengths only the device knows: units of one row tile then leave the second
// group idle (128 single tokens over 64 to 4096 cached ones, 32/8 heads: 200 us in
// a graph for T = 1, 255 for T = 33, 263 with one request of 33 rows among them).
AttendPlan attend_plan(int T, int group, int D, void* base) {
  AttendPlan p = {};
  p.dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  p.tok = 128 / group;
  p.mt = p.dp <= 128 && T > p.tok ? 2 : 1;
  p.slot_rows = p.mt == 2 ? 256 : (T < p.tok ? T : p.tok) * group;
  char* at = static_cast<char*>(base);
  auto take = [&](size_t n) {
    char* x = base ? at + p.bytes : nullptr;
    p.bytes += (n + 255) & ~size_t(255);
    return x;
  };
  const size_t slots = (size_t)2 * kMaxCtas * p.slot_rows;
  p.part = reinterpret_cast<float*>(take(slots * p.dp * sizeof(float)));
  p.stat = reinterpret_cast<float4*>(take(slots * sizeof(float4)));
  p.split = reinterpret_cast<ssv::AttendSplit*>(take(kMaxCtas * sizeof(ssv::AttendSplit)));
  return p;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiled>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// Boxes of 128 bytes (64 elements) along the first dimension, 128-byte swizzle; strides in elements.
template <int N>
bool make_map(CUtensorMap* m, const void* base, bool bf16, const long long (&size)[N], const long long (&stride)[N - 1],
              const int (&box)[N - 1]) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[N], strides[N - 1];
  cuuint32_t boxes[N], step[N];
  for (int i = 0; i < N; ++i) {
    dims[i] = (cuuint64_t)size[i];
    boxes[i] = i ? (cuuint32_t)box[i - 1] : 64;
    step[i] = 1;
    if (i) strides[i - 1] = (cuuint64_t)stride[i - 1] * 2;
  }
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, N, const_cast<void*>(base),
             dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class E, int DP, int MT>
spec_status_t run_attend(const spec_attention_t& A, const AttendPlan& p, uint32_t* status, cudaStream_t st) {
  using Sh = ssv::AttendShape<DP, MT>;
  constexpr bool bf = std::is_same<E, __nv_bfloat16>::value;
  int dev = 0;
  const int sms = device_sms(&dev);
  if (!sms) return SPEC_ERR_CUDA;
  static std::once_flag once[kMaxDevices];
  static cudaError_t made[kMaxDevices];
  std::call_once(once[dev], [dev]() {
    made[dev] = cudaFuncSetAttribute(ssv::attend_kernel<E, DP, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  });
  if (made[dev] != cudaSuccess) return SPEC_ERR_CUDA;
  ssv::AttendLaunch L = {};
  L.a = A;
  L.status = status;
  L.part = p.part;
  L.stat = p.stat;
  L.split = p.split;
  L.c = A.scale == 0.0f ? 1.0f : (float)(1.4426950408889634 * std::fabs((double)A.scale));
  L.flip = A.scale > 0.0f ? 1.0f : A.scale < 0.0f ? -1.0f : 0.0f;
  L.group = A.Hq / A.Hkv;
  L.tok = p.tok;
  L.q_rows = A.T < p.tok ? A.T : p.tok;
  L.slot_rows = p.slot_rows;
  L.box = Sh::NK;
  while (A.page_size % L.box) L.box /= 2;
  if (!make_map<3>(&L.q, A.q, bf, {A.D, A.Hq, A.rows}, {A.q_stride[1], A.q_stride[0]}, {L.group, L.q_rows}) ||
      !make_map<3>(&L.k_new, A.k_new, bf, {A.D, A.Hkv, A.rows}, {A.k_new_stride[1], A.k_new_stride[0]}, {1, 8}) ||
      !make_map<3>(&L.v_new, A.v_new, bf, {A.D, A.Hkv, A.rows}, {A.v_new_stride[1], A.v_new_stride[0]}, {1, 8}))
    return SPEC_ERR_CUDA;
  // Without a cache no context has a page to read: the maps then cover the pass's own keys.
  const bool cache = A.pages > 0;
  const void *kc = cache ? A.k_cache : A.k_new, *vc = cache ? A.v_cache : A.v_new;
  const long long pages = cache ? A.pages : 1, page = cache ? A.page_size : 1, heads = A.Hkv;
  L.beyond = (int)pages;
  const int chunks = (A.D + 63) / 64;
  auto fold_of = [&](const long long* s) {
    if (!cache || A.D % 64 || chunks == 1 || s[1] >= kMaxStride / 8) return 0;
    return s[2] == A.D ? 1 : s[0] == heads * s[2] && pages * heads <= 0x7FFFFFFFll ? 2 : 0;
  };
  L.fold_k = fold_of(A.k_stride);
  L.fold_v = fold_of(A.v_stride);
  if (!L.fold_k || !L.fold_v) L.fold_k = L.fold_v = 0;  // both tiles lie alike
  L.row8 = L.fold_k ? chunks * 1024 : 1024;
  L.col = L.fold_k ? 1024 : Sh::kChunk;
  for (int i = 0; i < 2; ++i) {
    const long long* s = i ? A.v_stride : A.k_stride;
    const long long same[3] = {A.D, A.D, A.D};
    if (!cache) s = same;
    for (int small = 0; small < 2; ++small) {
      CUtensorMap* m = i ? (small ? &L.v8 : &L.v) : (small ? &L.k8 : &L.k);
      const int fold = i ? L.fold_v : L.fold_k;
      if (fold && !small) {
        const long long cols = fold == 1 ? heads * chunks : chunks, last = fold == 1 ? pages : pages * heads;
        if (!make_map<5>(m, i ? vc : kc, bf, {64, 8, cols, page / 8, last}, {s[1], 64, 8 * s[1], s[fold == 1 ? 0 : 2]},
                         {8, chunks, L.box / 8, 1}))
          return SPEC_ERR_CUDA;
        continue;
      }
      if (!make_map<4>(m, i ? vc : kc, bf, {A.D, page, heads, pages}, {s[1], s[2], s[0]}, {small ? 8 : L.box, 1, 1}))
        return SPEC_ERR_CUDA;
    }
  }
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  ssv::attend_kernel<E, DP, MT><<<grid, Sh::kThreads, Sh::kSmem, st>>>(L);
  if (count_launch(cudaGetLastError()) != cudaSuccess) return SPEC_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  const int unit_rows = A.T < MT * p.tok ? A.T : MT * p.tok;  // of the pass, at most
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((unit_rows * L.group + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return from_cuda(count_launch(cudaLaunchKernelEx(&cfg, ssv::attend_join_kernel<E, DP, MT>, L)));
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  if (B < 0 || T < 1 || T > kMaxPassRows || Hkv < 1 || Hq < 1 || Hq % Hkv || D < 8 || D > 256 || D % 8 ||
      Hq / Hkv > ssv::kAttendMaxGroup)
    return 0;
  return attend_plan(T, Hq / Hkv, D, nullptr).bytes;
}

spec_status_t spec_tree_attention(const spec_attention_t* args, uint32_t* dev_status, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!args) return SPEC_ERR_INVALID_ARG;
  const spec_attention_t& A = *args;
  if (A.B < 0 || A.T < 1 || A.rows < 0 || A.Hkv < 1 || A.Hq < 1 || A.Hq % A.Hkv || A.D < 1 || A.pages < 0 ||
      A.page_size < 1 || A.table_width < 0 || (A.dtype != SPEC_BF16 && A.dtype != SPEC_F16) ||
      !std::isfinite(A.scale * 1.4426950409f))
    return SPEC_ERR_INVALID_ARG;
  if (!A.row_offsets && (long long)A.B * A.T != A.rows) return SPEC_ERR_INVALID_ARG;
  if (A.D > 256 || A.D % 8 || A.page_size % 8 || A.T > kMaxPassRows || A.Hq / A.Hkv > ssv::kAttendMaxGroup ||
      (long long)A.table_width * A.page_size > 0x7FFFFFFFll)
    return SPEC_ERR_UNSUPPORTED;
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
  if (!aligned(workspace, 256)) return SPEC_ERR_INVALID_ARG;
  const AttendPlan p = attend_plan(A.T, A.Hq / A.Hkv, A.D, workspace);
  const bool bf = A.dtype == SPEC_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSV_ATTEND(DP, MT) \
  return bf ? run_attend<__nv_bfloat16, DP, MT>(A, p, dev_status, st) : run_attend<__half, DP, MT>(A, p, dev_status, st)
  if (p.dp == 64) {
    if (p.mt == 1) SSV_ATTEND(64, 1);
    SSV_ATTEND(64, 2);
  }
  if (p.dp == 128) {
    if (p.mt == 1) SSV_ATTEND(128, 1);
    SSV_ATTEND(128, 2);
  }
  SSV_ATTEND(256, 1);
#undef SSV_ATTEND
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
  // Slices of 16 KB, twice that where reading the history for each of them would come to
  // more than a quarter of the logits' bytes, and shorter ones where requests are few.
  const long long short_slice = ssv::adjust_slice(es), least = 16ll * A.history_width * A.B / ((long long)A.rows * es);
  const long long want = least > short_slice ? 2 * short_slice : short_slice;
  int parts = (int)((A.V + want - 1) / want);
  while ((long long)A.B * (parts + 1) <= 4ll * sms && A.V / parts > 2048) ++parts;
  ssv::AdjustParams P = {A, dev_status, ((A.V + parts - 1) / parts + 63) / 64 * 64};
  const size_t smem = ssv::adjust_smem(P.slice, es, A.biases, A.T);
  static std::once_flag once[2][kMaxDevices];
  static cudaError_t made[2][kMaxDevices];
  const int which = A.dtype == SPEC_BF16;
  std::call_once(once[which][dev], [which, dev]() {
    const int el = which ? 2 : 4;
    const int most = (int)ssv::adjust_smem(2 * ssv::adjust_slice(el), el, ssv::kAdjustMaxBiases, ssv::kAdjustMaxRows);
    made[which][dev] =
        which ? cudaFuncSetAttribute(ssv::adjust_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)
              : cudaFuncSetAttribute(ssv::adjust_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (made[which][dev] != cudaSuccess) return SPEC_ERR_CUDA;
  const dim3 grid((unsigned)((A.V + P.slice - 1) / P.slice), (unsigned)A.B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (which)
    ssv::adjust_kernel<__nv_bfloat16><<<grid, ssv::adjust_threads(P.slice), smem, st>>>(P);
  else
    ssv::adjust_kernel<float><<<grid, ssv::adjust_threads(P.slice), smem, st>>>(P);
  return from_cuda(count_launch(cudaGetLastError()));
}

}  // extern "C"
