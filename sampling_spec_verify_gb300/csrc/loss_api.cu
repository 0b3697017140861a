// Host side of the drafter-training losses: argument checks, workspace layout,
// launch shapes and launches.  No entry point allocates device memory or
// synchronises the stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "distill.cuh"
#include "head.cuh"
#include "spec_verify.h"

namespace ssv {
cudaError_t count_launch(cudaError_t e);  // spec_api.cu
}

namespace {

using ssv::count_launch;

constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;
constexpr int kMaxDevices = 64;

spec_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int elem_size(spec_dtype_t dt) { return dt == SPEC_F32 ? 4 : 2; }
bool any_dtype(spec_dtype_t dt) { return dt == SPEC_F32 || dt == SPEC_BF16 || dt == SPEC_F16; }

struct Device {
  int sms = 0, smem_optin = 0;
};
bool device(Device* out, int* id) {
  static Device cache[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::call_once(once[dev], [dev]() {
    cudaDeviceGetAttribute(&cache[dev].sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&cache[dev].smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  });
  *out = cache[dev];
  *id = dev;
  return out->sms > 0 && out->smem_optin > 0;
}

// Launch facts of one kernel instantiation, looked up once per device, cluster
// size and shared-memory size: a fixed table, so that no lookup can throw.
struct Residency {
  struct Entry {
    int S, smem, clusters;
  };
  static constexpr int kEntries = 64;
  std::mutex mu;
  bool attrs[kMaxDevices] = {};
  Entry e[kMaxDevices][kEntries] = {};
  int n[kMaxDevices] = {};
};

// Clusters of S CTAs that fit on the device at once; sets the kernel's
// attributes on first use.  0 on failure.
int resident_clusters(Residency& r, const void* fn, int S, int smem, int threads, int dev, int smem_optin) {
  std::lock_guard<std::mutex> g(r.mu);
  for (int i = 0; i < r.n[dev]; ++i)
    if (r.e[dev][i].S == S && r.e[dev][i].smem == smem) return r.e[dev][i].clusters;
  if (!r.attrs[dev]) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess) return 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_optin - (int)fa.sharedSizeBytes) != cudaSuccess)
      return 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return 0;
    r.attrs[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (r.n[dev] < Residency::kEntries) r.e[dev][r.n[dev]++] = {S, smem, n};
  return n;
}

// Launches a kernel; all but the first of a call may start while the previous
// one drains (the kernels wait for it themselves).
template <class... P, class... A>
cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, int smem, int cluster, bool first, cudaStream_t st,
                   const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (!first) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return count_launch(cudaLaunchKernelEx(&cfg, fn, args...));
}

// Carves a workspace into 256-byte-aligned parts; with a null base it measures.
struct Carver {
  char* base;
  size_t used = 0;
  template <class T>
  T* take(size_t n) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += (n * sizeof(T) + 255) & ~size_t(255);
    return p;
  }
};

ssv::F2 split(double v) {
  const float hi = (float)v;
  return {hi, (float)(v - (double)hi)};
}

bool temperature_ok(float t) { return t > 0.0f && std::isfinite(t) && std::isfinite((float)(kLog2e / (double)t)); }

// ---- distillation of given logits ------------------------------------------------

struct DistillWs {
  ssv::LossScalars* scalars;
  float* t;
  ssv::RowTeacher* row;
  uint8_t* keep;
  float* zi;
  ssv::RowNorm* norm;
  float* row_loss;
  float4* part;
  size_t total;
};
DistillWs distill_ws(void* base, size_t N, size_t k) {
  Carver c{static_cast<char*>(base)};
  DistillWs w;
  w.scalars = c.take<ssv::LossScalars>(1);
  w.t = c.take<float>(N * k);
  w.row = c.take<ssv::RowTeacher>(N);
  w.keep = c.take<uint8_t>((N + 7) / 8 * 8);
  w.zi = c.take<float>(N * k);
  w.norm = c.take<ssv::RowNorm>(N);
  w.row_loss = c.take<float>(N);
  w.part = c.take<float4>((N + 7) / 8);
  w.total = c.used;
  return w;
}

// Rows of a call: the kernels count them in steps of 8 and 256 with 32-bit integers.
constexpr int kMaxRows = 1 << 30;

// Slices of a row: what a CTA's threads hold in registers (one stage: it is free
// again as soon as they do); rows too long for 16 such slices stay in shared memory, with
// two stages or one.  Short batches spread a row over more CTAs.
struct DistillShape {
  int S = 0, nst = 0;
  bool regs = false;
  uint32_t cap = 0;
};
DistillShape distill_shape(long long row_bytes, int N, int sms, bool wide) {
  const long long budget[3] = {wide ? ssv::kDVecs * ssv::kDThreads * 16 : -1, 104 * 1024, 208 * 1024};
  DistillShape d;
  for (int level = 0; level < 3 && !d.S; ++level)
    for (int s = 1; s <= ssv::kDMaxCluster; s *= 2)
      if ((row_bytes / 16 + s - 1) / s * 16 <= budget[level]) {
        d.S = s;
        d.regs = level == 0;
        d.nst = level == 1 ? 2 : 1;
        break;
      }
  if (!d.S) return d;
  while (d.S < 8 && (long long)N * d.S < sms && row_bytes / d.S > 8192) d.S *= 2;
  d.cap = (uint32_t)((((row_bytes / 16 + d.S - 1) / d.S) * 16 + 127) & ~127ll);
  if (!d.cap) d.cap = 128;
  return d;
}

template <class E, class O, int NV>
spec_status_t launch_distill_nv(ssv::DistillParams P, const DistillShape& sh, const Device& d, int dev,
                                cudaStream_t st) {
  static Residency res;
  const void* fn = (const void*)ssv::distill_kernel<E, O, NV>;
  P.nst = sh.nst;
  P.cap = sh.cap;
  const int smem = (int)(sh.cap * (uint32_t)sh.nst);
  const int fit = resident_clusters(res, fn, sh.S, smem, ssv::kDThreads, dev, d.smem_optin);
  if (fit <= 0) return SPEC_ERR_CUDA;
  const int G = P.N < fit ? P.N : fit;
  // Two CTAs take all registers of an SM: started around the previous kernel's
  // CTAs, a full grid lands unevenly (1792 x 151936: 353 us a pass against 288).
  const bool plain = G * sh.S > d.sms;
  return from_cuda(launch(ssv::distill_kernel<E, O, NV>, dim3((unsigned)(G * sh.S)), ssv::kDThreads, smem, sh.S, plain,
                          st, P));
}

template <class E, class O>
spec_status_t launch_distill(const ssv::DistillParams& P, cudaStream_t st) {
  Device d;
  int dev = 0;
  if (!device(&d, &dev)) return SPEC_ERR_CUDA;
  const DistillShape sh = distill_shape((long long)P.V * (long long)sizeof(E), P.N, d.sms, P.wide != 0);
  if (!sh.S) return SPEC_ERR_UNSUPPORTED;
  if (!sh.regs) return launch_distill_nv<E, O, 0>(P, sh, d, dev, st);
  const int vecs = (int)(sh.cap / 16 + ssv::kDThreads - 1) / ssv::kDThreads;
  switch (vecs <= 4 ? 0 : (vecs - 2) / 3) {  // the next of 4, 7, 10, ...
    case 0: return launch_distill_nv<E, O, 4>(P, sh, d, dev, st);
    case 1: return launch_distill_nv<E, O, 7>(P, sh, d, dev, st);
    case 2: return launch_distill_nv<E, O, 10>(P, sh, d, dev, st);
    case 3: return launch_distill_nv<E, O, 13>(P, sh, d, dev, st);
    case 4: return launch_distill_nv<E, O, 16>(P, sh, d, dev, st);
    default: return launch_distill_nv<E, O, ssv::kDVecs>(P, sh, d, dev, st);
  }
}

spec_status_t distill(const void* student, spec_dtype_t dtype, int N, int V, int k, float temperature,
                      float grad_scale, const int32_t* ids, const float* logits, const float* lse,
                      const float* weight, spec_reduction_t reduction, float* loss, float* row_loss, bool want_grad,
                      void* grad, spec_dtype_t grad_dtype, uint32_t* status, void* workspace, size_t bytes,
                      void* stream) {
  if (N < 0 || V < 1 || k < 1 || !any_dtype(dtype)) return SPEC_ERR_INVALID_ARG;
  if (reduction != SPEC_MEAN && reduction != SPEC_SUM) return SPEC_ERR_INVALID_ARG;
  if (!temperature_ok(temperature) || !std::isfinite(grad_scale)) return SPEC_ERR_INVALID_ARG;
  if (want_grad && grad_dtype != dtype && grad_dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
  if (!loss) return SPEC_ERR_INVALID_ARG;
  if (N > kMaxRows || k > ssv::kMaxEntries || !distill_shape((long long)V * elem_size(dtype), N, 1, false).S)
    return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) return from_cuda(cudaMemsetAsync(loss, 0, sizeof(float), st));
  if (!student || !ids || !logits || (want_grad && !grad)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(student, elem_size(dtype)) || (want_grad && !aligned(grad, elem_size(grad_dtype))))
    return SPEC_ERR_INVALID_ARG;
  const DistillWs ws = distill_ws(workspace, (size_t)N, (size_t)k);
  if (!workspace || bytes < ws.total || !aligned(workspace, 256)) return SPEC_ERR_INVALID_ARG;

  ssv::TargetParams tp = {};
  tp.ids = ids;
  tp.logits = logits;
  tp.lse = lse;
  tp.N = N;
  tp.V = V;
  tp.k = k;
  tp.inv_t = split(1.0 / (double)temperature);
  tp.t = ws.t;
  tp.row = ws.row;
  tp.keep = ws.keep;
  tp.scalars = ws.scalars;
  tp.status = status;
  const unsigned row_grid = (unsigned)((N + ssv::kTargetWarps - 1) / ssv::kTargetWarps);
  if (launch(ssv::targets_kernel<false>, dim3(row_grid), ssv::kTargetWarps * 32, 0, 0, true, st, tp) != cudaSuccess)
    return SPEC_ERR_CUDA;

  ssv::DistillParams P = {};
  P.z = student;
  P.grad = grad;
  P.N = N;
  P.V = V;
  P.k = k;
  P.skew = (int)((reinterpret_cast<uintptr_t>(student) & 15) / (uintptr_t)elem_size(dtype));
  P.odd = P.skew != 0 || ((long long)V * elem_size(dtype)) % 16 != 0;
  P.wide = 1;
  if (want_grad) {
    const uintptr_t o = reinterpret_cast<uintptr_t>(grad) - (uintptr_t)P.skew * (uintptr_t)elem_size(grad_dtype);
    P.wide = (o & (dtype != SPEC_F32 && grad_dtype == SPEC_F32 ? 31 : 15)) == 0;
  }
  P.s = (float)(kLog2e / (double)temperature);
  P.ids = ids;
  P.t = ws.t;
  P.row = ws.row;
  P.keep = ws.keep;
  P.weight = weight;
  P.mean = reduction == SPEC_MEAN;
  P.tail = lse != nullptr;
  P.gscale = (float)((double)grad_scale / (double)temperature);
  P.zi = ws.zi;
  P.norm = ws.norm;
  P.status = status;
  spec_status_t r;
  const bool wide = want_grad && grad_dtype == SPEC_F32;
  using B = __nv_bfloat16;
  using Hf = __half;
  if (dtype == SPEC_F32)
    r = want_grad ? launch_distill<float, float>(P, st) : launch_distill<float, ssv::NoGrad>(P, st);
  else if (dtype == SPEC_BF16)
    r = !want_grad ? launch_distill<B, ssv::NoGrad>(P, st)
                   : (wide ? launch_distill<B, float>(P, st) : launch_distill<B, B>(P, st));
  else
    r = !want_grad ? launch_distill<Hf, ssv::NoGrad>(P, st)
                   : (wide ? launch_distill<Hf, float>(P, st) : launch_distill<Hf, Hf>(P, st));
  if (r != SPEC_OK) return r;

  ssv::FinishParams F = {};
  F.N = N;
  F.k = k;
  F.inv_t = tp.inv_t;
  F.c = split((double)P.s * kLn2);  // the exponents' own factor
  F.part = ws.part;
  F.logits = logits;
  F.t = ws.t;
  F.row = ws.row;
  F.keep = ws.keep;
  F.weight = weight;
  F.zi = ws.zi;
  F.mean = P.mean;
  F.grad_scale = P.gscale;
  F.store_scale = 1.0f;
  F.loss = loss;
  F.row_loss = row_loss ? row_loss : ws.row_loss;
  F.scalars = ws.scalars;
  F.status = status;
  return from_cuda(launch(ssv::distill_finish_kernel, dim3((unsigned)((N + 7) / 8)), 256, 0, 0, false, st, F,
                          (const ssv::RowNorm*)ws.norm));
}

// ---- losses through the head --------------------------------------------------------

// CTA pairs in flight on this GPU's 152 SMs, for the split rule.  A constant: the size
// of a workspace, which the splits enter, is asked for without a device at hand.
constexpr int kPairs = 76;
// A batch whose probabilities fit kKeepBytes, a 64th of this GPU's memory (2 bytes
// an entry for bf16; 6 for fp16, which keeps them in fp32 beside D), keeps them
// between the passes; the others go in pieces of kPieceBytes and compute the logits
// twice.  Both gradients, kept against in pieces: bf16 1792 x 151936 x 2048 2.3 ms
// against 2.8, 8192 x 151936 x 2048 10.3 against 12.2; fp16 4096 x 129280 x 2048 4.7
// against 5.6.
constexpr size_t kKeepBytes = (size_t)4096 << 20;
constexpr size_t kPieceBytes = (size_t)256 << 20;
constexpr long long kLeastTiles = 8;

// How a call is cut: pieces of the vocabulary and splits of a piece's depth in
// the product that gives the hidden states' gradient.
struct HeadPlan {
  bool kept;       // one piece, pass 1's probabilities kept
  bool kept32;     // in fp32
  int piece;       // tokens per piece, a multiple of 256
  int pieces;
  int splits;
  int slot_rows;
};
// `most`: tiles of 256 tokens a piece has at most, for a caller whose workspace is
// smaller than the preferred one (head_fit); 0: the rule above.
HeadPlan head_plan(int N, int V, int H, bool bf16, long long most = 0) {
  HeadPlan p;
  const long long vt = ((long long)V + 255) / 256;
  long long cap = (long long)(kPieceBytes / 2 / (size_t)N) / 256;  // tiles of tokens
  if (cap < kLeastTiles) cap = kLeastTiles;
  p.kept32 = !bf16;
  p.kept = !most && (size_t)N * (size_t)vt * (bf16 ? 512 : 1536) <= kKeepBytes;
  if (p.kept) cap = vt;
  if (most && most < cap) cap = most;
  p.pieces = (int)((vt + cap - 1) / cap);
  p.piece = (int)((vt + p.pieces - 1) / p.pieces) * 256;
  p.pieces = (int)(((long long)V + p.piece - 1) / p.piece);
  p.slot_rows = (N + 255) / 256 * 256;
  // The tiles of N x H may be far fewer than the CTA pairs: the depth is split
  // until the last wave is full, at no less than 1024 tokens a split.
  const long long tiles = (long long)(p.slot_rows / 256) * ((H + 255) / 256);
  double best = 0.0;
  p.splits = 1;
  for (int s = 1; s <= 32 && (s == 1 || p.piece / s >= 1024); ++s) {
    const long long n = tiles * s;
    const double waves = (double)((n + kPairs - 1) / kPairs);
    const double eff = (double)n / (waves * kPairs) / (1.0 + 0.01 * s);
    if (eff > best) {
      best = eff;
      p.splits = s;
    }
  }
  return p;
}

// Rows that start off a 32-byte sector cost the products a quarter of their rate
// (1001 x 50257, bf16: H = 1536 94 us, 1544 125, 1552 103); the copy of the hidden
// states puts them on whole lines.  (The head is too large to copy.)
size_t pitch_of(size_t H) { return H % 16 ? (H + 63) / 64 * 64 : H; }

// A tensor map over less than 128 KB is read slowly (measured; the order of the reads
// makes no difference, the rows outside of the batch may hold anything).  Pass 1 of
// eight rows, by the bytes that the map of the hidden states covers, 32 KB / 64 / 128 /
// 256: 151936 x 2048 183 / 179 / 141 / 141 us, 151936 x 1024 109 / 107 / 94 / 92.  So
// calls with gradients extend their copy of the hidden states by rows that nothing
// looks at, and calls without copy them too where the head is longer than the L2
// (32000 x 1024: no difference).  Such calls also copy rows that start off a sector
// where several tiles of rows read the head (1000 x 151936 x 1544: 293 us against 322;
// 300 x 8000 x 1544: 32 against 28).
constexpr size_t kMapBytes = (size_t)128 << 10;
size_t copy_rows(size_t N, size_t H) {
  const size_t least = (kMapBytes / 2 + pitch_of(H) - 1) / pitch_of(H);
  return N > least ? N : least;
}
bool copies(size_t N, size_t V, size_t H, bool grads) {
  return grads || (V * H * 2 >= (size_t)128 << 20 && (N * H * 2 < kMapBytes || (H % 16 != 0 && N > 256)));
}

struct HeadWs {
  uint16_t* x;    // hidden states by place, at pitch_of(H), or null: as they lie
  int32_t* perm;  // row at each place
  uint32_t* keys;   // listed tokens in order, and where each tile of tokens begins
  uint16_t* starts; // (not for cross entropy)
  ssv::LossScalars* scalars;
  float* t;
  ssv::RowTeacher* row;
  uint8_t* keep;
  float* zi;
  float* row_loss;
  float* lse2;
  float4* sums;
  float2* part;
  float* hidden;
  uint16_t* d;
  float* e;  // fp32 probabilities
  size_t total;
};
HeadWs head_ws(void* base, const HeadPlan& p, size_t N, size_t V, size_t H, size_t k, bool listed, bool gh, bool gw) {
  Carver c{static_cast<char*>(base)};
  HeadWs w;
  w.scalars = c.take<ssv::LossScalars>(1);
  const bool grads = gh || gw;
  const bool copy = copies(N, V, H, grads);
  w.perm = copy ? c.take<int32_t>(N) : nullptr;
  w.t = c.take<float>(N * k);
  w.row = c.take<ssv::RowTeacher>(N);
  w.keep = c.take<uint8_t>((N + 7) / 8 * 8);
  w.zi = c.take<float>(N * k);
  w.row_loss = c.take<float>(N);
  w.lse2 = c.take<float>(N);
  w.sums = c.take<float4>((N + 7) / 8);
  w.keys = listed ? c.take<uint32_t>(N * k) : nullptr;
  w.starts = listed ? c.take<uint16_t>(N * ((V + 255) / 256 + 1)) : nullptr;
  w.part = c.take<float2>(N * ((V + 255) / 256));
  w.hidden = gh ? c.take<float>((size_t)p.splits * (size_t)p.slot_rows * H) : nullptr;
  w.d = grads ? c.take<uint16_t>(N * (size_t)p.piece) : nullptr;
  w.e = grads && p.kept && p.kept32 ? c.take<float>(N * (size_t)p.piece) : nullptr;
  w.x = copy ? c.take<uint16_t>(copy_rows(N, H) * pitch_of(H)) : nullptr;
  w.total = c.used;
  return w;
}

// The plan for a workspace of `bytes`: the preferred one where it fits, else without
// kept probabilities, in pieces of the vocabulary as long as they fit, down to kLeastTiles.
HeadPlan head_fit(int N, int V, int H, int k, bool bf16, bool listed, bool gh, bool gw, size_t bytes) {
  auto total = [&](const HeadPlan& p) {
    return head_ws(nullptr, p, (size_t)N, (size_t)V, (size_t)H, (size_t)k, listed, gh, gw).total;
  };
  HeadPlan p = head_plan(N, V, H, bf16);
  long long tiles = p.piece / 256;
  while (total(p) > bytes && (p.kept || tiles > kLeastTiles)) {
    if (!p.kept) tiles -= tiles / 8 > 1 ? tiles / 8 : 1;
    p = head_plan(N, V, H, bf16, tiles);
  }
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

// Row-major [rows, cols] matrix, tiles of box_rows x 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, spec_dtype_t dt, long long rows, long long cols, long long ld,
              int box_rows) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const int es = elem_size(dt);
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * (cuuint64_t)es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  const CUtensorMapDataType t = dt == SPEC_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dt == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  // Rows that start off a sector are read in 128-byte steps (1000 x 151936 x 1544,
  // bf16, without gradients: 333 us against 417 in 256-byte steps, with both 1080 against
  // 1115; of other rows the step makes no difference).
  const CUtensorMapL2promotion l2 =
      strides[0] % 32 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  return enc(m, t, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A product of M x N results, K deep.
ssv::Product product(int M, int N, int K, int splits, int b_off) {
  const int ksteps = (K + ssv::kTileK - 1) / ssv::kTileK;
  return {M, N, K, splits < ksteps ? splits : ksteps, b_off};
}
long long tiles_of(const ssv::Product& p) {
  return (long long)((p.M + ssv::kTileM - 1) / ssv::kTileM) * ((p.N + ssv::kTileN - 1) / ssv::kTileN) * p.splits;
}

// Launches the first (which & 1) and the second (which & 2) product of L.
template <ssv::HeadOp OP, bool OUT32>
spec_status_t launch_head(ssv::HeadLaunch& L, int which, cudaStream_t st) {
  static Residency res;
  const void* fn = (const void*)ssv::head_kernel<OP, OUT32>;
  Device d;
  int dev = 0;
  if (!device(&d, &dev)) return SPEC_ERR_CUDA;
  const int fit = resident_clusters(res, fn, 2, ssv::kHeadSmem, ssv::kHeadThreads, dev, d.smem_optin);
  if (fit <= 0) return SPEC_ERR_CUDA;
  const long long tiles = ((which & 1) ? tiles_of(L.p[0]) : 0) + ((which & 2) ? tiles_of(L.p[1]) : 0);
  if (tiles > 0x7FFFFFF) return SPEC_ERR_UNSUPPORTED;
  L.which = which;
  const int G = tiles < fit ? (int)tiles : fit;  // pairs without a tile leave at once
  return from_cuda(launch(ssv::head_kernel<OP, OUT32>, dim3((unsigned)(2 * G)), ssv::kHeadThreads, ssv::kHeadSmem, 0,
                          false, st, L));
}

struct HeadCall {
  const void *hidden, *weight;
  spec_dtype_t dtype;
  int N, V, H, k;
  float temperature, grad_scale;
  const int32_t* ids;
  const float* logits;  // null: cross entropy, ids are labels
  int ignore;
  const float* row_weight;
  spec_reduction_t reduction;
  float *loss, *row_loss, *lse;
  void *grad_hidden, *grad_weight;
  spec_dtype_t grad_dtype;
  uint32_t* status;
  void* workspace;
  size_t bytes;
  void* stream;
};

template <class E>
spec_status_t head_run(const HeadCall& c, const HeadPlan& plan, const HeadWs& ws) {
  cudaStream_t st = static_cast<cudaStream_t>(c.stream);
  const E* x = static_cast<const E*>(c.hidden);
  const E* w = static_cast<const E*>(c.weight);
  const double s = kLog2e / (double)c.temperature;
  const float store_scale = c.dtype == SPEC_F16 ? 32768.0f : 1.0f;
  const long long entries = (long long)c.N * c.k;

  ssv::TargetParams tp = {};
  tp.ids = c.ids;
  tp.logits = c.logits;
  tp.N = c.N;
  tp.V = c.V;
  tp.k = c.k;
  tp.ignore = c.ignore;
  tp.inv_t = split(1.0 / (double)c.temperature);
  tp.t = ws.t;
  tp.row = ws.row;
  tp.keep = ws.keep;
  tp.scalars = ws.scalars;
  tp.status = c.status;
  tp.tile = ssv::kTileN;
  tp.tiles = (c.V + ssv::kTileN - 1) / ssv::kTileN;
  tp.keys = ws.keys;
  tp.starts = ws.starts;
  const bool grads = c.grad_hidden || c.grad_weight;
  const int ldx = ws.x ? (int)pitch_of((size_t)c.H) : c.H;
  const void* xp = ws.x ? (const void*)ws.x : (const void*)x;
  const int per = 8 * ((c.N + 8191) / 8192);  // rows per CTA of the kernels that look at all rows
  const dim3 per_grid((unsigned)((c.N + per - 1) / per));
  const uint4* x16 = reinterpret_cast<const uint4*>(x);
  uint4* xp16 = reinterpret_cast<uint4*>(ws.x);
  if (!c.logits) {
    if (launch(ssv::label_rows_kernel, per_grid, 256, 0, 0, true, st, tp, per, x16, xp16, c.H / 8, ldx / 8, ws.perm) !=
        cudaSuccess)
      return SPEC_ERR_CUDA;
  } else {
    if (launch(ssv::targets_kernel<true>, dim3((unsigned)((c.N + ssv::kTargetWarps - 1) / ssv::kTargetWarps)),
               ssv::kTargetWarps * 32, 0, 0, true, st, tp) != cudaSuccess)
      return SPEC_ERR_CUDA;
    if (ws.x && launch(ssv::compact_kernel, per_grid, 256, 0, 0, false, st, (const uint8_t*)ws.keep, c.N, per, x16,
                        xp16, c.H / 8, ldx / 8, ws.perm, ws.scalars) != cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  const bool kept = grads && plan.kept;
  ssv::HeadLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.bf16 = c.dtype == SPEC_BF16;
  L.s = (float)s;
  L.part = ws.part;
  L.zi = ws.zi;
  L.labels = c.logits ? nullptr : c.ids;
  L.keys = ws.keys;
  L.starts = ws.starts;
  L.k = c.k;
  L.status = c.status;
  L.scalars = ws.scalars;
  L.lse2 = ws.lse2;
  L.weight = c.row_weight;
  L.keep = ws.keep;
  L.perm = ws.perm;
  L.store_scale = store_scale;
  L.slot_rows = plan.slot_rows;
  // 128-row boxes along K
  const long long map_rows = ws.x ? (long long)copy_rows((size_t)c.N, (size_t)c.H) : c.N;
  if (!make_map(&L.a[0], xp, c.dtype, map_rows, c.H, ldx, 128) || !make_map(&L.b[0], w, c.dtype, c.V, c.H, c.H, 128))
    return SPEC_ERR_CUDA;
  constexpr bool kWide = std::is_same<E, __half>::value;
  using S = typename std::conditional<kWide, float, __half>::type;  // of kept probabilities
  const void* room = kWide ? (const void*)ws.e : (const void*)ws.d;
  if (kept && !make_map(&L.out[0], room, kWide ? SPEC_F32 : SPEC_F16, c.N, c.V, plan.piece, 32)) return SPEC_ERR_CUDA;
  L.p[0] = product(c.N, c.V, c.H, 1, 0);
  spec_status_t r = kept ? launch_head<ssv::kHeadKeep, kWide>(L, 1, st) : launch_head<ssv::kHeadNorm, false>(L, 1, st);
  if (r != SPEC_OK) return r;

  ssv::FinishParams F = {};
  F.N = c.N;
  F.k = c.k;
  F.inv_t = tp.inv_t;
  F.c = split((double)L.s * kLn2);  // the exponents' own factor
  F.part = ws.sums;
  F.logits = c.logits;
  F.t = ws.t;
  F.row = ws.row;
  F.keep = ws.keep;
  F.weight = c.row_weight;
  F.zi = ws.zi;
  F.mean = c.reduction == SPEC_MEAN;
  F.grad_scale = (float)((double)c.grad_scale / (double)c.temperature);
  F.store_scale = store_scale;
  F.loss = c.loss;
  F.row_loss = c.row_loss ? c.row_loss : ws.row_loss;
  F.scalars = ws.scalars;
  F.status = c.status;
  if (launch(ssv::head_finish_kernel, dim3((unsigned)((c.N + 7) / 8)), 256, 0, 0, false, st, F,
             (const float2*)ws.part, (c.V + 255) / 256, (const int32_t*)ws.perm, c.lse, ws.lse2,
             reinterpret_cast<uint4*>(ws.x), ldx / 8) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (!grads) return SPEC_OK;

  L.count = &ws.scalars->count;  // from here on, only rows that count
  // the backward products: 64-row boxes along the other dimension
  ssv::HeadLaunch B = L;
  if (!make_map(&B.b[0], w, c.dtype, c.V, c.H, c.H, 64) || !make_map(&B.b[1], xp, c.dtype, c.N, c.H, ldx, 64))
    return SPEC_ERR_CUDA;
  if (c.grad_hidden &&
      !make_map(&B.out[0], ws.hidden, SPEC_F32, (long long)plan.splits * plan.slot_rows, c.H, c.H, 32))
    return SPEC_ERR_CUDA;
  ssv::ListedParams Q = {};
  Q.ids = c.ids;
  Q.t = ws.t;
  Q.zi = ws.zi;
  Q.lse2 = ws.lse2;
  Q.weight = c.row_weight;
  Q.keep = ws.keep;
  Q.perm = ws.perm;
  Q.scalars = ws.scalars;
  Q.N = c.N;
  Q.k = c.k;
  Q.ld = plan.piece;
  Q.s = (double)L.s;
  Q.store_scale = store_scale;
  E* d = reinterpret_cast<E*>(ws.d);
  int slots = 0;
  for (int i = 0; i < plan.pieces; ++i) {
    const int v0 = i * plan.piece;
    const int C = c.V - v0 < plan.piece ? c.V - v0 : plan.piece;
    Q.v0 = v0;
    Q.C = C;
    if (kept) {
      const dim3 grid((unsigned)c.N, (unsigned)((C + ssv::kDenseCols - 1) / ssv::kDenseCols));
      if (launch(ssv::dense_grads_kernel<E, S>, grid, 256, 0, 0, false, st, Q, (const float2*)ws.part,
                 static_cast<const S*>(room), d) != cudaSuccess)
        return SPEC_ERR_CUDA;
    } else {
      if (!make_map(&L.out[0], ws.d, c.dtype, c.N, C, plan.piece, 32)) return SPEC_ERR_CUDA;
      L.p[0] = product(c.N, C, c.H, 1, v0);
      if ((r = launch_head<ssv::kHeadGrad, false>(L, 1, st)) != SPEC_OK) return r;
      if (launch(ssv::listed_grads_kernel<E>, dim3((unsigned)((entries + 255) / 256)), 256, 0, 0, false, st, Q, d) !=
          cudaSuccess)
        return SPEC_ERR_CUDA;
    }

    if (!make_map(&B.a[0], ws.d, c.dtype, c.N, C, plan.piece, 128) ||
        !make_map(&B.a[1], ws.d, c.dtype, c.N, C, plan.piece, 64))
      return SPEC_ERR_CUDA;
    B.p[0] = product(c.N, c.H, C, plan.splits, v0);
    B.p[1] = product(C, c.H, c.N, 1, 0);
    B.first = i == 0;
    if (i == 0) slots = B.p[0].splits;  // later pieces are no longer than the first
    if (c.grad_weight) {
      const int es = elem_size(c.grad_dtype);
      if (!make_map(&B.out[1], static_cast<char*>(c.grad_weight) + (size_t)v0 * (size_t)c.H * (size_t)es, c.grad_dtype,
                    C, c.H, c.H, 32))
        return SPEC_ERR_CUDA;
    }
    const int which = (c.grad_hidden ? 1 : 0) | (c.grad_weight ? 2 : 0);
    r = c.grad_weight && c.grad_dtype == SPEC_F32 ? launch_head<ssv::kHeadBack, true>(B, which, st)
                                                  : launch_head<ssv::kHeadBack, false>(B, which, st);
    if (r != SPEC_OK) return r;
  }
  if (c.grad_hidden) {
    const long long elems = (long long)c.N * c.H;
    const long long slot = (long long)plan.slot_rows * c.H;
    const bool many = slots >= 8;
    const int per = many ? 64 : 256;
    const dim3 grid((unsigned)((elems / 4 + per - 1) / per));
    const ssv::LossScalars* sc = ws.scalars;
    const float* part = ws.hidden;
    const int32_t* perm = ws.perm;
    auto out = [&](auto* g) {
      using O = typename std::remove_pointer<decltype(g)>::type;
      return many ? launch(ssv::hidden_out_kernel<O, 4>, grid, 256, 0, 0, false, st, part, slots, slot, elems, c.H, perm, sc, g)
                  : launch(ssv::hidden_out_kernel<O, 1>, grid, 256, 0, 0, false, st, part, slots, slot, elems, c.H, perm, sc, g);
    };
    const cudaError_t e = c.grad_dtype == SPEC_F32 ? out(static_cast<float*>(c.grad_hidden))
                                                   : out(static_cast<E*>(c.grad_hidden));
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

bool head_dims_ok(int N, int V, int H, int k) { return N >= 0 && V >= 1 && H >= 8 && H % 8 == 0 && k >= 1; }
bool head_dims_fit(int N, int V, int H, int k) {
  return N <= (1 << 20) && V < (1 << 24) && H <= (1 << 16) && k <= ssv::kMaxEntries;
}

spec_status_t head_loss(const HeadCall& c, bool grads) {
  if (!head_dims_ok(c.N, c.V, c.H, c.k)) return SPEC_ERR_INVALID_ARG;
  if (c.dtype != SPEC_BF16 && c.dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
  if (c.reduction != SPEC_MEAN && c.reduction != SPEC_SUM) return SPEC_ERR_INVALID_ARG;
  if (!temperature_ok(c.temperature) || !std::isfinite(c.grad_scale) || !c.loss) return SPEC_ERR_INVALID_ARG;
  if (grads && ((!c.grad_hidden && !c.grad_weight && c.N > 0) ||
                (c.grad_dtype != c.dtype && c.grad_dtype != SPEC_F32)))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(c.grad_hidden, 16) || !aligned(c.grad_weight, 16)) return SPEC_ERR_INVALID_ARG;
  if (!head_dims_fit(c.N, c.V, c.H, c.k)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(c.stream);
  if (c.N == 0) {
    cudaError_t e = cudaMemsetAsync(c.loss, 0, sizeof(float), st);
    if (e == cudaSuccess && c.grad_weight)
      e = cudaMemsetAsync(c.grad_weight, 0, (size_t)c.V * (size_t)c.H * (size_t)elem_size(c.grad_dtype), st);
    return from_cuda(e);
  }
  if (!c.hidden || !c.weight || !c.ids || !aligned(c.hidden, 16) || !aligned(c.weight, 16)) return SPEC_ERR_INVALID_ARG;
  const HeadPlan plan = head_fit(c.N, c.V, c.H, c.k, c.dtype == SPEC_BF16, c.logits != nullptr,
                                 c.grad_hidden != nullptr, c.grad_weight != nullptr, c.bytes);
  const HeadWs ws = head_ws(c.workspace, plan, (size_t)c.N, (size_t)c.V, (size_t)c.H, (size_t)c.k, c.logits != nullptr,
                            c.grad_hidden != nullptr,
                            c.grad_weight != nullptr);
  if (!c.workspace || c.bytes < ws.total || !aligned(c.workspace, 256)) return SPEC_ERR_INVALID_ARG;
  return c.dtype == SPEC_BF16 ? head_run<__nv_bfloat16>(c, plan, ws) : head_run<__half>(c, plan, ws);
}

// Bytes of the workspace of a call that has room for `bytes`.
size_t head_workspace(spec_dtype_t dtype, int N, int V, int H, int k, bool gh, bool gw, size_t bytes) {
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return 0;
  if (!head_dims_ok(N, V, H, k) || !head_dims_fit(N, V, H, k)) return 0;
  if (N == 0) return 256;
  const HeadPlan p = head_fit(N, V, H, k, dtype == SPEC_BF16, true, gh, gw, bytes);
  return head_ws(nullptr, p, (size_t)N, (size_t)V, (size_t)H, (size_t)k, true, gh, gw).total;
}

}  // namespace

extern "C" {

size_t spec_topk_distill_workspace_bytes(int N, int V, int k) {
  if (N < 0 || N > kMaxRows || V < 1 || k < 1 || k > ssv::kMaxEntries) return 0;
  return distill_ws(nullptr, (size_t)N, (size_t)k).total;
}

spec_status_t spec_topk_distill(const void* student, spec_dtype_t dtype, int N, int V, int k, float temperature,
                                const int32_t* teacher_ids, const float* teacher_logits, const float* teacher_lse,
                                const float* row_weight, spec_reduction_t reduction, float* loss_out, float* row_loss,
                                uint32_t* dev_status, void* workspace, size_t workspace_bytes, void* stream) {
  return distill(student, dtype, N, V, k, temperature, 0.0f, teacher_ids, teacher_logits, teacher_lse, row_weight,
                 reduction, loss_out, row_loss, false, nullptr, dtype, dev_status, workspace, workspace_bytes, stream);
}

spec_status_t spec_topk_distill_fwd_bwd(const void* student, spec_dtype_t dtype, int N, int V, int k,
                                        float temperature, float grad_scale, const int32_t* teacher_ids,
                                        const float* teacher_logits, const float* teacher_lse,
                                        const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                        float* row_loss, void* grad, spec_dtype_t grad_dtype, uint32_t* dev_status,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  return distill(student, dtype, N, V, k, temperature, grad_scale, teacher_ids, teacher_logits, teacher_lse,
                 row_weight, reduction, loss_out, row_loss, true, grad, grad_dtype, dev_status, workspace,
                 workspace_bytes, stream);
}

size_t spec_linear_loss_workspace_bytes(spec_dtype_t dtype, int N, int V, int H, int k, int want_grad_hidden,
                                        int want_grad_weight) {
  return head_workspace(dtype, N, V, H, k, want_grad_hidden != 0, want_grad_weight != 0, SIZE_MAX);
}

size_t spec_linear_loss_workspace_least(spec_dtype_t dtype, int N, int V, int H, int k, int want_grad_hidden,
                                        int want_grad_weight) {
  return head_workspace(dtype, N, V, H, k, want_grad_hidden != 0, want_grad_weight != 0, 0);
}

spec_status_t spec_linear_cross_entropy_fwd_bwd(const void* hidden, const void* weight, spec_dtype_t dtype, int N,
                                                int V, int H, float temperature, float grad_scale,
                                                const int32_t* labels, int ignore_index, const float* row_weight,
                                                spec_reduction_t reduction, float* loss_out, float* row_loss,
                                                float* lse_out, void* grad_hidden, void* grad_weight,
                                                spec_dtype_t grad_dtype, uint32_t* dev_status, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  const HeadCall c{hidden,     weight,      dtype,        N,          V,          H,         1,        temperature,
                   grad_scale, labels,      nullptr,      ignore_index, row_weight, reduction, loss_out, row_loss,
                   lse_out,    grad_hidden, grad_weight,  grad_dtype, dev_status, workspace, workspace_bytes, stream};
  return head_loss(c, true);
}

spec_status_t spec_linear_cross_entropy(const void* hidden, const void* weight, spec_dtype_t dtype, int N, int V,
                                        int H, float temperature, const int32_t* labels, int ignore_index,
                                        const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                        float* row_loss, float* lse_out, uint32_t* dev_status, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const HeadCall c{hidden,  weight,  dtype,   N,            V,          H,         1,        temperature,
                   0.0f,    labels,  nullptr, ignore_index, row_weight, reduction, loss_out, row_loss,
                   lse_out, nullptr, nullptr, dtype,        dev_status, workspace, workspace_bytes, stream};
  return head_loss(c, false);
}

spec_status_t spec_linear_topk_distill_fwd_bwd(const void* hidden, const void* weight, spec_dtype_t dtype, int N,
                                               int V, int H, int k, float temperature, float grad_scale,
                                               const int32_t* teacher_ids, const float* teacher_logits,
                                               const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                               float* row_loss, float* lse_out, void* grad_hidden, void* grad_weight,
                                               spec_dtype_t grad_dtype, uint32_t* dev_status, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  if (N > 0 && !teacher_logits) return SPEC_ERR_INVALID_ARG;
  const HeadCall c{hidden,     weight,      dtype,          N,          V,          H,         k,        temperature,
                   grad_scale, teacher_ids, teacher_logits, -1,         row_weight, reduction, loss_out, row_loss,
                   lse_out,    grad_hidden, grad_weight,    grad_dtype, dev_status, workspace, workspace_bytes, stream};
  return head_loss(c, true);
}

spec_status_t spec_linear_topk_distill(const void* hidden, const void* weight, spec_dtype_t dtype, int N, int V, int H,
                                       int k, float temperature, const int32_t* teacher_ids,
                                       const float* teacher_logits, const float* row_weight,
                                       spec_reduction_t reduction, float* loss_out, float* row_loss, float* lse_out,
                                       uint32_t* dev_status, void* workspace, size_t workspace_bytes, void* stream) {
  if (N > 0 && !teacher_logits) return SPEC_ERR_INVALID_ARG;
  const HeadCall c{hidden,  weight,      dtype,          N,     V,          H,         k,        temperature,
                   0.0f,    teacher_ids, teacher_logits, -1,    row_weight, reduction, loss_out, row_loss,
                   lse_out, nullptr,     nullptr,        dtype, dev_status, workspace, workspace_bytes, stream};
  return head_loss(c, false);
}

}  // extern "C"
