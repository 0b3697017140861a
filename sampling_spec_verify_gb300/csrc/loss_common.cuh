// Pieces shared by the vocabulary losses (cross entropy of a head and
// distillation from a teacher's top logits): the teacher side of a row,
// scalars of a call, and the sum of the row losses.
//
// Every loss here has the form
//   L_n = sum_i t_i (log t_i - log q_i) + t_r (log t_r - log q_r)
// over at most kMaxEntries listed tokens per row, q the softmax of the whole
// vocabulary, t_r and q_r what the listed tokens leave over (t_r = 0 unless
// the teacher's normaliser is given).  Cross entropy is one entry with t = 1.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "spec_verify.h"

namespace ssv {

constexpr int kMaxEntries = 256;  // listed teacher tokens per row
constexpr int kTargetWarps = 8;   // rows per CTA of the kernels with a warp per row
constexpr int kHashSlots = 512;   // per row, at least twice kMaxEntries

struct RowTeacher {
  double shift;  // log of the teacher's normaliser: log t_i = x_i / T - shift
  float sum;     // sum of t_i
  float rest;    // t_r
};

struct RowNorm {  // of the student: sums of 2^((z - m) s), s = log2(e) / T
  float m, z;     // all tokens
  float mr, zr;   // the tokens that the teacher does not list
  float zl;       // the listed tokens, relative to m
};

// Scalars of a call, written by its kernels.
struct LossScalars {
  uint32_t ticket;
  uint32_t count;  // rows that count
  float inv_wmax;  // 1 / largest |row weight| of those (0 if there is none)
  float grad_mul;  // factor of the stored logit gradients in the results
};

// ---- elements ---------------------------------------------------------------------

template <class E>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int PV = 8;  // elements per 16-byte vector
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __forceinline__ __nv_bfloat16 neg_inf() { return __ushort_as_bfloat16(0xFF80u); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static constexpr int PV = 8;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static __forceinline__ float to_f32(__half v) { return __half2float(v); }
  __device__ static __forceinline__ __half neg_inf() { return __ushort_as_half(0xFC00u); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static constexpr int PV = 4;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  __device__ static __forceinline__ float to_f32(float v) { return v; }
  __device__ static __forceinline__ float neg_inf() { return -INFINITY; }
  __device__ static __forceinline__ float from_f32(float v) { return v; }
};

// ---- arithmetic ---------------------------------------------------------------------

// 2^(d (hi + lo)) to a few ulp: the rounding of the product is carried along.
// hi + lo = log2(e) / T with lo > 0 (the host rounds hi down), so that a logit
// of -inf stays -inf through d * hi + d * lo.
__device__ __forceinline__ float exp2_scaled(float d, float hi, float lo) {
  const float p = d * hi;
  if (!(fabsf(p) < INFINITY)) return p < 0.0f ? 0.0f : p;  // d = -inf; NaN and +inf pass on
  const float e = fmaf(d, lo, fmaf(d, hi, -p));
  return exp2f(p) * fmaf(e, 0.69314718f, 1.0f);
}

// Maximum of a float over the warp; NaN if any lane holds NaN.
__device__ __forceinline__ float redux_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void raise(uint32_t* status, uint32_t bits) {
  if (status && bits) atomicOr(status, bits);
}

// ---- the teacher side ---------------------------------------------------------

struct TargetParams {
  const int32_t* ids;    // [N, k]; one label per row when `logits` is null
  const float* logits;   // [N, k] teacher logits, or null
  const float* lse;      // [N] teacher normaliser, or null
  int N, V, k;
  int ignore;            // label of rows that are left out
  double inv_t;
  float* t;              // [N, k] out: teacher probabilities, 0 in unused slots
  RowTeacher* row;       // [N] out
  uint8_t* keep;         // [N] out: the row counts
  LossScalars* scalars;
  uint32_t* status;
};

// One warp per row.  Slots with id -1 are unused; an id outside [-1, V), an id
// listed twice, or a teacher row without a usable normaliser leaves the row out
// and is reported.  Duplicates are found with a hash set in shared memory: k
// inserts, against k^2 / 2 compares.
//
// log t_i is formed in fp64 (a few adds and multiplies per entry) because the
// loss is a small difference of such logarithms; the exponential is fp32.
__global__ void __launch_bounds__(kTargetWarps * 32) targets_kernel(const TargetParams P) {
  __shared__ int hash[kTargetWarps][kHashSlots];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) P.scalars->ticket = 0;
  const long long n = (long long)blockIdx.x * kTargetWarps + w;
  if (n >= P.N) return;

  if (!P.logits) {  // cross entropy: the label with probability 1
    if (lane == 0) {
      const int id = P.ids[n];
      const bool ok = id >= 0 && id < P.V && id != P.ignore;
      if (!ok && id != P.ignore) raise(P.status, SPEC_DEV_BAD_TOKEN);
      P.keep[n] = ok;
      P.t[n] = ok ? 1.0f : 0.0f;
      P.row[n] = RowTeacher{0.0, ok ? 1.0f : 0.0f, 0.0f};
    }
    return;
  }

  for (int i = lane; i < kHashSlots; i += 32) hash[w][i] = -1;
  __syncwarp();
  constexpr int kPer = kMaxEntries / 32;
  float x[kPer];
  bool bad = false, any = false;
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = lane + 32 * j;
    x[j] = -INFINITY;
    if (i < P.k) {
      const int id = P.ids[n * P.k + i];
      if (id < -1 || id >= P.V) bad = true;
      if (id >= 0 && id < P.V) {
        any = true;
        x[j] = P.logits[n * P.k + i];
        uint32_t s = ((uint32_t)id * 2654435761u) >> 23;  // 9 bits
        for (int probe = 0; probe < kHashSlots; ++probe) {
          const int old = atomicCAS(&hash[w][s], -1, id);
          if (old == -1) break;
          if (old == id) {
            bad = true;
            break;
          }
          s = (s + 1) & (kHashSlots - 1);
        }
        m = max_nan(m, x[j]);
      }
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  any = __any_sync(0xffffffffu, any);
  m = redux_max_nan(m);
  uint32_t bits = bad ? SPEC_DEV_BAD_TOKEN : 0u;
  double shift = 0.0;
  bool ok = any && !bad;
  const float lse = P.lse ? P.lse[n] : 0.0f;
  if (ok && (!(m < INFINITY) || (P.lse ? !(fabsf(lse) < INFINITY) : m == -INFINITY))) {
    bits |= SPEC_DEV_BAD_LOGITS;  // NaN or +inf, or nothing to normalise with
    ok = false;
  }
  float sum = 0.0f;
  if (ok) {
    shift = P.lse ? (double)lse : (double)m * P.inv_t;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {  // x becomes the (unnormalised) probability
      const double d = (double)x[j] * P.inv_t - shift;  // -inf where unused
      const float hi = (float)d;
      x[j] = hi > -INFINITY ? expf(hi) * (1.0f + (float)(d - (double)hi)) : 0.0f;
      sum += x[j];
    }
    sum = warp_sum(sum);
    if (!P.lse) {
      const float inv = 1.0f / sum;
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] *= inv;
      shift += log((double)sum);
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = lane + 32 * j;
    if (i < P.k) P.t[n * P.k + i] = ok ? x[j] : 0.0f;
  }
  if (lane == 0) {
    raise(P.status, bits);
    RowTeacher r{shift, 0.0f, 0.0f};
    if (ok) {
      r.sum = P.lse ? sum : 1.0f;
      const float rest = 1.0f - sum;
      // a remainder below 1e-6 is the rounding of the sum, not mass
      if (P.lse && rest > 1e-6f) r.rest = rest;
    }
    P.row[n] = r;
    P.keep[n] = ok;
  }
}

// ---- row losses and their sum --------------------------------------------------

struct FinishParams {
  int N, k;
  double inv_t;
  const float* logits;  // [N, k] teacher logits, or null (cross entropy)
  const float* t;       // [N, k]
  const RowTeacher* row;
  const uint8_t* keep;
  const float* weight;  // [N] or null
  const float* zi;      // [N, k] student logits of the entries
  int mean;
  float grad_scale;     // times 1 / T
  float store_scale;    // of the stored logit gradients (head losses)
  float* loss;          // [1]
  float* row_loss;      // [N]
  LossScalars* scalars;
  uint32_t* status;
};

// Loss of row n, by one warp (every lane gets it): log q_i = (z_i - m) / T -
// logz, log_qr the log of the unlisted tokens' mass.  The maximum is taken off
// first: rows masked with the type's lowest value would lose logz beside it.
__device__ __forceinline__ float row_loss_warp(const FinishParams& P, long long n, int lane, double m, double logz,
                                               double log_qr) {
  const RowTeacher r = P.row[n];
  float acc = 0.0f;
  for (int i = lane; i < P.k; i += 32) {
    const float t = P.t[n * P.k + i];
    if (t > 0.0f) {
      const double lt = P.logits ? (double)P.logits[n * P.k + i] * P.inv_t - r.shift : 0.0;
      acc += t * (float)(lt - (((double)P.zi[n * P.k + i] - m) * P.inv_t - logz));
    }
  }
  acc = warp_sum(acc);
  if (r.rest > 0.0f) {
    const double lr = r.sum < 0.5f ? log1p(-(double)r.sum) : log((double)r.rest);
    acc += (float)((double)r.rest * (lr - log_qr));
  }
  if (isnan(logz)) acc = NAN;  // also where the entries weigh nothing
  return acc;
}

// The last CTA to arrive sums the rows in one fixed order, in fp64.
__device__ __forceinline__ void finish_total(const FinishParams& P, int threads) {
  __shared__ uint32_t last;
  __shared__ double red[3][32];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&P.scalars->ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0, cnt = 0.0;
  float wmax = 0.0f;
  for (int n = threadIdx.x; n < P.N; n += threads) {
    if (!P.keep[n]) continue;
    const float w = P.weight ? P.weight[n] : 1.0f;
    sum += (double)w * (double)__ldcg(P.row_loss + n);
    cnt += 1.0;
    wmax = max_nan(wmax, fabsf(w));
  }
  sum = warp_sum(sum);
  cnt = warp_sum(cnt);
  wmax = redux_max_nan(wmax);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = threads >> 5;
  if (lane == 0) red[0][w] = sum, red[1][w] = cnt, red[2][w] = (double)wmax;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = cnt = 0.0;
    wmax = 0.0f;
    for (int i = 0; i < nw; ++i) sum += red[0][i], cnt += red[1][i], wmax = max_nan(wmax, (float)red[2][i]);
    const double den = P.mean ? (cnt > 0.0 ? cnt : 1.0) : 1.0;
    P.loss[0] = (float)(sum / den);
    P.scalars->count = (uint32_t)cnt;
    P.scalars->inv_wmax = wmax == 0.0f ? 0.0f : 1.0f / wmax;
    P.scalars->grad_mul = (float)((double)P.grad_scale * (double)wmax / (den * (double)P.store_scale));
  }
}

}  // namespace ssv
