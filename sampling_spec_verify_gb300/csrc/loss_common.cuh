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
constexpr int kHashSlots = 512;   // per row, twice kMaxEntries

struct __align__(16) RowTeacher {
  float shift, shift_lo;  // log of the teacher's normaliser: log t_i = x_i / T - (shift + shift_lo)
  float sum;              // sum of t_i
  float rest;             // t_r
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
  float inv_wmax;  // 1 / largest |row weight| of those (0 if there is none; one below 2^-126 counts as 2^-126)
  float grad_mul;  // factor of the stored logit gradients in the results
};

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

// ---- elements ---------------------------------------------------------------------

template <class E>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int PV = 8;  // elements per 16-byte vector
  // The 8 values as 4 packed pairs in element order (exact widening).
  __device__ static __forceinline__ void pairs(const uint4& w, f32x2 (&p)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  // Elementwise maximum of two vectors; NaN passes on.
  __device__ static __forceinline__ uint4 vmax(const uint4& a, const uint4& b) {
    return make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w));
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ static __forceinline__ float hmax(const uint4& w) {
    const uint32_t m = max2(max2(w.x, w.y), max2(w.z, w.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  static constexpr uint32_t kLow = 0xFF80FF80u;  // -inf in every element
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
  __device__ static __forceinline__ void pairs(const uint4& w, f32x2 (&p)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      p[i] = f2(f.x, f.y);
    }
  }
  __device__ static __forceinline__ uint4 vmax(const uint4& a, const uint4& b) {
    return make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w));
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ static __forceinline__ float hmax(const uint4& w) {
    const uint32_t m = max2(max2(w.x, w.y), max2(w.z, w.w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max_nan(f.x, f.y);
  }
  static constexpr uint32_t kLow = 0xFC00FC00u;
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
  __device__ static __forceinline__ void pairs(const uint4& w, f32x2 (&p)[2]) {
    p[0] = f2(__uint_as_float(w.x), __uint_as_float(w.y));
    p[1] = f2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ static __forceinline__ uint4 vmax(const uint4& a, const uint4& b) {
    return make_uint4(max1(a.x, b.x), max1(a.y, b.y), max1(a.z, b.z), max1(a.w, b.w));
  }
  __device__ static __forceinline__ uint32_t max1(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static __forceinline__ float hmax(const uint4& w) {
    return __uint_as_float(max1(max1(w.x, w.y), max1(w.z, w.w)));
  }
  static constexpr uint32_t kLow = 0xFF800000u;
  __device__ static __forceinline__ float to_f32(float v) { return v; }
  __device__ static __forceinline__ float neg_inf() { return -INFINITY; }
  __device__ static __forceinline__ float from_f32(float v) { return v; }
};

// ---- arithmetic ---------------------------------------------------------------------

__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^(d s) within 2^-21: the rounding of the product is carried along.  d = -inf
// gives 0; NaN and +inf pass on.
__device__ __forceinline__ float exp2_scaled(float d, float s) {
  const float p = d * s;
  const float e = fabsf(p) < INFINITY ? fmaf(d, s, -p) : 0.0f;
  return ex2(p) * fmaf(e, 0.69314718f, 1.0f);
}

// A sum of two floats kept as value and rounding error.
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ F2 two_mul(float a, F2 b) {
  const float p = a * b.hi;
  return {p, fmaf(a, b.lo, fmaf(a, b.hi, -p))};
}
__device__ __forceinline__ F2 pair_add(F2 a, F2 b) {
  F2 s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The kernels of a call follow each other by programmatic launches: a kernel
// starts its prologue while the previous one drains, and waits here before it
// touches anything that was written before it.
__device__ __forceinline__ void follow_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A pair's rounding, 0 where the value is not finite: the rounding of an infinite
// sum or product comes out as inf - inf and would turn it into NaN.
__device__ __forceinline__ F2 pair_of(float hi, float lo) { return {hi, fabsf(hi) < INFINITY ? lo : 0.0f}; }
// pair_add where infinite terms are ordinary.
__device__ __forceinline__ F2 sum_add(F2 a, F2 b) {
  const F2 s = pair_add(a, b);
  return pair_of(s.hi, s.lo);
}
// Sum over the lanes of a warp, roundings carried along (in every lane, the same).
__device__ __forceinline__ F2 warp_sum(F2 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = sum_add(v, F2{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

__device__ __forceinline__ void raise(uint32_t* status, uint32_t bits) {
  if (status && bits) atomicOr(status, bits);
}

// ---- the teacher side ---------------------------------------------------------

struct TargetParams {
  const int32_t* ids;    // [N, k] listed tokens (of cross entropy: the labels)
  const float* logits;   // [N, k] teacher logits (of cross entropy: null)
  const float* lse;      // [N] teacher normaliser, or null
  int N, V, k;
  int ignore;            // label of rows that are left out
  F2 inv_t;
  float* t;              // [N, k] out: teacher probabilities, 0 in unused slots
  RowTeacher* row;       // [N] out
  uint8_t* keep;         // [N, up to a multiple of eight] out: the row counts
  // through a head: the listed tokens in order, for each tile of tokens
  uint32_t* keys;        // [N, k] out: id << 8 | slot, ascending
  uint16_t* starts;      // [N, tiles + 1] out: first key of each tile (all 0 where the row is left out)
  int tiles, tile;       // tokens per tile
  LossScalars* scalars;
  uint32_t* status;
};

// One warp per row.  Slots with id -1 are unused; an id outside [-1, V), an id
// listed twice, or a teacher row without a usable normaliser leaves the row out
// and is reported.  Through a head (SORT) the ids are sorted in shared memory
// (key: id and slot; V is below 2^24) for the epilogue that looks them up, and
// duplicates are neighbours; otherwise a hash set finds them (1792 rows of 128: 5
// us against 9).
//
// log t_i is formed with its rounding carried along, because the loss is a
// small difference of such logarithms.  (In fp64 the kernel took 16 us for 1792
// rows of 128 entries, now 5: an SM does two fp64 operations a clock.)
template <bool SORT>
__global__ void __launch_bounds__(kTargetWarps * 32) targets_kernel(const TargetParams P) {
  __shared__ uint32_t room[kTargetWarps][SORT ? kMaxEntries : kHashSlots];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) P.scalars->ticket = 0;
  const long long n = (long long)blockIdx.x * kTargetWarps + w;
  if (n >= P.N) {
    if (lane == 0) P.keep[n] = 0;  // the flags' last word is whole
    return;
  }

  constexpr int kPer = kMaxEntries / 32;
  float x[kPer];
  int id[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = lane + 32 * j;
    id[j] = i < P.k ? P.ids[n * P.k + i] : -1;
    x[j] = i < P.k ? P.logits[n * P.k + i] : -INFINITY;
  }
  uint32_t* key = room[w];
  int size = 32;  // keys to sort
  while (size < P.k) size *= 2;
  if constexpr (!SORT) {
    for (int i = lane; i < kHashSlots; i += 32) key[i] = ~0u;
    __syncwarp();
  }
  bool bad = false, any = false;
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = lane + 32 * j;
    const bool used = id[j] >= 0 && id[j] < P.V;
    if constexpr (SORT) {
      if (i < size) key[i] = used ? (uint32_t)id[j] << 8 | (uint32_t)i : ~0u;
    }
    if (used) {
      any = true;
      m = max_nan(m, x[j]);
      if constexpr (!SORT) {
        uint32_t s = ((uint32_t)id[j] * 2654435761u) >> 23;  // 9 bits
        for (int probe = 0; probe < kHashSlots; ++probe) {
          const uint32_t old = atomicCAS(&key[s], ~0u, (uint32_t)id[j]);
          if (old == ~0u) break;
          if (old == (uint32_t)id[j]) {
            bad = true;
            break;
          }
          s = (s + 1) & (kHashSlots - 1);
        }
      }
    } else {
      bad |= id[j] != -1;
      x[j] = -INFINITY;
    }
  }
  if constexpr (SORT) {
    __syncwarp();
    for (int span = 2; span <= size; span *= 2) {
      for (int step = span / 2; step; step /= 2) {
        for (int i = lane; i < size / 2; i += 32) {
          const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
          const uint32_t a = key[lo], b = key[hi];
          const bool up = (lo & span) == 0;
          key[lo] = up ? min(a, b) : max(a, b);
          key[hi] = up ? max(a, b) : min(a, b);
        }
        __syncwarp();
      }
    }
    for (int i = lane; i + 1 < size; i += 32) bad |= key[i + 1] != ~0u && key[i] >> 8 == key[i + 1] >> 8;
  }
  bad = __any_sync(0xffffffffu, bad);
  any = __any_sync(0xffffffffu, any);
  m = redux_max_nan(m);
  uint32_t bits = bad ? SPEC_DEV_BAD_TOKEN : 0u;
  F2 shift{0.0f, 0.0f};
  bool ok = any && !bad;
  const float lse = P.lse ? P.lse[n] : 0.0f;
  if (ok && (!(m < INFINITY) || (P.lse ? !(fabsf(lse) < INFINITY) : m == -INFINITY))) {
    bits |= SPEC_DEV_BAD_LOGITS;  // NaN or +inf, or nothing to normalise with
    ok = false;
  }
  float sum = 0.0f;
  if (ok) {
    shift = P.lse ? F2{lse, 0.0f} : two_mul(m, P.inv_t);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {  // x becomes the (unnormalised) probability
      if (x[j] > -INFINITY) {
        const F2 d = pair_add(two_mul(x[j], P.inv_t), F2{-shift.hi, -shift.lo});
        x[j] = expf(d.hi) * (1.0f + d.lo);
      } else {
        x[j] = 0.0f;
      }
      sum += x[j];
    }
    sum = warp_sum(sum);
    if (!P.lse) {
      const float inv = 1.0f / sum;
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] *= inv;
      shift = pair_add(shift, F2{logf(sum), 0.0f});
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = lane + 32 * j;
    if (i < P.k) P.t[n * P.k + i] = ok ? x[j] : 0.0f;
  }
  if constexpr (SORT) {
    for (int i = lane; i < P.k; i += 32) P.keys[n * P.k + i] = key[i];
    for (int b = lane; b <= P.tiles; b += 32) {
      int lo = 0;
      if (ok) {
        const uint32_t first = (uint32_t)min((long long)b * P.tile, (long long)P.V) << 8;
        int len = P.k;
        while (len > 0) {  // first key that is not below
          const int half = len / 2;
          if (key[lo + half] < first)
            lo += half + 1, len -= half + 1;
          else
            len = half;
        }
      }
      P.starts[n * (P.tiles + 1) + b] = (uint16_t)lo;
    }
  }
  if (lane == 0) {
    raise(P.status, bits);
    RowTeacher r{shift.hi, shift.lo, 0.0f, 0.0f};
    if (ok) {
      r.sum = P.lse ? sum : 1.0f;
      // The remainder is as exact as the sum of 32-bit terms, about 1e-7 absolute: two
      // digits of one of 1e-5.  The inputs say no more: half a step of a float32
      // normaliser near 15 moves it by 5e-7.  (64-bit exponentials cost 16 us a
      // launch instead of 5.)  Below 1e-6 it is the rounding of the sum, not mass.
      const float rest = 1.0f - sum;
      if (P.lse && rest > 1e-6f) r.rest = rest;
    }
    P.row[n] = r;
    P.keep[n] = ok;
  }
  let_next_start();  // not before: kernels of whole SMs would be placed around this one's CTAs
}

// ---- row losses and their sum --------------------------------------------------

struct FinishParams {
  int N, k;
  F2 inv_t;             // teacher side
  F2 c;                 // student side: log q_i = (z_i - m) c - log Z
  const float* logits;  // [N, k] teacher logits, or null (cross entropy)
  const float* t;       // [N, k]
  const RowTeacher* row;
  const uint8_t* keep;
  const float* weight;  // [N] or null
  const float* zi;      // [N, k] student logits of the entries
  int mean;
  float grad_scale;     // times 1 / T
  float store_scale;    // of the stored logit gradients (head losses)
  float4* part;         // [CTAs] sums of a CTA's rows
  float* loss;          // [1]
  float* row_loss;      // [N]
  LossScalars* scalars;
  uint32_t* status;
};

// What a row's loss needs of the student.
struct RowLog {
  float m;        // taken off the student's logits first: rows masked with a
                  // type's lowest value would lose log Z beside it
  F2 base;        // log Z - (log of the teacher's normaliser)
  float extra;    // t_r (log t_r - log q_r)
};

// log z of a normal z > 0 within 2^-25: the exponent's part is exact in the high word,
// the mantissa's logarithm is below 0.41.  (The exponent's ln 2 is split in two words, the
// first short enough that its product is exact: the reduction of Cody and Waite.)
__device__ __forceinline__ F2 log_pair(float z) {
  int e;
  float f = frexpf(z, &e);  // [0.5, 1)
  if (f < 0.75f) f *= 2.0f, e -= 1;
  const float x = (float)e;
  // ln 2 = 0.693145751953125 (16 bits) + 1.42860682030941723e-6
  return two_sum(x * 0.693145751953125f, fmaf(x, 1.428606820309417e-6f, logf(f)));
}

// Row loss of row n, by one warp:
//   L_n = sum_i t_i ((x_i / T - shift) - ((z_i - m) c - log Z)) + extra
// with every difference carrying its rounding: the terms are small differences
// of logarithms near 10.
__device__ __forceinline__ float row_loss_warp(const FinishParams& P, long long n, int lane, const RowLog& g) {
  float acc = 0.0f;
#pragma unroll 4
  for (int i = lane; i < P.k; i += 32) {
    const float t = P.t[n * P.k + i], z = P.zi[n * P.k + i];
    const float x = P.logits ? P.logits[n * P.k + i] : 0.0f;
    if (t > 0.0f) {
      const F2 d = two_sum(z, -g.m);
      F2 lq = two_mul(d.hi, P.c);
      lq.lo = fmaf(d.lo, P.c.hi, lq.lo);
      F2 v = pair_add(two_mul(x, P.inv_t), F2{-lq.hi, -lq.lo});
      v = pair_add(v, g.base);
      acc = fmaf(t, lq.hi > -INFINITY ? v.hi + v.lo : INFINITY, acc);
    }
  }
  acc = warp_sum(acc) + g.extra;
  return isnan(g.base.hi) ? NAN : acc;  // also where the entries weigh nothing
}

// Sums of the CTA's eight rows (warp w's loss in every lane of it), and in the
// last CTA to arrive the call's, all in fixed orders, as pairs of floats (fp64
// additions here were a third of the kernel's time).  256 threads.  A row loss may
// be +inf (a listed token that the student gives no mass): so is the sum then.
__device__ __forceinline__ void finish_sums(const FinishParams& P, float loss, bool on, float weight) {
  __shared__ float4 red[8];  // {sum, its rounding, rows, largest |weight|}
  __shared__ uint32_t last;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto total = [&](float4 v) {  // over the lanes of a warp
    const F2 t = warp_sum(F2{v.x, v.y});
    return make_float4(t.hi, t.lo, warp_sum(v.z), redux_max_nan(v.w));
  };
  if (lane == 0) {
    const float p = on ? weight * loss : 0.0f;
    const F2 v = pair_of(p, on ? fmaf(weight, loss, -p) : 0.0f);
    red[w] = make_float4(v.hi, v.lo, on ? 1.0f : 0.0f, on ? fabsf(weight) : 0.0f);
  }
  __syncthreads();
  if (w == 0) {
    const float4 v = total(lane < 8 ? red[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (lane == 0) {
      if (gridDim.x > 1) {
        P.part[blockIdx.x] = v;
        __threadfence();
        last = atomicAdd(&P.scalars->ticket, 1u) == gridDim.x - 1;
      } else {
        last = 1;
      }
    }
  }
  __syncthreads();
  if (!last) return;
  if (gridDim.x > 1) {
    __threadfence();
    F2 sum{0.0f, 0.0f};
    float cnt = 0.0f, wmax = 0.0f;
#pragma unroll 4
    for (unsigned i = threadIdx.x; i < gridDim.x; i += 256) {
      const float4 v = __ldcg(P.part + i);
      sum = sum_add(sum, F2{v.x, v.y});
      cnt += v.z;
      wmax = max_nan(wmax, v.w);
    }
    const float4 v = total(make_float4(sum.hi, sum.lo, cnt, wmax));
    __syncthreads();
    if (lane == 0) red[w] = v;
    __syncthreads();
  }
  if (w == 0) {
    const float4 v = total(lane < 8 ? red[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (lane == 0) {
      const float den = P.mean && v.z > 0.0f ? v.z : 1.0f;  // counts are exact up to 2^24 rows
      P.loss[0] = (v.x + v.y) / den;
      P.scalars->count = (uint32_t)v.z;
      // the inverse of a smaller one would be infinite; (NaN passes on)
      const float wmax = v.w < 0x1p-126f ? 0x1p-126f : v.w;
      P.scalars->inv_wmax = v.w == 0.0f ? 0.0f : 1.0f / wmax;
      P.scalars->grad_mul = P.grad_scale * wmax / (den * P.store_scale);
    }
  }
}

}  // namespace ssv
