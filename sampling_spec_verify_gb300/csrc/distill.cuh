// Distillation of student logits from a teacher's top logits: loss and
// gradient in one read of the logits.
//
//   q = softmax(z / T) over the vocabulary; t the teacher's listed
//   probabilities, t_r what they leave (0 unless the teacher's normaliser is
//   given), q_r the student mass outside the list, M = sum t_i + t_r
//   L        = sum_i t_i (log t_i - log q_i) + t_r (log t_r - log q_r)
//   dL/dz_v  = (M q_v - t_v) / T                  v listed
//            = q_v / q_r (M q_r - t_r) / T        v not listed
// (without t_r the second line is M q_v / T).  M q_r - t_r is taken as
// sum t_i - M sum q_i where the list holds less than half of the student's
// mass: the difference of two masses near 1 would cancel.
//
// Bound: HBM.  A row is read once and its gradient written once; a row of
// 151936 bf16 logits is 304 KB, more than one SM holds, so a cluster of S CTAs
// keeps it in shared memory between the normaliser and the gradient.
#pragma once

#include <type_traits>

#include "loss_common.cuh"

namespace ssv {

constexpr int kDThreads = 512;
constexpr int kDWarps = kDThreads / 32;
constexpr int kDMaxCluster = 16;

struct DistillParams {
  const void* z;
  void* grad;
  int N, V, k;
  int nst;            // shared-memory stages (2: the next row's slice is prefetched)
  uint32_t cap;       // bytes of a stage
  int skew;           // elements by which the base lies past a 16-byte boundary
  int out_vec;        // gradient vectors may be written 16 bytes at a time
  float s_hi, s_lo;   // log2(e) / T
  const int32_t* ids; // [N, k]
  const float* t;     // [N, k]
  const RowTeacher* row;
  const uint8_t* keep;
  const float* weight;
  int mean, tail;
  float gscale;       // grad_scale / T
  float* zi;          // [N, k] out: student logits of the entries
  RowNorm* norm;      // [N] out
  uint32_t* status;
};

struct NoGrad {};

// Writes PV gradients of consecutive tokens.
template <class O, int PV>
__device__ __forceinline__ void store_grads(O* dst, const float (&g)[PV], bool vec) {
  if (vec) {
    if constexpr (sizeof(O) == 4) {
#pragma unroll
      for (int i = 0; i < PV; i += 4)
        __stcs(reinterpret_cast<float4*>(dst + i), make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]));
    } else {
      static_assert(PV == 8, "16-bit gradients come from 16-bit logits");
      uint4 w;
      w.x = Elem<O>::pack(g[0], g[1]), w.y = Elem<O>::pack(g[2], g[3]);
      w.z = Elem<O>::pack(g[4], g[5]), w.w = Elem<O>::pack(g[6], g[7]);
      __stcs(reinterpret_cast<uint4*>(dst), w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PV; ++i) dst[i] = Elem<O>::from_f32(g[i]);
  }
}

// One row's place in this CTA: the 16-byte vectors [v0, v1) of the row's
// aligned middle part, and the odd elements at either end of the row.
struct Slice {
  long long f0;        // flat index of the row's first element
  int a0, a1;          // the aligned part within the row
  int v0, v1;          // this CTA's vectors of it
  int head, tail;      // odd elements this CTA holds
};

template <int PV>
__device__ __forceinline__ Slice slice_of(long long n, int V, int skew, uint32_t rank, uint32_t S) {
  Slice s;
  s.f0 = n * V;
  int lead = (int)((PV - (s.f0 + skew) % PV) % PV);
  if (lead > V) lead = V;
  const int nv = (V - lead) / PV;
  s.a0 = lead;
  s.a1 = lead + nv * PV;
  s.v0 = (int)((long long)nv * rank / S);
  s.v1 = (int)((long long)nv * (rank + 1) / S);
  s.head = rank == 0 ? lead : 0;
  s.tail = rank == S - 1 ? V - s.a1 : 0;
  return s;
}

template <class E, class O>
__global__ void __launch_bounds__(kDThreads, 2) distill_kernel(const __grid_constant__ DistillParams P) {
  using T = Elem<E>;
  constexpr int PV = T::PV;
  constexpr bool kGrad = !std::is_same<O, NoGrad>::value;
  using OG = typename std::conditional<kGrad, O, float>::type;
  extern __shared__ __align__(128) unsigned char stage_mem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ float4 warp_part[kDWarps];    // {m, s} of the unlisted, {m, s} of the listed tokens
  __shared__ float4 box[2][kDMaxCluster];  // the same per CTA, pushed by every CTA of the cluster
  __shared__ float edge[16];               // odd elements: 0..7 before, 8..15 after the aligned part
  __shared__ RowNorm shared_norm;
  __shared__ uint32_t shared_count[kDWarps];
  __shared__ uint32_t abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int G = gridDim.x / S, c = blockIdx.x / S;
  const E* z = static_cast<const E*>(P.z);
  const uint32_t bar0 = smem_addr(bars);
  if (tid == 0) {
    mbar_init(bar0, 1);
    mbar_init(bar0 + 8, 1);
    fence_mbar_init();
    abort_flag = 0;
  }

  float coef0 = P.gscale;
  if (kGrad && P.mean) {  // rows that count
    uint32_t cnt = 0;
    for (int n = tid; n < P.N; n += kDThreads) cnt += P.keep[n];
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) shared_count[wid] = cnt;
  }
  cluster_sync();  // barriers initialised in every CTA, counts written
  if (kGrad && P.mean) {
    uint32_t cnt = 0;
#pragma unroll
    for (int i = 0; i < kDWarps; ++i) cnt += shared_count[i];
    coef0 = cnt ? coef0 / (float)cnt : 0.0f;
  }

  const uint64_t policy = l2_evict_first_policy();
  // Starts the copy of row n's slice into stage st; rows that are left out are
  // not read.
  auto fetch = [&](long long n, int st) {
    if (tid != 0 || n >= P.N || !P.keep[n]) return;
    const Slice s = slice_of<PV>(n, P.V, P.skew, rank, S);
    const uint32_t bytes = (uint32_t)(s.v1 - s.v0) * 16u;
    mbar_arrive_expect_tx(bar0 + 8 * st, bytes);
    if (bytes)
      bulk_load(smem_addr(stage_mem) + st * P.cap, z + s.f0 + s.a0 + (long long)s.v0 * PV, bytes, bar0 + 8 * st,
                policy);
  };

  // per-row values of the row about to be processed
  int my_id;
  float my_t, w, my_edge;
  bool live;
  RowTeacher rt;
  auto row_values = [&](long long n) {
    live = n < P.N && P.keep[n];
    my_id = -1;
    my_t = w = 0.0f;
    rt = RowTeacher{0.0, 0.0f, 0.0f};
    my_edge = -INFINITY;
    if (live) {
      if (tid < P.k) {
        my_id = P.ids[n * P.k + tid];
        my_t = P.t[n * P.k + tid];
      }
      rt = P.row[n];
      w = P.weight ? P.weight[n] : 1.0f;
      if (tid < 16) {
        const Slice s = slice_of<PV>(n, P.V, P.skew, rank, S);
        if (tid < s.head) my_edge = T::to_f32(z[s.f0 + tid]);
        if (tid >= 8 && tid - 8 < s.tail) my_edge = T::to_f32(z[s.f0 + s.a1 + tid - 8]);
      }
    }
  };

  uint32_t par = 0;  // phase parity of each stage, one bit per stage
  fetch(c, 0);
  if (P.nst == 2) fetch((long long)c + G, 1);
  row_values(c);
  int it = 0, ex = 0;
  uint32_t failed = 0;
  for (long long n = c; n < P.N; n += G, ++it) {
    const int st = P.nst == 2 ? (it & 1) : 0;
    const Slice s = slice_of<PV>(n, P.V, P.skew, rank, S);
    const int nvl = s.v1 - s.v0;
    OG* out = kGrad ? static_cast<OG*>(P.grad) + s.f0 : nullptr;
    if (!live) {  // left out: no gradient
      if (kGrad) {
        float zero[PV] = {};
        for (int i = tid; i < nvl; i += kDThreads) store_grads<OG, PV>(out + s.a0 + (s.v0 + i) * PV, zero, P.out_vec);
        if (tid < s.head) out[tid] = Elem<OG>::from_f32(0.0f);
        if (tid >= 8 && tid - 8 < s.tail) out[s.a1 + tid - 8] = Elem<OG>::from_f32(0.0f);
      }
      fetch(n + (long long)P.nst * G, st);
      row_values(n + G);
      continue;
    }
    E* buf = reinterpret_cast<E*>(stage_mem + st * P.cap);
    const uint4* vec = reinterpret_cast<const uint4*>(buf);
    const float coef = coef0 * w;

    if (tid < 16) edge[tid] = my_edge;
    // after a wait that ran out, the later ones are short: the call ends soon
    const bool got = mbar_wait_bounded(bar0 + 8 * st, (par >> st) & 1u, failed ? 100000ull : 2000000000ull);
    par ^= 1u << st;
    if (!got) failed = abort_flag = 1;
    __syncthreads();  // edges written

    // the listed tokens: taken out of the row, their logits kept by their threads
    float my_z = -INFINITY;
    bool mine = false;
    if (my_id >= 0) {
      if (my_id < s.a0) {
        mine = rank == 0;
        if (mine) {
          my_z = edge[my_id];
          edge[my_id] = -INFINITY;
        }
      } else if (my_id >= s.a1) {
        mine = rank == S - 1;
        if (mine) {
          my_z = edge[8 + my_id - s.a1];
          edge[8 + my_id - s.a1] = -INFINITY;
        }
      } else {
        const int v = (my_id - s.a0) / PV;
        mine = v >= s.v0 && v < s.v1;
        if (mine) {
          E* p = buf + (my_id - s.a0 - s.v0 * PV);
          my_z = T::to_f32(*p);
          *p = T::neg_inf();
        }
      }
      if (mine) P.zi[n * P.k + tid] = my_z;
    }
    __syncthreads();

    // normalisers: each warp relative to its own maximum
    float m = -INFINITY;
    for (int i = tid; i < nvl; i += kDThreads) {
      float x[PV];
      T::unpack(vec[i], x);
#pragma unroll
      for (int j = 0; j < PV; ++j) m = max_nan(m, x[j]);
    }
    if (tid < 16) m = max_nan(m, edge[tid]);
    m = redux_max_nan(m);
    float sum = 0.0f;
    if (m > -INFINITY && m < INFINITY) {
      for (int i = tid; i < nvl; i += kDThreads) {
        float x[PV];
        T::unpack(vec[i], x);
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          const float d = x[j] - m;
          a += ex2(fmaf(d, P.s_hi, d * P.s_lo));
        }
        sum += a;
      }
      if (tid < 16) sum += exp2_scaled(edge[tid] - m, P.s_hi, P.s_lo);
      sum = warp_sum(sum);
    } else if (!(m < INFINITY)) {  // NaN or +inf among the logits
      sum = NAN;
      m = 0.0f;
    }
    float mk = redux_max_nan(my_z), sk = 0.0f;
    if (mk > -INFINITY && mk < INFINITY) {
      sk = warp_sum(exp2_scaled(my_z - mk, P.s_hi, P.s_lo));
    } else if (!(mk < INFINITY)) {
      sk = NAN;
      mk = 0.0f;
    }
    if (lane == 0) warp_part[wid] = make_float4(m, sum, mk, sk);
    __syncthreads();
    const int slot = ex & 1;
    ++ex;
    // joins the {m, s} pairs of the lanes of a warp
    auto join = [&](float& mm, float& ss) {
      const float top = redux_max_nan(mm);
      ss = warp_sum(mm > -INFINITY ? ss * exp2_scaled(mm - top, P.s_hi, P.s_lo) : 0.0f);
      mm = top;
    };
    if (wid == 0) {
      float4 v = lane < kDWarps ? warp_part[lane] : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
      join(v.x, v.y);
      join(v.z, v.w);
      if (lane < (int)S) st_cluster_v4(map_rank(smem_addr(&box[slot][rank]), lane), v.x, v.y, v.z, v.w);
    }
    cluster_sync();
    if (wid == 0) {
      float4 v = lane < (int)S ? box[slot][lane] : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
      join(v.x, v.y);
      join(v.z, v.w);
      if (lane == 0) {
        const float top = fmaxf(v.x, v.z);
        RowNorm r;
        r.m = top;
        r.mr = v.x;
        r.zr = v.y;
        r.zl = v.z > -INFINITY ? v.w * exp2_scaled(v.z - top, P.s_hi, P.s_lo) : 0.0f;
        r.z = (v.x > -INFINITY ? v.y * exp2_scaled(v.x - top, P.s_hi, P.s_lo) : 0.0f) + r.zl;
        if (!(top > -INFINITY)) r.z = NAN;  // no finite logit
        shared_norm = r;
        if (rank == 0) {
          P.norm[n] = r;
          if (!(r.z < INFINITY)) raise(P.status, SPEC_DEV_BAD_LOGITS);
        }
      }
    }
    __syncthreads();

    // the next row's scalars travel while this one's gradient is written
    const int id = my_id;
    const float t = my_t;
    const RowTeacher rc = rt;
    row_values(n + G);

    if (kGrad) {
      const RowNorm r = shared_norm;
      const float mass = rc.sum + rc.rest;
      const float inv_z = 1.0f / r.z;
      const bool some = r.mr > -INFINITY;
      const float rest_scale = some ? exp2_scaled(r.mr - r.m, P.s_hi, P.s_lo) : 0.0f;
      const float mr = some ? r.mr : 0.0f;
      float cb;  // factor of 2^((z - mr) s) for tokens that are not listed
      if (P.tail) {
        const float ql = r.zl * inv_z;
        const float diff = ql < 0.5f ? rc.sum - mass * ql : mass * (r.zr * rest_scale * inv_z) - rc.rest;
        cb = some ? coef * diff / r.zr : coef * (r.z - r.z);
      } else {
        cb = coef * mass * rest_scale * inv_z;
      }
      for (int i = tid; i < nvl; i += kDThreads) {
        float x[PV], g[PV];
        T::unpack(vec[i], x);
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          const float d = x[j] - mr;
          g[j] = ex2(fmaf(d, P.s_hi, d * P.s_lo)) * cb;
        }
        store_grads<OG, PV>(out + s.a0 + (s.v0 + i) * PV, g, P.out_vec);
      }
      if (tid < 16) {
        const float g = exp2_scaled(edge[tid] - mr, P.s_hi, P.s_lo) * cb;
        if (tid < s.head) out[tid] = Elem<OG>::from_f32(g);
        if (tid >= 8 && tid - 8 < s.tail) out[s.a1 + tid - 8] = Elem<OG>::from_f32(g);
      }
      fence_proxy_async_smem();
      __syncthreads();  // the slice has been read, and the listed tokens' places hold 0
      if (mine) {
        const float q = exp2_scaled(my_z - r.m, P.s_hi, P.s_lo) * inv_z;
        out[id] = Elem<OG>::from_f32(coef * (mass * q - t));
      }
    } else {
      fence_proxy_async_smem();
      __syncthreads();
    }
    fetch(n + (long long)P.nst * G, st);
  }
  __syncthreads();
  if (tid == 0 && abort_flag) raise(P.status, SPEC_DEV_TIMEOUT);
  cluster_sync();  // no CTA leaves while others may still push into it
}

// Row losses and their sum: one warp per row.
__global__ void __launch_bounds__(kTargetWarps * 32) distill_finish_kernel(const FinishParams P,
                                                                          const RowNorm* norm) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = (long long)blockIdx.x * kTargetWarps + w;
  if (n < P.N) {
    float loss = 0.0f;
    if (P.keep[n]) {
      const RowNorm r = norm[n];
      const double logz = log((double)r.z);
      double log_qr = 0.0;
      if (P.row[n].rest > 0.0f) {
        // from the listed tokens' mass where that is the smaller part
        const double ql = (double)r.zl / (double)r.z;
        if (ql < 0.5)
          log_qr = log1p(-ql);
        else
          log_qr = r.mr > -INFINITY ? ((double)r.mr - (double)r.m) * P.inv_t + log((double)r.zr) - logz : -INFINITY;
      }
      loss = row_loss_warp(P, n, lane, (double)r.m, logz, log_qr);
    }
    if (lane == 0) P.row_loss[n] = loss;
  }
  finish_total(P, kTargetWarps * 32);
}

}  // namespace ssv
