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
// holds it between the normaliser and the gradient, each CTA a slice in its
// registers (up to NV vectors a thread; NV = 0: in shared memory, for slices that
// do not fit and gradients that start off a vector's boundary).  Slices land in
// shared memory by bulk copies a row ahead; two CTAs share an SM, so that one's
// exchange hides behind the other's work.  Measured: 896 x 129280 bf16 with its
// gradient 79 us (5.9 TB/s, 0.87 of the copy rate), 1792 x 151936 to fp32 257 us
// (0.94), 1024 x 151936 without gradient 65 us (0.71).
#pragma once

#include <type_traits>

#include "loss_common.cuh"

namespace ssv {

constexpr int kDThreads = 256;
constexpr int kDWarps = kDThreads / 32;
constexpr int kDMaxCluster = 16;
// Most vectors of a slice held by a thread.  Longer slices mean fewer warps a row
// and so less bookkeeping; more CTAs an SM hide more of the exchange.  Measured
// (us, 896 x 129280 bf16 with gradient; 1024 x 151936 loss alone): 10 vectors,
// three and four CTAs an SM 104; 66.  19 vectors, two CTAs 91; 70.  The loss
// alone takes the same slices as with its gradient, so that both give the same
// bits.  Kernels exist for every third length, 4, 7, ... 19: places beyond a slice hold
// -inf and are worked on without a test (a branch per vector cost 10%).  Against
// kernels for every length (us, rows of 2e8 bf16 logits in all with gradient; loss
// alone): slices of 17 vectors 149 in the kernel for 19, 149 in their own; 97, 95.
// 14: 152, 149; 106, 103.  11: 162, 156; 114, 111.  8: 192, 186; 138, 133.  5: 258,
// 245; 195, 182.  Rows of 2 vectors a thread (3300 tokens): 604, 555; 472, 333.
constexpr int kDVecs = 19;

struct DistillParams {
  const void* z;
  void* grad;
  int N, V, k;
  int nst;            // shared-memory stages: rows of this cluster in flight
  uint32_t cap;       // bytes of a stage
  int skew;           // elements by which the base lies past a 16-byte boundary
  int odd;            // rows may start off one
  int wide;           // gradients may be written a vector's at a time (always where NV > 0)
  float s;            // log2(e) / T
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

__device__ __forceinline__ void st_async_f4(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   addr),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}

// Writes the gradients of a vector's tokens.  32-byte stores where fp32
// gradients come from 16-bit logits: two 16-byte stores a thread would each
// touch half of every sector.
template <class O, int PV, int bytes>
__device__ __forceinline__ void store_grads(O* dst, const f32x2 (&g)[PV / 2]) {
  float x[PV];
#pragma unroll
  for (int i = 0; i < PV / 2; ++i) f2_split(g[i], x[2 * i], x[2 * i + 1]);
  if constexpr (bytes >= 16) {
    if constexpr (sizeof(O) == 2) {
      static_assert(PV == 8, "16-bit gradients come from 16-bit logits");
      uint4 w;
      w.x = Elem<O>::pack(x[0], x[1]), w.y = Elem<O>::pack(x[2], x[3]);
      w.z = Elem<O>::pack(x[4], x[5]), w.w = Elem<O>::pack(x[6], x[7]);
      __stcs(reinterpret_cast<uint4*>(dst), w);
    } else {
      if constexpr (PV == 8 && bytes == 32) {
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]), "f"(x[1]),
                       "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                       : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < PV; i += 4)
          __stcs(reinterpret_cast<float4*>(dst + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PV; ++i) dst[i] = Elem<O>::from_f32(x[i]);
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
  int lead = (PV - (int)((s.f0 + skew) & (PV - 1))) & (PV - 1);
  if (lead > V) lead = V;
  const uint32_t nv = (uint32_t)(V - lead) / PV;
  s.a0 = lead;
  s.a1 = lead + (int)nv * PV;
  s.v0 = (int)(nv * rank / S);  // nv * S < 2^31: rows of at most 16 slices of shared memory
  s.v1 = (int)(nv * (rank + 1) / S);
  s.head = rank == 0 ? lead : 0;
  s.tail = rank == S - 1 ? V - s.a1 : 0;
  return s;
}

template <class E, class O, int NV>
__global__ void __launch_bounds__(kDThreads, NV == 0 ? 1 : 2) distill_kernel(const __grid_constant__ DistillParams P) {
  using T = Elem<E>;
  constexpr int PV = T::PV;
  constexpr bool kGrad = !std::is_same<O, NoGrad>::value;
  using OG = typename std::conditional<kGrad, O, float>::type;
  constexpr int kWide = sizeof(OG) * PV;  // bytes of a vector's gradients
  extern __shared__ __align__(128) unsigned char stage_mem[];
  // {m, s} of the unlisted and {m, s} of the listed tokens, per warp of the
  // cluster, pushed by every CTA into every CTA; two rows in turn
  __shared__ float4 box[2][kDMaxCluster * kDWarps];
  __shared__ __align__(8) uint64_t bars[4];      // stages, boxes
  __shared__ float edge[16];  // odd elements: 0..7 before, 8..15 after the aligned part
  __shared__ float4 grad_of;  // {mr, cb, factor of a listed token's 2^((z - m) s), m}, see below
  __shared__ float grad_w;    // the row's coefficient
  __shared__ uint32_t shared_count[kDWarps];
  __shared__ uint32_t abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int G = gridDim.x / S, c = blockIdx.x / S;
  const E* z = static_cast<const E*>(P.z);
  const uint32_t bar0 = smem_addr(bars), xbar0 = bar0 + 16;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_mbar_init();
    abort_flag = 0;
  }
  let_next_start();
  follow_previous();

  const uint64_t policy = l2_evict_first_policy();
  // Starts the copy of row n's slice into stage st (thread 0; rows that are
  // left out are not read).
  auto fetch = [&](long long n, int st, bool on) {
    if (tid != 0 || n >= P.N || !on) return;
    const Slice s = slice_of<PV>(n, P.V, P.skew, rank, S);
    const uint32_t bytes = (uint32_t)(s.v1 - s.v0) * 16u;
    mbar_arrive_expect_tx(bar0 + 8 * st, bytes);
    if (bytes)
      bulk_load(smem_addr(stage_mem) + st * P.cap, z + s.f0 + s.a0 + (long long)s.v0 * PV, bytes, bar0 + 8 * st,
                policy);
  };

  // Per-row values, loaded a row ahead and independently of one another; the
  // row's own scalars by warp 0 alone.
  struct Row {
    int id;
    float t, w, sum, rest, edge;
    bool live;
  };
  auto row_values = [&](long long n) {
    Row r{-1, 0.0f, 0.0f, 0.0f, 0.0f, -INFINITY, false};
    if (n < P.N) {
      r.live = P.keep[n];
      if (tid < P.k) {
        r.id = P.ids[n * P.k + tid];
        if (kGrad) r.t = P.t[n * P.k + tid];
      }
      if (kGrad && wid == 0) {
        const RowTeacher rt = P.row[n];
        r.sum = rt.sum;
        r.rest = rt.rest;
        r.w = P.weight ? P.weight[n] : 1.0f;
      }
      if (P.odd && tid < 16) {
        const Slice s = slice_of<PV>(n, P.V, P.skew, rank, S);
        if (tid < s.head) r.edge = T::to_f32(z[s.f0 + tid]);
        if (tid >= 8 && tid - 8 < s.tail) r.edge = T::to_f32(z[s.f0 + s.a1 + tid - 8]);
      }
    }
    return r;
  };

  if (tid == 0) {
    fetch(c, 0, P.keep[c]);
    if (P.nst == 2 && c + G < P.N) fetch((long long)c + G, 1, P.keep[c + G]);
  }
  Row cur = row_values(c);
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

  uint32_t par = 0;  // phase parity of each stage, one bit per stage
  uint32_t it = 0, ex = 0, failed = 0;
  OG* late = nullptr;  // a listed token's gradient, written after the next barrier: its place
  float late_v = 0.0f;  // is first written, as 0, by the thread that holds its vector
  Slice s = slice_of<PV>(c, P.V, P.skew, rank, S);
  for (long long n = c; n < P.N; n += G, ++it) {
    const int st = P.nst == 2 ? (int)(it & 1) : 0;
    if (P.odd) s = slice_of<PV>(n, P.V, P.skew, rank, S);
    s.f0 = n * P.V;
    const int nvl = s.v1 - s.v0;
    OG* out = kGrad ? static_cast<OG*>(P.grad) + s.f0 : nullptr;
    const long long n_fetch = n + (long long)P.nst * G;
    const bool fetch_on = tid == 0 && n_fetch < P.N && P.keep[n_fetch];
    const uint4 low = make_uint4(T::kLow, T::kLow, T::kLow, T::kLow);
    if (!cur.live) {  // left out: no gradient
      if (kGrad) {
        const f32x2 zero[PV / 2] = {};
        for (int i = tid; i < nvl; i += kDThreads) {
          if (NV > 0 || P.wide)
            store_grads<OG, PV, kWide>(out + s.a0 + (s.v0 + i) * PV, zero);
          else
            store_grads<OG, PV, 0>(out + s.a0 + (s.v0 + i) * PV, zero);
        }
        if (tid < s.head) out[tid] = Elem<OG>::from_f32(0.0f);
        if (tid >= 8 && tid - 8 < s.tail) out[s.a1 + tid - 8] = Elem<OG>::from_f32(0.0f);
      }
      fetch(n_fetch, st, fetch_on);
      cur = row_values(n + G);
      continue;
    }
    E* buf = reinterpret_cast<E*>(stage_mem + st * P.cap);
    const uint4* vec = reinterpret_cast<const uint4*>(buf);
    const uint32_t slot = ex & 1, xpar = (ex >> 1) & 1;
    ++ex;
    if (tid == 0) mbar_arrive_expect_tx(xbar0 + 8 * slot, S * kDWarps * 16);

    // after a wait that ran out, the later ones are short: the call ends soon
    const uint64_t limit = failed ? 100000ull : 2000000000ull;
    if (!mbar_wait_bounded(bar0 + 8 * st, (par >> st) & 1u, limit)) failed = abort_flag = 1;
    par ^= 1u << st;
    if (P.odd) {
      if (tid < 16) edge[tid] = cur.edge;
      __syncthreads();
    }

    // the listed tokens: taken out of the row, their logits kept by their threads
    float my_z = -INFINITY;
    bool mine = false;
    if (cur.id >= 0) {
      if (cur.id < s.a0) {
        mine = rank == 0;
        if (mine) {
          my_z = edge[cur.id];
          edge[cur.id] = -INFINITY;
        }
      } else if (cur.id >= s.a1) {
        mine = rank == S - 1;
        if (mine) {
          my_z = edge[8 + cur.id - s.a1];
          edge[8 + cur.id - s.a1] = -INFINITY;
        }
      } else {
        const int v = (cur.id - s.a0) / PV;
        mine = v >= s.v0 && v < s.v1;
        if (mine) {
          E* p = buf + (cur.id - s.a0 - s.v0 * PV);
          my_z = T::to_f32(*p);
          *p = T::neg_inf();
        }
      }
      if (mine) P.zi[n * P.k + tid] = my_z;
    }
    __syncthreads();
    if (kGrad && late) *late = Elem<OG>::from_f32(late_v);
    late = nullptr;

    // the slice, from here on in registers
    uint4 v[NV ? NV : 1];
    uint4 top = low;
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[j] = low;
        if (tid + j * kDThreads < nvl) v[j] = vec[tid + j * kDThreads];
      }
    }
    const float my_edge = P.odd && tid < 16 ? edge[tid] : -INFINITY;
    const Row next = row_values(n + G);  // travels while this row is worked on
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) top = T::vmax(top, v[j]);
    } else {
      for (int i = tid; i < nvl; i += kDThreads) top = T::vmax(top, vec[i]);
    }

    // normalisers: each warp relative to its own maximum
    float m = redux_max_nan(max_nan(T::hmax(top), my_edge)), sum = 0.0f;
    if (m > -INFINITY && m < INFINITY) {
      const f32x2 s2 = f2(P.s, P.s), m2 = f2(-m, -m);
      f32x2 a0 = f2(0.0f, 0.0f), a1 = a0;
      auto add = [&](const uint4& u) {
        f32x2 p[PV / 2];
        T::pairs(u, p);
#pragma unroll
        for (int i = 0; i < PV / 2; ++i) {
          float x, y;
          f2_split(f2_mul(f2_add(p[i], m2), s2), x, y);
          const f32x2 e = f2(ex2(x), ex2(y));
          if (i & 1)
            a1 = f2_add(a1, e);
          else
            a0 = f2_add(a0, e);
        }
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) add(v[j]);
      } else {
        for (int i = tid; i < nvl; i += kDThreads) add(vec[i]);
      }
      sum = f2_hsum(f2_add(a0, a1));
      if (P.odd) sum += exp2_scaled(my_edge - m, P.s);
      sum = warp_sum(sum);
    } else if (!(m < INFINITY)) {  // NaN or +inf among the logits
      sum = NAN;
      m = 0.0f;
    }
    float mk = -INFINITY, sk = 0.0f;
    if (wid * 32 < P.k) {
      mk = redux_max_nan(my_z);
      if (mk > -INFINITY && mk < INFINITY) {
        sk = warp_sum(exp2_scaled(my_z - mk, P.s));
      } else if (!(mk < INFINITY)) {
        sk = NAN;
        mk = 0.0f;
      }
    }
    if (lane < (int)S)
      st_async_f4(map_rank(smem_addr(&box[slot][rank * kDWarps + wid]), lane), m, sum, mk, sk,
                  map_rank(xbar0 + 8 * slot, lane));
    if constexpr (NV > 0) {  // the stage is free: everyone has its part in registers
      fence_proxy_async_smem();
      __syncthreads();
      fetch(n_fetch, st, fetch_on);
    }

    // Warp 0 joins the cluster's pairs, in the same order in every CTA.  (Done
    // by every warp, this was a third of the kernel's instructions.)
    if (wid == 0) {
      if (!mbar_wait_bounded(xbar0 + 8 * slot, xpar, limit)) failed = abort_flag = 1;
      __syncwarp();
      const int entries = (int)S * kDWarps;
      float mu = -INFINITY, ml = -INFINITY;
      for (int i = lane; i < entries; i += 32) {
        const float4 b = box[slot][i];
        mu = max_nan(mu, b.x);
        ml = max_nan(ml, b.z);
      }
      mu = redux_max_nan(mu);
      ml = redux_max_nan(ml);
      float su = 0.0f, sl = 0.0f;
      for (int i = lane; i < entries; i += 32) {
        const float4 b = box[slot][i];
        if (b.x > -INFINITY) su += b.y * exp2_scaled(b.x - mu, P.s);
        if (b.z > -INFINITY) sl += b.w * exp2_scaled(b.z - ml, P.s);
      }
      su = warp_sum(su);
      sl = warp_sum(sl);
      const bool some = mu > -INFINITY;
      RowNorm r;
      r.m = fmaxf(mu, ml);
      r.mr = mu;
      r.zr = su;
      const float rest_scale = some ? exp2_scaled(mu - r.m, P.s) : 0.0f;
      r.zl = ml > -INFINITY ? sl * exp2_scaled(ml - r.m, P.s) : 0.0f;
      r.z = (some ? su * rest_scale : 0.0f) + r.zl;
      if (!(r.m > -INFINITY)) r.z = NAN;  // no finite logit
      if (rank == 0 && lane == 0) {
        P.norm[n] = r;
        if (!(r.z < INFINITY)) raise(P.status, SPEC_DEV_BAD_LOGITS);
      }
      if (kGrad && lane == 0) {
        const float coef = coef0 * cur.w;
        const float mass = cur.sum + cur.rest;
        const float inv_z = 1.0f / r.z;
        float cb;  // factor of 2^((z - mr) s) for tokens that are not listed
        if (P.tail) {
          const float ql = r.zl * inv_z;
          const float diff = ql < 0.5f ? cur.sum - mass * ql : mass * (r.zr * rest_scale * inv_z) - cur.rest;
          cb = some ? coef * diff / r.zr : coef * (r.z - r.z);
        } else {
          cb = coef * mass * rest_scale * inv_z;
        }
        grad_of = make_float4(some ? mu : 0.0f, cb, mass * inv_z, r.m);
        grad_w = coef;
      }
    }

    if (kGrad) {
      __syncthreads();
      const float4 go = grad_of;
      const float coef = grad_w;
      const f32x2 s2 = f2(P.s, P.s), m2 = f2(-go.x, -go.x), c2 = f2(go.y, go.y);
      OG* dst = out + s.a0 + (s.v0 + tid) * PV;
      auto grads = [&](const uint4& u, f32x2 (&p)[PV / 2]) {
        T::pairs(u, p);
#pragma unroll
        for (int j = 0; j < PV / 2; ++j) {
          float x, y;
          f2_split(f2_mul(f2_add(p[j], m2), s2), x, y);
          p[j] = f2_mul(f2(ex2(x), ex2(y)), c2);
        }
      };
      f32x2 p[PV / 2];
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          grads(v[j], p);
          if (tid + j * kDThreads < nvl) store_grads<OG, PV, kWide>(dst + j * kDThreads * PV, p);
        }
      } else {
        for (int i = tid; i < nvl; i += kDThreads) {
          grads(vec[i], p);
          if (P.wide)
            store_grads<OG, PV, kWide>(out + s.a0 + (s.v0 + i) * PV, p);
          else
            store_grads<OG, PV, 0>(out + s.a0 + (s.v0 + i) * PV, p);
        }
      }
      if (P.odd && tid < 16) {
        const float g = exp2_scaled(my_edge - go.x, P.s) * go.y;
        if (tid < s.head) out[tid] = Elem<OG>::from_f32(g);
        if (tid >= 8 && tid - 8 < s.tail) out[s.a1 + tid - 8] = Elem<OG>::from_f32(g);
      }
      if (mine) {
        late = out + cur.id;
        late_v = coef * (exp2_scaled(my_z - go.w, P.s) * go.z - cur.t);
      }
    }
    if constexpr (NV == 0) {
      fence_proxy_async_smem();
      __syncthreads();
      fetch(n_fetch, st, fetch_on);
    }
    cur = next;
  }
  __syncthreads();
  if (kGrad && late) *late = Elem<OG>::from_f32(late_v);
  if (tid == 0 && abort_flag) raise(P.status, SPEC_DEV_TIMEOUT);
  cluster_sync();  // no CTA leaves while others may still push into it
}

// Row losses and their sum: a warp per row.
__global__ void __launch_bounds__(256) distill_finish_kernel(const FinishParams P, const RowNorm* norm) {
  let_next_start();
  follow_previous();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = (long long)blockIdx.x * 8 + w;
  const bool on = n < P.N && P.keep[n];
  float loss = 0.0f, weight = 0.0f;
  if (on) {
    const RowNorm r = norm[n];
    const RowTeacher t = P.row[n];
    weight = P.weight ? P.weight[n] : 1.0f;
    const F2 logz = log_pair(r.z);
    RowLog g;
    g.m = r.m;
    g.base = pair_add(logz, F2{-t.shift, -t.shift_lo});
    g.extra = 0.0f;
    if (t.rest > 0.0f) {
      // each side from the listed tokens' mass where that is the smaller part
      const float lt = t.sum < 0.5f ? log1pf(-t.sum) : logf(t.rest);
      const float ql = r.zl / r.z;
      float lq = -INFINITY;
      if (ql < 0.5f) {
        lq = log1pf(-ql);
      } else if (r.mr > -INFINITY) {
        const F2 v = pair_add(pair_add(log_pair(r.zr), F2{-logz.hi, -logz.lo}), two_mul(r.mr - r.m, P.c));
        lq = v.hi + v.lo;
      }
      g.extra = t.rest * (lt - lq);
    }
    loss = row_loss_warp(P, n, lane, g);
  }
  if (lane == 0 && n < P.N) P.row_loss[n] = loss;
  finish_sums(P, loss, on, weight);
}

}  // namespace ssv
