// Attention of a pass's rows over a paged cache and the pass's own keys.
//
//   s_n = scale q . k_n,  out = sum_n e^(s_n - m) v_n / sum_n e^(s_n - m)
//
// over the cached tokens of the row's request and the rows of the pass that its
// mask names.  Running maximum m and sum in fp32.
#pragma once

#include "loss_common.cuh"

namespace ssv {

struct AttendParams {
  spec_attention_t a;
  uint32_t* status;
};

struct AttendRequest {
  int r0, rows, context;
  uint32_t bad;
};
__device__ __forceinline__ AttendRequest attend_request(const spec_attention_t& A, int b) {
  AttendRequest r;
  r.bad = 0;
  r.r0 = b * A.T;
  r.rows = A.T;
  if (A.row_offsets) {
    r.r0 = A.row_offsets[b];
    const int end = A.row_offsets[b + 1];
    if (r.r0 < 0 || end < r.r0 || end > A.rows || end - r.r0 > A.T) {
      r.bad = SPEC_DEV_BAD_OFFSETS;
      r.rows = 0;
    } else {
      r.rows = end - r.r0;
    }
  }
  r.context = A.context_lens[b];
  const int most = (int)min((long long)A.table_width * A.page_size, 0x7FFFFFFFll);
  if (r.context < 0 || r.context > most) {
    r.bad |= SPEC_DEV_BAD_OFFSETS;
    r.context = min(max(r.context, 0), most);
  }
  return r;
}

// A warp per (request, key head, row, head of the group).
template <class E>
__global__ void __launch_bounds__(128) attend_plain_kernel(const __grid_constant__ AttendParams P) {
  using El = Elem<E>;
  const spec_attention_t& A = P.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int b = blockIdx.y, h = blockIdx.z;
  __shared__ float qs[4][256];
  const AttendRequest R = attend_request(A, b);
  if (R.bad && threadIdx.x == 0 && P.status) atomicOr(P.status, R.bad);
  const int i = blockIdx.x * 4 + wid;
  if (i >= R.rows) return;
  const int kh = h / (A.Hq / A.Hkv);
  const E* q = (const E*)A.q + (long long)(R.r0 + i) * A.q_stride[0] + h * A.q_stride[1];
  for (int d = lane; d < A.D; d += 32) qs[wid][d] = El::to_f32(q[d]) * A.scale;
  __syncwarp();
  float m = -INFINITY, sum = 0.0f, acc[8] = {};
  const int n_all = R.context + R.rows;
  for (int n0 = 0; n0 < n_all; n0 += 32) {
    const int n = n0 + lane;
    const E *k = nullptr, *v = nullptr;
    bool sees = n < n_all;
    if (sees && n < R.context) {
      const int page = A.block_table[b * A.table_stride + n / A.page_size], at = n % A.page_size;
      if (page < 0 || page >= A.pages) {
        if (P.status) atomicOr(P.status, SPEC_DEV_BAD_PAGE);
      } else {
        k = (const E*)A.k_cache + page * A.k_stride[0] + at * A.k_stride[1] + kh * A.k_stride[2];
        v = (const E*)A.v_cache + page * A.v_stride[0] + at * A.v_stride[1] + kh * A.v_stride[2];
      }
    } else if (sees) {
      const int j = n - R.context;
      sees = A.mask ? A.mask[((long long)b * A.T + i) * A.T + j] != 0 : j <= i;
      k = (const E*)A.k_new + (long long)(R.r0 + j) * A.k_new_stride[0] + kh * A.k_new_stride[1];
      v = (const E*)A.v_new + (long long)(R.r0 + j) * A.v_new_stride[0] + kh * A.v_new_stride[1];
    }
    float s = sees ? 0.0f : -INFINITY;
    if (sees && k)
      for (int d = 0; d < A.D; ++d) s = fmaf(qs[wid][d], El::to_f32(k[d]), s);
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m1 = fmaxf(m, mx), off = m1 == -INFINITY ? 0.0f : m1;
    const float p = __expf(s - off), fix = __expf(m - off);
    m = m1;
    sum = sum * fix + warp_sum(p);
    for (int c = 0; c < 8; ++c) acc[c] *= fix;
    for (int j = 0; j < 32 && n0 + j < n_all; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const E* vj = (const E*)__shfl_sync(0xffffffffu, (unsigned long long)v, j);
      const bool see_j = __shfl_sync(0xffffffffu, (int)sees, j);
      if (!see_j || !vj) continue;
      for (int c = 0; c < 8; ++c)
        if (lane + 32 * c < A.D) acc[c] = fmaf(pj, El::to_f32(vj[lane + 32 * c]), acc[c]);
    }
  }
  E* out = (E*)A.out + ((long long)(R.r0 + i) * A.Hq + h) * A.D;
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  for (int c = 0; c < 8; ++c)
    if (lane + 32 * c < A.D) out[lane + 32 * c] = El::from_f32(acc[c] * inv);
  if (A.lse && lane == 0) A.lse[(long long)(R.r0 + i) * A.Hq + h] = m + logf(sum);
}

}  // namespace ssv
