// The cache around a decoding step: block tables, free pages and slot maps from
// request lengths, and the copy of committed keys and values into their slots.
#pragma once

#include <cstdint>

#include "spec_verify.h"

namespace ssv {

// ---- tables -----------------------------------------------------------------------

struct PlanParams {
  const int32_t *lens, *added, *table, *free, *count;
  int32_t *out_table, *out_free, *out_count, *out_lens, *slots;
  uint32_t* status;
  int B, T, width, capacity, page;
  int per;  // requests a CTA, from the grid
};

constexpr int kPlanThreads = 256;
constexpr int kNoSlot = 0x7FFFFFFF;  // beyond every cache: pages * page_size < 2^31

// A request's pages before and after the step.
struct PlanRequest {
  int held, want;
  bool fits;
  __device__ int back() const { return fits && held > want ? held - want : 0; }
  __device__ int need() const { return fits && want > held ? want - held : 0; }
};
__device__ __forceinline__ PlanRequest plan_request(const PlanParams& P, int len, int added) {
  const long long room = (long long)P.width * P.page, after = (long long)len + added;
  PlanRequest r;
  r.fits = len >= 0 && len <= room && after >= 0 && after <= room && added <= P.T;
  // below 2^31 each, as width * page is: 32 bits do
  r.held = r.fits ? (int)(((uint32_t)len + (uint32_t)P.page - 1u) / (uint32_t)P.page) : 0;
  r.want = r.fits ? (int)(((uint32_t)after + (uint32_t)P.page - 1u) / (uint32_t)P.page) : 0;
  return r;
}

// Request by request: pages given back go on the stack at count + (those of the
// requests before it), pages needed come from count + (all given back) - 1 -
// (those needed before it).  Every CTA sums the whole batch's lengths for
// itself (8 bytes a request, from L2) and then writes the rows of its own
// requests, so that one launch does without a pass over the batch before it;
// no CTA writes what another one reads, also in place: tables keep the entries
// of pages given back, and pushes lie above the stack's old top.
// Sums of pages are 32 bits: a request gives back or needs at most a row of the table, and
// the host refuses tables of 2^31 entries.
// Bound: latency at ordinary sizes (8 requests 4.8 us), else the copy of table and stack
// (1024 requests with 2048 pages each, 34 MB: 15 us warm, 18 cold), which a call in place leaves out.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams P) {
  __shared__ int back_at[kPlanThreads + 1];  // given back before each thread's requests
  __shared__ int need_at[kPlanThreads + 1];
  __shared__ int popped_max;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int first = blockIdx.x * P.per, last = min(first + P.per, P.B);
  // each thread sums a run of requests, then the runs are scanned
  const int run = (P.B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * run, P.B), r1 = min(r0 + run, P.B);
  int back = 0, need = 0;
  for (int b = r0; b < r1; ++b) {
    const PlanRequest r = plan_request(P, P.lens[b], P.added[b]);
    back += r.back();
    need += r.need();
  }
  __shared__ int warp_back[kPlanThreads / 32], warp_need[kPlanThreads / 32];
  int sb = back, sn = need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int xb = __shfl_up_sync(0xffffffffu, sb, o), xn = __shfl_up_sync(0xffffffffu, sn, o);
    if (lane >= o) sb += xb, sn += xn;
  }
  if (lane == 31) warp_back[wid] = sb, warp_need[wid] = sn;
  if (tid == 0) popped_max = 0;
  __syncthreads();
  for (int w = 0; w < wid; ++w) sb += warp_back[w], sn += warp_need[w];
  back_at[tid] = sb - back;
  need_at[tid] = sn - need;
  if (tid == kPlanThreads - 1) back_at[kPlanThreads] = sb, need_at[kPlanThreads] = sn;
  __syncthreads();
  const int count = *P.count, returned = back_at[kPlanThreads];
  const bool sound = count >= 0 && count <= P.capacity && returned <= P.capacity - count;
  const int have = sound ? count + returned : 0;

  // where the b-th request's pages start among those given back and needed
  auto sums_before = [&](int b, int& bk, int& nd) {
    const int t = b / run;
    bk = back_at[t], nd = need_at[t];
    for (int i = t * run; i < b; ++i) {
      const PlanRequest r = plan_request(P, P.lens[i], P.added[i]);
      bk += r.back();
      nd += r.need();
    }
  };
  // whole 16-byte pieces where both sides allow, entries at the ends
  auto copy = [&](const int32_t* from, int32_t* to, long long n, int at, int step) {
    const bool even = ((reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to)) & 15) == 0;
    const long long pieces = even ? n / 4 : 0;
    const int4* from4 = reinterpret_cast<const int4*>(from);
    int4* to4 = reinterpret_cast<int4*>(to);
#pragma unroll 4
    for (long long i = at; i < pieces; i += step) to4[i] = from4[i];
    for (long long i = pieces * 4 + at; i < n; i += step) to[i] = from[i];
  };
  // entry i of the stack once the pages given back lie on it
  auto stack_at = [&](int i) -> int {
    if (i < count) return P.free[i];
    i -= count;
    int lo = 0, hi = kPlanThreads;  // the thread run that holds the i-th page given back
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (back_at[mid] <= i ? lo : hi) = mid;
    }
    i -= back_at[lo];
    for (int b = lo * run;; ++b) {
      const PlanRequest r = plan_request(P, P.lens[b], P.added[b]);
      if (i < r.back()) return P.table[(long long)b * P.width + r.want + i];
      i -= r.back();
    }
  };

  const bool table_copy = P.out_table != P.table;
  for (int b = first; b < last; ++b) {
    const int len = P.lens[b], added = P.added[b];
    PlanRequest r = plan_request(P, len, added);
    int bk, nd;
    sums_before(b, bk, nd);
    const int needs = sound ? r.need() : 0;
    const bool served = sound && r.fits && (needs == 0 || nd + needs <= have);
    const long long row = (long long)b * P.width;
    if (table_copy) {
      copy(P.table + row, P.out_table + row, P.width, tid, kPlanThreads);
      if (served && needs) __syncthreads();  // the new pages go over the copy
    }
    if (served)
      for (int i = tid; i < needs; i += kPlanThreads) P.out_table[row + r.held + i] = stack_at(have - 1 - (nd + i));
    if (sound)
      for (int i = tid; i < r.back(); i += kPlanThreads) P.out_free[count + bk + i] = P.table[row + r.want + i];
    bool no_slot = false;
    for (int i = tid; i < P.T; i += kPlanThreads) {
      int slot = -1;
      if (served && i < added) {
        const int pos = len + i, p = pos / P.page;
        const int page = p < r.held ? P.table[row + p] : stack_at(have - 1 - (nd + p - r.held));
        // ids come from the caller: one that no cache has may wrap to another page's slot in 32 bits
        const long long at = (long long)page * P.page + (pos - p * P.page);
        const bool named = page >= 0 && at <= kNoSlot;
        slot = named ? (int)at : kNoSlot;
        no_slot |= !named;
      }
      P.slots[(long long)b * P.T + i] = slot;
    }
    if (no_slot && P.status) atomicOr(P.status, SPEC_DEV_BAD_PAGE);
    if (tid == 0) {
      P.out_lens[b] = served ? len + added : len;
      const uint32_t bits = (!r.fits || !sound ? SPEC_DEV_BAD_OFFSETS : 0u) |
                            (sound && r.fits && !served ? SPEC_DEV_NO_PAGES : 0u);
      if (bits && P.status) atomicOr(P.status, bits);
    }
  }
  // the stack below the pages given back, and above them
  if (P.out_free != P.free) {
    const int at = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    const int gap0 = sound ? count : 0, gap1 = sound ? have : 0, even = min((gap1 + 3) & ~3, P.capacity);
    copy(P.free, P.out_free, gap0, at, step);
    for (int i = gap1 + at; i < even; i += step) P.out_free[i] = P.free[i];
    copy(P.free + even, P.out_free + even, P.capacity - even, at, step);
  }
  // the new count: what is needed, or where that is too much, the longest start of it that is there
  if (blockIdx.x == 0) {
    int popped = sound ? need_at[kPlanThreads] : 0;
    if (popped > have) {
      int sum = need_at[tid], mine = 0;
      for (int b = r0; b < r1; ++b) {
        sum += plan_request(P, P.lens[b], P.added[b]).need();
        if (sum <= have) mine = sum;
      }
      if (mine) atomicMax(&popped_max, mine);
      __syncthreads();
      popped = popped_max;
    }
    if (tid == 0) *P.out_count = sound ? have - popped : count;
  }
}

// ---- commit -----------------------------------------------------------------------

struct CommitParams {
  spec_commit_t a;
  uint32_t* status;
};

// A warp per (layer, request, place): its row's keys and values, all heads, in
// 16-byte pieces, eight a lane in flight.  Bound: memory, the rows in and out (32 layers,
// 64 trees, 277 MB: 50 us, 5.5 TB/s).
constexpr int kCommitBatch = 4;
__global__ void __launch_bounds__(256) commit_kernel(const __grid_constant__ CommitParams P) {
  const spec_commit_t& A = P.a;
  const int lane = threadIdx.x & 31;
  const long long items = (long long)A.layers * A.B * A.S;
  const int per_head = A.D / 8, pieces = A.Hkv * per_head;
  for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 8) {
    const int i = (int)(it % A.S);
    const long long lb = it / A.S;
    const int b = (int)(lb % A.B), layer = (int)(lb / A.B);
    const int slot = A.slots[(long long)b * A.S + i];
    if (slot < 0) continue;
    int r0 = b * A.T, r1 = r0 + A.T;
    bool rows_ok = true;
    if (A.row_offsets) {
      r0 = A.row_offsets[b], r1 = A.row_offsets[b + 1];
      rows_ok = r0 >= 0 && r1 >= r0 && r1 <= A.rows && r1 - r0 <= A.T;
    }
    int row = i;
    if (i > 0 && A.path) {
      row = A.path[b * A.path_stride + i - 1];
      row = row < 0 || row >= 0x7FFFFFFF ? -1 : row + 1;
    }
    const bool page_ok = slot < A.pages * A.page_size;
    rows_ok = rows_ok && row >= 0 && row < r1 - r0;
    if (!rows_ok || !page_ok) {
      if (lane == 0 && P.status)
        atomicOr(P.status, (rows_ok ? 0u : SPEC_DEV_BAD_OFFSETS) | (page_ok ? 0u : SPEC_DEV_BAD_PAGE));
      continue;
    }
    const long long r = r0 + row, page = slot / A.page_size, place = slot % A.page_size;
    const uint16_t* kn = (const uint16_t*)A.k_new + layer * A.k_new_stride[0] + r * A.k_new_stride[1];
    const uint16_t* vn = (const uint16_t*)A.v_new + layer * A.v_new_stride[0] + r * A.v_new_stride[1];
    uint16_t* kc = (uint16_t*)A.k_cache + layer * A.k_stride[0] + page * A.k_stride[1] + place * A.k_stride[2];
    uint16_t* vc = (uint16_t*)A.v_cache + layer * A.v_stride[0] + page * A.v_stride[1] + place * A.v_stride[2];
    for (int p0 = lane; p0 < pieces; p0 += 32 * kCommitBatch) {
      uint4 k[kCommitBatch], v[kCommitBatch];
#pragma unroll
      for (int u = 0; u < kCommitBatch; ++u) {
        const int p = p0 + 32 * u, h = p / per_head, d = (p - h * per_head) * 8;
        if (p < pieces) {
          k[u] = __ldcs((const uint4*)(kn + h * A.k_new_stride[2] + d));
          v[u] = __ldcs((const uint4*)(vn + h * A.v_new_stride[2] + d));
        }
      }
#pragma unroll
      for (int u = 0; u < kCommitBatch; ++u) {
        const int p = p0 + 32 * u, h = p / per_head, d = (p - h * per_head) * 8;
        if (p < pieces) {
          *(uint4*)(kc + h * A.k_stride[3] + d) = k[u];
          *(uint4*)(vc + h * A.v_stride[3] + d) = v[u];
        }
      }
    }
  }
}

}  // namespace ssv
