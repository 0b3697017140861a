// Attention of a pass's rows over a paged cache and the pass's own keys, on the
// tensor cores.
//
//   s_n = q . k_n,  w_n = 2^(c (s_n - m) + h),  out = sum_n w_n v_n / sum_n w_n,  c = scale log2(e)
//
// over the cached tokens of the row's request and the rows of the pass that its
// mask names.  One pass over the keys: m is a running maximum, and where a weight
// would pass 2^(h + kLag) the sums so far are rescaled (a smaller growth leaves m
// behind the maximum, which changes no ratio).
//
// m is taken off the scores before they are multiplied by c.  c s_n - c m in one
// multiplication and addition would round c m first and scale all weights by 2 to the
// power of that error, which for scores from 2^26 on leaves the weights' range (it took 1%
// less for 33 rows).
//
// Scores, sums and the result are fp32.  The weights are rounded once to the operands'
// 16-bit type, which the tensor cores ask for both factors of the product with v: the
// result is off its 64-bit value by 2.3e-3 of its size in bf16 where rounding it alone
// would be 1.7e-3 (1.7e-4 and 1.5e-4 in fp16).  h is 0 in bf16; in fp16 it is 11,
// so that weights keep all bits down to 2^-25 of the largest and are off by at most 2^-36 of
// it below (with h = 0, the keys of a long context with 2^-25 each were lost, or
// counted twice).  The result is divided by the sum of the rounded weights, so that a row
// which one key dominates loses nothing; lse takes the sum before rounding.
//
// All query rows that share a key head (the pass's rows times the group's
// heads) form tiles of 128 rows, so that the cache is read once for all of
// them.  Bound: the cache's bytes, up to about 128 rows a key head; beyond, the
// products and the softmax.
//
// The batch is cut into units (request, key head, 128 or 256 rows), a unit into
// tiles of keys, and all units, one behind the other, into shares of equal cost, one a
// CTA and SM.  A unit that spans CTAs leaves one partial result (out, m, sum) a
// CTA; a second launch joins them.  The shares come from the lengths on the
// device: nothing of the launch depends on them, and the order of the sums
// follows from the lengths alone.
//
// A CTA: one warp loads q and the keys and one the values (through a ring of
// shared-memory tiles by TMA; a page's part of a tile is a box of the tensor map),
// one issues the products (scores into tensor memory, weights times values
// with the weights read from tensor memory), and two warpgroups do the softmax, a
// thread per row.
//
// Measured with heads of 128 in bf16: 128 requests of one token over 64 to 4096 cached
// ones (32/8 heads, pages of 16) 187 us, 5.8 TB/s; 2 x 8 rows over 131072 (64/8 heads)
// 169 us, 6.4 TB/s; 32 trees of 33 rows over 512 to 8192 (132 query rows a key head: two
// row tiles) 153 us, where the cache alone would take 89.  With two row tiles a group has
// one buffer of scores, so that a tile's scores, softmax and product follow each other and
// the tensor cores work 45% of the time; their products, of 256 rows of which 132 are live, would
// take 76 us at the measured rate.
#pragma once

#include "loss_common.cuh"
#include "tc05.cuh"

namespace ssv {

constexpr uint64_t kAttendWaitNs = 2000000000ull;
constexpr int kAttendMaxGroup = 128;

// DP: head size in shared memory.  MT: tiles of 128 query rows that a CTA works
// on.  GROUPS: warpgroups of the softmax.  Two groups take a row tile each, or
// take turns over the tiles of keys of one row tile, with a result, maximum and sum
// of their own that are joined at the end; a head beyond 128 leaves tensor
// memory for one result only.
template <int DP, int MT>
struct AttendShape {
  static constexpr int NK = DP > 128 ? 64 : 128;      // keys a tile
  static constexpr int GROUPS = DP > 128 ? 1 : 2;
  static constexpr bool kTurns = MT == 1 && GROUPS == 2;
  static constexpr int CH = DP / 64;                  // 128-byte columns of a row
  static constexpr int kChunk = NK * 128;             // bytes of one column of a tile
  static constexpr int kTile = CH * kChunk;           // keys or values of a tile
  static constexpr int kQChunk = 128 * 128;
  static constexpr int kQ = MT * CH * kQChunk;
  static constexpr int kRoom = 217 * 1024;
  static constexpr int kRing = (kRoom - kQ) / kTile > 12 ? 12 : (kRoom - kQ) / kTile;
  static constexpr int kSmem = kQ + kRing * kTile + 1024;
  // The groups' warps come first, then four of which three work: the products' and the keys'
  // warps share a scheduler (and its instruction cache) with no softmax of the first 64 rows.
  static constexpr int kValuesWarp = 4 * GROUPS + 1, kProductWarp = kValuesWarp + 1, kKeysWarp = kValuesWarp + 2;
  static constexpr int kThreads = 32 * (4 * GROUPS + 4);
  static constexpr int kOut = 256;                    // tensor-memory column of the results
  static_assert(2 * NK <= kOut && kOut + GROUPS * DP <= 512, "tensor memory");
  static_assert(kRing >= 4, "keys and values of two tiles");
};

struct AttendSplit {  // a unit that goes on in the next CTAs
  int unit, last;  // last: the CTA that holds its end; -1: none
  int r0, rows;    // of its request
};

struct AttendLaunch {
  CUtensorMap q, k_new, v_new;
  CUtensorMap k, v;    // boxes of `box` tokens of a page (see `fold`)
  CUtensorMap k8, v8;  // boxes of 8: the last tokens
  spec_attention_t a;
  uint32_t* status;
  float* part;         // [CTAs][2][slot_rows][DP]
  float4* stat;        // [CTAs][2][slot_rows]: m, sum of the rounded weights, sum of the weights
  AttendSplit* split;  // [CTAs]
  float c;             // |scale| log2(e), or 1 for a scale of 0
  float flip;          // 1, or what the scores are multiplied by first: -1 or 0
  int group, tok;      // heads a key head, rows of the pass in 128 query rows
  int box;             // tokens of a page that one copy takes
  int q_rows;          // rows of the pass that one copy of q takes
  int beyond;          // a page that the maps do not have: reads as zeros
  int slot_rows;       // query rows of a partial result
  // One copy takes all 64-element columns of a box where a head's columns continue an
  // even dimension of the cache: 1, its heads (one behind the other in a token), 2, its
  // pages (heads of pages evenly spaced); 0: a copy for each column.
  int fold_k, fold_v;
  int row8, col;       // bytes between groups of eight rows, 64-element columns of a tile in shared memory
};

// ---- requests, units and tiles ---------------------------------------------------

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
  const int most = A.table_width * A.page_size;  // below 2^31, checked
  if (r.context < 0 || r.context > most) {
    r.bad |= SPEC_DEV_BAD_OFFSETS;
    r.context = min(max(r.context, 0), most);
  }
  return r;
}

// A request's tiles of keys: `full` of the context alone, then the context's
// last `rest` tokens, a gap up to a multiple of 8, and the pass's rows.
constexpr int kAttendUnitCost = 3;

template <int NK>
struct AttendSpan {
  int r0, rows, full, rest, tiles;
  long long cost;  // of all units: their tiles and kAttendUnitCost each
  __device__ __forceinline__ void load(const spec_attention_t& A, int b, int tok_unit) {
    const AttendRequest r = attend_request(A, b);
    r0 = r.r0, rows = r.rows;
    full = r.context / NK;
    rest = r.context % NK;
    tiles = full + (((rest + 7) & ~7) + rows + NK - 1) / NK;
    cost = rows ? (long long)(tiles + kAttendUnitCost) * A.Hkv * ((rows + tok_unit - 1) / tok_unit) : 0;
  }
  // Tile t >= full: its cached tokens lie at [0, cached), the pass's rows [j0, j0 + fresh) from place `at` on.
  __device__ __forceinline__ void tail(int t, int& cached, int& at, int& j0, int& fresh) const {
    const int from = (t - full) * NK, r8 = (rest + 7) & ~7;
    cached = from == 0 ? rest : 0;
    at = max(0, r8 - from);
    j0 = max(0, from - r8);
    fresh = min(rows - j0, NK - at);
  }
};

// The CTA's share, unit by unit.  Every warp walks it by itself.  Shares are cut
// where costs are equal: a unit costs as much as its tiles and kAttendUnitCost more
// (its query rows, last tile and result), which come before its first tile.
template <int NK>
struct AttendWalk {
  long long at, end;  // costs of the batch
  long long off;      // of request b
  int b, tok_unit;
  AttendSpan<NK> s;
  // the segment
  int unit, t0, t1;
  long long unit_end; // of the unit, in the batch's costs
  __device__ __forceinline__ bool next(const spec_attention_t& A) {
    while (at < end) {
      while (off >= s.cost) {  // below the total there is another request
        if (b + 1 >= A.B) return false;  // the lengths changed under the call
        off = 0;
        s.load(A, ++b, tok_unit);
      }
      const int each = s.tiles + kAttendUnitCost;
      int from;
      if (s.cost <= 0x7FFFFFFF) {
        unit = (int)off / each;
        from = (int)off - unit * each;
      } else {
        unit = (int)(off / each);
        from = (int)(off - (long long)unit * each);
      }
      const int n = (int)min((long long)(each - from), end - at);
      unit_end = at + each - from;
      t0 = max(from - kAttendUnitCost, 0);
      t1 = from + n - kAttendUnitCost;
      at += n;
      off += n;
      if (t1 > t0) return true;
    }
    return false;
  }
};

// What a weight's exponent may lag by before the sums are rescaled, and what is added to it: together they
// stay below fp16's largest exponent, 15, by what the exponential's argument rounds by.
template <class E>
struct AttendRange {
  static constexpr bool kHalf = Elem<E>::kLow != 0xFF80FF80u;
  static constexpr float kLag = kHalf ? 4.0f : 8.0f, kUp = kHalf ? 11.0f : 0.0f;
};

template <class E>
__device__ __forceinline__ bool not_finite16(uint32_t x) {  // one element
  if constexpr (sizeof(E) == 2 && Elem<E>::kLow == 0xFF80FF80u)
    return (x & 0x7F80u) == 0x7F80u;
  else
    return (x & 0x7C00u) == 0x7C00u;
}

// ---- the kernel --------------------------------------------------------------------

template <class E, int DP, int MT>
__global__ void __launch_bounds__((AttendShape<DP, MT>::kThreads), 1)
    attend_kernel(const __grid_constant__ AttendLaunch L) {
  using El = Elem<E>;
  using Sh = AttendShape<DP, MT>;
  constexpr int NK = Sh::NK, CH = Sh::CH, R = Sh::kRing, kThreads = Sh::kThreads, GROUPS = Sh::GROUPS;
  constexpr bool kTurns = Sh::kTurns;
  constexpr bool kBf16 = El::kLow == 0xFF80FF80u;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * R + 16];
  __shared__ float4 row_stat[2][GROUPS][128];  // kTurns: maximum and sums of a group's rows, two segments in turn
  __shared__ uint32_t tmem_slot;
  __shared__ long long warp_sum_of[kThreads / 32];
  __shared__ long long start_off;
  __shared__ int start_b;
  __shared__ int not_finite[2];  // a value of the pass that is not finite was met: 1 + number of the segment

  const spec_attention_t& A = L.a;
  const int tid = threadIdx.x, wid = same_in_warp(tid >> 5), lane = tid & 31;
  const uint32_t q0 = (smem_addr(raw) + 1023u) & ~1023u, ring0 = q0 + Sh::kQ;
  const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * R;
  const uint32_t bar_q = bar_empty + 8 * R, bar_q_free = bar_q + 8;
  const uint32_t bar_s = bar_q_free + 8;      // scores written, two buffers
  const uint32_t bar_p = bar_s + 16;          // weights written, two
  const uint32_t bar_o = bar_p + 16;          // a product with the values done, per result
  const uint32_t bar_o_free = bar_o + 16;     // the result read, per result
  const uint32_t bar_fix = bar_o_free + 16;   // values of a last tile looked over, two in turn
  const uint32_t bar_join = bar_fix + 16;     // kTurns: both groups' maxima and sums are there
  const uint32_t bar_drain = bar_join + 8;
  const int tok_unit = L.tok * MT;

  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + 8 * i, 1);
      mbar_init(bar_p + 8 * i, 4);
      mbar_init(bar_o + 8 * i, 1);
      mbar_init(bar_o_free + 8 * i, kTurns ? 8 : 4);
      mbar_init(bar_fix + 8 * i, 4);
      not_finite[i] = 0;
    }
    mbar_init(bar_join, 8);
    mbar_init(bar_drain, 1);
    fence_mbar_init();
    prefetch_map(&L.q);
    prefetch_map(&L.k);
    prefetch_map(&L.v);
    prefetch_map(&L.k8);
    prefetch_map(&L.v8);
    prefetch_map(&L.k_new);
    prefetch_map(&L.v_new);
  }
  if (wid == Sh::kProductWarp) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  }
  // This CTA's share: each thread sums a run of requests, the runs are scanned.
  const int run = (A.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, A.B), b1 = min(b0 + run, A.B);
  AttendSpan<NK> mine;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    mine.load(A, b, tok_unit);
    sum += mine.cost;
    if (blockIdx.x == 0) raise(L.status, attend_request(A, b).bad);
  }
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) warp_sum_of[wid] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == wid) upto += total;
    total += warp_sum_of[w];
  }
  const int ctas = (int)min((long long)gridDim.x, total);
  const int cta = blockIdx.x;
  long long first = 0, end = 0;
  if (cta < ctas) first = total * cta / ctas, end = total * (cta + 1) / ctas;
  if (first < end && upto > first && upto - sum <= first) {
    long long off = first - (upto - sum);
    int b = b0;
    for (mine.load(A, b, tok_unit); off >= mine.cost && b + 1 < b1; mine.load(A, ++b, tok_unit)) off -= mine.cost;
    start_b = b;
    start_off = off;
  }
  __syncthreads();
  const uint32_t tmem = (uint32_t)same_in_warp((int)tmem_slot);
  AttendWalk<NK> w;
  w.at = first, w.end = end, w.tok_unit = tok_unit;
  if (first < end) {
    w.b = start_b, w.off = start_off;
    w.s.load(A, w.b, tok_unit);
  }
  const int chunks = (A.D + 63) / 64;  // 128-byte columns that hold anything

  // Place of tile i's keys and values among the 2n entries of the ring that a segment of n tiles takes.
  auto place_k = [](int i, int) { return MT == 2 ? 2 * i : i == 0 ? 0 : 2 * i - 1; };
  auto place_v = [](int i, int n) { return MT == 2 ? 2 * i + 1 : i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

  if (wid == Sh::kKeysWarp || wid == Sh::kValuesWarp) {
    // ---- loads: a warp for q and the keys, one for the values ----
    const bool values = wid == Sh::kValuesWarp;
    uint32_t base = 0, step = 0, seg = 0;
    uint32_t bad = 0;
    bool ok = true, any = false;
    for (; ok && __any_sync(0xffffffffu, w.next(A)); ++seg) {
      const int t0 = same_in_warp(w.t0), n = same_in_warp(w.t1) - t0, unit = same_in_warp(w.unit);
      const int kh = unit % A.Hkv, mg = unit / A.Hkv, full_tiles = same_in_warp(w.s.full);
      const int32_t* table = A.block_table + w.b * A.table_stride;
      for (int i = 0; ok && i < n; ++i) {
        const int t = t0 + i;
        step = base + (values ? place_v(i, n) : place_k(i, n));
        const uint32_t s = step % R, use = step / R, full = bar_full + 8 * s, dst = ring0 + s * Sh::kTile;
        // The tile's cached tokens in whole boxes of the map, then in boxes of 8, and the pass's
        // rows; a lane looks up the page and place of one box.
        int cached = NK, at = 0, j0 = 0, fresh = 0;
        if (t >= full_tiles) w.s.tail(t, cached, at, j0, fresh);
        cached = same_in_warp(cached);
        const int big = cached / L.box, small = (cached - big * L.box + 7) / 8, rows_new = same_in_warp((fresh + 7) / 8);
        const int pos = t * NK + (lane < big ? lane * L.box : big * L.box + (lane - big) * 8), p = pos / A.page_size;
        const int place = pos - p * A.page_size;
        int page = lane < big + small ? __ldg(table + p) : 0;
        if (use > 0) ok = mbar_wait_bounded(bar_empty + 8 * s, (use - 1) & 1u, kAttendWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        any = true;
        if (lane < big + small && (page < 0 || page >= A.pages)) page = L.beyond, bad = SPEC_DEV_BAD_PAGE;
        mbar_expect(full, (uint32_t)(chunks * (big * L.box + (small + rows_new) * 8) * 128));
        auto of_lane = [&](int x, int from) { return (int)__reduce_or_sync(0xffffffffu, lane == from ? (uint32_t)x : 0u); };
        int pl = t * NK % A.page_size, pg = of_lane(page, 0);  // the place is stepped along
        uint32_t to = dst;
        const CUtensorMap* map = values ? &L.v : &L.k;
        const int fold = values ? L.fold_v : L.fold_k;
        const int col0 = fold == 1 ? kh * chunks : 0, heads = fold == 1 ? 1 : A.Hkv, head0 = fold == 1 ? 0 : kh;
#pragma unroll 1
        for (int bx = 0; bx < big; ++bx) {
          const int next = of_lane(page, bx + 1);
          if (fold) {
            tma_load_5d(to, map, 0, 0, col0, pl >> 3, pg * heads + head0, full);
          } else {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
              if (ch < chunks) tma_load_4d(to + ch * L.col, map, ch * 64, pl, kh, pg, full);
          }
          pg = next;
          pl += L.box;
          if (pl == A.page_size) pl = 0;
          to += L.box / 8 * L.row8;
        }
        map = values ? &L.v8 : &L.k8;
#pragma unroll 1
        for (int bx = 0; bx < small; ++bx, to += L.row8) {
          const int pg8 = of_lane(page, big + bx), pl8 = of_lane(place, big + bx);
#pragma unroll
          for (int ch = 0; ch < CH; ++ch)
            if (ch < chunks) tma_load_4d(to + ch * L.col, map, ch * 64, pl8, kh, pg8, full);
        }
        map = values ? &L.v_new : &L.k_new;
        to = dst + same_in_warp(at) / 8 * L.row8;
        const int row_at = same_in_warp(w.s.r0 + j0);
#pragma unroll 1
        for (int bx = 0; bx < rows_new; ++bx, to += L.row8) {
#pragma unroll
          for (int ch = 0; ch < CH; ++ch)
            if (ch < chunks) tma_load_3d(to + ch * L.col, map, ch * 64, kh, row_at + bx * 8, full);
        }
        if (!values && i == (MT == 1 && n > 1 ? 1 : 0)) {  // q behind the first keys, which do not wait for the last segment
          const int first_row = same_in_warp(w.s.r0) + mg * tok_unit;  // of the pass
          const int tiles_m = min(MT, (same_in_warp(w.s.rows) - mg * tok_unit + L.tok - 1) / L.tok);
          if (seg > 0) ok = mbar_wait_bounded(bar_q_free, (seg - 1) & 1u, kAttendWaitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          mbar_expect(bar_q, (uint32_t)(tiles_m * chunks * L.q_rows * L.group * 128));
          for (int m = 0; m < tiles_m; ++m)
            for (int ch = 0; ch < chunks; ++ch)
              tma_load_3d(q0 + (m * CH + ch) * Sh::kQChunk, &L.q, ch * 64, kh * L.group, first_row + m * L.tok, bar_q);
        }
      }
      base += 2 * n;
    }
    raise(L.status, bad);
    if (!ok) {
      if (lane == 0) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        // the copies in flight, of either warp: what the ring's last uses are filled with
        for (int i = 0; any && i < R && (uint32_t)i <= step; ++i)
          mbar_wait_bounded(bar_full + 8 * ((step - i) % R), ((step - i) / R) & 1u, 10000000ull);
        if (!values) mbar_wait_bounded(bar_q, seg & 1u, 10000000ull);
      }
      __syncwarp();
    }
  } else if (wid == Sh::kProductWarp) {
    // ---- products ----
    constexpr uint64_t desc_q = smem_desc_base(16, 1024);
    const uint64_t desc_k = smem_desc_base(16, (uint32_t)L.row8), desc_v = smem_desc_base((uint32_t)L.col, (uint32_t)L.row8);
    const uint32_t idesc_s = mma_idesc_128(kBf16, NK, false);
    const uint32_t idesc_o = mma_idesc_128(kBf16, (A.D + 15) & ~15, true);
    const int ksteps = (A.D + 15) / 16;
    // per result: products with the values issued, known to be done; segments
    uint32_t slot = 0, phase = 0, seg = 0, fixes[2] = {0, 0}, tiles = 0, cnt[2] = {0, 0}, done[2] = {0, 0}, segs[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_short(bar, parity & 1u, kAttendWaitNs));
      return ok;
    };
    // All products of result g with the values are done, none of them skipped: the buffer of
    // scores that held their weights may be written (only products into one accumulator
    // keep their order by themselves).
    auto settle = [&](int g) {
      while (done[g] != cnt[g]) {
        if (!wait(bar_o + 8 * g, done[g])) return false;
        ++done[g];
      }
      return true;
    };
    // The ring's entries are taken in their order.
    auto next_entry = [&]() { return wait(bar_full + 8 * slot, phase); };
    auto pass = [&]() {
      if (++slot == R) slot = 0, phase ^= 1;
    };
    // scores of a tile against row tile m, into buffer sb
    auto scores = [&](uint32_t at, int m, int sb) {
      const uint32_t k0 = ring0 + at * Sh::kTile, qm = q0 + m * CH * Sh::kQChunk, d = tmem + sb * NK;
      // Descriptors are made anew for each product, and the count of products is a condition on each: stepped along,
      // with a loop of its own for fewer products, 33 rows took 171 us instead of 157.
#pragma unroll
      for (int j = 0; j < DP / 16; ++j)
        if (j < ksteps)
          mma_smem(d, smem_desc(desc_q, qm + j / 4 * Sh::kQChunk + j % 4 * 32),
                   smem_desc(desc_k, k0 + j / 4 * L.col + j % 4 * 32), idesc_s, j > 0 ? 1u : 0u);
      mma_commit(bar_s + 8 * sb);
    };
    auto weigh = [&](uint32_t at, int g, int sb, int keys, bool more) {
      const uint32_t v0 = ring0 + at * Sh::kTile, d = tmem + Sh::kOut + g * DP, p = tmem + sb * NK;
#pragma unroll
      for (int j = 0; j < NK / 16; ++j)
        if (j * 16 < keys) mma_tmem(d, p + j * 8, smem_desc(desc_v, v0 + j * 2 * L.row8), idesc_o, more || j > 0 ? 1u : 0u);
      mma_commit(bar_o + 8 * g);
    };
    for (; ok && __any_sync(0xffffffffu, w.next(A)); ++seg) {
      const int t0 = same_in_warp(w.t0), n = same_in_warp(w.t1) - t0, mg = same_in_warp(w.unit) / A.Hkv;
      const int full_tiles = same_in_warp(w.s.full);
      const int tiles_m = MT == 1 ? 1 : min(MT, (same_in_warp(w.s.rows) - mg * tok_unit + L.tok - 1) / L.tok);
      if (!next_entry() || !wait(bar_q, seg)) break;
      for (int g = 0; ok && g < GROUPS; ++g) settle(g);
      if (!ok) break;
      tc_fence_after();
      // tiles counts those before this segment: buffers take turns where one group has two
      for (int m = 0; m < tiles_m; ++m) scores(slot, m, MT == 2 ? m : kTurns ? 0 : tiles & 1);
      mma_commit(bar_empty + 8 * slot);
      pass();
      if (n == 1) mma_commit(bar_q_free);
      auto keys_of = [&](int t) {
        if (t < full_tiles) return NK;
        int cached, at, j0, fresh;
        w.s.tail(t, cached, at, j0, fresh);
        return same_in_warp(fresh > 0 ? at + fresh : cached);
      };
      if constexpr (MT == 2) {
        for (int i = 0; ok && i < n; ++i) {
          const int t = t0 + i;
          if (t >= full_tiles && !wait(bar_fix, fixes[0]++)) break;
          if (!next_entry()) break;
          const uint32_t this_v = slot;
          pass();
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= tiles_m || !wait(bar_p + 8 * m, cnt[m])) break;
            if (i == 0 && segs[m] > 0 && !wait(bar_o_free + 8 * m, segs[m] - 1)) break;
            // one row tile: the second group may still be at its last segment, whose word in
            // not_finite is the next segment's
            if (i == 0 && tiles_m == 1 && segs[1] > 0 && !wait(bar_o_free + 8, segs[1] - 1)) break;
            tc_fence_after();
            weigh(this_v, m, m, keys_of(t), i > 0);
            ++cnt[m];
            if (i + 1 < n) {
              if ((m == 0 && !next_entry()) || !settle(m)) break;
              tc_fence_after();
              scores(slot, m, m);
            }
          }
          if (!ok) break;
          mma_commit(bar_empty + 8 * this_v);
          if (i + 1 < n) {
            mma_commit(bar_empty + 8 * slot);
            pass();
            if (i + 2 == n) mma_commit(bar_q_free);
          }
        }
      } else {
        for (int i = 0; ok && i < n; ++i, ++tiles) {
          const int t = t0 + i, g = kTurns ? i & 1 : 0, sb = kTurns ? g : tiles & 1;
          if (!settle(kTurns ? g ^ 1 : 0)) break;
          if (i + 1 < n) {
            if (!next_entry()) break;
            tc_fence_after();
            scores(slot, 0, sb ^ 1);
            mma_commit(bar_empty + 8 * slot);
            pass();
            if (i + 2 == n) mma_commit(bar_q_free);
          }
          if (t >= full_tiles) {  // one group: two barriers in turn
            if (!wait(bar_fix + 8 * (kTurns ? g : fixes[0] & 1), kTurns ? fixes[g] : fixes[0] >> 1)) break;
            ++fixes[g];
          }
          if (!next_entry() || !wait(bar_p + 8 * sb, kTurns ? cnt[g] : tiles >> 1)) break;
          if (i == 0 && segs[0] > 0 && !wait(bar_o_free, segs[0] - 1)) break;
          tc_fence_after();
          weigh(slot, g, sb, keys_of(t), kTurns ? i > 1 : i > 0);
          ++cnt[g];
          mma_commit(bar_empty + 8 * slot);
          pass();
        }
      }
      for (int m = 0; m < tiles_m; ++m) ++segs[m];
    }
    if (!ok) {
      if (lane == 0) raise(L.status, SPEC_DEV_TIMEOUT);
      mma_commit(bar_drain);
      mbar_wait_bounded(bar_drain, 0, 10000000ull);
    }
    __syncwarp();
  } else if (wid < 4 * GROUPS) {
    // ---- softmax: a thread per row ----
    const int g = wid >> 2, m = MT == 2 ? g : 0;
    const int quad = wid & 3;  // the tensor-memory lanes that this warp may use
    const int r = quad * 32 + lane, tid_g = tid - g * 128;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t out_at = tmem + Sh::kOut + lanes;  // result 0
    uint32_t base = 0, cnt = 0, seg = 0, fixes = 0;
    bool ok = true, left_open = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait_short(bar, parity & 1u, kAttendWaitNs));
      return ok;
    };
    const int tok = r / L.group, head = r - tok * L.group;
    for (; w.next(A); ++seg) {
      const int n = w.t1 - w.t0, kh = w.unit % A.Hkv, mg = w.unit / A.Hkv;
      const int row0 = mg * tok_unit + m * L.tok;           // of the request, first of this tile
      const int rows = min(L.tok, w.s.rows - row0);          // of the pass in this tile
      if (rows <= 0) {
        base += 2 * n;
        continue;
      }
      const bool live = tok < rows;
      const bool warp_live = quad * 32 < rows * L.group;
      const int i_row = row0 + tok;
      float top = -INFINITY, total_w = 0.0f, exact_w = 0.0f;  // m; sums of the rounded weights and of the weights
      for (int i = kTurns ? g : 0; i < n; i += kTurns ? 2 : 1, ++cnt) {
        const bool opening = kTurns ? i < 2 : i == 0;
        const int t = w.t0 + i, sb = GROUPS == 1 ? cnt & 1 : g;
        const bool last = t >= w.s.full;
        int cached = 0, at = 0, j0 = 0, fresh = 0, keys = NK;
        uint32_t sees[NK / 32];
        if (last) {
          w.s.tail(t, cached, at, j0, fresh);
          keys = fresh > 0 ? at + fresh : cached;
#pragma unroll
          for (int u = 0; u < NK / 32; ++u) {
            const int k = cached - 32 * u;
            sees[u] = k >= 32 ? ~0u : k > 0 ? (1u << k) - 1 : 0u;
          }
          if (live) {
            const uint8_t* see = A.mask ? A.mask + ((long long)w.b * A.T + i_row) * A.T + j0 : nullptr;
#pragma unroll
            for (int u = 0; u < NK / 32; ++u)
              for (int k = max(at, 32 * u); k < min(at + fresh, 32 * u + 32); ++k)
                if (see ? see[k - at] != 0 : j0 + k - at <= i_row) sees[u] |= 1u << (k - 32 * u);
          }
        }
        if (!wait(bar_s + 8 * sb, GROUPS == 1 ? cnt >> 1 : cnt)) break;
        tc_fence_after();
        float fix = 1.0f;  // of the result so far
        if (warp_live) {
          const uint32_t score_at = tmem + sb * NK + lanes;
          // 64 columns at a time, in two passes and in loops that are not unrolled: the
          // registers hold no more, and a longer body waits for its instructions.
          uint32_t v[2][32];
          auto fetch = [&](int h) {
            tmem_start32(score_at + 64 * h, v[0]);
            tmem_start32(score_at + 64 * h + 32, v[1]);
            tmem_wait32(v[0]);
            tmem_wait32(v[1]);
            if (last | (L.flip != 1.0f)) {
              const uint32_t s0 = last ? h == 0 ? sees[0] : sees[NK / 32 - 2] : ~0u;
              const uint32_t s1 = last ? h == 0 ? sees[1] : sees[NK / 32 - 1] : ~0u;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                v[0][j] = (s0 >> j) & 1u ? __float_as_uint(__uint_as_float(v[0][j]) * L.flip) : 0xFF800000u;
                v[1][j] = (s1 >> j) & 1u ? __float_as_uint(__uint_as_float(v[1][j]) * L.flip) : 0xFF800000u;
              }
            }
          };
          const int halves = keys > 64 ? 2 : 1;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {
            fetch(h);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 32; j += 8)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  mx[c] = fmaxf(mx[c], fmaxf(__uint_as_float(v[u][j + c]), __uint_as_float(v[u][j + c + 4])));
          }
          // a larger maximum: the sums so far shrink, unless by less than 2^kLag
          const float grown = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          const bool grow = live && grown > top && !((grown - top) * L.c <= AttendRange<E>::kLag);
          if (grow) {
            fix = top == -INFINITY ? 0.0f : ex2((top - grown) * L.c);
            top = grown;
            total_w *= fix;
            exact_w *= fix;
          }
          const float off = top == -INFINITY ? 0.0f : top;
          const f32x2 c2 = f2(L.c, L.c), off2 = f2(-off, -off);
          f32x2 s0 = 0, s1 = 0, e0 = 0, e1 = 0;
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {  // a half's weights take the place of scores that are read
            fetch(h);
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const int u = j / 32;
              float a, b;
              const f32x2 d = f2_add(f2(__uint_as_float(v[u][j % 32]), __uint_as_float(v[u][j % 32 + 1])), off2);
              f2_split(kBf16 ? f2_mul(d, c2) : f2_fma(d, c2, f2(AttendRange<E>::kUp, AttendRange<E>::kUp)), a, b);
              a = ex2(a);
              b = ex2(b);
              const uint32_t pair = El::pack(a, b);
              p[j / 2] = pair;
              float ra, rb;  // as the product takes them
              if constexpr (kBf16) {
                ra = __uint_as_float(pair << 16);
                rb = __uint_as_float(pair & 0xFFFF0000u);
              } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pair));
                ra = f.x;
                rb = f.y;
              }
              if (j & 2) {
                s1 = f2_add(s1, f2(ra, rb));
                e1 = f2_add(e1, f2(a, b));
              } else {
                s0 = f2_add(s0, f2(ra, rb));
                e0 = f2_add(e0, f2(a, b));
              }
            }
            tmem_store32(score_at + 32 * h, p);
          }
          total_w += f2_hsum(f2_add(s0, s1));
          exact_w += f2_hsum(f2_add(e0, e1));
        }
        if (!opening) {
          // Two groups: the scores of this tile came behind the last product into the result.
          // One group: every product is waited for, the last one before this tile's here (a
          // wait that skips one could take it for the one two before).
          if (GROUPS == 1 && !wait(bar_o, cnt - 1)) break;
          if (__any_sync(0xffffffffu, fix != 1.0f)) {
            tc_fence_after();
            for (int d = 0; d < A.D; d += 32) {
              uint32_t o[32];
              tmem_start32(out_at + g * DP + d, o);
              tmem_wait32(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fix);
              tmem_store32(out_at + g * DP + d, o);
            }
          }
        }
        tmem_wait_stores();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 8 * sb);
        if (last && (MT == 1 || m == 0)) {
          // Values that no row may take in: the gaps become zeros; what is not finite among the
          // pass's values becomes zero here and is added to the rows that see it at the end.
          const uint32_t vs = base + place_v(i, n);
          if (!wait(bar_full + 8 * (vs % R), vs / R)) break;
          const uint32_t v0 = ring0 + vs % R * Sh::kTile;
          const int upto_k = (keys + 15) & ~15, gap = (fresh > 0 ? at : upto_k) - cached;
          const int zero_rows = gap + (fresh > 0 ? upto_k - keys : 0), per = 8 * chunks;
          for (int x = tid_g; x < zero_rows * per; x += 128) {
            const int z = x / per, y = x - z * per, row = z < gap ? cached + z : keys + z - gap;
            const uint32_t to = v0 + (y >> 3) * L.col + (row >> 3) * L.row8 + (row & 7) * 128 + (y & 7) * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
          }
          bool met = false;
          for (int x = tid_g; x < fresh * per; x += 128) {
            const int z = x / per, y = x - z * per, row = at + z;
            const uint32_t from = v0 + (y >> 3) * L.col + (row >> 3) * L.row8 + (row & 7) * 128 + (y & 7) * 16;
            uint32_t e[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(e[0]), "=r"(e[1]), "=r"(e[2]), "=r"(e[3])
                         : "r"(from)
                         : "memory");
            bool any = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (not_finite16<E>(e[q])) e[q] &= 0xFFFF0000u, any = true;
              if (not_finite16<E>(e[q] >> 16)) e[q] &= 0x0000FFFFu, any = true;
            }
            if (any) {
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(from), "r"(e[0]), "r"(e[1]), "r"(e[2]),
                           "r"(e[3])
                           : "memory");
              met = true;
            }
          }
          if (met) *(volatile int*)&not_finite[seg & 1] = (int)seg + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_fix + 8 * (GROUPS == 1 ? fixes & 1 : kTurns ? g : 0));
          ++fixes;
        }
      }
      if (!ok) break;
      // ---- the segment's result ----
      const bool mine_too = !kTurns || g == 0 || n > 1;  // this group had a tile
      if (mine_too && !wait(bar_o + 8 * g, cnt - 1)) break;
      float f0 = 1.0f, f1 = 0.0f;  // factors of the two groups' results
      if constexpr (kTurns) {
        row_stat[seg & 1][g][r] = make_float4(top, total_w, exact_w, 0.0f);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_join);
        if (!wait(bar_join, seg)) break;
        const float4 other = row_stat[seg & 1][g ^ 1][r];
        const float both = fmaxf(top, other.x), off = both == -INFINITY ? 0.0f : both;
        const float f = ex2((top - off) * L.c), fo = ex2((other.x - off) * L.c);
        total_w = total_w * f + other.y * fo;
        exact_w = exact_w * f + other.z * fo;
        top = both;
        f0 = g == 0 ? f : fo;
        f1 = g == 0 ? fo : f;
      }
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.s.tiles, opens = w.t0 == 0;
      const float inv = whole ? (total_w == 0.0f ? 0.0f : 1.0f / total_w) : 1.0f;
      f0 *= inv;
      f1 *= inv;
      const bool none = whole && total_w == 0.0f;  // only scores of -inf: zeros, also where they met values of inf
      const bool odd = w.t1 > w.s.full && *(volatile int*)&not_finite[seg & 1] == (int)seg + 1;
      const long long row = w.s.r0 + i_row, out_row = row * A.Hq + kh * L.group + head;
      const size_t slot = ((size_t)cta * 2 + (opens ? 1 : 0)) * L.slot_rows + m * 128 + r;
      if (warp_live) {
        for (int d = kTurns ? 32 * g : 0; d < A.D; d += kTurns ? 64 : 32) {  // the groups share the columns
          uint32_t o[32];
          tmem_start32(out_at + (MT == 2 ? g * DP : 0) + d, o);
          tmem_wait32(o);
          float x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(o[j]) * f0;
          if (kTurns && n > 1) {
            tmem_start32(out_at + DP + d, o);
            tmem_wait32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = fmaf(__uint_as_float(o[j]), f1, x[j]);
          }
          if (live) {
            if (odd) {
              int j_from, cached, at, j0, fresh;
              w.s.tail(max(w.t0, w.s.full), cached, at, j_from, fresh);
              w.s.tail(w.t1 - 1, cached, at, j0, fresh);
              const int j_to = j0 + max(fresh, 0);
              for (int j = j_from; j < j_to; ++j) {
                const bool seen = A.mask ? A.mask[((long long)w.b * A.T + i_row) * A.T + j] != 0 : j <= i_row;
                if (!seen) continue;
                const E* val = (const E*)A.v_new + (w.s.r0 + j) * A.v_new_stride[0] + kh * A.v_new_stride[1] + d;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  if (d + e >= A.D) break;
                  const float f = El::to_f32(val[e]);
                  if (!(fabsf(f) < INFINITY)) x[e] += f;
                }
              }
            }
            if (whole) {
              if (none)
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = 0.0f;
              E* to = (E*)A.out + out_row * A.D + d;
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                if (d + j < A.D)
                  *(uint4*)(to + j) = make_uint4(El::pack(x[j], x[j + 1]), El::pack(x[j + 2], x[j + 3]),
                                                 El::pack(x[j + 4], x[j + 5]), El::pack(x[j + 6], x[j + 7]));
            } else {
              float* to = L.part + slot * DP + d;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (d + j < A.D) *(float4*)(to + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
          }
          __syncwarp();  // the loads are the whole warp's
        }
        if (live && (!kTurns || g == 0)) {
          if (!whole)
            L.stat[slot] = make_float4(top, total_w, exact_w, 0.0f);
          else if (A.lse)
            A.lse[out_row] = 0.69314718055994531f * fmaf(top, L.c, __log2f(exact_w) - AttendRange<E>::kUp);
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o_free + 8 * (MT == 2 ? g : 0));
      if (opens && !whole && g == 0 && tid_g == 0) {
        L.split[cta] = {w.unit, (int)((w.unit_end * ctas - 1) / total), w.s.r0, w.s.rows};
        left_open = true;
      }
      base += 2 * n;
    }
    if (!ok) raise(L.status, SPEC_DEV_TIMEOUT);
    if (g == 0 && tid_g == 0 && !left_open) L.split[cta] = {0, -1, 0, 0};
  }
  tc_fence_before();
  __syncthreads();
  let_next_start();
  if (wid == Sh::kProductWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Joins the partial results of the unit that CTA blockIdx.x left open: a warp
// per row, the CTAs' parts in their order.
template <class E, int DP, int MT>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendLaunch L) {
  using El = Elem<E>;
  const spec_attention_t& A = L.a;
  follow_previous();
  const AttendSplit split = L.split[blockIdx.x];
  if (split.last < 0) return;
  const int lane = threadIdx.x & 31, x = blockIdx.y * 8 + (threadIdx.x >> 5), per = L.tok * L.group;
  const int m = x / per, r = x - m * per, tok = r / L.group, head = r - tok * L.group;
  if (m >= MT) return;
  const int kh = split.unit % A.Hkv, i_row = split.unit / A.Hkv * L.tok * MT + m * L.tok + tok;
  if (i_row >= split.rows) return;
  const int first = blockIdx.x, n = split.last - first + 1;
  const size_t at = m * 128 + r;
  auto slot = [&](int i) { return ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * L.slot_rows + at; };
  constexpr int PER = DP / 32, kAhead = 4;
  // The first parts are asked for with the maxima: most units have no more.
  float first_parts[kAhead][PER];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) first_parts[i][j] = i < n ? L.part[slot(i) * DP + lane * PER + j] : 0.0f;
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, L.stat[slot(i)].x);
  top = redux_max_f32(top);
  const float off = top == -INFINITY ? 0.0f : top;
  float acc[PER] = {}, sum = 0.0f, exact = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float wt = 0.0f, z = 0.0f, e = 0.0f;
    if (i0 + lane < n) {
      const float4 st = L.stat[slot(i0 + lane)];
      wt = ex2((st.x - off) * L.c);
      z = st.y * wt;
      e = st.z * wt;
    }
    sum += warp_sum(z);
    exact += warp_sum(e);
    int from = 0;
    if (i0 == 0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wt, i);
        if (i < n) {
#pragma unroll
          for (int j = 0; j < PER; ++j) acc[j] = fmaf(first_parts[i][j], wi, acc[j]);
        }
      }
      from = kAhead;
    }
    const int cnt = min(32, n - i0);
#pragma unroll 4
    for (int i = from; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
      const float* part = L.part + slot(i0 + i) * DP + lane * PER;
#pragma unroll
      for (int j = 0; j < PER; ++j) acc[j] = fmaf(part[j], wi, acc[j]);
    }
  }
  const float inv = 1.0f / sum;
  const long long out_row = (long long)(split.r0 + i_row) * A.Hq + kh * L.group + head;
  E* to = (E*)A.out + out_row * A.D + lane * PER;
#pragma unroll
  for (int j = 0; j < PER; j += 2)
    if (lane * PER + j < A.D) *(uint32_t*)(to + j) = sum == 0.0f ? 0u : El::pack(acc[j] * inv, acc[j + 1] * inv);
  if (A.lse && lane == 0) A.lse[out_row] = 0.69314718055994531f * fmaf(off, L.c, __log2f(exact) - AttendRange<E>::kUp);
}

}  // namespace ssv
