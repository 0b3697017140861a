// Attention of a pass's rows over a paged cache and the pass's own keys, on the
// tensor cores.
//
//   s_n = scale q . k_n,  out = sum_n 2^(c s_n - m) v_n / sum_n 2^(c s_n - m),  c = scale log2(e)
//
// over the cached tokens of the row's request and the rows of the pass that its
// mask names.  One pass over the keys: m is a running maximum, and where it
// grows by more than 2^8 the sums so far are rescaled (a smaller growth leaves
// it behind the maximum, which changes no ratio).  Scores, sums and the result
// are fp32; the weights are rounded to the operands' 16-bit type for the
// product with v.  The result is divided by the sum of the rounded weights, so
// that a row which one key dominates loses nothing; lse takes the sum before rounding.
//
// All query rows that share a key head (the pass's rows times the group's
// heads) form tiles of 128 rows, so that the cache is read once for all of
// them.  Bound: the cache's bytes, up to about 128 rows a key head; the
// exponentials beyond.
//
// The batch is cut into units (request, key head, 128 or 256 rows), a unit into
// tiles of keys, and all tiles, one unit behind the other, into equal shares, one a
// CTA and SM.  A unit that spans CTAs leaves one partial result (out, m, sum) a
// CTA; a second launch joins them.  The shares come from the lengths on the
// device: nothing of the launch depends on them, and the order of the sums
// follows from the lengths alone.
//
// A CTA: warp 0 loads (keys and values through a ring of shared-memory tiles by
// TMA, page by page; a page's part of a tile is a box of the tensor map),
// warp 1 issues the products (scores into tensor memory, weights times values
// with the weights read from tensor memory), four warps per 128 rows do the
// softmax, a thread per row.
#pragma once

#include "loss_common.cuh"
#include "tc05.cuh"

namespace ssv {

constexpr uint64_t kAttendWaitNs = 2000000000ull;
constexpr int kAttendMaxGroup = 128;

// DP: head size in shared memory.  MT: tiles of 128 rows that a CTA works on.
template <int DP, int MT>
struct AttendShape {
  static constexpr int NK = DP > 128 ? 64 : 128;      // keys a tile
  static constexpr int CH = DP / 64;                  // 128-byte columns of a row
  static constexpr int kChunk = NK * 128;             // bytes of one column of a tile
  static constexpr int kTile = CH * kChunk;           // keys or values of a tile
  static constexpr int kQChunk = 128 * 128;
  static constexpr int kQ = MT * CH * kQChunk;
  static constexpr int kRoom = 226 * 1024;
  static constexpr int kRing = (kRoom - kQ) / kTile > 12 ? 12 : (kRoom - kQ) / kTile;
  static constexpr int kSmem = kQ + kRing * kTile + 1024;
  static constexpr int kThreads = 64 + 128 * MT;
  static constexpr int kScores = 2;                   // buffers of scores: two of one row tile, or one each of two
  static constexpr int kOut = 256;                    // tensor-memory column of the results
  static_assert(kScores * NK <= kOut && kOut + MT * DP <= 512, "tensor memory");
  static_assert(kRing >= 4, "keys and values of two tiles");
};

struct AttendSplit {  // a unit that goes on in the next CTAs
  int b, unit, last;  // last: the CTA that holds its end; -1: none
};

struct AttendLaunch {
  CUtensorMap q, k_new, v_new;
  CUtensorMap k, v;    // boxes of `box` tokens of a page
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
  int slot_rows;       // query rows of a partial result
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
template <int NK>
struct AttendSpan {
  int r0, rows, full, rest, tiles;
  long long cost;  // tiles of all units
  __device__ __forceinline__ void load(const spec_attention_t& A, int b, int tok_unit) {
    const AttendRequest r = attend_request(A, b);
    r0 = r.r0, rows = r.rows;
    full = r.context / NK;
    rest = r.context % NK;
    tiles = full + (((rest + 7) & ~7) + rows + NK - 1) / NK;
    cost = rows ? (long long)tiles * A.Hkv * ((rows + tok_unit - 1) / tok_unit) : 0;
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

// The CTA's share of all tiles, unit by unit.  Every warp walks it by itself.
template <int NK>
struct AttendWalk {
  long long at, end;  // tiles of the batch
  long long off;      // of request b
  int b, tok_unit;
  AttendSpan<NK> s;
  // the segment
  int unit, t0, t1;
  long long from;     // its first tile in the batch's order
  __device__ __forceinline__ bool next(const spec_attention_t& A) {
    if (at >= end) return false;
    while (off >= s.cost) {  // below the total there is another request
      if (b + 1 >= A.B) return false;  // the lengths changed under the call
      off = 0;
      s.load(A, ++b, tok_unit);
    }
    if (s.cost <= 0x7FFFFFFF) {
      unit = (int)off / s.tiles;
      t0 = (int)off - unit * s.tiles;
    } else {
      unit = (int)(off / s.tiles);
      t0 = (int)(off - (long long)unit * s.tiles);
    }
    from = at;
    const int n = (int)min((long long)(s.tiles - t0), end - at);
    t1 = t0 + n;
    at += n;
    off += n;
    return true;
  }
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
__global__ void __launch_bounds__(64 + 128 * MT, 1) attend_kernel(const __grid_constant__ AttendLaunch L) {
  using El = Elem<E>;
  using Sh = AttendShape<DP, MT>;
  constexpr int NK = Sh::NK, CH = Sh::CH, R = Sh::kRing, kThreads = Sh::kThreads;
  constexpr bool kBf16 = El::kLow == 0xFF80FF80u;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * R + 16];
  __shared__ uint32_t tmem_slot;
  __shared__ long long warp_sum_of[kThreads / 32];
  __shared__ long long start_off;
  __shared__ int start_b;
  __shared__ int not_finite[2];  // a value of the pass that is not finite was met: 1 + number of the segment

  const spec_attention_t& A = L.a;
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const uint32_t q0 = (smem_addr(raw) + 1023u) & ~1023u, ring0 = q0 + Sh::kQ;
  const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * R;
  const uint32_t bar_q = bar_empty + 8 * R, bar_q_free = bar_q + 8;
  const uint32_t bar_s = bar_q_free + 8;      // scores written, two buffers
  const uint32_t bar_p = bar_s + 16;          // weights written, two
  const uint32_t bar_o = bar_p + 16;          // a product with the values done, per row tile
  const uint32_t bar_o_free = bar_o + 16;     // the result read, per row tile
  const uint32_t bar_fix = bar_o_free + 16;   // values of a last tile looked over, two in turn
  const uint32_t bar_drain = bar_fix + 16;
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
      mbar_init(bar_o_free + 8 * i, 4);
      mbar_init(bar_fix + 8 * i, 4);
      not_finite[i] = 0;
    }
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
  if (wid == 1) {
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
  const uint32_t tmem = tmem_slot;
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

  if (wid == 0) {
    // ---- loads ----
    uint32_t step = 0, seg = 0;
    uint32_t bad = 0;
    bool ok = true;
    for (; ok && w.next(A); ++seg) {
      const int n = w.t1 - w.t0, kh = w.unit % A.Hkv, mg = w.unit / A.Hkv;
      const int first_row = w.s.r0 + mg * tok_unit;  // of the pass
      const int tiles_m = min(MT, (w.s.rows - mg * tok_unit + L.tok - 1) / L.tok);
      const int32_t* table = A.block_table + w.b * A.table_stride;
      for (int x = 0; ok && x < 2 * n; ++x, ++step) {
        if (x == (MT == 1 && n > 1 ? 2 : 1)) {  // q behind the first keys, which do not wait for the last segment
          if (seg > 0) ok = mbar_wait_bounded(bar_q_free, (seg - 1) & 1u, kAttendWaitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, (uint32_t)(tiles_m * chunks * L.q_rows * L.group * 128));
            for (int m = 0; m < tiles_m; ++m)
              for (int ch = 0; ch < chunks; ++ch)
                tma_load_3d(q0 + (m * CH + ch) * Sh::kQChunk, &L.q, ch * 64, kh * L.group, first_row + m * L.tok, bar_q);
          }
        }
        bool values;
        int i;
        if constexpr (MT == 2) {
          values = x & 1;
          i = x >> 1;
        } else {
          values = x == 2 * n - 1 || (x > 0 && !(x & 1));
          i = x == 2 * n - 1 ? n - 1 : values ? (x - 2) >> 1 : (x + 1) >> 1;
        }
        const int t = w.t0 + i;
        const uint32_t s = step % R, use = step / R, full = bar_full + 8 * s, dst = ring0 + s * Sh::kTile;
        if (use > 0) ok = mbar_wait_bounded(bar_empty + 8 * s, (use - 1) & 1u, kAttendWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (t < w.s.full) {
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(chunks * NK * 128));
          __syncwarp();
          const CUtensorMap* map = values ? &L.v : &L.k;
          const int copies = NK / L.box * chunks;
          for (int y = lane; y < copies; y += 32) {
            const int bx = y / chunks, ch = y - bx * chunks, pos = t * NK + bx * L.box, p = pos / A.page_size;
            int page = __ldg(table + p);
            if (page < 0 || page >= A.pages) page = A.pages, bad = SPEC_DEV_BAD_PAGE;  // behind the end: zeros
            tma_load_4d(dst + ch * Sh::kChunk + bx * L.box * 128, map, ch * 64, pos - p * A.page_size, kh, page, full);
          }
        } else {
          int cached, at, j0, fresh;
          w.s.tail(t, cached, at, j0, fresh);
          const int old = (cached + 7) / 8, boxes = old + (fresh + 7) / 8;
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(chunks * boxes * 8 * 128));
          __syncwarp();
          for (int y = lane; y < boxes * chunks; y += 32) {
            const int bx = y / chunks, ch = y - bx * chunks;
            const uint32_t to = dst + ch * Sh::kChunk;
            if (bx < old) {
              const int pos = t * NK + bx * 8, p = pos / A.page_size;
              int page = __ldg(table + p);
              if (page < 0 || page >= A.pages) page = A.pages, bad = SPEC_DEV_BAD_PAGE;
              tma_load_4d(to + bx * 1024, values ? &L.v8 : &L.k8, ch * 64, pos - p * A.page_size, kh, page, full);
            } else {
              const int j = (bx - old) * 8;
              tma_load_3d(to + (at + j) * 128, values ? &L.v_new : &L.k_new, ch * 64, kh, w.s.r0 + j0 + j, full);
            }
          }
        }
      }
    }
    raise(L.status, bad);
    if (!ok) {
      if (lane == 0) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        for (int i = 0; i < R && step > 0; ++i, --step)  // the copies in flight
          mbar_wait_bounded(bar_full + 8 * ((step - 1) % R), ((step - 1) / R) & 1u, 10000000ull);
        mbar_wait_bounded(bar_q, seg & 1u, 10000000ull);
      }
      __syncwarp();
    }
  } else if (wid == 1) {
    // ---- products: one thread ----
    if (lane == 0) {
      constexpr uint64_t desc_k = smem_desc_base(16, 1024), desc_v = smem_desc_base(Sh::kChunk, 1024);
      const uint32_t idesc_s = mma_idesc_128(kBf16, NK, false);
      const uint32_t idesc_o = mma_idesc_128(kBf16, (A.D + 15) & ~15, true);
      const int ksteps = (A.D + 15) / 16;
      uint32_t base = 0, seg = 0, fixes = 0, cnt[2] = {0, 0}, done[2] = {0, 0}, segs[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = mbar_wait_bounded(bar, parity & 1u, kAttendWaitNs);
        return ok;
      };
      // All products with the values of row tile m are done, none of them skipped: the buffer
      // of scores that held their weights may be written (only products into one accumulator
      // keep their order by themselves).
      auto settle = [&](int m) {
        while (done[m] != cnt[m]) {
          if (!wait(bar_o + 8 * m, done[m])) return false;
          ++done[m];
        }
        return true;
      };
      // scores of a tile against row tile m, into buffer sb
      auto scores = [&](uint32_t at, int m, int sb) {
        const uint32_t k0 = ring0 + at % R * Sh::kTile;
        for (int j = 0; j < ksteps; ++j)
          mma_smem(tmem + sb * NK, smem_desc(desc_k, q0 + (m * CH + j / 4) * Sh::kQChunk + j % 4 * 32),
                   smem_desc(desc_k, k0 + j / 4 * Sh::kChunk + j % 4 * 32), idesc_s, j > 0 ? 1u : 0u);
        mma_commit(bar_s + 8 * sb);
      };
      auto weigh = [&](uint32_t at, int m, int sb, int keys, bool more) {
        const uint32_t v0 = ring0 + at % R * Sh::kTile;
        for (int j = 0; j * 16 < keys; ++j)
          mma_tmem(tmem + Sh::kOut + m * DP, tmem + sb * NK + j * 8, smem_desc(desc_v, v0 + j * 2048), idesc_o,
                   more || j > 0 ? 1u : 0u);
        mma_commit(bar_o + 8 * m);
      };
      for (; ok && w.next(A); ++seg) {
        const int n = w.t1 - w.t0, mg = w.unit / A.Hkv;
        const int tiles_m = MT == 1 ? 1 : min(MT, (w.s.rows - mg * tok_unit + L.tok - 1) / L.tok);
        auto full_at = [&](int place) { return wait(bar_full + 8 * ((base + place) % R), (base + place) / R); };
        if (!full_at(place_k(0, n)) || !wait(bar_q, seg)) break;
        for (int m = 0; ok && m < tiles_m; ++m) settle(m);
        if (!ok) break;
        tc_fence_after();
        for (int m = 0; m < tiles_m; ++m) scores(base, m, MT == 1 ? cnt[0] & 1 : m);
        mma_commit(bar_empty + 8 * (base % R));
        if (n == 1) mma_commit(bar_q_free);
        for (int i = 0; ok && i < n; ++i) {
          const int t = w.t0 + i;
          int keys = NK;
          if (t >= w.s.full) {
            int cached, at, j0, fresh;
            w.s.tail(t, cached, at, j0, fresh);
            keys = fresh > 0 ? at + fresh : cached;
          }
          const uint32_t next_k = base + (i + 1 < n ? place_k(i + 1, n) : 0), this_v = base + place_v(i, n);
          if (MT == 1 && !settle(0)) break;
          if (MT == 1 && i + 1 < n) {
            if (!full_at(place_k(i + 1, n))) break;
            tc_fence_after();
            scores(next_k, 0, (cnt[0] + 1) & 1);
            mma_commit(bar_empty + 8 * (next_k % R));
            if (i + 2 == n) mma_commit(bar_q_free);
          }
          if (t >= w.s.full) {
            if (!wait(bar_fix + 8 * (fixes & 1), fixes >> 1)) break;
            ++fixes;
          }
          if (!full_at(place_v(i, n))) break;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m >= tiles_m) break;
            const int sb = MT == 1 ? cnt[0] & 1 : m;
            if (!wait(bar_p + 8 * sb, MT == 1 ? cnt[0] >> 1 : cnt[m])) break;
            if (i == 0 && segs[m] > 0 && !wait(bar_o_free + 8 * m, segs[m] - 1)) break;
            tc_fence_after();
            weigh(this_v, m, sb, keys, i > 0);
            ++cnt[m];
            if (MT == 2 && i + 1 < n) {
              if ((m == 0 && !full_at(place_k(i + 1, n))) || !settle(m)) break;
              tc_fence_after();
              scores(next_k, m, m);
            }
          }
          if (!ok) break;
          mma_commit(bar_empty + 8 * (this_v % R));
          if (MT == 2 && i + 1 < n) {
            mma_commit(bar_empty + 8 * (next_k % R));
            if (i + 2 == n) mma_commit(bar_q_free);
          }
        }
        base += 2 * n;
        for (int m = 0; m < tiles_m; ++m) ++segs[m];
      }
      if (!ok) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        mma_commit(bar_drain);
        mbar_wait_bounded(bar_drain, 0, 10000000ull);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: a thread per row ----
    const int m = MT == 1 ? 0 : (wid - 2) >> 2, quad = wid & 3;  // the tensor-memory lanes that this warp may use
    const int r = quad * 32 + lane, tid_m = tid - 64 - m * 128;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t out_at = tmem + Sh::kOut + m * DP + lanes;
    uint32_t base = 0, cnt = 0, seg = 0, fixes = 0;
    bool ok = true, left_open = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, kAttendWaitNs));
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
      const bool live = tok < rows && tok < L.tok;
      const bool warp_live = quad * 32 < rows * L.group;
      const int i_row = row0 + tok;
      float top = -INFINITY, total_w = 0.0f, exact_w = 0.0f;  // m / c; sums of the rounded weights and of the weights
      for (int i = 0; i < n; ++i, ++cnt) {
        const int t = w.t0 + i, sb = MT == 1 ? cnt & 1 : m;
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
        if (!wait(bar_s + 8 * sb, MT == 1 ? cnt >> 1 : cnt)) break;
        // Every product with the values is waited for, the last one before this tile's
        // here: a wait that skips one could take it for the one two before.
        if (i > 0 && !wait(bar_o + 8 * m, cnt - 1)) break;
        tc_fence_after();
        if (warp_live) {
          const uint32_t score_at = tmem + sb * NK + lanes;
          uint32_t v[NK / 32][32];
#pragma unroll
          for (int u = 0; u < NK / 32; ++u)
            if (!last || 32 * u < keys) tmem_start32(score_at + 32 * u, v[u]);
          float mx = -INFINITY;
#pragma unroll
          for (int u = 0; u < NK / 32; ++u) {
            if (last && 32 * u >= keys) continue;
            tmem_wait32(v[u]);
            if (L.flip != 1.0f) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[u][j] = __float_as_uint(__uint_as_float(v[u][j]) * L.flip);
            }
            if (last) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((sees[u] >> j) & 1u)) v[u][j] = 0xFF800000u;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) mx = fmaxf(mx, __uint_as_float(v[u][j]));
          }
          // a larger maximum: the sums so far shrink, unless by less than 2^8
          const float grown = fmaxf(top, mx);
          const bool grow = live && grown > top && !((grown - top) * L.c <= 8.0f);
          if (__any_sync(0xffffffffu, grow)) {
            const float fix = !grow ? 1.0f : top == -INFINITY ? 0.0f : ex2((top - grown) * L.c);
            if (grow) top = grown;
            total_w *= fix;
            exact_w *= fix;
            if (i > 0) {
              for (int d = 0; d < A.D; d += 32) {
                uint32_t o[32];
                tmem_start32(out_at + d, o);
                tmem_wait32(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fix);
                tmem_store32(out_at + d, o);
              }
            }
          }
          const float off = top == -INFINITY ? 0.0f : top * L.c;
          const f32x2 c2 = f2(L.c, L.c), off2 = f2(-off, -off);
          f32x2 s0 = 0, s1 = 0, e0 = 0, e1 = 0;
#pragma unroll
          for (int u = 0; u < NK / 32; u += 2) {
            if (last && 32 * u >= keys) continue;
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const int uu = u + j / 32;
              float a = 0.0f, b = 0.0f;
              if (!last || 32 * uu < keys) {
                f2_split(f2_fma(f2(__uint_as_float(v[uu][j % 32]), __uint_as_float(v[uu][j % 32 + 1])), c2, off2), a, b);
                a = ex2(a);
                b = ex2(b);
              }
              const uint32_t h = El::pack(a, b);
              p[j / 2] = h;
              float ra, rb;  // as the product takes them
              if constexpr (kBf16) {
                ra = __uint_as_float(h << 16);
                rb = __uint_as_float(h & 0xFFFF0000u);
              } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
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
            tmem_store32(score_at + 16 * u, p);
          }
          total_w += f2_hsum(f2_add(s0, s1));
          exact_w += f2_hsum(f2_add(e0, e1));
          tmem_wait_stores();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 8 * sb);
        if (last && m == 0) {
          // Values that no row may take in: the gaps become zeros; what is not finite among the
          // pass's values becomes zero here and is added to the rows that see it at the end.
          const uint32_t vs = base + place_v(i, n);
          if (!wait(bar_full + 8 * (vs % R), vs / R)) break;
          const uint32_t v0 = ring0 + vs % R * Sh::kTile;
          const int upto_k = (keys + 15) & ~15, gap = (fresh > 0 ? at : upto_k) - cached;
          const int zero_rows = gap + (fresh > 0 ? upto_k - keys : 0), per = 8 * chunks;
          for (int x = tid_m; x < zero_rows * per; x += 128) {
            const int z = x / per, y = x - z * per, row = z < gap ? cached + z : keys + z - gap;
            const uint32_t to = v0 + (y >> 3) * Sh::kChunk + row * 128 + (y & 7) * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
          }
          bool met = false;
          for (int x = tid_m; x < fresh * per; x += 128) {
            const int z = x / per, y = x - z * per;
            const uint32_t from = v0 + (y >> 3) * Sh::kChunk + (at + z) * 128 + (y & 7) * 16;
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
          if (lane == 0) mbar_arrive(bar_fix + 8 * (fixes++ & 1));
          __syncwarp();
        }
      }
      if (!ok) break;
      // ---- the segment's result ----
      if (!wait(bar_o + 8 * m, cnt - 1)) break;
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.s.tiles, opens = w.t0 == 0;
      const float inv = whole ? (total_w == 0.0f ? 0.0f : 1.0f / total_w) : 1.0f;
      const bool odd = w.t1 > w.s.full && *(volatile int*)&not_finite[seg & 1] == (int)seg + 1;
      const long long row = w.s.r0 + i_row, out_row = row * A.Hq + kh * L.group + head;
      const size_t slot = ((size_t)cta * 2 + (opens ? 1 : 0)) * L.slot_rows + m * 128 + r;
      if (warp_live) {
        for (int d = 0; d < A.D; d += 32) {
          uint32_t o[32];
          tmem_start32(out_at + d, o);
          tmem_wait32(o);
          if (live) {
            float x[32];
  #pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(o[j]) * inv;
            if (odd) {
              int j_from, j_to, cached, at, j0, fresh;
              w.s.tail(max(w.t0, w.s.full), cached, at, j_from, fresh);
              w.s.tail(w.t1 - 1, cached, at, j0, fresh);
              j_to = j0 + max(fresh, 0);
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
        if (live) {
          const float top2 = top == -INFINITY ? -INFINITY : top * L.c;
          if (!whole)
            L.stat[slot] = make_float4(top2, total_w, exact_w, 0.0f);
          else if (A.lse)
            A.lse[out_row] = 0.69314718055994531f * (top2 + __log2f(exact_w));
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o_free + 8 * m);
      if (opens && !whole && m == 0 && tid_m == 0) {
        const long long last_tile = w.from + w.s.tiles - 1;
        L.split[cta] = {w.b, w.unit, (int)(((last_tile + 1) * ctas - 1) / total)};
        left_open = true;
      }
      base += 2 * n;
    }
    if (!ok) raise(L.status, SPEC_DEV_TIMEOUT);
    if (m == 0 && tid_m == 0 && !left_open) L.split[cta] = {0, 0, -1};
  }
  tc_fence_before();
  __syncthreads();
  let_next_start();
  if (wid == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Joins the partial results of the unit that CTA blockIdx.x left open: a warp
// per row, the CTAs' parts in their order.
template <class E, int DP, int MT>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendLaunch L) {
  using El = Elem<E>;
  constexpr int NK = AttendShape<DP, MT>::NK;
  const spec_attention_t& A = L.a;
  follow_previous();
  const AttendSplit split = L.split[blockIdx.x];
  if (split.last < 0) return;
  const int lane = threadIdx.x & 31, x = blockIdx.y * 8 + (threadIdx.x >> 5), per = L.tok * L.group;
  const int m = x / per, r = x - m * per, tok = r / L.group, head = r - tok * L.group;
  if (m >= MT) return;
  AttendSpan<NK> s;
  s.load(A, split.b, L.tok * MT);
  const int kh = split.unit % A.Hkv, i_row = split.unit / A.Hkv * L.tok * MT + m * L.tok + tok;
  if (i_row >= s.rows) return;
  const int first = blockIdx.x, n = split.last - first + 1;
  const size_t at = m * 128 + r;
  auto slot = [&](int i) { return ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * L.slot_rows + at; };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, L.stat[slot(i)].x);
  top = redux_max_f32(top);
  const float off = top == -INFINITY ? 0.0f : top;
  constexpr int PER = DP / 32;
  float acc[PER] = {}, sum = 0.0f, exact = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float wt = 0.0f, z = 0.0f, e = 0.0f;
    if (i0 + lane < n) {
      const float4 st = L.stat[slot(i0 + lane)];
      wt = ex2(st.x - off);
      z = st.y * wt;
      e = st.z * wt;
    }
    sum += warp_sum(z);
    exact += warp_sum(e);
    const int cnt = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
      const float* from = L.part + slot(i0 + i) * DP + lane * PER;
#pragma unroll
      for (int j = 0; j < PER; ++j) acc[j] = fmaf(from[j], wi, acc[j]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const long long out_row = (long long)(s.r0 + i_row) * A.Hq + kh * L.group + head;
  E* to = (E*)A.out + out_row * A.D + lane * PER;
#pragma unroll
  for (int j = 0; j < PER; j += 2)
    if (lane * PER + j < A.D) *(uint32_t*)(to + j) = El::pack(acc[j] * inv, acc[j + 1] * inv);
  if (A.lse && lane == 0) A.lse[out_row] = 0.69314718055994531f * (off + __log2f(exact));
}

}  // namespace ssv
