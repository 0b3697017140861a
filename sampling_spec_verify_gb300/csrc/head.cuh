// The vocabulary head's losses without its logits: matrix products on the
// tensor cores with the softmax in their epilogues.
//
//   z = X W^T / T                 X [N, H] hidden states, W [V, H] head
//   pass 1   per 256-token tile and row: maximum and sum of 2^z', z' = z log2(e)
//   pass 2   per piece of the vocabulary, C tokens wide:
//     D  = (softmax(z) - t) w     16 bits, [N, C]
//     dX += D W_piece             fp32, one partial per split of the piece
//     dW_piece = D^T X
//
// The piece lies in a workspace of bounded size.  Where the whole vocabulary is
// one piece, pass 1 leaves its unnormalised probabilities there and D is a
// rescaling of them (4 bytes of traffic an entry); otherwise D is recomputed
// from X and W piece by piece, a fourth product.
//
// D is rounded to the operands' 16-bit type because the products that consume
// it take that type: one rounding of half a step per entry, the size of the
// rounding of a 16-bit result.  Row weights are divided by the largest one and,
// for fp16, D is scaled by 2^15, so that probabilities down to 2^-29 keep
// their precision in fp16's short exponent.
//
// One kernel does all four products.  Bound: tensor cores (2 N V H operations
// a product).  A CTA pair owns a 256 x 256 tile: each CTA stages 128 rows of A
// and 128 of B per 64-deep step (32 KB, six stages), one thread of the even
// CTA issues tcgen05.mma for both, accumulators take half of tensor memory so
// that the epilogue of a tile overlaps the products of the next.  Measured at
// 1792 x 151936 x 2048, bf16: pass 1 574 us (1.94 PFLOP/s on a cold GPU, 1.65 under
// its power limit), both backward products 1140 us; at 60 rows, where the head's
// bytes count, pass 1 5.7 TB/s, dX 6.3 TB/s, dW 4.1 TB/s (a plain fill: 4.0).
#pragma once

#include "loss_common.cuh"
#include "tc05.cuh"

namespace ssv {

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * 128 * kTileK * 2;  // A and B halves of a CTA
constexpr int kEpiWarps = 4;
constexpr int kHeadThreads = 64 + 32 * kEpiWarps;
constexpr int kStageOut = 4096;  // per epilogue warp and buffer: 32 rows x 128 bytes
constexpr int kHeadSmem = kStages * kStageBytes + kEpiWarps * 2 * kStageOut + 1024;
constexpr uint64_t kWaitNs = 2000000000ull;

enum HeadOp {
  kHeadNorm,  // pass 1: row statistics of X W^T per tile
  kHeadKeep,  // pass 1, keeping the unnormalised probabilities
  kHeadGrad,  // D of a piece, recomputed
  kHeadBack   // dX partials (product 0) and dW (product 1) of a piece
};

// One product of a launch.  Rows of A and B run along K, or (mn) along the
// other dimension.
struct Product {
  int M, N, K;  // rows, columns, depth
  int splits;
  int b_off;    // the piece's start among the rows of B
};

struct HeadLaunch {
  CUtensorMap a[2], b[2], out[2];
  Product p[2];
  int which;          // bit 0: product 0, bit 1: product 1
  const uint32_t* count;  // rows that count; null: all of them
  const int32_t* perm;    // [rows] the batch's row at each place; null: the same
  int bf16;
  float s;            // log2(e) / T
  // kHeadNorm, kHeadKeep
  float2* part;       // [tiles_n, M]
  float* zi;          // [rows, k] logits of the listed tokens, by row and slot
  const int32_t* labels;   // cross entropy
  const uint32_t* keys;    // else: the listed tokens, sorted (see TargetParams)
  const uint16_t* starts;
  int k;
  // kHeadGrad
  const float* lse2;  // [M] log2 of the normaliser
  const float* weight;
  const uint8_t* keep;
  float store_scale;
  // kHeadBack
  int first;          // store (not add) the partials
  int slot_rows;      // rows between the partials of two splits
  const LossScalars* scalars;
  uint32_t* status;
};

// The launch's tiles.  Only rows that count take part in the backward products
// (and in a recomputed D): the batch's rows lie in such an order that they come
// first, and their number is read from device memory.
struct Tiles {
  int m[2], n[2], ksteps[2];
  int first, all;  // tiles of product 0, of the launch
};
template <HeadOp OP>
__device__ __forceinline__ Tiles tiles_of(const HeadLaunch& L) {
  const int rows = L.count ? max((int)*L.count, 1) : 0x7FFFFFFF;
  Tiles t;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int M = i == 0 ? min(L.p[i].M, rows) : L.p[i].M, K = i == 1 ? min(L.p[i].K, rows) : L.p[i].K;
    t.m[i] = (M + kTileM - 1) / kTileM;
    t.n[i] = (L.p[i].N + kTileN - 1) / kTileN;
    t.ksteps[i] = (K + kTileK - 1) / kTileK;
  }
  t.first = (L.which & 1) ? t.m[0] * t.n[0] * L.p[0].splits : 0;
  t.all = t.first + (OP == kHeadBack && (L.which & 2) ? t.m[1] * t.n[1] * L.p[1].splits : 0);
  return t;
}

// Tile `i` of the launch: bands of eight tile rows, down the rows first, so
// that the tiles in flight share operands in L2.
struct TileAt {
  int second;  // which product
  int m, n, split, k0, k1;
};
template <HeadOp OP>
__device__ __forceinline__ TileAt tile_at(const HeadLaunch& L, const Tiles& T, int i) {
  TileAt t;
  t.second = OP == kHeadBack && i >= T.first;
  if (t.second) i -= T.first;
  const int tiles_m = t.second ? T.m[1] : T.m[0], tiles_n = t.second ? T.n[1] : T.n[0];
  const int ksteps = t.second ? T.ksteps[1] : T.ksteps[0], splits = L.p[t.second].splits;
  const int per = tiles_m * tiles_n;
  t.split = i / per;
  i -= t.split * per;
  constexpr int kBand = 8;
  const int band = i / (kBand * tiles_n);
  const int rows = min(kBand, tiles_m - band * kBand);
  i -= band * kBand * tiles_n;
  t.m = band * kBand + i % rows;
  t.n = i / rows;
  t.k0 = (int)((long long)ksteps * t.split / splits);
  t.k1 = (int)((long long)ksteps * (t.split + 1) / splits);
  return t;
}

// Writes 16 bytes of a row into a 128-byte-swizzled staging tile.
__device__ __forceinline__ void stage_write(uint32_t base, int row, int unit, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + row * 128 + ((unit ^ (row & 7)) << 4)), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16) {
  return bf16 ? Elem<__nv_bfloat16>::pack(a, b) : Elem<__half>::pack(a, b);
}

// Unnormalised probabilities are kept as 2^(z' - m + 15), m the row's maximum in
// the tile: for bf16 operands in fp16, whose 11 bits (down to 2^-29 of the
// largest) leave rounding D to bf16 the one rounding that counts; for fp16
// operands in fp32.  (Calls that keep none use the same exponents, for the same
// bits.)
constexpr float kKeepShift = 15.0f;

// OUT32: kHeadKeep keeps fp32; dW of kHeadBack is fp32.
template <HeadOp OP, bool OUT32>
__global__ void __launch_bounds__(kHeadThreads, 1) __cluster_dims__(2, 1, 1)
    head_kernel(const __grid_constant__ HeadLaunch L) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_slot;

  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t tiles0 = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t out0 = tiles0 + kStages * kStageBytes;
  const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * kStages;
  const uint32_t bar_done = bar_empty + 8 * kStages;  // accumulators written, two
  const uint32_t bar_free = bar_done + 16;            // accumulators read, two
  const uint32_t bar_drain = bar_free + 16;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_done + 8 * i, 1);
      mbar_init(bar_free + 8 * i, 2 * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    fence_mbar_init();
    prefetch_map(&L.a[0]);
    prefetch_map(&L.b[0]);
  }
  let_next_start();
  if (wid == 0) {
    tmem_alloc_pair(smem_addr(&tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  follow_previous();
  const uint32_t tmem = tmem_slot;
  const int clusters = gridDim.x / 2, first_tile = blockIdx.x / 2;
  const Tiles T = tiles_of<OP>(L);

  if (wid == 0) {
    // ---- loads: one thread of each CTA ----
    if (lane == 0) {
      const uint32_t full0 = map_rank(bar_full, 0);
      uint32_t step = 0;
      bool ok = true;
      for (int i = first_tile; ok && i < T.all; i += clusters) {
        const TileAt t = tile_at<OP>(L, T, i);
        const CUtensorMap *map_a = &L.a[t.second], *map_b = &L.b[t.second];
        const int b_off = L.p[t.second].b_off;
        const bool a_mn = t.second, b_mn = OP == kHeadBack;
        const int row_a = t.m * kTileM + (int)rank * 128, row_b = t.n * kTileN + (int)rank * 128;
        for (int k = t.k0; k < t.k1; ++k, ++step) {
          const uint32_t s = step % kStages, use = step / kStages;
          if (use > 0 && !mbar_wait_bounded(bar_empty + 8 * s, (use - 1) & 1u, kWaitNs)) {
            ok = false;
            break;
          }
          const uint32_t a = tiles0 + s * kStageBytes, b = a + kStageBytes / 2;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * s, 2 * kStageBytes);
          const uint32_t full = full0 + 8 * s;
          if (a_mn) {
            tma_load_pair(a, map_a, row_a, k * kTileK, full);
            tma_load_pair(a + 8192, map_a, row_a + 64, k * kTileK, full);
          } else {
            tma_load_pair(a, map_a, k * kTileK, row_a, full);
          }
          if (b_mn) {
            tma_load_pair(b, map_b, row_b, b_off + k * kTileK, full);
            tma_load_pair(b + 8192, map_b, row_b + 64, b_off + k * kTileK, full);
          } else {
            tma_load_pair(b, map_b, k * kTileK, b_off + row_b, full);
          }
        }
      }
      if (!ok) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        // the copies in flight of the pair end on the even CTA's barriers
        if (rank == 0)
          for (int i = 0; i < kStages && step > 0; ++i, --step)
            mbar_wait_bounded(bar_full + 8 * ((step - 1) % kStages), ((step - 1) / kStages) & 1u, 10000000ull);
      }
    }
  } else if (wid == 1) {
    // ---- products: one thread of the even CTA ----
    if (rank == 0 && lane == 0) {
      constexpr uint64_t desc_k = smem_desc_base(16, 1024), desc_mn = smem_desc_base(8192, 1024);
      constexpr bool b_mn = OP == kHeadBack;
      constexpr uint64_t db = b_mn ? desc_mn : desc_k;
      constexpr uint32_t kb = b_mn ? 2048 : 32;  // bytes of 16 K steps
      uint32_t step = 0, it = 0;
      bool ok = true;
      for (int i = first_tile; ok && i < T.all; i += clusters, ++it) {
        const TileAt t = tile_at<OP>(L, T, i);
        const uint32_t idesc = mma_idesc(L.bf16 != 0, t.second, b_mn);
        const uint64_t da = t.second ? desc_mn : desc_k;
        const uint32_t ka = t.second ? 2048 : 32;
        const uint32_t acc = it & 1, use = it >> 1;
        if (use > 0 && !mbar_wait_bounded(bar_free + 8 * acc, (use - 1) & 1u, kWaitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * kTileN;
        for (int k = t.k0; k < t.k1; ++k, ++step) {
          const uint32_t s = step % kStages;
          if (!mbar_wait_bounded(bar_full + 8 * s, (step / kStages) & 1u, kWaitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = tiles0 + s * kStageBytes, b = a + kStageBytes / 2;
#pragma unroll
          for (int j = 0; j < kTileK / 16; ++j)
            mma_pair(d, smem_desc(da, a + j * ka), smem_desc(db, b + j * kb), idesc, (k > t.k0 || j > 0) ? 1u : 0u);
          mma_commit_pair(bar_empty + 8 * s);
        }
        if (ok) mma_commit_pair(bar_done + 8 * acc);
      }
      if (!ok) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        mma_commit_pair(bar_drain);
        mbar_wait_bounded(bar_drain, 0, 10000000ull);
      }
    }
  } else {
    // ---- epilogue: a thread per row of this CTA's half of the tile ----
    const int quad = wid & 3;  // the tensor-memory lanes that this warp may read
    const uint32_t stage = out0 + (wid - 2) * 2 * kStageOut;
    const uint32_t free0 = map_rank(bar_free, 0);
    uint32_t it = 0, buf = 0;
    // The next of the warp's two staging buffers, once its last store has read it.
    auto next_buffer = [&]() {
      const uint32_t dst = stage + buf * kStageOut;
      buf ^= 1;
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
      return dst;
    };
    // Sends a staged 32-row block of 128-byte rows to the result.
    auto send = [&](const CUtensorMap* map, uint32_t src, int x, int y, bool in, bool add) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (in) {
          if (add)
            tma_reduce_add(map, src, x, y);
          else
            tma_store(map, src, x, y);
        }
        bulk_commit();
      }
    };
    auto stage16 = [&](uint32_t dst, int unit, const float (&v)[32], bool bf) {
#pragma unroll
      for (int j = 0; j < 32; j += 8)
        stage_write(dst, lane, unit + j / 8, pack16(v[j], v[j + 1], bf), pack16(v[j + 2], v[j + 3], bf),
                    pack16(v[j + 4], v[j + 5], bf), pack16(v[j + 6], v[j + 7], bf));
    };
    auto stage32 = [&](uint32_t dst, const float (&v)[32]) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        stage_write(dst, lane, j / 4, __float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                    __float_as_uint(v[j + 3]));
    };

    for (int i = first_tile; i < T.all; i += clusters, ++it) {
      const TileAt t = tile_at<OP>(L, T, i);
      const uint32_t acc = it & 1, use = it >> 1;
      // pass 1: the listed tokens of this thread's row in this tile, looked up
      // while the products run
      long long n_row = 0;
      int from = 0, to = 0, col = -1;
      if constexpr (OP == kHeadNorm || OP == kHeadKeep) {
        const int r = t.m * kTileM + (int)rank * 128 + quad * 32 + lane;
        if (r < L.p[0].M) {
          n_row = L.perm ? L.perm[r] : r;
          if (L.labels) {
            col = L.labels[n_row] - t.n * kTileN;
            to = col >= 0 && col < min(kTileN, L.p[0].N - t.n * kTileN) && L.keep[n_row] ? 1 : 0;
          } else {
            const uint16_t* s = L.starts + n_row * (T.n[0] + 1) + t.n;
            from = s[0], to = s[1];
          }
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_done + 8 * acc, use & 1u, kWaitNs))) {
        raise(L.status, SPEC_DEV_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t src = tmem + acc * kTileN + ((uint32_t)(quad * 32) << 16);
      const int M = L.p[t.second].M, N = L.p[t.second].N;
      const int row0 = t.m * kTileM + (int)rank * 128 + quad * 32, row = row0 + lane;
      const int col0 = t.n * kTileN;

      if constexpr (OP == kHeadNorm || OP == kHeadKeep) {
        // the row's maximum over the tile, then the sum, in powers of two
        const int cols = N - col0;
        float m = -INFINITY, sum = 0.0f;
        for (int c = 0; c < kTileN; c += 32) {
          float v[32];
          tmem_load32(src + c, v);
          if (c + 32 <= cols) {
#pragma unroll
            for (int j = 0; j < 32; ++j) m = max_nan(m, v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) m = max_nan(m, c + j < cols ? v[j] : -INFINITY);
          }
        }
        m *= L.s;
        // A tile of nothing but -inf adds nothing: its terms are 2^(-inf - 0), and its
        // offset stays -inf, so that kept terms are rescaled by 0.
        const bool none = m == -INFINITY;
        const float off = none ? 0.0f : m - kKeepShift;
        constexpr int kCols = OP == kHeadKeep && OUT32 ? 32 : 64;
        for (int c = 0; c < kTileN; c += kCols) {
          if (c >= cols) break;
          uint32_t dst = 0;
          if constexpr (OP == kHeadKeep) dst = next_buffer();
#pragma unroll
          for (int h = 0; h < kCols; h += 32) {
            float v[32];
            tmem_load32(src + c + h, v);
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              v[j] = ex2(fmaf(v[j], L.s, -off));
              if (c + h + 32 > cols && c + h + j >= cols) v[j] = 0.0f;
              a += v[j];
            }
            sum += a;
            if constexpr (OP == kHeadKeep) {
              if constexpr (OUT32)
                stage32(dst, v);
              else
                stage16(dst, h / 8, v, false);
            }
          }
          if constexpr (OP == kHeadKeep) send(&L.out[0], dst, col0 + c, row0, row0 < M, false);
        }
        if (row < M) L.part[(long long)t.n * M + row] = make_float2(none ? -INFINITY : off, sum);
        // The listed tokens' logits are those of the same products that make the
        // normaliser: the tensor cores' sums are short of the exact ones by up to
        // 2.5e-6 of a logit, which would stand alone in the loss of a confident
        // row (0.6 +- 2e-5) but cancels between the two.
        for (uint32_t left; (left = __ballot_sync(0xffffffffu, from < to)) != 0;) {
          const int l = __ffs(left) - 1;
          uint32_t slot = 0;
          if (lane == l && !L.labels) {
            const uint32_t key = L.keys[n_row * L.k + from];
            slot = key & 255u;
            col = (int)(key >> 8) - t.n * kTileN;
          }
          const float z = tmem_load1(src + (uint32_t)__shfl_sync(0xffffffffu, col, l));
          if (lane == l) {
            L.zi[n_row * L.k + slot] = z;
            ++from;
          }
        }
      } else if constexpr (OP == kHeadGrad) {
        float lse = 0.0f, cf = 0.0f;
        const int n = row < M ? (L.perm ? L.perm[row] : row) : 0;
        if (row < M && L.keep[n]) {
          lse = L.lse2[row];
          cf = (L.weight ? L.weight[n] : 1.0f) * L.scalars->inv_wmax * L.store_scale;
        }
        for (int c = 0; c < kTileN; c += 64) {
          if (col0 + c >= N) break;
          const uint32_t dst = next_buffer();
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            float v[32];
            tmem_load32(src + c + h, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = cf != 0.0f ? ex2(fmaf(v[j], L.s, -lse)) * cf : 0.0f;
            stage16(dst, h / 8, v, L.bf16 != 0);
          }
          send(&L.out[0], dst, col0 + c, row0, row0 < M, false);
        }
      } else if (!t.second) {
        for (int c = 0; c < kTileN; c += 32) {
          if (col0 + c >= N) break;
          const uint32_t dst = next_buffer();
          float v[32];
          tmem_load32(src + c, v);
          stage32(dst, v);
          send(&L.out[0], dst, col0 + c, t.split * L.slot_rows + row0, row0 < M, !L.first);
        }
      } else {
        const float mul = L.scalars->grad_mul;
        constexpr int kCols = OUT32 ? 32 : 64;
        for (int c = 0; c < kTileN; c += kCols) {
          if (col0 + c >= N) break;
          const uint32_t dst = next_buffer();
#pragma unroll
          for (int h = 0; h < kCols; h += 32) {
            float v[32];
            tmem_load32(src + c + h, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= mul;
            if constexpr (OUT32)
              stage32(dst, v);
            else
              stage16(dst, h / 8, v, L.bf16 != 0);
          }
          send(&L.out[1], dst, col0 + c, row0, row0 < M, false);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free0 + 8 * acc);
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (wid == 0) tmem_free_pair(tmem, 512);
}

// Puts the rows that count before the others, each group in its order: perm[p] is
// the row at place p, and x is copied row by row to its place (at a pitch of
// whole lines where the batch's rows start off a sector).  A warp per row; every
// CTA counts all of `keep` (N bytes, zero-filled to whole words) for itself.
__global__ void __launch_bounds__(256) compact_kernel(const uint8_t* keep, int N, int per_cta, const uint4* x,
                                                      uint4* xp, int words, int ld_words, int32_t* perm,
                                                      LossScalars* scalars) {
  __shared__ int red[2][8];
  let_next_start();
  follow_previous();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = blockIdx.x * per_cta;  // a multiple of eight
  int all = 0, before = 0;
  const uint2* words8 = reinterpret_cast<const uint2*>(keep);
  for (int i = threadIdx.x; i < (N + 7) / 8; i += 256) {
    const uint2 v = words8[i];
    const int c = __popc(v.x) + __popc(v.y);
    all += c;
    if (i * 8 < base) before += c;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) red[0][w] = all, red[1][w] = before;
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) all += red[0][i], before += red[1][i];
  if (blockIdx.x == 0 && threadIdx.x == 0) scalars->count = (uint32_t)all;
  for (int r = 0; r < per_cta; r += 8) {
    const int n0 = base + r;
    if (n0 >= N) break;
    const uint2 v = words8[n0 / 8];
    const unsigned long long bits = (unsigned long long)v.y << 32 | v.x;
    const int n = n0 + w;
    if (n < N) {
      const bool on = (bits >> (8 * w)) & 1;
      const int ahead = before + __popcll(bits & ((1ull << (8 * w)) - 1));  // rows before this one that count
      const long long p = on ? ahead : all + (n - ahead);
      if (lane == 0) perm[p] = n;
      for (int i = lane; i < words; i += 32) xp[p * ld_words + i] = __ldcs(x + (long long)n * words + i);
    }
    before += __popcll(bits);
  }
}

// Cross entropy's preparation in one launch: whether a row counts and, where xp
// is given, what compact_kernel does.  Every CTA looks at all labels for itself
// (N <= 8192: 32 loads a thread at most).  One dependent launch less than a
// pass of its own for the flags: 6 us against 6 + 5, and a pass of 8 x 32000 x
// 1024 takes 70 instead of 71.
__global__ void __launch_bounds__(256) label_rows_kernel(const TargetParams P, int per_cta, const uint4* x, uint4* xp,
                                                         int words, int ld_words, int32_t* perm) {
  __shared__ int red[2][8];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = blockIdx.x * per_cta;
  auto counts = [&](int label) { return label >= 0 && label < P.V && label != P.ignore; };
  int all = 0, before = 0;
  if (xp) {
#pragma unroll 4
    for (int i = threadIdx.x; i < P.N; i += 256) {
      const int c = counts(P.ids[i]);
      all += c;
      before += i < base ? c : 0;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) red[0][w] = all, red[1][w] = before;
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all += red[0][i], before += red[1][i];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    P.scalars->ticket = 0;
    if (xp) P.scalars->count = (uint32_t)all;
  }
  for (int r = 0; r < per_cta && base + r < P.N; r += 8) {
    const int n0 = base + r, n = n0 + w;
    // the eight rows' flags, in every warp
    const int label = lane < 8 && n0 + lane < P.N ? P.ids[n0 + lane] : P.ignore;
    const uint32_t flags = __ballot_sync(0xffffffffu, counts(label));
    const int mine = __shfl_sync(0xffffffffu, label, w);
    if (n < P.N) {
      const bool on = (flags >> w) & 1;
      const int ahead = before + __popc(flags & ((1u << w) - 1));
      const long long p = on ? ahead : all + (n - ahead);
      if (lane == 0) {
        if (!on && mine != P.ignore) raise(P.status, SPEC_DEV_BAD_TOKEN);
        P.keep[n] = on;
        P.t[n] = on ? 1.0f : 0.0f;
        P.row[n] = RowTeacher{0.0f, 0.0f, on ? 1.0f : 0.0f, 0.0f};
        if (xp) perm[p] = n;
      }
      if (xp)
        for (int i = lane; i < words; i += 32) xp[p * ld_words + i] = __ldcs(x + (long long)n * words + i);
    }
    before += __popc(flags);
  }
  let_next_start();
}

// ---- the listed tokens -----------------------------------------------------------

// Puts the listed tokens' entries into a piece of D (tokens [v0, v0 + C)).
struct ListedParams {
  const int32_t* ids;
  const float* t;
  const float* zi;
  const float* lse2;
  const float* weight;
  const uint8_t* keep;
  const int32_t* perm;
  const LossScalars* scalars;
  int N, k, v0, C;
  long long ld;
  double s;  // log2(e) / T
  float store_scale;
};
template <class E>
__global__ void __launch_bounds__(256) listed_grads_kernel(const ListedParams P, E* d) {
  let_next_start();
  follow_previous();
  const long long j = (long long)blockIdx.x * 256 + threadIdx.x;
  if (j >= (long long)P.N * P.k) return;
  const long long p = j / P.k;
  if (p >= (long long)P.scalars->count) return;
  const long long n = P.perm[p], i = n * P.k + (j - p * P.k);
  const int id = P.ids[i];
  if (id < P.v0 || id >= P.v0 + P.C) return;
  const float cf = (P.weight ? P.weight[n] : 1.0f) * P.scalars->inv_wmax * P.store_scale;
  const float q = exp2f((float)((double)P.zi[i] * P.s - (double)P.lse2[p]));
  d[p * P.ld + (id - P.v0)] = Elem<E>::from_f32(cf == 0.0f ? 0.0f : (q - P.t[i]) * cf);
}

// Turns kept probabilities (S; fp16 ones lie where D goes) into D: one CTA per
// row and kDenseCols tokens (one read and one write, the listed tokens after).
// Bound: HBM (1613 x 151936: 167 us for 0.98 GB, 5.9 TB/s).
constexpr int kDenseCols = 8192;
template <class E, class S>
__global__ void __launch_bounds__(256) dense_grads_kernel(const ListedParams P, const float2* part, const S* kept,
                                                          E* d) {
  let_next_start();
  follow_previous();
  // place p; places up to the next 64-deep step get zeros, the rest is not read
  const long long p = blockIdx.x;
  const int count = (int)P.scalars->count;
  if (p >= max((count + kTileK - 1) / kTileK, 1) * kTileK) return;
  const bool on = p < count;
  const long long n = on ? P.perm[p] : 0;
  const int c0 = blockIdx.y * kDenseCols, c1 = min(P.C, c0 + kDenseCols);
  const float cf = on ? (P.weight ? P.weight[n] : 1.0f) * P.scalars->inv_wmax * P.store_scale : 0.0f;
  const float lse = on ? P.lse2[p] : 0.0f;
  constexpr int kWords = sizeof(S) / 2;  // 16-byte words of eight entries
  const uint4* src = reinterpret_cast<const uint4*>(kept + p * P.ld);
  uint4* dst = reinterpret_cast<uint4*>(d + p * P.ld);
  constexpr int kPer = kDenseCols / 8 / 256;
  uint4 v[kPer][kWords];
  float f[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = c0 + (i * 256 + threadIdx.x) * 8;
    if (c < c1) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) v[i][w] = __ldcs(src + c / 8 * kWords + w);
      f[i] = part[(long long)(c >> 8) * P.N + p].x;
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = c0 + (i * 256 + threadIdx.x) * 8;
    if (c < c1) {
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (cf != 0.0f) {
        const float m = ex2(f[i] - lse) * cf;
        float x[8];
        if constexpr (kWords == 1) {
          Elem<S>::unpack(v[i][0], x);
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            x[4 * w] = __uint_as_float(v[i][w].x), x[4 * w + 1] = __uint_as_float(v[i][w].y);
            x[4 * w + 2] = __uint_as_float(v[i][w].z), x[4 * w + 3] = __uint_as_float(v[i][w].w);
          }
        }
        o.x = Elem<E>::pack(x[0] * m, x[1] * m), o.y = Elem<E>::pack(x[2] * m, x[3] * m);
        o.z = Elem<E>::pack(x[4] * m, x[5] * m), o.w = Elem<E>::pack(x[6] * m, x[7] * m);
      }
      dst[c / 8] = o;
    }
  }
  __syncthreads();
  if (cf == 0.0f) return;
  for (int i = threadIdx.x; i < P.k; i += 256) {
    const int id = P.ids[n * P.k + i];
    if (id >= c0 && id < c1) {
      const float q = exp2f((float)((double)P.zi[n * P.k + i] * P.s - (double)lse));
      d[p * P.ld + id] = Elem<E>::from_f32((q - P.t[n * P.k + i]) * cf);
    }
  }
}

// ---- normalisers, row losses, their sum --------------------------------------------

// 8 rows per CTA.  The tiles' statistics of a row are joined by 32 threads (64
// contiguous bytes of every tile), each thread's loads independent of one
// another; then a warp per row.
//
// Rows are taken by place.  Where `spare` is given (the hidden states by place),
// the rows between the last one that counts and the next 64-deep step are
// zeroed: the head's gradient multiplies them by zeros, and hidden states of
// rows that are left out may hold anything.
__global__ void __launch_bounds__(256) head_finish_kernel(const FinishParams P, const float2* part, int tiles_n,
                                                          const int32_t* perm, float* lse_out, float* lse2,
                                                          uint4* spare, int ld_words) {
  __shared__ float2 sh[32][9];
  let_next_start();
  follow_previous();
  const int r8 = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long base = (long long)blockIdx.x * 8;
  // what the second half needs of row base + w, loaded beside the statistics
  const long long p = base + w;
  const bool in = p < P.N;
  const long long n = in && perm ? perm[p] : p;
  const bool on = in && P.keep[n];
  RowTeacher teacher{0.0f, 0.0f, 0.0f, 0.0f};
  float weight = 0.0f;
  if (in) {
    teacher = P.row[n];
    weight = P.weight ? P.weight[n] : 1.0f;
  }
  float m = -INFINITY, sum = 0.0f;
  if (base + r8 < P.N) {
    for (int t0 = g; t0 < tiles_n; t0 += 32 * 8) {
      float2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + 32 * j;
        v[j] = t < tiles_n ? __ldcs(part + (long long)t * P.N + base + r8) : make_float2(-INFINITY, 0.0f);
      }
      float nm = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) nm = max_nan(nm, v[j].x);
      if (nm > -INFINITY && nm < INFINITY) {
        sum *= exp2f(m - nm);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[j].y * exp2f(v[j].x - nm);
      }
      m = nm;
    }
  }
  sh[g][r8] = make_float2(m, sum);
  __syncthreads();
  float loss = 0.0f;
  if (in) {
    const float2 v = sh[lane][w];
    const float top = redux_max_nan(v.x);
    const bool fine = top > -INFINITY && top < INFINITY;
    const float z = warp_sum(fine ? v.y * exp2f(v.x - top) : 0.0f);
    // log2 Z as a pair: the maximum and a small logarithm
    const F2 l2 = fine ? two_sum(top, log2f(z)) : F2{NAN, 0.0f};
    const F2 ln2{0.693147182f, -1.90465421e-9f};
    F2 l = two_mul(l2.hi, ln2);
    l.lo = fmaf(l2.lo, ln2.hi, l.lo);
    if (lane == 0) {
      if (!fine && on) raise(P.status, SPEC_DEV_BAD_LOGITS);
      lse2[p] = l2.hi;
      if (lse_out) lse_out[n] = l.hi + l.lo;
    }
    if (on) loss = row_loss_warp(P, n, lane, RowLog{0.0f, pair_add(l, F2{-teacher.shift, -teacher.shift_lo}), 0.0f});
    if (lane == 0) P.row_loss[n] = loss;
    if (spare && !on && p < max((P.scalars->count + kTileK - 1) / kTileK, 1u) * (long long)kTileK)
      for (int i = lane; i < ld_words; i += 32) spare[p * ld_words + i] = make_uint4(0u, 0u, 0u, 0u);
  }
  finish_sums(P, loss, on, weight);
}

// grad_hidden = grad_mul * sum of the partials: Q threads for four elements, each
// every Q-th slot, joined in one order.  Q = 4 for many slots of few elements (19
// slots of 8 x 1024: 3.6 us against 6.1), 1 otherwise (4 slots of 1792 x 2048: 11
// against 20).
template <class O, int Q>
__global__ void __launch_bounds__(256) hidden_out_kernel(const float* part, int slots, long long slot_elems,
                                                         long long elems, int H, const int32_t* perm,
                                                         const LossScalars* scalars, O* out) {
  let_next_start();
  follow_previous();
  const long long i = ((long long)blockIdx.x * (256 / Q) + threadIdx.x / Q) * 4;
  const int q = threadIdx.x % Q;
  const bool in = i < elems;
  const long long p = in ? i / H : 0;
  const bool on = in && p < (long long)scalars->count;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (on) {
#pragma unroll 4
    for (int s = q; s < slots; s += Q) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(part + s * slot_elems + i));
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
#pragma unroll
  for (int o = 1; o < Q; o <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  if (!in || q != 0) return;
  const float mul = on ? scalars->grad_mul : 0.0f;
  O* dst = out + (long long)perm[p] * H + (i - p * H);
  if constexpr (sizeof(O) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(a.x * mul, a.y * mul, a.z * mul, a.w * mul);
  } else {
    uint2 v;
    v.x = Elem<O>::pack(a.x * mul, a.y * mul);
    v.y = Elem<O>::pack(a.z * mul, a.w * mul);
    *reinterpret_cast<uint2*>(dst) = v;
  }
}

}  // namespace ssv
