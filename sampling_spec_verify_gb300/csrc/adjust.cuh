// Sampling rules on the logits of a pass: penalties for repeated tokens, biases
// and grammar masks.
//
//   z = z > 0 ? z / r : z r         v seen: in the prompt, generated, or drafted on the row's path
//   z -= f c(v) + p                 c(v) > 0, occurrences that were generated or drafted
//   z += biases of v ;  z = -inf    v not allowed
//
// A CTA owns a slice of the vocabulary for one request.  The slices of the request's
// rows pass through a ring of shared-memory stages, in and out by bulk copies.
// While the first ones come in, the slice's occurrences are counted (32-bit
// counters, exact in any order), turned into what they add to a logit, and the
// touched tokens listed; then each row's listed tokens are computed in its stage, a
// lane per token, and a grammar's bits applied to whole vectors.  Bound: memory, the
// logits in and out, as long as there is little to compute (128 x 8 x 129280 in bf16 without
// rules 90 us, 5.9 TB/s); with a grammar, 4000 tokens of history and 300 biases 152 us, by the
// barriers between lanes per token and vectors (0.43 of the issue slots).  The form that passes
// logits through registers and computes touched ones in between took 157 us there and 78 us
// for 16 trees of 17 x 50257 (69 so), where the touched tokens lie close together.
#pragma once

#include <type_traits>

#include "loss_common.cuh"
#include "tc05.cuh"

namespace ssv {

constexpr int kAdjustThreads = 512;  // at most
// Threads of a CTA; a word of a row's grammar each.
inline int adjust_threads(int slice) { return slice > 8192 ? 512 : 256; }
constexpr int kAdjustMaxRows = 1024, kAdjustMaxBiases = 1024;
constexpr int kAdjustStages = 3, kAdjustNear = 64;
constexpr uint64_t kAdjustWaitNs = 2000000000ull;
// Tokens a CTA: 16 KB of logits, or twice that.  (Half of it, and twice the threads for
// as much, took 3% longer for 128 x 8 x 129280.)
__host__ __device__ constexpr int adjust_slice(int elem) { return 16384 / elem; }

struct AdjustParams {
  spec_adjust_t a;
  uint32_t* status;
  int slice;  // tokens a CTA, a multiple of 64
};

// A token's word: bit 31 the prompt holds it, bits 20..30 the length of the bias list
// less its first place there, bit 19 a row of the pass holds it, bits 0..18 its occurrences in
// the generated history.
constexpr uint32_t kSeenPrompt = 1u << 31, kDrafted = 1u << 19, kCountMask = kDrafted - 1;
constexpr int kBiasShift = 20;
constexpr int kAdjustMaxHistory = (int)kCountMask;

// Stages first, on 16-byte boundaries; a stage holds a slice and what its first vector is off one.
__host__ __device__ inline size_t adjust_stage(int slice, int elem) { return (size_t)slice * elem + 16; }
inline size_t adjust_smem(int slice, int elem, int biases, int rows) {
  return kAdjustStages * adjust_stage(slice, elem) + (size_t)slice * 6 + (size_t)slice / 8 * 5 + 8 + (size_t)biases * 9 +
         (size_t)rows * 4 + 64;
}

// Elements of a 16-byte vector to -inf where `no` has their bit.
template <class E>
__device__ __forceinline__ void drop_elements(uint4& w, uint32_t no) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      if ((no >> i) & 1u) x[i] = Elem<E>::kLow;
    } else {
      const uint32_t m = (((no >> (2 * i)) & 3u) * 0x8001u & 0x10001u) * 0xFFFFu;  // two bits to two halves
      x[i] = (x[i] & ~m) | (Elem<E>::kLow & m);
    }
  }
}

template <class E>
__global__ void __launch_bounds__(kAdjustThreads, 2) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using El = Elem<E>;
  constexpr int PV = El::PV;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[kAdjustStages];
  __shared__ int in_warp[kAdjustThreads / 32];
  __shared__ unsigned long long sees[kAdjustNear];  // rows that a row sees, where they are few
  const spec_adjust_t& A = P.a;
  const int S = P.slice, tid = threadIdx.x, threads = blockDim.x;  // 256, or 512 for a long slice
  const size_t stage = adjust_stage(S, sizeof(E));
  uint32_t* counts = reinterpret_cast<uint32_t*>(raw + kAdjustStages * stage);  // [S]
  uint32_t* touched = counts + S;                 // [S / 32] tokens with a bias, then all whose logits change
  uint32_t* seen = touched + S / 32;              // [S / 32] tokens of the history
  uint32_t* by_row = seen + S / 32;               // [S / 32] tokens whose count goes by the row
  uint32_t* grammar[2] = {by_row + S / 32, by_row + S / 16 + 1};  // [S / 32 + 1] a row's bits, two rows in turn
  float* bias = reinterpret_cast<float*>(by_row + 3 * (S / 32) + 2);            // [biases]
  int32_t* bias_id = reinterpret_cast<int32_t*>(bias + A.biases);
  int32_t* drafted = bias_id + A.biases;          // [T] a row's token in the slice, or -1
  uint16_t* list = reinterpret_cast<uint16_t*>(drafted + A.T);  // [S] the slice's touched tokens
  uint8_t* again = reinterpret_cast<uint8_t*>(list + S);        // [biases] later places have the token too
  const int b = blockIdx.y, v0 = blockIdx.x * S, v1 = min(v0 + S, A.V), n = v1 - v0;

  int r0 = b * A.T, r1 = r0 + A.T;
  if (A.row_offsets) {
    r0 = A.row_offsets[b], r1 = A.row_offsets[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > A.rows || r1 - r0 > A.T) {
      if (tid == 0) raise(P.status, SPEC_DEV_BAD_OFFSETS);
      return;
    }
  }
  const int rows = r1 - r0;
  if (rows == 0) return;

  // A row of the slice: elements before the first 16-byte boundary, whole vectors, the
  // rest.  What is not in vectors (all of it where input and output lie differently)
  // never enters a stage.
  struct Row {
    const E* in;
    E* out;
    int lead, vecs, pad;  // elements, vectors; the stage's bytes before the slice's first element
  };
  auto row_at = [&](int i) {
    Row r;
    const long long at = (long long)(r0 + i) * A.V + v0;
    r.in = static_cast<const E*>(A.logits) + at;
    r.out = static_cast<E*>(A.out) + at;
    const uintptr_t x = reinterpret_cast<uintptr_t>(r.in), y = reinterpret_cast<uintptr_t>(r.out);
    r.lead = ((x ^ y) & 15) ? n : min(n, (int)(((16 - (x & 15)) & 15) / sizeof(E)));
    r.vecs = (n - r.lead) / PV;
    r.pad = r.vecs > 0 && r.lead > 0 ? 16 - r.lead * (int)sizeof(E) : 0;
    return r;
  };
  const uint32_t stages0 = smem_addr(raw), bar0 = smem_addr(bars);
  const uint64_t policy = l2_evict_first_policy();
  auto load = [&](int i) {  // one thread
    const Row r = row_at(i);
    const uint32_t bar = bar0 + 8 * (i % kAdjustStages), bytes = (uint32_t)r.vecs * 16;
    mbar_arrive_expect_tx(bar, bytes);
    if (bytes)
      bulk_load(stages0 + (uint32_t)(i % kAdjustStages * stage) + r.pad + r.lead * (uint32_t)sizeof(E), r.in + r.lead,
                bytes, bar, policy);
  };
  if (tid == 0) {
    for (int s = 0; s < kAdjustStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    for (int i = 0; i < min(rows, kAdjustStages); ++i) load(i);
  }
  // All that the counting reads first is asked for at once, and used after the zeroing.
  const float* given = A.biases ? A.bias + (long long)b * A.biases : nullptr;
  const int32_t* given_ids = A.biases ? A.bias_ids + (long long)b * A.biases : nullptr;
  const int first_id = tid < A.biases ? __ldg(given_ids + tid) : -1;
  const float first_bias = tid < A.biases ? __ldg(given + tid) : 0.0f;
  const int first_token = tid < rows ? __ldg(A.tokens + r0 + tid) : -1;
  const int32_t* h = A.history + (long long)b * A.history_width;
  constexpr int kBatch = 8;
  int t[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) t[u] = tid + u * threads < A.history_width ? __ldg(h + tid + u * threads) : 0;
  int len = A.history_lens[b], prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
  const float rep = A.repetition ? A.repetition[b] : 1.0f;
  const float freq = A.frequency ? A.frequency[b] : 0.0f;
  const float pres = A.presence ? A.presence[b] : 0.0f;
  for (int i = tid; i < S + 3 * (S / 32); i += threads) counts[i] = 0;  // touched, seen and by_row too
  for (int i = tid; i < A.biases; i += threads) again[i] = 0;
  __syncthreads();

  uint32_t bad = 0;
  auto mark = [&](uint32_t* in, int v) {  // most occurrences are of tokens that occurred before
    const uint32_t bit = 1u << (v & 31);
    if (!(in[v >> 5] & bit)) atomicOr(&in[v >> 5], bit);
  };
  if (A.biases > 0) {
    // A token's first place in the list keeps its bias; those of later places are added
    // to it in the list's order.
    for (int i = tid; i < A.biases; i += threads) {
      const int t = i == tid ? first_id : given_ids[i];
      bias_id[i] = t;
      bias[i] = i == tid ? first_bias : given[i];
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
      if (t >= v0 && t < v1) {
        atomicMax(&counts[t - v0], (uint32_t)(A.biases - i) << kBiasShift);  // the first place is the largest
        mark(touched, t - v0);
      }
    }
    __syncthreads();
    auto first_of = [&](int t) { return A.biases - (int)(counts[t - v0] >> kBiasShift); };
    for (int i = tid; i < A.biases; i += threads) {
      const int t = bias_id[i];
      if (t >= v0 && t < v1 && first_of(t) != i) again[first_of(t)] = 1;
    }
    __syncthreads();
    for (int i = tid; i < A.biases; i += threads)
      if (again[i]) {
        float sum = bias[i];
        for (int j = i + 1; j < A.biases; ++j)
          if (bias_id[j] == bias_id[i]) sum += given[j];
        bias[i] = sum;
      }
  }
  {
    if (len < 0 || len > A.history_width) bad |= SPEC_DEV_BAD_OFFSETS;
    len = min(max(len, 0), A.history_width);
    if (prompt < 0 || prompt > len) bad |= SPEC_DEV_BAD_OFFSETS;
    for (int i0 = tid; i0 < len; i0 += kBatch * threads) {
      if (i0 != tid) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) t[u] = i0 + u * threads < len ? __ldg(h + i0 + u * threads) : 0;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * threads;
        if (i >= len) break;
        if (t[u] < 0 || t[u] >= A.V) {
          bad |= SPEC_DEV_BAD_TOKEN;
        } else if (t[u] >= v0 && t[u] < v1) {
          if (i < prompt)
            atomicOr(&counts[t[u] - v0], kSeenPrompt);
          else
            atomicAdd(&counts[t[u] - v0], 1u);
          mark(seen, t[u] - v0);
        }
      }
    }
    for (int j = tid; j < rows; j += threads) {
      const int t = j == tid ? first_token : A.tokens[r0 + j];
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
      const bool here = t >= v0 && t < v1;
      drafted[j] = here ? t - v0 : -1;
      if (here) {
        atomicOr(&counts[t - v0], kDrafted);
        mark(by_row, t - v0);
      }
    }
  }
  if (blockIdx.x == 0) raise(P.status, bad);  // every slice sees the same
  __syncthreads();

  // The touched tokens in their order, a word of the bitmap a thread.
  int n_list = 0;
  {
    const uint32_t word = tid < S / 32 ? touched[tid] | seen[tid] | by_row[tid] : 0u;
    if (tid < S / 32) touched[tid] = word;
    const int lane = tid & 31, wid = tid >> 5;
    int upto = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) in_warp[wid] = upto;
    __syncthreads();
    for (int k = 0; k < threads / 32; ++k) {
      if (k == wid) upto += n_list;
      n_list += in_warp[k];
    }
    int q = upto - __popc(word);
    for (uint32_t bits = word; bits; bits &= bits - 1) list[q++] = (uint16_t)(tid * 32 + __ffs(bits) - 1);
  }
  // Few rows: which of them a row sees as bits, and a drafted token with the rows that have it.
  const bool near = rows <= kAdjustNear;
  int own = -1;
  uint32_t own_word = 0;
  unsigned long long own_rows = 0;
  if (near && tid < rows) {
    unsigned long long see = (2ull << tid) - 1;
    if (A.mask) {
      const uint8_t* m = A.mask + ((long long)b * A.T + tid) * A.T;
      see = 0;
      for (int j = 0; j < rows; ++j) see |= (unsigned long long)(m[j] != 0) << j;
    }
    sees[tid] = see;
    own = drafted[tid];
    if (own >= 0) {
      for (int j = 0; j < rows; ++j) own_rows |= (unsigned long long)(drafted[j] == own) << j;
      if (own_rows & ((1ull << tid) - 1)) own = -1;  // an earlier row has the token too: its thread's
    }
    if (own >= 0) own_word = counts[own];
  }
  __syncthreads();
  auto in = [](const uint32_t* bits, int v) { return ((bits[v >> 5] >> (v & 31)) & 1u) != 0; };
  // The rule in two steps, each rounded as written, so that a token gives the same bits
  // whether or not another row drafted it: what a word and c occurrences add to a logit,
  // and the logit with the penalty and that.
  auto added = [&](uint32_t w, uint32_t c) {
    const int at = (int)((w & ~kSeenPrompt) >> kBiasShift);
    const float add = at ? bias[A.biases - at] : 0.0f;
    return c ? __fadd_rn(__fmaf_rn(-freq, (float)c, -pres), add) : add;
  };
  auto applied = [&](bool penalty, float add, float x) {
    // selected, not branched to: 16 trees of 17 x 50257 took 77 us with branches, 71 so
    const float q = __fdiv_rn(x, rep), y = x > 0.0f ? q : __fmul_rn(x, rep);
    return __fadd_rn(penalty ? y : x, add);
  };
  // Counts that are the same for all rows become what they add.
  for (int q = tid; q < n_list; q += threads) {
    const int v = list[q];
    if (in(by_row, v)) continue;
    const uint32_t w = counts[v];
    counts[v] = __float_as_uint(added(w, w & kCountMask));
  }
  __syncthreads();
  auto counted = [&](uint32_t w, uint32_t c, float x) {  // the whole rule, of c occurrences
    return applied(c || (w & kSeenPrompt), added(w, c), x);
  };
  auto rule = [&](int i, int v, float x) {  // row i, token v of the slice that goes by the row
    const uint32_t w = counts[v];
    uint32_t c = w & kCountMask;
    const uint8_t* see = A.mask ? A.mask + ((long long)b * A.T + i) * A.T : nullptr;
    const int upto = see ? rows : i + 1;
    for (int j = 0; j < upto; ++j)
      if (drafted[j] == v && (!see || see[j])) ++c;
    return counted(w, c, x);
  };
  auto computed = [&](int i, int v, float x) {
    return in(by_row, v) ? rule(i, v, x) : applied(in(seen, v), __uint_as_float(counts[v]), x);
  };

  // A row's bits of the slice are read while the row before it is at work, a word a thread.
  const int words = (A.V + 31) / 32, mine = min(S / 32, words - (v0 >> 5));
  uint32_t bits = 0;
  auto read_bits = [&](int i) {
    const uint32_t* from = A.allowed + (long long)(r0 + i) * words + (v0 >> 5);
    if (tid < mine) bits = __ldg(from + tid);
  };
  auto keep_bits = [&](int i) {
    if (tid < mine) grammar[i & 1][tid] = bits;
  };
  if (A.allowed) {
    read_bits(0);
    keep_bits(0);
    __syncthreads();
  }
  // A thread's first listed tokens stay in registers over the rows: token, what it adds.
  constexpr int kHold = 4;
  int held_at[kHold];  // -1: none, -2: goes by the row
  float held[kHold];
  uint32_t held_seen = 0;  // a bit each
#pragma unroll
  for (int u = 0; u < kHold; ++u) {
    const int q = tid + u * threads, v = q < n_list ? list[q] : -1;
    held_at[u] = v >= 0 && in(by_row, v) ? -2 : v;
    held[u] = v >= 0 ? __uint_as_float(counts[v]) : 0.0f;
    held_seen |= v >= 0 && in(seen, v) ? 1u << u : 0u;
  }
  auto read_edge = [&](int i) {
    const Row r = row_at(i);
    return tid < n - r.vecs * PV ? r.in[tid < r.lead ? tid : tid + r.vecs * PV] : El::neg_inf();
  };
  E edge = read_edge(0);
  bool ok = true;
  for (int i = 0; i < rows; ++i) {
    const Row r = row_at(i);
    const uint32_t* allow = A.allowed ? grammar[i & 1] : nullptr;  // by token of the slice
    if (allow && i + 1 < rows) read_bits(i + 1);
    // elements outside of the vectors, a thread's first one read a row ahead
    const int edges = n - r.vecs * PV;
    const E first = edge;
    if (i + 1 < rows) edge = read_edge(i + 1);
    for (int q = tid; q < edges; q += threads) {
      const int v = q < r.lead ? q : q + r.vecs * PV;
      const E was = q == tid ? first : r.in[v];
      const bool keep = !allow || ((allow[v >> 5] >> (v & 31)) & 1u);
      r.out[v] = !keep ? El::neg_inf() : in(touched, v) ? El::from_f32(computed(i, v, El::to_f32(was))) : was;
    }
    if (!r.vecs) {
      ok = ok && mbar_wait_short(bar0 + 8 * (i % kAdjustStages), (uint32_t)(i / kAdjustStages) & 1u, kAdjustWaitNs);
    } else {
      unsigned char* here = raw + i % kAdjustStages * stage;
      E* x = reinterpret_cast<E*>(here + r.pad);  // by token of the slice
      const int from = r.lead, to = r.lead + r.vecs * PV;
      ok = mbar_wait_short(bar0 + 8 * (i % kAdjustStages), (uint32_t)(i / kAdjustStages) & 1u, kAdjustWaitNs);
      if (ok) {
#pragma unroll
        for (int u = 0; u < kHold; ++u) {
          const int v = held_at[u];
          if (v >= from && v < to) x[v] = El::from_f32(applied((held_seen >> u) & 1u, held[u], El::to_f32(x[v])));
        }
        if (own >= from && own < to)
          x[own] = El::from_f32(counted(own_word, (own_word & kCountMask) + __popcll(sees[i] & own_rows), El::to_f32(x[own])));
        bool slow = false;
#pragma unroll
        for (int u = 0; u < kHold; ++u) slow |= held_at[u] < -1;
        if (slow && !near) {
#pragma unroll 1
          for (int q = tid; q < min(n_list, kHold * threads); q += threads) {
            const int v = list[q];
            if (in(by_row, v) && v >= from && v < to) x[v] = El::from_f32(rule(i, v, El::to_f32(x[v])));
          }
        }
#pragma unroll 1
        for (int q = tid + kHold * threads; q < n_list; q += threads) {
          const int v = list[q];
          if (v >= from && v < to && !(near && in(by_row, v))) x[v] = El::from_f32(computed(i, v, El::to_f32(x[v])));
        }
      }
      if (allow) {
        __syncthreads();
        uint4* vec = reinterpret_cast<uint4*>(x + from);
        if (from == 0) {  // the vectors' bits lie in one byte each
          const uint8_t* bytes = reinterpret_cast<const uint8_t*>(allow);
#pragma unroll 4
          for (int k = tid; k < r.vecs; k += threads) {
            const uint32_t keep = (uint32_t)bytes[k * PV >> 3] >> (k * PV & 7);
            uint4 w = vec[k];
            drop_elements<E>(w, ~keep);
            vec[k] = w;
          }
        } else {
#pragma unroll 4
          for (int k = tid; k < r.vecs; k += threads) {
            const int at = from + k * PV;
            const uint32_t keep = __funnelshift_r(allow[at >> 5], allow[(at >> 5) + 1], at & 31);
            uint4 w = vec[k];
            drop_elements<E>(w, ~keep);
            vec[k] = w;
          }
        }
      }
      fence_proxy_async_smem();
    }
    if (allow && i + 1 < rows) keep_bits(i + 1);
    ok = block_waited(ok);
    if (!ok) break;
    if (tid == 0) {
      if (r.vecs) {
        bulk_store(r.out + r.lead, stages0 + (uint32_t)(i % kAdjustStages * stage) + r.pad + r.lead * (uint32_t)sizeof(E),
                   (uint32_t)r.vecs * 16);
      }
      bulk_commit();
      // the stage of the row before is free once its store has read it
      const int next = i - 1 + kAdjustStages;
      if (i > 0 && next < rows) {
        bulk_wait_read<1>();
        load(next);
      }
    }
  }
  if (tid == 0) {
    if (!ok) {
      raise(P.status, SPEC_DEV_TIMEOUT);
      for (int i = 0; i < kAdjustStages; ++i)  // copies in flight, either phase of a stage
        for (uint32_t p = 0; p < 2; ++p) mbar_wait_bounded(bar0 + 8 * i, p, 10000000ull);
    }
    bulk_wait_all();
  }
}

}  // namespace ssv
