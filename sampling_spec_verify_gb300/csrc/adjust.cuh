// Sampling rules on the logits of a pass: penalties for repeated tokens, biases
// and grammar masks.
//
//   z = z > 0 ? z / r : z r         v seen: in the prompt, generated, or drafted on the row's path
//   z -= f c(v) + p                 c(v) > 0, occurrences that were generated or drafted
//   z += biases of v ;  z = -inf    v not allowed
//
// A CTA owns a slice of the vocabulary for one request: the slice's
// occurrences are counted once in shared memory (32-bit counters, exact in any
// order), then all the request's rows stream through it.  A row's own drafted
// tokens are compared only where a touched token is one of them, so that nothing
// has to be counted between the rows.  Bound: memory, the logits in and out; the
// counters are looked at only where a bitmap of touched tokens says so.
#pragma once

#include "loss_common.cuh"

namespace ssv {

constexpr int kAdjustThreads = 256;
constexpr int kAdjustMaxRows = 1024, kAdjustMaxBiases = 1024;
constexpr int kAdjustMaxSlice = 32768;

struct AdjustParams {
  spec_adjust_t a;
  uint32_t* status;
  int slice;  // tokens a CTA, a multiple of 64
};

// A token's word: bit 31 the prompt holds it, bits 20..30 the length of the bias list
// less its first place there, bit 19 a row of the pass holds it, bits 0..18 its occurrences in
// the generated history.
constexpr uint32_t kSeenPrompt = 1u << 31, kDrafted = 1u << 19, kCountMask = kDrafted - 1;
constexpr uint32_t kRare = 0x7FF80000u;  // a bias, or a row of the pass
constexpr int kBiasShift = 20;
constexpr int kAdjustMaxHistory = (int)kCountMask;

inline size_t adjust_smem(int slice, int biases, int rows) {
  return (size_t)slice * 4 + (size_t)slice / 8 + 8 + (size_t)biases * 9 + (size_t)rows * 4;
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
__global__ void __launch_bounds__(kAdjustThreads, 5) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using El = Elem<E>;
  constexpr int PV = El::PV, kVecs = 2;  // vectors a thread has in flight
  extern __shared__ uint32_t sh[];
  const spec_adjust_t& A = P.a;
  const int S = P.slice, tid = threadIdx.x;
  uint32_t* counts = sh;                          // [S]
  uint32_t* touched = counts + S;                 // [S / 32 + 2]
  float* bias = reinterpret_cast<float*>(touched + S / 32 + 2);  // [biases]
  int32_t* bias_id = reinterpret_cast<int32_t*>(bias + A.biases);
  int32_t* drafted = bias_id + A.biases;          // [T] a row's token in the slice, or -1
  uint8_t* again = reinterpret_cast<uint8_t*>(drafted + A.T);  // [biases] later places have the token too
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
  {
    uint4* zero = reinterpret_cast<uint4*>(sh);  // the slice is a multiple of 64 tokens
    for (int i = tid; i < S / 4; i += kAdjustThreads) zero[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < S / 32 + 2; i += kAdjustThreads) touched[i] = 0;
    for (int i = tid; i < A.biases; i += kAdjustThreads) again[i] = 0;
  }
  __syncthreads();

  uint32_t bad = 0;
  auto mark = [&](int v) { atomicOr(&touched[v >> 5], 1u << (v & 31)); };
  if (A.biases > 0) {
    // A token's first place in the list keeps its bias; those of later places are added
    // to it in the list's order.
    const float* given = A.bias + (long long)b * A.biases;
    for (int i = tid; i < A.biases; i += kAdjustThreads) {
      const int t = A.bias_ids[(long long)b * A.biases + i];
      bias_id[i] = t;
      bias[i] = given[i];
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
      if (t >= v0 && t < v1) {
        atomicMax(&counts[t - v0], (uint32_t)(A.biases - i) << kBiasShift);  // the first place is the largest
        mark(t - v0);
      }
    }
    __syncthreads();
    auto first_of = [&](int t) { return A.biases - (int)(counts[t - v0] >> kBiasShift); };
    for (int i = tid; i < A.biases; i += kAdjustThreads) {
      const int t = bias_id[i];
      if (t >= v0 && t < v1 && first_of(t) != i) again[first_of(t)] = 1;
    }
    __syncthreads();
    for (int i = tid; i < A.biases; i += kAdjustThreads)
      if (again[i]) {
        float sum = bias[i];
        for (int j = i + 1; j < A.biases; ++j)
          if (bias_id[j] == bias_id[i]) sum += given[j];
        bias[i] = sum;
      }
  }
  {
    int len = A.history_lens[b], prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
    if (len < 0 || len > A.history_width) bad |= SPEC_DEV_BAD_OFFSETS;
    len = min(max(len, 0), A.history_width);
    if (prompt < 0 || prompt > len) bad |= SPEC_DEV_BAD_OFFSETS;
    const int32_t* h = A.history + (long long)b * A.history_width;
    for (int i0 = tid; i0 < len; i0 += 8 * kAdjustThreads) {
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kAdjustThreads;
        t[u] = i < len ? __ldg(h + i) : v0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kAdjustThreads;
        if (i >= len) break;
        if (t[u] < 0 || t[u] >= A.V) {
          bad |= SPEC_DEV_BAD_TOKEN;
        } else if (t[u] >= v0 && t[u] < v1) {
          if (i < prompt)
            atomicOr(&counts[t[u] - v0], kSeenPrompt);
          else
            atomicAdd(&counts[t[u] - v0], 1u);
          mark(t[u] - v0);
        }
      }
    }
    for (int j = tid; j < rows; j += kAdjustThreads) {
      const int t = A.tokens[r0 + j];
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
      const bool here = t >= v0 && t < v1;
      drafted[j] = here ? t - v0 : -1;
      if (here) {
        atomicOr(&counts[t - v0], kDrafted);
        mark(t - v0);
      }
    }
  }
  if (blockIdx.x == 0) raise(P.status, bad);  // every slice sees the same
  __syncthreads();

  const float rep = A.repetition ? A.repetition[b] : 1.0f;
  const float inv_rep = 1.0f / rep;  // one rounding more than a division, and no code for it
  const float freq = A.frequency ? A.frequency[b] : 0.0f;
  const float pres = A.presence ? A.presence[b] : 0.0f;
  auto rule = [&](int i, int v, float x) {  // row i, token v of the slice
    const uint32_t w = counts[v];
    uint32_t c = w & kCountMask;
    if (w & kDrafted) {
      const uint8_t* see = A.mask ? A.mask + ((long long)b * A.T + i) * A.T : nullptr;
      const int upto = see ? rows : i + 1;
      for (int j = 0; j < upto; ++j)
        if (drafted[j] == v && (!see || see[j])) ++c;
    }
    if (c || (w & kSeenPrompt)) x = x > 0.0f ? x * inv_rep : x * rep;
    if (c) x = x - freq * (float)c - pres;
    const int at = (int)((w & ~kSeenPrompt) >> kBiasShift);
    if (at) x += bias[A.biases - at];
    return x;
  };

  const int words = (A.V + 31) / 32;
  const E* in_all = static_cast<const E*>(A.logits);
  E* out_all = static_cast<E*>(A.out);
  for (int i = 0; i < rows; ++i) {
    const long long row = (long long)(r0 + i) * A.V + v0;
    const E *in = in_all + row;
    E* out = out_all + row;
    const uint32_t* allow = A.allowed ? A.allowed + (long long)(r0 + i) * words : nullptr;
    // elements before the first 16-byte boundary, whole vectors, the rest
    const int lead = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / sizeof(E)));
    const int vecs = (n - lead) / PV;
    const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    auto one = [&](int v) {
      const bool ok = !allow || ((allow[(v0 + v) >> 5] >> ((v0 + v) & 31)) & 1u);
      const E raw = in[v];
      const bool hit = (touched[v >> 5] >> (v & 31)) & 1u;
      out[v] = !ok ? El::neg_inf() : hit ? El::from_f32(rule(i, v, El::to_f32(raw))) : raw;
    };
    if (!same) {
      for (int v = tid; v < n; v += kAdjustThreads) one(v);
      continue;
    }
    for (int v = tid; v < lead; v += kAdjustThreads) one(v);
    for (int v = lead + vecs * PV + tid; v < n; v += kAdjustThreads) one(v);
    const uint4* src = reinterpret_cast<const uint4*>(in + lead);
    uint4* dst = reinterpret_cast<uint4*>(out + lead);
    // The whole rule's code is there once a vector, in a loop over the elements that need
    // it: unrolled over them it waited for its instructions (128 x 8 x 129280: 426 us).
    // Dense places (a language's frequent tokens) take the short rule side by side.
    for (int k0 = tid; k0 < vecs; k0 += kVecs * kAdjustThreads) {
      uint4 w[kVecs];
      uint32_t ok[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int k = k0 + u * kAdjustThreads;
        ok[u] = ~0u;
        if (k < vecs) {
          w[u] = __ldcs(src + k);
          if (allow) {
            const int g = v0 + lead + k * PV, s = g & 31;
            uint32_t x = __ldg(allow + (g >> 5)) >> s;
            if (s > 32 - PV) x |= __ldg(allow + (g >> 5) + 1) << (32 - s);
            ok[u] = x;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int k = k0 + u * kAdjustThreads;
        if (k >= vecs) break;
        const int v = lead + k * PV, s = v & 31;
        uint32_t hit = __funnelshift_r(touched[v >> 5], touched[(v >> 5) + 1], s) & ((1u << PV) - 1) & ok[u];
        const uint4 raw = w[u];
        if (__popc(hit) > 2) {  // tokens that were merely counted, all elements at once
          E e[PV];
          *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            const uint32_t word = (hit >> j) & 1u ? counts[v + j] : kRare;
            const float x0 = El::to_f32(e[j]);
            float x = x0 > 0.0f ? x0 * inv_rep : x0 * rep;
            if (word & kCountMask) x = x - freq * (float)(word & kCountMask) - pres;
            if (!(word & kRare)) {
              hit &= ~(1u << j);
              e[j] = El::from_f32(x);
            }
          }
          w[u] = *reinterpret_cast<uint4*>(e);
        }
        if (allow) drop_elements<E>(w[u], ~ok[u]);
        __stcs(dst + k, w[u]);
        while (hit) {  // the others, one by one behind the vector
          const int j = __ffs(hit) - 1;
          hit &= hit - 1;
          float x;
          if constexpr (PV == 4) {
            x = __uint_as_float(j & 2 ? (j & 1 ? raw.w : raw.z) : (j & 1 ? raw.y : raw.x));
          } else {
            const uint32_t pair = j & 4 ? (j & 2 ? raw.w : raw.z) : (j & 2 ? raw.y : raw.x);
            x = __uint_as_float(j & 1 ? pair & 0xFFFF0000u : pair << 16);
          }
          out[v + j] = El::from_f32(rule(i, v + j, x));
        }
      }
    }
  }
}

}  // namespace ssv
