// Sampling rules on the logits of a pass: penalties for repeated tokens, biases
// and grammar masks.
//
//   z = z > 0 ? z / r : z r         v seen: in the prompt, generated, or drafted on the row's path
//   z -= f c(v) + p                 c(v) > 0, occurrences that were generated or drafted
//   z += biases of v ;  z = -inf    v not allowed
//
// A CTA owns a slice of the vocabulary for one request: the slice's
// occurrences are counted once in shared memory (32-bit counters, exact in any
// order), then the request's rows go by, each with its own drafted tokens
// counted in and out.  Bound: memory, the logits in and out; the counters are
// looked at only where a bitmap of touched tokens says so.
#pragma once

#include "loss_common.cuh"

namespace ssv {

constexpr int kAdjustThreads = 512;
constexpr int kAdjustMaxRows = 1024, kAdjustMaxBiases = 1024;
constexpr int kAdjustMaxSlice = 32768;

struct AdjustParams {
  spec_adjust_t a;
  uint32_t* status;
  int slice;  // tokens a CTA, a multiple of 64
};

// A token's word: bit 31 the prompt holds it, bits 20..30 one plus its first place
// in the bias list, bits 0..19 its occurrences.
constexpr uint32_t kSeenPrompt = 1u << 31, kCountMask = (1u << 20) - 1;
constexpr int kBiasShift = 20;
constexpr int kAdjustMaxHistory = 1000000;  // with kAdjustMaxRows more the count still fits

inline size_t adjust_smem(int slice, int biases, int rows) {
  return (size_t)slice * 4 + (size_t)slice / 8 + 8 + (size_t)biases * 8 + (size_t)rows * 4;
}

template <class E>
__global__ void __launch_bounds__(kAdjustThreads) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using El = Elem<E>;
  constexpr int PV = El::PV;
  extern __shared__ uint32_t sh[];
  const spec_adjust_t& A = P.a;
  const int S = P.slice, tid = threadIdx.x;
  uint32_t* counts = sh;                          // [S]
  uint32_t* touched = counts + S;                 // [S / 32 + 2]
  float* bias = reinterpret_cast<float*>(touched + S / 32 + 2);  // [biases]
  int32_t* bias_id = reinterpret_cast<int32_t*>(bias + A.biases);
  int32_t* drafted = bias_id + A.biases;          // [rows of the request] token in the slice, or -1
  const int b = blockIdx.y, v0 = blockIdx.x * S, v1 = min(v0 + S, A.V), n = v1 - v0;

  int r0 = b * A.T, r1 = r0 + A.T;
  if (A.row_offsets) {
    r0 = A.row_offsets[b], r1 = A.row_offsets[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > A.rows || r1 - r0 > A.T) {
      if (tid == 0 && P.status) atomicOr(P.status, SPEC_DEV_BAD_OFFSETS);
      return;
    }
  }
  const int rows = r1 - r0;
  if (rows == 0) return;
  for (int i = tid; i < S + S / 32 + 2; i += kAdjustThreads) counts[i] = 0;
  __syncthreads();

  uint32_t bad = 0;
  auto mark = [&](int v) { atomicOr(&touched[v >> 5], 1u << (v & 31)); };
  {
    int len = A.history_lens[b], prompt = A.prompt_lens ? A.prompt_lens[b] : 0;
    if (len < 0 || len > A.history_width) bad |= SPEC_DEV_BAD_OFFSETS;
    len = min(max(len, 0), A.history_width);
    if (prompt < 0 || prompt > len) bad |= SPEC_DEV_BAD_OFFSETS;
    const int32_t* h = A.history + (long long)b * A.history_width;
    for (int i = tid; i < len; i += kAdjustThreads) {
      const int t = h[i];
      if (t < 0 || t >= A.V) {
        bad |= SPEC_DEV_BAD_TOKEN;
      } else if (t >= v0 && t < v1) {
        if (i < prompt)
          atomicOr(&counts[t - v0], kSeenPrompt);
        else
          atomicAdd(&counts[t - v0], 1u);
        mark(t - v0);
      }
    }
    for (int i = tid; i < A.biases; i += kAdjustThreads) {
      const int t = A.bias_ids[(long long)b * A.biases + i];
      bias_id[i] = t;
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
    }
    for (int j = tid; j < rows; j += kAdjustThreads) {
      const int t = A.tokens[r0 + j];
      if (t < -1 || t >= A.V) bad |= SPEC_DEV_BAD_TOKEN;
      drafted[j] = t >= v0 && t < v1 ? t - v0 : -1;
    }
  }
  if (bad && P.status) atomicOr(P.status, bad);
  __syncthreads();
  // biases of a token that is listed more than once are added up in the list's order
  for (int i = tid; i < A.biases; i += kAdjustThreads) {
    const int t = bias_id[i];
    if (t < v0 || t >= v1) continue;
    bool first = true;
    for (int j = 0; j < i; ++j) first = first && bias_id[j] != t;
    if (!first) continue;
    const float* given = A.bias + (long long)b * A.biases;
    float sum = given[i];
    for (int j = i + 1; j < A.biases; ++j)
      if (bias_id[j] == t) sum += given[j];
    bias[i] = sum;
    atomicOr(&counts[t - v0], (uint32_t)(i + 1) << kBiasShift);
    mark(t - v0);
  }

  const float rep = A.repetition ? A.repetition[b] : 1.0f;
  const float freq = A.frequency ? A.frequency[b] : 0.0f;
  const float pres = A.presence ? A.presence[b] : 0.0f;
  auto rule = [&](int v, float x) {  // v within the slice
    const uint32_t w = counts[v];
    const uint32_t c = w & kCountMask;
    if (c || (w & kSeenPrompt)) x = x > 0.0f ? __fdiv_rn(x, rep) : x * rep;
    if (c) x = x - freq * (float)c - pres;
    const uint32_t at = (w & ~kSeenPrompt) >> kBiasShift;
    if (at) x += bias[at - 1];
    return x;
  };

  const int words = (A.V + 31) / 32;
  const E* in_all = static_cast<const E*>(A.logits);
  E* out_all = static_cast<E*>(A.out);
  for (int i = 0; i < rows; ++i) {
    // the drafted tokens that row i sees and row i - 1 did not, and the other way round
    __syncthreads();
    const uint8_t* see = A.mask ? A.mask + ((long long)b * A.T + i) * A.T : nullptr;
    for (int j = tid; j < rows; j += kAdjustThreads) {
      const int v = drafted[j];
      if (v < 0) continue;
      const bool now = see ? see[j] != 0 : j <= i;
      const bool was = i > 0 && (see ? see[j - (long long)A.T] != 0 : j < i);
      if (now != was) atomicAdd(&counts[v], now ? 1u : ~0u);
      if (now) mark(v);
    }
    __syncthreads();

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
      out[v] = !ok ? El::neg_inf() : hit ? El::from_f32(rule(v, El::to_f32(raw))) : raw;
    };
    if (!same) {
      for (int v = tid; v < n; v += kAdjustThreads) one(v);
      continue;
    }
    for (int v = tid; v < lead; v += kAdjustThreads) one(v);
    for (int v = lead + vecs * PV + tid; v < n; v += kAdjustThreads) one(v);
    const uint4* src = reinterpret_cast<const uint4*>(in + lead);
    uint4* dst = reinterpret_cast<uint4*>(out + lead);
    for (int k0 = tid; k0 < vecs; k0 += 4 * kAdjustThreads) {
      uint4 w[4];
      uint32_t ok[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * kAdjustThreads;
        ok[u] = ~0u;
        if (k < vecs) {
          w[u] = src[k];
          if (allow) {
            const int g = v0 + lead + k * PV, s = g & 31;
            uint32_t x = allow[g >> 5] >> s;
            if (s > 32 - PV) x |= allow[(g >> 5) + 1] << (32 - s);
            ok[u] = x;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * kAdjustThreads;
        if (k >= vecs) break;
        const int v = lead + k * PV, s = v & 31;
        const uint32_t hit = __funnelshift_r(touched[v >> 5], touched[(v >> 5) + 1], s) & ((1u << PV) - 1);
        const uint32_t no = ~ok[u] & ((1u << PV) - 1);
        if (hit | no) {
          E e[PV];
          *reinterpret_cast<uint4*>(e) = w[u];
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            if ((no >> j) & 1u)
              e[j] = El::neg_inf();
            else if ((hit >> j) & 1u)
              e[j] = El::from_f32(rule(v + j, El::to_f32(e[j])));
          }
          w[u] = *reinterpret_cast<uint4*>(e);
        }
        dst[k] = w[u];
      }
    }
  }
}

}  // namespace ssv
