// The merge of a split decode row's pieces, shared by the decode kernels.
#pragma once
#include "pka_device.cuh"
#include "pka_internal.h"

namespace pka {
namespace {

// n-way merge of the pieces of one split (request, kv head) for its G qo
// heads, all read from the float workspace ("Deep Dive - FlashInfer", "Core
// mechanism" and "A worked split-KV example"): with b_k the pieces' base-2
// statistics, m = max b_k and s = sum 2^(b_k - m), o = sum (2^(b_k - m) / s)
// o_k and lse = m + log2 s; pieces with b_k = -inf carry no weight, and if
// all are empty o = 0 and lse = -inf.  Every lane owns D / 32 dims of every
// head and folds the (piece, head) pairs in one at a time (a running max with
// rescaling), so all lanes hold the same statistics and nothing is exchanged.
// The states come from other SMs and are read through L2 (.cg), 16 pairs
// per round, all loads of a round issued before any is used.
template <int D, int G>
__device__ __noinline__ void join_merge_g(const AttnArgs& a, const PkaDecodeJoin j, int row,
                                          int head0, int lane) {
  constexpr int PER = D / 32;
  constexpr int CH = G == 8 ? 8 : 12;  // pairs per round; a multiple of G (pair q is head q % G)
  const int pairs = j.nslots * G;
  float m[G], s[G], acc[G][PER];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    s[h] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[h][e] = 0.f;
  }
  for (int p0 = 0; p0 < pairs; p0 += CH) {
    float b[CH], x[CH][PER];
#pragma unroll
    for (int q = 0; q < CH; ++q) {
      const int p = p0 + q;
      const bool ok = p < pairs;
      const int64_t rec = j.rec_first + (int64_t)(p / G) * j.rec_stride + q % G;
      b[q] = ok ? __ldcg(a.part_lse + rec) : -INFINITY;
      const float* src = a.part_o + (ok ? rec : 0) * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 v = ok ? __ldcg(reinterpret_cast<const float4*>(src))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        x[q][0] = v.x;
        x[q][1] = v.y;
        x[q][2] = v.z;
        x[q][3] = v.w;
      } else {
        const float2 v = ok ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
        x[q][0] = v.x;
        x[q][1] = v.y;
      }
    }
#pragma unroll
    for (int q = 0; q < CH; ++q) {
      const int h = q % G;
      if (b[q] == -INFINITY) continue;
      if (b[q] > m[h]) {
        const float sc = exp2f(m[h] - b[q]);  // 0 while m is -inf
        s[h] = s[h] * sc + 1.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[h][e] = acc[h][e] * sc + x[q][e];
        m[h] = b[q];
      } else {
        const float wq = exp2f(b[q] - m[h]);
        s[h] += wq;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[h][e] += wq * x[q][e];
      }
    }
  }
  const int Hq = a.num_qo_heads;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const bool any = s[h] > 0.f;
    const float inv = any ? 1.f / s[h] : 0.f;
    const int64_t oi = (int64_t)row * Hq + head0 + h;
    uint16_t* dst = a.o + oi * D + lane * PER;
    if constexpr (PER == 4) {
      uint2 pk;
      pk.x = float2_to_bf16x2(acc[h][0] * inv, acc[h][1] * inv);
      pk.y = float2_to_bf16x2(acc[h][2] * inv, acc[h][3] * inv);
      *reinterpret_cast<uint2*>(dst) = pk;
    } else {
      *reinterpret_cast<uint32_t*>(dst) = float2_to_bf16x2(acc[h][0] * inv, acc[h][1] * inv);
    }
    if (lane == 0 && a.lse) a.lse[oi] = any ? m[h] + log2f(s[h]) : -INFINITY;
  }
}

template <int D>
__device__ __forceinline__ void join_merge(const AttnArgs& a, const PkaDecodeJoin& j, int row,
                                           int head0, int G, int lane) {
  switch (G) {
    case 1: join_merge_g<D, 1>(a, j, row, head0, lane); break;
    case 2: join_merge_g<D, 2>(a, j, row, head0, lane); break;
    case 4: join_merge_g<D, 4>(a, j, row, head0, lane); break;
    default: join_merge_g<D, 8>(a, j, row, head0, lane); break;
  }
}

}  // namespace
}  // namespace pka
