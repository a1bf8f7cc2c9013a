// K/V held in 4 bits: the page format and the launches that know it.
//
// A page of the K (or V) pool is one run of bytes:
//   codes [P, Hk, D/2] (HND: [Hk, P, D/2]): element 2i of a head in the low
//     half of byte i, element 2i + 1 in the high half;
//   words [P, Hk, G] (HND: [Hk, P, G]): one 32-bit word for each of the G =
//     D / group groups of a head, a bf16 step in the low half and a bf16 origin
//     in the high half;
// padded to a multiple of 16 bytes.  Code c stands for origin + step * c.
// Codes and words lie apart so that both start on whole 16-byte pieces for
// every head count: a row of 64 bytes with its word beside it would start on
// multiples of 4.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "pka.h"
#include "pka_internal.h"

namespace pka {

// Elements of a group, or 0 for K/V in other types.
inline int kv4_group(int kv_dtype) {
  return kv_dtype == PKA_KV_INT4_G32    ? 32
         : kv_dtype == PKA_KV_INT4_G64  ? 64
         : kv_dtype == PKA_KV_INT4_G128 ? 128
                                        : 0;
}

// Bytes of the codes and of the words of one page.
inline int64_t kv4_code_bytes(const pka_params& p) {
  return (int64_t)p.page_size * p.num_kv_heads * (p.head_dim / 2);
}
inline int64_t kv4_word_bytes(const pka_params& p) {
  return (int64_t)p.page_size * p.num_kv_heads * (p.head_dim / kv4_group(p.kv_dtype)) * 4;
}

// Largest calls of the kernels in kv4.cu: heads make the second grid axis,
// rows the first.
constexpr int kKvMaxHeads = 4096;
constexpr int64_t kKvMaxRows = INT64_C(1) << 33;

// Whether 4-bit parameters describe something built: paged K/V, groups of at
// most a head, pages under 2 GB (a row's place in its page is 32 bits wide).
inline bool kv4_supported(const pka_params& p) {
  const int g = kv4_group(p.kv_dtype);
  if (g == 0) return true;
  if (g > p.head_dim || p.kv_ragged || p.num_kv_heads > kKvMaxHeads) return false;
  return (int64_t)p.num_kv_heads * (p.head_dim / 2 + p.head_dim / g * 4) <=
         (INT32_MAX - 15) / p.page_size;
}

// Elements of 16 bytes in a pool, less one: what a stride in elements may not have set.
inline int64_t kv_stride_mask(int kv_dtype) { return kv_dtype == PKA_KV_BF16 ? 7 : 15; }

// Where the rows of a call lie in the pools.
struct KvRows {
  // rows of requests: row t of request r is position begin[r] + t (begin null: 0
  // for a read, the request's last rows for an append)
  int32_t batch;
  const int32_t* begin;
  const int32_t* row_indptr;
  const int32_t* kv_indptr;
  const int32_t* last_page_len;
  int64_t num_pages;         // of the pools; INT64_MAX: page ids are trusted
  // or rows of the plan's units (units not null)
  const PkaDequantUnit* units;
  int32_t num_units;
  const int32_t* counts;     // graph mode: the plan's unit and row counts on the device
  int64_t rows;
  const int32_t* kv_indices;
  int64_t page_stride;       // elements
  int32_t page_size;
  int32_t layout;
  int32_t heads;
  int32_t* err;
};

// bf16 rows [rows, heads, D] quantised into 4-bit pools.
cudaError_t launch_append4(const KvRows& r, int head_dim, int group, const uint16_t* k_new,
                           const uint16_t* v_new, uint8_t* k, uint8_t* v, cudaStream_t stream);
// Rows of requests in pools of any type to bf16 [rows, heads, D]; an output may be null.
cudaError_t launch_read(const KvRows& r, int kv_dtype, int head_dim, float k_scale, float v_scale,
                        const void* k, const void* v, uint16_t* k_out, uint16_t* v_out,
                        cudaStream_t stream);
// The rows of a launch on the tensor cores, staged in f16 from 4-bit pools and
// bf16 queries: 11 bits where bf16 would round origin + step * code to 8.  Each
// of Q's heads, and each kv head of K and of V of a unit (a request's or a cascade
// node's keys), is scaled by the power of two that brings its largest element into
// [2^14, 2^15), so no magnitude leaves f16's range: an element keeps 11 bits down to
// 2^-28 of the largest.  A launch reads no other unit's scales with a unit's keys.
//   Where a kv head of a unit holds groups (of any of its keys, seen or not) whose
// largest elements lie more than 2^kF16Span apart, its rows are staged in bf16
// instead, unscaled, and Q and P are bf16 with them: 8 bits, at any magnitude, so that
// a row does not lose what it sees to a key that is hidden from it or has no weight.
// 16 leaves every group its 11 bits for elements down to 2^-12 of its largest.
constexpr uint32_t kF16Span = 16;
// Bits of the largest of a kv head's groups of K (x) and of V (y), and the complement
// of the bits of the smallest that is not 0 (z, w); all 0 where there is none.
typedef uint4 Kv4Range;
struct F16Scales {
  const float* q_down;       // [rows, Hq]: what Q's rows are to be multiplied by
  const Kv4Range* kv_range;  // [units, Hk]
  const uint16_t* q;         // bf16 Q
};
struct F16Stage {
  KvRows rows;               // units; rows: of the scratch (its capacity in graph mode)
  const uint8_t* k;
  const uint8_t* v;
  uint16_t* k16;             // [rows, Hk, D]
  uint16_t* v16;
  const uint16_t* q;         // [q_rows, Hq, D] bf16
  uint16_t* q16;
  float* q_down;
  int64_t q_rows;
  int q_heads;
  Kv4Range* kv_range;        // [rows.num_units, Hk]
};
cudaError_t launch_stage_f16(const F16Stage& s, int head_dim, int group, cudaStream_t stream);
cudaError_t launch_prefill_staged(const AttnArgs& a, const F16Scales& scales, int num_ctas,
                                  int head_dim, int group, int nnz_q, int64_t total_kv,
                                  MapCache* cache, cudaStream_t stream);
// Decode rows over 4-bit pools.
cudaError_t launch_decode4(const AttnArgs& a, int num_ctas, int head_dim, int group,
                           cudaStream_t stream);

#ifdef __CUDACC__
// 2^(14 - e) and 2^(e - 14) for the exponent e of a float given by its bits
// (kept from -100 on, so that both are normal).
__device__ __forceinline__ int f16_exponent(uint32_t bits) {
  return max((int)(bits >> 23) - 127, -100);
}
__device__ __forceinline__ float f16_up(uint32_t bits) {
  return __uint_as_float((uint32_t)(127 + 14 - f16_exponent(bits)) << 23);
}
__device__ __forceinline__ float f16_down(uint32_t bits) {
  return __uint_as_float((uint32_t)(127 - 14 + f16_exponent(bits)) << 23);
}

// Whether a kv head's rows are staged in bf16.
__device__ __forceinline__ bool f16_too_wide(const Kv4Range& r) {
  return (r.x >> 23) > kF16Span + (~r.z >> 23) || (r.y >> 23) > kF16Span + (~r.w >> 23);
}

// The step and origin of a group whose least and greatest elements are given,
// and the reciprocal that the codes are made with (0: every code is 0).
//   A step is the range's 15th and an origin the least element, each rounded to
// bf16: 8 significant bits leave a step within 2^-9, a 33rd of a step over 15
// codes, and 16 bits more a group would be spent on it.  A range that is not
// finite (an infinity or NaN in the group) makes both NaN, so the group reads
// back as NaN; a range too small for a normal bf16 step is held as its origin.
struct Group4 {
  uint32_t word;
  float step, origin, inv;
};

__device__ __forceinline__ Group4 group4(float lo, float hi) {
  Group4 g;
  const float range = hi - lo;
  if (!(fabsf(range) <= 3.402823466e38f)) {
    g.word = 0x7fc07fc0u;
    g.step = g.origin = g.inv = 0.f;
    return g;
  }
  // range / 15: the product with 1 / 15 corrected by its residual, exact where the
  // quotient is a float32, so that it rounds to bf16 as the quotient does
  const float fifteenth = 1.f / 15.f, near = range * fifteenth;
  const float step = fmaf(fmaf(-near, 15.f, range), fifteenth, near);
  uint32_t s;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(s) : "f"(lo), "f"(step));
  if ((s & 0x7fffu) < 0x0080u) s &= 0xffff0000u;
  g.word = s;
  g.step = __uint_as_float(s << 16);
  g.origin = __uint_as_float(s & 0xffff0000u);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.step));
  if (!(g.step > 0.f)) g.inv = 0.f;
  return g;
}

// 8 codes of a group, element i in bits 4i.
//   The quotient (x - origin) / step is the product with an approximate
// reciprocal, corrected by its residual (a step of Newton's iteration): exact where the quotient is a float32,
// so ties round to even as after a division, and elsewhere no quotient of 24-bit
// by 8-bit numbers that matters lies near a tie.  The sum with 1.5 * 2^23 rounds
// it; the code is then the low bits.  CLAMP: the origin may lie off the least
// element (which is no bf16), and quotients outside 0 .. 15.
template <bool CLAMP>
__device__ __forceinline__ uint32_t codes4(const float (&x)[8], const Group4& g) {
  const float2 less = make_float2(-g.origin, -g.origin), inv = make_float2(g.inv, g.inv);
  const float2 minus = make_float2(-g.step, -g.step), round = make_float2(12582912.f, 12582912.f);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 d = __fadd2_rn(make_float2(x[i], x[i + 1]), less);
    float2 q = __fmul2_rn(d, inv);
    q = __ffma2_rn(__ffma2_rn(q, minus, d), inv, q);
    if constexpr (CLAMP) {
      q.x = fminf(fmaxf(q.x, 0.f), 15.f);
      q.y = fminf(fmaxf(q.y, 0.f), 15.f);
    }
    q = __fadd2_rn(q, round);
    w += (__float_as_uint(q.x) << (4 * i)) + (__float_as_uint(q.y) << (4 * i + 4));
  }
  // each float's bits are 0x4b400000 + code: their sum, shifted, is taken off
  constexpr uint32_t kBias = 0x4b400000u;
  uint32_t off = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) off += kBias << (4 * i);
  return w - off;
}
#endif

}  // namespace pka
