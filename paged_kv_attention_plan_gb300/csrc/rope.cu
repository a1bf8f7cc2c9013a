// Rotary positions: pka_rope_init, pka_apply_rope and the append that rotates
// (pka_rope_append_paged_kv_cache).
//
// Pair i of a head, (a, b), at position n is the complex number a + i b times
// m exp(i n f_i).  The transposed map (the gradient) turns by -n f_i.
//
// Angles: f_i / 2 pi is held as a 64-bit fraction of a turn, F_i.  n * F_i
// modulo 2^64 is then the angle modulo one turn with no rounding at all, for
// every 32-bit n, from three integer instructions; its upper 32 bits, as a
// float in [-1, 1) half turns, go to sincospif.  A float32 product n * f_i
// would be off by up to 2^-24 n f_i radians, 0.06 at position 1,000,000.
#include <cmath>

#include "pka_cache.h"
#include "pka_device.cuh"
#include "pka_internal.h"
#include "pka_kv4.h"

namespace pka {
namespace {

// How the pairs of a head lie in it.
enum RopeLayout {
  kHalf = 0,       // (x[i], x[i + R/2]), R/2 a multiple of 8: whole 16-byte pieces
  kAdjacent = 1,   // (x[2i], x[2i + 1])
  kScattered = 2,  // (x[i], x[i + R/2]), any other R: through shared memory
  kPartOfHalf = 3,  // kHalf with R < D, where a lane's pieces lie elsewhere: 4-bit pools
};

// What the pools hold; any other number: 4 bits in groups of so many.
enum PoolType { kBf16 = 0, kE4m3 = 1 };

constexpr int kMaxHeads = 4096;            // of a row; keeps the second grid axis small
constexpr int64_t kMaxRows = INT64_C(1) << 33;  // eight a block

struct RopeArgs {
  const uint16_t* q;  // [rows, q_heads, D], row stride in elements
  const uint16_t* k;
  const uint16_t* v;  // append only
  uint16_t* q_out;
  uint16_t* k_out;    // apply only
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t rows;
  const int32_t* positions;  // [rows]; append: may be null (logical positions)
  int q_heads, k_heads;
  int rotary_dim;
  float magnitude;
  float sine_sign;           // -1 for the transposed map
  int steps_per_part;        // head steps that one warp takes of its row
  // append: the page table and the pools
  int32_t batch;
  const int32_t* append_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last_page_len;
  void* k_pool;
  void* v_pool;
  int64_t page_stride;
  int64_t num_pages;
  int page_size;
  int layout;
  float k_scale, v_scale;    // e4m3 pools
  float k_inv, v_inv;        // pow2_reciprocal of these
  int64_t code_bytes;        // 4-bit pools: where a page's words start
  int32_t* err;
  uint64_t turns[64];        // F_i
};

// 8 values divided by a pool's scale (correctly rounded; by the reciprocal of a
// power of two, which is as exact) and rounded to nearest even e4m3, magnitudes
// above 448 clamped; 8 codes, little-endian.  The general division costs a
// 9,216-row append into e4m3 pools 47 us where the product takes 41.
__device__ __forceinline__ uint2 to_e4m3x8(const float (&x)[8], float scale, float inv) {
  uint32_t pk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = inv > 0.f ? x[2 * i] * inv : __fdiv_rn(x[2 * i], scale);
    const float hi = inv > 0.f ? x[2 * i + 1] * inv : __fdiv_rn(x[2 * i + 1], scale);
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n cvt.u32.u16 %0, t;\n}"
        : "=r"(pk[i])
        : "f"(hi), "f"(lo));
  }
  return make_uint2(pk[0] | (pk[1] << 16), pk[2] | (pk[3] << 16));
}

__device__ __forceinline__ void unpack8(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[4]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  w[0] = x.x;
  w[1] = x.y;
  w[2] = x.z;
  w[3] = x.w;
}

__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Word w becomes (lo, hi) in bf16 where these are rotated: the first `turned`
// of the two elements.
__device__ __forceinline__ void round_turned(uint32_t& w, float lo, float hi, int turned) {
  if (turned <= 0) return;
  const uint32_t y = float2_to_bf16x2(lo, hi);
  w = turned > 1 ? y : (y & 0xffffu) | (w & 0xffff0000u);
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The least of 8 numbers, or of their negatives; NaN where one is.
template <bool NEGATED>
__device__ __forceinline__ float least8(const float (&x)[8]) {
  auto at = [&](int i) { return NEGATED ? -x[i] : x[i]; };
  const float a = min_nan(at(0), at(1), at(2)), b = min_nan(at(3), at(4), at(5));
  return min_nan(min_nan(at(6), at(7), a), b);
}

__device__ __forceinline__ void to_shared(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void from_shared(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x;
  x[1] = a.y;
  x[2] = a.z;
  x[3] = a.w;
  x[4] = b.x;
  x[5] = b.y;
  x[6] = b.z;
  x[7] = b.w;
}

// A warp takes a row, or a part of its heads, and walks the heads (q, then k,
// then v as one list).  A head is D/16 units of 8 pairs; a lane keeps one unit
// (u) and takes it from each of the 32 / (D/16) heads of a step, so its 8
// sines and cosines serve the whole row.  A lane reads and writes two 16-byte
// pieces A and B of a head.  Half layout: pair j is (A[j], B[j]).  Adjacent:
// the pairs inside A and inside B.  Scattered: the pieces meet as floats in
// shared memory, where a lane's pairs lie D/16 apart (no two lanes of a warp
// on one bank; the 16-byte moves in and out meet each bank twice) and are
// turned in place.  Elements past rotary_dim keep their bits.  The pieces of
// kInFlight steps are loaded before the first of them is used, the first ones
// before the row's page and sines are looked up.
//
// Whole pieces are bound by memory bandwidth: each element is read once and
// written once, and 16,387 rows of 64 heads of 128 take 79.4 us, 6.76 TB/s, the
// rate of a plain copy.  Two steps in flight at four blocks an SM are enough
// and leave the registers for it (16,387 rows of 40 heads, in us: one step
// 54.9, two 51.6, three at three blocks 51.8, four at two blocks 59.1).
// Scattered pairs wait for shared memory and take 1.5 to 1.9 times as long as
// a copy; the rotation alone spills 44 to 48 bytes there at four blocks an SM,
// 12 at three (in us, three / four blocks: 8,192 rows of 40 heads with 40 of
// 128 elements turned 46.6 / 42.4, 16,387 with 126 88.2 / 93.4, an append of
// 9,216 with 40 50.6 / 46.3).
// Into e4m3 pools both pieces are held as floats: three blocks, 80 registers
// and 12 to 36 bytes spilled.
//   Into 4-bit pools as well.  A lane's pieces are elements 8u .. and D/2 + 8u .. of
// a head, so a group is a power of two of lanes; only half layouts that rotate a part
// of a head (kPartOfHalf) hand their floats on through shared memory, 16 in a row to
// a lane.  Three blocks of 80 registers fill neither issue slots (54%) nor DRAM (50%):
// 9,101 rows of 48 heads of 128 with the read-back of what they wrote take 52.6 us with
// groups of a head, 55 with smaller ones, 59.4 where half of each head rotates (through
// shared memory for all: 61.3, 60.5 and 59.6; group sizes known at run time only: 64.1;
// four blocks an SM 59.4, two 62).
constexpr int kInFlight = 2;

template <int D, int L, bool APPEND, int POOL>
__global__ void __launch_bounds__(256, POOL != kBf16 ? 3 : 4)
rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr bool F8 = POOL == kE4m3, INT4 = POOL > kE4m3;
  constexpr int GR = POOL;  // elements of a group (4-bit pools)
  constexpr bool HALF = L == kHalf || L == kPartOfHalf;
  constexpr int UNITS = D / 16;      // lanes of a head
  constexpr int HPS = 32 / UNITS;    // heads of a step
  constexpr int K = 8 / HPS;         // pairs whose sine and cosine a lane computes
  // floats of a head in shared memory; kPartOfHalf reads it back 16 in a row, four
  // floats of padding apart so that the lanes of a head meet different banks
  constexpr int STRIDE = L == kPartOfHalf ? D + 4 * UNITS : D + UNITS;
  constexpr bool SHARED = L == kScattered || L == kPartOfHalf;
  __shared__ __align__(16) float heads_in_shared[SHARED ? 8 * HPS * STRIDE : 4];
  const int lane = threadIdx.x & 31;
  const int u = lane % UNITS, sub = lane / UNITS;
  const int rd = a.rotary_dim;
  const int heads = a.q_heads + (APPEND ? 2 : 1) * a.k_heads;
  const int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (row >= a.rows) return;

  // where the lane's pieces lie in a head (B `apart` elements behind A), and
  // which of its pairs rotate
  int off_a = 8 * u, apart = D / 2;
  if (HALF) {
    const int t = u - rd / 16;
    if (t >= 0) off_a = rd + 16 * t;
    apart = t < 0 ? rd / 2 : 8;
  }
  auto pair_of = [&](int j) {
    return HALF ? 8 * u + j
           : L == kScattered ? u + UNITS * j
                             : j < 4 ? 4 * u + j : D / 4 + 4 * u + j - 4;
  };
  uint32_t turning = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) turning |= (pair_of(j) < rd / 2 ? 1u : 0u) << j;
  uint64_t turn[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int p = pair_of(sub * K + i);
    turn[i] = p < rd / 2 ? a.turns[p] : 0;
  }

  // head h of the row starts at D * h of one of these
  const int64_t at_q = row * a.q_stride + off_a;
  const int64_t at_k = row * a.k_stride - (int64_t)a.q_heads * D + off_a;
  const int64_t at_v = APPEND ? row * a.v_stride - (int64_t)(a.q_heads + a.k_heads) * D + off_a : 0;
  const int k_end = a.q_heads + a.k_heads;
  const int h0 = blockIdx.y * a.steps_per_part * HPS;
  const int h1 = min(heads, h0 + a.steps_per_part * HPS);
  uint32_t wa[kInFlight][4], wb[kInFlight][4];
  auto load = [&](int hb) {  // the lane's pieces of heads hb + sub, + HPS, ...
#pragma unroll
    for (int t = 0; t < kInFlight; ++t) {
      const int h = hb + t * HPS + sub;
      if (h >= h1) continue;
      const uint16_t* src = h < a.q_heads               ? a.q + at_q
                            : !APPEND || h < k_end ? a.k + at_k
                                                   : a.v + at_v;
      src += h * D;
      load16(src, wa[t]);
      load16(src + apart, wb[t]);
    }
  };
  load(h0);

  int64_t pos = 0;
  int32_t page = -1;
  int slot = 0;
  if constexpr (APPEND) {
    // a decode step's rows are one a request: row r is tried as request r's
    // before the search
    const int guess = (int)min(row, (int64_t)a.batch - 1);
    int r = guess, first = a.append_indptr[guess], last = a.append_indptr[guess + 1];
    const int end = a.append_indptr[a.batch];
    if (row < first || row >= last) {
      if (row >= end) return;  // a row of no request
      r = warp_find(a.append_indptr, a.batch, row, lane);
      first = a.append_indptr[r];
      last = a.append_indptr[r + 1];
    }
    const int kv0 = a.kv_indptr[r], pages = a.kv_indptr[r + 1] - kv0;
    const int64_t kv_len = (int64_t)(pages - 1) * a.page_size + a.last_page_len[r];
    pos = kv_len - (last - first) + (row - first);
    const int64_t nth = pos < 0 ? -1
                        : pos <= UINT32_MAX ? (uint32_t)pos / (uint32_t)a.page_size
                                            : pos / a.page_size;
    if (nth >= 0 && nth < pages) {
      page = a.kv_indices[kv0 + nth];
      slot = (int)(pos - nth * a.page_size);
    }
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) note_error(a.err, PKA_ERR_METADATA);
      page = -1;
    }
  }
  if (!APPEND || a.positions) pos = a.positions[row];

  // sines and cosines: K pairs a lane, exchanged among the lanes of a unit
  float c[8], s[8];
  {
    float ck[K], sk[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const uint64_t phase = (uint64_t)pos * turn[i] + (1ull << 31);
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sk[i], &ck[i]);
      ck[i] *= a.magnitude;
      sk[i] *= a.magnitude * a.sine_sign;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = __shfl_sync(0xffffffffu, ck[j % K], (j / K) * UNITS + u);
      s[j] = __shfl_sync(0xffffffffu, sk[j % K], (j / K) * UNITS + u);
    }
  }

  // where head h goes: D * h behind out_q, or head_step * (its number) in the pool
  const int64_t out_q = row * a.q_out_stride + off_a;
  const int64_t out_k = row * a.k_out_stride - (int64_t)a.q_heads * D + off_a;
  const int64_t head_step = a.layout == PKA_NHD ? D : (int64_t)a.page_size * D;
  const int64_t in_pool = (int64_t)page * a.page_stride +
                          (int64_t)slot * (a.layout == PKA_NHD ? a.k_heads * D : D) + off_a;

  // 4-bit pools: the page's bytes, the row's place among the page's (slot, head) and a
  // head's step there (a page is under 2 GB)
  const int64_t pool_page = (int64_t)page * a.page_stride;
  const int pool_slot = a.layout == PKA_NHD ? slot * a.k_heads : slot;
  const int pool_head = a.layout == PKA_NHD ? 1 : a.page_size;

  for (int hb = h0;;) {
#pragma unroll
    for (int t = 0; t < kInFlight; ++t) {
      const int h = hb + t * HPS + sub;
      const bool is_v = APPEND && h >= k_end;
      const bool to_pool = APPEND && h >= a.q_heads;
      const bool store = h < h1 && !(to_pool && page < 0);
      if (L != kScattered && !store && !(INT4 && hb + (t + 1) * HPS > a.q_heads)) continue;
      float xa[8], xb[8];
      if constexpr (L == kScattered) {  // all lanes: the heads of a step meet the barriers together
        float* m = heads_in_shared + ((threadIdx.x >> 5) * HPS + sub) * STRIDE;
        unpack8(wa[t], xa);
        unpack8(wb[t], xb);
        if (!is_v) {
          to_shared(m + off_a, xa);
          to_shared(m + off_a + apart, xb);
        }
        __syncwarp();
        if (!is_v) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int p = u + UNITS * j;
            if (turning >> j & 1) {
              const float x = m[p], y = m[p + rd / 2];
              m[p] = x * c[j] - y * s[j];
              m[p + rd / 2] = x * s[j] + y * c[j];
            }
          }
        }
        __syncwarp();
        if (!is_v) {
          from_shared(m + off_a, xa);
          from_shared(m + off_a + apart, xb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            round_turned(wa[t][i], xa[2 * i], xa[2 * i + 1], rd - (off_a + 2 * i));
            round_turned(wb[t][i], xb[2 * i], xb[2 * i + 1], rd - (off_a + apart + 2 * i));
          }
        }
        __syncwarp();  // read before the next step writes
        if (!store && !(INT4 && hb + (t + 1) * HPS > a.q_heads)) continue;
      } else if (F8 || INT4 || (HALF && turning && !is_v)) {
        unpack8(wa[t], xa);
        unpack8(wb[t], xb);
        if (!is_v) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // pair j: (A[j], B[j]), or adjacent elements of A (j < 4) or of B
            float& x = HALF ? xa[j] : j < 4 ? xa[2 * j] : xb[2 * (j - 4)];
            float& y = HALF ? xb[j] : j < 4 ? xa[2 * j + 1] : xb[2 * (j - 4) + 1];
            if (HALF ? turning != 0 : (turning >> j & 1) != 0) {
              const float z = x * c[j] - y * s[j];
              y = x * s[j] + y * c[j];
              x = z;
              if (L == kAdjacent && !(INT4 && to_pool))
                (j < 4 ? wa[t][j & 3] : wb[t][j & 3]) = float2_to_bf16x2(x, y);
            }
          }
          if (HALF && turning && !(INT4 && to_pool)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              wa[t][i] = float2_to_bf16x2(xa[2 * i], xa[2 * i + 1]);
              wb[t][i] = float2_to_bf16x2(xb[2 * i], xb[2 * i + 1]);
            }
          }
        }
      } else if (L == kAdjacent && !is_v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t& w = j < 4 ? wa[t][j & 3] : wb[t][j & 3];
          const float2 f = bf16x2_to_float2(w);
          if (turning >> j & 1)
            w = float2_to_bf16x2(f.x * c[j] - f.y * s[j], f.x * s[j] + f.y * c[j]);
        }
      }
      // 4-bit pools: a group is pieces 8u .. and D/2 + 8u .. of all the head's lanes, or
      // one of the two of GR / 8 lanes.  A step of q heads alone has none.
      if constexpr (INT4) {
        if (hb + (t + 1) * HPS > a.q_heads) {  // the same for all lanes
          constexpr bool ROW = L == kPartOfHalf;  // its pieces now, through shared memory
          if constexpr (ROW) {
            float* m = heads_in_shared + ((threadIdx.x >> 5) * HPS + sub) * STRIDE;
            to_shared(m + off_a + (off_a >> 4) * 4, xa);
            to_shared(m + off_a + apart + ((off_a + apart) >> 4) * 4, xb);
            __syncwarp();
            from_shared(m + 20 * u, xa);
            from_shared(m + 20 * u + 8, xb);
            __syncwarp();  // read before the next step writes
          }
          constexpr int N = ROW || GR == D ? 1 : 2;  // groups that a lane is in
          constexpr int LANES = ROW ? GR / 16 : GR == D ? UNITS : GR / 8;
          const int at_head = pool_slot + (h - (is_v ? k_end : a.q_heads)) * pool_head;
          uint8_t* const p = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + pool_page;
          uint8_t* const codes = p + at_head * (D / 2) + (ROW ? 8 : 4) * u;
          uint8_t* const words = p + a.code_bytes + (at_head * (D / GR) + u / LANES) * 4;
          // least elements and negated greatest, of the lane and then of its groups
          float lo[2] = {least8<false>(xa), least8<false>(xb)};
          float hi[2] = {least8<true>(xa), least8<true>(xb)};
          if constexpr (N == 1) {
            lo[0] = min_nan(lo[0], lo[1]);
            hi[0] = min_nan(hi[0], hi[1]);
          }
#pragma unroll
          for (int off = 1; off < LANES; off <<= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
              hi[i] = min_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
            }
          }
          if (to_pool && store) {
            const Group4 g = group4(lo[0], -hi[0]);
            const Group4 gb = N == 1 ? g : group4(lo[1], -hi[1]);
            const uint32_t ca = codes4<true>(xa, g), cb = codes4<true>(xb, gb);
            if constexpr (ROW) {
              *reinterpret_cast<uint2*>(codes) = make_uint2(ca, cb);
            } else {
              *reinterpret_cast<uint32_t*>(codes) = ca;
              *reinterpret_cast<uint32_t*>(codes + D / 4) = cb;
            }
            if (u % LANES == 0) {
              *reinterpret_cast<uint32_t*>(words) = g.word;
              if constexpr (N == 2) *reinterpret_cast<uint32_t*>(words + D / GR * 2) = gb.word;
            }
          }
          if (to_pool || !store) continue;
        }
      }
      // rotated elements are rounded once, to bf16 or to a code; the others keep their bits
      if (!to_pool) {
        uint16_t* p = (h < a.q_heads ? a.q_out + out_q : a.k_out + out_k) + h * D;
        store16(p, wa[t]);
        store16(p + apart, wb[t]);
        continue;
      }
      const int64_t at = in_pool + (h - (is_v ? k_end : a.q_heads)) * head_step;
      if constexpr (F8) {
        const float scale = is_v ? a.v_scale : a.k_scale, inv = is_v ? a.v_inv : a.k_inv;
        uint8_t* p = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + at;
        *reinterpret_cast<uint2*>(p) = to_e4m3x8(xa, scale, inv);
        *reinterpret_cast<uint2*>(p + apart) = to_e4m3x8(xb, scale, inv);
      } else {
        uint16_t* p = static_cast<uint16_t*>(is_v ? a.v_pool : a.k_pool) + at;
        store16(p, wa[t]);
        store16(p + apart, wb[t]);
      }
    }
    hb += kInFlight * HPS;
    if (hb >= h1) break;
    load(hb);
  }
}

// How many of a row's head steps one warp takes.  First enough warps: 16 an SM
// (64 rows of 10 steps: 2.4 us with one step a warp, 5.8 with ten).  Then
// longer runs, which share one look-up of page and sines, to at most six steps:
// past that the last warps run alone (16,387 rows of 10 steps: one 97 us, two
// 60, four 56, six 55, ten 58; a 9,216-row append of 12: 83, 48, 39, 38, 38).
int steps_per_part(int64_t rows, int steps) {
  const int sms = current_device_sms();
  const int64_t warps = 16 * (int64_t)(sms > 0 ? sms : 1);
  const int64_t per = (rows * steps + warps - 1) / warps;
  const int most = per < 1 ? 1 : per > 6 ? 6 : (int)per;
  const int parts = (steps + most - 1) / most;
  return (steps + parts - 1) / parts;
}

template <int D, int L, bool APPEND, int POOL>
cudaError_t launch(const RopeArgs& args, cudaStream_t stream) {
  constexpr int HPS = 512 / D;  // heads of a step
  RopeArgs a = args;
  const int heads = a.q_heads + (APPEND ? 2 : 1) * a.k_heads;
  const int steps = (heads + HPS - 1) / HPS;
  a.steps_per_part = steps_per_part(a.rows, steps);
  const int parts = (steps + a.steps_per_part - 1) / a.steps_per_part;
  const dim3 grid((unsigned)((a.rows + 7) / 8), (unsigned)parts);
  rope_kernel<D, L, APPEND, POOL><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool APPEND, int POOL>
cudaError_t launch_layout(const RopeArgs& a, int l, cudaStream_t stream) {
  if constexpr (POOL > kE4m3)
    if (l == kPartOfHalf) return launch<D, kPartOfHalf, APPEND, POOL>(a, stream);
  return l == kAdjacent ? launch<D, kAdjacent, APPEND, POOL>(a, stream)
         : l == kHalf   ? launch<D, kHalf, APPEND, POOL>(a, stream)
                        : launch<D, kScattered, APPEND, POOL>(a, stream);
}

template <bool APPEND, int POOL>
cudaError_t launch_any(const RopeArgs& a, int head_dim, bool adjacent, cudaStream_t stream) {
  const int l = adjacent                                        ? kAdjacent
                : a.rotary_dim % 16                             ? kScattered
                : POOL > kE4m3 && a.rotary_dim < head_dim       ? kPartOfHalf
                                                                : kHalf;
  if (head_dim == 128) return launch_layout<128, APPEND, POOL>(a, l, stream);
  if constexpr (POOL <= 64) return launch_layout<64, APPEND, POOL>(a, l, stream);
  return cudaErrorInvalidValue;  // a group of more than a head
}

bool rope_valid(const pka_rope* r, int head_dim) {
  return r && r->rotary_dim >= 2 && r->rotary_dim % 2 == 0 && r->rotary_dim <= head_dim &&
         (r->interleaved == 0 || r->interleaved == 1) && r->reserved == 0 &&
         std::isfinite(r->magnitude);
}

void take_rope(RopeArgs* a, const pka_rope* r) {
  a->rotary_dim = r->rotary_dim;
  a->magnitude = r->magnitude;
  a->sine_sign = 1.f;
  for (int i = 0; i < r->rotary_dim / 2; ++i) a->turns[i] = r->turns[i];
}

// Rows of `heads` heads: 16-byte pieces at a row stride of whole pieces, rows apart.
bool rows_ok(const void* p, int64_t stride, int64_t rows, int heads, int head_dim) {
  if (!p || (reinterpret_cast<uintptr_t>(p) & 15) || (stride & 7)) return false;
  return rows <= 1 ? stride >= 0 : stride >= (int64_t)heads * head_dim;
}

// In place or apart: the same rows, or (as far as the first bytes tell) others.
bool out_ok(const void* in, int64_t in_stride, const void* out, int64_t out_stride) {
  return in != out || in_stride == out_stride;
}

}  // namespace
}  // namespace pka

extern "C" {

pka_status pka_rope_init(const pka_rope_params* p, pka_rope* rope) {
  if (!p || !rope) return PKA_ERR_INVALID_ARG;
  if (p->reserved != 0 || (p->interleaved != 0 && p->interleaved != 1)) return PKA_ERR_INVALID_ARG;
  if (p->rotary_dim < 2 || p->rotary_dim % 2) return PKA_ERR_INVALID_ARG;
  if (p->rotary_dim > 128) return PKA_ERR_UNSUPPORTED;
  if (!std::isfinite(static_cast<float>(p->magnitude))) return PKA_ERR_INVALID_ARG;
  if (!p->frequencies_h) {
    if (!(p->base >= 1.0) || !std::isfinite(p->base)) return PKA_ERR_INVALID_ARG;
    if (p->scaling < PKA_ROPE_PLAIN || p->scaling > PKA_ROPE_BY_PARTS) return PKA_ERR_INVALID_ARG;
    if (p->scaling != PKA_ROPE_PLAIN && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
      return PKA_ERR_INVALID_ARG;
    if (p->scaling == PKA_ROPE_BY_PARTS &&
        (!(p->original_len > 0.0) || !std::isfinite(p->original_len) ||
         !(p->low_rotations >= 0.0) || !(p->high_rotations > p->low_rotations) ||
         !std::isfinite(p->high_rotations)))
      return PKA_ERR_INVALID_ARG;
  }
  const double pi = 3.14159265358979323846;
  const int half = p->rotary_dim / 2;
  pka_rope out{};
  out.rotary_dim = p->rotary_dim;
  out.interleaved = p->interleaved;
  out.magnitude = p->magnitude > 0.0 ? static_cast<float>(p->magnitude) : 1.f;
  for (int i = 0; i < half; ++i) {
    double f;
    if (p->frequencies_h) {
      f = p->frequencies_h[i];
      if (!(std::fabs(f) <= pi)) return PKA_ERR_INVALID_ARG;
    } else {
      f = std::pow(p->base, -2.0 * i / p->rotary_dim);
      if (p->scaling == PKA_ROPE_LINEAR) f /= p->factor;
      if (p->scaling == PKA_ROPE_BY_PARTS) {
        const double turns = p->original_len * f / (2.0 * pi);
        double keep = (turns - p->low_rotations) / (p->high_rotations - p->low_rotations);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f = (1.0 - keep) * (f / p->factor) + keep * f;
      }
    }
    // |f| / 2 pi <= 1/2, so the fraction fits; a negative frequency is the
    // fraction's two's complement
    const uint64_t t = static_cast<uint64_t>(std::ldexp(std::fabs(f) / (2.0 * pi), 64));
    out.turns[i] = f < 0.0 ? 0 - t : t;
  }
  *rope = out;
  return PKA_OK;
}

pka_status pka_apply_rope(const pka_rope* rope, int32_t transpose, int32_t head_dim, int64_t rows,
                          const int32_t* positions_d, const void* q, int32_t q_heads,
                          int64_t q_row_stride, void* q_out, int64_t q_out_row_stride,
                          const void* k, int32_t k_heads, int64_t k_row_stride, void* k_out,
                          int64_t k_out_row_stride, void* stream) {
  if (!rope || (transpose != 0 && transpose != 1) || rows < 0 || q_heads < 0 || k_heads < 0)
    return PKA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKA_ERR_UNSUPPORTED;
  if (q_heads > pka::kMaxHeads || k_heads > pka::kMaxHeads || rows > pka::kMaxRows)
    return PKA_ERR_UNSUPPORTED;
  if (!pka::rope_valid(rope, head_dim)) return PKA_ERR_INVALID_ARG;
  if (rows == 0 || (q_heads == 0 && k_heads == 0)) return PKA_OK;
  if (!positions_d || pka::unaligned(positions_d)) return PKA_ERR_INVALID_ARG;
  if (q_heads > 0 && (!pka::rows_ok(q, q_row_stride, rows, q_heads, head_dim) ||
                      !pka::rows_ok(q_out, q_out_row_stride, rows, q_heads, head_dim) ||
                      !pka::out_ok(q, q_row_stride, q_out, q_out_row_stride)))
    return PKA_ERR_INVALID_ARG;
  if (k_heads > 0 && (!pka::rows_ok(k, k_row_stride, rows, k_heads, head_dim) ||
                      !pka::rows_ok(k_out, k_out_row_stride, rows, k_heads, head_dim) ||
                      !pka::out_ok(k, k_row_stride, k_out, k_out_row_stride)))
    return PKA_ERR_INVALID_ARG;
  pka::RopeArgs a{};
  pka::take_rope(&a, rope);
  if (transpose) a.sine_sign = -1.f;
  a.rows = rows;
  a.positions = positions_d;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.q_out_stride = q_out_row_stride;
  a.k_out_stride = k_out_row_stride;
  a.q_heads = q_heads;
  a.k_heads = k_heads;
  const cudaError_t e = pka::launch_any<false, pka::kBf16>(a, head_dim, rope->interleaved != 0,
                                                      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKA_OK : pka::cuda_failure(e, "rope launch");
}

pka_status pka_rope_append_paged_kv_cache(
    const pka_params* p, const pka_rope* rope, int32_t batch, int64_t nnz_new, const void* q,
    int64_t q_row_stride, void* q_out, const void* k_new, int64_t k_row_stride, const void* v_new,
    int64_t v_row_stride, const int32_t* positions_d, const int32_t* append_indptr_d,
    const int32_t* kv_indptr_d, const int32_t* kv_indices_d, const int32_t* last_page_len_d,
    void* k, void* v, int64_t page_stride, int64_t num_pool_pages, void* stream) {
  if (!pka::params_valid(p) || batch < 0 || nnz_new < 0 || num_pool_pages < 0)
    return PKA_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return PKA_ERR_UNSUPPORTED;
  if (p->kv_ragged || !pka::kv4_supported(*p)) return PKA_ERR_UNSUPPORTED;
  if (p->num_qo_heads > pka::kMaxHeads || p->num_kv_heads > pka::kMaxHeads ||
      nnz_new > pka::kMaxRows)
    return PKA_ERR_UNSUPPORTED;
  if (!pka::rope_valid(rope, p->head_dim)) return PKA_ERR_INVALID_ARG;
  if (nnz_new == 0 || batch == 0) return PKA_OK;
  if (!append_indptr_d || !kv_indptr_d || !kv_indices_d || !last_page_len_d || !k || !v ||
      page_stride <= 0)
    return PKA_ERR_INVALID_ARG;
  for (const int32_t* x :
       {positions_d, append_indptr_d, kv_indptr_d, kv_indices_d, last_page_len_d})
    if (pka::unaligned(x)) return PKA_ERR_INVALID_ARG;
  const bool f8 = p->kv_dtype == PKA_KV_FP8_E4M3;
  const int group = pka::kv4_group(p->kv_dtype);
  const uintptr_t mis = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  if ((mis & 15) || (page_stride & pka::kv_stride_mask(p->kv_dtype))) return PKA_ERR_INVALID_ARG;
  if (group && page_stride < pka::kv4_code_bytes(*p) + pka::kv4_word_bytes(*p))
    return PKA_ERR_INVALID_ARG;
  const int d = p->head_dim, hk = p->num_kv_heads;
  const int64_t q_out_stride = (int64_t)p->num_qo_heads * d;
  if (!pka::rows_ok(k_new, k_row_stride, nnz_new, hk, d) ||
      !pka::rows_ok(v_new, v_row_stride, nnz_new, hk, d))
    return PKA_ERR_INVALID_ARG;
  if (!q != !q_out) return PKA_ERR_INVALID_ARG;
  if (q && (!pka::rows_ok(q, q_row_stride, nnz_new, p->num_qo_heads, d) ||
            !pka::rows_ok(q_out, q_out_stride, nnz_new, p->num_qo_heads, d) ||
            !pka::out_ok(q, q_row_stride, q_out, q_out_stride)))
    return PKA_ERR_INVALID_ARG;
  pka::RopeArgs a{};
  pka::take_rope(&a, rope);
  a.rows = nnz_new;
  a.positions = positions_d;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_new);
  a.v = static_cast<const uint16_t*>(v_new);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.q_out_stride = q_out_stride;
  a.q_heads = q ? p->num_qo_heads : 0;
  a.k_heads = hk;
  a.batch = batch;
  a.append_indptr = append_indptr_d;
  a.kv_indptr = kv_indptr_d;
  a.kv_indices = kv_indices_d;
  a.last_page_len = last_page_len_d;
  a.k_pool = k;
  a.v_pool = v;
  a.page_stride = page_stride;
  a.num_pages = num_pool_pages;
  a.page_size = p->page_size;
  a.layout = p->layout;
  a.k_scale = p->k_scale > 0.f ? p->k_scale : 1.f;
  a.v_scale = p->v_scale > 0.f ? p->v_scale : 1.f;
  a.k_inv = pka::pow2_reciprocal(a.k_scale);
  a.v_inv = pka::pow2_reciprocal(a.v_scale);
  a.code_bytes = pka::kv4_code_bytes(*p);
  a.err = pka::device_error_word();
  const bool adjacent = rope->interleaved != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = group == 32    ? pka::launch_any<true, 32>(a, d, adjacent, st)
                        : group == 64  ? pka::launch_any<true, 64>(a, d, adjacent, st)
                        : group == 128 ? pka::launch_any<true, 128>(a, d, adjacent, st)
                        : f8           ? pka::launch_any<true, pka::kE4m3>(a, d, adjacent, st)
                                       : pka::launch_any<true, pka::kBf16>(a, d, adjacent, st);
  return e == cudaSuccess ? PKA_OK : pka::cuda_failure(e, "rope append launch");
}

}  // extern "C"
