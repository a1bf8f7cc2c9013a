// K/V held in 4 bits: the append that quantises, the read-back of cached rows
// (of pools of every type), and the f16 rows of the tensor-core launch.  The
// page format and the rounding rules are in pka_kv4.h.
#include "pka_cache.h"
#include "pka_device.cuh"
#include "pka_kv4.h"

namespace pka {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// A row's place in the pools.
struct Place {
  int32_t page;  // or one of these
  int32_t slot;
};
constexpr int32_t kBad = -1;   // outside its request's keys, or a page id out of range
constexpr int32_t kNone = -2;  // a row of no request
constexpr int32_t kZero = -3;  // a row of the scratch behind the last: zeros

// The place of logical position `pos` of request r.
__device__ __forceinline__ Place place_of(const KvRows& a, int r, int64_t pos) {
  Place p{kBad, 0};
  const int kv0 = a.kv_indptr[r], pages = a.kv_indptr[r + 1] - kv0;
  const int64_t kv_len = (int64_t)(pages - 1) * a.page_size + a.last_page_len[r];
  if (pos < 0 || pos >= kv_len) return p;
  const int64_t nth = pos <= UINT32_MAX ? (uint32_t)pos / (uint32_t)a.page_size
                                        : pos / a.page_size;
  p.page = a.kv_indices[kv0 + nth];
  p.slot = (int)(pos - nth * a.page_size);
  if (p.page < 0 || p.page >= a.num_pages) p.page = kBad;
  return p;
}

// The place of row `row` of a batch: a read's rows count from `begin`, an
// append's are its request's last.  A decode step's rows are one a request, so
// row r is tried as request r's first.
__device__ __forceinline__ Place row_place(const KvRows& a, int64_t row, bool append) {
  int r = (int)min(row, (int64_t)a.batch - 1);
  if (row < a.row_indptr[r] || row >= a.row_indptr[r + 1]) {
    if (row >= a.row_indptr[a.batch]) return Place{kNone, 0};
    int hi = a.batch - 1;  // the last request that starts at or before the row
    r = 0;
    while (r < hi) {
      const int mid = (int)(((int64_t)r + hi + 1) >> 1);
      if (a.row_indptr[mid] <= row) r = mid; else hi = mid - 1;
    }
  }
  int64_t pos = row - a.row_indptr[r];
  if (append) {
    const int pages = a.kv_indptr[r + 1] - a.kv_indptr[r];
    pos += (int64_t)(pages - 1) * a.page_size + a.last_page_len[r] -
           (a.row_indptr[r + 1] - a.row_indptr[r]);
  } else if (a.begin) {
    pos += a.begin[r];
  }
  return place_of(a, r, pos);
}

// The request of row `row`, or -1 for a row of none, found by a whole warp.
__device__ __forceinline__ int warp_request(const KvRows& a, int64_t row, int lane) {
  const int guess = (int)min(row, (int64_t)a.batch - 1);
  if (row >= a.row_indptr[guess] && row < a.row_indptr[guess + 1]) return guess;
  if (row >= a.row_indptr[a.batch]) return -1;
  return warp_find(a.row_indptr, a.batch, row, lane);
}

// How a call's rows are dealt to warps: a step is 256 elements of a row (8 a lane,
// one to four heads); a warp keeps one step, so that what its lanes' heads need is
// worked out once, and walks `rows` rows at a time, kAhead of them in flight.  Its
// lanes look up the places of all these rows at once, since a look-up is a chain of
// four or more dependent loads.
struct Deal {
  int steps;  // of a row
  int rows;
};
constexpr int kAhead = 4;

struct Walk {
  int step;
  int64_t row0, turn;  // the warp's first rows, and how far it goes on
  bool any;
  __device__ __forceinline__ Walk(const Deal& d) {
    const uint32_t warps = gridDim.x * 8, groups = warps / d.steps;
    const uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5), group = w / d.steps;
    step = (int)(w - group * d.steps);
    row0 = (int64_t)group * d.rows;
    turn = (int64_t)groups * d.rows;
    any = group < groups;
  }
};

// Where the rows of a slot lie in a page: `row` bytes a head, at slot * per_slot +
// head * per_head.
struct Rows {
  int32_t per_slot;
  int64_t per_head;
  __device__ __forceinline__ Rows(const KvRows& t, int row)
      : per_slot(t.layout == PKA_NHD ? t.heads * row : row),
        per_head(t.layout == PKA_NHD ? row : (int64_t)t.page_size * row) {}
};

__device__ __forceinline__ float word_step(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float word_origin(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

// The largest magnitude under a word, that of code 0 or of code 15; infinity where one
// of them is not finite or would not be in bf16.
__device__ __forceinline__ float word_bound(uint32_t w) {
  const float a = fabsf(word_origin(w)), b = fabsf(fmaf(15.f, word_step(w), word_origin(w)));
  constexpr float kPastBf16 = 0x1.ffp127f;
  return a < kPastBf16 && b < kPastBf16 ? fmaxf(a, b) : INFINITY;
}

// origin + step * c of the 8 codes c of a word, each pair as (even, odd).  A code
// becomes the float 2^23 + c by one byte permutation, and c by a subtraction;
// step * c is exact (8 by 4 bits), so the sum is rounded once.
__device__ __forceinline__ void values4(uint32_t codes, float step, float origin,
                                        float2 (&out)[4]) {
  const uint32_t even = codes & 0x0f0f0f0fu, odd = codes >> 4 & 0x0f0f0f0fu;
  const float2 s = make_float2(step, step), z = make_float2(origin, origin);
  const float2 less = make_float2(-8388608.f, -8388608.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t sel = 0x7540u + i;  // code i, 0, 0, 0x4b
    const float2 c = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(even, 0x4b000000u, sel)),
                                            __uint_as_float(__byte_perm(odd, 0x4b000000u, sel))),
                                less);
    out[i] = __ffma2_rn(s, c, z);
  }
}

// ---------------------------------------------------------------------------
// Append.  A row's steps are K's heads, then V's.  The lanes of a group exchange
// its least and greatest element (exact in bf16, both in one word: the least and
// the negated greatest under one minimum), then every lane makes its 8 codes, one
// 32-bit store.
//   On long appends nothing is full (9,101 rows of 8 heads of 128: issue slots 58%,
// DRAM 28%): each four rows are asked for when the four before are stored.  A decode
// step waits for the dependent look-ups of request, page and slot.
// ---------------------------------------------------------------------------

struct Append4Args {
  KvRows rows;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint8_t* k;
  uint8_t* v;
  int64_t code_bytes;  // of a page
  Deal deal;
};

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D, int GR>
__global__ void __launch_bounds__(256) append4_kernel(const __grid_constant__ Append4Args a) {
  constexpr int LPH = D / 8;      // lanes of a head
  constexpr int HPS = 32 / LPH;   // heads of a step
  constexpr int LPG = GR / 8;     // lanes of a group
  constexpr int G = D / GR;
  const int lane = threadIdx.x & 31;
  const int piece = lane % LPH;
  const KvRows& t = a.rows;
  const Walk walk(a.deal);
  if (!walk.any) return;
  const int hk = t.heads, h = walk.step * HPS + lane / LPH;
  const bool have = h < 2 * hk, is_v = h >= hk;
  const int hh = !have ? 0 : is_v ? h - hk : h;
  const Rows codes(t, D / 2), words(t, 4 * G);
  const uint16_t* const src = (is_v ? a.v_new : a.k_new) + hh * D + piece * 8;
  uint8_t* const pool = is_v ? a.v : a.k;
  uint8_t* const code_pool = pool + hh * codes.per_head + piece * 4;
  uint8_t* const word_pool = pool + a.code_bytes + hh * words.per_head + piece / LPG * 4;
  const int64_t row_elems = (int64_t)hk * D;
  for (int64_t row0 = walk.row0; row0 < t.rows; row0 += walk.turn) {
    const int n = (int)min((int64_t)a.deal.rows, t.rows - row0);
    uint4 x[kAhead];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (have && i0 + u < n)
          x[u] = *reinterpret_cast<const uint4*>(src + (row0 + i0 + u) * row_elems);
      }
    };
    load(0);  // before the look-ups, which take longer
    Place mine{kNone, 0};
    if (lane < n) mine = row_place(t, row0 + lane, true);
    if (mine.page == kBad) note_error(t.err, PKA_ERR_METADATA);
    for (int i0 = 0;;) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i0 + u >= n) break;
        const int32_t page = __shfl_sync(kAll, mine.page, i0 + u);
        const int32_t slot = __shfl_sync(kAll, mine.slot, i0 + u);
        // {least, -greatest} of the lane's 8 elements, then of its group
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        const uint32_t lo = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
        const uint32_t hi = min2_nan(min2_nan(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                                     min2_nan(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
        uint32_t both = min2_nan(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
        for (int off = 1; off < LPG; off <<= 1)
          both = min2_nan(both, __shfl_xor_sync(kAll, both, off));
        if (!have || page < 0) continue;
        const Group4 g = group4(__uint_as_float(both << 16),
                                -__uint_as_float(both & 0xffff0000u));
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = bf16x2_to_float2(w[i]);
          f[2 * i] = v.x;
          f[2 * i + 1] = v.y;
        }
        const int64_t at = (int64_t)page * t.page_stride;
        *reinterpret_cast<uint32_t*>(code_pool + at + (int64_t)slot * codes.per_slot) =
            codes4<false>(f, g);
        if (piece % LPG == 0)
          *reinterpret_cast<uint32_t*>(word_pool + at + (int64_t)slot * words.per_slot) = g.word;
      }
      i0 += kAhead;
      if (i0 >= n) break;
      load(i0);
    }
  }
}

// ---------------------------------------------------------------------------
// Read-back.  A row's steps are the heads of the outputs asked for, K's first; a
// lane takes 4 bytes of codes, 8 of e4m3 or 16 of bf16 a step and writes 16.  Here
// a warp takes a row (or a part of its steps), eight steps in flight, and looks it
// up alone: with most of its bytes in the rows that go out, 2 an element whatever they
// came in, it is faster where a warp writes K's and V's whole rows (walking rows as
// above, 40,710 rows of 8 heads of 128: 40.9 us for 39.9 out of 4-bit pools, issue
// slots 70% there, 53.8 for 43.7 out of e4m3 ones).
// ---------------------------------------------------------------------------

struct ReadArgs {
  KvRows rows;
  const uint8_t* k;
  const uint8_t* v;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t code_bytes;
  float k_scale, v_scale;
  int steps_per_part;
};

constexpr int kReadSteps = 8;  // in flight

// Element type of the pools: 0 bf16, 1 e4m3, otherwise 4 bits in groups of so many.
template <int D, int KIND>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int LPH = D / 8, HPS = 32 / LPH;
  constexpr int IN = KIND == 0 ? 16 : KIND == 1 ? 8 : 4;  // bytes a lane takes a step
  constexpr int G = KIND > 1 ? D / KIND : 1;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, piece = lane % LPH;
  const KvRows& t = a.rows;
  const int hk = t.heads;
  const Rows codes(t, LPH * IN), words(t, 4 * G);
  // the outputs asked for, as one list of heads
  const int k_end = a.k_out ? hk : 0, heads = k_end + (a.v_out ? hk : 0);
  const int h0 = blockIdx.y * a.steps_per_part * HPS;
  const int h1 = min(heads, h0 + a.steps_per_part * HPS);
  for (int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < t.rows; row += gridDim.x * 8ll) {
    const int r = warp_request(t, row, lane);
    if (r < 0) break;  // this row and those behind it belong to no request
    const Place p = place_of(t, r, (t.begin ? t.begin[r] : 0ll) + (row - t.row_indptr[r]));
    if (p.page < 0) {
      if (lane == 0) note_error(t.err, PKA_ERR_METADATA);
      continue;
    }
    const int64_t page = (int64_t)p.page * t.page_stride * (KIND == 0 ? 2 : 1);
    // 64 bits: pages of bf16 and e4m3 pools may be larger than 2 GB
    const int64_t code_at = page + (int64_t)p.slot * codes.per_slot + piece * IN;
    const int64_t word_at = page + a.code_bytes + (int64_t)p.slot * words.per_slot +
                            piece / (KIND > 1 ? KIND / 8 : 1) * 4;
    for (int hb = h0; hb < h1; hb += kReadSteps * HPS) {
      uint4 x[kReadSteps];
#pragma unroll
      for (int s = 0; s < kReadSteps; ++s) {
        const int h = hb + s * HPS + sub;
        if (h >= h1) continue;
        const int hh = h < k_end ? h : h - k_end;
        const uint8_t* pool = h < k_end ? a.k : a.v;
        const uint8_t* src = pool + code_at + hh * codes.per_head;
        if constexpr (KIND == 0) {
          x[s] = *reinterpret_cast<const uint4*>(src);
        } else if constexpr (KIND == 1) {
          const uint2 c = *reinterpret_cast<const uint2*>(src);
          x[s].x = c.x;
          x[s].y = c.y;
        } else {
          x[s].x = *reinterpret_cast<const uint32_t*>(src);
          x[s].y = *reinterpret_cast<const uint32_t*>(pool + word_at + hh * words.per_head);
        }
      }
#pragma unroll
      for (int s = 0; s < kReadSteps; ++s) {
        const int h = hb + s * HPS + sub;
        if (h >= h1) continue;
        const bool is_k = h < k_end;
        uint32_t out[4];
        if constexpr (KIND == 0) {
          out[0] = x[s].x;
          out[1] = x[s].y;
          out[2] = x[s].z;
          out[3] = x[s].w;
        } else if constexpr (KIND == 1) {
          const float scale = is_k ? a.k_scale : a.v_scale;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t two = (i < 2 ? x[s].x : x[s].y) >> (16 * (i & 1)) & 0xffffu;
            uint32_t h2;
            asm("{\n .reg .b16 c;\n cvt.u16.u32 c, %1;\n cvt.rn.f16x2.e4m3x2 %0, c;\n}"
                : "=r"(h2)
                : "r"(two));
            float lo, hi;
            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n"
                " cvt.f32.f16 %1, h;\n}"
                : "=f"(lo), "=f"(hi)
                : "r"(h2));
            out[i] = float2_to_bf16x2(lo * scale, hi * scale);
          }
        } else {
          float2 v[4];
          values4(x[s].x, word_step(x[s].y), word_origin(x[s].y), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = float2_to_bf16x2(v[i].x, v[i].y);
        }
        uint16_t* dst = (is_k ? a.k_out : a.v_out) +
                        (row * hk + (is_k ? h : h - k_end)) * (int64_t)D + piece * 8;
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(out[0], out[1], out[2], out[3]));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The f16 rows of a launch on the tensor cores (F16Stage), in two launches: Q
// and, from the words alone, bounds of the largest magnitude in each kv head of
// each unit, and of the smallest of its groups, then K and V with their scales.  The
// words are read twice: 16, 32 or 64 times as many bytes go out in groups of 32, 64 or
// 128.  40,710 keys of 8 heads of 128 and 9,101 rows of Q take 26 and 44 us, DRAM 53%
// and 54%, issue slots 54% and 62%: neither is full, loads wait for the stores before.
// ---------------------------------------------------------------------------

// The rows of this plan: in graph mode what the device image says.
__device__ __forceinline__ int64_t staged_rows(const KvRows& t, int* units) {
  *units = t.num_units;
  if (!t.counts) return t.rows;
  *units = min(max(t.counts[0], 0), t.num_units);
  return *units > 0 ? min((int64_t)max(t.counts[2], 0), t.rows) : 0;
}

// Page and slot of scratch row `row`, and its unit (the last that starts at or before it).
__device__ __forceinline__ Place unit_place(const KvRows& t, int units, int64_t row,
                                            int* unit) {
  int lo = 0, hi = units - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.units[mid].dst_row0 <= row) lo = mid; else hi = mid - 1;
  }
  *unit = lo;
  const PkaDequantUnit u = t.units[lo];
  const uint32_t j = (uint32_t)(row - u.dst_row0), nth = j / (uint32_t)t.page_size;
  Place p;
  p.page = t.kv_indices[u.kv_base + nth];
  p.slot = (int)(j - nth * (uint32_t)t.page_size);
  return p;
}

// The bounds of one kv head in all units: block `block_id` of `blocks` takes its rows,
// 256 rows at a time, most often of one unit: then the block adds to its bounds at
// once, otherwise each warp for the lanes of a unit.
template <int G>
__device__ __forceinline__ void range_of_words(const F16Stage& a, int64_t code_bytes, int head,
                                               unsigned block_id, unsigned blocks) {
  const KvRows& t = a.rows;
  int units;
  const int64_t rows = staged_rows(t, &units);
  const int lane = threadIdx.x & 31;
  __shared__ uint32_t of_block[4];
  __shared__ int block_unit;
  for (int64_t row0 = block_id * 256ll; row0 < rows; row0 += blocks * 256ll) {
    const int64_t row = row0 + threadIdx.x;
    uint32_t most[4] = {0u, 0u, 0u, 0u};  // as in Kv4Range
    int unit = -1;
    if (row < rows) {
      const Place p = unit_place(t, units, row, &unit);
      const int64_t idx = t.layout == PKA_NHD ? (int64_t)p.slot * t.heads + head
                                              : (int64_t)head * t.page_size + p.slot;
      const int64_t at = (int64_t)p.page * t.page_stride + code_bytes + idx * (4 * G);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>((kv ? a.v : a.k) + at);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float b = word_bound(w[g]);
          if (!(b > 0.f && b < INFINITY)) continue;
          most[kv] = max(most[kv], __float_as_uint(b));
          most[2 + kv] = max(most[2 + kv], ~__float_as_uint(b));
        }
      }
    }
    if (threadIdx.x == 0) block_unit = unit;
    if (threadIdx.x < 4) of_block[threadIdx.x] = 0;
    __syncthreads();
    const bool one = __syncthreads_and(unit == block_unit || unit < 0);
    const unsigned with = one ? kAll : __match_any_sync(kAll, unit);
    uint32_t* const range =
        reinterpret_cast<uint32_t*>(a.kv_range + (int64_t)max(unit, 0) * t.heads + head);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = __reduce_max_sync(with, most[i]);  // 0 of lanes without a row
      if (m && lane == __ffs(with) - 1) atomicMax(one ? of_block + i : range + i, m);
    }
    __syncthreads();
    if (one && threadIdx.x < 4 && of_block[threadIdx.x])
      atomicMax(range + threadIdx.x, of_block[threadIdx.x]);
    __syncthreads();
  }
}

__device__ __forceinline__ uint32_t float2_to_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// 8 codes under a step and an origin -> f16, or bf16.
__device__ __forceinline__ uint4 codes_to_16(uint32_t codes, float step, float origin,
                                             bool bf16) {
  float2 v[4];
  values4(codes, step, origin, v);
  if (bf16)
    return make_uint4(float2_to_bf16x2(v[0].x, v[0].y), float2_to_bf16x2(v[1].x, v[1].y),
                      float2_to_bf16x2(v[2].x, v[2].y), float2_to_bf16x2(v[3].x, v[3].y));
  return make_uint4(float2_to_f16x2(v[0].x, v[0].y), float2_to_f16x2(v[1].x, v[1].y),
                    float2_to_f16x2(v[2].x, v[2].y), float2_to_f16x2(v[3].x, v[3].y));
}

// A warp's rows as above, K and V of a head together.  A key whose V is not finite in
// a group gets zeros there and NaN in K instead: the rows that see it become NaN, and
// the others, whose probability of it is 0, do not (0 * NaN in the P V product
// would reach every row of a tile).  For the same reason the up to 127 rows behind
// the last one that a tile may read, old ones of another plan in graph mode, become
// zeros.
template <int D, int GR>
__global__ void __launch_bounds__(256)
    stage_kernel(const __grid_constant__ F16Stage a, const int64_t code_bytes, const Deal deal) {
  constexpr int LPH = D / 8, HPS = 32 / LPH, G = D / GR, LPG = GR / 8;
  const int lane = threadIdx.x & 31;
  const int piece = lane % LPH;
  const KvRows& t = a.rows;
  const Walk walk(deal);
  if (!walk.any) return;
  const int hk = t.heads, h = walk.step * HPS + lane / LPH;
  const bool have = h < hk;
  const int hh = have ? h : 0;
  const Rows codes(t, D / 2), words(t, 4 * G);
  const int64_t code_off = hh * codes.per_head + piece * 4;
  const int64_t word_off = code_bytes + hh * words.per_head + piece / LPG * 4;
  float ku = 0.f, vu = 0.f;  // the scales of the lane's head in unit `scaled`
  bool wide = false;
  int scaled = -1;
  const int64_t row_elems = (int64_t)hk * D, out_off = hh * D + piece * 8;
  int units;
  const int64_t rows = staged_rows(t, &units), end = min(rows + 127, t.rows);
  for (int64_t row0 = walk.row0; row0 < end; row0 += walk.turn) {
    const int n = (int)min((int64_t)deal.rows, end - row0);
    Place mine{kZero, 0};
    int my_unit = 0;
    if (lane < n && row0 + lane < rows) mine = unit_place(t, units, row0 + lane, &my_unit);
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      uint32_t kc[kAhead], vc[kAhead], kw[kAhead], vw[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int32_t page = __shfl_sync(kAll, mine.page, (i0 + u) & 31);
        const int32_t slot = __shfl_sync(kAll, mine.slot, (i0 + u) & 31);
        kc[u] = vc[u] = kw[u] = vw[u] = 0u;  // zeros under a step and an origin of 0
        if (!have || i0 + u >= n || page == kZero) continue;
        const int64_t at = (int64_t)page * t.page_stride;
        const int64_t c = at + (int64_t)slot * codes.per_slot + code_off;
        const int64_t w = at + (int64_t)slot * words.per_slot + word_off;
        kc[u] = *reinterpret_cast<const uint32_t*>(a.k + c);
        vc[u] = *reinterpret_cast<const uint32_t*>(a.v + c);
        kw[u] = *reinterpret_cast<const uint32_t*>(a.k + w);
        vw[u] = *reinterpret_cast<const uint32_t*>(a.v + w);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int unit = __shfl_sync(kAll, my_unit, (i0 + u) & 31);
        if (!have || i0 + u >= n) continue;
        if (unit != scaled) {
          const Kv4Range r = a.kv_range[(int64_t)unit * hk + hh];
          wide = f16_too_wide(r);
          ku = wide ? 1.f : f16_up(r.x);
          vu = wide ? 1.f : f16_up(r.y);
          scaled = unit;
        }
        uint4 k = codes_to_16(kc[u], word_step(kw[u]) * ku, word_origin(kw[u]) * ku, wide);
        uint4 v = codes_to_16(vc[u], word_step(vw[u]) * vu, word_origin(vw[u]) * vu, wide);
        if (!(word_bound(vw[u]) < INFINITY)) {
          k = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);  // NaN in both
          v = make_uint4(0u, 0u, 0u, 0u);
        }
        const int64_t at = (row0 + i0 + u) * row_elems + out_off;
        *reinterpret_cast<uint4*>(a.k16 + at) = k;
        *reinterpret_cast<uint4*>(a.v16 + at) = v;
      }
    }
  }
}

// The first word_blocks blocks take the words, kv head by kv head; the others Q: D
// / 8 lanes a (row, head), 8 elements a lane.
template <int D, int G>
__global__ void __launch_bounds__(256)
    stage_q_kernel(const __grid_constant__ F16Stage a, const int64_t code_bytes,
                   const unsigned word_blocks) {
  constexpr int LPH = D / 8;
  if (blockIdx.x < word_blocks) {
    const unsigned heads = a.rows.heads;
    range_of_words<G>(a, code_bytes, blockIdx.x % heads, blockIdx.x / heads, word_blocks / heads);
    return;
  }
  const int64_t total = a.q_rows * a.q_heads * LPH, turn = (gridDim.x - word_blocks) * 256ll;
  // whole warps: 32 is a multiple of LPH and the rounded-up lanes only shuffle
  for (int64_t at = (blockIdx.x - word_blocks) * 256ll + threadIdx.x;
       at - (threadIdx.x & 31) < total; at += turn) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (at < total) x = reinterpret_cast<const uint4*>(a.q)[at];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float most = 0.f, f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf16x2_to_float2(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
      most = fmaxf(most, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
#pragma unroll
    for (int off = 1; off < LPH; off <<= 1)
      most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
    if (at >= total) continue;
    const float up = f16_up(__float_as_uint(most));
    reinterpret_cast<uint4*>(a.q16)[at] =
        make_uint4(float2_to_f16x2(f[0] * up, f[1] * up), float2_to_f16x2(f[2] * up, f[3] * up),
                   float2_to_f16x2(f[4] * up, f[5] * up), float2_to_f16x2(f[6] * up, f[7] * up));
    if (at % LPH == 0) a.q_down[at / LPH] = f16_down(__float_as_uint(most));
  }
}

// Rows a warp takes at a time: up to 16, as many as leave 24 warps an SM (an
// append of 9,101 rows of 8 heads of 128 with its read-back, in us, in groups of 32
// and of 128: at most four rows 26.0 and 26.2, eight 24.2 and 24.7, sixteen 23.6 and
// 24.2, thirty-two 23.6 and 24.2).
Deal deal_of(int64_t rows, int steps) {
  const int sms = current_device_sms();
  const int64_t per = rows * steps / (24 * (int64_t)(sms > 0 ? sms : 1));
  const int n = per < 1 ? 1 : per > 16 ? 16 : (int)per;
  return {steps, n < kAhead ? n : n / kAhead * kAhead};
}

// Whole turns of all steps, at most 2^20 blocks.
unsigned blocks_of(int64_t rows, const Deal& d) {
  const int64_t groups = (rows + d.rows - 1) / d.rows;
  const int64_t blocks = (groups * d.steps + 7) / 8, most = (int64_t)1 << 20;
  return (unsigned)(blocks < 1 ? 1 : blocks > most ? most : blocks);
}

template <int D, int KIND>
cudaError_t launch_read_t(const ReadArgs& args, cudaStream_t stream) {
  ReadArgs a = args;
  constexpr int HPS = 256 / D;
  const int heads = a.rows.heads * ((a.k_out ? 1 : 0) + (a.v_out ? 1 : 0));
  const int steps = (heads + HPS - 1) / HPS;
  // enough warps first (16 an SM, for which a row is split), then whole rows
  const int sms = current_device_sms();
  const int64_t warps = 16 * (int64_t)(sms > 0 ? sms : 1), rows = a.rows.rows;
  const int64_t per = (rows * steps + warps - 1) / warps;
  int parts = per >= kReadSteps ? 1 : (steps + (int)per - 1) / (int)per;
  if (parts == 1) parts = (steps + kReadSteps - 1) / kReadSteps;
  a.steps_per_part = (steps + parts - 1) / parts;
  const int64_t blocks = (rows + 7) / 8, most = (int64_t)1 << 24;
  const dim3 grid((unsigned)(blocks > most ? most : blocks),
                  (unsigned)((steps + a.steps_per_part - 1) / a.steps_per_part));
  read_kernel<D, KIND><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int GR>
cudaError_t launch_append_t(const Append4Args& args, cudaStream_t stream) {
  Append4Args a = args;
  constexpr int HPS = 256 / D;
  const int steps = (2 * a.rows.heads + HPS - 1) / HPS;
  a.deal = deal_of(a.rows.rows, steps);
  append4_kernel<D, GR><<<blocks_of(a.rows.rows, a.deal), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

unsigned blocks_of(int64_t work, int per_block, int per_sm) {
  const int sms = current_device_sms();
  const int64_t most = (int64_t)per_sm * (sms > 0 ? sms : 1);
  const int64_t b = (work + per_block - 1) / per_block;
  return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}

template <int D, int GR>
cudaError_t launch_stage_t(const F16Stage& a, cudaStream_t stream) {
  constexpr int HPS = 256 / D;
  const KvRows& t = a.rows;
  const int64_t code_bytes = (int64_t)t.page_size * t.heads * (D / 2);
  cudaError_t e = cudaMemsetAsync(
      a.kv_range, 0, (size_t)t.num_units * t.heads * sizeof(*a.kv_range), stream);
  if (e != cudaSuccess) return e;
  // the words of all heads beside Q's rows: neither waits for the other
  const unsigned word_blocks = blocks_of(t.rows, 256, 1) * (unsigned)t.heads;
  const unsigned q_blocks = blocks_of(a.q_rows * a.q_heads * (D / 8), 256, 32);
  stage_q_kernel<D, D / GR>
      <<<word_blocks + q_blocks, 256, 0, stream>>>(a, code_bytes, word_blocks);
  const int steps = (t.heads + HPS - 1) / HPS;
  const Deal d = deal_of(t.rows, steps);
  stage_kernel<D, GR><<<blocks_of(t.rows, d), 256, 0, stream>>>(a, code_bytes, d);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_stage_f16(const F16Stage& s, int head_dim, int group, cudaStream_t stream) {
  if (head_dim == 128)
    return group == 32   ? launch_stage_t<128, 32>(s, stream)
           : group == 64 ? launch_stage_t<128, 64>(s, stream)
                         : launch_stage_t<128, 128>(s, stream);
  return group == 32 ? launch_stage_t<64, 32>(s, stream) : launch_stage_t<64, 64>(s, stream);
}

cudaError_t launch_append4(const KvRows& r, int head_dim, int group, const uint16_t* k_new,
                           const uint16_t* v_new, uint8_t* k, uint8_t* v, cudaStream_t stream) {
  Append4Args a{};
  a.rows = r;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k = k;
  a.v = v;
  a.code_bytes = (int64_t)r.page_size * r.heads * (head_dim / 2);
  if (head_dim == 128)
    return group == 32   ? launch_append_t<128, 32>(a, stream)
           : group == 64 ? launch_append_t<128, 64>(a, stream)
                         : launch_append_t<128, 128>(a, stream);
  return group == 32 ? launch_append_t<64, 32>(a, stream) : launch_append_t<64, 64>(a, stream);
}

cudaError_t launch_read(const KvRows& r, int kv_dtype, int head_dim, float k_scale, float v_scale,
                        const void* k, const void* v, uint16_t* k_out, uint16_t* v_out,
                        cudaStream_t stream) {
  if (r.rows <= 0 || (!k_out && !v_out)) return cudaSuccess;
  ReadArgs a{};
  a.rows = r;
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.k_out = k_out;
  a.v_out = v_out;
  a.code_bytes = (int64_t)r.page_size * r.heads * (head_dim / 2);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int group = kv4_group(kv_dtype);
  if (head_dim == 128)
    return kv_dtype == PKA_KV_BF16       ? launch_read_t<128, 0>(a, stream)
           : kv_dtype == PKA_KV_FP8_E4M3 ? launch_read_t<128, 1>(a, stream)
           : group == 32                 ? launch_read_t<128, 32>(a, stream)
           : group == 64                 ? launch_read_t<128, 64>(a, stream)
                                         : launch_read_t<128, 128>(a, stream);
  return kv_dtype == PKA_KV_BF16       ? launch_read_t<64, 0>(a, stream)
         : kv_dtype == PKA_KV_FP8_E4M3 ? launch_read_t<64, 1>(a, stream)
         : group == 32                 ? launch_read_t<64, 32>(a, stream)
                                       : launch_read_t<64, 64>(a, stream);
}

}  // namespace pka
