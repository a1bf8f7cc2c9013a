// Decode attention (one query row per request) over a cache held in 4 bits.
//
// The work list, the splits and the join of their pieces are the decode
// kernel's (decode.cu); what differs is how a key's bytes become operands.
// With origin z and step s of a key's group of elements and q the query,
//   score = scale * sum over groups (s * (q . c) + z * sum(q)),
//   o     = (sum p * s * c + sum p * z) / sum p,
// so the codes c go to the tensor cores as they are and the words are applied
// to scores and probabilities, one product a key and group instead of one an
// element.
//
// A code becomes an f16 operand by one AND: four bits at the bottom of an f16
// are the subnormal c * 2^-24, and at bits 4..7 16 c * 2^-24, exact and taken
// at full rate by the MMA.  So a word of 8 codes takes one shift and four ANDs;
// the 2^24 and the 16 are taken back in Q (K's products) and at the end (V's).
// An OR with 1024's or 128's exponent would leave an offset of 1024 or 128 in
// every product, whose cancellation costs the statistics 2^-17 or so.
//   Q is scaled to f16 by a power of two per head that puts its largest element
// in [2^14, 2^15): bf16 values down to 2^-27 of it stay exact.
//   The second 8 keys of each 16 take V's codes from above, as 15 - c under -P,
// with 15 of the same rounded P beside them: an output's sum then runs up by as much
// as down.  With c alone all its terms are positive, it grows with the keys, and so
// does what each MMA cuts off of it: 2% of an output that is the mean of 160,000
// values.
//   P goes to f16 with V's step in it, 11 bits against the 8 of bf16: p * s times a
// power of two of its own for each head and group, which puts the largest p * s seen
// at 2^11 (a larger one may pass it by 2^4 before the state is rescaled).  So the 11
// bits reach down to 2^-25 of the largest p * s of the group, however the groups of a
// head and the keys differ in size (one power of two for all groups of a head took 6%
// of outputs whose group's steps were 2^-24 of another's).
//
// Warps: each kv head of the CTA is served by several warps that take the item's
// 32-key tiles in turn, so 16 warps work whatever the head count; their states
// meet in shared memory at the end of an item.  Every warp brings its own tiles
// in with cp.async, two stages ahead, and waits only for its own copies: there
// is no producer, no barrier wait that could run out, and any page size, layout
// and stride is one address a key.
//   A CTA fills an SM (16 warps of 128 registers), at most one is launched on each.
//
// What bounds it: long rows run at 6.6 TB/s with groups of 128 of a head of 128
// (25 ns a key of 8 heads on an SM), 6.4 with 64 and 4.7 with 32, where two or four
// words a key instead of one are applied to the scores (and, with 32, registers spill);
// D = 64 at 5.2 and 4.8 (groups of 64 and 32), pages of one key at 4.3, one kv head a
// CTA at 4.7.  Groups of 128 are bound by memory, the others by the warps' chains of
// MMA, vote and exponential (issue slots 40 to 61% used, 16 warps).  An item's start and
// end are 3 us, the kernel's about 10: the first copies, four look-ups deep, the first
// tile's rescaling (0.3 us, most of it instructions on their way), and at the end the
// states' meeting, the write, the count and the join, each a round trip.
#include "pka_device.cuh"
#include "pka_kv4.h"

namespace pka {
namespace {

constexpr int kTile = 32;        // keys of a warp's step
// More warps have too few registers: heads of 64 in 24 warps of 80 take 31.8 us for 28.2
// with 16 (64 requests, groups of 64), and 122.5 for 108.8 (8 of 32K to 128K keys).
constexpr int kMaxWarps = 16;
// Tiles a warp has on their way.  More do not help: 37 requests over a token pool of
// heads of 64 take 28.1 us with two, 28.4 with three, 28.8 with four.
constexpr int kStages = 2;
// p is 2^-kBelow at the running maximum: its products with values up to 2^115 and
// their sums over a row stay finite.  The state is rescaled when the maximum grows by
// more than 2^kRescale (as in decode.cu).
constexpr float kBelow = 12.0f;
constexpr float kRescale = 8.0f;
// The largest P after a rescaling, and the largest that goes on without one (f16 bits).
constexpr int kHeadroom = 11;
constexpr uint32_t kMostP = 0x7800u;  // 2^15
// Steps below it count as it for their group's power of two, which stays finite.
constexpr float kLeastStep = 0x1p-100f;

template <int D, int GR>
struct Shape {
  static constexpr int G = D / GR;        // groups of a head
  static constexpr int CH = D / 32;       // 16-byte chunks of a row of codes
  static constexpr int ROW = D / 2;       // bytes of a row of codes
  static constexpr int MT = D / 16;       // 16-row blocks of V^T
  static constexpr int DL = GR / 8;       // elements of a group that a lane's V rows hold
  static constexpr int CODES = kTile * ROW;
  static constexpr int WORDS = kTile * G * 4;
  static constexpr int STAGE = 2 * (CODES + WORDS);  // K codes, V codes, K words, V words
  static constexpr int STATE = MT * 4 + 4 + 2 * G;   // floats of a lane's state
  static constexpr int SLOT = STATE * 128;           // bytes of a warp's state
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The larger of each half; NaN only of two.
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 2^n for a whole n up to 127; 0 below -126.
__device__ __forceinline__ float pow2(float n) {
  return n < -126.f ? 0.f : __uint_as_float((uint32_t)((int)n + 127) << 23);
}
// 1 / w for a power of two w in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float w) {
  return __uint_as_float(0x7f000000u - __float_as_uint(w));
}
// Keeps 2^-n, and 2^24 2^n, normal numbers.
__device__ __forceinline__ float clamp_log(float n) { return fminf(fmaxf(n, -126.f), 100.f); }
__device__ __forceinline__ float pow2_log(float w) {
  return (float)((int)(__float_as_uint(w) >> 23) - 127);
}

// d += a . b for a 16x16 (row) and 16x8 (col) f16 fragment pair.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t float2_to_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) {
  float2 f;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(x));
  return f;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Copy BYTES (4, 8 or 16) to shared memory, or zeros where `there` is false.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  const int n = there ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(n)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// The G words of a key.
template <int G>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[G]) {
  if constexpr (G == 1) {
    w[0] = lds32(addr);
  } else if constexpr (G == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  }
}

__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float origin_of(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

struct Decode4Args {
  AttnArgs a;
  int64_t code_bytes;  // of a page
  int64_t v_from_k;    // V's pool, seen from K's
  int splits;          // warps of a kv head
};

// Rows are held as they lie in the page, 16-byte chunk j of key i at chunk
// j ^ chunk_swap(i).  K's words are read by 8 keys (lane / 4) at a time and V's
// by 4 keys (lane % 4), and both meet every bank once.
template <int D>
__device__ __forceinline__ int chunk_swap(int key) {
  return D == 128 ? (key & 2) | (key >> 2 & 1) : key >> 2 & 1;
}

// The largest and the sum over the lanes that hold one head's keys.
template <bool HALF, int N>
__device__ __forceinline__ void max_keys(float2 (&x)[N]) {
#pragma unroll
  for (int off = HALF ? 2 : 4; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i].x = fmaxf(x[i].x, __shfl_xor_sync(0xffffffffu, x[i].x, off));
      x[i].y = fmaxf(x[i].y, __shfl_xor_sync(0xffffffffu, x[i].y, off));
    }
  }
}
template <bool HALF>
__device__ __forceinline__ float sum_keys(float x) {
#pragma unroll
  for (int off = HALF ? 2 : 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Merge the pieces of a split (request, kv head) for its qo heads first, first +
// step, ...: with b_k the pieces' base-2 statistics, m = max b_k and s = sum
// 2^(b_k - m), o = sum (2^(b_k - m) / s) o_k and lse = m + log2 s; pieces with b_k
// = -inf carry no weight, and if all are empty o = 0 and lse = -inf.  Lane k takes
// the statistics of pieces k, k + 32, ..; then the rows come in, from other SMs
// through L2 (.cg).  Two heads at a time, R rows of each in flight: the call is a
// chain of such round trips at the end of the kernel.  With R = 8 it is shorter, but
// its registers are taken from the main loop's (64 requests 45.1 us, 41.2 with 4).
template <int D>
__device__ __noinline__ void join_heads(const AttnArgs& a, const PkaDecodeJoin j, int row,
                                        int head0, int group, int first, int step, int lane) {
  constexpr int PER = D / 32, R = 4;
  for (int h0 = first; h0 < group; h0 += 2 * step) {
    const int heads[2] = {h0, h0 + step < group ? h0 + step : h0};
    auto stat = [&](int k, int h) {
      return k < j.nslots ? __ldcg(a.part_lse + j.rec_first + (int64_t)k * j.rec_stride + h)
                          : -INFINITY;
    };
    float b0[2], m[2], sum[2], acc[2][PER];
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = b0[i] = stat(lane, heads[i]);
    for (int k = lane + 32; k < j.nslots; k += 32)
#pragma unroll
      for (int i = 0; i < 2; ++i) m[i] = fmaxf(m[i], stat(k, heads[i]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
      if (m[i] == -INFINITY) m[i] = 0.f;
      sum[i] = exp2f(b0[i] - m[i]);
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[i][e] = 0.f;
    }
    for (int base = 0; base < j.nslots; base += 32) {
      float weight[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        weight[i] = exp2f((base ? stat(base + lane, heads[i]) : b0[i]) - m[i]);
        if (base) sum[i] += weight[i];
      }
      const int n = min(32, j.nslots - base);
      for (int k0 = 0; k0 < n; k0 += R) {
        float x[2][R][PER];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int q = 0; q < R; ++q) {
#pragma unroll
            for (int e = 0; e < PER; ++e) x[i][q][e] = 0.f;
            const float* src =
                a.part_o + lane * PER +
                (j.rec_first + (int64_t)(base + k0 + q) * j.rec_stride + heads[i]) * D;
            if (k0 + q < n) {
              if constexpr (PER == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                x[i][q][0] = v.x, x[i][q][1] = v.y, x[i][q][2] = v.z, x[i][q][3] = v.w;
              } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                x[i][q][0] = v.x, x[i][q][1] = v.y;
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int q = 0; q < R; ++q) {  // past the last piece: weight 0 of zeros
            const float w = __shfl_sync(0xffffffffu, weight[i], (k0 + q) & 31);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[i][e] = fmaf(w, x[i][q][e], acc[i][e]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
      if (i && heads[1] == heads[0]) continue;
      const bool none = sum[i] == 0.f;
      const float inv = none ? 0.f : 1.f / sum[i];
      const int64_t out = (int64_t)row * a.num_qo_heads + head0 + heads[i];
      uint16_t* dst = a.o + out * D + lane * PER;
      if constexpr (PER == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(float2_to_bf16x2(acc[i][0] * inv, acc[i][1] * inv),
                       float2_to_bf16x2(acc[i][2] * inv, acc[i][3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) =
            float2_to_bf16x2(acc[i][0] * inv, acc[i][1] * inv);
      if (lane == 0 && a.lse) a.lse[out] = none ? -INFINITY : m[i] + log2f(sum[i]);
    }
  }
}

// HALF (at most 4 qo heads a kv head): Q's columns 4..7 repeat columns 0..3, so
// every lane has scores of its heads for both 16-key blocks of a tile, and lanes
// 0, 1 of a quad go on with the first block, lanes 2, 3 with the second: half the
// exponentials, words and products a tile.  P^T then holds the blocks in columns
// 0..3 and 4..7; each block's V takes its own columns (the others as zeros), and
// the two halves of O meet at the end.  With 4 qo heads a kv head: 8 requests of
// 32K to 128K keys 139.2 us (152.7 without), 64 of 512 to 4096 41.2 (42.3).
template <int D, int GR, bool HALF>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    decode4_kernel(const __grid_constant__ Decode4Args p) {
  using S = Shape<D, GR>;
  constexpr int G = S::G, CH = S::CH, MT = S::MT;
  constexpr int NB = HALF ? 1 : 2;  // blocks of a tile whose scores a lane keeps
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int merging[8];  // per kv head of the CTA
  const AttnArgs& a = p.a;
  const int i0 = a.cta_ptr[blockIdx.x], i1 = a.cta_ptr[blockIdx.x + 1];
  if (i0 >= i1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hpc = a.heads_per_cta, n_split = p.splits;
  const int hl = warp % hpc, split = warp / hpc;
  const int Hq = a.num_qo_heads, group = Hq / a.num_kv_heads;
  const int qd = lane & 3, grp = lane >> 2;
  const int h0 = HALF ? (2 * qd) & 3 : 2 * qd;  // the lane's heads: h0, h0 + 1
  const int my_block = HALF ? qd >> 1 : 0;
  const float sc = a.scale_log2;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * S::STAGE);
  // states that meet: floor(splits / 2) slots a head
  float* const slots = reinterpret_cast<float*>(
      smem + hpc * n_split * (kStages * S::STAGE) + hl * (n_split >> 1) * S::SLOT);

  // ---- what this warp copies: its tiles of all items, one after another ----
  const uint8_t* const kp = reinterpret_cast<const uint8_t*>(a.k);
  const uint8_t* const k_chunk = kp + lane % CH * 16;
  // Lane i follows key c_key + i through the table: its page's index, slot and id.
  // (Unsigned: a key count may end right below 2^31.)
  const uint32_t P = a.page_size, stride = kTile * n_split;
  const uint32_t step_pages = stride / P, step_slots = stride % P;
  const uint32_t per_slot = a.layout == PKA_NHD ? a.num_kv_heads : 1;
  const uint32_t per_head = a.layout == PKA_NHD ? 1 : P;
  uint32_t c_key = 0, c_end = 0, c_pi = 0, c_last = 0, c_slot = 0, c_row0 = 0;
  int c_item = i0;
  const int32_t* c_table = nullptr;
  int32_t c_page = 0;
  auto next_item = [&]() {  // to the next item that has a tile for this warp
    while (c_key >= c_end && c_item < i1) {
      const PkaWorkItem* w = a.items + c_item++;
      c_key = w->t0 + kTile * split;
      c_end = w->t1;
      c_row0 = (uint32_t)(w->kv_head0 + hl) * per_head;
      c_table = a.kv_indices + w->kv_base;
      c_pi = (c_key + lane) / P;
      c_slot = (c_key + lane) - c_pi * P;
      c_last = (c_end - 1) / P;
    }
    if (c_key < c_end) c_page = c_table[min(c_pi, c_last)];
  };
  auto copy_tile = [&](int stage) {
    if (c_key < c_end) {
      const uint32_t at = ring + stage * S::STAGE;
      const uint32_t idx = c_slot * per_slot + c_row0;
      const int64_t page = (int64_t)c_page * a.page_stride;
      const uint32_t left = c_end - c_key;
      const int64_t words = page + p.code_bytes + (int64_t)idx * (4 * G);
      copy_async<4 * G>(at + 2 * S::CODES + lane * (4 * G), kp + words, lane < left);
      copy_async<4 * G>(at + 2 * S::CODES + S::WORDS + lane * (4 * G), kp + words + p.v_from_k,
                        lane < left);
      const int64_t row = page + (int64_t)idx * S::ROW;
      const int ch = lane % CH;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int k = lane / CH + i * (32 / CH);
        const uint8_t* from = k_chunk + __shfl_sync(0xffffffffu, row, k);
        const uint32_t to = at + k * S::ROW + ((ch ^ chunk_swap<D>(k)) << 4);
        copy_async<16>(to, from, k < left);
        copy_async<16>(to + S::CODES, from + p.v_from_k, k < left);
      }
      c_key += stride;
      c_pi += step_pages;
      c_slot += step_slots;
      if (c_slot >= P) {
        c_slot -= P;
        ++c_pi;
      }
      next_item();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  next_item();
#pragma unroll
  for (int s = 0; s < kStages; ++s) copy_tile(s);

  // rows of the MMA's A fragments: row r of a 16-key block is key
  // (r & 1) * 4 + (r & 7) / 2 (+ 8), so that V's lanes read keys t, t + 4, t + 8
  // and t + 12 (t = lane % 4)
  const int my_key = (grp & 1) * 4 + (grp >> 1);
  const int k_swap = chunk_swap<D>(my_key);
  const uint32_t k_lane = my_key * S::ROW + qd * 4;
  // halves of a word: elements 0..3 and 4..7; groups of 32 give a lane one half
  const uint32_t half_lo = S::DL == 4 && (grp & 1) ? 0x7632u : 0x5410u;

  int stage = 0;
  for (int ii = i0; ii < i1; ++ii) {
    const PkaWorkItem w = a.items[ii];
    const int head_base = (w.kv_head0 + hl) * group;
    // Q^T fragments of column grp: elements 8 qd .. 8 qd + 7 of each 32-element
    // chunk, in the order of K's operands, and the sums of q over the groups
    uint32_t qf[2 * CH][2];
    float2 cs, qs[G];
    {
      const int col = HALF ? grp & 3 : grp;
      const bool real = col < group;
      const uint4* row = reinterpret_cast<const uint4*>(
          a.q + ((int64_t)w.q_row0 * Hq + head_base + (real ? col : 0)) * D);
      float x[CH][8], most = 0.f, sum[G];
#pragma unroll
      for (int g = 0; g < G; ++g) sum[g] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const uint4 v = real ? row[4 * j + qd] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(u[i]);
          x[j][2 * i] = f.x;
          x[j][2 * i + 1] = f.y;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          most = fmaxf(most, fabsf(x[j][i]));
          sum[j * 32 / GR] += x[j][i];
        }
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
#pragma unroll
        for (int g = 0; g < G; ++g) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
      }
      const float up = f16_up(__float_as_uint(most));
      const float down = f16_down(__float_as_uint(most)) * (16777216.f * sc);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[j][i] * ((i & 1) ? up * 0.0625f : up);
        qf[2 * j][0] = float2_to_f16x2(y[0], y[4]);
        qf[2 * j][1] = float2_to_f16x2(y[1], y[5]);
        qf[2 * j + 1][0] = float2_to_f16x2(y[2], y[6]);
        qf[2 * j + 1][1] = float2_to_f16x2(y[3], y[7]);
      }
      // the sums in the units of q . c: Q's scale and the codes' 2^-24
      auto of_heads = [&](float x) {
        return make_float2(__shfl_sync(0xffffffffu, x, h0 * 4),
                           __shfl_sync(0xffffffffu, x, (h0 + 1) * 4));
      };
      cs = of_heads(down);
#pragma unroll
      for (int g = 0; g < G; ++g) qs[g] = of_heads(sum[g] * up * 0x1p-24f);
    }
    float acc[MT][4];
    float2 zs[G];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) zs[g] = make_float2(0.f, 0.f);
    // references of the exponents (log2, whole numbers), this lane's share of the sums of
    // p, and the powers of two of P
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float2 pw[G];
#pragma unroll
    for (int g = 0; g < G; ++g) pw[g] = make_float2(1.f, 1.f);
    bool begun = false;  // whether a tile had a key
    const int64_t mrow = ((int64_t)w.mask_hi << 32 | (uint32_t)w.mask_lo) +
                         (int64_t)w.q_local0 * w.kv_len;
    const uint32_t t1 = w.t1;

    // One tile of keys a0 .. a0 + 31.  ALL: every key is there and seen.  Pairs are of the
    // lane's two heads; b and y name the keys: my_key + 8 y of the lane's blocks.
    auto tile = [&](auto all, uint32_t a0) {
      constexpr bool ALL = decltype(all)::value;
      const uint32_t at = ring + stage * S::STAGE;
      auto key_of = [&](int b, int y) { return 16 * (HALF ? my_block : b) + 8 * y + my_key; };
      auto v_words = [&](int b, int y, uint32_t (&vw)[G]) {
        lds_words<G>(at + 2 * S::CODES + S::WORDS + key_of(b, y) * (4 * G), vw);
      };
      float2 s[NB][2];  // scores
      {
        uint32_t kw[NB][2][G];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            lds_words<G>(at + 2 * S::CODES + key_of(b, y) * (4 * G), kw[b][y]);
            s[b][y] = make_float2(0.f, 0.f);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float d[2][4];  // q . c over the group
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            d[b][0] = d[b][1] = d[b][2] = d[b][3] = 0.f;
#pragma unroll
            for (int j = g * (GR / 32); j < (g + 1) * (GR / 32); ++j) {
              const uint32_t from = at + k_lane + b * 16 * S::ROW + ((j ^ k_swap) << 4);
              const uint32_t w0 = lds32(from), w1 = lds32(from + 8 * S::ROW);
              const uint32_t u0 = w0 >> 8, u1 = w1 >> 8;
              mma16816(d[b], w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u,
                       w1 & 0x00f000f0u, qf[2 * j][0], qf[2 * j][1]);
              mma16816(d[b], u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u,
                       u1 & 0x00f000f0u, qf[2 * j + 1][0], qf[2 * j + 1][1]);
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float2 x = make_float2(d[b][2 * y], d[b][2 * y + 1]);
              if constexpr (HALF)
                if (my_block) x = make_float2(d[1][2 * y], d[1][2 * y + 1]);
              const float ks = step_of(kw[b][y][g]), kz = origin_of(kw[b][y][g]);
              s[b][y] = __ffma2_rn(make_float2(kz, kz), qs[g], s[b][y]);
              s[b][y] = __ffma2_rn(make_float2(ks, ks), x, s[b][y]);
            }
          }
        }
      }
      float most = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          s[b][y] = __fmul2_rn(s[b][y], cs);
          if constexpr (!ALL) {
            const int key = key_of(b, y);
            bool seen = a0 + key < t1;
            if (a.mask_mode == PKA_MASK_CUSTOM && seen) {
              const int64_t bit = mrow + a0 + key;
              seen = (a.mask[bit >> 3] >> (bit & 7)) & 1;
            }
            if (!seen) s[b][y] = make_float2(-INFINITY, -INFINITY);
          }
          most = max3(most, s[b][y].x - m[0], s[b][y].y - m[1]);
        }
      }
      // the first tile with a key (m = -inf) or a maximum well past its reference: the state
      // is rescaled, the same in all lanes of a column, and P's powers of two found anew,
      // from this tile's p * step and the earlier ones' (at most 2^kHeadroom / pw)
      if (__any_sync(0xffffffffu, most > kRescale - kBelow)) {
        // (all reductions a level at a time: a first tile waits for them)
        float2 top[1] = {make_float2(-INFINITY, -INFINITY)}, grown[G];
#pragma unroll
        for (int b = 0; b < NB; ++b)
          top[0] = make_float2(max3(top[0].x, s[b][0].x, s[b][1].x),
                               max3(top[0].y, s[b][0].y, s[b][1].y));
        max_keys<HALF>(top);
        const float2 to = make_float2(fmaxf(m[0], ceilf(top[0].x) + kBelow),
                                      fmaxf(m[1], ceilf(top[0].y) + kBelow));
#pragma unroll
        for (int g = 0; g < G; ++g) grown[g] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t vw[G];
            v_words(b, y, vw);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const float step = lg2(fmaxf(fabsf(step_of(vw[g])), kLeastStep));
              grown[g].x = fmaxf(grown[g].x, s[b][y].x - to.x + step);
              grown[g].y = fmaxf(grown[g].y, s[b][y].y - to.y + step);
            }
          }
        }
        max_keys<HALF>(grown);
        float al[2][G + 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int g = 0; g <= G; ++g) al[h][g] = 1.f;
          const float ref = h ? to.y : to.x;
          if (ref == -INFINITY) continue;  // no key yet
          const float far = fmaxf(m[h] - ref, -1000.f);  // -1000: no key before
          m[h] = ref;
          al[h][G] = pow2(far);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float& w = h ? pw[g].y : pw[g].x;
            const float before = far - pow2_log(w);
            const float now = clamp_log(
                fmaxf(before, ceilf(h ? grown[g].y : grown[g].x) - kHeadroom));
            al[h][g] = pow2(before - now);
            w = pow2(-now);
          }
        }
        if (begun) {  // not all zeros
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            l[h] *= al[h][G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
              (h ? zs[g].y : zs[g].x) *= al[h][G];
#pragma unroll
              for (int mt = g * (MT / G); mt < (g + 1) * (MT / G); ++mt) {
                acc[mt][h] *= al[h][g];
                acc[mt][2 + h] *= al[h][g];
              }
            }
          }
        }
        begun = true;
      }
      float2 e[NB][2];  // p
      uint32_t vw[NB][2][G];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          v_words(b, y, vw[b][y]);
          e[b][y] = make_float2(ex2(s[b][y].x - m[0]), ex2(s[b][y].y - m[1]));
          if constexpr (!ALL) {
            if (s[b][y].x == -INFINITY) e[b][y].x = 0.f;  // not -inf + inf
            if (s[b][y].y == -INFINITY) e[b][y].y = 0.f;
            // an unseen key's words may hold anything
            if (s[b][y].x == -INFINITY && s[b][y].y == -INFINITY)
#pragma unroll
              for (int g = 0; g < G; ++g) vw[b][y][g] = 0u;
          }
          l[0] += e[b][y].x;
          l[1] += e[b][y].y;
        }
      }
      // O^T += V^T . P^T, with P = p * step * pw
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t pb[2][2];
        auto weigh = [&]() {
          uint32_t most_p = 0;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float step = step_of(vw[b][y][g]);
              const float2 p = __fmul2_rn(e[b][y], __fmul2_rn(make_float2(step, step), pw[g]));
              pb[b][y] = float2_to_f16x2(p.x, p.y);
              most_p = max_f16x2(most_p, pb[b][y] & 0x7fff7fffu);
            }
          }
          return ((most_p + (0x7fffu - kMostP) * 0x10001u) & 0x80008000u) != 0;
        };
        if (__any_sync(0xffffffffu, weigh())) {  // a P past f16's middle: a smaller power of two
          float2 grown[1] = {make_float2(0.f, 0.f)};
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float step = fabsf(step_of(vw[b][y][g]));
              grown[0].x = fmaxf(grown[0].x, e[b][y].x * step);
              grown[0].y = fmaxf(grown[0].y, e[b][y].y * step);
            }
          }
          max_keys<HALF>(grown);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float before = -pow2_log(h ? pw[g].y : pw[g].x);
            const float now =
                clamp_log(fmaxf(before, ceilf(lg2(h ? grown[0].y : grown[0].x)) - kHeadroom));
            const float al = pow2(before - now);
            (h ? pw[g].y : pw[g].x) = pow2(-now);
#pragma unroll
            for (int mt = g * (MT / G); mt < (g + 1) * (MT / G); ++mt) {
              acc[mt][h] *= al;
              acc[mt][2 + h] *= al;
            }
          }
          weigh();
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float z = origin_of(vw[b][y][g]);
            zs[g] = __ffma2_rn(e[b][y], make_float2(z, z), zs[g]);
          }
          // 15 of the second keys' P as it is rounded, which the MMAs take (15 - c) of
          const float2 p = f16x2_to_float2(pb[b][1]);
          zs[g] = __ffma2_rn(p, make_float2(15.f * pow2_inverse(pw[g].x),
                                            15.f * pow2_inverse(pw[g].y)), zs[g]);
          pb[b][0] = transpose8x8(pb[b][0]);
          pb[b][1] = transpose8x8(pb[b][1] ^ 0x80008000u);
        }
        if constexpr (HALF) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            pb[1][y] = grp < 4 ? 0u : pb[0][y];
            pb[0][y] = grp < 4 ? pb[0][y] : 0u;
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // the lane's elements of keys t, t + 4, t + 8, t + 12 of this group
          const uint32_t vat = at + S::CODES + (16 * b + qd) * S::ROW;
          const int swap0 = chunk_swap<D>(qd), swap4 = chunk_swap<D>(qd + 4);
          constexpr int WL = S::DL < 8 ? 1 : S::DL / 8;  // words
          uint32_t v0[WL], v4[WL], v8[WL], v12[WL];
          const int word = g * (GR / 8) + (grp * S::DL >> 3);  // of the row
          const uint32_t c0 = vat + (((word >> 2) ^ swap0) << 4) + ((word & 3) << 2);
          const uint32_t c4 = vat + 4 * S::ROW + (((word >> 2) ^ swap4) << 4) + ((word & 3) << 2);
          if constexpr (WL == 2) {
            const uint2 x0 = lds64(c0), x4 = lds64(c4), x8 = lds64(c0 + 8 * S::ROW),
                        x12 = lds64(c4 + 8 * S::ROW);
            v0[0] = x0.x, v0[1] = x0.y, v4[0] = x4.x, v4[1] = x4.y;
            v8[0] = x8.x, v8[1] = x8.y, v12[0] = x12.x, v12[1] = x12.y;
          } else {
            v0[0] = lds32(c0), v4[0] = lds32(c4);
            v8[0] = lds32(c0 + 8 * S::ROW), v12[0] = lds32(c4 + 8 * S::ROW);
          }
#pragma unroll
          for (int q = 0; q < S::DL / 4; ++q) {  // four elements, two 16-row blocks
            const uint32_t sel = S::DL == 4 ? half_lo : (q & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(v0[q >> 1], v4[q >> 1], sel);
            const uint32_t y = __byte_perm(v8[q >> 1], v12[q >> 1], sel);
            const uint32_t x8 = x >> 8, y8 = y >> 8;
            const int mt = (g * (S::DL / 4) + q) * 2;
            mma16816(acc[mt], x & 0x000f000fu, x & 0x00f000f0u, ~y & 0x000f000fu,
                     ~y & 0x00f000f0u, pb[b][0], pb[b][1]);
            mma16816(acc[mt + 1], x8 & 0x000f000fu, x8 & 0x00f000f0u, ~y8 & 0x000f000fu,
                     ~y8 & 0x00f000f0u, pb[b][0], pb[b][1]);
          }
        }
      }
    };
    const uint32_t all_end = a.mask_mode == PKA_MASK_CUSTOM ? 0u : t1;
    for (uint32_t a0 = w.t0 + kTile * split; a0 < t1; a0 += stride) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      if (a0 + kTile <= all_end)
        tile(Yes{}, a0);
      else
        tile(No{}, a0);
      __syncwarp();
      copy_tile(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // from P's powers of two and the codes' 2^-24 and 2^-20 to what p weighs
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float2 w = pw[mt / (MT / G)];
      const float inv[2] = {pow2_inverse(w.x), pow2_inverse(w.y)};
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[mt][x] *= inv[x & 1] * (x < 2 ? 16777216.f : 1048576.f);
    }

    // ---- the head's warps bring their states together, pair by pair; which warp
    // ends an item goes round, so that the others are at the next one meanwhile ----
    const int turn = (ii - i0) % n_split;
    const int rank = split >= turn ? split - turn : split - turn + n_split;
    for (int n = n_split; n > 1;) {
      const int half = (n + 1) >> 1;
      float* const slot = slots + (rank >= half ? rank - half : rank) * (S::SLOT / 4) + lane;
      if (rank >= half && rank < n) {
        int i = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x) slot[32 * i++] = acc[mt][x];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          slot[32 * i++] = m[h];
          slot[32 * i++] = l[h];
#pragma unroll
          for (int g = 0; g < G; ++g) slot[32 * i++] = h ? zs[g].y : zs[g].x;
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(hl + 1), "r"(32 * n_split) : "memory");
      if (rank < n - half) {
        const float* const tail = slot + 32 * 4 * MT;
        float mine[2], other[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float om = tail[32 * (h * (2 + G))];
          const float to = fmaxf(m[h], om);
          mine[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - to);
          other[h] = om == -INFINITY ? 0.f : ex2(om - to);
          m[h] = to;
          l[h] = l[h] * mine[h] + tail[32 * (h * (2 + G) + 1)] * other[h];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float& z = h ? zs[g].y : zs[g].x;
            z = z * mine[h] + tail[32 * (h * (2 + G) + 2 + g)] * other[h];
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            acc[mt][x] = acc[mt][x] * mine[x & 1] + slot[32 * (4 * mt + x)] * other[x & 1];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(hl + 1), "r"(32 * n_split) : "memory");
      n = half;
    }
    if (rank == 0) {

    // ---- normalise and write: O and the LSE, or this piece's partial state ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = sum_keys<HALF>(l[h]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float& z = h ? zs[g].y : zs[g].x;
        z = sum_keys<HALF>(z);
      }
    }
    if constexpr (HALF) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] += __shfl_xor_sync(0xffffffffu, acc[mt][i], 2);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int head = head_base + h0 + h;
      if (h0 + h >= group || my_block) continue;
      // a NaN among the words of a seen key makes the sums NaN, which is not "no key"
      const bool none = l[h] == 0.f;
      const float inv = none ? 0.f : 1.f / l[h];
      const float lse = none ? -INFINITY : m[h] + log2f(l[h]);
      const int rec = w.out_rec + (head - w.kv_head0 * group);
      uint16_t* orow = a.o + ((int64_t)w.q_row0 * Hq + head) * D;
      float* prow = a.part_o + (int64_t)rec * D;
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int q = 0; q < S::DL / 4; ++q) {
          const int mt = (g * (S::DL / 4) + q) * 2;
          const float z = (h ? zs[g].y : zs[g].x) * inv;
          const float x0 = fmaf(acc[mt][h], inv, z), x1 = fmaf(acc[mt][2 + h], inv, z);
          const float x2 = fmaf(acc[mt + 1][h], inv, z), x3 = fmaf(acc[mt + 1][2 + h], inv, z);
          const int d = g * GR + grp * S::DL + 4 * q;
          if (w.out_rec < 0)
            *reinterpret_cast<uint2*>(orow + d) =
                make_uint2(float2_to_bf16x2(x0, x1), float2_to_bf16x2(x2, x3));
          else
            *reinterpret_cast<float4*>(prow + d) = make_float4(x0, x1, x2, x3);
        }
      }
      if (grp == 0) {
        if (w.out_rec >= 0)
          a.part_lse[rec] = lse;
        else if (a.lse)
          a.lse[(int64_t)w.q_row0 * Hq + head] = lse;
      }
    }
    }  // rank 0
    if (w.join >= 0 && a.joins) {
      // count the piece in once its state is visible; the last one merges: for a
      // CTA's last item all warps of the head, before it the one that ended the item
      PkaDecodeJoin* const jp = a.joins + w.join + hl;
      const bool together = ii + 1 == i1 && n_split > 1;
      int last = 0;
      if (rank == 0) {
        __threadfence();
        __syncwarp();
        if (lane == 0) last = atomicAdd(&jp->arrived, 1) == jp->nslots - 1;
        if (together && lane == 0) merging[hl] = last;
        last = __shfl_sync(0xffffffffu, last, 0);
      }
      if (together) {
        asm volatile("bar.sync %0, %1;" ::"r"(hl + 1), "r"(32 * n_split) : "memory");
        last = merging[hl];
      }
      if (last) {
        __threadfence();
        join_heads<D>(a, *jp, w.q_row0, head_base, group, together ? rank : 0,
                      together ? n_split : 1, lane);
        __syncwarp();
        if (together)  // every warp has read the fixed fields
          asm volatile("bar.sync %0, %1;" ::"r"(hl + 1), "r"(32 * n_split) : "memory");
        if (rank == 0 && lane == 0) jp->arrived = 0;  // re-armed for the next run
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int GR, bool HALF>
cudaError_t launch_t(const AttnArgs& a, int num_ctas, cudaStream_t stream) {
  using S = Shape<D, GR>;
  Decode4Args p{};
  p.a = a;
  p.code_bytes = (int64_t)a.page_size * a.num_kv_heads * (D / 2);
  p.v_from_k = reinterpret_cast<intptr_t>(a.v) - reinterpret_cast<intptr_t>(a.k);
  const int hpc = a.heads_per_cta;
  p.splits = kMaxWarps / hpc;
  const int warps = hpc * p.splits;
  const int smem = warps * kStages * S::STAGE + hpc * (p.splits / 2) * S::SLOT;
  static_assert(kMaxWarps * kStages * S::STAGE + kMaxWarps / 2 * S::SLOT <= 227 * 1024,
                "shared memory");
  cudaError_t e = ensure_dynamic_smem<decode4_kernel<D, GR, HALF>>(smem);
  if (e != cudaSuccess) return e;
  decode4_kernel<D, GR, HALF><<<num_ctas, 32 * warps, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int GR>
cudaError_t launch_any(const AttnArgs& a, int num_ctas, bool half, cudaStream_t stream) {
  return half ? launch_t<D, GR, true>(a, num_ctas, stream)
              : launch_t<D, GR, false>(a, num_ctas, stream);
}

}  // namespace

cudaError_t launch_decode4(const AttnArgs& a, int num_ctas, int head_dim, int group,
                           cudaStream_t stream) {
  const bool half = a.num_qo_heads <= 4 * a.num_kv_heads;
  if (head_dim == 128)
    return group == 32   ? launch_any<128, 32>(a, num_ctas, half, stream)
           : group == 64 ? launch_any<128, 64>(a, num_ctas, half, stream)
                         : launch_any<128, 128>(a, num_ctas, half, stream);
  return group == 32 ? launch_any<64, 32>(a, num_ctas, half, stream)
                     : launch_any<64, 64>(a, num_ctas, half, stream);
}

}  // namespace pka
