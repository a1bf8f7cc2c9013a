// K/V held in 4 bits: the append that quantises, and the read-back of cached
// rows (of pools of every type), also as the bf16 scratch of the tensor-core
// rows.  The page format and the rounding rules are in pka_kv4.h.
#include "pka_cache.h"
#include "pka_device.cuh"
#include "pka_kv4.h"

namespace pka {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// A row's place in the pools; page < 0: nowhere.
struct Place {
  int32_t page;
  int32_t slot;
};

// The logical position `pos` of request r, looked up in its table.
__device__ __forceinline__ Place place_of(const KvRows& a, int r, int64_t pos) {
  Place p{-1, 0};
  const int kv0 = a.kv_indptr[r], pages = a.kv_indptr[r + 1] - kv0;
  const int64_t kv_len = (int64_t)(pages - 1) * a.page_size + a.last_page_len[r];
  if (pos < 0 || pos >= kv_len) return p;
  const int64_t nth = pos <= UINT32_MAX ? (uint32_t)pos / (uint32_t)a.page_size
                                        : pos / a.page_size;
  p.page = a.kv_indices[kv0 + nth];
  p.slot = (int)(pos - nth * a.page_size);
  if (p.page >= a.num_pages) p.page = -1;
  return p;
}

// The request of row `row` of a batch, or -1 for a row of none.  A decode
// step's rows are one a request, so row r is tried as request r's first.
__device__ __forceinline__ int request_of(const KvRows& a, int64_t row, int lane) {
  const int guess = (int)min(row, (int64_t)a.batch - 1);
  if (row >= a.row_indptr[guess] && row < a.row_indptr[guess + 1]) return guess;
  if (row >= a.row_indptr[a.batch]) return -1;
  return warp_find(a.row_indptr, a.batch, row, lane);
}

// ---------------------------------------------------------------------------
// Append.  A warp takes a row, or a part of its heads (K's, then V's, as one
// list), in steps of 256 elements: 8 a lane, four steps in flight.  The lanes
// of a group exchange its least and greatest element (exact in bf16, both in
// one word: the least and the negated greatest under one minimum), then every
// lane makes its 8 codes, one 32-bit store.
//   Bound by memory on long appends; on a decode step by the dependent look-ups
// of request, page and slot.
// ---------------------------------------------------------------------------

struct Append4Args {
  KvRows rows;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint8_t* k;
  uint8_t* v;
  int64_t code_bytes;  // of a page
  int steps_per_part;
};

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr int kAppendSteps = 4;  // in flight

template <int D, int GR>
__global__ void __launch_bounds__(256) append4_kernel(const __grid_constant__ Append4Args a) {
  constexpr int LPH = D / 8;      // lanes of a head
  constexpr int HPS = 32 / LPH;   // heads of a step
  constexpr int LPG = GR / 8;     // lanes of a group
  constexpr int G = D / GR;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, piece = lane % LPH;
  const KvRows& t = a.rows;
  const int hk = t.heads, heads = 2 * hk;
  const int h0 = blockIdx.y * a.steps_per_part * HPS;
  const int h1 = min(heads, h0 + a.steps_per_part * HPS);
  for (int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < t.rows; row += gridDim.x * 8ll) {
    const int64_t at = row * hk * D + piece * 8;
    uint4 x[kAppendSteps];
    auto load = [&](int hb) {
#pragma unroll
      for (int s = 0; s < kAppendSteps; ++s) {
        const int h = hb + s * HPS + sub;
        x[s] = make_uint4(0u, 0u, 0u, 0u);
        if (h >= h1) continue;
        const uint16_t* src = h < hk ? a.k_new + at + (int64_t)h * D
                                     : a.v_new + at + (int64_t)(h - hk) * D;
        x[s] = *reinterpret_cast<const uint4*>(src);
      }
    };
    load(h0);
    const int r = request_of(t, row, lane);
    if (r < 0) break;  // this row and those behind it belong to no request
    const int first = t.row_indptr[r], n = t.row_indptr[r + 1] - first;
    const int kv0 = t.kv_indptr[r], pages = t.kv_indptr[r + 1] - kv0;
    const int64_t kv_len = (int64_t)(pages - 1) * t.page_size + t.last_page_len[r];
    const Place p = place_of(t, r, kv_len - n + (row - first));
    if (p.page < 0) {
      if (lane == 0) note_error(t.err, PKA_ERR_METADATA);
      continue;
    }
    const int64_t page = (int64_t)p.page * t.page_stride;
    for (int hb = h0;;) {
#pragma unroll
      for (int s = 0; s < kAppendSteps; ++s) {
        const int h = hb + s * HPS + sub;
        // {least, -greatest} of the lane's 8 elements, then of its group
        const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
        const uint32_t lo = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
        const uint32_t hi = min2_nan(min2_nan(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                                     min2_nan(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
        uint32_t both = min2_nan(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
        for (int off = 1; off < LPG; off <<= 1)
          both = min2_nan(both, __shfl_xor_sync(kAll, both, off));
        if (h >= h1) continue;
        const Group4 g = group4(__uint_as_float(both << 16),
                                -__uint_as_float(both & 0xffff0000u));
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = bf16x2_to_float2(w[i]);
          f[2 * i] = v.x;
          f[2 * i + 1] = v.y;
        }
        const bool is_v = h >= hk;
        const int hh = is_v ? h - hk : h;
        const int64_t idx = t.layout == PKA_NHD ? (int64_t)p.slot * hk + hh
                                                : (int64_t)hh * t.page_size + p.slot;
        uint8_t* pool = (is_v ? a.v : a.k) + page;
        *reinterpret_cast<uint32_t*>(pool + idx * (D / 2) + piece * 4) = codes4(f, g);
        if (piece % LPG == 0)
          *reinterpret_cast<uint32_t*>(pool + a.code_bytes + (idx * G + piece / LPG) * 4) = g.word;
      }
      hb += kAppendSteps * HPS;
      if (hb >= h1) break;
      load(hb);
    }
  }
}

// ---------------------------------------------------------------------------
// Read-back.  A warp takes a row or a part of its heads as above, 8 elements a
// lane and step (4 bytes of codes, 8 of e4m3, 16 of bf16 in; 16 out), eight
// steps in flight.  Bound by memory: the rows go out in 2 bytes an element
// whatever they came in.
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
  // the outputs asked for, as one list of heads
  const int k_end = a.k_out ? hk : 0, heads = k_end + (a.v_out ? hk : 0);
  const int h0 = blockIdx.y * a.steps_per_part * HPS;
  const int h1 = min(heads, h0 + a.steps_per_part * HPS);
  int64_t rows = t.rows;
  int units = t.num_units;
  if (t.counts) {  // this plan's counts, within what the launch was sized for
    units = min(max(t.counts[0], 0), units);
    rows = min((int64_t)max(t.counts[2], 0), rows);
    if (units <= 0) return;
  }
  for (int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < rows; row += gridDim.x * 8ll) {
    Place p;
    if (t.units) {
      // the last unit that starts at or before the row
      int lo = 0, n = units;
      while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const bool le = at < n && t.units[lo + at].dst_row0 <= row;
        const int below = max(__popc(__ballot_sync(kAll, le)) - 1, 0);
        lo += below * step;
        n = min(step, n - below * step);
      }
      const PkaDequantUnit u = t.units[lo];
      const uint32_t j = (uint32_t)(row - u.dst_row0), nth = j / (uint32_t)t.page_size;
      p.page = t.kv_indices[u.kv_base + nth];
      p.slot = (int)(j - nth * (uint32_t)t.page_size);
    } else {
      const int r = request_of(t, row, lane);
      if (r < 0) break;
      p = place_of(t, r, (t.begin ? t.begin[r] : 0ll) + (row - t.row_indptr[r]));
      if (p.page < 0) {
        if (lane == 0) note_error(t.err, PKA_ERR_METADATA);
        continue;
      }
    }
    const int64_t page = (int64_t)p.page * t.page_stride * (KIND == 0 ? 2 : 1);
    for (int hb = h0; hb < h1; hb += kReadSteps * HPS) {
      uint4 x[kReadSteps];
#pragma unroll
      for (int s = 0; s < kReadSteps; ++s) {
        const int h = hb + s * HPS + sub;
        if (h >= h1) continue;
        const int hh = h < k_end ? h : h - k_end;
        const int64_t idx = t.layout == PKA_NHD ? (int64_t)p.slot * hk + hh
                                                : (int64_t)hh * t.page_size + p.slot;
        const uint8_t* pool = (h < k_end ? a.k : a.v) + page;
        const uint8_t* src = pool + (idx * LPH + piece) * IN;
        if constexpr (KIND == 0) {
          x[s] = *reinterpret_cast<const uint4*>(src);
        } else if constexpr (KIND == 1) {
          const uint2 c = *reinterpret_cast<const uint2*>(src);
          x[s].x = c.x;
          x[s].y = c.y;
        } else {
          x[s].x = *reinterpret_cast<const uint32_t*>(src);
          x[s].y = *reinterpret_cast<const uint32_t*>(pool + a.code_bytes +
                                                      (idx * G + piece / (KIND / 8)) * 4);
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
          const float step = __uint_as_float(x[s].y << 16);
          const float origin = __uint_as_float(x[s].y & 0xffff0000u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the code as a float: 2^23 + c less 2^23
            const uint32_t w = x[s].x >> (8 * i);
            const float c0 = __uint_as_float((w & 15u) | 0x4b000000u) - 8388608.f;
            const float c1 = __uint_as_float((w >> 4 & 15u) | 0x4b000000u) - 8388608.f;
            // step * c is exact (8 by 4 bits), so this rounds twice: the sum to
            // float32 and the result to bf16
            out[i] = float2_to_bf16x2(fmaf(step, c0, origin), fmaf(step, c1, origin));
          }
        }
        uint16_t* dst = (is_k ? a.k_out : a.v_out) +
                        (row * hk + (is_k ? h : h - k_end)) * (int64_t)D + piece * 8;
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

// How many of a row's steps one warp takes: enough warps first (16 an SM), then
// as many steps as are in flight at once.
int steps_per_part(int64_t rows, int steps, int most) {
  const int sms = current_device_sms();
  const int64_t warps = 16 * (int64_t)(sms > 0 ? sms : 1);
  const int64_t per = (rows * steps + warps - 1) / warps;
  const int n = per < 1 ? 1 : per > most ? most : (int)per;
  const int parts = (steps + n - 1) / n;
  return (steps + parts - 1) / parts;
}

dim3 grid_of(int64_t rows, int steps, int per_part) {
  const int parts = (steps + per_part - 1) / per_part;
  const int64_t blocks = (rows + 7) / 8;
  const int64_t most = (int64_t)1 << 24;
  return dim3((unsigned)(blocks < 1 ? 1 : blocks > most ? most : blocks), (unsigned)parts);
}

template <int D, int KIND>
cudaError_t launch_read_t(const ReadArgs& args, cudaStream_t stream) {
  ReadArgs a = args;
  constexpr int HPS = 256 / D;
  const int heads = a.rows.heads * ((a.k_out ? 1 : 0) + (a.v_out ? 1 : 0));
  const int steps = (heads + HPS - 1) / HPS;
  a.steps_per_part = steps_per_part(a.rows.rows, steps, kReadSteps);
  read_kernel<D, KIND><<<grid_of(a.rows.rows, steps, a.steps_per_part), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int GR>
cudaError_t launch_append_t(const Append4Args& args, cudaStream_t stream) {
  Append4Args a = args;
  constexpr int HPS = 256 / D;
  const int steps = (2 * a.rows.heads + HPS - 1) / HPS;
  a.steps_per_part = steps_per_part(a.rows.rows, steps, 2 * kAppendSteps);
  append4_kernel<D, GR><<<grid_of(a.rows.rows, steps, a.steps_per_part), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

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
