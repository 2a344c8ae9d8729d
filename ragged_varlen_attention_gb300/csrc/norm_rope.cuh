// Per-head RMS norm with the position rotation: forward, backward, and the serving
// form that writes K and V into the paged cache.
//
//   r = 1/sqrt(mean x^2 + eps), y = x r w, z = R(pos) y on the first rot elements
//   backward: g = R(pos)^T dz, a = g w, xh = x r, dx = r (a - xh mean(a xh)), dw = sum g xh
//
// Every element is read once and written once; the arithmetic is a few fma per
// element, so memory bounds all three forms. A head's row is one group of G = 8 .. 32
// lanes with 8 elements each, and its sums are shuffles inside the group. A rotated
// pair never leaves its lane: in the halves layout lane i holds elements 4i .. 4i+3
// and their partners rot/2 + 4i .., in the adjacent layout 8i .. 8i+7; either way as
// four a's and their four b's, in packed pairs (half the fma instructions; with scalar
// ones the backward was bound by them, 41 % of the copy bandwidth). A warp's unit is kUnroll x
// (32/G) consecutive rows of one tensor, and the next unit's rows are loaded before
// this one's are computed, so that loads are always in flight.
//
// Measured, bf16, 32 + 8 heads of d = 128, against a copy at 6.79 TB/s: forward 32768 tokens
// 106 us (94 %), backward 16384 tokens 83 us (90 %), serving form 8192 tokens of 40 + 8 + 8
// fp16 heads 40 us (88 %); 48 tokens of a decode step 2.6 us, where the launch and two memory
// latencies are all there is. Where a unit spans tokens (heads that its rows do not divide)
// each row has a table row of its own: 23889 tokens of 16 + 4 heads 46 us (79 %).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace thd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// rows in flight for each group of lanes: 4, as far as the registers hold two such sets
constexpr int norm_rope_unroll(int elem, bool back) { return back && elem == 4 ? 2 : 4; }

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Sums N values over the group's lanes at once: each step hands half of the values to the
// other half of the lanes, so that N + log2(G/N) shuffles do what N log2(G) would. Lane l of
// the group returns the sum of value l / (G / N).
template <int G, int N>
__device__ __forceinline__ float sum_each(float (&v)[N]) {
  int bit = G / 2;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, bit >>= 1) {
    const bool upper = threadIdx.x & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[i + n] : v[i], give = upper ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
    }
  }
#pragma unroll
  for (; bit > 0; bit >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  return v[0];
}

// A lane's 8 elements of a row as loaded: 4 from e0, 4 from e1.
template <typename T>
struct Raw {
  uint2 lo, hi;
  __device__ __forceinline__ void load(const T* row, int e0, int e1) {
    lo = *reinterpret_cast<const uint2*>(row + e0);
    hi = *reinterpret_cast<const uint2*>(row + e1);
  }
  __device__ __forceinline__ void zero() { lo = hi = make_uint2(0u, 0u); }
  __device__ __forceinline__ void store(T* row, int e0, int e1) const {
    *reinterpret_cast<uint2*>(row + e0) = lo;
    *reinterpret_cast<uint2*>(row + e1) = hi;
  }
};
template <>
struct Raw<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* row, int e0, int e1) {
    lo = *reinterpret_cast<const float4*>(row + e0);
    hi = *reinterpret_cast<const float4*>(row + e1);
  }
  __device__ __forceinline__ void zero() { lo = hi = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void store(float* row, int e0, int e1) const {
    *reinterpret_cast<float4*>(row + e0) = lo;
    *reinterpret_cast<float4*>(row + e1) = hi;
  }
};

// the two elements of a 32-bit word
template <typename T>
__device__ __forceinline__ float2 split(uint32_t w);
template <>
__device__ __forceinline__ float2 split<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 split<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t merge(float x, float y);
template <>
__device__ __forceinline__ uint32_t merge<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t merge<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The lane's elements as pairs (a_k, b_k), k = 0 .. 3, in packed float32:
// v[0] = (a_0, a_1), v[1] = (a_2, a_3), v[2] = (b_0, b_1), v[3] = (b_2, b_3).
// Halves layout: a from lo, b from hi. ADJ: lo = a_0 b_0 a_1 b_1, hi = a_2 b_2 a_3 b_3.
struct Eight {
  uint64_t v[4];
  template <typename T, bool ADJ>
  __device__ __forceinline__ void get(const Raw<T>& r) {
    float2 x[4];
    if constexpr (sizeof(T) == 2) {
      x[0] = split<T>(r.lo.x); x[1] = split<T>(r.lo.y); x[2] = split<T>(r.hi.x); x[3] = split<T>(r.hi.y);
    } else {
      x[0] = make_float2(r.lo.x, r.lo.y); x[1] = make_float2(r.lo.z, r.lo.w);
      x[2] = make_float2(r.hi.x, r.hi.y); x[3] = make_float2(r.hi.z, r.hi.w);
    }
    if (ADJ) {
      v[0] = ptx::f2_pack(x[0].x, x[1].x); v[1] = ptx::f2_pack(x[2].x, x[3].x);
      v[2] = ptx::f2_pack(x[0].y, x[1].y); v[3] = ptx::f2_pack(x[2].y, x[3].y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = ptx::f2_pack(x[i].x, x[i].y);
    }
  }
  template <typename T, bool ADJ>
  __device__ __forceinline__ void put(Raw<T>& r) const {
    float2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::f2_unpack(v[i], y[i].x, y[i].y);
    if (ADJ) {
      x[0] = make_float2(y[0].x, y[2].x); x[1] = make_float2(y[0].y, y[2].y);
      x[2] = make_float2(y[1].x, y[3].x); x[3] = make_float2(y[1].y, y[3].y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = y[i];
    }
    if constexpr (sizeof(T) == 2) {
      r.lo = make_uint2(merge<T>(x[0].x, x[0].y), merge<T>(x[1].x, x[1].y));
      r.hi = make_uint2(merge<T>(x[2].x, x[2].y), merge<T>(x[3].x, x[3].y));
    } else {
      r.lo = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
      r.hi = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
  }
};

__device__ __forceinline__ uint64_t both(float x) { return ptx::f2_pack(x, x); }
__device__ __forceinline__ float fold(uint64_t x) {
  float a, b;
  ptx::f2_unpack(x, a, b);
  return a + b;
}
// <x, y> over the lane's elements
__device__ __forceinline__ float dot(const Eight& x, const Eight& y) {
  return fold(ptx::f2_fma(x.v[3], y.v[3], ptx::f2_fma(x.v[2], y.v[2], ptx::f2_fma(x.v[1], y.v[1], ptx::f2_mul(x.v[0], y.v[0])))));
}

// The angles of a lane's four pairs; neg = -sin.
struct Angles {
  uint64_t cos[2], sin[2], neg[2];
  __device__ __forceinline__ void load(const float* row, int half) {
    set(*reinterpret_cast<const float4*>(row), *reinterpret_cast<const float4*>(row + half));
  }
  __device__ __forceinline__ void set(const float4& c, const float4& s) {
    cos[0] = ptx::f2_pack(c.x, c.y); cos[1] = ptx::f2_pack(c.z, c.w);
    sin[0] = ptx::f2_pack(s.x, s.y); sin[1] = ptx::f2_pack(s.z, s.w);
    neg[0] = ptx::f2_pack(-s.x, -s.y); neg[1] = ptx::f2_pack(-s.z, -s.w);
  }
  // (a, b) -> (a c - b s, b c + a s), or by the opposite angle
  template <bool BACK>
  __device__ __forceinline__ void turn(Eight& y) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = y.v[i], b = y.v[2 + i];
      y.v[i] = ptx::f2_fma(a, cos[i], ptx::f2_mul(b, BACK ? sin[i] : neg[i]));
      y.v[2 + i] = ptx::f2_fma(b, cos[i], ptx::f2_mul(a, BACK ? neg[i] : sin[i]));
    }
  }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The cache row that row t of tensor `which` (1 K, 2 V) goes to; false: it goes nowhere.
template <typename T>
__device__ __forceinline__ bool cache_row(const NormRopeParams& p, int which, int slot, T*& dst) {
  if (slot < 0 || slot >= p.num_slots) return false;
  const int page = slot / p.page_size;
  dst = static_cast<T*>(p.out[which]) + (int64_t)page * p.out_page[which] +
        (int64_t)(slot - page * p.page_size) * p.out_tok[which];
  return true;
}

// Strides of a view: the row of token t and head h is base + t tok + h head.
struct Where {
  int64_t tok, head;
  template <typename P>
  __device__ __forceinline__ P* at(P* base, int t, int h) const { return base + t * tok + h * head; }
};

// One tensor's rows (WHICH: 0 Q, 1 K, 2 V) among the launch's units. `u` is the warp's first
// unit counted from the tensor's; on return, counted from the next tensor's. ONE: the heads
// are a multiple of a unit's rows, so that a unit is of one token, with one position and one
// row of the table. `acc`: the lane's part of the weight gradient (backward).
template <typename T, int G, int FORM, bool ADJ, bool ONE, int WHICH>
__device__ __forceinline__ void rows_of(const NormRopeParams& p, int64_t& u, Eight& acc, uint32_t& status) {
  constexpr bool kBack = FORM == THD_NORM_ROPE_BWD;
  constexpr bool kCached = FORM == THD_NORM_ROPE_PAGED && WHICH != 0;  // rows go to the cache
  constexpr int kUnroll = norm_rope_unroll(sizeof(T), kBack);
  constexpr int kAtOnce = 32 / G;
  constexpr int kRows = kAtOnce * kUnroll;
  const int lane = threadIdx.x & 31;
  const int item = lane % G, sub = lane / G;
  const bool active = item * 8 < p.d;
  const bool rotated = item * 8 < p.rot;
  const int e0 = rotated && !ADJ ? 4 * item : 8 * item;
  const int e1 = rotated && !ADJ ? p.rot / 2 + 4 * item : 8 * item + 4;
  const float inv_d = 1.f / (float)p.d;
  const FastDiv by_heads = p.by_heads[WHICH ? 1 : 0];
  const int rows = p.rows * by_heads.d;  // below 2^31 by the caller's choice of kernel
  const int64_t units = (rows + kRows - 1) / kRows;
  const int64_t stride = (int64_t)gridDim.x * kWarps;

  Eight w;
  if constexpr (WHICH < 2) {
    Raw<T> r;
    if (p.w[WHICH] && active) {
      r.load(static_cast<const T*>(p.w[WHICH]), e0, e1);
      w.get<T, ADJ>(r);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w.v[i] = both(1.f);
    }
  }

  // the lane's rows of a unit (ONE: a constant stride apart, and a whole number of units)
  struct Unit {
    Raw<T> x[kUnroll], g[kBack ? kUnroll : 1];
    int pos[ONE ? 1 : kUnroll];
  };
  const Where in = {p.in_tok[WHICH], p.in_head[WHICH]};
  const Where gin = {p.in_tok[kBack ? 2 + WHICH : 0], p.in_head[kBack ? 2 + WHICH : 0]};
  const Where out = {p.out_tok[WHICH], p.out_head[WHICH]};
  const T* const x_base = static_cast<const T*>(p.in[WHICH]);
  const T* const g_base = static_cast<const T*>(p.in[kBack ? 2 + WHICH : 0]);
  const auto load = [&](Unit& n, int64_t unit) {
    const int first = (int)unit * kRows;
    const T *x = nullptr, *g = nullptr;
    if (ONE) {
      const int t = by_heads.div(first), h = first - t * by_heads.d + sub;
      if (!kBack) n.pos[0] = p.positions[t];
      x = in.at(x_base, t, h);
      if constexpr (kBack) g = gin.at(g_base, t, h);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int row = first + sub + i * kAtOnce;
      if (!ONE) {
        const int t = by_heads.div(min(row, rows - 1)), h = row - t * by_heads.d;
        n.pos[i] = p.positions[t];
        x = in.at(x_base, t, h);
        if constexpr (kBack) g = gin.at(g_base, t, h);
      }
      if (active && (ONE || row < rows)) {
        n.x[i].load(x, e0, e1);
        if constexpr (kBack) n.g[i].load(g, e0, e1);
      } else {
        n.x[i].zero();
        if constexpr (kBack) n.g[i].zero();
      }
      if (ONE) {
        x += kAtOnce * in.head;
        if constexpr (kBack) g += kAtOnce * gin.head;
      }
    }
  };
  // Backward and ONE: the next unit's row of the table is in flight too, by a position that was
  // loaded a unit earlier still (the rotation is the first thing done to dz: without this a warp
  // waited for the table for 1700 of the 4300 cycles of a unit).
  constexpr bool kAhead = kBack && ONE;
  float4 next_cos, next_sin;
  int pos_after = -1;  // of the unit after the next
  const auto load_angles = [&](int pos) {
    if (rotated && pos >= 0 && pos < p.max_pos) {
      const float* row = p.cos_sin + (int64_t)pos * p.rot + 4 * item;
      next_cos = *reinterpret_cast<const float4*>(row);
      next_sin = *reinterpret_cast<const float4*>(row + p.rot / 2);
    }
  };
  const auto position = [&](int64_t unit) { return unit < units ? p.positions[by_heads.div((int)unit * kRows)] : -1; };
  Unit next;
  if (u < units) {
    load(next, u);
    if constexpr (kAhead) {
      next.pos[0] = position(u);
      load_angles(next.pos[0]);
      pos_after = position(u + stride);
    }
  }
  for (; u < units; u += stride) {
    Unit now = next;
    Angles angles[ONE || WHICH == 2 ? 1 : kUnroll];
    if constexpr (kAhead) angles[0].set(next_cos, next_sin);
    if (u + stride < units) {
      load(next, u + stride);
      if constexpr (kAhead) {
        next.pos[0] = pos_after;
        load_angles(pos_after);
        pos_after = position(u + 2 * stride);
      }
    }
    const int first = (int)u * kRows;
    // where the rows go, and the angles: all rows' loads before the first is used
    T* dst[kUnroll];
    bool write[kUnroll], skip[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (ONE && i > 0) {
        skip[i] = skip[0];
        write[i] = write[0];
        dst[i] = dst[i - 1] + kAtOnce * out.head;
        continue;
      }
      const int row = first + sub + i * kAtOnce;
      const int t = by_heads.div(ONE ? first : min(row, rows - 1)), h = row - t * by_heads.d;
      const int pos = now.pos[i];
      skip[i] = pos < 0 || pos >= p.max_pos;
      if (pos >= p.max_pos) status |= THD_DEV_BAD_POSITION;
      if constexpr (kCached) {
        const int slot = p.slot_map[t];
        if (slot >= p.num_slots) status |= THD_DEV_BAD_PAGE;
        write[i] = !skip[i] && cache_row(p, WHICH, slot, dst[i]);
        dst[i] += (int64_t)h * out.head;
      } else {
        dst[i] = out.at(static_cast<T*>(p.out[WHICH]), t, h);
        write[i] = !skip[i] || p.zero_skipped;
      }
      write[i] = write[i] && active && (ONE || row < rows);
      if constexpr (WHICH < 2 && !kAhead)
        if (rotated && !skip[i]) angles[i].load(p.cos_sin + (int64_t)pos * p.rot + 4 * item, p.rot / 2);
    }
    if constexpr (WHICH == 2) {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (write[i]) now.x[i].store(dst[i], e0, e1);
    } else if constexpr (!kBack) {
      Eight x[kUnroll];
      float ss[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        x[i].template get<T, ADJ>(now.x[i]);
        ss[i] = dot(x[i], x[i]);
      }
      const float r_mine = rsqrtf(sum_each<G, kUnroll>(ss) * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const float r = __shfl_sync(0xffffffffu, r_mine, i * (G / kUnroll), G);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i].v[k] = ptx::f2_mul(ptx::f2_mul(x[i].v[k], both(r)), w.v[k]);
        if (rotated && !skip[i]) angles[ONE ? 0 : i].template turn<false>(x[i]);
        Raw<T> raw;
        if (skip[i]) raw.zero();
        else x[i].template put<T, ADJ>(raw);
        if (write[i]) raw.store(dst[i], e0, e1);
      }
    } else {
      // two rows at a time: dx = r a + c x with a = g w, c = -r^3 <a, x> / d
#pragma unroll
      for (int i = 0; i < kUnroll; i += 2) {
        Eight x[2], g[2], a[2];
        float sums[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[j].template get<T, ADJ>(now.x[i + j]);
          g[j].template get<T, ADJ>(now.g[i + j]);
          if (rotated && !skip[i + j]) angles[ONE ? 0 : i + j].template turn<true>(g[j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) a[j].v[k] = ptx::f2_mul(g[j].v[k], w.v[k]);
          sums[j] = dot(x[j], x[j]);
          sums[2 + j] = dot(a[j], x[j]);
        }
        const float mine = sum_each<G, 4>(sums), other = __shfl_xor_sync(0xffffffffu, mine, G / 2);
        const bool upper = threadIdx.x & (G / 2);
        const float r_mine = rsqrtf((upper ? other : mine) * inv_d + p.eps);
        const float c_mine = -(r_mine * r_mine * r_mine) * ((upper ? mine : other) * inv_d);
        const float give = upper ? c_mine : r_mine;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float r = __shfl_sync(0xffffffffu, give, j * (G / 4), G);
          const float c = __shfl_sync(0xffffffffu, give, (2 + j) * (G / 4), G);
          const bool counts = !skip[i + j] && (ONE || first + sub + (i + j) * kAtOnce < rows);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (counts) acc.v[k] = ptx::f2_fma(g[j].v[k], ptx::f2_mul(x[j].v[k], both(r)), acc.v[k]);
            x[j].v[k] = ptx::f2_fma(x[j].v[k], both(c), ptx::f2_mul(a[j].v[k], both(r)));
          }
          Raw<T> raw;
          if (skip[i + j]) raw.zero();
          else x[j].template put<T, ADJ>(raw);
          if (write[i + j]) raw.store(dst[i + j], e0, e1);
        }
      }
    }
  }
  u -= units;
}

// Blocks of an SM: with the next unit in flight, 20 to 24 warps of 2 KB (16 bits, forward) or
// 12 of 4 KB keep the 45 KB in flight that the memory's latency takes. (Loading each row of
// the next unit as soon as this unit's is taken holds half the registers, but spreads the
// loads between the computations: 140 us instead of 113 for the forward, 134 instead of 107
// for the backward.)
constexpr int norm_rope_blocks(int elem, int form, bool one) {
  return form == THD_NORM_ROPE_BWD || elem == 4 ? 3 : !one ? 4 : form == THD_NORM_ROPE_PAGED ? 5 : 6;
}

// ONEQ / ONEK: see rows_of.
template <typename T, int G, int FORM, bool ADJ, bool ONEQ, bool ONEK>
__global__ void __launch_bounds__(kThreads, norm_rope_blocks(sizeof(T), FORM, ONEK)) norm_rope_kernel(NormRopeParams p) {
  constexpr bool kBack = FORM == THD_NORM_ROPE_BWD;
  ptx::pdl_wait();
  ptx::pdl_release();
  __shared__ float part[kBack ? kWarps : 1][2][kBack ? G * 8 : 1];
  uint32_t status = 0;
  int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  Eight acc;
  // the block's weight gradients: over the warp's groups, then over the warps in order
  const auto flush = [&](int which) {
    const int lane = threadIdx.x & 31, item = lane % G;
    const bool rotated = item * 8 < p.rot;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[2];
      ptx::f2_unpack(acc.v[k], v[0], v[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int s = G; s < 32; s <<= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], s);
        // pair number and half of v[j], see Eight
        const int pair = (k & 1) * 2 + j, b = k >> 1;
        const int e = ADJ ? 8 * item + 2 * pair + b
                          : rotated ? (b ? p.rot / 2 : 0) + 4 * item + pair : 8 * item + 4 * b + pair;
        if (lane < G && item * 8 < p.d) part[threadIdx.x / 32][which][e] = v[j];
      }
      acc.v[k] = 0;
    }
  };
#pragma unroll
  for (int k = 0; k < 4; ++k) acc.v[k] = 0;
  rows_of<T, G, FORM, ADJ, ONEQ, 0>(p, u, acc, status);
  if constexpr (kBack) flush(0);
  rows_of<T, G, FORM, ADJ, ONEK, 1>(p, u, acc, status);
  if constexpr (kBack) {
    flush(1);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
      const int j = i / p.d, e = i - j * p.d;
      float v = 0.f;
#pragma unroll
      for (int wp = 0; wp < kWarps; ++wp) v += part[wp][j][e];
      p.part_dw[(int64_t)blockIdx.x * 2 * p.d + i] = v;
    }
  }
  if constexpr (FORM == THD_NORM_ROPE_PAGED) rows_of<T, G, FORM, ADJ, ONEK, 2>(p, u, acc, status);
  write_status(p.status, status);
}

// Any d <= 256, any rot, any strides: a warp per (row, head), elements strided over
// the lanes, partners exchanged through shared memory.
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(NormRopeParams p) {
  constexpr bool kBack = FORM == THD_NORM_ROPE_BWD;
  constexpr bool kPaged = FORM == THD_NORM_ROPE_PAGED;
  __shared__ float buf[kWarps][256];
  __shared__ float part[kBack ? kWarps : 1][2][kBack ? 256 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int per_token = p.h_q + p.h_kv * (kPaged ? 2 : 1);
  const int64_t units = (int64_t)p.rows * per_token;
  const int half = p.rot / 2;
  ptx::pdl_wait();
  ptx::pdl_release();
  uint32_t status = 0;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;

  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(u / per_token);
    int h = (int)(u - (int64_t)t * per_token);
    const int which = h < p.h_q ? 0 : h < p.h_q + p.h_kv ? 1 : 2;
    h -= which == 0 ? 0 : which == 1 ? p.h_q : p.h_q + p.h_kv;
    const int pos = p.positions[t];
    const bool skip = pos < 0 || pos >= p.max_pos;
    if (pos >= p.max_pos) status |= THD_DEV_BAD_POSITION;
    T* dst;
    bool write;
    if (kPaged && which != 0) {
      const int slot = p.slot_map[t];
      if (slot >= p.num_slots) status |= THD_DEV_BAD_PAGE;
      write = !skip && cache_row(p, which, slot, dst);
    } else {
      dst = static_cast<T*>(p.out[which]) + (int64_t)t * p.out_tok[which];
      write = !skip || p.zero_skipped;
    }
    if (!write) continue;
    dst += (int64_t)h * p.out_head[which];
    const T* x = static_cast<const T*>(p.in[which]) + (int64_t)t * p.in_tok[which] + (int64_t)h * p.in_head[which];
    if (which == 2) {
      for (int e = lane; e < p.d; e += 32) dst[e] = x[e];
      continue;
    }
    if (skip) {
      for (int e = lane; e < p.d; e += 32) dst[e] = from_f<T>(0.f);
      continue;
    }
    const T* wr = static_cast<const T*>(p.w[which]);
    const float* angles = p.cos_sin + (int64_t)pos * p.rot;
    float v[8], w[8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < p.d ? to_f(x[e]) : 0.f;
      w[i] = e < p.d && wr ? to_f(wr[e]) : 1.f;
      ss += v[i] * v[i];
    }
    const float r = rsqrtf(group_sum<32>(ss) / (float)p.d + p.eps);
    const T* gz = nullptr;
    if constexpr (kBack)
      gz = static_cast<const T*>(p.in[2 + which]) + (int64_t)t * p.in_tok[2 + which] +
           (int64_t)h * p.in_head[2 + which];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < p.d) buf[warp][e] = kBack ? to_f(gz[e]) : v[i] * r * w[i];
    }
    __syncwarp();
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e >= p.d) {
        z[i] = 0.f;
      } else if (e >= p.rot) {
        z[i] = buf[warp][e];
      } else {
        const int pair = p.interleaved ? e / 2 : (e < half ? e : e - half);
        const bool first = p.interleaved ? (e & 1) == 0 : e < half;
        const int other = p.interleaved ? (e ^ 1) : (first ? e + half : e - half);
        const float sn = kBack ? -angles[half + pair] : angles[half + pair];
        const float mine = buf[warp][e], theirs = buf[warp][other];
        z[i] = first ? mine * angles[pair] - theirs * sn : mine * angles[pair] + theirs * sn;
      }
    }
    if constexpr (kBack) {
      float ax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ax += z[i] * w[i] * v[i];
      const float mean = group_sum<32>(ax) * r / (float)p.d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = v[i] * r, gx = z[i] * xh;
        dw[0][i] += which == 0 ? gx : 0.f;
        dw[1][i] += which == 0 ? 0.f : gx;
        z[i] = r * (z[i] * w[i] - xh * mean);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < p.d) dst[e] = from_f<T>(z[i]);
    }
  }
  if constexpr (kBack) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) part[warp][j][lane + 32 * i] = dw[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
      const int j = i / p.d, e = i - j * p.d;
      float s = 0.f;
#pragma unroll
      for (int wp = 0; wp < kWarps; ++wp) s += part[wp][j][e];
      p.part_dw[(int64_t)blockIdx.x * 2 * p.d + i] = s;
    }
  }
  write_status(p.status, status);
}

// dw = sum over the blocks' partial rows in a fixed order: 8 columns (a 32-byte sector) to a
// block, 64 rows at a time, then over the 64 in shared memory.
constexpr int kDwColumns = 8, kDwRows = 64;
__global__ void __launch_bounds__(kDwColumns * kDwRows) norm_rope_dw_kernel(NormRopeParams p, int blocks) {
  __shared__ float part[kDwRows][kDwColumns + 1];
  ptx::pdl_wait();
  ptx::pdl_release();
  const int x = threadIdx.x % kDwColumns, y = threadIdx.x / kDwColumns;
  const int col = blockIdx.x * kDwColumns + x;
  float v = 0.f;
  if (col < 2 * p.d) {
#pragma unroll 8
    for (int b = y; b < blocks; b += kDwRows) v += p.part_dw[(int64_t)b * 2 * p.d + col];
  }
  part[y][x] = v;
  __syncthreads();
  if (threadIdx.x >= 32 * kDwColumns) return;
  const int lane = threadIdx.x & 31, c = threadIdx.x / 32, e = blockIdx.x * kDwColumns + c;
  v = group_sum<32>(part[lane][c] + part[lane + 32][c]);
  if (lane == 0 && e < 2 * p.d) {
    float* dw = p.dw[e < p.d ? 0 : 1];
    if (dw) dw[e < p.d ? e : e - p.d] = v;
  }
}

template <typename T, int G, int FORM, bool ADJ>
cudaError_t launch_vec(const NormRopeParams& p, int sms, cudaStream_t stream, int& blocks) {
  constexpr int kRows = 32 / G * norm_rope_unroll(sizeof(T), FORM == THD_NORM_ROPE_BWD);
  const bool one_q = p.h_q % kRows == 0, one_k = one_q && p.h_kv % kRows == 0;
  const int64_t tensors = FORM == THD_NORM_ROPE_PAGED ? 2 : 1;
  const int64_t units = ((int64_t)p.rows * p.h_q + kRows - 1) / kRows +
                        tensors * (((int64_t)p.rows * p.h_kv + kRows - 1) / kRows);
  blocks = sms * norm_rope_blocks(sizeof(T), FORM, one_k);
  if (units < (int64_t)blocks * kWarps) blocks = units > 0 ? (int)((units + kWarps - 1) / kWarps) : 1;
  const auto kernel = one_k   ? norm_rope_kernel<T, G, FORM, ADJ, true, true>
                      : one_q ? norm_rope_kernel<T, G, FORM, ADJ, true, false>
                              : norm_rope_kernel<T, G, FORM, ADJ, false, false>;
  return launch_overlapped(kernel, blocks, kThreads, 0, stream, p);
}

template <typename T, int FORM>
cudaError_t launch_form(const NormRopeParams& p, bool vec, int num_sms, cudaStream_t stream) {
  const int sms = num_sms < kMaxSmsForSizing ? num_sms : kMaxSmsForSizing;
  int blocks = 1;
  cudaError_t e;
  if (!vec) {
    const int64_t units = (int64_t)p.rows * (p.h_q + (int64_t)p.h_kv * (FORM == THD_NORM_ROPE_PAGED ? 2 : 1));
    blocks = sms * 8;
    if (units < (int64_t)blocks * kWarps) blocks = units > 0 ? (int)((units + kWarps - 1) / kWarps) : 1;
    e = launch_overlapped(norm_rope_any_kernel<T, FORM>, blocks, kThreads, 0, stream, p);
  } else if (p.interleaved) {
    e = p.d <= 64    ? launch_vec<T, 8, FORM, true>(p, sms, stream, blocks)
        : p.d <= 128 ? launch_vec<T, 16, FORM, true>(p, sms, stream, blocks)
                     : launch_vec<T, 32, FORM, true>(p, sms, stream, blocks);
  } else {
    e = p.d <= 64    ? launch_vec<T, 8, FORM, false>(p, sms, stream, blocks)
        : p.d <= 128 ? launch_vec<T, 16, FORM, false>(p, sms, stream, blocks)
                     : launch_vec<T, 32, FORM, false>(p, sms, stream, blocks);
  }
  if (e != cudaSuccess || FORM != THD_NORM_ROPE_BWD || !(p.dw[0] || p.dw[1])) return e;
  return launch_overlapped(norm_rope_dw_kernel, (2 * p.d + kDwColumns - 1) / kDwColumns, kDwColumns * kDwRows, 0, stream,
                           p, blocks);
}

}  // namespace

// The operator for one storage type: included by one source file for each.
template <typename T>
cudaError_t norm_rope_type(const NormRopeParams& p, thd_norm_rope_form_t form, bool vec, int num_sms,
                           cudaStream_t stream) {
  switch (form) {
    case THD_NORM_ROPE_FWD: return launch_form<T, THD_NORM_ROPE_FWD>(p, vec, num_sms, stream);
    case THD_NORM_ROPE_BWD: return launch_form<T, THD_NORM_ROPE_BWD>(p, vec, num_sms, stream);
    default: return launch_form<T, THD_NORM_ROPE_PAGED>(p, vec, num_sms, stream);
  }
}

}  // namespace thd
