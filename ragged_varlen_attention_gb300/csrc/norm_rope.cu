// Per-head RMS norm with the position rotation: forward, backward, and the serving
// form that writes K and V into the paged cache.
//
//   r = 1/sqrt(mean x^2 + eps), y = x r w, z = R(pos) y on the first rot elements
//   backward: g = R(pos)^T dz, a = g w, xh = x r, dx = r (a - xh mean(a xh)), dw = sum g xh
//
// Every element is read once and written once; the arithmetic is a few fma per
// element, so memory bounds all three forms. A head is one group of G = 8 .. 32
// lanes with 8 elements each, and its sums are shuffles inside the group. A rotated
// pair never leaves its lane: in the halves layout lane i holds elements 4i .. 4i+3
// and their partners rot/2 + 4i .., in the adjacent layout 8i .. 8i+7. A warp's unit
// is one token x kUnroll x (32/G) heads of one tensor, so that the loads of all its
// heads are in flight together and the rotation's row and the weight are read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace thd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;

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

// four consecutive elements as loaded (8 bytes, or 16 of float32)
template <typename T>
struct Quad {
  uint2 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { raw = make_uint2(0u, 0u); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint2*>(p) = raw; }
  __device__ __forceinline__ void get(float* f) const {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = to_f(e[i]);
  }
  __device__ __forceinline__ void set(const float* f) {
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = from_f<T>(f[i]);
  }
};
template <>
struct Quad<float> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = raw; }
  __device__ __forceinline__ void get(float* f) const { f[0] = raw.x; f[1] = raw.y; f[2] = raw.z; f[3] = raw.w; }
  __device__ __forceinline__ void set(const float* f) { raw = make_float4(f[0], f[1], f[2], f[3]); }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// z = R y for the lane's 8 elements (BACK: the transpose). c and s are the 4 angles
// of the lane's pairs: (k, k + 4) in the halves layout, (2k, 2k + 1) in the adjacent one.
template <bool BACK>
__device__ __forceinline__ void rotate(float (&y)[8], const float (&c)[4], const float (&s)[4], bool interleaved) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float sn = BACK ? -s[k] : s[k];
    const float a = interleaved ? y[2 * k] : y[k];
    const float b = interleaved ? y[2 * k + 1] : y[k + 4];
    const float za = a * c[k] - b * sn, zb = b * c[k] + a * sn;
    if (interleaved) {
      y[2 * k] = za;
      y[2 * k + 1] = zb;
    } else {
      y[k] = za;
      y[k + 4] = zb;
    }
  }
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

template <typename T, int G, int FORM>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeParams p) {
  constexpr bool kBack = FORM == THD_NORM_ROPE_BWD;
  constexpr bool kPaged = FORM == THD_NORM_ROPE_PAGED;
  constexpr int kHeadsAtOnce = 32 / G;
  constexpr int kHeads = kHeadsAtOnce * kUnroll;
  const int lane = threadIdx.x & 31;
  const int item = lane % G, sub = lane / G;
  const bool active = item * 8 < p.d;
  const bool rotated = item * 8 < p.rot;
  const int e0 = rotated && !p.interleaved ? 4 * item : 8 * item;
  const int e1 = rotated && !p.interleaved ? p.rot / 2 + 4 * item : 8 * item + 4;
  const float inv_d = 1.f / (float)p.d;

  const int cq = (p.h_q + kHeads - 1) / kHeads, ck = (p.h_kv + kHeads - 1) / kHeads;
  const int per_token = cq + ck + (kPaged ? ck : 0);
  const int64_t units = (int64_t)p.rows * per_token;
  ptx::pdl_wait();
  ptx::pdl_release();
  uint32_t status = 0;
  float dw[2][8];
  if constexpr (kBack) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  }

  for (int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; u < units; u += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(u / per_token);
    int c = (int)(u - (int64_t)t * per_token);
    const int which = c < cq ? 0 : c < cq + ck ? 1 : 2;
    c -= which == 0 ? 0 : which == 1 ? cq : cq + ck;
    const int heads = which == 0 ? p.h_q : p.h_kv;
    const int head0 = c * kHeads + sub;
    // the unit's loads, all in flight before the position is looked at
    const T* x = static_cast<const T*>(p.in[which]) + (int64_t)t * p.in_tok[which];
    Quad<T> lo[kUnroll], hi[kUnroll], glo[kBack ? kUnroll : 1], ghi[kBack ? kUnroll : 1];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = head0 + i * kHeadsAtOnce;
      if (active && h < heads) {
        const T* row = x + (int64_t)h * p.in_head[which];
        lo[i].load(row + e0);
        hi[i].load(row + e1);
        if constexpr (kBack) {
          const T* grow = static_cast<const T*>(p.in[2 + which]) + (int64_t)t * p.in_tok[2 + which] +
                          (int64_t)h * p.in_head[2 + which];
          glo[i].load(grow + e0);
          ghi[i].load(grow + e1);
        }
      } else {
        lo[i].zero();
        hi[i].zero();
        if constexpr (kBack) {
          glo[i].zero();
          ghi[i].zero();
        }
      }
    }
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
    float cs[4], sn[4], w[8];
    if (which != 2 && !skip) {
      if (rotated) {
        const float* row = p.cos_sin + (int64_t)pos * p.rot + 4 * item;
        const float4 a = *reinterpret_cast<const float4*>(row);
        const float4 b = *reinterpret_cast<const float4*>(row + p.rot / 2);
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
        sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
      }
      if (p.w[which] && active) {
        const T* wr = static_cast<const T*>(p.w[which]);
        Quad<T> a, b;
        a.load(wr + e0);
        b.load(wr + e1);
        a.get(w);
        b.get(w + 4);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 1.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = head0 + i * kHeadsAtOnce;
      if (which != 2) {
        float v[8];
        lo[i].get(v);
        hi[i].get(v + 4);
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += v[k] * v[k];
        if (skip) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.f;
        } else if constexpr (!kBack) {
          const float r = rsqrtf(group_sum<G>(ss) * inv_d + p.eps);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[k] * r * w[k];
          if (rotated) rotate<false>(v, cs, sn, p.interleaved);
        } else {
          float g[8];
          glo[i].get(g);
          ghi[i].get(g + 4);
          if (rotated) rotate<true>(g, cs, sn, p.interleaved);
          float ax = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) ax += g[k] * w[k] * v[k];
          const float r = rsqrtf(group_sum<G>(ss) * inv_d + p.eps);
          const float mean = group_sum<G>(ax) * r * inv_d;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = v[k] * r;
            const float gx = h < heads ? g[k] * xh : 0.f;  // xh of no head at all may be 0 * inf
            dw[0][k] += which == 0 ? gx : 0.f;
            dw[1][k] += which == 0 ? 0.f : gx;
            v[k] = r * (g[k] * w[k] - xh * mean);
          }
        }
        lo[i].set(v);
        hi[i].set(v + 4);
      }
      if (active && h < heads) {
        T* row = dst + (int64_t)h * p.out_head[which];
        lo[i].store(row + e0);
        hi[i].store(row + e1);
      }
    }
  }

  if constexpr (kBack) {
    // the block's weight gradients: over the warp's groups, then over the warps in order
    __shared__ float part[kWarps][2][G * 8];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v = dw[j][k];
#pragma unroll
        for (int s = G; s < 32; s <<= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        if (sub == 0 && active) part[threadIdx.x / 32][j][k < 4 ? e0 + k : e1 + k - 4] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
      const int j = i / p.d, e = i - j * p.d;
      float v = 0.f;
#pragma unroll
      for (int wp = 0; wp < kWarps; ++wp) v += part[wp][j][e];
      p.part_dw[(int64_t)blockIdx.x * 2 * p.d + i] = v;
    }
  }
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

// dw = sum over the blocks' partial rows, 32 columns to a block, in a fixed order.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(NormRopeParams p, int blocks) {
  __shared__ float part[32][33];
  ptx::pdl_wait();
  ptx::pdl_release();
  const int col = blockIdx.x * 32 + threadIdx.x % 32, row = threadIdx.x / 32;
  float v = 0.f;
  if (col < 2 * p.d)
    for (int b = row; b < blocks; b += 32) v += p.part_dw[(int64_t)b * 2 * p.d + col];
  part[row][threadIdx.x % 32] = v;
  __syncthreads();
  v = group_sum<32>(part[threadIdx.x % 32][row]);
  const int c = blockIdx.x * 32 + row;
  if (threadIdx.x % 32 == 0 && c < 2 * p.d) {
    float* dw = p.dw[c < p.d ? 0 : 1];
    if (dw) dw[c < p.d ? c : c - p.d] = v;
  }
}

template <typename T, int FORM>
cudaError_t launch_form(const NormRopeParams& p, bool vec, int num_sms, cudaStream_t stream) {
  const int sms = num_sms < kMaxSmsForSizing ? num_sms : kMaxSmsForSizing;
  const int g = p.d <= 64 ? 8 : p.d <= 128 ? 16 : 32;
  const int heads = vec ? 32 / g * kUnroll : 1;
  const int64_t per_token = (p.h_q + heads - 1) / heads + (int64_t)((p.h_kv + heads - 1) / heads) *
                                                              (FORM == THD_NORM_ROPE_PAGED ? 2 : 1);
  const int64_t need = (p.rows * per_token + kWarps - 1) / kWarps;
  int blocks = sms * 8;
  if (need < blocks) blocks = need > 0 ? (int)need : 1;
  const auto kernel = !vec ? norm_rope_any_kernel<T, FORM>
                      : g == 8 ? norm_rope_kernel<T, 8, FORM>
                      : g == 16 ? norm_rope_kernel<T, 16, FORM>
                                : norm_rope_kernel<T, 32, FORM>;
  const cudaError_t e = launch_overlapped(kernel, blocks, kThreads, 0, stream, p);
  if (e != cudaSuccess || FORM != THD_NORM_ROPE_BWD || !(p.dw[0] || p.dw[1])) return e;
  return launch_overlapped(norm_rope_dw_kernel, (2 * p.d + 31) / 32, 1024, 0, stream, p, blocks);
}

template <typename T>
cudaError_t launch_type(const NormRopeParams& p, thd_norm_rope_form_t form, bool vec, int num_sms,
                        cudaStream_t stream) {
  switch (form) {
    case THD_NORM_ROPE_FWD: return launch_form<T, THD_NORM_ROPE_FWD>(p, vec, num_sms, stream);
    case THD_NORM_ROPE_BWD: return launch_form<T, THD_NORM_ROPE_BWD>(p, vec, num_sms, stream);
    default: return launch_form<T, THD_NORM_ROPE_PAGED>(p, vec, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, thd_dtype_t dtype, thd_norm_rope_form_t form, bool vec,
                             int num_sms, cudaStream_t stream) {
  switch (dtype) {
    case THD_BF16: return launch_type<__nv_bfloat16>(p, form, vec, num_sms, stream);
    case THD_FP16: return launch_type<__half>(p, form, vec, num_sms, stream);
    default: return launch_type<float>(p, form, vec, num_sms, stream);
  }
}

}  // namespace thd
