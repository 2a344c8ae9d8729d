// Attention of one new token per request over a paged key-value cache.
//
//   s_j = scale <q, k_j>, O = sum_j softmax(s)_j v_j, LSE = ln sum_j exp s_j
//
// Every visible K and V row is read once and used by the query heads of its group
// only: 2 G operations per byte in 16 bits, far below the tensor cores' rate, so
// memory bounds the kernel. What matters is that every SM streams at its share of
// the bandwidth until the end, whatever the lengths are:
//   - A segment is (request, kv head, up to 8/16/32 query heads of its group). All
//     segments' key tiles (64 keys) form one line, and CTA c of n takes the tiles
//     [c W / n, (c + 1) W / n) of it, across segment borders. The border positions
//     follow from the lengths on the device; no setup kernel, no work list.
//   - Each warp streams its own 16 of a tile's 64 keys through its own ring of
//     cp.async stages and keeps its own running maximum, sum and output; warps meet
//     only at the end of a segment, where their four results are joined.
//   - A segment that lies inside one CTA is finished there. One that crosses a border
//     leaves normalised partial outputs in the workspace, and the join kernel merges
//     them in CTA order (no atomics: equal inputs give equal bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace thd {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;                    // keys of a warp's stage
constexpr int kTile = kChunk * kWarps;        // keys of a CTA's step
static_assert(kTile == kDecodeKeysPerTile, "the plan's bound counts these tiles");
constexpr float kLn2 = 0.69314718055994530942f;

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

// ------------------------------------------------------------------ schedule
// Visible keys [lo, n) of a request; `base` = lo rounded down to a chunk.
struct Span {
  int32_t n, lo, base, tiles;
  bool bad;
};
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  s.n = p.seq_lens[b];
  s.bad = s.n < 0 || (int64_t)s.n > (int64_t)p.max_pages * p.page_size;
  if (s.bad) s.n = 0;
  const int w = p.window ? p.window[b] : -1;
  s.lo = w >= 0 && w < s.n - 1 ? s.n - 1 - w : 0;
  s.base = s.lo & ~(kChunk - 1);
  s.tiles = (s.n - s.base + kTile - 1) / kTile;
  return s;
}

// Position in the line of tiles: request b, segment seg of its `segs`, tile of the
// segment; sp is the request's span.
struct Cursor {
  int32_t b, seg, tile;
  Span sp;
  // the next request with keys (the caller knows that there is one)
  __device__ __forceinline__ void skip_empty(const DecodeParams& p) {
    const int lane = threadIdx.x & 31;
    while (b < p.batch) {
      const int mine = b + lane;
      const bool some = mine < p.batch && span_of(p, mine).tiles > 0;
      const uint32_t any = __ballot_sync(0xffffffffu, some);
      if (any) {
        b += __ffs(any) - 1;
        sp = span_of(p, b);
        return;
      }
      b += 32;
    }
  }
  __device__ __forceinline__ void advance(const DecodeParams& p, int segs, bool more) {
    if (++tile < sp.tiles) return;
    tile = 0;
    if (++seg < segs) return;
    seg = 0;
    ++b;
    if (more) skip_empty(p);
  }
};

struct Range {
  int64_t total, begin, end;
  int32_t ctas;
};

// First tile of CTA c of n over a line of w tiles.
__device__ __forceinline__ int64_t cta_start(int64_t c, int64_t w, int32_t n) { return c * w / n; }

// The CTA's range and the cursor at its beginning. Every thread calls it.
__device__ __forceinline__ Range locate(const DecodeParams& p, int segs, Cursor& cur, uint32_t& status) {
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int32_t found_b;
  __shared__ int64_t found_before;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int strip = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, (int)threadIdx.x * strip), b1 = min(p.batch, b0 + strip);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Span s = span_of(p, b);
    if (s.bad) status |= THD_DEV_BAD_LENGTH;
    mine += s.tiles;
  }
  int64_t upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += o;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  Range r;
  r.total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += warp_sums[w];
    r.total += warp_sums[w];
  }
  r.total *= segs;
  r.ctas = (int32_t)min64(gridDim.x, max64(r.total, 1));
  r.begin = r.end = 0;
  if ((int)blockIdx.x < r.ctas) {
    r.begin = cta_start(blockIdx.x, r.total, r.ctas);
    r.end = cta_start(blockIdx.x + 1, r.total, r.ctas);
  }
  if (r.begin < r.end) {
    int64_t before = (upto - mine) * segs;
    if (before <= r.begin && r.begin < upto * segs) {
      for (int b = b0; b < b1; ++b) {
        const int64_t n = (int64_t)span_of(p, b).tiles * segs;
        if (r.begin < before + n) {
          found_b = b;
          found_before = before;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    cur.b = found_b;
    cur.sp = span_of(p, cur.b);
    const int64_t rel = r.begin - found_before;
    cur.seg = (int)(rel / cur.sp.tiles);
    cur.tile = (int)(rel - (int64_t)cur.seg * cur.sp.tiles);
  }
  return r;
}

// Rows without a visible key: O = 0, LSE = -inf.
template <typename T>
__device__ __forceinline__ void write_empty(const DecodeParams& p) {
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    const Span s = span_of(p, b);
    if (s.bad || s.tiles > 0) continue;
    for (int i = threadIdx.x; i < p.h_q * p.d; i += kThreads) {
      const int h = i / p.d, e = i - h * p.d;
      static_cast<T*>(p.o)[(int64_t)b * p.o_tok + (int64_t)h * p.o_head + e] = from_f<T>(0.f);
      if (e == 0 && p.stats) p.stats[(int64_t)b * p.stats_tok + (int64_t)h * p.stats_head] = -INFINITY;
    }
  }
}

// First query head of a segment, and how many it has.
template <int HEADS>
__device__ __forceinline__ int segment_heads(const DecodeParams& p, int seg, int& head0) {
  const int per = (p.group + HEADS - 1) / HEADS;
  const int g = seg / per, c = seg - g * per;
  head0 = g * p.group + c * HEADS;
  return min(HEADS, p.group - c * HEADS);
}

// Joins the four warps' results for 8 heads of a segment (`h8` the first of them) and
// writes the rows, or the partial rows when the segment goes on in another CTA.
// part_max / part_sum / part_o hold each warp's base-2 maximum, sum and output.
template <typename T, int D, int HEADS>
__device__ __forceinline__ void join_warps(const DecodeParams& p, const float (&part_max)[kWarps][8],
                                           const float (&part_sum)[kWarps][8],
                                           const float (&part_o)[kWarps][8][D + 4], int b, int head0, int heads,
                                           int h8, int slot) {
  for (int i = threadIdx.x; i < 8 * (D / 4); i += kThreads) {
    const int h = i / (D / 4), e = (i - h * (D / 4)) * 4;
    float top = part_max[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, part_max[w][h]);
    const bool dead = top == -INFINITY;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!dead) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(part_max[w][h] - top);
        const float4 a = *reinterpret_cast<const float4*>(&part_o[w][h][e]);
        sum += f * part_sum[w][h];
        o.x += f * a.x; o.y += f * a.y; o.z += f * a.z; o.w += f * a.w;
      }
    }
    const float inv = dead ? 0.f : 1.f / sum;
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    const float lse2 = dead ? -INFINITY : top + log2f(sum);
    if (slot >= 0) {
      const int64_t row = (int64_t)slot * HEADS + h8 + h;
      *reinterpret_cast<float4*>(p.part_o + row * D + e) = o;
      if (e == 0) p.part_lse[row] = lse2;
    } else if (h8 + h < heads) {
      T* dst = static_cast<T*>(p.o) + (int64_t)b * p.o_tok + (int64_t)(head0 + h8 + h) * p.o_head;
      const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + k < p.d) dst[e + k] = from_f<T>(v[k]);
      if (e == 0 && p.stats)
        p.stats[(int64_t)b * p.stats_tok + (int64_t)(head0 + h8 + h) * p.stats_head] = dead ? -INFINITY : lse2 * kLn2;
    }
  }
}

// What the CTA records for the join kernel.
__device__ __forceinline__ void write_record(const DecodeParams& p, const Range& range, const Cursor& cur) {
  if (threadIdx.x != 0) return;
  if (blockIdx.x == 0) {
    p.total[0] = range.total;
    p.total[1] = range.ctas;
  }
  DecodeRec rec = {0, 0, 0, 0};
  if (range.begin < range.end) rec = {cur.b, cur.seg, cur.sp.tiles, cur.tile};
  p.recs[blockIdx.x] = rec;
}

// ------------------------------------------------------------- matrix pieces
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int bytes = real ? 16 : 0;  // 0: the 16 bytes are zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// d += a (16 x 16, row) * b (16 x 8, column)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// ------------------------------------------------- matrix-instruction kernel
// A stage's 16 keys are the 16 rows of the instruction and the query heads its 8
// columns: S^T = K Q^T, then O^T += V^T P^T, so a group of 8 heads fills the tile (the
// other way round heads would be padded to 16). P^T's fragment is S^T's, transposed 8 x 8
// by movmatrix; P is rounded to the storage type for the product (at most half a step
// of a value <= 1), its sum is kept in float32.
template <int D>
struct MmaSmem {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kStageBytes = 2 * kChunk * kRowBytes;  // K rows, then V rows
  unsigned char ring[kWarps][kStages][kStageBytes];
  float part_o[kWarps][8][D + 4];
  float part_max[kWarps][8], part_sum[kWarps][8];
  uint32_t seen[kWarps][kStages];  // bit r: key r of the stage is visible
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kDecodeCtasPerSm) paged_decode_mma_kernel(DecodeParams p) {
  using Smem = MmaSmem<D>;
  constexpr int kStages = Smem::kStages;
  constexpr int kHeads = 8 * NT;
  constexpr int kRowBytes = Smem::kRowBytes;
  constexpr int kVecs = D / 8;            // 16-byte pieces of a row
  constexpr int kRowsAtOnce = 32 / kVecs; // rows one warp-wide cp.async covers
  extern __shared__ __align__(128) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int per = (p.group + kHeads - 1) / kHeads;   // segments of a kv head
  const int segs = p.h_kv * per;
  uint32_t status = 0;
  Cursor cur;
  const Range range = locate(p, segs, cur, status);
  write_record(p, range, cur);
  write_empty<T>(p);

  const int steps = (int)(range.end - range.begin);  // below 2^31 by the plan's bound
  Cursor load = cur;
  int issued = 0;
  // the page of key `lane` of the warp's chunk at `load` (-1: none), looked up one step
  // before it is used
  const int vec = lane % kVecs, row_in = lane / kVecs;
  const bool vec_real = vec * 8 < p.d;
  int key_page = -1, key_row = 0;
  auto look_up = [&]() {
    key_page = -1;
    if (issued >= steps) return;
    const int key = load.sp.base + load.tile * kTile + warp * kChunk + (lane & (kChunk - 1));
    if (key >= load.sp.lo && key < load.sp.n) {
      const int column = key / p.page_size;
      key_row = key - column * p.page_size;
      key_page = p.block_table[(int64_t)load.b * p.table_stride + column];
      if (key_page < 0 || key_page >= p.num_pages) {
        status |= THD_DEV_BAD_PAGE;
        key_page = -1;
      }
    }
  };
  auto issue = [&]() {
    if (issued < steps) {
      const int stage = issued % kStages;
      const uint32_t seen = __ballot_sync(0xffffffffu, key_page >= 0) & 0xffffu;
      if (lane == 0) sm.seen[warp][stage] = seen;
      const uint32_t dst = ptx::smem_u32(sm.ring[warp][stage]);
      const int g = load.seg / per;
      const T* kh = static_cast<const T*>(p.k) + (int64_t)g * p.k_head + vec * 8;
      const T* vh = static_cast<const T*>(p.v) + (int64_t)g * p.v_head + vec * 8;
#pragma unroll
      for (int i = 0; i < kChunk / kRowsAtOnce; ++i) {
        const int row = i * kRowsAtOnce + row_in;
        const int page = __shfl_sync(0xffffffffu, key_page, row);
        const int in_page = __shfl_sync(0xffffffffu, key_row, row);
        const bool real = page >= 0 && vec_real;
        const uint32_t at = dst + row * kRowBytes + ((vec ^ (row & 7)) << 4);
        const T* ks = static_cast<const T*>(p.k);
        const T* vs = static_cast<const T*>(p.v);
        if (real) {
          ks = kh + (int64_t)page * p.k_page + (int64_t)in_page * p.k_tok;
          vs = vh + (int64_t)page * p.v_page + (int64_t)in_page * p.v_tok;
        }
        cp_async16(at, ks, real);
        cp_async16(at + kChunk * kRowBytes, vs, real);
      }
      ++issued;
      load.advance(p, segs, issued < steps);
      look_up();
    }
    cp_commit();  // an empty group when there is nothing left: the count stays one per step
  };
  look_up();
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t qf[D / 16][NT][2];
  float acc[D / 16][NT][4];
  float top[NT][2], sum[NT][2];
  int head0 = 0, heads = 0, first_tile = 0;
  bool fresh = true;
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      first_tile = cur.tile;
      heads = segment_heads<kHeads>(p, cur.seg, head0);
      const T* q = static_cast<const T*>(p.q) + (int64_t)cur.b * p.q_tok;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + lane / 4;
        const T* row = q + (int64_t)(head0 + h) * p.q_head;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int e = kk * 16 + j * 8 + (lane % 4) * 2;
            qf[kk][nt][j] = h < heads && e < p.d ? *reinterpret_cast<const uint32_t*>(row + e) : 0u;
          }
        top[nt][0] = top[nt][1] = -INFINITY;
        sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[dt][nt][j] = 0.f;
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const int stage = step % kStages;
    const uint32_t seen = sm.seen[warp][stage];
    if (seen != 0) {
      const uint32_t kbase = ptx::smem_u32(sm.ring[warp][stage]);
      const uint32_t vbase = kbase + kChunk * kRowBytes;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      {
        const int row = lane & 15, half = lane >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[4];
          ldsm4(a, kbase + row * kRowBytes + (((kk * 2 + half) ^ (row & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<T>(s[nt], a, qf[kk][nt][0], qf[kk][nt][1]);
        }
      }
      const bool see0 = (seen >> (lane / 4)) & 1, see1 = (seen >> (lane / 4 + 8)) & 1;
      uint32_t pb[NT][2];
      float scale[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[nt][j] = see0 ? s[nt][j] * p.scale_log2 : -INFINITY;
          s[nt][j + 2] = see1 ? s[nt][j + 2] * p.scale_log2 : -INFINITY;
          float m = fmaxf(s[nt][j], s[nt][j + 2]);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          m = fmaxf(m, top[nt][j]);
          const float ref = m == -INFINITY ? 0.f : m;
          scale[nt][j] = exp2f(top[nt][j] - ref);
          moved |= m != top[nt][j];
          top[nt][j] = m;
          s[nt][j] = exp2f(s[nt][j] - ref);
          s[nt][j + 2] = exp2f(s[nt][j + 2] - ref);
          sum[nt][j] = sum[nt][j] * scale[nt][j] + (s[nt][j] + s[nt][j + 2]);
        }
        pb[nt][0] = transpose8x8(pack2<T>(s[nt][0], s[nt][1]));
        pb[nt][1] = transpose8x8(pack2<T>(s[nt][2], s[nt][3]));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[dt][nt][j] *= scale[nt][j & 1];
      }
      {
        // matrices in order: keys 0-7 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 0-7, keys 8-15 / d 8-15
        const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t a[4];
          ldsm4_t(a, vbase + row * kRowBytes + (((dt * 2 + half) ^ (row & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<T>(acc[dt][nt], a, pb[nt][0], pb[nt][1]);
        }
      }
    }
    __syncwarp();  // the stage is read by every lane before it is filled again
    issue();

    const bool last = cur.tile + 1 == cur.sp.tiles || step + 1 == steps;
    if (last) {
      // -1: the CTA holds the whole segment; 2c: it began before CTA c; 2c + 1: it goes on behind it
      const int slot =
          first_tile > 0 ? 2 * (int)blockIdx.x : cur.tile + 1 < cur.sp.tiles ? 2 * (int)blockIdx.x + 1 : -1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= heads) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l = sum[nt][j];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int h = (lane % 4) * 2 + j;
          if (lane < 4) {
            sm.part_max[warp][h] = top[nt][j];
            sm.part_sum[warp][h] = l;
          }
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            sm.part_o[warp][h][dt * 16 + lane / 4] = acc[dt][nt][j];
            sm.part_o[warp][h][dt * 16 + lane / 4 + 8] = acc[dt][nt][j + 2];
          }
        }
        __syncthreads();
        join_warps<T, D, kHeads>(p, sm.part_max, sm.part_sum, sm.part_o, cur.b, head0, heads, nt * 8, slot);
        __syncthreads();
      }
      fresh = true;
    }
    cur.advance(p, segs, step + 1 < steps);
  }
  cp_wait<0>();
  write_status(p.status, kDecodeMaxCtas, status);
}

// --------------------------------------------------------------- SIMT kernel
// float32 caches, and any d <= 128 and alignment: the same schedule and join, each warp's
// 16 keys taken 4 at a time with the head's elements spread over the lanes.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_decode_simt_kernel(DecodeParams p) {
  constexpr int kHeads = 8;
  constexpr int kPer = D / 32;  // elements of a lane: e = lane + 32 i
  constexpr int kKeys = 4;
  __shared__ __align__(16) float part_o[kWarps][8][D + 4];
  __shared__ float part_max[kWarps][8], part_sum[kWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int per = (p.group + kHeads - 1) / kHeads;
  const int segs = p.h_kv * per;
  uint32_t status = 0;
  Cursor cur;
  const Range range = locate(p, segs, cur, status);
  write_record(p, range, cur);
  write_empty<T>(p);

  const int steps = (int)(range.end - range.begin);  // below 2^31 by the plan's bound
  float q[8][kPer], acc[8][kPer], top[8], sum[8];
  int head0 = 0, heads = 0, first_tile = 0;
  bool fresh = true;
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      first_tile = cur.tile;
      heads = segment_heads<kHeads>(p, cur.seg, head0);
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const T* row = static_cast<const T*>(p.q) + (int64_t)cur.b * p.q_tok + (int64_t)(head0 + h) * p.q_head;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          q[h][i] = h < heads && lane + 32 * i < p.d ? to_f(row[lane + 32 * i]) * p.scale_log2 : 0.f;
          acc[h][i] = 0.f;
        }
        top[h] = -INFINITY;
        sum[h] = 0.f;
      }
    }
    const int g = cur.seg / per;
    const T* kh = static_cast<const T*>(p.k) + (int64_t)g * p.k_head;
    const T* vh = static_cast<const T*>(p.v) + (int64_t)g * p.v_head;
    int page = -1, in_page = 0;
    {
      const int key = cur.sp.base + cur.tile * kTile + warp * kChunk + (lane & (kChunk - 1));
      if (key >= cur.sp.lo && key < cur.sp.n) {
        const int column = key / p.page_size;
        in_page = key - column * p.page_size;
        page = p.block_table[(int64_t)cur.b * p.table_stride + column];
        if (page < 0 || page >= p.num_pages) {
          status |= THD_DEV_BAD_PAGE;
          page = -1;
        }
      }
    }
    const uint32_t seen = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    for (int k0 = 0; k0 < kChunk; k0 += kKeys) {
      if (((seen >> k0) & ((1u << kKeys) - 1)) == 0) continue;
      float kv[kKeys][kPer], vv[kKeys][kPer];
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        const int pg = __shfl_sync(0xffffffffu, page, k0 + j);
        const int64_t ip = __shfl_sync(0xffffffffu, in_page, k0 + j);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = lane + 32 * i;
          const bool real = pg >= 0 && e < p.d;
          kv[j][i] = real ? to_f(kh[(int64_t)pg * p.k_page + ip * p.k_tok + e]) : 0.f;
          vv[j][i] = real ? to_f(vh[(int64_t)pg * p.v_page + ip * p.v_tok + e]) : 0.f;
        }
      }
      // lane 4 h + j ends with the score of head h and key j: 32 sums over the lanes,
      // folded in half at each of five shuffles
      float v[32];
#pragma unroll
      for (int h = 0; h < 8; ++h)
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
          float a = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) a += q[h][i] * kv[j][i];
          v[h * kKeys + j] = a;
        }
#pragma unroll
      for (int bit = 16; bit > 0; bit >>= 1) {
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < bit; ++i) {
          const float keep = upper ? v[i + bit] : v[i], give = upper ? v[i] : v[i + bit];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
        }
      }
      const bool visible = (seen >> (k0 + lane % kKeys)) & 1;
      const float score = visible ? v[0] : -INFINITY;
      float m = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const float now = fmaxf(top[h], __shfl_sync(0xffffffffu, m, h * kKeys));
        const float ref = now == -INFINITY ? 0.f : now;
        const float f = exp2f(top[h] - ref);
        top[h] = now;
        sum[h] *= f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[h][i] *= f;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
          const float e = exp2f(__shfl_sync(0xffffffffu, score, h * kKeys + j) - ref);
          sum[h] += e;
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[h][i] += e * vv[j][i];
        }
      }
    }
    if (cur.tile + 1 == cur.sp.tiles || step + 1 == steps) {
      const int slot =
          first_tile > 0 ? 2 * (int)blockIdx.x : cur.tile + 1 < cur.sp.tiles ? 2 * (int)blockIdx.x + 1 : -1;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        if (lane == 0) {
          part_max[warp][h] = top[h];
          part_sum[warp][h] = sum[h];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) part_o[warp][h][lane + 32 * i] = acc[h][i];
      }
      __syncthreads();
      join_warps<T, D, kHeads>(p, part_max, part_sum, part_o, cur.b, head0, heads, 0, slot);
      __syncthreads();
      fresh = true;
    }
    cur.advance(p, segs, step + 1 < steps);
  }
  write_status(p.status, kDecodeMaxCtas, status);
}

// ----------------------------------------------------------------- join kernel
// Block (c, h): if CTA c's range is the first to begin inside a segment, merge the
// segment's pieces for its head h. The piece that begins the segment is slot
// 2 (c - 1) + 1, the others are slots 2c, 2 (c + 1), ... The four warps take the
// pieces in turn, then their results are merged in warp order.
template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(kThreads) paged_decode_join_kernel(DecodeParams p) {
  __shared__ __align__(16) float part_o[kWarps][D];
  __shared__ float part_max[kWarps], part_sum[kWarps];
  const int64_t total = p.total[0];
  const int32_t ctas = (int32_t)p.total[1];
  const int c = blockIdx.x;
  if (c == 0 || c >= ctas || total == 0) return;
  const DecodeRec rec = p.recs[c];
  if (rec.before == 0) return;
  int head0;
  const int heads = segment_heads<HEADS>(p, rec.seg, head0);
  const int h = blockIdx.y;
  if (h >= heads) return;
  const int64_t begin = cta_start(c, total, ctas) - rec.before, end = begin + rec.tiles;
  if (cta_start(c - 1, total, ctas) > begin) return;  // an earlier block's
  // the CTA that holds the segment's last tile
  const int c_last = (int)((end * ctas - 1) / total);
  const int pieces = c_last - c + 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  constexpr int kPer = D / 32;
  float top = -INFINITY, sum = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int i = warp; i < pieces; i += kWarps) {
    const int slot = i == 0 ? 2 * (c - 1) + 1 : 2 * (c + i - 1);
    const int64_t row = (int64_t)slot * HEADS + h;
    const float lse = p.part_lse[row];
    float o[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = p.part_o[row * D + lane * kPer + k];
    const float now = fmaxf(top, lse), ref = now == -INFINITY ? 0.f : now;
    const float f = exp2f(top - ref), g = exp2f(lse - ref);
    top = now;
    sum = sum * f + g;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = acc[k] * f + g * o[k];
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) part_o[warp][lane * kPer + k] = acc[k];
  if (lane == 0) {
    part_max[warp] = top;
    part_sum[warp] = sum;
  }
  __syncthreads();
  float all = part_max[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) all = fmaxf(all, part_max[w]);
  const bool dead = all == -INFINITY;
  float l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) l += dead ? 0.f : exp2f(part_max[w] - all) * part_sum[w];
  T* dst = static_cast<T*>(p.o) + (int64_t)rec.b * p.o_tok + (int64_t)(head0 + h) * p.o_head;
  for (int e = threadIdx.x; e < p.d; e += kThreads) {
    float o = 0.f;
    if (!dead) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) o += exp2f(part_max[w] - all) * part_o[w][e];
      o /= l;
    }
    dst[e] = from_f<T>(o);
  }
  if (threadIdx.x == 0 && p.stats)
    p.stats[(int64_t)rec.b * p.stats_tok + (int64_t)(head0 + h) * p.stats_head] =
        dead ? -INFINITY : (all + log2f(l)) * kLn2;
}

template <typename T, int D, int NT>
cudaError_t launch_mma(const DecodeParams& p, int ctas, cudaStream_t stream) {
  constexpr int bytes = (int)sizeof(MmaSmem<D>);
  const cudaError_t e = cudaFuncSetAttribute(paged_decode_mma_kernel<T, D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  paged_decode_mma_kernel<T, D, NT><<<ctas, kThreads, bytes, stream>>>(p);
  paged_decode_join_kernel<T, D, 8 * NT><<<dim3(ctas, 8 * NT), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_mma_heads(const DecodeParams& p, int ctas, cudaStream_t stream) {
  switch (decode_seg_heads(p.group, true)) {
    case 8: return launch_mma<T, D, 1>(p, ctas, stream);
    case 16: return launch_mma<T, D, 2>(p, ctas, stream);
    default: return launch_mma<T, D, 4>(p, ctas, stream);
  }
}

template <typename T>
cudaError_t launch_type(const DecodeParams& p, bool mma, int ctas, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (mma) return decode_pad_d(p.d) == 64 ? launch_mma_heads<T, 64>(p, ctas, stream)
                                            : launch_mma_heads<T, 128>(p, ctas, stream);
  }
  if (decode_pad_d(p.d) == 64) {
    paged_decode_simt_kernel<T, 64><<<ctas, kThreads, 0, stream>>>(p);
    paged_decode_join_kernel<T, 64, 8><<<dim3(ctas, 8), kThreads, 0, stream>>>(p);
  } else {
    paged_decode_simt_kernel<T, 128><<<ctas, kThreads, 0, stream>>>(p);
    paged_decode_join_kernel<T, 128, 8><<<dim3(ctas, 8), kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_decode(const DecodeParams& p, thd_dtype_t dtype, bool mma, int num_sms, cudaStream_t stream) {
  const int sms = num_sms < kMaxSmsForSizing ? num_sms : kMaxSmsForSizing;
  const int ctas = sms * kDecodeCtasPerSm;
  switch (dtype) {
    case THD_BF16: return launch_type<__nv_bfloat16>(p, mma, ctas, stream);
    case THD_FP16: return launch_type<__half>(p, mma, ctas, stream);
    default: return launch_type<float>(p, false, ctas, stream);
  }
}

}  // namespace thd
