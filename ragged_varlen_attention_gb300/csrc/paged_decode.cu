// Attention of one new token per request over a paged key-value cache.
//
//   s_j = scale <q, k_j>, O = sum_j softmax(s)_j v_j, LSE = ln sum_j exp s_j
//
// Every visible K and V row is read once and used by the query heads of its group
// only: 2 G operations per byte in 16 bits, far below the tensor cores' rate, so
// memory bounds the kernel. What matters is that every SM streams at its share of
// the bandwidth until the end, whatever the lengths are:
//   - A segment is (request, kv head, up to 8/16/32 query heads of its group). All
//     segments' key chunks (16 or 32 keys) form one line, which the warps share in equal
//     ranges, in order and across segment borders. The border positions follow from the
//     lengths on the device; no setup kernel, no work list.
//   - A warp streams its chunks through its own ring of stages and keeps its own
//     running maximum, sum and output: no warp waits for another one.
//   - A segment that lies inside one warp's range is finished there. One that crosses a
//     border leaves normalised partial outputs in the workspace, and the join kernel
//     merges them in the line's order (no atomics: equal inputs give equal bits).
//
// Measured (both kernels), against a copy at 6.79 TB/s: bf16, 64 requests of 1 to 8192 keys, 32 + 8
// heads of d = 128 (1.07 GB) 169 us (94 %); fp16, 2 x 131072 keys, 64 + 8 heads 168 us (94 %);
// 1024 x 256 keys 187 us (86 %: a segment's beginning and end cost about a chunk's time each);
// d = 64, one query head per kv head, pages of 24, a window of 1023 keys (142 MB) 34 us (61 %);
// 1.07 GB in pages of one row 206 us (77 %: every row's address by shuffles); float32, 32 + 8 heads
// 174 us (91 %), 64 + 8 heads 243 us (65 %: bound by fma and shuffles). One request of 700 keys
// takes 8.2 us: 0.85 for the launch, 1.1 until each warp knows its range, 0.9 until its keys are
// there, 2.3 to compute and write, the rest in the join kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace thd {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLn2 = 0.69314718055994530942f;
// keys of a chunk: half of the rows that a warp's stage holds (K and V) with d = 128, all
// of them with d = 64, so that a stage is 8 KB either way
constexpr int chunk_keys(int pad_d) { return pad_d == 128 ? 16 : 32; }
constexpr int simt_chunk_keys(int pad_d) { return pad_d == 128 ? 8 : 16; }  // 8 KB of float32
static_assert(simt_chunk_keys(128) >= kDecodeMinChunk, "the plan's bound counts these chunks");
static_assert(kWarps * kDecodeMaxCtas == kDecodeMaxWorkers, "the workspace is sized for these workers");

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
// Visible keys [lo, n) of a request; `base` = lo rounded down to a multiple of 16.
struct Span {
  int32_t n, lo, base, chunks;
  bool bad;
};
template <int KC>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  s.n = p.seq_lens[b];
  s.bad = s.n < 0 || (int64_t)s.n > (int64_t)p.max_pages * p.page_size;
  if (s.bad) s.n = 0;
  const int w = p.window ? p.window[b] : -1;
  s.lo = w >= 0 && w < s.n - 1 ? s.n - 1 - w : 0;
  s.base = s.lo & ~15;
  s.chunks = (s.n - s.base + KC - 1) / KC;
  return s;
}

// Position in the line of chunks: request b, segment seg of its `segs`, chunk of the
// segment; sp is the request's span. The warp's lanes hold the same cursor.
template <int KC>
struct Cursor {
  int32_t b, seg, chunk;
  Span sp;
  // the next request with keys (the caller knows that there is one)
  __device__ __forceinline__ void skip_empty(const DecodeParams& p) {
    const int lane = threadIdx.x & 31;
    while (b < p.batch) {
      const int mine = b + lane;
      const bool some = mine < p.batch && span_of<KC>(p, mine).chunks > 0;
      const uint32_t any = __ballot_sync(0xffffffffu, some);
      if (any) {
        b += __ffs(any) - 1;
        sp = span_of<KC>(p, b);
        return;
      }
      b += 32;
    }
  }
  __device__ __forceinline__ void advance(const DecodeParams& p, int segs, bool more) {
    if (++chunk < sp.chunks) return;
    chunk = 0;
    if (++seg < segs) return;
    seg = 0;
    ++b;
    if (more) skip_empty(p);
  }
};

// a / b below 2^31 of non-negative numbers; a 64-bit division, a few hundred cycles, only
// where one is needed
__device__ __forceinline__ int32_t quotient(int64_t a, int32_t b) {
  return (a >> 32) == 0 ? (int32_t)((uint32_t)a / (uint32_t)b) : (int32_t)(a / b);
}

// The line's `total` chunks over the workers (warps): `each` of them, the first `extra`
// workers one more.
struct Line {
  int64_t total;
  int32_t workers, each, extra;
  __device__ __forceinline__ int64_t start(int32_t w) const { return (int64_t)w * each + min(w, extra); }
  // the worker that holds chunk t
  __device__ __forceinline__ int32_t holder(int64_t t) const {
    const int64_t big = (int64_t)extra * (each + 1);
    return t < big ? quotient(t, each + 1) : extra + quotient(t - big, each);
  }
};

__device__ __forceinline__ Line line_of(int64_t total) {
  Line line;
  line.total = total;
  line.workers = (int32_t)min64((int64_t)gridDim.x * kWarps, max64(total, 1));
  line.each = quotient(total, line.workers);  // below 2^31 by the plan's bound
  line.extra = (int32_t)(total - (int64_t)line.each * line.workers);
  return line;
}

__device__ __forceinline__ int32_t inclusive_scan(int32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// The number of chunks in the warp's range, and the cursor at its beginning. All lanes call
// it. Each warp finds its own range, without a barrier: up to 256 requests, 128 at a time in
// flight; lane l keeps the sum of requests 32 l .. 32 l + 31. The chunks of the line fit 31
// bits. (With more requests the block shares them: locate_many.) A quarter of a small call's
// time was here with the block-wide search.
template <int KC>
__device__ __forceinline__ int locate_few(const DecodeParams& p, int segs, Cursor<KC>& cur, Line& line,
                                          uint32_t& status) {
  const int lane = threadIdx.x & 31;
  int32_t tile_sum = 0, total = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 128) {
    int32_t mine[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int b = b0 + 32 * t + lane;
      mine[t] = 0;
      if (b < p.batch) {
        const Span s = span_of<KC>(p, b);
        if (s.bad) status |= THD_DEV_BAD_LENGTH;
        mine[t] = s.chunks;
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int32_t sum = __reduce_add_sync(0xffffffffu, mine[t]);
      if (lane == b0 / 32 + t) tile_sum = sum;
      total += sum;
    }
  }
  line = line_of((int64_t)total * segs);
  const int32_t worker = blockIdx.x * kWarps + threadIdx.x / 32;
  if (worker >= line.workers || total == 0) return 0;
  const int32_t begin = (int32_t)line.start(worker);
  int32_t before = 0, b0 = 0;
  if (p.batch > 32) {
    const int32_t upto = inclusive_scan(tile_sum);
    const int tile = __ffs(__ballot_sync(0xffffffffu, begin < upto * segs)) - 1;
    before = __shfl_sync(0xffffffffu, upto - tile_sum, tile);
    b0 = tile * 32;
  }
  const int32_t mine = b0 + lane < p.batch ? span_of<KC>(p, b0 + lane).chunks : 0;
  const int32_t upto = before + inclusive_scan(mine);
  const int at = __ffs(__ballot_sync(0xffffffffu, begin < upto * segs)) - 1;
  cur.b = b0 + at;
  cur.sp = span_of<KC>(p, cur.b);
  const int32_t rel = begin - __shfl_sync(0xffffffffu, upto - mine, at) * segs;
  cur.seg = (int)((uint32_t)rel / (uint32_t)cur.sp.chunks);
  cur.chunk = rel - cur.seg * cur.sp.chunks;
  return (int)(line.start(worker + 1) - line.start(worker));
}

// The same for any number of requests and chunks: the block's threads share the requests.
template <int KC>
__device__ __forceinline__ int locate_many(const DecodeParams& p, int segs, Cursor<KC>& cur, Line& line,
                                           uint32_t& status) {
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int32_t found_b[kWarps];
  __shared__ int64_t found_before[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int strip = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, (int)threadIdx.x * strip), b1 = min(p.batch, b0 + strip);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Span s = span_of<KC>(p, b);
    if (s.bad) status |= THD_DEV_BAD_LENGTH;
    mine += s.chunks;
  }
  int64_t upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += o;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += warp_sums[w];
    total += warp_sums[w];
  }
  line = line_of(total * segs);
  // the request that each of the block's workers begins in
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t at = line.start(blockIdx.x * kWarps + w);
    int64_t before = (upto - mine) * segs;
    if (before <= at && at < upto * segs) {
      for (int b = b0; b < b1; ++b) {
        const int64_t n = (int64_t)span_of<KC>(p, b).chunks * segs;
        if (at < before + n) {
          found_b[w] = b;
          found_before[w] = before;
          break;
        }
        before += n;
      }
    }
  }
  __syncthreads();
  const int32_t worker = blockIdx.x * kWarps + warp;
  if (worker >= line.workers || line.total == 0) return 0;
  cur.b = found_b[warp];
  cur.sp = span_of<KC>(p, cur.b);
  const int64_t rel = line.start(worker) - found_before[warp];  // below segs x chunks
  cur.seg = quotient(rel, cur.sp.chunks);
  cur.chunk = (int)(rel - (int64_t)cur.seg * cur.sp.chunks);
  return (int)(line.start(worker + 1) - line.start(worker));
}

template <int KC>
__device__ __forceinline__ int locate(const DecodeParams& p, int segs, Cursor<KC>& cur, Line& line, uint32_t& status) {
  return p.few ? locate_few(p, segs, cur, line, status) : locate_many(p, segs, cur, line, status);
}

// The worker's record for the join kernel, from the cursor at the beginning of its range.
template <int KC>
__device__ __forceinline__ void write_record(const DecodeParams& p, const Line& line, const Cursor<KC>& cur, int steps) {
  if ((threadIdx.x & 31) != 0) return;
  const int32_t worker = blockIdx.x * kWarps + threadIdx.x / 32;
  DecodeRec rec = {0, 0, 0, 0};
  if (steps > 0 && cur.chunk > 0) {
    const int64_t begin = line.start(worker) - cur.chunk;
    if (line.start(worker - 1) <= begin)
      rec = {cur.b, cur.seg, line.holder(begin + cur.sp.chunks - 1) - worker + 2, 0};
  }
  p.recs[worker] = rec;
}

// Rows without a visible key: O = 0, LSE = -inf.
template <typename T>
__device__ __forceinline__ void write_empty(const DecodeParams& p) {
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    const Span s = span_of<16>(p, b);
    if (s.bad || s.chunks > 0) continue;
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

// Where a worker leaves its piece of a segment: -1 when it holds the whole segment, 2w when
// the segment began before worker w's range, 2w + 1 when it begins there and goes on.
__device__ __forceinline__ int piece_slot(int worker, int first, int last, int chunks) {
  return first > 0 ? 2 * worker : last + 1 < chunks ? 2 * worker + 1 : -1;
}

// --------------------------------------------------- copies and matrix pieces
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes of zeros when not `real`: src is not read then, and is any valid aligned address
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int bytes = real ? 16 : 0;
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

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// the larger magnitudes of two pairs (a NaN gives the other), and whether one is infinite
template <typename T>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_magnitude<__nv_bfloat16>(uint32_t a, uint32_t b) {
  const __nv_bfloat162 v = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t max_magnitude<__half>(uint32_t a, uint32_t b) {
  const __half2 v = __hmax2(*reinterpret_cast<__half2*>(&a), __habs2(*reinterpret_cast<__half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ bool is_infinite(uint32_t magnitudes);
template <>
__device__ __forceinline__ bool is_infinite<__nv_bfloat16>(uint32_t m) {
  return (m & 0xffffu) == 0x7f80u || (m >> 16) == 0x7f80u;
}
template <>
__device__ __forceinline__ bool is_infinite<__half>(uint32_t m) {
  return (m & 0xffffu) == 0x7c00u || (m >> 16) == 0x7c00u;
}

// ------------------------------------------------- matrix-instruction kernel
// 16 keys are the rows of the instruction and the query heads its 8 columns: S^T = K Q^T,
// then O^T += V^T P^T, so a group of 8 heads fills the tile (the other way round heads
// would be padded to 16). P^T's fragment is S^T's, transposed 8 x 8 by movmatrix. P goes into
// the product as two 16-bit parts, its rounding and what that left over: rounded once, its
// error would be as large as O's own rounding (1.35 to 1.45 times the error in all, measured
// against 64 bits). The second part is left out where a V is infinite, which a negative or
// zero remainder would turn into NaN. Its sum is kept in float32.
//
// A stage is filled by cp.async, 16 bytes a lane, 2 (d = 128) or 4 rows at a time. Where a
// page holds a multiple of 8 rows and the whole chunk is visible, 8 rows are a constant
// stride apart and cost an addition each; otherwise each row's page comes from the lane that
// looked it up. The 16-byte piece c of row r lies at c ^ (r & 7), so that ldmatrix's eight rows
// fall into different banks. (Rows 16 bytes apart from a multiple of 128 do that too, with
// addresses that are constants away from the stage's, but then half of the 32-byte sectors end
// in two lines of shared memory and are requested twice: 38 % hits in L2 where nothing is read
// again. One bulk copy per row, by the lane that knows the page, takes the copy unit 11 to 15
// cycles: 3.4 TB/s at d = 64, 4.95 at d = 128.)
template <int D>
struct MmaSmem {
  static constexpr int kKeys = chunk_keys(D);
  static constexpr int kStages = 3;
  static constexpr int kPitch = 2 * D;
  static constexpr int kStageBytes = 2 * kKeys * kPitch;  // K rows, then V rows
  alignas(256) unsigned char ring[kWarps][kStages][kStageBytes];
  uint32_t seen[kWarps][kStages];  // bit r: key r of the stage is visible
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kDecodeCtasPerSm) paged_decode_mma_kernel(DecodeParams p) {
  using Smem = MmaSmem<D>;
  constexpr int kStages = Smem::kStages;
  constexpr int kKeys = Smem::kKeys;
  constexpr int MT = kKeys / 16;          // 16-key rows of the instruction in a chunk
  constexpr int kHeads = 8 * NT;
  constexpr int kPitch = Smem::kPitch;
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int worker = blockIdx.x * kWarps + warp;
  const int per = (p.group + kHeads - 1) / kHeads;   // segments of a kv head
  const int segs = p.h_kv * per;
  ptx::pdl_wait();
  ptx::pdl_release();
  uint32_t status = 0;
  const uint32_t ring = ptx::smem_u32(sm.ring[warp]);
  if (p.d < D)  // the columns past d, which no copy of a whole chunk fills
    for (int i = lane; i < (int)sizeof(sm.ring[0]) / 16; i += 32)
      reinterpret_cast<uint4*>(sm.ring[warp])[i] = make_uint4(0u, 0u, 0u, 0u);
  Cursor<kKeys> cur;
  Line line;
  const int steps = locate<kKeys>(p, segs, cur, line, status);

  Cursor<kKeys> load = cur;
  int issued = 0;
  uint32_t load_stage = 0;
  // key lane % kKeys of the chunk at `load`: whether it is visible, and where it is, looked
  // up one step before it is used
  bool key_seen = false;
  int64_t key_k = 0, key_v = 0;  // its rows' offsets in the caches
  // the plan gives this kernel strides below 2^31: a product is one 32 x 32 -> 64 instruction
  const int k_page = (int)p.k_page, k_tok = (int)p.k_tok, k_head = (int)p.k_head;
  const int v_page = (int)p.v_page, v_tok = (int)p.v_tok, v_head = (int)p.v_head;
  const bool same = k_page == v_page && k_tok == v_tok;
  auto look_up = [&]() {
    key_seen = false;
    if (issued >= steps) return;
    const int key = load.sp.base + load.chunk * kKeys + (lane & (kKeys - 1));
    if (key >= load.sp.lo && key < load.sp.n) {
      const int column = p.by_page.div(key), row = key - column * p.page_size;
      const int page = p.block_table[(int64_t)load.b * p.table_stride + column];
      key_seen = page >= 0 && page < p.num_pages;
      if (!key_seen) status |= THD_DEV_BAD_PAGE;
      key_k = (int64_t)page * k_page + (int64_t)row * k_tok;
      key_v = same ? key_k : (int64_t)page * v_page + (int64_t)row * v_tok;
    }
  };
  constexpr uint32_t kAll = kKeys == 16 ? 0xffffu : 0xffffffffu;
  constexpr int kVecs = D / 8;             // 16-byte pieces of a row
  constexpr int kRowsAtOnce = 32 / kVecs;  // rows of one warp-wide copy
  const int vec = lane % kVecs, row_in = lane / kVecs;
  const bool vec_real = vec * 8 < p.d;
  const bool whole_pages = (p.page_size & 7) == 0;  // 8 rows from a multiple of 8 are in one page
  const uint32_t piece = (vec ^ row_in) * 16;  // of row row_in (below 8); rows i kRowsAtOnce on: ^ their number
  const T* const k_lane = static_cast<const T*>(p.k) + vec * 8;
  const T* const v_lane = static_cast<const T*>(p.v) + vec * 8;
  const int64_t k_row = (int64_t)row_in * k_tok, v_row = (int64_t)row_in * v_tok;
  const int64_t k_step = (int64_t)kRowsAtOnce * k_tok, v_step = (int64_t)kRowsAtOnce * v_tok;
  auto issue = [&]() {
    if (issued < steps) {
      const uint32_t seen = __ballot_sync(0xffffffffu, key_seen) & kAll;
      if (lane == 0) sm.seen[warp][load_stage] = seen;
      const uint32_t dst = ring + load_stage * Smem::kStageBytes + row_in * kPitch;
      const int g = per == 1 ? load.seg : load.seg / per;
      const T* kh = k_lane + (int64_t)g * k_head;
      const T* vh = v_lane + (int64_t)g * v_head;
      if (whole_pages && seen == kAll) {
#pragma unroll
        for (int r8 = 0; r8 < kKeys; r8 += 8) {
          const int64_t at_k = __shfl_sync(0xffffffffu, key_k, r8);
          const int64_t at_v = same ? at_k : __shfl_sync(0xffffffffu, key_v, r8);
          const T* ks = kh + (at_k + k_row);
          const T* vs = vh + (at_v + v_row);
#pragma unroll
          for (int i = 0; i < 8 / kRowsAtOnce; ++i) {
            const uint32_t at = dst + (r8 + i * kRowsAtOnce) * kPitch + (piece ^ (i * kRowsAtOnce * 16));
            if (vec_real) {
              cp_async16(at, ks);
              cp_async16(at + kKeys * kPitch, vs);
            }
            ks += k_step;
            vs += v_step;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kKeys / kRowsAtOnce; ++i) {
          const int row = i * kRowsAtOnce + row_in;
          const int64_t at_k = __shfl_sync(0xffffffffu, key_k, row);
          const int64_t at_v = same ? at_k : __shfl_sync(0xffffffffu, key_v, row);
          const bool real = ((seen >> row) & 1) && vec_real;
          const uint32_t at = dst + i * kRowsAtOnce * kPitch + (piece ^ ((i * kRowsAtOnce & 7) * 16));
          const void* ks = real ? static_cast<const void*>(kh + at_k) : p.status;
          const void* vs = real ? static_cast<const void*>(vh + at_v) : p.status;
          cp_async16(at, ks, real);
          cp_async16(at + kKeys * kPitch, vs, real);
        }
      }
      ++issued;
      load_stage = load_stage + 1 == kStages ? 0 : load_stage + 1;
      load.advance(p, segs, issued < steps);
      look_up();
    }
    cp_commit();  // an empty group when there is nothing left: the count stays one per step
  };
  __syncwarp();
  look_up();
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t qf[D / 16][NT][2];
  float acc[D / 16][NT][4];
  float top[NT][2], sum[NT][2];
  int head0 = 0, heads = 0, first = 0;
  // the query rows of the segment at `cur`; with 8 heads there are registers to load them
  // ahead of the last segment's end
  constexpr bool kAhead = NT == 1;
  auto load_q = [&]() {
    first = cur.chunk;
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
    }
  };
  auto clear = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt][0] = top[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[dt][nt][j] = 0.f;
    }
  };
  if (steps > 0) load_q();
  clear();
  write_record<kKeys>(p, line, cur, steps);
  write_empty<T>(p);
  uint32_t stage = 0;
  for (int step = 0; step < steps; ++step) {
    cp_wait<kStages - 2>();
    __syncwarp();  // this stage has arrived for every lane, and every lane has read the last one
    issue();       // which is filled again
    const uint32_t seen = sm.seen[warp][stage];
    const uint32_t kbase = ring + stage * Smem::kStageBytes;
    const uint32_t vbase = kbase + kKeys * kPitch;
    if (seen != 0) {
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float odd[NT][4];  // two chains of products, half as long each
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][nt][j] = odd[nt][j] = 0.f;
        // matrices in order: keys 0-7 / d 0-7, keys 8-15 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 8-15
        const uint32_t at = kbase + (mt * 16 + (lane & 15)) * kPitch + (((lane >> 4) ^ (lane & 7)) * 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[4];
          ldsm4(a, at ^ (kk * 32));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<T>(kk & 1 ? odd[nt] : s[mt][nt], a, qf[kk][nt][0], qf[kk][nt][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][nt][j] += odd[nt][j];
      }
      // The reference of the exponentials moves only when a score passes it by 2^8: weights up
      // to 256 cost no precision (P is rounded relative to itself), and most chunks need neither
      // the maximum over the lanes nor the rescaling.
      bool over = false;
      float m[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          m[nt][j] = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float& v = s[mt][nt][j + 2 * half];
              v *= p.scale_log2;
              if (seen != kAll && !((seen >> (mt * 16 + half * 8 + lane / 4)) & 1)) v = -INFINITY;
              m[nt][j] = fmaxf(m[nt][j], v);
            }
          over |= m[nt][j] > top[nt][j] + 8.f;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float now = m[nt][j];
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 4));
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
            now = fmaxf(now, top[nt][j]);
            const float scale = ptx::ex2(top[nt][j] - (now == -INFINITY ? 0.f : now));
            top[nt][j] = now;
            sum[nt][j] *= scale;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
              acc[dt][nt][j] *= scale;
              acc[dt][nt][j + 2] *= scale;
            }
          }
      }
      uint32_t pb[MT][NT][2], rest[MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float ref = top[nt][j] == -INFINITY ? 0.f : top[nt][j];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float& v = s[mt][nt][j + 2 * half];
              v = ptx::ex2(v - ref);
              sum[nt][j] += v;
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float x = s[mt][nt][2 * half], y = s[mt][nt][2 * half + 1];
            const uint32_t rounded = pack2<T>(x, y);
            const float2 back = unpack2<T>(rounded);
            pb[mt][nt][half] = transpose8x8(rounded);
            rest[mt][nt][half] = transpose8x8(pack2<T>(x - back.x, y - back.y));
          }
      }
      // matrices in order: keys 0-7 / d 0-7, keys 0-7 / d 8-15, keys 8-15 / d 0-7, keys 8-15 / d 8-15
      const uint32_t v_at =
          vbase + ((lane & 7) + ((lane >> 4) << 3)) * kPitch + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
      uint32_t largest = 0;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t a[4];
          ldsm4_t(a, (v_at + mt * 16 * kPitch) ^ (dt * 32));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<T>(acc[dt][nt], a, pb[mt][nt][0], pb[mt][nt][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) largest = max_magnitude<T>(largest, a[i]);
        }
      if (!__any_sync(0xffffffffu, is_infinite<T>(largest))) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t a[4];
            ldsm4_t(a, (v_at + mt * 16 * kPitch) ^ (dt * 32));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<T>(acc[dt][nt], a, rest[mt][nt][0], rest[mt][nt][1]);
          }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;

    const bool last = cur.chunk + 1 == cur.sp.chunks || step + 1 == steps;
    const int slot = piece_slot(worker, first, cur.chunk, cur.sp.chunks);
    const int b_done = cur.b, head0_done = head0, heads_done = heads;
    cur.advance(p, segs, step + 1 < steps);
    if (last) {
      if (kAhead && step + 1 < steps) load_q();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= heads_done) break;
        float inv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l = sum[nt][j];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int h = nt * 8 + (lane % 4) * 2 + j;
          const bool dead = top[nt][j] == -INFINITY;
          inv[j] = dead ? 0.f : 1.f / l;
          const float lse2 = dead ? -INFINITY : top[nt][j] + log2f(l);
          if (lane < 4) {
            if (slot >= 0) p.part_lse[(int64_t)slot * kHeads + h] = lse2;
            else if (h < heads_done && p.stats)
              p.stats[(int64_t)b_done * p.stats_tok + (int64_t)(head0_done + h) * p.stats_head] = lse2 * kLn2;
          }
        }
        if (slot >= 0) {
          // 8 lanes write 32 consecutive bytes of a head's row
          float* row = p.part_o + ((int64_t)slot * kHeads + nt * 8 + (lane % 4) * 2) * D + lane / 4;
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j) row[(j & 1) * D + dt * 16 + (j >> 1) * 8] = acc[dt][nt][j] * inv[j & 1];
        } else {
          const int h = nt * 8 + lane / 4;
          T* row = static_cast<T*>(p.o) + (int64_t)b_done * p.o_tok + (int64_t)(head0_done + h) * p.o_head;
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t v = transpose8x8(pack2<T>(acc[dt][nt][2 * half] * inv[0], acc[dt][nt][2 * half + 1] * inv[1]));
              const int e = dt * 16 + half * 8 + (lane % 4) * 2;
              if (h < heads_done && e < p.d) *reinterpret_cast<uint32_t*>(row + e) = v;
            }
        }
      }
      if (!kAhead && step + 1 < steps) load_q();
      clear();
    }
  }
  write_status(p.status, status);
}

// --------------------------------------------------------------- SIMT kernel
// float32 caches, and any d <= 128 and alignment: the same schedule and ring of stages,
// products by packed fma. A lane holds D / 32 consecutive elements of the HB query rows and of
// their outputs. NK = 32 / HB keys at a time: each lane multiplies its elements for all 32
// (head, key) pairs, the 32 sums over the lanes are folded in half at each of five shuffles
// until lane h NK + j has the score of head h and key j, and its weight goes to all lanes
// through shared memory. About 85 instructions a key with 8 heads, 45 with 4, of the 170 that
// an SM issues while its share of the bandwidth brings a key (1 KB at d = 128).
template <typename T, int D>
struct SimtSmem {
  static constexpr int kKeys = simt_chunk_keys(D);
  static constexpr int kStages = 3;
  T ring[kWarps][kStages][2 * kKeys][D];  // K rows, then V rows
  float2 weight[kWarps][32];
  uint32_t seen[kWarps][kStages];
};

template <typename T, int N>
__device__ __forceinline__ void read_row(float (&f)[N], const T* row) {
  if constexpr (sizeof(T) == 4 && N == 4) {
    const float4 v = *reinterpret_cast<const float4*>(row);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else if constexpr (sizeof(T) == 4) {
    const float2 v = *reinterpret_cast<const float2*>(row);
    f[0] = v.x; f[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(row[i]);
  }
}

template <typename T, int D, int HB>
__global__ void __launch_bounds__(kThreads, kDecodeCtasPerSm) paged_decode_simt_kernel(DecodeParams p) {
  using Smem = SimtSmem<T, D>;
  constexpr int kKeys = Smem::kKeys, kStages = Smem::kStages;
  constexpr int kPer = D / 32, kPairs = kPer / 2;
  constexpr int NK = 32 / HB;
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int worker = blockIdx.x * kWarps + warp;
  const int per = (p.group + HB - 1) / HB;
  const int segs = p.h_kv * per;
  ptx::pdl_wait();
  ptx::pdl_release();
  uint32_t status = 0;
  Cursor<kKeys> cur;
  Line line;
  const int steps = locate<kKeys>(p, segs, cur, line, status);

  Cursor<kKeys> load = cur;
  int issued = 0, load_stage = 0;
  bool key_seen = false;
  int64_t key_k = 0, key_v = 0;
  auto look_up = [&]() {  // as in the matrix kernel
    key_seen = false;
    if (issued >= steps) return;
    const int key = load.sp.base + load.chunk * kKeys + (lane & (kKeys - 1));
    if (key >= load.sp.lo && key < load.sp.n) {
      const int column = p.by_page.div(key), row = key - column * p.page_size;
      const int page = p.block_table[(int64_t)load.b * p.table_stride + column];
      key_seen = page >= 0 && page < p.num_pages;
      if (!key_seen) status |= THD_DEV_BAD_PAGE;
      key_k = page * p.k_page + row * p.k_tok;
      key_v = page * p.v_page + row * p.v_tok;
    }
  };
  constexpr int kVecs = D * (int)sizeof(T) / 16, kRowsAtOnce = kVecs >= 32 ? 1 : 32 / kVecs;
  auto issue = [&]() {
    if (issued < steps) {
      const uint32_t seen = __ballot_sync(0xffffffffu, key_seen) & ((1u << kKeys) - 1);
      if (lane == 0) sm.seen[warp][load_stage] = seen;
      const int g = load.seg / per;
      const T* kh = static_cast<const T*>(p.k) + (int64_t)g * p.k_head;
      const T* vh = static_cast<const T*>(p.v) + (int64_t)g * p.v_head;
      T(*rows)[D] = sm.ring[warp][load_stage];
      if (p.aligned) {
        const int vec = lane % kVecs * (16 / (int)sizeof(T)), row_in = lane / kVecs;
#pragma unroll
        for (int i = 0; i < kKeys / kRowsAtOnce; ++i) {
          const int row = i * kRowsAtOnce + row_in;
          const int64_t at_k = __shfl_sync(0xffffffffu, key_k, row), at_v = __shfl_sync(0xffffffffu, key_v, row);
          const bool real = ((seen >> row) & 1) && vec < p.d;
          cp_async16(ptx::smem_u32(&rows[row][vec]), real ? static_cast<const void*>(kh + at_k + vec) : p.status, real);
          cp_async16(ptx::smem_u32(&rows[kKeys + row][vec]), real ? static_cast<const void*>(vh + at_v + vec) : p.status, real);
        }
      } else {
        for (int row = 0; row < kKeys; ++row) {
          const int64_t at_k = __shfl_sync(0xffffffffu, key_k, row), at_v = __shfl_sync(0xffffffffu, key_v, row);
#pragma unroll
          for (int e = lane; e < D; e += 32) {
            const bool real = ((seen >> row) & 1) && e < p.d;
            rows[row][e] = real ? kh[at_k + e] : from_f<T>(0.f);
            rows[kKeys + row][e] = real ? vh[at_v + e] : from_f<T>(0.f);
          }
        }
      }
      ++issued;
      load_stage = load_stage + 1 == kStages ? 0 : load_stage + 1;
      load.advance(p, segs, issued < steps);
      look_up();
    }
    cp_commit();
  };
  look_up();
  for (int i = 0; i < kStages - 1; ++i) issue();
  write_record<kKeys>(p, line, cur, steps);
  write_empty<T>(p);

  uint64_t q[HB][kPairs], acc[HB][kPairs];
  float top = 0.f, sum = 0.f;  // of head lane / NK (the sum: of this lane's keys)
  int head0 = 0, heads = 0, first = 0, stage = 0;
  bool fresh = true;
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      first = cur.chunk;
      heads = segment_heads<HB>(p, cur.seg, head0);
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const T* row = static_cast<const T*>(p.q) + (int64_t)cur.b * p.q_tok + (int64_t)(head0 + h) * p.q_head;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float v[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int e = lane * kPer + 2 * i + j;
            v[j] = h < heads && e < p.d ? to_f(row[e]) * p.scale_log2 : 0.f;
          }
          q[h][i] = ptx::f2_pack(v[0], v[1]);
          acc[h][i] = 0;
        }
      }
      top = -INFINITY;
      sum = 0.f;
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    issue();
    const uint32_t seen = sm.seen[warp][stage];
    const T(*rows)[D] = sm.ring[warp][stage];
#pragma unroll
    for (int k0 = 0; k0 < kKeys; k0 += NK) {
      if (((seen >> k0) & ((1u << NK) - 1)) == 0) continue;
      float v[32];
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        float f[kPer];
        read_row(f, &rows[k0 + j][lane * kPer]);
        uint64_t kk[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) kk[i] = ptx::f2_pack(f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          uint64_t a = ptx::f2_mul(q[h][0], kk[0]);
          if (kPairs == 2) a = ptx::f2_fma(q[h][kPairs - 1], kk[kPairs - 1], a);
          float lo, hi;
          ptx::f2_unpack(a, lo, hi);
          v[h * NK + j] = lo + hi;
        }
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
      const float score = (seen >> (k0 + lane % NK)) & 1 ? v[0] : -INFINITY;
      float m = score;
#pragma unroll
      for (int bit = 1; bit < NK; bit <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, bit));
      m = fmaxf(m, top);
      const float ref = m == -INFINITY ? 0.f : m;
      const float scale = ptx::ex2(top - ref);
      if (__any_sync(0xffffffffu, m != top)) {
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          const float f = __shfl_sync(0xffffffffu, scale, h * NK);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) acc[h][i] = ptx::f2_mul(acc[h][i], ptx::f2_pack(f, f));
        }
      }
      top = m;
      const float weight = ptx::ex2(score - ref);
      sum = sum * scale + weight;
      __syncwarp();
      sm.weight[warp][lane] = make_float2(weight, weight);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        float f[kPer];
        read_row(f, &rows[kKeys + k0 + j][lane * kPer]);
        uint64_t vv[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) vv[i] = ptx::f2_pack(f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          const uint64_t w = *reinterpret_cast<const uint64_t*>(&sm.weight[warp][h * NK + j]);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) acc[h][i] = ptx::f2_fma(w, vv[i], acc[h][i]);
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;

    if (cur.chunk + 1 == cur.sp.chunks || step + 1 == steps) {
      const int slot = piece_slot(worker, first, cur.chunk, cur.sp.chunks);
      float all = sum;
#pragma unroll
      for (int bit = 1; bit < NK; bit <<= 1) all += __shfl_xor_sync(0xffffffffu, all, bit);
      const bool dead = top == -INFINITY;
      const float inv_mine = dead ? 0.f : 1.f / all;
      const float lse2 = dead ? -INFINITY : top + log2f(all);
      const int mine = lane / NK;
      if (lane % NK == 0 && mine < heads) {
        if (slot >= 0) p.part_lse[(int64_t)slot * HB + mine] = lse2;
        else if (p.stats) p.stats[(int64_t)cur.b * p.stats_tok + (int64_t)(head0 + mine) * p.stats_head] = lse2 * kLn2;
      }
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const float inv = __shfl_sync(0xffffffffu, inv_mine, h * NK);
        if (h >= heads) break;
        T* row = static_cast<T*>(p.o) + (int64_t)cur.b * p.o_tok + (int64_t)(head0 + h) * p.o_head;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float v[2];
          ptx::f2_unpack(acc[h][i], v[0], v[1]);
          const int e = lane * kPer + 2 * i;
          if (slot >= 0) {
            *reinterpret_cast<float2*>(p.part_o + ((int64_t)slot * HB + h) * D + e) = make_float2(v[0] * inv, v[1] * inv);
          } else {
            if (e < p.d) row[e] = from_f<T>(v[0] * inv);
            if (e + 1 < p.d) row[e + 1] = from_f<T>(v[1] * inv);
          }
        }
      }
      fresh = true;
    }
    cur.advance(p, segs, step + 1 < steps);
  }
  cp_wait<0>();
  write_status(p.status, status);
}

// ----------------------------------------------------------------- join kernel
// Block (x, h) looks at the records of 16 workers and merges the pieces of the segments that
// they own for one head. The piece that begins the segment is slot 2 (w - 1) + 1, the others
// are slots 2w, 2 (w + 1), ... Up to 8 pieces are one warp's work, more are shared by the
// block's warps (every eighth piece) and merged in warp order: a long request alone leaves
// hundreds, and a warp would read them one latency after another. Every warp reads the 16
// records and knows its share, so that only shared segments meet a barrier.
constexpr int kJoinWorkers = 16;
constexpr int kJoinWarps = 8;

// The running result of a warp: base-2 maximum and sum, and the lane's elements.
template <int D>
struct Merged {
  static constexpr int kPer = D / 32;
  float top, sum, o[kPer];
  __device__ __forceinline__ void clear() {
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = 0.f;
  }
  __device__ __forceinline__ void add(float lse, float weight, const float (&x)[kPer]) {
    const float now = fmaxf(top, lse), ref = now == -INFINITY ? 0.f : now;
    const float f = ptx::ex2(top - ref), g = ptx::ex2(lse - ref);
    top = now;
    sum = sum * f + g * weight;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = o[k] * f + g * x[k];
  }
  // pieces first, first + step, ... of worker w's segment, N at a time in flight
  template <int HEADS, int N>
  __device__ __forceinline__ void read(const DecodeParams& p, int w, int h, int pieces, int first, int step) {
    for (int i0 = first; i0 < pieces; i0 += N * step) {
      float lse[N], x[N][kPer];
#pragma unroll
      for (int a = 0; a < N; ++a) {
        const int i = i0 + a * step;
        lse[a] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[a][k] = 0.f;
        if (i < pieces) {
          const int row = (i == 0 ? 2 * w - 1 : 2 * (w + i - 1)) * HEADS + h;
          lse[a] = p.part_lse[row];
          const float* src = p.part_o + (int64_t)row * D + (threadIdx.x & 31) * kPer;
          if constexpr (kPer == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[a][0] = v.x; x[a][1] = v.y; x[a][2] = v.z; x[a][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[a][0] = v.x; x[a][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int a = 0; a < N; ++a) add(lse[a], 1.f, x[a]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void write(const DecodeParams& p, int b, int head) {
    const bool dead = top == -INFINITY;
    const float inv = dead ? 0.f : 1.f / sum;
    const int lane = threadIdx.x & 31;
    T* dst = static_cast<T*>(p.o) + (int64_t)b * p.o_tok + (int64_t)head * p.o_head;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (lane * kPer + k < p.d) dst[lane * kPer + k] = from_f<T>(o[k] * inv);
    if (lane == 0 && p.stats)
      p.stats[(int64_t)b * p.stats_tok + (int64_t)head * p.stats_head] = dead ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
};

template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(32 * kJoinWarps, 4) paged_decode_join_kernel(DecodeParams p) {
  __shared__ float part_o[kJoinWarps][D];
  __shared__ float part_max[kJoinWarps], part_sum[kJoinWarps];
  ptx::pdl_wait();
  ptx::pdl_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, h = blockIdx.y;
  const int w0 = blockIdx.x * kJoinWorkers;
  // lane i: the record of worker w0 + i, if it owns a segment that has this head
  DecodeRec rec = {0, 0, 0, 0};
  if (lane < kJoinWorkers && w0 + lane < p.workers) rec = p.recs[w0 + lane];
  int head0 = 0;
  if (rec.pieces > 0 && h >= segment_heads<HEADS>(p, rec.seg, head0)) rec.pieces = 0;
  const uint32_t few = __ballot_sync(0xffffffffu, rec.pieces > 0 && rec.pieces <= kJoinWarps);
  const uint32_t many = __ballot_sync(0xffffffffu, rec.pieces > kJoinWarps);
  Merged<D> m;
  int turn = 0;
  for (uint32_t todo = few; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    if (turn++ % kJoinWarps != warp) continue;
    m.clear();
    m.template read<HEADS, 4>(p, w0 + i, h, __shfl_sync(0xffffffffu, rec.pieces, i), 0, 1);
    m.template write<T>(p, __shfl_sync(0xffffffffu, rec.b, i), __shfl_sync(0xffffffffu, head0, i) + h);
  }
  for (uint32_t todo = many; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    m.clear();
    m.template read<HEADS, 8>(p, w0 + i, h, __shfl_sync(0xffffffffu, rec.pieces, i), warp, kJoinWarps);
    __syncthreads();  // the last segment's results have been read
#pragma unroll
    for (int k = 0; k < m.kPer; ++k) part_o[warp][lane * m.kPer + k] = m.o[k];
    if (lane == 0) {
      part_max[warp] = m.top;
      part_sum[warp] = m.sum;
    }
    __syncthreads();
    if (warp != 0) continue;
    m.clear();
#pragma unroll
    for (int o = 0; o < kJoinWarps; ++o) {
      float x[m.kPer];
#pragma unroll
      for (int k = 0; k < m.kPer; ++k) x[k] = part_o[o][lane * m.kPer + k];
      m.add(part_max[o], part_sum[o], x);
    }
    m.template write<T>(p, __shfl_sync(0xffffffffu, rec.b, i), __shfl_sync(0xffffffffu, head0, i) + h);
  }
}

template <typename T, int D, int NT>
cudaError_t launch_mma(const DecodeParams& p, int ctas, cudaStream_t stream) {
  constexpr int bytes = (int)sizeof(MmaSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(paged_decode_mma_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       bytes);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(paged_decode_mma_kernel<T, D, NT>, ctas, kThreads, bytes, stream, p);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_decode_join_kernel<T, D, 8 * NT>, dim3((p.workers + kJoinWorkers - 1) / kJoinWorkers, 8 * NT),
                           32 * kJoinWarps, 0, stream, p);
}

template <typename T, int D, int HB>
cudaError_t launch_simt(const DecodeParams& p, int ctas, cudaStream_t stream) {
  constexpr int bytes = (int)sizeof(SimtSmem<T, D>);
  cudaError_t e = cudaFuncSetAttribute(paged_decode_simt_kernel<T, D, HB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       bytes);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(paged_decode_simt_kernel<T, D, HB>, ctas, kThreads, bytes, stream, p);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_decode_join_kernel<T, D, HB>, dim3((p.workers + kJoinWorkers - 1) / kJoinWorkers, HB), 32 * kJoinWarps, 0,
                           stream, p);
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
  if (decode_pad_d(p.d) == 64)
    return p.group <= 4 ? launch_simt<T, 64, 4>(p, ctas, stream) : launch_simt<T, 64, 8>(p, ctas, stream);
  return p.group <= 4 ? launch_simt<T, 128, 4>(p, ctas, stream) : launch_simt<T, 128, 8>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_paged_decode(DecodeParams p, thd_dtype_t dtype, bool mma, int num_sms, cudaStream_t stream) {
  const int sms = num_sms < kMaxSmsForSizing ? num_sms : kMaxSmsForSizing;
  const int ctas = sms * kDecodeCtasPerSm;
  p.workers = ctas * kWarps;
  switch (dtype) {
    case THD_BF16: return launch_type<__nv_bfloat16>(p, mma, ctas, stream);
    case THD_FP16: return launch_type<__half>(p, mma, ctas, stream);
    default: return launch_type<float>(p, false, ctas, stream);
  }
}

}  // namespace thd
