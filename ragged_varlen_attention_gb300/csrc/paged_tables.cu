// Page tables of one step: pages for the new tokens from the free list, each new
// token's slot and position, the lengths after the step.
//
//   old_b = ceil(len_b / P), need_b = ceil((len_b + n_b) / P) - old_b
//   page i < need_b of request b is free[begin + sum_{a<b} need_a + i]
//
// A few integers per token: the launch and three memory latencies in a row (lengths, page
// number, slot) bound it, 3.9 us for 24 requests and 5.4 us for 512 requests with 65536 new
// tokens, so it is one launch with no step that waits for another block. Every block scans the need of all requests for
// itself (batch x 8 bytes from L2), and a token finds its page without the table being
// written first: an old page from the table, a new one from the free list. The token
// at the start of a new page writes the page's table entry, so nothing else has to.
#include "internal.h"
#include "ptx.cuh"

namespace thd {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = kPagedTablesRowsPerBlock / kThreads;

// Inclusive scan over the block's threads of a non-negative value.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, s);
    if (lane >= s) v += o;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  return v + before;
}

// pages that n >= 0 tokens take
__device__ __forceinline__ int32_t pages_of(const PagedTablesParams& p, int32_t n) {
  return n > 0 ? p.by_page.div(n - 1) + 1 : 0;
}

struct Request {
  int32_t len, need;
  bool bad, bad_cu;  // takes no part; its offsets are outside the rows or decrease
};
__device__ __forceinline__ Request request_of(const PagedTablesParams& p, int b) {
  Request r;
  const int lo = p.cu_new[b], hi = p.cu_new[b + 1];
  r.len = p.seq_lens[b];
  r.bad_cu = lo < 0 || hi < lo || hi > p.cap_rows;
  const int64_t after = (int64_t)r.len + (r.bad_cu ? 0 : hi - lo);
  r.bad = r.bad_cu || r.len < 0 || after > (int64_t)p.max_pages * p.page_size;
  r.need = r.bad ? 0 : pages_of(p, (int32_t)after) - pages_of(p, r.len);
  return r;
}

__global__ void __launch_bounds__(kThreads) paged_tables_kernel(PagedTablesParams p) {
  // first free page of each request, counted from `begin` and capped at what there is;
  // -1 for a request that takes no part
  __shared__ int32_t start[kPagedMaxBatch];
  __shared__ int64_t warp_sums[kThreads / 32];
  ptx::pdl_wait();
  ptx::pdl_release();
  uint32_t status = 0;
  const int strip = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, (int)threadIdx.x * strip), b1 = min(p.batch, b0 + strip);

  // the lengths, the offsets and the free list's span in one round of loads
  int64_t begin = p.free_span[0], end = p.free_span[1];
  int bad_cu = 0;
  int64_t need = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    bad_cu |= r.bad_cu;
    need += r.need;
  }
  bad_cu = __syncthreads_or(bad_cu);
  if (begin < 0 || end < begin || end > p.cap_free) {
    status |= THD_DEV_BAD_OFFSET;
    end = begin;
  }
  const int64_t avail = end - begin;
  if (bad_cu) {
    status |= THD_DEV_BAD_LENGTH;
    need = 0;
  }
  const int64_t upto = block_scan(need, warp_sums);
  int64_t at = upto - need;
  for (int b = b0; b < b1; ++b) {
    int32_t n = 0;
    bool bad = true;
    int64_t len = 0;
    if (!bad_cu) {
      const Request r = request_of(p, b);
      n = r.need;
      bad = r.bad;
      len = r.len;
      if (bad) status |= THD_DEV_BAD_LENGTH;
    }
    const int64_t first = min64(at, avail), got = min64(at + n, avail) - first;
    start[b] = bad ? -1 : (int32_t)first;
    if (got < n) status |= THD_DEV_OUT_OF_PAGES;
    if (blockIdx.x == 0) {
      if (bad) {
        p.seq_lens_out[b] = p.seq_lens[b];
      } else {
        const int64_t old = pages_of(p, (int32_t)len);
        const int64_t after = len + (p.cu_new[b + 1] - p.cu_new[b]);
        p.seq_lens_out[b] = (int32_t)min64(after, (old + got) * p.page_size);
      }
    }
    at += n;
  }
  // the last thread's sum is the sum over all requests
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) *p.free_begin_out = (int32_t)(begin + min64(upto, avail));
  __syncthreads();

  const int row0 = (blockIdx.x * kThreads + threadIdx.x) * kPerThread;
  if (row0 < p.cap_rows) {
    const bool owned = !bad_cu && p.batch > 0;
    const int cu_first = owned ? p.cu_new[0] : 0, cu_last = owned ? p.cu_new[p.batch] : 0;
    int b = 0;
    int slot[kPerThread], position[kPerThread];
    bool found = false;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int row = row0 + i;
      slot[i] = position[i] = -1;
      if (row >= cu_last || row < cu_first) continue;
      if (!found) {  // the last request that begins at or before the row
        int lo = 0, hi = p.batch - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (p.cu_new[mid] <= row) lo = mid;
          else hi = mid - 1;
        }
        b = lo;
        found = true;
      }
      while (p.cu_new[b + 1] <= row) ++b;
      const int first = start[b];
      if (first < 0) continue;
      const int len = p.seq_lens[b];
      const int pos = len + (row - p.cu_new[b]);
      const int column = p.by_page.div(pos), in_page = pos - column * p.page_size;
      const int old = pages_of(p, len);
      position[i] = pos;
      int page;
      if (column < old) {
        page = p.block_table[(int64_t)b * p.table_stride + column];
        if (page < 0 || page >= p.num_pages) {
          status |= THD_DEV_BAD_PAGE;
          page = -1;
        }
      } else {
        const int64_t entry = (int64_t)first + (column - old);
        page = -1;
        if (entry < avail) {
          page = p.free_pages[begin + entry];
          if (page < 0 || page >= p.num_pages) {
            status |= THD_DEV_BAD_PAGE;
            page = -1;
          }
        }
        if (in_page == 0) p.block_table[(int64_t)b * p.table_stride + column] = page;
      }
      if (page >= 0) slot[i] = page * p.page_size + in_page;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (row0 + i < p.cap_rows) {
        p.slot_map[row0 + i] = slot[i];
        p.positions[row0 + i] = position[i];
      }
  }
  write_status(p.status, status);
}

}  // namespace

cudaError_t launch_paged_tables(const PagedTablesParams& p, cudaStream_t stream) {
  const int blocks = p.cap_rows > 0 ? (p.cap_rows + kPagedTablesRowsPerBlock - 1) / kPagedTablesRowsPerBlock : 1;
  return launch_overlapped(paged_tables_kernel, blocks, kThreads, 0, stream, p);
}

}  // namespace thd
