// Host side of the operators beside attention (declared in include/thd_attn.h): the
// per-head norm with the position rotation, the page tables, and one-token attention
// over pages. Descriptors are validated once, at plan time; a call checks its pointers
// and enqueues. Every check that can fail comes before the first launch.
#include <cmath>
#include <cstring>
#include <new>

#include "internal.h"

namespace {

constexpr int64_t kAlign = 256;
constexpr int64_t kInt32End = int64_t(1) << 31;

int64_t align_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
int elem_bytes(thd_dtype_t t) { return t == THD_FP32 ? 4 : 2; }
bool known_dtype(thd_dtype_t t) { return t == THD_BF16 || t == THD_FP16 || t == THD_FP32; }
bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

thd_attn_plan_s* new_plan(int kind, int status_blocks) {
  auto* p = new (std::nothrow) thd_attn_plan_s;
  if (!p) return nullptr;
  std::memset(p, 0, sizeof(*p));
  p->kind = kind;
  p->kernel = THD_KERNEL_SIMT;
  p->status_blocks = status_blocks;
  return p;
}

bool bad_workspace(const void* ws) { return !ws || !aligned(ws, kAlign); }

// span in bytes of a paged view [pages, page_size, heads, d]
int64_t cache_span(int64_t pages, int64_t page_size, int64_t heads, int64_t d, int64_t sp, int64_t st, int64_t sh,
                   int64_t eb) {
  if (pages <= 0) return 0;
  return ((pages - 1) * sp + (page_size - 1) * st + (heads - 1) * sh + d) * eb;
}

}  // namespace

extern "C" {

// ------------------------------------------------------ per-head norm and rotation

thd_status_t thd_qk_norm_rope_plan(thd_attn_plan_t* out, const thd_norm_rope_desc_t* desc, size_t* ws_bytes) {
  if (!out || !desc || !ws_bytes) return THD_ERR_INVALID_ARG;
  *out = nullptr;
  const thd_norm_rope_desc_t& d = *desc;
  if (!known_dtype(d.dtype)) return THD_ERR_INVALID_ARG;
  if (d.form != THD_NORM_ROPE_FWD && d.form != THD_NORM_ROPE_BWD && d.form != THD_NORM_ROPE_PAGED)
    return THD_ERR_INVALID_ARG;
  if (d.rows < 0 || d.h_q < 1 || d.h_kv < 1 || d.d < 1) return THD_ERR_INVALID_ARG;
  if (d.rot < 0 || d.rot % 2 != 0 || d.rot > d.d || d.max_pos < 0) return THD_ERR_INVALID_ARG;
  if (!(d.eps >= 0.f) || !std::isfinite(d.eps)) return THD_ERR_INVALID_ARG;
  if (d.flags & ~(uint32_t)THD_FLAG_ZERO_SKIPPED) return THD_ERR_INVALID_ARG;
  if (d.d > 256) return THD_ERR_UNSUPPORTED;
  if (d.h_q > 65536 || d.h_kv > 65536) return THD_ERR_UNSUPPORTED;
  const bool paged = d.form == THD_NORM_ROPE_PAGED;
  if (paged) {
    if (d.page_size < 1 || d.num_pages < 0) return THD_ERR_INVALID_ARG;
    if ((int64_t)d.page_size * d.num_pages >= kInt32End) return THD_ERR_UNSUPPORTED;
  }
  const int eb = elem_bytes(d.dtype);
  const bool used[6] = {true, true, d.form != THD_NORM_ROPE_FWD, true, true, d.form != THD_NORM_ROPE_FWD};
  const bool q_heads[6] = {true, false, d.form == THD_NORM_ROPE_BWD, d.form != THD_NORM_ROPE_BWD,
                           d.form == THD_NORM_ROPE_BWD, false};
  for (int i = 0; i < 6; ++i) {
    if (!used[i]) continue;
    const bool cache = paged && i >= 4;
    if (d.stride_tok[i] < 0 || d.stride_head[i] < 0 || d.bytes[i] < 0) return THD_ERR_INVALID_ARG;
    if (cache && d.stride_page[i] < 0) return THD_ERR_INVALID_ARG;
    if (d.bytes[i] == 0) continue;
    const int64_t heads = q_heads[i] ? d.h_q : d.h_kv;
    const int64_t span = cache ? cache_span(d.num_pages, d.page_size, heads, d.d, d.stride_page[i], d.stride_tok[i],
                                            d.stride_head[i], eb)
                               : thd_attn_view_span_bytes(d.rows, heads, d.d, d.stride_tok[i], d.stride_head[i], eb);
    if (span > d.bytes[i]) return THD_ERR_CAPACITY;
  }
  auto* p = new_plan(kPlanNormRope, thd::kNormRopeMaxBlocks);
  if (!p) return THD_ERR_INVALID_ARG;
  p->ndesc = d;
  p->elem_bytes = eb;
  int64_t off = align_up(4 * (1 + thd::kNormRopeMaxBlocks));
  p->ws_off[1] = off;
  if (d.form == THD_NORM_ROPE_BWD) off = align_up(off + (int64_t)thd::kNormRopeMaxBlocks * 2 * d.d * 4);
  p->ws_bytes = (size_t)off;
  *ws_bytes = p->ws_bytes;
  *out = p;
  return THD_OK;
}

namespace {

// Fills what the three forms share and launches. `views` in the descriptor's order.
thd_status_t run_norm_rope(thd_attn_plan_t plan, const void* const (&views)[6], const void* w_q, const void* w_k,
                           const float* cos_sin, const int32_t* positions, const int32_t* slot_map, float* dw_q,
                           float* dw_k, void* workspace, void* stream_ptr) {
  const thd_norm_rope_desc_t& d = plan->ndesc;
  const bool paged = d.form == THD_NORM_ROPE_PAGED, back = d.form == THD_NORM_ROPE_BWD;
  if (bad_workspace(workspace)) return THD_ERR_WORKSPACE;
  if (d.rows > 0) {
    if (!positions || (paged && !slot_map)) return THD_ERR_INVALID_ARG;
    if (!cos_sin && d.rot > 0 && d.max_pos > 0) return THD_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i) {
      if ((i == 2 || i == 5) && d.form == THD_NORM_ROPE_FWD) continue;
      if (!views[i] && !(paged && i >= 4 && d.num_pages == 0)) return THD_ERR_INVALID_ARG;
    }
  }
  thd::NormRopeParams np;
  std::memset(&np, 0, sizeof(np));
  // inputs: Q, K, then V (paged) or dQ out, dK out (backward); outputs of Q, K, V
  const int in_view[4] = {0, 1, 2, 3};
  const int out_view[3] = {back ? 4 : 3, back ? 5 : 4, 5};
  const int inputs = back ? 4 : paged ? 3 : 2, outputs = paged ? 3 : 2;
  const int64_t vec_bytes = 4 * plan->elem_bytes;
  const int64_t most_heads = d.h_q > d.h_kv ? d.h_q : d.h_kv;
  // 64 spare: the last unit's rows are numbered past the tensor's end
  bool vec = d.d % 8 == 0 && d.rot % 8 == 0 && d.rows * most_heads < kInt32End - 64 && aligned(cos_sin, 16) && aligned(w_q, vec_bytes) &&
             aligned(w_k, vec_bytes);
  for (int i = 0; i < inputs; ++i) {
    const int v = in_view[i];
    np.in[i] = views[v];
    np.in_tok[i] = d.stride_tok[v];
    np.in_head[i] = d.stride_head[v];
    vec = vec && aligned(views[v], vec_bytes) && d.stride_tok[v] % 4 == 0 && d.stride_head[v] % 4 == 0;
  }
  for (int i = 0; i < outputs; ++i) {
    const int v = out_view[i];
    np.out[i] = const_cast<void*>(views[v]);
    np.out_page[i] = d.stride_page[v];
    np.out_tok[i] = d.stride_tok[v];
    np.out_head[i] = d.stride_head[v];
    vec = vec && aligned(views[v], vec_bytes) && d.stride_tok[v] % 4 == 0 && d.stride_head[v] % 4 == 0 &&
          (!paged || i == 0 || d.stride_page[v] % 4 == 0);
  }
  np.w[0] = w_q; np.w[1] = w_k;
  np.cos_sin = cos_sin; np.positions = positions; np.slot_map = slot_map;
  char* ws = static_cast<char*>(workspace);
  np.status = reinterpret_cast<uint32_t*>(ws);
  np.part_dw = reinterpret_cast<float*>(ws + plan->ws_off[1]);
  np.dw[0] = dw_q; np.dw[1] = dw_k;
  np.rows = d.rows; np.h_q = d.h_q; np.h_kv = d.h_kv; np.d = d.d; np.rot = d.rot;
  np.by_heads[0] = thd::FastDiv(d.h_q);
  np.by_heads[1] = thd::FastDiv(d.h_kv);
  np.interleaved = d.interleaved ? 1 : 0;
  np.max_pos = d.max_pos;
  np.page_size = d.page_size;
  np.num_slots = (int64_t)d.page_size * d.num_pages;
  np.eps = d.eps;
  np.zero_skipped = (d.flags & THD_FLAG_ZERO_SKIPPED) ? 1 : 0;
  const int sms = thd::current_device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  const auto launch = d.dtype == THD_BF16   ? thd::launch_norm_rope_bf16
                      : d.dtype == THD_FP16 ? thd::launch_norm_rope_fp16
                                            : thd::launch_norm_rope_fp32;
  return launch(np, d.form, vec, sms, static_cast<cudaStream_t>(stream_ptr)) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

bool is_form(thd_attn_plan_t plan, thd_norm_rope_form_t form) {
  return plan && plan->kind == kPlanNormRope && plan->ndesc.form == form;
}

}  // namespace

thd_status_t thd_qk_norm_rope_fwd(thd_attn_plan_t plan, const void* q, const void* k, const void* w_q,
                                  const void* w_k, const float* cos_sin, const int32_t* positions, void* q_out,
                                  void* k_out, void* workspace, void* stream) {
  if (!is_form(plan, THD_NORM_ROPE_FWD)) return THD_ERR_INVALID_ARG;
  const void* views[6] = {q, k, nullptr, q_out, k_out, nullptr};
  return run_norm_rope(plan, views, w_q, w_k, cos_sin, positions, nullptr, nullptr, nullptr, workspace, stream);
}

thd_status_t thd_qk_norm_rope_bwd(thd_attn_plan_t plan, const void* q, const void* k, const void* dq_out,
                                  const void* dk_out, const void* w_q, const void* w_k, const float* cos_sin,
                                  const int32_t* positions, void* dq, void* dk, float* dw_q, float* dw_k,
                                  void* workspace, void* stream) {
  if (!is_form(plan, THD_NORM_ROPE_BWD)) return THD_ERR_INVALID_ARG;
  const void* views[6] = {q, k, dq_out, dk_out, dq, dk};
  return run_norm_rope(plan, views, w_q, w_k, cos_sin, positions, nullptr, dw_q, dw_k, workspace, stream);
}

thd_status_t thd_qk_norm_rope_paged(thd_attn_plan_t plan, const void* q, const void* k, const void* v,
                                    const void* w_q, const void* w_k, const float* cos_sin,
                                    const int32_t* positions, const int32_t* slot_map, void* q_out, void* k_cache,
                                    void* v_cache, void* workspace, void* stream) {
  if (!is_form(plan, THD_NORM_ROPE_PAGED)) return THD_ERR_INVALID_ARG;
  const void* views[6] = {q, k, v, q_out, k_cache, v_cache};
  return run_norm_rope(plan, views, w_q, w_k, cos_sin, positions, slot_map, nullptr, nullptr, workspace, stream);
}

// --------------------------------------------------------------------- page tables

thd_status_t thd_paged_tables_plan(thd_attn_plan_t* out, const thd_paged_tables_desc_t* desc, size_t* ws_bytes) {
  if (!out || !desc || !ws_bytes) return THD_ERR_INVALID_ARG;
  *out = nullptr;
  const thd_paged_tables_desc_t& d = *desc;
  if (d.batch < 0 || d.page_size < 1 || d.num_pages < 0 || d.max_pages < 0 || d.cap_rows < 0 || d.cap_free < 0)
    return THD_ERR_INVALID_ARG;
  if (d.table_stride < d.max_pages || d.flags != 0) return THD_ERR_INVALID_ARG;
  if (d.batch > thd::kPagedMaxBatch || d.cap_rows > thd::kPagedTablesMaxBlocks * thd::kPagedTablesRowsPerBlock)
    return THD_ERR_UNSUPPORTED;
  if ((int64_t)d.page_size * d.num_pages >= kInt32End || (int64_t)d.page_size * d.max_pages >= kInt32End)
    return THD_ERR_UNSUPPORTED;
  auto* p = new_plan(kPlanPagedTables, thd::kPagedTablesMaxBlocks);
  if (!p) return THD_ERR_INVALID_ARG;
  p->tdesc = d;
  p->ws_bytes = (size_t)align_up(4 * (1 + thd::kPagedTablesMaxBlocks));
  *ws_bytes = p->ws_bytes;
  *out = p;
  return THD_OK;
}

thd_status_t thd_paged_tables(thd_attn_plan_t plan, const int32_t* seq_lens, const int32_t* cu_new,
                              const int32_t* free_pages, const int32_t* free_span, int32_t* block_table,
                              int32_t* slot_map, int32_t* positions, int32_t* seq_lens_out, int32_t* free_begin_out,
                              void* workspace, void* stream) {
  if (!plan || plan->kind != kPlanPagedTables) return THD_ERR_INVALID_ARG;
  const thd_paged_tables_desc_t& d = plan->tdesc;
  if (bad_workspace(workspace)) return THD_ERR_WORKSPACE;
  if (!free_span || !free_begin_out || free_span == free_begin_out || free_span + 1 == free_begin_out)
    return THD_ERR_INVALID_ARG;
  if (d.batch > 0 && (!seq_lens || !cu_new || !seq_lens_out || seq_lens == seq_lens_out)) return THD_ERR_INVALID_ARG;
  if (d.batch > 0 && d.max_pages > 0 && !block_table) return THD_ERR_INVALID_ARG;
  if (d.cap_rows > 0 && (!slot_map || !positions)) return THD_ERR_INVALID_ARG;
  if (d.cap_free > 0 && !free_pages) return THD_ERR_INVALID_ARG;
  thd::PagedTablesParams tp;
  tp.seq_lens = seq_lens; tp.cu_new = cu_new; tp.free_pages = free_pages; tp.free_span = free_span;
  tp.block_table = block_table; tp.slot_map = slot_map; tp.positions = positions;
  tp.seq_lens_out = seq_lens_out; tp.free_begin_out = free_begin_out;
  tp.table_stride = d.table_stride;
  tp.batch = d.batch; tp.page_size = d.page_size; tp.num_pages = d.num_pages; tp.max_pages = d.max_pages;
  tp.cap_rows = d.cap_rows; tp.cap_free = d.cap_free;
  tp.by_page = thd::FastDiv(d.page_size);
  tp.status = static_cast<uint32_t*>(workspace);
  return thd::launch_paged_tables(tp, static_cast<cudaStream_t>(stream)) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

// --------------------------------------------------- one-token attention over pages

thd_status_t thd_paged_decode_plan(thd_attn_plan_t* out, const thd_paged_decode_desc_t* desc, size_t* ws_bytes) {
  if (!out || !desc || !ws_bytes) return THD_ERR_INVALID_ARG;
  *out = nullptr;
  const thd_paged_decode_desc_t& d = *desc;
  if (!known_dtype(d.dtype)) return THD_ERR_INVALID_ARG;
  if (d.batch < 0 || d.h_q < 1 || d.h_kv < 1 || d.h_q % d.h_kv != 0 || d.d < 1) return THD_ERR_INVALID_ARG;
  if (d.page_size < 1 || d.num_pages < 0 || d.max_pages < 0 || d.table_stride < d.max_pages)
    return THD_ERR_INVALID_ARG;
  if (d.stats_layout != THD_STATS_TOKEN_MAJOR && d.stats_layout != THD_STATS_HEAD_MAJOR) return THD_ERR_INVALID_ARG;
  if (d.kernel != THD_KERNEL_AUTO && d.kernel != THD_KERNEL_SIMT && d.kernel != THD_KERNEL_MMA)
    return THD_ERR_INVALID_ARG;
  if (d.flags != 0) return THD_ERR_INVALID_ARG;
  if (d.d > 128 || d.batch > thd::kPagedMaxBatch || d.h_q > 65536) return THD_ERR_UNSUPPORTED;
  // a key's number, rounded up to a step of the kernel, stays an int
  if ((int64_t)d.page_size * d.num_pages >= kInt32End || (int64_t)d.page_size * d.max_pages >= kInt32End - 256)
    return THD_ERR_UNSUPPORTED;
  const float scale = std::isnan(d.softmax_scale) ? 1.0f / std::sqrt((float)d.d) : d.softmax_scale;
  if (!std::isfinite(scale)) return THD_ERR_INVALID_ARG;
  const int eb = elem_bytes(d.dtype);
  const int64_t heads[4] = {d.h_q, d.h_kv, d.h_kv, d.h_q};
  bool mma = d.dtype != THD_FP32 && d.d % 8 == 0;
  for (int i = 0; i < 4; ++i) {
    const bool cache = i == 1 || i == 2;
    if (d.stride_tok[i] < 0 || d.stride_head[i] < 0 || d.bytes[i] < 0 || (cache && d.stride_page[i] < 0))
      return THD_ERR_INVALID_ARG;
    if (cache)
      mma = mma && d.stride_tok[i] * eb % 16 == 0 && d.stride_head[i] * eb % 16 == 0 &&
            d.stride_page[i] * eb % 16 == 0 && d.stride_tok[i] < kInt32End && d.stride_head[i] < kInt32End &&
            d.stride_page[i] < kInt32End;
    else
      mma = mma && d.stride_tok[i] % 2 == 0 && d.stride_head[i] % 2 == 0;  // Q and O are accessed in pairs
    if (d.bytes[i] == 0) continue;
    const int64_t span = cache ? cache_span(d.num_pages, d.page_size, heads[i], d.d, d.stride_page[i], d.stride_tok[i],
                                            d.stride_head[i], eb)
                               : thd_attn_view_span_bytes(d.batch, heads[i], d.d, d.stride_tok[i], d.stride_head[i], eb);
    if (span > d.bytes[i]) return THD_ERR_CAPACITY;
  }
  if (d.kernel == THD_KERNEL_MMA && !mma) return THD_ERR_UNSUPPORTED;
  if (d.kernel == THD_KERNEL_SIMT) mma = false;
  const int group = d.h_q / d.h_kv;
  const int seg_heads = thd::decode_seg_heads(group, mma);
  const int64_t segs = (int64_t)d.h_kv * ((group + seg_heads - 1) / seg_heads);
  const int64_t max_chunks = (int64_t)d.max_pages * d.page_size / thd::kDecodeMinChunk + 3;
  // the line's chunks: below 2^31 for each worker, and chunks x workers inside 64 bits
  if ((double)d.batch * (double)segs * (double)max_chunks >= (double)(int64_t(1) << 38)) return THD_ERR_UNSUPPORTED;
  const bool few = d.batch <= 256 && d.batch * segs * max_chunks < kInt32End;
  auto* p = new_plan(kPlanPagedDecode, thd::kDecodeMaxCtas);
  if (!p) return THD_ERR_INVALID_ARG;
  p->ddesc = d;
  p->few_requests = few;
  p->elem_bytes = eb;
  p->scale = scale;
  p->kernel = mma ? THD_KERNEL_MMA : THD_KERNEL_SIMT;
  p->rows_per_unit = seg_heads;
  p->keys_per_tile = thd::kDecodeMinChunk;
  p->stats_tok = d.stats_layout == THD_STATS_TOKEN_MAJOR ? d.h_q : 1;
  p->stats_head = d.stats_layout == THD_STATS_TOKEN_MAJOR ? 1 : d.batch;
  const int64_t rows = 2 * (int64_t)thd::kDecodeMaxWorkers * seg_heads;
  int64_t off = align_up(4 * (1 + thd::kDecodeMaxCtas));
  p->ws_off[1] = off; off = align_up(off + thd::kDecodeMaxWorkers * (int64_t)sizeof(thd::DecodeRec));
  p->ws_off[3] = off; off = align_up(off + rows * thd::decode_pad_d(d.d) * 4);
  p->ws_off[4] = off; off = align_up(off + rows * 4);
  p->ws_bytes = (size_t)off;
  *ws_bytes = p->ws_bytes;
  *out = p;
  return THD_OK;
}

thd_status_t thd_paged_decode(thd_attn_plan_t plan, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* window_left,
                              void* o, float* stats, void* workspace, void* stream) {
  if (!plan || plan->kind != kPlanPagedDecode) return THD_ERR_INVALID_ARG;
  const thd_paged_decode_desc_t& d = plan->ddesc;
  if (bad_workspace(workspace)) return THD_ERR_WORKSPACE;
  if (d.batch > 0 && (!q || !o || !seq_lens)) return THD_ERR_INVALID_ARG;
  if (d.batch > 0 && d.max_pages > 0 && !block_table) return THD_ERR_INVALID_ARG;
  if (d.num_pages > 0 && (!k_cache || !v_cache)) return THD_ERR_INVALID_ARG;
  if (plan->kernel == THD_KERNEL_MMA && (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 4) || !aligned(o, 4)))
    return THD_ERR_ALIGNMENT;
  thd::DecodeParams dp;
  dp.q = q; dp.k = k_cache; dp.v = v_cache; dp.o = o; dp.stats = stats;
  dp.block_table = block_table; dp.seq_lens = seq_lens; dp.window = window_left;
  dp.q_tok = d.stride_tok[0]; dp.q_head = d.stride_head[0];
  dp.k_page = d.stride_page[1]; dp.k_tok = d.stride_tok[1]; dp.k_head = d.stride_head[1];
  dp.v_page = d.stride_page[2]; dp.v_tok = d.stride_tok[2]; dp.v_head = d.stride_head[2];
  dp.o_tok = d.stride_tok[3]; dp.o_head = d.stride_head[3];
  dp.table_stride = d.table_stride;
  dp.stats_tok = plan->stats_tok; dp.stats_head = plan->stats_head;
  dp.batch = d.batch; dp.h_q = d.h_q; dp.h_kv = d.h_kv; dp.d = d.d; dp.group = d.h_q / d.h_kv;
  dp.page_size = d.page_size; dp.num_pages = d.num_pages; dp.max_pages = d.max_pages;
  dp.by_page = thd::FastDiv(d.page_size);
  dp.few = plan->few_requests;
  const int64_t eb = plan->elem_bytes;
  dp.aligned = aligned(k_cache, 16) && aligned(v_cache, 16) && d.d * eb % 16 == 0;
  for (int i = 1; i < 3; ++i)
    dp.aligned = dp.aligned && d.stride_tok[i] * eb % 16 == 0 && d.stride_head[i] * eb % 16 == 0 &&
                 d.stride_page[i] * eb % 16 == 0;
  dp.scale_log2 = plan->scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  dp.status = reinterpret_cast<uint32_t*>(ws);
  dp.recs = reinterpret_cast<thd::DecodeRec*>(ws + plan->ws_off[1]);
  dp.part_o = reinterpret_cast<float*>(ws + plan->ws_off[3]);
  dp.part_lse = reinterpret_cast<float*>(ws + plan->ws_off[4]);
  const int sms = thd::current_device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  return thd::launch_paged_decode(dp, d.dtype, plan->kernel == THD_KERNEL_MMA, sms,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? THD_OK
             : THD_ERR_CUDA;
}

}  // extern "C"
