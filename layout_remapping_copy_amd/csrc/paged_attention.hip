// Attention of one new token over a paged cache: lr_paged_attention_plan and lr_paged_attention, and the plans and
// launches that the other passes over such a cache share with it.
#include "attention.h"

namespace lr {

int attention_shapes(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages, int32_t dtype,
                     AttentionArgs* a, lr_attention_plan* out) {
  if (int rc = lr_cache_validate(c)) return rc;
  if (!is_model_type(dtype) || (!is_quantised(c->dtype) && c->dtype != dtype)) return LR_ERR_TYPE;
  int rc = check_tensor(Lq, 3, INT64_MAX, false);
  if (rc || (rc = check_tensor(Lo, 3, INT64_MAX, true))) return rc;
  std::memset(a, 0, sizeof(*a));
  const Mode qd = mode_of(*Lq, 0), qh = mode_of(*Lq, 1), qb = mode_of(*Lq, 2);
  const Mode od = mode_of(*Lo, 0), oh = mode_of(*Lo, 1), ob = mode_of(*Lo, 2);
  if (one_leaf(qd, &a->qd) || one_leaf(qh, &a->qh) || one_leaf(qb, &a->qb) || one_leaf(od, &a->od) ||
      one_leaf(oh, &a->oh) || one_leaf(ob, &a->ob))
    return LR_ERR_INVALID;
  const Mode kd = mode_of(c->k_layout, 0), kh = mode_of(c->k_layout, 1), ks = mode_of(c->k_layout, 2);
  const Mode kp = mode_of(c->k_layout, 3), vd = mode_of(c->v_layout, 0), vh = mode_of(c->v_layout, 1);
  const Mode vs = mode_of(c->v_layout, 2), vp = mode_of(c->v_layout, 3);
  one_leaf(kd, &a->kd), one_leaf(kh, &a->kh), one_leaf(ks, &a->ksl), one_leaf(kp, &a->kp);  // checked above
  one_leaf(vd, &a->vd), one_leaf(vh, &a->vh), one_leaf(vs, &a->vsl), one_leaf(vp, &a->vp);
  if (is_quantised(c->dtype)) {
    one_leaf(mode_of(c->scale_layout, 0), &a->sh);
    one_leaf(mode_of(c->scale_layout, 1), &a->ssl);
    one_leaf(mode_of(c->scale_layout, 2), &a->sp);
  }
  if (qd.size != kd.size || od.size != vd.size || oh.size != qh.size || ob.size != qb.size) return LR_ERR_SIZE_MISMATCH;
  if (qh.size % kh.size) return LR_ERR_SIZE_MISMATCH;
  if (kd.size > kAttentionDim || vd.size > kAttentionDim || max_pages < 1) return LR_ERR_INVALID;
  if (max_pages > kMaxCount / ks.size) return LR_ERR_OVERFLOW;
  a->dk = (int32_t)kd.size;
  a->dv = (int32_t)vd.size;
  a->heads = (uint32_t)qh.size;
  a->kv_heads = (uint32_t)kh.size;
  a->group = a->row_heads = (uint32_t)(qh.size / kh.size);
  a->fd_rows = make_fastdiv(a->row_heads);
  a->page_size = (uint32_t)ks.size;
  a->fd_page = make_fastdiv(a->page_size);
  a->pages = (uint32_t)kp.size;
  a->max_pages = (uint32_t)max_pages;
  a->k = c->k;
  a->v = c->v;
  a->ks = c->k_scale;
  a->vs = c->v_scale;
  // The matrix kernel wants rows of whole chunks: a multiple of 8 elements (4 in fp32), contiguous and
  // that much aligned, and keys of at least one chunk of 16 codes.
  const int64_t v = c->dtype == LR_F32 ? 4 : 8;
  const bool matrix = (kd.size >= 16 || !is_quantised(c->dtype)) && kd.size % v == 0 && vd.size % v == 0 &&
                      rows_aligned(c->k_layout, nullptr, dtype_bytes(c->dtype), v) &&
                      rows_aligned(c->v_layout, nullptr, dtype_bytes(c->dtype), v);
  out->path = matrix ? LR_ATTENTION_MATRIX : LR_ATTENTION_ELEMENT;
  const int64_t widest = std::max(kd.size, vd.size);
  // Loads past a row's end are not free, though they ask for what another lane does: rows of 72 in the width of 128
  // took 190 us where the width of 96 takes 155 (16 sequences of up to 30000 bf16 tokens, 8 heads), of 160 in 192
  // 284 and 264, of 32 in 64 81 and 68.  Rows of codes, loaded 64 at a time, have no use for 32, 96 and 160.
  const bool codes = is_quantised(c->dtype);
  a->wide = widest <= 32 && !codes ? 32 : widest <= 64 ? 64 : widest <= 96 && !codes ? 96 : widest <= 128 ? 128
            : widest <= 160 && !codes ? 160 : widest <= 192 ? 192 : 256;
  return LR_OK;
}

int attention_split(int64_t sequences, int64_t span, bool listed, AttentionArgs* a, lr_attention_plan* out) {
  a->unit_heads = out->path != LR_ATTENTION_MATRIX ? 1 : a->group > 16 && a->wide <= 128 ? 32 : 16;
  a->tiles = (a->group + a->unit_heads - 1) / a->unit_heads;
  // Four cache heads a workgroup, one a wave, where a token's heads lie next to each other: their rows then share
  // lines and pages of memory (16 sequences of up to 30000 tokens, 8 heads: 174 us against 198 in bf16 of 128, 73
  // against 111 in e4m3 of 64).  Where a head's tokens lie next to each other, the four waves take tokens of one
  // head; also where a run would be under 8 steps, as four heads leave four times the parts to join (one sequence of
  // 4000 tokens: 16 us against 21).
  const int64_t ktok = std::abs(a->page_size > 1 ? a->ksl : a->kp), vtok = std::abs(a->page_size > 1 ? a->vsl : a->vp);
  out->head_tiles = (int32_t)a->tiles;
  // Parts of a sequence: short ones stay whole, which saves the second launch; otherwise as many as there
  // are blocks, up to 8192 parts in all (their sums are some 66 MB for 16 heads of 128), or 8 a unit.
  const int64_t steps = (int64_t)((double)sequences * a->kv_heads / 4 * a->tiles * (double)((span + 31) / 32));
  const bool by_heads = out->path == LR_ATTENTION_MATRIX && !listed && a->kv_heads % 4 == 0 && std::abs(a->kh) < ktok &&
                        std::abs(a->vh) < vtok && span <= (int64_t(1) << 30) && steps >= 8 * kRuns;
  a->wide_heads = by_heads ? 4 : 1;
  // Heads that end inside a line: their waves keep in step, so that the line is still near for the second of them
  // (as above: heads of 72 in bf16 153 to 144 us, of 112 201 to 185, of 160 265 to 254).  Heads of 64 would lose 6 %
  // by it and whole lines up to 1 %; codes of 80 to 192 gain 2 to 4 %, but lose as much with heads of up to 64.
  a->in_step = by_heads && a->dk > 64 && a->dk % 64;
  a->block = by_heads ? kWideBlock : kBlock;
  a->units = a->kv_heads / a->wide_heads * a->tiles;
  const int64_t blocks = (span + a->block - 1) / a->block;
  const double units = (double)sequences * a->units;
  int64_t most = blocks <= 4 ? 1 : std::min(blocks, std::max<int64_t>((int64_t)(8192 / units), 8));
  out->chunk = (span + most - 1) / most;
  out->splits = (span + out->chunk - 1) / out->chunk;
  const double parts = (double)sequences * a->heads * (double)out->splits;
  if (parts > (double)kMaxCount / 256 || units > (double)kMaxCount || units * blocks > 0x1p50) return LR_ERR_OVERFLOW;
  a->min_share = out->splits > 1 ? (uint32_t)((blocks - 2) / (out->splits - 1) + 1) : 1;
  out->workspace_bytes = out->splits == 1 ? 0 : (int64_t)parts * (a->dv + 2) * 4;
  a->splits = (uint32_t)out->splits;
  return LR_OK;
}

void attention_buffers(const lr_cache* c, const lr_layout* Lq, const void* q, int32_t dtype, int32_t path, AttentionArgs* a) {
  const uintptr_t align = is_quantised(c->dtype) ? 8 : 16;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  a->path = path;
  if (a->path == LR_ATTENTION_MATRIX && ((uintptr_t)c->k % align || (uintptr_t)c->v % align)) a->path = LR_ATTENTION_ELEMENT;
  if (a->path == LR_ATTENTION_ELEMENT) {
    a->unit_heads = 1;
    a->wide_heads = 1;
    a->block = kBlock;
    a->tiles = a->group;
    a->units = a->kv_heads * a->group;
  }
  a->q_wide = rows_aligned(*Lq, q, e, 16 / e);
  // Two workgroups a CU where a step is too short for one to keep enough loads under way: rows of 64 bytes 74 us with
  // one, 60 with two; of 80 bytes 89 and 84; of 128 bytes 91 and 95.  Four heads at once ask for enough.
  const bool small_step = a->wide_heads == 1 && (a->dk + a->dv) * ce <= 192;
  a->grid = (uint32_t)(a->path == LR_ATTENTION_ELEMENT ? 8 * kRuns : small_step ? 2 * kRuns : kRuns);
}

int launch_attention_pass(const AttentionArgs& a, int32_t dtype, int32_t ctype, hipStream_t st) {
  return with_model_type(dtype, [&](auto dt) {
    constexpr int D = decltype(dt)::value;
    if (ctype == LR_E4M3) return launch_pass<D, LR_E4M3, false>(a, st);
    if (ctype == LR_INT8) return launch_pass<D, LR_INT8, false>(a, st);
    return launch_pass<D, D, false>(a, st);
  });
}

int launch_attention_join(const AttentionArgs& a, int32_t dtype, hipStream_t st) {
  return with_model_type(dtype, [&](auto dt) {
    hipLaunchKernelGGL((k_attention_join<decltype(dt)::value>), dim3(a.batch * a.heads), dim3(256), 0, st, a);
    return check_op_launch();
  });
}

static int plan_attention(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages, int32_t dtype,
                          int64_t window, AttentionArgs* a, lr_attention_plan* out) {
  if (int rc = attention_shapes(Lq, c, Lo, max_pages, dtype, a, out)) return rc;
  if (window < 0) return LR_ERR_INVALID;
  a->window = std::min(window, kMaxCount);
  int64_t span = max_pages * a->page_size;
  if (a->window > 0) span = std::min(span, a->window + 31);
  return attention_split(mode_of(*Lq, 2).size, span, false, a, out);
}

}  // namespace lr

using namespace lr;

extern "C" {

int lr_paged_attention_plan(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages,
                            int32_t dtype, int64_t window, lr_attention_plan* out) {
  if (!out) return LR_ERR_INVALID;
  AttentionArgs a;
  return plan_attention(Lq, c, Lo, max_pages, dtype, window, &a, out);
}

int lr_paged_attention(const void* q, const lr_layout* Lq, int64_t q_capacity, const lr_cache* c, const int32_t* table,
                       int64_t table_stride, int64_t max_pages, const int32_t* lens, int64_t batch, void* out,
                       const lr_layout* Lo, int64_t out_capacity, float* lse, int32_t dtype, float scale, int64_t window,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !out || batch < 0 || (batch > 0 && (!table || !lens)) || !std::isfinite(scale)) return LR_ERR_INVALID;
  AttentionArgs a;
  lr_attention_plan p;
  if (int rc = plan_attention(Lq, c, Lo, max_pages, dtype, window, &a, &p)) return rc;
  if (cosize_bound(Lq) > q_capacity || cosize_bound(Lo) > out_capacity || batch > mode_of(*Lq, 2).size)
    return LR_ERR_BOUNDS;
  if (table_stride < 0) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  const int64_t lse_bytes = lse ? batch * a.heads * 4 : 0;
  const int64_t table_bytes = batch ? ((batch - 1) * table_stride + max_pages) * 4 : 0;
  const Buffer in[] = {{q, q_capacity * e}, {c->k, c->k_capacity * ce}, {c->v, c->v_capacity * ce},
      {c->k_scale, c->scale_capacity * 4}, {c->v_scale, c->scale_capacity * 4}, {table, table_bytes}, {lens, batch * 4}};
  const Buffer made[] = {{out, out_capacity * e}, {lse, lse_bytes}, {workspace, p.workspace_bytes}};
  if (p.workspace_bytes && (!workspace || workspace_bytes < p.workspace_bytes)) return LR_ERR_CAPACITY;
  if (p.workspace_bytes && (uintptr_t)workspace % 16) return LR_ERR_INVALID;
  if (int rc = check_overlaps(in, 7, made, 3)) return rc;
  if (batch == 0) return LR_OK;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.batch = (uint32_t)batch;
  a.scale2 = scale * kLog2e;
  a.part_o = (float*)workspace;
  a.part_ml = (float*)workspace + (p.workspace_bytes / 4 - 2 * (int64_t)mode_of(*Lq, 2).size * a.heads * p.splits);
  attention_buffers(c, Lq, q, dtype, p.path, &a);
  const hipStream_t st = (hipStream_t)stream;
  if (int rc = launch_attention_pass(a, dtype, c->dtype, st)) return rc;
  return a.splits == 1 ? LR_OK : launch_attention_join(a, dtype, st);
}

}  // extern "C"
