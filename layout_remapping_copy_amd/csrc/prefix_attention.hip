// Attention of a batch that shares a prefix: lr_prefix_attention_plan and lr_prefix_attention.
//
// The softmax over a sequence's tokens is split at the prefix's end: one pass over the prefix serves all sequences, whose
// query heads of one cache head are the rows of one product with its keys; a second pass takes each sequence's own
// tokens; parts (m, l, o) of both are joined by the rule that joins the parts of one sequence.
#include "attention.h"

namespace lr {

struct PrefixJoin {
  const float *ml, *o;  // parts of the prefix, for row b * group + r of cache head g: (g, row, split)
  uint32_t splits, group, batch;
  FastDiv fd_group;
};

template <int DT>
__global__ void __launch_bounds__(256) k_prefix_join(AttentionArgs a, PrefixJoin p) {
  __shared__ __attribute__((aligned(16))) float os[256 * 4];
  const uint32_t b = blockIdx.x / a.heads, h = blockIdx.x % a.heads, g = op_div(h, p.fd_group);
  const Columns q4 = columns_of(a.dv);
  const uint64_t own = (uint64_t)blockIdx.x * a.splits;
  const uint64_t pre = ((uint64_t)(g * p.batch + b) * p.group + (h - g * p.group)) * p.splits;
  Joined j{-__builtin_inff(), 0.f, F4{}};
  join_list(p.ml + 2 * pre, p.o + pre * a.dv, p.splits, a.dv, q4, false, &j);
  join_list(a.part_ml + 2 * own, a.part_o + own * a.dv, a.splits, a.dv, q4, false, &j);
  join_out<DT>(a, b, h, q4, j, a.lens[b] < 0, os);
}

// The arguments of both passes and what they leave.
struct PrefixPlan {
  AttentionArgs own, pre;
  lr_attention_plan p_own, p_pre;
  int64_t rows;             // sequences * heads
  int64_t o_own, o_pre;     // in the workspace, floats: sums; maxima and sums of weights come first
  int64_t workspace_bytes;
};
static int plan_prefix(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t prefix_pages,
                       int64_t max_pages, int32_t dtype, PrefixPlan* p) {
  if (int rc = attention_shapes(Lq, c, Lo, max_pages, dtype, &p->own, &p->p_own)) return rc;
  if (prefix_pages < 1) return LR_ERR_INVALID;
  if (prefix_pages > kMaxCount / p->own.page_size) return LR_ERR_OVERFLOW;
  const int64_t sequences = mode_of(*Lq, 2).size;
  p->rows = sequences * p->own.heads;
  if (p->rows > kMaxCount) return LR_ERR_OVERFLOW;
  p->own.parts = true;
  p->pre = p->own;
  p->p_pre = p->p_own;
  if (int rc = attention_split(sequences, max_pages * p->own.page_size, false, &p->own, &p->p_own)) return rc;
  p->pre.max_pages = (uint32_t)prefix_pages;
  p->pre.group = (uint32_t)(sequences * p->own.group);
  p->pre.heads = (uint32_t)p->rows;
  if (int rc = attention_split(1, prefix_pages * p->own.page_size, false, &p->pre, &p->p_pre)) return rc;
  const int64_t parts = p->rows * (p->p_own.splits + p->p_pre.splits), dv = p->own.dv;
  p->o_own = (2 * parts + 3) / 4 * 4;
  p->o_pre = p->o_own + (p->rows * p->p_own.splits * dv + 3) / 4 * 4;
  p->workspace_bytes = (p->o_pre + p->rows * p->p_pre.splits * dv) * 4;
  return LR_OK;
}

}  // namespace lr

using namespace lr;

extern "C" {

int lr_prefix_attention_plan(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t prefix_pages,
                             int64_t max_pages, int32_t dtype, lr_prefix_plan* out) {
  if (!out) return LR_ERR_INVALID;
  PrefixPlan p;
  if (int rc = plan_prefix(Lq, c, Lo, prefix_pages, max_pages, dtype, &p)) return rc;
  out->path = p.p_own.path;
  out->row_tiles = (int32_t)p.pre.tiles;
  out->prefix_splits = p.p_pre.splits;
  out->own_splits = p.p_own.splits;
  out->workspace_bytes = p.workspace_bytes;
  return LR_OK;
}

int lr_prefix_attention(const void* q, const lr_layout* Lq, int64_t q_capacity, const lr_cache* c, const int32_t* prefix,
                        int64_t prefix_pages, const int32_t* prefix_len, const int32_t* table, int64_t table_stride,
                        int64_t max_pages, const int32_t* lens, int64_t batch, void* out, const lr_layout* Lo,
                        int64_t out_capacity, float* lse, int32_t dtype, float scale, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  if (!q || !out || batch < 0 || (batch > 0 && (!prefix || !prefix_len || !table || !lens)) || !std::isfinite(scale) ||
      table_stride < 0)
    return LR_ERR_INVALID;
  PrefixPlan p;
  if (int rc = plan_prefix(Lq, c, Lo, prefix_pages, max_pages, dtype, &p)) return rc;
  if (cosize_bound(Lq) > q_capacity || cosize_bound(Lo) > out_capacity || batch > mode_of(*Lq, 2).size)
    return LR_ERR_BOUNDS;
  if (!workspace || workspace_bytes < p.workspace_bytes) return LR_ERR_CAPACITY;
  if ((uintptr_t)workspace % 16) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  const Buffer in[] = {{q, q_capacity * e}, {c->k, c->k_capacity * ce}, {c->v, c->v_capacity * ce},
                       {c->k_scale, c->scale_capacity * 4}, {c->v_scale, c->scale_capacity * 4}, {prefix, prefix_pages * 4},
                       {prefix_len, 4}, {table, batch ? ((batch - 1) * table_stride + max_pages) * 4 : 0}, {lens, batch * 4}};
  const Buffer made[] = {{out, out_capacity * e}, {lse, lse ? batch * p.own.heads * 4 : 0}, {workspace, p.workspace_bytes}};
  if (int rc = check_overlaps(in, 9, made, 3)) return rc;
  if (batch == 0) return LR_OK;
  AttentionArgs &a = p.own, &x = p.pre;
  float* ws = (float*)workspace;
  a.q = x.q = q;
  a.out = out;
  a.lse = lse;
  a.scale2 = x.scale2 = scale * kLog2e;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.batch = (uint32_t)batch;
  a.part_ml = ws;
  a.part_o = ws + p.o_own;
  // the prefix: one sequence, whose rows are those of the whole batch
  x.table = prefix;
  x.table_stride = 0;
  x.lens = prefix_len;
  x.batch = 1;
  x.group = (uint32_t)(batch * a.group);
  x.heads = (uint32_t)(batch * a.heads);
  x.tiles = (x.group + x.unit_heads - 1) / x.unit_heads;
  x.units = x.kv_heads / x.wide_heads * x.tiles;
  x.part_ml = ws + 2 * p.rows * p.p_own.splits;
  x.part_o = ws + p.o_pre;
  attention_buffers(c, Lq, q, dtype, p.p_own.path, &a);
  attention_buffers(c, Lq, q, dtype, p.p_pre.path, &x);
  const hipStream_t st = (hipStream_t)stream;
  if (int rc = launch_attention_pass(x, dtype, c->dtype, st)) return rc;
  if (int rc = launch_attention_pass(a, dtype, c->dtype, st)) return rc;
  const PrefixJoin j{x.part_ml, x.part_o, x.splits, a.group, a.batch, make_fastdiv(a.group)};
  return with_model_type(dtype, [&](auto dt) {
    hipLaunchKernelGGL((k_prefix_join<decltype(dt)::value>), dim3((unsigned)(batch * a.heads)), dim3(256), 0, st, a, j);
    return check_op_launch();
  });
}

}  // extern "C"
