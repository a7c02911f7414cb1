// Attention of one new token over a paged cache: lr_paged_attention_plan and lr_paged_attention.
//
// With s_t = scale q . k_t over the tokens t a sequence sees, out = sum_t e^(s_t - m) v_t / l with
// m = max s_t and l = sum_t e^(s_t - m).  One pass holds (m, l, o) for the tokens seen so far and
// rescales l and o by e^(m - m') when m grows to m'; parts of a sequence are joined by the same rule.
// Scores are held in base-2 units (scale * log2 e folded in), so that e^x is one v_exp_f32.
#include "op_common.h"

namespace lr {

constexpr int kAttentionDim = 256;  // head_dim at most
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttentionArgs {
  const void *q, *k, *v;
  const float *ks, *vs;
  const int32_t *table, *lens;
  void* out;
  float* lse;
  float *part_o, *part_ml;    // per (sequence, head, split): Dv sums; maximum and sum
  int64_t qd, qh, qb, od, oh, ob;
  int64_t kd, kh, ksl, kp, vd, vh, vsl, vp;  // cache strides: head dimension, heads, slots, pages
  int64_t sh, ssl, sp;
  int64_t table_stride;
  int32_t dk, dv;
  uint32_t heads, kv_heads, group, page_size, pages, max_pages, batch;
  FastDiv fd_page;
  uint32_t chunk, splits;
  int64_t window;
  float scale2;  // scale * log2 e
};

// The tokens [first, n) a sequence sees; chunks start at `base`, first rounded down so
// that their tiles stay aligned to 32 tokens.
struct Span {
  uint32_t base, first, n;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& a, uint32_t b) {
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : n > cap ? cap : n;
  const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
  return Span{(uint32_t)first & ~31u, (uint32_t)first, (uint32_t)n};
}

// Weight 2^(m - top) of a part with maximum m among parts with maximum top; 0 for a part
// without tokens.
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

// Any types, strides and alignment.  A workgroup has one chunk of one query head; its
// waves take tiles of 64 tokens in turn, a lane a token for the scores and every 64th
// value column for the sums.
template <int DT, int CT>
__global__ void __launch_bounds__(256) k_attention_element(AttentionArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  __shared__ float qs[kAttentionDim];
  __shared__ float ps[4][64];
  __shared__ int64_t at[4][64];
  __shared__ float os[4][kAttentionDim];
  __shared__ float ms[4], ls[4];
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x / 64;
  const uint32_t split = blockIdx.x % a.splits, bh = blockIdx.x / a.splits, b = bh / a.heads, h = bh % a.heads;
  const uint32_t g = h / a.group;
  const Span sp = span_of(a, b);
  const uint64_t lo = (uint64_t)sp.base + (uint64_t)split * a.chunk;
  if (split && lo >= sp.n) return;
  const uint32_t hi = (uint32_t)(lo + a.chunk < sp.n ? lo + a.chunk : sp.n);
  for (uint32_t e = threadIdx.x; e < (uint32_t)a.dk; e += 256)
    qs[e] = value_of<DT>(((const T*)a.q)[(int64_t)b * a.qb + (int64_t)h * a.qh + (int64_t)e * a.qd]) * a.scale2;
  __syncthreads();
  float m = -__builtin_inff(), l = 0, o[kAttentionDim / 64] = {};
  for (uint64_t t0 = lo + 64 * w; t0 < hi; t0 += 256) {
    const uint32_t t = (uint32_t)t0 + lane;
    bool seen = t < hi && t >= sp.first;
    int64_t page = 0;
    const uint32_t pg = op_div(t, a.fd_page), in = t - pg * a.page_size;
    if (seen) {
      page = a.table[(int64_t)b * a.table_stride + pg];
      seen = page >= 0 && page < (int64_t)a.pages;
    }
    float s = -__builtin_inff(), vscale = 1;
    if (seen) {
      const C* k = (const C*)a.k + page * a.kp + (int64_t)in * a.ksl + (int64_t)g * a.kh;
      float dot = 0;
      for (int e = 0; e < a.dk; ++e) dot += qs[e] * value_of<CT>(k[(int64_t)e * a.kd]);
      if constexpr (CT == LR_E4M3 || CT == LR_INT8) {
        const int64_t so = page * a.sp + (int64_t)in * a.ssl + (int64_t)g * a.sh;
        dot *= a.ks[so];
        vscale = a.vs[so];
      }
      s = dot;
    }
    float top = s;
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    top = fmaxf(m, top);
    const float keep = weight_of(m, top);
    const float p = seen ? __builtin_amdgcn_exp2f(s - (top == -__builtin_inff() ? 0.f : top)) : 0.f;
    float sum = p;
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = top;
    ps[w][lane] = p * vscale;
    at[w][lane] = seen ? page * a.vp + (int64_t)in * a.vsl + (int64_t)g * a.vh : -1;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kAttentionDim / 64; ++i) {
      const int e = (int)lane + 64 * i;
      if (64 * i >= a.dv) break;
      float acc = o[i] * keep;
      for (int j = 0; j < 64; ++j) {
        const int64_t off = at[w][j];
        if (off >= 0 && e < a.dv) acc += ps[w][j] * value_of<CT>(((const C*)a.v)[off + (int64_t)e * a.vd]);
      }
      o[i] = acc;
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (lane == 0) {
    ms[w] = m;
    ls[w] = l;
  }
#pragma unroll
  for (int i = 0; i < kAttentionDim / 64; ++i) os[w][lane + 64 * i] = o[i];
  __syncthreads();
  const float top = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
  float total = 0, wt[4];
  for (int i = 0; i < 4; ++i) {
    wt[i] = weight_of(ms[i], top);
    total += ls[i] * wt[i];
  }
  const uint32_t e = threadIdx.x;
  if (e < (uint32_t)a.dv) {
    float acc = 0;
    for (int i = 0; i < 4; ++i) acc += os[i][e] * wt[i];
    if (a.splits == 1)
      ((T*)a.out)[(int64_t)b * a.ob + (int64_t)h * a.oh + (int64_t)e * a.od] = (T)(total > 0 ? acc / total : 0.f * acc);
    else
      a.part_o[((uint64_t)bh * a.splits + split) * a.dv + e] = acc;
  }
  if (threadIdx.x == 0) {
    if (a.splits > 1) {
      a.part_ml[2 * ((uint64_t)bh * a.splits + split)] = top;
      a.part_ml[2 * ((uint64_t)bh * a.splits + split) + 1] = total;
    } else if (a.lse) {
      a.lse[bh] = top == -__builtin_inff() ? top : (top + __log2f(total)) * kLn2;
    }
  }
}

// Joins the chunks of one query head in their order.
template <int DT>
__global__ void __launch_bounds__(256) k_attention_join(AttentionArgs a) {
  using T = typename ElemOf<DT>::T;
  const uint32_t bh = blockIdx.x, b = bh / a.heads, h = bh % a.heads;
  const Span sp = span_of(a, b);
  const uint32_t used = sp.n > sp.base ? (sp.n - sp.base + a.chunk - 1) / a.chunk : 1;  // chunk 0 always writes
  const float* ml = a.part_ml + 2 * (uint64_t)bh * a.splits;
  float top = -__builtin_inff();
  for (uint32_t s = 0; s < used; ++s) top = fmaxf(top, ml[2 * s]);
  float total = 0, acc = 0;
  const uint32_t e = threadIdx.x;
  for (uint32_t s = 0; s < used; ++s) {
    const float wt = weight_of(ml[2 * s], top);
    total += ml[2 * s + 1] * wt;
    if (e < (uint32_t)a.dv) acc += a.part_o[((uint64_t)bh * a.splits + s) * a.dv + e] * wt;
  }
  if (e < (uint32_t)a.dv)
    ((T*)a.out)[(int64_t)b * a.ob + (int64_t)h * a.oh + (int64_t)e * a.od] = (T)(total > 0 ? acc / total : 0.f * acc);
  if (e == 0 && a.lse) a.lse[bh] = top == -__builtin_inff() ? top : (top + __log2f(total)) * kLn2;
}

// ------------------------------------------------------------------ host

// Everything but the buffers: the layouts' checks, the plan and the kernel arguments.
static int plan_attention(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages, int32_t dtype,
                          int64_t window, AttentionArgs* a, lr_attention_plan* out) {
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
  if (kd.size > kAttentionDim || vd.size > kAttentionDim || max_pages < 1 || window < 0) return LR_ERR_INVALID;
  if (max_pages > kMaxCount / ks.size) return LR_ERR_OVERFLOW;
  a->dk = (int32_t)kd.size;
  a->dv = (int32_t)vd.size;
  a->heads = (uint32_t)qh.size;
  a->kv_heads = (uint32_t)kh.size;
  a->group = (uint32_t)(qh.size / kh.size);
  a->page_size = (uint32_t)ks.size;
  a->fd_page = make_fastdiv(a->page_size);
  a->pages = (uint32_t)kp.size;
  a->max_pages = (uint32_t)max_pages;
  window = std::min(window, kMaxCount);
  a->window = window;
  a->k = c->k;
  a->v = c->v;
  a->ks = c->k_scale;
  a->vs = c->v_scale;
  out->path = LR_ATTENTION_ELEMENT;
  out->head_tiles = (int32_t)a->group;
  int64_t span = max_pages * ks.size;
  if (window > 0) span = std::min(span, window + 31);
  const double work = (double)span * (double)qb.size * a->kv_heads * out->head_tiles;
  int64_t chunk = (int64_t)(work / 1024 / 128 + 1) * 128;
  chunk = std::min<int64_t>(std::max<int64_t>(chunk, 128), 2048);
  out->chunk = chunk;
  out->splits = (span + chunk - 1) / chunk;
  const double parts = (double)qb.size * a->heads * (double)out->splits;
  if (parts > (double)kMaxCount / 256) return LR_ERR_OVERFLOW;
  out->workspace_bytes = out->splits == 1 ? 0 : (int64_t)parts * (a->dv + 2) * 4;
  a->chunk = (uint32_t)chunk;
  a->splits = (uint32_t)out->splits;
  return LR_OK;
}

template <int DT, int CT>
static int launch_attention(const AttentionArgs& a, hipStream_t st) {
  const uint32_t rows = a.batch * a.heads;
  hipLaunchKernelGGL((k_attention_element<DT, CT>), dim3(rows * a.splits), dim3(256), 0, st, a);
  if (int rc = check_op_launch()) return rc;
  if (a.splits == 1) return LR_OK;
  hipLaunchKernelGGL((k_attention_join<DT>), dim3(rows), dim3(256), 0, st, a);
  return check_op_launch();
}

template <int DT>
static int launch_attention_of(const AttentionArgs& a, int32_t ctype, hipStream_t st) {
  if (ctype == LR_E4M3) return launch_attention<DT, LR_E4M3>(a, st);
  if (ctype == LR_INT8) return launch_attention<DT, LR_INT8>(a, st);
  return launch_attention<DT, DT>(a, st);
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
  if (!q || !out || !table || !lens || batch < 0 || !std::isfinite(scale)) return LR_ERR_INVALID;
  AttentionArgs a;
  lr_attention_plan p;
  if (int rc = plan_attention(Lq, c, Lo, max_pages, dtype, window, &a, &p)) return rc;
  if (cosize_bound(Lq) > q_capacity || cosize_bound(Lo) > out_capacity || batch > mode_of(*Lq, 2).size) return LR_ERR_BOUNDS;
  if (table_stride < 0) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  const int64_t lse_bytes = lse ? batch * a.heads * 4 : 0, table_bytes = batch ? ((batch - 1) * table_stride + max_pages) * 4 : 0;
  struct { const void* p; int64_t n; } in[] = {{q, q_capacity * e}, {c->k, c->k_capacity * ce}, {c->v, c->v_capacity * ce},
      {c->k_scale, c->k_scale ? c->scale_capacity * 4 : 0}, {c->v_scale, c->v_scale ? c->scale_capacity * 4 : 0},
      {table, table_bytes}, {lens, batch * 4}};
  struct { const void* p; int64_t n; } made[] = {{out, out_capacity * e}, {lse, lse_bytes}, {workspace, p.workspace_bytes}};
  if (p.workspace_bytes && (!workspace || workspace_bytes < p.workspace_bytes)) return LR_ERR_CAPACITY;
  if (p.workspace_bytes && (uintptr_t)workspace % 16) return LR_ERR_INVALID;
  for (int i = 0; i < 3; ++i) {
    if (!made[i].p || !made[i].n) continue;
    for (auto& x : in)
      if (x.n && overlap(x.p, x.n, made[i].p, made[i].n)) return LR_ERR_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (made[j].p && made[j].n && overlap(made[j].p, made[j].n, made[i].p, made[i].n)) return LR_ERR_OVERLAP;
  }
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
  const hipStream_t st = (hipStream_t)stream;
  if (dtype == LR_F32) return launch_attention_of<LR_F32>(a, c->dtype, st);
  if (dtype == LR_F16) return launch_attention_of<LR_F16>(a, c->dtype, st);
  return launch_attention_of<LR_BF16>(a, c->dtype, st);
}

}  // extern "C"
