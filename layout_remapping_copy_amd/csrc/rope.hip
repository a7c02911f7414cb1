// Rotary positions: lr_rope_table and lr_rope.
#include "op_common.h"

namespace lr {

struct RopeArgs {
  const void* x;
  void* y;
  const int64_t* turns;
  const int64_t* positions;
  ModeArg xh, yh, xt, yt, p;  // heads and tokens of x and y, positions
  int64_t xd, yd;             // strides of the head dimension
  int32_t dim, rot, pairs;
  uint32_t heads, n, units;
  FastDiv fd_units, fd_heads;
  float magnitude, sign;
};

struct RopeChunkArgs {
  const void* x;
  void* y;
  const int64_t* turns;
  const int64_t* positions;
  ModePair xh, yh, xt, yt, p;
  Units un;
  RowGrid grid;
  uint32_t heads, n;
  int32_t pairs;
  float magnitude, sign;
};

// Rows in chunks of V elements: a lane has one unit of a token's rows, computes its V angles once and turns
// `per_lane` heads with them, their loads two at a time ahead of the arithmetic.  An angle costs some 40
// instructions, a pair's turn 6: over 8 heads the arithmetic is 37 % of the vector units' time and memory the bound.
// 16 x 4096 x 32 x 128 bf16, heads regrouped on the way (1 GiB moved): 179 us, 6.0 TB/s, against 157 for a plain
// copy and 170 for the same regrouping without arithmetic.  Eight tokens of one step: 4.2 us, two dependent reads
// of memory after the arguments'; a call is 6.9 us of the host.
template <int DT, int V, bool NT>
__global__ void __launch_bounds__(256) k_rope_chunks(RopeChunkArgs a) {
  using T = typename ElemOf<DT>::T;
  using Vec = typename Chunk<T, V>::Vec;
  uint32_t u, h, t;
  if (!row_lane(a.grid, threadIdx.x, &u, &h, &t)) return;
  const uint64_t token = (uint64_t)blockIdx.x * a.grid.tokens + t;
  if (token >= a.n) return;
  t = (uint32_t)token;
  h += blockIdx.y * a.grid.per_lane << a.grid.head_shift;
  uint32_t i, j;
  chunks_of(a.un, u, V, &i, &j);
  const bool turned = u < (uint32_t)a.un.turned, two = j < (uint32_t)a.un.dim, half = a.pairs == LR_PAIRS_HALF;
  const T* x = (const T*)a.x + mode_offset(a.xt, t);
  T* y = (T*)a.y + mode_offset(a.yt, t);
  const uint32_t step = 1u << a.grid.head_shift, last = a.heads - 1;
  Vec v[2], w[2];
  auto load = [&](uint32_t n) {  // heads h + n step and the next
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const T* p = x + mode_offset(a.xh, min(h + (n + z) * step, last));
      v[z] = load_chunk<NT, Vec>(p + i);
      w[z] = load_chunk<NT, Vec>(p + (two ? j : i));
    }
  };
  load(0);
  float c[V], s[V];
  if (turned) angles_of<V>(a.turns, a.positions[mode_offset(a.p, t)], u, a.un.rot, half, a.magnitude, a.sign, c, s);
  const uint32_t left = (a.heads - (blockIdx.y * a.grid.per_lane << a.grid.head_shift) + step - 1) >> a.grid.head_shift;
  const uint32_t count = min(a.grid.per_lane, left);  // the same for all lanes
  for (uint32_t n = 0; n < count; n += 2) {
    Vec f2[2], g2[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) f2[z] = v[z], g2[z] = w[z];
    if (n + 2 < count) load(n + 2);
    if (turned) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float f[V], g[V];
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = value_of<DT>(f2[z][k]), g[k] = value_of<DT>(g2[z][k]);
        rotate_unit<V>(f, g, c, s, half);
#pragma unroll
        for (int k = 0; k < V; ++k) f2[z][k] = (T)f[k], g2[z][k] = (T)g[k];
      }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (n + z >= count || h + (n + z) * step > last) continue;
      T* q = y + mode_offset(a.yh, h + (n + z) * step);
      store_chunk<NT>(q + i, f2[z]);
      if (two) store_chunk<NT>(q + j, g2[z]);
    }
  }
}

// Any strides and sizes: one pair of a head (or two elements past the rotated part) per lane (635 us for the 1 GiB
// above).
template <int DT>
__global__ void __launch_bounds__(256) k_rope(RopeArgs a) {
  using T = typename ElemOf<DT>::T;
  const uint64_t count = (uint64_t)a.heads * a.n * a.units;
  for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < count; at += (uint64_t)gridDim.x * 256) {
    const uint64_t row = at / a.units;
    const uint32_t u = (uint32_t)(at - row * a.units), t = (uint32_t)(row / a.heads), h = (uint32_t)(row % a.heads);
    const T* x = (const T*)a.x + mode_offset(a.xh, h) + mode_offset(a.xt, t);
    T* y = (T*)a.y + mode_offset(a.yh, h) + mode_offset(a.yt, t);
    const uint32_t half = (uint32_t)a.rot / 2;
    if (u >= half) {  // past the rotated part
      for (uint32_t e = (uint32_t)a.rot + 2 * (u - half), k = 0; k < 2 && e < (uint32_t)a.dim; ++e, ++k)
        y[(int64_t)e * a.yd] = x[(int64_t)e * a.xd];
      continue;
    }
    const uint32_t i = a.pairs == LR_PAIRS_HALF ? u : 2 * u, j = a.pairs == LR_PAIRS_HALF ? u + half : 2 * u + 1;
    float s, c;
    sincos_turn((uint64_t)a.positions[mode_offset(a.p, t)] * (uint64_t)a.turns[u], &s, &c);
    s *= a.magnitude * a.sign;
    c *= a.magnitude;
    const float v = value_of<DT>(x[(int64_t)i * a.xd]), w = value_of<DT>(x[(int64_t)j * a.xd]);
    y[(int64_t)i * a.yd] = (T)(v * c - w * s);
    y[(int64_t)j * a.yd] = (T)(w * c + v * s);
  }
}

template <int DT, int V>
static void launch_chunks(const RopeChunkArgs& a, double bytes, hipStream_t st) {
  const dim3 grid(a.grid.blocks_x, a.grid.blocks_y);
  if (bytes > kStreamBytes)
    hipLaunchKernelGGL((k_rope_chunks<DT, V, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_rope_chunks<DT, V, false>), grid, dim3(256), 0, st, a);
}

template <int DT>
static void launch_chunks_of(const RopeChunkArgs& a, int64_t v, double bytes, hipStream_t st) {
  if constexpr (DT != LR_F32) {
    if (v == 8) return launch_chunks<DT, 8>(a, bytes, st);
  }
  if (v == 4) return launch_chunks<DT, 4>(a, bytes, st);
  launch_chunks<DT, 2>(a, bytes, st);
}

static bool same_leaves(const Mode& a, const Mode& b) {
  if (a.n != b.n) return false;
  for (int i = 0; i < a.n; ++i)
    if (a.leaf[i].n != b.leaf[i].n || a.leaf[i].d != b.leaf[i].d) return false;
  return true;
}

int check_rotation(const lr_rotation* r, int64_t dim, int64_t n) {
  if (!r || !r->turns || (n > 0 && !r->positions)) return LR_ERR_INVALID;
  if (r->rot_dim < 2 || r->rot_dim > 1024 || r->rot_dim % 2 || r->rot_dim > dim) return LR_ERR_INVALID;
  if (r->pairs != LR_PAIRS_HALF && r->pairs != LR_PAIRS_INTERLEAVED) return LR_ERR_INVALID;
  return LR_OK;
}

}  // namespace lr

using namespace lr;

extern "C" {

int lr_rope_table(const lr_rope_params* p, int64_t* turns, double* magnitude) {
  if (!p || !turns || !magnitude) return LR_ERR_INVALID;
  const int rot = p->rot_dim;
  if (rot < 2 || rot > 1024 || rot % 2 || !(p->base > 1) || !std::isfinite(p->base)) return LR_ERR_INVALID;
  if (p->scaling < LR_ROPE_PLAIN || p->scaling > LR_ROPE_BANDS) return LR_ERR_INVALID;
  if (p->scaling != LR_ROPE_PLAIN && !(p->factor > 0 && std::isfinite(p->factor))) return LR_ERR_INVALID;
  const bool blended = p->scaling == LR_ROPE_PARTS || p->scaling == LR_ROPE_BANDS;
  if (blended && !(p->original_len > 0 && std::isfinite(p->original_len) && p->low > 0 && p->high > p->low &&
                   std::isfinite(p->high)))
    return LR_ERR_INVALID;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  long double base = p->base, factor = p->scaling == LR_ROPE_PLAIN ? 1.0L : (long double)p->factor;
  if (p->scaling == LR_ROPE_BASE && rot > 2) base *= powl(factor, (long double)rot / (rot - 2));
  if (!(base > 1) || !std::isfinite((double)base)) return LR_ERR_INVALID;
  long double from = 0, to = 0;  // LR_ROPE_PARTS: the ramp over the pair's index
  if (p->scaling == LR_ROPE_PARTS) {
    auto turning = [&](long double times) {
      return rot * logl((long double)p->original_len / (times * two_pi)) / (2 * logl(base));
    };
    from = std::max(floorl(turning(p->high)), 0.0L);
    to = std::min(ceill(turning(p->low)), (long double)rot - 1);
  }
  for (int i = 0; i < rot / 2; ++i) {
    long double w = powl(base, -2.0L * i / rot);
    if (p->scaling == LR_ROPE_LINEAR) w /= factor;
    if (blended) {
      const long double k = p->scaling == LR_ROPE_PARTS
                                ? 1 - (i - from) / std::max(to - from, 0.001L)
                                : ((long double)p->original_len * w / two_pi - p->low) / ((long double)p->high - p->low);
      const long double keep = std::min(std::max(k, 0.0L), 1.0L);
      w = w / factor * (1 - keep) + w * keep;
    }
    // the fraction of a turn, whole turns dropped: a turn is a turn
    long double t = w / two_pi;
    t -= floorl(t);
    const long double scaled = t * 18446744073709551616.0L + 0.5L;
    turns[i] = scaled >= 18446744073709551616.0L ? 0 : (int64_t)(uint64_t)scaled;
  }
  *magnitude = p->scaling == LR_ROPE_PARTS && p->factor > 1 ? 0.1 * std::log(p->factor) + 1 : 1.0;
  return LR_OK;
}

int lr_rope(const void* x, const lr_layout* Lx, int64_t x_capacity, void* y, const lr_layout* Ly, int64_t y_capacity,
            int32_t dtype, const lr_rotation* r, const lr_layout* Lp, int64_t p_capacity, int64_t n, uint32_t flags,
            void* stream) {
  if (!x || !y || (flags & ~LR_ROPE_BACKWARD)) return LR_ERR_INVALID;
  if (!is_model_type(dtype)) return LR_ERR_TYPE;
  int rc = check_tensor(Lx, 3, x_capacity, false);
  if (rc || (rc = check_tensor(Ly, 3, y_capacity, true))) return rc;
  const Mode xd = mode_of(*Lx, 0), yd = mode_of(*Ly, 0), xh = mode_of(*Lx, 1), yh = mode_of(*Ly, 1);
  const Mode xt = mode_of(*Lx, 2), yt = mode_of(*Ly, 2);
  if (xd.size != yd.size || xh.size != yh.size || xt.size != yt.size) return LR_ERR_SIZE_MISMATCH;
  if ((rc = check_rotation(r, xd.size, n))) return rc;
  if (n < 0) return LR_ERR_INVALID;
  if (n > xt.size) return LR_ERR_BOUNDS;
  Mode p{0, {}, 1};
  if (Lp) {
    if ((rc = check_tensor(Lp, Lp->nmodes, p_capacity, false))) return rc;
    lr_layout flat = *Lp;  // one mode: the token index runs over all of it
    flat.nmodes = 1;
    flat.mode_end[0] = flat.nleaves;
    p = mode_of(flat, 0);
    if (p.size != xt.size) return LR_ERR_SIZE_MISMATCH;
    if (p.n > kMaxModeLeaves) return LR_ERR_INVALID;
  } else {
    if (p_capacity < n) return LR_ERR_BOUNDS;
    p.size = xt.size;
    if (xt.size > 1) p.leaf[p.n++] = Leaf{xt.size, 1};
  }
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  if (one_leaf(xd, &a.xd) || one_leaf(yd, &a.yd)) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype);
  // in place: each element is read and written by the same lane
  const bool in_place = x == y && same_leaves(xd, yd) && same_leaves(xh, yh) && same_leaves(xt, yt);
  if (!in_place && overlap(x, x_capacity * e, y, y_capacity * e)) return LR_ERR_OVERLAP;
  if (overlap(r->positions, p_capacity * 8, y, y_capacity * e) || overlap(r->turns, r->rot_dim * 4, y, y_capacity * e))
    return LR_ERR_OVERLAP;
  if (n == 0) return LR_OK;
  a.x = x;
  a.y = y;
  a.turns = r->turns;
  a.positions = r->positions;
  a.xh = mode_arg(xh);
  a.yh = mode_arg(yh);
  a.xt = mode_arg(xt);
  a.yt = mode_arg(yt);
  a.p = mode_arg(p);
  a.dim = (int32_t)xd.size;
  a.rot = r->rot_dim;
  a.pairs = r->pairs;
  a.heads = (uint32_t)xh.size;
  a.n = (uint32_t)n;
  a.magnitude = r->magnitude;
  a.sign = flags & LR_ROPE_BACKWARD ? -1.f : 1.f;
  const hipStream_t st = (hipStream_t)stream;
  // the widest chunks that halves, rest and rows are whole numbers of
  int64_t v = 16 / e;
  while (v > 1 && (a.rot / 2 % v || (a.dim - a.rot) % v || !rows_aligned(*Lx, x, e, v) || !rows_aligned(*Ly, y, e, v)))
    v /= 2;
  const double bytes = 2.0 * (double)a.heads * (double)n * a.dim * (double)e;
  RopeChunkArgs k;
  bool chunked = v > 1 && mode_pair(xh, &k.xh) && mode_pair(yh, &k.yh) && mode_pair(xt, &k.xt) &&
                 mode_pair(yt, &k.yt) && mode_pair(p, &k.p);
  if (chunked) {
    k.un = units_of(a.rot, a.dim, (int32_t)v);
    chunked = k.un.count <= 256;
  }
  if (chunked) {
    // four heads side by side: runs of four rows on the side where heads are neighbours, while the other lanes
    // are neighbouring tokens for the side where those are (1, 2, 4, 8, 32 took 213, 194, 185, 197, 272 us for a
    // head split of 512 MiB)
    k.grid = row_grid((uint32_t)k.un.count, a.heads, a.n, 1, 4);
    chunked = row_grid_fits(k.grid);
    k.x = x;
    k.y = y;
    k.turns = r->turns;
    k.positions = r->positions;
    k.heads = a.heads;
    k.n = a.n;
    k.pairs = r->pairs;
    k.magnitude = a.magnitude;
    k.sign = a.sign;
  }
  if (chunked && dtype == LR_F32) {
    launch_chunks_of<LR_F32>(k, v, bytes, st);
  } else if (chunked && dtype == LR_F16) {
    launch_chunks_of<LR_F16>(k, v, bytes, st);
  } else if (chunked) {
    launch_chunks_of<LR_BF16>(k, v, bytes, st);
  } else {
    a.units = (uint32_t)(a.rot / 2 + (a.dim - a.rot + 1) / 2);
    const double lanes = (double)a.heads * (double)n * a.units;
    const int64_t groups = lanes > 1e9 ? 1 << 22 : ((int64_t)lanes + 255) / 256;
    if (dtype == LR_F32)
      hipLaunchKernelGGL(k_rope<LR_F32>, dim3((unsigned)groups), dim3(256), 0, st, a);
    else if (dtype == LR_F16)
      hipLaunchKernelGGL(k_rope<LR_F16>, dim3((unsigned)groups), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL(k_rope<LR_BF16>, dim3((unsigned)groups), dim3(256), 0, st, a);
  }
  return check_op_launch();
}

}  // extern "C"
