// Shared by the attention operators (rope.hip, kv_cache.hip, paged_attention.hip):
// host checks of their tensors, and the device side of element types, token and head
// modes, and the angle of a rotation.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "lr_internal.h"

namespace lr {

// ------------------------------------------------------------------ host checks

constexpr int kMaxModeLeaves = LR_MAX_LEAVES - 2;  // a tensor has at least three modes

// One top-level mode, coalesced: leaves of extent 1 dropped, neighbours merged.
struct Mode {
  int n;
  Leaf leaf[LR_MAX_LEAVES];
  int64_t size;
};

inline Mode mode_of(const lr_layout& L, int mode) {
  Mode m{0, {}, 1};
  for (int i = mode ? L.mode_end[mode - 1] : 0; i < L.mode_end[mode]; ++i) {
    m.size *= L.shape[i];
    if (L.shape[i] == 1) continue;
    if (m.n && L.stride[i] == m.leaf[m.n - 1].n * m.leaf[m.n - 1].d)
      m.leaf[m.n - 1].n *= L.shape[i];
    else
      m.leaf[m.n++] = Leaf{L.shape[i], L.stride[i]};
  }
  return m;
}

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;

// A tensor's layout: valid, unswizzled, `modes` top-level modes, extents below 2^31,
// inside a buffer of `capacity` elements; an output's has to be injective too.
inline int check_tensor(const lr_layout* L, int modes, int64_t capacity, bool output) {
  if (!L) return LR_ERR_INVALID;
  if (int rc = validate(L)) return rc;
  if (L->swz_b > 0) return LR_ERR_SWIZZLE;
  if (L->nmodes != modes) return LR_ERR_INVALID;
  for (int m = 0; m < modes; ++m)
    if (mode_of(*L, m).size > kMaxCount) return LR_ERR_OVERFLOW;
  if (cosize_bound(L) > capacity) return LR_ERR_BOUNDS;
  if (output && !injective(L)) return LR_ERR_ALIAS;
  return LR_OK;
}

// The stride of a mode that has to be one leaf (0 when its extent is 1).
inline int one_leaf(const Mode& m, int64_t* stride) {
  if (m.n > 1) return LR_ERR_INVALID;
  *stride = m.n ? m.leaf[0].d : 0;
  return LR_OK;
}

inline int dtype_bytes(int32_t t) {
  return t == LR_F32 ? 4 : t == LR_F16 || t == LR_BF16 ? 2 : t == LR_E4M3 || t == LR_INT8 ? 1 : 0;
}
inline bool is_model_type(int32_t t) { return t == LR_F32 || t == LR_F16 || t == LR_BF16; }
inline bool is_quantised(int32_t t) { return t == LR_E4M3 || t == LR_INT8; }

// Whether the storage of two buffers overlaps.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// Whether rows of a tensor can be moved `v` elements at a time: the head dimension
// (mode 0) contiguous, every other stride and the buffer a multiple of v elements.
inline bool rows_aligned(const lr_layout& L, const void* p, int64_t elem, int64_t v) {
  const Mode d = mode_of(L, 0);
  if (d.n && (d.n != 1 || d.leaf[0].d != 1)) return false;
  if ((uintptr_t)p % (uintptr_t)(elem * v)) return false;
  for (int m = 1; m < L.nmodes; ++m) {
    const Mode o = mode_of(L, m);
    for (int i = 0; i < o.n; ++i)
      if (o.leaf[i].d % v) return false;
  }
  return true;
}

inline int check_op_launch() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return LR_OK;
  set_hip_error(hipGetErrorString(e));
  return LR_ERR_HIP;
}

// ------------------------------------------------------------------ modes on the device

struct ModeArg {
  int32_t n;
  uint32_t ext[kMaxModeLeaves];
  FastDiv fd[kMaxModeLeaves];
  int64_t stride[kMaxModeLeaves];
};

inline ModeArg mode_arg(const Mode& m) {
  ModeArg a;
  std::memset(&a, 0, sizeof(a));
  a.n = m.n;
  for (int i = 0; i < m.n; ++i) {
    a.ext[i] = (uint32_t)m.leaf[i].n;
    a.fd[i] = make_fastdiv((uint32_t)m.leaf[i].n);
    a.stride[i] = m.leaf[i].d;
  }
  return a;
}

__device__ __forceinline__ uint32_t op_div(uint32_t x, FastDiv f) { return f.m ? (__umulhi(x, f.m) >> f.s) : x; }

// Offset of index i in a mode (colexicographic; the last leaf takes what is left).
__device__ __forceinline__ int64_t mode_offset(const ModeArg& m, uint32_t i) {
  int64_t off = 0;
  for (int k = 0; k + 1 < m.n; ++k) {
    const uint32_t q = op_div(i, m.fd[k]);
    off += (int64_t)(i - q * m.ext[k]) * m.stride[k];
    i = q;
  }
  return m.n ? off + (int64_t)i * m.stride[m.n - 1] : 0;
}

// A mode of at most two leaves, without loops and in few bytes: arguments come from host memory, and a kernel
// of a few microseconds waits for each line of them that it reads on its way.
struct ModePair {
  FastDiv fd;  // by the first leaf's extent, at least 2
  uint32_t ext;
  int64_t stride[2];
};
inline bool mode_pair(const Mode& m, ModePair* a) {
  if (m.n > 2) return false;
  a->ext = m.n == 2 ? (uint32_t)m.leaf[0].n : (uint32_t)kMaxCount;  // one leaf: never reached by an index
  a->fd = make_fastdiv(a->ext);
  a->stride[0] = m.n ? m.leaf[0].d : 0;
  a->stride[1] = m.n == 2 ? m.leaf[1].d : 0;
  return true;
}
__device__ __forceinline__ int64_t mode_offset(const ModePair& m, uint32_t i) {
  const uint32_t q = __umulhi(i, m.fd.m) >> m.fd.s;
  return (int64_t)(i - q * m.ext) * m.stride[0] + (int64_t)q * m.stride[1];
}

// ------------------------------------------------------------------ element types

template <int DT> struct ElemOf;
template <> struct ElemOf<LR_F32> { using T = float; };
template <> struct ElemOf<LR_F16> { using T = _Float16; };
template <> struct ElemOf<LR_BF16> { using T = __bf16; };
template <> struct ElemOf<LR_E4M3> { using T = uint8_t; };
template <> struct ElemOf<LR_INT8> { using T = int8_t; };

// The number an element or a code stands for (a code's scale aside).
template <int DT>
__device__ __forceinline__ float value_of(typename ElemOf<DT>::T x) {
  if constexpr (DT == LR_E4M3)
    return __builtin_amdgcn_cvt_f32_fp8((int)x, 0);
  else
    return (float)x;
}

// ------------------------------------------------------------------ angles

// sin and cos of a fraction of a turn given in 64 bits, as a signed lower half and an upper one.  The upper half is
// reduced to a quadrant and a rest within an eighth of a turn either way, the lower one is joined to the rest in one
// rounding, so that small angles have all their bits too.  The rest's Taylor sums to x^9 and x^10 are off by under
// 2e-9, below a half step of fp32.  With the roundings of the rest and of the sums, sin and cos of 26 million random
// angles are off by up to 1.7 * 2^-24 (0.34 root mean square; their last rounding alone is up to 0.5), and sin of a
// small angle by up to 3.1 * 2^-24 of itself.
__device__ __forceinline__ void sincos_turn(uint64_t t, float* sin_out, float* cos_out) {
  const uint32_t hi = (uint32_t)(t >> 32) + ((uint32_t)t >> 31);
  const uint32_t q = (hi + 0x20000000u) >> 30;
  constexpr float kAngle = 1.4629180792671596e-09f;  // 2 pi / 2^32
  const float low = (float)(int32_t)(uint32_t)t * (kAngle * 0x1p-32f);
  const float x = __builtin_fmaf((float)(int32_t)(hi - (q << 30)), kAngle, low);
  const float z = x * x;
  const float s = x + x * z * (-1.f / 6 + z * (1.f / 120 + z * (-1.f / 5040 + z * (1.f / 362880))));
  const float c = 1.f + z * (-0.5f + z * (1.f / 24 + z * (-1.f / 720 + z * (1.f / 40320 + z * (-1.f / 3628800)))));
  const float a = q & 1 ? c : s, b = q & 1 ? s : c;
  *sin_out = q & 2 ? -a : a;
  *cos_out = (q + 1) & 2 ? -b : b;
}

// ------------------------------------------------------------------ rows in chunks

// A row of `dim` elements, the first `rot` of them rotated, as units of two chunks of V elements each: a
// rotated unit has the chunks that pairs of the half layout lie in (i and i + rot/2), a unit past them two
// chunks that are as far apart, so that neighbouring lanes' chunks are neighbours in memory.
struct Units {
  int32_t rot, dim, turned, rest;  // turned: rotated units; rest: distance of the two chunks past them
  int32_t count;
};
inline Units units_of(int32_t rot, int32_t dim, int32_t V) {
  Units u{rot, dim, rot / (2 * V), 0, 0};
  const int32_t chunks = (dim - rot) / V;
  u.rest = (chunks + 1) / 2 * V;
  u.count = u.turned + (chunks + 1) / 2;
  return u;
}
// First elements of unit u's chunks; the second is past the row's end when there is none.
__device__ __forceinline__ void chunks_of(const Units& n, uint32_t u, uint32_t V, uint32_t* i, uint32_t* j) {
  const bool turned = u < (uint32_t)n.turned;
  *i = turned ? u * V : n.rot + (u - n.turned) * V;
  *j = *i + (turned ? n.rot / 2 : n.rest);
}

// V elements of type T, moved at once.
template <class T, int V> struct Chunk {
  typedef T Vec __attribute__((ext_vector_type(V)));
};
template <bool NT, class Vec> __device__ __forceinline__ Vec load_chunk(const void* p) {
  return NT ? __builtin_nontemporal_load((const Vec*)p) : *(const Vec*)p;
}
template <bool NT, class Vec> __device__ __forceinline__ void store_chunk(void* p, Vec x) {
  if (NT)
    __builtin_nontemporal_store(x, (Vec*)p);
  else
    *(Vec*)p = x;
}

// Work beyond the 256 MiB of the memory-side cache streams past the caches: reads reach 7.2 TB/s instead
// of 6.3, and what is written would not be found there anyway (131072 tokens read back: 146 us streaming, 200
// with plain loads).  Below, what was just written and what is read next are there: 39 MB of gradient take 9.1 us
// with plain accesses and 14.4 with streaming ones when the caches hold them (17 either way when not).
constexpr double kStreamBytes = 256.0 * (1 << 20);

// Positions on several axes: pair i turns by the position on axis[i], whose positions lie `stride` after the axis before.
constexpr int kMaxAxes = 4;
struct AxesArg {
  const int32_t* axis;  // of each pair; null for one axis
  int64_t stride;
  int32_t axes;
};
// A token's positions on all axes, read side by side: reading the one that a pair asks for would wait for its axis first.
struct AxisPositions {
  int64_t p0, p1, p2, p3;  // no array: one that a lane's own axis indexes would be kept in shared memory
  // Of the first axis for a pair whose axis is none.  By masks: a choice of four values becomes branches, in which
  // the lanes of each axis take turns and the loads after them wait (3069 x 16 x 80 fp32: 21.5 us).
  __device__ __forceinline__ int64_t of(int32_t axis) const {
    const int64_t m1 = -(int64_t)(axis == 1), m2 = -(int64_t)(axis == 2), m3 = -(int64_t)(axis == 3);
    return (p0 & ~(m1 | m2 | m3)) | (p1 & m1) | (p2 & m2) | (p3 & m3);
  }
};
__device__ __forceinline__ AxisPositions axis_positions(const int64_t* first, const AxesArg& x) {
  return AxisPositions{first[0], first[x.axes > 1 ? x.stride : 0], first[x.axes > 2 ? 2 * x.stride : 0],
                       first[x.axes > 3 ? 3 * x.stride : 0]};
}

// cos and sin of the angles of one unit's V pairs: pair k of a half layout is element k of both chunks, pairs
// of an interleaved one lie inside the first chunk, then the second.  `position`: the token's first.
template <int V, bool AXES>
__device__ __forceinline__ void angles_of(const int64_t* turns, const int64_t* position, const AxesArg& x, uint32_t u,
                                          int32_t rot, bool half, float magnitude, float sign, float* c, float* s) {
  AxisPositions p;
  int64_t turn[V], one = 0;
  int32_t axis[V];
  auto pair_of = [&](int k) { return half ? u * V + k : u * (V / 2) + (k < V / 2 ? k : rot / 4 + k - V / 2); };
  if constexpr (AXES) {
    p = axis_positions(position, x);
#pragma unroll
    for (int k = 0; k < V; ++k) axis[k] = x.axis[pair_of(k)];
  } else {
    one = *position;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) turn[k] = turns[pair_of(k)];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if constexpr (AXES) one = p.of(axis[k]);
    sincos_turn((uint64_t)one * (uint64_t)turn[k], &s[k], &c[k]);
    s[k] *= magnitude * sign;
    c[k] *= magnitude;
  }
}
template <int V>
__device__ __forceinline__ void rotate_unit(float* a, float* b, const float* c, const float* s, bool half) {
  if (half) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float v = a[k], w = b[k];
      a[k] = v * c[k] - w * s[k];
      b[k] = w * c[k] + v * s[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float* x = k < V / 2 ? a + 2 * k : b + 2 * (k - V / 2);
      const float v = x[0], w = x[1];
      x[0] = v * c[k] - w * s[k];
      x[1] = w * c[k] + v * s[k];
    }
  }
}

// How a workgroup of 256 lanes covers rows: `lanes` a row (2^row_shift where lanes of a row reduce among each
// other), 2^head_shift heads next to each other, the rest tokens; a lane then takes `per_lane` heads,
// 2^head_shift apart, so that what depends on the token alone is computed once for them.
struct RowGrid {
  uint32_t lanes, head_shift, tokens, per_lane;
  FastDiv fd_lanes;
  uint32_t blocks_x, blocks_y;  // token blocks, head blocks
};
inline RowGrid row_grid(uint32_t lanes, uint32_t heads, uint32_t n, uint32_t sides, uint32_t side_by_side) {
  RowGrid g;
  g.lanes = lanes;
  g.fd_lanes = make_fastdiv(lanes);
  g.head_shift = 0;
  while (2u << g.head_shift <= std::min(heads, side_by_side) && lanes << g.head_shift <= 64) ++g.head_shift;
  g.tokens = (256 / lanes) >> g.head_shift;
  if (!g.tokens) g.tokens = 1, g.head_shift = 0;
  g.blocks_x = (n + g.tokens - 1) / g.tokens;
  const uint32_t steps = (heads + (1u << g.head_shift) - 1) >> g.head_shift;
  // several heads a lane once there are 8 workgroups a CU without
  const uint64_t all = (uint64_t)g.blocks_x * steps * sides;
  g.per_lane = (uint32_t)std::min<uint64_t>({steps, 8, std::max<uint64_t>(all / 2048, 1)});
  g.blocks_y = (steps + g.per_lane - 1) / g.per_lane;
  return g;
}
// Within the launch's limits: 2^32 lanes along x, 65535 workgroups along y.
inline bool row_grid_fits(const RowGrid& g) { return g.blocks_x < 1u << 24 && g.blocks_y <= 65535; }
// Lane's unit, first head and token; false for a lane without work.
__device__ __forceinline__ bool row_lane(const RowGrid& g, uint32_t lane, uint32_t* u, uint32_t* h, uint32_t* t) {
  const uint32_t row = op_div(lane, g.fd_lanes);
  *u = lane - row * g.lanes;
  *h = row & ((1u << g.head_shift) - 1);
  *t = row >> g.head_shift;
  return *t < g.tokens;
}

}  // namespace lr
