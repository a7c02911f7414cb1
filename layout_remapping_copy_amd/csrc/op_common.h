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

// sin and cos of a fraction of a turn given in 64 bits.  The upper 32 bits are
// reduced to a quadrant and a rest within an eighth of a turn either way; the rest's
// Taylor sums to x^9 and x^10 are off by under 2e-9, below a half step of fp32.
__device__ __forceinline__ void sincos_turn(uint64_t t, float* sin_out, float* cos_out) {
  const uint32_t hi = (uint32_t)(t >> 32);
  const uint32_t q = (hi + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(hi - (q << 30)) * 1.4629180792671596e-09f;  // 2 pi / 2^32
  const float z = x * x;
  const float s = x + x * z * (-1.f / 6 + z * (1.f / 120 + z * (-1.f / 5040 + z * (1.f / 362880))));
  const float c = 1.f + z * (-0.5f + z * (1.f / 24 + z * (-1.f / 720 + z * (1.f / 40320 + z * (-1.f / 3628800)))));
  const float a = q & 1 ? c : s, b = q & 1 ? s : c;
  *sin_out = q & 2 ? -a : a;
  *cos_out = (q + 1) & 2 ? -b : b;
}

}  // namespace lr
