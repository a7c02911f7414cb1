// The paged cache of keys and values: lr_cache_validate, lr_cache_write, lr_cache_read.
#include "op_common.h"

namespace lr {

int check_rotation(const lr_rotation* r, int64_t dim, int64_t n);

constexpr int kCacheDim = 512;  // head_dim at most

struct CacheSide {  // keys or values
  void* cache;
  float* scale;
  void* rows;                 // the tensor written from or read to
  ModeArg rh, rt;             // its heads and tokens
  int64_t rd;                 // its head-dimension stride
  int64_t cd, ch, cs, cp;     // cache strides: head dimension, heads, slots, pages
  int32_t dim, rot;           // rot: rotated elements, 0 for none
};

struct CacheArgs {
  CacheSide side[2];
  int64_t sh, ss, sp;  // scale strides
  const int64_t* slots;
  const int64_t* turns;
  const int64_t* positions;
  float magnitude;
  int32_t pairs;
  int64_t cache_slots;
  uint32_t page_size, heads, n;
};

// The code nearest x / scale, exactly: the fp32 quotient's remainder says which side of
// the quotient the true value lies on, and a quotient that could be a tie (an even last
// bit) is moved one step towards it.  The remainder of x and scale has to be a number of
// fp32: rows of small numbers are scaled up by the caller.
template <int DT>
__device__ __forceinline__ typename ElemOf<DT>::T code_of(float x, float scale) {
  constexpr float top = DT == LR_E4M3 ? 448.f : 127.f;
  if (DT == LR_INT8 && x != x) return 0;
  const float inv = 1.f / scale;  // finite
  const float q0 = x * inv;
  float q = __builtin_fmaf(__builtin_fmaf(-q0, scale, x), inv, q0);
  const float rest = __builtin_fmaf(-q, scale, x);
  const uint32_t bits = __float_as_uint(q);
  if (!(bits & 1) && q != 0 && rest != 0 && __builtin_fabsf(q) < 2 * top)
    q = __uint_as_float((rest > 0) == (q > 0) ? bits + 1 : bits - 1);
  if (__builtin_fabsf(x) == __builtin_inff()) q = x;
  if constexpr (DT == LR_E4M3) {
    if (q == q) q = __builtin_fminf(__builtin_fmaxf(q, -top), top);
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xff);
  } else {
    return (int8_t)(int)__builtin_rintf(__builtin_fminf(__builtin_fmaxf(q, -top), top));
  }
}

// The chunked kernels' arguments: both sides' rows in chunks of V elements.
struct ChunkSide {
  void* cache;
  float* scale;
  void* rows;
  ModePair rt;
  int64_t rh, ch, cs, cp;
  Units un;
};
struct ChunkArgs {
  ChunkSide side[2];
  RowGrid grid;
  const int64_t* slots;
  const int64_t* turns;
  const int64_t* positions;
  int64_t sh, ss, sp;
  int64_t cache_slots;
  FastDiv fd_page;
  uint32_t page_size, heads, n;
  float magnitude;
  int32_t pairs;
};

// Page and slot of a token's place; false for none.
__device__ __forceinline__ bool place_of(const ChunkArgs& a, int64_t slot, uint32_t* page, uint32_t* in) {
  const bool held = (uint64_t)slot < (uint64_t)a.cache_slots;
  const uint32_t s = held ? (uint32_t)slot : 0;
  *page = op_div(s, a.fd_page);
  *in = s - *page * a.page_size;
  return held;
}

// V numbers, none infinite, as codes, exactly, without a division each.  p = x * (1 / scale), the reciprocal off by a
// step at most, is within 3 steps of fp32 of the quotient.  A candidate T next to p is taken such that no tie but T
// itself can lie between T and the quotient; the side of T that the quotient is on is the sign of x - T scale, which
// one fma has right (T has 21 bits at most), and T moved a little to that side rounds as the quotient does.
// Looking at ties only where p is near one is no cheaper: numbers of 16 bits often are simple parts of their row's
// largest, which are ties or next to them (16389 tokens of fp16 stored: 26.9 us that way, 22.1 us this way).
template <int DT, int CT, int V>
__device__ __forceinline__ void codes_of(const float* v, float scale, float inv, uint32_t* code) {
  if constexpr (CT == LR_E4M3) {
    // T: p to a multiple of 8 steps.  Ties and codes are multiples of 2^19 steps.
    float q[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int32_t t = (int32_t)((__float_as_uint(v[k] * inv) + 4) & ~7u);
      const float r = __builtin_fmaf(-__builtin_fabsf(__int_as_float(t)), scale, __builtin_fabsf(v[k]));
      // the sign of r, whose bits have the order of integers (a zero here is +0), in one instruction
      int32_t side;
      asm("v_med3_i32 %0, %1, -1, 1" : "=v"(side) : "v"(r));
      q[k] = __int_as_float(t + side);
      // a NaN with ones at its end would be carried out of the NaN; one of 16 bits has zeros there
      if (DT == LR_F32) q[k] = v[k] == v[k] ? q[k] : v[k];
    }
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[k], q[k + 1], 0, false);
      code[k / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[k + 2], q[k + 3], lo, true);
    }
  } else {
    // T: the half between the whole numbers around p.  The sum with 1.5 * 2^23 is rounded to a whole number, to
    // the even one of two as near, and has it as its last bits.
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = v[k + e], t = __builtin_floorf(x * inv) + 0.5f;
        const float r = __builtin_fmaf(-t, scale, x) * 0x1p100f;
        const float q = t + __builtin_amdgcn_fmed3f(r, -0.25f, 0.25f);
        // a NaN of 16 bits has zeros there
        c[e] = DT == LR_F32 && x != x ? 0 : __float_as_uint(q + 12582912.f);
      }
      const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400);
      code[k / 4] = lo | __builtin_amdgcn_perm(c[3], c[2], 0x04000c0c);
    }
  }
}

// max(x, |y|, |z|) in one instruction, of which fmaxf would make four; NaN if one of them is.  (v_max3_f32 passes
// over a quiet NaN, but a signalling one, as bf16 or fp32 in memory may be, makes its result NaN, and the next
// one passes over that with all that went in before.)
__device__ __forceinline__ float max_abs(float x, float y, float z) {
  float r;
  asm("v_maximum3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}

// The largest x >= 0 (as its bits, which have the same order, NaN above all) over the `lanes` lanes, a power of two,
// of a row: within 16 lanes by exchanges that are part of the instruction (neighbours, pairs, mirrors of 8 and 16).
__device__ __forceinline__ float row_max(float value, uint32_t lanes) {
  uint32_t x = __float_as_uint(value);
  if (lanes > 1) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xb1, 0xf, 0xf, true));
  if (lanes > 2) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4e, 0xf, 0xf, true));
  if (lanes > 4) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true));
  if (lanes > 8) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, true));
  if (lanes > 16) x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  if (lanes > 32) x = max(x, (uint32_t)__shfl_xor((int)x, 32));
  return __uint_as_float(x);
}

// amax / Q, rounded to nearest: with the rounded reciprocal of Q, one step on the remainder is exact (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
template <int CT> __device__ __forceinline__ float scale_of(float amax) {
  constexpr float kTop = CT == LR_E4M3 ? 448.f : 127.f, kInv = 1.f / kTop;
  const float q = amax * kInv;
  return fmaxf(__builtin_fmaf(__builtin_fmaf(-kTop, q, amax), kInv, q), 0x1p-126f);
}
// 16389 tokens of 8 heads of 128 fp16, rotated and stored in e4m3 (102 MB moved): 20 us, as long as
// a copy of the same bytes; the vector units are busy 96 % of it.  65536 tokens: 79 us (5.2 TB/s); the same many from
// fp32, not rotated, 131 us, and of bf16 into a bf16 cache, rotated, 102 us (5.2 and 5.3 TB/s).
//
// Rows in chunks: a lane has one unit of a token's rows, its angles in registers for `per_lane` heads; the
// lanes of a row (a power of two next to each other) find its largest value by exchange.  A row that holds an
// infinity or a NaN is told by that value, and is done again with the care that it needs.
template <int DT, int CT, int V, bool NT>
__global__ void __launch_bounds__(256) k_cache_write_chunks(ChunkArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  using Vec = typename Chunk<T, V>::Vec;
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  const ChunkSide& sd = a.side[blockIdx.z];
  uint32_t u, h, t;
  row_lane(a.grid, threadIdx.x, &u, &h, &t);  // lanes of a row are all there, for the exchange
  const uint64_t token = (uint64_t)blockIdx.x * a.grid.tokens + t;
  const bool there = token < a.n;
  t = there ? (uint32_t)token : a.n - 1;
  h += blockIdx.y * a.grid.per_lane << a.grid.head_shift;
  uint32_t i, j, page, in;
  chunks_of(sd.un, u, V, &i, &j);
  const bool one = u < (uint32_t)sd.un.count, two = one && j < (uint32_t)sd.un.dim, turned = u < (uint32_t)sd.un.turned;
  const bool half = a.pairs == LR_PAIRS_HALF;
  const bool ragged = sd.un.count * 2 * V != sd.un.dim || (uint32_t)sd.un.count != a.grid.lanes;
  const bool held = place_of(a, a.slots[t], &page, &in) && there;
  const T* x = (const T*)sd.rows + mode_offset(sd.rt, t);
  C* y = (C*)sd.cache + (int64_t)page * sd.cp + (int64_t)in * sd.cs;
  float* scales = sd.scale + (int64_t)page * a.sp + (int64_t)in * a.ss;
  const uint32_t step = 1u << a.grid.head_shift, last = a.heads - 1;
  const uint32_t left = (a.heads - (blockIdx.y * a.grid.per_lane << a.grid.head_shift) + step - 1) >> a.grid.head_shift;
  const uint32_t count = min(a.grid.per_lane, left);  // the same for all lanes
  Vec v, w, vn, wn;
  auto load = [&](uint32_t head) {  // a lane past its row's end reads the row's first chunk, and stores nothing
    const T* p = x + (int64_t)min(head, last) * sd.rh;
    vn = load_chunk<NT, Vec>(p + (one ? i : 0));
    wn = load_chunk<NT, Vec>(p + (two ? j : 0));
  };
  load(h);
  float c[V], s[V];
  if (turned) angles_of<V>(a.turns, a.positions[t], u, sd.un.rot, half, a.magnitude, 1.f, c, s);
  for (uint32_t n = 0; n < count; ++n, h += step) {
    const bool mine = held && h < a.heads;
    v = vn, w = wn;
    if (n + 1 < count) load(h + step);
    C* q = y + (int64_t)h * sd.ch;
    if constexpr (!kQuant) {
      if (turned) {
        float f[V], g[V];
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = value_of<DT>(v[k]), g[k] = value_of<DT>(w[k]);
        rotate_unit<V>(f, g, c, s, half);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = (T)f[k], w[k] = (T)g[k];
      }
      if (mine && one) store_chunk<NT>(q + i, v);
      if (mine && two) store_chunk<NT>(q + j, w);
    } else {
      float f[V], g[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = value_of<DT>(v[k]), g[k] = value_of<DT>(w[k]);
      if (turned) rotate_unit<V>(f, g, c, s, half);
      if (ragged) {  // lanes past their row's end read something else
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = one ? f[k] : 0.f, g[k] = two ? g[k] : 0.f;
      }
      auto largest = [&](float bound) {
        float z = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float x = __builtin_fabsf(f[k]), y = __builtin_fabsf(g[k]);
          z = fmaxf(z, x < bound ? x : 0.f);
          z = fmaxf(z, y < bound ? y : 0.f);
        }
        return row_max(z, a.grid.lanes);
      };
      float amax = 0;
#pragma unroll
      for (int k = 0; k < V; ++k) amax = max_abs(amax, f[k], g[k]);
      amax = row_max(amax, a.grid.lanes);
      const bool special = !(amax < __builtin_inff());  // an infinity or a NaN
      if (__any(special)) amax = largest(__builtin_inff());
      const float scale = scale_of<CT>(amax);
      float unit = scale;
      if (__any(special || amax < 0x1p-90f)) {
        // infinities become the largest code; rows so small that a product's last bits were lost are scaled up
        const float up = amax < 0x1p-90f ? 0x1p64f : 1.f;
        unit = scale * up;
        const float most = unit * (CT == LR_E4M3 ? 448.f : 127.f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          f[k] = __builtin_fabsf(f[k]) == __builtin_inff() ? __builtin_copysignf(most, f[k]) : f[k] * up;
          g[k] = __builtin_fabsf(g[k]) == __builtin_inff() ? __builtin_copysignf(most, g[k]) : g[k] * up;
        }
      }
      const float inv = __builtin_amdgcn_rcpf(unit);
      uint32_t cv[V / 4], cw[V / 4];
      codes_of<DT, CT, V>(f, unit, inv, cv);
      codes_of<DT, CT, V>(g, unit, inv, cw);
      using CVec = typename Chunk<uint32_t, V / 4>::Vec;
      if (mine && one) store_chunk<NT>(q + i, *(const CVec*)cv);
      if (mine && two) store_chunk<NT>(q + j, *(const CVec*)cw);
      if (mine && u == 0) scales[(int64_t)h * a.sh] = scale;
    }
  }
}

// Rows in chunks, the other way: codes times their scale, or the elements as they are.  131072 tokens of 8 heads of
// 128 e4m3 to bf16 (814 MB moved): 146 us, 5.6 TB/s, bound by memory (119 us at a plain copy's rate; the codes come
// in runs of 512 bytes).  From a bf16 cache (1.07 GB): 184 us, 5.8 TB/s.  Four heads in flight instead of two: 159 us.
template <int DT, int CT, int V, bool NT>
__global__ void __launch_bounds__(256) k_cache_read_chunks(ChunkArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  using Vec = typename Chunk<T, V>::Vec;
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  using CVec = typename Chunk<C, V>::Vec;
  const ChunkSide& sd = a.side[blockIdx.z];
  uint32_t u, h, t, page, in, i, j;
  if (!row_lane(a.grid, threadIdx.x, &u, &h, &t) || u >= (uint32_t)sd.un.count) return;
  const uint64_t token = (uint64_t)blockIdx.x * a.grid.tokens + t;
  if (token >= a.n) return;
  t = (uint32_t)token;
  h += blockIdx.y * a.grid.per_lane << a.grid.head_shift;
  chunks_of(sd.un, u, V, &i, &j);
  const bool two = j < (uint32_t)sd.un.dim, held = place_of(a, a.slots[t], &page, &in);
  const C* x = (const C*)sd.cache + (int64_t)page * sd.cp + (int64_t)in * sd.cs;
  const float* scales = sd.scale + (int64_t)page * a.sp + (int64_t)in * a.ss;
  T* y = (T*)sd.rows + mode_offset(sd.rt, t);
  const uint32_t step = 1u << a.grid.head_shift, last = a.heads - 1;
  const uint32_t left = (a.heads - (blockIdx.y * a.grid.per_lane << a.grid.head_shift) + step - 1) >> a.grid.head_shift;
  const uint32_t count = min(a.grid.per_lane, left);  // the same for all lanes
  auto made = [&](CVec v, float scale) -> Vec {
    Vec r;
    if constexpr (CT == LR_E4M3) {
      const uint32_t* d = (const uint32_t*)&v;
      typedef float F2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const F2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(d[k / 4], false);
        const F2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(d[k / 4], true);
        r[k] = (T)(lo[0] * scale), r[k + 1] = (T)(lo[1] * scale);
        r[k + 2] = (T)(hi[0] * scale), r[k + 3] = (T)(hi[1] * scale);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if constexpr (kQuant)
          r[k] = (T)(value_of<CT>(v[k]) * scale);
        else
          r[k] = v[k];
    }
    return held ? r : Vec{};
  };
  CVec v[2], w[2];
  float sc[2] = {1, 1};
  auto load = [&](uint32_t n) {  // heads h + n step and the next
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint32_t hd = min(h + (n + z) * step, last);
      const C* p = x + (int64_t)hd * sd.ch;
      if constexpr (kQuant) sc[z] = load_chunk<NT, float>(scales + (int64_t)hd * a.sh);
      v[z] = load_chunk<NT, CVec>(p + i);
      w[z] = load_chunk<NT, CVec>(p + (two ? j : i));
    }
  };
  load(0);
  for (uint32_t n = 0; n < count; n += 2) {
    CVec f[2], g[2];
    float m[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) f[z] = v[z], g[z] = w[z], m[z] = sc[z];
    if (n + 2 < count) load(n + 2);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (n + z >= count || h + (n + z) * step > last) continue;
      T* q = y + (int64_t)(h + (n + z) * step) * sd.rh;
      store_chunk<NT>(q + i, made(f[z], m[z]));
      if (two) store_chunk<NT>(q + j, made(g[z], m[z]));
    }
  }
}

// Any strides and sizes (177 us and 1047 us for the two sizes above): one wave per row (token, head) of one side; a
// lane holds pairs lane, lane + 64, ...
template <int DT, int CT>
__global__ void __launch_bounds__(256) k_cache_write(CacheArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t rows = 2ull * a.n * a.heads;
  for (uint64_t row = (uint64_t)blockIdx.x * 4 + threadIdx.x / 64; row < rows; row += (uint64_t)gridDim.x * 4) {
    const CacheSide& s = a.side[row & 1];
    const uint32_t t = (uint32_t)((row >> 1) / a.heads), h = (uint32_t)((row >> 1) % a.heads);
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.cache_slots) continue;
    const uint32_t page = (uint32_t)slot / a.page_size, in = (uint32_t)slot % a.page_size;
    const T* x = (const T*)s.rows + mode_offset(s.rh, h) + mode_offset(s.rt, t);
    C* y = (C*)s.cache + (int64_t)page * s.cp + (int64_t)in * s.cs + (int64_t)h * s.ch;
    const uint32_t half = (uint32_t)s.rot / 2, units = half + (uint32_t)(s.dim - s.rot + 1) / 2;
    float v[kCacheDim / 64];
    float amax = 0;
#pragma unroll
    for (int k = 0; k < kCacheDim / 128; ++k) {
      const uint32_t u = lane + 64 * k;
      v[2 * k] = v[2 * k + 1] = 0;
      if (u >= units) continue;
      const bool turned = u < half;
      const uint32_t i = !turned ? s.rot + 2 * (u - half) : a.pairs == LR_PAIRS_HALF ? u : 2 * u;
      const uint32_t j = turned && a.pairs == LR_PAIRS_HALF ? u + half : i + 1;
      float p = value_of<DT>(x[(int64_t)i * s.rd]), q = j < (uint32_t)s.dim ? value_of<DT>(x[(int64_t)j * s.rd]) : 0.f;
      if (turned) {
        float sn, cs;
        sincos_turn((uint64_t)a.positions[t] * (uint64_t)a.turns[u], &sn, &cs);
        sn *= a.magnitude;
        cs *= a.magnitude;
        const float w = p * cs - q * sn;
        q = q * cs + p * sn;
        p = w;
      }
      v[2 * k] = p;
      v[2 * k + 1] = q;
      if (__builtin_fabsf(p) < __builtin_inff()) amax = fmaxf(amax, __builtin_fabsf(p));
      if (__builtin_fabsf(q) < __builtin_inff()) amax = fmaxf(amax, __builtin_fabsf(q));
    }
    float scale = 1, up = 1;
    if constexpr (CT == LR_E4M3 || CT == LR_INT8) {
      for (int m = 32; m; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
      scale = fmaxf(amax / (CT == LR_E4M3 ? 448.f : 127.f), 0x1p-126f);
      up = amax < 0x1p-90f ? 0x1p64f : 1.f;
      if (lane == 0) s.scale[(int64_t)page * a.sp + (int64_t)in * a.ss + (int64_t)h * a.sh] = scale;
    }
#pragma unroll
    for (int k = 0; k < kCacheDim / 128; ++k) {
      const uint32_t u = lane + 64 * k;
      if (u >= units) continue;
      const bool turned = u < half;
      const uint32_t i = !turned ? s.rot + 2 * (u - half) : a.pairs == LR_PAIRS_HALF ? u : 2 * u;
      const uint32_t j = turned && a.pairs == LR_PAIRS_HALF ? u + half : i + 1;
      if constexpr (CT == LR_E4M3 || CT == LR_INT8) {
        y[(int64_t)i * s.cd] = code_of<CT>(v[2 * k] * up, scale * up);
        if (j < (uint32_t)s.dim) y[(int64_t)j * s.cd] = code_of<CT>(v[2 * k + 1] * up, scale * up);
      } else {
        y[(int64_t)i * s.cd] = (C)v[2 * k];
        if (j < (uint32_t)s.dim) y[(int64_t)j * s.cd] = (C)v[2 * k + 1];
      }
    }
  }
}

// Any strides and sizes.
template <int DT, int CT>
__global__ void __launch_bounds__(256) k_cache_read(CacheArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t rows = 2ull * a.n * a.heads;
  for (uint64_t row = (uint64_t)blockIdx.x * 4 + threadIdx.x / 64; row < rows; row += (uint64_t)gridDim.x * 4) {
    const CacheSide& s = a.side[row & 1];
    const uint32_t t = (uint32_t)((row >> 1) / a.heads), h = (uint32_t)((row >> 1) % a.heads);
    const int64_t slot = a.slots[t];
    T* y = (T*)s.rows + mode_offset(s.rh, h) + mode_offset(s.rt, t);
    const bool held = slot >= 0 && slot < a.cache_slots;
    const uint32_t page = held ? (uint32_t)slot / a.page_size : 0, in = held ? (uint32_t)slot % a.page_size : 0;
    const C* x = (const C*)s.cache + (int64_t)page * s.cp + (int64_t)in * s.cs + (int64_t)h * s.ch;
    float scale = 1;
    if constexpr (CT == LR_E4M3 || CT == LR_INT8)
      scale = s.scale[(int64_t)page * a.sp + (int64_t)in * a.ss + (int64_t)h * a.sh];
    for (uint32_t e = lane; e < (uint32_t)s.dim; e += 64)
      y[(int64_t)e * s.rd] = held ? (T)(value_of<CT>(x[(int64_t)e * s.cd]) * scale) : (T)0.f;
  }
}

// Whether `bytes` at p overlap the cache's codes or its scales.
static bool in_cache(const lr_cache* c, const void* p, int64_t bytes) {
  const int64_t e = dtype_bytes(c->dtype);
  if (overlap(p, bytes, c->k, c->k_capacity * e) || overlap(p, bytes, c->v, c->v_capacity * e)) return true;
  return is_quantised(c->dtype) &&
         (overlap(p, bytes, c->k_scale, c->scale_capacity * 4) || overlap(p, bytes, c->v_scale, c->scale_capacity * 4));
}

// The cache's own checks, and the part of the kernel arguments that comes from it.
static int fill_cache(const lr_cache* c, CacheArgs* a) {
  if (!c || !c->k || !c->v) return LR_ERR_INVALID;
  const bool quant = is_quantised(c->dtype);
  if (!quant && !is_model_type(c->dtype)) return LR_ERR_TYPE;
  if (quant ? !c->k_scale || !c->v_scale : c->k_scale || c->v_scale) return LR_ERR_INVALID;
  std::memset(a, 0, sizeof(*a));
  const lr_layout* L[2] = {&c->k_layout, &c->v_layout};
  const int64_t cap[2] = {c->k_capacity, c->v_capacity};
  int64_t heads = 0, slots = 0, pages = 0;
  for (int i = 0; i < 2; ++i) {
    if (int rc = check_tensor(L[i], 4, cap[i], true)) return rc;
    CacheSide& s = a->side[i];
    const Mode d = mode_of(*L[i], 0), h = mode_of(*L[i], 1), p = mode_of(*L[i], 2), g = mode_of(*L[i], 3);
    if (one_leaf(d, &s.cd) || one_leaf(h, &s.ch) || one_leaf(p, &s.cs) || one_leaf(g, &s.cp)) return LR_ERR_INVALID;
    if (d.size > kCacheDim) return LR_ERR_INVALID;
    if (i && (h.size != heads || p.size != slots || g.size != pages)) return LR_ERR_SIZE_MISMATCH;
    heads = h.size;
    slots = p.size;
    pages = g.size;
    s.dim = (int32_t)d.size;
    s.cache = i ? c->v : c->k;
    s.scale = i ? c->v_scale : c->k_scale;
  }
  if (pages > kMaxCount / slots) return LR_ERR_OVERFLOW;
  const int64_t e = dtype_bytes(c->dtype);
  if (overlap(c->k, c->k_capacity * e, c->v, c->v_capacity * e)) return LR_ERR_OVERLAP;
  if (quant) {
    if (int rc = check_tensor(&c->scale_layout, 3, c->scale_capacity, true)) return rc;
    const Mode h = mode_of(c->scale_layout, 0), p = mode_of(c->scale_layout, 1), g = mode_of(c->scale_layout, 2);
    if (h.size != heads || p.size != slots || g.size != pages) return LR_ERR_SIZE_MISMATCH;
    if (one_leaf(h, &a->sh) || one_leaf(p, &a->ss) || one_leaf(g, &a->sp)) return LR_ERR_INVALID;
    const int64_t bytes = c->scale_capacity * 4;
    if (overlap(c->k_scale, bytes, c->v_scale, bytes)) return LR_ERR_OVERLAP;
    for (const float* scale : {c->k_scale, c->v_scale})
      if (overlap(scale, bytes, c->k, c->k_capacity * e) || overlap(scale, bytes, c->v, c->v_capacity * e))
        return LR_ERR_OVERLAP;
  }
  a->heads = (uint32_t)heads;
  a->page_size = (uint32_t)slots;
  a->cache_slots = pages * slots;
  return LR_OK;
}

// The rows written from or read to.
static int fill_rows(const lr_cache* c, CacheArgs* a, const void* k, const lr_layout* Lk, int64_t k_capacity,
                     const void* v, const lr_layout* Lv, int64_t v_capacity, int32_t dtype, const int64_t* slots,
                     int64_t n, bool output) {
  if (!k || !v || n < 0 || (n > 0 && !slots)) return LR_ERR_INVALID;
  if (!is_model_type(dtype) || (!is_quantised(c->dtype) && c->dtype != dtype)) return LR_ERR_TYPE;
  const lr_layout* L[2] = {Lk, Lv};
  const void* p[2] = {k, v};
  const int64_t cap[2] = {k_capacity, v_capacity};
  const int64_t e = dtype_bytes(dtype);
  for (int i = 0; i < 2; ++i) {
    if (int rc = check_tensor(L[i], 3, cap[i], output)) return rc;
    CacheSide& s = a->side[i];
    const Mode d = mode_of(*L[i], 0), h = mode_of(*L[i], 1), t = mode_of(*L[i], 2);
    if (one_leaf(d, &s.rd)) return LR_ERR_INVALID;
    if (d.size != s.dim || h.size != (int64_t)a->heads) return LR_ERR_SIZE_MISMATCH;
    if (n > t.size) return LR_ERR_BOUNDS;
    s.rh = mode_arg(h);
    s.rt = mode_arg(t);
    s.rows = const_cast<void*>(p[i]);
    if (in_cache(c, p[i], cap[i] * e) || (output && overlap(p[i], cap[i] * e, slots, n * 8))) return LR_ERR_OVERLAP;
  }
  if (output ? overlap(k, k_capacity * e, v, v_capacity * e) : in_cache(c, slots, n * 8)) return LR_ERR_OVERLAP;
  a->slots = slots;
  a->n = (uint32_t)n;
  return LR_OK;
}

// Calls f<dtype, cache type>() for the pairs of types the cache takes.
template <class F>
static int with_types(int32_t dtype, int32_t ctype, F&& f) {
#define LR_CACHE_CASE(D)                                                                  \
  if (dtype == D) {                                                                       \
    if (ctype == D) return f(std::integral_constant<int, D>{}, std::integral_constant<int, D>{});             \
    if (ctype == LR_E4M3) return f(std::integral_constant<int, D>{}, std::integral_constant<int, LR_E4M3>{}); \
    if (ctype == LR_INT8) return f(std::integral_constant<int, D>{}, std::integral_constant<int, LR_INT8>{}); \
  }
  LR_CACHE_CASE(LR_F32)
  LR_CACHE_CASE(LR_F16)
  LR_CACHE_CASE(LR_BF16)
#undef LR_CACHE_CASE
  return LR_ERR_TYPE;
}

// The chunked kernels' arguments; the elements of a chunk, or 0 where rows are no whole chunks: 16 bytes of
// the rows' type, or 8.  `reduce`: the lanes of a row are a power of two within a wave.
static int fill_chunks(const lr_cache* c, const CacheArgs& a, const lr_layout* Lk, const lr_layout* Lv, int32_t dtype,
                       bool reduce, ChunkArgs* k, double* bytes) {
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  const lr_layout *L[2] = {Lk, Lv}, *cl[2] = {&c->k_layout, &c->v_layout};
  *bytes = 0;
  int v = (int)(16 / e);
  for (int i = 0; i < 2; ++i) {
    const CacheSide& s = a.side[i];
    if (one_leaf(mode_of(*L[i], 1), &k->side[i].rh) || !mode_pair(mode_of(*L[i], 2), &k->side[i].rt)) return 0;
    while (v > 1 && (s.rot / 2 % v || (s.dim - s.rot) % v || !rows_aligned(*L[i], s.rows, e, v) ||
                     !rows_aligned(*cl[i], s.cache, ce, v)))
      v /= 2;
  }
  if (v < 4) return 0;
  uint32_t lanes = 1;
  for (int i = 0; i < 2; ++i) {
    const CacheSide& s = a.side[i];
    ChunkSide& d = k->side[i];
    d.cache = s.cache;
    d.scale = s.scale;
    d.rows = s.rows;
    d.ch = s.ch;
    d.cs = s.cs;
    d.cp = s.cp;
    d.un = units_of(s.rot, s.dim, v);
    lanes = std::max(lanes, (uint32_t)d.un.count);
    *bytes += (double)a.n * a.heads * (double)(s.dim * (e + ce));
  }
  if (reduce)
    while (lanes & (lanes - 1)) lanes += lanes & -lanes;
  if (lanes > 64) return 0;
  k->grid = row_grid(lanes, a.heads, a.n, 2, reduce ? 2 : 4);
  k->slots = a.slots;
  k->turns = a.turns;
  k->positions = a.positions;
  k->sh = a.sh;
  k->ss = a.ss;
  k->sp = a.sp;
  k->cache_slots = a.cache_slots;
  k->fd_page = make_fastdiv(a.page_size);
  k->page_size = a.page_size;
  k->heads = a.heads;
  k->n = a.n;
  k->magnitude = a.magnitude;
  k->pairs = a.pairs;
  return row_grid_fits(k->grid) ? v : 0;
}

}  // namespace lr

using namespace lr;

extern "C" {

int lr_cache_validate(const lr_cache* c) {
  CacheArgs a;
  return fill_cache(c, &a);
}

int lr_cache_write(const lr_cache* c, const void* k, const lr_layout* Lk, int64_t k_capacity, const void* v,
                   const lr_layout* Lv, int64_t v_capacity, int32_t dtype, const int64_t* slots, int64_t n,
                   const lr_rotation* r, void* stream) {
  CacheArgs a;
  int rc = fill_cache(c, &a);
  if (rc || (rc = fill_rows(c, &a, k, Lk, k_capacity, v, Lv, v_capacity, dtype, slots, n, false))) return rc;
  if (r) {
    if ((rc = check_rotation(r, a.side[0].dim, n))) return rc;
    if (in_cache(c, r->positions, n * 8) || in_cache(c, r->turns, r->rot_dim * 4)) return LR_ERR_OVERLAP;
    a.side[0].rot = r->rot_dim;
    a.turns = r->turns;
    a.positions = r->positions;
    a.pairs = r->pairs;
    a.magnitude = r->magnitude;
  }
  if (n == 0) return LR_OK;
  const hipStream_t st = (hipStream_t)stream;
  ChunkArgs chunks;
  double bytes;
  const int wide = fill_chunks(c, a, Lk, Lv, dtype, true, &chunks, &bytes);
  const bool nt = bytes > kStreamBytes;
  if (wide)
    return with_types(dtype, c->dtype, [&](auto dt, auto ct) {
      constexpr int D = decltype(dt)::value, C = decltype(ct)::value;
      const dim3 grid(chunks.grid.blocks_x, chunks.grid.blocks_y, 2);
      if constexpr (D != LR_F32) {
        if (wide == 8) {
          if (nt)
            hipLaunchKernelGGL((k_cache_write_chunks<D, C, 8, true>), grid, dim3(256), 0, st, chunks);
          else
            hipLaunchKernelGGL((k_cache_write_chunks<D, C, 8, false>), grid, dim3(256), 0, st, chunks);
          return check_op_launch();
        }
      }
      if (nt)
        hipLaunchKernelGGL((k_cache_write_chunks<D, C, 4, true>), grid, dim3(256), 0, st, chunks);
      else
        hipLaunchKernelGGL((k_cache_write_chunks<D, C, 4, false>), grid, dim3(256), 0, st, chunks);
      return check_op_launch();
    });
  const int64_t rows = 2 * n * (int64_t)a.heads, groups = std::min<int64_t>((rows + 3) / 4, 1 << 22);
  return with_types(dtype, c->dtype, [&](auto dt, auto ct) {
    hipLaunchKernelGGL((k_cache_write<decltype(dt)::value, decltype(ct)::value>), dim3((unsigned)groups), dim3(256), 0,
                       st, a);
    return check_op_launch();
  });
}

int lr_cache_read(const lr_cache* c, const int64_t* slots, int64_t n, void* k, const lr_layout* Lk, int64_t k_capacity,
                  void* v, const lr_layout* Lv, int64_t v_capacity, int32_t dtype, void* stream) {
  CacheArgs a;
  int rc = fill_cache(c, &a);
  if (rc || (rc = fill_rows(c, &a, k, Lk, k_capacity, v, Lv, v_capacity, dtype, slots, n, true))) return rc;
  if (n == 0) return LR_OK;
  const hipStream_t st = (hipStream_t)stream;
  ChunkArgs chunks;
  double bytes;
  const int wide = fill_chunks(c, a, Lk, Lv, dtype, false, &chunks, &bytes);
  const bool nt = bytes > kStreamBytes;
  if (wide)
    return with_types(dtype, c->dtype, [&](auto dt, auto ct) {
      constexpr int D = decltype(dt)::value, C = decltype(ct)::value;
      const dim3 grid(chunks.grid.blocks_x, chunks.grid.blocks_y, 2);
      if constexpr (D != LR_F32) {
        if (wide == 8) {
          if (nt)
            hipLaunchKernelGGL((k_cache_read_chunks<D, C, 8, true>), grid, dim3(256), 0, st, chunks);
          else
            hipLaunchKernelGGL((k_cache_read_chunks<D, C, 8, false>), grid, dim3(256), 0, st, chunks);
          return check_op_launch();
        }
      }
      if (nt)
        hipLaunchKernelGGL((k_cache_read_chunks<D, C, 4, true>), grid, dim3(256), 0, st, chunks);
      else
        hipLaunchKernelGGL((k_cache_read_chunks<D, C, 4, false>), grid, dim3(256), 0, st, chunks);
      return check_op_launch();
    });
  const int64_t rows = 2 * n * (int64_t)a.heads, groups = std::min<int64_t>((rows + 3) / 4, 1 << 22);
  return with_types(dtype, c->dtype, [&](auto dt, auto ct) {
    hipLaunchKernelGGL((k_cache_read<decltype(dt)::value, decltype(ct)::value>), dim3((unsigned)groups), dim3(256), 0,
                       st, a);
    return check_op_launch();
  });
}

}  // extern "C"
