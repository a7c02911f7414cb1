// The kernels of attention over a paged cache, for lr_paged_attention, lr_prefix_attention and lr_block_attention.
//
// With s_t = scale q . k_t over the tokens t a sequence sees, out = sum_t e^(s_t - m) v_t / l with
// m = max s_t and l = sum_t e^(s_t - m).  One pass holds (m, l, o) for the tokens seen so far and
// rescales l and o by e^(m - m') when m grows to m'; parts of a sequence are joined by the same rule.
// Scores are held in base-2 units (scale * log2 e folded in), so that e^x is one v_exp_f32.
#pragma once

#include <type_traits>

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
  uint32_t unit_heads, tiles, units;  // query heads of a wave, their tiles in a cache head, units of a sequence
  uint32_t wide_heads, block;         // cache heads of a unit (1, or 4: one a wave); tokens of a block
  uint32_t splits, min_share;         // parts of a unit at most; blocks of a workgroup at least
  uint32_t grid;                      // workgroups (splits > 1; else one a unit)
  int64_t window;
  bool q_wide;   // query rows are contiguous and 16-byte aligned
  bool in_step;  // the four waves of four cache heads keep in step
  bool parts;    // every unit leaves its parts, also a whole one
  float scale2;  // scale * log2 e
  // Row r of cache head g's `group` rows is query head g * row_heads + r % row_heads of sequence b + r / row_heads:
  // row_heads is group where a sequence has tokens of its own, and a sequence's share of them where the rows of a
  // whole batch attend to the same tokens (b is then 0).
  uint32_t row_heads;
  FastDiv fd_rows;
  // The blocks that each cache head attends to, (sequence, cache head, count), or null: pages of the sequence.
  const int32_t* blocks;
  uint32_t count;
  int32_t path, wide;         // host only: lr_attention_path and the matrix kernel's variant
};

// The work is split evenly however uneven the sequences are.  A unit is one sequence's tokens for the
// query heads that one workgroup takes together (unit_heads of one cache head, or of four); its tokens are
// cut into blocks.  All blocks of all units, in order, are dealt out to `used` workgroups in equal runs:
// workgroup w has the blocks [w T / used, (w + 1) T / used) of T.  A run that starts or ends inside a unit
// leaves a part of it, joined by a second launch.  A unit of n blocks meets at most
// 1 + ceil((n - 1) / min_share) runs, as none is shorter than min_share.  That has to be at most `splits`, the
// parts of a unit that the workspace has room for, so min_share grows with the longest unit that the page table
// admits; where the lengths are far below it, fewer than all workgroups have a run (64 sequences of 1000 tokens, 32
// heads on 8 of 128: 54 us under a table just wide enough, 129 with 63 runs under one for 131072 tokens).
constexpr int64_t kRuns = 256;                     // one a CU
constexpr uint32_t kBlock = 128, kWideBlock = 32;  // a step of four waves over tokens, or over heads

// The tokens [first, n) a sequence sees; blocks start at `base`, first rounded down so that steps of 32
// tokens stay aligned.  A sequence without tokens has one (empty) block, so that it is written too.
// Where blocks are listed, the tokens are those of the list's pages one after another, `len` the sequence's own.
struct Span {
  uint32_t base, first, n, blocks, len;
};
// LISTED: blocks may be listed (a.blocks says whether they are).
template <bool LISTED> __device__ __forceinline__ Span span_of(const AttentionArgs& a, int32_t len) {
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t n = len;
  n = n < 0 ? 0 : n > cap ? cap : n;
  const uint32_t own = (uint32_t)n;
  if (LISTED && a.blocks) {
    const uint32_t pages = own ? op_div(own - 1, a.fd_page) + 1 : 0;
    n = (int64_t)(pages < a.count ? pages : a.count) * a.page_size;
  }
  const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
  const uint32_t base = (uint32_t)first & ~31u;
  const uint32_t blocks = ((uint32_t)n - base + a.block - 1) / a.block;
  return Span{base, (uint32_t)first, (uint32_t)n, blocks ? blocks : 1, own};
}
// Offset of row r of cache head g's rows in the queries.
__device__ __forceinline__ int64_t query_at(const AttentionArgs& a, uint32_t b, uint32_t g, uint32_t r) {
  const uint32_t s = op_div(r, a.fd_rows);
  return (int64_t)(b + s) * a.qb + (int64_t)(g * a.row_heads + r - s * a.row_heads) * a.qh;
}

struct Deal {
  uint64_t total;
  uint32_t used;
};
// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
  return uniform((uint32_t)x) | (uint64_t)uniform((uint32_t)(x >> 32)) << 32;
}
// blocks: of all sequences, one unit each.
__device__ __forceinline__ Deal deal_of(const AttentionArgs& a, uint64_t blocks) {
  const uint64_t total = uniform64(blocks) * a.units, most = total / a.min_share;
  return Deal{total, (uint32_t)(most < 1 ? 1 : most < a.grid ? most : a.grid)};
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, uint32_t lane) {  // inclusive; 64 sequences stay below 2^32
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(v, d);
    if (lane >= (uint32_t)d) v += u;
  }
  return v;
}
__device__ __forceinline__ uint64_t run_start(const Deal& d, uint64_t w) { return w * d.total / d.used; }
__device__ __forceinline__ uint32_t run_of(const Deal& d, uint64_t block) {
  return (uint32_t)(((block + 1) * d.used - 1) / d.total);
}

// One workgroup's way through its run, a unit at a time.
struct Run {
  Deal deal;
  uint32_t w;        // which run
  uint64_t at, end;  // blocks
  uint64_t start;    // of the current unit
  uint32_t b, u;     // the current unit: sequence, and its number there
  uint32_t split;    // the part of it that this run has
  bool whole, last;  // all of it; its end
  Span sp;
  uint32_t lo, hi;   // its tokens
};
__device__ __forceinline__ void run_unit(const AttentionArgs& a, uint32_t w, Run* r) {
  const uint64_t left = r->start + r->sp.blocks, stop = r->end < left ? r->end : left;
  r->last = stop == left;
  r->whole = !a.parts && r->at == r->start && r->last;
  r->split = r->whole ? 0 : w - run_of(r->deal, r->start);
  r->lo = r->sp.base + (uint32_t)(r->at - r->start) * a.block;
  const uint64_t hi = (uint64_t)r->sp.base + (stop - r->start) * a.block;
  r->hi = hi < r->sp.n ? (uint32_t)hi : r->sp.n;
}
template <bool LISTED> __device__ __forceinline__ bool run_begin(const AttentionArgs& a, uint32_t block, Run* r) {
  const uint32_t lane = threadIdx.x & 63;
  if (a.splits == 1) {  // one unit a workgroup
    r->b = block / a.units;
    r->u = block % a.units;
    r->sp = span_of<LISTED>(a, a.lens[r->b]);
    r->deal = Deal{1, 1};
    r->w = 0;
    r->at = r->start = 0;
    r->end = r->sp.blocks;
  } else {
    int32_t len = lane < a.batch ? a.lens[lane] : 0;
    uint32_t v = lane < a.batch ? span_of<LISTED>(a, len).blocks : 0;
    uint32_t upto = wave_scan(v, lane);  // the first 64 sequences
    uint64_t all = __shfl(upto, 63);
    if (a.batch > 64) {
      uint64_t more = 0;
      for (uint32_t i = 64 + lane; i < a.batch; i += 64) more += span_of<LISTED>(a, a.lens[i]).blocks;
      for (int x = 32; x; x >>= 1) more += __shfl_xor((unsigned long long)more, x);
      all += more;
    }
    r->deal = deal_of(a, all);
    if (block >= r->deal.used) return false;
    // Workgroups go to the eight dies in turn; neighbouring runs, which are often heads of the same tokens, go
    // to one die, whose cache then holds the lines they share: a token's scales for all heads lie in one line
    // (64 x 16384 e4m3 tokens: 466 to 441 us; runs that share no lines are within 1 %).
    r->w = r->deal.used % 8 ? block : block % 8 * (r->deal.used / 8) + block / 8;
    r->at = run_start(r->deal, r->w);
    r->end = run_start(r->deal, r->w + 1);
    uint64_t past = 0;  // blocks of the sequences before the 64 looked at
    for (uint32_t i = 0;; i += 64) {
      const uint64_t hit = __ballot((past + upto) * a.units > r->at);
      if (hit) {
        const int f = __ffsll((unsigned long long)hit) - 1;
        r->b = i + f;
        r->start = (past + uniform(__shfl(upto - v, f))) * a.units;
        r->sp = span_of<LISTED>(a, (int32_t)uniform(__shfl(len, f)));
        break;
      }
      past += uniform(__shfl(upto, 63));
      len = i + 64 + lane < a.batch ? a.lens[i + 64 + lane] : 0;
      v = i + 64 + lane < a.batch ? span_of<LISTED>(a, len).blocks : 0;
      upto = wave_scan(v, lane);
    }
    r->u = (uint32_t)((r->at - r->start) / r->sp.blocks);
    r->start += (uint64_t)r->u * r->sp.blocks;
  }
  run_unit(a, r->w, r);
  return true;
}
template <bool LISTED> __device__ __forceinline__ bool run_next(const AttentionArgs& a, Run* r) {
  r->start += r->sp.blocks;
  r->at = r->start;
  if (r->at >= r->end) return false;
  if (++r->u == a.units) {
    r->u = 0;
    r->sp = span_of<LISTED>(a, a.lens[++r->b]);
  }
  run_unit(a, r->w, r);
  return true;
}

// A part's maximum and sum for the second launch; the sign of the sum tells the last part of a unit.  A whole
// unit is written at once, and leaves a first part that is the last, for which there is nothing to join.
__device__ __forceinline__ void leave_part(const AttentionArgs& a, const Run& run, uint32_t bh, float m, float l) {
  float* ml = a.part_ml + 2 * ((uint64_t)bh * a.splits + run.split);
  ml[0] = m;
  ml[1] = __uint_as_float((__float_as_uint(l) & 0x7fffffffu) | (run.last ? 0x80000000u : 0));
}

// Weight 2^(m - top) of a part with maximum m among parts with maximum top; 0 for a part
// without tokens.
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

// log sum e^s of a part with maximum top and sum total: -inf without a token (0 is -inf in log2), NaN where a score
// is, for which the maximum says nothing.
__device__ __forceinline__ float lse_of(float top, float total) { return (top + __log2f(total)) * kLn2; }

// Orders this wave's accesses to shared memory; one wave's are done in their order, so no wait is needed.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Any types, strides and alignment (23.8 ms for the 2.15 GB below).  A unit is one query head; a workgroup's
// waves take tiles of 64 tokens of its run in turn, a lane a token for the scores and every 64th
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
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64);
  Run run;
  if (!run_begin<true>(a, blockIdx.x, &run)) return;
  do {
    const uint32_t b = run.b, h = run.u, g = h / a.group, bh = b * a.heads + h, split = run.split, hi = run.hi;
    const uint64_t lo = run.lo;
    const Span sp = run.sp;
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < (uint32_t)a.dk; e += 256)
      qs[e] = value_of<DT>(((const T*)a.q)[query_at(a, b, g, h - g * a.group) + (int64_t)e * a.qd]) * a.scale2;
    __syncthreads();
    float m = -__builtin_inff(), l = 0, o[kAttentionDim / 64] = {};
    for (uint64_t t0 = lo + 64 * w; t0 < hi; t0 += 256) {
      const uint32_t t = (uint32_t)t0 + lane;
      bool seen = t < hi && t >= sp.first;
      int64_t page = 0;
      uint32_t pg = op_div(t, a.fd_page);
      const uint32_t in = t - pg * a.page_size;
      if (seen && a.blocks) {
        pg = (uint32_t)a.blocks[((uint64_t)b * a.kv_heads + g) * a.count + pg];
        seen = pg < a.max_pages && pg * a.page_size + in < sp.len;
      }
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
      wave_fence();
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
      wave_fence();
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
      if (run.whole)
        ((T*)a.out)[(int64_t)b * a.ob + (int64_t)h * a.oh + (int64_t)e * a.od] =
            (T)(total > 0 ? acc / total : 0.f * acc);
      else
        a.part_o[((uint64_t)bh * a.splits + split) * a.dv + e] = acc;
    }
    if (threadIdx.x == 0) {
      if (a.splits > 1 || a.parts) leave_part(a, run, bh, top, total);
      if (run.whole && a.lse) a.lse[bh] = lse_of(top, total);
    }
  } while (run_next<true>(a, &run));
}

// ------------------------------------------------------------------ matrix instructions

typedef float F4 __attribute__((ext_vector_type(4)));
typedef __bf16 B2 __attribute__((ext_vector_type(2)));
typedef __bf16 B8 __attribute__((ext_vector_type(8)));
typedef _Float16 H2 __attribute__((ext_vector_type(2)));
typedef _Float16 H8 __attribute__((ext_vector_type(8)));
typedef uint32_t U4 __attribute__((ext_vector_type(4)));

template <int BYTES> struct Raw { typedef uint32_t T __attribute__((ext_vector_type(BYTES / 4))); };
template <> struct Raw<4> { typedef uint32_t T; };

__device__ __forceinline__ F4 mfma(B8 a, B8 b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(H8 a, H8 b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(F4 a, F4 b, F4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

template <int DT> struct MatrixOf { typedef F4 T; };
template <> struct MatrixOf<LR_BF16> { typedef B8 T; };
template <> struct MatrixOf<LR_F16> { typedef H8 T; };

// Eight codes (8 bytes) as matrix elements of the model's type: both 8-bit types are exact in it.
template <int DT, int CT>
__device__ __forceinline__ typename MatrixOf<DT>::T decode(typename Raw<8>::T x) {
  typename MatrixOf<DT>::T y;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    if constexpr (CT == LR_E4M3 && DT == LR_BF16) {
      const B2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[d], 1.f, false);
      const B2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[d], 1.f, true);
      y[4 * d] = a[0], y[4 * d + 1] = a[1], y[4 * d + 2] = b[0], y[4 * d + 3] = b[1];
    } else if constexpr (CT == LR_E4M3) {
      const H2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[d], 1.f, false);
      const H2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[d], 1.f, true);
      y[4 * d] = a[0], y[4 * d + 1] = a[1], y[4 * d + 2] = b[0], y[4 * d + 3] = b[1];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[4 * d + e] = (typename ElemOf<DT>::T)(float)(int8_t)(x[d] >> (8 * e));
    }
  }
  return y;
}

// Four codes as fp32.
template <int CT> __device__ __forceinline__ F4 decode4(uint32_t x) {
  F4 y;
  if constexpr (CT == LR_E4M3) {
    typedef float F2 __attribute__((ext_vector_type(2)));
    const F2 a = __builtin_amdgcn_cvt_pk_f32_fp8(x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(x, true);
    y = F4{a[0], a[1], b[0], b[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)(int8_t)(x >> (8 * e));
  }
  return y;
}

// Two codes (the low or the high half of x) as bf16.
template <int CT, bool HIGH>
__device__ __forceinline__ uint32_t decode_pair(uint32_t x) {
  if constexpr (CT == LR_E4M3) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.f, HIGH));
  } else {
    const B2 y = {(__bf16)(float)(int8_t)(x >> (HIGH ? 16 : 0)), (__bf16)(float)(int8_t)(x >> (HIGH ? 24 : 8))};
    return __builtin_bit_cast(uint32_t, y);
  }
}

// Two 16-bit numbers with infinities and NaN replaced by the largest finite number of their sign.  As signed integers
// the positive ones have their order and the negative ones are below zero; as unsigned integers the negative
// ones have the order of their size, above all positive ones.
template <int DT> __device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
  typedef short I2 __attribute__((ext_vector_type(2)));
  typedef unsigned short W2 __attribute__((ext_vector_type(2)));
  constexpr unsigned short kMost = DT == LR_F16 ? 0x7bff : 0x7f7f;
  const I2 y = __builtin_elementwise_min(__builtin_bit_cast(I2, x), I2{(short)kMost, (short)kMost});
  constexpr unsigned short kLeast = kMost | 0x8000;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(W2, y), W2{kLeast, kLeast}));
}

// x itself, unknown to the compiler: what is computed from it is not kept in registers over the loop around.
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float across_groups_max(float x) {  // over lanes l, l ^ 16, l ^ 32
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float across_groups_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
// What the four waves of a workgroup take: tokens of one cache head, a cache head each, or tokens of the blocks that
// are listed for one cache head.
enum Waves { kOverTokens, kOverHeads, kOverBlocks };
// Keys and values up to DC wide; HT tiles of 16 query heads of one cache head.
template <int DT, int CT, int DC, int HT>
struct MatrixShape {
  static constexpr bool kF32 = DT == LR_F32;
  static constexpr int kElem = CT == LR_F32 ? 4 : CT == LR_E4M3 || CT == LR_INT8 ? 1 : 2;
  static constexpr int kTiles = kF32 ? 1 : 2;                  // 16-token tiles of a wave's step
  static constexpr int kTokens = 16 * kTiles;
  static constexpr int kPart = kF32 ? 4 : 8;                   // inner elements a lane gives one product
  static constexpr int kKeyChunk = 16 / kElem;                 // key elements a lane loads at a time
  static constexpr int kKeyParts = kKeyChunk / kPart;
  static constexpr int kKeySteps = (DC + 4 * kKeyChunk - 1) / (4 * kKeyChunk);
  static constexpr int kValChunk = kF32 || (DC % 128 && DC != 96) ? 4 : 8;   // value elements a lane loads at a time
  static constexpr int kValSteps = (DC + 16 * kValChunk - 1) / (16 * kValChunk);
  static constexpr int kVals = 4 * kTiles;                     // value rows a lane loads in a step
  // waves of a SIMD, the most that needs no spills
  static constexpr int kMinWaves = (DC >= 160 && kElem > 1) || (kF32 && DC * HT > 128) ? 1 : 2;
};

// A workgroup has one chunk of one sequence and HT * 16 query heads that share a cache head; its four
// waves take steps of 32 tokens (16 in fp32) in turn and join at the end.
//
// The scores of 16 tokens x 16 heads are a product of keys (rows) and queries (columns), so that a lane
// (head = lane % 16, j = lane / 16) gets tokens 4j .. 4j + 3 of each tile: exactly the operand that the
// second product, values transposed x weights, wants from it when its inner index runs over the tokens
// in that order.  Weights never leave their lane.  Keys come from memory as the operand itself (16 rows,
// each lane a chunk).  Values come as whole rows (a row a group of 16 lanes), eight rows a lane, and are
// transposed within the lane by byte permutes; the output's column 8 r + m is then row r of product m.
//
// What bounds it is the reading of the cache: 64 sequences of up to 16384 bf16 tokens, 64 query heads on 8 of 128
// (2.15 GB) take 338 us a call, 6.4 TB/s, and 2 of 131071 e4m3 tokens 93 us, 6.0 TB/s, where a bare streaming read
// reaches 7.2 (299 and 77 us); as many fp16 tokens 339 us, 2.21 GB of fp32 (32 sequences, 32 heads) 340 us, 6.5 TB/s,
// and fp32 queries over 0.57 GB of e4m3 228 us, 2.5 TB/s, where the fp32 products are the bound.  The vector units are
// busy 19 % of the first, 37 % of the second, with the matrix units' part.
// One workgroup a CU keeps enough loads under way; two and three a CU (512 and 768 runs) took 359 and 367 us against
// 353, as more rows of memory are open at once.  Plain loads took 20 % longer than streaming ones.
template <int DT, int CT, int DC, int HT, int WAVES> struct MatrixShared {
  static constexpr int kRow = 16 * MatrixShape<DT, CT, DC, HT>::kValChunk + 4;  // floats; the 4 keep 16 heads' accesses off one bank
  static constexpr int kJoin = WAVES == kOverHeads ? 1 : 16;                    // four heads are not joined
  int64_t offs[4][64];
  __attribute__((aligned(16))) float scales[4][64];
  float ms[4][kJoin * HT], ls[4][kJoin * HT];
  __attribute__((aligned(16))) float os[4][kJoin * kRow];
};
// The run of workgroup `block` of the pass.  The arguments come by value: by reference the compiler reckons with what is
// written in between changing them, and keeps up to three times as many aside (48 sequences of up to 9001 int8 tokens under
// a window of 2048, 20 heads of 80 fp16 on one: 21.6 us a call so, 21.0 now).
template <int DT, int CT, int DC, int HT, int WAVES>
__device__ __forceinline__ void attention_run(AttentionArgs a, uint32_t block,
                                              MatrixShared<DT, CT, DC, HT, WAVES>& shared) {
  constexpr bool by_heads = WAVES == kOverHeads, listed = WAVES == kOverBlocks;
  using S = MatrixShape<DT, CT, DC, HT>;
  using T = typename ElemOf<DT>::T;
  using M = typename MatrixOf<DT>::T;
  typedef U4 KR __attribute__((aligned(8)));  // rows of 8-bit caches are aligned to 8 elements
  typedef typename Raw<8>::T KHalf;
  using VR = typename Raw<S::kValChunk * S::kElem>::T;
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  constexpr int kRow = MatrixShared<DT, CT, DC, HT, WAVES>::kRow;
  auto& ms = shared.ms;
  auto& ls = shared.ls;
  auto& os = shared.os;
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64), r = lane & 15, j = lane >> 4;
  int64_t* offs = shared.offs[w];
  float* scales = shared.scales[w];

  Run run;
  if (!run_begin<listed>(a, block, &run)) return;
  for (bool again = false;; again = true) {
    const uint32_t b = run.b, split = run.split, hi = run.hi;
    const uint32_t g = by_heads ? run.u / a.tiles * 4 + w : run.u / a.tiles;
    const uint32_t in_group = run.u % a.tiles * 16 * HT;  // first query head of this unit within its group
    const Span sp = run.sp;
    const uint32_t lo = run.lo;

    // queries: lane r's head, dimensions chunk kk * 4 + j
    const uint32_t rq = here(r), jq = here(j);
    M q[HT][S::kKeySteps * S::kKeyParts];
    auto dim_at = [&](int kk) -> uint32_t {
      return ((kk / S::kKeyParts * 4 + jq) * S::kKeyParts + kk % S::kKeyParts) * S::kPart;
    };
    auto load_queries = [&](auto wide) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const uint32_t h = in_group + 16 * ht + rq;
        const T* x = (const T*)a.q + query_at(a, b, g, h < a.group ? h : 0);
#pragma unroll
        for (int kk = 0; kk < S::kKeySteps * S::kKeyParts; ++kk) {
          const uint32_t e0 = dim_at(kk) < (uint32_t)a.dk ? dim_at(kk) : 0;
          if constexpr (decltype(wide)::value) {
            q[ht][kk] = *(const M*)(x + e0);
          } else {
#pragma unroll
            for (int e = 0; e < S::kPart; ++e) q[ht][kk][e] = x[(int64_t)(e0 + e) * a.qd];
          }
        }
      }
    };
    if (a.q_wide)
      load_queries(std::true_type{});
    else
      load_queries(std::false_type{});
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int kk = 0; kk < S::kKeySteps * S::kKeyParts; ++kk)
        if (in_group + 16 * ht + rq >= a.group || dim_at(kk) >= (uint32_t)a.dk) q[ht][kk] = M{};

    // Page lookup: lanes 0 .. and 32 .. find the pages of a step's tokens, the first for keys, the second
    // for values.  All loads of the loop below are unconditional, so that each wait is for the loads it
    // needs and no younger ones: what is not there is read from a place that is, and left out after.
    const uint32_t li = lane & (S::kTokens - 1);
    const bool for_v = lane >= 32;
    const int32_t* table = a.table + (int64_t)b * a.table_stride;
    const uint32_t one = a.fd_page.m ? 0 : ~0u;  // pages of one slot: the quotient is the dividend
    auto page_index = [&](uint32_t t) -> uint32_t { return (__umulhi(t, a.fd_page.m) >> a.fd_page.s) + (t & one); };
    const int32_t* list = a.blocks + ((uint64_t)b * a.kv_heads + g) * a.count;  // only looked at where blocks are listed
    auto page_of = [&](uint32_t t0) -> int32_t {
      const uint32_t t = t0 + li < hi ? t0 + li : hi - 1, at = page_index(t);
      if constexpr (listed) {
        const uint32_t block = (uint32_t)list[at], in = t - at * a.page_size;
        const bool ok = block < a.max_pages && block * a.page_size + in < sp.len;
        const int32_t page = table[ok ? block : 0];
        return ok ? page : -1;
      } else {
        return table[at];
      }
    };
    const int64_t page_step = (for_v ? a.vp : a.kp) * S::kElem, slot_step = (for_v ? a.vsl : a.ksl) * S::kElem;
    const float* scale_base = nullptr;
    if constexpr (kQuant) scale_base = (for_v ? a.vs : a.ks) + (int64_t)g * a.sh;
    const char* kbase = (const char*)a.k + (int64_t)g * a.kh * S::kElem;
    const char* vbase = (const char*)a.v + (int64_t)g * a.vh * S::kElem;

    // The step's row offsets to shared memory (0, the cache's first row, for a token that is not seen);
    // returns the mask of its seen tokens.
    auto place = [&](uint32_t t0, int32_t page, float* scale) -> uint32_t {
      const uint32_t t = t0 + li;
      const bool ok = (t >= sp.first) & (t < hi) & ((uint32_t)page < a.pages);
      const uint32_t in = ok ? t - page_index(t) * a.page_size : 0, pg = ok ? page : 0;
      wave_fence();
      offs[lane] = (int64_t)(pg * (uint64_t)page_step + in * (uint64_t)slot_step);
      wave_fence();
      if constexpr (kQuant)  // streaming too: plain loads of the scales alone took 132 us where these take 109
        *scale = __builtin_nontemporal_load(scale_base + (pg * (uint64_t)a.sp + in * (uint64_t)a.ssl));
      return (uint32_t)__ballot(ok);
    };

    KR kr[S::kTiles][S::kKeySteps];
    VR vr[S::kVals][S::kValSteps];
    // Where a lane's chunk kk of a row is read: past the row's end where the group's first lane reads, or the
    // load before, so that it asks for no other line; half past it (8 elements of 16 are left) 8 before, whose
    // upper half they are.
    auto key_at = [&](int kk) -> uint32_t {
      const uint32_t dk = (uint32_t)a.dk, e0 = (kk * 4 + j) * S::kKeyChunk, g0 = kk * 4 * S::kKeyChunk;
      const uint32_t past = g0 + S::kKeyChunk <= dk ? g0 : e0 >= 4 * S::kKeyChunk ? e0 - 4 * S::kKeyChunk : 0;
      return e0 >= dk ? (past + S::kKeyChunk <= dk ? past : 0) : e0 + S::kKeyChunk > dk ? e0 - 8 : e0;
    };
    const bool ragged = a.dk != DC;
    auto load_keys = [&]() {
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t) {
        const char* row = kbase + offs[16 * t + r];
#pragma unroll
        for (int kk = 0; kk < S::kKeySteps; ++kk) {
          kr[t][kk] = __builtin_nontemporal_load((const KR*)(row + key_at(kk) * S::kElem));
        }
      }
    };
    auto load_values = [&]() {
#pragma unroll
      for (int x = 0; x < S::kVals; ++x) {
        const char* row = vbase + offs[32 + 16 * (x / 4) + 4 * j + x % 4];
#pragma unroll
        for (int p = 0; p < S::kValSteps; ++p) {
          const uint32_t e0 = (p * 16 + r) * S::kValChunk, g0 = p * 16 * S::kValChunk;
          const uint32_t at = e0 < (uint32_t)a.dv ? e0 : g0 < (uint32_t)a.dv ? g0 : 0;  // past dv: rows of no output
          vr[x][p] = __builtin_nontemporal_load((const VR*)(row + at * S::kElem));
        }
      }
    };

    F4 o[HT][S::kValSteps][S::kValChunk] = {};
    // Scores are taken off `base`, at most 8 below the running maximum; weights in fp16 parts, whose smallest is
    // 2^-24, off a base 7 to 15 below it: the largest is then 2^7 to 2^15, and one of 2^-32 of it still counts.
    constexpr float kLow = std::is_same_v<M, H8> && !kQuant ? 7.f : 0.f;
    float base[HT], l[HT];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) base[ht] = -__FLT_MAX__, l[ht] = 0;
    constexpr uint32_t kAll = 0xffffffffu;  // of 16 tokens the mask has every bit twice

    const uint32_t step = by_heads ? S::kTokens : 4 * S::kTokens;
    uint32_t t0 = by_heads ? lo : lo + w * S::kTokens;
    if (t0 < hi) {
      float sc = 0;
      uint32_t seen = place(t0, page_of(t0), &sc);
      int32_t page = page_of(t0 + step);
      load_keys();
      load_values();
      // The last round's loads are of the cache's first row, so that they need no branch either.
      do {
        // scores
        if (ragged)
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int kk = 0; kk < S::kKeySteps; ++kk) {
              const uint32_t e0 = (kk * 4 + j) * S::kKeyChunk;
              if (kQuant && e0 + 8 == (uint32_t)a.dk) kr[t][kk] = KR{kr[t][kk][2], kr[t][kk][3], 0, 0};
              if (e0 >= (uint32_t)a.dk) kr[t][kk] = KR{};
            }
        F4 s[HT][S::kTiles];
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) {
            s[ht][t] = F4{};
#pragma unroll
            for (int kk = 0; kk < S::kKeySteps; ++kk) {
              if constexpr (kQuant && S::kF32) {
#pragma unroll
                for (int d = 0; d < 4; ++d) s[ht][t] = mfma(decode4<CT>(kr[t][kk][d]), q[ht][4 * kk + d], s[ht][t]);
              } else if constexpr (kQuant) {
                s[ht][t] = mfma(decode<DT, CT>(KHalf{kr[t][kk][0], kr[t][kk][1]}), q[ht][2 * kk], s[ht][t]);
                s[ht][t] = mfma(decode<DT, CT>(KHalf{kr[t][kk][2], kr[t][kk][3]}), q[ht][2 * kk + 1], s[ht][t]);
              } else {
                s[ht][t] = mfma(__builtin_bit_cast(M, kr[t][kk]), q[ht][kk], s[ht][t]);
              }
            }
          }
        F4 ksc[S::kTiles], vsc[S::kTiles];
        if constexpr (kQuant) {
          wave_fence();
          scales[lane] = (seen >> li) & 1 ? sc : 0.f;
          wave_fence();
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t) {
            ksc[t] = *(const F4*)&scales[16 * t + 4 * j] * a.scale2;
            vsc[t] = *(const F4*)&scales[32 + 16 * t + 4 * j];
          }
        }
        const uint32_t seen_next = place(t0 + step, page, &sc);
        page = page_of(t0 + 2 * step);
        if constexpr (by_heads && !kQuant && !S::kF32)
          if (a.in_step) __builtin_amdgcn_s_barrier();  // the four waves make equally many rounds
        load_keys();
        // weights
        // Of 16-bit products' weights two parts are taken, the value and what its rounding left, 16 bits in bf16 and 22
        // in fp16: a bf16 alone would add as much error to the output as its own rounding does, and cost an fp16
        // model with an 8-bit cache its last three bits; a third part would add nothing that an output of 8 or 11
        // bits shows.  The second part may be zero or negative, so that an infinite value must meet
        // the first one only: times zero, or taken off itself, it would be NaN.  An fp16 first part is not rounded to
        // zero for the same reason; the second takes off what is too much.
        using P = std::conditional_t<kQuant && !S::kF32, B8, M>;
        using PE = std::conditional_t<kQuant && !S::kF32, __bf16, T>;
        P phi[HT], plo[HT];
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          float top = -__builtin_inff();
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t) {
            if constexpr (kQuant)
              s[ht][t] *= ksc[t];
            else
              s[ht][t] *= a.scale2;
            if (seen != kAll)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[ht][t][i] = (seen >> (16 * t + 4 * j + i)) & 1 ? s[ht][t][i] : -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[ht][t][i]);
          }
          if (__any(top > base[ht] + (8.f + kLow))) {
            top = fmaxf(base[ht], across_groups_max(top) - kLow);
            const float keep = __builtin_amdgcn_exp2f(base[ht] - top);
            base[ht] = top;
            l[ht] *= keep;
#pragma unroll
            for (int p = 0; p < S::kValSteps; ++p)
#pragma unroll
              for (int m = 0; m < S::kValChunk; ++m) o[ht][p][m] *= keep;
          }
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = __builtin_amdgcn_exp2f(s[ht][t][i] - base[ht]);
              l[ht] += x;
              if constexpr (kQuant) x *= vsc[t][i];
              phi[ht][4 * t + i] = (PE)(std::is_same_v<PE, _Float16> ? fmaxf(x, 0x1p-24f) : x);
              if constexpr (!S::kF32) plo[ht][4 * t + i] = (PE)(x - (float)phi[ht][4 * t + i]);
            }
        }
        if (seen != kAll)  // what is not seen may hold NaN
#pragma unroll
          for (int x = 0; x < S::kVals; ++x)
            if (!((seen >> (16 * (x / 4) + 4 * j + x % 4)) & 1))
#pragma unroll
              for (int p = 0; p < S::kValSteps; ++p) vr[x][p] = VR{};
        // values
#pragma unroll
        for (int p = 0; p < S::kValSteps; ++p) {
          if constexpr (S::kF32) {
            F4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if constexpr (kQuant)
                v[x] = decode4<CT>(vr[x][p]);
              else
                v[x] = __builtin_bit_cast(F4, vr[x][p]);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
                o[ht][p][m] = mfma(F4{v[0][m], v[1][m], v[2][m], v[3][m]}, phi[ht], o[ht][p][m]);
          } else if constexpr (kQuant) {
#pragma unroll
            for (int d = 0; d < S::kValChunk / 4; ++d) {
              auto word = [&](int x) { if constexpr (S::kValChunk == 4) return vr[x][p]; else return vr[x][p][d]; };
#pragma unroll
              for (int half = 0; half < 2; ++half) {  // columns 4 d + 2 half and the next
                U4 v0, v1;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const uint32_t y = __builtin_amdgcn_perm(word(2 * x + 1), word(2 * x), half ? 0x07030602 : 0x05010400);
                  v0[x] = decode_pair<CT, false>(y);
                  v1[x] = decode_pair<CT, true>(y);
                }
#pragma unroll
                for (int ht = 0; ht < HT; ++ht) {
                  F4& oa = o[ht][p][4 * d + 2 * half];
                  F4& ob = o[ht][p][4 * d + 2 * half + 1];
                  oa = mfma(__builtin_bit_cast(B8, v0), phi[ht], oa);
                  ob = mfma(__builtin_bit_cast(B8, v1), phi[ht], ob);
                  oa = mfma(__builtin_bit_cast(B8, v0), plo[ht], oa);
                  ob = mfma(__builtin_bit_cast(B8, v1), plo[ht], ob);
                }
              }
            }
          } else {
#pragma unroll
            for (int d = 0; d < S::kValChunk / 2; ++d) {  // columns 2 d and the next
              U4 v0, v1;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                v0[x] = __builtin_amdgcn_perm(vr[2 * x + 1][p][d], vr[2 * x][p][d], 0x05040100);
                v1[x] = __builtin_amdgcn_perm(vr[2 * x + 1][p][d], vr[2 * x][p][d], 0x07060302);
              }
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                F4& oa = o[ht][p][2 * d];
                F4& ob = o[ht][p][2 * d + 1];
                oa = mfma(__builtin_bit_cast(M, v0), phi[ht], oa);
                ob = mfma(__builtin_bit_cast(M, v1), phi[ht], ob);
              }
#pragma unroll
              for (int x = 0; x < 4; ++x) v0[x] = finite_pair<DT>(v0[x]), v1[x] = finite_pair<DT>(v1[x]);
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                F4& oa = o[ht][p][2 * d];
                F4& ob = o[ht][p][2 * d + 1];
                oa = mfma(__builtin_bit_cast(M, v0), plo[ht], oa);
                ob = mfma(__builtin_bit_cast(M, v1), plo[ht], ob);
              }
            }
          }
        }
        load_values();
        seen = seen_next;
        t0 += step;
      } while (t0 < hi);
    }

    const uint32_t re = here(r), je = here(j);
    if constexpr (by_heads) {
      // a wave has all of its head's part
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const float total = across_groups_sum(l[ht]);
        const float top = base[ht] == -__FLT_MAX__ ? -__builtin_inff() : base[ht];
        const uint32_t h = in_group + 16 * ht + re;
        if (h >= a.group) continue;
        const uint32_t bh = b * a.heads + g * a.group + h;
        T* out = (T*)a.out + (int64_t)b * a.ob + (int64_t)(g * a.group + h) * a.oh;
        const float inv = total > 0 ? 1.f / total : 0.f;
#pragma unroll
        for (int p = 0; p < S::kValSteps; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < S::kValChunk; m += 4) {
              const uint32_t e = (p * 16 + 4 * je + i) * S::kValChunk + m;
              if (e >= (uint32_t)a.dv) continue;
              const F4 x = {o[ht][p][m][i], o[ht][p][m + 1][i], o[ht][p][m + 2][i], o[ht][p][m + 3][i]};
              if (run.whole) {
#pragma unroll
                for (int y = 0; y < 4; ++y) out[(int64_t)(e + y) * a.od] = (T)(total != total ? total : x[y] * inv);
              } else {
                *(F4*)&a.part_o[((uint64_t)bh * a.splits + split) * a.dv + e] = x;
              }
            }
        if (je == 0) {
          if (a.splits > 1 || a.parts) leave_part(a, run, bh, top, total);
          if (run.whole && a.lse) a.lse[bh] = lse_of(top, total);
        }
      }
    } else {
      // join the waves: maxima and sums, then 16 heads x 16 chunks of columns at a time
      const uint32_t lane256 = here(threadIdx.x);
      if (again) __syncthreads();
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const float sum = across_groups_sum(l[ht]);
        if (je == 0) {
          ms[w][16 * ht + re] = base[ht] == -__FLT_MAX__ ? -__builtin_inff() : base[ht];
          ls[w][16 * ht + re] = sum;
        }
      }
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int p = 0; p < S::kValSteps; ++p) {
          if (ht || p) __syncthreads();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < S::kValChunk; m += 4)
              *(F4*)&os[w][re * kRow + (4 * je + i) * S::kValChunk + m] =
                  F4{o[ht][p][m][i], o[ht][p][m + 1][i], o[ht][p][m + 2][i], o[ht][p][m + 3][i]};
          __syncthreads();
#pragma unroll
          for (int x = 0; x < S::kValChunk / 4; ++x) {
            const uint32_t at = lane256 + 256 * x, hd = at / (4 * S::kValChunk), c4 = at % (4 * S::kValChunk) * 4;
            const uint32_t h = in_group + 16 * ht + hd, e = p * 16 * S::kValChunk + c4;
            if (h >= a.group || e >= (uint32_t)a.dv) continue;
            float m4[4], top = -__builtin_inff(), total = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, m4[i] = ms[i][16 * ht + hd]);
            F4 acc = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float wt = weight_of(m4[i], top);
              total += ls[i][16 * ht + hd] * wt;
              acc += *(const F4*)&os[i][hd * kRow + c4] * wt;
            }
            const uint32_t bh = b * a.heads + g * a.group + h;
            if (run.whole) {
              T* out = (T*)a.out + (int64_t)b * a.ob + (int64_t)(g * a.group + h) * a.oh;
              const float inv = total > 0 ? 1.f / total : 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) out[(int64_t)(e + i) * a.od] = (T)(total != total ? total : acc[i] * inv);
            } else {
              *(F4*)&a.part_o[((uint64_t)bh * a.splits + split) * a.dv + e] = acc;
            }
            if (e == 0) {
              if (a.splits > 1 || a.parts) leave_part(a, run, bh, top, total);
              if (run.whole && a.lse) a.lse[bh] = lse_of(top, total);
            }
          }
        }
    }
    if (!run_next<listed>(a, &run)) break;
  }
}

template <int DT, int CT, int DC, int HT, int WAVES>
__global__ void __launch_bounds__(256, (MatrixShape<DT, CT, DC, HT>::kMinWaves)) k_attention_matrix(AttentionArgs a) {
  __shared__ MatrixShared<DT, CT, DC, HT, WAVES> shared;
  attention_run<DT, CT, DC, HT, WAVES>(a, blockIdx.x, shared);
}

// The parts of one query head, joined by a workgroup or a wave: a wave has the weights of 64 parts at a time, one a lane;
// the LANES lanes are groups of lanes with four columns each, a group takes every next part, and the groups' sums are added
// in their order.
struct Joined {
  float top, total;
  F4 acc;
};
struct Columns {  // of this lane: four from 4 c on, for the parts grp, grp + groups, ...
  uint32_t wide, groups, grp, c;
};
template <int LANES> __device__ __forceinline__ Columns columns_of(int32_t dv) {
  const uint32_t wide = ((uint32_t)dv + 3) / 4, lane = threadIdx.x % LANES, grp = lane / wide;
  return Columns{wide, LANES / wide, grp, lane - grp * wide};
}
typedef float F2 __attribute__((ext_vector_type(2)));
// Maximum and sum of this lane's part among the 64 from s on.
__device__ __forceinline__ F2 part_at(const float* part_ml, uint32_t s, uint32_t splits) {
  const uint32_t i = s + (threadIdx.x & 63);
  return i < splits ? ((const F2*)part_ml)[i] : F2{-__builtin_inff(), 0.f};
}
// Adds the parts of the list at part_ml (the first 64 of which are `x`) and part_o; false for a unit that is whole, where
// that is asked for.
__device__ __forceinline__ bool join_list(F2 x, const float* part_ml, const float* part_o, uint32_t splits, int32_t dv,
                                          const Columns& q4, bool ask_whole, Joined* j) {
  const uint32_t lane = threadIdx.x & 63, c = q4.c;
  const float* po = part_o + 4 * c;
  float top = j->top, total = j->total;
  F4 acc = j->acc;
  for (uint32_t s = 0; s < splits; s += 64) {
    if (s) x = part_at(part_ml, s, splits);
    const uint64_t hit = __ballot(__float_as_uint(x[1]) >> 31);  // what is past the last part means nothing
    const uint32_t parts = hit ? __ffsll((unsigned long long)hit) : 64;
    if (ask_whole && s == 0 && parts == 1) return false;  // whole: written already
    const float m = lane < parts ? x[0] : -__builtin_inff();
    float most = m;
    for (int d = 32; d; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
    most = fmaxf(top, most);
    const float keep = weight_of(top, most), wt = weight_of(m, most);
    float sum = lane < parts ? __builtin_fabsf(x[1]) * wt : 0.f;
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    total = total * keep + sum;
    top = most;
    acc *= keep;
    for (uint32_t q = 0; q < parts; q += q4.groups) {
      const uint32_t p = q + q4.grp;
      const float w = __shfl(wt, p & 63);
      if (p >= parts || q4.grp >= q4.groups) continue;
      const float* y = po + (uint64_t)(s + p) * dv;
      if (dv % 4 == 0) {
        acc += *(const F4*)y * w;
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          if (4 * c + i < (uint32_t)dv) acc[i] += y[i] * w;
      }
    }
    if (hit) break;
  }
  *j = Joined{top, total, acc};
  return true;
}
// The groups' sums added, and the head's output; `os`: LANES * 4 floats of these lanes, `blank`: zeros instead.
template <int DT, int LANES>
__device__ __forceinline__ void join_out(const AttentionArgs& a, uint32_t b, uint32_t h, const Columns& q4, Joined j, bool blank,
                                         float* os) {
  using T = typename ElemOf<DT>::T;
  F4 acc = j.acc;
  *(F4*)&os[4 * (threadIdx.x % LANES)] = acc;
  if constexpr (LANES == 64)
    wave_fence();
  else
    __syncthreads();
  if (q4.grp) return;
  for (uint32_t i = 1; i < q4.groups; ++i) acc += *(const F4*)&os[4 * (i * q4.wide + q4.c)];
  T* out = (T*)a.out + (int64_t)b * a.ob + (int64_t)h * a.oh;
  const float inv = j.total > 0 ? 1.f / j.total : 0.f;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    if (4 * q4.c + i < (uint32_t)a.dv)
      out[(int64_t)(4 * q4.c + i) * a.od] = (T)(blank ? 0.f : j.total != j.total ? j.total : acc[i] * inv);
  if (q4.c == 0 && a.lse) a.lse[(uint64_t)b * a.heads + h] = blank ? -__builtin_inff() : lse_of(j.top, j.total);
}

// 4096 heads: 6 us; 32 heads: 4 us, most of it the launch.
template <int DT>
__global__ void __launch_bounds__(256) k_attention_join(AttentionArgs a) {
  __shared__ __attribute__((aligned(16))) float os[256 * 4];
  const uint64_t at = (uint64_t)blockIdx.x * a.splits;
  const Columns q4 = columns_of<256>(a.dv);
  Joined j{-__builtin_inff(), 0.f, F4{}};
  const float* ml = a.part_ml + 2 * at;
  if (!join_list(part_at(ml, 0, a.splits), ml, a.part_o + at * a.dv, a.splits, a.dv, q4, true, &j)) return;
  join_out<DT, 256>(a, blockIdx.x / a.heads, blockIdx.x % a.heads, q4, j, false, os);
}

// ------------------------------------------------------------------ host

// The layouts' checks and what follows from them: strides, sizes, the cache's arrays, and whether the matrix kernel
// takes buffers that are aligned (out->path).  max_pages: of the page table.
int attention_shapes(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages, int32_t dtype,
                     AttentionArgs* a, lr_attention_plan* out);
// How `sequences` units of work of up to `span` tokens each, for a->group rows of each cache head, are cut up.
int attention_split(int64_t sequences, int64_t span, bool listed, AttentionArgs* a, lr_attention_plan* out);
// What the call adds to the plan: the kernel that buffers aligned like these take, and its workgroups.
void attention_buffers(const lr_cache* c, const lr_layout* Lq, const void* q, int32_t dtype, int32_t path, AttentionArgs* a);

template <int DT, int CT, int DC, int HT, bool LISTED>
static void launch_matrix(const AttentionArgs& a, dim3 grid, hipStream_t st) {
  if constexpr (LISTED)
    hipLaunchKernelGGL((k_attention_matrix<DT, CT, DC, HT, kOverBlocks>), grid, dim3(256), 0, st, a);
  else if (a.wide_heads > 1)
    hipLaunchKernelGGL((k_attention_matrix<DT, CT, DC, HT, kOverHeads>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_attention_matrix<DT, CT, DC, HT, kOverTokens>), grid, dim3(256), 0, st, a);
}

// Widths that caches of codes have no use for.
template <int DT, int CT, int DC, bool LISTED>
static void launch_plain(const AttentionArgs& a, dim3 grid, hipStream_t st) {
  if constexpr (DT == CT) {
    if constexpr (DC <= 128) {
      if (a.unit_heads == 32) return launch_matrix<DT, CT, DC, 2, LISTED>(a, grid, st);
    }
    launch_matrix<DT, CT, DC, 1, LISTED>(a, grid, st);
  }
}

template <int DT, int CT, int DC, bool LISTED>
static void launch_tiles(const AttentionArgs& a, dim3 grid, hipStream_t st) {
  a.unit_heads == 16 ? launch_matrix<DT, CT, DC, 1, LISTED>(a, grid, st) : launch_matrix<DT, CT, DC, 2, LISTED>(a, grid, st);
}

// The pass over the tokens; what it cuts is left as parts.
template <int DT, int CT, bool LISTED>
static int launch_pass(const AttentionArgs& a, hipStream_t st) {
  const dim3 grid(a.splits == 1 ? a.batch * a.units : a.grid);
  if (a.path == LR_ATTENTION_ELEMENT)
    hipLaunchKernelGGL((k_attention_element<DT, CT>), grid, dim3(256), 0, st, a);
  else if (a.wide == 32)
    launch_plain<DT, CT, 32, LISTED>(a, grid, st);
  else if (a.wide == 64)
    launch_tiles<DT, CT, 64, LISTED>(a, grid, st);
  else if (a.wide == 96)
    launch_plain<DT, CT, 96, LISTED>(a, grid, st);
  else if (a.wide == 128)
    launch_tiles<DT, CT, 128, LISTED>(a, grid, st);
  else if (a.wide == 160)
    launch_plain<DT, CT, 160, LISTED>(a, grid, st);
  else if (a.wide == 192)
    launch_matrix<DT, CT, 192, 1, LISTED>(a, grid, st);
  else
    launch_matrix<DT, CT, 256, 1, LISTED>(a, grid, st);
  return check_op_launch();
}
// The pass of paged attention and of a shared prefix, for a cache of type ctype; the join of its parts.
int launch_attention_pass(const AttentionArgs& a, int32_t dtype, int32_t ctype, hipStream_t st);
int launch_attention_join(const AttentionArgs& a, int32_t dtype, hipStream_t st);

// Calls f<type>() for a model type.
template <class F> static int with_model_type(int32_t dtype, F&& f) {
  if (dtype == LR_F32) return f(std::integral_constant<int, LR_F32>{});
  if (dtype == LR_F16) return f(std::integral_constant<int, LR_F16>{});
  return f(std::integral_constant<int, LR_BF16>{});
}

// The overlaps of a call: every output against every input and the outputs before it.
struct Buffer {
  const void* p;
  int64_t bytes;
};
inline int check_overlaps(const Buffer* in, int inputs, const Buffer* made, int outputs) {
  for (int i = 0; i < outputs; ++i) {
    if (!made[i].p || !made[i].bytes) continue;
    for (int j = 0; j < inputs; ++j)
      if (in[j].p && in[j].bytes && overlap(in[j].p, in[j].bytes, made[i].p, made[i].bytes)) return LR_ERR_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (made[j].p && made[j].bytes && overlap(made[j].p, made[j].bytes, made[i].p, made[i].bytes)) return LR_ERR_OVERLAP;
  }
  return LR_OK;
}

}  // namespace lr
