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
  uint32_t unit_heads, tiles, units;  // query heads of a wave, their tiles in a cache head, units of a sequence
  uint32_t wide_heads, block;         // cache heads of a unit (1, or 4: one a wave); tokens of a block
  uint32_t splits, min_share;         // parts of a unit at most; blocks of a workgroup at least
  uint32_t grid;                      // workgroups (splits > 1; else one a unit)
  int64_t window;
  bool q_wide;   // query rows are contiguous and 16-byte aligned
  bool in_step;  // the four waves of four cache heads keep in step
  float scale2;  // scale * log2 e
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
// heads on 8 of 128: 48 us under a table just wide enough, 127 with 63 runs under one for 131072 tokens).
constexpr int64_t kRuns = 256;                     // one a CU
constexpr uint32_t kBlock = 128, kWideBlock = 32;  // a step of four waves over tokens, or over heads

// The tokens [first, n) a sequence sees; blocks start at `base`, first rounded down so that steps of 32
// tokens stay aligned.  A sequence without tokens has one (empty) block, so that it is written too.
struct Span {
  uint32_t base, first, n, blocks;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& a, int32_t len) {
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t n = len;
  n = n < 0 ? 0 : n > cap ? cap : n;
  const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
  const uint32_t base = (uint32_t)first & ~31u;
  const uint32_t blocks = ((uint32_t)n - base + a.block - 1) / a.block;
  return Span{base, (uint32_t)first, (uint32_t)n, blocks ? blocks : 1};
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
  r->whole = r->at == r->start && r->last;
  r->split = r->whole ? 0 : w - run_of(r->deal, r->start);
  r->lo = r->sp.base + (uint32_t)(r->at - r->start) * a.block;
  const uint64_t hi = (uint64_t)r->sp.base + (stop - r->start) * a.block;
  r->hi = hi < r->sp.n ? (uint32_t)hi : r->sp.n;
}
__device__ __forceinline__ bool run_begin(const AttentionArgs& a, Run* r) {
  const uint32_t lane = threadIdx.x & 63;
  if (a.splits == 1) {  // one unit a workgroup
    r->b = blockIdx.x / a.units;
    r->u = blockIdx.x % a.units;
    r->sp = span_of(a, a.lens[r->b]);
    r->deal = Deal{1, 1};
    r->w = 0;
    r->at = r->start = 0;
    r->end = r->sp.blocks;
  } else {
    int32_t len = lane < a.batch ? a.lens[lane] : 0;
    uint32_t v = lane < a.batch ? span_of(a, len).blocks : 0;
    uint32_t upto = wave_scan(v, lane);  // the first 64 sequences
    uint64_t all = __shfl(upto, 63);
    if (a.batch > 64) {
      uint64_t more = 0;
      for (uint32_t i = 64 + lane; i < a.batch; i += 64) more += span_of(a, a.lens[i]).blocks;
      for (int x = 32; x; x >>= 1) more += __shfl_xor((unsigned long long)more, x);
      all += more;
    }
    r->deal = deal_of(a, all);
    if (blockIdx.x >= r->deal.used) return false;
    // Workgroups go to the eight dies in turn; neighbouring runs, which are often heads of the same tokens, go
    // to one die, whose cache then holds the lines they share: a token's scales for all heads lie in one line
    // (64 x 16384 e4m3 tokens: 466 to 441 us; runs that share no lines are within 1 %).
    r->w = r->deal.used % 8 ? blockIdx.x : blockIdx.x % 8 * (r->deal.used / 8) + blockIdx.x / 8;
    r->at = run_start(r->deal, r->w);
    r->end = run_start(r->deal, r->w + 1);
    uint64_t past = 0;  // blocks of the sequences before the 64 looked at
    for (uint32_t i = 0;; i += 64) {
      const uint64_t hit = __ballot((past + upto) * a.units > r->at);
      if (hit) {
        const int f = __ffsll((unsigned long long)hit) - 1;
        r->b = i + f;
        r->start = (past + uniform(__shfl(upto - v, f))) * a.units;
        r->sp = span_of(a, (int32_t)uniform(__shfl(len, f)));
        break;
      }
      past += uniform(__shfl(upto, 63));
      len = i + 64 + lane < a.batch ? a.lens[i + 64 + lane] : 0;
      v = i + 64 + lane < a.batch ? span_of(a, len).blocks : 0;
      upto = wave_scan(v, lane);
    }
    r->u = (uint32_t)((r->at - r->start) / r->sp.blocks);
    r->start += (uint64_t)r->u * r->sp.blocks;
  }
  run_unit(a, r->w, r);
  return true;
}
__device__ __forceinline__ bool run_next(const AttentionArgs& a, Run* r) {
  r->start += r->sp.blocks;
  r->at = r->start;
  if (r->at >= r->end) return false;
  if (++r->u == a.units) {
    r->u = 0;
    r->sp = span_of(a, a.lens[++r->b]);
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
  if (!run_begin(a, &run)) return;
  do {
    const uint32_t b = run.b, h = run.u, g = h / a.group, bh = b * a.heads + h, split = run.split, hi = run.hi;
    const uint64_t lo = run.lo;
    const Span sp = run.sp;
    __syncthreads();
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
      if (a.splits > 1) leave_part(a, run, bh, top, total);
      if (run.whole && a.lse) a.lse[bh] = lse_of(top, total);
    }
  } while (run_next(a, &run));
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
// (2.15 GB) take 352 us a call, 6.1 TB/s, and 2 of 131071 e4m3 tokens 97 us, 5.7 TB/s, where a bare streaming read
// reaches 7.2 (299 and 77 us); as many fp16 tokens 352 us, 2.21 GB of fp32 (32 sequences, 32 heads) 363 us, 6.1 TB/s,
// and fp32 queries over 0.57 GB of e4m3 234 us, 2.4 TB/s, where the fp32 products are the bound.  The vector units are
// busy 19 % of the first, 37 % of the second, with the matrix units' part.
// One workgroup a CU keeps enough loads under way; two and three a CU (512 and 768 runs) took 359 and 367 us against
// 353, as more rows of memory are open at once.  Plain loads took 20 % longer than streaming ones.
template <int DT, int CT, int DC, int HT, bool by_heads>
__global__ void __launch_bounds__(256, (MatrixShape<DT, CT, DC, HT>::kMinWaves)) k_attention_matrix(AttentionArgs a) {
  using S = MatrixShape<DT, CT, DC, HT>;
  using T = typename ElemOf<DT>::T;
  using M = typename MatrixOf<DT>::T;
  typedef U4 KR __attribute__((aligned(8)));  // rows of 8-bit caches are aligned to 8 elements
  typedef typename Raw<8>::T KHalf;
  using VR = typename Raw<S::kValChunk * S::kElem>::T;
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  constexpr int kRow = 16 * S::kValChunk + 4;  // floats; the 4 keep 16 heads' accesses off one bank
  __shared__ int64_t offs_all[4][64];
  __shared__ __attribute__((aligned(16))) float scale_all[4][64];
  constexpr int kJoin = by_heads ? 1 : 16;  // four heads are not joined
  __shared__ float ms[4][kJoin * HT], ls[4][kJoin * HT];
  __shared__ __attribute__((aligned(16))) float os[4][kJoin * kRow];
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64), r = lane & 15, j = lane >> 4;
  int64_t* offs = offs_all[w];
  float* scales = scale_all[w];

  Run run;
  if (!run_begin(a, &run)) return;
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
    const T* qb = (const T*)a.q + (int64_t)b * a.qb + (int64_t)(g * a.group) * a.qh;
    auto load_queries = [&](auto wide) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const uint32_t h = in_group + 16 * ht + rq;
        const T* x = qb + (int64_t)(h < a.group ? h : 0) * a.qh;
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
    auto page_of = [&](uint32_t t0) -> int32_t {
      const uint32_t t = t0 + li;
      return table[page_index(t < hi ? t : hi - 1)];
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
          if (a.splits > 1) leave_part(a, run, bh, top, total);
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
              if (a.splits > 1) leave_part(a, run, bh, top, total);
              if (run.whole && a.lse) a.lse[bh] = lse_of(top, total);
            }
          }
        }
    }
    if (!run_next(a, &run)) break;
  }
}

// 4096 heads: 6 us; 32 heads: 4 us, most of it the launch.
//
// Joins the parts of one query head: a wave has the weights of 64 parts at a time, one a lane; 256 lanes are
// groups of lanes with four columns each, a group takes every next part, and the groups' sums are added in
// their order.
template <int DT>
__global__ void __launch_bounds__(256) k_attention_join(AttentionArgs a) {
  using T = typename ElemOf<DT>::T;
  typedef float F2 __attribute__((ext_vector_type(2)));
  __shared__ __attribute__((aligned(16))) float os[256 * 4];
  const uint32_t bh = blockIdx.x, lane = threadIdx.x & 63;
  const uint32_t wide = ((uint32_t)a.dv + 3) / 4, groups = 256 / wide, grp = threadIdx.x / wide, c = threadIdx.x % wide;
  const F2* ml = (const F2*)a.part_ml + (uint64_t)bh * a.splits;
  const float* po = a.part_o + (uint64_t)bh * a.splits * a.dv + 4 * c;
  float top = -__builtin_inff(), total = 0;
  F4 acc = {};
  for (uint32_t s = 0; s < a.splits; s += 64) {
    F2 x = {-__builtin_inff(), 0.f};
    if (s + lane < a.splits) x = ml[s + lane];
    const uint64_t hit = __ballot(__float_as_uint(x[1]) >> 31);  // what is past the last part means nothing
    const uint32_t parts = hit ? __ffsll((unsigned long long)hit) : 64;
    if (s == 0 && parts == 1) return;  // whole: written already
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
    for (uint32_t q = 0; q < parts; q += groups) {
      const uint32_t p = q + grp;
      const float w = __shfl(wt, p & 63);
      if (p >= parts || grp >= groups) continue;
      const float* y = po + (uint64_t)(s + p) * a.dv;
      if (a.dv % 4 == 0) {
        acc += *(const F4*)y * w;
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          if (4 * c + i < (uint32_t)a.dv) acc[i] += y[i] * w;
      }
    }
    if (hit) break;
  }
  *(F4*)&os[4 * threadIdx.x] = acc;
  __syncthreads();
  if (grp) return;
  for (uint32_t i = 1; i < groups; ++i) acc += *(const F4*)&os[4 * (i * wide + c)];
  const uint32_t b = bh / a.heads, h = bh % a.heads;
  T* out = (T*)a.out + (int64_t)b * a.ob + (int64_t)h * a.oh;
  const float inv = total > 0 ? 1.f / total : 0.f;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    if (4 * c + i < (uint32_t)a.dv) out[(int64_t)(4 * c + i) * a.od] = (T)(total != total ? total : acc[i] * inv);
  if (c == 0 && a.lse) a.lse[bh] = lse_of(top, total);
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
  a->unit_heads = !matrix ? 1 : a->group > 16 && a->wide <= 128 ? 32 : 16;
  a->tiles = (a->group + a->unit_heads - 1) / a->unit_heads;
  // Four cache heads a workgroup, one a wave, where a token's heads lie next to each other: their rows then share
  // lines and pages of memory (16 sequences of up to 30000 tokens, 8 heads: 174 us against 198 in bf16 of 128, 73
  // against 111 in e4m3 of 64).  Where a head's tokens lie next to each other, the four waves take tokens of one
  // head; also where a run would be under 8 steps, as four heads leave four times the parts to join (one sequence of
  // 4000 tokens: 16 us against 21).
  const int64_t ktok = std::abs(ks.size > 1 ? a->ksl : a->kp), vtok = std::abs(ks.size > 1 ? a->vsl : a->vp);
  out->head_tiles = (int32_t)a->tiles;
  // Parts of a sequence: short ones stay whole, which saves the second launch; otherwise as many as there
  // are blocks, up to 8192 parts in all (their sums are some 66 MB for 16 heads of 128), or 8 a unit.
  int64_t span = max_pages * ks.size;
  if (window > 0) span = std::min(span, window + 31);
  const int64_t steps = (int64_t)((double)qb.size * a->kv_heads / 4 * a->tiles * (double)((span + 31) / 32));
  const bool by_heads = matrix && a->kv_heads % 4 == 0 && std::abs(a->kh) < ktok && std::abs(a->vh) < vtok &&
                        span <= (int64_t(1) << 30) && steps >= 8 * kRuns;
  a->wide_heads = by_heads ? 4 : 1;
  // Heads that end inside a line: their waves keep in step, so that the line is still near for the second of them
  // (as above: heads of 72 in bf16 153 to 144 us, of 112 201 to 185, of 160 265 to 254).  Heads of 64 would lose 6 %
  // by it and whole lines up to 1 %; codes of 80 to 192 gain 2 to 4 %, but lose as much with heads of up to 64.
  a->in_step = by_heads && kd.size > 64 && kd.size % 64;
  a->block = by_heads ? kWideBlock : kBlock;
  a->units = a->kv_heads / a->wide_heads * a->tiles;
  const int64_t blocks = (span + a->block - 1) / a->block;
  const double units = (double)qb.size * a->units;
  int64_t most = blocks <= 4 ? 1 : std::min(blocks, std::max<int64_t>((int64_t)(8192 / units), 8));
  out->chunk = (span + most - 1) / most;
  out->splits = (span + out->chunk - 1) / out->chunk;
  const double parts = (double)qb.size * a->heads * (double)out->splits;
  if (parts > (double)kMaxCount / 256 || units > (double)kMaxCount || units * blocks > 0x1p50) return LR_ERR_OVERFLOW;
  a->min_share = out->splits > 1 ? (uint32_t)((blocks - 2) / (out->splits - 1) + 1) : 1;
  out->workspace_bytes = out->splits == 1 ? 0 : (int64_t)parts * (a->dv + 2) * 4;
  a->splits = (uint32_t)out->splits;
  return LR_OK;
}

template <int DT, int CT, int DC, int HT>
static void launch_matrix(const AttentionArgs& a, dim3 grid, hipStream_t st) {
  if (a.wide_heads > 1)
    hipLaunchKernelGGL((k_attention_matrix<DT, CT, DC, HT, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_attention_matrix<DT, CT, DC, HT, false>), grid, dim3(256), 0, st, a);
}

// Widths that caches of codes have no use for.
template <int DT, int CT, int DC>
static void launch_plain(const AttentionArgs& a, dim3 grid, hipStream_t st) {
  if constexpr (DT == CT) {
    if constexpr (DC <= 128) {
      if (a.unit_heads == 32) return launch_matrix<DT, CT, DC, 2>(a, grid, st);
    }
    launch_matrix<DT, CT, DC, 1>(a, grid, st);
  }
}

template <int DT, int CT>
static int launch_attention(const AttentionArgs& a, hipStream_t st) {
  const dim3 grid(a.splits == 1 ? a.batch * a.units : a.grid);
  if (a.path == LR_ATTENTION_ELEMENT) {
    hipLaunchKernelGGL((k_attention_element<DT, CT>), grid, dim3(256), 0, st, a);
  } else {
    if (a.wide == 32)
      launch_plain<DT, CT, 32>(a, grid, st);
    else if (a.wide == 64)
      a.unit_heads == 16 ? launch_matrix<DT, CT, 64, 1>(a, grid, st) : launch_matrix<DT, CT, 64, 2>(a, grid, st);
    else if (a.wide == 96)
      launch_plain<DT, CT, 96>(a, grid, st);
    else if (a.wide == 160)
      launch_plain<DT, CT, 160>(a, grid, st);
    else if (a.wide == 128)
      a.unit_heads == 16 ? launch_matrix<DT, CT, 128, 1>(a, grid, st) : launch_matrix<DT, CT, 128, 2>(a, grid, st);
    else if (a.wide == 192)
      launch_matrix<DT, CT, 192, 1>(a, grid, st);
    else
      launch_matrix<DT, CT, 256, 1>(a, grid, st);
  }
  if (int rc = check_op_launch()) return rc;
  if (a.splits == 1) return LR_OK;
  hipLaunchKernelGGL((k_attention_join<DT>), dim3(a.batch * a.heads), dim3(256), 0, st, a);
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
  const uintptr_t align = is_quantised(c->dtype) ? 8 : 16;
  a.path = p.path;
  if (a.path == LR_ATTENTION_MATRIX && ((uintptr_t)c->k % align || (uintptr_t)c->v % align)) {
    a.path = LR_ATTENTION_ELEMENT;
    a.unit_heads = 1;
    a.wide_heads = 1;
    a.block = kBlock;
    a.tiles = a.group;
    a.units = a.heads;
  }
  a.q_wide = rows_aligned(*Lq, q, e, 16 / e);
  // Two workgroups a CU where a step is too short for one to keep enough loads under way: rows of 64 bytes 74 us with
  // one, 60 with two; of 80 bytes 89 and 84; of 128 bytes 91 and 95.  Four heads at once ask for enough.
  const bool small_step = a.wide_heads == 1 && (a.dk + a.dv) * ce <= 192;
  a.grid = (uint32_t)(a.path == LR_ATTENTION_ELEMENT ? 8 * kRuns : small_step ? 2 * kRuns : kRuns);
  const hipStream_t st = (hipStream_t)stream;
  if (dtype == LR_F32) return launch_attention_of<LR_F32>(a, c->dtype, st);
  if (dtype == LR_F16) return launch_attention_of<LR_F16>(a, c->dtype, st);
  return launch_attention_of<LR_BF16>(a, c->dtype, st);
}

}  // extern "C"
