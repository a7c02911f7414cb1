// Attention of a batch that shares a prefix: lr_prefix_attention_plan and lr_prefix_attention.
//
// The softmax over a sequence's tokens is split at the prefix's end: one pass over the prefix serves all sequences, whose
// query heads of one cache head are the rows of one product with its keys; a second pass takes each sequence's own
// tokens; parts (m, l, o) of both are joined by the rule that joins the parts of one sequence.
#include "attention.h"

namespace lr {

// ------------------------------------------------------------------ many rows on one prefix

typedef float F16x __attribute__((ext_vector_type(16)));
typedef short S4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) S4 LdsS4;
typedef uint32_t U2 __attribute__((ext_vector_type(2)));
typedef unsigned short W2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ F16x mfma32(B8 a, B8 b, F16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ F16x mfma32(H8 a, H8 b, F16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

constexpr uint32_t kTileTokens = 64, kPitch = 256;  // of a step; bytes of a row in shared memory

// Where chunk c (16 bytes) of a row lies in its 256 bytes of shared memory: 16 rows' chunks of one number spread over
// all banks, for the keys' operand, and 4 rows' groups of four chunks, for the values' (4 cycles of a read for each;
// the row's number itself in place of its halves swapped: 8 for the values').
__device__ __forceinline__ uint32_t place_in_row(uint32_t row, uint32_t c) {
  return row * kPitch + (c ^ ((row & 3) << 2 | (row >> 2 & 3))) * 16;
}

// 128 or 256 rows (query heads of one cache head, of all sequences) share the keys and values of a run of tokens: a
// workgroup of four or eight waves brings 64 tokens at a time to shared memory, 8-bit codes as 16-bit numbers, while
// its waves work on the 64 before, 32 rows each.  The scores of 32 tokens x 32 rows are a product of keys (first operand,
// from shared memory) and queries (in registers), so that a lane has scores of one row alone: its maximum and sum need
// one exchange.  They are also the second operand of the next product, values transposed x weights, when its inner index
// runs over the tokens as they lie in the lane; the values' operand comes by transpose reads of shared memory.
//
// What bounds it is that vector and matrix instructions take turns: a SIMD's two waves go from barrier to barrier through
// products, exponentials and products in step.  8192 rows on 32768 tokens (8 cache heads of 128 bf16, 137 GFLOP) 212 us,
// 648 TFLOP/s, where a large library product reaches 1270; with the second part of the weights the matrix units do
// half as much again.  They are busy 48 % of it, the vector units 56 %: all of it together, where both at once could be
// less.  With four waves (244 us, 44 % and 55 %) leaving out that part saved 47 us, the exponentials 15, bringing tiles 38.
template <int CT, int WAVES> struct RowsShared {
  __attribute__((aligned(16))) char keys[2 * kTileTokens * kPitch], values[2 * kTileTokens * kPitch];  // two tiles each
  __attribute__((aligned(16))) int64_t offs[WAVES][kTileTokens][2];
  __attribute__((aligned(16))) float scales[CT == LR_E4M3 || CT == LR_INT8 ? WAVES : 1][2][2][kTileTokens];
  // of each tile, whether the values that a wave brought hold an infinity or a NaN
  __attribute__((aligned(16))) uint32_t odd[2][CT == LR_E4M3 || CT == LR_INT8 ? 1 : WAVES];
};
template <int DT, int CT, int DC, int WAVES>
__device__ __forceinline__ void rows_run(const AttentionArgs& a, uint32_t block, RowsShared<CT, WAVES>& shared) {
  constexpr int kRows = 16 / WAVES, kApart = 4 * WAVES;  // rows of a tile that a lane brings a chunk of, and their distance
  using T = typename ElemOf<DT>::T;
  using M = typename MatrixOf<DT>::T;  // 8 numbers of the model's type
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  constexpr int kElem = kQuant ? 1 : 2, kKeySteps = DC / 16, kValSteps = DC / 32;
  // weights meet the values in the model's type, in bf16 where those are codes
  using P = std::conditional_t<kQuant, B8, M>;
  using PE = std::conditional_t<kQuant, __bf16, T>;
  using CT8 = std::conditional_t<kQuant, U2, U4>;  // 8 elements of the cache
  constexpr uint32_t kTile = kTileTokens * kPitch;
  char *keys = shared.keys, *values = shared.values;
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64), r = lane & 31, half = lane >> 5;
  auto offs = shared.offs[w];
  auto scales = shared.scales[kQuant ? w : 0];
  const uint32_t row0 = threadIdx.x / 16, chunk = threadIdx.x % 16;  // of the rows row0 + kApart x this lane brings one chunk
  // Where this lane reads its operands: of the keys row r, of the values four columns of a token (below).  The other
  // chunks of the row are at the same place but for bits 5 to 7, in which their numbers differ.
  const uint32_t key_at = place_in_row(r, half), val_row = 4 * half + (lane & 15) / 4;
  uint32_t val_at[2];
#pragma unroll
  for (int y = 0; y < 2; ++y)
    val_at[y] = place_in_row(val_row + 8 * y, 2 * (lane >> 4 & 1) + (lane & 3) / 2) + (lane & 1) * 8;
  const bool key_chunk = chunk * 8 < (uint32_t)a.dk, val_chunk = chunk * 8 < (uint32_t)a.dv;

  // Scores times `unit` are in base-2 units: the scale where tokens have none of their own, its sign in the queries so
  // that the largest product is the largest score.
  const float sign = a.scale2 < 0 ? -1.f : a.scale2 > 0 ? 1.f : 0.f;
  const float unit = kQuant || a.scale2 == 0 ? 1.f : __builtin_fabsf(a.scale2);

  Run run;
  if (!run_begin<false>(a, block, &run)) return;
  do {
    const uint32_t g = run.u / a.tiles, tile0 = run.u % a.tiles * (32 * WAVES) + w * 32, row = tile0 + here(r);
    const uint32_t lo = run.lo, hi = run.hi;
    const bool idle = tile0 >= a.group;

    M q[kKeySteps];
    {
      const uint32_t hq = here(half);
      const T* x = (const T*)a.q + query_at(a, run.b, g, row < a.group ? row : 0);
#pragma unroll
      for (int kk = 0; kk < kKeySteps; ++kk) {
        const uint32_t e0 = kk * 16 + hq * 8, e = e0 < (uint32_t)a.dk ? e0 : 0;
        if (a.q_wide) {
          q[kk] = *(const M*)(x + e);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[kk][i] = x[(int64_t)(e + i) * a.qd];
        }
        if (row >= a.group || e0 >= (uint32_t)a.dk) q[kk] = M{};
        if constexpr (!kQuant) q[kk] *= (T)sign;
      }
    }

    const char* kbase = (const char*)a.k + ((int64_t)g * a.kh + (key_chunk ? chunk * 8 : 0)) * kElem;
    const char* vbase = (const char*)a.v + ((int64_t)g * a.vh + (val_chunk ? chunk * 8 : 0)) * kElem;
    const uint32_t one = a.fd_page.m ? 0 : ~0u;  // pages of one slot: the quotient is the dividend
    auto page_index = [&](uint32_t t) -> uint32_t { return (__umulhi(t, a.fd_page.m) >> a.fd_page.s) + (t & one); };
    // Lane l's page of token t0 + l; loads past the end are of the last token's, and left out after.
    auto page_of = [&](uint32_t t0) -> int32_t { return a.table[page_index(t0 + lane < hi ? t0 + lane : hi - 1)]; };
    // Row offsets to shared memory (the cache's first row for what is not seen); returns the mask of the seen tokens.
    auto place = [&](uint32_t t0, int32_t page, float* ks, float* vs) -> uint64_t {
      const uint32_t t = t0 + lane;
      const bool ok = (t < hi) & ((uint32_t)page < a.pages);
      const uint32_t in = ok ? t - page_index(t) * a.page_size : 0, pg = ok ? page : 0;
      wave_fence();
      offs[lane][0] = (int64_t)(pg * (uint64_t)a.kp + in * (uint64_t)a.ksl) * kElem;
      offs[lane][1] = (int64_t)(pg * (uint64_t)a.vp + in * (uint64_t)a.vsl) * kElem;
      wave_fence();
      if constexpr (kQuant) {
        const uint64_t at = pg * (uint64_t)a.sp + in * (uint64_t)a.ssl + (uint64_t)g * a.sh;
        *ks = ok ? a.ks[at] * a.scale2 : 0.f;
        *vs = ok ? a.vs[at] : 0.f;
      }
      return __ballot(ok);
    };
    CT8 kr[kRows], vr[kRows];
    uint32_t bad = 0;  // of this lane's rows, those not seen
    auto load = [&](uint64_t seen) {
      bad = 0;
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        const uint32_t t = row0 + kApart * x;
        kr[x] = *(const CT8*)(kbase + offs[t][0]);
        vr[x] = *(const CT8*)(vbase + offs[t][1]);
        bad |= (uint32_t)(~(seen >> t) & 1) << x;
      }
    };
    auto store = [&](uint32_t buf) {
      W2 most = {};  // of the values' upper bits, without signs
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        const uint32_t at = place_in_row(row0 + kApart * x, chunk);
        U4 k, v;
        if constexpr (kQuant) {
          k = __builtin_bit_cast(U4, decode<DT, CT>(kr[x]));
          v = __builtin_bit_cast(U4, decode<LR_BF16, CT>(vr[x]));
        } else {
          k = kr[x];
          v = vr[x];
        }
        if (!key_chunk) k = U4{};
        if (bad >> x & 1) v = U4{};  // what is not seen may hold NaN
        *(U4*)&keys[buf * kTile + at] = k;
        *(U4*)&values[buf * kTile + at] = v;
        if constexpr (!kQuant)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            most = __builtin_elementwise_max(most, __builtin_bit_cast(W2, v[y] & 0x7fff7fffu));
      }
      if constexpr (!kQuant) {
        constexpr unsigned short kInf = DT == LR_F16 ? 0x7c00 : 0x7f80;
        const bool any = __any(most[0] >= kInf || most[1] >= kInf);
        if (lane == 0) shared.odd[buf][w] = any;
      }
    };

    F16x o[kValSteps];
#pragma unroll
    for (int d = 0; d < kValSteps; ++d) o[d] = F16x{};
    // Scores are taken off `base`, at most 8 below the running maximum; weights in fp16 parts off a base 7 to 15 below
    // it, so that one of 2^-32 of the largest still counts.
    constexpr float kLow = std::is_same_v<PE, _Float16> ? 7.f : 0.f;
    float base = -__FLT_MAX__, l = 0;
    if (lo < hi) {
      float ks[2] = {}, vs[2] = {};
      uint64_t seen = place(lo, page_of(lo), &ks[0], &vs[0]);
      load(seen);
      int32_t page = page_of(lo + kTileTokens);
      store(0);
      if constexpr (kQuant) scales[0][0][lane] = ks[0], scales[0][1][lane] = vs[0];
      uint64_t seen_next = place(lo + kTileTokens, page, &ks[1], &vs[1]);
      load(seen_next);
      page = page_of(lo + 2 * kTileTokens);
      __syncthreads();
      uint32_t buf = 0;
      for (uint32_t t0 = lo; t0 < hi; t0 += kTileTokens, buf ^= 1) {
        store(buf ^ 1);
        if constexpr (kQuant) scales[buf ^ 1][0][lane] = ks[1], scales[buf ^ 1][1][lane] = vs[1];
        const uint64_t seen_after = place(t0 + 2 * kTileTokens, page, &ks[1], &vs[1]);
        load(seen_after);
        page = page_of(t0 + 3 * kTileTokens);
        if (!idle) {
          uint32_t odd = 0;
          if constexpr (!kQuant) {
            U4 any = *(const U4*)&shared.odd[buf][0];
            if constexpr (WAVES == 8) any |= *(const U4*)&shared.odd[buf][4];
            odd = uniform(any[0] | any[1] | any[2] | any[3]);
          }
#pragma unroll 1
          for (uint32_t tt = 0; tt < 2; ++tt) {
            const uint32_t from = buf * kTile + tt * 32 * kPitch;
            const uint32_t mask = (uint32_t)(seen >> (32 * tt));
            // Operands are read ahead of the products that need them, by addresses made here: kept over the loop, they
            // would take the registers for that.
            const uint32_t kp = here(from + key_at), vp[2] = {here(from + val_at[0]), here(from + val_at[1])};
            auto key = [&](int kk) -> M { return __builtin_bit_cast(M, *(const U4*)&keys[kp ^ 32 * kk]); };
            // Column 32 d + r of this lane in the tokens 16 z + 4 half + (0 .. 3) and 8 further: a lane addresses four columns
            // of one token, and receives its own column of the tokens that its group of 16 lanes addresses.
            auto value = [&](int d, int z) -> U4 {
              U4 v;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const char* at = &values[(vp[y] ^ 64 * d) + 16 * z * kPitch];
                const U2 x = __builtin_bit_cast(U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4*)const_cast<char*>(at)));
                v[2 * y] = x[0], v[2 * y + 1] = x[1];
              }
              return v;
            };
            F16x s = {};
            M k0 = key(0), k1 = key(1);
#pragma unroll
            for (int kk = 0; kk < kKeySteps; ++kk) {
              const M k2 = kk + 2 < kKeySteps ? key(kk + 2) : k1;
              s = mfma32(k0, q[kk], s);
              k0 = k1, k1 = k2;
            }
            U4 v0 = value(0, 0), v1 = value(0, 1);
            // element i is token 8 (i / 4) + 4 half + i % 4 of the 32
            F4 vsc[4];
            if constexpr (kQuant) {
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const F4 ksc = *(const F4*)&scales[buf][0][32 * tt + 8 * z + 4 * half];
                vsc[z] = *(const F4*)&scales[buf][1][32 * tt + 8 * z + 4 * half];
#pragma unroll
                for (int i = 0; i < 4; ++i) s[4 * z + i] *= ksc[i];
              }
            }
            if (mask != ~0u)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                s[i] = mask >> (8 * (i / 4) + 4 * half + i % 4) & 1 ? s[i] : -__builtin_inff();
            float top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
            top *= unit;
            if (__any(top > base + (8.f + kLow))) {
              top = fmaxf(base, fmaxf(top, __shfl_xor(top, 32)) - kLow);
              const float keep = __builtin_amdgcn_exp2f(base - top);
              base = top;
              l *= keep;
#pragma unroll
              for (int d = 0; d < kValSteps; ++d) o[d] *= keep;
            }
            // The weights in two 16-bit parts as in k_attention_matrix: the number, rounded, and what that left.  The second
            // may be zero or negative, and meets finite values; which tiles hold others is found as they are brought (first
            // parts cut off, whose rests are never negative, need no finite values, but have a bit less; finite values
            // made in every tile take 344 us where prefix large takes 321).
            U4 phi[2], plo[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float x[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                x[y] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + y], unit, -base));
                l += x[y];
                if constexpr (kQuant) x[y] *= vsc[i / 4][i % 4 + y];
              }
              uint32_t up, rest;  // pairs, converted together
              if constexpr (std::is_same_v<PE, _Float16>) {
                const H2 z = {(PE)fmaxf(x[0], 0x1p-24f), (PE)fmaxf(x[1], 0x1p-24f)};
                up = __builtin_bit_cast(uint32_t, z);
                rest = __builtin_bit_cast(uint32_t, H2{(PE)(x[0] - (float)z[0]), (PE)(x[1] - (float)z[1])});
              } else {
                up = __builtin_bit_cast(uint32_t, __builtin_convertvector((F2{x[0], x[1]}), B2));
                const F2 left = {x[0] - __uint_as_float(up << 16), x[1] - __uint_as_float(up & 0xffff0000u)};
                rest = __builtin_bit_cast(uint32_t, __builtin_convertvector(left, B2));
              }
              phi[i / 8][i % 8 / 2] = up, plo[i / 8][i % 8 / 2] = rest;
            }
#pragma unroll
            for (int d = 0; d < kValSteps; ++d) {
              U4 n0 = v0, n1 = v1;
              if (d + 1 < kValSteps) n0 = value(d + 1, 0), n1 = value(d + 1, 1);
              o[d] = mfma32(__builtin_bit_cast(P, v0), __builtin_bit_cast(P, phi[0]), o[d]);
              o[d] = mfma32(__builtin_bit_cast(P, v1), __builtin_bit_cast(P, phi[1]), o[d]);
              if (!kQuant && odd)
#pragma unroll
                for (int y = 0; y < 4; ++y) v0[y] = finite_pair<DT>(v0[y]), v1[y] = finite_pair<DT>(v1[y]);
              o[d] = mfma32(__builtin_bit_cast(P, v0), __builtin_bit_cast(P, plo[0]), o[d]);
              o[d] = mfma32(__builtin_bit_cast(P, v1), __builtin_bit_cast(P, plo[1]), o[d]);
              v0 = n0, v1 = n1;
            }
          }
        }
        seen = seen_next;
        seen_next = seen_after;
        __syncthreads();
      }
    }
    const float total = l + __shfl_xor(l, 32);
    if (row < a.group) {
      const uint32_t he = here(half);
      const uint64_t at = (uint64_t)(g * a.group + row) * a.splits + run.split;
#pragma unroll
      for (int d = 0; d < kValSteps; ++d)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t e = 32 * d + 8 * z + 4 * he;
          if (e < (uint32_t)a.dv)
            *(F4*)&a.part_o[at * a.dv + e] = F4{o[d][4 * z], o[d][4 * z + 1], o[d][4 * z + 2], o[d][4 * z + 3]};
        }
      if (he == 0) leave_part(a, run, g * a.group + row, base == -__FLT_MAX__ ? -__builtin_inff() : base, total);
    }
  } while (run_next<false>(a, &run));
}

template <int DT, int CT, int DC, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 2) k_prefix_rows(AttentionArgs a) {
  __shared__ RowsShared<CT, WAVES> shared;
  rows_run<DT, CT, DC, WAVES>(a, blockIdx.x, shared);
}

// Both passes in one launch where one workgroup a CU has the prefix: the first `first` workgroups.  The others have the
// sequences' own tokens, whose bound is the reading of them, on the other half of each CU (32 sequences of up to 1024 tokens
// behind 8191: 51 us with a launch for each pass, 40 this way).
template <int DT, int CT, int DC, int OWN>
__global__ void __launch_bounds__(256, 2) k_prefix_mixed(AttentionArgs prefix, AttentionArgs own, uint32_t first) {
  constexpr int kOwn = DC == 96 && (CT == LR_E4M3 || CT == LR_INT8) ? 128 : DC;
  __shared__ union {
    RowsShared<CT, 4> rows;
    MatrixShared<DT, CT, kOwn, 1, OWN> matrix;
  } shared;
  if (blockIdx.x < first)
    rows_run<DT, CT, DC, 4>(prefix, blockIdx.x, shared.rows);
  else
    attention_run<DT, CT, kOwn, 1, OWN>(own, blockIdx.x - first, shared.matrix);
}

// Both passes in one launch, for calls whose time is mostly that of launches: the first `first` workgroups have the
// prefix, the others the sequences' own tokens.  4 sequences of up to 60 tokens behind 1000, 32 heads on 8 of 128 bf16:
// 8.7 us, 8.2 and 5.7 with a launch for each.
template <int DT, int CT, int DC>
__global__ void __launch_bounds__(256, (MatrixShape<DT, CT, DC, 1>::kMinWaves)) k_prefix_pair(
    AttentionArgs prefix, AttentionArgs own, uint32_t first) {
  __shared__ MatrixShared<DT, CT, DC, 1, kOverTokens> shared;
  if (blockIdx.x < first)
    attention_run<DT, CT, DC, 1, kOverTokens>(prefix, blockIdx.x, shared);
  else
    attention_run<DT, CT, DC, 1, kOverTokens>(own, blockIdx.x - first, shared);
}

struct PrefixJoin {
  const float *ml, *o;  // parts of the prefix, for row b * group + r of cache head g: (g, row, split)
  uint32_t splits, group, batch;
  FastDiv fd_group;
};

// LANES lanes a query head: a workgroup, as k_attention_join, whose four waves go over the weights each; or a wave where
// heads are many enough to keep the device busy so.  In us, by workgroups and by waves, of some 12 parts of 128 bf16 a
// head: 1024 heads 7.2 and 11.2, 2048 10.6 and 11.6, 2560 11 and 10.7 (of 96, 34 parts; of 64 9 and 6.4), 4096 14 and 10.3,
// 8192 21.7 and 12 (3.7 TB/s).
constexpr uint32_t kManyHeads = 10 * kRuns;
template <int DT, int LANES>
__global__ void __launch_bounds__(256) k_prefix_join(AttentionArgs a, PrefixJoin p) {
  __shared__ __attribute__((aligned(16))) float os[256 * 4];
  const uint32_t w = LANES == 64 ? uniform(threadIdx.x / 64) : 0, bh = blockIdx.x * (256 / LANES) + w;
  if (bh >= a.batch * a.heads) return;
  const uint32_t b = bh / a.heads, h = bh - b * a.heads, g = op_div(h, p.fd_group);
  const Columns q4 = columns_of<LANES>(a.dv);
  const uint64_t own = (uint64_t)bh * a.splits;
  const uint64_t pre = ((uint64_t)(g * p.batch + b) * p.group + (h - g * p.group)) * p.splits;
  Joined j{-__builtin_inff(), 0.f, F4{}};
  const float *ml = p.ml + 2 * pre, *ml2 = a.part_ml + 2 * own;
  const F2 x = part_at(ml, 0, p.splits), x2 = part_at(ml2, 0, a.splits);  // both lists' first, side by side
  const bool blank = a.lens[b] < 0;
  join_list(x, ml, p.o + pre * a.dv, p.splits, a.dv, q4, false, &j);
  join_list(x2, ml2, a.part_o + own * a.dv, a.splits, a.dv, q4, false, &j);
  join_out<DT, LANES>(a, b, h, q4, j, blank, os + 4 * LANES * w);
}

// From so many rows of a cache head on they share what a workgroup brings to shared memory, if there is work enough for
// that to pay.  32 query heads on 8 of 128 bf16, in us with k_attention_matrix and with k_prefix_rows: 64 rows on 8191
// tokens 30 and 33, on 65536 109 and 80; 96 on 8191 39 and 35; 128 on 1000 24 and 26; 192 on 1000 31 and 29, on 65536
// 270 and 131; 32 rows on 65536 69 and 73.  Over e4m3 the lines cross at the same places.
constexpr uint32_t kManyRows = 64;
constexpr int64_t kEnoughWork = 600000, kEnoughCodes = 1 << 20;  // rows times tokens
static bool much_work(const AttentionArgs& x, int32_t ctype) {
  return (int64_t)x.group * x.max_pages * x.page_size >= (is_quantised(ctype) ? kEnoughCodes : kEnoughWork);
}

// Whether k_prefix_rows takes such a call: 16-bit products, heads of up to 128.
static bool rows_fit(const AttentionArgs& a, int32_t dtype) {
  return a.path == LR_ATTENTION_MATRIX && dtype != LR_F32 && a.dk <= 128 && a.dv <= 128;
}
// How the prefix's pass runs: by k_prefix_rows in workgroups of so many waves, by k_prefix_pair, or as that of a batch
// of one sequence; and whether the sequences' own tokens go along in its launch.
struct PrefixWay {
  enum { kRows, kPair, kAlone } how;
  uint32_t waves;
  bool mixed;
};
// Chooses it, and sets the tiles and runs that go with it.
static PrefixWay prefix_way(int32_t dtype, int32_t ctype, AttentionArgs* x, AttentionArgs* a) {
  const bool matrix = x->path == LR_ATTENTION_MATRIX && a->path == LR_ATTENTION_MATRIX;
  if (rows_fit(*x, dtype) && x->group >= kManyRows && much_work(*x, ctype)) {
    // Eight waves share a tile's staging (1024 rows on 32768 tokens 244 us with four, 204 with eight), but four where that
    // spares codes, whose staging costs more, half a tile of rows that are none (384 rows on 65536: 218 and 236).  Where
    // one workgroup of four waves a CU has no more than 8 blocks of 128 tokens (5 of codes), the other half of the CU takes
    // the sequences' own tokens in the same launch (up to 64 each: 128 rows on 8191 tokens 38 us without and 29 with, 512
    // rows 65 and 58, 256 rows on 30000 82 and 84; over e4m3 256 rows on 8191 47 and 42, on 16000 60 and 63).
    const uint32_t fours = (x->group + 127) / 128;
    const int64_t blocks = (int64_t)x->kv_heads * fours * ((int64_t)x->max_pages * x->page_size / kBlock);
    const bool mixed = blocks <= (is_quantised(ctype) ? 5 : 8) * kRuns && matrix && a->unit_heads == 16;
    const uint32_t waves = !mixed && fours > 1 && !(is_quantised(ctype) && fours % 2) ? 8 : 4;
    x->tiles = waves == 8 ? (fours + 1) / 2 : fours;
    x->units = x->kv_heads * x->tiles;
    x->wide_heads = 1;
    x->block = kBlock;
    x->grid = (uint32_t)(waves == 8 || mixed ? kRuns : 2 * kRuns);
    return {PrefixWay::kRows, waves, mixed};
  }
  if (!matrix || much_work(*x, ctype) || x->wide_heads > 1 || a->wide_heads > 1) return {PrefixWay::kAlone, 4, false};
  for (AttentionArgs* y : {x, a}) {
    y->unit_heads = 16;
    y->tiles = (y->group + 15) / 16;
    y->units = y->kv_heads * y->tiles;
  }
  return {PrefixWay::kPair, 4, true};
}
template <int DT, int CT, int DC>
static int launch_rows_wide(const AttentionArgs& x, const AttentionArgs& a, PrefixWay how, hipStream_t st) {
  const unsigned grid = x.splits == 1 ? x.units : x.grid, second = a.splits == 1 ? a.batch * a.units : a.grid;
  if (how.mixed && a.wide_heads > 1)
    hipLaunchKernelGGL((k_prefix_mixed<DT, CT, DC, kOverHeads>), dim3(grid + second), dim3(256), 0, st, x, a, grid);
  else if (how.mixed)
    hipLaunchKernelGGL((k_prefix_mixed<DT, CT, DC, kOverTokens>), dim3(grid + second), dim3(256), 0, st, x, a, grid);
  else if (how.waves == 8)
    hipLaunchKernelGGL((k_prefix_rows<DT, CT, DC, 8>), dim3(grid), dim3(512), 0, st, x);
  else
    hipLaunchKernelGGL((k_prefix_rows<DT, CT, DC, 4>), dim3(grid), dim3(256), 0, st, x);
  return check_op_launch();
}
template <int DT, int CT>
static int launch_rows_of(const AttentionArgs& x, const AttentionArgs& a, PrefixWay how, hipStream_t st) {
  const int32_t widest = std::max(a.dk, a.dv);
  return widest <= 64   ? launch_rows_wide<DT, CT, 64>(x, a, how, st)
         : widest <= 96 ? launch_rows_wide<DT, CT, 96>(x, a, how, st)
                        : launch_rows_wide<DT, CT, 128>(x, a, how, st);
}
template <int DT>
static int launch_rows_from(const AttentionArgs& x, const AttentionArgs& a, PrefixWay how, int32_t ctype, hipStream_t st) {
  if (ctype == LR_E4M3) return launch_rows_of<DT, LR_E4M3>(x, a, how, st);
  if (ctype == LR_INT8) return launch_rows_of<DT, LR_INT8>(x, a, how, st);
  return launch_rows_of<DT, DT>(x, a, how, st);
}

template <int DT, int CT, int DC>
static int launch_pair_wide(const AttentionArgs& x, const AttentionArgs& a, hipStream_t st) {
  const unsigned first = x.splits == 1 ? x.units : x.grid, second = a.splits == 1 ? a.batch * a.units : a.grid;
  hipLaunchKernelGGL((k_prefix_pair<DT, CT, DC>), dim3(first + second), dim3(256), 0, st, x, a, first);
  return check_op_launch();
}
// In the widths of 64, 128 and 256: reading is not what such calls wait for.
template <int DT, int CT> static int launch_pair_of(const AttentionArgs& x, const AttentionArgs& a, hipStream_t st) {
  return a.wide <= 64    ? launch_pair_wide<DT, CT, 64>(x, a, st)
         : a.wide <= 128 ? launch_pair_wide<DT, CT, 128>(x, a, st)
                         : launch_pair_wide<DT, CT, 256>(x, a, st);
}
static int launch_pair(const AttentionArgs& x, const AttentionArgs& a, int32_t dtype, int32_t ctype, hipStream_t st) {
  return with_model_type(dtype, [&](auto dt) {
    constexpr int D = decltype(dt)::value;
    if (ctype == LR_E4M3) return launch_pair_of<D, LR_E4M3>(x, a, st);
    if (ctype == LR_INT8) return launch_pair_of<D, LR_INT8>(x, a, st);
    return launch_pair_of<D, D>(x, a, st);
  });
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
  p.own.path = p.p_own.path;
  p.pre.path = p.p_pre.path;
  prefix_way(dtype, c->dtype, &p.pre, &p.own);
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
  const PrefixWay way = prefix_way(dtype, c->dtype, &x, &a);
  if (way.how == PrefixWay::kRows) {
    const int rc = dtype == LR_F16 ? launch_rows_from<LR_F16>(x, a, way, c->dtype, st)
                                   : launch_rows_from<LR_BF16>(x, a, way, c->dtype, st);
    if (rc) return rc;
  } else if (way.how == PrefixWay::kPair) {
    if (int rc = launch_pair(x, a, dtype, c->dtype, st)) return rc;
  } else {
    if (int rc = launch_attention_pass(x, dtype, c->dtype, st)) return rc;
  }
  if (!way.mixed)
    if (int rc = launch_attention_pass(a, dtype, c->dtype, st)) return rc;
  const PrefixJoin j{x.part_ml, x.part_o, x.splits, a.group, a.batch, make_fastdiv(a.group)};
  const unsigned rows = (unsigned)(batch * a.heads);
  return with_model_type(dtype, [&](auto dt) {
    if (rows >= kManyHeads)
      hipLaunchKernelGGL((k_prefix_join<decltype(dt)::value, 64>), dim3((rows + 3) / 4), dim3(256), 0, st, a, j);
    else
      hipLaunchKernelGGL((k_prefix_join<decltype(dt)::value, 256>), dim3(rows), dim3(256), 0, st, a, j);
    return check_op_launch();
  });
}

}  // extern "C"
