// Attention over the blocks of a paged cache that a cheap score selects: lr_block_keys, lr_block_select and
// lr_block_attention, with their plans.  A block is a page.
#include "attention.h"

namespace lr {

// ------------------------------------------------------------------ the blocks' keys

struct BlockKeysArgs {
  const void* k;
  const float* ks;
  void* out;
  const int64_t* slots;
  int64_t kd, kh, ksl, kp, sh, ssl, sp, od, oh, op;
  int64_t cache_slots;
  FastDiv fd_page;
  uint32_t page_size, heads, n, chunk, heads_y;  // heads_y: of a workgroup
  int32_t dim;
};

// The upper half of the lanes' x exchanged with the lower half's y (of each 32 lanes, where not WIDE), in one instruction
// for 32 bits: x + y is then what either half keeps of a sum by halves.
template <bool WIDE> __device__ __forceinline__ void halves_swapped(double* x, double* y) {
  uint64_t a = (uint64_t)__double_as_longlong(*x), b = (uint64_t)__double_as_longlong(*y), c[2], d[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto r = WIDE ? __builtin_amdgcn_permlane32_swap((uint32_t)(a >> (32 * h)), (uint32_t)(b >> (32 * h)), false, false)
                        : __builtin_amdgcn_permlane16_swap((uint32_t)(a >> (32 * h)), (uint32_t)(b >> (32 * h)), false, false);
    c[h] = r[0], d[h] = r[1];
  }
  *x = __longlong_as_double((long long)(c[1] << 32 | c[0]));
  *y = __longlong_as_double((long long)(d[1] << 32 | d[0]));
}

// Adds the sums of lanes that are D, D / 2, ... `lanes` apart: of N columns each half of them keeps half, of one both.
template <int D, int N>
__device__ __forceinline__ void add_halves(double* sum, uint32_t lanes, uint32_t lane, uint32_t* first, uint32_t* left) {
  if ((uint32_t)D < lanes) return;
  const bool high = lane & D;
  if constexpr (N > 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      double low = sum[i], up = sum[N / 2 + i];
      if constexpr (D >= 16) {
        halves_swapped<(D >= 32)>(&low, &up);
        sum[i] = low + up;
      } else {
        asm("" : "+v"(low), "+v"(up));  // values: not one element of sum at an index of the lane's own
        sum[i] = (high ? up : low) + __shfl_xor(high ? low : up, D);
      }
    }
    *first += high ? N / 2 : 0;
    *left = N / 2;
  } else {
    sum[0] += __shfl_xor(sum[0], D);
  }
  if constexpr (D > 1) add_halves<D / 2, (N > 1 ? N / 2 : 1)>(sum, lanes, lane, first, left);
}

// The first slot inside the cache among the entries from `from` on, or -1: each wave of the workgroup takes every fourth
// 1024 entries, half of the next ones under way, until it meets one or is past one that another wave met.  Padding behind
// the last token is looked through to its end, as fast as one CU reads (some 65 GB/s): 8 heads of 128 bf16, 131071 entries
// the first 101 of which have a slot, 23 us (8 if only the next entry were looked at), 262144 and 100001 65 us (47).
__device__ __forceinline__ int64_t first_inside(const BlockKeysArgs& a, uint32_t from, uint32_t lane, uint32_t w) {
  __shared__ uint32_t met;
  if (threadIdx.x == 0) met = ~0u;
  __syncthreads();
  const uint32_t most = a.n - 1;
  int64_t x[2][8];
  auto load = [&](int half, uint32_t i) {
#pragma unroll
    for (uint32_t z = 0; z < 8; ++z) x[half][z] = a.slots[min(i + 64 * z + lane, most)];
  };
  auto look = [&](int half, uint32_t i) {
    uint32_t high = ~0u;  // 0 where one is no negative number: then they are looked at one by one
#pragma unroll
    for (int z = 0; z < 8; ++z) high = min(high, (uint32_t)((uint64_t)x[half][z] >> 32));
    if (!__any(high == 0)) return;
#pragma unroll
    for (uint32_t z = 0; z < 8; ++z)
      if ((uint64_t)x[half][z] < (uint64_t)a.cache_slots) atomicMin(&met, min(i + 64 * z + lane, most));
  };
  load(0, from + 1024 * w);
  load(1, from + 1024 * w + 512);
  for (uint32_t i = from + 1024 * w; i < a.n; i += 4096) {
    look(0, i);
    load(0, i + 4096);
    look(1, i + 512);
    load(1, i + 4608);
    if (*(volatile uint32_t*)&met < i + 4096) break;
  }
  __syncthreads();
  return met == ~0u ? -1 : a.slots[met];
}

// A workgroup has `chunk` entries of slots and makes the mean of every page whose newest slot is among them; its waves
// take cache heads of one page side by side, which share lines of memory, their scales above all.  A row of a page is a
// group of lanes with V elements each, as many rows at a time as the wave has groups, four loads ahead, and the next
// rows or page asked for before these are added.  Sums are held in 64 bits, in which those of a page of codes or 16-bit
// keys are exact but for extreme ranges: which blocks a score selects does not hang on the order of a sum.  Codes times
// scales are rounded to the 32 bits that lr_cache_read gives where keys have 16, so that a caller who makes keys of those
// numbers gets the same ones, and from them the same choice (whole products turn 640 of the 16.8 million elements of the
// first size below); keys of 32 bits, in which that rounding would show, are made of the whole products.  The groups'
// sums are added by halves, each half of the lanes keeping half of the columns, so that a lane ends with few to divide
// and store (all lanes with all columns: 254 us for the first size below).
//
// 262142 tokens of 8 heads of 128 e4m3 in pages of 16 (tokens first): 85 us, 3.3 TB/s.  Vector instructions are busy 83 % of
// it, but adding nothing took no less: what bounds it is the loads, 8 bytes a lane, that a wave has under way (bf16, 16
// bytes a lane: 115 us, 5.0 TB/s).  16 tokens, each the newest of its page of 64: 5 us, slot, keys and store one after
// another.
template <int DT, int CT, int V>
__global__ void __launch_bounds__(256) k_block_keys(BlockKeysArgs a) {
  using T = typename ElemOf<DT>::T;
  using C = typename ElemOf<CT>::T;
  using Vec = typename Chunk<C, V>::Vec;
  constexpr bool kQuant = CT == LR_E4M3 || CT == LR_INT8;
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64);
  const uint64_t at = (uint64_t)blockIdx.x * a.chunk + lane;
  const bool mine = lane < a.chunk && at < a.n;
  const int64_t slot = mine ? a.slots[at] : -1;
  int64_t next = mine && at + 1 < a.n ? a.slots[at + 1] : -1;
  const bool held = (uint64_t)slot < (uint64_t)a.cache_slots;
  const uint32_t page = held ? op_div((uint32_t)slot, a.fd_page) : 0, in = held ? (uint32_t)slot - page * a.page_size : 0;
  // The newest of its page, unless the next entry inside the cache is a later slot of the same page.  Where others stand
  // between, that is looked for in the chunk, for the chunk's last in the 64 entries behind, and if its page has later
  // slots at all in those behind them.
  if (__builtin_expect(__any(held && (uint64_t)next >= (uint64_t)a.cache_slots), 0)) {
    const uint64_t inside = __ballot(held), after = inside & ~(((uint64_t)2 << lane) - 1);
    next = __shfl((long long)slot, after ? __ffsll((unsigned long long)after) - 1 : 0);
    const uint64_t behind = (blockIdx.x + (uint64_t)1) * a.chunk;
    int64_t first = behind + lane < a.n ? a.slots[behind + lane] : -1;
    const uint64_t near = __ballot((uint64_t)first < (uint64_t)a.cache_slots);
    first = __shfl((long long)first, near ? __ffsll((unsigned long long)near) - 1 : 0);
    if (!near) {
      const uint32_t newest = uniform(__shfl(in, 63 - __builtin_clzll(inside)));
      first = newest + 1 < a.page_size && behind + 64 < a.n ? first_inside(a, (uint32_t)behind + 64, lane, w) : -1;
    }
    if (!after) next = first;
  }
  const bool later = next > slot && next < (int64_t)(page + (uint64_t)1) * a.page_size;
  uint64_t todo = __ballot(held && !later);
  uint32_t lanes = 1;  // of a row, a power of two
  while (lanes * V < (uint32_t)a.dim && lanes < 64) lanes *= 2;
  const uint32_t rows = 64 / lanes, row = lane / lanes, col = lane % lanes * V;
  // This lane's row among those read at a time, as offsets; where it is past the newest slot, the first of them is read.
  const int64_t k_row = (int64_t)row * a.ksl, s_row = (int64_t)row * a.ssl;
  // Cache heads side by side, one a wave, as many as there are up to 4; the waves left over take other pages.
  const uint32_t side = a.heads > 2 ? 2 : a.heads - 1;  // as a power of two
  const uint32_t mine_h = w & ((1u << side) - 1), mine_p = w >> side, others = (4u >> side) - 1;
  const uint32_t h_end = min(a.heads, (blockIdx.y + 1) * a.heads_y);
  // A wave's work in order: its pages, the cache heads of each, the columns of each that the lanes cover at a time.
  uint32_t p = 0, count = 0, h = h_end, e0 = 0, rank = 0;
  auto next_work = [&]() -> bool {
    e0 += lanes * V;
    if (h < h_end && e0 < (uint32_t)a.dim) return true;
    e0 = 0;
    h += 1u << side;
    if (h < h_end) return true;
    while (todo) {
      const int f = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      if ((rank++ & others) != mine_p) continue;
      p = uniform(__shfl(page, f)), count = uniform(__shfl(in, f)) + 1;
      h = blockIdx.y * a.heads_y + mine_h;
      return h < h_end;  // the same for every page
    }
    return false;
  };
  // Rows t0 .. t0 + 4 rows - 1 of it, and their scales.
  Vec x[4];
  float sc[4];
  auto load = [&](uint32_t t0) {
    const C* k = (const C*)a.k + (int64_t)p * a.kp + (int64_t)h * a.kh;
    const float* ks = kQuant ? a.ks + (int64_t)p * a.sp + (int64_t)h * a.sh : nullptr;
    const int64_t at_col = e0 + col < (uint32_t)a.dim ? (int64_t)(e0 + col) * (V > 1 ? 1 : a.kd) : 0, at_row = k_row + at_col;
#pragma unroll
    for (uint32_t z = 0; z < 4; ++z) {
      const uint32_t t = t0 + z * rows;
      if (t >= count) continue;  // the same for all lanes
      int64_t at = at_row, at_s = s_row;
      if (t + rows > count && t + row >= count) at = at_col, at_s = 0;
      x[z] = __builtin_nontemporal_load((const Vec*)(k + (int64_t)t * a.ksl + at));
      if constexpr (kQuant) sc[z] = (ks + (int64_t)t * a.ssl)[at_s];
    }
  };
  bool more = next_work();
  if (more) load(0);
  while (more) {
    const uint32_t n = count, at = e0 + col;
    T* out = (T*)a.out + (int64_t)p * a.op + (int64_t)h * a.oh;
    double sum[V] = {};
    for (uint32_t t0 = 0; t0 < n; t0 += 4 * rows) {
      Vec y[4];
      float s[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) y[z] = x[z], s[z] = sc[z];
      if (t0 + 4 * rows < n) {
        load(t0 + 4 * rows);
      } else {
        more = next_work();
        if (more) load(0);
      }
#pragma unroll
      for (uint32_t z = 0; z < 4; ++z) {
        const uint32_t t = t0 + z * rows;
        if (t >= n || (t + rows > n && t + row >= n)) continue;
        float v[V];
        if constexpr (kQuant && V > 1) {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const F4 d = decode4<CT>(((const uint32_t*)&y[z])[i / 4]);
            v[i] = d[0], v[i + 1] = d[1], v[i + 2] = d[2], v[i + 3] = d[3];
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = value_of<CT>(y[z][i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
          sum[i] = kQuant && DT == LR_F32 ? __builtin_fma((double)v[i], (double)s[z], sum[i])
                                          : sum[i] + (double)(kQuant ? v[i] * s[z] : v[i]);
      }
    }
    uint32_t first = 0, left = V;  // the columns that this lane is left with
    add_halves<32, V>(sum, lanes, lane, &first, &left);
    // The quotient itself, as times 1 / n a mean between two numbers would be rounded to the wrong one; a full page of a
    // power of two, the usual case, has it without a division (with one for all pages 3 % more of the first size above).
    if (__builtin_expect(n & (n - 1), 0)) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] /= (double)n;
    } else {
      const int down = -(31 - __builtin_clz(n));
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = __builtin_ldexp(sum[i], down);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float mean = (float)sum[i];
      asm("" : "+v"(mean));  // two roundings: the compiler makes one of them otherwise, with other bits next to a tie
      if ((uint32_t)i < left && at < (uint32_t)a.dim) out[(int64_t)(at + first + i) * a.od] = (T)mean;
    }
  }
}

// ------------------------------------------------------------------ scores and the choice

struct SelectArgs {
  const void *q, *keys;
  const int32_t *table, *lens;
  int32_t* out;
  double* scores;  // (sequence, cache head, max_pages)
  int64_t qd, qh, qb, kd, kh, kp;
  int64_t table_stride;
  FastDiv fd_page, fd_heads, fd_runs;  // by the page's size, by kv_heads, by runs
  uint32_t page_size, pages, max_pages, kv_heads, group, batch;
  uint32_t count, first, last;
  uint32_t runs, rounds;  // workgroups of a row of scores, 64 blocks of each
  int32_t dim;
};
__device__ __forceinline__ uint32_t blocks_of(const SelectArgs& a, int32_t len) {
  const uint32_t b = len > 0 ? op_div((uint32_t)len - 1, a.fd_page) + 1 : 0;
  return b < a.max_pages ? b : a.max_pages;
}

typedef double D4 __attribute__((ext_vector_type(4)));

// The largest x over the 16 lanes of each row of lanes, passing over NaN, by exchanges that are part of an instruction
// (neighbours, pairs, mirrors of 8 and 16).
template <int CTRL> __device__ __forceinline__ double exchanged(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double row_largest(double x) {
  x = fmax(x, exchanged<0xb1>(x));
  x = fmax(x, exchanged<0x4e>(x));
  x = fmax(x, exchanged<0x141>(x));
  return fmax(x, exchanged<0x140>(x));
}

// What comes in chunks of 16 bytes: nothing, the keys, or the queries too.
enum ScoreChunks { kNoChunks, kKeyChunks, kAllChunks };

// score(b, g, j) = max over the query heads h of cache head g of q[b, h] . key[table[b, j], g], in 64 bits: which blocks
// are chosen hangs on scores that differ in their last bits, so these are as good as exact.  16 blocks x 16 heads are a
// product of 64-bit matrix instructions, as fast as the vector units' 64 bits, with the sums over the lanes done; they
// take 2048 cycles of a SIMD for 16 blocks of 128.  Keys and queries come from memory as the products' operands
// themselves (16 rows, each lane a chunk of 16 bytes), so that waves share nothing; a wave takes every fourth tile of
// its workgroup's, the next one's keys under way.  2 sequences of 8192 blocks, 64 heads on 8 of 128 bf16 (34 MB): 17 us,
// of which the products are 7; 16 sequences of up to 512 blocks, 32 heads (8 MB): 11 us, length, page, key and product
// one after another (12.7 with the first tile's keys asked for before the length is known).  Queries whose rows are not
// made of chunks leave the keys' as they are, in a kernel of their own: a branch between both cost 2 us of each.
template <int DT, int DC, int CHUNKS>
__global__ void __launch_bounds__(256) k_block_scores(SelectArgs a) {
  using T = typename ElemOf<DT>::T;
  constexpr uint32_t E = DT == LR_F32 ? 4 : 8;  // elements of a chunk
  using Vec = typename Chunk<T, (int)E>::Vec;
  constexpr uint32_t kChunks = DC / (4 * E);
  constexpr std::bool_constant<CHUNKS != kNoChunks> keys_wide{};
  constexpr std::bool_constant<CHUNKS == kAllChunks> queries_wide{};
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x / 64), r = lane & 15, j = lane >> 4;
  const uint32_t bg = op_div(blockIdx.x, a.fd_runs), b = op_div(bg, a.fd_heads), g = bg - b * a.kv_heads;
  const uint32_t begin = (blockIdx.x - bg * a.runs) * 64 * a.rounds + 16 * w;
  const uint32_t many = blocks_of(a, a.lens[b]), end = min(begin + 64 * a.rounds, many);
  if (begin >= end || many <= a.count) return;  // all are taken: nothing to compare
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  double* scores = a.scores + (uint64_t)bg * a.max_pages;
  auto load = [&](auto wide, const T* row, int64_t stride, bool there, Vec* x) {
#pragma unroll
    for (uint32_t c = 0; c < kChunks; ++c) {
      const uint32_t e0 = (c * 4 + j) * E;
      if constexpr (decltype(wide)::value) {
        x[c] = *(const Vec*)(row + (e0 < (uint32_t)a.dim ? e0 : 0));
        if (!there || e0 >= (uint32_t)a.dim) x[c] = Vec{};
      } else {
#pragma unroll
        for (uint32_t i = 0; i < E; ++i)
          x[c][i] = there && e0 + i < (uint32_t)a.dim ? row[(int64_t)(e0 + i) * stride] : (T)0.f;
      }
    }
  };
  auto page_at = [&](uint32_t j0) { return j0 + r < many ? table[j0 + r] : -1; };
  auto key_of = [&](int32_t page) {
    return (const T*)a.keys + (int64_t)((uint32_t)page < a.pages ? page : 0) * a.kp + (int64_t)g * a.kh;
  };
  for (uint32_t h0 = 0; h0 < a.group; h0 += 16) {
    Vec q[kChunks], next[kChunks];
    int32_t page = page_at(begin);
    const bool head = h0 + r < a.group;
    const T* query = (const T*)a.q + (int64_t)b * a.qb + (int64_t)(g * a.group + (head ? h0 + r : 0)) * a.qh;
    load(queries_wide, query, a.qd, head, q);
    load(keys_wide, key_of(page), a.kd, true, next);
    for (uint32_t j0 = begin; j0 < end; j0 += 64) {
      Vec k[kChunks];
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c) k[c] = next[c];
      const uint64_t seen = __ballot((uint32_t)page < a.pages);
      if (j0 + 64 < end) {
        page = page_at(j0 + 64);
        load(keys_wide, key_of(page), a.kd, true, next);
      }
      D4 acc = {};
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c)
#pragma unroll
        for (uint32_t i = 0; i < E; ++i)
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)value_of<DT>(k[c][i]), (double)value_of<DT>(q[c][i]), acc, 0, 0, 0);
      // lane r, j has head r of blocks j, 4 + j, 8 + j, 12 + j
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        double x = row_largest(head ? acc[i] : -__builtin_inf());
        const uint32_t row = 4 * i + j;
        if (r == 0 && j0 + row < many) {
          x = x == x && (seen >> row & 1) ? x : -__builtin_inf();
          if (h0) x = fmax(x, scores[j0 + row]);
          scores[j0 + row] = x;
        }
      }
    }
  }
}

// A score's bits as an integer of the same order (-0 as 0).
__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | (uint64_t)1 << 63;
}

// One workgroup chooses for one sequence and cache head: the first and the last blocks, and of the others the best.
// The score at the border is found a digit of 8 bits at a time, from the highest bit in which any two scores differ,
// until a digit's scores are all taken or all bits are known; the chosen blocks are then written in their order, of
// equal scores at the border the first ones.  A lane keeps the first HELD scores of its own; those of longer rows are
// read again for each digit.  16 rows of 8191 scores: 18 us, a chain of reading, four digits and three sums over the
// workgroup; 128 rows of up to 512, by four waves each: 6 us.
template <int LANES, int HELD>
__global__ void __launch_bounds__(LANES) k_block_choose(SelectArgs a) {
  constexpr uint32_t kWaves = LANES / 64;
  __shared__ uint32_t hist[256];
  __shared__ uint64_t ends[2][kWaves];
  __shared__ uint32_t found[3];
  __shared__ uint32_t before[2][2][HELD * kWaves];
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x / 64, bg = blockIdx.x;
  int32_t* out = a.out + (uint64_t)bg * a.count;
  const double* scores = a.scores + (uint64_t)bg * a.max_pages;
  const uint32_t many = blocks_of(a, a.lens[op_div(bg, a.fd_heads)]);
  if (many <= a.count) {
    for (uint32_t i = threadIdx.x; i < a.count; i += LANES) out[i] = i < many ? (int32_t)i : -1;
    return;
  }
  const uint32_t lo = a.first, hi = many - a.last;  // of these is chosen
  uint32_t need = a.count - a.first - a.last;
  uint64_t border = ~(uint64_t)0;  // taken: above it, and the first `equal` of those on it
  uint32_t equal = 0;
  uint64_t held[HELD];
#pragma unroll
  for (uint32_t k = 0; k < HELD; ++k) {
    const uint32_t i = k * LANES + threadIdx.x;
    held[k] = order_of(i >= lo && i < hi ? scores[i] : 0.0);
  }
  // f(i, score) for this lane's blocks that are chosen from
  auto each = [&](auto f) {
#pragma unroll
    for (uint32_t k = 0; k < HELD; ++k) {
      const uint32_t i = k * LANES + threadIdx.x;
      if (i >= lo && i < hi) f(held[k]);
    }
    for (uint32_t i = HELD * LANES + threadIdx.x; i < hi; i += LANES)
      if (i >= lo) f(order_of(scores[i]));
  };
  if (need) {
    uint64_t least = ~(uint64_t)0, most = 0;
    each([&](uint64_t s) {
      least = s < least ? s : least;
      most = s > most ? s : most;
    });
    for (int d = 32; d; d >>= 1) {
      const uint64_t x = __shfl_xor((unsigned long long)least, d), y = __shfl_xor((unsigned long long)most, d);
      least = x < least ? x : least;
      most = y > most ? y : most;
    }
    if (lane == 0) ends[0][w] = least, ends[1][w] = most;
    for (uint32_t i = threadIdx.x; i < 256; i += LANES) hist[i] = 0;
    __syncthreads();
    for (uint32_t i = 0; i < kWaves; ++i) {
      least = ends[0][i] < least ? ends[0][i] : least;
      most = ends[1][i] > most ? ends[1][i] : most;
    }
    uint32_t bit = least == most ? 0 : 64 - (uint32_t)__builtin_clzll(least ^ most);  // bits not known yet
    border = bit < 64 ? most >> bit << bit : 0;
    equal = need;
    while (bit) {
      const uint32_t from = bit > 8 ? bit - 8 : 0, bins = 1u << (bit - from);
      each([&](uint64_t s) {
        if (bit == 64 || s >> bit == border >> bit) atomicAdd(&hist[(uint32_t)(s >> from) & (bins - 1)], 1u);
      });
      __syncthreads();
      if (w == 0) {  // four bins a lane, from the highest down; empty again for the next digit
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          sum += c[z] = hist[255 - (4 * lane + z)];
          hist[255 - (4 * lane + z)] = 0;
        }
        uint32_t above = wave_scan(sum, lane) - sum;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          if (above < need && above + c[z] >= need) found[0] = 255 - (4 * lane + z), found[1] = need - above, found[2] = c[z];
          above += c[z];
        }
      }
      __syncthreads();
      border |= (uint64_t)found[0] << from;
      need = equal = found[1];
      bit = from;
      if (found[2] == need) {  // all scores that begin so
        equal = ~0u;
        break;
      }
    }
  }
  const bool some = equal && equal != ~0u;  // of equal scores the first ones
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  uint32_t done = 0, level = 0;             // written; met on the border
  // HELD runs of LANES blocks at a time: each wave's counts of all of them, and the sums of those before it
  for (uint32_t i0 = 0, turn = 0; i0 < many; i0 += HELD * LANES, turn ^= 1) {
    uint64_t s[HELD];
    bool take[HELD];
#pragma unroll
    for (uint32_t k = 0; k < HELD; ++k) {
      const uint32_t i = i0 + k * LANES + threadIdx.x;
      const bool choice = i >= lo && i < hi;
      s[k] = i0 == 0 ? held[k] : choice ? order_of(scores[i]) : 0;
      const bool on = choice && equal && s[k] == border;
      take[k] = i < many && (!choice || (equal && (s[k] > border || (on && !some))));
      s[k] = on;  // from here on only that
    }
    auto counts = [&](uint32_t which, auto flag) {
#pragma unroll
      for (uint32_t k = 0; k < HELD; ++k) {
        const uint64_t x = __ballot(flag(k));
        if (lane == 0) before[turn][which][k * kWaves + w] = (uint32_t)__popcll(x);
      }
      __syncthreads();
      if (w == 0) {  // running sums over HELD * kWaves counts
        uint32_t sum = 0;
        for (uint32_t x = 0; x < HELD * kWaves; x += 64) {
          const uint32_t c = x + lane < HELD * kWaves ? before[turn][which][x + lane] : 0;
          const uint32_t upto = wave_scan(c, lane);
          if (x + lane < HELD * kWaves) before[turn][which][x + lane] = sum + upto;
          sum += uniform(__shfl(upto, 63));
        }
      }
      __syncthreads();
    };
    auto start = [&](uint32_t which, uint32_t k) { return k * kWaves + w ? before[turn][which][k * kWaves + w - 1] : 0; };
    if (some) {
      counts(0, [&](uint32_t k) { return s[k] != 0; });
#pragma unroll
      for (uint32_t k = 0; k < HELD; ++k) {
        const uint32_t rank = level + start(0, k) + (uint32_t)__popcll(__ballot(s[k] != 0) & below);
        take[k] = take[k] || (s[k] && rank < equal);
      }
      level += before[turn][0][HELD * kWaves - 1];
    }
    counts(1, [&](uint32_t k) { return take[k]; });
#pragma unroll
    for (uint32_t k = 0; k < HELD; ++k) {
      const uint32_t at = done + start(1, k) + (uint32_t)__popcll(__ballot(take[k]) & below);
      if (take[k]) out[at] = (int32_t)(i0 + k * LANES + threadIdx.x);
    }
    done += before[turn][1][HELD * kWaves - 1];
  }
}

// ------------------------------------------------------------------ host

// A tensor of one row of head_dim elements for each head and item: layout (head_dim, heads, items).
struct Rows {
  int64_t dim, heads, items, d, h, i;  // extents and strides
};
static int rows_of(const lr_layout* L, int64_t capacity, bool output, Rows* r) {
  if (int rc = check_tensor(L, 3, capacity, output)) return rc;
  const Mode d = mode_of(*L, 0), h = mode_of(*L, 1), i = mode_of(*L, 2);
  if (one_leaf(d, &r->d) || one_leaf(h, &r->h) || one_leaf(i, &r->i)) return LR_ERR_INVALID;
  r->dim = d.size;
  r->heads = h.size;
  r->items = i.size;
  return LR_OK;
}

template <int DT, int CT, int V>
static int launch_keys(const BlockKeysArgs& a, dim3 grid, hipStream_t st) {
  hipLaunchKernelGGL((k_block_keys<DT, CT, V>), grid, dim3(256), 0, st, a);
  return check_op_launch();
}
// In chunks of v elements, or one at a time.
template <int DT, int CT>
static int launch_keys_of(const BlockKeysArgs& a, int64_t v, dim3 grid, hipStream_t st) {
  constexpr int kMost = CT == LR_F32 ? 4 : 8;
  if (v == kMost) return launch_keys<DT, CT, kMost>(a, grid, st);
  return launch_keys<DT, CT, 1>(a, grid, st);
}

template <int DT, int DC> static int launch_scores(const SelectArgs& a, ScoreChunks chunks, dim3 grid, hipStream_t st) {
  if (chunks == kAllChunks)
    hipLaunchKernelGGL((k_block_scores<DT, DC, kAllChunks>), grid, dim3(256), 0, st, a);
  else if (chunks == kKeyChunks)
    hipLaunchKernelGGL((k_block_scores<DT, DC, kKeyChunks>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_block_scores<DT, DC, kNoChunks>), grid, dim3(256), 0, st, a);
  return check_op_launch();
}

static int plan_select(const lr_layout* Lq, int64_t q_capacity, const lr_layout* Lk, int64_t keys_capacity,
                       int64_t max_pages, Rows* q, Rows* k, int64_t* bytes) {
  int rc = rows_of(Lq, q_capacity, false, q);
  if (rc || (rc = rows_of(Lk, keys_capacity, false, k))) return rc;
  if (q->dim != k->dim || q->heads % k->heads) return LR_ERR_SIZE_MISMATCH;
  if (q->dim > kAttentionDim || max_pages < 1) return LR_ERR_INVALID;
  const double runs = (double)q->items * (double)k->heads * (double)((max_pages + 63) / 64);
  if (max_pages > kMaxCount || runs > (double)kMaxCount) return LR_ERR_OVERFLOW;
  *bytes = q->items * k->heads * max_pages * 8;
  return LR_OK;
}

static int plan_blocks(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t max_pages, int64_t count,
                       int32_t dtype, AttentionArgs* a, lr_attention_plan* out) {
  if (int rc = attention_shapes(Lq, c, Lo, max_pages, dtype, a, out)) return rc;
  if (count < 1) return LR_ERR_INVALID;
  if (count > kMaxCount / a->page_size) return LR_ERR_OVERFLOW;
  if ((double)mode_of(*Lq, 2).size * a->kv_heads * count > 0x1p60) return LR_ERR_OVERFLOW;
  a->count = (uint32_t)count;
  return attention_split(mode_of(*Lq, 2).size, count * a->page_size, true, a, out);
}

}  // namespace lr

using namespace lr;

extern "C" {

int lr_block_keys(const lr_cache* c, const int64_t* slots, int64_t n, void* keys, const lr_layout* Lkeys,
                  int64_t keys_capacity, int32_t dtype, void* stream) {
  if (int rc = lr_cache_validate(c)) return rc;
  if (!keys || n < 0 || (n > 0 && !slots)) return LR_ERR_INVALID;
  if (!is_model_type(dtype) || (!is_quantised(c->dtype) && c->dtype != dtype)) return LR_ERR_TYPE;
  Rows o;
  if (int rc = rows_of(Lkeys, keys_capacity, true, &o)) return rc;
  const Mode kd = mode_of(c->k_layout, 0), kh = mode_of(c->k_layout, 1), ks = mode_of(c->k_layout, 2);
  const Mode kp = mode_of(c->k_layout, 3);
  if (o.dim != kd.size || o.heads != kh.size || o.items != kp.size) return LR_ERR_SIZE_MISMATCH;
  if (kh.size > 4 * 65535 || n > kMaxCount) return LR_ERR_OVERFLOW;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype);
  const Buffer in[] = {{slots, n * 8}, {c->k, c->k_capacity * ce}, {c->v, c->v_capacity * ce},
                       {c->k_scale, c->scale_capacity * 4}, {c->v_scale, c->scale_capacity * 4}};
  const Buffer made[] = {{keys, keys_capacity * e}};
  if (int rc = check_overlaps(in, 5, made, 1)) return rc;
  if (n == 0) return LR_OK;
  BlockKeysArgs a;
  std::memset(&a, 0, sizeof(a));
  a.k = c->k;
  a.ks = c->k_scale;
  a.out = keys;
  a.slots = slots;
  one_leaf(kd, &a.kd), one_leaf(kh, &a.kh), one_leaf(ks, &a.ksl), one_leaf(kp, &a.kp);  // checked with the cache
  if (is_quantised(c->dtype)) {
    one_leaf(mode_of(c->scale_layout, 0), &a.sh);
    one_leaf(mode_of(c->scale_layout, 1), &a.ssl);
    one_leaf(mode_of(c->scale_layout, 2), &a.sp);
  }
  a.od = o.d;
  a.oh = o.h;
  a.op = o.i;
  a.page_size = (uint32_t)ks.size;
  a.fd_page = make_fastdiv(a.page_size);
  a.cache_slots = kp.size * ks.size;
  a.heads = (uint32_t)kh.size;
  a.n = (uint32_t)n;
  a.dim = (int32_t)kd.size;
  // 64 entries and all heads a workgroup, fewer where that would leave part of the device without one: a step's
  // entries are each the newest of their page, a prompt's one in page_size
  a.chunk = (uint32_t)std::min<int64_t>(64, std::max<int64_t>(1, n / 2048));
  a.heads_y = a.chunk < 64 ? 4 : a.heads;
  int64_t v = ce == 4 ? 4 : 8;
  while (v > 1 && (a.dim % v || !rows_aligned(c->k_layout, c->k, ce, v))) v /= 2;
  const dim3 grid((unsigned)((n + a.chunk - 1) / a.chunk), (a.heads + a.heads_y - 1) / a.heads_y);
  const hipStream_t st = (hipStream_t)stream;
  return with_model_type(dtype, [&](auto dt) {
    constexpr int D = decltype(dt)::value;
    if (c->dtype == LR_E4M3) return launch_keys_of<D, LR_E4M3>(a, v, grid, st);
    if (c->dtype == LR_INT8) return launch_keys_of<D, LR_INT8>(a, v, grid, st);
    return launch_keys_of<D, D>(a, v, grid, st);
  });
}

int lr_block_select_plan(const lr_layout* Lq, const lr_layout* Lkeys, int64_t max_pages, int64_t* workspace_bytes) {
  if (!workspace_bytes) return LR_ERR_INVALID;
  Rows q, k;
  return plan_select(Lq, INT64_MAX, Lkeys, INT64_MAX, max_pages, &q, &k, workspace_bytes);
}

int lr_block_select(const void* q, const lr_layout* Lq, int64_t q_capacity, const void* keys, const lr_layout* Lkeys,
                    int64_t keys_capacity, int32_t dtype, const int32_t* table, int64_t table_stride, int64_t max_pages,
                    const int32_t* lens, int64_t page_size, int64_t batch, int64_t first, int64_t last, int32_t* blocks,
                    int64_t count, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !keys || batch < 0 || (batch > 0 && (!blocks || !table || !lens)) || table_stride < 0) return LR_ERR_INVALID;
  if (!is_model_type(dtype)) return LR_ERR_TYPE;
  Rows r, k;
  int64_t need;
  if (int rc = plan_select(Lq, q_capacity, Lkeys, keys_capacity, max_pages, &r, &k, &need)) return rc;
  if (batch > r.items) return LR_ERR_BOUNDS;
  if (page_size < 1 || first < 0 || last < 0 || count < 1 || first > count || last > count - first) return LR_ERR_INVALID;
  if (max_pages > kMaxCount / page_size || count > kMaxCount || (double)batch * k.heads * count > 0x1p60)
    return LR_ERR_OVERFLOW;
  if (!workspace || workspace_bytes < need) return LR_ERR_CAPACITY;
  if ((uintptr_t)workspace % 16) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype);
  const Buffer in[] = {{q, q_capacity * e}, {keys, keys_capacity * e}, {lens, batch * 4},
                       {table, batch ? ((batch - 1) * table_stride + max_pages) * 4 : 0}};
  const Buffer made[] = {{blocks, batch * k.heads * count * 4}, {workspace, need}};
  if (int rc = check_overlaps(in, 4, made, 2)) return rc;
  if (batch == 0) return LR_OK;
  SelectArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q;
  a.keys = keys;
  a.table = table;
  a.lens = lens;
  a.out = blocks;
  a.scores = (double*)workspace;
  a.qd = r.d, a.qh = r.h, a.qb = r.i;
  a.kd = k.d, a.kh = k.h, a.kp = k.i;
  a.table_stride = table_stride;
  a.page_size = (uint32_t)page_size;
  a.fd_page = make_fastdiv(a.page_size);
  a.pages = (uint32_t)k.items;
  a.max_pages = (uint32_t)max_pages;
  a.kv_heads = (uint32_t)k.heads;
  a.fd_heads = make_fastdiv(a.kv_heads);
  a.group = (uint32_t)(r.heads / k.heads);
  a.batch = (uint32_t)batch;
  a.count = (uint32_t)count;
  a.first = (uint32_t)first;
  a.last = (uint32_t)last;
  a.dim = (int32_t)r.dim;
  const hipStream_t st = (hipStream_t)stream;
  const int64_t rows = batch * k.heads;
  if (max_pages > count) {  // else nothing is compared
    const int64_t tiles = (max_pages + 63) / 64;
    a.rounds = (uint32_t)std::min<int64_t>(8, std::max<int64_t>(1, rows * tiles / 2048));
    a.runs = (uint32_t)((tiles + a.rounds - 1) / a.rounds);
    a.fd_runs = make_fastdiv(a.runs);
    const bool wide = r.dim % (16 / e) == 0 && rows_aligned(*Lkeys, keys, e, 16 / e);
    const ScoreChunks chunks = !wide ? kNoChunks : rows_aligned(*Lq, q, e, 16 / e) ? kAllChunks : kKeyChunks;
    const dim3 grid((unsigned)(rows * a.runs));
    const int rc = with_model_type(dtype, [&](auto dt) {
      constexpr int D = decltype(dt)::value;
      if (a.dim <= 64) return launch_scores<D, 64>(a, chunks, grid, st);
      if (a.dim <= 128) return launch_scores<D, 128>(a, chunks, grid, st);
      return launch_scores<D, 256>(a, chunks, grid, st);
    });
    if (rc) return rc;
  }
  // a row of up to 1024 scores by four waves, longer ones by sixteen
  if (max_pages > 1024)
    hipLaunchKernelGGL((k_block_choose<1024, 8>), dim3((unsigned)rows), dim3(1024), 0, st, a);
  else
    hipLaunchKernelGGL((k_block_choose<256, 4>), dim3((unsigned)rows), dim3(256), 0, st, a);
  return check_op_launch();
}

int lr_block_attention_plan(const lr_layout* Lq, const lr_cache* c, const lr_layout* Lo, int64_t count, int32_t dtype,
                            lr_attention_plan* out) {
  if (!out) return LR_ERR_INVALID;
  AttentionArgs a;
  return plan_blocks(Lq, c, Lo, 1, count, dtype, &a, out);
}

int lr_block_attention(const void* q, const lr_layout* Lq, int64_t q_capacity, const lr_cache* c, const int32_t* blocks,
                       int64_t count, const int32_t* table, int64_t table_stride, int64_t max_pages,
                       const int32_t* lens, int64_t batch, void* out, const lr_layout* Lo, int64_t out_capacity,
                       float* lse, int32_t dtype, float scale, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !out || batch < 0 || (batch > 0 && (!blocks || !table || !lens)) || !std::isfinite(scale) || table_stride < 0)
    return LR_ERR_INVALID;
  AttentionArgs a;
  lr_attention_plan p;
  if (int rc = plan_blocks(Lq, c, Lo, max_pages, count, dtype, &a, &p)) return rc;
  if (cosize_bound(Lq) > q_capacity || cosize_bound(Lo) > out_capacity || batch > mode_of(*Lq, 2).size)
    return LR_ERR_BOUNDS;
  if (p.workspace_bytes && (!workspace || workspace_bytes < p.workspace_bytes)) return LR_ERR_CAPACITY;
  if (p.workspace_bytes && (uintptr_t)workspace % 16) return LR_ERR_INVALID;
  const int64_t e = dtype_bytes(dtype), ce = dtype_bytes(c->dtype), rows = batch * a.heads;
  const Buffer in[] = {{q, q_capacity * e}, {c->k, c->k_capacity * ce}, {c->v, c->v_capacity * ce},
                       {c->k_scale, c->scale_capacity * 4}, {c->v_scale, c->scale_capacity * 4},
                       {table, batch ? ((batch - 1) * table_stride + max_pages) * 4 : 0}, {lens, batch * 4},
                       {blocks, batch * a.kv_heads * count * 4}};
  const Buffer made[] = {{out, out_capacity * e}, {lse, lse ? rows * 4 : 0}, {workspace, p.workspace_bytes}};
  if (int rc = check_overlaps(in, 8, made, 3)) return rc;
  if (batch == 0) return LR_OK;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.blocks = blocks;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.batch = (uint32_t)batch;
  a.scale2 = scale * kLog2e;
  a.part_o = (float*)workspace;
  a.part_ml = (float*)workspace + (p.workspace_bytes / 4 - 2 * mode_of(*Lq, 2).size * a.heads * p.splits);
  attention_buffers(c, Lq, q, dtype, p.path, &a);
  const hipStream_t st = (hipStream_t)stream;
  const int rc = with_model_type(dtype, [&](auto dt) {
    constexpr int D = decltype(dt)::value;
    if (c->dtype == LR_E4M3) return launch_pass<D, LR_E4M3, true>(a, st);
    if (c->dtype == LR_INT8) return launch_pass<D, LR_INT8, true>(a, st);
    return launch_pass<D, D, true>(a, st);
  });
  return rc || a.splits == 1 ? rc : launch_attention_join(a, dtype, st);
}

}  // extern "C"
