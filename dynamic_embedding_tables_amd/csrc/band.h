// band.h -- attention of a sequence to its own past: what the kernels for it share
// (band_fwd.hip, band_bwd.hip over strided or packed keys, paged.hip over a paged
// cache).
//
// The query at position p sees the keys j <= p with p - j < window or j < sinks
// (and mask[j] != 0).  The q_heads / kv_heads query heads that share a key head are
// folded into the rows of a pair (batch entry, key head): row = query * group + g.
//
// Matrix products are 32x32: an operand holds, per lane, 8 consecutive k of one row
// (lane % 32), k from 8 * (lane / 32); a result holds column lane % 32 and rows
// 8 * (i / 4) + 4 * (lane / 32) + i % 4 for i = 0 .. 15.  Scores are computed with
// the side that is reduced over as rows, so two of a result's quarters are, after
// rounding, the operand of the next product over 16 of them: slot j of lane half h
// is row 4 h + j for j < 4, and 8 + 4 h + j - 4 above, and the other operand is read
// in that order.
#pragma once

#include "attn.h"
#include "divide.h"

namespace recis {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct BandArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  float* lse;
  const int* offsets;          // of packed queries (and, without pages, of the keys); or null
  const int* lens;             // keys an entry has; or null
  const int* table;            // paged: [batch][width] pages
  const unsigned char* kv_mask;
  unsigned* error;
  long long mask_stride, total_rows, table_stride, pages;
  long long qs[3], os[3], dos[3], dqs[3];      // batch, position, head
  long long ks[3], vs[3], dks[3], dvs[3];      // the same, or page, slot, head
  int batch, q_len, q_heads, kv_heads, group, head_dim;
  int max_len;                 // most keys an entry has
  int rows;                    // most rows a pair has: q_len * group
  int causal, window, sinks;   // window: more than any length where there is none
  Quick by_page, by_group, by_kv_heads;
  int row_tiles, key_tiles, splits, q_splits, kv_splits, sink_splits;
  int part_keys, far_keys;     // keys that have parts of dK and dV, and sinks in whole blocks of 32
  int die_bits, unit;          // `unit` pairs share a die, 2^die_bits units lie side by side
  int ranked;                  // entries take their turns by length, the longest first
  int pairs_inner;             // in a unit: a tile's pairs next to each other, else a pair's tiles
  int per;                     // blocks of a pair, in this launch
  Quick by_inner, by_across, by_splits;  // blocks of the inner order, of a unit and of a tile, in this launch
  float scale;
  float *part_o, *part_ml;     // parts of key ranges: [pair][split][rows][head_dim], [..][2]
  float* part_kv;              // parts of row ranges: [pair][split][part_keys][2][head_dim], then far ones
  f32x2* stats;                // [pair][rows]: L and delta, from dQ's kernel to dK and dV's
};

// Sizes a launch of one of the many-row kernels needs (band_fwd.hip, band_bwd.hip).
constexpr int kBandWaves = 4, kBandRows = 32 * kBandWaves;
constexpr int kDies = 8, kDieBits = 3;
constexpr int kLeastTiles = 2;      // tiles of keys a split has where there are so many
constexpr int kMaxSplits = 256;     // parts that keys or rows are split into
inline int band_dp(int head_dim) { return (head_dim + 31) / 32 * 32; }
// Keys of a tile.  (float32 of more than 32 elements: 32, since its products hold the matrix
// unit sixteen times as long as bfloat16's and a few tiles must go round: 33 entries of up to
// 999 keys, 50 rows, 6 heads of 40: 49 us with 64, 39 with 32.)
inline int band_keys(int dtype, int head_dim) { return dtype == RECIS_DTYPE_F32 && head_dim > 32 ? 32 : 64; }
// The grid of a launch of `tiles` tiles a pair in `splits` parts each.
inline dim3 band_grid(BandArgs* a, int64_t tiles, int64_t splits) {
  const int64_t per = tiles * splits, unit = a->unit;
  a->per = (int)per;
  a->by_inner = Quick(a->pairs_inner ? unit : per);
  a->by_across = Quick(per * unit);
  a->by_splits = Quick(splits);
  return grid_of(round_up((int64_t)a->batch * a->kv_heads, unit << a->die_bits) * per);
}
// How the blocks of a call are laid over the dies.
//  - All pairs of an entry on one die where its keys are read about once (one tile of
//    rows), a pair's blocks side by side, which reads a pair's keys in one stretch.
//  - The same where the heads are shorter than a 128-byte line, which would be fetched by
//    several dies, but the pairs of a tile side by side, as they meet in the lines.
//  - With few pairs a pair's blocks go to every die.
constexpr int kEntriesForDies = 64, kPairsForDies = 128;
inline void place_pairs(BandArgs* a, int dtype) {
  const bool once = a->row_tiles <= 1, together = once || a->head_dim * dtype_size(dtype) < 128;
  a->unit = together && a->batch >= kEntriesForDies ? a->kv_heads : 1;
  a->pairs_inner = !once;
  a->die_bits = (int64_t)a->batch * a->kv_heads >= kPairsForDies ? kDieBits : 0;
}
// Elements an access takes: 8 where rows are aligned to 16 bytes, 2 where all are to pairs, else 1.
inline int band_access(int dtype, int head_dim, std::initializer_list<const void*> ptrs,
                       std::initializer_list<const long long*> strides) {
  for (int w : {8, 2}) {
    const int bytes = w == 8 ? 16 : 2 * dtype_size(dtype), per = bytes / dtype_size(dtype);
    bool all = head_dim % w == 0;
    for (const void* p : ptrs) all = all && aligned_to(p, bytes);
    for (const long long* s : strides)
      for (int i = 0; i < 3; ++i) all = all && s[i] % per == 0;
    if (all) return w;
  }
  return 1;
}
void launch_band_fwd(int dtype, bool paged, int access, const BandArgs& a, hipStream_t s);

namespace {

__device__ __forceinline__ int page_of(const BandArgs& a, int key) { return divided(key, a.by_page); }

// --------------------------------------------------------------- an entry
struct Entry {
  long long row0;  // first packed row
  int n;           // queries whose results are written
  int len;         // keys
  int step, shift; // position of query q: q * step + shift; not causal: the last key's, for all
};

template <bool PAGED>
__device__ __forceinline__ Entry entry_at(const BandArgs& a, int b, bool tell = true) {
  long long lo = 0, hi = a.q_len;
  bool bad = false;
  if (a.offsets) {
    lo = a.offsets[b], hi = a.offsets[b + 1];
    bad = lo < 0 || hi < lo || hi > a.total_rows || hi - lo > a.q_len;
    if (bad) lo = hi = 0;
  }
  const int n = (int)(hi - lo);
  int len = PAGED || !a.offsets ? a.max_len : n;
  if (a.lens) {
    len = a.lens[b];
    if (len < 0 || len > a.max_len) {
      bad = true;
      len = 0;
    }
  }
  if (bad && tell && a.error && threadIdx.x == 0) atomicOr(a.error, kErrInvalid);
  const int causal = a.causal ? 1 : 0;
  return Entry{lo, n, len, causal, causal ? (PAGED ? len - n : 0) : len - 1};
}

// Position of a query: below 0 it sees nothing (rows past the length among them).
__device__ __forceinline__ int position(const BandArgs& a, Entry e, int query) {
  const int p = query * e.step + e.shift;
  return p < e.len ? p : -1;
}

// Positions of the rows row0 .. row1 of a pair that the entry has: the lowest and the
// highest that see a key (high < low: none does).
struct Reach {
  int low, high;
};
__device__ __forceinline__ Reach reach_of(const BandArgs& a, Entry e, int row0, int row1) {
  const int last = std::min(std::min(divided(row1, a.by_group), e.n - 1) * e.step + e.shift, e.len - 1);
  return Reach{divided(row0, a.by_group) * e.step + e.shift, row0 < e.n * a.group ? last : -1};
}

// A key, or where no row of a reach sees it -- behind the sinks, before the window, where
// a cache's pages may be gone -- the first of the window.
__device__ __forceinline__ int in_reach(const BandArgs& a, int key, int window_lo) {
  return key < a.sinks ? key : std::max(key, window_lo);
}

// The tiles of K keys that rows of a reach see, in order: tiles of sinks that lie
// before the window, then the window's.
struct Walk {
  int sink_tiles, first, n;
  __device__ __forceinline__ int tile(int i) const { return i < sink_tiles ? i : first + i - sink_tiles; }
};
template <int K>
__device__ __forceinline__ Walk walk_of(const BandArgs& a, Reach r) {
  Walk w{0, 0, 0};
  if (r.high < r.low || r.high < 0) return w;
  const int lo = std::max(0, r.low - a.window + 1);
  w.sink_tiles = (std::min(a.sinks, lo) + K - 1) / K;
  w.first = std::max(w.sink_tiles, lo / K);
  w.n = w.sink_tiles + std::max(0, r.high / K - w.first + 1);
  return w;
}
// Every row of the reach sees every one of K keys from `first`.
template <int K>
__device__ __forceinline__ bool all_seen(const BandArgs& a, Reach r, int first) {
  return first + K - 1 <= r.low && (first > r.high - a.window || first + K <= a.sinks);
}
// No row of the reach sees any of them.
template <int K>
__device__ __forceinline__ bool none_seen(const BandArgs& a, Reach r, int first) {
  return first > r.high || (first + K - 1 <= r.low - a.window && first >= a.sinks);
}
__device__ __forceinline__ bool seen(const BandArgs& a, int p, int key) {
  return key <= p && (p - key < a.window || key < a.sinks);
}

// Bits of the keys first .. first + 63 that the row at position p sees.
__device__ __forceinline__ unsigned long long seen_bits(const BandArgs& a, int p, int first) {
  const int hi = p - first, lo = hi - a.window + 1, sinks = a.sinks - first;
  const unsigned long long upto = hi < 0 ? 0 : hi >= 63 ? ~0ull : (2ull << hi) - 1;
  const unsigned long long near = lo <= 0 ? ~0ull : lo >= 64 ? 0 : ~0ull << lo;
  const unsigned long long sink = sinks <= 0 ? 0 : sinks >= 64 ? ~0ull : (1ull << sinks) - 1;
  return upto & (near | sink);
}

// Split `s` of `splits` of a walk: `per` tiles, `least` where there are so many.
__device__ __forceinline__ int split_size(int n, int splits, int least) {
  if (splits == 1) return n > 0 ? n : 1;
  const int per = (n + splits - 1) / splits;
  return per > least ? per : least;
}

// Consecutive blocks go to the eight dies in turn; a unit is the pairs of an entry, or one
// pair, and shares a die and its L2.
__device__ __forceinline__ bool band_place(const BandArgs& a, int* b, int* h, int* tile, int* split) {
  const int id = block_id(), slot = id >> a.die_bits, turn = divided(slot, a.by_across);
  const int rest = slot - turn * a.by_across.d, outer = divided(rest, a.by_inner);
  const int inner = rest - outer * a.by_inner.d;
  const int t = a.pairs_inner ? outer : inner, in_unit = a.pairs_inner ? inner : outer;
  const int pair = ((turn << a.die_bits) + (id & ((1 << a.die_bits) - 1))) * a.unit + in_unit;
  *tile = divided(t, a.by_splits);
  *split = t - *tile * a.by_splits.d;
  *b = divided(pair, a.by_kv_heads);
  *h = pair - *b * a.kv_heads;
  return *b < a.batch;
}

// The entry that is `rank`th by length, of 64 at most, those without rows last: blocks of a
// long walk that start late run alone at the end.  Found by every wave for itself, in less
// than a microsecond.
__device__ __forceinline__ int entry_of_rank(const BandArgs& a, int rank) {
  const int lane = threadIdx.x & 63;
  int mine = -1;
  if (lane < a.batch) {
    const Entry e = entry_at<true>(a, lane, false);
    mine = e.n > 0 ? e.len : -1;
  }
  int before = 0;
  for (int i = 0; i < a.batch; ++i) {
    const int other = __builtin_amdgcn_readlane(mine, i);
    before += other > mine || (other == mine && i < lane);
  }
  return __ffsll((unsigned long long)__ballot(lane < a.batch && before == rank)) - 1;
}

// Offset of query q, head g of the group, in a tensor of queries.
__device__ __forceinline__ long long query_at(const BandArgs& a, const long long (&st)[3], Entry e, int b,
                                              int h, int r) {
  const int q = divided(r, a.by_group), g = r - q * a.group;
  return (a.offsets ? e.row0 * st[1] : (long long)b * st[0]) + (long long)q * st[1] +
         (long long)(h * a.group + g) * st[2];
}
__device__ __forceinline__ long long lse_at(const BandArgs& a, Entry e, int b, int h, int r) {
  const int q = divided(r, a.by_group), g = r - q * a.group;
  return ((a.offsets ? e.row0 : (long long)b * a.q_len) + q) * a.q_heads + h * a.group + g;
}

// Offset of key head h of an entry in a tensor of keys that is not paged.
__device__ __forceinline__ long long keys_at(const BandArgs& a, const long long (&st)[3], Entry e, int b,
                                             int h) {
  return (a.offsets ? e.row0 * st[1] : (long long)b * st[0]) + (long long)h * st[2];
}

// Bit i: key first + i is there and not masked (not paged).
__device__ __forceinline__ unsigned long long band_bits(const BandArgs& a, Entry e, int b, int first, int lane) {
  const int n = e.len - first;
  if (!a.kv_mask) return n >= 64 ? ~0ull : n <= 0 ? 0 : (1ull << n) - 1;
  bool in = lane < n;
  if (in) in = a.kv_mask[(a.offsets ? e.row0 : (long long)b * a.mask_stride) + first + lane] != 0;
  return __ballot(in);
}

constexpr float kSlack = 8.f;
template <typename T, int DP>
constexpr int kBandKeys = sizeof(T) == 4 && DP > 32 ? 32 : 64;

// Zeros for `heads` heads from h of the packed rows that no entry writes: those before
// the first and after the last, a part of them from each of the head's blocks, and those
// of an entry that is taken as empty (entry_at), from its own `per` blocks (t of them).
template <typename T>
__device__ __forceinline__ void zero_rows(T* to, const long long (&st)[3], int h, int heads, int dim, long long lo,
                                          long long hi, long long end, int block, int blocks) {
  const long long per = (long long)heads * dim, n = (lo + end - hi) * per;
  for (long long i = (long long)block * kThreads + threadIdx.x; i < n; i += (long long)blocks * kThreads) {
    const long long at = i / per, in = i - at * per, row = at < lo ? at : hi + (at - lo);
    to[row * st[1] + (h + in / dim) * st[2] + in % dim] = (T)0.f;
  }
}
template <typename T>
__device__ __forceinline__ void zero_spare(const BandArgs& a, void* to, const long long (&st)[3], int h, int heads,
                                           int b, int t, int per) {
  if (!a.offsets) return;
  auto at = [&](int i) { return std::min<long long>(std::max(a.offsets[i], 0), a.total_rows); };
  const long long first = at(0), last = at(a.batch), lo = at(b), hi = at(b + 1);
  if (first > 0 || last < a.total_rows)
    zero_rows(static_cast<T*>(to), st, h, heads, a.head_dim, first, std::max(first, last), a.total_rows, b * per + t,
              a.batch * per);
  if (hi - lo > a.q_len || a.offsets[b] < 0 || a.offsets[b + 1] > a.total_rows)
    zero_rows(static_cast<T*>(to), st, h, heads, a.head_dim, 0, lo, hi, t, per);
}

// ------------------------------------------------------------ 32x32 products
__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
// Whether chunk c of a head is worth its products: float32's take eight instructions, each of
// twice bfloat16's cycles, so those past the head are left out.
template <typename T>
__device__ __forceinline__ bool chunk_counts(int c, int dim) {
  return sizeof(T) == 2 || c * 16 < dim;
}
__device__ __forceinline__ f32x16 zeros16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}
// Row (of 32) that element i of a lane's result is.
__device__ __forceinline__ int result_row(int lane, int i) { return 8 * (i / 4) + 4 * (lane >> 5) + i % 4; }

__device__ __forceinline__ float halves_max(float x) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float halves_add(float x) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Half G of a result (its rows 16 G .. 16 G + 15) as the next product's operand.
template <typename T, int G>
__device__ __forceinline__ Frag<T> half_of(const f32x16& x) {
  const f32x8 y = G == 0 ? __builtin_shufflevector(x, x, 0, 1, 2, 3, 4, 5, 6, 7)
                         : __builtin_shufflevector(x, x, 8, 9, 10, 11, 12, 13, 14, 15);
  return __builtin_convertvector(y, Frag<T>);
}

// Elements 32 * block .. of a lane's row of a result (columns are rows of the tensor), times
// `by`.  A lane and the one 32 away hold alternate 4 elements; bfloat16 pairs are exchanged
// so that each stores 8 in a row.
template <typename T, int W>
__device__ __forceinline__ void store_result(T* row, int block, int lane, int dim, const f32x16& x, float by) {
  if constexpr (W == 8 && sizeof(T) == 2) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    auto two = [&](int i) { return __builtin_bit_cast(unsigned, bf16x2{(__bf16)(x[i] * by), (__bf16)(x[i + 1] * by)}); };
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const auto lo = __builtin_amdgcn_permlane32_swap(two(i), two(i + 4), false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(two(i + 2), two(i + 6), false, false);
      const int d0 = block * 32 + 2 * i + 8 * (lane >> 5);
      if (d0 < dim) *reinterpret_cast<u32x4*>(row + d0) = u32x4{lo[0], hi[0], lo[1], hi[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store4<T, W == 8>(row, block * 32 + result_row(lane, i), dim,
                     f32x4{x[i] * by, x[i + 1] * by, x[i + 2] * by, x[i + 3] * by});
  }
}

// 8 elements from d0 of a row that is there, W at a time; past its `dim` elements anything,
// which zero_past() makes zeros.  By 2, those past the end are the last pair again, since a
// load behind a branch would be waited for there (16 entries of 1024, 8 heads of 74, bfloat16:
// 142 us against 214 by 1 and with branches); by 1 eight such addresses cost more than the
// branches (heads of 77: 227 us against 206).
template <typename T, int W>
__device__ __forceinline__ Frag<T> load_any(const T* row, int d0, int dim) {
  Frag<T> f;
  if constexpr (W == 8) {
    f = *reinterpret_cast<const Frag<T>*>(row + (d0 < dim ? d0 : 0));
  } else if constexpr (W == 2) {
    typedef T Part __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const Part x = *reinterpret_cast<const Part*>(row + std::min(d0 + i, dim - 2));
      f[i] = x[0], f[i + 1] = x[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = d0 + i < dim ? row[d0 + i] : (T)0.f;
  }
  return f;
}
template <typename T, int W>
__device__ __forceinline__ void zero_past(Frag<T>& f, int d0, int dim) {
  if constexpr (W == 8) {
    if (d0 >= dim) f = Frag<T>{};
  } else if (W == 2 && d0 + 8 > dim) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d0 + i >= dim) f[i] = (T)0.f;
  }
}

// A lane's operands for the KK chunks (16 elements each) of a row that is there; zeros
// past its `dim` elements.
template <typename T, int KK, int W>
__device__ __forceinline__ void load_row16(Frag<T> (&f)[KK], const T* row, int lane, int dim) {
#pragma unroll
  for (int c = 0; c < KK; ++c) f[c] = load_any<T, W>(row, c * 16 + (lane >> 5) * 8, dim);
  if (dim < KK * 16) {
#pragma unroll
    for (int c = 0; c < KK; ++c) zero_past<T, W>(f[c], c * 16 + (lane >> 5) * 8, dim);
  }
}

// A lane's operand for chunk c of rows row0 .. row0 + 31 of a tile in LDS.
template <int DP>
__device__ __forceinline__ bf16x8 rows32(const __bf16* tile, int row0, int c, int lane) {
  // (the exchange leaves all but the low 3 bits of a chunk's number alone: four addresses
  // serve all chunks)
  return *reinterpret_cast<const bf16x8*>(tile + row0 * kLd<__bf16, DP> + (c & ~3) * 16 +
                                          chunk_at<__bf16, DP>(lane & 31, (c & 3) * 2 + (lane >> 5)));
}
template <int DP>
__device__ __forceinline__ f32x8 rows32(const float* tile, int row0, int c, int lane) {
  const float* p = tile + (row0 + (lane & 31)) * kLd<float, DP> + c * 16 + (lane >> 5) * 8;
  const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Column c0 + lane % 32 of the 16 rows from row0, in half_of()'s order.
template <int DP>
__device__ __forceinline__ bf16x8 cols32(const __bf16* tile, int row0, int c0, int lane) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int row = (lane >> 5) * 4 + ((lane & 15) >> 2);
  const __bf16* p = tile + row0 * kLd<__bf16, DP> + (c0 & ~63) +
                    chunk_at<__bf16, DP>(row, (c0 & 63) / 8 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) +
                    (lane & 1) * 4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * kLd<__bf16, DP>));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int DP>
__device__ __forceinline__ f32x8 cols32(const float* tile, int row0, int c0, int lane) {
  const float* p = tile + (row0 + (lane >> 5) * 4) * kLd<float, DP> + c0 + (lane & 31);
  f32x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = p[(j < 4 ? j : j + 4) * kLd<float, DP>];
  return x;
}

// A tile of K keys of K and V in registers on its way to LDS.  What is not there -- keys
// past the length or masked, elements past the head -- is loaded from a place that is,
// and replaced by zeros on the way to LDS: no load stands behind a branch, after which
// the compiler would wait for it (that wait took a third of the forward's time).
template <typename T, int DP, int K, bool PAGED, int W>
struct KeyStage {
  static constexpr int kAcross = kCols<DP> / 8, kStep = kThreads / kAcross, kPer = K / kStep;
  static_assert(K % kStep == 0, "every thread has the same number of chunks");
  Frag<T> fk[kPer], fv[kPer];
  int page;        // paged: of key `lane` of the tile that comes next
  int row, d0, window_lo;
  unsigned at_d;   // bytes into the head
  bool bad;
  __device__ __forceinline__ void start(const BandArgs& a, int from = 0) {
    window_lo = from;  // paged: the first key of the block's window
    row = threadIdx.x / kAcross;
    d0 = (threadIdx.x % kAcross) * 8;
    at_d = d0 < a.head_dim ? d0 * (unsigned)sizeof(T) : 0;
    bad = false;
  }
  __device__ __forceinline__ void ask_pages(const BandArgs& a, const int* table, int first, int len) {
    page = table[page_of(a, in_reach(a, std::min(first + ((int)threadIdx.x & (K - 1)), len - 1), window_lo))];
  }
  // Bit i: key first + i of the tile that comes next is there, its page's number one of the
  // cache's.  (Asked once a tile by each wave, a key a lane, and passed on by exchange.)  A page
  // out of range is read as page 0, which is there.
  __device__ __forceinline__ unsigned long long paged_bits(const BandArgs& a, int first, int len) {
    const bool in = (unsigned)page < (unsigned long long)a.pages;
    if (!in) page = 0, bad = true;
    return __ballot(in && first + ((int)threadIdx.x & (K - 1)) < len);
  }
  static __device__ __forceinline__ Frag<T> at_bytes(const T* base, unsigned bytes) {
    return *reinterpret_cast<const Frag<T>*>(reinterpret_cast<const char*>(base) + bytes);
  }
  __device__ __forceinline__ void load(const BandArgs& a, const T* kb, const T* vb, int first, int len) {
    const T* tile_k = kb + (long long)first * a.ks[1];
    const T* tile_v = vb + (long long)first * a.vs[1];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int in_tile = row + i * kStep;
      if constexpr (PAGED) {
        const int key = in_reach(a, std::min(first + in_tile, len - 1), window_lo);
        const int slot = key - page_of(a, key) * a.by_page.d;
        const int p = __shfl(page, in_tile);
        if constexpr (W == 8) {  // (strides are below 2^31)
          fk[i] = at_bytes(kb + ((unsigned long long)(unsigned)p * (unsigned)a.ks[0] +
                                 (unsigned long long)(unsigned)slot * (unsigned)a.ks[1]), at_d);
          fv[i] = at_bytes(vb + ((unsigned long long)(unsigned)p * (unsigned)a.vs[0] +
                                 (unsigned long long)(unsigned)slot * (unsigned)a.vs[1]), at_d);
        } else {
          fk[i] = load_any<T, W>(kb + (long long)p * a.ks[0] + (long long)slot * a.ks[1], d0, a.head_dim);
          fv[i] = load_any<T, W>(vb + (long long)p * a.vs[0] + (long long)slot * a.vs[1], d0, a.head_dim);
        }
      } else if constexpr (W == 8) {  // (a tile's bytes are below 2^31)
        const unsigned r = std::min(in_tile, len - 1 - first);
        fk[i] = at_bytes(tile_k, r * (unsigned)(a.ks[1] * sizeof(T)) + at_d);
        fv[i] = at_bytes(tile_v, r * (unsigned)(a.vs[1] * sizeof(T)) + at_d);
      } else {
        const int r = std::min(in_tile, len - 1 - first);
        fk[i] = load_any<T, W>(tile_k + (long long)r * a.ks[1], d0, a.head_dim);
        fv[i] = load_any<T, W>(tile_v + (long long)r * a.vs[1], d0, a.head_dim);
      }
    }
  }
  // `bits`: the keys of the loaded tile that are there
  __device__ __forceinline__ void store(const BandArgs& a, T* tk, T* tv, unsigned long long bits) {
    if ((K == 64 ? bits != ~0ull : (unsigned)bits != ~0u) || a.head_dim < kCols<DP>) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (W == 2) zero_past<T, W>(fk[i], d0, a.head_dim), zero_past<T, W>(fv[i], d0, a.head_dim);
        if (!(bits >> (row + i * kStep) & 1) || d0 >= a.head_dim) fk[i] = fv[i] = Frag<T>{};
      }
    }
    if (kCols<DP> > DP && d0 >= DP) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = chunk_at<T, DP>(row + i * kStep, d0 / 8);
      *reinterpret_cast<Frag<T>*>(tk + at) = fk[i];
      *reinterpret_cast<Frag<T>*>(tv + at) = fv[i];
    }
  }
  __device__ __forceinline__ void tell(const BandArgs& a) const {
    if (PAGED && bad && a.error) atomicOr(a.error, kErrInvalid);
  }
};

// -------------------------------------------------------------------- joins
// Joins the key ranges of a row, V elements a thread; rows of one range are done.
template <typename T, int V, bool PAGED, int K, int ROWS, int LEAST>
__global__ __launch_bounds__(kThreads) void k_band_join(BandArgs a) {
  const unsigned per_row = a.head_dim / V;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;
  const unsigned row = id / per_row, d = (id - row * per_row) * V;
  const unsigned pair = row / a.rows, r = row - pair * a.rows;
  if (pair >= (unsigned)(a.batch * a.kv_heads)) return;
  const int b = divided((int)pair, a.by_kv_heads), h = (int)pair - b * a.kv_heads;
  const Entry e = entry_at<PAGED>(a, b, false);
  if ((int)r >= e.n * a.group) return;
  const int tile_row = r / ROWS * ROWS;
  const int n = walk_of<K>(a, reach_of(a, e, tile_row, tile_row + ROWS - 1)).n, per = split_size(n, a.splits, LEAST);
  if (n <= per) return;
  const int used = (n + per - 1) / per;
  const long long at = (long long)pair * a.splits * a.rows + r;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.part_ml);
  float top = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < used; ++s) top = fmaxf(top, ml[at + (long long)s * a.rows][0]);
  const float ref = top == -INFINITY ? 0.f : top;
  float o[V] = {}, l = 0.f;
#pragma unroll 4
  for (int s = 0; s < used; ++s) {
    const long long p = at + (long long)s * a.rows;
    const f32x2 x = ml[p];
    const float weight = __builtin_amdgcn_exp2f(x[0] - ref);
    l += weight * x[1];
    float v[V];
    load_f32<float, V>(a.part_o + p * a.head_dim + d, v);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] += weight * v[i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + query_at(a, a.os, e, b, h, r) + d;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = (T)(o[i] * inv);
  if (a.lse && d == 0) a.lse[lse_at(a, e, b, h, r)] = l == 0.f ? -INFINITY : top * kLn2 + __logf(l);
}

// The same for few rows and many ranges: a block a row, consecutive ranges for each
// wave.
template <typename T, bool PAGED, int K, int ROWS, int LEAST>
__global__ __launch_bounds__(kThreads) void k_band_join_few(BandArgs a) {
  constexpr int kParts = kMaxHeadDim / 64;
  __shared__ float part[kBandWaves][kMaxHeadDim + 1];
  const int lane = threadIdx.x & 63, wave = wave_of();
  const int r = (int)(blockIdx.x % a.rows), pair = (int)(blockIdx.x / a.rows);
  const int b = divided(pair, a.by_kv_heads), h = pair - b * a.kv_heads;
  const Entry e = entry_at<PAGED>(a, b, false);
  if (r >= e.n * a.group) return;
  const int tile_row = r / ROWS * ROWS;
  const int n = walk_of<K>(a, reach_of(a, e, tile_row, tile_row + ROWS - 1)).n, per = split_size(n, a.splits, LEAST);
  if (n <= per) return;
  const int used = (n + per - 1) / per;
  const long long at = (long long)pair * a.splits * a.rows + r;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.part_ml);
  float top = -INFINITY, o[kParts] = {}, l = 0.f;
  for (int s = lane; s < used; s += 64) top = fmaxf(top, ml[at + (long long)s * a.rows][0]);
  top = group_max(top);
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
  const float ref = top == -INFINITY ? 0.f : top;
  const int mine = (used + kBandWaves - 1) / kBandWaves, s1 = std::min(used, (wave + 1) * mine);
#pragma unroll 4
  for (int s = wave * mine; s < s1; ++s) {
    const long long p = at + (long long)s * a.rows;
    const f32x2 x = ml[p];
    const float weight = __builtin_amdgcn_exp2f(x[0] - ref);
    l += weight * x[1];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (lane + 64 * i < a.head_dim) o[i] += weight * a.part_o[p * a.head_dim + lane + 64 * i];
  }
#pragma unroll
  for (int i = 0; i < kParts; ++i) part[wave][lane + 64 * i] = o[i];
  if (lane == 0) part[wave][kMaxHeadDim] = l;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int k = 1; k < kBandWaves; ++k) {
    l += part[k][kMaxHeadDim];
#pragma unroll
    for (int i = 0; i < kParts; ++i) o[i] += part[k][lane + 64 * i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + query_at(a, a.os, e, b, h, r);
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    if (lane + 64 * i < a.head_dim) out[lane + 64 * i] = (T)(o[i] * inv);
  if (a.lse && lane == 0) a.lse[lse_at(a, e, b, h, r)] = l == 0.f ? -INFINITY : top * kLn2 + __logf(l);
}

// A block a row where the rows alone do not fill the chip.
template <typename T, bool PAGED, int K, int ROWS, int LEAST>
void launch_join(const BandArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  const int v = a.head_dim % 4 ? 1 : 4;
  const int64_t threads = rows * (a.head_dim / v);
  const dim3 blocks((unsigned)((threads + kThreads - 1) / kThreads));
  if (rows <= 2048)
    hipLaunchKernelGGL((k_band_join_few<T, PAGED, K, ROWS, LEAST>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
  else if (v == 4)
    hipLaunchKernelGGL((k_band_join<T, 4, PAGED, K, ROWS, LEAST>), blocks, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_band_join<T, 1, PAGED, K, ROWS, LEAST>), blocks, dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace recis
