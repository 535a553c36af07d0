// band_fwd.hip -- attention of a sequence to its own past, forward, for many rows:
// over strided or packed keys, and over the pages of a cache.
//
//   S = scale Q K^T over the keys a row sees,  L = log sum exp S,  O = exp(S - L) V
//
// Scores, the running maximum and sum, and every product's sum are float32; with
// bfloat16 the softmax weights are rounded to bfloat16 where they meet V (the matrix
// unit takes no wider operand beside a bfloat16 one).
//
// A wave holds 32 rows (of 32x32 products); the block's four waves share the keys,
// staged in LDS in two buffers, one barrier a tile, the next tile's loads in flight
// meanwhile.  Only the tiles that some row of the block sees are walked: those of the
// sinks, then those from the window of the first row to the position of the last.
// The running maximum that the weights are taken relative to is raised only once a
// score exceeds it by 2^kSlack in weight.
//
// Bound, at long walks, by the matrix unit's and the vector unit's turns at two to four
// waves a SIMD (causal, 32 entries of 4096 positions, 8 heads, bfloat16: heads of 64 796 us,
// 690 TFLOP/s, of 128 1365 us, 806 TFLOP/s; there the matrix unit is busy 35% of the
// cycles, the vector unit 46%, LDS 44%, two fifths of that for conflicts; without the
// exponentials it would take 1503 us, without loads and barriers 1110, with the products
// and their LDS reads alone 960).  Short windows are bound by the tiles at a window's
// ends, computed whole or by halves of 32 keys, and by each block's start: window 512 of
// up to 4096, 8 heads of 64 160 us, of up to 1000 packed, window 128, 4 heads of 32 90 us.
// Over a cache, 32 entries of up to 512 rows and 8192 keys, 16 heads of 128 that share 4:
// 406 to 436 us, 620 to 660 TFLOP/s.  Float32: 51 to 95 TFLOP/s of the 154 that a large
// product reaches, padded head sizes and half-seen tiles counted as lost.
//
// Tried, for the same time: raised wave priority around the products, a fixed order of
// products, exponentials and LDS reads, the LDS reads ahead of the products, two blocks'
// scores interleaved; slower: masks by comparison in place of bits.
#include <algorithm>
#include <cmath>

#include "band.h"

namespace recis {
namespace {

// Waves a SIMD, as many as leave no more than a few spilled registers.
template <typename T, int DP>
constexpr int kForwardWaves = DP > 64 ? 2 : sizeof(T) == 2 ? 4 : DP > 32 ? 2 : 3;

template <typename T, int DP, bool PAGED, int W>
__global__ __launch_bounds__(kThreads, (kForwardWaves<T, DP>)) void k_band_fwd(BandArgs a) {
  constexpr int KK = DP / 16, DB = DP / 32, K = kBandKeys<T, DP>, KB = K / 32;
  constexpr int kTile = K * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  int b, h, tile, split;
  if (!band_place(a, &b, &h, &tile, &split)) return;
  if (PAGED && a.ranked) b = entry_of_rank(a, b);
  if constexpr (!PAGED) zero_spare<T>(a, a.out, a.os, h * a.group, a.group, b, tile * a.splits + split, a.per);
  tile = a.row_tiles - 1 - tile;  // the last rows see the most keys: they start first
  const Entry e = entry_at<PAGED>(a, b);
  const int tile_row = tile * kBandRows, rows = e.n * a.group;
  if (tile_row >= rows) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Reach block_reach = reach_of(a, e, tile_row, tile_row + kBandRows - 1);
  const Walk walk = walk_of<K>(a, block_reach);
  const Reach reach = reach_of(a, e, tile_row + wave * 32, tile_row + wave * 32 + 31);
  const int per = split_size(walk.n, a.splits, kLeastTiles);
  const int i0 = split * per, i1 = std::min(walk.n, i0 + per);
  if (split > 0 && i0 >= walk.n) return;
  const T *kb, *vb;
  const int* table = nullptr;
  if constexpr (PAGED) {
    table = a.table + (long long)b * a.table_stride;
    kb = static_cast<const T*>(a.k) + (long long)h * a.ks[2];
    vb = static_cast<const T*>(a.v) + (long long)h * a.vs[2];
  } else {
    kb = static_cast<const T*>(a.k) + keys_at(a, a.ks, e, b, h);
    vb = static_cast<const T*>(a.v) + keys_at(a, a.vs, e, b, h);
  }
  const int r = tile_row + wave * 32 + (lane & 31);
  const bool exists = r < rows;
  const int p = exists ? position(a, e, divided(r, a.by_group)) : -1;
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = zeros16();
  // maximum, the same in log2 of the weight (0 before the first key), how far a
  // score may go before both are raised, sum
  float m = -INFINITY, ref = 0.f, most = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;
  KeyStage<T, DP, K, PAGED, W> st;
  st.start(a, block_reach.low - a.window + 1);  // (below 0: all of them)
  auto keys_there = [&](int first) {
    if constexpr (PAGED)
      return st.paged_bits(a, first, e.len);
    else
      return band_bits(a, e, b, first, lane);
  };
  unsigned long long bits = 0;
  if (i0 < i1) {
    const int first = walk.tile(i0) * K;
    if constexpr (PAGED) st.ask_pages(a, table, first, e.len);
    bits = keys_there(first);
    st.load(a, kb, vb, first, e.len);
    if constexpr (PAGED) st.ask_pages(a, table, walk.tile(std::min(i0 + 1, i1 - 1)) * K, e.len);
  }
  Frag<T> q[KK];  // (after the first keys' loads, which take longer)
  load_row16<T, KK, W>(q, static_cast<const T*>(a.q) + query_at(a, a.qs, e, b, h, std::min(r, rows - 1)), lane,
                         a.head_dim);
  int buffer = 0;
  for (int i = i0; i < i1; ++i, buffer ^= 1) {
    const int first = walk.tile(i) * K;
    T* tk = tiles + buffer * 2 * kTile;
    T* tv = tk + kTile;
    const unsigned long long now = bits;
    st.store(a, tk, tv, now);
    __syncthreads();
    {  // (after the last tile, that one again: a branch would have its loads waited for)
      const int next = walk.tile(std::min(i + 1, i1 - 1)) * K;
      bits = keys_there(next);
      st.load(a, kb, vb, next, e.len);
      if constexpr (PAGED) st.ask_pages(a, table, walk.tile(std::min(i + 2, i1 - 1)) * K, e.len);
    }
    if (none_seen<K>(a, reach, first)) continue;
    f32x16 s[KB];
    auto scores = [&](int n) {
      s[n] = zeros16();
#pragma unroll
      for (int c = 0; c < KK; ++c)
        if (chunk_counts<T>(c, a.head_dim)) s[n] = mma32(rows32<DP>(tk, n * 32, c, lane), q[c], s[n]);
    };
    auto mask = [&](int n) {
      const int at = first + n * 32;
      const unsigned there = (unsigned)(now >> (n * 32));
      if (there == ~0u && all_seen<32>(a, reach, at)) return;
      const unsigned mine = (unsigned)(seen_bits(a, p, at) & there) >> (4 * (lane >> 5));
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (!(mine >> (8 * (x / 4) + x % 4) & 1)) s[n][x] = -INFINITY;
    };
    auto highest = [&](int n) {
      float top = s[n][0];
#pragma unroll
      for (int x = 1; x < 16; ++x) top = fmaxf(top, s[n][x]);
      return halves_max(top);
    };
    auto raise = [&](float top) {
      if (!__any(top * c2 > most)) return;
      const float to = fmaxf(m, top);
      ref = to == -INFINITY ? 0.f : to * c2;
      const float alpha = __builtin_amdgcn_exp2f(m * c2 - ref);
      m = to;
      most = to == -INFINITY ? -INFINITY : ref + kSlack;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= alpha;
    };
    auto weights = [&](int n) {
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        s[n][x] = __builtin_amdgcn_exp2f(s[n][x] * c2 - ref);
        l += s[n][x];
      }
    };
    auto products = [&](int n) {
      const Frag<T> p0 = half_of<T, 0>(s[n]), p1 = half_of<T, 1>(s[n]);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        o[d] = mma32(cols32<DP>(tv, n * 32, d * 32, lane), p0, o[d]);
        o[d] = mma32(cols32<DP>(tv, n * 32 + 16, d * 32, lane), p1, o[d]);
      }
    };
    auto finish = [&](int n) {
      mask(n);
      raise(highest(n));
      weights(n);
      products(n);
    };
    if constexpr (DP > 64 && KB == 2) {
      // both blocks' scores first: at two waves a SIMD the products of one run behind the
      // exponentials of the other
      scores(0);
      scores(1);
      finish(0);
      finish(1);
    } else {
#pragma unroll
      for (int n = 0; n < KB; ++n) {
        if (none_seen<32>(a, reach, first + n * 32)) continue;
        scores(n);
        finish(n);
      }
    }
  }
  st.tell(a);
  l = halves_add(l);
  if (!exists) return;
  if (p < 0) {  // a row that sees nothing, whatever its block walked
    l = 0.f;
    m = -INFINITY;
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = zeros16();
  }
  if (walk.n > per) {
    const long long at = (((long long)b * a.kv_heads + h) * a.splits + split) * a.rows + r;
    float* po = a.part_o + at * a.head_dim;
#pragma unroll
    for (int d = 0; d < DB; ++d) store_result<float, 1>(po, d, lane, a.head_dim, o[d], 1.f);
    if (lane < 32) {
      a.part_ml[2 * at] = m * c2;
      a.part_ml[2 * at + 1] = l;
    }
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + query_at(a, a.os, e, b, h, r);
#pragma unroll
  for (int d = 0; d < DB; ++d) store_result<T, W>(out, d, lane, a.head_dim, o[d], inv);
  if (a.lse && lane < 32) a.lse[lse_at(a, e, b, h, r)] = l == 0.f ? -INFINITY : m * a.scale + __logf(l);
}

template <typename T, int DP, bool PAGED>
void launch_fwd(int access, BandArgs a, hipStream_t s) {
  const dim3 grid = band_grid(&a, a.row_tiles, a.splits);
  if (access == 8)
    hipLaunchKernelGGL((k_band_fwd<T, DP, PAGED, 8>), grid, dim3(kThreads), 0, s, a);
  else if (access == 2)
    hipLaunchKernelGGL((k_band_fwd<T, DP, PAGED, 2>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_band_fwd<T, DP, PAGED, 1>), grid, dim3(kThreads), 0, s, a);
  if (a.splits <= 1) return;
  launch_join<T, PAGED, kBandKeys<T, DP>, kBandRows, kLeastTiles>(a, s);
}

template <typename T, bool PAGED>
void launch_fwd_dp(int access, const BandArgs& a, hipStream_t s) {
  switch (band_dp(a.head_dim)) {
    case 32: return launch_fwd<T, 32, PAGED>(access, a, s);
    case 64: return launch_fwd<T, 64, PAGED>(access, a, s);
    case 96: return launch_fwd<T, 96, PAGED>(access, a, s);
    default: return launch_fwd<T, 128, PAGED>(access, a, s);
  }
}

}  // namespace

void launch_band_fwd(int dtype, bool paged, int access, const BandArgs& a, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16)
    paged ? launch_fwd_dp<__bf16, true>(access, a, s) : launch_fwd_dp<__bf16, false>(access, a, s);
  else
    paged ? launch_fwd_dp<float, true>(access, a, s) : launch_fwd_dp<float, false>(access, a, s);
}

}  // namespace recis
