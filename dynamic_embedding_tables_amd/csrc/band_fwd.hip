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
#include <algorithm>
#include <cmath>

#include "band.h"

namespace recis {
namespace {

// A tile of K keys of K and V in registers on its way to LDS.
template <typename T, int DP, int K, bool PAGED, bool ALN>
struct KeyStage {
  static constexpr int kAcross = kCols<DP> / 8, kStep = kThreads / kAcross;
  static constexpr int kPer = (K + kStep - 1) / kStep;
  Frag<T> fk[kPer], fv[kPer];
  int page[kPer];  // of the tile that comes next
  int row, d0;
  __device__ __forceinline__ void start() {
    row = threadIdx.x / kAcross;
    d0 = (threadIdx.x % kAcross) * 8;
  }
  __device__ __forceinline__ void ask_pages(const BandArgs& a, const int* table, int first, int len) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int key = first + row + i * kStep;
      page[i] = key < len ? table[page_of(a, key)] : 0;
    }
  }
  // rows whose bit is clear, and those past the length, are zero, whatever memory holds there
  __device__ __forceinline__ void load(const BandArgs& a, const T* kb, const T* vb, int first, int len,
                                       unsigned long long bits) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int in_tile = row + i * kStep, key = first + in_tile;
      bool in = in_tile < K;
      const T *pk, *pv;
      if constexpr (PAGED) {
        in = in && key < len;
        if (in && (unsigned)page[i] >= (unsigned long long)a.pages) {
          in = false;
          if (a.error) atomicOr(a.error, kErrInvalid);
        }
        const int slot = key - page_of(a, key) * a.page_size;
        pk = kb + (long long)page[i] * a.ks[0] + (long long)slot * a.ks[1];
        pv = vb + (long long)page[i] * a.vs[0] + (long long)slot * a.vs[1];
      } else {
        in = in && (bits >> in_tile & 1);
        pk = kb + (long long)key * a.ks[1];
        pv = vb + (long long)key * a.vs[1];
      }
      fk[i] = load8<T, ALN>(pk, d0, a.head_dim, in);
      fv[i] = load8<T, ALN>(pv, d0, a.head_dim, in);
    }
  }
  __device__ __forceinline__ void store(T* tk, T* tv) const {
    if (d0 >= DP) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (K == kPer * kStep || row + i * kStep < K) {
        const int at = chunk_at<T, DP>(row + i * kStep, d0 / 8);
        *reinterpret_cast<Frag<T>*>(tk + at) = fk[i];
        *reinterpret_cast<Frag<T>*>(tv + at) = fv[i];
      }
  }
};

template <typename T, int DP, bool PAGED, bool ALN>
__global__ __launch_bounds__(kThreads, 2) void k_band_fwd(BandArgs a) {
  constexpr int KK = DP / 16, DB = DP / 32, K = kBandKeys<T, DP>, KB = K / 32;
  constexpr int kTile = K * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  int b, h, t;
  if (!band_place(a, a.row_tiles * a.splits, &b, &h, &t)) return;
  if constexpr (!PAGED) zero_spare<T>(a, a.out, a.os, h * a.group, a.group, b, t, a.row_tiles * a.splits);
  // the last rows see the most keys: they start first
  const int split = t % a.splits, tile = a.row_tiles - 1 - t / a.splits;
  const Entry e = entry_at<PAGED>(a, b);
  const int tile_row = tile * kBandRows, rows = e.n * a.group;
  if (tile_row >= rows) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Walk walk = walk_of<K>(a, reach_of(a, e, tile_row, tile_row + kBandRows - 1));
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
  const int p = exists ? position(a, e, r / a.group) : -1;
  Frag<T> q[KK];
  {
    const T* from = static_cast<const T*>(a.q) + (exists ? query_at(a, a.qs, e, b, h, r) : 0);
#pragma unroll
    for (int c = 0; c < KK; ++c) q[c] = load_head16<T, ALN>(from, c, lane, a.head_dim, exists);
  }
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = zeros16();
  // maximum, the same in log2 of the weight (0 before the first key), how far a
  // score may go before both are raised, sum
  float m = -INFINITY, ref = 0.f, most = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;
  KeyStage<T, DP, K, PAGED, ALN> st;
  st.start();
  unsigned long long bits = ~0ull;
  if (i0 < i1) {
    const int first = walk.tile(i0) * K;
    if constexpr (PAGED)
      st.ask_pages(a, table, first, e.len);
    else
      bits = band_bits(a, e, b, first, lane);
    st.load(a, kb, vb, first, e.len, bits);
    if constexpr (PAGED)
      if (i0 + 1 < i1) st.ask_pages(a, table, walk.tile(i0 + 1) * K, e.len);
  }
  int buffer = 0;
  for (int i = i0; i < i1; ++i, buffer ^= 1) {
    const int first = walk.tile(i) * K;
    T* tk = tiles + buffer * 2 * kTile;
    T* tv = tk + kTile;
    st.store(tk, tv);
    __syncthreads();
    const unsigned long long now = bits;
    if (i + 1 < i1) {
      const int next = walk.tile(i + 1) * K;
      if constexpr (!PAGED) bits = band_bits(a, e, b, next, lane);
      st.load(a, kb, vb, next, e.len, bits);
      if constexpr (PAGED)
        if (i + 2 < i1) st.ask_pages(a, table, walk.tile(i + 2) * K, e.len);
    }
    if (none_seen<K>(a, reach, first)) continue;
    f32x16 s[KB];
#pragma unroll
    for (int n = 0; n < KB; ++n) {
      s[n] = zeros16();
#pragma unroll
      for (int c = 0; c < KK; ++c) s[n] = mma32(rows32<DP>(tk, n * 32, c, lane), q[c], s[n]);
    }
    const bool whole = K == 64 ? now == ~0ull : (unsigned)now == ~0u;
    if (!whole || !all_seen<K>(a, reach, first)) {
      const unsigned long long mine = (seen_bits(a, p, first) & now) >> (4 * (lane >> 5));
#pragma unroll
      for (int n = 0; n < KB; ++n)
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!((mine >> (n * 32 + 8 * (x / 4) + x % 4)) & 1)) s[n][x] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < KB; ++n)
#pragma unroll
      for (int x = 0; x < 16; ++x) top = fmaxf(top, s[n][x]);
    top = halves_max(top);
    if (__any(top * c2 > most)) {
      const float to = fmaxf(m, top);
      ref = to == -INFINITY ? 0.f : to * c2;
      const float alpha = __builtin_amdgcn_exp2f(m * c2 - ref);
      m = to;
      most = to == -INFINITY ? -INFINITY : ref + kSlack;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= alpha;
    }
#pragma unroll
    for (int n = 0; n < KB; ++n)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        s[n][x] = __builtin_amdgcn_exp2f(s[n][x] * c2 - ref);
        l += s[n][x];
      }
#pragma unroll
    for (int n = 0; n < KB; ++n) {
      const Frag<T> p0 = half_of<T, 0>(s[n]), p1 = half_of<T, 1>(s[n]);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        o[d] = mma32(cols32<DP>(tv, n * 32, d * 32, lane), p0, o[d]);
        o[d] = mma32(cols32<DP>(tv, n * 32 + 16, d * 32, lane), p1, o[d]);
      }
    }
  }
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
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int x = 0; x < 16; x += 4)
        store4<float, false>(po, d * 32 + result_row(lane, x), a.head_dim,
                             f32x4{o[d][x], o[d][x + 1], o[d][x + 2], o[d][x + 3]});
    if (lane < 32) {
      a.part_ml[2 * at] = m * c2;
      a.part_ml[2 * at + 1] = l;
    }
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + query_at(a, a.os, e, b, h, r);
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int x = 0; x < 16; x += 4)
      store4<T, ALN>(out, d * 32 + result_row(lane, x), a.head_dim,
                     f32x4{o[d][x] * inv, o[d][x + 1] * inv, o[d][x + 2] * inv, o[d][x + 3] * inv});
  if (a.lse && lane < 32) a.lse[lse_at(a, e, b, h, r)] = l == 0.f ? -INFINITY : m * a.scale + __logf(l);
}

template <typename T, int DP, bool PAGED>
void launch_fwd(bool aln, const BandArgs& a, hipStream_t s) {
  const dim3 grid = band_grid(a, (int64_t)a.row_tiles * a.splits);
  if (aln)
    hipLaunchKernelGGL((k_band_fwd<T, DP, PAGED, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_band_fwd<T, DP, PAGED, false>), grid, dim3(kThreads), 0, s, a);
  if (a.splits <= 1) return;
  launch_join<T, PAGED, kBandKeys<T, DP>, kBandRows, kLeastTiles>(a, s);
}

template <typename T, bool PAGED>
void launch_fwd_dp(bool aln, const BandArgs& a, hipStream_t s) {
  switch (band_dp(a.head_dim)) {
    case 32: return launch_fwd<T, 32, PAGED>(aln, a, s);
    case 64: return launch_fwd<T, 64, PAGED>(aln, a, s);
    case 96: return launch_fwd<T, 96, PAGED>(aln, a, s);
    default: return launch_fwd<T, 128, PAGED>(aln, a, s);
  }
}

}  // namespace

void launch_band_fwd(int dtype, bool paged, bool aln, const BandArgs& a, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16)
    paged ? launch_fwd_dp<__bf16, true>(aln, a, s) : launch_fwd_dp<__bf16, false>(aln, a, s);
  else
    paged ? launch_fwd_dp<float, true>(aln, a, s) : launch_fwd_dp<float, false>(aln, a, s);
}

}  // namespace recis
