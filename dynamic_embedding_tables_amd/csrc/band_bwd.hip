// band_bwd.hip -- attention of a sequence to its own past: the backward pass, and the
// host side of both passes.
//
//   P = exp(S - L),  dV = P^T dO,  dP = dO V^T,  delta = sum dO O,  dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  over the pairs (row, key) that see each other
//
// Sums are float32; with bfloat16, P and dS are rounded to bfloat16 where they enter a
// matrix product.  dQ has a kernel of its own, which walks the keys of 128 rows; dK and
// dV's walks the rows of 128 keys.  So S and dP are computed twice, 7 products for 5:
// a single kernel would add up dQ over its blocks, by atomics, whose order would change
// the result, or through memory.
//
// The sinks' keys are seen by all later rows, many times a window.  Their rows past the
// window are walked by blocks of their own (FAR), split over the rows, whose four waves
// share 32 keys; the parts are added in order at the end.
//
// Bound by dependent products, exponentials and LDS reads at few waves a SIMD (registers hold
// the operands of 32 rows or keys and both sums): dQ's kernel has two to four; dK and dV's two
// to four at heads of up to 32, two up to 64, and above that one in most forms, above 96 in
// all.  In float32 dK and dV's spills 72 to 92 bytes a lane at heads of 33 to 64, its far form
// 168 to 196 there, and dQ's 248 to 288 at heads above 96.  The matrix unit is busy about a
// quarter of the cycles.  32 entries of up to 4096 positions, 8 heads of 64, window
// 512, 4 sinks, bfloat16: dQ 235 us, dK and dV 250 (at three waves, spilling, 392; tiles of
// 32 rows 281), the sinks' far rows 38 (memory: they read Q and dO once more; in parts of
// 2 steps instead of 8 62; in the near rows' launch no less), the parts 5.  Causal, 4096
// positions: 2309 us with heads of 64, 595 TFLOP/s of the formula's five products, and
// 5388 of 128, 510.
#include <algorithm>
#include <cmath>

#include "band.h"

namespace recis {
namespace {

// Waves a SIMD of dQ's kernel: its time goes by them (32 entries of up to 4096 positions, 8
// heads of 64, window 512, bfloat16: 2 265 us, 3 233).
template <typename T, int DP>
constexpr int kBackwardWaves = DP > 64 || (sizeof(T) == 4 && DP > 32) ? 2 : sizeof(T) == 2 && DP <= 32 ? 4 : 3;

// dQ, and each row's L (in log2 of the weight) and delta for dK and dV.
template <typename T, int DP, int W>
__global__ __launch_bounds__(kThreads, (kBackwardWaves<T, DP>)) void k_band_bwd_q(BandArgs a) {
  constexpr int KK = DP / 16, DB = DP / 32, K = kBandKeys<T, DP>, KB = K / 32;
  constexpr int kTile = K * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  int b, h, tile, split;
  if (!band_place(a, &b, &h, &tile, &split)) return;
  zero_spare<T>(a, a.dq, a.dqs, h * a.group, a.group, b, tile * a.q_splits + split, a.per);
  tile = a.row_tiles - 1 - tile;
  const Entry e = entry_at<false>(a, b);
  const int tile_row = tile * kBandRows, rows = e.n * a.group;
  if (tile_row >= rows) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Walk walk = walk_of<K>(a, reach_of(a, e, tile_row, tile_row + kBandRows - 1));
  const int per = split_size(walk.n, a.q_splits, kLeastTiles);
  const int i0 = split * per, i1 = std::min(walk.n, i0 + per);
  if (split > 0 && i0 >= walk.n) return;
  const Reach reach = reach_of(a, e, tile_row + wave * 32, tile_row + wave * 32 + 31);
  const T* kb = static_cast<const T*>(a.k) + keys_at(a, a.ks, e, b, h);
  const T* vb = static_cast<const T*>(a.v) + keys_at(a, a.vs, e, b, h);
  const int r = tile_row + wave * 32 + (lane & 31);
  const bool exists = r < rows;
  const int p = exists ? position(a, e, divided(r, a.by_group)) : -1;
  const float c2 = a.scale * kLog2e;
  f32x16 dq[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dq[d] = zeros16();
  KeyStage<T, DP, K, false, W> st;
  st.start(a);
  unsigned long long bits = 0;
  if (i0 < i1) {
    const int first = walk.tile(i0) * K;
    bits = band_bits(a, e, b, first, lane);
    st.load(a, kb, vb, first, e.len);
  }
  Frag<T> q[KK], g[KK];  // (after the first keys' loads, which take longer)
  float delta = 0.f;
  {
    const int in = std::min(r, rows - 1);
    Frag<T> out[KK];
    load_row16<T, KK, W>(q, static_cast<const T*>(a.q) + query_at(a, a.qs, e, b, h, in), lane, a.head_dim);
    load_row16<T, KK, W>(g, static_cast<const T*>(a.dout) + query_at(a, a.dos, e, b, h, in), lane, a.head_dim);
    load_row16<T, KK, W>(out, static_cast<const T*>(a.o) + query_at(a, a.os, e, b, h, in), lane, a.head_dim);
#pragma unroll
    for (int c = 0; c < KK; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) delta += (float)g[c][i] * (float)out[c][i];
    delta = halves_add(delta);
  }
  const float lse = a.lse[lse_at(a, e, b, h, std::min(r, rows - 1))];
  const float lse2 = p >= 0 && lse != -INFINITY ? lse * kLog2e : INFINITY;  // exp2(s - inf) = 0
  if (p < 0) delta = 0.f;
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
      bits = band_bits(a, e, b, next, lane);
      st.load(a, kb, vb, next, e.len);
    }
    if (none_seen<K>(a, reach, first)) continue;
    // delta from out carries out's rounding, which a key with nearly all the weight
    // sees whole: rows that see one tile of keys get it from P and dP
    if (sizeof(T) == 2 && walk.n == 1) {
      delta = 0.f;
#pragma unroll
      for (int n = 0; n < KB; ++n) {
        f32x16 s = zeros16(), dp = zeros16();
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          s = mma32(rows32<DP>(tk, n * 32, c, lane), q[c], s);
          dp = mma32(rows32<DP>(tv, n * 32, c, lane), g[c], dp);
        }
        const unsigned mine =
            (unsigned)((seen_bits(a, p, first + n * 32) & (now >> (n * 32))) >> (4 * (lane >> 5)));
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (mine >> (8 * (x / 4) + x % 4) & 1) delta += __builtin_amdgcn_exp2f(s[x] * c2 - lse2) * dp[x];
      }
      delta = halves_add(delta);
    }
#pragma unroll
    for (int n = 0; n < KB; ++n) {
      if (none_seen<32>(a, reach, first + n * 32)) continue;
      f32x16 s = zeros16(), dp;
#pragma unroll
      for (int x = 0; x < 16; ++x) dp[x] = -delta;
#pragma unroll
      for (int c = 0; c < KK; ++c) {
        if (!chunk_counts<T>(c, a.head_dim)) continue;
        s = mma32(rows32<DP>(tk, n * 32, c, lane), q[c], s);
        dp = mma32(rows32<DP>(tv, n * 32, c, lane), g[c], dp);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) s[x] = __builtin_amdgcn_exp2f(s[x] * c2 - lse2) * dp[x];
      const int at = first + n * 32;
      const unsigned there = (unsigned)(now >> (n * 32));
      if (there != ~0u || !all_seen<32>(a, reach, at)) {
        const unsigned mine = (unsigned)(seen_bits(a, p, at) & there) >> (4 * (lane >> 5));
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!(mine >> (8 * (x / 4) + x % 4) & 1)) s[x] = 0.f;
      }
      const Frag<T> d0 = half_of<T, 0>(s), d1 = half_of<T, 1>(s);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        dq[d] = mma32(cols32<DP>(tk, n * 32, d * 32, lane), d0, dq[d]);
        dq[d] = mma32(cols32<DP>(tk, n * 32 + 16, d * 32, lane), d1, dq[d]);
      }
    }
  }
  if (!exists) return;
  if (lane < 32 && split == 0) a.stats[((long long)b * a.kv_heads + h) * a.rows + r] = f32x2{lse2, delta};
  if (p < 0) {
#pragma unroll
    for (int d = 0; d < DB; ++d) dq[d] = zeros16();
  }
  if (walk.n > per) {
    float* to = a.part_o + ((((long long)b * a.kv_heads + h) * a.q_splits + split) * a.rows + r) * a.head_dim;
#pragma unroll
    for (int d = 0; d < DB; ++d) store_result<float, 1>(to, d, lane, a.head_dim, dq[d], 1.f);
    return;
  }
  T* to = static_cast<T*>(a.dq) + query_at(a, a.dqs, e, b, h, r);
#pragma unroll
  for (int d = 0; d < DB; ++d) store_result<T, W>(to, d, lane, a.head_dim, dq[d], a.scale);
}

// Adds the key ranges' parts of dQ, in order: V elements of a row a thread.
template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void k_band_join_q(BandArgs a) {
  const unsigned per_row = a.head_dim / V;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;
  const unsigned row = id / per_row, d = (id - row * per_row) * V;
  const unsigned pair = row / a.rows, r = row - pair * a.rows;
  if (pair >= (unsigned)(a.batch * a.kv_heads)) return;
  const int b = divided((int)pair, a.by_kv_heads), h = (int)pair - b * a.kv_heads;
  const Entry e = entry_at<false>(a, b, false);
  if ((int)r >= e.n * a.group) return;
  const int tile_row = r / kBandRows * kBandRows;
  const int n = walk_of<K>(a, reach_of(a, e, tile_row, tile_row + kBandRows - 1)).n;
  const int per = split_size(n, a.q_splits, kLeastTiles);
  if (n <= per) return;
  const int used = (n + per - 1) / per;
  const float* from = a.part_o + ((long long)pair * a.q_splits * a.rows + r) * a.head_dim + d;
  float sum[V] = {};
#pragma unroll 4
  for (int s = 0; s < used; ++s) {
    float v[V];
    load_f32<float, V>(from + (long long)s * a.rows * a.head_dim, v);
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += v[i];
  }
  T* out = static_cast<T*>(a.dq) + query_at(a, a.dqs, e, b, h, r) + d;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = (T)(sum[i] * a.scale);
}

// ------------------------------------------------------------------ dK, dV
// Rows of a tile: of the near walk, and of the far one, where each wave has 32 of its own.
template <int DP, bool FAR>
constexpr int kWalkRows = FAR ? 128 : DP <= 64 ? 64 : 32;

// A thread's chunks of R folded rows of Q and dO on their way to LDS.  Rows from `until` on
// are loaded from the one before it and zeroed by store(): no load stands behind a branch.
// OWN: each wave stages 32 rows of its own.
template <typename T, int DP, int R, bool OWN, int W>
struct RowStage {
  static constexpr int kAcross = kCols<DP> / 8, kStep = (OWN ? 64 : kThreads) / kAcross, kPer = (OWN ? 32 : R) / kStep;
  static_assert((OWN ? 32 : R) % kStep == 0, "every thread has the same number of chunks");
  Frag<T> fq[kPer], fg[kPer];
  int row, d0, here;
  __device__ __forceinline__ void start() {
    row = OWN ? wave_of() * 32 + (threadIdx.x & 63) / kAcross : threadIdx.x / kAcross;
    d0 = (threadIdx.x % kAcross) * 8;
  }
  __device__ __forceinline__ void load(const BandArgs& a, Entry e, int b, int h, int first, int until) {
    here = until - first;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = std::min(first + row + i * kStep, until - 1);
      const T* pq = static_cast<const T*>(a.q) + query_at(a, a.qs, e, b, h, r);
      const T* pg = static_cast<const T*>(a.dout) + query_at(a, a.dos, e, b, h, r);
      fq[i] = load_any<T, W>(pq, d0, a.head_dim);
      fg[i] = load_any<T, W>(pg, d0, a.head_dim);
    }
  }
  __device__ __forceinline__ void store(const BandArgs& a, T* tq, T* tg) {
    if (here < R || a.head_dim < kCols<DP>) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (W == 2) zero_past<T, W>(fq[i], d0, a.head_dim), zero_past<T, W>(fg[i], d0, a.head_dim);
        if (row + i * kStep >= here || d0 >= a.head_dim) fq[i] = fg[i] = Frag<T>{};
      }
    }
    if (kCols<DP> > DP && d0 >= DP) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = chunk_at<T, DP>(row + i * kStep, d0 / 8);
      *reinterpret_cast<Frag<T>*>(tq + at) = fq[i];
      *reinterpret_cast<Frag<T>*>(tg + at) = fg[i];
    }
  }
};

constexpr int kTileKeys128 = 32 * kBandWaves;  // keys of a near block
constexpr int kMostFarSinks = 128;             // more sinks: their tiles walk all rows themselves

// Where a key's part of dK and dV lies: near parts first, [pair][split][keys], then far.
__device__ __forceinline__ float* part_near(const BandArgs& a, long long pair, int split, int key) {
  return a.part_kv + ((pair * a.kv_splits + split) * a.part_keys + key) * 2 * a.head_dim;
}
__device__ __forceinline__ float* part_far(const BandArgs& a, long long pair, int split, int key) {
  const long long near = (long long)a.batch * a.kv_heads * a.kv_splits * a.part_keys;
  return a.part_kv + (near + (pair * a.sink_splits + split) * a.far_keys + key) * 2 * a.head_dim;
}

template <typename T, int DP, int W, bool FAR>
__global__ __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) void k_band_bwd_kv(BandArgs a) {
  constexpr int KK = DP / 16, DB = DP / 32;
  constexpr int R = kWalkRows<DP, FAR>, kTile = R * kLd<T, DP>;
  // (the far walk's waves have rows of their own, so one buffer and no barrier)
  constexpr int kBuffers = FAR ? 1 : 2;
  constexpr int kTileBytes = kBuffers * 2 * kTile * (int)sizeof(T);
  constexpr int kJoinBytes = FAR ? 32 * DP * 4 : 0;
  __shared__ __attribute__((aligned(128))) char tile_bytes[kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes];
  T* const tiles = reinterpret_cast<T*>(tile_bytes);
  __shared__ __attribute__((aligned(16))) float stat_l[kBuffers][R], stat_d[kBuffers][R];
  __shared__ __attribute__((aligned(16))) int stat_p[kBuffers][R];
  int b, h, tile, split;
  if (!band_place(a, &b, &h, &tile, &split)) return;
  const int splits = a.by_splits.d;
  const long long pair = (long long)b * a.kv_heads + h;
  const int lane = threadIdx.x & 63, wave = wave_of();
  if constexpr (!FAR) {
    zero_spare<T>(a, a.dk, a.dks, h, 1, b, tile * splits + split, a.per);
    zero_spare<T>(a, a.dv, a.dvs, h, 1, b, tile * splits + split, a.per);
  }
  const Entry e = entry_at<false>(a, b);
  const int block_key = FAR ? tile * 32 : tile * kTileKeys128;
  // padded keys past the length still get their (zero) gradient
  const int end = a.offsets ? e.len : a.max_len;
  if (block_key >= (FAR ? std::min(e.len, a.sinks) : end)) return;
  // rows that see a key of the tile: near, from the first key's to the last one's
  // window's end; far, the rest
  const int tile_end = std::min(e.len, (block_key / kTileKeys128 + 1) * kTileKeys128);  // of the near tile
  const int near_end = (int)std::min<long long>(e.len, (long long)tile_end - 1 + a.window);
  const bool all_rows = !FAR && block_key < a.sinks && a.sink_splits == 0;
  const int from = (FAR ? near_end : block_key) * a.group;
  const int until = (FAR || all_rows ? e.len : near_end) * a.group;
  const int steps = until > from ? (until - from + R - 1) / R : 0;
  const int per = split_size(steps, splits, 1);
  const int s0 = split * per, s1 = std::min(steps, s0 + per);
  const T* kb = static_cast<const T*>(a.k) + keys_at(a, a.ks, e, b, h);
  const T* vb = static_cast<const T*>(a.v) + keys_at(a, a.vs, e, b, h);
  const float c2 = a.scale * kLog2e;
  const int key_lo = FAR ? block_key : block_key + wave * 32, key = key_lo + (lane & 31);
  bool in = key < e.len;
  if (in && a.kv_mask) in = a.kv_mask[(a.offsets ? e.row0 : (long long)b * a.mask_stride) + key] != 0;
  Frag<T> k[KK], v[KK];
  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dk[d] = dv[d] = zeros16();
  const f32x2* row_stats = a.stats + pair * a.rows;
  const f32x2 none{INFINITY, 0.f};  // rows that do not exist: weight 0
  RowStage<T, DP, R, FAR, W> st;
  f32x2 stat = none;
  // the row whose L and delta the thread takes (twice over in a wave of its own rows)
  const int stat_row = FAR ? wave * 32 + (lane & 31) : (int)threadIdx.x;
  auto load = [&](int first) {  // (past the last row: that one again)
    st.load(a, e, b, h, first, until);
    stat = row_stats[std::min(first + stat_row, until - 1)];
    if (first + stat_row >= until) stat = none;
  };
  if (s0 < s1) {
    st.start();
    load(from + s0 * R);
  }
  if (e.len > 0) {  // (a key that does not count spoils its own column only, which is zero at the end)
    const int there = std::min(key, e.len - 1);
    load_row16<T, KK, W>(k, kb + (long long)there * a.ks[1], lane, a.head_dim);
    load_row16<T, KK, W>(v, vb + (long long)there * a.vs[1], lane, a.head_dim);
  }
  int buffer = 0;
  for (int step = s0; step < s1; ++step, buffer ^= kBuffers - 1) {
    const int first = from + step * R;
    T* tq = tiles + buffer * 2 * kTile;
    T* tg = tq + kTile;
    st.store(a, tq, tg);
    if (stat_row < R) {
      stat_l[buffer][stat_row] = stat[0];
      stat_d[buffer][stat_row] = -stat[1];
      stat_p[buffer][stat_row] = divided(first + stat_row, a.by_group);
    }
    if constexpr (FAR)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are executed in order
    else
      __syncthreads();
    load(first + R);
#pragma unroll
    for (int n0 = 0; n0 < (FAR ? 32 : R); n0 += 32) {
      const int n = FAR ? wave * 32 : n0;
      const int p_lo = divided(first + n, a.by_group), p_hi = divided(first + n + 31, a.by_group);
      // (of the far walk's rows every one sees every sink)
      const bool far_sinks = key_lo < a.sinks;
      if (!FAR && (p_hi < key_lo || (p_lo - (key_lo + 31) >= a.window && !far_sinks))) continue;
      const bool whole = FAR ? key_lo + 32 <= a.sinks
                             : p_lo >= key_lo + 31 && (p_hi - key_lo < a.window || key_lo + 32 <= a.sinks);
      f32x16 s = zeros16(), dp;
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        const f32x4 d4 = *reinterpret_cast<const f32x4*>(&stat_d[buffer][n + result_row(lane, x)]);
#pragma unroll
        for (int y = 0; y < 4; ++y) dp[x + y] = d4[y];
      }
#pragma unroll
      for (int c = 0; c < KK; ++c) {
        if (!chunk_counts<T>(c, a.head_dim)) continue;
        s = mma32(rows32<DP>(tq, n, c, lane), k[c], s);
        dp = mma32(rows32<DP>(tg, n, c, lane), v[c], dp);
      }
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(&stat_l[buffer][n + result_row(lane, x)]);
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x + y] = __builtin_amdgcn_exp2f(s[x + y] * c2 - l4[y]);
      }
      if (!whole) {
        typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const i32x4 p4 = *reinterpret_cast<const i32x4*>(&stat_p[buffer][n + result_row(lane, x)]);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (!seen(a, p4[y], key)) s[x + y] = dp[x + y] = 0.f;
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) dp[x] *= s[x];
      const Frag<T> p0 = half_of<T, 0>(s), p1 = half_of<T, 1>(s), d0 = half_of<T, 0>(dp), d1 = half_of<T, 1>(dp);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        dv[d] = mma32(cols32<DP>(tg, n, d * 32, lane), p0, dv[d]);
        dk[d] = mma32(cols32<DP>(tq, n, d * 32, lane), d0, dk[d]);
        dv[d] = mma32(cols32<DP>(tg, n + 16, d * 32, lane), p1, dv[d]);
        dk[d] = mma32(cols32<DP>(tq, n + 16, d * 32, lane), d1, dk[d]);
      }
    }
    if constexpr (FAR) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if constexpr (FAR) {
    // the waves' sums, one wave after the other, dK and then dV
    float* sums = reinterpret_cast<float*>(tile_bytes);
    for (int half = 0; half < 2; ++half) {
      for (int w = 0; w < kBandWaves; ++w) {
        __syncthreads();
        if (wave != w) continue;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float* at = sums + (d * 32 + result_row(lane, x)) * 32 + (lane & 31);
            const float mine = half ? dv[d][x] : dk[d][x];
            *at = w ? *at + mine : mine;
          }
      }
      __syncthreads();
      const int keys = std::min(32, a.sinks - block_key);
      for (int i = threadIdx.x; i < keys * a.head_dim; i += kThreads) {
        const int at_key = i / a.head_dim, d = i - at_key * a.head_dim;
        part_far(a, pair, split, block_key + at_key)[half * a.head_dim + d] = sums[d * 32 + at_key];
      }
    }
    return;
  } else {
    if (key >= end) return;
    const bool sink = key < a.sinks && a.sink_splits > 0 && key < e.len;
    if (a.kv_splits > 1 || sink) {
      float* to = part_near(a, pair, split, key);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        store_result<float, 1>(to, d, lane, a.head_dim, dk[d], 1.f);
        store_result<float, 1>(to + a.head_dim, d, lane, a.head_dim, dv[d], 1.f);
      }
      return;
    }
    T* tk = static_cast<T*>(a.dk) + keys_at(a, a.dks, e, b, h) + (long long)key * a.dks[1];
    T* tv = static_cast<T*>(a.dv) + keys_at(a, a.dvs, e, b, h) + (long long)key * a.dvs[1];
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      if (!in) dk[d] = dv[d] = zeros16();
      store_result<T, W>(tk, d, lane, a.head_dim, dk[d], a.scale);
      store_result<T, W>(tv, d, lane, a.head_dim, dv[d], 1.f);
    }
  }
}

// Adds a key's parts of dK and dV, near ones and then far ones, in order: V elements a
// thread, of the keys 0 .. part_keys - 1.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_band_join_kv(BandArgs a) {
  const unsigned per_key = 2 * a.head_dim / V;
  const long long id = (long long)block_id() * kThreads + threadIdx.x;
  const long long at = id / per_key;
  const int d = (int)(id - at * per_key) * V;
  const long long pair = at / a.part_keys;
  const int key = (int)(at - pair * a.part_keys);
  if (pair >= (long long)a.batch * a.kv_heads) return;
  const int h = (int)(pair % a.kv_heads), b = (int)(pair / a.kv_heads);
  const Entry e = entry_at<false>(a, b, false);
  const bool sink = key < a.sinks && a.sink_splits > 0 && key < e.len;
  if (key >= (a.offsets ? e.len : a.max_len) || !(a.kv_splits > 1 || sink)) return;
  float sum[V] = {};
  bool in = key < e.len;
  if (in && a.kv_mask) in = a.kv_mask[(a.offsets ? e.row0 : (long long)b * a.mask_stride) + key] != 0;
  if (in) {
#pragma unroll 4
    for (int s = 0; s < a.kv_splits; ++s) {
      float v[V];
      load_f32<float, V>(part_near(a, pair, s, key) + d, v);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += v[i];
    }
    if (sink) {
#pragma unroll 4
      for (int s = 0; s < a.sink_splits; ++s) {
        float v[V];
        load_f32<float, V>(part_far(a, pair, s, key) + d, v);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += v[i];
      }
    }
  }
  T* to;
  if (d < a.head_dim) {
    to = static_cast<T*>(a.dk) + keys_at(a, a.dks, e, b, h) + (long long)key * a.dks[1] + d;
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] *= a.scale;
  } else {
    to = static_cast<T*>(a.dv) + keys_at(a, a.dvs, e, b, h) + (long long)key * a.dvs[1] + (d - a.head_dim);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) to[i] = (T)sum[i];
}

// ----------------------------------------------------------- sizes, launches
template <typename T, int DP, int W>
void launch_bwd(BandArgs a, hipStream_t s) {
  constexpr int K = kBandKeys<T, DP>;
  const int64_t pairs = (int64_t)a.batch * a.kv_heads;
  const int v = a.head_dim % 4 ? 1 : 4;
  dim3 grid = band_grid(&a, a.row_tiles, a.q_splits);
  hipLaunchKernelGGL((k_band_bwd_q<T, DP, W>), grid, dim3(kThreads), 0, s, a);
  if (a.q_splits > 1) {
    const dim3 blocks((unsigned)((pairs * a.rows * (a.head_dim / v) + kThreads - 1) / kThreads));
    if (v == 4)
      hipLaunchKernelGGL((k_band_join_q<T, 4, K>), blocks, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_band_join_q<T, 1, K>), blocks, dim3(kThreads), 0, s, a);
  }
  grid = band_grid(&a, a.key_tiles, a.kv_splits);
  hipLaunchKernelGGL((k_band_bwd_kv<T, DP, W, false>), grid, dim3(kThreads), 0, s, a);
  if (a.sink_splits) {
    grid = band_grid(&a, a.far_keys / 32, a.sink_splits);
    hipLaunchKernelGGL((k_band_bwd_kv<T, DP, W, true>), grid, dim3(kThreads), 0, s, a);
  }
  if (a.sink_splits || a.kv_splits > 1) {
    const dim3 blocks = grid_of((pairs * a.part_keys * 2 * (a.head_dim / v) + kThreads - 1) / kThreads);
    if (v == 4)
      hipLaunchKernelGGL((k_band_join_kv<T, 4>), blocks, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_band_join_kv<T, 1>), blocks, dim3(kThreads), 0, s, a);
  }
}

template <typename T, int DP>
void launch_bwd_by(int access, const BandArgs& a, hipStream_t s) {
  if (access == 8)
    launch_bwd<T, DP, 8>(a, s);
  else if (access == 2)
    launch_bwd<T, DP, 2>(a, s);
  else
    launch_bwd<T, DP, 1>(a, s);
}

template <typename T>
void launch_bwd_dp(int access, const BandArgs& a, hipStream_t s) {
  switch (band_dp(a.head_dim)) {
    case 32: return launch_bwd_by<T, 32>(access, a, s);
    case 64: return launch_bwd_by<T, 64>(access, a, s);
    case 96: return launch_bwd_by<T, 96>(access, a, s);
    default: return launch_bwd_by<T, 128>(access, a, s);
  }
}

recis_status check_self(const recis_self_attn_desc* d) {
  if (!d || !dtype_known(d->dtype) || d->batch < 0 || d->len < 0 || d->q_heads < 1 || d->kv_heads < 1 ||
      d->head_dim < 1 || d->q_heads % d->kv_heads || !(d->scale > 0.f) || !std::isfinite(d->scale) || d->window < 0 ||
      d->sinks < 0)
    return RECIS_ERR_INVALID_ARG;
  if (d->offsets && (d->lens || d->rows < 0)) return RECIS_ERR_INVALID_ARG;
  if (!aligned_to(d->offsets, 4) || !aligned_to(d->lens, 4) || !aligned_to(d->error, 4)) return RECIS_ERR_INVALID_ARG;
  if (d->head_dim > kMaxHeadDim) return RECIS_ERR_UNSUPPORTED;
  if ((int64_t)d->len * (d->q_heads / d->kv_heads) > (1 << 30) || (int64_t)d->batch * d->kv_heads > (1 << 24))
    return RECIS_ERR_UNSUPPORTED;
  return RECIS_OK;
}

struct SelfPlan {
  int window, sinks;
  int row_tiles, key_tiles, splits, q_splits, kv_splits, sink_splits;
  int64_t part_keys, far_keys;
  int64_t ml_at, fwd_bytes, dq_at, kv_at, bwd_bytes;
  bool launchable[2];
};

SelfPlan self_plan(const recis_self_attn_desc* d) {
  SelfPlan p;
  const int group = d->q_heads / d->kv_heads;
  const int64_t rows = (int64_t)d->len * group, pairs = (int64_t)d->batch * d->kv_heads;
  const int keys = band_keys(d->dtype, d->head_dim);
  // a window that no row fills: none, and nothing for sinks to add
  const bool band = d->window && d->window < d->len;
  p.window = band ? d->window : 1 << 30;
  p.sinks = band ? std::min(d->sinks, d->len) : 0;
  p.row_tiles = std::max<int64_t>(1, (rows + kBandRows - 1) / kBandRows);
  p.key_tiles = std::max(1, (d->len + kTileKeys128 - 1) / kTileKeys128);
  const int64_t near = band ? (int64_t)d->window + kBandRows / group + 1 + p.sinks : d->len;
  const int64_t walk = d->len ? std::min<int64_t>(d->len, near) / keys + 2 : 0;  // (no keys: packed rows of no entry)
  // keys (rows) are split until there are `want` blocks
  auto split = [&](int64_t blocks, int64_t want, int64_t most) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, want / std::max<int64_t>(1, blocks), most}));
  };
  p.splits = p.q_splits = split(pairs * p.row_tiles, 1024, (walk + kLeastTiles - 1) / kLeastTiles);
  const int64_t row_steps = (std::min<int64_t>(d->len, band ? d->window + kTileKeys128 : d->len) * group + 63) / 64;
  p.kv_splits = split(pairs * p.key_tiles, 512, (row_steps + 1) / 2);
  p.sink_splits = 0;
  p.far_keys = p.part_keys = 0;
  if (p.sinks > 0 && p.sinks <= kMostFarSinks) {
    p.far_keys = round_up(p.sinks, 32);
    p.part_keys = p.far_keys;
    // parts of 8 steps of 128 rows, less where that leaves the chip empty
    const int64_t steps = std::max<int64_t>(1, rows / 128);
    p.sink_splits = (int)std::max<int64_t>(
        1, std::min<int64_t>({64, steps, std::max<int64_t>(steps / 8, 512 / std::max<int64_t>(1, pairs))}));
  }
  if (p.kv_splits > 1) p.part_keys = (int64_t)p.key_tiles * kTileKeys128;
  const int64_t cells = std::max<int64_t>(pairs * rows, 1);
  p.ml_at = p.splits > 1 ? round_up(cells * p.splits * d->head_dim * 4, 256) : 0;
  p.fwd_bytes = p.splits > 1 ? p.ml_at + round_up(cells * p.splits * 8, 256) : 0;
  p.dq_at = round_up(cells * 8, 256);
  p.kv_at = p.dq_at + (p.q_splits > 1 ? round_up(cells * p.q_splits * d->head_dim * 4, 256) : 0);
  p.bwd_bytes = p.kv_at;
  if (p.part_keys)
    p.bwd_bytes += round_up(std::max<int64_t>(pairs, 1) * (p.kv_splits * p.part_keys + p.sink_splits * p.far_keys) * 2 *
                                d->head_dim * 4, 256);
  auto fits = [&](int64_t per) { return round_up(pairs, (int64_t)kDies * d->kv_heads) * per <= kMaxBlocks; };
  p.launchable[0] = fits((int64_t)p.row_tiles * p.splits);
  p.launchable[1] = p.launchable[0] && fits((int64_t)p.key_tiles * p.kv_splits) &&
                    fits(std::max<int64_t>(1, p.far_keys / 32) * std::max(1, p.sink_splits)) &&
                    pairs * p.part_keys * 2 * d->head_dim / kThreads < kMaxBlocks;
  return p;
}

void fill_self(const recis_self_attn_desc* d, const SelfPlan& p, BandArgs* a) {
  *a = BandArgs{};
  a->offsets = d->offsets;
  a->lens = d->lens;
  a->kv_mask = d->kv_mask;
  a->error = d->error;
  a->mask_stride = d->mask_stride;
  a->total_rows = d->rows;
  const int64_t lead[2] = {d->offsets ? 1 : d->batch, d->offsets ? d->rows : d->len};
  const int64_t q_axes[3] = {lead[0], lead[1], d->q_heads}, kv_axes[3] = {lead[0], lead[1], d->kv_heads};
  for (int i = 0; i < 3; ++i) {
    a->qs[i] = stride_of(d->q_strides[i], q_axes[i]);
    a->ks[i] = stride_of(d->k_strides[i], kv_axes[i]);
    a->vs[i] = stride_of(d->v_strides[i], kv_axes[i]);
    a->os[i] = stride_of(d->o_strides[i], q_axes[i]);
    a->dos[i] = stride_of(d->do_strides[i], q_axes[i]);
    a->dqs[i] = stride_of(d->dq_strides[i], q_axes[i]);
    a->dks[i] = stride_of(d->dk_strides[i], kv_axes[i]);
    a->dvs[i] = stride_of(d->dv_strides[i], kv_axes[i]);
  }
  a->batch = d->batch;
  a->q_len = a->max_len = d->len;
  a->q_heads = d->q_heads;
  a->kv_heads = d->kv_heads;
  a->group = d->q_heads / d->kv_heads;
  a->head_dim = d->head_dim;
  a->rows = d->len * a->group;
  a->causal = 1;
  a->window = p.window;
  a->sinks = p.sinks;
  a->by_page = Quick(1);
  a->by_group = Quick(a->group);
  a->by_kv_heads = Quick(d->kv_heads);
  a->row_tiles = p.row_tiles;
  a->key_tiles = p.key_tiles;
  a->splits = p.splits;
  a->q_splits = p.q_splits;
  a->kv_splits = p.kv_splits;
  a->sink_splits = p.sink_splits;
  a->part_keys = (int)p.part_keys;
  a->far_keys = (int)p.far_keys;
  place_pairs(a, d->dtype);
  a->scale = d->scale;
}

// Rows can be moved 16 bytes at a time.
int self_access(int dtype, const BandArgs& a, std::initializer_list<const void*> ptrs,
                std::initializer_list<const long long*> strides) {
  const int access = band_access(dtype, a.head_dim, ptrs, strides);
  // a tile's rows stay within 32 bits of byte offset
  for (const long long* s : {a.ks, a.vs})
    if (access == 8 && (s[1] < 0 || s[1] >= (1 << 23))) return 1;
  return access;
}

bool all_there(const recis_self_attn_desc* d, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p || !aligned_to(p, dtype_size(d->dtype))) return false;
  return true;
}

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

int64_t recis_self_attn_workspace_bytes(const recis_self_attn_desc* desc, int32_t backward) {
  if (check_self(desc) != RECIS_OK) return -1;
  const SelfPlan p = self_plan(desc);
  if (!p.launchable[backward ? 1 : 0]) return -1;
  return backward ? p.bwd_bytes : p.fwd_bytes;
}

recis_status recis_self_attn_fwd(const recis_self_attn_desc* desc, const void* q, const void* k, const void* v,
                                 void* out, float* lse, void* workspace, int64_t workspace_bytes, hipStream_t s) {
  const recis_status st = check_self(desc);
  if (st != RECIS_OK) return st;
  if (desc->batch == 0 || (desc->offsets ? desc->rows : desc->len) == 0) return RECIS_OK;
  if (!all_there(desc, {q, k, v, out}) || !aligned_to(lse, 4)) return RECIS_ERR_INVALID_ARG;
  const SelfPlan p = self_plan(desc);
  if (!p.launchable[0]) return RECIS_ERR_UNSUPPORTED;
  if (p.fwd_bytes && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.fwd_bytes))
    return RECIS_ERR_INVALID_ARG;
  BandArgs a;
  fill_self(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ml_at);
  const int access = self_access(desc->dtype, a, {q, k, v, out}, {a.qs, a.ks, a.vs, a.os});
  launch_band_fwd(desc->dtype, false, access, a, s);
  return launch_status();
}

recis_status recis_self_attn_bwd(const recis_self_attn_desc* desc, const void* grad_out, const void* q, const void* k,
                                 const void* v, const void* out, const float* lse, void* grad_q, void* grad_k,
                                 void* grad_v, void* workspace, int64_t workspace_bytes, hipStream_t s) {
  const recis_status st = check_self(desc);
  if (st != RECIS_OK) return st;
  if (desc->batch == 0 || (desc->offsets ? desc->rows : desc->len) == 0) return RECIS_OK;
  if (!all_there(desc, {grad_out, q, k, v, out, grad_q, grad_k, grad_v}) || !lse || !aligned_to(lse, 4))
    return RECIS_ERR_INVALID_ARG;
  const SelfPlan p = self_plan(desc);
  if (!p.launchable[1]) return RECIS_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bwd_bytes) return RECIS_ERR_INVALID_ARG;
  BandArgs a;
  fill_self(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = out;
  a.dout = grad_out;
  a.lse = const_cast<float*>(lse);
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  a.stats = static_cast<f32x2*>(workspace);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.dq_at);
  a.part_kv = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.kv_at);
  const int access = self_access(desc->dtype, a, {q, k, v, out, grad_out, grad_q, grad_k, grad_v},
                                 {a.qs, a.ks, a.vs, a.os, a.dos, a.dqs, a.dks, a.dvs});
  if (desc->dtype == RECIS_DTYPE_BF16)
    launch_bwd_dp<__bf16>(access, a, s);
  else
    launch_bwd_dp<float>(access, a, s);
  return launch_status();
}

}  // extern "C"
