// attn.hip -- cross attention of queries to the keys and values of another
// sequence, forward and backward.
//
// For each batch entry and key head h, with the G = q_heads / kv_heads query
// heads that share it folded into the rows (row = query * G + g; no mask here
// tells rows of a batch entry apart, so the fold changes nothing):
//
//   S = scale Q K^T (masked keys left out),  L = log sum exp S,  P = exp(S - L),  O = P V
//   dV = P^T dO,  dP = dO V^T,  delta = sum dO O,  dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q
//
// Scores, the running maximum and sum, and every product's sum are float32.
// P and dS are rounded to the inputs' type where they enter a matrix product
// (the matrix unit takes no wider operand beside a bfloat16 one).
//
// All products run on 16x16 matrix instructions.  A product's operands hold,
// per lane, 8 consecutive k of one row (lane % 16), k from 8 * (lane / 16);
// its result holds column lane % 16 and rows 4 * (lane / 16) + 0..3.  The
// scores are computed transposed (keys as rows, queries as columns), so a lane
// holds keys of one query: the softmax needs two shuffles a tile, and two
// result tiles of 16 keys are, after rounding, the operand of the next product
// for 32 keys -- in an order of keys that the other operand follows (slot j of
// lane group g is key 4 g + j for j < 4, and 16 + 4 g + j - 4 above).
#include <algorithm>
#include <cmath>

#include "attn.h"

namespace recis {
namespace {

struct AttnArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  float* lse;
  f32x2* stats;  // [batch * kv_heads][rows], from k_attn_bwd_q to k_attn_bwd_kv
  const int *kv_offsets, *kv_lens;
  const unsigned char* kv_mask;
  long long mask_stride, kv_rows;
  long long qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];  // batch, row, head
  int batch, q_len, kv_len, q_heads, kv_heads, group, head_dim;
  int rows;                // q_len * group
  int row_tiles, key_tiles;
  int dies, unit;              // `unit` pairs of (batch entry, key head) share a die, `dies` units lie side by side
  int splits, split_keys;      // forward: key ranges of a row tile, joined by k_attn_join
  int q_splits, q_split_keys;  // dQ: the same, joined by k_attn_join_q
  float scale;
  float *part_o, *part_ml;     // [batch * kv_heads][splits][rows][head_dim], [..][2]
  int* kept;                   // [batch][kKeptWords], from k_attn_kept to k_attn_bwd_q; or null
  unsigned* error;
};

// ---------------------------------------------------------- keys of an entry
struct Span {
  long long row0;  // first row of the packed keys (0 when padded)
  int len;
};

__device__ __forceinline__ Span kv_span(const AttnArgs& a, int b) {
  Span s{0, a.kv_len};
  bool bad = false;
  if (a.kv_offsets) {
    long long lo = a.kv_offsets[b], hi = a.kv_offsets[b + 1];
    bad = lo < 0 || hi < lo || hi > a.kv_rows || hi - lo > a.kv_len;
    if (bad) lo = hi = 0;
    s.row0 = lo;
    s.len = (int)(hi - lo);
  } else if (a.kv_lens) {
    const int n = a.kv_lens[b];
    bad = n < 0 || n > a.kv_len;
    s.len = bad ? 0 : n;
  }
  if (bad && a.error && threadIdx.x == 0) atomicOr(a.error, kErrInvalid);
  return s;
}

template <typename T>
__device__ __forceinline__ const T* kv_base(const void* p, const long long (&st)[3], const AttnArgs& a, const Span& s,
                                            int b, int h) {
  return static_cast<const T*>(p) + (a.kv_offsets ? s.row0 * st[1] : (long long)b * st[0]) + (long long)h * st[2];
}

// Bit i: key first + i counts.
__device__ __forceinline__ unsigned long long key_bits(const AttnArgs& a, const Span& s, int b, int first, int lane) {
  const int key = first + lane;
  bool in = key < s.len;
  if (in && a.kv_mask) in = a.kv_mask[(a.kv_offsets ? s.row0 : (long long)b * a.mask_stride) + key] != 0;
  return __ballot(in);
}

// The same for a tile of KEYS keys; the bits past it are set (a whole tile is all ones).
template <int KEYS>
__device__ __forceinline__ unsigned long long tile_bits(const AttnArgs& a, const Span& s, int b, int first, int lane) {
  const unsigned long long bits = key_bits(a, s, b, first, lane);
  return KEYS == 64 ? bits : bits | (~0ull << 32);
}
template <int KEYS>
__device__ __forceinline__ bool no_key(unsigned long long bits) {
  return KEYS == 64 ? bits == 0 : (unsigned)bits == 0;
}

// Consecutive blocks go to the eight dies in turn; `unit` (batch entry, key
// head) pairs, all blocks of each, share a die and its L2.
//  - Where the keys are read once (one row tile), all heads of an entry: its
//    positions' memory is then read by one die, in one stretch (single queries,
//    up to 8192 keys, 4 heads of 128 bfloat16: 64 entries 116 us against 126,
//    128 232 against 256), and heads shorter than a 128-byte line are not
//    fetched once per die (50 queries, up to 1000 keys, 4 heads of 32: 512
//    entries 29 us against 46).  Below 64 entries both take the same time
//    within 5% (16: 40.3 and 40.4, 48: 89 and 91; 11.0 and 11.0 with 32).
//  - Where there is more to compute than to read, one pair, so that entries of
//    unequal length spread over the dies (512 queries, up to 1000 keys, 8 heads
//    of 64 bfloat16, both passes: 512 pairs 271 us against 303, 256 156 against
//    169, 128 149 against 151).
//  - With few pairs that leaves dies idle, and a pair's blocks go to every die
//    (the same: 16 pairs 64 us against 69, 32 91 against 97, 64 112 against
//    114; 96 123 against 122).
constexpr int kDies = 8, kEntriesForDies = 64, kPairsForDies = 128;
__device__ __forceinline__ bool place(const AttnArgs& a, int per, int* b, int* h, int* t) {
  const int id = block_id(), slot = id / a.dies, across = per * a.unit;
  const int rest = slot % across;
  const int bh = ((slot / across) * a.dies + id % a.dies) * a.unit + rest / per;
  *t = rest % per;
  *b = bh / a.kv_heads;
  *h = bh % a.kv_heads;
  return bh < a.batch * a.kv_heads;
}

// Row r of the folded queries: offset of its head vector in a tensor.
__device__ __forceinline__ long long row_at(const AttnArgs& a, const long long (&st)[3], int b, int h, int r) {
  const int q = r / a.group, g = r - q * a.group;
  return (long long)b * st[0] + (long long)q * st[1] + (long long)(h * a.group + g) * st[2];
}

__device__ __forceinline__ long long stat_at(const AttnArgs& a, int b, int h, int r) {
  const int q = r / a.group, g = r - q * a.group;
  return ((long long)b * a.q_len + q) * a.q_heads + h * a.group + g;
}

// 8 elements at a base that every lane shares plus the lane's own byte offset
// (one 32-bit register of address for all of a thread's loads).
template <typename T>
__device__ __forceinline__ Frag<T> load_at(const T* base, unsigned bytes) {
  return *reinterpret_cast<const Frag<T>*>(reinterpret_cast<const char*>(base) + bytes);
}

// A tile of R rows x DP held in registers on its way to LDS.
template <typename T, int DP, int R, bool ALN>
struct Stage {
  static constexpr int kAcross = kCols<DP> / 8;     // chunks of 8 columns
  static constexpr int kStep = kThreads / kAcross;  // rows between a thread's chunks
  static constexpr int kPer = (R + kStep - 1) / kStep;
  Frag<T> f[kPer];
  const T* base;
  int row, d0;
  unsigned at;
  __device__ __forceinline__ void start(const T* from, long long stride, int first) {
    row = threadIdx.x / kAcross;
    d0 = (threadIdx.x % kAcross) * 8;
    at = (unsigned)((row * stride + d0) * (long long)sizeof(T));  // ALN: fits (rows_aligned)
    base = from + (long long)first * stride;
  }
  // rows whose bit is clear are zero, whatever memory holds there
  __device__ __forceinline__ void load(long long stride, unsigned long long bits, int dim) {
    if (ALN && R == kPer * kStep && bits == ~0ull) {
      if (dim == kCols<DP>) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = load_at<T>(base + (long long)(i * kStep) * stride, at);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = Frag<T>{};
        if (d0 < dim) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) f[i] = load_at<T>(base + (long long)(i * kStep) * stride, at);
        }
      }
    } else {
      const unsigned long long mine = bits >> row;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = row + i * kStep < R && ((mine >> (i * kStep)) & 1);
        if constexpr (ALN) {
          f[i] = Frag<T>{};
          if (in && d0 < dim) f[i] = load_at<T>(base + (long long)(i * kStep) * stride, at);
        } else {
          f[i] = load8<T, ALN>(base + (long long)(row + i * kStep) * stride, d0, dim, in);
        }
      }
    }
    base += (long long)R * stride;
  }
  __device__ __forceinline__ void store(T* tile) const {
    if (d0 >= DP) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (R == kPer * kStep || row + i * kStep < R)
        *reinterpret_cast<Frag<T>*>(tile + chunk_at<T, DP>(row + i * kStep, d0 / 8)) = f[i];
  }
};

// Keys a tile: 64, or 32 where two buffers of 64 would leave one block a CU.
constexpr int kBlockKeys = 64;
template <typename T, int DP>
constexpr int kTileKeys = sizeof(T) == 4 && DP > 64 ? 32 : 64;
constexpr int kAttnWaves = kThreads / 64;

// ------------------------------------------------------------------ forward
// Bound by vector instructions, mostly: a 16 x 16 tile of scores takes 4 matrix
// instructions (head 64) of 16 cycles, and per lane 4 scores' multiply-add,
// exponential (at a quarter of the rate), sum and maximum.  Vector instructions
// take 58% of the SIMDs' busy cycles and the exponentials' rate some 20% more,
// the matrix unit 26%.  128 entries, 512 queries, 8 heads of 64, 0 to 1000 keys,
// bfloat16: 150 us, 447 TFLOP/s of the keys that count (32 queries a wave, 2
// tiles; 16: 182 us).  50 queries, 4 heads of 32, 512 entries: 35 us, 144 MB of
// unavoidable traffic at 4.1 TB/s.
//
// A wave holds QT tiles of 16 queries; the block walks the keys 64 at a time,
// staged in LDS for its four waves in two buffers (one barrier a tile), the
// next tile's loads in flight meanwhile.  The running maximum that the weights
// are taken relative to is raised only once a score exceeds it by 2^kSlack in
// weight: the sum and the output stay exact relative to it, far from float32's
// range, and most tiles need no rescaling of the output.
constexpr float kSlack = 8.f;
template <typename T, int DP, int QT, bool ALN>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && DP <= 64 ? 3 : 1) void k_attn_fwd(AttnArgs a) {
  constexpr int KK = kChunks32<DP>, DT = DP / 16, kKeys = kTileKeys<T, DP>, NT = kKeys / 16;
  constexpr int kTile = kKeys * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  int b, h, t;
  if (!place(a, a.row_tiles * a.splits, &b, &h, &t)) return;
  const int split = t % a.splits, tile = t / a.splits;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Span sp = kv_span(a, b);
  const int key0 = split * a.split_keys;
  const int key1 = std::min(sp.len, key0 + a.split_keys);
  const T* kb = kv_base<T>(a.k, a.ks, a, sp, b, h);
  const T* vb = kv_base<T>(a.v, a.vs, a, sp, b, h);
  const int row0 = tile * (16 * QT * kAttnWaves) + wave * 16 * QT + (lane & 15);
  Frag<T> q[QT][KK];
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    const int r = row0 + j * 16;
    const bool in = r < a.rows;
    const T* p = static_cast<const T*>(a.q) + (in ? row_at(a, a.qs, b, h, r) : 0);
#pragma unroll
    for (int c = 0; c < KK; ++c) q[j][c] = load_head<T, ALN>(p, c, lane, a.head_dim, in);
  }
  f32x4 o[QT][DT];
  // maximum, the same in log2 of the weight (0 before the first key), how far a
  // score may go before both are raised, sum
  float m[QT], ref[QT], most[QT], l[QT];
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    m[j] = most[j] = -INFINITY;
    ref[j] = l[j] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float c2 = a.scale * kLog2e;
  const f32x4 zero = zeros();
  Stage<T, DP, kKeys, ALN> sk, sv;
  unsigned long long bits = 0;
  if (key0 < key1) {
    sk.start(kb, a.ks[1], key0);
    sv.start(vb, a.vs[1], key0);
    bits = tile_bits<kKeys>(a, sp, b, key0, lane);
    sk.load(a.ks[1], bits, a.head_dim);
    sv.load(a.vs[1], bits, a.head_dim);
  }
  int buffer = 0;
  for (int first = key0; first < key1; first += kKeys, buffer ^= 1) {
    T* tk = tiles + buffer * 2 * kTile;
    T* tv = tk + kTile;
    sk.store(tk);
    sv.store(tv);
    __syncthreads();
    const unsigned long long now = bits;
    if (first + kKeys < key1) {
      bits = tile_bits<kKeys>(a, sp, b, first + kKeys, lane);
      sk.load(a.ks[1], bits, a.head_dim);
      sv.load(a.vs[1], bits, a.head_dim);
    }
    if (no_key<kKeys>(now)) continue;
    f32x4 s[NT][QT];
    // as many operands ahead as 32 registers hold
    constexpr int kAhead = std::max(1, std::min(NT, 16 * 4 / (KK * (int)sizeof(Frag<T>))));
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kAhead) {
      Frag<T> f[kAhead][KK];
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
#pragma unroll
        for (int c = 0; c < KK; ++c) f[n][c] = read_rows<DP>(tk, (n0 + n) * 16, c, lane);
      reads_before();
      // a sum's next product is issued as late as it can be
#pragma unroll
      for (int c = 0; c < KK; ++c)
#pragma unroll
        for (int n = 0; n < kAhead; ++n)
#pragma unroll
          for (int j = 0; j < QT; ++j) s[n0 + n][j] = mma_head<DP>(f[n][c], q[j][c], c == 0 ? zero : s[n0 + n][j], c);
    }
    if (now != ~0ull) {
      const unsigned long long mine = now >> ((lane >> 4) * 4);  // this lane's keys: constant bits from here on
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((mine >> (n * 16 + i)) & 1))
#pragma unroll
            for (int j = 0; j < QT; ++j) s[n][j][i] = -INFINITY;
    }
    float top[QT];
    bool raise = false;
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      top[j] = s[0][j][0];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[j] = fmaxf(top[j], s[n][j][i]);
      top[j] = group_max(top[j]);
      raise |= top[j] * c2 > most[j];
    }
    if (__any(raise)) {
#pragma unroll
      for (int j = 0; j < QT; ++j) {
        const float to = fmaxf(m[j], top[j]);
        ref[j] = to == -INFINITY ? 0.f : to * c2;
        const float alpha = __builtin_amdgcn_exp2f(m[j] * c2 - ref[j]);
        m[j] = to;
        most[j] = to == -INFINITY ? -INFINITY : ref[j] + kSlack;
        l[j] *= alpha;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[j][d] *= alpha;
      }
    }
#pragma unroll
    for (int j = 0; j < QT; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[n][j][i] = __builtin_amdgcn_exp2f(s[n][j][i] * c2 - ref[j]);
          l[j] += s[n][j][i];
        }
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      Frag<T> p[QT];
#pragma unroll
      for (int j = 0; j < QT; ++j) p[j] = pack<T>(s[n][j], s[n + 1][j]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const Frag<T> f = read_cols<DP>(tv, n * 16, d * 16, lane);
#pragma unroll
        for (int j = 0; j < QT; ++j) o[j][d] = mma(f, p[j], o[j][d]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    const int r = row0 + j * 16;
    l[j] = group_add(l[j]);
    if (r >= a.rows) continue;
    if (a.splits > 1) {
      const long long at = (((long long)b * a.kv_heads + h) * a.splits + split) * a.rows + r;
      float* po = a.part_o + at * a.head_dim;
#pragma unroll
      for (int d = 0; d < DT; ++d) store4<float, false>(po, d * 16 + (lane >> 4) * 4, a.head_dim, o[j][d]);
      if (lane < 16) {
        a.part_ml[2 * at] = m[j] * c2;
        a.part_ml[2 * at + 1] = l[j];
      }
      continue;
    }
    const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
    T* out = static_cast<T*>(a.out) + row_at(a, a.os, b, h, r);
#pragma unroll
    for (int d = 0; d < DT; ++d) store4<T, ALN>(out, d * 16 + (lane >> 4) * 4, a.head_dim, o[j][d] * inv);
    if (a.lse && lane < 16)
      a.lse[stat_at(a, b, h, r)] = l[j] == 0.f ? -INFINITY : m[j] * a.scale + __logf(l[j]);
  }
}

// Bound by memory: the keys and values are read once.  64 entries of 0 to 8192
// keys, 16 query heads on 4 of 128, bfloat16: 537 MB in 113 us, 4.8 TB/s, the
// rate of a large copy (with the join, 118; the many-rows kernel took 120 and
// 10 to join).  4 entries of up to 200 keys, 4 heads of 32, float32: 6.3 us
// (10.4 with four waves sharing a tile).
//
// Few rows (16 at most: single queries, and their heads): the block's waves
// take turns of 32 keys and meet once, at the end.  Keys go from memory into
// the product's operand directly, values through LDS of the wave's own, so no
// wave waits for another while the keys stream.
constexpr int kFewRows = 16, kFewKeys = 32;

template <typename T, int DP, bool ALN>
__global__ __launch_bounds__(kThreads) void k_attn_few(AttnArgs a) {
  constexpr int KK = kChunks32<DP>, DT = DP / 16;
  constexpr int kAcross = kCols<DP> / 8, kRows = 64 / kAcross, kPer = kFewKeys / kRows;  // chunks of values a lane
  constexpr int kTile = kFewKeys * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[kAttnWaves * kTile];
  __shared__ float refs[kAttnWaves][kFewRows], sums[kAttnWaves][kFewRows];
  static_assert(kTile * (int)sizeof(T) >= kFewRows * DP * 4, "a wave's output fits its tile");
  int b, h, split;
  if (!place(a, a.splits, &b, &h, &split)) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Span sp = kv_span(a, b);
  const int key0 = split * a.split_keys;
  const int key1 = std::min(sp.len, key0 + a.split_keys);
  const T* kb = kv_base<T>(a.k, a.ks, a, sp, b, h);
  const T* vb = kv_base<T>(a.v, a.vs, a, sp, b, h);
  const float c2 = a.scale * kLog2e;
  const f32x4 zero = zeros();
  Frag<T> q[KK];
  {
    const int r = lane & 15;
    const bool in = r < a.rows;
    const T* p = static_cast<const T*>(a.q) + (in ? row_at(a, a.qs, b, h, r) : 0);
#pragma unroll
    for (int c = 0; c < KK; ++c) q[c] = load_head<T, ALN>(p, c, lane, a.head_dim, in);
  }
  Frag<T> kf[2][KK], vf[kPer];
  // a lane's key in the operand of 16 keys, and its place in 64 chunks of values
  const int kr = lane & 15, vr = lane / kAcross, vd = (lane % kAcross) * 8;
  constexpr int kHalf = sizeof(T) == 2 ? 8 : 4;  // the operand's first elements (load_head)
  const int kd = (lane >> 4) * kHalf;
  const unsigned k_at = (unsigned)((kr * a.ks[1] + kd) * (long long)sizeof(T));  // ALN: fits (rows_aligned)
  const unsigned v_at = (unsigned)((vr * a.vs[1] + vd) * (long long)sizeof(T));
  auto fetch = [&](int first, unsigned bits) {
    const T* kp = kb + (long long)first * a.ks[1];
    const T* vp = vb + (long long)first * a.vs[1];
    if (ALN && bits == ~0u && a.head_dim == kCols<DP>) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          const T* from = kp + u * 16 * a.ks[1] + c * 32;
          if constexpr (sizeof(T) == 2) {
            kf[u][c] = load_at<T>(from, k_at);
          } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(from) + k_at);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(from + 16) + k_at);
            kf[u][c] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        }
#pragma unroll
      for (int i = 0; i < kPer; ++i) vf[i] = load_at<T>(vp + (long long)(i * kRows) * a.vs[1], v_at);
      return;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < KK; ++c)
        kf[u][c] = load_head<T, ALN>(kp + (long long)(u * 16 + kr) * a.ks[1], c, lane, a.head_dim,
                                     (bits >> (u * 16 + kr)) & 1);
    const unsigned mine = bits >> vr;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool in = (mine >> (i * kRows)) & 1;
      if constexpr (ALN) {
        vf[i] = Frag<T>{};
        if (in && vd < a.head_dim) vf[i] = load_at<T>(vp + (long long)(i * kRows) * a.vs[1], v_at);
      } else {
        vf[i] = load8<T, ALN>(vp + (long long)(i * kRows + vr) * a.vs[1], vd, a.head_dim, in);
      }
    }
  };
  f32x4 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = zero;
  float m = -INFINITY, ref = 0.f, most = -INFINITY, l = 0.f;
  T* tv = tiles + wave * kTile;
  constexpr int kStep = kFewKeys * kAttnWaves;
  unsigned bits = 0;
  int first = key0 + wave * kFewKeys;
  if (first < key1) {
    bits = (unsigned)key_bits(a, sp, b, first, lane);
    fetch(first, bits);
  }
  for (; first < key1; first += kStep) {
    const unsigned now = bits;
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = zero;
#pragma unroll
      for (int c = 0; c < KK; ++c) s[u] = mma_head<DP>(kf[u][c], q[c], s[u], c);
    }
    if (vd < DP) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        *reinterpret_cast<Frag<T>*>(tv + chunk_at<T, DP>(i * kRows + vr, vd / 8)) = vf[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are executed in order
    if (first + kStep < key1) {
      bits = (unsigned)key_bits(a, sp, b, first + kStep, lane);
      fetch(first + kStep, bits);
    }
    if (now != ~0u) {
      const unsigned mine = now >> ((lane >> 4) * 4);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((mine >> (u * 16 + i)) & 1)) s[u][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[u][i]);
    top = group_max(top);
    if (__any(top * c2 > most)) {
      const float to = fmaxf(m, top);
      ref = to == -INFINITY ? 0.f : to * c2;
      const float alpha = __builtin_amdgcn_exp2f(m * c2 - ref);
      m = to;
      most = to == -INFINITY ? -INFINITY : ref + kSlack;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= alpha;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[u][i] = __builtin_amdgcn_exp2f(s[u][i] * c2 - ref);
        l += s[u][i];
      }
    const Frag<T> p = pack<T>(s[0], s[1]);
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = mma(read_cols<DP>(tv, 0, d * 16, lane), p, o[d]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  l = group_add(l);
  float* mine = reinterpret_cast<float*>(tv);  // [row][DP]
#pragma unroll
  for (int d = 0; d < DT; ++d)
    *reinterpret_cast<f32x4*>(mine + (lane & 15) * DP + d * 16 + (lane >> 4) * 4) = o[d];
  if (lane < 16) {
    refs[wave][lane] = m * c2;
    sums[wave][lane] = l;
  }
  __syncthreads();
  // 16 threads a row, DT elements each
  const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * DT;
  if (r >= a.rows) return;
  float top = refs[0][r];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, refs[w][r]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, out[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) out[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    const float weight = __builtin_amdgcn_exp2f(refs[w][r] - base);
    sum += weight * sums[w][r];
    const float* from = reinterpret_cast<const float*>(tiles + w * kTile) + r * DP + d0;
#pragma unroll
    for (int i = 0; i < DT; ++i) out[i] += weight * from[i];
  }
  if (a.splits > 1) {
    const long long at = (((long long)b * a.kv_heads + h) * a.splits + split) * a.rows + r;
#pragma unroll
    for (int i = 0; i < DT; ++i)
      if (d0 + i < a.head_dim) a.part_o[at * a.head_dim + d0 + i] = out[i];
    if (d0 == 0) {
      a.part_ml[2 * at] = top;
      a.part_ml[2 * at + 1] = sum;
    }
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* to = static_cast<T*>(a.out) + row_at(a, a.os, b, h, r);
#pragma unroll
  for (int i = 0; i < DT; ++i)
    if (d0 + i < a.head_dim) to[d0 + i] = (T)(out[i] * inv);
  if (a.lse && d0 == 0) a.lse[stat_at(a, b, h, r)] = sum == 0.f ? -INFINITY : top * kLn2 + __logf(sum);
}

// Joins the key ranges of many rows: V elements of a row a thread.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_attn_join_many(AttnArgs a) {
  const unsigned per = a.head_dim / V;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;
  const unsigned row = id / per, d = (id - row * per) * V;
  const unsigned bh = row / a.rows, r = row - bh * a.rows;
  if (bh >= (unsigned)(a.batch * a.kv_heads)) return;
  const int h = (int)bh % a.kv_heads, b = (int)bh / a.kv_heads;
  const long long at = (long long)bh * a.splits * a.rows + r;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.part_ml);
  float top = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, ml[at + (long long)s * a.rows][0]);
  const float ref = top == -INFINITY ? 0.f : top;
  float o[V] = {}, l = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
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
  T* out = static_cast<T*>(a.out) + row_at(a, a.os, b, h, r) + d;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = (T)(o[i] * inv);
  if (a.lse && d == 0) a.lse[stat_at(a, b, h, r)] = l == 0.f ? -INFINITY : top * kLn2 + __logf(l);
}

// The same for few rows: a block a row, consecutive ranges for each wave.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn_join_few(AttnArgs a) {
  constexpr int kParts = kMaxHeadDim / 64;
  __shared__ float part[kAttnWaves][kMaxHeadDim + 1];
  const int lane = threadIdx.x & 63, wave = wave_of();
  const int r = (int)(blockIdx.x % a.rows), bh = (int)(blockIdx.x / a.rows);
  const int h = bh % a.kv_heads, b = bh / a.kv_heads;
  const long long at = (long long)bh * a.splits * a.rows + r;
  float top = -INFINITY, o[kParts] = {}, l = 0.f;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.part_ml[2 * (at + (long long)s * a.rows)]);
  top = group_max(top);
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
  const float ref = top == -INFINITY ? 0.f : top;
  const int per = (a.splits + kAttnWaves - 1) / kAttnWaves;
  const int s1 = std::min(a.splits, (wave + 1) * per);
#pragma unroll 4
  for (int s = wave * per; s < s1; ++s) {
    const long long p = at + (long long)s * a.rows;
    const float weight = __builtin_amdgcn_exp2f(a.part_ml[2 * p] - ref);
    l += weight * a.part_ml[2 * p + 1];
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
  for (int k = 1; k < kAttnWaves; ++k) {
    l += part[k][kMaxHeadDim];
#pragma unroll
    for (int i = 0; i < kParts; ++i) o[i] += part[k][lane + 64 * i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + row_at(a, a.os, b, h, r);
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    if (lane + 64 * i < a.head_dim) out[lane + 64 * i] = (T)(o[i] * inv);
  if (a.lse && lane == 0) a.lse[stat_at(a, b, h, r)] = l == 0.f ? -INFINITY : top * kLn2 + __logf(l);
}

// ----------------------------------------------------------------- backward
// The keys that a mask leaves an entry, where they are 64 at most: their number
// and places, in order.  (More: a number above 64.)  A block an entry, 8 * 64
// keys a wave and round.  A kernel of its own because k_attn_bwd_q's blocks would
// each count again: 4 entries of 8192 keys, 50 queries, 8 heads of 64, about 40
// keys left, the backward takes 71 us so, 111 us otherwise and 58 with delta from
// out; with 90% left 68 us, 71 and 65.
constexpr int kMostKept = 64, kKeptWords = 1 + kMostKept;
__global__ __launch_bounds__(kThreads) void k_attn_kept(AttnArgs a) {
  __shared__ int counts[kAttnWaves];
  const int b = block_id(), lane = threadIdx.x & 63, wave = wave_of();
  if (b >= a.batch) return;
  const Span sp = kv_span(a, b);
  int* list = a.kept + (long long)b * kKeptWords;
  constexpr int kTiles = 8;
  int kept = 0;
  for (int round = 0; round < sp.len && kept <= kMostKept; round += kAttnWaves * kTiles * 64) {
    const int first = round + wave * kTiles * 64;
    unsigned long long bits[kTiles];
    int mine = 0;
#pragma unroll
    for (int u = 0; u < kTiles; ++u) bits[u] = key_bits(a, sp, b, first + u * 64, lane);
#pragma unroll
    for (int u = 0; u < kTiles; ++u) mine += __popcll(bits[u]);
    if (lane == 0) counts[wave] = mine;
    __syncthreads();
    int at = kept;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      if (w < wave) at += counts[w];
      kept += counts[w];
    }
    if (kept <= kMostKept) {
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        if ((bits[u] >> lane) & 1)
          list[1 + at + __popcll(bits[u] & ((1ull << lane) - 1))] = first + u * 64 + lane;
        at += __popcll(bits[u]);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) list[0] = kept;
}

// Three products of the forward's two sizes and the exponentials again.  The
// registers of Q, dO and dQ leave two waves a SIMD; held to three the kernel
// spills (222 us against 207 for the case above, 100 GFLOP: 485 TFLOP/s).
//
// dQ, and for k_attn_bwd_kv each row's L and delta in the form it starts its
// sums with: the forward's walk over the keys, with P from the saved L.
template <typename T, int DP, int QT, bool ALN, bool MASKED>
__global__ __launch_bounds__(kThreads) void k_attn_bwd_q(AttnArgs a) {
  constexpr int KK = kChunks32<DP>, DT = DP / 16;
  constexpr int kKeys = kTileKeys<T, DP>, kTile = kKeys * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  int b, h, tile;
  if (!place(a, a.row_tiles * a.q_splits, &b, &h, &tile)) return;
  const int split = tile % a.q_splits;
  tile /= a.q_splits;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Span sp = kv_span(a, b);
  const T* kb = kv_base<T>(a.k, a.ks, a, sp, b, h);
  const T* vb = kv_base<T>(a.v, a.vs, a, sp, b, h);
  const int row0 = tile * (16 * QT * kAttnWaves) + wave * 16 * QT + (lane & 15);
  const float c2 = a.scale * kLog2e;
  const f32x4 zero = zeros();
  Frag<T> q[QT][KK], g[QT][KK];
  f32x4 dq[QT][DT];
  float lse2[QT];
  f32x4 start[QT];  // -delta
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    const int r = row0 + j * 16;
    const bool in = r < a.rows;
    const T* pq = static_cast<const T*>(a.q) + (in ? row_at(a, a.qs, b, h, r) : 0);
    const T* po = static_cast<const T*>(a.o) + (in ? row_at(a, a.os, b, h, r) : 0);
    const T* pg = static_cast<const T*>(a.dout) + (in ? row_at(a, a.dos, b, h, r) : 0);
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < KK; ++c) {
      q[j][c] = load_head<T, ALN>(pq, c, lane, a.head_dim, in);
      g[j][c] = load_head<T, ALN>(pg, c, lane, a.head_dim, in);
      const Frag<T> o = load_head<T, ALN>(po, c, lane, a.head_dim, in);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += (float)g[j][c][i] * (float)o[i];
    }
    sum = group_add(sum);
    start[j] = f32x4{-sum, -sum, -sum, -sum};
    const float lse = in ? a.lse[stat_at(a, b, h, r)] : 0.f;
    lse2[j] = in && lse != -INFINITY ? lse * kLog2e : INFINITY;  // exp2(s - inf) = 0
#pragma unroll
    for (int d = 0; d < DT; ++d) dq[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // delta from out carries out's rounding, which a key with nearly all the
  // weight sees whole.  So with bfloat16 an entry of which 64 keys at most count
  // gets delta from P and dP: in the loop where it has one tile, and where a
  // mask leaves so few (MASKED), from a tile of their own.
  Stage<T, DP, kKeys, ALN> sk, sv;
  float from_p[QT];
  auto add_delta = [&](const T* tk, const T* tv, unsigned long long now) {
#pragma unroll
    for (int n = 0; n < kKeys; n += 16) {
      f32x4 s[QT], dp[QT];
#pragma unroll
      for (int c = 0; c < KK; ++c) {
        const Frag<T> fk = read_rows<DP>(tk, n, c, lane), fv = read_rows<DP>(tv, n, c, lane);
#pragma unroll
        for (int j = 0; j < QT; ++j) {
          s[j] = mma_head<DP>(fk, q[j][c], c == 0 ? zero : s[j], c);
          dp[j] = mma_head<DP>(fv, g[j][c], c == 0 ? zero : dp[j], c);
        }
      }
      const unsigned mine = (unsigned)(now >> (n + (lane >> 4) * 4));
#pragma unroll
      for (int j = 0; j < QT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((mine >> i) & 1) from_p[j] += __builtin_amdgcn_exp2f(s[j][i] * c2 - lse2[j]) * dp[j][i];
    }
  };
  auto take_delta = [&] {
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      const float x = -group_add(from_p[j]);
      start[j] = f32x4{x, x, x, x};
    }
  };
#pragma unroll
  for (int j = 0; j < QT; ++j) from_p[j] = 0.f;
  const bool short_entry = sizeof(T) == 2 && sp.len <= kKeys;
  if constexpr (MASKED) {
    const int* list = a.kept + (long long)b * kKeptWords;
    const int kept = list[0];
    if (!short_entry && kept <= kKeys) {  // in every block of the entry
      const int row = threadIdx.x / sk.kAcross, d0 = (threadIdx.x % sk.kAcross) * 8;
      sk.row = sv.row = row;
      sk.d0 = sv.d0 = d0;
#pragma unroll
      for (int i = 0; i < sk.kPer; ++i) {
        const bool in = row + i * sk.kStep < kept;
        const long long key = in ? list[1 + row + i * sk.kStep] : 0;
        sk.f[i] = load8<T, ALN>(kb + key * a.ks[1], d0, a.head_dim, in);
        sv.f[i] = load8<T, ALN>(vb + key * a.vs[1], d0, a.head_dim, in);
      }
      sk.store(tiles);
      sv.store(tiles + kTile);
      __syncthreads();
      add_delta(tiles, tiles + kTile, kept < 64 ? (1ull << kept) - 1 : ~0ull);
      take_delta();
      __syncthreads();  // the loop starts with the same buffer
    }
  }
  unsigned long long bits = 0;
  const int key0 = split * a.q_split_keys;
  const int key1 = std::min(sp.len, key0 + a.q_split_keys);
  if (key0 < key1) {
    sk.start(kb, a.ks[1], key0);
    sv.start(vb, a.vs[1], key0);
    bits = tile_bits<kKeys>(a, sp, b, key0, lane);
    sk.load(a.ks[1], bits, a.head_dim);
    sv.load(a.vs[1], bits, a.head_dim);
  }
  int buffer = 0;
  for (int first = key0; first < key1; first += kKeys, buffer ^= 1) {
    T* tk = tiles + buffer * 2 * kTile;
    T* tv = tk + kTile;
    sk.store(tk);
    sv.store(tv);
    __syncthreads();
    const unsigned long long now = bits;
    if (first + kKeys < key1) {
      bits = tile_bits<kKeys>(a, sp, b, first + kKeys, lane);
      sk.load(a.ks[1], bits, a.head_dim);
      sv.load(a.vs[1], bits, a.head_dim);
    }
    if (no_key<kKeys>(now)) continue;
    if (short_entry) {
      add_delta(tk, tv, now);
      take_delta();
    }
#pragma unroll
    for (int n = 0; n < kKeys; n += 32) {
      f32x4 s[2][QT], dp[2][QT];
      Frag<T> fk[2][KK], fv[2][KK];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          fk[u][c] = read_rows<DP>(tk, n + u * 16, c, lane);
          fv[u][c] = read_rows<DP>(tv, n + u * 16, c, lane);
        }
      if constexpr (sizeof(T) == 2) reads_before();
#pragma unroll
      for (int c = 0; c < KK; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < QT; ++j) {
            s[u][j] = mma_head<DP>(fk[u][c], q[j][c], c == 0 ? zero : s[u][j], c);
            dp[u][j] = mma_head<DP>(fv[u][c], g[j][c], c == 0 ? start[j] : dp[u][j], c);  // dP - delta, for nothing
          }
      Frag<T> ft[DT];  // on their way during the exponentials
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int d = 0; d < DT; ++d) ft[d] = read_cols<DP>(tk, n, d * 16, lane);
        reads_before();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < QT; ++j)
            s[u][j][i] = __builtin_amdgcn_exp2f(s[u][j][i] * c2 - lse2[j]) * dp[u][j][i];
      }
      if (now != ~0ull) {
        const unsigned long long mine = now >> ((lane >> 4) * 4);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((mine >> (n + u * 16 + i)) & 1))
#pragma unroll
              for (int j = 0; j < QT; ++j) s[u][j][i] = 0.f;
      }
      Frag<T> ds[QT];
#pragma unroll
      for (int j = 0; j < QT; ++j) ds[j] = pack<T>(s[0][j], s[1][j]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const Frag<T> f = sizeof(T) == 2 ? ft[d] : read_cols<DP>(tk, n, d * 16, lane);
#pragma unroll
        for (int j = 0; j < QT; ++j) dq[j][d] = mma(f, ds[j], dq[j][d]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    const int r = row0 + j * 16;
    if (r >= a.rows) continue;
    if (lane < 16 && split == 0)
      a.stats[((long long)b * a.kv_heads + h) * a.rows + r] =
          f32x2{sizeof(T) == 2 ? -lse2[j] / c2 : lse2[j], start[j][0]};
    if (a.q_splits > 1) {
      const long long at = (((long long)b * a.kv_heads + h) * a.q_splits + split) * a.rows + r;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        store4<float, false>(a.part_o + at * a.head_dim, d * 16 + (lane >> 4) * 4, a.head_dim, dq[j][d]);
      continue;
    }
    T* out = static_cast<T*>(a.dq) + row_at(a, a.dqs, b, h, r);
#pragma unroll
    for (int d = 0; d < DT; ++d) store4<T, ALN>(out, d * 16 + (lane >> 4) * 4, a.head_dim, dq[j][d] * a.scale);
  }
}

// Adds the key ranges' parts of dQ, in order: V elements of a row a thread.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_attn_join_q(AttnArgs a) {
  const unsigned per = a.head_dim / V;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;
  const unsigned row = id / per, d = (id - row * per) * V;
  const unsigned bh = row / a.rows, r = row - bh * a.rows;
  if (bh >= (unsigned)(a.batch * a.kv_heads)) return;
  const float* from = a.part_o + ((long long)bh * a.q_splits * a.rows + r) * a.head_dim + d;
  T* out = static_cast<T*>(a.dq) + row_at(a, a.dqs, (int)bh / a.kv_heads, (int)bh % a.kv_heads, r) + d;
  float sum[V] = {};
#pragma unroll 4
  for (int s = 0; s < a.q_splits; ++s) {
    float v[V];
    load_f32<float, V>(from + (long long)s * a.rows * a.head_dim, v);
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = (T)(sum[i] * a.scale);
}

// Four products; 300 us for the case above, 134 GFLOP: 447 TFLOP/s.  Vector
// instructions take 47% of the SIMDs' busy cycles (the exponentials' rate
// included), the matrix unit 28%: its two waves wait for their own results.  It
// is the products that cost
// (without the last two 220 us, without the exponentials 290, without reading
// the rows 280).  32 keys a wave, or 16 at four waves a SIMD: 305 and 318 us; 32
// rows a tile instead of 64: 314.  dQ has a kernel of its own (S and dP are
// computed twice, 7 products for 5) because its sum runs over the blocks here:
// without atomics, whose order would change the result, each block's part would
// go through memory, 2 GB for this case.
//
// dK and dV: a wave holds KT tiles of 16 keys and walks the rows, kBlockRows
// at a time, staged in LDS.  Here the scores have rows as rows, so a lane
// holds rows of one key.  A key that does not count spoils its own column
// only, which is written as zero at the end.
template <int DP>
constexpr int kBlockRows = DP <= 64 ? 64 : 32;

// Walks a thread's chunks of the folded rows of two tensors (Q and dO).
template <typename T, int DP, bool ALN>
struct RowStage {
  static constexpr int R = kBlockRows<DP>;
  static constexpr int kAcross = kCols<DP> / 8, kStep = kThreads / kAcross, kPer = (R + kStep - 1) / kStep;
  Frag<T> fq[kPer], fg[kPer];
  const T *pq[kPer], *pg[kPer];  // of the row that comes next
  int head[kPer];                // its head in the group
  int row, d0;
  __device__ __forceinline__ void start(const AttnArgs& a, int b, int h) {
    row = threadIdx.x / kAcross;
    d0 = (threadIdx.x % kAcross) * 8;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = row + i * kStep;
      head[i] = r % a.group;
      pq[i] = static_cast<const T*>(a.q) + row_at(a, a.qs, b, h, r);
      pg[i] = static_cast<const T*>(a.dout) + row_at(a, a.dos, b, h, r);
    }
  }
  // `left` rows from the next one on exist; the others are zero
  __device__ __forceinline__ void load(const AttnArgs& a, int left) {
    const int dq = R / a.group, dh = R % a.group;  // R rows on
    if (ALN && R == kPer * kStep && left >= R && a.head_dim == kCols<DP>) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        fq[i] = *reinterpret_cast<const Frag<T>*>(pq[i] + d0);
        fg[i] = *reinterpret_cast<const Frag<T>*>(pg[i] + d0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = row + i * kStep < std::min(left, R);
        fq[i] = load8<T, ALN>(pq[i], d0, a.head_dim, in);
        fg[i] = load8<T, ALN>(pg[i], d0, a.head_dim, in);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pq[i] += dq * a.qs[1] + dh * a.qs[2];
      pg[i] += dq * a.dos[1] + dh * a.dos[2];
      if (dh) {
        head[i] += dh;
        if (head[i] >= a.group) {
          head[i] -= a.group;
          pq[i] += a.qs[1] - a.group * a.qs[2];
          pg[i] += a.dos[1] - a.group * a.dos[2];
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* tq, T* tg) const {
    if (d0 >= DP) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (R == kPer * kStep || row + i * kStep < R) {
        const int at = chunk_at<T, DP>(row + i * kStep, d0 / 8);
        *reinterpret_cast<Frag<T>*>(tq + at) = fq[i];
        *reinterpret_cast<Frag<T>*>(tg + at) = fg[i];
      }
  }
};

// Zero gradients for head h of the packed rows 0 .. lo - 1 and hi .. end - 1, a
// part of them from block `block` of `blocks`.
template <typename T, int DP, bool ALN>
__device__ __forceinline__ void zero_rows(const AttnArgs& a, int h, long long lo, long long hi, long long end,
                                          int block, int blocks) {
  constexpr int V = ALN ? 8 : 1, kAcross = kCols<DP> / V, kRows = kThreads / kAcross;
  const long long n = lo + end - hi;
  const int d = (int)(threadIdx.x % kAcross) * V;
  if (d >= a.head_dim) return;
  for (long long i = (long long)block * kRows + threadIdx.x / kAcross; i < n; i += (long long)blocks * kRows) {
    const long long r = i < lo ? i : hi + (i - lo);
    T* dk = static_cast<T*>(a.dk) + r * a.dks[1] + h * a.dks[2] + d;
    T* dv = static_cast<T*>(a.dv) + r * a.dvs[1] + h * a.dvs[2] + d;
    if constexpr (ALN) {
      *reinterpret_cast<Frag<T>*>(dk) = Frag<T>{};
      *reinterpret_cast<Frag<T>*>(dv) = Frag<T>{};
    } else {
      *dk = *dv = (T)0.f;
    }
  }
}

template <typename T, int DP, int KT, bool ALN>
__global__ __launch_bounds__(kThreads) void k_attn_bwd_kv(AttnArgs a) {
  constexpr int KK = kChunks32<DP>, DT = DP / 16;
  constexpr int R = kBlockRows<DP>, kTile = R * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[4 * kTile];
  __shared__ __attribute__((aligned(16))) float stats[2][2 * R];
  int b, h, tile;
  if (!place(a, a.key_tiles, &b, &h, &tile)) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Span sp = kv_span(a, b);
  const int block_key = tile * (16 * KT * kAttnWaves);
  // Packed rows that no entry has: before the first and after the last, by all
  // blocks of the head (512 entries of 0 to 1000 keys, 4 heads of 32 bfloat16, 50
  // queries, in a buffer of twice the rows in use: the backward takes 151 us, 141
  // without the spare rows, and 7.1 ms with one block a head for all of them),
  // and those of an entry of too many, by its own.
  if (a.kv_offsets) {
    auto row = [&](int i) { return std::min<long long>(std::max(a.kv_offsets[i], 0), a.kv_rows); };
    zero_rows<T, DP, ALN>(a, h, row(0), row(a.batch), a.kv_rows, b * a.key_tiles + tile, a.batch * a.key_tiles);
    if (sp.len == 0) zero_rows<T, DP, ALN>(a, h, 0, row(b), row(b + 1), tile, a.key_tiles);
  }
  // padded keys past the length still get their (zero) gradient
  const int end = a.kv_offsets ? sp.len : a.kv_len;
  if (block_key >= end) return;
  const T* kb = kv_base<T>(a.k, a.ks, a, sp, b, h);
  const T* vb = kv_base<T>(a.v, a.vs, a, sp, b, h);
  const float c2 = a.scale * kLog2e;
  const int key0 = block_key + wave * 16 * KT + (lane & 15);
  Frag<T> k[KT][KK], v[KT][KK];
  f32x4 dk[KT][DT], dv[KT][DT];
  bool in[KT];
#pragma unroll
  for (int j = 0; j < KT; ++j) {
    const int key = key0 + j * 16;
    in[j] = key < sp.len;
    if (in[j] && a.kv_mask)
      in[j] = a.kv_mask[(a.kv_offsets ? sp.row0 : (long long)b * a.mask_stride) + key] != 0;
#pragma unroll
    for (int c = 0; c < KK; ++c) {
      k[j][c] = load_head<T, ALN>(kb + (long long)key * a.ks[1], c, lane, a.head_dim, in[j]);
      v[j][c] = load_head<T, ALN>(vb + (long long)key * a.vs[1], c, lane, a.head_dim, in[j]);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[j][d] = dv[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const f32x2* row_stats = a.stats + ((long long)b * a.kv_heads + h) * a.rows;
  const int rows = block_key < sp.len ? a.rows : 0;
  // rows that do not exist: weight 0
  const f32x2 none{sizeof(T) == 2 ? -INFINITY : INFINITY, 0.f};
  RowStage<T, DP, ALN> st;
  f32x2 stat = none;
  if (rows > 0) {
    st.start(a, b, h);
    st.load(a, rows);
    if ((int)threadIdx.x < std::min(rows, R)) stat = row_stats[threadIdx.x];
  }
  int buffer = 0;
  for (int first = 0; first < rows; first += R, buffer ^= 1) {
    T* tq = tiles + buffer * 2 * kTile;
    T* tg = tq + kTile;
    float* tl = stats[buffer];
    float* td = tl + R;
    st.store(tq, tg);
    if (threadIdx.x < R) {
      tl[threadIdx.x] = stat[0];
      td[threadIdx.x] = stat[1];
    }
    __syncthreads();
    const int left = rows - first - R;
    if (left > 0) {
      st.load(a, left);
      stat = (int)threadIdx.x < std::min(left, R) ? row_stats[first + R + threadIdx.x] : none;
    }
#pragma unroll
    for (int n = 0; n < R; n += 32) {
      f32x4 s[2][KT], dp[2][KT], l4[2], d4[2];
      Frag<T> fq[2][KK], fg[2][KK];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        l4[u] = *reinterpret_cast<const f32x4*>(tl + n + u * 16 + (lane >> 4) * 4);
        d4[u] = *reinterpret_cast<const f32x4*>(td + n + u * 16 + (lane >> 4) * 4);
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          fq[u][c] = read_rows<DP>(tq, n + u * 16, c, lane);
          fg[u][c] = read_rows<DP>(tg, n + u * 16, c, lane);
        }
      }
      if constexpr (sizeof(T) == 2) reads_before();
      // the products' sums start at -L / scale and -delta (in float32 the
      // scores start at 0: there the extra rounding would show)
#pragma unroll
      for (int c = 0; c < KK; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < KT; ++j) {
            const f32x4 from = sizeof(T) == 2 ? l4[u] : f32x4{0.f, 0.f, 0.f, 0.f};
            s[u][j] = mma_head<DP>(fq[u][c], k[j][c], c == 0 ? from : s[u][j], c);
            dp[u][j] = mma_head<DP>(fg[u][c], v[j][c], c == 0 ? d4[u] : dp[u][j], c);
          }
      Frag<T> tgf[DT], tqf[DT];  // on their way during the exponentials
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          tgf[d] = read_cols<DP>(tg, n, d * 16, lane);
          tqf[d] = read_cols<DP>(tq, n, d * 16, lane);
        }
        reads_before();
      }
      Frag<T> p[KT], ds[KT];
#pragma unroll
      for (int j = 0; j < KT; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = sizeof(T) == 2 ? s[u][j][i] * c2 : s[u][j][i] * c2 - l4[u][i];
            s[u][j][i] = __builtin_amdgcn_exp2f(x);
            dp[u][j][i] *= s[u][j][i];
          }
        p[j] = pack<T>(s[0][j], s[1][j]);
        ds[j] = pack<T>(dp[0][j], dp[1][j]);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const Frag<T> cg = sizeof(T) == 2 ? tgf[d] : read_cols<DP>(tg, n, d * 16, lane);
        const Frag<T> cq = sizeof(T) == 2 ? tqf[d] : read_cols<DP>(tq, n, d * 16, lane);
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          dv[j][d] = mma(cg, p[j], dv[j][d]);
          dk[j][d] = mma(cq, ds[j], dk[j][d]);
        }
      }
    }
  }
  T* dkb = const_cast<T*>(kv_base<T>(a.dk, a.dks, a, sp, b, h));
  T* dvb = const_cast<T*>(kv_base<T>(a.dv, a.dvs, a, sp, b, h));
#pragma unroll
  for (int j = 0; j < KT; ++j) {
    const int key = key0 + j * 16;
    if (key >= end) continue;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int d0 = d * 16 + (lane >> 4) * 4;
      const f32x4 zero{0.f, 0.f, 0.f, 0.f};
      store4<T, ALN>(dkb + (long long)key * a.dks[1], d0, a.head_dim, in[j] ? dk[j][d] * a.scale : zero);
      store4<T, ALN>(dvb + (long long)key * a.dvs[1], d0, a.head_dim, in[j] ? dv[j][d] : zero);
    }
  }
}

// ----------------------------------------------------------- sizes, launches
struct AttnPlan {
  int dp, qt, kt;
  bool few;
  int row_tiles, key_tiles, splits, split_keys, q_splits, q_split_keys;
  int64_t part_ml, part_dq, kept, fwd_bytes, bwd_bytes;
};

recis_status check_desc(const recis_attn_desc* d) {
  if (!d || !dtype_known(d->dtype) || d->batch < 0 || d->q_len < 0 || d->kv_len < 0 || d->q_heads < 1 ||
      d->kv_heads < 1 || d->head_dim < 1 || d->q_heads % d->kv_heads || !(d->scale > 0.f) || !std::isfinite(d->scale))
    return RECIS_ERR_INVALID_ARG;
  if (d->kv_offsets && (d->kv_lens || d->kv_rows < 0)) return RECIS_ERR_INVALID_ARG;
  if (!aligned_to(d->kv_offsets, 4) || !aligned_to(d->kv_lens, 4) || !aligned_to(d->error, 4))
    return RECIS_ERR_INVALID_ARG;
  if (d->head_dim > kMaxHeadDim) return RECIS_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)d->q_len * (d->q_heads / d->kv_heads);
  if (rows > (1 << 30) || d->kv_len > (1 << 30) || (int64_t)d->batch * d->kv_heads > (1 << 24))
    return RECIS_ERR_UNSUPPORTED;
  return RECIS_OK;
}

constexpr int kMaxSplits = 256, kBlocksForOutside = 512;

AttnPlan attn_plan(const recis_attn_desc* d) {
  AttnPlan p;
  const bool f32 = d->dtype == RECIS_DTYPE_F32;
  p.dp = d->head_dim <= 32 ? 32 : f32 && d->head_dim <= 48 ? 48 : d->head_dim <= 64 ? 64 : d->head_dim <= 96 ? 96 : 128;
  const int group = d->q_heads / d->kv_heads;
  const int64_t rows = (int64_t)d->q_len * group, bh = (int64_t)d->batch * d->kv_heads;
  // Two tiles a wave at head sizes to 64.  Above, they take a backward wave past
  // 256 registers, so that one runs a SIMD (128 entries, 512 queries, up to 1000
  // keys, 8 heads of 128: 1128 us against 981), and small forward calls have
  // half the blocks (16 entries: 86 us against 51); large forward calls would
  // gain (226 against 316) and would need a rule of their own.
  p.qt = rows > 64 && d->dtype == RECIS_DTYPE_BF16 && p.dp <= 64 ? 2 : 1;
  p.kt = d->dtype == RECIS_DTYPE_BF16 && p.dp <= 64 ? 2 : 1;
  p.row_tiles = (int)((rows + 64 * p.qt - 1) / (64 * p.qt));
  p.key_tiles = std::max(1, (int)(((int64_t)d->kv_len + 64 * p.kt - 1) / (64 * p.kt)));
  // few pairs over a large packed buffer: further tiles, without keys, for its
  // rows outside the entries (zero_rows; one entry, 2 heads of 64, 2M spare
  // rows: 232 us, 53 ms from its two blocks)
  if (d->kv_offsets && bh > 0 && bh < kBlocksForOutside)
    p.key_tiles = std::max(p.key_tiles, (int)std::min<int64_t>((kBlocksForOutside + bh - 1) / bh,
                                                               d->kv_rows / ((int64_t)d->batch * kBlockKeys)));
  p.few = rows <= kFewRows;
  // keys are split until there are `want` blocks (of unequal length where the
  // entries' are), `least` keys each, kMaxSplits ranges at most
  auto split = [&](int64_t blocks, int64_t want, int64_t least, int* splits, int* keys) {
    const int64_t n = std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, want / std::max<int64_t>(1, blocks)));
    *keys = (int)std::max<int64_t>(least, round_up((d->kv_len + n - 1) / n, 2 * kBlockKeys));
    *splits = std::max(1, (int)(((int64_t)d->kv_len + *keys - 1) / *keys));
  };
  split(bh * p.row_tiles, p.few || f32 ? 2048 : 1024, p.few ? 256 : 128, &p.splits, &p.split_keys);
  split(bh * p.row_tiles, f32 ? 2048 : 1024, 128, &p.q_splits, &p.q_split_keys);
  p.part_ml = p.splits > 1 ? round_up(bh * p.splits * rows * d->head_dim * 4, 256) : 0;
  p.fwd_bytes = p.splits > 1 ? p.part_ml + round_up(bh * p.splits * rows * 8, 256) : 0;
  p.part_dq = round_up(std::max<int64_t>(bh * rows, 1) * 8, 256);
  p.kept = p.part_dq + (p.q_splits > 1 ? round_up(bh * p.q_splits * rows * d->head_dim * 4, 256) : 0);
  p.bwd_bytes = p.kept + (f32 ? 0 : round_up((int64_t)d->batch * kKeptWords * 4, 256));
  return p;
}

void fill_args(const recis_attn_desc* d, const AttnPlan& p, AttnArgs* a) {
  *a = AttnArgs{};
  a->kv_offsets = d->kv_offsets;
  a->kv_lens = d->kv_lens;
  a->kv_mask = d->kv_mask;
  a->mask_stride = d->mask_stride;
  a->kv_rows = d->kv_rows;
  for (int i = 0; i < 3; ++i) {
    a->qs[i] = d->q_strides[i];
    a->ks[i] = d->k_strides[i];
    a->vs[i] = d->v_strides[i];
    a->os[i] = d->o_strides[i];
    a->dos[i] = d->do_strides[i];
    a->dqs[i] = d->dq_strides[i];
    a->dks[i] = d->dk_strides[i];
    a->dvs[i] = d->dv_strides[i];
  }
  a->batch = d->batch;
  a->q_len = d->q_len;
  a->kv_len = d->kv_len;
  a->q_heads = d->q_heads;
  a->kv_heads = d->kv_heads;
  a->group = d->q_heads / d->kv_heads;
  a->head_dim = d->head_dim;
  a->rows = d->q_len * a->group;
  a->row_tiles = p.row_tiles;
  a->unit = p.row_tiles <= 1 && d->batch >= kEntriesForDies ? d->kv_heads : 1;
  a->dies = (int64_t)d->batch * d->kv_heads >= kPairsForDies ? kDies : 1;
  a->key_tiles = p.key_tiles;
  a->splits = p.splits;
  a->split_keys = p.split_keys;
  a->q_splits = p.q_splits;
  a->q_split_keys = p.q_split_keys;
  a->scale = d->scale;
  a->error = d->error;
}

// Rows can be moved 16 bytes at a time.
bool rows_aligned(const recis_attn_desc* d, std::initializer_list<const void*> ptrs,
                  std::initializer_list<const int64_t*> strides) {
  const int per = 16 / dtype_size(d->dtype);
  if (d->head_dim % 8) return false;
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return false;
  for (const int64_t* s : strides)
    for (int i = 0; i < 3; ++i)
      if (s[i] % per) return false;
  // 64 rows stay within 32 bits of byte offset
  for (const int64_t* s : {d->k_strides, d->v_strides})
    if (s[1] < 0 || s[1] >= (1 << 23)) return false;
  return true;
}

bool elements_aligned(const recis_attn_desc* d, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p || !aligned_to(p, dtype_size(d->dtype))) return false;
  return true;
}

dim3 attn_grid(const AttnArgs& a, int per) {
  return grid_of(round_up((int64_t)a.batch * a.kv_heads, a.dies * a.unit) * per);
}

enum AttnPass { kFwd, kFew, kBwdQ, kBwdKv };

template <typename T, int DP, int N, bool ALN>
void launch_pass(AttnPass pass, const AttnArgs& a, hipStream_t s) {
  if (pass == kFwd)
    hipLaunchKernelGGL((k_attn_fwd<T, DP, N, ALN>), attn_grid(a, a.row_tiles * a.splits), dim3(kThreads), 0, s, a);
  else if (pass == kFew) {
    if constexpr (N == 1) hipLaunchKernelGGL((k_attn_few<T, DP, ALN>), attn_grid(a, a.splits), dim3(kThreads), 0, s, a);
  } else if (pass == kBwdQ) {
    const dim3 grid = attn_grid(a, a.row_tiles * a.q_splits);
    if (sizeof(T) == 2 && a.kept)
      hipLaunchKernelGGL((k_attn_bwd_q<T, DP, N, ALN, sizeof(T) == 2>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_attn_bwd_q<T, DP, N, ALN, false>), grid, dim3(kThreads), 0, s, a);
  } else
    hipLaunchKernelGGL((k_attn_bwd_kv<T, DP, N, ALN>), attn_grid(a, a.key_tiles), dim3(kThreads), 0, s, a);
}

template <typename T, int DP>
void launch_dp(AttnPass pass, const AttnPlan& p, bool aln, const AttnArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2 && DP <= 64) {
    if ((pass == kBwdKv ? p.kt : p.qt) == 2)
      return aln ? launch_pass<T, DP, 2, true>(pass, a, s) : launch_pass<T, DP, 2, false>(pass, a, s);
  }
  aln ? launch_pass<T, DP, 1, true>(pass, a, s) : launch_pass<T, DP, 1, false>(pass, a, s);
}

template <typename T>
void launch_type(AttnPass pass, const AttnPlan& p, bool aln, const AttnArgs& a, hipStream_t s) {
  switch (p.dp) {
    case 32: return launch_dp<T, 32>(pass, p, aln, a, s);
    case 48:
      if constexpr (sizeof(T) == 4) launch_dp<T, 48>(pass, p, aln, a, s);
      return;
    case 64: return launch_dp<T, 64>(pass, p, aln, a, s);
    case 96: return launch_dp<T, 96>(pass, p, aln, a, s);
    default: return launch_dp<T, 128>(pass, p, aln, a, s);
  }
}

void launch_attn(AttnPass pass, int dtype, const AttnPlan& p, bool aln, const AttnArgs& a, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16)
    launch_type<__bf16>(pass, p, aln, a, s);
  else
    launch_type<float>(pass, p, aln, a, s);
}

// Blocks for every V elements of every row of the folded queries; split calls
// have few row tiles (attn_plan), so this is far below 2^31 threads.
dim3 join_grid(const AttnArgs& a, int v) {
  const int64_t threads = (int64_t)a.batch * a.kv_heads * a.rows * (a.head_dim / v);
  return dim3((unsigned)((threads + kThreads - 1) / kThreads));
}

// A block a row where the rows alone do not fill the chip (1024 rows of 8
// ranges, head size 128: 6 us against 10).
template <typename T>
void launch_join(const AttnArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  if (rows <= 2048)
    hipLaunchKernelGGL((k_attn_join_few<T>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
  else if (a.head_dim % 4 == 0)
    hipLaunchKernelGGL((k_attn_join_many<T, 4>), join_grid(a, 4), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_join_many<T, 1>), join_grid(a, 1), dim3(kThreads), 0, s, a);
}

template <typename T>
void launch_join_q(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim % 4 == 0)
    hipLaunchKernelGGL((k_attn_join_q<T, 4>), join_grid(a, 4), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_join_q<T, 1>), join_grid(a, 1), dim3(kThreads), 0, s, a);
}

// A pass's blocks can be launched.
bool grid_fits(const recis_attn_desc* d, const AttnPlan& p, bool backward) {
  const int64_t per = backward ? std::max<int64_t>((int64_t)p.row_tiles * p.q_splits, p.key_tiles)
                               : (int64_t)p.row_tiles * p.splits;
  return round_up((int64_t)d->batch * d->kv_heads, (int64_t)kDies * d->kv_heads) * per <= kMaxBlocks;
}

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

int64_t recis_cross_attn_workspace_bytes(const recis_attn_desc* desc, int32_t backward) {
  if (check_desc(desc) != RECIS_OK) return -1;
  const AttnPlan p = attn_plan(desc);
  if (!grid_fits(desc, p, backward)) return -1;
  return backward ? p.bwd_bytes : p.fwd_bytes;
}

recis_status recis_cross_attn_fwd(const recis_attn_desc* desc, const void* q, const void* k, const void* v, void* out,
                                  float* lse, void* workspace, int64_t workspace_bytes, hipStream_t s) {
  const recis_status st = check_desc(desc);
  if (st != RECIS_OK) return st;
  if (desc->batch == 0 || desc->q_len == 0) return RECIS_OK;
  const bool keys = desc->kv_offsets ? desc->kv_rows > 0 : desc->kv_len > 0;
  if (!elements_aligned(desc, {q, out}) || (keys && !elements_aligned(desc, {k, v})) || !aligned_to(lse, 4))
    return RECIS_ERR_INVALID_ARG;
  const AttnPlan p = attn_plan(desc);
  if (!grid_fits(desc, p, false)) return RECIS_ERR_UNSUPPORTED;
  if (p.fwd_bytes && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.fwd_bytes))
    return RECIS_ERR_INVALID_ARG;
  AttnArgs a;
  fill_args(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_ml);
  const bool aln = rows_aligned(desc, {q, k, v, out},
                                {desc->q_strides, desc->k_strides, desc->v_strides, desc->o_strides});
  launch_attn(p.few ? kFew : kFwd, desc->dtype, p, aln, a, s);
  if (p.splits > 1) {
    if (desc->dtype == RECIS_DTYPE_BF16)
      launch_join<__bf16>(a, s);
    else
      launch_join<float>(a, s);
  }
  return launch_status();
}

recis_status recis_cross_attn_bwd(const recis_attn_desc* desc, const void* grad_out, const void* q, const void* k,
                                  const void* v, const void* out, const float* lse, void* grad_q, void* grad_k,
                                  void* grad_v, void* workspace, int64_t workspace_bytes, hipStream_t s) {
  const recis_status st = check_desc(desc);
  if (st != RECIS_OK) return st;
  if (desc->batch == 0) return RECIS_OK;
  const bool keys = desc->kv_offsets ? desc->kv_rows > 0 : desc->kv_len > 0;
  const bool rows = desc->q_len > 0;
  if ((rows && !elements_aligned(desc, {grad_out, q, out, grad_q})) ||
      (keys && !elements_aligned(desc, {k, v, grad_k, grad_v})) || (rows && !lse) || !aligned_to(lse, 4))
    return RECIS_ERR_INVALID_ARG;
  const AttnPlan p = attn_plan(desc);
  if (!grid_fits(desc, p, true)) return RECIS_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bwd_bytes) return RECIS_ERR_INVALID_ARG;
  AttnArgs a;
  fill_args(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = out;
  a.dout = grad_out;
  a.lse = const_cast<float*>(lse);
  a.stats = static_cast<f32x2*>(workspace);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_dq);
  // a mask over more than a tile of keys may leave few
  if (desc->dtype == RECIS_DTYPE_BF16 && desc->kv_mask && desc->kv_len > kBlockKeys)
    a.kept = reinterpret_cast<int*>(static_cast<char*>(workspace) + p.kept);
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  const bool aln = rows_aligned(desc, {q, k, v, out, grad_out, grad_q, grad_k, grad_v},
                                {desc->q_strides, desc->k_strides, desc->v_strides, desc->o_strides,
                                 desc->do_strides, desc->dq_strides, desc->dk_strides, desc->dv_strides});
  if (rows && a.kept) hipLaunchKernelGGL(k_attn_kept, grid_of(desc->batch), dim3(kThreads), 0, s, a);
  if (rows) launch_attn(kBwdQ, desc->dtype, p, aln, a, s);
  if (rows && p.q_splits > 1) {
    if (desc->dtype == RECIS_DTYPE_BF16)
      launch_join_q<__bf16>(a, s);
    else
      launch_join_q<float>(a, s);
  }
  if (keys) launch_attn(kBwdKv, desc->dtype, p, aln, a, s);
  return launch_status();
}

}  // extern "C"
