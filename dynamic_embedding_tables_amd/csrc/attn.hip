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

#include "seq.h"

namespace recis {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  float *lse, *delta;
  const int *kv_offsets, *kv_lens;
  const unsigned char* kv_mask;
  long long mask_stride, kv_rows;
  long long qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];  // batch, row, head
  int batch, q_len, kv_len, q_heads, kv_heads, group, head_dim;
  int rows;                // q_len * group
  int row_tiles, key_tiles;
  int splits, split_keys;  // forward: key ranges of a row tile, joined by k_attn_join
  float scale;
  float *part_o, *part_ml;  // [batch * kv_heads][splits][rows][head_dim], [..][2]
  unsigned* error;
};

// ---------------------------------------------------------------- fragments
template <typename T>
struct FragOf;
template <>
struct FragOf<__bf16> {
  typedef bf16x8 type;
};
template <>
struct FragOf<float> {
  typedef f32x8 type;
};
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Eight products of k = 4: the j-th takes element j of every lane, so the
// operands' layout is the bfloat16 one.
__device__ __forceinline__ f32x4 mma(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

template <typename T>
__device__ __forceinline__ Frag<T> pack(f32x4 lo, f32x4 hi) {
  const f32x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_convertvector(x, Frag<T>);
}

// 8 elements of a row of `dim`, from d0; ALN: rows are 16-byte aligned and dim
// is a multiple of 8.
template <typename T, bool ALN>
__device__ __forceinline__ Frag<T> load8(const T* row, int d0, int dim, bool in) {
  Frag<T> f;
  if constexpr (ALN) {
    if (in && d0 < dim) {
      f = *reinterpret_cast<const Frag<T>*>(row + d0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = (T)0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in && d0 + i < dim ? row[d0 + i] : (T)0.f;
  }
  return f;
}

template <typename T, bool ALN>
__device__ __forceinline__ void store4(T* row, int d0, int dim, f32x4 x) {
  if constexpr (ALN) {
    if (d0 < dim) {
      float v[4] = {x[0], x[1], x[2], x[3]};
      store_f32<T, 4>(row + d0, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d0 + i < dim) row[d0 + i] = (T)x[i];
  }
}

// LDS tile rows are padded by 16 bytes: 16 lanes reading one column of 16
// rows then fall on distinct banks.
template <typename T, int DP>
constexpr int kLd = DP + 16 / (int)sizeof(T);

template <typename T, int DP>
__device__ __forceinline__ Frag<T> read_rows(const T* tile, int row0, int c0, int lane) {
  return *reinterpret_cast<const Frag<T>*>(tile + (row0 + (lane & 15)) * kLd<T, DP> + c0 + (lane >> 4) * 8);
}

// Column c0 + lane % 16 of 32 rows, in the slot order of pack().
template <int DP>
__device__ __forceinline__ bf16x8 read_cols(const __bf16* tile, int row0, int c0, int lane) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const __bf16* p = tile + (row0 + (lane >> 4) * 4 + ((lane & 15) >> 2)) * kLd<__bf16, DP> + c0 + (lane & 3) * 4;
  // within 16 lanes: lane i names 4 columns of row i / 4, and receives column i of the 4 rows
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * kLd<__bf16, DP>));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, x);
}
template <int DP>
__device__ __forceinline__ f32x8 read_cols(const float* tile, int row0, int c0, int lane) {
  const float* p = tile + (row0 + (lane >> 4) * 4) * kLd<float, DP> + c0 + (lane & 15);
  f32x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = p[(j < 4 ? j : j + 12) * kLd<float, DP>];
  return x;
}

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

// Consecutive blocks go to the eight dies in turn; the blocks of one (batch
// entry, key head) are given to the same die, so its keys stay in one L2.
constexpr int kDies = 8;
__device__ __forceinline__ bool place(const AttnArgs& a, int per, int* b, int* h, int* t) {
  const int slot = blockIdx.x / kDies;
  const int bh = (slot / per) * kDies + blockIdx.x % kDies;
  *t = slot % per;
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

// A tile of R rows x DP held in registers on its way to LDS.
template <typename T, int DP, int R, bool ALN>
struct Stage {
  static constexpr int kChunks = R * (DP / 8);
  static constexpr int kPer = (kChunks + kThreads - 1) / kThreads;
  Frag<T> f[kPer];
  // rows whose bit is clear are zero, whatever memory holds there
  __device__ __forceinline__ void load(const T* base, long long stride, int first, unsigned long long bits, int dim) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * kThreads + threadIdx.x;
      const int r = c / (DP / 8), d0 = (c % (DP / 8)) * 8;
      const bool in = (kChunks % kThreads == 0 || c < kChunks) && ((bits >> r) & 1);
      f[i] = load8<T, ALN>(base + (long long)(first + r) * stride, d0, dim, in);
    }
  }
  __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * kThreads + threadIdx.x;
      if (kChunks % kThreads == 0 || c < kChunks)
        *reinterpret_cast<Frag<T>*>(tile + (c / (DP / 8)) * kLd<T, DP> + (c % (DP / 8)) * 8) = f[i];
    }
  }
};

constexpr int kBlockKeys = 64;
constexpr int kAttnWaves = kThreads / 64;

// ------------------------------------------------------------------ forward
// A wave holds QT tiles of 16 queries; the block walks the keys 64 at a time,
// staged in LDS for its four waves, the next tile's loads in flight meanwhile.
template <typename T, int DP, int QT, bool ALN>
__global__ __launch_bounds__(kThreads) void k_attn_fwd(AttnArgs a) {
  constexpr int KK = DP / 32, DT = DP / 16, NT = kBlockKeys / 16;
  __shared__ __attribute__((aligned(16))) T tk[kBlockKeys * kLd<T, DP>];
  __shared__ __attribute__((aligned(16))) T tv[kBlockKeys * kLd<T, DP>];
  int b, h, t;
  if (!place(a, a.row_tiles * a.splits, &b, &h, &t)) return;
  const int split = t % a.splits, tile = t / a.splits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    for (int c = 0; c < KK; ++c) q[j][c] = load8<T, ALN>(p, c * 32 + (lane >> 4) * 8, a.head_dim, in);
  }
  f32x4 o[QT][DT];
  float m[QT], l[QT];
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float c2 = a.scale * kLog2e;
  Stage<T, DP, kBlockKeys, ALN> sk, sv;
  unsigned long long bits = 0;
  if (key0 < key1) {
    bits = key_bits(a, sp, b, key0, lane);
    sk.load(kb, a.ks[1], key0, bits, a.head_dim);
    sv.load(vb, a.vs[1], key0, bits, a.head_dim);
  }
  for (int first = key0; first < key1; first += kBlockKeys) {
    __syncthreads();
    sk.store(tk);
    sv.store(tv);
    __syncthreads();
    const unsigned long long now = bits;
    if (first + kBlockKeys < key1) {
      bits = key_bits(a, sp, b, first + kBlockKeys, lane);
      sk.load(kb, a.ks[1], first + kBlockKeys, bits, a.head_dim);
      sv.load(vb, a.vs[1], first + kBlockKeys, bits, a.head_dim);
    }
    if (now == 0) continue;
    f32x4 s[NT][QT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < QT; ++j) s[n][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KK; ++c) {
        const Frag<T> f = read_rows<T, DP>(tk, n * 16, c * 32, lane);
#pragma unroll
        for (int j = 0; j < QT; ++j) s[n][j] = mma(f, q[j][c], s[n][j]);
      }
    }
    if (now != ~0ull) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((now >> (n * 16 + (lane >> 4) * 4 + i)) & 1))
#pragma unroll
            for (int j = 0; j < QT; ++j) s[n][j][i] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      float top = m[j];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[n][j][i]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float ref = top == -INFINITY ? 0.f : top * c2;
      const float alpha = __builtin_amdgcn_exp2f(m[j] * c2 - ref);
      m[j] = top;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[n][j][i] = __builtin_amdgcn_exp2f(s[n][j][i] * c2 - ref);
          sum += s[n][j][i];
        }
      l[j] = l[j] * alpha + sum;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[j][d] *= alpha;
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
    l[j] += __shfl_xor(l[j], 16);
    l[j] += __shfl_xor(l[j], 32);
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

// Joins the key ranges of a row: one wave a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a) {
  const long long id = (long long)blockIdx.x * kAttnWaves + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (id >= (long long)a.batch * a.kv_heads * a.rows) return;
  const int r = (int)(id % a.rows);
  const long long bh = id / a.rows;
  const int h = (int)(bh % a.kv_heads), b = (int)(bh / a.kv_heads);
  const long long at = bh * a.splits * a.rows + r;
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.part_ml[2 * (at + (long long)s * a.rows)]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  float o[2] = {0.f, 0.f}, l = 0.f;  // head_dim <= 128
  for (int s = 0; s < a.splits; ++s) {
    const long long p = at + (long long)s * a.rows;
    const float w = __builtin_amdgcn_exp2f(a.part_ml[2 * p] - ref);
    if (w == 0.f) continue;
    l += w * a.part_ml[2 * p + 1];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64 * i < a.head_dim) o[i] += w * a.part_o[p * a.head_dim + lane + 64 * i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + row_at(a, a.os, b, h, r);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < a.head_dim) out[lane + 64 * i] = (T)(o[i] * inv);
  if (a.lse && lane == 0) a.lse[stat_at(a, b, h, r)] = l == 0.f ? -INFINITY : top * kLn2 + __logf(l);
}

// ----------------------------------------------------------------- backward
// dQ (and delta, which k_attn_bwd_kv reads): the forward's walk over the keys,
// with P from the saved L.
template <typename T, int DP, int QT, bool ALN>
__global__ __launch_bounds__(kThreads) void k_attn_bwd_q(AttnArgs a) {
  constexpr int KK = DP / 32, DT = DP / 16;
  __shared__ __attribute__((aligned(16))) T tk[kBlockKeys * kLd<T, DP>];
  __shared__ __attribute__((aligned(16))) T tv[kBlockKeys * kLd<T, DP>];
  int b, h, tile;
  if (!place(a, a.row_tiles, &b, &h, &tile)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Span sp = kv_span(a, b);
  const T* kb = kv_base<T>(a.k, a.ks, a, sp, b, h);
  const T* vb = kv_base<T>(a.v, a.vs, a, sp, b, h);
  const int row0 = tile * (16 * QT * kAttnWaves) + wave * 16 * QT + (lane & 15);
  const float c2 = a.scale * kLog2e;
  Frag<T> q[QT][KK], g[QT][KK];
  f32x4 dq[QT][DT];
  float lse2[QT], delta[QT];
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
      const int d0 = c * 32 + (lane >> 4) * 8;
      q[j][c] = load8<T, ALN>(pq, d0, a.head_dim, in);
      g[j][c] = load8<T, ALN>(pg, d0, a.head_dim, in);
      const Frag<T> o = load8<T, ALN>(po, d0, a.head_dim, in);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += (float)g[j][c][i] * (float)o[i];
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    delta[j] = sum;
    const float lse = in ? a.lse[stat_at(a, b, h, r)] : 0.f;
    lse2[j] = in && lse != -INFINITY ? lse * kLog2e : INFINITY;  // exp2(s - inf) = 0
    if (in && lane < 16) a.delta[((long long)b * a.kv_heads + h) * a.rows + r] = sum;
#pragma unroll
    for (int d = 0; d < DT; ++d) dq[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  Stage<T, DP, kBlockKeys, ALN> sk, sv;
  unsigned long long bits = 0;
  if (sp.len > 0) {
    bits = key_bits(a, sp, b, 0, lane);
    sk.load(kb, a.ks[1], 0, bits, a.head_dim);
    sv.load(vb, a.vs[1], 0, bits, a.head_dim);
  }
  for (int first = 0; first < sp.len; first += kBlockKeys) {
    __syncthreads();
    sk.store(tk);
    sv.store(tv);
    __syncthreads();
    const unsigned long long now = bits;
    if (first + kBlockKeys < sp.len) {
      bits = key_bits(a, sp, b, first + kBlockKeys, lane);
      sk.load(kb, a.ks[1], first + kBlockKeys, bits, a.head_dim);
      sv.load(vb, a.vs[1], first + kBlockKeys, bits, a.head_dim);
    }
    if (now == 0) continue;
#pragma unroll
    for (int n = 0; n < kBlockKeys; n += 32) {
      f32x4 s[2][QT], dp[2][QT];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < QT; ++j) s[u][j] = dp[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          const Frag<T> fk = read_rows<T, DP>(tk, n + u * 16, c * 32, lane);
          const Frag<T> fv = read_rows<T, DP>(tv, n + u * 16, c * 32, lane);
#pragma unroll
          for (int j = 0; j < QT; ++j) {
            s[u][j] = mma(fk, q[j][c], s[u][j]);
            dp[u][j] = mma(fv, g[j][c], dp[u][j]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = (now >> (n + u * 16 + (lane >> 4) * 4 + i)) & 1;
#pragma unroll
          for (int j = 0; j < QT; ++j) {
            const float p = __builtin_amdgcn_exp2f(s[u][j][i] * c2 - lse2[j]);
            s[u][j][i] = in ? p * (dp[u][j][i] - delta[j]) : 0.f;
          }
        }
      }
      Frag<T> ds[QT];
#pragma unroll
      for (int j = 0; j < QT; ++j) ds[j] = pack<T>(s[0][j], s[1][j]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const Frag<T> f = read_cols<DP>(tk, n, d * 16, lane);
#pragma unroll
        for (int j = 0; j < QT; ++j) dq[j][d] = mma(f, ds[j], dq[j][d]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < QT; ++j) {
    const int r = row0 + j * 16;
    if (r >= a.rows) continue;
    T* out = static_cast<T*>(a.dq) + row_at(a, a.dqs, b, h, r);
#pragma unroll
    for (int d = 0; d < DT; ++d) store4<T, ALN>(out, d * 16 + (lane >> 4) * 4, a.head_dim, dq[j][d] * a.scale);
  }
}

// dK and dV: a wave holds KT tiles of 16 keys and walks the rows, kBlockRows
// at a time, staged in LDS.  Here the scores have rows as rows, so a lane
// holds rows of one key.
constexpr int kBlockRows = 32;

template <typename T, int DP, int KT, bool ALN>
__global__ __launch_bounds__(kThreads) void k_attn_bwd_kv(AttnArgs a) {
  constexpr int KK = DP / 32, DT = DP / 16;
  __shared__ __attribute__((aligned(16))) T tq[kBlockRows * kLd<T, DP>];
  __shared__ __attribute__((aligned(16))) T tg[kBlockRows * kLd<T, DP>];
  __shared__ __attribute__((aligned(16))) float tl[kBlockRows];
  __shared__ __attribute__((aligned(16))) float td[kBlockRows];
  int b, h, tile;
  if (!place(a, a.key_tiles, &b, &h, &tile)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Span sp = kv_span(a, b);
  const int block_key = tile * (16 * KT * kAttnWaves);
  if (tile == 0 && a.kv_offsets) {  // packed rows before the first entry and after the last: zero
    const long long lo = std::min<long long>(std::max(a.kv_offsets[0], 0), a.kv_rows);
    const long long hi = std::min<long long>(std::max(a.kv_offsets[a.batch], 0), a.kv_rows);
    const long long n0 = b == 0 ? lo : 0, n = n0 + (b == a.batch - 1 ? a.kv_rows - hi : 0);
    for (long long i = wave; i < n; i += kAttnWaves) {
      const long long r = i < n0 ? i : hi + (i - n0);
      for (int d = lane; d < a.head_dim; d += 64) {
        static_cast<T*>(a.dk)[r * a.dks[1] + h * a.dks[2] + d] = (T)0.f;
        static_cast<T*>(a.dv)[r * a.dvs[1] + h * a.dvs[2] + d] = (T)0.f;
      }
    }
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
      const int d0 = c * 32 + (lane >> 4) * 8;
      k[j][c] = load8<T, ALN>(kb + (long long)key * a.ks[1], d0, a.head_dim, in[j]);
      v[j][c] = load8<T, ALN>(vb + (long long)key * a.vs[1], d0, a.head_dim, in[j]);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[j][d] = dv[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const long long stat0 = ((long long)b * a.kv_heads + h) * a.rows;
  const int rows = block_key < sp.len ? a.rows : 0;
  constexpr int kChunks = kBlockRows * (DP / 8), kPer = (kChunks + kThreads - 1) / kThreads;
  Frag<T> sq[kPer], sg[kPer];
  float sl = INFINITY, sd = 0.f;
  auto stage = [&](int first) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * kThreads + threadIdx.x;
      const int r = first + c / (DP / 8), d0 = (c % (DP / 8)) * 8;
      const bool ok = c < kChunks && r < rows;
      sq[i] = load8<T, ALN>(static_cast<const T*>(a.q) + (ok ? row_at(a, a.qs, b, h, r) : 0), d0, a.head_dim, ok);
      sg[i] = load8<T, ALN>(static_cast<const T*>(a.dout) + (ok ? row_at(a, a.dos, b, h, r) : 0), d0, a.head_dim, ok);
    }
    if (threadIdx.x < kBlockRows) {
      const int r = first + threadIdx.x;
      const float lse = r < rows ? a.lse[stat_at(a, b, h, r)] : -INFINITY;
      sl = lse == -INFINITY ? INFINITY : lse * kLog2e;
      sd = r < rows ? a.delta[stat0 + r] : 0.f;
    }
  };
  if (rows > 0) stage(0);
  for (int first = 0; first < rows; first += kBlockRows) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * kThreads + threadIdx.x;
      if (c < kChunks) {
        const int at = (c / (DP / 8)) * kLd<T, DP> + (c % (DP / 8)) * 8;
        *reinterpret_cast<Frag<T>*>(tq + at) = sq[i];
        *reinterpret_cast<Frag<T>*>(tg + at) = sg[i];
      }
    }
    if (threadIdx.x < kBlockRows) {
      tl[threadIdx.x] = sl;
      td[threadIdx.x] = sd;
    }
    __syncthreads();
    if (first + kBlockRows < rows) stage(first + kBlockRows);
    f32x4 s[2][KT], dp[2][KT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < KT; ++j) s[u][j] = dp[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KK; ++c) {
        const Frag<T> fq = read_rows<T, DP>(tq, u * 16, c * 32, lane);
        const Frag<T> fg = read_rows<T, DP>(tg, u * 16, c * 32, lane);
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          s[u][j] = mma(fq, k[j][c], s[u][j]);
          dp[u][j] = mma(fg, v[j][c], dp[u][j]);
        }
      }
      const f32x4 l4 = *reinterpret_cast<const f32x4*>(tl + u * 16 + (lane >> 4) * 4);
      const f32x4 d4 = *reinterpret_cast<const f32x4*>(td + u * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = in[j] ? __builtin_amdgcn_exp2f(s[u][j][i] * c2 - l4[i]) : 0.f;
          s[u][j][i] = p;
          dp[u][j][i] = in[j] ? p * (dp[u][j][i] - d4[i]) : 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      const Frag<T> p = pack<T>(s[0][j], s[1][j]), ds = pack<T>(dp[0][j], dp[1][j]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        dv[j][d] = mma(read_cols<DP>(tg, 0, d * 16, lane), p, dv[j][d]);
        dk[j][d] = mma(read_cols<DP>(tq, 0, d * 16, lane), ds, dk[j][d]);
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
      store4<T, ALN>(dkb + (long long)key * a.dks[1], d0, a.head_dim, dk[j][d] * a.scale);
      store4<T, ALN>(dvb + (long long)key * a.dvs[1], d0, a.head_dim, dv[j][d]);
    }
  }
}

// ----------------------------------------------------------- sizes, launches
struct AttnPlan {
  int dp, qt, kt;
  int row_tiles, key_tiles, splits, split_keys;
  int64_t part_o, part_ml, fwd_bytes, bwd_bytes;
};

constexpr int kMaxHeadDim = 128;

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

AttnPlan attn_plan(const recis_attn_desc* d) {
  AttnPlan p;
  p.dp = d->head_dim <= 32 ? 32 : d->head_dim <= 64 ? 64 : 128;
  const int group = d->q_heads / d->kv_heads;
  const int64_t rows = (int64_t)d->q_len * group, bh = (int64_t)d->batch * d->kv_heads;
  p.qt = rows > 64 && d->dtype == RECIS_DTYPE_BF16 && p.dp <= 64 ? 2 : 1;
  p.kt = d->dtype == RECIS_DTYPE_BF16 && p.dp <= 64 ? 2 : 1;
  p.row_tiles = (int)((rows + 64 * p.qt - 1) / (64 * p.qt));
  p.key_tiles = std::max(1, (int)(((int64_t)d->kv_len + 64 * p.kt - 1) / (64 * p.kt)));
  // keys are split until there are some 2048 blocks, at least 256 keys each
  const int64_t blocks = std::max<int64_t>(1, bh * p.row_tiles);
  const int64_t want = std::max<int64_t>(1, 2048 / blocks);
  p.split_keys = (int)std::max<int64_t>(256, round_up((d->kv_len + want - 1) / want, kBlockKeys));
  p.splits = std::max(1, (int)(((int64_t)d->kv_len + p.split_keys - 1) / p.split_keys));
  p.part_o = 0;
  p.part_ml = round_up(bh * p.splits * rows * d->head_dim * 4, 256);
  p.fwd_bytes = p.splits > 1 ? p.part_ml + round_up(bh * p.splits * rows * 8, 256) : 0;
  p.bwd_bytes = round_up(std::max<int64_t>(bh * rows, 1) * 4, 256);
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
  a->key_tiles = p.key_tiles;
  a->splits = p.splits;
  a->split_keys = p.split_keys;
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
  return true;
}

bool elements_aligned(const recis_attn_desc* d, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p || !aligned_to(p, dtype_size(d->dtype))) return false;
  return true;
}

dim3 attn_grid(const AttnArgs& a, int per) {
  return dim3((unsigned)(round_up((int64_t)a.batch * a.kv_heads, kDies) * per));
}

enum AttnPass { kFwd, kBwdQ, kBwdKv };

template <typename T, int DP, int N, bool ALN>
void launch_pass(AttnPass pass, const AttnArgs& a, hipStream_t s) {
  if (pass == kFwd)
    hipLaunchKernelGGL((k_attn_fwd<T, DP, N, ALN>), attn_grid(a, a.row_tiles * a.splits), dim3(kThreads), 0, s, a);
  else if (pass == kBwdQ)
    hipLaunchKernelGGL((k_attn_bwd_q<T, DP, N, ALN>), attn_grid(a, a.row_tiles), dim3(kThreads), 0, s, a);
  else
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

void launch_attn(AttnPass pass, int dtype, const AttnPlan& p, bool aln, const AttnArgs& a, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16) {
    p.dp == 32 ? launch_dp<__bf16, 32>(pass, p, aln, a, s)
               : p.dp == 64 ? launch_dp<__bf16, 64>(pass, p, aln, a, s) : launch_dp<__bf16, 128>(pass, p, aln, a, s);
  } else {
    p.dp == 32 ? launch_dp<float, 32>(pass, p, aln, a, s)
               : p.dp == 64 ? launch_dp<float, 64>(pass, p, aln, a, s) : launch_dp<float, 128>(pass, p, aln, a, s);
  }
}

bool grid_fits(const recis_attn_desc* d, int64_t per) {
  return round_up((int64_t)d->batch * d->kv_heads, kDies) * per < (1ll << 31);
}

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

int64_t recis_cross_attn_workspace_bytes(const recis_attn_desc* desc, int32_t backward) {
  if (check_desc(desc) != RECIS_OK) return -1;
  const AttnPlan p = attn_plan(desc);
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
  if (p.fwd_bytes && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.fwd_bytes))
    return RECIS_ERR_INVALID_ARG;
  if (!grid_fits(desc, (int64_t)p.row_tiles * p.splits)) return RECIS_ERR_UNSUPPORTED;
  AttnArgs a;
  fill_args(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_o);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_ml);
  const bool aln = rows_aligned(desc, {q, k, v, out},
                                {desc->q_strides, desc->k_strides, desc->v_strides, desc->o_strides});
  launch_attn(kFwd, desc->dtype, p, aln, a, s);
  if (p.splits > 1) {
    const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
    const dim3 grid((unsigned)((rows + kAttnWaves - 1) / kAttnWaves));
    if (desc->dtype == RECIS_DTYPE_BF16)
      hipLaunchKernelGGL((k_attn_join<__bf16>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_attn_join<float>), grid, dim3(kThreads), 0, s, a);
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
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bwd_bytes) return RECIS_ERR_INVALID_ARG;
  if (!grid_fits(desc, std::max(p.row_tiles, p.key_tiles))) return RECIS_ERR_UNSUPPORTED;
  AttnArgs a;
  fill_args(desc, p, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = out;
  a.dout = grad_out;
  a.lse = const_cast<float*>(lse);
  a.delta = static_cast<float*>(workspace);
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  const bool aln = rows_aligned(desc, {q, k, v, out, grad_out, grad_q, grad_k, grad_v},
                                {desc->q_strides, desc->k_strides, desc->v_strides, desc->o_strides,
                                 desc->do_strides, desc->dq_strides, desc->dk_strides, desc->dv_strides});
  if (rows) launch_attn(kBwdQ, desc->dtype, p, aln, a, s);
  if (keys) launch_attn(kBwdKv, desc->dtype, p, aln, a, s);
  return launch_status();
}

}  // extern "C"
