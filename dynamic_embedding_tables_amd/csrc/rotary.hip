// rotary.hip -- positions as rotations of the heads' pairs, alone and on the way
// into a paged cache of keys and values.
//
//   angle = position * freqs[i];  (a, b) -> A (a cos - b sin, b cos + a sin)
//
// for pair i of the first rot_dim elements of each head: (i, i + rot_dim / 2), or
// (2i, 2i + 1) interleaved; the rest of the head is copied.  The gradient is the
// rotation by the negative angle.  Angles are products in 64 bits, reduced to one
// turn there (a position of 10^6 leaves 32 bits an error of 0.06 radians); cosine,
// sine and the rotation are float32, results are rounded once.
//
// Bound by memory.  A block takes whole tokens: their cosines and sines once, into
// LDS, for all heads; then its threads walk the tokens' elements in order, V pairs
// at a time, 16 bytes of either element.  The table is small, 8 KB, so that eight
// blocks stay on a CU: at 32 KB four do, and appending 2048 packed histories of up to
// 1000 events (1.57 GB; 4 heads of 32, bf16) took 457 us, at 8 KB 355.  Values are
// copied by a loop of their own, since a wave that holds both kinds rotates with half
// its lanes: 338 -> 307 us, 5.1 TB/s, where a large copy reaches 4.9.  Rotating 2048 x
// 1000 events alone, 4 heads: 184 us a pass, 5.7 TB/s of requests, some of which the
// last-level cache answers.  One event each for 64 users: 3 to 4 us, the launch.
#include <algorithm>

#include "seq.h"
#include "divide.h"

namespace recis {
namespace {

constexpr int kMaxTurnDim = 1024;           // elements a head
constexpr int kMaxTokenElems = 1 << 18;     // elements a token
constexpr int kTurnTable = 1024;            // pairs of LDS a block: 8 KB
constexpr int kMaxTokens = 64;              // tokens a block

struct Turns {
  const double* freqs;
  int half;  // pairs
  float amp_c, amp_s;
};

// Cosine and sine of `tokens` positions into the table, token by token.
__device__ __forceinline__ void fill_turns(const Turns& a, const long long* pos, int tokens, Div half, f32x2* table) {
  constexpr double kInvTurn = 0.15915494309189535;  // 1 / (2 pi)
  for (unsigned i = threadIdx.x; i < (unsigned)(tokens * a.half); i += kThreads) {
    const unsigned t = divided(i, half);
    const double turns = (double)pos[t] * a.freqs[i - t * half.d] * kInvTurn;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    table[i] = f32x2{c * a.amp_c, s * a.amp_s};
  }
}

// V pairs, held as lo and hi: of halves the first and the second elements, of
// neighbours the first and the second V of 2 V elements.
template <int V, bool NEIGHBOURS>
__device__ __forceinline__ void turn(const f32x2* table, float (&lo)[V], float (&hi)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const f32x2 t = table[i];
    float *pa, *pb;
    if constexpr (NEIGHBOURS) {
      pa = 2 * i < V ? &lo[(2 * i) % V] : &hi[(2 * i) % V];
      pb = 2 * i + 1 < V ? &lo[(2 * i + 1) % V] : &hi[(2 * i + 1) % V];
    } else {
      pa = &lo[i];
      pb = &hi[i];
    }
    const float a = *pa, b = *pb;
    *pa = a * t[0] - b * t[1];
    *pb = b * t[0] + a * t[1];
  }
}

// Item j of a head: V pairs, or past those V elements of the rest.
template <typename T, int V, bool NEIGHBOURS>
__device__ __forceinline__ void turn_item(const T* from, T* to, const f32x2* table, int j, int turned, int half) {
  if (j < turned) {
    const int e0 = NEIGHBOURS ? 2 * j * V : j * V, e1 = NEIGHBOURS ? e0 + V : e0 + half;
    float lo[V], hi[V];
    load_f32<T, V>(from + e0, lo);
    load_f32<T, V>(from + e1, hi);
    turn<V, NEIGHBOURS>(table + j * V, lo, hi);
    store_f32<T, V>(to + e0, lo);
    store_f32<T, V>(to + e1, hi);
  } else {
    const int e = 2 * half + (j - turned) * V;
    *reinterpret_cast<Vec<T, V>*>(to + e) = *reinterpret_cast<const Vec<T, V>*>(from + e);
  }
}

// ------------------------------------------------------------ rotation alone
struct RotaryArgs {
  const void* x;
  void* out;
  const int64_t* positions;  // or null: the place in the sequence
  Turns turns;
  int64_t tokens, seq;
  int64_t xs[3], os[3], ps[2];  // batch, position, head
  int per_block, turned;  // turned: items of a head that are V pairs, the rest's being V elements
  Div by_half, by_token, by_head;
};

template <typename T, int V, bool NEIGHBOURS>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a) {
  __shared__ f32x2 table[kTurnTable];
  __shared__ long long pos[kMaxTokens], at_x[kMaxTokens], at_o[kMaxTokens];
  const int64_t first = (int64_t)block_id() * a.per_block;
  if (first >= a.tokens) return;
  const int tokens = (int)std::min<int64_t>(a.per_block, a.tokens - first);
  if ((int)threadIdx.x < tokens) {
    const int64_t n = first + threadIdx.x, b = n / a.seq, s = n - b * a.seq;
    pos[threadIdx.x] = a.positions ? a.positions[b * a.ps[0] + s * a.ps[1]] : s;
    at_x[threadIdx.x] = b * a.xs[0] + s * a.xs[1];
    at_o[threadIdx.x] = b * a.os[0] + s * a.os[1];
  }
  __syncthreads();
  fill_turns(a.turns, pos, tokens, a.by_half, table);
  __syncthreads();
  const unsigned all = tokens * a.by_token.d;
  for (unsigned i = threadIdx.x; i < all; i += kThreads) {
    const unsigned t = a.per_block == 1 ? 0 : divided(i, a.by_token);
    const unsigned in = i - t * a.by_token.d, h = divided(in, a.by_head), j = in - h * a.by_head.d;
    turn_item<T, V, NEIGHBOURS>(static_cast<const T*>(a.x) + at_x[t] + h * a.xs[2],
                                static_cast<T*>(a.out) + at_o[t] + h * a.os[2], table + t * a.turns.half, j, a.turned,
                                a.turns.half);
  }
}

// ----------------------------------------------------------------- appending
struct AppendArgs {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  const int *offsets, *lens, *table;
  unsigned* error;
  Turns turns;
  int64_t rows, table_stride, pages;
  int64_t qs[3], qos[3], ks[3], vs[3];  // batch, position, head
  int64_t kcs[3], vcs[3];               // page, slot, head
  int batch, new_len, width, page_size;
  int q_heads, per_block, turned;  // turned: as in RotaryArgs, of a head of q and k
  Div by_half, by_token, by_head, by_v_token, by_copied;  // by_token: of q and k
};

// The entry of a packed row: the largest b in [lo, hi] with offsets[b] <= row.
__device__ __forceinline__ int entry_of(const int* offsets, int lo, int hi, int64_t row) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= row)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The same for one row by a whole wave, 64 probes a round.
__device__ __forceinline__ int wave_entry_of(const int* offsets, int batch, int64_t row) {
  int lo = 0, n = batch;  // among lo .. lo + n - 1
  const int lane = threadIdx.x & 63;
  while (n > 1) {
    const int step = (n + 63) / 64, at = lane * step;
    const unsigned long long under = __ballot(at < n && offsets[lo + at] <= row);
    const int last = under ? 63 - __clzll(under) : 0;
    lo += last * step;
    n = std::min(step, n - last * step);
  }
  return lo;
}

template <typename T, int V, bool NEIGHBOURS>
__global__ __launch_bounds__(kThreads) void k_cache_append(AppendArgs a) {
  __shared__ f32x2 table[kTurnTable];
  __shared__ long long pos[kMaxTokens], at_q[kMaxTokens], at_qo[kMaxTokens], at_k[kMaxTokens], at_v[kMaxTokens];
  __shared__ long long at_kc[kMaxTokens], at_vc[kMaxTokens];  // -1: not stored
  __shared__ int ends[2], none[kMaxTokens];
  const int64_t first = (int64_t)block_id() * a.per_block;
  if (first >= a.rows) return;
  const int tokens = (int)std::min<int64_t>(a.per_block, a.rows - first);
  const int64_t room = (int64_t)a.width * a.page_size;
  bool bad = false;
  if (first == 0 && a.error) {  // what no row's own checks see
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      bad |= a.lens[b] < 0 || a.lens[b] > room;
      if (a.offsets) bad |= a.offsets[b] < 0 || a.offsets[b + 1] < a.offsets[b] || a.offsets[b + 1] > a.rows;
    }
  }
  if (a.offsets) {
    const int wave = threadIdx.x >> 6;
    if (wave < 2) {
      const int e = wave_entry_of(a.offsets, a.batch, wave ? first + tokens - 1 : first);
      if ((threadIdx.x & 63) == 0) ends[wave] = e;
    }
    __syncthreads();
  }
  if ((int)threadIdx.x < tokens) {
    const int t = threadIdx.x;
    const int64_t n = first + t;
    int64_t b, i, count = a.new_len;
    bool in = true;
    if (a.offsets) {
      b = entry_of(a.offsets, ends[0], ends[1], n);
      i = n - a.offsets[b];
      count = (int64_t)a.offsets[b + 1] - a.offsets[b];
      in = i >= 0 && i < count && a.offsets[b] >= 0 && a.offsets[b + 1] <= a.rows;
    } else {
      b = n / a.new_len;
      i = n - b * a.new_len;
    }
    const int64_t len = in ? a.lens[b] : 0;
    if (len < 0 || len > room) in = false;
    const int64_t p = len - count + i;
    const int64_t bb = a.offsets ? 0 : b, ii = a.offsets ? n : i;
    at_q[t] = bb * a.qs[0] + ii * a.qs[1];
    at_qo[t] = bb * a.qos[0] + ii * a.qos[1];
    at_k[t] = bb * a.ks[0] + ii * a.ks[1];
    at_v[t] = bb * a.vs[0] + ii * a.vs[1];
    pos[t] = in ? p : 0;
    none[t] = !in;
    at_kc[t] = at_vc[t] = -1;
    if (in && p >= 0) {
      const int64_t turn = (unsigned)p / (unsigned)a.page_size, slot = p - turn * a.page_size;
      const int64_t page = a.table[b * a.table_stride + turn];
      if (page >= 0 && page < a.pages) {
        at_kc[t] = page * a.kcs[0] + slot * a.kcs[1];
        at_vc[t] = page * a.vcs[0] + slot * a.vcs[1];
      } else {
        bad = true;
      }
    }
  }
  if (bad && a.error) atomicOr(a.error, kErrInvalid);
  __syncthreads();
  fill_turns(a.turns, pos, tokens, a.by_half, table);
  __syncthreads();
  const unsigned turned = tokens * a.by_token.d;
  for (unsigned x = threadIdx.x; x < turned; x += kThreads) {
    const unsigned t = a.per_block == 1 ? 0 : divided(x, a.by_token);
    const unsigned in = x - t * a.by_token.d, head = divided(in, a.by_head), j = in - head * a.by_head.d;
    const T* from;
    T* to;
    if (head < (unsigned)a.q_heads) {
      from = static_cast<const T*>(a.q) + at_q[t] + head * a.qs[2];
      to = static_cast<T*>(a.qo) + at_qo[t] + head * a.qos[2];
      if (none[t]) {  // a row of no entry
        const float zero[V] = {};
        if ((int)j < a.turned) {
          const int e0 = NEIGHBOURS ? 2 * j * V : j * V, e1 = NEIGHBOURS ? e0 + V : e0 + a.turns.half;
          store_f32<T, V>(to + e0, zero);
          store_f32<T, V>(to + e1, zero);
        } else {
          store_f32<T, V>(to + 2 * a.turns.half + (j - a.turned) * V, zero);
        }
        continue;
      }
    } else {
      if (at_kc[t] < 0) continue;
      from = static_cast<const T*>(a.k) + at_k[t] + (head - a.q_heads) * a.ks[2];
      to = static_cast<T*>(a.kc) + at_kc[t] + (head - a.q_heads) * a.kcs[2];
    }
    turn_item<T, V, NEIGHBOURS>(from, to, table + t * a.turns.half, j, a.turned, a.turns.half);
  }
  const unsigned copied = tokens * a.by_v_token.d;
  for (unsigned x = threadIdx.x; x < copied; x += kThreads) {
    const unsigned t = a.per_block == 1 ? 0 : divided(x, a.by_v_token);
    const unsigned in = x - t * a.by_v_token.d, h = divided(in, a.by_copied), j = in - h * a.by_copied.d;
    if (at_vc[t] < 0) continue;
    *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.vc) + at_vc[t] + h * a.vcs[2] + j * V) =
        *reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.v) + at_v[t] + h * a.vs[2] + j * V);
  }
}

// Tokens a block: about 2048 items, but 4096 blocks -- two turns of all that the
// chip holds -- before any takes a second token, and their turns fit the table.
// (Items 1024 / 2048: appending those histories 310 / 307 us; blocks 512 / 4096
// with 47 397 tokens of 42 items: 25.6 / 23.1 us a pass.)
int tokens_a_block(int64_t tokens, int64_t items, int half) {
  int64_t n = std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, 2048 / std::max<int64_t>(1, items)));
  if (half) n = std::min<int64_t>(n, kTurnTable / half);
  return (int)std::max<int64_t>(1, std::min(n, (tokens + 4095) / 4096));
}

// The widest access of a head's halves (or neighbours) and its rest.
int turn_width(int size, int head_dim, int half, std::initializer_list<const void*> ptrs,
               std::initializer_list<int64_t> strides) {
  int v = access_width(size, head_dim, ptrs, strides);
  while (v > 1 && half % v) v /= 2;
  return v;
}

template <typename T, int V>
void launch_rotary(bool neighbours, const RotaryArgs& a, dim3 grid, hipStream_t s) {
  if (neighbours)
    hipLaunchKernelGGL((k_rotary<T, V, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_rotary<T, V, false>), grid, dim3(kThreads), 0, s, a);
}
template <typename T, int V>
void launch_append(bool neighbours, const AppendArgs& a, dim3 grid, hipStream_t s) {
  if (neighbours)
    hipLaunchKernelGGL((k_cache_append<T, V, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_cache_append<T, V, false>), grid, dim3(kThreads), 0, s, a);
}

#define RECIS_BY_WIDTH(launch, dtype, v, ...)              \
  do {                                                     \
    if ((dtype) == RECIS_DTYPE_BF16) {                     \
      if ((v) == 8) launch<__bf16, 8>(__VA_ARGS__);        \
      else if ((v) == 4) launch<__bf16, 4>(__VA_ARGS__);   \
      else if ((v) == 2) launch<__bf16, 2>(__VA_ARGS__);   \
      else launch<__bf16, 1>(__VA_ARGS__);                 \
    } else {                                               \
      if ((v) == 4) launch<float, 4>(__VA_ARGS__);         \
      else if ((v) == 2) launch<float, 2>(__VA_ARGS__);    \
      else launch<float, 1>(__VA_ARGS__);                  \
    }                                                      \
  } while (0)

bool turn_known(int dtype, int head_dim, int rot_dim, float amplitude, const double* freqs) {
  return dtype_known(dtype) && head_dim >= 1 && rot_dim >= 0 && rot_dim <= head_dim && rot_dim % 2 == 0 &&
         amplitude - amplitude == 0.f && (rot_dim == 0 || freqs) && aligned_to(freqs, 8);
}

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

recis_status recis_rotary(const recis_rotary_desc* d, int32_t backward, const void* x, void* out, hipStream_t s) {
  if (!d || !turn_known(d->dtype, d->head_dim, d->rot_dim, d->amplitude, d->freqs) || d->batch < 0 || d->seq < 0 ||
      d->heads < 1 || !aligned_to(d->positions, 8))
    return RECIS_ERR_INVALID_ARG;
  if (d->head_dim > kMaxTurnDim || (int64_t)d->heads * d->head_dim > kMaxTokenElems || d->batch > (1ll << 40) ||
      d->seq > (1ll << 40) || (d->seq > 0 && d->batch > (1ll << 40) / d->seq))
    return RECIS_ERR_UNSUPPORTED;
  const int size = dtype_size(d->dtype);
  if (!aligned_to(x, size) || !aligned_to(out, size)) return RECIS_ERR_INVALID_ARG;
  if (d->batch == 0 || d->seq == 0) return RECIS_OK;
  if (!x || !out) return RECIS_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.x = x;
  a.out = out;
  a.positions = d->positions;
  a.turns.freqs = d->freqs;
  a.turns.half = d->rot_dim / 2;
  a.turns.amp_c = d->amplitude;
  a.turns.amp_s = backward ? -d->amplitude : d->amplitude;
  a.tokens = d->batch * d->seq;
  a.seq = d->seq;
  bool same = x == out;
  const int64_t axes[3] = {d->batch, d->seq, d->heads};
  for (int i = 0; i < 3; ++i) {
    a.xs[i] = stride_of(d->x_strides[i], axes[i]);
    a.os[i] = stride_of(d->out_strides[i], axes[i]);
    same = same && a.xs[i] == a.os[i];
  }
  if (x == out && !same) return RECIS_ERR_INVALID_ARG;
  a.ps[0] = d->pos_strides[0];
  a.ps[1] = d->pos_strides[1];
  const int v = turn_width(size, d->head_dim, a.turns.half, {x, out},
                           {a.xs[0], a.xs[1], a.xs[2], a.os[0], a.os[1], a.os[2]});
  a.turned = a.turns.half / v;
  const int items = a.turned + (same ? 0 : (d->head_dim - d->rot_dim) / v);  // of a head (in place the rest is there)
  if (items == 0) return RECIS_OK;
  const int64_t per_token = (int64_t)d->heads * items;
  a.per_block = tokens_a_block(a.tokens, per_token, a.turns.half);
  a.by_half = div_by(std::max(1, a.turns.half));
  a.by_token = div_by(per_token);
  a.by_head = div_by(items);
  const int64_t blocks = (a.tokens + a.per_block - 1) / a.per_block;
  if (blocks > kMaxBlocks) return RECIS_ERR_UNSUPPORTED;
  RECIS_BY_WIDTH(launch_rotary, d->dtype, v, d->interleaved != 0, a, grid_of(blocks), s);
  return launch_status();
}

recis_status recis_cache_append(const recis_append_desc* d, const void* q, const void* k, const void* v, void* q_out,
                                void* k_cache, void* v_cache, hipStream_t s) {
  if (!d || !turn_known(d->dtype, d->head_dim, d->rot_dim, d->amplitude, d->freqs) || d->batch < 0 || d->new_len < 0 ||
      d->q_heads < 0 || d->kv_heads < 1 || d->page_size < 1 || d->pages < 0 || d->table_width < 0 ||
      d->table_stride < d->table_width || !aligned_to(d->kv_lens, 4) || !aligned_to(d->q_offsets, 4) ||
      !aligned_to(d->page_table, 4) || !aligned_to(d->error, 4) ||
      (d->q_offsets && d->rows < 0))
    return RECIS_ERR_INVALID_ARG;
  if (d->head_dim > kMaxTurnDim || (int64_t)(d->q_heads + 2ll * d->kv_heads) * d->head_dim > kMaxTokenElems ||
      d->page_size > (1 << 30) || (int64_t)d->table_width * d->page_size > (1 << 30) || d->pages > (1ll << 31) ||
      (d->q_offsets && d->rows > (1ll << 31)))
    return RECIS_ERR_UNSUPPORTED;
  const int size = dtype_size(d->dtype);
  for (const void* p : {q, k, v, (const void*)q_out, (const void*)k_cache, (const void*)v_cache})
    if (!aligned_to(p, size)) return RECIS_ERR_INVALID_ARG;
  const int64_t rows = d->q_offsets ? d->rows : (int64_t)d->batch * d->new_len;
  if (d->batch == 0 || rows == 0) return RECIS_OK;
  if (!k || !v || !d->kv_lens || (d->q_heads && (!q || !q_out))) return RECIS_ERR_INVALID_ARG;
  if (d->pages > 0 && d->table_width > 0 && (!k_cache || !v_cache || !d->page_table)) return RECIS_ERR_INVALID_ARG;
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.kc = k_cache;
  a.vc = v_cache;
  a.offsets = d->q_offsets;
  a.lens = d->kv_lens;
  a.table = d->page_table;
  a.error = d->error;
  a.turns.freqs = d->freqs;
  a.turns.half = d->rot_dim / 2;
  a.turns.amp_c = a.turns.amp_s = d->amplitude;
  a.rows = rows;
  a.table_stride = d->table_stride;
  a.pages = d->pages;
  const int64_t lead[2] = {d->q_offsets ? 1 : d->batch, d->q_offsets ? rows : d->new_len};
  const int64_t q_axes[3] = {lead[0], lead[1], d->q_heads}, kv_axes[3] = {lead[0], lead[1], d->kv_heads};
  const int64_t cache_axes[3] = {d->pages, d->page_size, d->kv_heads};
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = stride_of(d->q_strides[i], q_axes[i]);
    a.qos[i] = stride_of(d->q_out_strides[i], q_axes[i]);
    a.ks[i] = stride_of(d->k_strides[i], kv_axes[i]);
    a.vs[i] = stride_of(d->v_strides[i], kv_axes[i]);
    a.kcs[i] = stride_of(d->k_cache_strides[i], cache_axes[i]);
    a.vcs[i] = stride_of(d->v_cache_strides[i], cache_axes[i]);
    if (d->q_heads && q == q_out && a.qs[i] != a.qos[i]) return RECIS_ERR_INVALID_ARG;
  }
  a.batch = d->batch;
  a.new_len = d->new_len;
  a.width = d->table_width;
  a.page_size = d->page_size;
  a.q_heads = d->q_heads;
  int w = turn_width(size, d->head_dim, a.turns.half, {k, v, k_cache, v_cache},
                     {a.ks[0], a.ks[1], a.ks[2], a.vs[0], a.vs[1], a.vs[2], a.kcs[0], a.kcs[1], a.kcs[2], a.vcs[0],
                      a.vcs[1], a.vcs[2]});
  if (d->q_heads)
    w = std::min(w, turn_width(size, d->head_dim, a.turns.half, {q, q_out},
                               {a.qs[0], a.qs[1], a.qs[2], a.qos[0], a.qos[1], a.qos[2]}));
  a.turned = a.turns.half / w;
  // items of a head of q and k, and of one of v
  const int items = a.turned + (d->head_dim - d->rot_dim) / w, copied = d->head_dim / w;
  const int64_t per_token = (int64_t)(d->q_heads + d->kv_heads) * items + (int64_t)d->kv_heads * copied;
  a.per_block = tokens_a_block(rows, per_token, a.turns.half);
  a.by_half = div_by(std::max(1, a.turns.half));
  a.by_token = div_by((int64_t)(d->q_heads + d->kv_heads) * items);
  a.by_head = div_by(items);
  a.by_v_token = div_by((int64_t)d->kv_heads * copied);
  a.by_copied = div_by(copied);
  const int64_t blocks = (rows + a.per_block - 1) / a.per_block;
  if (blocks > kMaxBlocks) return RECIS_ERR_UNSUPPORTED;
  RECIS_BY_WIDTH(launch_append, d->dtype, w, d->interleaved != 0, a, grid_of(blocks), s);
  return launch_status();
}

}  // extern "C"
