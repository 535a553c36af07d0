// paged.hip -- attention of new events to a paged cache of keys and values.
//
//   O = softmax(scale q k^T) v over the keys of the entry that the row sees (band.h)
//
// An entry's key j lies in slot j % page_size of page page_table[entry][j / page_size].
// Up to 16 rows a pair (batch entry, key head) -- single events and the query heads
// that share the key head -- run here; more run in band_fwd.hip's kernel.
//
// Bound by memory: the keys and values are read once.  The block's waves take turns of
// 32 keys and meet once, at the end.  Keys go from memory into the product's operand
// directly, values through LDS of the wave's own, so no wave waits for another while
// the keys stream.  A lane asks for one key's page a turn ahead; the others get its
// address by an exchange, or, where 16 keys share a page, from scalar registers.
//
// The keys an entry sees are split evenly over `splits` blocks, whatever its length;
// an entry short enough for one needs no join.
//
// 64 single events over up to 8192 keys, 16 heads of 128 that share 4, bfloat16: 120 us a
// call, 4.5 TB/s, where a large copy reaches 4.9 (all pairs of an entry on one die, a pair's
// blocks side by side; with the pairs of a tile side by side 127).  The same over 8192 keys
// each in float32, 2.15 GB: 399 to 437 us, 4.9 to 5.4 TB/s, although heads above 96 leave it
// one wave a SIMD.  4 events over up to 200 keys, 4 heads of 32, float32: 6 us, the launch
// and three dependent reads.
#include <algorithm>
#include <cmath>

#include "band.h"

namespace recis {
namespace {

constexpr int kFewRows = 16, kFewKeys = 32, kFewLeast = 8;  // a split has 8 turns where there are so many

__device__ __forceinline__ long long lane_value(long long x, int lane) {
  const int lo = __builtin_amdgcn_readlane((int)x, lane), hi = __builtin_amdgcn_readlane((int)(x >> 32), lane);
  return ((long long)hi << 32) | (unsigned)lo;
}

// 8 elements from d0 of a row, W at a time; zeros past its `dim` elements and where it is not
// `in` (then `row` is one that is there all the same: by 2, it is read and replaced).  (64
// single events over 4096 keys, 16 heads of 74 that share 4: bfloat16 197 us by 1, 161 by 2,
// float32 314, 205.)
template <typename T, int W>
__device__ __forceinline__ Frag<T> few_row(const T* row, int d0, int dim, bool in) {
  if constexpr (W == 2) {
    Frag<T> f = load_any<T, 2>(row, d0, dim);
    zero_past<T, 2>(f, in ? d0 : dim, dim);
    return f;
  } else {
    return load8<T, W == 8>(row, d0, dim, in);
  }
}
// The operand for chunk c of a row (load_head), likewise.
template <typename T, int W>
__device__ __forceinline__ Frag<T> few_head(const T* row, int c, int lane, int dim, bool in) {
  if constexpr (W != 2) {
    return load_head<T, W == 8>(row, c, lane, dim, in);
  } else if constexpr (sizeof(T) == 2) {
    return few_row<T, 2>(row, c * 32 + (lane >> 4) * 8, dim, in);
  } else {
    typedef T Part __attribute__((ext_vector_type(2)));
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const int d = c * 32 + i / 4 * 16 + (lane >> 4) * 4 + i % 4;
      const Part x = *reinterpret_cast<const Part*>(row + std::min(d, dim - 2));
      f[i] = in && d < dim ? x[0] : 0.f;
      f[i + 1] = in && d < dim ? x[1] : 0.f;
    }
    return f;
  }
}

template <typename T, int DP, int W>
__global__ __launch_bounds__(kThreads) void k_paged_few(BandArgs a) {
  constexpr int KK = kChunks32<DP>, DT = DP / 16;
  constexpr int kAcross = kCols<DP> / 8, kRows = 64 / kAcross, kPer = kFewKeys / kRows;  // chunks of values a lane
  constexpr int kTile = kFewKeys * kLd<T, DP>;
  __shared__ __attribute__((aligned(128))) T tiles[kBandWaves * kTile];
  __shared__ float refs[kBandWaves][kFewRows], sums[kBandWaves][kFewRows];
  static_assert(kTile * (int)sizeof(T) >= kFewRows * DP * 4, "a wave's output fits its tile");
  int b, h, tile, split;
  if (!band_place(a, &b, &h, &tile, &split)) return;
  const int lane = threadIdx.x & 63, wave = wave_of();
  const Entry e = entry_at<true>(a, b);
  const int rows = e.n * a.group;
  const Reach reach = reach_of(a, e, 0, kFewRows - 1);
  const Walk walk = walk_of<kFewKeys>(a, reach);
  const int per = split_size(walk.n, a.splits, kFewLeast);
  const int i0 = split * per, i1 = std::min(walk.n, i0 + per);
  if (rows == 0 || (split > 0 && i0 >= walk.n)) return;
  const int* table = a.table + (long long)b * a.table_stride;
  const T* kb = static_cast<const T*>(a.k) + (long long)h * a.ks[2];
  const T* vb = static_cast<const T*>(a.v) + (long long)h * a.vs[2];
  const float c2 = a.scale * kLog2e;
  const f32x4 zero = zeros();
  const int kr = lane & 15;  // the lane's row of the queries, and its key of 16
  const int p = kr < rows ? position(a, e, divided(kr, a.by_group)) : -1;
  Frag<T> q[KK];
  {
    const bool in = kr < rows;
    const T* from = static_cast<const T*>(a.q) + (in ? query_at(a, a.qs, e, b, h, kr) : 0);
#pragma unroll
    for (int c = 0; c < KK; ++c) q[c] = few_head<T, W>(from, c, lane, a.head_dim, in);
  }
  Frag<T> kf[2][KK], vf[kPer];
  const int vr = lane / kAcross, vd = (lane % kAcross) * 8;  // the lane's place in 64 chunks of values
  constexpr int kHalf = sizeof(T) == 2 ? 8 : 4;              // the operand's first elements (load_head)
  const unsigned k_at = (unsigned)((kr * a.ks[1] + (lane >> 4) * kHalf) * (long long)sizeof(T));  // W = 8: fits
  const unsigned v_at = (unsigned)((vr * a.vs[1] + vd) * (long long)sizeof(T));
  const bool by16 = W == 8 && a.by_page.d % 16 == 0 && a.head_dim == kCols<DP>;
  const int window_lo = reach.low - a.window + 1;  // before it no row sees a key but the sinks
  auto wanted = [&](int key) { return key < e.len && (key >= window_lo || key < a.sinks); };
  auto ask_page = [&](int first) {
    const int key = first + (lane & 31);
    return wanted(key) ? table[page_of(a, key)] : 0;
  };
  auto at_bytes = [](const T* base, unsigned bytes) {
    return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + bytes);
  };
  // 32 keys from `first`, whose page the lane was told; returns the keys that are there
  auto fetch = [&](int first, int page) {
    const int key = first + (lane & 31);
    bool in = wanted(key);
    if (in && (unsigned)page >= (unsigned long long)a.pages) {
      in = false;
      if (a.error) atomicOr(a.error, kErrInvalid);
    }
    const unsigned bits = (unsigned)__ballot(in);
    const int slot = key - page_of(a, key) * a.by_page.d;
    const long long ko = in ? (long long)page * a.ks[0] + (long long)slot * a.ks[1] : 0;
    const long long vo = in ? (long long)page * a.vs[0] + (long long)slot * a.vs[1] : 0;
    if (by16 && bits == ~0u) {
      const T *k16[2], *v16[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        k16[u] = kb + lane_value(ko, u * 16);
        v16[u] = vb + lane_value(vo, u * 16);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < KK; ++c) {
          const T* from = at_bytes(k16[u] + c * 32, k_at);
          if constexpr (sizeof(T) == 2) {
            kf[u][c] = *reinterpret_cast<const Frag<T>*>(from);
          } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(from);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(from + 16);
            kf[u][c] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        constexpr int kIn16 = 16 / kRows;
        vf[i] = *reinterpret_cast<const Frag<T>*>(
            at_bytes(v16[i / kIn16] + (long long)(i % kIn16 * kRows) * a.vs[1], v_at));
      }
      return bits;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const T* from = kb + __shfl(ko, u * 16 + kr);
#pragma unroll
      for (int c = 0; c < KK; ++c)
        kf[u][c] = few_head<T, W>(from, c, lane, a.head_dim, (bits >> (u * 16 + kr)) & 1);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      vf[i] = few_row<T, W>(vb + __shfl(vo, i * kRows + vr), vd, a.head_dim, (bits >> (i * kRows + vr)) & 1);
    return bits;
  };
  f32x4 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = zero;
  float m = -INFINITY, ref = 0.f, most = -INFINITY, l = 0.f;
  T* tv = tiles + wave * kTile;
  unsigned bits = 0;
  int page = 0, i = i0 + wave;
  if (i < i1) {
    const int first = walk.tile(i) * kFewKeys;
    bits = fetch(first, ask_page(first));
    if (i + kBandWaves < i1) page = ask_page(walk.tile(i + kBandWaves) * kFewKeys);
  }
  for (; i < i1; i += kBandWaves) {
    const int first = walk.tile(i) * kFewKeys;
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
      for (int x = 0; x < kPer; ++x)
        *reinterpret_cast<Frag<T>*>(tv + chunk_at<T, DP>(x * kRows + vr, vd / 8)) = vf[x];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are executed in order
    if (i + kBandWaves < i1) {
      bits = fetch(walk.tile(i + kBandWaves) * kFewKeys, page);
      if (i + 2 * kBandWaves < i1) page = ask_page(walk.tile(i + 2 * kBandWaves) * kFewKeys);
    }
    if (now != ~0u || !all_seen<kFewKeys>(a, reach, first)) {
      const unsigned mine = ((unsigned)seen_bits(a, p, first) & now) >> ((lane >> 4) * 4);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (!((mine >> (u * 16 + x)) & 1)) s[u][x] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) top = fmaxf(top, s[u][x]);
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
      for (int x = 0; x < 4; ++x) {
        s[u][x] = __builtin_amdgcn_exp2f(s[u][x] * c2 - ref);
        l += s[u][x];
      }
    const Frag<T> w = pack<T>(s[0], s[1]);
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = mma(read_cols<DP>(tv, 0, d * 16, lane), w, o[d]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  l = group_add(l);
  if (p < 0) {  // a row that sees nothing, whatever its block walked
    l = 0.f;
    m = -INFINITY;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = zero;
  }
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
  if (r >= rows) return;
  float top = refs[0][r];
#pragma unroll
  for (int w = 1; w < kBandWaves; ++w) top = fmaxf(top, refs[w][r]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, out[DT];
#pragma unroll
  for (int x = 0; x < DT; ++x) out[x] = 0.f;
#pragma unroll
  for (int w = 0; w < kBandWaves; ++w) {
    const float weight = __builtin_amdgcn_exp2f(refs[w][r] - base);
    sum += weight * sums[w][r];
    const float* from = reinterpret_cast<const float*>(tiles + w * kTile) + r * DP + d0;
#pragma unroll
    for (int x = 0; x < DT; ++x) out[x] += weight * from[x];
  }
  if (walk.n > per) {
    const long long at = (((long long)b * a.kv_heads + h) * a.splits + split) * a.rows + r;
#pragma unroll
    for (int x = 0; x < DT; ++x)
      if (d0 + x < a.head_dim) a.part_o[at * a.head_dim + d0 + x] = out[x];
    if (d0 == 0) {
      a.part_ml[2 * at] = top;
      a.part_ml[2 * at + 1] = sum;
    }
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* to = static_cast<T*>(a.out) + query_at(a, a.os, e, b, h, r);
#pragma unroll
  for (int x = 0; x < DT; ++x)
    if (d0 + x < a.head_dim) to[d0 + x] = (T)(out[x] * inv);
  if (a.lse && d0 == 0) a.lse[lse_at(a, e, b, h, r)] = sum == 0.f ? -INFINITY : top * kLn2 + __logf(sum);
}

template <typename T, int DP>
void launch_few(int access, BandArgs a, hipStream_t s) {
  const dim3 grid = band_grid(&a, 1, a.splits);
  if (access == 8)
    hipLaunchKernelGGL((k_paged_few<T, DP, 8>), grid, dim3(kThreads), 0, s, a);
  else if (access == 2)
    hipLaunchKernelGGL((k_paged_few<T, DP, 2>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_paged_few<T, DP, 1>), grid, dim3(kThreads), 0, s, a);
}

template <typename T>
void launch_few_dp(int access, const BandArgs& a, hipStream_t s) {
  const int d = a.head_dim;
  if (d <= 32)
    launch_few<T, 32>(access, a, s);
  else if (sizeof(T) == 4 && d <= 48)
    launch_few<T, sizeof(T) == 4 ? 48 : 64>(access, a, s);
  else if (d <= 64)
    launch_few<T, 64>(access, a, s);
  else if (d <= 96)
    launch_few<T, 96>(access, a, s);
  else
    launch_few<T, 128>(access, a, s);
  if (a.splits > 1) launch_join<T, true, kFewKeys, kFewRows, kFewLeast>(a, s);
}

// ----------------------------------------------------------- sizes, launches
struct PagedPlan {
  bool few;
  int row_tiles, splits;
  int64_t ml_at, bytes;
};

recis_status check_paged(const recis_paged_attn_desc* d) {
  if (!d || !dtype_known(d->dtype) || d->batch < 0 || d->q_len < 0 || d->q_heads < 1 || d->kv_heads < 1 ||
      d->head_dim < 1 || d->q_heads % d->kv_heads || !(d->scale > 0.f) || !std::isfinite(d->scale) ||
      d->window < 0 || d->sinks < 0 || (!d->causal && d->window) || d->page_size < 1 || d->pages < 0 ||
      d->table_width < 0 || d->table_stride < d->table_width || (d->q_offsets && d->q_rows < 0))
    return RECIS_ERR_INVALID_ARG;
  if (!aligned_to(d->q_offsets, 4) || !aligned_to(d->kv_lens, 4) || !aligned_to(d->page_table, 4) ||
      !aligned_to(d->error, 4))
    return RECIS_ERR_INVALID_ARG;
  if (d->head_dim > kMaxHeadDim || (int64_t)d->table_width * d->page_size > (1 << 30) || d->page_size > (1 << 30) ||
      d->pages > (1ll << 31) || (int64_t)d->q_len * (d->q_heads / d->kv_heads) > (1 << 30) ||
      (int64_t)d->batch * d->kv_heads > (1 << 24))
    return RECIS_ERR_UNSUPPORTED;
  return RECIS_OK;
}

int window_of(int window) { return window ? std::min(window, 1 << 30) : 1 << 30; }

PagedPlan paged_plan(const recis_paged_attn_desc* d) {
  PagedPlan p;
  const int group = d->q_heads / d->kv_heads;
  const int64_t rows = (int64_t)d->q_len * group, pairs = (int64_t)d->batch * d->kv_heads;
  const int64_t room = (int64_t)d->table_width * d->page_size;
  p.few = rows <= kFewRows;
  const int tile = p.few ? kFewRows : kBandRows, keys = p.few ? kFewKeys : band_keys(d->dtype, d->head_dim);
  p.row_tiles = (int)((rows + tile - 1) / tile);
  // a block's walk at most: the window of its rows and the sinks
  const int64_t near = d->window ? (int64_t)d->window + tile / group + 1 + d->sinks : room;
  const int64_t walk = std::min(room, near) / keys + 2;
  // keys are split until there are `want` blocks, `least` tiles each where an entry has them
  const int64_t blocks = std::max<int64_t>(1, pairs * p.row_tiles), want = p.few ? 2048 : 1024;
  const int least = p.few ? kFewLeast : kLeastTiles;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, want / blocks, (walk + least - 1) / least}));
  p.ml_at = p.splits > 1 ? round_up(pairs * p.splits * rows * d->head_dim * 4, 256) : 0;
  p.bytes = p.splits > 1 ? p.ml_at + round_up(pairs * p.splits * rows * 8, 256) : 0;
  return p;
}

bool paged_grid_fits(const recis_paged_attn_desc* d, const PagedPlan& p) {
  return round_up((int64_t)d->batch * d->kv_heads, (int64_t)kDies * d->kv_heads) * p.row_tiles * p.splits <= kMaxBlocks;
}

int paged_access(int dtype, const BandArgs& a, std::initializer_list<const void*> ptrs) {
  const int access = band_access(dtype, a.head_dim, ptrs, {a.qs, a.os, a.ks, a.vs});
  // a wave's slots stay within 32 bits of byte offset
  for (const long long* s : {a.ks, a.vs})
    if (access == 8 && (s[1] < 0 || s[1] >= (1 << 23) || s[0] < 0 || s[0] >= (1ll << 31))) return 1;
  return access;
}

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

int64_t recis_paged_attn_workspace_bytes(const recis_paged_attn_desc* desc) {
  if (check_paged(desc) != RECIS_OK) return -1;
  const PagedPlan p = paged_plan(desc);
  return paged_grid_fits(desc, p) ? p.bytes : -1;
}

recis_status recis_paged_attn_fwd(const recis_paged_attn_desc* d, const void* q, const void* k_cache,
                                  const void* v_cache, void* out, float* lse, void* workspace,
                                  int64_t workspace_bytes, hipStream_t s) {
  const recis_status st = check_paged(d);
  if (st != RECIS_OK) return st;
  if (d->batch == 0 || d->q_len == 0 || (d->q_offsets && d->q_rows == 0)) return RECIS_OK;
  const int size = dtype_size(d->dtype);
  const bool keys = d->pages > 0 && d->table_width > 0;
  if (!q || !out || !d->kv_lens || (keys && (!k_cache || !v_cache || !d->page_table)) || !aligned_to(q, size) ||
      !aligned_to(out, size) || !aligned_to(k_cache, size) || !aligned_to(v_cache, size) || !aligned_to(lse, 4))
    return RECIS_ERR_INVALID_ARG;
  const PagedPlan p = paged_plan(d);
  if (!paged_grid_fits(d, p)) return RECIS_ERR_UNSUPPORTED;
  if (p.bytes && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bytes)) return RECIS_ERR_INVALID_ARG;
  BandArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.out = out;
  a.lse = lse;
  a.offsets = d->q_offsets;
  a.lens = d->kv_lens;
  a.table = d->page_table;
  a.error = d->error;
  a.total_rows = d->q_rows;
  a.table_stride = d->table_stride;
  a.pages = d->pages;
  const int64_t q_axes[3] = {d->q_offsets ? 1 : d->batch, d->q_offsets ? d->q_rows : d->q_len, d->q_heads};
  const int64_t cache_axes[3] = {d->pages, d->page_size, d->kv_heads};
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = stride_of(d->q_strides[i], q_axes[i]);
    a.os[i] = stride_of(d->o_strides[i], q_axes[i]);
    a.ks[i] = stride_of(d->k_strides[i], cache_axes[i]);
    a.vs[i] = stride_of(d->v_strides[i], cache_axes[i]);
  }
  a.batch = d->batch;
  a.q_len = d->q_len;
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.group = d->q_heads / d->kv_heads;
  a.head_dim = d->head_dim;
  a.max_len = d->pages > 0 ? d->table_width * d->page_size : 0;
  a.rows = d->q_len * a.group;
  a.causal = d->causal != 0;
  a.window = window_of(d->window);
  a.sinks = std::min(d->sinks, 1 << 30);
  a.by_page = Quick(d->page_size);
  a.by_group = Quick(a.group);
  a.by_kv_heads = Quick(d->kv_heads);
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.ranked = !p.few && !d->window && d->batch > 1 && d->batch <= 64;
  place_pairs(&a, d->dtype);
  a.scale = d->scale;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ml_at);
  const int access = paged_access(d->dtype, a, {q, out, k_cache, v_cache});
  if (!p.few)
    launch_band_fwd(d->dtype, true, access, a, s);
  else if (d->dtype == RECIS_DTYPE_BF16)
    launch_few_dp<__bf16>(access, a, s);
  else
    launch_few_dp<float>(access, a, s);
  return launch_status();
}

}  // extern "C"
