// embed.hip -- token embedding with scaling, and its gradient by sorted tokens.
//
//   y[i]  = scale * W[t[i]]                      (0 where t[i] < 0)
//   dW[v] = scale * sum over i with t[i] = v of dY[i]
//
// The gradient's sum runs over the tokens in sorted order, equal tokens in
// the order of the call, so it does not depend on which block runs first: two
// calls on the same inputs return the same bits.
#include <algorithm>

#include "seq.h"

namespace recis {
namespace {

// ------------------------------------------------------------------ forward
// A thread carries one access of V elements of one row.  A block takes
// kFwdTile consecutive (row, access) places; per_row accesses a row, m =
// ceil(2^32 / per_row) replaces the division inside the block (exact: the
// dividend stays below per_row + kFwdTile).
constexpr int kFwdBatch = 4;
constexpr int kFwdTile = kThreads * kFwdBatch;

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void k_embed_fwd(const long long* __restrict__ tokens, long long n,
                                                        const T* __restrict__ w, long long rows, long long w_stride,
                                                        int per_row, unsigned m, float scale, T* __restrict__ out,
                                                        long long out_stride, unsigned* error) {
  const long long first = (long long)blockIdx.x * kFwdTile;
  const long long row0 = first / per_row;
  const unsigned rem = (unsigned)(first - row0 * per_row);
  long long row[kFwdBatch], tok[kFwdBatch];
  int col[kFwdBatch];
#pragma unroll
  for (int b = 0; b < kFwdBatch; ++b) {
    const unsigned f = rem + b * kThreads + threadIdx.x;
    const unsigned r = per_row == 1 ? f : __umulhi(f, m);
    row[b] = row0 + r;
    col[b] = (int)(f - r * per_row) * V;
    tok[b] = row[b] < n ? tokens[row[b]] : -1;
  }
  float v[kFwdBatch][V];
#pragma unroll
  for (int b = 0; b < kFwdBatch; ++b) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[b][i] = 0.f;
    if (tok[b] >= rows) {
      if (error) atomicOr(error, kErrKeyRange);
    } else if (tok[b] >= 0) {
      load_f32<T, V>(w + tok[b] * w_stride + col[b], v[b]);
    }
  }
#pragma unroll
  for (int b = 0; b < kFwdBatch; ++b) {
    if (row[b] >= n) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) v[b][i] *= scale;
    store_f32<T, V>(out + row[b] * out_stride + col[b], v[b]);
  }
}

template <typename T, int V>
void launch_fwd(const int64_t* tokens, int64_t n, const void* w, int64_t rows, int dim, int64_t w_stride, float scale,
                void* out, int64_t out_stride, uint32_t* error, hipStream_t s) {
  const int per_row = dim / V;
  const unsigned m = (unsigned)(((1ull << 32) + per_row - 1) / per_row);
  const int64_t blocks = (n * per_row + kFwdTile - 1) / kFwdTile;
  hipLaunchKernelGGL((k_embed_fwd<T, V>), dim3((unsigned)blocks), dim3(kThreads), 0, s,
                     reinterpret_cast<const long long*>(tokens), (long long)n, static_cast<const T*>(w),
                     (long long)rows, (long long)w_stride, per_row, m, scale, static_cast<T*>(out),
                     (long long)out_stride, error);
}

// ------------------------------------------------------------- sorted tokens
// Least-significant-digit radix sort of (token, place), stable.  Tokens that
// take no gradient (negative, or beyond the table) get the key `rows` and end
// up behind every row.  Per pass: a histogram of each tile's digits, the
// tiles' exclusive offsets, and a scatter that ranks the keys of a tile in
// order: the wave's lanes with the same digit find each other by ballots, the
// four waves of a block follow each other through per-wave counters in LDS.
constexpr int kDigitBits = 8;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kWaves = kThreads / 64;
constexpr int kSortPerThread = 16;
constexpr int kSortTile = kThreads * kSortPerThread;  // 4096

template <bool FIRST>
__device__ __forceinline__ unsigned sort_key(const long long* tokens, const unsigned* keys, long long i,
                                             unsigned rows, unsigned* error) {
  if constexpr (FIRST) {
    const long long t = tokens[i];
    if (t >= (long long)rows && error) atomicOr(error, kErrKeyRange);
    return t < 0 || t >= (long long)rows ? rows : (unsigned)t;
  } else {
    return keys[i];
  }
}

template <bool FIRST>
__global__ __launch_bounds__(kThreads) void k_sort_hist(const long long* __restrict__ tokens,
                                                        const unsigned* __restrict__ keys, long long n, unsigned rows,
                                                        int shift, unsigned* __restrict__ hist, unsigned* error) {
  __shared__ unsigned h[kDigits];
  h[threadIdx.x] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * kSortTile;
#pragma unroll
  for (int j = 0; j < kSortPerThread; ++j) {
    const long long i = base + j * kThreads + threadIdx.x;
    if (i < n) atomicAdd(&h[(sort_key<FIRST>(tokens, keys, i, rows, error) >> shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
  hist[(long long)blockIdx.x * kDigits + threadIdx.x] = h[threadIdx.x];
}

// One block a digit: its counts over the tiles become exclusive offsets, its
// total goes to totals[digit].
__global__ __launch_bounds__(kThreads) void k_sort_scan(unsigned* __restrict__ hist, int tiles,
                                                        unsigned* __restrict__ totals) {
  __shared__ unsigned part[kThreads];
  const int d = blockIdx.x;
  unsigned run = 0;
  for (int t0 = 0; t0 < tiles; t0 += kThreads) {
    const int t = t0 + (int)threadIdx.x;
    const unsigned c = t < tiles ? hist[(long long)t * kDigits + d] : 0u;
    part[threadIdx.x] = c;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
      const unsigned x = (int)threadIdx.x >= o ? part[threadIdx.x - o] : 0u;
      __syncthreads();
      part[threadIdx.x] += x;
      __syncthreads();
    }
    if (t < tiles) hist[(long long)t * kDigits + d] = run + part[threadIdx.x] - c;
    run += part[kThreads - 1];
    __syncthreads();
  }
  if (threadIdx.x == 0) totals[d] = run;
}

template <bool FIRST>
__global__ __launch_bounds__(kThreads) void k_sort_scatter(const long long* __restrict__ tokens,
                                                           const unsigned* __restrict__ keys,
                                                           const unsigned* __restrict__ places, long long n,
                                                           unsigned rows, int shift, const unsigned* __restrict__ hist,
                                                           const unsigned* __restrict__ totals,
                                                           unsigned* __restrict__ keys_out,
                                                           unsigned* __restrict__ places_out) {
  __shared__ unsigned cnt[kWaves][kDigits];
  __shared__ unsigned scan[kThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) cnt[w][threadIdx.x] = 0;
  // where each digit's keys begin
  const unsigned total = totals[threadIdx.x];
  scan[threadIdx.x] = total;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const unsigned x = (int)threadIdx.x >= o ? scan[threadIdx.x - o] : 0u;
    __syncthreads();
    scan[threadIdx.x] += x;
    __syncthreads();
  }
  const unsigned begin = scan[threadIdx.x] - total + hist[(long long)blockIdx.x * kDigits + threadIdx.x];
  __syncthreads();

  // each wave owns kSortTile / kWaves consecutive keys, 64 at a time
  const long long base = (long long)blockIdx.x * kSortTile + wave * (kSortTile / kWaves);
  unsigned key[kSortPerThread], place[kSortPerThread], rank[kSortPerThread];
#pragma unroll
  for (int j = 0; j < kSortPerThread; ++j) {
    const long long i = base + j * 64 + lane;
    const bool in = i < n;
    key[j] = in ? sort_key<FIRST>(tokens, keys, i, rows, nullptr) : 0u;
    place[j] = in ? (FIRST ? (unsigned)i : places[i]) : 0u;
  }
#pragma unroll
  for (int j = 0; j < kSortPerThread; ++j) {
    const bool in = base + j * 64 + lane < n;
    const unsigned d = (key[j] >> shift) & (kDigits - 1);
    unsigned long long same = __ballot(in);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
      const unsigned long long set = __ballot((d >> b) & 1u);
      same &= (d >> b) & 1u ? set : ~set;
    }
    rank[j] = 0;
    if (in) {
      const unsigned before = (unsigned)__popcll(same & ((1ull << lane) - 1));
      rank[j] = cnt[wave][d] + before;
      // the last lane of the digit leaves the counter for the next 64 keys
      // (a wave's LDS accesses are executed in order)
      if (before + 1 == (unsigned)__popcll(same)) cnt[wave][d] = rank[j] + 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __syncthreads();
  unsigned run = begin;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const unsigned c = cnt[w][threadIdx.x];
    cnt[w][threadIdx.x] = run;
    run += c;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortPerThread; ++j) {
    if (base + j * 64 + lane < n) {
      const unsigned to = cnt[wave][(key[j] >> shift) & (kDigits - 1)] + rank[j];
      keys_out[to] = key[j];
      places_out[to] = place[j];
    }
  }
}

// ------------------------------------------------------------------ the sums
// The sorted tokens and the table's rows are merged: a token is one unit of
// work (a gradient row read), the end of a row another (a gradient row
// written).  Every group of lanes takes `quantum` consecutive units of the
// merge, so neither a token that fills the batch nor a long stretch of
// untouched rows makes one group longer than another.  A row that spans
// groups of a block is joined in LDS, in order; one that spans blocks leaves a
// float32 part per block for k_embed_join.
struct SumArgs {
  const unsigned* tok;    // [n] sorted keys
  const unsigned* place;  // [n] their places in the call
  long long n, rows;
  const void* grad;
  long long grad_stride;
  void* out;
  long long out_stride;
  float scale;
  int dim, quantum;
  // per block: the row it starts in, whether that row has earlier tokens, and
  // the parts it leaves: `head` ends the first row, `tail` belongs to the row
  // the next block starts in
  int* first_row;
  int* began;
  float* head;
  float* tail;
};

// Tokens consumed when the merge has made d steps (a token t goes before the
// end of row r iff t <= r).
__device__ __forceinline__ long long merge_tokens(const unsigned* tok, long long n, long long rows, long long d) {
  long long lo = d > rows ? d - rows : 0, hi = d < n ? d : n;
  while (lo < hi) {
    const long long mid = (lo + hi) >> 1;
    if ((long long)tok[mid] <= d - 1 - mid)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// TG: gradient type, TW: type of the result, V elements an access, L lanes a
// row (a block covers L * V columns; blockIdx.y counts column tiles).
template <typename TG, typename TW, int V, int L>
__global__ __launch_bounds__(kThreads) void k_embed_sum(SumArgs a) {
  constexpr int kGroups = kThreads / L;
  constexpr int kBatch = 8;
  constexpr int C = L * V;
  __shared__ float head[kGroups][C];
  __shared__ float tail[kGroups][C];
  __shared__ int first[kGroups + 1];
  __shared__ int begun[kGroups];
  const int g = threadIdx.x / L, lane = threadIdx.x % L;
  const int col = blockIdx.y * C + lane * V;
  const bool live = col < a.dim;
  const TG* grad = static_cast<const TG*>(a.grad);
  TW* out = static_cast<TW*>(a.out);

  const long long total = a.n + a.rows;
  const long long d0 = std::min(total, ((long long)blockIdx.x * kGroups + g) * a.quantum);
  const long long d1 = std::min(total, d0 + a.quantum);
  const long long i0 = merge_tokens(a.tok, a.n, a.rows, d0), i1 = merge_tokens(a.tok, a.n, a.rows, d1);
  int row = (int)(d0 - i0);
  const int row_end = (int)(d1 - i1);
  const int row_first = row;
  const bool began = i0 > 0 && (long long)a.tok[i0 - 1] == row;

  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  auto finish_row = [&]() {
    if (live) {
      if (row == row_first && began) {
#pragma unroll
        for (int i = 0; i < V; ++i) head[g][lane * V + i] = acc[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a.scale;
        store_f32<TW, V>(out + (long long)row * a.out_stride + col, acc);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    ++row;
  };
  for (long long i = i0; i < i1; i += kBatch) {
    unsigned t[kBatch];
    float x[kBatch][V];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool in = i + b < i1;
      t[b] = in ? a.tok[i + b] : (unsigned)a.rows;
      if (live && t[b] < (unsigned)a.rows) {
        load_f32<TG, V>(grad + (long long)a.place[i + b] * a.grad_stride + col, x[b]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[b][k] = 0.f;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (t[b] < (unsigned)a.rows) {
        while (row < (int)t[b]) finish_row();
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += x[b][k];
      }
    }
  }
  while (row < row_end) finish_row();
#pragma unroll
  for (int i = 0; i < V; ++i) tail[g][lane * V + i] = acc[i];
  if (lane == 0) {
    first[g] = row_first;
    begun[g] = began;
    if (g == kGroups - 1) first[kGroups] = row_end;
  }
  __syncthreads();
  // join the rows that span groups: thread c carries column c through the
  // groups in order
  for (int c = threadIdx.x; c < C; c += kThreads) {
    const int column = blockIdx.y * C + c;
    if (column >= a.dim) break;
    float run = 0.f;
    bool open = begun[0];  // the row in `run` has tokens before this block
    for (int k = 0; k < kGroups; ++k) {
      const int r = first[k];
      if (first[k + 1] > r) {  // the group ends row r
        if (open) {
          a.head[(long long)blockIdx.x * a.dim + column] = run + head[k][c];
        } else if (begun[k]) {
          out[(long long)r * a.out_stride + column] = (TW)((run + head[k][c]) * a.scale);
        }
        run = tail[k][c];
        open = false;
      } else {
        run += tail[k][c];
      }
    }
    a.tail[(long long)blockIdx.x * a.dim + column] = run;
  }
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    a.first_row[blockIdx.x] = first[0];
    a.began[blockIdx.x] = begun[0];
    if (blockIdx.x == gridDim.x - 1) a.first_row[gridDim.x] = first[kGroups];
  }
}

// Rows that span blocks of k_embed_sum: the block that ends the row adds the
// tails of the blocks before it that the row runs through, in order.
template <typename TW>
__global__ __launch_bounds__(kThreads) void k_embed_join(SumArgs a) {
  const int b = blockIdx.x;
  const int r = a.first_row[b];
  if (!a.began[b] || a.first_row[b + 1] == r) return;
  int k = b - 1;  // the first block with tokens of the row
  while (k > 0 && a.first_row[k] == r && a.began[k]) --k;
  for (int c = threadIdx.x; c < a.dim; c += kThreads) {
    float sum = 0.f;
    for (int j = k; j < b; ++j) sum += a.tail[(long long)j * a.dim + c];
    sum += a.head[(long long)b * a.dim + c];
    static_cast<TW*>(a.out)[(long long)r * a.out_stride + c] = (TW)(sum * a.scale);
  }
}

// ----------------------------------------------------------- sizes, launches
struct BwdPlan {
  int bits, passes, tiles;
  int v, lanes, groups, quantum, col_tiles;
  int64_t blocks;
  // byte offsets in the workspace
  int64_t keys[2], places[2], hist, totals, first_row, began, head, tail, bytes;
};

BwdPlan bwd_plan(int64_t n, int64_t rows, int dim, int v) {
  BwdPlan p;
  p.bits = 1;
  while ((rows >> p.bits) != 0) ++p.bits;  // keys 0 .. rows
  p.passes = (p.bits + kDigitBits - 1) / kDigitBits;
  p.tiles = (int)((n + kSortTile - 1) / kSortTile);
  p.v = v;
  p.lanes = 8;
  while (p.lanes < 64 && p.lanes * v < dim) p.lanes *= 2;
  p.groups = kThreads / p.lanes;
  p.col_tiles = (dim + p.lanes * v - 1) / (p.lanes * v);
  const int64_t units = n + rows;
  p.quantum = (int)std::min<int64_t>(128, std::max<int64_t>(8, units / ((int64_t)p.groups * 1024)));
  p.blocks = (units + (int64_t)p.groups * p.quantum - 1) / ((int64_t)p.groups * p.quantum);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  for (int k = 0; k < 2; ++k) {
    p.keys[k] = take(4 * n);
    p.places[k] = take(4 * n);
  }
  p.hist = take(4ll * kDigits * p.tiles);
  p.totals = take(4ll * kDigits);
  p.first_row = take(4 * (p.blocks + 1));
  p.began = take(4 * p.blocks);
  p.head = take(4 * p.blocks * dim);
  p.tail = take(4 * p.blocks * dim);
  p.bytes = at;
  return p;
}

template <typename TG, typename TW, int V>
void launch_sum_v(const BwdPlan& p, const SumArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)p.blocks, (unsigned)p.col_tiles), block(kThreads);
  switch (p.lanes) {
    case 8: hipLaunchKernelGGL((k_embed_sum<TG, TW, V, 8>), grid, block, 0, s, a); break;
    case 16: hipLaunchKernelGGL((k_embed_sum<TG, TW, V, 16>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((k_embed_sum<TG, TW, V, 32>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_embed_sum<TG, TW, V, 64>), grid, block, 0, s, a); break;
  }
}

template <typename TG, typename TW>
void launch_sum(const BwdPlan& p, const SumArgs& a, hipStream_t s) {
  if (p.v == 4)
    launch_sum_v<TG, TW, 4>(p, a, s);
  else if (p.v == 2)
    launch_sum_v<TG, TW, 2>(p, a, s);
  else
    launch_sum_v<TG, TW, 1>(p, a, s);
  hipLaunchKernelGGL((k_embed_join<TW>), dim3((unsigned)p.blocks), dim3(kThreads), 0, s, a);
}

constexpr int64_t kMaxTokens = (1ll << 31) - kSortTile;
constexpr int64_t kMaxVocab = 1ll << 30;
constexpr int kMaxDim = 1 << 16;

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

recis_status recis_embed_fwd(const int64_t* tokens, int64_t n, const void* weight, int32_t dtype, int64_t rows,
                             int32_t dim, int64_t weight_stride, float scale, void* out, int64_t out_stride,
                             uint32_t* error, hipStream_t s) {
  if (!dtype_known(dtype) || n < 0 || rows < 1 || dim < 1 || weight_stride < dim || out_stride < dim)
    return RECIS_ERR_INVALID_ARG;
  if (n > kMaxTokens || rows > kMaxVocab || dim > kMaxDim) return RECIS_ERR_UNSUPPORTED;
  if (n == 0) return RECIS_OK;
  const int size = dtype_size(dtype);
  if (!tokens || !weight || !out || !aligned_to(tokens, 8) || !aligned_to(weight, size) || !aligned_to(out, size) ||
      !aligned_to(error, 4))
    return RECIS_ERR_INVALID_ARG;
  const int v = access_width(size, dim, {weight, out}, {weight_stride, out_stride});
  if ((n * (dim / v) + kFwdTile - 1) / kFwdTile > (1ll << 31) - 1) return RECIS_ERR_UNSUPPORTED;
  auto go = [&](auto launch) {
    launch(tokens, n, weight, rows, dim, weight_stride, scale, out, out_stride, error, s);
  };
  if (dtype == RECIS_DTYPE_BF16) {
    v == 8 ? go(launch_fwd<__bf16, 8>) : v == 4 ? go(launch_fwd<__bf16, 4>) : v == 2 ? go(launch_fwd<__bf16, 2>)
                                                                                      : go(launch_fwd<__bf16, 1>);
  } else {
    v == 4 ? go(launch_fwd<float, 4>) : v == 2 ? go(launch_fwd<float, 2>) : go(launch_fwd<float, 1>);
  }
  return launch_status();
}

int64_t recis_embed_bwd_workspace_bytes(int64_t n, int64_t rows, int32_t dim) {
  if (n < 0 || rows < 1 || dim < 1 || n > kMaxTokens || rows > kMaxVocab || dim > kMaxDim) return -1;
  int64_t most = 0;
  for (int v : {1, 2, 4}) most = std::max(most, bwd_plan(n, rows, dim, v).bytes);
  return most;
}

recis_status recis_embed_bwd(const int64_t* tokens, int64_t n, const void* grad_out, int32_t grad_dtype,
                             int64_t grad_stride, int64_t rows, int32_t dim, float scale, void* grad_weight,
                             int32_t weight_dtype, int64_t weight_stride, void* workspace, int64_t workspace_bytes,
                             uint32_t* error, hipStream_t s) {
  if (!dtype_known(grad_dtype) || !dtype_known(weight_dtype) || n < 0 || rows < 1 || dim < 1 || weight_stride < dim ||
      grad_stride < dim || !grad_weight)
    return RECIS_ERR_INVALID_ARG;
  if (n > kMaxTokens || rows > kMaxVocab || dim > kMaxDim) return RECIS_ERR_UNSUPPORTED;
  const int gs = dtype_size(grad_dtype), ws = dtype_size(weight_dtype);
  if ((n > 0 && (!tokens || !grad_out)) || !aligned_to(tokens, 8) || !aligned_to(grad_out, gs) ||
      !aligned_to(grad_weight, ws) || !aligned_to(error, 4))
    return RECIS_ERR_INVALID_ARG;
  // one access width for both sides: the gradients' and the result's rows
  const int v = std::min(4, std::min(access_width(gs, dim, {grad_out}, {grad_stride}),
                                     access_width(ws, dim, {grad_weight}, {weight_stride})));
  const BwdPlan p = bwd_plan(n, rows, dim, v);
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bytes) return RECIS_ERR_INVALID_ARG;
  if (p.blocks > (1ll << 31) - 1) return RECIS_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(workspace);
  unsigned* hist = reinterpret_cast<unsigned*>(w + p.hist);
  unsigned* totals = reinterpret_cast<unsigned*>(w + p.totals);
  const long long* tok = reinterpret_cast<const long long*>(tokens);
  int cur = 0;
  if (n > 0) {
    for (int pass = 0; pass < p.passes; ++pass) {
      const unsigned* kin = reinterpret_cast<const unsigned*>(w + p.keys[cur]);
      const unsigned* pin = reinterpret_cast<const unsigned*>(w + p.places[cur]);
      unsigned* kout = reinterpret_cast<unsigned*>(w + p.keys[cur ^ 1]);
      unsigned* pout = reinterpret_cast<unsigned*>(w + p.places[cur ^ 1]);
      const int shift = pass * kDigitBits;
      const dim3 grid((unsigned)p.tiles), block(kThreads);
      if (pass == 0)
        hipLaunchKernelGGL((k_sort_hist<true>), grid, block, 0, s, tok, kin, (long long)n, (unsigned)rows, shift, hist,
                           error);
      else
        hipLaunchKernelGGL((k_sort_hist<false>), grid, block, 0, s, tok, kin, (long long)n, (unsigned)rows, shift,
                           hist, error);
      hipLaunchKernelGGL(k_sort_scan, dim3(kDigits), block, 0, s, hist, p.tiles, totals);
      if (pass == 0)
        hipLaunchKernelGGL((k_sort_scatter<true>), grid, block, 0, s, tok, kin, pin, (long long)n, (unsigned)rows,
                           shift, hist, totals, kout, pout);
      else
        hipLaunchKernelGGL((k_sort_scatter<false>), grid, block, 0, s, tok, kin, pin, (long long)n, (unsigned)rows,
                           shift, hist, totals, kout, pout);
      cur ^= 1;
    }
  }
  SumArgs a;
  a.tok = reinterpret_cast<const unsigned*>(w + p.keys[cur]);
  a.place = reinterpret_cast<const unsigned*>(w + p.places[cur]);
  a.n = n;
  a.rows = rows;
  a.grad = grad_out;
  a.grad_stride = grad_stride;
  a.out = grad_weight;
  a.out_stride = weight_stride;
  a.scale = scale;
  a.dim = dim;
  a.quantum = p.quantum;
  a.first_row = reinterpret_cast<int*>(w + p.first_row);
  a.began = reinterpret_cast<int*>(w + p.began);
  a.head = reinterpret_cast<float*>(w + p.head);
  a.tail = reinterpret_cast<float*>(w + p.tail);
  const bool gb = grad_dtype == RECIS_DTYPE_BF16, wb = weight_dtype == RECIS_DTYPE_BF16;
  if (gb && wb)
    launch_sum<__bf16, __bf16>(p, a, s);
  else if (gb)
    launch_sum<__bf16, float>(p, a, s);
  else if (wb)
    launch_sum<float, __bf16>(p, a, s);
  else
    launch_sum<float, float>(p, a, s);
  return launch_status();
}

}  // extern "C"
