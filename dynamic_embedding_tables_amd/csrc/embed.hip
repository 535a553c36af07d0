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
// Bound by the stores: 2.05M tokens on 100000 rows of 128 bfloat16 write 524 MB
// and read 42 in 79 us, 7.2 TB/s (a fill of 2 GiB reaches 6.9; stored through
// the caches 143 us).  32 tokens: 2 us, of 8 that the call takes on the host.
//
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
                                                        long long out_stride, int stream, unsigned* error) {
  const long long first = (long long)block_id() * kFwdTile;
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
    const float by = tok[b] >= 0 && tok[b] < rows ? scale : 0.f;  // (a scale may be infinite)
#pragma unroll
    for (int i = 0; i < V; ++i) v[b][i] *= by;
    store_or_stream<T, V>(stream, out + row[b] * out_stride + col[b], v[b]);
  }
}

template <typename T, int V>
void launch_fwd(const int64_t* tokens, int64_t n, const void* w, int64_t rows, int dim, int64_t w_stride, float scale,
                void* out, int64_t out_stride, uint32_t* error, hipStream_t s) {
  const int per_row = dim / V;
  const unsigned m = (unsigned)(((1ull << 32) + per_row - 1) / per_row);
  const int64_t blocks = (n * per_row + kFwdTile - 1) / kFwdTile;
  hipLaunchKernelGGL((k_embed_fwd<T, V>), grid_of(blocks), dim3(kThreads), 0, s,
                     reinterpret_cast<const long long*>(tokens), (long long)n, static_cast<const T*>(w),
                     (long long)rows, (long long)w_stride, per_row, m, scale, static_cast<T*>(out),
                     (long long)out_stride, (int)(n * dim * (int64_t)sizeof(T) > kStreamBytes), error);
}

// ------------------------------------------------------------- sorted tokens
// 2.05M tokens on 1M rows (two passes of 10 bits): 10 us to count, 8 to scan and
// 16 to 24 to scatter a pass, the scattered 8-byte words bounding it.  Digits of
// 8 bits took three passes, 92 us against 82; separate words for key and place
// 38 us a scatter.  4096 keys a block above 2^18 tokens, 1024 below, where more
// blocks count for more.
//
// Least-significant-digit radix sort of (token, place), stable.  Tokens that
// take no gradient (negative, or beyond the table) get the key `rows` and end
// up behind every row.  Digits of up to 11 bits: one pass for tables of 2047
// rows, two up to 4M rows.  Per pass: a histogram of each tile's digits, where
// each tile's share of a digit begins, and a scatter that ranks the keys of a
// tile in order: the wave's lanes with the same digit find each other by
// ballots, the waves of a block follow each other through counters in LDS.
constexpr int kMaxDigitBits = 11;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kWaves = kThreads / 64;

// A key and its place travel as one 8-byte word: half the scattered writes.
struct __align__(8) Keyed {
  unsigned key, place;
};

template <bool FIRST>
__device__ __forceinline__ Keyed sort_key(const long long* tokens, const Keyed* in, long long i, unsigned rows,
                                          unsigned* error) {
  if constexpr (FIRST) {
    const long long t = tokens[i];
    if (t >= (long long)rows && error) atomicOr(error, kErrKeyRange);
    return Keyed{t < 0 || t >= (long long)rows ? rows : (unsigned)t, (unsigned)i};
  } else {
    return in[i];
  }
}

struct SortArgs {
  const long long* tokens;
  const Keyed* in;
  Keyed* out;
  long long n;
  unsigned rows;
  int shift, digits, tiles;
  unsigned* hist;    // [tiles][digits] counts, exclusive offsets after k_sort_scan
  unsigned* totals;  // [digits], written by k_sort_scan
  unsigned* error;
};

// PER keys a thread, PER * kThreads a tile.
template <bool FIRST, int PER>
__global__ __launch_bounds__(kThreads) void k_sort_hist(SortArgs a) {
  __shared__ unsigned h[kMaxDigits];
  for (int d = threadIdx.x; d < a.digits; d += kThreads) h[d] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * PER * kThreads;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const long long i = base + j * kThreads + threadIdx.x;
    if (i >= a.n) continue;
    const unsigned key = sort_key<FIRST>(a.tokens, a.in, i, a.rows, a.error).key;
    atomicAdd(&h[(key >> a.shift) & (a.digits - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.digits; d += kThreads) a.hist[(long long)blockIdx.x * a.digits + d] = h[d];
}

// 16 digits a block, the tiles in 16 consecutive ranges: counts become
// exclusive offsets over the tiles, a digit's total goes to totals[digit].
constexpr int kScanDigits = 16, kScanParts = kThreads / kScanDigits;
__global__ __launch_bounds__(kThreads) void k_sort_scan(SortArgs a) {
  __shared__ unsigned part[kScanParts][kScanDigits];
  const int c = threadIdx.x % kScanDigits, p = threadIdx.x / kScanDigits;
  const int d = blockIdx.x * kScanDigits + c;
  const int per = (a.tiles + kScanParts - 1) / kScanParts;
  const int t0 = p * per, t1 = std::min(a.tiles, t0 + per);
  unsigned sum = 0;
  if (d < a.digits)
#pragma unroll 8
    for (int t = t0; t < t1; ++t) sum += a.hist[(long long)t * a.digits + d];
  part[p][c] = sum;
  __syncthreads();
  if (d >= a.digits) return;
  unsigned run = 0;
  for (int k = 0; k < p; ++k) run += part[k][c];
  if (p == kScanParts - 1) a.totals[d] = run + sum;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) {
    const unsigned x = a.hist[(long long)t * a.digits + d];
    a.hist[(long long)t * a.digits + d] = run;
    run += x;
  }
}

// SCANNED: hist and totals are k_sort_scan's; otherwise hist holds the counts
// of a few tiles and every block adds them up itself (a launch less).
template <bool FIRST, int PER, bool SCANNED>
__global__ __launch_bounds__(kThreads) void k_sort_scatter(SortArgs a) {
  __shared__ unsigned cnt[kWaves][kMaxDigits];
  __shared__ unsigned wave_sum[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // each wave owns PER * 64 consecutive keys, 64 at a time
  const long long base = (long long)blockIdx.x * PER * kThreads + wave * (PER * 64);
  Keyed key[PER];
  unsigned rank[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const long long i = base + j * 64 + lane;
    key[j] = i < a.n ? sort_key<FIRST>(a.tokens, a.in, i, a.rows, nullptr) : Keyed{0u, 0u};
  }
  // where the tile's share of each digit begins: thread t has digits
  // t * per_thread and the next ones
  const int per_thread = (a.digits + kThreads - 1) / kThreads;
  unsigned begin[kMaxDigits / kThreads];
  unsigned mine = 0;
#pragma unroll
  for (int k = 0; k < kMaxDigits / kThreads; ++k) {
    const int d = threadIdx.x * per_thread + k;
    unsigned before = 0, total = 0;
    if (k < per_thread && d < a.digits) {
      if constexpr (SCANNED) {
        total = a.totals[d];
        before = a.hist[(long long)blockIdx.x * a.digits + d];
      } else {
        for (int t0 = 0; t0 < a.tiles; t0 += 16) {  // 16 loads under way
          unsigned x[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) x[t] = t0 + t < a.tiles ? a.hist[(long long)(t0 + t) * a.digits + d] : 0u;
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            total += x[t];
            if (t0 + t < (int)blockIdx.x) before += x[t];
          }
        }
      }
      for (int w = 0; w < kWaves; ++w) cnt[w][d] = 0;
    }
    begin[k] = mine + before;
    mine += total;
  }
  unsigned incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned x = __shfl_up(incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  unsigned first = incl - mine;
  for (int w = 0; w < wave; ++w) first += wave_sum[w];

#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool in = base + j * 64 + lane < a.n;
    const unsigned d = (key[j].key >> a.shift) & (a.digits - 1);
    unsigned long long same = __ballot(in);
    for (int b = 1; b < a.digits; b <<= 1) {
      const unsigned long long set = __ballot((d & b) != 0);
      same &= d & b ? set : ~set;
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
#pragma unroll
  for (int k = 0; k < kMaxDigits / kThreads; ++k) {
    const int d = threadIdx.x * per_thread + k;
    if (k >= per_thread || d >= a.digits) continue;
    unsigned run = first + begin[k];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const unsigned c = cnt[w][d];
      cnt[w][d] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (base + j * 64 + lane < a.n) {
      const unsigned to = cnt[wave][(key[j].key >> a.shift) & (a.digits - 1)] + rank[j];
      a.out[to] = key[j];
    }
  }
}

// ------------------------------------------------------------------ the sums
// Bound by memory where there is much: 2.05M gradient rows of 128 bfloat16 and
// 1M rows of result, 780 MB in 175 us, 4.5 TB/s (a large copy: 4.8).  By its
// chain of dependent reads where there is little: 20011 tokens on 50021 rows of
// 64 float32, 18 MB in 12 us (8 units a group; 4: 14 us, 16: 15 us).
//
// The sorted tokens and the table's rows are merged: a token is one unit of
// work (a gradient row read), the end of a row another (a gradient row
// written).  Every group of lanes takes `quantum` consecutive units of the
// merge, so neither a token that fills the batch nor a long stretch of
// untouched rows makes one group longer than another.  A row that spans
// groups of a block is joined in LDS, in order; one that spans blocks leaves a
// float32 part per block for k_embed_join.
constexpr int kMaxUnits = 2048;  // units a block

struct SumArgs {
  const Keyed* tok;  // [n] sorted tokens with their places in the call
  long long n, rows;
  const void* grad;
  long long grad_stride;
  void* out;
  long long out_stride;
  float scale;
  int dim, quantum, stream;
  int lane_bits;  // 2^lane_bits lanes a row; blockIdx.y counts tiles of 2^lane_bits * V columns
  // per block: the row it starts in, whether that row has earlier tokens, and
  // the parts it leaves: `head` ends the first row, `tail` belongs to the row
  // the next block starts in
  int* first_row;
  int* began;
  float* head;
  float* tail;
  // few tokens: unsorted, with the rows of a block
  const long long* raw;
  int block_rows;
  unsigned* error;
};

// Tokens consumed when the merge has made d steps (a token t goes before the
// end of row r iff t <= r): 64 probes a round.
__device__ __forceinline__ long long merge_tokens(const SumArgs& a, long long d, int lane) {
  long long lo = d > a.rows ? d - a.rows : 0, hi = d < a.n ? d : a.n;
  while (lo < hi) {
    const long long step = (hi - lo + 63) >> 6;
    const long long at = lo + (lane + 1) * step - 1;
    const bool before = at < hi && (long long)a.tok[at].key <= d - 1 - at;
    lo += __popcll(__ballot(before)) * step;
    hi = std::min(hi, lo + step - 1);
  }
  return lo;
}

// Few tokens are not sorted beforehand: every block looks all of them through
// for those of its own `block_rows` rows, and puts them in order itself (one
// launch in place of six; 32 tokens on 4096 rows: 10 us against 22).
constexpr int kFewTokens = 1024, kFewPer = kFewTokens / kThreads;

// The block's tokens in order, in `slice`; `scratch` has room for kFewTokens.
// Returns their number.
__device__ __forceinline__ int pick_tokens(const long long* tokens, int n, long long row0, int rows, long long all_rows,
                                           unsigned* error, Keyed* slice, Keyed* scratch, int* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Keyed mine[kFewPer];
  int count = 0;
#pragma unroll
  for (int k = 0; k < kFewPer; ++k) {
    const int i = threadIdx.x * kFewPer + k;
    const long long t = i < n ? tokens[i] : -1;
    if (t >= all_rows && error && blockIdx.x == 0) atomicOr(error, kErrKeyRange);
    if (t >= row0 && t < row0 + rows) mine[count++] = Keyed{(unsigned)t, (unsigned)i};
  }
  int incl = count;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int at = incl - count, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at += wave_sum[w];
    total += wave_sum[w];
  }
#pragma unroll
  for (int k = 0; k < kFewPer; ++k)
    if (k < count) scratch[at + k] = mine[k];
  __syncthreads();
  // a token's place in order: the smaller ones, and the equal ones before it
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const unsigned key = scratch[i].key;
    int before = 0;
    for (int k = 0; k < total; ++k) before += scratch[k].key < key || (scratch[k].key == key && k < i);
    slice[before] = scratch[i];
  }
  return total;
}

// TG: gradient type, TW: type of the result, V elements an access.
template <typename TG, typename TW, int V, bool FEW>
__global__ __launch_bounds__(kThreads) void k_embed_sum(SumArgs a) {
  constexpr int kBatch = 8;
  __shared__ Keyed slice[kMaxUnits];   // the block's tokens; later the groups' tails
  __shared__ float head[kThreads * V];  // [groups][columns]
  __shared__ long long ends[2];
  __shared__ int before_first;  // the token before the slice, -1 without one
  __shared__ unsigned short starts[kThreads + 1];  // tokens before each group
  static_assert(sizeof(slice) >= sizeof(head), "tails fit the slice");
  const int lanes = 1 << a.lane_bits, groups = kThreads >> a.lane_bits, C = lanes * V;
  const int g = threadIdx.x >> a.lane_bits, lane = threadIdx.x & (lanes - 1);
  const int col = blockIdx.y * C + lane * V;
  const bool live = col < a.dim;
  const TG* grad = static_cast<const TG*>(a.grad);
  TW* out = static_cast<TW*>(a.out);

  // the block's part of the merge: `count` tokens from `first` on, rows from
  // block_row on, `left` units in all, `quantum` a group
  int count, block_row, left, quantum = a.quantum;
  if constexpr (FEW) {
    __shared__ int wave_sum[kWaves];
    block_row = (int)blockIdx.x * a.block_rows;
    const int rows = (int)std::min<long long>(a.block_rows, a.rows - block_row);
    count = pick_tokens(a.raw, (int)a.n, block_row, rows, a.rows, a.error, slice, slice + kFewTokens, wave_sum);
    left = count + rows;
    quantum = (left + groups - 1) / groups;
    if (threadIdx.x == 0) before_first = -1;
  } else {
    const long long total = a.n + a.rows;
    const int units = groups * quantum;
    const long long d0 = (long long)blockIdx.x * units;
    const int wave = threadIdx.x >> 6;
    if (wave < 2) {
      const long long i = merge_tokens(a, std::min(total, d0 + wave * units), threadIdx.x & 63);
      if ((threadIdx.x & 63) == 0) ends[wave] = i;
    }
    __syncthreads();
    const long long first = ends[0];
    count = (int)(ends[1] - first);
    block_row = (int)(d0 - first);
    left = (int)std::min<long long>(total - d0, units);
    for (int i = threadIdx.x; i < count; i += kThreads) slice[i] = a.tok[first + i];
    if (threadIdx.x == kThreads - 1) before_first = first > 0 ? (int)a.tok[first - 1].key : -1;
  }
  __syncthreads();
  // the same search inside the block
  if (threadIdx.x == 0) starts[groups] = (unsigned short)count;
  if (threadIdx.x < groups) {
    const int d = std::min(left, (int)threadIdx.x * quantum);
    int lo = std::max(0, d - (left - count)), hi = std::min(d, count);
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((int)slice[mid].key - block_row <= d - 1 - mid)
        lo = mid + 1;
      else
        hi = mid;
    }
    starts[threadIdx.x] = (unsigned short)lo;
  }
  __syncthreads();
  auto row_of = [&](int k) {  // the row group k starts in
    return block_row + std::min(left, k * quantum) - (int)starts[k];
  };
  auto has_tokens = [&](int k) {  // whether that row has tokens before the group
    return (starts[k] > 0 ? (int)slice[starts[k] - 1].key : before_first) == row_of(k);
  };
  const int i0 = starts[g], i1 = starts[g + 1];
  const int row_first = row_of(g), row_end = row_of(g + 1);
  const bool began = has_tokens(g);
  int row = row_first;

  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  auto finish_row = [&]() {
    if (live) {
      if (row == row_first && began) {
#pragma unroll
        for (int i = 0; i < V; ++i) head[g * C + lane * V + i] = acc[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a.scale;
        store_or_stream<TW, V>(a.stream, out + (long long)row * a.out_stride + col, acc);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    ++row;
  };
  // rows up to `to`: the first may have tokens (`open`), the others have none
  // and are zero whatever the scale
  bool open = began;
  auto advance = [&](int to) {
    if (row >= to) return;
    if (open) finish_row();
    const float none[V] = {};
    for (; row < to; ++row)
      if (live) store_or_stream<TW, V>(a.stream, out + (long long)row * a.out_stride + col, none);
  };
  // the next batch's gradient rows are on their way while one is added up
  Vec<TG, V> x[kBatch], ahead[kBatch];
  auto fetch = [&](int i, Vec<TG, V>(&to)[kBatch]) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (live && i + b < i1 && slice[i + b].key < (unsigned)a.rows)
        to[b] = *reinterpret_cast<const Vec<TG, V>*>(grad + (long long)slice[i + b].place * a.grad_stride + col);
    }
  };
  fetch(i0, x);
  for (int i = i0; i < i1; i += kBatch) {
    fetch(i + kBatch, ahead);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const unsigned t = i + b < i1 ? slice[i + b].key : (unsigned)a.rows;
      if (t < (unsigned)a.rows) {
        advance((int)t);
        open = true;
        if (live) {
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] += (float)x[b].e[k];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) x[b] = ahead[b];
  }
  advance(row_end);
  const int rows_of = threadIdx.x < groups ? row_of(threadIdx.x) : 0;
  const int begun_of = threadIdx.x < groups ? has_tokens(threadIdx.x) : 0;
  const int last_row = row_of(groups);
  __shared__ int group_row[kThreads + 1];
  __shared__ unsigned char group_began[kThreads];
  if (threadIdx.x < groups) {
    group_row[threadIdx.x] = rows_of;
    group_began[threadIdx.x] = begun_of;
  }
  if (threadIdx.x == 0) group_row[groups] = last_row;
  __syncthreads();  // the slice is free from here on
  float* tail = reinterpret_cast<float*>(slice);
#pragma unroll
  for (int i = 0; i < V; ++i) tail[g * C + lane * V + i] = acc[i];
  __syncthreads();
  // join the rows that span groups, one (group that ends such a row, column) a
  // thread: the tails of the groups the row runs through, in order, and the
  // group's head.  Past the last group the same gives the block's tail.
  for (int item = threadIdx.x; item < C * (groups + (FEW ? 0 : 1)); item += kThreads) {
    const int k = item / C, c = item % C, column = blockIdx.y * C + c;
    if (column >= a.dim) continue;
    const int r = group_row[k];
    if (k < groups && (group_row[k + 1] == r || !group_began[k])) continue;
    int j = k;
    while (j > 0 && (j == k || group_row[j] == r)) --j;
    float sum = 0.f;
    for (int g0 = j; g0 < k; ++g0) sum += tail[g0 * C + c];
    if (k == groups) {
      a.tail[(long long)blockIdx.x * a.dim + column] = sum;
      continue;
    }
    sum += head[k * C + c];
    // does the row have tokens before this block?
    if (j == 0 && group_row[0] == r && group_began[0])
      a.head[(long long)blockIdx.x * a.dim + column] = sum;
    else
      out[(long long)r * a.out_stride + column] = (TW)(sum * a.scale);
  }
  if (!FEW && threadIdx.x == 0 && blockIdx.y == 0) {
    a.first_row[blockIdx.x] = group_row[0];
    a.began[blockIdx.x] = group_began[0];
    if (blockIdx.x == gridDim.x - 1) a.first_row[gridDim.x] = last_row;
  }
}

// Rows that span blocks of k_embed_sum: the block that ends the row adds the
// tails of the blocks before it that the row runs through.  The tails are
// taken in kJoinParts consecutive ranges at a time, joined in order.
constexpr int kJoinLanes = 32, kJoinParts = kThreads / kJoinLanes;
template <typename TW, int V>
__global__ __launch_bounds__(kThreads) void k_embed_join(SumArgs a) {
  __shared__ float part[kJoinParts][kJoinLanes * V];
  const int b = blockIdx.x;
  const int r = a.first_row[b], next = a.first_row[b + 1], began = a.began[b];
  if (!began || next == r) return;
  // the first block with tokens of the row: every block after it starts in
  // the row, which has begun by then (64 blocks a step)
  int k = b;
  const int lane = threadIdx.x & 63;
  for (;;) {
    const int at = k - lane;
    const bool inside = at > 0 && a.first_row[at] == r && a.began[at];
    const unsigned long long out_of_it = ~__ballot(inside);
    const int steps = out_of_it ? __ffsll(out_of_it) - 1 : 64;
    k -= steps;
    if (steps < 64) break;
  }
  const int l = threadIdx.x % kJoinLanes, p = threadIdx.x / kJoinLanes;
  const int per = (b - k + kJoinParts - 1) / kJoinParts;
  const int j0 = std::min(b, k + p * per), j1 = std::min(b, j0 + per);
  for (int c0 = 0; c0 < a.dim; c0 += kJoinLanes * V) {
    const int c = c0 + l * V;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    if (c < a.dim) {
#pragma unroll 8
      for (int j = j0; j < j1; ++j) {
        float x[V];
        load_f32<float, V>(a.tail + (long long)j * a.dim + c, x);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += x[i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[p][l * V + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinLanes * V && c0 + i < a.dim; i += kThreads) {
      float x = part[0][i];
#pragma unroll
      for (int q = 1; q < kJoinParts; ++q) x += part[q][i];
      x += a.head[(long long)b * a.dim + c0 + i];
      static_cast<TW*>(a.out)[(long long)r * a.out_stride + c0 + i] = (TW)(x * a.scale);
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------- sizes, launches
struct BwdPlan {
  int passes, digit_bits, per, tiles;
  bool scanned, few;
  int block_rows = 0;
  int lane_bits, quantum, col_tiles;
  int64_t blocks;
  // byte offsets in the workspace
  int64_t sorted[2], hist, totals, first_row, began, head, tail, bytes;
};

BwdPlan bwd_plan(int64_t n, int64_t rows, int dim, int v) {
  BwdPlan p;
  int bits = 1;
  while ((rows >> bits) != 0) ++bits;  // keys 0 .. rows
  p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  const int digits = 1 << p.digit_bits;
  p.per = n <= (1 << 18) ? 4 : 16;
  p.tiles = (int)((n + p.per * kThreads - 1) / (p.per * kThreads));
  p.scanned = p.tiles > 64;
  p.lane_bits = 0;
  while (p.lane_bits < 6 && (v << p.lane_bits) < dim) ++p.lane_bits;
  const int groups = kThreads >> p.lane_bits, columns = v << p.lane_bits;
  p.col_tiles = (dim + columns - 1) / columns;
  const int64_t units = n + rows;
  const int64_t most = std::min(128, kMaxUnits / groups);
  p.quantum = (int)std::min<int64_t>(most, std::max<int64_t>(8, units / ((int64_t)groups * 1024)));
  // (512 units a block or more in large calls: 2^23 blocks at most)
  p.blocks = (units + (int64_t)groups * p.quantum - 1) / ((int64_t)groups * p.quantum);
  p.few = n <= kFewTokens;
  if (p.few) {
    p.block_rows = (int)std::max<int64_t>(1, (rows + 1023) / 1024);
    p.blocks = (rows + p.block_rows - 1) / p.block_rows;
  }
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  for (int k = 0; k < 2; ++k) p.sorted[k] = take(8 * n);
  p.hist = take(4ll * digits * p.tiles);
  p.totals = take(4ll * digits);
  p.first_row = take(4 * (p.blocks + 1));
  p.began = take(4 * p.blocks);
  p.head = take(4 * p.blocks * dim);
  p.tail = take(4 * p.blocks * dim);
  p.bytes = at;
  return p;
}

template <bool FIRST, int PER>
void launch_sort(const BwdPlan& p, const SortArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)p.tiles), block(kThreads);
  hipLaunchKernelGGL((k_sort_hist<FIRST, PER>), grid, block, 0, s, a);
  if (p.scanned || PER > 4) {  // (tiles of 4096 keys are more than 64: bwd_plan)
    hipLaunchKernelGGL(k_sort_scan, dim3((a.digits + kScanDigits - 1) / kScanDigits), block, 0, s, a);
    hipLaunchKernelGGL((k_sort_scatter<FIRST, PER, true>), grid, block, 0, s, a);
  } else if constexpr (PER == 4) {
    hipLaunchKernelGGL((k_sort_scatter<FIRST, PER, false>), grid, block, 0, s, a);
  }
}

template <typename TG, typename TW, bool FEW>
void launch_sum_as(const BwdPlan& p, int v, const SumArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)p.blocks, (unsigned)p.col_tiles), block(kThreads);
  switch (v) {
    case 8:
      if constexpr (sizeof(TG) == 2) hipLaunchKernelGGL((k_embed_sum<TG, TW, 8, FEW>), grid, block, 0, s, a);
      break;
    case 4: hipLaunchKernelGGL((k_embed_sum<TG, TW, 4, FEW>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_embed_sum<TG, TW, 2, FEW>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_embed_sum<TG, TW, 1, FEW>), grid, block, 0, s, a); break;
  }
}

template <typename TG, typename TW>
void launch_sum(const BwdPlan& p, int v, const SumArgs& a, hipStream_t s) {
  if (p.few) return launch_sum_as<TG, TW, true>(p, v, a, s);
  launch_sum_as<TG, TW, false>(p, v, a, s);
  const dim3 grid((unsigned)p.blocks), block(kThreads);
  if (a.dim % 4 == 0)
    hipLaunchKernelGGL((k_embed_join<TW, 4>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_embed_join<TW, 1>), grid, block, 0, s, a);
}

constexpr int64_t kMaxTokens = (1ll << 31) - 4096;
constexpr int64_t kMaxVocab = 1ll << 30;
constexpr int kMaxDim = 1 << 16;
constexpr int64_t kMaxElements = 1ll << 40;  // of the forward's result
static_assert(kMaxElements / kFwdTile <= kMaxBlocks, "the forward's blocks can be launched");

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

recis_status recis_embed_fwd(const int64_t* tokens, int64_t n, const void* weight, int32_t dtype, int64_t rows,
                             int32_t dim, int64_t weight_stride, float scale, void* out, int64_t out_stride,
                             uint32_t* error, hipStream_t s) {
  if (!dtype_known(dtype) || n < 0 || rows < 1 || dim < 1 || weight_stride < dim || out_stride < dim)
    return RECIS_ERR_INVALID_ARG;
  if (n > kMaxTokens || rows > kMaxVocab || dim > kMaxDim || n * dim > kMaxElements) return RECIS_ERR_UNSUPPORTED;
  if (n == 0) return RECIS_OK;
  const int size = dtype_size(dtype);
  if (!tokens || !weight || !out || !aligned_to(tokens, 8) || !aligned_to(weight, size) || !aligned_to(out, size) ||
      !aligned_to(error, 4))
    return RECIS_ERR_INVALID_ARG;
  const int v = access_width(size, dim, {weight, out}, {weight_stride, out_stride});
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
  for (int v : {1, 2, 4, 8}) most = std::max(most, bwd_plan(n, rows, dim, v).bytes);
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
  // (a bfloat16 side may ask for eight elements, a float32 one for four; the
  // float32 result of a bfloat16 gradient is then written in two accesses)
  const int gv = access_width(gs, dim, {grad_out}, {grad_stride});
  const int wv = access_width(ws, dim, {grad_weight}, {weight_stride});
  const int v = gv == 8 && wv == 4 && ws == 4 ? 8 : std::min(gv, wv);
  const BwdPlan p = bwd_plan(n, rows, dim, v);
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < p.bytes) return RECIS_ERR_INVALID_ARG;
  char* w = static_cast<char*>(workspace);
  SortArgs o;
  o.tokens = reinterpret_cast<const long long*>(tokens);
  o.n = n;
  o.rows = (unsigned)rows;
  o.digits = 1 << p.digit_bits;
  o.tiles = p.tiles;
  o.hist = reinterpret_cast<unsigned*>(w + p.hist);
  o.totals = reinterpret_cast<unsigned*>(w + p.totals);
  o.error = error;
  int cur = 0;
  for (int pass = 0; !p.few && pass < p.passes; ++pass) {
    o.in = reinterpret_cast<const Keyed*>(w + p.sorted[cur]);
    o.out = reinterpret_cast<Keyed*>(w + p.sorted[cur ^ 1]);
    o.shift = pass * p.digit_bits;
    if (p.per == 4)
      pass == 0 ? launch_sort<true, 4>(p, o, s) : launch_sort<false, 4>(p, o, s);
    else
      pass == 0 ? launch_sort<true, 16>(p, o, s) : launch_sort<false, 16>(p, o, s);
    cur ^= 1;
  }
  SumArgs a;
  a.tok = reinterpret_cast<const Keyed*>(w + p.sorted[cur]);
  a.n = n;
  a.rows = rows;
  a.grad = grad_out;
  a.grad_stride = grad_stride;
  a.out = grad_weight;
  a.out_stride = weight_stride;
  a.scale = scale;
  a.dim = dim;
  a.quantum = p.quantum;
  a.stream = rows * dim * ws > kStreamBytes;
  a.lane_bits = p.lane_bits;
  a.raw = o.tokens;
  a.block_rows = p.block_rows;
  a.error = error;
  a.first_row = reinterpret_cast<int*>(w + p.first_row);
  a.began = reinterpret_cast<int*>(w + p.began);
  a.head = reinterpret_cast<float*>(w + p.head);
  a.tail = reinterpret_cast<float*>(w + p.tail);
  const bool gb = grad_dtype == RECIS_DTYPE_BF16, wb = weight_dtype == RECIS_DTYPE_BF16;
  if (gb && wb)
    launch_sum<__bf16, __bf16>(p, v, a, s);
  else if (gb)
    launch_sum<__bf16, float>(p, v, a, s);
  else if (wb)
    launch_sum<float, __bf16>(p, v, a, s);
  else
    launch_sum<float, float>(p, v, a, s);
  return launch_status();
}

}  // extern "C"
