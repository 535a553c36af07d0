// norm.hip -- layer norm, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  xh = (x - mean) rstd
//   y  = xh w + b
//   dx = rstd (g w - sum(g w) / D - xh sum(g w xh) / D),   dw = sum_rows g xh,   db = sum_rows g
//
// A row stays in the registers of the L lanes that share it (K accesses of V
// elements a lane), so it is read once: the mean first, the squared distances
// from it second.  Everything is held in float32.
//
// Bound by memory.  2.05M rows of 128 bfloat16: forward 1.05 GB in 180 us, 5.8
// TB/s, backward 1.57 GB in 296 us, 5.3 TB/s (above a large copy's 4.8: part of
// the rows is still in the memory-side cache from the pass before).  12289 rows
// of 777 float32, whose rows allow no wider access than 4 bytes: 16.4 and 21.7
// us, 4.6 and 5.3 TB/s, and 4.5 us to add up the blocks' weight gradients.
// Bfloat16 rows that allow no 16-byte access are read and written by single
// elements, and bound by the number of accesses: 2.05M rows of 100, 516 and 755
// us, 1.6 TB/s.  Above 8192 elements a row takes 1024 lanes, whose 128 registers
// do not hold all of the backward's values: 8 to 62 words a lane go through
// scratch memory (10000 rows of 16384 float32: forward 241 us, 5.4 TB/s,
// backward 385, 5.1; of 16383: 269 and 731).
#include <algorithm>
#include <atomic>

#include "seq.h"

namespace recis {
namespace {

// Sums of N values over the L lanes of a group, or over the block (L = its size).
template <int L, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*shared)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lane_sum<(L < 64 ? L : 64)>(v[n]);
  if constexpr (L > 64) {
    constexpr int kW = L / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) shared[threadIdx.x >> 6][n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) v[n] += shared[w][n];
    }
    __syncthreads();
  }
}

struct NormArgs {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  void* y;  // y forward, dx backward
  float* mean;
  float* rstd;
  float* partial;  // [blocks][2][dim]
  int64_t m, x_stride, dy_stride, y_stride;
  int dim, w_bf16;
  float eps;
};

// The lane's columns of the weight (or `none` without one).
template <int V, int K, int L>
__device__ __forceinline__ void load_weight(const void* w, int bf16, int dim, int lane, float none, float (&v)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = none;
    const int c = (k * L + lane) * V;
    if (!w || c >= dim) continue;
    if (bf16) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = (float)static_cast<const __bf16*>(w)[c + i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = static_cast<const float*>(w)[c + i];
    }
  }
}

template <typename T, int V, int K, int L>
__device__ __forceinline__ void load_row(const T* row, int dim, int lane, float (&v)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * L + lane) * V;
    if (c < dim) {
      load_f32<T, V>(row + c, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = 0.f;
    }
  }
}

// s / n to the last bit or nearly: a constant row has its constant as mean.
__device__ __forceinline__ float over(float s, float n, float inv) {
  const float q = s * inv;
  return fmaf(fmaf(-q, n, s), inv, q);
}

// R rows a group at a time: their loads are all under way before the first sum.
template <typename T, int V, int L, int K, int THREADS, int R>
__global__ __launch_bounds__(THREADS) void k_norm_fwd(NormArgs a) {
  constexpr int kGroups = THREADS / L;
  __shared__ float shared[THREADS / 64][R];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const float n = (float)a.dim, inv = 1.f / n;
  float w[K][V], b[K][V];
  load_weight<V, K, L>(a.w, a.w_bf16, a.dim, lane, 1.f, w);
  load_weight<V, K, L>(a.b, a.w_bf16, a.dim, lane, 0.f, b);
  for (int64_t r0 = (int64_t)blockIdx.x * (kGroups * R); r0 < a.m; r0 += (int64_t)gridDim.x * (kGroups * R)) {
    float v[R][K][V], s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r * kGroups + group;
      load_row<T, V, K, L>(static_cast<const T*>(a.x) + row * a.x_stride, row < a.m ? a.dim : 0, lane, v[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) s[r] += v[r][k][i];
    }
    group_sums<L, R>(s, shared);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = over(s[r], n, inv);
      s[r] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = (k * L + lane) * V < a.dim ? v[r][k][i] - mean[r] : 0.f;
          v[r][k][i] = d;
          s[r] += d * d;
        }
    }
    group_sums<L, R>(s, shared);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r * kGroups + group;
      if (row >= a.m) continue;
      const float rstd = __builtin_amdgcn_rsqf(over(s[r], n, inv) + a.eps);
      if (lane == 0 && a.mean) {
        a.mean[row] = mean[r];
        a.rstd[row] = rstd;
      }
      T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * V;
        if (c >= a.dim) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) v[r][k][i] = v[r][k][i] * rstd * w[k][i] + b[k][i];
        store_f32<T, V>(y + c, v[r][k]);
      }
    }
  }
}

// dx, and the block's part of dw and db: every lane adds up its columns over
// the rows its group takes, the groups are joined in LDS in order, and
// k_norm_bwd_weight adds the blocks' parts in order.
template <typename T, int V, int L, int K, int THREADS, int R>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(NormArgs a) {
  constexpr int kGroups = THREADS / L;
  __shared__ float shared[THREADS / 64][2 * R];
  __shared__ float join[kGroups > 1 ? THREADS * K * V : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const float n = (float)a.dim, inv = 1.f / n;
  float w[K][V], dw[K][V], db[K][V];
  load_weight<V, K, L>(a.w, a.w_bf16, a.dim, lane, 1.f, w);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * (kGroups * R); r0 < a.m; r0 += (int64_t)gridDim.x * (kGroups * R)) {
    float x[R][K][V], g[R][K][V], rstd[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r * kGroups + group;
      const bool in = row < a.m;
      load_row<T, V, K, L>(static_cast<const T*>(a.x) + row * a.x_stride, in ? a.dim : 0, lane, x[r]);
      load_row<T, V, K, L>(static_cast<const T*>(a.dy) + row * a.dy_stride, in ? a.dim : 0, lane, g[r]);
      s[r] = in ? a.mean[row] : 0.f;
      rstd[r] = in ? a.rstd[row] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mean = s[r];
      s[r] = s[R + r] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // (a row that does not exist has gradient 0 and rstd 0)
        const bool live = (k * L + lane) * V < a.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = live ? (x[r][k][i] - mean) * rstd[r] : 0.f;
          dw[k][i] += g[r][k][i] * xh;
          db[k][i] += g[r][k][i];
          x[r][k][i] = xh;
          g[r][k][i] *= w[k][i];
          s[r] += g[r][k][i];
          s[R + r] += g[r][k][i] * xh;
        }
      }
    }
    group_sums<L, 2 * R>(s, shared);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r * kGroups + group;
      if (row >= a.m) continue;
      T* dx = static_cast<T*>(a.y) + row * a.y_stride;
      const float m1 = s[r] * inv, m2 = s[R + r] * inv;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * V;
        if (c >= a.dim) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) g[r][k][i] = (g[r][k][i] - m1 - x[r][k][i] * m2) * rstd[r];
        store_f32<T, V>(dx + c, g[r][k]);
      }
    }
  }
  if (!a.partial) return;
  float* part = a.partial + (int64_t)blockIdx.x * 2 * a.dim;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (k * L + lane) * V + i;
        if (c < a.dim) {
          part[c] = dw[k][i];
          part[a.dim + c] = db[k][i];
        }
      }
  } else {
    constexpr int C = L * K * V;  // columns of a group
    for (int half = 0; half < 2; ++half) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) join[group * C + (k * L + lane) * V + i] = half ? db[k][i] : dw[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < C; c += THREADS) {
        if (c >= a.dim) break;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kGroups; ++r) sum += join[r * C + c];
        part[half * a.dim + c] = sum;
      }
    }
  }
}

constexpr int kJoinCols = 16, kJoinRows = 64;

// Columns 0 .. 2 dim - 1 of the blocks' parts: dw, then db.
__global__ __launch_bounds__(kJoinCols* kJoinRows) void k_norm_bwd_weight(const float* __restrict__ partial,
                                                                          int blocks, int dim, void* dw, void* db,
                                                                          int w_bf16) {
  __shared__ float join[kJoinRows][kJoinCols + 1];
  const int tc = threadIdx.x % kJoinCols, tr = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + tc;
  float sum = 0.f;
  if (c < 2 * dim)
#pragma unroll 8
    for (int b = tr; b < blocks; b += kJoinRows) sum += partial[(int64_t)b * 2 * dim + c];
  join[tr][tc] = sum;
  __syncthreads();
  if (tr == 0 && c < 2 * dim) {
    sum = 0.f;
    for (int r = 0; r < kJoinRows; ++r) sum += join[r][tc];
    void* to = c < dim ? dw : db;
    const int at = c < dim ? c : c - dim;
    if (to) {
      if (w_bf16)
        static_cast<__bf16*>(to)[at] = (__bf16)sum;
      else
        static_cast<float*>(to)[at] = sum;
    }
  }
}

// How a row of `dim` elements read V at a time is laid over lanes: L lanes
// of K accesses.
struct RowPlan {
  int v, lanes, k, threads;
};

// Rows a group holds at once, of `held` floats a lane each.  Forward: more
// loads under way (2.05M rows of 128 bf16: 2 rows 180 us, 1 row 188, 4 rows
// 199).  Backward: one, the registers are better spent on more waves (1 row
// 298 us, 2 rows 314, 4 rows 449).
constexpr int forward_rows(int held) { return held <= 4 ? 4 : held <= 8 ? 2 : 1; }
constexpr int backward_rows(int held) { return held <= 4 ? 2 : 1; }

constexpr int kMaxNormDim = 16384;
constexpr int most_accesses(int v, int lanes) {  // K * V <= 32 floats of a row a lane
  return lanes == 16 ? 1 : std::min(16, 32 / v);
}

// Whether row_plan takes this form for any row length.
constexpr bool row_form(int v, int lanes, int k) {
  const int fewer_lanes = lanes > 16 ? lanes / 4 * most_accesses(v, lanes / 4) : 0, fewer = k > 1 ? lanes * k / 2 : 0;
  return k <= most_accesses(v, lanes) && std::max(fewer_lanes, fewer) < std::min(lanes * k, kMaxNormDim / v);
}

bool row_plan(int dim, int v, RowPlan* p) {
  const int acc = (dim + v - 1) / v;
  p->v = v;
  p->threads = 256;
  for (int l : {16, 64, 256, 1024}) {
    for (int k = 1; k <= most_accesses(v, l); k *= 2) {
      if ((int64_t)l * k < acc) continue;
      p->lanes = l;
      p->k = k;
      if (l > 256) p->threads = l;
      return true;
    }
  }
  return false;
}

// The backward's blocks stay for the whole call, each with a part of dw and db
// to write: as many as run at once (the same case: 1536 blocks, 6 a CU, 298 us;
// with 2048 a third of the work waits for a second turn, 379 us).
constexpr int kMaxBwdThreads = 256 * 6 * 256;

template <void (*KERNEL)(NormArgs)>
int blocks_at_once(int threads) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0: not asked yet
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess || device >= kDevices) device = 0;
  int n = known[device].load(std::memory_order_relaxed);
  if (n) return n;
  int per_cu = 0, cus = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, KERNEL, threads, 0) != hipSuccess || per_cu < 1)
    per_cu = 1;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || cus < 1) cus = 256;
  (void)hipGetLastError();
  n = std::min(per_cu * cus, kMaxBwdThreads / threads);
  known[device].store(n, std::memory_order_relaxed);
  return n;
}

// Returns the blocks of the launch.
template <typename T, int V, int L, int K, int THREADS>
int launch_norm(bool bwd, const NormArgs& a, hipStream_t s) {
  if constexpr (row_form(V, L, K)) {
    auto blocks_of = [&](int64_t rows, int64_t most) { return (int)std::min<int64_t>(most, (a.m + rows - 1) / rows); };
    if (bwd) {
      constexpr int R = backward_rows(K * V);
      const int most = blocks_at_once<k_norm_bwd<T, V, L, K, THREADS, R>>(THREADS);
      const int blocks = blocks_of(THREADS / L * R, most);
      hipLaunchKernelGGL((k_norm_bwd<T, V, L, K, THREADS, R>), dim3(blocks), dim3(THREADS), 0, s, a);
      return blocks;
    }
    constexpr int R = forward_rows(K * V);
    const int blocks = blocks_of(THREADS / L * R, 1 << 14);
    hipLaunchKernelGGL((k_norm_fwd<T, V, L, K, THREADS, R>), dim3(blocks), dim3(THREADS), 0, s, a);
    return blocks;
  }
  return 0;
}

template <typename T, int V, int L, int THREADS>
int launch_norm_k(bool bwd, int k, const NormArgs& a, hipStream_t s) {
  switch (k) {
    case 1: return launch_norm<T, V, L, 1, THREADS>(bwd, a, s);
    case 2: return launch_norm<T, V, L, 2, THREADS>(bwd, a, s);
    case 4: return launch_norm<T, V, L, 4, THREADS>(bwd, a, s);
    case 8: return launch_norm<T, V, L, 8, THREADS>(bwd, a, s);
    default: return launch_norm<T, V, L, 16, THREADS>(bwd, a, s);
  }
}

template <typename T, int V>
int launch_norm_v(bool bwd, const RowPlan& p, const NormArgs& a, hipStream_t s) {
  switch (p.lanes) {
    case 16: return launch_norm<T, V, 16, 1, 256>(bwd, a, s);
    case 64: return launch_norm_k<T, V, 64, 256>(bwd, p.k, a, s);
    case 256: return launch_norm_k<T, V, 256, 256>(bwd, p.k, a, s);
    default: return launch_norm_k<T, V, 1024, 1024>(bwd, p.k, a, s);
  }
}

int launch_norm_any(bool bwd, int dtype, const RowPlan& p, const NormArgs& a, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16) {
    return p.v == 8 ? launch_norm_v<__bf16, 8>(bwd, p, a, s) : launch_norm_v<__bf16, 1>(bwd, p, a, s);
  } else {
    return p.v == 4 ? launch_norm_v<float, 4>(bwd, p, a, s) : launch_norm_v<float, 1>(bwd, p, a, s);
  }
}

// Parts of dw and db that a call of either access width may write.
int64_t most_bwd_blocks(int64_t m, int dim) {
  int64_t most = 0;
  for (int v : {1, 4, 8}) {
    RowPlan p;
    if (row_plan(dim, v, &p)) most = std::max<int64_t>(most, kMaxBwdThreads / p.threads);
  }
  return std::min(most, std::max<int64_t>(m, 1));
}

int whole_or_one(int dtype, int v) { return v == 16 / dtype_size(dtype) ? v : 1; }

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" {

recis_status recis_layernorm_fwd(const void* x, int32_t dtype, int64_t x_stride, int64_t m, int32_t dim,
                                 const void* weight, const void* bias, int32_t weight_dtype, float eps, void* y,
                                 int64_t y_stride, float* mean, float* rstd, hipStream_t s) {
  if (!dtype_known(dtype) || !dtype_known(weight_dtype) || m < 0 || dim < 1 || x_stride < dim || y_stride < dim ||
      !(eps >= 0.f) || !mean != !rstd)
    return RECIS_ERR_INVALID_ARG;
  if (dim > kMaxNormDim) return RECIS_ERR_UNSUPPORTED;
  const int size = dtype_size(dtype), ws = dtype_size(weight_dtype);
  if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(weight, ws) || !aligned_to(bias, ws) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RECIS_ERR_INVALID_ARG;
  if (m == 0) return RECIS_OK;
  if (!x || !y) return RECIS_ERR_INVALID_ARG;
  RowPlan p;
  if (!row_plan(dim, whole_or_one(dtype, access_width(size, dim, {x, y}, {x_stride, y_stride})), &p))
    return RECIS_ERR_UNSUPPORTED;
  NormArgs a{};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.m = m;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.dim = dim;
  a.w_bf16 = weight_dtype == RECIS_DTYPE_BF16;
  a.eps = eps;
  launch_norm_any(false, dtype, p, a, s);
  return launch_status();
}

int64_t recis_layernorm_bwd_workspace_bytes(int64_t m, int32_t dim) {
  if (m < 0 || dim < 1 || dim > kMaxNormDim) return -1;
  return round_up(most_bwd_blocks(m, dim) * 2 * dim * 4, 256);
}

recis_status recis_layernorm_bwd(const void* grad_y, int64_t grad_stride, const void* x, int64_t x_stride,
                                 int32_t dtype, int64_t m, int32_t dim, const float* mean, const float* rstd,
                                 const void* weight, int32_t weight_dtype, void* grad_x, int64_t grad_x_stride,
                                 void* grad_weight, void* grad_bias, void* workspace, int64_t workspace_bytes,
                                 hipStream_t s) {
  if (!dtype_known(dtype) || !dtype_known(weight_dtype) || m < 0 || dim < 1 || x_stride < dim || grad_stride < dim ||
      grad_x_stride < dim)
    return RECIS_ERR_INVALID_ARG;
  if (dim > kMaxNormDim) return RECIS_ERR_UNSUPPORTED;
  const int size = dtype_size(dtype), ws = dtype_size(weight_dtype);
  if (!aligned_to(x, size) || !aligned_to(grad_y, size) || !aligned_to(grad_x, size) || !aligned_to(weight, ws) ||
      !aligned_to(grad_weight, ws) || !aligned_to(grad_bias, ws) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RECIS_ERR_INVALID_ARG;
  if (m > 0 && (!x || !grad_y || !grad_x || !mean || !rstd)) return RECIS_ERR_INVALID_ARG;
  const bool sums = grad_weight || grad_bias;
  if (sums && (!workspace || !aligned_to(workspace, 256) ||
               workspace_bytes < recis_layernorm_bwd_workspace_bytes(m, dim)))
    return RECIS_ERR_INVALID_ARG;
  RowPlan p;
  if (!row_plan(dim, whole_or_one(dtype, access_width(size, dim, {x, grad_y, grad_x},
                                                      {x_stride, grad_stride, grad_x_stride})), &p))
    return RECIS_ERR_UNSUPPORTED;
  NormArgs a{};
  a.x = x;
  a.dy = grad_y;
  a.w = weight;
  a.y = grad_x;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.m = m;
  a.x_stride = x_stride;
  a.dy_stride = grad_stride;
  a.y_stride = grad_x_stride;
  a.dim = dim;
  a.w_bf16 = weight_dtype == RECIS_DTYPE_BF16;
  const int blocks = m > 0 ? launch_norm_any(true, dtype, p, a, s) : 0;
  if (sums)
    hipLaunchKernelGGL(k_norm_bwd_weight, dim3((2 * dim + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinRows), 0,
                       s, a.partial, blocks, dim, grad_weight, grad_bias, a.w_bf16);
  return launch_status();
}

}  // extern "C"
