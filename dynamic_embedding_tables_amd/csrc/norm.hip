// norm.hip -- layer norm, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  xh = (x - mean) rstd
//   y  = xh w + b
//   dx = rstd (g w - sum(g w) / D - xh sum(g w xh) / D),   dw = sum_rows g xh,   db = sum_rows g
//
// A row stays in the registers of the L lanes that share it (K accesses of V
// elements a lane), so it is read once: the mean first, the squared distances
// from it second.  Everything is held in float32.
#include <algorithm>

#include "seq.h"

namespace recis {
namespace {

// Sum over the L lanes of a group (L <= 64), or over the block (L = blockDim).
template <int L>
__device__ __forceinline__ float group_sum(float v, float* shared) {
#pragma unroll
  for (int o = 1; o < (L < 64 ? L : 64); o <<= 1) v += __shfl_xor(v, o);
  if constexpr (L > 64) {
    constexpr int kW = L / 64;
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) v += shared[w];
    __syncthreads();
  }
  return v;
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

__device__ __forceinline__ float weight_at(const void* w, int bf16, int i) {
  return bf16 ? (float)static_cast<const __bf16*>(w)[i] : static_cast<const float*>(w)[i];
}

template <typename T, int V, int K>
__device__ __forceinline__ void load_row(const T* row, int dim, int lane, int lanes, float (&v)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * lanes + lane) * V;
    if (c < dim) {
      load_f32<T, V>(row + c, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = 0.f;
    }
  }
}

template <typename T, int V, int L, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_fwd(NormArgs a) {
  constexpr int kRows = THREADS / L;
  __shared__ float shared[THREADS / 64];
  const int lane = threadIdx.x % L;
  float w[K][V], b[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (k * L + lane) * V + i;
      w[k][i] = a.w && c < a.dim ? weight_at(a.w, a.w_bf16, c) : 1.f;
      b[k][i] = a.b && c < a.dim ? weight_at(a.b, a.w_bf16, c) : 0.f;
    }
  // divided, not multiplied by 1 / dim: a constant row has its constant as mean
  const float dim_f = (float)a.dim;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.m; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool in = row < a.m;
    float v[K][V];
    load_row<T, V, K>(static_cast<const T*>(a.x) + row * a.x_stride, in ? a.dim : 0, lane, L, v);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[k][i];
    const float mean = group_sum<L>(s, shared) / dim_f;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = (k * L + lane) * V < a.dim ? v[k][i] - mean : 0.f;
        v[k][i] = d;
        q += d * d;
      }
    const float rstd = 1.f / sqrtf(group_sum<L>(q, shared) / dim_f + a.eps);
    if (!in) continue;
    if (lane == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c >= a.dim) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rstd * w[k][i] + b[k][i];
      store_f32<T, V>(y + c, v[k]);
    }
  }
}

// dx, and the block's part of dw and db: every lane adds up its columns over
// the rows its group takes, the groups are joined in LDS in order, and
// k_norm_bwd_weight adds the blocks' parts in order.
template <typename T, int V, int L, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(NormArgs a) {
  constexpr int kRows = THREADS / L;
  __shared__ float shared[THREADS / 64];
  __shared__ float join[kRows > 1 ? THREADS * K * V : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  float w[K][V], dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (k * L + lane) * V + i;
      w[k][i] = a.w && c < a.dim ? weight_at(a.w, a.w_bf16, c) : 1.f;
      dw[k][i] = db[k][i] = 0.f;
    }
  const float dim_f = (float)a.dim;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.m; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + group;
    const bool in = row < a.m;
    const int dim = in ? a.dim : 0;
    float x[K][V], g[K][V];
    load_row<T, V, K>(static_cast<const T*>(a.x) + row * a.x_stride, dim, lane, L, x);
    load_row<T, V, K>(static_cast<const T*>(a.dy) + row * a.dy_stride, dim, lane, L, g);
    const float mean = in ? a.mean[row] : 0.f, rstd = in ? a.rstd[row] : 0.f;
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool live = (k * L + lane) * V < dim;
        const float xh = live ? (x[k][i] - mean) * rstd : 0.f;
        dw[k][i] += g[k][i] * xh;
        db[k][i] += g[k][i];
        x[k][i] = xh;
        g[k][i] *= w[k][i];
        s += g[k][i];
        q += g[k][i] * xh;
      }
    s = group_sum<L>(s, shared) / dim_f;
    q = group_sum<L>(q, shared) / dim_f;
    if (!in) continue;
    T* dx = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c >= a.dim) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) g[k][i] = (g[k][i] - s - x[k][i] * q) * rstd;
      store_f32<T, V>(dx + c, g[k]);
    }
  }
  if (!a.partial) return;
  float* part = a.partial + (int64_t)blockIdx.x * 2 * a.dim;
  if constexpr (kRows == 1) {
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
        for (int r = 0; r < kRows; ++r) sum += join[r * C + c];
        part[half * a.dim + c] = sum;
      }
    }
  }
}

constexpr int kJoinCols = 32, kJoinRows = 32;

// Columns 0 .. 2 dim - 1 of the blocks' parts: dw, then db.
__global__ __launch_bounds__(kJoinCols* kJoinRows) void k_norm_bwd_weight(const float* __restrict__ partial,
                                                                          int blocks, int dim, void* dw, void* db,
                                                                          int w_bf16) {
  __shared__ float join[kJoinRows][kJoinCols + 1];
  const int tc = threadIdx.x % kJoinCols, tr = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + tc;
  float sum = 0.f;
  if (c < 2 * dim)
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

constexpr int kMaxNormDim = 16384;

bool row_plan(int dim, int v, RowPlan* p) {
  const int acc = (dim + v - 1) / v;
  const int most = std::min(16, 32 / v);  // K * V <= 32 floats of a row a lane
  p->v = v;
  p->threads = 256;
  for (int l : {16, 64, 256, 1024}) {
    for (int k = 1; k <= (l == 16 ? 1 : most); k *= 2) {
      if ((int64_t)l * k < acc) continue;
      p->lanes = l;
      p->k = k;
      if (l > 256) p->threads = l;
      return true;
    }
  }
  return false;
}

template <typename T, int V, int L, int K, int THREADS>
void launch_norm(bool bwd, const NormArgs& a, int blocks, hipStream_t s) {
  if constexpr (K * V <= 32) {
    if (bwd)
      hipLaunchKernelGGL((k_norm_bwd<T, V, L, K, THREADS>), dim3(blocks), dim3(THREADS), 0, s, a);
    else
      hipLaunchKernelGGL((k_norm_fwd<T, V, L, K, THREADS>), dim3(blocks), dim3(THREADS), 0, s, a);
  }
}

template <typename T, int V, int L, int THREADS>
void launch_norm_k(bool bwd, int k, const NormArgs& a, int blocks, hipStream_t s) {
  switch (k) {
    case 1: return launch_norm<T, V, L, 1, THREADS>(bwd, a, blocks, s);
    case 2: return launch_norm<T, V, L, 2, THREADS>(bwd, a, blocks, s);
    case 4: return launch_norm<T, V, L, 4, THREADS>(bwd, a, blocks, s);
    case 8: return launch_norm<T, V, L, 8, THREADS>(bwd, a, blocks, s);
    default: return launch_norm<T, V, L, 16, THREADS>(bwd, a, blocks, s);
  }
}

template <typename T, int V>
void launch_norm_v(bool bwd, const RowPlan& p, const NormArgs& a, int blocks, hipStream_t s) {
  switch (p.lanes) {
    case 16: return launch_norm<T, V, 16, 1, 256>(bwd, a, blocks, s);
    case 64: return launch_norm_k<T, V, 64, 256>(bwd, p.k, a, blocks, s);
    case 256: return launch_norm_k<T, V, 256, 256>(bwd, p.k, a, blocks, s);
    default: return launch_norm_k<T, V, 1024, 1024>(bwd, p.k, a, blocks, s);
  }
}

void launch_norm_any(bool bwd, int dtype, const RowPlan& p, const NormArgs& a, int blocks, hipStream_t s) {
  if (dtype == RECIS_DTYPE_BF16) {
    p.v == 8 ? launch_norm_v<__bf16, 8>(bwd, p, a, blocks, s) : launch_norm_v<__bf16, 1>(bwd, p, a, blocks, s);
  } else {
    p.v == 4 ? launch_norm_v<float, 4>(bwd, p, a, blocks, s) : launch_norm_v<float, 1>(bwd, p, a, blocks, s);
  }
}

constexpr int kBwdBlocks = 1024;

int norm_blocks(int64_t m, const RowPlan& p, int most) {
  const int64_t rows = p.threads / p.lanes;
  return (int)std::min<int64_t>(most, (m + rows - 1) / rows);
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
  launch_norm_any(false, dtype, p, a, norm_blocks(m, p, 1 << 14), s);
  return launch_status();
}

int64_t recis_layernorm_bwd_workspace_bytes(int64_t m, int32_t dim) {
  if (m < 0 || dim < 1 || dim > kMaxNormDim) return -1;
  return round_up(std::min<int64_t>(kBwdBlocks, std::max<int64_t>(m, 1)) * 2 * dim * 4, 256);
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
  const int blocks = norm_blocks(m, p, kBwdBlocks);
  if (m > 0) launch_norm_any(true, dtype, p, a, blocks, s);
  if (sums)
    hipLaunchKernelGGL(k_norm_bwd_weight, dim3((2 * dim + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinRows), 0,
                       s, a.partial, m > 0 ? blocks : 0, dim, grad_weight, grad_bias, a.w_bf16);
  return launch_status();
}

}  // extern "C"
