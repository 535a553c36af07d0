// seq.h -- shared helpers of the sequence operators (embed.hip, norm.hip, attn.hip).
#pragma once

#include "internal.h"

namespace recis {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// V consecutive elements of type T as one aligned memory access (16 bytes at most).
template <typename T, int V>
struct __attribute__((aligned(sizeof(T) * V))) Vec {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[V]) {
  const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = (float)x.e[i];
}

// One rounding, to nearest with ties to even, where T is bfloat16; 16 bytes a
// store at most.
template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[V]) {
  constexpr int W = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
#pragma unroll
  for (int j = 0; j < V; j += W) {
    Vec<T, W> x;
#pragma unroll
    for (int i = 0; i < W; ++i) x.e[i] = (T)v[j + i];
    *reinterpret_cast<Vec<T, W>*>(p + j) = x;
  }
}

// Results of more bytes than the L2s hold together are stored past them: no
// reader would find them there, and the stores would push out what the kernel
// itself reads again (embedding of 2.05M tokens, 128 bf16: 79 us against 143).
constexpr int64_t kStreamBytes = 32ll << 20;

template <typename T, int V>
__device__ __forceinline__ void stream_f32(T* p, const float (&v)[V]) {
  constexpr int W = V * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : V;
  typedef T TV __attribute__((ext_vector_type(W)));
#pragma unroll
  for (int j = 0; j < V; j += W) {
    if constexpr (W == 1) {
      __builtin_nontemporal_store((T)v[j], p + j);
    } else {
      TV x;
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = (T)v[j + i];
      __builtin_nontemporal_store(x, reinterpret_cast<TV*>(p + j));
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_or_stream(bool stream, T* p, const float (&v)[V]) {
  if (stream)
    stream_f32<T, V>(p, v);
  else
    store_f32<T, V>(p, v);
}

// Sum over the L lanes of an aligned group (a power of two up to 64), in every
// lane, by register permutations.
template <int CTRL>
__device__ __forceinline__ float add_permuted(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (L > 1) v = add_permuted<0xB1>(v);    // lanes 1 0 3 2
  if constexpr (L > 2) v = add_permuted<0x4E>(v);    // lanes 2 3 0 1
  if constexpr (L > 4) v = add_permuted<0x141>(v);   // 8 lanes reversed
  if constexpr (L > 8) v = add_permuted<0x140>(v);   // 16 lanes reversed
  if constexpr (L > 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (L > 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return v;
}

// Widest access, in elements of `size` bytes, that the pointers, the row
// strides (in elements) and the row length allow: 16 bytes down to one element.
inline int access_width(int size, int64_t dim, std::initializer_list<const void*> ptrs,
                        std::initializer_list<int64_t> strides) {
  int v = 16 / size;
  auto fits = [&](int w) {
    if (dim % w) return false;
    for (const void* p : ptrs)
      if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)(w * size)) return false;
    for (int64_t s : strides)
      if (s % w) return false;
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  return v;
}

inline int dtype_size(int dtype) { return dtype == RECIS_DTYPE_BF16 ? 2 : 4; }
inline bool dtype_known(int dtype) { return dtype == RECIS_DTYPE_F32 || dtype == RECIS_DTYPE_BF16; }

// Tensors hold naturally aligned elements; anything else is refused.
inline bool aligned_to(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)size == 0; }

// The blocks (of kThreads) of a launch that may have very many: a dimension of a
// launch holds 2^32 - 1 threads at most, so from kRowBlocks on they lie in rows
// of that many.  The last row's blocks past `blocks` have ids past it too, which
// the kernel has to leave alone.  kRowBlocks is a multiple of the dies, so the
// order in which blocks go to them is that of the ids.
constexpr int64_t kRowBlocks = 1 << 22;
constexpr int64_t kMaxBlocks = (1ll << 31) - kRowBlocks;  // every id fits an int
inline dim3 grid_of(int64_t blocks) {
  if (blocks <= kRowBlocks) return dim3((unsigned)blocks);
  return dim3((unsigned)kRowBlocks, (unsigned)((blocks + kRowBlocks - 1) / kRowBlocks));
}
__device__ __forceinline__ int block_id() { return (int)(blockIdx.y * (unsigned)kRowBlocks + blockIdx.x); }

inline recis_status launch_status() {
  return hipGetLastError() == hipSuccess ? RECIS_OK : RECIS_ERR_HIP;
}

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace recis
