// seq.h -- shared helpers of the sequence operators (embed.hip, norm.hip, attn.hip).
#pragma once

#include "internal.h"

namespace recis {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
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

inline recis_status launch_status() {
  return hipGetLastError() == hipSuccess ? RECIS_OK : RECIS_ERR_HIP;
}

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace recis
