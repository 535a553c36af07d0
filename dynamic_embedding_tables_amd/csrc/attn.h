// attn.h -- what the attention kernels share: operands of the matrix
// instructions, LDS tiles, and the exchanges between a wave's lanes.
#pragma once

#include <cmath>

#include "seq.h"

namespace recis {
namespace {

constexpr int kMaxHeadDim = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The wave's number, known to be the same in all its lanes.
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

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
// Eight products of k = 4: the j-th takes element j of every lane.
template <int N = 8>
__device__ __forceinline__ f32x4 mma(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < N; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// Head sizes are padded to DP: 32, 48 (float32), 64, 96 or 128.  A product
// over the head runs in KK chunks of 32; float32's operand of a chunk holds 4
// elements from 4 * (lane / 16) and 4 from 16 further on, so that a last chunk
// of 16 costs half of the products.
template <int DP>
constexpr int kChunks32 = (DP + 31) / 32;
template <int DP>
__device__ __forceinline__ f32x4 mma_head(bf16x8 a, bf16x8 b, f32x4 c, int) {
  return mma(a, b, c);
}
template <int DP>
__device__ __forceinline__ f32x4 mma_head(f32x8 a, f32x8 b, f32x4 c, int chunk) {
  return DP % 32 && chunk == kChunks32<DP> - 1 ? mma<4>(a, b, c) : mma<8>(a, b, c);
}

// Four zeros that stay in registers: a product that starts from them needs no
// moves (the compiler would clear its accumulator each time).
__device__ __forceinline__ f32x4 zeros() {
  f32x4 z{0.f, 0.f, 0.f, 0.f};
  asm volatile("" : "+v"(z));
  return z;
}

// LDS reads stay on their side of this point (everything else may cross): a
// product's operands are all asked for before the first one is needed, where
// the compiler, short of registers, would ask for two and wait, and so on.
__device__ __forceinline__ void reads_before() { __builtin_amdgcn_sched_barrier(0x47F); }

// The larger / the sum of a lane's value and those of the lanes 16, 32 and 48
// away, by register swaps (no LDS access).
template <typename F>
__device__ __forceinline__ float across_groups(float x, F f) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_max(float x) {
  return across_groups(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float group_add(float x) {
  return across_groups(x, [](float a, float b) { return a + b; });
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
    // (one unaligned access for the 8 was measured too, and is slower: dK and dV
    // of head size 77, 573 us against 329)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in && d0 + i < dim ? row[d0 + i] : (T)0.f;
  }
  return f;
}

// A lane's operand for chunk c of a row of `dim`.
template <typename T, bool ALN>
__device__ __forceinline__ Frag<T> load_head(const T* row, int c, int lane, int dim, bool in) {
  if constexpr (sizeof(T) == 2) {
    return load8<T, ALN>(row, c * 32 + (lane >> 4) * 8, dim, in);
  } else {
    Frag<T> f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d0 = c * 32 + h * 16 + (lane >> 4) * 4;
      f32x4 x{0.f, 0.f, 0.f, 0.f};
      if constexpr (ALN) {
        if (in && d0 < dim) x = *reinterpret_cast<const f32x4*>(row + d0);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in && d0 + i < dim) x[i] = row[d0 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) f[h * 4 + i] = x[i];
    }
    return f;
  }
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

// LDS tiles.  A bfloat16 tile is read by rows (8 lanes at a time take 16 bytes
// of one column of 8 rows) and by columns (16 lanes take 32 bytes of 4 rows).
// The 16-byte chunks of a row are exchanged by a number that differs over any
// 8 rows, and in its upper bits over any aligned 4, which spreads both over the
// banks without padding.  The column reads still count 4 conflict cycles each,
// 40% of the LDS cycles of the training kernels.  (Rows padded by 16 bytes took
// the same time, with the same conflicts and an eighth more LDS.)
// Float32 rows are padded by 16 bytes.
template <int DP>
constexpr int kCols = DP == 48 ? 64 : DP == 96 ? 128 : DP;  // columns that threads stage
template <typename T, int DP>
constexpr int kLd = sizeof(T) == 2 ? kCols<DP> : DP + 4;

template <int DP>
__device__ __forceinline__ int exchange(int row) {
  if constexpr (DP == 32)  // two rows to the 128 bytes of all banks
    return ((row >> 1 & 1) << 1) | (row >> 2 & 1);
  else
    return ((row & 3) << 1) | (row >> 2 & 1);
}

// Offset of 8 elements of a tile's row.
template <typename T, int DP>
__device__ __forceinline__ int chunk_at(int row, int chunk) {
  return row * kLd<T, DP> + (sizeof(T) == 2 ? chunk ^ exchange<DP>(row) : chunk) * 8;
}

// A lane's operand for chunk c of rows row0 .. row0 + 15.
template <int DP>
__device__ __forceinline__ bf16x8 read_rows(const __bf16* tile, int row0, int c, int lane) {
  return *reinterpret_cast<const bf16x8*>(tile + row0 * kLd<__bf16, DP> +
                                          chunk_at<__bf16, DP>(lane & 15, c * 4 + (lane >> 4)));
}
template <int DP>
__device__ __forceinline__ f32x8 read_rows(const float* tile, int row0, int c, int lane) {
  const float* p = tile + (row0 + (lane & 15)) * kLd<float, DP> + c * 32 + (lane >> 4) * 4;
  const f32x4 lo = *reinterpret_cast<const f32x4*>(p);
  f32x4 hi{0.f, 0.f, 0.f, 0.f};
  if (c * 32 + 16 < DP) hi = *reinterpret_cast<const f32x4*>(p + 16);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Column c0 + lane % 16 of 32 rows, in the slot order of pack().
template <int DP>
__device__ __forceinline__ bf16x8 read_cols(const __bf16* tile, int row0, int c0, int lane) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int row = (lane >> 4) * 4 + ((lane & 15) >> 2);
  const __bf16* p =
      tile + row0 * kLd<__bf16, DP> + chunk_at<__bf16, DP>(row, c0 / 8 + ((lane & 3) >> 1)) + (lane & 1) * 4;
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

}  // namespace
}  // namespace recis
