// Rows of a matrix held in registers by W warps each, eight elements or more a lane: loads,
// stores, sums over a row, and the asynchronous copies of the next row.  Used by
// the norms.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_common.cuh"

namespace ssd {
namespace rows {

constexpr int kL = 8;  // elements of a lane where a kernel takes no other number (L)

template <int W>
struct Shape {
  static constexpr int kRows = W >= 8 ? 1 : 8 / W;  // rows of a CTA at a time
  static constexpr int kThreads = kRows * W * 32;
};

// Column of element i of a lane (`lane` counts over the row's W warps): VEC
// lanes hold 16-byte vectors that are contiguous over the lanes.
template <typename T, bool VEC, int W>
__device__ __forceinline__ int column(int lane, int i) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
  return ((i / E) * W * 32 + lane) * E + i % E;
}

// v[i] = row[column(i)], zero past the width.  In the vector case the width is
// a multiple of the vector; U: the type of the column rule (that of y), T: the
// type of the row, whose vectors may be twice as long.
template <typename U, bool VEC, int W, typename T, int L>
__device__ __forceinline__ void load_row(const T* row, int lane, int width, float (&v)[L]) {
  if constexpr (VEC) {
    constexpr int E = 16 / (int)sizeof(U);
#pragma unroll
    for (int j = 0; j < L; j += E) {
      const int c = column<U, VEC, W>(lane, j);
      if (c < width) {
        if constexpr (sizeof(T) == 2) {
          const uint4 q = *(const uint4*)(row + c);
          const __nv_bfloat162* h = (const __nv_bfloat162*)&q;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            v[j + 2 * i] = f.x;
            v[j + 2 * i + 1] = f.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; i += 4) {
            const float4 f = *(const float4*)(row + c + i);
            v[j + i] = f.x; v[j + i + 1] = f.y; v[j + i + 2] = f.z; v[j + i + 3] = f.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[j + i] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = column<U, VEC, W>(lane, i);
      v[i] = c < width ? to_f32(row[c]) : 0.f;
    }
  }
}

template <typename U, bool VEC, int W, typename T, int L>
__device__ __forceinline__ void store_row(T* row, int lane, int width, const float (&v)[L]) {
  if constexpr (VEC) {
    constexpr int E = 16 / (int)sizeof(U);
#pragma unroll
    for (int j = 0; j < L; j += E) {
      const int c = column<U, VEC, W>(lane, j);
      if (c >= width) continue;
      if constexpr (sizeof(T) == 2) {
        uint4 q;
        __nv_bfloat162* h = (__nv_bfloat162*)&q;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
        *(uint4*)(row + c) = q;
      } else {
#pragma unroll
        for (int i = 0; i < E; i += 4)
          *(float4*)(row + c + i) = make_float4(v[j + i], v[j + i + 1], v[j + i + 2], v[j + i + 3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = column<U, VEC, W>(lane, i);
      if (c < width) row[c] = from_f32<T>(v[i]);
    }
  }
}

// Sums of NV values over the W warps of a row, the warps' totals added in
// order.  red: [2][rows][W][NV] floats, alternated by the caller (buf).
template <int W, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* red, int buf, int group) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (W > 1) {
    const int warp = (threadIdx.x >> 5) % W;
    float* r = red + ((buf * Shape<W>::kRows + group) * W) * NV;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i * W + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) t += r[i * W + j];
      v[i] = t;
    }
  }
}

// One operand's eight elements of a lane as they come from memory: 16-byte
// pieces in the vector case.  The vector case copies the next row's pieces into
// shared memory (cp.async, two stages) while the current row is worked on; a
// thread reads back only what it copied itself.
template <typename T, bool VEC, int L = kL>
struct Pieces {
  static constexpr int n = VEC ? L * (int)sizeof(T) / 16 : 0;
};
// (not for CTAs of 1024 threads: two stages of a norm's backward do not fit beside
// the weights in a CTA's shared memory, and its forward follows the same rule)
template <bool VEC, int W>
constexpr bool kStaged = VEC && W < 32;

__device__ __forceinline__ void cp_async16(uint4* smem, const void* gmem, bool in) {
  // (0 bytes of the source: zeros are written)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (unsigned)__cvta_generic_to_shared(smem)),
               "l"(gmem), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void cp_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// The pieces of a row into slots [piece][thread]; U: the type of the column rule.
template <typename U, int W, int L = kL, typename T>
__device__ __forceinline__ void fetch(uint4* slot, const T* row, int lane, int width) {
#pragma unroll
  for (int i = 0; i < Pieces<T, true, L>::n; ++i) {
    const int c = column<U, true, W>(lane, i * (16 / (int)sizeof(T)));
    const bool in = c < width;
    cp_async16(slot + i * Shape<W>::kThreads, in ? row + c : row, in);
  }
}
template <typename T, int W, int L>
__device__ __forceinline__ void unpack(const uint4* slot, float (&v)[L]) {
#pragma unroll
  for (int i = 0; i < Pieces<T, true, L>::n; ++i) {
    const uint4 q = slot[i * Shape<W>::kThreads];
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162* h = (const __nv_bfloat162*)&q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __bfloat1622float2(h[j]);
        v[8 * i + 2 * j] = f.x;
        v[8 * i + 2 * j + 1] = f.y;
      }
    } else {
      const float4 f = *(const float4*)&q;
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  }
}

}  // namespace rows
}  // namespace ssd
