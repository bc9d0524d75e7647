// Layer norm over the rows of a matrix, one pass in each direction.  Per row, with
// mean over the width,
//   mu = mean x,  i = 1/sqrt(mean (x - mu)^2 + eps),  n = (x - mu) i,  y = n w + b
// backward, t = dy w:
//   dx = i (t - mean t - n mean(t n)),  dw = sum over the rows of dy n,  db = of dy
// The mean is taken off before the squares are summed (the row is in registers), so
// that a large mean costs no digits.
//
// Bound by memory: x and y, or x, dy and dx, each once.  W warps hold a row; a CTA
// walks groups of rows, the next row's 16-byte pieces on their way while it works
// on the current one (rows.cuh).  The backward's column sums are kept by the
// threads over all rows of a CTA and added up, CTA by CTA in order, by a second
// kernel.
#include <cuda_bf16.h>

#include "persistent_grid.h"
#include "rows.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

using namespace rows;

template <typename T, bool VEC, int W>
__global__ void __launch_bounds__(Shape<W>::kThreads) k_layer_norm_fwd(const LayerNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads, nT = Pieces<T, VEC>::n;
  constexpr bool S = kStaged<VEC, W>;
  __shared__ __align__(16) float red[2 * R * W];
  extern __shared__ uint4 stage[];  // [2][piece][thread]
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const float inv_w = 1.f / (float)p.width;
  const long long steps = (p.rows + R - 1) / R;
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    fetch<T, W>(stage + st * nT * NT + threadIdx.x, (const T*)p.x + (in ? row : 0) * p.x_stride, lane,
                in ? p.width : 0);
    cp_commit();
  };
  float w[kL], b[kL];
#pragma unroll
  for (int e = 0; e < kL; ++e) {
    w[e] = 1.f;
    b[e] = 0.f;
  }
  if (p.weight) load_row<T, VEC, W>(p.weight, lane, p.width, w);
  if (p.bias) load_row<T, VEC, W>(p.bias, lane, p.width, b);
  int st = 0;
  if constexpr (S) prefetch(blockIdx.x, 0);
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float x[kL];
    if constexpr (S) {
      prefetch(i + gridDim.x, st ^ 1);
      cp_wait1();
      unpack<T, W>(stage + st * nT * NT + threadIdx.x, x);
    } else {
      load_row<T, VEC, W>((const T*)p.x + row * p.x_stride, lane, width, x);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < kL; ++e) s[0] += x[e];
    row_sums<W>(s, red, 0, group);
    const float mean = s[0] * inv_w;
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      x[e] -= mean;
      if (column<T, VEC, W>(lane, e) < p.width) s[0] = fmaf(x[e], x[e], s[0]);
    }
    row_sums<W>(s, red, 1, group);
    const float inv = 1.f / sqrtf(s[0] * inv_w + p.eps);
#pragma unroll
    for (int e = 0; e < kL; ++e) x[e] = fmaf(x[e] * inv, w[e], b[e]);
    store_row<T, VEC, W>((T*)p.y + row * p.width, lane, width, x);
    if (p.stats && in && lane == 0) ((float2*)p.stats)[row] = make_float2(mean, inv);
  }
  if constexpr (S) cp_wait0();
}

// part: [grid][2][width] sums of dy n and of dy over a CTA's rows.
template <typename T, bool VEC, int W>
__global__ void __launch_bounds__(Shape<W>::kThreads) k_layer_norm_bwd(const LayerNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads, nT = Pieces<T, VEC>::n;
  constexpr bool S = kStaged<VEC, W>;
  __shared__ __align__(16) float red[3 * 2 * R * W];
  extern __shared__ uint4 stage[];  // [2][x, dy][piece][thread]; after the rows [R][2][width]
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const float inv_w = 1.f / (float)p.width;
  const long long steps = (p.rows + R - 1) / R;
  auto slot = [&](int st, int at) { return stage + (st * 2 + at) * nT * NT + threadIdx.x; };
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    const long long r = in ? row : 0;
    const int width = in ? p.width : 0;
    fetch<T, W>(slot(st, 0), (const T*)p.x + r * p.x_stride, lane, width);
    fetch<T, W>(slot(st, 1), (const T*)p.dy + r * p.width, lane, width);
    cp_commit();
  };
  float w[kL], cw[kL], cb[kL];
#pragma unroll
  for (int e = 0; e < kL; ++e) {
    w[e] = 1.f;
    cw[e] = cb[e] = 0.f;
  }
  if (p.weight) load_row<T, VEC, W>(p.weight, lane, p.width, w);
  int st = 0;
  if constexpr (S) prefetch(blockIdx.x, 0);
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float x[kL], dy[kL], mean, inv;
    if (p.stats) {
      const float2 m = in ? ((const float2*)p.stats)[row] : make_float2(0.f, 0.f);
      mean = m.x;
      inv = m.y;
    }
    if constexpr (S) {
      prefetch(i + gridDim.x, st ^ 1);
      cp_wait1();
      unpack<T, W>(slot(st, 0), x);
      unpack<T, W>(slot(st, 1), dy);
    } else {
      load_row<T, VEC, W>((const T*)p.x + row * p.x_stride, lane, width, x);
      load_row<T, VEC, W>((const T*)p.dy + row * p.width, lane, width, dy);
    }
    if (!p.stats) {
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < kL; ++e) s[0] += x[e];
      row_sums<W>(s, red, 0, group);
      mean = s[0] * inv_w;
      s[0] = 0.f;
#pragma unroll
      for (int e = 0; e < kL; ++e) {
        const float d = x[e] - mean;
        if (column<T, VEC, W>(lane, e) < p.width) s[0] = fmaf(d, d, s[0]);
      }
      row_sums<W>(s, red, 1, group);
      inv = in ? 1.f / sqrtf(s[0] * inv_w + p.eps) : 0.f;
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      x[e] = (x[e] - mean) * inv;
      cw[e] = fmaf(dy[e], x[e], cw[e]);
      cb[e] += dy[e];
      dy[e] *= w[e];  // (zero past the width, as dy is)
      s[0] += dy[e];
      s[1] = fmaf(dy[e], x[e], s[1]);
    }
    row_sums<W>(s, red + 2 * R * W, st, group);
    const float a = s[0] * inv_w, c = s[1] * inv_w;
#pragma unroll
    for (int e = 0; e < kL; ++e) x[e] = inv * (dy[e] - fmaf(x[e], c, a));
    store_row<T, VEC, W>((T*)p.dx + row * p.width, lane, width, x);
  }
  if constexpr (S) cp_wait0();
  float* part = p.part + (size_t)blockIdx.x * 2 * p.width;
  if constexpr (R == 1) {
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      const int c = column<T, VEC, W>(lane, e);
      if (c < p.width) {
        part[c] = cw[e];
        part[p.width + c] = cb[e];
      }
    }
  } else {
    float* cols = (float*)stage;
    __syncthreads();  // every thread has read its last row
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      const int c = column<T, VEC, W>(lane, e);
      if (c < p.width) {
        cols[(group * 2) * p.width + c] = cw[e];
        cols[(group * 2 + 1) * p.width + c] = cb[e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.width; c += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < R; ++g) t += cols[g * 2 * p.width + c];
      part[c] = t;
    }
  }
}

// The CTAs' partial rows summed in order: a CTA takes 32 columns of dw or db, 32
// slices of the partials each, then the slices in order.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) k_layer_norm_dw(int ncta, LayerNorm p) {
  __shared__ float sum[kSlices][33];
  const int j = threadIdx.x & 31, sl = threadIdx.x >> 5, which = blockIdx.y;
  const int c = blockIdx.x * 32 + j;
  float* out = which ? p.dbias : p.dweight;
  if (!out) return;
  float a = 0.f;
  if (c < p.width)
    for (int i = sl; i < ncta; i += kSlices) a += p.part[((size_t)i * 2 + which) * p.width + c];
  sum[sl][j] = a;
  __syncthreads();
  if (sl == 0 && c < p.width) {
    a = 0.f;
    for (int i = 0; i < kSlices; ++i) a += sum[i][j];
    out[c] = a;
  }
}

template <typename T, bool VEC, int W>
cudaError_t launch(const LayerNorm& p, bool backward, int* grid_out, cudaStream_t s) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  const long long steps = (p.rows + R - 1) / R;
  int grid = 1;
  constexpr size_t one = kStaged<VEC, W> ? (size_t)2 * Pieces<T, VEC>::n * NT * 16 : 0;
  if (!backward) {
    static FitOf fit;
    const cudaError_t e =
        persistent_grid(k_layer_norm_fwd<T, VEC, W>, NT, one, steps, 1 << 20, &fit, &grid);
    if (e != cudaSuccess) return e;
    LaunchScope ls("layer_norm_fwd", s);
    k_layer_norm_fwd<T, VEC, W><<<grid, NT, one, s>>>(p);
    return cudaGetLastError();
  }
  // the widest row's column sums
  constexpr size_t cols = R > 1 ? (size_t)R * 2 * W * 32 * kL * sizeof(float) : 0;
  constexpr size_t smem = 2 * one > cols ? 2 * one : cols;
  static FitOf fit;
  const cudaError_t e = persistent_grid(k_layer_norm_bwd<T, VEC, W>, NT, smem, steps,
                                        kLayerNormMaxCtas, &fit, &grid);
  if (e != cudaSuccess) return e;
  *grid_out = grid;
  LaunchScope ls("layer_norm_bwd", s);
  k_layer_norm_bwd<T, VEC, W><<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_w(const LayerNorm& p, bool backward, int* grid, cudaStream_t s) {
  const int w = (p.width + 32 * kL - 1) / (32 * kL);  // warps that a row needs
  if (w <= 1) return launch<T, VEC, 1>(p, backward, grid, s);
  if (w <= 2) return launch<T, VEC, 2>(p, backward, grid, s);
  if (w <= 4) return launch<T, VEC, 4>(p, backward, grid, s);
  if (w <= 8) return launch<T, VEC, 8>(p, backward, grid, s);
  if (w <= 16) return launch<T, VEC, 16>(p, backward, grid, s);
  return launch<T, VEC, 32>(p, backward, grid, s);
}

cudaError_t dispatch(const LayerNorm& p, bool bf16, bool backward, int* grid, cudaStream_t s) {
  // 16-byte vectors need every row of every tensor to start on such a boundary
  // and the width to be whole vectors
  const int unit = bf16 ? 8 : 4;
  bool vec = p.width % unit == 0 && p.x_stride % unit == 0;
  const void* ptrs[] = {p.x, p.weight, p.bias, p.y, p.dy, p.dx};
  for (const void* q : ptrs) vec = vec && ((uintptr_t)q & 15u) == 0;
  if (bf16)
    return vec ? launch_w<__nv_bfloat16, true>(p, backward, grid, s)
               : launch_w<__nv_bfloat16, false>(p, backward, grid, s);
  return vec ? launch_w<float, true>(p, backward, grid, s) : launch_w<float, false>(p, backward, grid, s);
}

}  // namespace

cudaError_t layer_norm_forward(const LayerNorm& p, bool bf16, cudaStream_t s) {
  return dispatch(p, bf16, false, nullptr, s);
}

cudaError_t layer_norm_backward(const LayerNorm& p, bool bf16, cudaStream_t s) {
  int grid = 1;
  const cudaError_t e = dispatch(p, bf16, true, &grid, s);
  if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
  LaunchScope ls("layer_norm_dw", s);
  k_layer_norm_dw<<<dim3((p.width + 31) / 32, 2), 32 * kSlices, 0, s>>>(grid, p);
  return cudaGetLastError();
}

}  // namespace ssd
