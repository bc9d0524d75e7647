// Layer norm over the rows of a matrix, one pass in each direction.  Per row, with
// mean over the width,
//   mu = mean x,  i = 1/sqrt(mean (x - mu)^2 + eps),  n = (x - mu) i,  y = n w + b
// backward, t = dy w:
//   dx = i (t - mean t - n mean(t n)),  dw = sum over the rows of dy n,  db = of dy
// A warp takes its own columns' mean off (they are in registers) and sums what is left
// and its squares; the mean of what is left is what the first one was off by, and the
// warps' means are joined as differences to one of them.  So a large mean costs n no
// digits, and a row takes one exchange between its warps.  (From statistics, the
// gradients' n is off by the rounding of the stored mean.)
//
// Bound by memory: x and y, or x, dy and dx, each once.  W warps hold a row; a CTA
// walks groups of rows, the next three rows' 16-byte pieces on their way while it works
// on the current one (rows.cuh).  The backward's column sums are kept by the
// threads over all rows of a CTA and added up, CTA by CTA in order, by a second
// kernel.  8192 x 2048 in bf16: 16.6 us forward and 31.0 with the gradients' second kernel
// (6), where the bytes at the copy rate take 10 and 15; in fp32 24.5 and 41.6 (20 and 30).
// Figures are of calls back to back on tensors larger than the caches.
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "persistent_grid.h"
#include "rows.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

using namespace rows;

// Rows on their way and worked on.  From flushed caches the gradients of 8192 x 2048 in
// bf16 take 32.4 us with four and 34.5 with two (the row kernel), the forward 18.8 with
// either; back to back 31.0 and 31.0, 16.6 and 16.0.  (Three in fp32, whose pieces are
// twice as long, for two CTAs an SM.)
template <typename T>
constexpr int kStagesOf = sizeof(T) == 2 ? 4 : 3;
template <int N>
__device__ __forceinline__ void cp_wait_row() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N - 1) : "memory");
}

// Pairs of a lane's elements are worked on by one instruction each (f32x2.cuh).
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
template <int L>
__device__ __forceinline__ float2 pair(const float (&x)[L], int e) { return make_float2(x[e], x[e + 1]); }
template <int L>
__device__ __forceinline__ void set_pair(float (&x)[L], int e, float2 v) {
  x[e] = v.x;
  x[e + 1] = v.y;
}
// v for elements e and e + 1, zero past the width (a vector is whole or not there)
template <typename T, bool VEC, int W>
__device__ __forceinline__ float2 inside(float v, int lane, int e, int width) {
  if constexpr (VEC) {
    constexpr int E = 16 / (int)sizeof(T);
    return both(column<T, VEC, W>(lane, e / E * E) < width ? v : 0.f);
  }
  return make_float2(column<T, VEC, W>(lane, e) < width ? v : 0.f,
                     column<T, VEC, W>(lane, e + 1) < width ? v : 0.f);
}

// Columns of a row that one of its warps has.
template <typename T, bool VEC, int W, int L>
__device__ __forceinline__ float warp_columns(int warp, int width) {
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
  int n = 0;
#pragma unroll
  for (int j = 0; j < L; j += E) n += min(max(width - (j / E * W + warp) * 32 * E, 0), 32 * E);
  return (float)n;
}

__device__ __forceinline__ float sum_warp(float sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Of a row: mean, 1 / sqrt(variance + eps), and what is to be added to x as it is left.
struct RowStats {
  float mean, inv, rest;
};
// x: zeros past the width, on return less the mean of the warp's own columns (zeros past
// the width).  red: [2][R][W] float4, alternated by the caller (buf).
template <typename T, bool VEC, int W, int L>
__device__ __forceinline__ RowStats row_stats(float (&x)[L], int lane, int width, float eps, float4* red,
                                              int buf, int group) {
  const int warp = lane >> 5;
  float2 sums = both(0.f);
#pragma unroll
  for (int e = 0; e < L; e += 2) sums = add2(sums, pair(x, e));
  const float n = warp_columns<T, VEC, W, L>(warp, width), inv_n = n > 0.f ? 1.f / n : 0.f;
  // The sum's rounding goes by the mean, what is left goes by the spread: its own mean is
  // what the first one was off by.
  const float off = sum_warp(sums.x + sums.y) * inv_n;
  float2 squares = sums = both(0.f);
#pragma unroll
  for (int e = 0; e < L; e += 2) {
    const float2 d = add2(pair(x, e), inside<T, VEC, W>(-off, lane, e, width));
    set_pair(x, e, d);
    sums = add2(sums, d);
    squares = fma2(d, d, squares);
  }
  const float more = sum_warp(sums.x + sums.y) * inv_n;
  float m2 = sum_warp(squares.x + squares.y), mean = off + more, rest = -more;
  if (m2 < INFINITY) m2 = fmaxf(fmaf(-n * more, more, m2), 0.f);
  if constexpr (W > 1) {
    // lane j: warp j's, as differences to the first warp's mean
    float4* r = red + (buf * Shape<W>::kRows + group) * W;
    if ((lane & 31) == 0) r[warp] = make_float4(off, more, m2, 0.f);
    __syncthreads();
    const int j = lane & (W - 1);
    const float4 theirs = r[j];
    const float first = r[0].x, m = warp_columns<T, VEC, W, L>(j, width);
    const float diff = (theirs.x - first) + theirs.y;
    float to = m * diff;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) to += __shfl_xor_sync(0xffffffffu, to, o);
    to /= (float)width;
    mean = first + to;
    rest = (off - first) - to;
    m2 = fmaf(m * (diff - to), diff - to, theirs.z);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
  }
  return {mean, 1.f / sqrtf(m2 / (float)width + eps), rest};
}

template <typename T, bool VEC, int W, int L>
__global__ void __launch_bounds__(Shape<W>::kThreads, W <= 8 ? 2 : 1) k_layer_norm_fwd(const LayerNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads, nT = Pieces<T, VEC, L>::n;
  constexpr bool S = VEC;
  constexpr int kStages = kStagesOf<T>;
  __shared__ float4 red[2 * R * W];
  extern __shared__ uint4 stage[];  // [kStages][piece][thread]
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const long long steps = (p.rows + R - 1) / R;
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    fetch<T, W, L>(stage + st * nT * NT + threadIdx.x, (const T*)p.x + (in ? row : 0) * p.x_stride, lane,
                in ? p.width : 0);
    cp_commit();
  };
  float w[L], b[L];
#pragma unroll
  for (int e = 0; e < L; ++e) {
    w[e] = 1.f;
    b[e] = 0.f;
  }
  if constexpr (S)
    for (int k = 0; k < kStages - 1; ++k) prefetch(blockIdx.x + (long long)k * gridDim.x, k);
  if (p.weight) load_row<T, VEC, W>(p.weight, lane, p.width, w);
  if (p.bias) load_row<T, VEC, W>(p.bias, lane, p.width, b);
  int st = 0, buf = 0;
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st = (st + 1) % kStages, buf ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float x[L];
    if constexpr (S) {
      prefetch(i + (long long)(kStages - 1) * gridDim.x, (st + kStages - 1) % kStages);
      cp_wait_row<kStages>();
      unpack<T, W>(stage + st * nT * NT + threadIdx.x, x);
    } else {
      load_row<T, VEC, W>((const T*)p.x + row * p.x_stride, lane, width, x);
    }
    const RowStats m = row_stats<T, VEC, W, L>(x, lane, p.width, p.eps, red, buf, group);
    const float2 rest = both(m.rest * m.inv), inv = both(m.inv);
#pragma unroll
    for (int e = 0; e < L; e += 2)
      set_pair(x, e, fma2(fma2(pair(x, e), inv, rest), pair(w, e), pair(b, e)));
    store_row<T, VEC, W>((T*)p.y + row * p.width, lane, width, x);
    if (p.stats && in && lane == 0) ((float2*)p.stats)[row] = make_float2(m.mean, m.inv);
  }
  if constexpr (S) cp_wait0();
}

// part: [grid][2][width] sums of dy n and of dy over a CTA's rows.
template <typename T, bool VEC, int W, int L>
__global__ void __launch_bounds__(Shape<W>::kThreads, W <= 8 ? 2 : 1) k_layer_norm_bwd(const LayerNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads, nT = Pieces<T, VEC, L>::n;
  constexpr bool S = VEC;
  constexpr int kStages = kStagesOf<T>;
  __shared__ float4 red2[2 * R * W];
  __shared__ __align__(16) float red[2 * 2 * R * W];
  extern __shared__ uint4 stage[];  // [kStages][x, dy][piece][thread]; after the rows [R][2][width]
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const float inv_w = 1.f / (float)p.width;
  const long long steps = (p.rows + R - 1) / R;
  auto slot = [&](int st, int at) { return stage + (st * 2 + at) * nT * NT + threadIdx.x; };
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    const long long r = in ? row : 0;
    const int width = in ? p.width : 0;
    fetch<T, W, L>(slot(st, 0), (const T*)p.x + r * p.x_stride, lane, width);
    fetch<T, W, L>(slot(st, 1), (const T*)p.dy + r * p.width, lane, width);
    cp_commit();
  };
  float w[L], cw[L], cb[L];
#pragma unroll
  for (int e = 0; e < L; ++e) {
    w[e] = 1.f;
    cw[e] = cb[e] = 0.f;
  }
  if constexpr (S)
    for (int k = 0; k < kStages - 1; ++k) prefetch(blockIdx.x + (long long)k * gridDim.x, k);
  if (p.weight) load_row<T, VEC, W>(p.weight, lane, p.width, w);
  int st = 0, buf = 0;
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st = (st + 1) % kStages, buf ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float x[L], dy[L], mean, inv;
    if (p.stats) {
      const float2 m = in ? ((const float2*)p.stats)[row] : make_float2(0.f, 0.f);
      mean = m.x;
      inv = m.y;
    }
    if constexpr (S) {
      prefetch(i + (long long)(kStages - 1) * gridDim.x, (st + kStages - 1) % kStages);
      cp_wait_row<kStages>();
      unpack<T, W>(slot(st, 0), x);
      unpack<T, W>(slot(st, 1), dy);
    } else {
      load_row<T, VEC, W>((const T*)p.x + row * p.x_stride, lane, width, x);
      load_row<T, VEC, W>((const T*)p.dy + row * p.width, lane, width, dy);
    }
    float rest = 0.f;  // without statistics n = x inv + rest, x less the warp's own mean
    if (!p.stats) {
      const RowStats m = row_stats<T, VEC, W, L>(x, lane, p.width, p.eps, red2, buf, group);
      inv = in ? m.inv : 0.f;
      rest = m.rest * inv;
    }
    const float2 inv2 = both(inv), rest2 = both(rest);
    float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
    for (int e = 0; e < L; e += 2) {
      const float2 n = p.stats ? mul2(add2(pair(x, e), both(-mean)), inv2) : fma2(pair(x, e), inv2, rest2);
      const float2 g = pair(dy, e), t = mul2(g, pair(w, e));  // (zero past the width, as dy is)
      set_pair(x, e, n);
      set_pair(dy, e, t);
      set_pair(cw, e, fma2(g, n, pair(cw, e)));
      set_pair(cb, e, add2(g, pair(cb, e)));
      s0 = add2(s0, t);
      s1 = fma2(t, n, s1);
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sums<W>(s, red, buf, group);
    const float2 a = both(-s[0] * inv_w * inv), c = both(-s[1] * inv_w * inv);
#pragma unroll
    for (int e = 0; e < L; e += 2)  // inv (t - mean t - n mean(t n))
      set_pair(x, e, fma2(pair(dy, e), inv2, fma2(pair(x, e), c, a)));
    store_row<T, VEC, W>((T*)p.dx + row * p.width, lane, width, x);
  }
  // (the kernel behind this one is the sum over `part`, which waits for its end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (S) cp_wait0();
  float* part = p.part + (size_t)blockIdx.x * 2 * p.width;
  if constexpr (R == 1) {
#pragma unroll
    for (int e = 0; e < L; ++e) {
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
    for (int e = 0; e < L; ++e) {
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
  // (launched while the kernel that writes `part` runs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int j = threadIdx.x & 31, sl = threadIdx.x >> 5, which = blockIdx.y;
  const int c = blockIdx.x * 32 + j;
  float* out = which ? p.dbias : p.dweight;
  if (!out) return;
  float a = 0.f;
  if (c < p.width)
#pragma unroll 8
    for (int i = sl; i < ncta; i += kSlices) a += p.part[((size_t)i * 2 + which) * p.width + c];
  sum[sl][j] = a;
  __syncthreads();
  if (sl == 0 && c < p.width) {
    a = 0.f;
    for (int i = 0; i < kSlices; ++i) a += sum[i][j];
    out[c] = a;
  }
}

template <typename T, bool VEC, int W, int L>
cudaError_t forward(const LayerNorm& p, cudaStream_t s) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  constexpr size_t smem = (size_t)kStagesOf<T> * Pieces<T, VEC, L>::n * NT * 16;
  static FitOf fit;
  int grid = 1;
  const cudaError_t e = persistent_grid(k_layer_norm_fwd<T, VEC, W, L>, NT, smem, (p.rows + R - 1) / R,
                                        1 << 20, &fit, &grid);
  if (e != cudaSuccess) return e;
  LaunchScope ls("layer_norm_fwd", s);
  k_layer_norm_fwd<T, VEC, W, L><<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}
template <typename T, bool VEC, int W, int L>
cudaError_t backward(const LayerNorm& p, int* grid, cudaStream_t s) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  constexpr size_t staged = (size_t)kStagesOf<T> * 2 * Pieces<T, VEC, L>::n * NT * 16;
  // the widest row's column sums
  constexpr size_t cols = R > 1 ? (size_t)R * 2 * W * 32 * L * sizeof(float) : 0;
  constexpr size_t smem = staged > cols ? staged : cols;
  static FitOf fit;
  const cudaError_t e = persistent_grid(k_layer_norm_bwd<T, VEC, W, L>, NT, smem, (p.rows + R - 1) / R,
                                        kLayerNormMaxCtas, &fit, grid);
  if (e != cudaSuccess) return e;
  LaunchScope ls("layer_norm_bwd", s);
  k_layer_norm_bwd<T, VEC, W, L><<<*grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}

// Elements of a lane and warps of a row by its width: at eight elements what a warp does
// once a row (the sums over its lanes, the row's statistics) is more than their work
// (8192 x 2048 bf16: 21.2 us forward, 16.6 with 32 on two warps).  The backward has five
// values an element in registers, the forward three.  A forward of few rows has no such
// choice: rows on few warps leave SMs idle, and a row's own time counts (250 x 1537 in
// fp32: 4.3 us with eight elements, 6.3 with 32).
template <typename T, bool VEC>
cudaError_t launch(const LayerNorm& p, bool back, int* grid, cudaStream_t s) {
  const int w = p.width;
  if (back) {
    if (w <= 256) return backward<T, VEC, 1, 8>(p, grid, s);
    if (w <= 512) return backward<T, VEC, 1, 16>(p, grid, s);
    if (w <= 1024) return backward<T, VEC, 2, 16>(p, grid, s);
    if (w <= 2048) return backward<T, VEC, 4, 16>(p, grid, s);
    if (w <= 4096) return backward<T, VEC, 8, 16>(p, grid, s);
    return backward<T, VEC, 16, 16>(p, grid, s);
  }
  if (w <= 256) return forward<T, VEC, 1, 8>(p, s);
  if (p.rows < 4 * kLaSms) {
    if (w <= 512) return forward<T, VEC, 2, 8>(p, s);
    if (w <= 1024) return forward<T, VEC, 4, 8>(p, s);
    if (w <= 2048) return forward<T, VEC, 8, 8>(p, s);
    if (w <= 4096) return forward<T, VEC, 16, 8>(p, s);
    return forward<T, VEC, 32, 8>(p, s);
  }
  if (w <= 512) return forward<T, VEC, 1, 16>(p, s);
  if (w <= 1024) return forward<T, VEC, 1, 32>(p, s);
  if (w <= 2048) return forward<T, VEC, 2, 32>(p, s);
  if (w <= 4096) return forward<T, VEC, 4, 32>(p, s);
  return forward<T, VEC, 8, 32>(p, s);
}

cudaError_t dispatch(const LayerNorm& p, bool bf16, bool back, int* grid, cudaStream_t s) {
  // 16-byte vectors need every row of every tensor to start on such a boundary
  // and the width to be whole vectors; other rows go element by element, with nothing on
  // its way ahead (8192 x 2049: 55 us forward and 58 backward in bf16, 35 and 51 in fp32)
  const int unit = bf16 ? 8 : 4;
  bool vec = p.width % unit == 0 && p.x_stride % unit == 0;
  const void* ptrs[] = {p.x, p.weight, p.bias, p.y, p.dy, p.dx};
  for (const void* q : ptrs) vec = vec && ((uintptr_t)q & 15u) == 0;
  if (bf16)
    return vec ? launch<__nv_bfloat16, true>(p, back, grid, s)
               : launch<__nv_bfloat16, false>(p, back, grid, s);
  return vec ? launch<float, true>(p, back, grid, s) : launch<float, false>(p, back, grid, s);
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
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((p.width + 31) / 32, 2);
  c.blockDim = dim3(32 * kSlices);
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k_layer_norm_dw, grid, p);
}

}  // namespace ssd
