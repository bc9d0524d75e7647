// Norms before and after a block with its gate and residual scale, one pass
// over the rows in each direction.  Per row, with mean over the width,
//   iy = 1/sqrt(mean y^2 + eps),  n = y iy,  s = silu(z)
//   r' = r + alpha n w_post s,    ir = 1/sqrt(mean r'^2 + eps),  x = r' ir w_pre
// backward, from dx and dn (the gradient that reaches r' on later paths):
//   t  = dx w_pre,  dr = dn + ir t - r' ir^3 mean(t r')
//   e  = alpha dr,  dz = e n w_post silu'(z)
//   q  = e s w_post,  dy = iy q - y iy^3 mean(q y)
//   over the rows: c = sum dr n s,  dw_post = alpha c,  dalpha = w_post c,
//   dw_pre = sum dx r' ir
// (alpha and w_post are constants of a column, so one column sum serves both
// of their gradients).
//
// Bound by memory: the forward moves r, y, z, r', x, the backward y, z, r',
// dx, dn, dr, dy, dz, each once.  W warps hold a row, eight elements a lane in
// registers; a CTA of 256 threads or more walks groups of rows, the next row's
// 16-byte pieces on their way while it works on the current one, up to 4096
// columns and where the rows are aligned for that; else what a row needs is
// loaded when its turn comes, unaligned rows element by element.  Measured on
// 8192 x 2048 bf16 with an fp32 residual: 48 us forward (72 % of the copy rate),
// 91 us backward with its column sums (60 %).
//
// Device times of the other variants (bf16, fp32 residual; forward, backward;
// 52 and 97 us for 8192 x 2048 measured so).
//   2048 x 8192, 1024 threads without stages: 70 and 128.  Two stages of the
//   backward do not fit beside the weights in the 227 KB of a CTA; the forward's
//   would (56 us), it follows the same rule.  The backward, at 64 registers a
//   thread, keeps its column sums in shared memory and spills up to 176 bytes.
//   Unaligned rows are built for 1, 4 and 32 warps alone: 16384 x 1023 on four
//   takes 83 and 109, 2048 x 8191 on 32 83 and 154; widths between pay for idle
//   warps (8192 x 2047 on 32: 226 and 404, where eight would take 80 and 108;
//   16384 x 511 on four: 74 and 85, on two 44 and 62).
#include <cuda_bf16.h>

#include "persistent_grid.h"
#include "rows.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

using namespace rows;

// 1 / (1 + e^-z) for a gate of type T.  fp32 gates take the exact functions.
// bf16 gates, which are rounded by up to 2^-8 themselves, take the hardware's
// base-2 exponential and reciprocal: the rounding of z log2 e is |z| 2^-24 of the
// result, 2^-18 at z = -80 (2^(+large) = inf gives 0, 2^(-large) = 0 gives 1).
// Measured on 8192 x 2048, bf16 with a bf16 residual: 33 us forward and 64 us
// backward, with the exact functions 40 and 75; in fp32, which more bytes bound,
// 60 and 102, exactly 62 and 103.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 4) {
    return 1.f / (1.f + expf(-z));
  } else {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
  }
}

template <typename T, typename TR, bool VEC, int W>
__global__ void __launch_bounds__(Shape<W>::kThreads) k_block_norm_fwd(const BlockNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  constexpr bool S = kStaged<VEC, W>;
  constexpr int nT = Pieces<T, VEC>::n, nR = Pieces<TR, VEC>::n, nS = 2 * nT + nR;
  __shared__ __align__(16) float red[2 * 2 * R * W];
  extern __shared__ uint4 stage[];  // [2][y, z, residual][piece][thread]
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const float inv_w = 1.f / (float)p.width;
  const long long steps = (p.rows + R - 1) / R;
  auto slot = [&](int st, int at) { return stage + (st * nS + at) * NT + threadIdx.x; };
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    const long long r = in ? row : 0;
    const int width = in ? p.width : 0;
    fetch<T, W>(slot(st, 0), (const T*)p.y + r * p.y_stride, lane, width);
    if (p.z) fetch<T, W>(slot(st, nT), (const T*)p.z + r * p.z_stride, lane, width);
    fetch<T, W>(slot(st, 2 * nT), (const TR*)p.residual + r * p.width, lane, width);
    cp_commit();
  };
  float wa[kL], wq[kL];  // res_scale w_post, w_pre
  load_row<T, VEC, W>(p.w_post, lane, p.width, wa);
  if (p.res_scale) {
    load_row<T, VEC, W>(p.res_scale, lane, p.width, wq);
#pragma unroll
    for (int e = 0; e < kL; ++e) wa[e] *= wq[e];
  }
  load_row<T, VEC, W>(p.w_pre, lane, p.width, wq);
  int st = 0;
  if constexpr (S) prefetch(blockIdx.x, 0);
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float y[kL], z[kL], r[kL];
    if constexpr (S) {
      prefetch(i + gridDim.x, st ^ 1);
      cp_wait1();
      unpack<T, W>(slot(st, 0), y);
      if (p.z) unpack<T, W>(slot(st, nT), z);
      unpack<TR, W>(slot(st, 2 * nT), r);
    } else {
      load_row<T, VEC, W>((const T*)p.y + row * p.y_stride, lane, width, y);
      if (p.z) load_row<T, VEC, W>((const T*)p.z + row * p.z_stride, lane, width, z);
      load_row<T, VEC, W>((const TR*)p.residual + row * p.width, lane, width, r);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < kL; ++e) s[0] = fmaf(y[e], y[e], s[0]);
    if (p.z)
#pragma unroll
      for (int e = 0; e < kL; ++e) y[e] *= z[e] * sigmoid<T>(z[e]);
    row_sums<W>(s, red, 0, group);
    const float iy = 1.f / sqrtf(s[0] * inv_w + p.eps);
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      r[e] = fmaf(y[e] * iy, wa[e], r[e]);
      s[0] = fmaf(r[e], r[e], s[0]);
    }
    store_row<T, VEC, W>((TR*)p.new_residual + row * p.width, lane, width, r);
    row_sums<W>(s, red, 1, group);
    const float ir = 1.f / sqrtf(s[0] * inv_w + p.eps);
#pragma unroll
    for (int e = 0; e < kL; ++e) r[e] *= ir * wq[e];
    store_row<T, VEC, W>((T*)p.x + row * p.width, lane, width, r);
    if (p.stats && in && lane == 0) ((float2*)p.stats)[row] = make_float2(iy, ir);
  }
  if constexpr (S) cp_wait0();
}

// part: [grid][2][width] sums of dr n s and of dx r' ir over a CTA's rows.
template <typename T, typename TR, bool VEC, int W>
__global__ void __launch_bounds__(Shape<W>::kThreads, W <= 8 ? 3 : 1) k_block_norm_bwd(const BlockNorm p) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  constexpr bool S = kStaged<VEC, W>;
  constexpr int nT = Pieces<T, VEC>::n, nR = Pieces<TR, VEC>::n, nS = 3 * nT + 2 * nR;
  __shared__ __align__(16) float red[2 * 3 * R * W];
  // [2][8][lane of the row]: w_pre, res_scale w_post by element, then
  // [2][y, z, dx, r', dn][piece][thread]; after the rows [R][2][width] (R > 1)
  extern __shared__ uint4 shared[];
  constexpr int NL = W * 32;
  float* weights = (float*)shared;
  uint4* stage = shared + 2 * kL * NL / 4;
  const int group = threadIdx.x / (W * 32), lane = threadIdx.x % (W * 32);
  const float inv_w = 1.f / (float)p.width;
  const long long steps = (p.rows + R - 1) / R;
  auto slot = [&](int st, int at) { return stage + (st * nS + at) * NT + threadIdx.x; };
  auto prefetch = [&](long long i, int st) {
    const long long row = i * R + group;
    const bool in = i < steps && row < p.rows;
    const long long r = in ? row : 0;
    const int width = in ? p.width : 0;
    fetch<T, W>(slot(st, 0), (const T*)p.y + r * p.y_stride, lane, width);
    if (p.z) fetch<T, W>(slot(st, nT), (const T*)p.z + r * p.z_stride, lane, width);
    fetch<T, W>(slot(st, 2 * nT), (const T*)p.dx + r * p.width, lane, width);
    fetch<T, W>(slot(st, 3 * nT), (const TR*)p.residual + r * p.width, lane, width);
    if (p.dnew) fetch<T, W>(slot(st, 3 * nT + nR), (const TR*)p.dnew + r * p.width, lane, width);
    cp_commit();
  };
  // the column sums: registers, or for rows of 1024 threads (64 registers each)
  // shared memory, [sum][element][thread]
  constexpr int nA = W == 32 ? 1 : kL;
  float cp[nA], cq[nA];
  float* sums = (float*)stage + threadIdx.x;
#pragma unroll
  for (int e = 0; e < kL; ++e) {
    if constexpr (W == 32) sums[e * NT] = sums[(kL + e) * NT] = 0.f;
    else cp[e] = cq[e] = 0.f;
  }
  auto add_p = [&](int e, float a, float b) {
    if constexpr (W == 32) sums[e * NT] = fmaf(a, b, sums[e * NT]);
    else cp[e] = fmaf(a, b, cp[e]);
  };
  auto add_q = [&](int e, float a, float b) {
    if constexpr (W == 32) sums[(kL + e) * NT] = fmaf(a, b, sums[(kL + e) * NT]);
    else cq[e] = fmaf(a, b, cq[e]);
  };
  int st = 0;
  if constexpr (S) prefetch(blockIdx.x, 0);
  if (group == 0) {
    float a[kL], q[kL], al[kL];
    load_row<T, VEC, W>(p.w_post, lane, p.width, a);
    load_row<T, VEC, W>(p.w_pre, lane, p.width, q);
    if (p.res_scale) load_row<T, VEC, W>(p.res_scale, lane, p.width, al);
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      weights[e * NL + lane] = q[e];
      weights[(kL + e) * NL + lane] = p.res_scale ? a[e] * al[e] : a[e];
    }
  }
  __syncthreads();
  for (long long i = blockIdx.x; i < steps; i += gridDim.x, st ^= 1) {
    const long long row = i * R + group;
    const bool in = row < p.rows;
    const int width = in ? p.width : 0;
    float y[kL], r[kL], dx[kL], dr[kL], w[kL];
    if constexpr (S) {
      prefetch(i + gridDim.x, st ^ 1);
      cp_wait1();
      unpack<T, W>(slot(st, 0), y);
      unpack<T, W>(slot(st, 2 * nT), dx);
      unpack<TR, W>(slot(st, 3 * nT), r);
      if (p.dnew) unpack<TR, W>(slot(st, 3 * nT + nR), dr);
    } else {
      load_row<T, VEC, W>((const T*)p.y + row * p.y_stride, lane, width, y);
      load_row<T, VEC, W>((const T*)p.dx + row * p.width, lane, width, dx);
      load_row<T, VEC, W>((const TR*)p.residual + row * p.width, lane, width, r);
      if (p.dnew) load_row<T, VEC, W>((const TR*)p.dnew + row * p.width, lane, width, dr);
    }
    if (!p.dnew)
#pragma unroll
      for (int e = 0; e < kL; ++e) dr[e] = 0.f;
#pragma unroll
    for (int e = 0; e < kL; ++e) w[e] = weights[e * NL + lane];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      s[0] = fmaf(dx[e] * w[e], r[e], s[0]);
      s[1] = fmaf(r[e], r[e], s[1]);
      s[2] = fmaf(y[e], y[e], s[2]);
    }
    row_sums<W>(s, red, 0, group);
    float ir, iy;
    if (p.stats) {
      const float2 stt = in ? ((const float2*)p.stats)[row] : make_float2(0.f, 0.f);
      iy = stt.x;
      ir = stt.y;
    } else {
      ir = 1.f / sqrtf(s[1] * inv_w + p.eps);
      iy = 1.f / sqrtf(s[2] * inv_w + p.eps);
    }
    const float kr = s[0] * inv_w * ir * ir * ir;
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      dr[e] += fmaf(ir * dx[e], w[e], -kr * r[e]);
      add_q(e, dx[e] * ir, r[e]);
    }
    store_row<T, VEC, W>((TR*)p.dresidual + row * p.width, lane, width, dr);
    // from here w = res_scale w_post, dx = dr n with n = y iy
#pragma unroll
    for (int e = 0; e < kL; ++e) w[e] = weights[(kL + e) * NL + lane];
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      dx[e] = dr[e] * y[e] * iy;
      dr[e] *= w[e];
    }
    float t[1] = {0.f};
    if (p.z) {
      if constexpr (S) unpack<T, W>(slot(st, nT), r);
      else load_row<T, VEC, W>((const T*)p.z + row * p.z_stride, lane, width, r);
#pragma unroll
      for (int e = 0; e < kL; ++e) {
        const float sg = sigmoid<T>(r[e]), g = r[e] * sg;
        add_p(e, dx[e], g);
        dx[e] *= w[e] * (sg * fmaf(r[e], 1.f - sg, 1.f));
        dr[e] *= g;
        t[0] = fmaf(dr[e], y[e], t[0]);
      }
      store_row<T, VEC, W>((T*)p.dz + row * p.width, lane, width, dx);
    } else {
#pragma unroll
      for (int e = 0; e < kL; ++e) {
        add_p(e, dx[e], 1.f);
        t[0] = fmaf(dr[e], y[e], t[0]);
      }
    }
    row_sums<W>(t, red + 3 * R * W, 0, group);
    const float ky = t[0] * inv_w * iy * iy * iy;
#pragma unroll
    for (int e = 0; e < kL; ++e) dr[e] = fmaf(iy, dr[e], -ky * y[e]);
    store_row<T, VEC, W>((T*)p.dy + row * p.width, lane, width, dr);
  }
  if constexpr (S) cp_wait0();
  float* part = p.part + (size_t)blockIdx.x * 2 * p.width;
  if constexpr (R == 1) {
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      const int c = column<T, VEC, W>(lane, e);
      if (c < p.width) {
        part[c] = W == 32 ? sums[e * NT] : cp[W == 32 ? 0 : e];
        part[p.width + c] = W == 32 ? sums[(kL + e) * NT] : cq[W == 32 ? 0 : e];
      }
    }
  } else {
    float* cols = (float*)stage;
    __syncthreads();  // every thread has read its last row
#pragma unroll
    for (int e = 0; e < kL; ++e) {
      const int c = column<T, VEC, W>(lane, e);
      if (c < p.width) {
        cols[(group * 2) * p.width + c] = cp[W == 32 ? 0 : e];
        cols[(group * 2 + 1) * p.width + c] = cq[W == 32 ? 0 : e];
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

// The CTAs' partial rows summed in order: a CTA takes 32 columns, 32 slices of
// the partials each, then the slices in order.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) k_block_norm_dw(int ncta, BlockNorm p) {
  __shared__ float sum[2][kSlices][33];
  const int j = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + j;
  float a = 0.f, b = 0.f;
  if (c < p.width)
    for (int i = sl; i < ncta; i += kSlices) {
      a += p.part[(size_t)i * 2 * p.width + c];
      b += p.part[((size_t)i * 2 + 1) * p.width + c];
    }
  sum[0][sl][j] = a;
  sum[1][sl][j] = b;
  __syncthreads();
  if (sl == 0 && c < p.width) {
    a = b = 0.f;
    for (int i = 0; i < kSlices; ++i) {
      a += sum[0][i][j];
      b += sum[1][i][j];
    }
    p.dw_post[c] = p.res_scale ? a * p.res_scale[c] : a;
    if (p.dres_scale) p.dres_scale[c] = a * p.w_post[c];
    p.dw_pre[c] = b;
  }
}

template <typename T, typename TR, bool VEC, int W>
cudaError_t launch(const BlockNorm& p, bool backward, int* grid_out, cudaStream_t s) {
  constexpr int R = Shape<W>::kRows, NT = Shape<W>::kThreads;
  const long long steps = (p.rows + R - 1) / R;
  int grid = 1;
  if (!backward) {
    constexpr size_t smem =
        kStaged<VEC, W> ? (size_t)2 * (2 * Pieces<T, VEC>::n + Pieces<TR, VEC>::n) * NT * 16 : 0;
    static FitOf fit;
    cudaError_t e =
        persistent_grid(k_block_norm_fwd<T, TR, VEC, W>, NT, smem, steps, 1 << 20, &fit, &grid);
    if (e != cudaSuccess) return e;
    LaunchScope ls("block_norm_fwd", s);
    k_block_norm_fwd<T, TR, VEC, W><<<grid, NT, smem, s>>>(p);
    return cudaGetLastError();
  }
  constexpr size_t staged =
      kStaged<VEC, W> ? (size_t)2 * (3 * Pieces<T, VEC>::n + 2 * Pieces<TR, VEC>::n) * NT * 16 : 0;
  // the widest row's column sums
  constexpr size_t cols = (R > 1 ? (size_t)R * 2 * W * 32 * kL : W == 32 ? (size_t)2 * kL * NT : 0) * sizeof(float);
  constexpr size_t smem = (staged > cols ? staged : cols) + (size_t)2 * kL * W * 32 * sizeof(float);
  static FitOf fit;
  cudaError_t e =
      persistent_grid(k_block_norm_bwd<T, TR, VEC, W>, NT, smem, steps, kBlockNormMaxCtas, &fit,
                      &grid);
  if (e != cudaSuccess) return e;
  *grid_out = grid;
  LaunchScope ls("block_norm_bwd", s);
  k_block_norm_bwd<T, TR, VEC, W><<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t launch_t(const BlockNorm& p, bool vec, bool backward, int* grid, cudaStream_t s) {
  const int w = (p.width + 32 * kL - 1) / (32 * kL);  // warps that a row needs
  if (vec) {
    if (w <= 1) return launch<T, TR, true, 1>(p, backward, grid, s);
    if (w <= 2) return launch<T, TR, true, 2>(p, backward, grid, s);
    if (w <= 4) return launch<T, TR, true, 4>(p, backward, grid, s);
    if (w <= 8) return launch<T, TR, true, 8>(p, backward, grid, s);
    if (w <= 16) return launch<T, TR, true, 16>(p, backward, grid, s);
    return launch<T, TR, true, 32>(p, backward, grid, s);
  }
  if (w <= 1) return launch<T, TR, false, 1>(p, backward, grid, s);
  if (w <= 4) return launch<T, TR, false, 4>(p, backward, grid, s);
  return launch<T, TR, false, 32>(p, backward, grid, s);
}

cudaError_t dispatch(const BlockNorm& p, bool bf16, bool res_bf16, bool backward, int* grid,
                     cudaStream_t s) {
  // 16-byte vectors need every row of every tensor to start on such a boundary
  // and the width to be whole vectors
  const int unit = bf16 ? 8 : 4;
  bool vec = p.width % unit == 0 && p.y_stride % unit == 0 && (!p.z || p.z_stride % unit == 0);
  const void* ptrs[] = {p.residual, p.y, p.z, p.w_post, p.res_scale, p.w_pre, p.new_residual,
                        p.x, p.dx, p.dnew, p.dresidual, p.dy, p.dz};
  for (const void* q : ptrs) vec = vec && ((uintptr_t)q & 15u) == 0;
  if (!bf16) return launch_t<float, float>(p, vec, backward, grid, s);
  if (res_bf16) return launch_t<__nv_bfloat16, __nv_bfloat16>(p, vec, backward, grid, s);
  return launch_t<__nv_bfloat16, float>(p, vec, backward, grid, s);
}

}  // namespace

cudaError_t block_norm_forward(const BlockNorm& p, bool bf16, bool res_bf16, cudaStream_t s) {
  return dispatch(p, bf16, res_bf16, false, nullptr, s);
}

cudaError_t block_norm_backward(const BlockNorm& p, bool bf16, bool res_bf16, cudaStream_t s) {
  int grid = 1;
  const cudaError_t e = dispatch(p, bf16, res_bf16, true, &grid, s);
  if (e != cudaSuccess) return e;
  LaunchScope ls("block_norm_dw", s);
  k_block_norm_dw<<<(p.width + 31) / 32, 32 * kSlices, 0, s>>>(grid, p);
  return cudaGetLastError();
}

}  // namespace ssd
