// Global gradient norm over many tensors and clipping by it, two launches:
//   k_clip_norm:  the sum of squares of a CTA's chunks, one partial per CTA
//   k_clip_apply: every CTA adds the partials in order (n, c), then out = c g
// The tensors are cut into chunks; chunk j belongs to CTA j mod grid.  The
// table of tensors travels in the launch's parameters.
//
// Bound by memory: g is read twice (the second time from L2 as far as it fits
// there, which is why the second kernel takes its chunks in reverse) and out
// written once.  Measured on 240 tensors, 1.2 GB: 595 us, 87 % of the copy rate
// for those three passes (chunks of sixteen times the size were slower).
//
// Squares are added in fp32, at most eight after one another (their roundings
// may all go the same way), and those sums over a thread's part of a chunk, of
// any length, in two fp32 parts; above that in fp64.  A part whose sum is so large
// or so small that squares may have left fp32's range is added again in fp64.
#include <cuda_bf16.h>

#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <int N>
struct Table {
  int count;          // tensors
  int chunks;         // chunks of all of them
  int shift;          // log2 of a chunk's bytes
  ClipEntry e[N];
};

// Table entry and first byte of chunk j.
template <int N>
__device__ __forceinline__ int find(const Table<N>& t, int j) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first_chunk <= j) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The sum of a vector's squares.
template <typename T>
__device__ __forceinline__ float squares(uint4 q, unsigned& any) {
  any |= q.x | q.y | q.z | q.w;
  if constexpr (sizeof(T) == 4) {
    const float4 f = *(const float4*)&q;
    return fmaf(f.x, f.x, fmaf(f.y, f.y, fmaf(f.z, f.z, f.w * f.w)));
  } else {
    const __nv_bfloat162* h = (const __nv_bfloat162*)&q;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
    return s;
  }
}

// A sum and, apart from it, the rounding errors of its additions (each of them
// exactly, by Knuth's two-sum).
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = hi + x, y = t - hi;
    lo += (hi - (t - y)) + (x - y);
    hi = t;
  }
};

// Elements [0, n) at g: those before the first 16-byte boundary, whole
// vectors, and the rest.
struct Split {
  int head, vecs, tail;
};
template <typename T>
__device__ __forceinline__ Split split(const T* g, int n) {
  Split s;
  s.head = min(n, (int)(((16 - ((uintptr_t)g & 15)) & 15) / sizeof(T)));
  s.vecs = (n - s.head) / (16 / (int)sizeof(T));
  s.tail = s.head + s.vecs * (16 / (int)sizeof(T));
  return s;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int n) {
  const Split sp = split(g, n);
  const uint4* v = (const uint4*)(g + sp.head);
  const int t = threadIdx.x;
  Sum s;
  unsigned any = 0;
  int i = t;
  for (; i + 3 * kThreads < sp.vecs; i += 4 * kThreads) {
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = v[i + u * kThreads];
    s.add((squares<T>(q[0], any) + squares<T>(q[1], any)) +
          (squares<T>(q[2], any) + squares<T>(q[3], any)));
  }
  for (; i < sp.vecs; i += kThreads) s.add(squares<T>(v[i], any));
  // at most 7 elements before the vectors and 7 behind them
  const int edge = t < sp.head ? t : t >= 32 && sp.tail + t - 32 < n ? sp.tail + t - 32 : -1;
  if (edge >= 0) {
    const float f = to_f32(g[edge]);
    s.add(f * f);
    any |= f != 0.f;
  }
  // squares of |g| in [2^-48, 2^48] and any sum of them stay well inside fp32
  // (a sign bit alone only costs the second pass)
  if (s.hi < 0x1p+96f && (s.hi > 0x1p-96f || any == 0)) return (double)s.hi + (double)s.lo;
  double d = 0.0;
  constexpr int E = 16 / (int)sizeof(T);
  for (i = t; i < sp.vecs; i += kThreads)
    for (int u = 0; u < E; ++u) {
      const double x = (double)to_f32(g[sp.head + i * E + u]);
      d = fma(x, x, d);
    }
  if (edge >= 0) {
    const double x = (double)to_f32(g[edge]);
    d = fma(x, x, d);
  }
  return d;
}

__device__ __forceinline__ double block_sum_f64(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
k_clip_norm(const __grid_constant__ Table<N> t, double* __restrict__ part) {
  double sum = 0.0;
  for (int j = blockIdx.x; j < t.chunks; j += gridDim.x) {
    const ClipEntry& e = t.e[find(t, j)];
    const int esz = e.bf16 ? 1 : 2;  // log2 of an element's bytes
    const long long at = (long long)(j - e.first_chunk) << (t.shift - esz);
    const int n = (int)min((long long)1 << (t.shift - esz), e.numel - at);
    sum += e.bf16 ? chunk_squares((const __nv_bfloat16*)e.g + at, n)
                  : chunk_squares((const float*)e.g + at, n);
  }
  sum = block_sum_f64(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 q, float c) {
  if constexpr (sizeof(T) == 4) {
    float4* f = (float4*)&q;
    f->x *= c; f->y *= c; f->z *= c; f->w *= c;
  } else {
    __nv_bfloat162* h = (__nv_bfloat162*)&q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      h[i] = __floats2bfloat162_rn(f.x * c, f.y * c);
    }
  }
  return q;
}

template <typename T>
__device__ __forceinline__ void chunk_apply(const T* g, T* out, int n, float c) {
  const int t = threadIdx.x;
  if ((((uintptr_t)g ^ (uintptr_t)out) & 15) != 0) {  // never on a 16-byte boundary together
    for (int i = t; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(g[i]) * c);
    return;
  }
  const Split sp = split(g, n);
  const uint4* v = (const uint4*)(g + sp.head);
  uint4* o = (uint4*)(out + sp.head);
  int i = t;
  for (; i + 3 * kThreads < sp.vecs; i += 4 * kThreads) {
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = v[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[i + u * kThreads] = scaled<T>(q[u], c);
  }
  for (; i < sp.vecs; i += kThreads) o[i] = scaled<T>(v[i], c);
  const int edge = t < sp.head ? t : t >= 32 && sp.tail + t - 32 < n ? sp.tail + t - 32 : -1;
  if (edge >= 0) out[edge] = from_f32<T>(to_f32(g[edge]) * c);
}

template <int N>
__global__ void __launch_bounds__(kThreads)
k_clip_apply(const __grid_constant__ Table<N> t, const double* __restrict__ part, int parts,
             float max_norm, float eps, float* __restrict__ norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
  sum = sqrt(block_sum_f64(sum));
  // min(1, max_norm / (n + eps)); NaN stays NaN, nothing is scaled where n + eps is 0
  const double den = sum + (double)eps;
  double cd = den == 0.0 ? 1.0 : (double)max_norm / den;
  if (cd > 1.0) cd = 1.0;
  const float c = (float)cd;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)sum;
  for (int i = (t.chunks - 1 - (int)blockIdx.x) / (int)gridDim.x; i >= 0; --i) {
    const int j = i * gridDim.x + blockIdx.x;
    if (j >= t.chunks) continue;
    const ClipEntry& e = t.e[find(t, j)];
    if (c == 1.f && e.g == e.out) continue;
    const int esz = e.bf16 ? 1 : 2;
    const long long at = (long long)(j - e.first_chunk) << (t.shift - esz);
    const int n = (int)min((long long)1 << (t.shift - esz), e.numel - at);
    if (e.bf16) chunk_apply((const __nv_bfloat16*)e.g + at, (__nv_bfloat16*)e.out + at, n, c);
    else chunk_apply((const float*)e.g + at, (float*)e.out + at, n, c);
  }
}

// One launch's worth of tensors (each not empty) from `src`.
template <int N>
void fill(Table<N>& t, const ClipEntry* src, int count, int shift) {
  t.count = count;
  t.shift = shift;
  int chunks = 0;
  for (int i = 0; i < count; ++i) {
    t.e[i] = src[i];
    t.e[i].first_chunk = chunks;
    chunks += (int)(((src[i].numel << (src[i].bf16 ? 1 : 2)) + (1ll << shift) - 1) >> shift);
  }
  t.chunks = chunks;
}

int grid_of(int chunks) { return chunks < kClipMaxCtas ? chunks : kClipMaxCtas; }

template <int N>
cudaError_t run(const ClipEntry* src, int count, int shift, bool apply, double* part, int* parts,
                float max_norm, float eps, float* norm, cudaStream_t s) {
  Table<N> t;
  fill(t, src, count, shift);
  if (!apply) {
    const int grid = grid_of(t.chunks);
    LaunchScope ls("clip_norm", s);
    k_clip_norm<N><<<grid, kThreads, 0, s>>>(t, part + *parts);
    *parts += grid;
  } else {
    const int grid = t.chunks ? grid_of(t.chunks) : 1;
    LaunchScope ls("clip_apply", s);
    k_clip_apply<N><<<grid, kThreads, 0, s>>>(t, part, *parts, max_norm, eps, norm);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t clip_grad_norm(const ClipEntry* e, int count, int shift, double* part, float max_norm,
                           float eps, float* norm, cudaStream_t s) {
  int parts = 0;
  for (int pass = 0; pass < 2; ++pass)
    for (int at = 0; at < count || (pass == 1 && at == 0); at += kClipTable) {
      const int n = count - at < kClipTable ? count - at : kClipTable;
      float* to = at == 0 ? norm : nullptr;
      const cudaError_t err =
          n <= 48 ? run<48>(e + at, n, shift, pass == 1, part, &parts, max_norm, eps, to, s)
                  : run<kClipTable>(e + at, n, shift, pass == 1, part, &parts, max_norm, eps, to, s);
      if (err != cudaSuccess) return err;
    }
  return cudaSuccess;
}

}  // namespace ssd
