// Linear attention with a decay for each head: the walk over the steps of a
// row (forward, and with exchanged roles the gradients), the sum over a
// group's heads, and the step of one token.
//
// With a = e^{log_decay_h} and chunks of C steps, S the state before a chunk
// and positions i, j inside it,
//   o_i = s sum_{j <= i} a^{i-j} (q_i . k_j) v_j + s a^{i+1} S q_i
//   S  <- a^C S + sum_j a^{C-1-j} v_j k_j^T
// which is the recurrence S_t = a S_{t-1} + v_t k_t^T, o_t = s S_t q_t
// regrouped.  The gradients of L = sum(do . o) + sum(dS . S_T) are
//   dq_i = s sum_{j <= i} a^{i-j} (do_i . v_j) k_j + s a^{i+1} S0^T do_i
//   dk_j = s sum_{i >= j} a^{i-j} (v_j . do_i) q_i + a^{T-1-j} dS^T v_j
//   dv_j = s sum_{i >= j} a^{i-j} (k_j . q_i) do_i + a^{T-1-j} dS k_j
//   dS0  = a^T dS + s sum_i a^{i+1} do_i q_i^T
// i.e. the same walk with the operands' roles exchanged, the last three from
// the last step back (off = 0: the incoming dS belongs to the last step
// itself, not to the one before the first).
#include "f32x2.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

// a^e for e >= 0 from log a; a^0 = 1 also where a = 0 (log a = -inf)
__device__ __forceinline__ float decay_pow(float la, float e) { return e == 0.f ? 1.f : expf(la * e); }

// ---- the walk in fp32 on the CUDA cores ---------------------------------------
//
// One CTA per (h, 32 columns of v, b, segment of the row), chunks of 64 steps.
// 128 threads as 16 x 8: thread (ty, tx) forms 4 x 4 blocks of the products
//   u = Q X              rows 4 ty + a, columns 4 tx + e
//   P = mask(Q K^T)      rows 4 ty + a, columns tx + 8 e
//   o = lead u + P V     rows 4 ty + a, columns 4 tx + e
//   X = a^n X + K^T w V  rows 4 ty + a (+ 64), columns 4 tx + e, in registers
// two products an instruction (fma.f32x2): the first three add up even and odd
// terms of their sums apart, from operands that lie along the sum (V and X are
// kept transposed for that); the last forms pairs of rows k, with each w V held
// twice.  Eight 16-byte loads then serve 32 instructions of 64 products.  P
// replaces the rows of Q that a warp is done with, which leaves room for three
// CTAs on an SM to hide one another's loads; P and P V leave out the columns
// that the mask empties for a warp's sixteen rows.  fp32 throughout: the
// operands' type leaves no other choice that keeps their precision.
constexpr int kC = 64;         // steps of a chunk
constexpr int kB = 32;         // columns of v of a CTA
constexpr int kThreads = 128;

template <int DK, bool kStates>
struct Simt {
  static constexpr int LK = DK + 4;  // rows 16 bytes apart in the banks
  static constexpr int LV = kC + 4;
  // K and w V (twice); Q or P, V and X transposed
  static constexpr int kFloats =
      kC * LK + 2 * kC * kB + (kStates ? 0 : kC * LK + kB * LV + kB * LK);
  static constexpr size_t smem = kFloats * sizeof(float);
};

struct SimtWalk {
  LaWalk w;
  int nseg, span;  // steps of a segment
};

__device__ __forceinline__ float4 ld4(const float* p) { return *(const float4*)p; }
// 16 bytes, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
// acc += l . r over four terms, even and odd ones apart
__device__ __forceinline__ float2 dot4(float4 l, float4 r, float2 acc) {
  return fma2(make_float2(l.x, l.y), make_float2(r.x, r.y),
              fma2(make_float2(l.z, l.w), make_float2(r.z, r.w), acc));
}

// acc[a][e] += rows a of `left` . rows 8 e of `right`, terms [from, to)
template <int LL, int LR>
__device__ __forceinline__ void block4x4(const float* left, const float* right, int from, int to,
                                         float2 (&acc)[4][4]) {
#pragma unroll 2
  for (int d = from; d < to; d += 4) {
    float4 l[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) l[a] = ld4(left + a * LL + d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 r = ld4(right + 8 * e * LR + d);
#pragma unroll
      for (int a = 0; a < 4; ++a) acc[a][e] = dot4(l[a], r, acc[a][e]);
    }
  }
}

// kStates: only the state, each segment from zero, into w.last
// [nseg][B][H][dv][dk].
template <int DK, bool kStates>
__global__ void __launch_bounds__(kThreads, DK == 64 ? 3 : 2)
k_la_walk(const __grid_constant__ SimtWalk args) {
  using G = Simt<DK, kStates>;
  constexpr int LK = G::LK, LV = G::LV;
  const LaWalk& w = args.w;
  extern __shared__ __align__(16) float sm[];
  float* K = sm;
  float* W = K + kC * LK;       // w V: [step][columns 4 tx, 4 tx + 1, then + 2, + 3][twice]
  float* Q = W + 2 * kC * kB;   // P once the warp is done with its rows
  float* V = Q + kC * LK;       // column 4 i + c in row i + 8 c
  float* X = V + kB * LV;       // the same
  __shared__ float pw[kC + 2];
  const int vblocks = (w.dv + kB - 1) / kB;
  const int h = blockIdx.x / vblocks, v0 = (blockIdx.x % vblocks) * kB;
  const int b = blockIdx.y, seg = blockIdx.z, t = threadIdx.x, tx = t & 7, ty = t >> 3, wp = t >> 5;
  const float la = w.log_decay[h];
  int len = w.T;
  if (w.lens) len = min(max(w.lens[b], 0), w.T);
  if (t < kC + 2) pw[t] = decay_pow(la, (float)t);
  const int dv = min(kB, w.dv - v0);
  const size_t sbase = (((size_t)seg * w.B + b) * w.H + h) * w.dv * w.dk;
  // state element (k, v) of this thread
  auto state_at = [&](int k, int v) {
    return sbase + (!kStates && w.first_swapped ? (size_t)k * w.dv + v0 + v : (size_t)(v0 + v) * w.dk + k);
  };
  float2 x[DK / 32][4];  // rows k = 4 ty + 2 (i & 1) + 64 (i >> 1) and the next
#pragma unroll
  for (int i = 0; i < DK / 32; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = 4 * ty + 2 * (i & 1) + (i >> 1) * 64, v = 4 * tx + c;
      const bool in = !kStates && w.first && k < w.dk && v < dv;
      x[i][c] = in ? make_float2(w.first[state_at(k, v)], w.first[state_at(k + 1, v)])
                   : make_float2(0.f, 0.f);
    }
  const float* qp = (const float*)w.q.p + b * w.q.batch + (long long)(h / w.q.share) * w.dk;
  const float* kp = (const float*)w.k.p + b * w.k.batch + (long long)(h / w.k.share) * w.dk;
  const float* vp = (const float*)w.v.p + b * w.v.batch + (long long)(h / w.v.share) * w.dv + v0;
  float* op = (float*)w.o + ((long long)b * w.T * w.H + h) * w.dv + v0;
  const int s0 = seg * args.span, s1 = min(s0 + args.span, len);  // the segment's steps
  const int nc = s1 > s0 ? (s1 - s0 + kC - 1) / kC : 0;
  for (int ci = 0; ci < nc; ++ci) {
    const int t0 = s0 + (w.reverse ? nc - 1 - ci : ci) * kC, n = min(kC, s1 - t0);
    __syncthreads();
    for (int i = t; i < kC * (DK / 4); i += kThreads) {
      const int r = i / (DK / 4), d = i % (DK / 4) * 4;
      const bool in = r < n && d < w.dk;
      if (!kStates) copy16(Q + r * LK + d, in ? qp + (long long)(t0 + r) * w.q.step + d : qp, in);
      copy16(K + r * LK + d, in ? kp + (long long)(t0 + r) * w.k.step + d : kp, in);
    }
    float4 v[kC * (kB / 4) / kThreads];
#pragma unroll
    for (int i = 0; i < kC * (kB / 4) / kThreads; ++i) {
      const int r = (t + i * kThreads) / (kB / 4);
      v[i] = r < n && 4 * tx < dv ? ld4(vp + (long long)(t0 + r) * w.v.step + 4 * tx)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (!kStates)
#pragma unroll
      for (int g = 0; g < DK / 64; ++g)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *(float4*)(X + (tx + 8 * c) * LK + 4 * ty + 64 * g) =
              make_float4(x[2 * g][c].x, x[2 * g][c].y, x[2 * g + 1][c].x, x[2 * g + 1][c].y);
#pragma unroll
    for (int i = 0; i < kC * (kB / 4) / kThreads; ++i) {
      const int r = (t + i * kThreads) / (kB / 4);
      const float f = r < n ? w.s_inject * pw[(w.reverse ? r : n - 1 - r) + 1 - w.off] : 0.f;
      const float4 y = make_float4(f * v[i].x, f * v[i].y, f * v[i].z, f * v[i].w);
      *(float4*)(W + r * 2 * kB + 4 * tx) = make_float4(y.x, y.x, y.y, y.y);
      *(float4*)(W + r * 2 * kB + kB + 4 * tx) = make_float4(y.z, y.z, y.w, y.w);
      if (!kStates) {
        V[tx * LV + r] = v[i].x;
        V[(tx + 8) * LV + r] = v[i].y;
        V[(tx + 16) * LV + r] = v[i].z;
        V[(tx + 24) * LV + r] = v[i].w;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!kStates) {
      float2 o[4][4];
      auto clear = [](float2 (&acc)[4][4]) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][e] = make_float2(0.f, 0.f);
      };
      clear(o);
      block4x4<LK, LK>(Q + 4 * ty * LK, X + tx * LK, 0, DK, o);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int i = min(4 * ty + a, n - 1);  // (a row past the end is not written)
        const float lead = w.s_carry * pw[(w.reverse ? n - 1 - i : i) + w.off];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][e] = make_float2(lead * (o[a][e].x + o[a][e].y), 0.f);
      }
      // groups of 32 columns (tx + 8 e) that the warp's rows 16 wp ... 16 wp + 15
      // need: the diagonal one, and the one before (after) it for half of the warps
      const int c0 = wp / 2;
      const bool both = w.reverse ? c0 == 0 : c0 == 1;
      float2 s[4][4];
      float p[4][4];
      if (both) {
        clear(s);
        block4x4<LK, LK>(Q + 4 * ty * LK, K + (tx + 32 * (1 - c0)) * LK, 0, DK, s);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[a][e] = s[a][e].x + s[a][e].y;
      }
      clear(s);
      block4x4<LK, LK>(Q + 4 * ty * LK, K + (tx + 32 * c0) * LK, 0, DK, s);
      __syncwarp();  // (the rows of Q are the warp's own)
      auto put = [&](int c, int a, int e, float f) {
        const int i = 4 * ty + a, j = tx + 32 * c + 8 * e, d = w.reverse ? j - i : i - j;
        Q[i * LK + j] = d >= 0 ? w.s_intra * pw[d] * f : 0.f;
      };
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          put(c0, a, e, s[a][e].x + s[a][e].y);
          if (both) put(1 - c0, a, e, p[a][e]);
        }
      __syncwarp();
      block4x4<LK, LV>(Q + 4 * ty * LK, V + tx * LV, w.reverse ? 16 * wp : 0,
                       w.reverse ? kC : 16 * wp + 16, o);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int i = 4 * ty + a;
        if (i < n && 4 * tx < dv)
          *(float4*)(op + (long long)(t0 + i) * w.H * w.dv + 4 * tx) =
              make_float4(o[a][0].x + o[a][0].y, o[a][1].x + o[a][1].y, o[a][2].x + o[a][2].y,
                          o[a][3].x + o[a][3].y);
      }
    }
    const float2 an = make_float2(pw[n], pw[n]);
#pragma unroll
    for (int i = 0; i < DK / 32; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i][c] = mul2(x[i][c], an);
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float4 ya = ld4(W + j * 2 * kB + 4 * tx), yb = ld4(W + j * 2 * kB + kB + 4 * tx);
      const float2 y[4] = {make_float2(ya.x, ya.y), make_float2(ya.z, ya.w),
                           make_float2(yb.x, yb.y), make_float2(yb.z, yb.w)};
#pragma unroll
      for (int g = 0; g < DK / 64; ++g) {
        const float4 k = ld4(K + j * LK + 4 * ty + 64 * g);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[2 * g][c] = fma2(make_float2(k.x, k.y), y[c], x[2 * g][c]);
          x[2 * g + 1][c] = fma2(make_float2(k.z, k.w), y[c], x[2 * g + 1][c]);
        }
      }
    }
  }
  if (!kStates) {  // past the row's end
    const int z0 = max(s0, min(len, s0 + args.span)), z1 = min(s0 + args.span, w.T);
    const int d = t % (kB / 4) * 4;
    if (d < dv)
      for (int r = z0 + t / (kB / 4); r < z1; r += kThreads / (kB / 4))
        *(float4*)(op + (long long)r * w.H * w.dv + d) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (w.last)
#pragma unroll
    for (int i = 0; i < DK / 32; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = 4 * ty + 2 * (i & 1) + (i >> 1) * 64, v = 4 * tx + c;
        if (k < w.dk && v < dv) {
          w.last[state_at(k, v)] = x[i][c].x;
          w.last[state_at(k + 1, v)] = x[i][c].y;
        }
      }
}

// The states before each segment from the segments' own: in walk order
//   X_0 = first, X_{s+1} = a^{steps of s} X_s + local_s;  last = X_nseg.
// seg [nseg][B][H][dv][dk], overwritten in place.
__global__ void __launch_bounds__(256) k_la_segments(const LaSegments p) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int i = blockIdx.x * 256 + threadIdx.x, n = p.dk * p.dv;
  if (i >= n) return;
  const float la = p.log_decay[h];
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const size_t row = ((size_t)b * p.H + h) * n, stride = (size_t)p.B * p.H * n;
  const size_t at = row + (p.swapped ? (size_t)(i % p.dk) * p.dv + i / p.dk : (size_t)i);
  float x = p.first ? p.first[at] : 0.f;
  for (int j0 = 0; j0 < p.nseg; j0 += 8) {
    float local[8];  // read ahead: the loads do not wait for one another
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int s = p.reverse ? p.nseg - 1 - j0 - u : j0 + u;
      local[u] = j0 + u < p.nseg ? p.seg[s * stride + row + i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + u >= p.nseg) break;
      const int s = p.reverse ? p.nseg - 1 - j0 - u : j0 + u;
      const int steps = min(max(len - s * p.span, 0), p.span);
      p.seg[s * stride + row + i] = x;
      x = fmaf(decay_pow(la, (float)steps), x, local[u]);
    }
  }
  if (p.last) p.last[at] = x;
}

template <int DK, bool kStates>
cudaError_t walk_t(const SimtWalk& a, cudaStream_t s) {
  constexpr int smem = (int)Simt<DK, kStates>::smem;
  cudaError_t e = cudaFuncSetAttribute(k_la_walk<DK, kStates>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "linattn_states" : a.w.reverse ? "linattn_walk_back" : "linattn_walk", s);
  const int vblocks = (a.w.dv + kB - 1) / kB;
  k_la_walk<DK, kStates><<<dim3(a.w.H * vblocks, a.w.B, a.nseg), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

// part [rows][G][share][D] -> out [rows][G][D]
__global__ void k_la_group_sum(long long n, int share, int D, const float* __restrict__ part,
                               float* __restrict__ out) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const float* p = part + i / D * share * D + i % D;
    float s = 0.f;
    for (int j = 0; j < share; ++j) s += p[(long long)j * D];
    out[i] = s;
  }
}

// One token: S' = a S + v k^T, o = s S' q.  A row of the state (dk floats) is
// held by LPR lanes, four floats each; a warp takes NR rows a lane at once, so
// that as many 16-byte loads are in flight, and adds the NR dot products up
// together: while a lane holds several, each exchange halves them (lanes of one
// half keep one half of the values), nine exchanges for eight sums over 32
// lanes instead of forty.
//
// Bound by the states' bytes, read and written once.  Measured on 256 rows of
// 64 heads, 128 x 64 (1.08 GB): 191 us with one row a lane at a time and sixteen
// rows a CTA, 160 us with eight.
constexpr int kStepWarps = 4;

// four consecutive operands of a lane
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 f = *(const float4*)p;
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 q = *(const uint2*)p;
  const float2 a = __bfloat1622float2(*(const __nv_bfloat162*)&q.x);
  const float2 b = __bfloat1622float2(*(const __nv_bfloat162*)&q.y);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

template <typename T, int LPR, int NR>
__global__ void __launch_bounds__(kStepWarps * 32) k_la_step(const LaStep p) {
  constexpr int RPW = 32 / LPR;                  // rows of a warp side by side
  constexpr int kRows = kStepWarps * RPW * NR;   // rows of a CTA
  const int h = blockIdx.y, b = blockIdx.z, g = h / (p.H / p.G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, k0 = sub * 4;
  const bool kin = k0 < p.dk;
  long long row = b;
  if (p.slots) {
    row = p.slots[b];
    if (row < 0 || row >= p.nslots) row = -1;
  }
  const int vb = blockIdx.x * kRows + warp * (RPW * NR) + lane / LPR;  // row of slot i: + i RPW
  const long long at = ((row * p.H + h) * p.dv + vb) * p.dk + k0;
  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i)
    s[i] = kin && row >= 0 && vb + i * RPW < p.dv
               ? *(const float4*)(p.state_in + at + (long long)i * RPW * p.dk)
               : make_float4(0.f, 0.f, 0.f, 0.f);
  const float a = decay_pow(p.log_decay[b * p.decay_batch + h], 1.f);
  float q[4] = {0.f, 0.f, 0.f, 0.f}, k[4] = {0.f, 0.f, 0.f, 0.f};
  if (kin) {
    load4((const T*)p.q + b * p.q_batch + (long long)g * p.dk + k0, q);
    load4((const T*)p.k + b * p.k_batch + (long long)g * p.dk + k0, k);
  }
  const T* vp = (const T*)p.v + b * p.v_batch + (long long)h * p.dv;
  float o[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int v = vb + i * RPW;
    const float x = v < p.dv ? to_f32(vp[v]) : 0.f;
    s[i].x = fmaf(a, s[i].x, x * k[0]);
    s[i].y = fmaf(a, s[i].y, x * k[1]);
    s[i].z = fmaf(a, s[i].z, x * k[2]);
    s[i].w = fmaf(a, s[i].w, x * k[3]);
    if (kin && row >= 0 && v < p.dv) *(float4*)(p.state_out + at + (long long)i * RPW * p.dk) = s[i];
    o[i] = fmaf(s[i].x, q[0], fmaf(s[i].y, q[1], fmaf(s[i].z, q[2], s[i].w * q[3])));
  }
  int n = NR, first = 0;  // this lane holds the sums first ... first + n - 1
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) {
    if (n > 1) {
      const bool up = (sub & d) != 0;
      n /= 2;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i)
        if (i < n) {
          const float send = up ? o[i] : o[i + n], keep = up ? o[i + n] : o[i];
          o[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
      if (up) first += n;
    } else {
      o[0] += __shfl_xor_sync(0xffffffffu, o[0], d);
    }
  }
  // lanes that differ below the exchanges that halved hold the same sums
  if (sub % (LPR * n / NR > 1 ? LPR * n / NR : 1) == 0)
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i < n && vb + (first + i) * RPW < p.dv)
        ((T*)p.o)[((long long)b * p.H + h) * p.dv + vb + (first + i) * RPW] =
            from_f32<T>(row >= 0 ? p.scale * o[i] : 0.f);
}

template <typename T, int LPR>
cudaError_t step_l(const LaStep& p, cudaStream_t s) {
  LaunchScope ls("linattn_step", s);
  constexpr int rows = kStepWarps * (32 / LPR);
  // eight rows a lane once that leaves work for every SM (with fewer rows the
  // latency of one counts: 32 heads of one row ran in 8.1 us with two a lane)
  if ((long long)p.B * p.H * ((p.dv + 8 * rows - 1) / (8 * rows)) >= 304)
    k_la_step<T, LPR, 8><<<dim3((p.dv + 8 * rows - 1) / (8 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  else
    k_la_step<T, LPR, 2><<<dim3((p.dv + 2 * rows - 1) / (2 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const LaStep& p, cudaStream_t s) {
  const int lanes = p.dk / 4;
  if (lanes <= 4) return step_l<T, 4>(p, s);
  if (lanes <= 8) return step_l<T, 8>(p, s);
  if (lanes <= 16) return step_l<T, 16>(p, s);
  return step_l<T, 32>(p, s);
}

}  // namespace

int la_segments(long long rows, long long chunks, long long slots) {
  // A row's chunks go to one CTA unless that leaves SMs idle.  Splitting a row
  // costs a pass for the segments' states (about half a walk) and two more
  // launches, and every wave of CTAs its start (about two chunks), so it has to
  // pay for that.
  auto waves = [&](long long n) { return (rows * n + slots - 1) / slots; };
  double best = (double)(waves(1) * (chunks + 2));
  int at = 1;
  for (int n = 2; n <= chunks && n <= 32; ++n) {
    const long long per = (chunks + n - 1) / n;
    const double cost = 1.5 * (double)(waves(n) * (per + 2)) + 4.0 + 0.25 * n;
    if (cost < best) {
      best = cost;
      at = n;
    }
  }
  return at;
}

cudaError_t la_segment_states(const LaSegments& p, cudaStream_t s) {
  LaunchScope ls("linattn_segments", s);
  k_la_segments<<<dim3((p.dk * p.dv + 255) / 256, p.H, p.B), 256, 0, s>>>(p);
  return cudaGetLastError();
}

// CTAs of the fp32 walk that run at once on 152 SMs (three of 69 KB, or two of 110)
static int simt_segments(int B, int H, int T, int dk, int dv) {
  return la_segments((long long)B * H * ((dv + kB - 1) / kB), (T + kC - 1) / kC,
                     dk <= 64 ? 456 : 304);
}

size_t la_scratch_floats(int B, int H, int T, int dk, int dv, bool bf16) {
  if (bf16) return la_tc_scratch_floats(B, H, T, dk, dv);
  // (the walks of a backward pass have dk and dv in either order)
  const int a = simt_segments(B, H, T, dk, dv), b = simt_segments(B, H, T, dv, dk), n = a > b ? a : b;
  return n > 1 ? (size_t)n * B * H * dk * dv : 0;
}

cudaError_t la_walk(const LaWalk& w, bool bf16, bool beside, float* scratch, cudaStream_t s) {
  if (bf16) return la_walk_tc(w, beside, scratch, s);
  SimtWalk a;
  a.w = w;
  const int nc = (w.T + kC - 1) / kC;
  int n = simt_segments(w.B, w.H, w.T, w.dk, w.dv);
  a.span = (nc + n - 1) / n * kC;
  n = (w.T + a.span - 1) / a.span;
  a.nseg = n;
  if (n > 1) {
    a.w.last = scratch;
    cudaError_t e = w.dk <= 64 ? walk_t<64, true>(a, s) : walk_t<128, true>(a, s);
    if (e != cudaSuccess) return e;
    const LaSegments g = {w.B, w.H, w.T, w.dk, w.dv, n, a.span, w.log_decay, w.lens, scratch,
                          w.first, w.last, w.first_swapped, w.reverse};
    if ((e = la_segment_states(g, s)) != cudaSuccess) return e;
    a.w.first = scratch;
    a.w.first_swapped = false;
    a.w.last = nullptr;
  }
  return w.dk <= 64 ? walk_t<64, false>(a, s) : walk_t<128, false>(a, s);
}

cudaError_t la_group_sum(long long rows, int G, int share, int D, const float* part, float* out,
                         cudaStream_t s) {
  const long long n = rows * G * D;
  const long long want = (n + 255) / 256;
  LaunchScope ls("linattn_group_sum", s);
  k_la_group_sum<<<(int)(want < 8192 ? want : 8192), 256, 0, s>>>(n, share, D, part, out);
  return cudaGetLastError();
}

cudaError_t la_step(const LaStep& p, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace ssd
