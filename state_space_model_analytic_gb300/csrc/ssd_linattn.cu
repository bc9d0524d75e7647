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
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

// a^e for e >= 0 from log a; a^0 = 1 also where a = 0 (log a = -inf)
__device__ __forceinline__ float decay_pow(float la, float e) { return e == 0.f ? 1.f : expf(la * e); }

constexpr int kC = 32;        // steps of a chunk
constexpr int kThreads = 256;

// One CTA per (h, b).  Shared memory (fp32): q, k [C][dk + 1], v [C][dv + 1],
// P [C][C + 1], S [dv][dk + 1].
__global__ void __launch_bounds__(kThreads) k_la_walk(LaWalk w) {
  using T = float;
  extern __shared__ float sm[];
  const int dk = w.dk, dv = w.dv, lk = dk + 1, lv = dv + 1;
  float* Q = sm;
  float* K = Q + kC * lk;
  float* V = K + kC * lk;
  float* P = V + kC * lv;
  float* S = P + kC * (kC + 1);
  __shared__ float pw[kC + 2];
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  const float la = w.log_decay[h];
  int len = w.T;
  if (w.lens) len = min(max(w.lens[b], 0), w.T);
  if (t < kC + 2) pw[t] = decay_pow(la, (float)t);
  const size_t sbase = ((size_t)b * w.H + h) * dv * dk;
  for (int i = t; i < dv * dk; i += kThreads) {
    const int v = i / dk, k = i % dk;
    S[v * lk + k] = !w.first ? 0.f : w.first[sbase + (w.first_swapped ? (size_t)k * dv + v : i)];
  }
  const T* qp = (const T*)w.q.p + b * w.q.batch + (long long)(h / w.q.share) * dk;
  const T* kp = (const T*)w.k.p + b * w.k.batch + (long long)(h / w.k.share) * dk;
  const T* vp = (const T*)w.v.p + b * w.v.batch + (long long)(h / w.v.share) * dv;
  T* op = (T*)w.o + ((long long)b * w.T * w.H + h) * dv;
  const int nc = (len + kC - 1) / kC;
  for (int ci = 0; ci < nc; ++ci) {
    const int c = w.reverse ? nc - 1 - ci : ci;
    const int n = min(kC, len - c * kC);
    const long long t0 = (long long)c * kC;
    __syncthreads();
    for (int i = t; i < kC * dk; i += kThreads) {
      const int r = i / dk, d = i % dk;
      Q[r * lk + d] = r < n ? to_f32(qp[(t0 + r) * w.q.step + d]) : 0.f;
      K[r * lk + d] = r < n ? to_f32(kp[(t0 + r) * w.k.step + d]) : 0.f;
    }
    for (int i = t; i < kC * dv; i += kThreads) {
      const int r = i / dv, d = i % dv;
      V[r * lv + d] = r < n ? to_f32(vp[(t0 + r) * w.v.step + d]) : 0.f;
    }
    __syncthreads();
    for (int e = t; e < kC * kC; e += kThreads) {
      const int i = e / kC, j = e % kC;
      const int d = w.reverse ? j - i : i - j;
      float s = 0.f;
      if (d >= 0 && i < n && j < n) {
        for (int x = 0; x < dk; ++x) s = fmaf(Q[i * lk + x], K[j * lk + x], s);
        s *= w.s_intra * pw[d];
      }
      P[i * (kC + 1) + j] = s;
    }
    __syncthreads();
    for (int e = t; e < n * dv; e += kThreads) {
      const int i = e / dv, v = e % dv;
      float s = 0.f, u = 0.f;
      for (int j = 0; j < kC; ++j) s = fmaf(P[i * (kC + 1) + j], V[j * lv + v], s);
      for (int x = 0; x < dk; ++x) u = fmaf(S[v * lk + x], Q[i * lk + x], u);
      const int lead = (w.reverse ? n - 1 - i : i) + w.off;
      op[(t0 + i) * w.H * dv + v] = fmaf(w.s_carry * pw[lead], u, s);
    }
    __syncthreads();
    const float an = decay_pow(la, (float)n);
    for (int e = t; e < dv * dk; e += kThreads) {
      const int v = e / dk, k = e % dk;
      float s = 0.f;
      for (int j = 0; j < n; ++j)
        s = fmaf(V[j * lv + v] * pw[(w.reverse ? j : n - 1 - j) + 1 - w.off], K[j * lk + k], s);
      S[v * lk + k] = fmaf(an, S[v * lk + k], w.s_inject * s);
    }
  }
  __syncthreads();
  for (long long i = t; i < (long long)(w.T - len) * dv; i += kThreads)
    op[(len + i / dv) * w.H * dv + i % dv] = 0.f;
  if (w.last)
    for (int i = t; i < dv * dk; i += kThreads) {
      const int v = i / dk, k = i % dk;
      w.last[sbase + (w.first_swapped ? (size_t)k * dv + v : i)] = S[v * lk + k];
    }
}

// part [rows][G][share][D] fp32 -> out [rows][G][D]
template <typename T>
__global__ void k_la_group_sum(long long n, int share, int D, const float* __restrict__ part,
                               T* __restrict__ out) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const long long rg = i / D;
    const float* p = part + rg * share * D + i % D;
    float s = 0.f;
    for (int j = 0; j < share; ++j) s += p[(long long)j * D];
    out[i] = from_f32<T>(s);
  }
}

// One token: S' = a S + v k^T, o = s S' q.  A warp takes rows v of the state,
// 32 / LPR at a time (a row of dk floats is held by LPR lanes, four floats
// each).
constexpr int kStepWarps = 4;
constexpr int kStepRows = 16;  // rows of a CTA

template <typename T, int LPR>
__global__ void __launch_bounds__(kStepWarps * 32) k_la_step(LaStep p) {
  const int h = blockIdx.y, b = blockIdx.z, g = h / (p.H / p.G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, k0 = sub * 4;
  const bool kin = k0 < p.dk;
  long long row = b;
  if (p.slots) {
    row = p.slots[b];
    if (row < 0 || row >= p.nslots) row = -1;
  }
  const float a = decay_pow(p.log_decay[b * p.decay_batch + h], 1.f);
  float q[4], k[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = kin ? to_f32(((const T*)p.q)[b * p.q_batch + (long long)g * p.dk + k0 + i]) : 0.f;
    k[i] = kin ? to_f32(((const T*)p.k)[b * p.k_batch + (long long)g * p.dk + k0 + i]) : 0.f;
  }
  constexpr int RPW = 32 / LPR;
  for (int v0 = blockIdx.x * kStepRows + warp * RPW; v0 < min(p.dv, (int)(blockIdx.x + 1) * kStepRows);
       v0 += kStepWarps * RPW) {
    const int v = v0 + lane / LPR;
    const bool in = kin && v < p.dv && row >= 0;
    const long long at = ((row * p.H + h) * p.dv + v) * p.dk + k0;
    float4 s = in ? *(const float4*)(p.state_in + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float x = v < p.dv ? to_f32(((const T*)p.v)[b * p.v_batch + (long long)h * p.dv + v]) : 0.f;
    s.x = fmaf(a, s.x, x * k[0]);
    s.y = fmaf(a, s.y, x * k[1]);
    s.z = fmaf(a, s.z, x * k[2]);
    s.w = fmaf(a, s.w, x * k[3]);
    if (in) *(float4*)(p.state_out + at) = s;
    float o = fmaf(s.x, q[0], fmaf(s.y, q[1], fmaf(s.z, q[2], s.w * q[3])));
#pragma unroll
    for (int d = LPR / 2; d > 0; d >>= 1) o += __shfl_xor_sync(0xffffffffu, o, d);
    if (sub == 0 && v < p.dv)
      ((T*)p.o)[((long long)b * p.H + h) * p.dv + v] = from_f32<T>(row >= 0 ? p.scale * o : 0.f);
  }
}

template <typename T>
cudaError_t step_t(const LaStep& p, cudaStream_t s) {
  const dim3 grid((p.dv + kStepRows - 1) / kStepRows, p.H, p.B);
  const int lanes = p.dk / 4;
  LaunchScope ls("linattn_step", s);
  if (lanes <= 4) k_la_step<T, 4><<<grid, kStepWarps * 32, 0, s>>>(p);
  else if (lanes <= 8) k_la_step<T, 8><<<grid, kStepWarps * 32, 0, s>>>(p);
  else if (lanes <= 16) k_la_step<T, 16><<<grid, kStepWarps * 32, 0, s>>>(p);
  else k_la_step<T, 32><<<grid, kStepWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t la_scratch_floats(int B, int H, int T, int dk, int dv, bool bf16) {
  return bf16 ? la_tc_scratch_floats(B, H, T, dk, dv) : 0;
}

cudaError_t la_walk(const LaWalk& w, bool bf16, float* scratch, cudaStream_t s) {
  if (bf16) return la_walk_tc(w, scratch, s);
  const size_t smem =
      sizeof(float) * ((size_t)2 * kC * (w.dk + 1) + (size_t)kC * (w.dv + 1) + kC * (kC + 1) +
                       (size_t)w.dv * (w.dk + 1));
  cudaError_t e =
      cudaFuncSetAttribute(k_la_walk, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(w.reverse ? "linattn_walk_back" : "linattn_walk", s);
  k_la_walk<<<dim3(w.H, w.B), kThreads, smem, s>>>(w);
  return cudaGetLastError();
}

cudaError_t la_group_sum(long long rows, int G, int share, int D, bool bf16, const float* part,
                         void* out, cudaStream_t s) {
  const long long n = rows * G * D;
  const long long want = (n + 255) / 256;
  const int grid = (int)(want < 8192 ? want : 8192);
  LaunchScope ls("linattn_group_sum", s);
  if (bf16) k_la_group_sum<<<grid, 256, 0, s>>>(n, share, D, part, (__nv_bfloat16*)out);
  else k_la_group_sum<<<grid, 256, 0, s>>>(n, share, D, part, (float*)out);
  return cudaGetLastError();
}

cudaError_t la_step(const LaStep& p, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace ssd
