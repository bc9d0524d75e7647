// Gated delta rule: the gradients of q, k, the decays and the write strengths of
// every chunk, from the state H before it, the gradient D of the state after it, E
// and y (ssd_delta.cuh, ssd_delta.cu have the formulas), no chunk waiting for
// another.  With dv = beta y, U = beta E,
//   MP_ij = s Gamma_ij dO_i . U_j (j <= i),  ML_ij = -Gamma_ij dv_i . U_j (j < i)
//   dq = s e^g dO H + MP K
//   dk = r + w,  r = ML K - e^g dv H,  w = MP^T Q + ML^T K + e^{G-g} U D
//   dbeta_i = E_i . y_i
// e^{g_i} stands with q_i and with k_i where it is read, e^{-g_i} with k_i where it
// is written, and e^G with the state that is handed on, so
//   dg_i = q_i . dq_i + k_i . r_i - k_i . w_i,  dG = <H', D>
//   <H', D> = e^G <H, D> + sum_j k_j . (e^{G-g} U D)_j
// and a step's log decay gets the sum of dg from it to the chunk's end.  These terms
// cancel to a thirtieth of their size or less, which is why every operand here has
// all its parts; two parts (2^-17) gave 9e-5 of dlog_decay.
//
// One CTA per (chunk, head, row), eight warps: 16 rows (steps) and a share of the
// columns each; operands of 64 columns of v at a time.  Heads that share q and k
// write their own gradients in fp32, summed in head order by a second kernel.
#include <cuda_bf16.h>

#include "ssd_delta3.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace delta3;

constexpr int kThreads = 256;

template <int NI, int DK>
struct Geom {
  static constexpr int C = kSteps<NI>;
  static constexpr int RB = DK * 2, VR = kVB * 2, PB = C * 2;
  static constexpr int KT = NI * C * RB;                 // Q, K
  static constexpr int OT = NI * C * VR;                 // dO
  static constexpr int HT = kParts * kVB * RB;           // H, D
  static constexpr int UT = kParts * C * VR;             // U, dv
  static constexpr int MT = kParts * C * PB;             // MP, ML: in the place of H, D
  static_assert(MT <= HT, "");
  static constexpr int kK = KT, kO = 2 * KT, kH = kO + OT, kD = kH + HT, kU = kD + HT, kV = kU + UT;
  static constexpr size_t smem = kV + UT;
  static constexpr int WR = C / 16, WC = 8 / WR;         // strips of rows, groups of columns
  static constexpr int NK = DK / 8 / WC;                 // eights of columns of dq, dk of a warp
  static constexpr int NM = C / 8 / (WC / 2);            // of MP or ML
};

// a row-major tile's two elements at (row, column c, c + 1)
template <int NI, int RB, int C>
__device__ __forceinline__ float2 pair_at(const uint8_t* tile, int row, int c) {
  const uint8_t* at = tile + at16<RB>(row, c >> 3) + (c & 7) * 2;
  float2 f = make_float2(0.f, 0.f);
#pragma unroll
  for (int p = NI - 1; p >= 0; --p) {
    const uint32_t x = *(const uint32_t*)(at + p * C * RB);
    f.x += __uint_as_float(x << 16);
    f.y += __uint_as_float(x & 0xffff0000u);
  }
  return f;
}

// sum over 16 lanes
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <typename T>
__device__ __forceinline__ void put_pair(T* at, float x, float y) {
  if constexpr (sizeof(T) == 2) *(uint32_t*)at = pack2(x, y);
  else *(float2*)at = make_float2(x, y);
}

// kShared: dq, dk of the head in fp32 to part (dq's, then dk's, [B][T][H][dk])
template <int NI, int DK, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) k_delta_grads(const DeltaGrads p, float* part) {
  using G = Geom<NI, DK>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  using TO = typename std::conditional<kShared, float, T>::type;
  constexpr int C = G::C, RB = G::RB, VR = G::VR, PB = G::PB, NK = G::NK, NM = G::NM, NB = C / 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ Gates<C> g;
  __shared__ float dbeta[C], red[G::WC][C], sums[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int h = blockIdx.y, b = blockIdx.z, t0 = blockIdx.x * C;
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const int n = min(C, len - t0), rows = min(C, p.T - t0);
  const long long token = (long long)b * p.T + t0;
  // where dq and dk go: rows of `heads` heads
  const int heads = kShared ? p.H : p.G;
  TO* dq_out = (kShared ? (TO*)part : (TO*)p.dq) + (token * heads + h) * p.dk;
  TO* dk_out = (kShared ? (TO*)(part + (long long)p.B * p.T * p.H * p.dk) : (TO*)p.dk_out) +
               (token * heads + h) * p.dk;
  const long long out_step = (long long)heads * p.dk;
  // past the row's end: zeros
  const int z0 = max(n, 0);
  for (int i = tid; i < (rows - z0) * (p.dk / 8); i += kThreads) {
    const int r = z0 + i / (p.dk / 8), c = i % (p.dk / 8) * 8;
#pragma unroll
    for (int e = 0; e < 8; e += 16 / (int)sizeof(TO)) {
      *(uint4*)(dq_out + r * out_step + c + e) = make_uint4(0, 0, 0, 0);
      *(uint4*)(dk_out + r * out_step + c + e) = make_uint4(0, 0, 0, 0);
    }
  }
  const long long gate0 = token * p.H + h;
  for (int r = z0 + tid; r < rows; r += kThreads)
    p.dlog_decay[gate0 + (long long)r * p.H] = p.dbeta[gate0 + (long long)r * p.H] = 0.f;
  if (n <= 0) return;
  const int chunks = (p.T + C - 1) / C;
  const long long unit = ((long long)b * p.H + h) * chunks + blockIdx.x;
  const float* hs = p.hist_s + unit * p.dv * p.dk;
  const float* hd = p.hist_d + unit * p.dv * p.dk;
  const float* ep = p.err + unit * C * p.dv;
  const float* yp = p.y + unit * C * p.dv;
  const T* qp = (const T*)p.q.p + b * p.q.batch + t0 * p.q.step + (long long)(h / p.q.share) * p.dk;
  const T* kp = (const T*)p.k.p + b * p.k.batch + t0 * p.k.step + (long long)(h / p.k.share) * p.dk;
  const T* gp = (const T*)p.dout.p + b * p.dout.batch + t0 * p.dout.step + (long long)h * p.dv;
  load_tile<NI, C, DK, kThreads>(sm, qp, p.q.step, n, p.dk, tid);
  load_tile<NI, C, DK, kThreads>(sm + G::kK, kp, p.k.step, n, p.dk, tid);
  if (tid < C) dbeta[tid] = 0.f;
  if (warp == 0) {
    RawGates<C> raw;
    load_gates<C>(raw, p.log_decay, p.beta, gate0, p.H, n, lane);
    scan_gates<C>(g, raw, lane);
  }
  __syncthreads();
  const int strip = warp % G::WR, group = warp / G::WR;
  const bool is_l = group >= G::WC / 2;        // this warp's scores: ML's, else MP's
  const int mg = group % (G::WC / 2);
  const int m0 = mg * NM;                      // their first eight of columns
  const uint32_t sQ = smem32(sm), sK = sQ + G::kK, sO = sQ + G::kO, sH = sQ + G::kH,
                 sD = sQ + G::kD, sU = sQ + G::kU, sV = sQ + G::kV;
  float dq[NK][4], rd[NK][4], wr[NK][4], mm[NM][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int i = 0; i < NK; ++i) dq[i][e] = rd[i][e] = wr[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NM; ++i) mm[i][e] = 0.f;
  }
  float hdot = 0.f;  // <H, D>
  for (int v0 = 0; v0 < p.dv; v0 += kVB) {
    const int width = min(kVB, p.dv - v0);
    if (v0) __syncthreads();
    load_tile<NI, C, kVB, kThreads>(sm + G::kO, gp + v0, p.dout.step, n, width, tid);
    if (NI == 1) copy_commit();
#pragma unroll 2
    for (int i = tid; i < kVB * (DK / 4); i += kThreads) {
      const int r = i / (DK / 4), x = i % (DK / 4);
      const bool in = r < width && x * 4 < p.dk;
      const long long at = (long long)(v0 + r) * p.dk + x * 4;
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 s = in ? *(const float4*)(hs + at) : z, d = in ? *(const float4*)(hd + at) : z;
      hdot = fmaf(s.x, d.x, fmaf(s.y, d.y, fmaf(s.z, d.z, fmaf(s.w, d.w, hdot))));
      uint8_t* to = sm + G::kH + at16<RB>(r, x >> 1) + (x & 1) * 8;
      uint32_t a[kParts], c[kParts];
      split2<kParts>(s.x, s.y, a);
      split2<kParts>(s.z, s.w, c);
#pragma unroll
      for (int q = 0; q < kParts; ++q) *(uint2*)(to + q * kVB * RB) = make_uint2(a[q], c[q]);
      split2<kParts>(d.x, d.y, a);
      split2<kParts>(d.z, d.w, c);
      to += G::HT;
#pragma unroll
      for (int q = 0; q < kParts; ++q) *(uint2*)(to + q * kVB * RB) = make_uint2(a[q], c[q]);
    }
#pragma unroll
    for (int i0 = 0; i0 < C * (kVB / 4); i0 += kThreads) {
      const int i = i0 + tid, r = i / (kVB / 4), x = i % (kVB / 4);
      float4 e = make_float4(0.f, 0.f, 0.f, 0.f), y = e;
      if (x * 4 < width) {
        e = *(const float4*)(ep + (long long)r * p.dv + v0 + x * 4);
        y = *(const float4*)(yp + (long long)r * p.dv + v0 + x * 4);
      }
      const float d = sum16(fmaf(e.x, y.x, fmaf(e.y, y.y, fmaf(e.z, y.z, e.w * y.w))));
      if (x == 0) dbeta[r] += d;
      const float be = g.beta[r];
      uint8_t* to = sm + G::kU + at16<VR>(r, x >> 1) + (x & 1) * 8;
      uint32_t a[kParts], c[kParts];
      split2<kParts>(be * e.x, be * e.y, a);
      split2<kParts>(be * e.z, be * e.w, c);
#pragma unroll
      for (int q = 0; q < kParts; ++q) *(uint2*)(to + q * C * VR) = make_uint2(a[q], c[q]);
      split2<kParts>(be * y.x, be * y.y, a);
      split2<kParts>(be * y.z, be * y.w, c);
      to += G::UT;
#pragma unroll
      for (int q = 0; q < kParts; ++q) *(uint2*)(to + q * C * VR) = make_uint2(a[q], c[q]);
    }
    copy_wait<0>();
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < width; k += 16) {
      uint32_t ao[NI][4], au[kParts][4], av[kParts][4];
#pragma unroll
      for (int q = 0; q < NI; ++q) ldm4(ao[q], sO + q * C * VR + left<VR>(lane, 16 * strip, k));
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        ldm4(au[q], sU + q * C * VR + left<VR>(lane, 16 * strip, k));
        ldm4(av[q], sV + q * C * VR + left<VR>(lane, 16 * strip, k));
      }
#pragma unroll
      for (int i = 0; i < NK; i += 2) {
        const int c = (group * NK + i) * 8;
        uint32_t r[kParts][2][2];
        load_right_t<RB, kParts, 2>(r, sH, kVB * RB, lane, c, k);
        mma_parts<NI, kParts, 2>(dq + i, ao, r);
        mma_parts<kParts, kParts, 2>(rd + i, av, r);
        load_right_t<RB, kParts, 2>(r, sD, kVB * RB, lane, c, k);
        mma_parts<kParts, kParts, 2>(wr + i, au, r);
      }
#pragma unroll
      for (int i = 0; i < NM; i += 2)
        if (m0 + i <= 2 * strip) {
          uint32_t r[kParts][2][2];
          load_right<VR, kParts, 2>(r, sU, C * VR, lane, 8 * (m0 + i), k);
          if (is_l) mma_parts<kParts, kParts, 2>(mm + i, av, r);
          else mma_parts<NI, kParts, 2>(mm + i, ao, r);
        }
    }
  }
  __syncthreads();  // H and D have been read
  const int i0 = 16 * strip + (lane >> 2), c2 = (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < NM; ++i)
    if (m0 + i <= 2 * strip + 1) {
      const int col = 8 * (m0 + i) + c2;
      const float2 hj = *(const float2*)&g.hi[col], lj = *(const float2*)&g.lo[col];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = i0 + 8 * u;
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = is_l ? col + e < row : col + e <= row;
          x[e] = in ? mm[i][2 * u + e] * (is_l ? -1.f : p.scale) *
                          decay(g.hi[row], g.lo[row], e ? hj.y : hj.x, e ? lj.y : lj.x)
                    : 0.f;
        }
        uint32_t a[kParts];
        split2<kParts>(x[0], x[1], a);
        uint8_t* at = sm + (is_l ? G::kD : G::kH) + at16<PB>(row, m0 + i) + c2 * 2;
#pragma unroll
        for (int q = 0; q < kParts; ++q) *(uint32_t*)(at + q * C * PB) = a[q];
      }
    }
  float state_dot = 0.f;  // sum over this warp's rows and columns of k . (e^{G-g} U D)
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float l = g.lead[i0 + 8 * u], t = g.tail[i0 + 8 * u];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const float2 kk = pair_at<NI, RB, C>(sm + G::kK, i0 + 8 * u, (group * NK + i) * 8 + c2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dq[i][2 * u + e] *= p.scale * l;
        rd[i][2 * u + e] *= -l;
        wr[i][2 * u + e] *= t;
        state_dot = fmaf(e ? kk.y : kk.x, wr[i][2 * u + e], state_dot);
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < NB; ++k) {
    if (k <= strip) {  // columns 16 k ... of MP, ML
      uint32_t ap[kParts][4], al[kParts][4];
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        ldm4(ap[q], sH + q * C * PB + left<PB>(lane, 16 * strip, 16 * k));
        ldm4(al[q], sD + q * C * PB + left<PB>(lane, 16 * strip, 16 * k));
      }
#pragma unroll
      for (int i = 0; i < NK; i += 2) {
        uint32_t r[NI][2][2];
        load_right_t<RB, NI, 2>(r, sK, C * RB, lane, (group * NK + i) * 8, 16 * k);
        mma_parts<kParts, NI, 2>(dq + i, ap, r);
        mma_parts<kParts, NI, 2>(rd + i, al, r);
      }
    }
    if (k >= strip) {  // rows 16 k ...
      uint32_t ap[kParts][4], al[kParts][4];
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        ldm4t(ap[q], sH + q * C * PB + left_t<PB>(lane, 16 * strip, 16 * k));
        ldm4t(al[q], sD + q * C * PB + left_t<PB>(lane, 16 * strip, 16 * k));
      }
#pragma unroll
      for (int i = 0; i < NK; i += 2) {
        uint32_t r[NI][2][2];
        load_right_t<RB, NI, 2>(r, sQ, C * RB, lane, (group * NK + i) * 8, 16 * k);
        mma_parts<kParts, NI, 2>(wr + i, ap, r);
        load_right_t<RB, NI, 2>(r, sK, C * RB, lane, (group * NK + i) * 8, 16 * k);
        mma_parts<kParts, NI, 2>(wr + i, al, r);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int row = i0 + 8 * u;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int c = (group * NK + i) * 8 + c2;
      const float2 q = pair_at<NI, RB, C>(sm, row, c), k = pair_at<NI, RB, C>(sm + G::kK, row, c);
      const float *x = &dq[i][2 * u], *r = &rd[i][2 * u], *w = &wr[i][2 * u];
      s += fmaf(q.x, x[0], k.x * (r[0] - w[0])) + fmaf(q.y, x[1], k.y * (r[1] - w[1]));
      if (row < n && c < p.dk) {
        put_pair(dq_out + row * out_step + c, x[0], x[1]);
        put_pair(dk_out + row * out_step + c, r[0] + w[0], r[1] + w[1]);
      }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if ((lane & 3) == 0) red[group][row] = s;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    hdot += __shfl_xor_sync(0xffffffffu, hdot, d);
    state_dot += __shfl_xor_sync(0xffffffffu, state_dot, d);
  }
  if (lane == 0) {
    sums[0][warp] = hdot;
    sums[1][warp] = state_dot;
  }
  __syncthreads();
  if (warp == 0) {
    // dg, and its sums from each step to the end, in 64 bits (they cancel)
    constexpr int N = C / 32;
    double x[N], total = 0.0, last = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) last += (double)g.last * sums[0][i] + sums[1][i];
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
      const int r = lane * N + i;
      double d = 0.0;
#pragma unroll
      for (int c = 0; c < G::WC; ++c) d += red[c][r];
      if (r == C - 1) d += last;
      total += d;
      x[i] = total;
    }
    double after = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_down_sync(0xffffffffu, after, o);
      if (lane + o < 32) after += y;
    }
    after = __shfl_down_sync(0xffffffffu, after, 1);
    if (lane == 31) after = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = lane * N + i;
      if (r < n) p.dlog_decay[gate0 + (long long)r * p.H] = (float)(x[i] + after);
    }
  }
  if (tid < n) p.dbeta[gate0 + (long long)tid * p.H] = dbeta[tid];
}

// part [2][rows][G][share][D] -> dq, dk [rows][G][D], a group's heads in order;
// four elements a thread
template <typename T>
__global__ void __launch_bounds__(256) k_delta_group_sum(long long n, int share, int D,
                                                         const float* __restrict__ part, T* dq, T* dk) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < 2 * n;
       i += (long long)gridDim.x * 256) {
    const long long e = (i < n ? i : i - n) * 4;
    const float* p = part + (i < n ? 0 : n * 4 * share) + e / D * share * D + e % D;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < share; ++j) {
      const float4 f = *(const float4*)(p + (long long)j * D);
      s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
    }
    T* to = (i < n ? dq : dk) + e;
    put_pair(to, s.x, s.y);
    put_pair(to + 2, s.z, s.w);
  }
}

template <int NI, int DK, bool kShared>
cudaError_t grads_s(const DeltaGrads& p, float* part, cudaStream_t s) {
  using G = Geom<NI, DK>;
  static_assert(G::smem + 4096 <= 232448, "");
  const cudaError_t e = cudaFuncSetAttribute(k_delta_grads<NI, DK, kShared>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls("delta_grads", s);
  k_delta_grads<NI, DK, kShared>
      <<<dim3((p.T + G::C - 1) / G::C, p.H, p.B), kThreads, G::smem, s>>>(p, part);
  return cudaGetLastError();
}

template <int NI, int DK>
cudaError_t grads_t(const DeltaGrads& p, float* part, cudaStream_t s) {
  if (p.H == p.G) return grads_s<NI, DK, false>(p, part, s);
  const cudaError_t e = grads_s<NI, DK, true>(p, part, s);
  if (e != cudaSuccess) return e;
  const long long n = (long long)p.B * p.T * p.G * (p.dk / 4), want = (2 * n + 255) / 256;
  LaunchScope ls("delta_group_sum", s);
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  k_delta_group_sum<T><<<(int)(want < 8192 ? want : 8192), 256, 0, s>>>(n, p.H / p.G, p.dk, part,
                                                                       (T*)p.dq, (T*)p.dk_out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_grads(const DeltaGrads& p, float* part, bool bf16, cudaStream_t s) {
  if (bf16) return p.dk <= 64 ? grads_t<1, 64>(p, part, s) : grads_t<1, 128>(p, part, s);
  return p.dk <= 64 ? grads_t<3, 64>(p, part, s) : grads_t<3, 128>(p, part, s);
}

}  // namespace ssd
