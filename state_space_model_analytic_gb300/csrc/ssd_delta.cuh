// What the kernels of the gated delta rule share: products of operands that are
// carried as several bf16 parts, and what a chunk of steps needs besides its
// operands.
//
// The rule: e_t = v_t - a_t S_{t-1} k_t, S_t = a_t S_{t-1} + beta_t e_t k_t^T,
// o_t = s S_t q_t, with a_t = e^{log_decay_t}.  In a chunk of C steps, with g_i
// the sum of the log decays up to step i, Gamma_ij = e^{g_i - g_j} for j <= i, H
// the state before the chunk ([dv][dk]) and L_ij = Gamma_ij k_i . k_j for j < i,
//   F = V - e^g K H^T,  (I + L beta) E = F,  U = beta E
//   O = s e^g Q H^T + P U,  P_ij = s Gamma_ij q_i . k_j for j <= i
//   H <- e^G H + U^T (e^{G-g} K),  G = g at the last step
// E is found by forward substitution over blocks of 16 steps: inside a block
// (I + L beta)^-1 = I - X beta, X = L (I + beta L)^-1 (strictly lower), and what a
// solved block contributes is taken off the later ones.  (An inverse of the whole
// chunk by repeated squaring would lose everything to cancellation where keys are
// alike: powers of L grow like binomials.)
//
// Precision: every operand of a matrix instruction is a sum of bf16 parts of 8
// significant bits, exact for bf16 tensors and three parts for everything held in
// 32 bits; of the products of parts those up to 2^-16 are formed, what is left out
// is below 2^-24 of the product.  Sums are fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd_common.cuh"
#include "ssd_layer_internal.h"

namespace ssd {
namespace delta {

constexpr int kPrep = 128;   // threads that prepare the next chunk
constexpr int kVB = 64;      // columns of v of a CTA: up to four warps of 16
constexpr int kParts = 3;    // parts of a value held in 32 bits

// Byte offset of a 16-byte piece of a tile whose rows are RB bytes: pieces of
// eight consecutive rows fall on all 32 banks.
template <int RB>
__device__ __forceinline__ uint32_t at16(int row, int piece) {
  if constexpr (RB >= 128) return row * RB + ((piece ^ (row & 7)) << 4);
  if constexpr (RB == 64) return row * RB + ((piece ^ ((row >> 1) & 3)) << 4);
  return row * RB + ((piece ^ ((row >> 2) & 1)) << 4);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// two values as N bf16 parts each
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = pack2(x, y);
    x -= __uint_as_float(p[i] << 16);
    y -= __uint_as_float(p[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t smem32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // 8 x 8 of 16 bits
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// d += a b, 16 x 16 times 16 x 8.  With g = lane / 4, t = lane % 4: d row g,
// columns 2 t and 2 t + 1, then row g + 8; a row g, terms 2 t and 2 t + 1, row
// g + 8, then both at terms + 8; b terms 2 t and 2 t + 1 of column g, then + 8.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where lane `lane` points for the four 8 x 8 pieces of ldmatrix, in a tile with
// rows of RB bytes:
// rows m, terms along the row: a left operand of rows m ... m + 15, terms k ... k + 15
template <int RB>
__device__ __forceinline__ uint32_t left(int lane, int m, int k) {
  return at16<RB>(m + (lane & 15), (k >> 3) + (lane >> 4));
}
// terms down the rows: the same left operand from its transpose
template <int RB>
__device__ __forceinline__ uint32_t left_t(int lane, int m, int k) {
  return at16<RB>(k + (lane & 7) + (lane >> 4 << 3), (m >> 3) + (lane >> 3 & 1));
}
// columns n down the rows, terms along them: right operands of columns n ... n + 7
// (r[0], r[1]) and n + 8 ... (r[2], r[3])
template <int RB>
__device__ __forceinline__ uint32_t right(int lane, int n, int k) {
  return at16<RB>(n + (lane & 7) + (lane >> 4 << 3), (k >> 3) + (lane >> 3 & 1));
}
// terms down the rows
template <int RB>
__device__ __forceinline__ uint32_t right_t(int lane, int n, int k) {
  return at16<RB>(k + (lane & 7) + ((lane >> 3 & 1) << 3), (n >> 3) + (lane >> 4));
}

// d[n] += a b[n] for N columns of eight, all products of parts i + j < max(PA, PB),
// the small ones first; the columns take turns, since an instruction waits for the
// one before it on the same sum.
template <int PA, int PB, int N>
__device__ __forceinline__ void mma_parts(float (*d)[4], const uint32_t (&a)[PA][4],
                                          const uint32_t (&b)[PB][N][2]) {
  constexpr int M = PA > PB ? PA : PB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        if (i + j == s)
#pragma unroll
          for (int n = 0; n < N; ++n) mma(d[n], a[i], b[j][n][0], b[j][n][1]);
}
// right operands of N (even) columns of eight, PB parts `step` bytes apart
template <int RB, int PB, int N>
__device__ __forceinline__ void load_right(uint32_t (&b)[PB][N][2], uint32_t tile, uint32_t step,
                                           int lane, int n, int k) {
#pragma unroll
  for (int p = 0; p < PB; ++p)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t r[4];
      ldm4(r, tile + p * step + right<RB>(lane, n + 8 * i, k));
      b[p][i][0] = r[0];
      b[p][i][1] = r[1];
      b[p][i + 1][0] = r[2];
      b[p][i + 1][1] = r[3];
    }
}
template <int RB, int PB, int N>
__device__ __forceinline__ void load_right_t(uint32_t (&b)[PB][N][2], uint32_t tile, uint32_t step,
                                             int lane, int n, int k) {
#pragma unroll
  for (int p = 0; p < PB; ++p)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t r[4];
      ldm4t(r, tile + p * step + right_t<RB>(lane, n + 8 * i, k));
      b[p][i][0] = r[0];
      b[p][i][1] = r[1];
      b[p][i + 1][0] = r[2];
      b[p][i + 1][1] = r[3];
    }
}
// Two columns of eight of a product's result as the left operand of 16 terms of
// the next one.
template <int P>
__device__ __forceinline__ void as_left(uint32_t (&a)[P][4], const float (&x)[4], const float (&y)[4]) {
  uint32_t r[P];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    split2<P>(x[2 * e], x[2 * e + 1], r);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][e] = r[p];
    split2<P>(y[2 * e], y[2 * e + 1], r);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][2 + e] = r[p];
  }
}

__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem32(dst)), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- a chunk's tiles ------------------------------------------------------------

// NI: parts of an element of q, k, v (bf16: one; fp32: three).  fp32 takes chunks
// of 32 steps, since three parts of 64 would not fit beside each other.
template <int NI>
constexpr int kSteps = NI == 1 ? 64 : 32;

// C rows of D elements (a multiple of 64) as NI part tiles `C * D * 2` bytes apart,
// from rows `stride` elements apart; past row n and past `width` (a multiple of 8)
// zeros.  bf16: asynchronous copies, to be committed by the caller.
template <int NI, int C, int D, int NT>
__device__ __forceinline__ void load_tile(uint8_t* tile, const void* src, long long stride, int n,
                                          int width, int tid) {
  constexpr int RB = D * 2;
  if constexpr (NI == 1) {
    const __nv_bfloat16* s = (const __nv_bfloat16*)src;
#pragma unroll 4
    for (int i = tid; i < C * (D / 8); i += NT) {
      const int r = i / (D / 8), x = i % (D / 8);
      const bool in = r < n && x * 8 < width;
      copy16(tile + at16<RB>(r, x), in ? s + r * stride + x * 8 : s, in);
    }
  } else {
    const float* s = (const float*)src;
    constexpr int per = C * (D / 4) / NT;
    static_assert(C * (D / 4) % NT == 0, "");
#pragma unroll
    for (int b = 0; b < per; b += 8) {  // eight 16-byte loads on their way at a time
      float4 f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (b + u < per) {
          const int i = tid + (b + u) * NT, r = i / (D / 4), x = i % (D / 4);
          f[u] = r < n && x * 4 < width ? *(const float4*)(s + r * stride + x * 4)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (b + u < per) {
          const int i = tid + (b + u) * NT, r = i / (D / 4), x = i % (D / 4);
          uint32_t p[NI], q[NI];
          split2<NI>(f[u].x, f[u].y, p);
          split2<NI>(f[u].z, f[u].w, q);
          uint8_t* at = tile + at16<RB>(r, x >> 1) + (x & 1) * 8;
#pragma unroll
          for (int k = 0; k < NI; ++k) *(uint2*)(at + k * C * RB) = make_uint2(p[k], q[k]);
        }
    }
  }
}

// Per step of a chunk: the sum of the log decays as two floats (a difference of
// two sums is then good to its own last bit however long they have grown), the
// write strength, and e^g, e^{G-g}.
template <int C>
struct alignas(16) Gates {
  float hi[C], lo[C], beta[C], lead[C], tail[C];
  float last;  // e^G
};

// log_decay below -200 is as good as -inf (e^-104 is the smallest float) and keeps
// sums finite; NaN stays
__device__ __forceinline__ float clamp_decay(float x) { return x < -200.f ? -200.f : x; }

// One warp; raw: C log decays (zero past the chunk's end).
template <int C>
__device__ __forceinline__ void scan_gates(Gates<C>& g, const float* raw, int lane) {
  constexpr int N = C / 32;
  double s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = raw[lane * N + i] + (i ? s[i ? i - 1 : 0] : 0.0);
  double before = s[N - 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  const double total = __shfl_sync(0xffffffffu, before, 31);
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) before = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double x = before + s[i];
    const float hi = (float)x;
    g.hi[lane * N + i] = hi;
    g.lo[lane * N + i] = (float)(x - hi);
    g.lead[lane * N + i] = expf(hi);
    g.tail[lane * N + i] = expf((float)(total - x));
  }
  if (lane == 0) g.last = expf((float)total);
}
// Gamma_ij
template <int C>
__device__ __forceinline__ float decay(const Gates<C>& g, int i, int j) {
  return expf((g.hi[i] - g.hi[j]) + (g.lo[i] - g.lo[j]));
}

// What the walks read of a chunk besides its operands: -X in the blocks of 16 on
// the diagonal and -L below them, and P, in parts (tiles [C][C]).
constexpr int kDiag = 20;  // floats of a row of a diagonal block
template <int C>
struct alignas(16) Scratch {
  float raw[C];
  float diag[C / 16][16][kDiag];
};

// Rows 16 s ... 16 s + 15 of A K^T, columns up to the diagonal block's end, times
// the decays: -L (below the diagonal blocks to `out`, in them to the scratch), or
// factor * (values on and below the diagonal) to `out`.
template <int NI, int DK, int PO, bool kL>
__device__ __forceinline__ void scores(uint32_t A, uint32_t K, uint8_t* out, int s,
                                       const Gates<kSteps<NI>>& g, Scratch<kSteps<NI>>& sc,
                                       float factor, int lane, int wait_bar) {
  constexpr int C = kSteps<NI>, RB = DK * 2, OB = C * 2, NT = C / 8;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll 2
  for (int k = 0; k < DK; k += 16) {
    uint32_t a[NI][4];
#pragma unroll
    for (int p = 0; p < NI; ++p) ldm4(a[p], A + p * C * RB + left<RB>(lane, 16 * s, k));
#pragma unroll
    for (int n = 0; n < NT; n += 2)
      if (n <= 2 * s) {
        uint32_t b[NI][2][2];
        load_right<RB, NI, 2>(b, K, C * RB, lane, 8 * n, k);
        mma_parts<NI, NI, 2>(acc + n, a, b);
      }
  }
  if (wait_bar) bar(wait_bar, kPrep);  // the gates are there
  const int r0 = 16 * s + (lane >> 2), c0 = (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (n <= 2 * s + 1) {
      const bool diag = n >= 2 * s;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = r0 + 8 * u, j = 8 * n + c0;
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[e] = (kL ? j + e < i : j + e <= i) ? acc[n][2 * u + e] * factor * decay(g, i, j + e) : 0.f;
        if (kL && diag) {
          float* d = &sc.diag[s][i & 15][j & 15];
          d[0] = x[0];
          d[1] = x[1];
        } else {
          uint32_t p[PO];
          split2<PO>(kL ? -x[0] : x[0], kL ? -x[1] : x[1], p);
          uint8_t* at = out + at16<OB>(i, n) + c0 * 2;
#pragma unroll
          for (int q = 0; q < PO; ++q) *(uint32_t*)(at + q * C * OB) = p[q];
        }
      }
    }
}

// One thread a column of a diagonal block: with T = (I + beta L)^-1 column j by
// forward substitution, X_ij = sum_m L_im T_mj and T_ij = -beta_i X_ij.
template <int C>
__device__ __forceinline__ void invert_diag(uint8_t* out, const Gates<C>& g, const Scratch<C>& sc,
                                            int tid) {
  constexpr int OB = C * 2;
  const int s = tid >> 4, j = tid & 15;
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x = 0.f;
#pragma unroll
    for (int m = 0; m < i; m += 4) {
      const float4 l = *(const float4*)&sc.diag[s][i][m];
      x = fmaf(l.x, t[m], x);
      if (m + 1 < i) x = fmaf(l.y, t[m + 1 < 16 ? m + 1 : 0], x);
      if (m + 2 < i) x = fmaf(l.z, t[m + 2 < 16 ? m + 2 : 0], x);
      if (m + 3 < i) x = fmaf(l.w, t[m + 3 < 16 ? m + 3 : 0], x);
    }
    t[i] = i == j ? 1.f : -g.beta[16 * s + i] * x;
    uint32_t p[kParts];
    split2<kParts>(i > j ? -x : 0.f, 0.f, p);
    uint8_t* at = out + at16<OB>(16 * s + i, 2 * s + (j >> 3)) + (j & 7) * 2;
#pragma unroll
    for (int q = 0; q < kParts; ++q) *(uint16_t*)(at + q * C * OB) = (uint16_t)p[q];
  }
}

// The gates' next values of a thread (one step a thread).
struct NextGates {
  float decay = 0.f, beta = 0.f;
};
template <int C>
__device__ __forceinline__ NextGates load_gates(const float* log_decay, const float* beta,
                                                long long at, long long stride, int n, int tid) {
  NextGates x;
  if (tid < C && tid < n) {
    x.decay = clamp_decay(log_decay[at + tid * stride]);
    x.beta = beta[at + tid * stride];
  }
  return x;
}

// Everything of a chunk whose operands are in shared memory, by the kPrep threads
// (bar 1); kP: P too, times `scale`.
template <int NI, int DK, int PP, bool kP>
__device__ __forceinline__ void prepare(const uint8_t* Qt, const uint8_t* Kt, uint8_t* M, uint8_t* P,
                                        Gates<kSteps<NI>>& g, Scratch<kSteps<NI>>& sc, NextGates ng,
                                        float scale, int tid) {
  constexpr int C = kSteps<NI>, NB = C / 16;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid < C) {
    sc.raw[tid] = ng.decay;
    g.beta[tid] = ng.beta;
  }
  bar(1, kPrep);
  if (warp == 3) scan_gates<C>(g, sc.raw, lane);
  const uint32_t K = smem32(Kt), Q = smem32(Qt);
  if constexpr (kP) {
    // strips of 2, 4, 6, 8 columns of eight: the first with the last
    if (warp < 2) {
      scores<NI, DK, kParts, true>(K, K, M, warp, g, sc, 1.f, lane, 1);
      if constexpr (NB == 4) scores<NI, DK, kParts, true>(K, K, M, 3 - warp, g, sc, 1.f, lane, 0);
    } else {
      scores<NI, DK, PP, false>(Q, K, P, warp - 2, g, sc, scale, lane, 1);
      if constexpr (NB == 4) scores<NI, DK, PP, false>(Q, K, P, 5 - warp, g, sc, scale, lane, 0);
    }
  } else {
    if (warp < NB) scores<NI, DK, kParts, true>(K, K, M, warp, g, sc, 1.f, lane, 1);
    else bar(1, kPrep);
  }
  bar(1, kPrep);
  if (tid < C) invert_diag<C>(M, g, sc, tid);
}

}  // namespace delta
}  // namespace ssd
