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
namespace delta3 {

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

// Per step of a chunk: the sum g of the log decays (of base 2), as two floats, so that
// a difference of two sums is good to its own last bit however long they have grown;
// the write strength; and e^g, e^{G-g}.
template <int C>
struct alignas(16) Gates {
  float hi[C], lo[C], beta[C], lead[C], tail[C];
  float last;  // e^G
};

struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^x: the hardware's (2^-22) with the second float's share
__device__ __forceinline__ float exp2_of(Two x) {
  const float e = exp2_fast(x.hi);
  return fmaf(e, x.lo * 0.693147181f, e);
}

// A warp's gates of a chunk on their way: C / 32 steps a lane.
template <int C>
struct RawGates {
  float decay[C / 32], beta[C / 32];
};
// (log decays of base 2; below -200 a log decay is as good as -inf, as e^-104 is the
// smallest float, and keeps sums finite; NaN stays; past n 0)
template <int C>
__device__ __forceinline__ void load_gates(RawGates<C>& x, const float* log_decay, const float* beta,
                                           long long at, long long stride, int n, int lane) {
#pragma unroll
  for (int i = 0; i < C / 32; ++i) {
    const int r = lane * (C / 32) + i;
    float d = 0.f, b = 0.f;
    if (r < n) {
      d = log_decay[at + r * stride];
      b = beta[at + r * stride];
    }
    x.decay[i] = d < -200.f ? -200.f : d;
    x.beta[i] = b;
  }
}
template <int C>
__device__ __forceinline__ void scan_gates(Gates<C>& g, const RawGates<C>& raw, int lane) {
  constexpr int N = C / 32;
  constexpr float kLog2e = 1.44269504f, kLog2eLo = 1.92596303e-8f;  // their sum: 48 bits
  Two s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = raw.decay[i], hi = d * kLog2e;
    s[i] = {hi, fmaf(d, kLog2e, -hi) + d * kLog2eLo};
    if (i) s[i] = add(s[i ? i - 1 : 0], s[i]);
  }
  Two before = s[N - 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two x = {__shfl_up_sync(0xffffffffu, before.hi, o), __shfl_up_sync(0xffffffffu, before.lo, o)};
    if (lane >= o) before = add(x, before);
  }
  const Two total = {__shfl_sync(0xffffffffu, before.hi, 31), __shfl_sync(0xffffffffu, before.lo, 31)};
  before = {__shfl_up_sync(0xffffffffu, before.hi, 1), __shfl_up_sync(0xffffffffu, before.lo, 1)};
  if (lane == 0) before = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Two x = add(before, s[i]), rest = add(total, {-x.hi, -x.lo});
    const int r = lane * N + i;
    g.hi[r] = x.hi;
    g.lo[r] = x.lo;
    g.beta[r] = raw.beta[i];
    g.lead[r] = exp2_of(x);
    g.tail[r] = exp2_of(rest);
  }
  if (lane == 0) g.last = exp2_of(total);
}
// Gamma_ij
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
  return exp2_fast((hi_i - hi_j) + (lo_i - lo_j));
}

// What the walks read of a chunk besides its operands, in parts (tiles [C][C]): in M
// -L below the blocks of 16 on the diagonal and in them -X^T, and P.
constexpr int kDiag = 20;  // floats of a column of a diagonal block
template <int C>
struct alignas(16) Scratch {
  float diag[C / 16][16][kDiag];  // L[i][j] at [j][i], a warp each
};

// One block of 16 x 16 of A K^T, rows 16 bi ..., columns 16 bj ..., times the decays
// and `factor`: to the tile `out` in PO parts, or to `diag`, transposed.  On the
// diagonal what lies above it is zero (kL: and on it).
template <int NI, int DK, int PO, bool kDiagL>
__device__ __forceinline__ void score_block(uint32_t A, uint32_t K, uint8_t* out,
                                            const Gates<kSteps<NI>>& g, float (*diag)[kDiag], int bi,
                                            int bj, float factor, int lane) {
  constexpr int C = kSteps<NI>, RB = DK * 2, OB = C * 2;
  float acc[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  constexpr int U = NI == 1 ? DK / 16 : 2;  // (every operand of a bf16 block on its way at once)
#pragma unroll(U)
  for (int k = 0; k < DK; k += 16) {
    uint32_t a[NI][4], b[NI][2][2];
#pragma unroll
    for (int p = 0; p < NI; ++p) ldm4(a[p], A + p * C * RB + left<RB>(lane, 16 * bi, k));
    load_right<RB, NI, 2>(b, K, C * RB, lane, 16 * bj, k);
    mma_parts<NI, NI, 2>(acc, a, b);
  }
  const int c0 = (lane & 3) * 2, i0 = 16 * bi + (lane >> 2);
  const float hi0 = g.hi[i0], lo0 = g.lo[i0], hi1 = g.hi[i0 + 8], lo1 = g.lo[i0 + 8];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int j = 16 * bj + 8 * n + c0;
    const float2 hj = *(const float2*)&g.hi[j], lj = *(const float2*)&g.lo[j];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + 8 * u;
      const float hi = u ? hi1 : hi0, lo = u ? lo1 : lo0;
      float x = acc[n][2 * u] * factor * decay(hi, lo, hj.x, lj.x);
      float y = acc[n][2 * u + 1] * factor * decay(hi, lo, hj.y, lj.y);
      if (kDiagL ? j >= i : j > i) x = 0.f;
      if (kDiagL ? j + 1 >= i : j + 1 > i) y = 0.f;
      if constexpr (kDiagL) {
        diag[j & 15][i & 15] = x;
        diag[(j & 15) + 1][i & 15] = y;
      } else {
        uint32_t p[PO];
        split2<PO>(x, y, p);
        uint8_t* at = out + at16<OB>(i, 2 * bj + n) + c0 * 2;
#pragma unroll
        for (int q = 0; q < PO; ++q) *(uint32_t*)(at + q * C * OB) = p[q];
      }
    }
  }
}

// Lanes 0 - 15, a column j each of diagonal block s: with T = (I + beta L)^-1, X = L T
// and T = I - beta X, so once X_mj is whole, T_mj = -beta_m X_mj (1 for m = j) adds
// L_im T_mj to every later X_ij.
template <int C>
__device__ __forceinline__ void invert_diag(uint8_t* out, const Gates<C>& g, const float (*diag)[kDiag],
                                            int s, int j) {
  constexpr int OB = C * 2;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
  for (int m = 0; m < 15; ++m) {
    const float t = m == j ? 1.f : -g.beta[16 * s + m] * x[m];
#pragma unroll
    for (int i = (m + 1) / 4 * 4; i < 16; i += 4) {
      const float4 l = *(const float4*)&diag[m][i];
      if (i > m) x[i] = fmaf(l.x, t, x[i]);
      if (i + 1 > m) x[i + 1] = fmaf(l.y, t, x[i + 1]);
      if (i + 2 > m) x[i + 2] = fmaf(l.z, t, x[i + 2]);
      if (i + 3 > m) x[i + 3] = fmaf(l.w, t, x[i + 3]);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4][kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<kParts>(-x[8 * h + 2 * i], -x[8 * h + 2 * i + 1], p[i]);
    uint8_t* at = out + at16<OB>(16 * s + j, 2 * s + h);
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      *(uint4*)(at + q * C * OB) = make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
  }
}

// M and, with kP, P times `scale` of a chunk whose operands and gates are in shared
// memory, by the kPrep threads: a warp takes one of L's diagonal blocks and inverts
// it, then its share of the other blocks of L and of P.  (The blocks go through one
// loop: as straight code with the strips known at compile time the four warps' code
// and the walk's did not fit the instruction caches together, and waiting for
// instructions was the largest of all stalls.)  The last warp has `aside` to do as
// well (the gates of a later chunk).
template <int NI, int DK, int PP, bool kP, typename F>
__device__ __forceinline__ void prepare(const uint8_t* Qt, const uint8_t* Kt, uint8_t* M, uint8_t* P,
                                        const Gates<kSteps<NI>>& g, Scratch<kSteps<NI>>& sc,
                                        float scale, int tid, F aside) {
  constexpr int C = kSteps<NI>, NB = C / 16, W = kPrep / 32;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t K = smem32(Kt), Q = smem32(Qt);
  if (warp < NB) {
    score_block<NI, DK, kParts, true>(K, K, nullptr, g, sc.diag[warp], warp, warp, 1.f, lane);
    __syncwarp();
    if (lane < 16) invert_diag<C>(M, g, sc.diag[warp], warp, lane);
    __syncwarp();
  }
  // L's blocks below the diagonal, rows and columns (hexadecimal digits, the first one last)
  constexpr uint32_t kLi = NB == 4 ? 0x333221 : 0x1, kLj = NB == 4 ? 0x210100 : 0x0;
  constexpr uint64_t kPi = NB == 4 ? 0x3333222110ull : 0x110, kPj = NB == 4 ? 0x3210210100ull : 0x100;
  constexpr int nL = NB * (NB - 1) / 2, nP = NB * (NB + 1) / 2;
#pragma unroll 1
  for (int r = warp; r < nL; r += W)
    score_block<NI, DK, kParts, false>(K, K, M, g, nullptr, kLi >> 4 * r & 15, kLj >> 4 * r & 15, -1.f,
                                       lane);
  if constexpr (kP) {
    // (in the order that leaves every warp the same number of blocks)
#pragma unroll 1
    for (int r = (warp + W - nL % W) % W; r < nP; r += W)
      score_block<NI, DK, PP, false>(Q, K, P, g, nullptr, kPi >> 4 * r & 15, kPj >> 4 * r & 15, scale,
                                     lane);
  }
  if (warp == W - 1) aside();
}

}  // namespace delta3
}  // namespace ssd
