// What the kernels of the gated delta rule share: products of operands that are
// carried as fp16 parts, and what a chunk of steps needs besides its operands.
//
// The rule: e_t = v_t - a_t S_{t-1} k_t, S_t = a_t S_{t-1} + beta_t e_t k_t^T,
// o_t = s S_t q_t, with a_t = e^{log_decay_t}.  In a chunk of C steps, with g_i
// the sum of the log decays up to step i, Gamma_ij = e^{g_i - g_j} for j <= i, H
// the state before the chunk ([dv][dk]) and L_ij = Gamma_ij k_i . k_j for j < i,
//   F = V - e^g K H^T,  (I + L beta) E = F,  U = beta E
//   O = s e^g Q H^T + s P U,  P_ij = Gamma_ij q_i . k_j for j <= i
//   H <- e^G H + U^T (e^{G-g} K),  G = g at the last step
// E is found by forward substitution over blocks of 16 steps: inside a block
// (I + L beta)^-1 = I - X beta, X = L (I + beta L)^-1 (strictly lower), and what a
// solved block contributes is taken off the later ones.  (An inverse of the whole
// chunk by repeated squaring would lose everything to cancellation where keys are
// alike: powers of L grow like binomials.)
//
// Precision: a matrix instruction takes fp16 operands of 11 significant bits and
// sums in fp32.  A value held in 32 bits is two such parts, hi + lo (22 bits), and a
// product of two of them hi hi + hi lo + lo hi; what is left out is below 2^-22 of
// it.  A bf16 element is one part.  Three bf16 parts (24 bits) need six products
// instead of three, and one more a product with a bf16 tensor; two (16 bits) left
// 4e-6 of the states and 9e-5 of dlog_decay.
//
// fp16 has few powers of two, so every operand is scaled by one.  Keys: the rule does
// not change with k 2^n, v 2^n, beta 2^-2n in place of k, v, beta for a step, and n is
// taken such that the largest element of k is in [1, 2); L, X, E and U below are those
// of the rows so scaled ("of k's scale").  Queries the same way, 2^-n going into the
// output.  Left operands (the state, U and so on) are scaled row by row, by the
// largest element.
//
// Every tile and left operand holds its values times 2^kLift more than that (L and P,
// which are below 2^9, times 2^kScore), so that the second part, whose last bit is 2^-24,
// is whole down to 2^-16 of a row's largest element; from there on an element has a bit
// less for each power of two, and below 2^-39 it is zero.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "ssd_common.cuh"
#include "ssd_layer_internal.h"

namespace ssd {
namespace delta {

constexpr int kPrep = 256;   // threads that prepare the next chunk
constexpr int kVB = 64;      // columns of v of a tile
constexpr int kParts = 2;    // parts of a value held in 32 bits
constexpr int kLift = 14, kScore = 6;

// Byte offset of a 16-byte piece of a tile whose rows are RB bytes: pieces of
// eight consecutive rows fall on all 32 banks.
template <int RB>
__device__ __forceinline__ uint32_t at16(int row, int piece) {
  if constexpr (RB >= 128) return row * RB + ((piece ^ (row & 7)) << 4);
  if constexpr (RB == 64) return row * RB + ((piece ^ ((row >> 1) & 3)) << 4);
  return row * RB + ((piece ^ ((row >> 2) & 1)) << 4);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
  return __half22float2(*(const __half2*)&x);
}
__device__ __forceinline__ float2 unpack_bf(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// two values as N fp16 parts each
template <int N>
__device__ __forceinline__ void split2(float2 x, uint32_t (&p)[N]) {
  p[0] = pack_half(x.x, x.y);
  if constexpr (N == 2) {
    const float2 r = fma2(unpack_half(p[0]), make_float2(-1.f, -1.f), x);
    p[1] = pack_half(r.x, r.y);
  }
}
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[N]) {
  split2<N>(make_float2(x, y), p);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// a product's values (columns 2 t and 2 t + 1) of row g (u = 0) or g + 8
__device__ __forceinline__ float2 pair(const float (&x)[4], int u) { return make_float2(x[2 * u], x[2 * u + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[4], int u, float2 v) {
  x[2 * u] = v.x;
  x[2 * u + 1] = v.y;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

constexpr float pow2(int n) { return n < 0 ? 0.5f * pow2(n + 1) : n ? 2.f * pow2(n - 1) : 1.f; }

// The power of two that brings m > 0 into [2^T, 2^{T+1}), and the inverse of 2^kLess times
// it (kLess: what the other operand is multiplied by); infinities and NaN stay what they
// are, and what is below 2^-87 is multiplied as if it were that.
struct Scale {
  float up, down;
};
template <int T, int kLess = 0>
__device__ __forceinline__ Scale scale_to(float m) {
  static_assert(T + kLess < 40, "");
  int e = (int)(__float_as_uint(m) >> 23);  // (m >= 0)
  e = e < 40 ? 40 : e > 254 ? 254 : e;
  return {__uint_as_float((uint32_t)(254 + T - e) << 23), __uint_as_float((uint32_t)(e - T - kLess) << 23)};
}
// The same for a row of steps: into [1, 2), by 2^kFar at most.  For k kFar is kFarKey (beta
// is divided by the square) and rows of zeros stay as they are (v is multiplied by k's
// factor).
constexpr int kFarKey = 63, kFarStep = 110;
template <int kFar>
__device__ __forceinline__ float row_exponent(float m) {
  static_assert(kFar + kLift <= 127, "");
  int e = (int)(__float_as_uint(m) >> 23);
  e = kFar == kFarKey && m == 0.f ? 127 : e < 127 - kFar ? 127 - kFar : e > 253 ? 253 : e;
  return __uint_as_float((uint32_t)(254 - e) << 23);
}
__device__ __forceinline__ float inverse_pow2(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}
// the largest over the four lanes that hold a row of a product
__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <int N>
__device__ __forceinline__ void zero(float (&d)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
}

// Where a lane points for the four 8 x 8 pieces of ldmatrix, in a tile with rows of RB
// bytes whose address is a multiple of RB.  Both row and piece being multiples of 16
// elements apart, an address is the tile's, whole rows, and the lane's own offset in the
// first rows with the piece's bits exchanged: one instruction for a piece's column.
template <int RB>
struct Lane {
  uint32_t a, b;
  __device__ __forceinline__ explicit Lane(int lane)
      : a(at16<RB>(lane & 15, lane >> 4)),
        b(at16<RB>((lane & 7) + (lane >> 4 << 3), lane >> 3 & 1)) {}
  // rows m, terms along the row: a left operand of rows m ... m + 15, terms k ... k + 15
  __device__ __forceinline__ uint32_t left(uint32_t tile, int m, int k) const {
    return tile + (a ^ (k * 2)) + m * RB;
  }
  // terms down the rows: the same left operand from its transpose
  __device__ __forceinline__ uint32_t left_t(uint32_t tile, int m, int k) const {
    return tile + (b ^ (m * 2)) + k * RB;
  }
  // columns n down the rows, terms along them: right operands of columns n ... n + 7
  // (r[0], r[1]) and n + 8 ... (r[2], r[3])
  __device__ __forceinline__ uint32_t right(uint32_t tile, int n, int k) const {
    return tile + (b ^ (k * 2)) + n * RB;
  }
  // terms down the rows
  __device__ __forceinline__ uint32_t right_t(uint32_t tile, int n, int k) const {
    return tile + (a ^ (n * 2)) + k * RB;
  }
};

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
// the same, the sums beginning with zero
template <int PA, int PB, int N>
__device__ __forceinline__ void mma_parts0(float (*d)[4], const uint32_t (&a)[PA][4],
                                           const uint32_t (&b)[PB][N][2]) {
  constexpr int M = PA > PB ? PA : PB;
#pragma unroll
  for (int s = M - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        if (i + j == s) {
          const bool first = s == M - 1 && (i == 0 || (i > 0 && s - (i - 1) >= PB));
#pragma unroll
          for (int n = 0; n < N; ++n) {
            if (first) mma0(d[n], a[i], b[j][n][0], b[j][n][1]);
            else mma(d[n], a[i], b[j][n][0], b[j][n][1]);
          }
        }
}
// right operands of N (even) columns of eight, PB parts `step` bytes apart
template <int PB, int N, int RB>
__device__ __forceinline__ void load_right(uint32_t (&b)[PB][N][2], uint32_t tile, uint32_t step,
                                           const Lane<RB>& at, int n, int k) {
#pragma unroll
  for (int p = 0; p < PB; ++p)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t r[4];
      ldm4(r, at.right(tile, n + 8 * i, k) + p * step);
      b[p][i][0] = r[0];
      b[p][i][1] = r[1];
      b[p][i + 1][0] = r[2];
      b[p][i + 1][1] = r[3];
    }
}
template <int PB, int N, int RB>
__device__ __forceinline__ void load_right_t(uint32_t (&b)[PB][N][2], uint32_t tile, uint32_t step,
                                             const Lane<RB>& at, int n, int k) {
#pragma unroll
  for (int p = 0; p < PB; ++p)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t r[4];
      ldm4t(r, at.right_t(tile, n + 8 * i, k) + p * step);
      b[p][i][0] = r[0];
      b[p][i][1] = r[1];
      b[p][i + 1][0] = r[2];
      b[p][i + 1][1] = r[3];
    }
}
// Two columns of eight of a product's result, rows g times s0 and g + 8 times s1, as
// the left operand of 16 terms of the next one.
template <int P>
__device__ __forceinline__ void as_left(uint32_t (&a)[P][4], const float (&x)[4], const float (&y)[4],
                                        float s0, float s1) {
  uint32_t r[P];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 s = both(e ? s1 : s0);
    split2<P>(mul2(pair(x, e), s), r);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][e] = r[p];
    split2<P>(mul2(pair(y, e), s), r);
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
// Registers of a warp group from here on (kernels of 384 threads start with 168).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- a chunk's tiles ------------------------------------------------------------

// NI: parts of an element of q, k, v (bf16: one; fp32: two).  fp32 takes chunks of 32
// steps.
template <int NI>
constexpr int kSteps = NI == 1 ? 64 : 32;

// bf16: C rows of D elements from rows `stride` elements apart, as asynchronous copies
// to be committed by the caller; past row n and past `width` (a multiple of 8) zeros.
template <int C, int D, int NT>
__device__ __forceinline__ void load_tile(uint8_t* tile, const __nv_bfloat16* s, long long stride,
                                          int n, int width, int tid) {
  constexpr int RB = D * 2, LPR = D / 8, R = NT / LPR;  // R rows at a time
  static_assert(C % R == 0 && R % 8 == 0, "");
  const int r = tid / LPR, x = tid % LPR;
  const uint32_t to = smem32(tile) + at16<RB>(r, x);
  const __nv_bfloat16* from = s + r * stride + x * 8;
  const bool in = x * 8 < width;
#pragma unroll
  for (int i = 0; i < C / R; ++i) {  // (the pieces' places repeat every eight rows)
    const bool here = in && r + i * R < n;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * R * RB),
                 "l"(here ? from : s), "r"(here ? 16 : 0)
                 : "memory");
    from += R * stride;
  }
}
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *(const __nv_bfloat162*)&x; }
// The largest magnitudes of eight bf16's even and odd elements (NaN is passed over).
__device__ __forceinline__ __nv_bfloat162 max_bf(const uint4& q) {
  return __hmax2(__hmax2(__habs2(as_bf2(q.x)), __habs2(as_bf2(q.y))),
                 __hmax2(__habs2(as_bf2(q.z)), __habs2(as_bf2(q.w))));
}
// eight bf16 times a power of two as fp16
__device__ __forceinline__ uint4 bf_to_half(const uint4& q, float s) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = mul2(unpack_bf((&q.x)[i]), both(s));
    (&r.x)[i] = pack_half(f.x, f.y);
  }
  return r;
}
__device__ __forceinline__ float no_least(int) { return 0.f; }
// A bf16 tile to fp16 in its place: a thread's elements are read, and written row by
// row, each scaled into [1, 2) (and by 2^kLift), or by no more than `least(row)` would be; done(row,
// scale, largest) by one lane a row.
template <int C, int DK, int NT>
struct HalfRows {
  static constexpr int LPR = DK / 8, N = C * LPR / NT;
  static_assert(C * LPR % NT == 0, "");
  uint4 q[N];
  __device__ __forceinline__ void read(const uint8_t* tile, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * NT + tid;
      q[i] = *(const uint4*)(tile + at16<DK * 2>(at / LPR, at % LPR));
    }
  }
  template <int kFar, typename F, typename L>
  __device__ __forceinline__ void write(uint8_t* tile, int tid, L least, F done) const {
    __nv_bfloat162 m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = max_bf(q[i]);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = __hmax2(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * NT + tid, r = at / LPR, x = at % LPR;
      const float most = fmaxf(fmaxf(__low2float(m[i]), __high2float(m[i])), least(r));
      const float s = row_exponent<kFar>(most);
      *(uint4*)(tile + at16<DK * 2>(r, x)) = bf_to_half(q[i], s * pow2(kLift));
      if (x == 0) done(r, s, most);
    }
  }
};

// fp32: C rows of D elements one behind the other, as asynchronous copies.
template <int C, int D, int NT>
__device__ __forceinline__ void load_tile(uint8_t* tile, const float* s, long long stride, int n,
                                          int width, int tid) {
  constexpr int LPR = D / 4, R = NT / LPR;
  static_assert(C % R == 0, "");
  const int r = tid / LPR, x = tid % LPR;
  const uint32_t to = smem32(tile) + tid * 16;
  const float* from = s + r * stride + x * 4;
  const bool in = x * 4 < width;
#pragma unroll
  for (int i = 0; i < C / R; ++i) {
    const bool here = in && r + i * R < n;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * NT * 16),
                 "l"(here ? from : s), "r"(here ? 16 : 0)
                 : "memory");
    from += R * stride;
  }
}
// Such a tile to two fp16 parts in its place, C * DK * 2 bytes apart: a thread's
// elements are read, and after a barrier of all threads written.
template <int C, int DK, int NT>
struct FloatRows {
  static constexpr int LPR = DK / 4, N = C * LPR / NT;
  static_assert(C * LPR % NT == 0 && LPR <= 32, "");
  float4 f[N];
  __device__ __forceinline__ void read(const uint8_t* tile, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = ((const float4*)tile)[i * NT + tid];
  }
  __device__ __forceinline__ void put(uint8_t* tile, int i, float s, int tid) const {
    const int at = i * NT + tid, r = at / LPR, x = at % LPR;
    uint32_t p[2], q[2];
    split2<2>(f[i].x * s, f[i].y * s, p);
    split2<2>(f[i].z * s, f[i].w * s, q);
    uint8_t* to = tile + at16<DK * 2>(r, x >> 1) + (x & 1) * 8;
    *(uint2*)to = make_uint2(p[0], q[0]);
    *(uint2*)(to + C * DK * 2) = make_uint2(p[1], q[1]);
  }
  // each row scaled into [1, 2) (and by 2^kLift), or by no more than `least(row)` would
  // be; done(row, scale, largest) by one lane a row
  template <int kFar, typename F, typename L>
  __device__ __forceinline__ void write(uint8_t* tile, int tid, L least, F done) const {
    float m[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      m[i] = fmaxf(max3_abs(f[i].x, f[i].y, f[i].z), fabsf(f[i].w));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * NT + tid;
      m[i] = fmaxf(m[i], least(at / LPR));
      const float s = row_exponent<kFar>(m[i]);
      put(tile, i, s * pow2(kLift), tid);
      if (at % LPR == 0) done(at / LPR, s, m[i]);
    }
  }
};

// Per step of a chunk: the sum g of the log decays (of base 2), as two floats, so that
// a difference of two sums is good to its own last bit however long they have grown;
// e^g, e^{G-g}; the write strength, of k's scale; the power of two that k was multiplied
// by; what to multiply q's results by; what X's column was divided by, and that times
// the write strength.
template <int C>
struct alignas(16) Gates {
  float hi[C], lo[C], lead[C], tail[C], beta[C], kup[C], qdown[C], xs[C], bx[C];
  float last;    // e^G
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
// a += b, the rounding put aside (one addition waits for the one before)
__device__ __forceinline__ void put_in(Two& a, float b) {
  const float s = a.hi + b, t = s - a.hi;
  a.lo += (a.hi - (s - t)) + (b - t);
  a.hi = s;
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
// (log decays below -200 are as good as -inf, as e^-104 is the smallest float, and keep
// sums finite; NaN stays; past n 0)
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

// What the walks read of a chunk besides its operands, in parts: a tile M [C][C] with -L
// below the blocks of 16 on the diagonal, in them -X^T, its rows scaled, and above them
// P, block (i, j) in the place of block (j, i), as it is (L and P times 2^kScore); and P's diagonal blocks, a tile
// [C][16] (kPRow bytes a row).
constexpr int kPRow = 32;
constexpr int kDiag = 20;  // floats of a column of a diagonal block
template <int C>
struct alignas(16) Scratch {
  float diag[C / 16][16][kDiag];  // L[i][j] at [j][i], a warp each
  uint8_t t[C / 16][kParts * 512];  // T of the diagonal blocks, transposed like X, in parts
};

// One block of 16 x 16, rows 16 bi ..., columns 16 bj ..., of L and, with kP, of P, which
// share the decays and the right operand.  -L goes to the tile M in parts, or on the
// diagonal (kDiagonal) L to `diag`, transposed; P to M's upper blocks or to P.  On the
// diagonal P is zero above it and L on it too.
template <int NI, int DK, bool kP, bool kDiagonal>
__device__ __forceinline__ void score_block(uint32_t Q, uint32_t K, uint8_t* M, uint8_t* P,
                                            const Gates<kSteps<NI>>& g, float (*diag)[kDiag], int bi,
                                            int bj, int lane) {
  constexpr int C = kSteps<NI>, RB = DK * 2, OB = C * 2, NA = kP ? 2 : 1;
  const Lane<RB> at(lane);
  float acc[NA][2][4];
  const uint32_t A[2] = {K + bi * 16 * RB, Q + bi * 16 * RB}, B = K + bj * 16 * RB;
#pragma unroll
  for (int w = 0; w < NA; ++w) zero(acc[w]);
  constexpr int U = NI == 1 ? 4 : 2;
#pragma unroll(U)
  for (int k = 0; k < DK; k += 16) {
    uint32_t a[NA][NI][4], b[NI][2][2];
#pragma unroll
    for (int w = 0; w < NA; ++w)
#pragma unroll
      for (int p = 0; p < NI; ++p) ldm4(a[w][p], at.left(A[w], 0, k) + p * C * RB);
    load_right<NI, 2>(b, B, C * RB, at, 0, k);
#pragma unroll
    for (int w = 0; w < NA; ++w) mma_parts<NI, NI, 2>(acc[w], a[w], b);
  }
  const int c0 = (lane & 3) * 2, r0 = lane >> 2;
  const float* gi = &g.hi[16 * bi + r0];
  const float* gj = &g.hi[16 * bj + c0];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float2 hj = *(const float2*)(gj + 8 * n), lj = *(const float2*)(gj + C + 8 * n);
    const int j = 8 * n + c0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = r0 + 8 * u;
      // Gamma_ij = 2^((hi_i - hi_j) + (lo_i - lo_j))
      const float2 minus = both(-1.f);
      const float2 t = add2(fma2(hj, minus, both(gi[8 * u])), fma2(lj, minus, both(gi[C + 8 * u])));
      // (the operands' factors off, the scores' on)
      const float2 gamma = mul2(make_float2(exp2_fast(t.x), exp2_fast(t.y)),
                                both(pow2(kScore - 2 * kLift)));
      float2 l = mul2(pair(acc[0][n], u), gamma);
      const uint32_t to = at16<OB>(16 * bi + i, 2 * bj + n) + c0 * 2;
      if constexpr (kDiagonal) {
        diag[j][i] = j < i ? l.x * pow2(-kScore) : 0.f;
        diag[j + 1][i] = j + 1 < i ? l.y * pow2(-kScore) : 0.f;
      } else {
        uint32_t p[kParts];
        split2<kParts>(make_float2(-l.x, -l.y), p);
#pragma unroll
        for (int q = 0; q < kParts; ++q) *(uint32_t*)(M + to + q * C * OB) = p[q];
      }
      if constexpr (kP) {
        float2 v = mul2(pair(acc[NA - 1][n], u), gamma);
        if (kDiagonal && j > i) v.x = 0.f;
        if (kDiagonal && j + 1 > i) v.y = 0.f;
        uint32_t p[kParts];
        split2<kParts>(v, p);
        uint8_t* at = kDiagonal ? P + at16<kPRow>(16 * bi + i, n) + c0 * 2
                                : M + at16<OB>(16 * bj + i, 2 * bi + n) + c0 * 2;
#pragma unroll
        for (int q = 0; q < kParts; ++q) *(uint32_t*)(at + q * C * (kDiagonal ? kPRow : OB)) = p[q];
      }
    }
  }
}

// Lanes 0 - 15, a column j each of diagonal block s: with T = (I + beta L)^-1, X = L T
// and T = I - beta X, so once X_mj is whole, T_mj = -beta_m X_mj (1 for m = j) adds
// L_im T_mj to every later X_ij.  kT: T to `tt` too, and the columns of both scaled by T's
// largest (X, which comes to |k|^2 times T, would leave T's second part no exponents).
template <int C, bool kT>
__device__ __forceinline__ void invert_diag(uint8_t* out, uint8_t* tt, Gates<C>& g,
                                            const float (*diag)[kDiag], int s, int j) {
  constexpr int OB = C * 2;
  float x[16], tm[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
  for (int m = 0; m < (kT ? 16 : 15); ++m) {
    const float t = m == j ? 1.f : -g.beta[16 * s + m] * x[m];
    tm[m] = t;
    if (m == 15) break;
#pragma unroll
    for (int i = (m + 1) / 4 * 4; i < 16; i += 4) {
      const float4 l = *(const float4*)&diag[m][i];
      if (i > m) x[i] = fmaf(l.x, t, x[i]);
      if (i + 1 > m) x[i + 1] = fmaf(l.y, t, x[i + 1]);
      if (i + 2 > m) x[i + 2] = fmaf(l.z, t, x[i + 2]);
      if (i + 3 > m) x[i + 3] = fmaf(l.w, t, x[i + 3]);
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(kT ? tm[i] : x[i]));
  // (an element of L is at most 2^9, so one of X = L T, and of the folded blocks, is below
  // 2^15 where T's are below 4)
  const Scale sx = scale_to<kT ? 1 : kLift>(m);
  g.xs[16 * s + j] = sx.down;
  g.bx[16 * s + j] = sx.down * g.beta[16 * s + j];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4][kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      split2<kParts>(-x[8 * h + 2 * i] * sx.up, -x[8 * h + 2 * i + 1] * sx.up, p[i]);
    uint8_t* at = out + at16<OB>(16 * s + j, 2 * s + h);
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      *(uint4*)(at + q * C * OB) = make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
    if constexpr (kT) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        split2<kParts>(tm[8 * h + 2 * i] * sx.up, tm[8 * h + 2 * i + 1] * sx.up, p[i]);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        *(uint4*)(tt + q * 512 + at16<32>(j, h)) = make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
    }
  }
}

// A block of M below the diagonal, rows 16 bi ..., columns 16 bj ...: -L T in the place
// of -L (as it is: T has its own factor).
template <int C>
__device__ __forceinline__ void fold_block(uint8_t* M, const uint8_t* tt, int bi, int bj, int lane) {
  constexpr int OB = C * 2;
  const Lane<OB> at(lane);
  const Lane<32> t(lane);
  uint32_t a[kParts][4], b[kParts][2][2];
  float d[2][4];
#pragma unroll
  for (int q = 0; q < kParts; ++q) ldm4(a[q], at.left(smem32(M), 16 * bi, 16 * bj) + q * C * OB);
  load_right<kParts, 2>(b, smem32(tt), 512, t, 0, 0);
  mma_parts0<kParts, kParts, 2>(d, a, b);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t p[kParts];
      split2<kParts>(mul2(pair(d[n], u), both(pow2(-kScore))), p);
      uint8_t* to = M + at16<OB>(16 * bi + (lane >> 2) + 8 * u, 2 * bj + n) + (lane & 3) * 4;
#pragma unroll
      for (int q = 0; q < kParts; ++q) *(uint32_t*)(to + q * C * OB) = p[q];
    }
}

// M and, with kP, P of a chunk whose operands and gates are in shared memory, by the
// kPrep threads: a warp takes a diagonal block and inverts L's, the others the blocks
// below the diagonal.  (These go through one loop: as straight code, with the strips of
// a warp known at compile time, the warps' code and the walk's did not fit the
// instruction caches together, and waiting for instructions was the largest of all
// stalls.)  The last warp has `aside` to do as well (the gates of a later chunk).
template <int NI, int DK, bool kP, bool kFold, typename F>
__device__ __forceinline__ void prepare(const uint8_t* Qt, const uint8_t* Kt, uint8_t* M, uint8_t* P,
                                        Gates<kSteps<NI>>& g, Scratch<kSteps<NI>>& sc, int tid,
                                        F aside) {
  constexpr int C = kSteps<NI>, NB = C / 16, W = kPrep / 32 - NB;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t K = smem32(Kt), Q = smem32(Qt);
  // rows and columns (hexadecimal digits, the first last)
  constexpr uint32_t kI = NB == 4 ? 0x333221 : 0x1, kJ = NB == 4 ? 0x210100 : 0x0;
  if (warp < NB) {
    score_block<NI, DK, kP, true>(Q, K, M, P, g, sc.diag[warp], warp, warp, lane);
    __syncwarp();
    if (lane < 16) invert_diag<C, kFold>(M, sc.t[warp], g, sc.diag[warp], warp, lane);
    __syncwarp();
  } else {
#pragma unroll 1
    for (int r = warp - NB; r < NB * (NB - 1) / 2; r += W)
      score_block<NI, DK, kP, false>(Q, K, M, P, g, nullptr, kI >> 4 * r & 15, kJ >> 4 * r & 15, lane);
    if (warp == kPrep / 32 - 1) aside();
  }
  if constexpr (kFold) {
    bar(2, kPrep);
    if (warp < NB * (NB - 1) / 2) {
      const int bj = kJ >> 4 * warp & 15;
      fold_block<C>(M, sc.t[bj], kI >> 4 * warp & 15, bj, lane);
    }
  }
}

}  // namespace delta
}  // namespace ssd
