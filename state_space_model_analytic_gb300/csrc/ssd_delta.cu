// Gated delta rule: the walk over the chunks of a row (outputs and state, or the
// states before every chunk and the errors E), the walk back (the gradients of the
// states and of v), and the step of one token.  The formulas of a chunk stand in
// ssd_delta.cuh; the gradients of L = sum(do . o) + sum(dS . S_T) are, with D the
// gradient of the state after a chunk,
//   dU = s P^T dO + e^{G-g} K D^T,  (I + L^T beta) y = dU,  dv = beta y,
//   dbeta_i = E_i . y_i,  D <- e^G D + (s e^g dO)^T Q - (e^g dv)^T K
// and those of q, k and the decays need no walk (ssd_delta_grads.cu).
//
// One CTA per (head, columns of v, row): the rows of the state are independent of each
// other.  Four warps hold 16 rows of the state each, in registers, in the layout in
// which matrix instructions leave their results.  That is also the layout in which
// they take a left operand, and every product of the chain that one chunk has to pass
// on to the next has such a one: F^T = V^T - H K^T from the state, E^T from F^T, the
// new state from U^T.  So that chain runs within a warp, without a word through shared
// memory; eight other warps meanwhile prepare the next chunk (L, X, P: all that does not
// depend on the state) and load the one after it, and one barrier a chunk hands over.
//
// Where rows are few, WK = 2 or 4 warps share 16 rows of the state, a part of dk each:
// the products with the state are split, F's parts added up through shared memory, and
// the solution of the triangular system, which all of them need, is found by each.
//
// Bound by that chain and, where o is formed, by the warps that form it: at 4 x 2048 steps
// of 32 heads 128/64 (bf16, 175 us; memory alone would take 31) a chunk of 64 steps takes
// 10 thousand cycles.  The chain has 2.2 of them for the products with the state, 3.4 for
// the system and 1.7 for the new state; o takes 188 matrix instructions a warp, 84 when
// one part of the state, P and U was taken (153 us, but o off by 2^-12 of |q| |S|).
// Tensor pipe 45 % and issue slots 42 % busy.  The walk that keeps the states takes 144
// us, the walk back 232.  fp32 (8 x 1024 steps of 24 heads 64/64): 154 us.  (These and the
// times below: events around the kernel, caches flushed.)
#include <cuda_bf16.h>

#include "ssd_delta.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace delta;

constexpr int kWalkers = 4;  // warps of a walk

template <int NI, int DK, int WK, int kExchanged, bool kHelped = false>
struct Geom {
  static constexpr int kThreads = kPrep + 32 * kWalkers * (kHelped ? 2 : 1);
  // Registers of those that walk and of the others, of what a CTA starts with.
  static constexpr int kPrepRegs = kHelped ? 96 : 128, kWalkRegs = kHelped ? 224 : 240;
  static_assert((kThreads - 32 * kWalkers) * kPrepRegs + 32 * kWalkers * kWalkRegs <=
                    kThreads * (kHelped ? 128 : 168), "");
  static constexpr int C = kSteps<NI>, NC = C / 8;
  static constexpr int RB = DK * 2, PB = C * 2;      // bytes of a row of K, of M
  static constexpr int KT = NI * C * RB;             // K's or Q's tile, all parts
  // V in the walk (bf16 as it is, fp32 as floats whose rows are 4 banks apart),
  // dO in the walk back (parts)
  static constexpr int LV = kVB + 4;
  static constexpr int VT = NI == 1 ? C * kVB * 2 : C * LV * 4;
  static_assert(VT >= NI * C * kVB * 2, "");
  static constexpr int NS = 3;                       // stages of the operands
  static constexpr int MT = kParts * C * PB, PT = kParts * C * kPRow;
  static constexpr int kStage = 2 * KT + VT;
  static constexpr int kM = NS * kStage, kP = kM + 2 * MT;
  static constexpr int kG = kP + 2 * PT, kS = kG + 3 * (int)sizeof(Gates<C>);
  static constexpr int kX = kS + (int)sizeof(Scratch<C>);  // sums of WK warps on their way
  // of a walking warp, for those that form its o: the state and U as left operands, what
  // their rows were multiplied by
  static constexpr int NB = C / 16, kHS = kParts * DK / 16 * 512, kUS = kParts * NB * 512;
  static constexpr int kGiven = kHS + kUS + (1 + NB) * 64;
  static constexpr size_t smem =
      kX + (WK > 1 ? kExchanged * kWalkers * NC * 512 : 0) + (kHelped ? kWalkers * kGiven : 0);
  static_assert(kStage % 16 == 0 && kX % 16 == 0 && kGiven % 16 == 0, "");
};

// fp32 rows of v: C x kVB floats
template <int C, int LV>
__device__ __forceinline__ void load_floats(uint8_t* tile, const float* src, long long stride, int n,
                                            int width, int tid) {
  float* t = (float*)tile;
#pragma unroll 4
  for (int i = tid; i < C * (kVB / 4); i += kPrep) {
    const int r = i / (kVB / 4), x = i % (kVB / 4) * 4;
    const bool in = r < n && x < width;
    copy16(t + r * LV + x, in ? src + r * stride + x : src, in);
  }
}

// A warp's rows of a state [dv][dk], from column k0: x[j]: row v (+ 8 for e >= 2),
// column k0 + 8 j + 2 t (+ 1 for odd e), from or to memory.
template <int NK>
__device__ __forceinline__ void get_state(float (&x)[NK][4], const float* p, int v, int dv, int k0,
                                          int dk, int lane) {
  const int c = k0 + (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < NK; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float2 f = make_float2(0.f, 0.f);
      if (p && v + 8 * u < dv && k0 + 8 * j < dk) f = *(const float2*)(p + (v + 8 * u) * dk + 8 * j + c);
      x[j][2 * u] = f.x;
      x[j][2 * u + 1] = f.y;
    }
}
template <int NK>
__device__ __forceinline__ void put_state(const float (*x)[4], float* p, int v, int dv, int k0,
                                          int dk, int lane) {
  const int c = k0 + (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < NK; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (v + 8 * u < dv && k0 + 8 * j < dk)
        *(float2*)(p + (v + 8 * u) * dk + 8 * j + c) = make_float2(x[j][2 * u], x[j][2 * u + 1]);
}
// the largest magnitudes of a lane's values in its rows g and g + 8
template <int N>
__device__ __forceinline__ float2 row_max(const float (*x)[4], float2 m = make_float2(0.f, 0.f)) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    m.x = max3_abs(m.x, x[j][0], x[j][1]);
    m.y = max3_abs(m.y, x[j][2], x[j][3]);
  }
  return m;
}
// x times the factors of its columns
__device__ __forceinline__ void times(float (&x)[4], float2 f) {
#pragma unroll
  for (int u = 0; u < 2; ++u) set_pair(x, u, mul2(pair(x, u), f));
}
// the scales of a warp's rows from its lanes' largest values, for products with a tile
// that holds 2^kLess times its values
struct RowScales {
  float up0, down0, up1, down1;
};
template <int kLess>
__device__ __forceinline__ RowScales row_scales(float2 m) {
  const Scale a = scale_to<kLift, kLess>(quad_max(m.x)), b = scale_to<kLift, kLess>(quad_max(m.y));
  return {a.up, a.down, b.up, b.down};
}

// x <- x + d, d's rows scaled back
__device__ __forceinline__ void add_rows(float (&x)[4], const float (&d)[4], const RowScales& s) {
  set_pair(x, 0, fma2(pair(d, 0), both(s.down0), pair(x, 0)));
  set_pair(x, 1, fma2(pair(d, 1), both(s.down1), pair(x, 1)));
}
__device__ __forceinline__ void scale_back(float (&x)[4], const RowScales& s) {
  set_pair(x, 0, mul2(pair(x, 0), both(s.down0)));
  set_pair(x, 1, mul2(pair(x, 1), both(s.down1)));
}

// x (rows v, columns c0 ... of steps, eight) transposed to rows of memory: row i of
// step i, n steps, `step` elements apart; at: the first step's element v0.
template <typename T>
__device__ __forceinline__ void put_steps(const float (&x)[4], T* at, long long step, int c0, int n,
                                          int v0, int dv, int lane) {
  const int g = lane >> 2, c = (lane & 3) * 2;
  if constexpr (sizeof(T) == 2) {
    const uint32_t a = transpose8(pack_bf(x[0], x[1])), b = transpose8(pack_bf(x[2], x[3]));
    if (c0 + g < n) {
      T* row = at + (c0 + g) * step + c;
      if (v0 < dv) *(uint32_t*)row = a;
      if (v0 + 8 < dv) *(uint32_t*)(row + 8) = b;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = c0 + c + (e & 1), v = g + 8 * (e >> 1);
      if (i < n && v0 + v < dv) at[i * step + v] = x[e];
    }
  }
}

// rows of a row's end up to T: zeros
template <typename T>
__device__ __forceinline__ void clear_rows(T* out, long long step, int from, int to, int width,
                                           int tid, int threads) {
  constexpr int E = 16 / (int)sizeof(T);
  const int per = width / E;  // (dv is a multiple of 8)
  const long long n = (long long)(to - from) * per;
  for (long long i = tid; i < n; i += threads) {
    const long long r = from + i / per;
    *(uint4*)(out + r * step + i % per * E) = make_uint4(0, 0, 0, 0);
  }
}

// f[n] = X K^T for the C steps of a tile whose rows are steps, X the warp's columns k0
// ... of the state, scaled; and with kO o[n] = X Q^T.  The right operands of a group of
// columns are loaded while the group before is multiplied.  given(k, a): the state's
// parts as left operands of columns 16 k ..., as soon as there are any.
template <int NI, bool kO, int DK, int NK, int NC, typename F>
__device__ __forceinline__ void state_times(float (&f)[NC][4], float (&o)[NC][4],
                                            const float (&x)[NK][4], const RowScales& s, uint32_t K,
                                            uint32_t Q, int k0, const Lane<DK * 2>& at, F given) {
  constexpr int C = kSteps<NI>, RB = DK * 2;
  constexpr int GN = NC < 4 ? NC : 4;                     // columns of eight of a group
  constexpr int GF = NC / GN, GK = kO ? 2 * GF : GF;  // groups of 16 terms
  constexpr int NG = NK / 2 * GK;
  uint32_t a[2][kParts][4], b[2][NI][GN][2];
  auto load = [&](int i) {
    const int k = i / GK, g = i % GK;
    load_right<NI, GN>(b[i & 1], g < GF ? K : Q, C * RB, at, 8 * GN * (g % GF), k0 + 16 * k);
  };
  as_left<kParts>(a[0], x[0], x[1], s.up0, s.up1);
  load(0);
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int k = i / GK, g = i % GK;
    if (i + 1 < NG) load(i + 1);
    if (g == 0) {
      given(k, a[k & 1]);
      if (2 * k + 2 < NK) as_left<kParts>(a[(k + 1) & 1], x[2 * k + 2], x[2 * k + 3], s.up0, s.up1);
    }
    if (g < GF) {
      if (k == 0) mma_parts0<kParts, NI, GN>(f + GN * g, a[0], b[i & 1]);
      else mma_parts<kParts, NI, GN>(f + GN * g, a[k & 1], b[i & 1]);
    } else if constexpr (kO) {
      if (k == 0) mma_parts0<kParts, NI, GN>(o + GN * (g - GF), a[0], b[i & 1]);
      else mma_parts<kParts, NI, GN>(o + GN * (g - GF), a[k & 1], b[i & 1]);
    }
  }
}

// Block (i, k) of P, 16 rows and 16 columns, as a right operand: its rows as columns.
template <int C>
__device__ __forceinline__ void load_scores(uint32_t (&r)[kParts][2][2], uint32_t M, uint32_t P,
                                            const Lane<C * 2>& lm, const Lane<kPRow>& lp, int i, int k) {
  if (i == k) load_right<kParts, 2>(r, P, C * kPRow, lp, 16 * k, 0);
  else load_right<kParts, 2>(r, M, C * C * 2, lm, 16 * k, 16 * i);
}

// d = a b for two columns of eight, all parts of both; the small products go to a sum
// of their own, so that fewer wait for one another.
__device__ __forceinline__ void mma_short(float (&d)[2][4], const uint32_t (&a)[kParts][4],
                                          const uint32_t (&b)[kParts][2][2]) {
  float e[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) mma0(e[n], a[0], b[1][n][0], b[1][n][1]);
#pragma unroll
  for (int n = 0; n < 2; ++n) mma0(d[n], a[0], b[0][n][0], b[0][n][1]);
#pragma unroll
  for (int n = 0; n < 2; ++n) mma(e[n], a[1], b[0][n][0], b[0][n][1]);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u) set_pair(d[n], u, add2(pair(d[n], u), pair(e[n], u)));
}

// x <- scale x + Y tile for columns n, GN eights of them, Y (rows v, C steps) as parts of
// left operands that were scaled by s; x: columns k0 ... of the state.  beside(): work
// that is issued between the products.
template <int NI, int DK, int GN, int NB, typename F>
__device__ __forceinline__ void columns_add(float (*x)[4], float scale, const uint32_t (*y)[kParts][4],
                                            const RowScales& s, uint32_t tile, int n, const Lane<DK * 2>& at,
                                            F beside) {
  constexpr int C = kSteps<NI>, RB = DK * 2;
  float d[GN][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t r[NI][GN][2];
    load_right_t<NI, GN>(r, tile, C * RB, at, n, 16 * b);
    if (b == 0) mma_parts0<kParts, NI, GN>(d, y[b], r);
    else mma_parts<kParts, NI, GN>(d, y[b], r);
    if (b == 0) beside();
  }
#pragma unroll
  for (int i = 0; i < GN; ++i) {
    times(x[i], both(scale));
    add_rows(x[i], d[i], s);
  }
}
// The same for all columns, beside(i) beside group i of ceil(NK / 4).  Returns the
// largest values of the lane's rows.
template <int NI, int DK, int NK, int NB, typename F>
__device__ __forceinline__ float2 state_add(float (&x)[NK][4], float scale, const uint32_t (*y)[kParts][4],
                                            const RowScales& s, uint32_t tile, int k0, const Lane<DK * 2>& at,
                                            F beside) {
  constexpr int GN = NK < 4 ? NK : 4;
  float2 m = make_float2(0.f, 0.f);
#pragma unroll
  for (int n = 0; n < NK; n += GN) {
    columns_add<NI, DK, GN, NB>(x + n, scale, y, s, tile, k0 + 8 * n, at, [&] { beside(n / GN); });
    m = row_max<GN>(x + n, m);
  }
  return m;
}

// The sum over WK warps of t[n], in the same order for each; ex: the warps' NC * 32
// float4, from the first warp of the group.
template <int WK, int NC>
__device__ __forceinline__ void add_warps(float (&t)[NC][4], const float4* ex, int kg, int lane) {
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < WK; ++q) {
      const float4 f = q == kg ? make_float4(t[n][0], t[n][1], t[n][2], t[n][3])
                               : ex[(q * NC + n) * 32 + lane];
      s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
    }
    t[n][0] = s.x; t[n][1] = s.y; t[n][2] = s.z; t[n][3] = s.w;
  }
}

// The row of a CTA.  Of rows with lengths, where the CTAs outnumber the SMs, the longest go
// first, so that none of them begins when the others are done (16 rows of up to 1003
// steps, 24 heads 64/64: 130 us against 151).
constexpr int kOrdered = 256;  // rows that are put in order
// len: kOrdered + 1 words of shared memory that are free again afterwards.
__device__ __forceinline__ int row_of(const int* lens, int B, int T, int tid, int* len) {
  if (!lens || B > kOrdered || gridDim.x * gridDim.y <= kLaSms) return blockIdx.y;
  if (tid < B) len[tid] = min(max(lens[tid], 0), T);
  __syncthreads();
  if (tid < B) {
    int before = 0;
    const int mine = len[tid];
    for (int i = 0; i < B; ++i) before += len[i] > mine || (len[i] == mine && i < tid);
    if (before == blockIdx.y) len[kOrdered] = tid;
  }
  __syncthreads();
  const int row = len[kOrdered];
  __syncthreads();
  return row;
}

// Whether o is formed by four warps of their own: the walking ones hand them the state and
// U as they have them for their own products.  4 x 2048 steps of 32 heads 128/64: 175 us
// against 190; at 64/64 there is less to take over and the four need their issue slots (16
// rows of up to 1003, 24 heads: 131 against 130), in fp32, whose chunks are half as long, the
// state is handed over twice as often (187 against 154), and with WK > 1 the preparation is
// what takes longest.  Where they are, the preparing warps have time to multiply the rows of
// later blocks by the inverse of the earlier ones as well, and the chain has one product a
// block less.
template <int NI, int DK, int WK, bool kStates>
constexpr bool helped() {
  return !kStates && WK == 1 && NI == 1 && DK == 128;
}

// What a walking warp hands to the warp that forms its o: the parts of the state and
// of U's blocks as left operands, with what their rows were multiplied by.
template <typename G>
struct Given {
  uint8_t* at;
  __device__ __forceinline__ uint4* state(int k, int q, int lane) const {
    return (uint4*)(at + (k * kParts + q) * 512) + lane;
  }
  __device__ __forceinline__ uint4* u(int k, int q, int lane) const {
    return (uint4*)(at + G::kHS + (k * kParts + q) * 512) + lane;
  }
  // of rows g and g + 8: the state's (0), those of U's block k (1 + k)
  __device__ __forceinline__ float2* down(int k, int lane) const {
    return (float2*)(at + G::kHS + G::kUS + k * 64) + (lane >> 2);
  }
  __device__ __forceinline__ void put(uint4* to, const uint32_t (&a)[4]) const {
    *to = make_uint4(a[0], a[1], a[2], a[3]);
  }
};

// o of a chunk, 16 columns of v: s e^g H q + s P U.
template <int NI, int DK, typename G, typename T>
__device__ __forceinline__ void form_o(const Given<G>& x, int vg, uint32_t Q, uint32_t M, uint32_t P,
                                       const Gates<G::C>& g, T* out, long long out_step, int n, int v,
                                       int dv, int lane) {
  constexpr int C = G::C, NB = G::NB;
  const Lane<G::RB> la(lane);
  const Lane<G::PB> lm(lane);
  const Lane<kPRow> lp(lane);
  const int c2 = (lane & 3) * 2;
  auto scales = [&](int k) {
    const float2 d = *x.down(k, lane);
    return RowScales{0.f, d.x, 0.f, d.y};
  };
  auto fetch = [&](uint32_t (&a)[4], const uint4* from) {
    const uint4 t = *from;
    a[0] = t.x; a[1] = t.y; a[2] = t.z; a[3] = t.w;
  };
  float o[2 * NB][4];
  zero(o);
  bar(3 + vg, 64);
#pragma unroll
  for (int k = 0; k < DK / 16; ++k) {
    uint32_t a[kParts][4];
#pragma unroll
    for (int q = 0; q < kParts; ++q) fetch(a[q], x.state(k, q, lane));
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      uint32_t r[NI][2][2];
      load_right<NI, 2>(r, Q, C * G::RB, la, 16 * j, 16 * k);
      mma_parts<kParts, NI, 2>(o + 2 * j, a, r);
    }
  }
  {
    const RowScales s = scales(0);
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {
      scale_back(o[j], s);
      times(o[j], *(const float2*)&g.lead[8 * j + c2]);
    }
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    if (k == 0) bar(3 + kWalkers + vg, 64);
    if (k == NB / 2) bar(3 + 2 * kWalkers + vg, 64);
    uint32_t a[kParts][4];
    const RowScales s = scales(1 + k);
#pragma unroll
    for (int q = 0; q < kParts; ++q) fetch(a[q], x.u(k, q, lane));
#pragma unroll
    for (int j = k; j < NB; ++j) {
      uint32_t r[kParts][2][2];
      float d[2][4];
      load_scores<C>(r, M, P, lm, lp, j, k);
      mma_parts0<kParts, kParts, 2>(d, a, r);
      add_rows(o[2 * j], d[0], s);
      add_rows(o[2 * j + 1], d[1], s);
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
    times(o[j], *(const float2*)&g.qdown[8 * j + c2]);
    put_steps<T>(o[j], out, out_step, 8 * j, n, v, dv, lane);
  }
}

template <int NI, int DK, int WK, bool kStates>
__global__ void __launch_bounds__(kPrep + 32 * kWalkers * (helped<NI, DK, WK, kStates>() ? 2 : 1), 1)
    k_delta_walk(const DeltaWalk p) {
  // o: formed by the preparing warps, or by the walking ones
  constexpr bool kHelped = helped<NI, DK, WK, kStates>(), kOwn = !kStates && !kHelped;
  using G = Geom<NI, DK, WK, kStates ? 1 : 2, kHelped>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  constexpr int C = G::C, NC = G::NC, NB = C / 16, NK = DK / 8 / WK, VB = kVB / WK;
  // blocks of 16 steps of o and E that a warp writes
  constexpr int OB = NB / WK > 0 ? NB / WK : 1;
  extern __shared__ __align__(1024) uint8_t sm[];
  Gates<C>* gates = (Gates<C>*)(sm + G::kG);
  Scratch<C>& scratch = *(Scratch<C>*)(sm + G::kS);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (p.dv + VB - 1) / VB;
  const int h = blockIdx.x / vblocks, v0 = blockIdx.x % vblocks * VB;
  const int b = row_of(p.lens, p.B, p.T, tid, (int*)sm);
  const int width = min(VB, p.dv - v0);
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const int nc = (len + C - 1) / C;
  const long long gate0 = (long long)b * p.T * p.H + h;
  T* out = kStates ? nullptr : (T*)p.o + ((long long)b * p.T * p.H + h) * p.dv + v0;
  const long long out_step = (long long)p.H * p.dv;
  const int chunks = (p.T + C - 1) / C;
  const long long unit = (long long)b * p.H + h;
  float* hist = kStates ? p.hist + unit * chunks * p.dv * p.dk : nullptr;
  float* err = kStates ? p.err + unit * chunks * C * p.dv + v0 : nullptr;
  auto stage = [&](int c) { return sm + c % G::NS * G::kStage; };  // Q, K, V
  if (warp < kPrep / 32) {
    fewer_registers<G::kPrepRegs>();
    const T* qp = (const T*)p.q.p + b * p.q.batch + (long long)(h / p.q.share) * p.dk;
    const T* kp = (const T*)p.k.p + b * p.k.batch + (long long)(h / p.k.share) * p.dk;
    const T* vp = (const T*)p.v.p + b * p.v.batch + (long long)h * p.dv + v0;
    // what is copied asynchronously
    auto load = [&](int c) {
      const int n = len - c * C;
      const long long t0 = (long long)c * C;
      uint8_t* st = stage(c);
      load_tile<C, DK, kPrep>(st + G::KT, kp + t0 * p.k.step, p.k.step, n, p.dk, tid);
      if (!kStates) load_tile<C, DK, kPrep>(st, qp + t0 * p.q.step, p.q.step, n, p.dk, tid);
      if constexpr (NI == 1)
        load_tile<C, kVB, kPrep>(st + 2 * G::KT, vp + t0 * p.v.step, p.v.step, n, width, tid);
      else
        load_floats<C, G::LV>(st + 2 * G::KT, vp + t0 * p.v.step, p.v.step, n, width, tid);
    };
    // the gates of chunk c + 1 are made ready beside the preparation of chunk c, by
    // the last warp, which has loaded them one chunk earlier
    RawGates<C> raw;
    auto load_raw = [&](int c) {
      load_gates<C>(raw, p.log_decay, p.beta, gate0 + (long long)c * C * p.H, p.H, len - c * C, lane);
    };
    auto prep = [&](int c) {
      Gates<C>& g = gates[c % 3];
      uint8_t* st = stage(c);
      auto k_done = [&](int r, float s, float) {
        g.kup[r] = s;
        const float d = inverse_pow2(s);
        g.beta[r] = g.beta[r] * d * d;
      };
      auto q_done = [&](int r, float s, float) { g.qdown[r] = p.scale * inverse_pow2(s); };
      if constexpr (NI == 1) {
        HalfRows<C, DK, kPrep> k, q;
        k.read(st + G::KT, tid);
        if (!kStates) q.read(st, tid);
        k.template write<kFarKey>(st + G::KT, tid, no_least, k_done);
        if (!kStates) q.template write<kFarStep>(st, tid, no_least, q_done);
      } else {
        FloatRows<C, DK, kPrep> k, q;
        k.read(st + G::KT, tid);
        if (!kStates) q.read(st, tid);
        bar(1, kPrep);
        k.template write<kFarKey>(st + G::KT, tid, no_least, k_done);
        if (!kStates) q.template write<kFarStep>(st, tid, no_least, q_done);
      }
      bar(1, kPrep);
      prepare<NI, DK, !kStates, kHelped>(st, st + G::KT, sm + G::kM + (c & 1) * G::MT,
                                    sm + G::kP + (c & 1) * G::PT, g, scratch, tid, [&] {
                                      scan_gates<C>(gates[(c + 1) % 3], raw, lane);
                                      load_raw(c + 2);
                                    });
    };
    if (nc > 0) {
      load(0);
      copy_commit();
      if (nc > 1) load(1);
      copy_commit();
      if (warp == kPrep / 32 - 1) {
        load_raw(0);
        scan_gates<C>(gates[0], raw, lane);
        load_raw(1);
      }
      copy_wait<1>();
      bar(1, kPrep);
      prep(0);
    }
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      if (c + 1 < nc) {
        // (the stage that the walk has left)
        if (c + 2 < nc) load(c + 2);
        copy_commit();
        copy_wait<1>();
        bar(1, kPrep);
        prep(c + 1);
      }
      __syncthreads();
    }
  } else if (kHelped && warp >= kPrep / 32 + kWalkers) {
    fewer_registers<G::kPrepRegs>();
    const int vg = warp % kWalkers, w0 = 16 * vg;
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      if (w0 < width)
        form_o<NI, DK, G, T>({sm + G::kX + vg * G::kGiven}, vg, smem32(stage(c)),
                             smem32(sm + G::kM + (c & 1) * G::MT), smem32(sm + G::kP + (c & 1) * G::PT),
                             gates[c % 3], out + (long long)c * C * out_step + w0, out_step,
                             min(C, len - c * C), v0 + w0, p.dv, lane);
      __syncthreads();
    }
  } else {
    more_registers<G::kWalkRegs>();
    const int wi = warp - kPrep / 32, vg = wi / WK, kg = wi % WK;
    const int w0 = vg * 16;        // this warp's columns of v in the block
    const int k0 = kg * (DK / WK);  // and its columns of the state
    const int v = v0 + w0 + (lane >> 2), c2 = (lane & 3) * 2;
    auto owns = [&](int block) { return WK == 1 || block / OB == kg; };
    float4* ex = (float4*)(sm + G::kX) + (long long)vg * WK * NC * 32;
    const bool idle = w0 >= width;  // (fewer columns than warps for them)
    const Lane<G::RB> la(lane);
    const Lane<G::PB> lm(lane);
    const Lane<kPRow> lp(lane);
    const Given<G> given = {sm + G::kX + vg * G::kGiven};
    float x[NK][4];
    get_state<NK>(x, p.first ? p.first + unit * p.dv * p.dk : nullptr, v, p.dv, k0, p.dk, lane);
    float2 most = row_max<NK>(x);
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      if (idle) {
        __syncthreads();
        continue;
      }
      const uint8_t* st = stage(c);
      const uint32_t Q = smem32(st), K = Q + G::KT, V = K + G::KT;
      const uint32_t M = smem32(sm + G::kM + (c & 1) * G::MT), P = smem32(sm + G::kP + (c & 1) * G::PT);
      const Gates<C>& g = gates[c % 3];
      const int n = min(C, len - c * C);
      // f: F^T, then U^T.  o: O^T of the blocks that this warp writes, without s and of
      // q's scale
      float f[NC][4], o[2 * OB][4];
      const RowScales sx = row_scales<kLift>(most);
      {
        float qx[NC][4];
        state_times<NI, kOwn, DK, NK, NC>(f, qx, x, sx, K, Q, k0, la,
                                                   [&](int k, const uint32_t (&a)[kParts][4]) {
          if constexpr (kHelped) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) given.put(given.state(k, q, lane), a[q]);
            if (k == 0 && (lane & 3) == 0) *given.down(0, lane) = make_float2(sx.down0, sx.down1);
            if (k == NK / 2 - 1) bar_arrive(3 + vg, 64);
          }
          if constexpr (kStates)
            put_state<2>(x + 2 * k, hist + (long long)c * p.dv * p.dk, v, p.dv, k0 + 16 * k, p.dk, lane);
        });
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          scale_back(f[i], sx);
          if (kOwn) scale_back(qx[i], sx);
        }
        if constexpr (WK > 1) {
          float4* mine = ex + kg * NC * 32 + lane;
          constexpr int kO = kWalkers * NC * 32;  // o's after f's
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            mine[i * 32] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
            if (kOwn) mine[kO + i * 32] = make_float4(qx[i][0], qx[i][1], qx[i][2], qx[i][3]);
          }
          bar(3 + vg, 32 * WK);
          add_warps<WK, NC>(f, ex, kg, lane);
          if constexpr (kOwn) {
            zero(o);
            if (kg * OB < NB)
#pragma unroll
              for (int i = 0; i < 2 * OB; ++i)
#pragma unroll
                for (int q = 0; q < WK; ++q) {
                  const float4 t = ex[kO + (q * NC + kg * 2 * OB + i) * 32 + lane];
                  o[i][0] += t.x; o[i][1] += t.y; o[i][2] += t.z; o[i][3] += t.w;
                }
          }
        } else if constexpr (kOwn) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = qx[i][e];
        }
      }
#pragma unroll
      for (int i = 0; i < NC; i += 2) {
        float val[2][4];
        if constexpr (NI == 1) {
          uint32_t r[4];
          // steps 8 i ..., columns w0 ... as rows: the layout of a left operand's transpose
          ldm4t(r, V + at16<kVB * 2>(8 * i + (lane & 7) + (lane >> 4 << 3), w0 / 8 + (lane >> 3 & 1)));
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 t = unpack_bf(r[2 * q + u]);
              val[q][2 * u] = t.x;
              val[q][2 * u + 1] = t.y;
            }
        } else {
          const float* vf = (const float*)(st + 2 * G::KT);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              val[q][e] = vf[(8 * (i + q) + c2 + (e & 1)) * G::LV + w0 + (lane >> 2) + 8 * (e >> 1)];
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 l = *(const float2*)&g.lead[8 * (i + q) + c2];
          const float2 ku = *(const float2*)&g.kup[8 * (i + q) + c2];
          const float2 minus = make_float2(-l.x, -l.y);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            set_pair(f[i + q], u, fma2(minus, pair(f[i + q], u), mul2(ku, pair(val[q], u))));
        }
      }
      if constexpr (kOwn) {
#pragma unroll
        for (int i = 0; i < 2 * OB; ++i)
          times(o[i], *(const float2*)&g.lead[(WK == 1 ? 0 : min(kg * OB, NB - OB) * 16) + 8 * i + c2]);
      }
      if constexpr (kHelped) {
        // block by block, with y = beta F: E = F - X y, U = beta E, and y takes off F of the
        // later blocks what their rows of L T say.  The next block waits for its own share
        // alone; all else is beside the chain.
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          uint32_t a[kParts][4], r[kParts][2][2];
          float d[2][4], y[2][4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 bx = *(const float2*)&g.bx[16 * k + 8 * q + c2];
#pragma unroll
            for (int u = 0; u < 2; ++u) set_pair(y[q], u, mul2(pair(f[2 * k + q], u), bx));
          }
          const RowScales sy = row_scales<0>(row_max<2>(y));
          as_left<kParts>(a, y[0], y[1], sy.up0, sy.up1);
#pragma unroll
          for (int i = 2 * k + 2; i < NC; i += 2) {
            load_right<kParts, 2>(r, M, C * G::PB, lm, 8 * i, 16 * k);
            mma_short(d, a, r);
            add_rows(f[i], d[0], sy);
            add_rows(f[i + 1], d[1], sy);
          }
          load_right_t<kParts, 2>(r, M, C * G::PB, lm, 16 * k, 16 * k);
          mma_short(d, a, r);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int at = 16 * k + 8 * q + c2;
            add_rows(f[2 * k + q], d[q], sy);
            times(f[2 * k + q], *(const float2*)&g.beta[at]);
          }
          uint32_t ao[kParts][4];  // U for o
          const RowScales su = row_scales<kScore>(row_max<2>(f + 2 * k));
          as_left<kParts>(ao, f[2 * k], f[2 * k + 1], su.up0, su.up1);
#pragma unroll
          for (int q = 0; q < kParts; ++q) given.put(given.u(k, q, lane), ao[q]);
          if ((lane & 3) == 0) *given.down(1 + k, lane) = make_float2(su.down0, su.down1);
          // (in halves: all at once left what U adds to o to the end of the chunk, 179 us
          // against 175)
          if (k == NB / 2 - 1) bar_arrive(3 + kWalkers + vg, 64);
          if (k == NB - 1) bar_arrive(3 + 2 * kWalkers + vg, 64);
        }
      } else {
        // block by block: E = F - X beta F, U = beta E, and what U takes off F of the
        // later blocks and adds to O.  The next block waits for its own share alone; the
        // rest is issued while the next one's first product is on its way.
        uint32_t au[kParts][4];
        RowScales su;
        auto add_scaled = [&](float (*to)[4], const float (&d)[2][4]) {
          add_rows(to[0], d[0], su);
          add_rows(to[1], d[1], su);
        };
        auto rest = [&](int k) {
#pragma unroll
          for (int i = 2 * k + 4; i < NC; i += 2) {
            uint32_t r[kParts][2][2];
            float d[2][4];
            load_right<kParts, 2>(r, M, C * G::PB, lm, 8 * i, 16 * k);
            mma_short(d, au, r);
            add_scaled(f + i, d);
          }
          if constexpr (kOwn) {
#pragma unroll
            for (int j = 0; j < OB; ++j) {
              const int i = WK == 1 ? j : kg * OB + j;  // block
              if (i >= k && (WK == 1 || i < NB)) {
                uint32_t rp[kParts][2][2];
                float d[2][4];
                load_scores<C>(rp, M, P, lm, lp, i, k);
                mma_parts0<kParts, kParts, 2>(d, au, rp);
                add_scaled(o + 2 * j, d);
              }
            }
          }
        };
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          uint32_t a[kParts][4], r[kParts][2][2];
          float d[2][4], y[2][4];
          load_right_t<kParts, 2>(r, M, C * G::PB, lm, 16 * k, 16 * k);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int at = 16 * k + 8 * q + c2;
            const float2 bx = *(const float2*)&g.bx[at];
#pragma unroll
            for (int u = 0; u < 2; ++u) set_pair(y[q], u, mul2(pair(f[2 * k + q], u), bx));
          }
          const RowScales sy = row_scales<0>(row_max<2>(y));
          as_left<kParts>(a, y[0], y[1], sy.up0, sy.up1);
          mma_short(d, a, r);
          if (k > 0) rest(k - 1);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int at = 16 * k + 8 * q + c2;
            const float2 be = *(const float2*)&g.beta[at];
            add_rows(f[2 * k + q], d[q], sy);
            if (kStates)
#pragma unroll
              for (int e = 0; e < 4; ++e) d[q][e] = f[2 * k + q][e];
            times(f[2 * k + q], be);
            if constexpr (kStates) {
              const float2 ku = *(const float2*)&g.kup[at];
              float* ep = err + (long long)c * C * p.dv;
              if (owns(k))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int i = at + (e & 1), vv = w0 + (lane >> 2) + 8 * (e >> 1);
                  if (vv < width) ep[(long long)i * p.dv + vv] = d[q][e] * inverse_pow2(e & 1 ? ku.y : ku.x);
                }
            }
          }
          su = row_scales<kScore>(row_max<2>(f + 2 * k));
          as_left<kParts>(au, f[2 * k], f[2 * k + 1], su.up0, su.up1);
          if (k + 1 < NB) {
            load_right<kParts, 2>(r, M, C * G::PB, lm, 16 * k + 16, 16 * k);
            mma_short(d, au, r);
            add_scaled(f + 2 * k + 2, d);
          }
        }
        rest(NB - 1);
      }
      uint32_t y[NB][kParts][4];
#pragma unroll
      for (int i = 0; i < NC; ++i) times(f[i], *(const float2*)&g.tail[8 * i + c2]);
      const RowScales sw = row_scales<kLift>(row_max<NC>(f));
#pragma unroll
      for (int k = 0; k < NB; ++k) as_left<kParts>(y[k], f[2 * k], f[2 * k + 1], sw.up0, sw.up1);
      constexpr int kGroups = NK < 4 ? 1 : NK / 4;
      most = state_add<NI, DK, NK, NB>(x, g.last, y, sw, K, k0, la, [&](int i) {
        if constexpr (kOwn) {  // o's columns, shared out over the products
          constexpr int per = (2 * OB + kGroups - 1) / kGroups;
#pragma unroll
          for (int j = 0; j < per; ++j) {
            const int m = i * per + j;
            if (m < 2 * OB) {
              const int first = (WK == 1 ? 0 : kg * OB * 16) + 8 * m;  // step
              if (WK == 1 || first < C) {
                times(o[m], *(const float2*)&g.qdown[first + c2]);
                put_steps<T>(o[m], out + (long long)c * C * out_step + w0, out_step, first, n, v0 + w0, p.dv,
                             lane);
              }
            }
          }
        }
      });
      __syncthreads();
    }
    if (p.last) put_state<NK>(x, p.last + unit * p.dv * p.dk, v, p.dv, k0, p.dk, lane);
  }
  if (!kStates) clear_rows<T>(out, out_step, len, p.T, width, tid, blockDim.x);
}

// The walk back.  The sums are those of k's and q's scales: dU and y of 2^-n, dv of 2^n
// times theirs, and dO's rows are divided by q's.  dO's columns are scaled each by its own
// largest of the chunk: they are the rows of the left operands, and what is in one of
// them, infinities too, stays in it.
template <int NI, int DK, int WK>
__global__ void __launch_bounds__(kPrep + 32 * kWalkers, 1) k_delta_back(const DeltaBack p) {
  using G = Geom<NI, DK, WK, 1>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  constexpr int C = G::C, NC = G::NC, NB = C / 16, NK = DK / 8 / WK, VB = kVB / WK;
  constexpr int OB = NB / WK > 0 ? NB / WK : 1;
  extern __shared__ __align__(1024) uint8_t sm[];
  Gates<C>* gates = (Gates<C>*)(sm + G::kG);
  Scratch<C>& scratch = *(Scratch<C>*)(sm + G::kS);
  // of dO's columns: the bits of the largest of this chunk and the next, and what they
  // were divided by
  __shared__ __align__(16) uint32_t top_out[2][kVB];
  __shared__ float out_down[2][kVB];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (p.dv + VB - 1) / VB;
  const int h = blockIdx.x / vblocks, v0 = blockIdx.x % vblocks * VB;
  const int b = row_of(p.lens, p.B, p.T, tid, (int*)sm);
  const int width = min(VB, p.dv - v0);
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const int nc = (len + C - 1) / C;
  const long long gate0 = (long long)b * p.T * p.H + h;
  T* out = (T*)p.dv_out + ((long long)b * p.T * p.H + h) * p.dv + v0;
  const long long out_step = (long long)p.H * p.dv;
  const int chunks = (p.T + C - 1) / C;
  const long long unit = (long long)b * p.H + h;
  float* hist = p.hist + unit * chunks * p.dv * p.dk;
  float* ys = p.y + unit * chunks * C * p.dv + v0;
  auto stage = [&](int c) { return sm + c % G::NS * G::kStage; };  // Q, K, dO
  if (warp < kPrep / 32) {
    fewer_registers<G::kPrepRegs>();
    const T* qp = (const T*)p.q.p + b * p.q.batch + (long long)(h / p.q.share) * p.dk;
    const T* kp = (const T*)p.k.p + b * p.k.batch + (long long)(h / p.k.share) * p.dk;
    const T* gp = (const T*)p.dout.p + b * p.dout.batch + (long long)h * p.dv + v0;
    auto load = [&](int c) {
      const int n = len - c * C;
      const long long t0 = (long long)c * C;
      uint8_t* st = stage(c);
      load_tile<C, DK, kPrep>(st + G::KT, kp + t0 * p.k.step, p.k.step, n, p.dk, tid);
      load_tile<C, DK, kPrep>(st, qp + t0 * p.q.step, p.q.step, n, p.dk, tid);
      load_tile<C, kVB, kPrep>(st + 2 * G::KT, gp + t0 * p.dout.step, p.dout.step, n, width, tid);
    };
    RawGates<C> raw;
    auto load_raw = [&](int c) {  // (a chunk before the first has no steps)
      load_gates<C>(raw, p.log_decay, p.beta, gate0 + (long long)c * C * p.H, p.H,
                    c < 0 ? 0 : len - c * C, lane);
    };
    auto prep = [&](int c) {
      Gates<C>& g = gates[c % 3];
      uint8_t* st = stage(c);
      auto k_done = [&](int r, float s, float) {
        g.kup[r] = s;
        const float d = inverse_pow2(s);
        g.beta[r] = g.beta[r] * d * d;
      };
      auto q_done = [&](int r, float s, float) { g.qdown[r] = inverse_pow2(s); };
      // dO: a thread's eights (NI == 1) or fours of elements, of the same columns
      constexpr int E = NI == 1 ? 8 : 4, LPR = kVB / E, ND = C * LPR / kPrep;
      static_assert(C * LPR % kPrep == 0 && kPrep % LPR == 0, "");
      const int v8 = tid % LPR * E;
      float d[ND][E];
      if constexpr (NI == 1) {
        HalfRows<C, DK, kPrep> k, q;
        k.read(st + G::KT, tid);
        q.read(st, tid);
        k.template write<kFarKey>(st + G::KT, tid, no_least, k_done);
        q.template write<kFarStep>(st, tid, no_least, q_done);
      } else {
        FloatRows<C, DK, kPrep> k, q;
        k.read(st + G::KT, tid);
        q.read(st, tid);
#pragma unroll
        for (int i = 0; i < ND; ++i) {
          const float4 f = ((const float4*)(st + 2 * G::KT))[i * kPrep + tid];
          d[i][0] = f.x; d[i][1] = f.y; d[i][2] = f.z; d[i][3] = f.w;
        }
        bar(1, kPrep);
        k.template write<kFarKey>(st + G::KT, tid, no_least, k_done);
        q.template write<kFarStep>(st, tid, no_least, q_done);
      }
      bar(1, kPrep);
      float m[E];
#pragma unroll
      for (int e = 0; e < E; ++e) m[e] = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int r = (i * kPrep + tid) / LPR;
        if constexpr (NI == 1) {
          const uint4 q = *(const uint4*)(st + 2 * G::KT + at16<kVB * 2>(r, tid % LPR));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf((&q.x)[e]);
            d[i][2 * e] = f.x;
            d[i][2 * e + 1] = f.y;
          }
        }
        const float s = g.qdown[r];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          d[i][e] *= s;
          m[e] = fmaxf(m[e], fabsf(d[i][e]));
        }
      }
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
        for (int e = 0; e < E; ++e) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
      if (lane < LPR)
#pragma unroll
        for (int e = 0; e < E; ++e) atomicMax(&top_out[c & 1][v8 + e], __float_as_uint(m[e]));
      bar(1, kPrep);
      if (tid < kVB) {
        top_out[(c & 1) ^ 1][tid] = 0;  // (read a chunk ago)
        out_down[c & 1][tid] = scale_to<kLift>(__uint_as_float(top_out[c & 1][tid])).down;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) m[e] = scale_to<kLift>(__uint_as_float(top_out[c & 1][v8 + e])).up;
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int r = (i * kPrep + tid) / LPR;
        uint32_t q[E / 2][NI];
#pragma unroll
        for (int e = 0; e < E; e += 2) split2<NI>(d[i][e] * m[e], d[i][e + 1] * m[e + 1], q[e / 2]);
        if constexpr (NI == 1) {
          *(uint4*)(st + 2 * G::KT + at16<kVB * 2>(r, tid % LPR)) =
              make_uint4(q[0][0], q[1][0], q[2][0], q[3][0]);
        } else {
          const int x = tid % LPR;
          uint8_t* to = st + 2 * G::KT + at16<kVB * 2>(r, x >> 1) + (x & 1) * 8;
#pragma unroll
          for (int k = 0; k < NI; ++k) *(uint2*)(to + k * C * kVB * 2) = make_uint2(q[0][k], q[1][k]);
        }
      }
      prepare<NI, DK, true, false>(st, st + G::KT, sm + G::kM + (c & 1) * G::MT,
                                    sm + G::kP + (c & 1) * G::PT, g, scratch, tid, [&] {
                                      scan_gates<C>(gates[(c + 2) % 3], raw, lane);  // (c - 1)
                                      load_raw(c - 2);
                                    });
    };
    if (nc > 0) {
      if (tid < kVB) top_out[(nc - 1) & 1][tid] = 0;
      load(nc - 1);
      copy_commit();
      if (nc > 1) load(nc - 2);
      copy_commit();
      if (warp == kPrep / 32 - 1) {
        load_raw(nc - 1);
        scan_gates<C>(gates[(nc - 1) % 3], raw, lane);
        load_raw(nc - 2);
      }
      copy_wait<1>();
      bar(1, kPrep);
      prep(nc - 1);
    }
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      if (c > 0) {
        if (c > 1) load(c - 2);
        copy_commit();
        copy_wait<1>();
        bar(1, kPrep);
        prep(c - 1);
      }
      __syncthreads();
    }
  } else {
    more_registers<G::kWalkRegs>();
    const int wi = warp - kPrep / 32, vg = wi / WK, kg = wi % WK;
    const int w0 = vg * 16, k0 = kg * (DK / WK);
    const int v = v0 + w0 + (lane >> 2), c2 = (lane & 3) * 2;
    auto owns = [&](int block) { return WK == 1 || block / OB == kg; };
    float4* ex = (float4*)(sm + G::kX) + (long long)vg * WK * NC * 32;
    const bool idle = w0 >= width;
    const Lane<G::RB> la(lane);
    const Lane<G::PB> lm(lane);
    const Lane<kPRow> lp(lane);
    const Lane<kVB * 2> lv(lane);
    float x[NK][4];  // D
    get_state<NK>(x, p.first ? p.first + unit * p.dv * p.dk : nullptr, v, p.dv, k0, p.dk, lane);
    float2 most = row_max<NK>(x);
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      if (idle) {
        __syncthreads();
        continue;
      }
      const uint32_t Q = smem32(stage(c)), K = Q + G::KT, dO = K + G::KT;
      const uint32_t M = smem32(sm + G::kM + (c & 1) * G::MT), P = smem32(sm + G::kP + (c & 1) * G::PT);
      const Gates<C>& g = gates[c % 3];
      const int n = min(C, len - c * C);
      float f[NC][4];  // dU^T, then dv^T
      {
        const RowScales sx = row_scales<kLift>(most);
        // (the state is stored between the products: all at once the warp waited 1400
        // cycles for its own stores)
        state_times<NI, false, DK, NK, NC>(f, f, x, sx, K, K, k0, la, [&](int k, const uint32_t (&)[kParts][4]) {
          put_state<2>(x + 2 * k, hist + (long long)c * p.dv * p.dk, v, p.dv, k0 + 16 * k, p.dk, lane);
        });
#pragma unroll
        for (int i = 0; i < NC; ++i) scale_back(f[i], sx);
        if constexpr (WK > 1) {
          float4* mine = ex + kg * NC * 32 + lane;
#pragma unroll
          for (int i = 0; i < NC; ++i) mine[i * 32] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
          bar(3 + vg, 32 * WK);
          add_warps<WK, NC>(f, ex, kg, lane);
        }
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) times(f[i], *(const float2*)&g.tail[8 * i + c2]);
      // of rows g and g + 8
      const float so[2] = {p.scale * out_down[c & 1][w0 + (lane >> 2)],
                           p.scale * out_down[c & 1][w0 + (lane >> 2) + 8]};
      // dO's rows v, steps 16 k ... as a left operand
      auto dout_left = [&](uint32_t (&a)[NI][4], int k) {
#pragma unroll
        for (int q = 0; q < NI; ++q)
          ldm4t(a[q], lv.left_t(dO, w0, 16 * k) + q * C * kVB * 2);
      };
      // P^T dO for the steps of block k
      auto from_out = [&](int k) {
        float d[2][4];
#pragma unroll
        for (int i = k; i < NB; ++i) {
          uint32_t a[NI][4], r[kParts][2][2];
          dout_left(a, i);
          if (i == k) load_right_t<kParts, 2>(r, P, C * kPRow, lp, 0, 16 * k);
          else load_right_t<kParts, 2>(r, M, C * G::PB, lm, 16 * i, 16 * k);
          if (i == k) mma_parts0<NI, kParts, 2>(d, a, r);
          else mma_parts<NI, kParts, 2>(d, a, r);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            set_pair(f[2 * k + q], u,
                     fma2(both(so[u] * pow2(-kScore)), pair(d[q], u), pair(f[2 * k + q], u)));
      };
      // what dO adds to D waits for nothing of this chunk: its products go between the
      // steps of the solution, each of which waits for the one before
      uint32_t zo[NB][kParts][4];
      RowScales sz;
      {
        float z[NC][4];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          uint32_t a[NI][4];
          dout_left(a, k);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float2 s = unpack_half(a[0][w]);
            if (NI == 2) {
              const float2 t = unpack_half(a[NI - 1][w]);
              s.x += t.x;
              s.y += t.y;
            }
            // registers 0, 1: rows g, g + 8 of the first eight steps; 2, 3: of the others
            const float2 l = *(const float2*)&g.lead[16 * k + 8 * (w >> 1) + c2];
            z[2 * k + (w >> 1)][2 * (w & 1)] = s.x * so[w & 1] * l.x;
            z[2 * k + (w >> 1)][2 * (w & 1) + 1] = s.y * so[w & 1] * l.y;
          }
        }
        sz = row_scales<kLift>(row_max<NC>(z));
#pragma unroll
        for (int k = 0; k < NB; ++k) as_left<kParts>(zo[k], z[2 * k], z[2 * k + 1], sz.up0, sz.up1);
      }
      constexpr int GN = NK < 4 ? NK : 4, kGroups = NK / GN, kPer = (kGroups + NB - 1) / NB;
      auto add_out = [&](int k) {
#pragma unroll
        for (int i = k * kPer; i < (k + 1) * kPer && i < kGroups; ++i)
          columns_add<NI, DK, GN, NB>(x + i * GN, g.last, zo, sz, Q, k0 + 8 * GN * i, la, [] {});
      };
      // from the last block back: y = dU - X^T beta dU, dv = beta y, and what dv takes
      // off dU of the earlier blocks (the order of issue as in the walk)
      uint32_t av[kParts][4];
      RowScales su;
      auto add_scaled = [&](float (*to)[4], const float (&d)[2][4]) {
        add_rows(to[0], d[0], su);
        add_rows(to[1], d[1], su);
      };
      auto rest = [&](int k) {
#pragma unroll
        for (int i = 0; i < 2 * k - 2; i += 2) {
          uint32_t r[kParts][2][2];
          float d[2][4];
          load_right_t<kParts, 2>(r, M, C * G::PB, lm, 8 * i, 16 * k);
          mma_short(d, av, r);
          add_scaled(f + i, d);
        }
      };
      from_out(NB - 1);
#pragma unroll
      for (int k = NB - 1; k >= 0; --k) {
        uint32_t a[kParts][4], r[kParts][2][2];
        float d[2][4], y[2][4];
        load_right<kParts, 2>(r, M, C * G::PB, lm, 16 * k, 16 * k);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 be = *(const float2*)&g.beta[16 * k + 8 * q + c2];
#pragma unroll
          for (int u = 0; u < 2; ++u) set_pair(y[q], u, mul2(pair(f[2 * k + q], u), be));
        }
        const RowScales sy = row_scales<0>(row_max<2>(y));
        as_left<kParts>(a, y[0], y[1], sy.up0, sy.up1);
        mma_short(d, a, r);
        if (k + 1 < NB) rest(k + 1);
        if (k > 0) from_out(k - 1);
        add_out(k);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at = 16 * k + 8 * q + c2;
          const float2 be = *(const float2*)&g.beta[at], xs = *(const float2*)&g.xs[at];
          const float2 ku = *(const float2*)&g.kup[at];
          float* yp = ys + (long long)c * C * p.dv;
          float yv[4];
          times(d[q], xs);
          add_rows(f[2 * k + q], d[q], sy);
#pragma unroll
          for (int e = 0; e < 4; ++e) yv[e] = f[2 * k + q][e];
          times(f[2 * k + q], be);
          if (owns(k)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = at + (e & 1), vv = w0 + (lane >> 2) + 8 * (e >> 1);
              if (vv < width) yp[(long long)i * p.dv + vv] = yv[e] * inverse_pow2(e & 1 ? ku.y : ku.x);
            }
            const float* z = f[2 * k + q];
            const float r4[4] = {z[0] * ku.x, z[1] * ku.y, z[2] * ku.x, z[3] * ku.y};
            put_steps<T>(r4, out + (long long)c * C * out_step + w0, out_step, 16 * k + 8 * q, n, v0 + w0,
                         p.dv, lane);
          }
        }
        su = row_scales<kScore>(row_max<2>(f + 2 * k));
        as_left<kParts>(av, f[2 * k], f[2 * k + 1], su.up0, su.up1);
        if (k > 0) {
          load_right_t<kParts, 2>(r, M, C * G::PB, lm, 16 * k - 16, 16 * k);
          mma_short(d, av, r);
          add_scaled(f + 2 * k - 2, d);
        }
      }
      uint32_t y[NB][kParts][4];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const float2 l = *(const float2*)&g.lead[8 * i + c2];
        times(f[i], make_float2(-l.x, -l.y));
      }
      {
        const RowScales sw = row_scales<kLift>(row_max<NC>(f));
#pragma unroll
        for (int k = 0; k < NB; ++k) as_left<kParts>(y[k], f[2 * k], f[2 * k + 1], sw.up0, sw.up1);
        most = state_add<NI, DK, NK, NB>(x, 1.f, y, sw, K, k0, la, [](int) {});
      }
      __syncthreads();
    }
    if (p.last) put_state<NK>(x, p.last + unit * p.dv * p.dk, v, p.dv, k0, p.dk, lane);
  }
  clear_rows<T>(out, out_step, len, p.T, width, tid, blockDim.x);
}

// CTAs of a walk
dim3 walk_grid(int H, int B, int dv, int wk) { return dim3(H * ((dv + kVB / wk - 1) / (kVB / wk)), B); }

template <int NI, int DK, int WK, bool kStates>
cudaError_t walk_t(const DeltaWalk& p, cudaStream_t s) {
  using G = Geom<NI, DK, WK, kStates ? 1 : 2, helped<NI, DK, WK, kStates>()>;
  constexpr size_t smem = G::smem;
  static_assert(smem <= 232448, "");
  const cudaError_t e = cudaFuncSetAttribute(k_delta_walk<NI, DK, WK, kStates>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "delta_states" : "delta_walk", s);
  k_delta_walk<NI, DK, WK, kStates>
      <<<walk_grid(p.H, p.B, p.dv, WK), G::kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <int NI, int DK, int WK>
cudaError_t back_t(const DeltaBack& p, cudaStream_t s) {
  using G = Geom<NI, DK, WK, 1>;
  constexpr size_t smem = G::smem;
  static_assert(smem + 16 * kVB <= 232448, "");
  const cudaError_t e = cudaFuncSetAttribute(k_delta_back<NI, DK, WK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls("delta_back", s);
  k_delta_back<NI, DK, WK><<<walk_grid(p.H, p.B, p.dv, WK), G::kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

// Warps that share 16 columns of v: as many as leave every CTA an SM of its own.  Below
// that the shared rows' shorter chain gains, above it the second wave costs more (us of the
// walk that keeps the states, one, two, four warps; CTAs with one):
//   1 x 4096, 32 heads 128/64 (32): 267 226 211    2 x 2048, 32 heads 128/64 (64): 142 123 222
//   1 x 4096, 16 heads 64/64 (16): 185 178 169     2 x 2048, 24 heads 64/64 (48): 97 95 175
//   3 x 2048, 32 heads 128/64 (96): 143 232 327    8 x 1024, 24 heads 64/64 (192): 103 144 261
int warps_per_rows(int B, int H, int dv) {
  for (int wk = 4; wk > 1; wk /= 2) {
    const dim3 g = walk_grid(H, B, dv, wk);
    if ((long long)g.x * g.y <= kLaSms) return wk;
  }
  return 1;
}
template <int NI, int DK, bool kStates>
cudaError_t walk_k(const DeltaWalk& p, cudaStream_t s) {
  const int wk = warps_per_rows(p.B, p.H, p.dv);
  return wk == 4   ? walk_t<NI, DK, 4, kStates>(p, s)
         : wk == 2 ? walk_t<NI, DK, 2, kStates>(p, s)
                   : walk_t<NI, DK, 1, kStates>(p, s);
}
template <int NI, int DK>
cudaError_t back_k(const DeltaBack& p, cudaStream_t s) {
  const int wk = warps_per_rows(p.B, p.H, p.dv);
  return wk == 4 ? back_t<NI, DK, 4>(p, s) : wk == 2 ? back_t<NI, DK, 2>(p, s) : back_t<NI, DK, 1>(p, s);
}

// One token: A = a S, e = v - A k, S' = A + beta e k^T, o = s S' q.  A row of the
// state (dk floats) is held by LPR lanes, four floats each, and a warp takes NR rows
// a lane at once: their loads are in flight together, and their dot products with k
// are added up together (while a lane holds several sums, each exchange halves
// them), as are those with q.  o needs no second pass: S' q = A q + beta e (k . q).
//
// Bound by the states' bytes, read and written once: 256 rows of 64 heads 128/64 take 160
// us, the copy rate.  Eight rows a lane where that leaves two CTAs an SM, else two, so that
// a single row (32 heads 128/64: 6.7 us) is on 256 CTAs.
constexpr int kStepWarps = 4;

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
// every lane of LPR gets the sum over them
template <int LPR>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <typename T, int LPR, int NR>
__global__ void __launch_bounds__(kStepWarps * 32) k_delta_step(const DeltaStep p) {
  constexpr int RPW = 32 / LPR;                 // rows of a warp side by side
  constexpr int kRows = kStepWarps * RPW * NR;  // rows of a CTA
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
  const float a = expf(p.log_decay[(long long)b * p.H + h]), beta = p.beta[(long long)b * p.H + h];
  float q[4] = {0.f, 0.f, 0.f, 0.f}, k[4] = {0.f, 0.f, 0.f, 0.f};
  if (kin) {
    load4((const T*)p.q + b * p.q_batch + (long long)g * p.dk + k0, q);
    load4((const T*)p.k + b * p.k_batch + (long long)g * p.dk + k0, k);
  }
  const float kq = sum_lanes<LPR>(fmaf(k[0], q[0], fmaf(k[1], q[1], fmaf(k[2], q[2], k[3] * q[3]))));
  const T* vp = (const T*)p.v + b * p.v_batch + (long long)h * p.dv;
  float r[NR], o[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    s[i].x *= a; s[i].y *= a; s[i].z *= a; s[i].w *= a;
    r[i] = fmaf(s[i].x, k[0], fmaf(s[i].y, k[1], fmaf(s[i].z, k[2], s[i].w * k[3])));
    o[i] = fmaf(s[i].x, q[0], fmaf(s[i].y, q[1], fmaf(s[i].z, q[2], s[i].w * q[3])));
  }
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      r[i] += __shfl_xor_sync(0xffffffffu, r[i], d);
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], d);
    }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int v = vb + i * RPW;
    if (v >= p.dv) continue;
    const float u = beta * (to_f32(vp[v]) - r[i]);
    s[i].x = fmaf(u, k[0], s[i].x);
    s[i].y = fmaf(u, k[1], s[i].y);
    s[i].z = fmaf(u, k[2], s[i].z);
    s[i].w = fmaf(u, k[3], s[i].w);
    if (kin && row >= 0) *(float4*)(p.state_out + at + (long long)i * RPW * p.dk) = s[i];
    if (sub == 0)
      ((T*)p.o)[((long long)b * p.H + h) * p.dv + v] =
          from_f32<T>(row >= 0 ? p.scale * fmaf(u, kq, o[i]) : 0.f);
  }
}

template <typename T, int LPR>
cudaError_t step_l(const DeltaStep& p, cudaStream_t s) {
  LaunchScope ls("delta_step", s);
  constexpr int rows = kStepWarps * (32 / LPR);
  if ((long long)p.B * p.H * ((p.dv + 8 * rows - 1) / (8 * rows)) >= 2 * kLaSms)
    k_delta_step<T, LPR, 8><<<dim3((p.dv + 8 * rows - 1) / (8 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  else
    k_delta_step<T, LPR, 2><<<dim3((p.dv + 2 * rows - 1) / (2 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t step_t(const DeltaStep& p, cudaStream_t s) {
  const int lanes = p.dk / 4;
  if (lanes <= 4) return step_l<T, 4>(p, s);
  if (lanes <= 8) return step_l<T, 8>(p, s);
  if (lanes <= 16) return step_l<T, 16>(p, s);
  return step_l<T, 32>(p, s);
}

}  // namespace

cudaError_t delta_walk(const DeltaWalk& p, bool bf16, cudaStream_t s) {
  if (p.hist) {
    if (bf16) return p.dk <= 64 ? walk_k<1, 64, true>(p, s) : walk_k<1, 128, true>(p, s);
    return p.dk <= 64 ? walk_k<2, 64, true>(p, s) : walk_k<2, 128, true>(p, s);
  }
  if (bf16) return p.dk <= 64 ? walk_k<1, 64, false>(p, s) : walk_k<1, 128, false>(p, s);
  return p.dk <= 64 ? walk_k<2, 64, false>(p, s) : walk_k<2, 128, false>(p, s);
}

cudaError_t delta_back(const DeltaBack& p, bool bf16, cudaStream_t s) {
  if (bf16) return p.dk <= 64 ? back_k<1, 64>(p, s) : back_k<1, 128>(p, s);
  return p.dk <= 64 ? back_k<2, 64>(p, s) : back_k<2, 128>(p, s);
}

cudaError_t delta_step(const DeltaStep& p, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

int delta_chunk(bool bf16) { return bf16 ? kSteps<1> : kSteps<2>; }

}  // namespace ssd
