// Gated delta rule: the walk over the chunks of a row (outputs and state, or the
// states before every chunk and the errors E), the walk back (the gradients of the
// states and of v), and the step of one token.  The formulas of a chunk stand in
// ssd_delta.cuh; the gradients of L = sum(do . o) + sum(dS . S_T) are, with D the
// gradient of the state after a chunk,
//   dU = P^T dO + e^{G-g} K D^T,  (I + L^T beta) y = dU,  dv = beta y,
//   dbeta_i = E_i . y_i,  D <- e^G D + (s e^g dO)^T Q - (e^g dv)^T K
// and those of q, k and the decays need no walk (ssd_delta_grads.cu).
//
// One CTA per (head, 64 columns of v, row): the rows of the state are independent
// of each other.  Four warps hold 16 rows of the state each, in registers, in the
// layout in which matrix instructions leave their results.  That is also the layout
// in which they take a left operand, and every product of the chain that one chunk
// has to pass on to the next has such a one: F^T = V^T - H K^T from the state, E^T
// from F^T, the new state from U^T.  So that chain runs within a warp, without a
// word through shared memory; four other warps meanwhile prepare the next chunk (L,
// X, P: all that does not depend on the state) and load the one after it, and one
// barrier a chunk hands over.
#include <cuda_bf16.h>

#include "ssd_delta.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace delta;

// Parts of the state, P and U where they make o alone.  A bf16 o has 8 bits: two
// parts (16) leave it its own rounding, 0.0017 of its root mean square; with one
// part of the state and of P it was off by 0.0028 where o is small beside its terms.
template <int NI>
constexpr int kOutParts = NI == 1 ? 2 : 3;

template <int NI, int DK, int PP>
struct Geom {
  static constexpr int C = kSteps<NI>;
  static constexpr int RB = DK * 2, PB = C * 2;      // bytes of a row of K, of M
  static constexpr int KT = NI * C * RB;             // K's or Q's tile, all parts
  // V in the walk (bf16 as it is, fp32 as floats whose rows are 4 banks apart),
  // dO in the walk back (parts)
  static constexpr int LV = kVB + 4;
  static constexpr int VT = NI == 1 ? C * kVB * 2 : C * kVB * 2 * NI;
  static_assert(NI == 1 || C * LV * 4 <= VT, "");
  static constexpr int NS = NI == 1 ? 3 : 2;         // stages of the operands
  static constexpr int MT = kParts * C * PB, PT = PP * C * PB;
  static constexpr int kStage = 2 * KT + VT;
  static constexpr int kM = NS * kStage, kP = kM + 2 * MT;
  static constexpr int kG = kP + 2 * PT, kS = kG + 3 * (int)sizeof(Gates<C>);
  static constexpr size_t smem = kS + sizeof(Scratch<C>);
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

// A warp's rows of a state [dv][dk]: x[j]: row v (+ 8 for e >= 2), column 8 j + 2 t
// (+ 1 for odd e), from or to memory.
template <int NK>
__device__ __forceinline__ void get_state(float (&x)[NK][4], const float* p, int v, int dv, int dk,
                                          int lane) {
  const int c = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < NK; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float2 f = make_float2(0.f, 0.f);
      if (p && v + 8 * u < dv && 8 * j < dk) f = *(const float2*)(p + (v + 8 * u) * dk + 8 * j + c);
      x[j][2 * u] = f.x;
      x[j][2 * u + 1] = f.y;
    }
}
template <int NK>
__device__ __forceinline__ void put_state(const float (&x)[NK][4], float* p, int v, int dv, int dk,
                                          int lane) {
  const int c = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < NK; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (v + 8 * u < dv && 8 * j < dk)
        *(float2*)(p + (v + 8 * u) * dk + 8 * j + c) = make_float2(x[j][2 * u], x[j][2 * u + 1]);
}

// x (rows v, columns c0 ... of steps, eight) transposed to rows of memory: row i of
// step i, n steps, `step` elements apart; at: the first step's element v0.
template <typename T>
__device__ __forceinline__ void put_steps(const float (&x)[4], T* at, long long step, int c0, int n,
                                          int v0, int dv, int lane) {
  const int g = lane >> 2, c = (lane & 3) * 2;
  if constexpr (sizeof(T) == 2) {
    const uint32_t a = transpose8(pack2(x[0], x[1])), b = transpose8(pack2(x[2], x[3]));
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

// f[n] += X K^T for the C steps of a tile whose rows are steps, X the state with all
// its parts; and with PO > 0 o[n] += X Q^T with PO of them.  The right operands of a
// group of columns are loaded while the group before is multiplied.
template <int NI, int PO, int DK, int NK, int NC>
__device__ __forceinline__ void state_times(float (&f)[NC][4], float (&o)[NC][4],
                                            const float (&x)[NK][4], uint32_t K, uint32_t Q, int lane) {
  constexpr int C = kSteps<NI>, RB = DK * 2;
  constexpr int GN = NI == 1 ? 4 : 2;                   // columns of eight of a group
  constexpr int GF = NC / GN, GK = PO > 0 ? 2 * GF : GF;  // groups of 16 terms
  constexpr int NG = NK / 2 * GK;
  uint32_t a[2][kParts][4], b[2][NI][GN][2];
  auto load = [&](int s) {
    const int k = s / GK, g = s % GK;
    load_right<RB, NI, GN>(b[s & 1], g < GF ? K : Q, C * RB, lane, 8 * GN * (g % GF), 16 * k);
  };
  as_left<kParts>(a[0], x[0], x[1]);
  load(0);
#pragma unroll
  for (int s = 0; s < NG; ++s) {
    const int k = s / GK, g = s % GK;
    if (s + 1 < NG) load(s + 1);
    if (g == 0 && 2 * k + 2 < NK) as_left<kParts>(a[(k + 1) & 1], x[2 * k + 2], x[2 * k + 3]);
    if (g < GF) {
      mma_parts<kParts, NI, GN>(f + GN * g, a[k & 1], b[s & 1]);
    } else if constexpr (PO > 0) {
      uint32_t ao[PO][4];
#pragma unroll
      for (int q = 0; q < PO; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) ao[q][e] = a[k & 1][q][e];
      mma_parts<PO, NI, GN>(o + GN * (g - GF), ao, b[s & 1]);
    }
  }
}

// d += a b for two columns of eight, all parts of both; the products of one order of
// size go to a sum of their own, so that fewer wait for one another.
__device__ __forceinline__ void mma_short(float (&d)[2][4], const uint32_t (&a)[kParts][4],
                                          const uint32_t (&b)[kParts][2][2]) {
  float e[2][2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) e[i][n][c] = 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
#pragma unroll
    for (int n = 0; n < 2; ++n) mma(e[0][n], a[i], b[2 - i][n][0], b[2 - i][n][1]);
    if (i < 2)
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(e[1][n], a[i], b[1 - i][n][0], b[1 - i][n][1]);
    if (i == 0)
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(d[n], a[0], b[0][n][0], b[0][n][1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) d[n][c] += e[0][n][c] + e[1][n][c];
}

// x <- scale x + Y tile, Y (rows v, C steps) as parts of left operands.  beside(i),
// i < NK / 4: work that is issued between the products.
template <int NI, int DK, int NK, int NB, typename F>
__device__ __forceinline__ void state_add(float (&x)[NK][4], float scale, const uint32_t (*y)[kParts][4],
                                          uint32_t tile, int lane, F beside) {
  constexpr int C = kSteps<NI>, RB = DK * 2;
#pragma unroll
  for (int n = 0; n < NK; n += 4) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t r[NI][4][2];
      load_right_t<RB, NI, 4>(r, tile, C * RB, lane, 8 * n, 16 * b);
      mma_parts<kParts, NI, 4>(d, y[b], r);
      if (b == 0) beside(n / 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n + i][e] = fmaf(scale, x[n + i][e], d[i][e]);
  }
}

template <int NI, int DK, bool kStates>
__global__ void __launch_bounds__(256, 1) k_delta_walk(const DeltaWalk p) {
  constexpr int PP = kOutParts<NI>;
  using G = Geom<NI, DK, PP>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  constexpr int C = G::C, NC = C / 8, NB = C / 16, NK = DK / 8;
  extern __shared__ __align__(1024) uint8_t sm[];
  Gates<C>* gates = (Gates<C>*)(sm + G::kG);
  Scratch<C>& scratch = *(Scratch<C>*)(sm + G::kS);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (p.dv + kVB - 1) / kVB;
  const int h = blockIdx.x / vblocks, v0 = blockIdx.x % vblocks * kVB, b = blockIdx.y;
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
    const T* qp = (const T*)p.q.p + b * p.q.batch + (long long)(h / p.q.share) * p.dk;
    const T* kp = (const T*)p.k.p + b * p.k.batch + (long long)(h / p.k.share) * p.dk;
    const T* vp = (const T*)p.v.p + b * p.v.batch + (long long)h * p.dv + v0;
    auto load = [&](int c) {
      const int n = len - c * C;
      const long long t0 = (long long)c * C;
      uint8_t* st = stage(c);
      load_tile<NI, C, DK, kPrep>(st + G::KT, kp + t0 * p.k.step, p.k.step, n, p.dk, tid);
      if (!kStates) load_tile<NI, C, DK, kPrep>(st, qp + t0 * p.q.step, p.q.step, n, p.dk, tid);
      if constexpr (NI == 1)
        load_tile<1, C, kVB, kPrep>(st + 2 * G::KT, vp + t0 * p.v.step, p.v.step, n, p.dv - v0, tid);
      else
        load_floats<C, G::LV>(st + 2 * G::KT, (const float*)vp + t0 * p.v.step, p.v.step, n,
                              p.dv - v0, tid);
    };
    // the gates of chunk c + 1 are made ready beside the preparation of chunk c, by
    // the last warp, which has loaded them one chunk earlier
    RawGates<C> raw;
    auto load_raw = [&](int c) {
      load_gates<C>(raw, p.log_decay, p.beta, gate0 + (long long)c * C * p.H, p.H, len - c * C, lane);
    };
    auto prep = [&](int c) {
      prepare<NI, DK, PP, !kStates>(stage(c), stage(c) + G::KT, sm + G::kM + (c & 1) * G::MT,
                                    sm + G::kP + (c & 1) * G::PT, gates[c % 3], scratch, p.scale, tid,
                                    [&] {
                                      scan_gates<C>(gates[(c + 1) % 3], raw, lane);
                                      load_raw(c + 2);
                                    });
    };
    if (nc > 0) {
      load(0);
      copy_commit();
      if (G::NS > 2 && nc > 1) load(1);
      copy_commit();
      if (warp == 3) {
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
        if (G::NS > 2 ? c + 2 < nc : true) load(G::NS > 2 ? c + 2 : c + 1);
        copy_commit();
        copy_wait<G::NS - 2>();
        bar(1, kPrep);
        prep(c + 1);
      }
      __syncthreads();
    }
  } else {
    const int w0 = (warp - kPrep / 32) * 16;  // this warp's columns of v in the block
    const int v = v0 + w0 + (lane >> 2), c2 = (lane & 3) * 2;
    float x[NK][4];
    get_state<NK>(x, p.first ? p.first + unit * p.dv * p.dk : nullptr, v, p.dv, p.dk, lane);
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      const uint8_t* st = stage(c);
      const uint32_t Q = smem32(st), K = Q + G::KT, V = K + G::KT;
      const uint32_t M = smem32(sm + G::kM + (c & 1) * G::MT), P = smem32(sm + G::kP + (c & 1) * G::PT);
      const Gates<C>& g = gates[c % 3];
      const int n = min(C, len - c * C);
      if (kStates) put_state<NK>(x, hist + (long long)c * p.dv * p.dk, v, p.dv, p.dk, lane);
      // f: F^T, then U^T; o: O^T
      float f[NC][4], o[NC][4];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = o[i][e] = 0.f;
      state_times<NI, kStates ? 0 : PP, DK, NK, NC>(f, o, x, K, Q, lane);
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
              val[q][2 * u] = __uint_as_float(r[2 * q + u] << 16);
              val[q][2 * u + 1] = __uint_as_float(r[2 * q + u] & 0xffff0000u);
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
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            f[i + q][2 * u] = fmaf(-l.x, f[i + q][2 * u], val[q][2 * u]);
            f[i + q][2 * u + 1] = fmaf(-l.y, f[i + q][2 * u + 1], val[q][2 * u + 1]);
            if (!kStates) {
              o[i + q][2 * u] *= l.x * p.scale;
              o[i + q][2 * u + 1] *= l.y * p.scale;
            }
          }
        }
      }
      // block by block: E = F - X beta F, U = beta E, and what U takes off F of the
      // later blocks and adds to O.  The next block waits for its own share alone; the
      // rest is issued while the next one's first product is on its way.
      uint32_t au[kParts][4];
      auto rest = [&](int k) {
#pragma unroll
        for (int i = 2 * k + 4; i < NC; i += 2) {
          uint32_t r[kParts][2][2];
          load_right<G::PB, kParts, 2>(r, M, C * G::PB, lane, 8 * i, 16 * k);
          mma_parts<kParts, kParts, 2>(f + i, au, r);
        }
        if constexpr (!kStates) {
          uint32_t ao[PP][4];
#pragma unroll
          for (int q = 0; q < PP; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) ao[q][e] = au[q][e];
#pragma unroll
          for (int i = 2 * k; i < NC; i += 2) {
            uint32_t rp[PP][2][2];
            load_right<G::PB, PP, 2>(rp, P, C * G::PB, lane, 8 * i, 16 * k);
            mma_parts<PP, PP, 2>(o + i, ao, rp);
          }
        }
      };
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t a[kParts][4], r[kParts][2][2];
        float d[2][4], y[2][4];
        load_right_t<G::PB, kParts, 2>(r, M, C * G::PB, lane, 16 * k, 16 * k);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 be = *(const float2*)&g.beta[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[q][e] = 0.f;
            y[q][e] = f[2 * k + q][e] * (e & 1 ? be.y : be.x);
          }
        }
        as_left<kParts>(a, y[0], y[1]);
        mma_short(d, a, r);
        if (k > 0) rest(k - 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 be = *(const float2*)&g.beta[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ev = f[2 * k + q][e] + d[q][e];
            if (kStates) d[q][e] = ev;
            f[2 * k + q][e] = ev * (e & 1 ? be.y : be.x);
          }
          if constexpr (kStates) {
            float* ep = err + (long long)c * C * p.dv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 16 * k + 8 * q + c2 + (e & 1), vv = w0 + (lane >> 2) + 8 * (e >> 1);
              if (v0 + vv < p.dv) ep[(long long)i * p.dv + vv] = d[q][e];
            }
          }
        }
        as_left<kParts>(au, f[2 * k], f[2 * k + 1]);
        if (k + 1 < NB) {
          load_right<G::PB, kParts, 2>(r, M, C * G::PB, lane, 16 * k + 16, 16 * k);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[q][e] = f[2 * k + 2 + q][e];
          mma_short(d, au, r);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[2 * k + 2 + q][e] = d[q][e];
        }
      }
      rest(NB - 1);
      uint32_t y[NB][kParts][4];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 t = *(const float2*)&g.tail[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[2 * k + q][e] *= e & 1 ? t.y : t.x;
        }
        as_left<kParts>(y[k], f[2 * k], f[2 * k + 1]);
      }
      state_add<NI, DK, NK, NB>(x, g.last, y, K, lane, [&](int i) {
        if constexpr (!kStates) {  // o's columns, shared out over the products
          constexpr int per = NC / (NK / 4) > 0 ? NC / (NK / 4) : 1;
#pragma unroll
          for (int j = 0; j < per; ++j)
            if (i * per + j < NC)
              put_steps<T>(o[i * per + j], out + (long long)c * C * out_step + w0, out_step,
                           8 * (i * per + j), n, v0 + w0, p.dv, lane);
        }
      });
      __syncthreads();
    }
    if (p.last) put_state<NK>(x, p.last + unit * p.dv * p.dk, v, p.dv, p.dk, lane);
  }
  if (!kStates) clear_rows<T>(out, out_step, len, p.T, min(kVB, p.dv - v0), tid, blockDim.x);
}

// The walk back.
template <int NI, int DK>
__global__ void __launch_bounds__(256, 1) k_delta_back(const DeltaBack p) {
  using G = Geom<NI, DK, kParts>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  constexpr int C = G::C, NC = C / 8, NB = C / 16, NK = DK / 8;
  extern __shared__ __align__(1024) uint8_t sm[];
  Gates<C>* gates = (Gates<C>*)(sm + G::kG);
  Scratch<C>& scratch = *(Scratch<C>*)(sm + G::kS);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (p.dv + kVB - 1) / kVB;
  const int h = blockIdx.x / vblocks, v0 = blockIdx.x % vblocks * kVB, b = blockIdx.y;
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
    const T* qp = (const T*)p.q.p + b * p.q.batch + (long long)(h / p.q.share) * p.dk;
    const T* kp = (const T*)p.k.p + b * p.k.batch + (long long)(h / p.k.share) * p.dk;
    const T* gp = (const T*)p.dout.p + b * p.dout.batch + (long long)h * p.dv + v0;
    auto load = [&](int c) {
      const int n = len - c * C;
      const long long t0 = (long long)c * C;
      uint8_t* st = stage(c);
      load_tile<NI, C, DK, kPrep>(st + G::KT, kp + t0 * p.k.step, p.k.step, n, p.dk, tid);
      load_tile<NI, C, DK, kPrep>(st, qp + t0 * p.q.step, p.q.step, n, p.dk, tid);
      load_tile<NI, C, kVB, kPrep>(st + 2 * G::KT, gp + t0 * p.dout.step, p.dout.step, n, p.dv - v0,
                                   tid);
    };
    RawGates<C> raw;
    auto load_raw = [&](int c) {  // (a chunk before the first has no steps)
      load_gates<C>(raw, p.log_decay, p.beta, gate0 + (long long)c * C * p.H, p.H,
                    c < 0 ? 0 : len - c * C, lane);
    };
    auto prep = [&](int c) {
      prepare<NI, DK, kParts, true>(stage(c), stage(c) + G::KT, sm + G::kM + (c & 1) * G::MT,
                                    sm + G::kP + (c & 1) * G::PT, gates[c % 3], scratch, p.scale, tid,
                                    [&] {
                                      scan_gates<C>(gates[(c + 2) % 3], raw, lane);  // (c - 1)
                                      load_raw(c - 2);
                                    });
    };
    if (nc > 0) {
      load(nc - 1);
      copy_commit();
      if (G::NS > 2 && nc > 1) load(nc - 2);
      copy_commit();
      if (warp == 3) {
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
        if (G::NS > 2 ? c > 1 : true) load(G::NS > 2 ? c - 2 : c - 1);
        copy_commit();
        copy_wait<G::NS - 2>();
        bar(1, kPrep);
        prep(c - 1);
      }
      __syncthreads();
    }
  } else {
    const int w0 = (warp - kPrep / 32) * 16;
    const int v = v0 + w0 + (lane >> 2), c2 = (lane & 3) * 2;
    float x[NK][4];  // D
    get_state<NK>(x, p.first ? p.first + unit * p.dv * p.dk : nullptr, v, p.dv, p.dk, lane);
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      const uint32_t Q = smem32(stage(c)), K = Q + G::KT, dO = K + G::KT;
      const uint32_t M = smem32(sm + G::kM + (c & 1) * G::MT), P = smem32(sm + G::kP + (c & 1) * G::PT);
      const Gates<C>& g = gates[c % 3];
      const int n = min(C, len - c * C);
      put_state<NK>(x, hist + (long long)c * p.dv * p.dk, v, p.dv, p.dk, lane);
      float f[NC][4];  // dU^T, then dv^T
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = 0.f;
      state_times<NI, 0, DK, NK, NC>(f, f, x, K, K, lane);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const float2 t = *(const float2*)&g.tail[8 * i + c2];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] *= e & 1 ? t.y : t.x;
      }
      // dO's rows v, steps 16 k ... as a left operand
      auto dout_left = [&](uint32_t (&a)[NI][4], int k) {
#pragma unroll
        for (int q = 0; q < NI; ++q)
          ldm4t(a[q], dO + q * C * kVB * 2 + left_t<kVB * 2>(lane, w0, 16 * k));
      };
      // P^T dO for the steps of block k
      auto from_out = [&](int k) {
#pragma unroll
        for (int i = k; i < NB; ++i) {
          uint32_t a[NI][4], r[kParts][2][2];
          dout_left(a, i);
          load_right_t<G::PB, kParts, 2>(r, P, C * G::PB, lane, 16 * k, 16 * i);
          mma_parts<NI, kParts, 2>(f + 2 * k, a, r);
        }
      };
      // from the last block back: y = dU - X^T beta dU, dv = beta y, and what dv takes
      // off dU of the earlier blocks (the order of issue as in the walk)
      uint32_t av[kParts][4];
      auto rest = [&](int k) {
#pragma unroll
        for (int i = 0; i < 2 * k - 2; i += 2) {
          uint32_t r[kParts][2][2];
          load_right_t<G::PB, kParts, 2>(r, M, C * G::PB, lane, 8 * i, 16 * k);
          mma_parts<kParts, kParts, 2>(f + i, av, r);
        }
      };
      from_out(NB - 1);
#pragma unroll
      for (int k = NB - 1; k >= 0; --k) {
        uint32_t a[kParts][4], r[kParts][2][2];
        float d[2][4], y[2][4];
        load_right<G::PB, kParts, 2>(r, M, C * G::PB, lane, 16 * k, 16 * k);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 be = *(const float2*)&g.beta[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[q][e] = 0.f;
            y[q][e] = f[2 * k + q][e] * (e & 1 ? be.y : be.x);
          }
        }
        as_left<kParts>(a, y[0], y[1]);
        mma_short(d, a, r);
        if (k + 1 < NB) rest(k + 1);
        if (k > 0) from_out(k - 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 be = *(const float2*)&g.beta[16 * k + 8 * q + c2];
          float* yp = ys + (long long)c * C * p.dv;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float yv = f[2 * k + q][e] + d[q][e];
            const int i = 16 * k + 8 * q + c2 + (e & 1), vv = w0 + (lane >> 2) + 8 * (e >> 1);
            if (v0 + vv < p.dv) yp[(long long)i * p.dv + vv] = yv;
            f[2 * k + q][e] = yv * (e & 1 ? be.y : be.x);
          }
        }
        as_left<kParts>(av, f[2 * k], f[2 * k + 1]);
        if (k > 0) {
          load_right_t<G::PB, kParts, 2>(r, M, C * G::PB, lane, 16 * k - 16, 16 * k);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[q][e] = f[2 * k - 2 + q][e];
          mma_short(d, av, r);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[2 * k - 2 + q][e] = d[q][e];
        }
      }
      T* at = out + (long long)c * C * out_step + w0;
#pragma unroll
      for (int i = 0; i < NC; ++i) put_steps<T>(f[i], at, out_step, 8 * i, n, v0 + w0, p.dv, lane);
      uint32_t y[NB][kParts][4];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 l = *(const float2*)&g.lead[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[2 * k + q][e] *= -(e & 1 ? l.y : l.x);
        }
        as_left<kParts>(y[k], f[2 * k], f[2 * k + 1]);
      }
      state_add<NI, DK, NK, NB>(x, g.last, y, K, lane, [](int) {});
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t a[NI][4];
        dout_left(a, k);
        float d[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 l = *(const float2*)&g.lead[16 * k + 8 * q + c2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int w = 2 * q + (e >> 1);
            float s = 0.f;
#pragma unroll
            for (int i = NI - 1; i >= 0; --i)
              s += __uint_as_float(e & 1 ? a[i][w] & 0xffff0000u : a[i][w] << 16);
            d[q][e] = s * p.scale * (e & 1 ? l.y : l.x);
          }
        }
        as_left<kParts>(y[k], d[0], d[1]);
      }
      state_add<NI, DK, NK, NB>(x, 1.f, y, Q, lane, [](int) {});
      __syncthreads();
    }
    if (p.last) put_state<NK>(x, p.last + unit * p.dv * p.dk, v, p.dv, p.dk, lane);
  }
  clear_rows<T>(out, out_step, len, p.T, min(kVB, p.dv - v0), tid, blockDim.x);
}

// CTAs of a walk: four warps that prepare, and one for 16 columns of v.
dim3 walk_grid(int H, int B, int dv) { return dim3(H * ((dv + kVB - 1) / kVB), B); }
int walk_threads(int dv) { return kPrep + 32 * ((min(dv, kVB) + 15) / 16); }

template <int NI, int DK, bool kStates>
cudaError_t walk_t(const DeltaWalk& p, cudaStream_t s) {
  constexpr size_t smem = Geom<NI, DK, kOutParts<NI>>::smem;
  static_assert(smem <= 232448, "");
  const cudaError_t e = cudaFuncSetAttribute(k_delta_walk<NI, DK, kStates>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "delta_states" : "delta_walk", s);
  k_delta_walk<NI, DK, kStates><<<walk_grid(p.H, p.B, p.dv), walk_threads(p.dv), smem, s>>>(p);
  return cudaGetLastError();
}
template <int NI, int DK>
cudaError_t back_t(const DeltaBack& p, cudaStream_t s) {
  constexpr size_t smem = Geom<NI, DK, kParts>::smem;
  static_assert(smem <= 232448, "");
  const cudaError_t e = cudaFuncSetAttribute(k_delta_back<NI, DK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls("delta_back", s);
  k_delta_back<NI, DK><<<walk_grid(p.H, p.B, p.dv), walk_threads(p.dv), smem, s>>>(p);
  return cudaGetLastError();
}

// One token: A = a S, e = v - A k, S' = A + beta e k^T, o = s S' q.  A row of the
// state (dk floats) is held by LPR lanes, four floats each, and a warp takes NR rows
// a lane at once: their loads are in flight together, and their dot products with k
// are added up together (while a lane holds several sums, each exchange halves
// them), as are those with q.  o needs no second pass: S' q = A q + beta e (k . q).
//
// Bound by the states' bytes, read and written once.
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
    if (bf16) return p.dk <= 64 ? walk_t<1, 64, true>(p, s) : walk_t<1, 128, true>(p, s);
    return p.dk <= 64 ? walk_t<3, 64, true>(p, s) : walk_t<3, 128, true>(p, s);
  }
  if (bf16) return p.dk <= 64 ? walk_t<1, 64, false>(p, s) : walk_t<1, 128, false>(p, s);
  return p.dk <= 64 ? walk_t<3, 64, false>(p, s) : walk_t<3, 128, false>(p, s);
}

cudaError_t delta_back(const DeltaBack& p, bool bf16, cudaStream_t s) {
  if (bf16) return p.dk <= 64 ? back_t<1, 64>(p, s) : back_t<1, 128>(p, s);
  return p.dk <= 64 ? back_t<3, 64>(p, s) : back_t<3, 128>(p, s);
}

cudaError_t delta_step(const DeltaStep& p, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

int delta_chunk(bool bf16) { return bf16 ? kSteps<1> : kSteps<3>; }

}  // namespace ssd
