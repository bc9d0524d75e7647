// Gated delta rule: the gradients of q, k, the decays and the write strengths of
// every chunk, from the state H before it, the gradient D of the state after it, E
// and y (ssd_delta.cuh, ssd_delta.cu have the formulas), no chunk waiting for
// another.  With dv = beta y, U = beta E, (Q K^T) and (K K^T) the plain scores,
//   MP_ij = s Gamma_ij dO_i . U_j (j <= i),  ML_ij = -Gamma_ij dv_i . U_j (j < i)
//   dq = a + MP K,      a = s e^g dO H
//   dk = r + w,         r = b + ML K, b = -e^g dv H,  w = MP^T Q + ML^T K + c, c = e^{G-g} U D
//   dbeta_i = E_i . y_i
// A step's log decay acts on everything that is written before it and read from it on:
// with m_ij = MP_ij (q_i . k_j) + ML_ij (k_i . k_j), what a pair of steps contributes,
//   dlog_decay_t = sum_{i >= t > j} m_ij + sum_{i >= t} (q_i . a_i + k_i . b_i)
//                + sum_{j < t} k_j . c_j + e^G <H, D>
// found as the sums from the chunk's end of rows minus columns of m and so on, in two floats.  (Rows
// and columns are sums of the same m_ij, whose errors then cancel like the pairs within
// [t, C) do.  With q . dq - k . w in their place, from products of their own, what
// should cancel was thirty times the result.)
//
// One persistent CTA an SM walks over (chunk, head, row); a warp has 16 rows (steps) and
// a share of the columns, operands come 64 columns of v at a time and are split into
// parts in the place where they arrive.  H and D of the next piece are on their way
// while this one is multiplied, E, y and dO of the next chunk while MP and ML are; K and
// Q come during the first products, which need neither.  Heads that share q and k
// write their own gradients in fp32, summed in head order by a second kernel.
//
// Scales.  With rows of dO, dv, U, q and k in [1, 2) times a power of two each, the tiles
// of MP and ML hold Gamma_ij times the products of such rows: at most 2^9, whatever the
// rows' powers are.  The power of the output's row is multiplied in at the end; the other
// one goes by the share that a step has in the sum (what it writes, U_j k_j, for dq and
// dk's first part; what it reads, dO_i q_i or dv_i k_i, for its second) and is multiplied
// into the right operand's rows, relative to the chunk's largest share.  So a step's dq
// does not depend on the size of its q, nor dk on that of k.
//
// 4 x 2048 steps of 32 heads 128/64 (bf16): 432 us for 4096 items of 30 thousand cycles,
// where the 709 MB it reads and writes take 106 (events around the kernel, caches flushed;
// tensor pipe 26 % and issue slots 43 % busy).  Of an item the splitting takes 6 thousand
// cycles, the products with H and D 6 (tensor pipe and shared memory), the scores and masks
// 4, the products with MP and ML 7, loads and barriers the rest.  MP and ML as one part
// each: 24 us less, and dq and dk off by 2^-11 of their size; held in q's and k's scales: 20
// less, and steps of short q and k without their bits.  When it took 423 us, two CTAs an SM
// with half the columns each took 510, since both take E, y and dO apart, and one CTA an
// item instead of persistent ones 543.
#include <cuda_bf16.h>

#include "persistent_grid.h"
#include "ssd_delta.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace delta;

template <int NI, int DK>
struct Geom {
  static constexpr int C = kSteps<NI>, NT = C * 8;       // threads
  static constexpr int RB = DK * 2, VR = kVB * 2, PB = C * 2;
  static constexpr int KT = NI * C * RB;                 // Q, K
  static constexpr int OT = NI * C * VR;                 // dO
  static constexpr int HT = kParts * kVB * RB;           // H, D
  static constexpr int UT = kParts * C * VR;             // U, dv
  static constexpr int MT = kParts * C * PB;     // MP, ML: in the place of H, D
  static_assert(MT <= HT, "");
  static constexpr int kK = KT, kO = 2 * KT, kU = kO + OT, kV = kU + UT, kH = kV + UT;
  static constexpr size_t smem = kH + 4 * HT;            // H, D; the next ones
  static constexpr int WR = C / 16, WC = 4;              // strips of rows, groups of columns
  static constexpr int NK = DK / 8 / WC;                 // eights of columns of dq, dk of a warp
  static constexpr int NM = C / 16;                      // of MP or ML
  static_assert(WR * WC * 32 == NT && NK % 2 == 0 && NM % 2 == 0, "");
};

// a row-major tile's two elements at `at`
template <int NI, int RB, int C>
__device__ __forceinline__ float2 pair_at(const uint8_t* at) {
  float2 f = unpack_half(*(const uint32_t*)at);
  if (NI == 2) f = add2(f, unpack_half(*(const uint32_t*)(at + C * RB)));
  return f;
}
template <typename T>
__device__ __forceinline__ void put_pair(T* at, float2 x) {
  if constexpr (sizeof(T) == 2) *(uint32_t*)at = pack_bf(x.x, x.y);
  else *(float2*)at = x;
}
template <int N>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// the power of two below |x| (1 for zero, infinities and NaN)
__device__ __forceinline__ float pow2_of(float x) {
  const uint32_t e = __float_as_uint(x) & 0x7f800000u;
  return e == 0 || e == 0x7f800000u ? 1.f : __uint_as_float(e);
}
// a right operand's terms 2 t, 2 t + 1 times lo, those at + 8 times hi
template <int NI>
__device__ __forceinline__ void times_terms(uint32_t (&r)[NI][2][2], const uint32_t (&b)[NI][2][2],
                                            __half2 lo, __half2 hi) {
#pragma unroll
  for (int q = 0; q < NI; ++q)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2 x = __hmul2(*(const __half2*)&b[q][n][e], e ? hi : lo);
        r[q][n][e] = *(const uint32_t*)&x;
      }
}
// the largest of x >= 0 over a warp and *top, whose bits are in the order of the values
__device__ __forceinline__ void max_of_all(uint32_t* top, float x, int lane) {
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
  if (lane == 0) atomicMax(top, m);
}

// kShared: dq, dk of the head in fp32 to part (dq's, then dk's, [B][T][H][dk])
template <int NI, int DK, bool kShared>
__global__ void __launch_bounds__(Geom<NI, DK>::NT, 1) k_delta_grads(const DeltaGrads p, float* part,
                                                                    uint32_t items) {
  using G = Geom<NI, DK>;
  using T = typename std::conditional<NI == 1, __nv_bfloat16, float>::type;
  using TO = typename std::conditional<kShared, float, T>::type;
  constexpr int C = G::C, NT = G::NT, NW = NT / 32, RB = G::RB, VR = G::VR, PB = G::PB, NK = G::NK,
                NM = G::NM, NB = C / 16;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ Gates<C> gates[2];
  // Of the steps: the largest of U, dv and dO and what they were divided by (of this
  // piece and the one before), what q and k were; dbeta; sums over columns and rows.
  __shared__ float most[2][3][C], down[2][3][C], qdown[C], kdown[C], dbeta[C];
  __shared__ float rows_of[G::WC][C], cols_of[2][G::WR][C], reads[G::WC][C], writes[G::WC][C];
  __shared__ float hdots[NW];
  // the bits of the largest of H and D
  __shared__ __align__(8) uint32_t top_state[2][2];
  // the largest of the steps' q and k; their shares (written; read by q and by k), as
  // powers of two of at most 1, and what these were divided by
  __shared__ float qmost[C], kmost[C], share_down[2];
  __shared__ __align__(4) __half share[3][C];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // (the warps of a sub-core, four apart, have different strips: the later ones have more
  // of MP and ML)
  const int strip = (warp + warp / 4) % G::WR, group = warp / G::WR;
  const bool is_l = group >= 2;   // this warp's scores: ML's, else MP's
  const int m0 = (group & 1) * NM;  // their first eight of columns
  const uint32_t sQ = smem32(sm), sK = sQ + G::kK, sO = sQ + G::kO, sU = sQ + G::kU, sV = sQ + G::kV;
  const Lane<RB> lk(lane);
  const Lane<VR> lv(lane);
  const Lane<PB> lm(lane);
  const int chunks = (p.T + C - 1) / C, vblocks = (p.dv + kVB - 1) / kVB;
  const long long out_step = (long long)(kShared ? p.H : p.G) * p.dk;

  struct Item {
    int b, h, t0, n, rows;  // n: steps, `rows` up to T
    long long unit;
  };
  auto item_of = [&](uint32_t i) {
    Item x;
    const uint32_t bh = i / (uint32_t)chunks, c = i - bh * chunks;
    x.b = (int)(bh / (uint32_t)p.H);
    x.h = (int)(bh - x.b * p.H);
    x.t0 = (int)c * C;
    int len = p.T;
    if (p.lens) len = min(max(p.lens[x.b], 0), p.T);
    x.n = min(C, len - x.t0);
    x.rows = min(C, p.T - x.t0);
    x.unit = i;
    return x;
  };
  auto load_state = [&](const Item& x, int vb, int buf) {
    const int v0 = vb * kVB, width = p.dv - v0;
    const long long at = (x.unit * p.dv + v0) * p.dk;
    uint8_t* to = sm + G::kH + buf * 2 * G::HT;
    load_tile<kVB, DK, NT>(to, p.hist_s + at, p.dk, width, p.dk, tid);
    load_tile<kVB, DK, NT>(to + G::HT, p.hist_d + at, p.dk, width, p.dk, tid);
  };
  auto load_steps = [&](const Item& x, int vb) {
    const int v0 = vb * kVB, width = p.dv - v0;
    const long long at = x.unit * C * p.dv + v0;
    load_tile<C, kVB, NT>(sm + G::kU, p.err + at, p.dv, C, width, tid);
    load_tile<C, kVB, NT>(sm + G::kV, p.y + at, p.dv, C, width, tid);
    load_tile<C, kVB, NT>(sm + G::kO,
                          (const T*)p.dout.p + x.b * p.dout.batch + x.t0 * p.dout.step + (long long)x.h * p.dv + v0,
                          p.dout.step, x.n, width, tid);
  };
  auto next_of = [&](uint32_t i, Item& x) {  // the first item with steps from i on
    for (; i < items; i += gridDim.x) {
      x = item_of(i);
      if (x.n > 0) break;
    }
    return i;
  };

  // past the rows' ends: zeros, and nothing else to do
  for (uint32_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item x = item_of(i);
    const int z0 = max(x.n, 0);
    if (z0 >= x.rows) continue;
    const long long token = (long long)x.b * p.T + x.t0;
    TO* dq_out = (kShared ? (TO*)part : (TO*)p.dq) + token * out_step + (long long)x.h * p.dk;
    TO* dk_out = (kShared ? (TO*)(part + (long long)p.B * p.T * p.H * p.dk) : (TO*)p.dk_out) +
                 token * out_step + (long long)x.h * p.dk;
    for (int e = tid; e < (x.rows - z0) * (p.dk / 8); e += NT) {
      const int r = z0 + e / (p.dk / 8), c = e % (p.dk / 8) * 8;
#pragma unroll
      for (int k = 0; k < 8; k += 16 / (int)sizeof(TO)) {
        *(uint4*)(dq_out + r * out_step + c + k) = make_uint4(0, 0, 0, 0);
        *(uint4*)(dk_out + r * out_step + c + k) = make_uint4(0, 0, 0, 0);
      }
    }
    for (int r = z0 + tid; r < x.rows; r += NT)
      p.dlog_decay[(token + r) * p.H + x.h] = p.dbeta[(token + r) * p.H + x.h] = 0.f;
  }

  if (tid < 2) top_state[0][tid] = top_state[1][tid] = 0;
  // scale: a power of two and a factor of at most 2
  const float s2 = pow2_of(p.scale), s1 = p.scale / s2;
  Item x, nx;
  nx.n = 0;
  uint32_t i = next_of(blockIdx.x, x);
  int buf = 0, turn = 0;
  RawGates<C> raw;  // warp 1: the next item's gates
  auto load_raw = [&](const Item& x) {
    load_gates<C>(raw, p.log_decay, p.beta, ((long long)x.b * p.T + x.t0) * p.H + x.h, p.H, x.n, lane);
  };
  if (i < items) {
    load_state(x, 0, 0);
    load_steps(x, 0);
    copy_commit();
    if (warp == 1) {
      load_raw(x);
      scan_gates<C>(gates[0], raw, lane);
    }
  }
  while (i < items) {
    const uint32_t in = next_of(i + gridDim.x, nx);
    const long long token = (long long)x.b * p.T + x.t0;
    const T* qp = (const T*)p.q.p + x.b * p.q.batch + x.t0 * p.q.step + (long long)(x.h / p.q.share) * p.dk;
    const T* kp = (const T*)p.k.p + x.b * p.k.batch + x.t0 * p.k.step + (long long)(x.h / p.k.share) * p.dk;
    load_tile<C, DK, NT>(sm, qp, p.q.step, x.n, p.dk, tid);
    load_tile<C, DK, NT>(sm + G::kK, kp, p.k.step, x.n, p.dk, tid);
    copy_commit();
    const Gates<C>& g = gates[turn];
    if (tid < C) dbeta[tid] = 0.f;
    float dq[NK][4], rd[NK][4], wr[NK][4], mm[NM][4];
    zero(dq);
    zero(rd);
    zero(wr);
    zero(mm);
    float hdot = 0.f;  // <H, D>
    // H's and D's divisors, this lane's largest elements
    float hs = 0.f, ds = 0.f, mh = 0.f, md = 0.f;
    const int i0 = 16 * strip + (lane >> 2), c2 = (lane & 3) * 2;
#pragma unroll 1
    for (int vb = 0; vb < vblocks; ++vb) {
      const int width = min(kVB, p.dv - vb * kVB), now = vb & 1;
      uint8_t* Ht = sm + G::kH + buf * 2 * G::HT;
      if (vb == 0) {
        copy_wait<1>();  // (all but K and Q)
      } else {
        __syncthreads();
        load_steps(x, vb);
        copy_commit();
        copy_wait<0>();
      }
      __syncthreads();
      // the pieces into parts, in their place
      const float hs0 = hs, ds0 = ds;
      {
        FloatRows<kVB, DK, NT> fh, fd;
        FloatRows<C, kVB, NT> fe, fy;
        typename std::conditional<NI == 1, HalfRows<C, kVB, NT>, FloatRows<C, kVB, NT>>::type fo;
        fh.read(Ht, tid);
        fd.read(Ht + G::HT, tid);
        fe.read(sm + G::kU, tid);
        fy.read(sm + G::kV, tid);
        fo.read(sm + G::kO, tid);
        // (later pieces are not scaled up by more than the earlier ones, rows of zeros by the
        // most there is, so that sums of these may be scaled to them by factors of at most 1)
#pragma unroll
        for (int k = 0; k < fh.N; ++k) {
          const float4 s = fh.f[k], d = fd.f[k];
          mh = max3_abs(max3_abs(mh, s.x, s.y), s.z, s.w);
          md = max3_abs(max3_abs(md, d.x, d.y), d.z, d.w);
          hdot = fmaf(s.x, d.x, fmaf(s.y, d.y, fmaf(s.z, d.z, fmaf(s.w, d.w, hdot))));
        }
        max_of_all(&top_state[buf][0], mh, lane);
        max_of_all(&top_state[buf][1], md, lane);
#pragma unroll
        for (int k = 0; k < fe.N; ++k) {
          const int at = k * NT + tid, r = at / fe.LPR;
          float4 &e = fe.f[k], &y = fy.f[k];
          const float d = sum_lanes<fe.LPR>(fmaf(e.x, y.x, fmaf(e.y, y.y, fmaf(e.z, y.z, e.w * y.w))));
          if (at % fe.LPR == 0) dbeta[r] += d;
          const float be = g.beta[r];
          e.x *= be; e.y *= be; e.z *= be; e.w *= be;
          y.x *= be; y.y *= be; y.z *= be; y.w *= be;
        }
        __syncthreads();
        const uint2 top = *(const uint2*)top_state[buf];
        // (their products are with U, dv and dO, which have kLift of their own)
        const Scale sh = scale_to<kLift, kLift>(__uint_as_float(top.x)),
                    sd = scale_to<kLift, kLift>(__uint_as_float(top.y));
        hs = sh.down;
        ds = sd.down;
#pragma unroll
        for (int k = 0; k < fh.N; ++k) {
          fh.put(Ht, k, sh.up, tid);
          fd.put(Ht + G::HT, k, sd.up, tid);
        }
        auto least = [&](int which) {
          return [=](int r) { return vb ? most[now ^ 1][which][r] : 0.f; };
        };
        auto done = [&](int which) {
          return [=](int r, float s, float m) {
            most[now][which][r] = m;
            down[now][which][r] = inverse_pow2(s);
          };
        };
        fe.template write<kFarStep>(sm + G::kU, tid, least(0), done(0));
        fy.template write<kFarStep>(sm + G::kV, tid, least(1), done(1));
        fo.template write<kFarStep>(sm + G::kO, tid, least(2), done(2));
      }
      __syncthreads();
      if (tid < 2) top_state[buf][tid] = 0;  // (all have read it)
      if (vb + 1 < vblocks) load_state(x, vb + 1, buf ^ 1);
      else if (in < items) load_state(nx, 0, buf ^ 1);
      copy_commit();
      if (vb > 0) {
        const float fh = hs0 / hs, fd = ds0 / ds;
        const auto ratio = [&](int which, int r) { return down[now ^ 1][which][r] / down[now][which][r]; };
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = i0 + 8 * u;
          const float fu = ratio(0, r), fv = ratio(1, r), fo = ratio(2, r);
#pragma unroll
          for (int e = 0; e < NK; ++e) {
            set_pair(dq[e], u, mul2(pair(dq[e], u), both(fo * fh)));
            set_pair(rd[e], u, mul2(pair(rd[e], u), both(fv * fh)));
            set_pair(wr[e], u, mul2(pair(wr[e], u), both(fu * fd)));
          }
#pragma unroll
          for (int e = 0; e < NM; ++e) {
            const int c = 8 * (m0 + e) + c2;
            const float f = is_l ? fv : fo;
            set_pair(mm[e], u, mul2(pair(mm[e], u), make_float2(f * ratio(0, c), f * ratio(0, c + 1))));
          }
        }
      }
      const uint32_t sH = smem32(Ht), sD = sH + G::HT;
#pragma unroll 2
      for (int k = 0; k < width; k += 16) {
        uint32_t ao[NI][4], au[kParts][4], av[kParts][4];
#pragma unroll
        for (int q = 0; q < NI; ++q) ldm4(ao[q], lv.left(sO, 16 * strip, k) + q * C * VR);
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          ldm4(au[q], lv.left(sU, 16 * strip, k) + q * C * VR);
          ldm4(av[q], lv.left(sV, 16 * strip, k) + q * C * VR);
        }
#pragma unroll
        for (int e = 0; e < NK; e += 2) {
          const int c = (group * NK + e) * 8;
          uint32_t r[kParts][2][2];
          load_right_t<kParts, 2>(r, sH, kVB * RB, lk, c, k);
          mma_parts<NI, kParts, 2>(dq + e, ao, r);
          mma_parts<kParts, kParts, 2>(rd + e, av, r);
          load_right_t<kParts, 2>(r, sD, kVB * RB, lk, c, k);
          mma_parts<kParts, kParts, 2>(wr + e, au, r);
        }
#pragma unroll
        for (int e = 0; e < NM; e += 2)
          if (m0 + e <= 2 * strip) {
            uint32_t r[kParts][2][2];
            load_right<kParts, 2>(r, sU, C * VR, lv, 8 * (m0 + e), k);
            if (is_l) mma_parts<kParts, kParts, 2>(mm + e, av, r);
            else mma_parts<NI, kParts, 2>(mm + e, ao, r);
          }
      }
      buf ^= 1;
    }
    copy_wait<1>();  // K and Q (not the next H and D)
    __syncthreads();
    if (in < items) {
      load_steps(nx, 0);
      if (warp == 1) load_raw(nx);
    }
    copy_commit();
    {
      auto q_done = [&](int r, float s, float m) {
        qdown[r] = inverse_pow2(s) * pow2(-kLift);
        qmost[r] = m;
      };
      auto k_done = [&](int r, float s, float m) {
        kdown[r] = inverse_pow2(s) * pow2(-kLift);
        kmost[r] = m;
      };
      if constexpr (NI == 2) {
        FloatRows<C, DK, NT> q, k;
        q.read(sm, tid);
        k.read(sm + G::kK, tid);
        __syncthreads();
        q.template write<kFarStep>(sm, tid, no_least, q_done);
        k.template write<kFarKey>(sm + G::kK, tid, no_least, k_done);
      } else {
        HalfRows<C, DK, NT> q, k;
        q.read(sm, tid);
        k.read(sm + G::kK, tid);
        q.template write<kFarStep>(sm, tid, no_least, q_done);
        k.template write<kFarKey>(sm + G::kK, tid, no_least, k_done);
      }
    }
    __syncthreads();
    const int last = (vblocks - 1) & 1;
    const float *udown = down[last][0], *vdown = down[last][1], *odown = down[last][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = i0 + 8 * u;
      const float fq = p.scale * g.lead[r] * odown[r], fr = -g.lead[r] * vdown[r],
                  fw = g.tail[r] * udown[r];
      float2 read_q = both(0.f), read_k = both(0.f), write2 = both(0.f);
      // (a row's pieces: their index exchanged by r's last bits)
      const uint8_t* row = sm + r * RB + c2 * 2;
#pragma unroll
      for (int e = 0; e < NK; ++e) {
        const uint8_t* at = row + (((group * NK + e) ^ (r & 7)) << 4);
        const float2 q = pair_at<NI, RB, C>(at), k = pair_at<NI, RB, C>(at + G::kK);
        // (the state's factor first: the product of both may be below what fp32 holds)
        const float2 a = mul2(mul2(pair(dq[e], u), both(hs)), both(fq)),
                     b = mul2(mul2(pair(rd[e], u), both(hs)), both(fr)),
                     w = mul2(mul2(pair(wr[e], u), both(ds)), both(fw));
        set_pair(dq[e], u, a);
        set_pair(rd[e], u, b);
        set_pair(wr[e], u, w);
        read_q = fma2(q, a, read_q);
        read_k = fma2(k, b, read_k);
        write2 = fma2(k, w, write2);
      }
      const float s = sum_lanes<4>((read_q.x + read_q.y) * qdown[r] + (read_k.x + read_k.y) * kdown[r]);
      const float write = sum_lanes<4>((write2.x + write2.y) * kdown[r]);
      if ((lane & 3) == 0) {
        reads[group][r] = s;
        writes[group][r] = write;
      }
    }
    uint8_t* Mt = sm + G::kH + (buf ^ 1) * 2 * G::HT;  // the last piece's H and D
    if (group == 1 && strip == 0) {  // (a warp without columns of MP)
      float w[C / 32], rq[C / 32], rk[C / 32], top_w = 0.f, top_r = 0.f;
#pragma unroll
      for (int k = 0; k < C / 32; ++k) {
        const int r = k * 32 + lane;
        const bool uu = most[last][0][r] > 0.f, vv = most[last][1][r] > 0.f, oo = most[last][2][r] > 0.f;
        const bool kk = kmost[r] > 0.f, qq = qmost[r] > 0.f;
        w[k] = uu && kk ? udown[r] * kdown[r] : 0.f;
        rq[k] = oo && qq ? s2 * odown[r] * qdown[r] : 0.f;
        rk[k] = vv && kk ? vdown[r] * kdown[r] : 0.f;
        top_w = fmaxf(top_w, w[k]);
        top_r = fmaxf(top_r, fmaxf(rq[k], rk[k]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        top_w = fmaxf(top_w, __shfl_xor_sync(0xffffffffu, top_w, o));
        top_r = fmaxf(top_r, __shfl_xor_sync(0xffffffffu, top_r, o));
      }
      // (the quotient of two powers of two; of zero there is no share)
      const auto part_of = [](float x, float top) { return __float2half_rn(top > 0.f ? x / top : 0.f); };
#pragma unroll
      for (int k = 0; k < C / 32; ++k) {
        const int r = k * 32 + lane;
        share[0][r] = part_of(w[k], top_w);
        share[1][r] = part_of(rq[k], top_r);
        share[2][r] = part_of(rk[k], top_r);
      }
      if (lane == 0) {
        share_down[0] = top_w;
        share_down[1] = top_r;
      }
    }
    // MP or ML as their tiles hold them (times 2^kMask), and the products with the scores
    constexpr int kMask = 5;
    constexpr float kMaskDown = pow2(-kMask);
    {
      const uint32_t A = is_l ? sK : sQ;
      uint8_t* tile = Mt + (is_l ? G::HT : 0);
      const float held = (is_l ? -1.f : s1) * pow2(kMask - 2 * kLift);  // (the operands' factors off)
      float row[2] = {0.f, 0.f}, f[2], hi[2], lo[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + 8 * u;
        f[u] = (is_l ? vdown[i] * kdown[i] : s2 * odown[i] * qdown[i]) * kMaskDown;
        hi[u] = g.hi[i];
        lo[u] = g.lo[i];
      }
#pragma unroll
      for (int e = 0; e < NM; e += 2) {
        float s[2][4];
        zero(s);
        if (m0 + e <= 2 * strip) {
#pragma unroll 2
          for (int k = 0; k < DK; k += 16) {
            uint32_t a[NI][4], r[NI][2][2];
#pragma unroll
            for (int q = 0; q < NI; ++q) ldm4(a[q], lk.left(A, 16 * strip, k) + q * C * RB);
            load_right<NI, 2>(r, sK, C * RB, lk, 8 * (m0 + e), k);
            mma_parts<NI, NI, 2>(s, a, r);
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int j = 8 * (m0 + e + q) + c2;
          float (&m)[4] = mm[e + q];
          float2 col = make_float2(0.f, 0.f);
          if (m0 + e <= 2 * strip) {
            const float2 hj = *(const float2*)&g.hi[j], lj = *(const float2*)&g.lo[j];
            const float2 fj = mul2(*(const float2*)&udown[j], *(const float2*)&kdown[j]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int i = i0 + 8 * u;
              const float2 minus = both(-1.f);
              const float2 t = add2(fma2(hj, minus, both(hi[u])), fma2(lj, minus, both(lo[u])));
              float2 v = mul2(mul2(pair(m, u), both(held)), make_float2(exp2_fast(t.x), exp2_fast(t.y)));
              if (m0 + e == 2 * strip) {  // (the diagonal's columns)
                const int above = is_l ? 1 : 0;
                if (j + above > i) v.x = 0.f;
                if (j + 1 + above > i) v.y = 0.f;
              }
              uint32_t a[kParts];
              split2<kParts>(v, a);
              uint8_t* at = tile + at16<PB>(i, m0 + e + q) + c2 * 2;
#pragma unroll
              for (int w = 0; w < kParts; ++w) *(uint32_t*)(at + w * C * PB) = a[w];
              const float2 c = mul2(mul2(v, both(f[u])), mul2(fj, pair(s[q], u)));
              row[u] += c.x + c.y;
              col = add2(col, c);
            }
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            col.x += __shfl_xor_sync(0xffffffffu, col.x, d);
            col.y += __shfl_xor_sync(0xffffffffu, col.y, d);
          }
          if (lane < 4) *(float2*)&cols_of[is_l][strip][j] = col;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        row[u] = sum_lanes<4>(row[u]);
        if ((lane & 3) == 0) rows_of[group][i0 + 8 * u] = row[u];
      }
    }
    hdot = sum_lanes<32>(hdot);
    if (lane == 0) hdots[warp] = hdot;
    __syncthreads();
    if (warp == 0) {
      // dg, and its sums from each step to the end, in two floats
      constexpr int N = C / 32;
      Two d[N], total = {0.f, 0.f};
      float tails = 0.f, hd = 0.f;
      for (int k = lane; k < NW; k += 32) hd += hdots[k];
      hd = sum_lanes<32>(hd);
#pragma unroll
      for (int k = N - 1; k >= 0; --k) {
        const int r = lane * N + k;
        float w = 0.f;
#pragma unroll
        for (int c = 0; c < G::WC; ++c) {
          put_in(total, rows_of[c][r]);
          put_in(total, reads[c][r]);
          w += writes[c][r];
        }
#pragma unroll
        for (int c = 0; c < G::WR; ++c) {
          put_in(total, -cols_of[0][c][r]);
          put_in(total, -cols_of[1][c][r]);
        }
        tails += w;
        put_in(total, -w);
        d[k] = total;
      }
      tails = sum_lanes<32>(tails);
      Two after = total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two y = {__shfl_down_sync(0xffffffffu, after.hi, o), __shfl_down_sync(0xffffffffu, after.lo, o)};
        if (lane + o < 32) after = add(after, y);
      }
      after = {__shfl_down_sync(0xffffffffu, after.hi, 1), __shfl_down_sync(0xffffffffu, after.lo, 1)};
      if (lane == 31) after = {0.f, 0.f};
      after = add(after, {fmaf(g.last, hd, tails), 0.f});
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int r = lane * N + k;
        const Two t = add(d[k], after);
        if (r < x.n) p.dlog_decay[(token + r) * p.H + x.h] = t.hi + t.lo;
      }
    }
    if (warp == 1 && in < items) scan_gates<C>(gates[turn ^ 1], raw, lane);
    if (tid < x.n) p.dbeta[(token + tid) * p.H + x.h] = dbeta[tid];
    // the products with MP and ML, and the results
    TO* dq_out = (kShared ? (TO*)part : (TO*)p.dq) + token * out_step + (long long)x.h * p.dk;
    TO* dk_out = (kShared ? (TO*)(part + (long long)p.B * p.T * p.H * p.dk) : (TO*)p.dk_out) +
                 token * out_step + (long long)x.h * p.dk;
    const uint32_t sP = smem32(Mt), sL = sP + G::HT;
    // of the rows of MP K, ML K and of the sum of MP^T Q and ML^T K
    float up_q[2], up_r[2], up_w[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = i0 + 8 * u;
      up_q[u] = s2 * odown[r] * (share_down[0] * kMaskDown);
      up_r[u] = vdown[r] * (share_down[0] * kMaskDown);
      up_w[u] = udown[r] * (share_down[1] * kMaskDown);
    }
    // the shares of steps 16 k + 2 t, 16 k + 2 t + 1 and those at + 8
    const auto share_of = [&](int which, int at) { return *(const __half2*)&share[which][at + c2]; };
#pragma unroll
    for (int e = 0; e < NK; e += 2) {
      const int c = (group * NK + e) * 8;
      float d[3][2][4];
      zero(d[0]);
      zero(d[1]);
      zero(d[2]);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t a[kParts][4], rk[NI][2][2];
        load_right_t<NI, 2>(rk, sK, C * RB, lk, c, 16 * k);
        if (k <= strip) {  // columns 16 k ... of MP, ML
#pragma unroll
          for (int q = 0; q < kParts; ++q) ldm4(a[q], lm.left(sP, 16 * strip, 16 * k) + q * C * PB);
          uint32_t rw[NI][2][2];
          times_terms<NI>(rw, rk, share_of(0, 16 * k), share_of(0, 16 * k + 8));
          mma_parts<kParts, NI, 2>(d[0], a, rw);
#pragma unroll
          for (int q = 0; q < kParts; ++q) ldm4(a[q], lm.left(sL, 16 * strip, 16 * k) + q * C * PB);
          mma_parts<kParts, NI, 2>(d[1], a, rw);
        }
        if (k >= strip) {  // rows 16 k ...
          uint32_t rq[NI][2][2];
          load_right_t<NI, 2>(rq, sQ, C * RB, lk, c, 16 * k);
#pragma unroll
          for (int q = 0; q < kParts; ++q) ldm4t(a[q], lm.left_t(sP, 16 * strip, 16 * k) + q * C * PB);
          times_terms<NI>(rq, rq, share_of(1, 16 * k), share_of(1, 16 * k + 8));
          mma_parts<kParts, NI, 2>(d[2], a, rq);
#pragma unroll
          for (int q = 0; q < kParts; ++q) ldm4t(a[q], lm.left_t(sL, 16 * strip, 16 * k) + q * C * PB);
          times_terms<NI>(rk, rk, share_of(2, 16 * k), share_of(2, 16 * k + 8));
          mma_parts<kParts, NI, 2>(d[2], a, rk);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = i0 + 8 * u, cc = c + 8 * q + c2;
          if (r < x.n && cc < p.dk) {
            put_pair(dq_out + r * out_step + cc,
                     fma2(pair(d[0][q], u), both(up_q[u]), pair(dq[e + q], u)));
            const float2 dk = fma2(pair(d[1][q], u), both(up_r[u]),
                                   fma2(pair(d[2][q], u), both(up_w[u]),
                                        add2(pair(rd[e + q], u), pair(wr[e + q], u))));
            put_pair(dk_out + r * out_step + cc, dk);
          }
        }
    }
    __syncthreads();
    x = nx;
    i = in;
    turn ^= 1;
  }
  copy_wait<0>();
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
    put_pair(to, make_float2(s.x, s.y));
    put_pair(to + 2, make_float2(s.z, s.w));
  }
}

template <int NI, int DK, bool kShared>
cudaError_t grads_s(const DeltaGrads& p, float* part, cudaStream_t s) {
  using G = Geom<NI, DK>;
  static_assert(G::smem + 16384 <= 232448, "");
  // (B T H is at most 4e10, and an item 32 steps or more)
  const long long items = (long long)p.B * p.H * ((p.T + G::C - 1) / G::C);
  int grid = 1;
  static FitOf fit;
  const cudaError_t e = persistent_grid(k_delta_grads<NI, DK, kShared>, G::NT, G::smem, items, 1 << 16,
                                        &fit, &grid);
  if (e != cudaSuccess) return e;
  LaunchScope ls("delta_grads", s);
  k_delta_grads<NI, DK, kShared><<<grid, G::NT, G::smem, s>>>(p, part, (uint32_t)items);
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
  return p.dk <= 64 ? grads_t<2, 64>(p, part, s) : grads_t<2, 128>(p, part, s);
}

}  // namespace ssd
