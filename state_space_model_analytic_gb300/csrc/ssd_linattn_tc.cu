// Tensor-core walk of linear attention with a decay for each head (bf16
// operands, fp32 state): the forward and, with exchanged roles, the gradients
// (the formulas stand in ssd_linattn.cu).
//
// Chunks of 128 steps, one CTA per (head, row, segment of the row).  Per chunk,
// with w_j the decay from step j to the chunk's end and X the state before it
// ([dk][dv], rows k),
//   S  = Q K^T              128 x 128, masked and decayed into P (bf16, TMEM)
//   O  = P V                A from TMEM
//   Oc = Q X                X in bf16; o = O + lead_i Oc
//   U  = K^T (w o V)        X <- a^n X + U, X in fp32 registers
// All accumulators are in TMEM (512 columns, one CTA per SM).
//
// Precision.  P is rounded to bf16 once (the scores are the A operand of the
// second product) and X once as an operand; the output is bf16 itself.  The
// state is an fp32 result, so w o V is carried as three bf16 parts (hi, mid,
// lo: 24 bits) and U is three products; the one of V and K that is narrower is
// scaled.
//
// Bound by memory: a chunk moves dk, dk, dv, dv columns of 128 rows once, at
// 45 GB/s an SM some 4100 cycles for dk = 128, dv = 64, against 1800 cycles of
// products.  The work is split over warps so that these overlap with the
// loads: warps 0-3 turn S into P and write o (thread = row), warps 4-7 build
// the parts of w o V and carry X (thread = row k), one thread issues the TMA
// loads of the next chunks, one the products.
//
// Rows past the end of a batch row (its length, or T) take part as zeros: TMA
// fills what lies past T; between a shorter row's end and T warps 0-3 clear
// the tile's rows before any product reads them.
#include <cuda.h>
#include <cuda_bf16.h>

#include <mutex>

#include "f32x2.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"
#include "tc_util.cuh"

namespace ssd {

using namespace tc;

namespace {

constexpr int kQ = 128;
constexpr int kThreads = 320;  // 4 + 4 warps, the loader and the issuer
constexpr uint64_t kWaitNs = 1000000000ull;

__device__ unsigned int g_la_error;

struct Maps {
  CUtensorMap q, k, v, o;
};

struct TcWalk {
  int B, T, H, dk, dv;
  int qs, ks, vs;  // heads that share an operand's head
  int nseg, seg_chunks;
  const float* log_decay;
  const float* first;  // state before the row (nseg == 1) or before each segment
  float* last;         // state after it; after each segment alone in a states walk
  int first_swapped;
  const int* lens;
  void* o;
  int o_f32;
  float s_intra, s_carry, s_inject;
  int off, reverse;
};

// ---- PTX that only this file uses ----------------------------------------------

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int c0, int c1, int c2,
                                            int c3, uint64_t* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(mbar))
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const void* tmap, const void* src, int c0, int c1,
                                             int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          tmap),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(src))
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: A's row i is lane i, two bf16 a column
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 16 columns of 32 bits from registers
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ float decay_pow(float la, float e) { return e == 0.f ? 1.f : expf(la * e); }

// ---- shared memory -----------------------------------------------------------------

// NS: stages of the loads; WH: buffers of half a chunk's scaled parts.  The
// sums stay below the 227 KB of a CTA.
template <int DK, int DV>
struct Geom {
  static constexpr bool scale_k = DK < DV;
  static constexpr int DS = scale_k ? DK : DV;  // width of the scaled operand
  static constexpr int NS = DK + DV == 256 ? 1 : 2;
  static constexpr int WH = DS == 64 && DK + DV != 192 ? 2 : DK < DV ? 2 : 1;
  static constexpr int QT = DK * 256, VT = DV * 256;  // bytes of 128 rows
  static constexpr int WP = DS * 128;                  // one part of half a chunk
  static constexpr int kQo = 0;
  static constexpr int kKo = kQo + NS * QT;
  static constexpr int kVo = kKo + NS * QT;
  static constexpr int kWo = kVo + NS * VT;
  static constexpr int kXo = kWo + WH * 3 * WP;
  static constexpr int kSo = kXo + DK * DV * 2;        // 16 KB staging of o
  static constexpr int kBytes = kSo + 16384;
  static constexpr size_t smem = kBytes + 1024;
};

struct Bars {
  uint64_t fullQ[2], fullK[2], fullV[2], emptyQ[2], emptyK[2], emptyV[2];
  uint64_t s, p, o, ofree, x, xfree, w[2], wfree[2], u, fix, drain;
  uint32_t tmem;
  volatile int abort;
};

// Bounded wait that also ends when another role of the CTA has given up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Bars* B) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (B->abort) return false;
    if (globaltimer_ns() - t0 > kWaitNs) {
      B->abort = 1;
      atomicOr(&g_la_error, 1u);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* B) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, B);
}

__device__ __forceinline__ void unpack8(const uint4& q, float* f) {
  const __nv_bfloat162* h = (const __nv_bfloat162*)&q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __bfloat1622float2(h[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// kStates: only the states (K, V, U, X), each segment from zero.
template <int DK, int DV, bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
k_la_walk_tc(const __grid_constant__ Maps maps, const TcWalk p) {
  using G = Geom<DK, DV>;
  constexpr int NS = G::NS, WH = G::WH;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = align1024(raw);
  __shared__ Bars bars;
  Bars* B = &bars;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, seg = blockIdx.z;
  const float la = p.log_decay[h];
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const int c0 = seg * p.seg_chunks;
  const int c1 = min(c0 + p.seg_chunks, (len + kQ - 1) / kQ);
  const int nit = max(c1 - c0, 0);
  auto chunk = [&](int it) { return p.reverse ? c1 - 1 - it : c0 + it; };
  auto valid = [&](int c) { return min(kQ, len - c * kQ); };
  // rows of chunk c that lie past the row's end but not past T
  auto ragged = [&](int c) { return valid(c) < kQ && len < p.T; };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->fullQ[i], 1);
      mbar_init(&B->fullK[i], 1);
      mbar_init(&B->fullV[i], 1);
      mbar_init(&B->emptyQ[i], 1);
      mbar_init(&B->emptyK[i], 1);
      mbar_init(&B->emptyV[i], 1);
      mbar_init(&B->w[i], 128);
      mbar_init(&B->wfree[i], 1);
    }
    mbar_init(&B->s, 1);
    mbar_init(&B->p, 128);
    mbar_init(&B->o, 1);
    mbar_init(&B->ofree, 128);
    mbar_init(&B->x, 128);
    mbar_init(&B->xfree, 1);
    mbar_init(&B->u, 1);
    mbar_init(&B->fix, 128);
    mbar_init(&B->drain, 1);
    B->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&B->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tS = B->tmem, tO = tS + 128, tC = tS + 256, tU = tS + 384;

  if (warp == 8) {
    // ---- loads ----
    if (tid == 8 * 32) {
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
      int issued = 0;
      for (int it = 0; it < nit; ++it) {
        const int s = it % NS, t0 = chunk(it) * kQ;
        const uint32_t free = ((it / NS) & 1) ^ 1;
        if (!wait(&B->emptyK[s], free, B)) break;
        uint8_t* d = sm + G::kKo + s * G::QT;
        mbar_expect_tx(&B->fullK[s], G::QT);
        for (int x = 0; x < DK; x += 64)
          tma_load_4d(d + x * 256, &maps.k, x, h / p.ks, t0, b, &B->fullK[s]);
        if (!kStates) {
          if (!wait(&B->emptyQ[s], free, B)) break;
          d = sm + G::kQo + s * G::QT;
          mbar_expect_tx(&B->fullQ[s], G::QT);
          for (int x = 0; x < DK; x += 64)
            tma_load_4d(d + x * 256, &maps.q, x, h / p.qs, t0, b, &B->fullQ[s]);
        }
        if (!wait(&B->emptyV[s], free, B)) break;
        d = sm + G::kVo + s * G::VT;
        mbar_expect_tx(&B->fullV[s], G::VT);
        for (int x = 0; x < DV; x += 64)
          tma_load_4d(d + x * 256, &maps.v, x, h / p.vs, t0, b, &B->fullV[s]);
        issued = it + 1;
      }
      if (B->abort) {
        // no copy may be in flight when the CTA ends: those of the last stages
        // (a barrier that nothing was issued on in that phase runs out its limit)
        for (int it = issued > NS ? issued - NS : 0; it <= issued && it < nit; ++it) {
          const int s = it % NS;
          const uint32_t ph = (it / NS) & 1;
          const uint64_t lim = 50000000ull;
          mbar_wait(&B->fullK[s], ph, lim);
          if (!kStates) mbar_wait(&B->fullQ[s], ph, lim);
          mbar_wait(&B->fullV[s], ph, lim);
        }
      }
    }
  } else if (warp == 9) {
    // ---- products ----
    if (tid == 9 * 32) {
      const uint32_t id_s = idesc_bf16(128, 128, false, false);
      const uint32_t id_x = idesc_bf16(128, DV, false, true);
      const uint32_t id_u = idesc_bf16(128, DV, true, true);
      for (int it = 0; it < nit; ++it) {
        const int s = it % NS;
        const uint32_t full = (it / NS) & 1, ph = it & 1;
        const uint32_t aQ = smem_u32(sm + G::kQo + s * G::QT), aK = smem_u32(sm + G::kKo + s * G::QT);
        const uint32_t aV = smem_u32(sm + G::kVo + s * G::VT), aX = smem_u32(sm + G::kXo);
        if (!wait(&B->fullK[s], full, B)) break;
        if (!kStates) {
          if (!wait(&B->fullQ[s], full, B)) break;
          if (ragged(chunk(it)) && !wait(&B->fix, 0, B)) break;
          // S takes the columns of the previous chunk's P
          if (it > 0 && !wait(&B->o, ph ^ 1, B)) break;
          fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_bf16(tS, desc_sw128(aQ + off, 16, 1024), desc_sw128(aK + off, 16, 1024), id_s, kk > 0);
          }
          mma_commit(&B->s);
          if (!wait(&B->x, ph, B)) break;
          if (it > 0 && !wait(&B->ofree, ph ^ 1, B)) break;
          fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_bf16(tC, desc_sw128(aQ + off, 16, 1024), desc_sw128(aX + kk * 2048, DK * 128, 1024),
                     id_x, kk > 0);
          }
          mma_commit(&B->emptyQ[s]);
          mma_commit(&B->xfree);
        } else if (ragged(chunk(it)) && !wait(&B->fix, 0, B)) {
          break;
        }
        if (!wait(&B->fullV[s], full, B)) break;
        bool go = true;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int u = 2 * it + half, wb = u % WH;
          if (!wait(&B->w[wb], (u / WH) & 1, B)) {
            go = false;
            break;
          }
          fence_after_sync();
          const uint32_t aW = smem_u32(sm + G::kWo + wb * 3 * G::WP);
          // rows 64 half ... of the tile that is not scaled
          const uint32_t aT = (G::scale_k ? aV : aK) + half * 8192;
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t dw = desc_sw128(aW + part * G::WP + kk * 2048, 8192, 1024);
              const uint64_t dt = desc_sw128(aT + kk * 2048, 16384, 1024);
              mma_bf16(tU, G::scale_k ? dw : dt, G::scale_k ? dt : dw, id_u,
                       half + part + kk > 0);
            }
          mma_commit(&B->wfree[wb]);
        }
        if (!go) break;
        mma_commit(&B->emptyK[s]);
        mma_commit(&B->u);
        if (kStates) {
          mma_commit(&B->emptyV[s]);
        } else {
          if (!wait(&B->p, ph, B)) break;
          fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tO, tS + kk * 8, desc_sw128(aV + kk * 2048, 16384, 1024), id_x, kk > 0);
          mma_commit(&B->o);
          mma_commit(&B->emptyV[s]);
        }
      }
      mma_commit(&B->drain);
      mbar_wait(&B->drain, 0, kWaitNs);
    }
  } else if (warp < 4) {
    // ---- P and o: thread = row i of the chunk ----
    const int row = tid, il = row & 31, ib = warp;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // a^{|i-j|} of a column j of another 32-column block: a^(steps between the
    // blocks' facing edges) split into a factor of the row and one of the
    // column; inside the row's own block one factor per element
    float col[32], diag[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      col[j] = decay_pow(la, (float)(p.reverse ? j : 31 - j));
      const int d = p.reverse ? j - il : il - j;
      diag[j] = d >= 0 ? p.s_intra * decay_pow(la, (float)d) : 0.f;
    }
    float near[3];
#pragma unroll
    for (int x = 0; x < 3; ++x)
      near[x] = p.s_intra * decay_pow(la, (float)((p.reverse ? 32 - il : il + 1) + 32 * x));
    // (after a wait that gave up the four warps still meet at their barriers,
    // without touching the data)
    bool ok = true;
    for (int it = 0; it < nit; ++it) {
      const int c = chunk(it), n = valid(c), s = it % NS;
      const uint32_t ph = it & 1;
      if (ragged(c)) {
        const uint32_t full = (it / NS) & 1;
        ok = ok && wait(&B->fullK[s], full, B) && wait(&B->fullV[s], full, B) &&
             (kStates || wait(&B->fullQ[s], full, B));
        if (ok) {
          const uint4 z = make_uint4(0, 0, 0, 0);
          if (row >= n) {
            for (int x = 0; x < 2 * DK; x += 16) {
              const int at = (x >> 7) * 16384 + row * 128 + (x & 127);
              if (!kStates) *(uint4*)(sm + G::kQo + s * G::QT + at) = z;
              *(uint4*)(sm + G::kKo + s * G::QT + at) = z;
            }
            for (int x = 0; x < 2 * DV; x += 16)
              *(uint4*)(sm + G::kVo + s * G::VT + (x >> 7) * 16384 + row * 128 + (x & 127)) = z;
          }
          fence_async_smem();
          mbar_arrive(&B->fix);
        }
      }
      if (kStates) continue;
      ok = __all_sync(0xffffffffu, ok && wait(&B->s, ph, B));
      if (ok) {
        fence_after_sync();
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          const int dist = p.reverse ? jb - ib : ib - jb;
          uint32_t r[16];
          if (dist < 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = 0;
          } else {
            float v[32];
            tmem_ld32(tS + lane_base + jb * 32, v);
            tmem_wait_ld();
            if (dist == 0) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float2 x = mul2(make_float2(v[2 * j], v[2 * j + 1]),
                                make_float2(diag[2 * j], diag[2 * j + 1]));
                // a step that comes later has no part, whatever its product is
                if (p.reverse ? 2 * j < il : 2 * j > il) x.x = 0.f;
                if (p.reverse ? 2 * j + 1 < il : 2 * j + 1 > il) x.y = 0.f;
                r[j] = pack_bf16(x.x, x.y);
              }
            } else {
              const float f = dist == 1 ? near[0] : dist == 2 ? near[1] : near[2];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 x = mul2(mul2(make_float2(v[2 * j], v[2 * j + 1]), make_float2(f, f)),
                                      make_float2(col[2 * j], col[2 * j + 1]));
                r[j] = pack_bf16(x.x, x.y);
              }
            }
          }
          tmem_st16(tS + lane_base + jb * 16, r);
        }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(&B->p);
      }
      const int e = (p.reverse ? n - 1 - row : row) + p.off;
      const float lead = row < n ? p.s_carry * decay_pow(la, (float)e) : 0.f;
      ok = __all_sync(0xffffffffu, ok && wait(&B->o, ph, B));
      fence_after_sync();
      uint8_t* st = sm + G::kSo;
#pragma unroll
      for (int x = 0; x < DV; x += 32) {
        float v[32];
        if (ok) {
          float y[32];
          tmem_ld32(tO + lane_base + x, v);
          tmem_ld32(tC + lane_base + x, y);
          tmem_wait_ld();
          if (x == DV - 32) {
            fence_before_sync();
            mbar_arrive(&B->ofree);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = row < n ? fmaf(lead, y[j], v[j]) : 0.f;
        }
        // 16 KB of staging: 64 columns of bf16, or 32 of fp32
        if (p.o_f32 || x % 64 == 0) {
          if (tid == 0) bulk_wait_read0();
          named_sync(1, 128);
        }
        if (ok) {
          if (p.o_f32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *(float4*)(st + sw128(row, j)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *(uint4*)(st + sw128(row, (x % 64) / 8 + j)) = pack8(v + 8 * j);
          }
        }
        if (p.o_f32 || x % 64 == 32) {
          fence_async_smem();
          named_sync(1, 128);
          // (a box that starts past the width would start out of range)
          const int x0 = p.o_f32 ? x : x - 32;
          if (tid == 0 && ok && x0 < p.dv) {
            tma_store_4d(&maps.o, st, x0, h, c * kQ, b);
            bulk_commit();
          }
        }
      }
    }
    if (!kStates && tid == 0) bulk_wait0();
  } else {
    // ---- w o V (or K), X: thread = row j of a half, row k of the state ----
    const int t = tid - 128, k = t;
    const uint32_t lane_base = (uint32_t)((warp - 4) * 32) << 16;
    const bool mine = k < DK;
    float X[DV];
#pragma unroll
    for (int v = 0; v < DV; ++v) X[v] = 0.f;
    const size_t sbase = (((size_t)seg * p.B + b) * p.H + h) * p.dk * p.dv;
    if (!kStates && p.first && k < p.dk) {
      const float* f = p.first + sbase;
      // (unrolled: X stays in registers)
#pragma unroll
      for (int v = 0; v < DV; ++v)
        if (v < p.dv) X[v] = f[p.first_swapped ? (size_t)k * p.dv + v : (size_t)v * p.dk + k];
    }
    auto put_x = [&] {
      if (mine)
#pragma unroll
        for (int v = 0; v < DV; v += 8)
          *(uint4*)(sm + G::kXo + (v >> 6) * DK * 128 + sw128(k, (v & 63) >> 3)) = pack8(X + v);
      fence_async_smem();
      mbar_arrive(&B->x);
    };
    if (!kStates && nit > 0) put_x();
    auto all_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity, B)) != 0;
    };
    bool ok = true;
    for (int it = 0; it < nit && ok; ++it) {
      const int c = chunk(it), n = valid(c), s = it % NS;
      const uint32_t full = (it / NS) & 1;
      if (!all_wait(G::scale_k ? &B->fullK[s] : &B->fullV[s], full)) break;
      if (ragged(c) && !all_wait(&B->fix, 0)) break;
      const uint8_t* src = sm + (G::scale_k ? G::kKo + s * G::QT : G::kVo + s * G::VT);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int u = 2 * it + half, wb = u % WH;
        if (!all_wait(&B->wfree[wb], ((u / WH) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const int r = t & 63, j = half * 64 + r;
        const int e = (p.reverse ? j : n - 1 - j) + 1 - p.off;
        const float w = j < n ? p.s_inject * decay_pow(la, (float)e) : 0.f;
        uint8_t* dst = sm + G::kWo + wb * 3 * G::WP;
        // a thread takes half of the row: 32 columns of each 64
#pragma unroll
        for (int x = 0; x < G::DS; x += 64)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int ch = (t >> 6) * 4 + q;
            float f[8], m[8];
            unpack8(*(const uint4*)(src + (x >> 6) * 16384 + sw128(j, ch)), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= w;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint4 o = pack8(f);
              *(uint4*)(dst + part * G::WP + (x >> 6) * 8192 + sw128(r, ch)) = o;
              unpack8(o, m);
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] -= m[i];
            }
          }
        fence_async_smem();
        fence_before_sync();
        mbar_arrive(&B->w[wb]);
      }
      if (!ok || !all_wait(&B->u, it & 1)) break;
      fence_after_sync();
      const float an = decay_pow(la, (float)n);
#pragma unroll
      for (int x = 0; x < DV; x += 32) {
        float v[32];
        tmem_ld32(tU + lane_base + x, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) X[x + i] = fmaf(an, X[x + i], v[i]);
      }
      fence_before_sync();
      if (!kStates && it + 1 < nit) {
        if (!all_wait(&B->xfree, it & 1)) break;
        put_x();
      }
    }
    if (p.last && k < p.dk) {
      float* l = p.last + sbase;
#pragma unroll
      for (int v = 0; v < DV; ++v)
        if (v < p.dv) l[!kStates && p.first_swapped ? (size_t)k * p.dv + v : (size_t)v * p.dk + k] = X[v];
    }
  }
  if (!kStates) {
    // whole chunks of the segment past the row's end
    const int z0 = max(c1, c0) * kQ, z1 = min((c0 + p.seg_chunks) * kQ, p.T);
    const int esz = p.o_f32 ? 4 : 2, row16 = p.dv * esz / 16;
    for (long long i = tid; i < (long long)(z1 - z0) * row16; i += kThreads) {
      const long long t = z0 + i / row16;
      uint8_t* o = (uint8_t*)p.o + (((size_t)b * p.T + t) * p.H + h) * p.dv * esz;
      *(uint4*)(o + (i % row16) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tmem_dealloc(tS, 512);
  }
}

// The states before each segment from the segments' own: in walk order
//   X_0 = first, X_{s+1} = a^{steps of s} X_s + local_s;  last = X_nseg.
// seg [nseg][B][H][dv][dk], overwritten in place.
__global__ void __launch_bounds__(256) k_la_segments(const TcWalk p, float* seg, const float* first,
                                                     float* last) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int i = blockIdx.x * 256 + threadIdx.x, n = p.dk * p.dv;
  if (i >= n) return;
  const float la = p.log_decay[h];
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const size_t row = ((size_t)b * p.H + h) * n, stride = (size_t)p.B * p.H * n;
  const size_t at = row + (p.first_swapped ? (size_t)(i % p.dk) * p.dv + i / p.dk : (size_t)i);
  float x = first ? first[at] : 0.f;
  for (int j = 0; j < p.nseg; ++j) {
    const int s = p.reverse ? p.nseg - 1 - j : j;
    const int span = p.seg_chunks * kQ;
    const int steps = min(max(len - s * span, 0), span);
    float* q = seg + s * stride + row + i;
    const float local = *q;
    *q = x;
    x = fmaf(decay_pow(la, (float)steps), x, local);
  }
  if (last) last[at] = x;
}

// ---- host --------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  });
  return fn;
}

// [B][T][heads][D] with {128 bytes of D, one head, 128 steps, one row} boxes.
bool map_4d(CUtensorMap* m, const void* base, bool f32, int D, int heads, int T, int B,
            long long step, long long batch) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = f32 ? 4 : 2;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {D * e, (cuuint64_t)step * e, (cuuint64_t)batch * e};
  cuuint32_t box[4] = {f32 ? 32u : 64u, 1, kQ, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool kStates>
cudaError_t launch(const Maps& m, const TcWalk& p, cudaStream_t s) {
  constexpr size_t smem = Geom<DK, DV>::smem;
  static_assert(smem + sizeof(Bars) <= 232448, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(k_la_walk_tc<DK, DV, kStates>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "linattn_states" : p.reverse ? "linattn_walk_back" : "linattn_walk", s);
  k_la_walk_tc<DK, DV, kStates><<<dim3(p.H, p.B, p.nseg), kThreads, smem, s>>>(m, p);
  return cudaGetLastError();
}

template <bool kStates>
cudaError_t launch_d(const Maps& m, const TcWalk& p, cudaStream_t s) {
  if (p.dk <= 64) return p.dv <= 64 ? launch<64, 64, kStates>(m, p, s) : launch<64, 128, kStates>(m, p, s);
  return p.dv <= 64 ? launch<128, 64, kStates>(m, p, s) : launch<128, 128, kStates>(m, p, s);
}

}  // namespace

int la_tc_segments(int B, int H, int T) {
  // One CTA an SM: a row's nc chunks go to one CTA unless that leaves SMs idle.
  // Splitting a row costs a pass over K and V for the segments' states (about
  // half a walk) and two more launches, so it has to pay for that.
  const long long nc = (T + kQ - 1) / kQ, rows = (long long)B * H, sms = 152;
  auto waves = [&](long long n) { return (rows * n + sms - 1) / sms; };
  double best = (double)(waves(1) * nc);
  long long at = 1;
  for (long long n = 2; n <= nc && n <= 64; ++n) {
    const long long per = (nc + n - 1) / n;
    const double cost = 1.5 * (double)(waves(n) * per) + 4.0;
    if (cost < best) {
      best = cost;
      at = n;
    }
  }
  return (int)at;
}

size_t la_tc_scratch_floats(int B, int H, int T, int dk, int dv) {
  const int n = la_tc_segments(B, H, T);
  return n > 1 ? (size_t)n * B * H * dk * dv : 0;
}

cudaError_t la_walk_tc(const LaWalk& w, float* scratch, cudaStream_t s) {
  Maps m;
  if (!map_4d(&m.q, w.q.p, false, w.dk, w.H / w.q.share, w.T, w.B, w.q.step, w.q.batch) ||
      !map_4d(&m.k, w.k.p, false, w.dk, w.H / w.k.share, w.T, w.B, w.k.step, w.k.batch) ||
      !map_4d(&m.v, w.v.p, false, w.dv, w.H / w.v.share, w.T, w.B, w.v.step, w.v.batch) ||
      !map_4d(&m.o, w.o, w.o_f32, w.dv, w.H, w.T, w.B, (long long)w.H * w.dv,
              (long long)w.T * w.H * w.dv))
    return cudaErrorNotSupported;
  TcWalk p = {};
  p.B = w.B;
  p.T = w.T;
  p.H = w.H;
  p.dk = w.dk;
  p.dv = w.dv;
  p.qs = w.q.share;
  p.ks = w.k.share;
  p.vs = w.v.share;
  p.log_decay = w.log_decay;
  p.lens = w.lens;
  p.o = w.o;
  p.o_f32 = w.o_f32;
  p.s_intra = w.s_intra;
  p.s_carry = w.s_carry;
  p.s_inject = w.s_inject;
  p.off = w.off;
  p.reverse = w.reverse;
  const int nc = (w.T + kQ - 1) / kQ;
  int n = la_tc_segments(w.B, w.H, w.T);
  p.seg_chunks = (nc + n - 1) / n;
  n = (nc + p.seg_chunks - 1) / p.seg_chunks;
  p.nseg = n;
  p.first = w.first;
  p.last = w.last;
  p.first_swapped = w.first_swapped;
  if (n > 1) {
    p.last = scratch;
    cudaError_t e = launch_d<true>(m, p, s);
    if (e != cudaSuccess) return e;
    {
      LaunchScope ls("linattn_segments", s);
      k_la_segments<<<dim3((w.dk * w.dv + 255) / 256, w.H, w.B), 256, 0, s>>>(p, scratch, w.first,
                                                                              w.last);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    p.first = scratch;
    p.first_swapped = 0;
    p.last = nullptr;
  }
  return launch_d<false>(m, p, s);
}

cudaError_t la_read_and_clear_error(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_la_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_la_error, &zero, sizeof(unsigned int));
}

}  // namespace ssd
