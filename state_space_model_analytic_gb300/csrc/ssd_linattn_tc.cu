// Tensor-core walk of linear attention with a decay for each head (bf16
// operands, fp32 state): the forward and, with exchanged roles, the gradients
// (the formulas stand in ssd_linattn.cu).
//
// Chunks of 128 steps; one CTA per (head, 64 columns of v, row, segment of the
// row).  Per chunk, with w_j the decay from step j to the chunk's end and X the
// state before it ([dk][64], rows k),
//   S  = Q K^T              128 x 128, masked and decayed into P (bf16, TMEM)
//   O  = P V                A from TMEM
//   Oc = Q X                X in bf16; o = O + lead_i Oc
//   U  = K^T (w o V)        X <- a^n X + U, X in fp32 registers
// All accumulators are in TMEM (512 columns, one CTA per SM).
//
// Precision.  P is rounded to bf16 once (the scores are the A operand of the
// second product) and X once as an operand; the output is bf16 itself.  The
// state is an fp32 result, so w o V is carried exactly, as three bf16 parts of
// 8 bits each, side by side in one product of 192 columns.
//
// Bound by memory: a chunk moves dk, dk, 64, 64 columns of 128 rows once, at
// 45 GB/s an SM some 4100 cycles for dk = 128, against 1900 cycles of products
// and 3200 of shared-memory traffic.  The work is split over warps so that it
// overlaps with the loads and with itself: warps 0-7 turn S into P and write o
// of the chunk before (thread = row and half of the columns), warps 8-15 build
// the parts of w o V and carry X (thread = row k and half of the columns), one
// warp each issues the TMA loads of the next chunks, the products of S, of O
// and Oc, and of U.  128 columns of v are two CTAs, which read q
// and k twice (from L2) and form S twice: at 64 columns the accumulators leave
// room for P beside S, so that S of the next chunk does not wait for P V.
//
// Rows past the end of a batch row (its length, or T) take part as zeros: TMA
// fills what lies past T; between a shorter row's end and T warps 0-7 clear
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
constexpr int kThreads = 640;  // 8 + 8 warps, and four of which three issue loads and products
constexpr long long kWaitClocks = 3000000000ll;
constexpr uint64_t kWaitNs = 1000000000ull;  // at the end, for what is still in flight

__device__ unsigned int g_la_error;

struct Maps {
  CUtensorMap q, k, v, o;
};

// What of a walk a kernel needs.
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
  float s_intra, s_carry, s_inject;
  int off, reverse;
  int beside;  // launched beside the kernel before it, whose end it waits for last
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
// The products are issued by one lane; the predicate is on the instruction and
// not on a branch around it, so that the operands stay in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t issue, uint32_t d_tmem, uint64_t a_desc,
                                       uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
// the same with A in TMEM: its row i is lane i, two bf16 a column
__device__ __forceinline__ void mma_ts(uint32_t issue, uint32_t d_tmem, uint32_t a_tmem,
                                       uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t issue, uint64_t* mbar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(mbar)),
      "r"(issue)
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
// 32 lanes x 8 columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// One arrival for the warp, after what its lanes did before (each lane has
// issued the fences that its writes need).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}


__device__ __forceinline__ float decay_pow(float la, float e) { return e == 0.f ? 1.f : expf(la * e); }

// ---- shared memory and tensor memory --------------------------------------------

constexpr int kV = 64;      // columns of v of a CTA
constexpr int kPiece = 32;  // steps of a piece of w o V
constexpr int kDiagRow = 36;  // (16-byte pieces of 8 rows fall on all 32 banks)

// NS: stages of the loads; NW: buffers of a piece's three parts; NB: 16 KB
// buffers that o is staged in.  The sums stay below the 227 KB of a CTA.
template <int DK, bool kStates>
struct Geom {
  static constexpr int NS = kStates || DK == 64 ? 3 : 2;
  static constexpr int NW = kStates ? 4 : 2;
  static constexpr int NB = kStates ? 0 : DK == 64 ? 2 : 1;
  static constexpr int QT = DK * 256, VT = kV * 256;  // bytes of 128 rows
  static constexpr int WP = kPiece * 128;              // one part of a piece
  static constexpr int kQo = 0;
  static constexpr int kKo = kStates ? 0 : NS * QT;
  static constexpr int kVo = kKo + NS * QT;
  static constexpr int kWo = kVo + NS * VT;
  static constexpr int kXo = kWo + NW * 3 * WP;
  static constexpr int kSo = kXo + (kStates ? 0 : DK * kV * 2);
  static constexpr int kDo = kSo + NB * 16384;          // kDiagRow floats a row, 32 rows
  static constexpr int kBytes = kDo + (kStates ? 0 : 32 * kDiagRow * 4);
  static constexpr size_t smem = kBytes + 1024;
};

// TMEM columns
constexpr int cS = 0, cP = 128, cO = 192, cC = 256, cU = 320;

struct Bars {
  uint64_t fullQ[3], fullK[3], fullV[3], emptyQ[3], emptyK[3], emptyV[3];
  uint64_t w[4], wfree[4], s, sfree, p, o, ofree, x, xfree, u, fix, drain[3];
  uint32_t tmem;
  volatile int abort;
  float pw[132];  // a^0 ... a^130
  alignas(16) float col[32];
};

// Bounded wait that also ends when another role of the CTA has given up.  The
// bound is in SM clocks (about a second and a half): reading the nanosecond
// timer takes about a microsecond, which every wait that is not over at once
// would pay.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Bars* B) {
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (B->abort) return false;
    if (clock64() - t0 > kWaitClocks) {
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

// kStates: only the states (K, V, U, X), each segment from zero.  kF32: o is
// fp32 (partial sums), else bf16.
template <int DK, bool kStates, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
k_la_walk_tc(const __grid_constant__ Maps maps, const TcWalk p) {
  using G = Geom<DK, kStates>;
  constexpr int NS = G::NS, NW = G::NW;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = align1024(raw);
  __shared__ Bars bars;
  Bars* B = &bars;
  // (the shuffles tell the compiler what is the same in a warp's lanes: the roles'
  // branches and loops and the products' operands then stay in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (p.dv + kV - 1) / kV;
  const int h = blockIdx.x / vblocks, v0 = (blockIdx.x % vblocks) * kV;
  const int b = blockIdx.y, seg = blockIdx.z;
  grid_dep_launch();  // a kernel that needs nothing of this one may start beside it
  const float la = p.log_decay[h];
  int len = p.T;
  if (p.lens) len = __shfl_sync(0xffffffffu, min(max(p.lens[b], 0), p.T), 0);
  const int c0 = seg * p.seg_chunks;
  const int c1 = min(c0 + p.seg_chunks, (len + kQ - 1) / kQ);
  const int nit = max(c1 - c0, 0);
  auto chunk = [&](int it) { return p.reverse ? c1 - 1 - it : c0 + it; };
  auto valid = [&](int c) { return min(kQ, len - c * kQ); };
  // rows of chunk c that lie past the row's end but not past T
  auto ragged = [&](int c) { return valid(c) < kQ && len < p.T; };
  auto all_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity, B)) != 0;
  };
  // w o V of pieces [first, end) of chunk `it`, by 256 threads (t): a row of the
  // piece and one of its 16-byte chunks each
  auto pieces = [&](int it, const int first, const int end, int t) {
    const int r = t & 31, ch = t >> 5, n = valid(chunk(it));
    const uint8_t* src = sm + G::kVo + (it % NS) * G::VT;
    uint4 in[4];
#pragma unroll
    for (int i = first; i < end; ++i) in[i] = *(const uint4*)(src + sw128(i * kPiece + r, ch));
#pragma unroll
    for (int piece = first; piece < end; ++piece) {
      // the three parts, before the wait for the buffer they go to
      const int j = piece * kPiece + r;
      const float w = j < n ? p.s_inject * bars.pw[(p.reverse ? j : n - 1 - j) + 1 - p.off] : 0.f;
      const float2 w2 = make_float2(w, w);
      float2 f[4];
      unpack8(in[piece], (float*)f);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w2);
      uint4 o[3];
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        o[part] = pack8((const float*)f);
        float2 m[4];
        unpack8(o[part], (float*)m);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = fma2(m[i], make_float2(-1.f, -1.f), f[i]);
      }
      const int wb = piece % NW;  // (its turn: 4 / NW times a chunk)
      if (!all_wait(&B->wfree[wb], ((it * (4 / NW) + piece / NW) & 1) ^ 1)) return false;
      uint8_t* dst = sm + G::kWo + wb * 3 * G::WP + sw128(r, ch);
#pragma unroll
      for (int part = 0; part < 3; ++part) *(uint4*)(dst + part * G::WP) = o[part];
      fence_async_smem();
      fence_before_sync();
      warp_arrive(&B->w[wb]);
    }
    return true;
  };
  // zeros into a row of a stage: 64 bytes of each 128-byte row of each tile
  auto clear_row = [&](int s, int row, int hf) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    const int at = row * 128 + hf * 64;
#pragma unroll 1
    for (int x = 0; x < 2 * DK / 128 * 4; ++x) {
      const int o = (x >> 2) * 16384 + at + (x & 3) * 16;
      if (!kStates) *(uint4*)(sm + G::kQo + s * G::QT + o) = z;
      *(uint4*)(sm + G::kKo + s * G::QT + o) = z;
    }
#pragma unroll 1
    for (int x = 0; x < 4; ++x) *(uint4*)(sm + G::kVo + s * G::VT + at + x * 16) = z;
  };

  // the loads of chunk `it` of the walk, each once its buffer is free
  auto load = [&](int it) {
    const int s = it % NS, t0 = chunk(it) * kQ;
    const uint32_t free = ((it / NS) & 1) ^ 1;
    if (!wait(&B->emptyK[s], free, B)) return false;
    uint8_t* d = sm + G::kKo + s * G::QT;
    mbar_expect_tx(&B->fullK[s], G::QT);
    for (int x = 0; x < DK; x += 64)
      tma_load_4d(d + x * 256, &maps.k, x, h / p.ks, t0, b, &B->fullK[s]);
    if (!kStates) {
      if (!wait(&B->emptyQ[s], free, B)) return false;
      d = sm + G::kQo + s * G::QT;
      mbar_expect_tx(&B->fullQ[s], G::QT);
      for (int x = 0; x < DK; x += 64)
        tma_load_4d(d + x * 256, &maps.q, x, h / p.qs, t0, b, &B->fullQ[s]);
    }
    if (!wait(&B->emptyV[s], free, B)) return false;
    mbar_expect_tx(&B->fullV[s], G::VT);
    tma_load_4d(sm + G::kVo + s * G::VT, &maps.v, v0, h / p.vs, t0, b, &B->fullV[s]);
    return true;
  };
  // (the loading thread sets the barriers up and starts on the first stages at once)
  if (tid == 19 * 32) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&B->fullQ[i], 1);
      mbar_init(&B->fullK[i], 1);
      mbar_init(&B->fullV[i], 1);
      mbar_init(&B->emptyQ[i], 1);
      mbar_init(&B->emptyK[i], kStates ? 1 : 2);
      mbar_init(&B->emptyV[i], kStates ? 1 : 2);
    }
    for (int i = 0; i < NW; ++i) {
      mbar_init(&B->w[i], 8);
      mbar_init(&B->wfree[i], 1);
    }
    mbar_init(&B->s, 1);
    mbar_init(&B->sfree, 8);
    mbar_init(&B->p, 8);
    mbar_init(&B->o, 1);
    mbar_init(&B->ofree, 8);
    mbar_init(&B->x, 8);
    mbar_init(&B->xfree, 1);
    mbar_init(&B->u, 1);
    mbar_init(&B->fix, 8);
    mbar_init(&B->drain[0], 1);
    mbar_init(&B->drain[1], 1);
    mbar_init(&B->drain[2], 1);
    B->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.v);
#pragma unroll 1
    for (int it = 0; it < min(nit, NS); ++it) load(it);
  }
  for (int i = tid; i < 131; i += kThreads) bars.pw[i] = decay_pow(la, (float)i);
  if (tid >= 160 && tid < 192) {
    const int j = tid - 160;
    bars.col[j] = decay_pow(la, (float)(p.reverse ? j : 31 - j));
  }
  // s_intra a^{|i-j|} inside a 32 x 32 block on the diagonal, 0 for later steps
  float* diag = (float*)(sm + G::kDo);
  if (!kStates)
    for (int i = tid; i < 1024; i += kThreads) {
      const int d = p.reverse ? (i & 31) - (i >> 5) : (i >> 5) - (i & 31);
      diag[(i >> 5) * kDiagRow + (i & 31)] = d >= 0 ? p.s_intra * decay_pow(la, (float)d) : 0.f;
    }
  if (warp == 16) {
    tmem_alloc(&B->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = __shfl_sync(0xffffffffu, B->tmem, 0);

  if (warp == 19) {
    // ---- loads ----
    if (tid == 19 * 32) {
      int it = min(nit, NS);
#pragma unroll 1
      for (; it < nit; ++it)
        if (!load(it)) break;
      if (B->abort) {
        // no copy may be in flight when the CTA ends: those of the last stages
        // (a barrier that nothing was issued on in that phase runs out its limit)
        for (int j = it > NS ? it - NS : 0; j <= it && j < nit; ++j) {
          const int s = j % NS;
          const uint32_t ph = (j / NS) & 1;
          const uint64_t lim = 50000000ull;
          mbar_wait(&B->fullK[s], ph, lim);
          if (!kStates) mbar_wait(&B->fullQ[s], ph, lim);
          mbar_wait(&B->fullV[s], ph, lim);
        }
      }
    }
  } else if (warp == 17) {
    // ---- products of the scores: S (once S of the last chunk is read) ----
    // The whole warp walks the loop (so that descriptors stay warp-uniform), one
    // lane issues.  Descriptors of a tile differ in their start address alone
    // (16-byte units): K-major steps of 16 are 2 units apart and 1024 units after
    // every four, MN-major ones 128.
    const uint32_t lead = (tid & 31) == 0;
    constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
    const uint64_t dQ0 = desc_sw128(smem_u32(sm + G::kQo), 16, 1024);
    const uint64_t dK0 = desc_sw128(smem_u32(sm + G::kKo), 16, 1024);
#pragma unroll 1
    for (int it = 0; it < nit && !kStates; ++it) {
      const int s = it % NS;
      const uint32_t full = (it / NS) & 1;
      if (!all_wait(&B->fullK[s], full) || !all_wait(&B->fullQ[s], full)) break;
      if (ragged(chunk(it)) && !all_wait(&B->fix, 0)) break;
      if (it > 0 && !all_wait(&B->sfree, (it - 1) & 1)) break;
      fence_after_sync();
      const uint64_t dQ = dQ0 + s * (G::QT >> 4), dK = dK0 + s * (G::QT >> 4);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const int off = (kk >> 2) * 1024 + (kk & 3) * 2;
        mma_ss(lead, tm + cS, dQ + off, dK + off, id_s, kk > 0);
      }
      commit_if(lead, &B->s);
      commit_if(lead, &B->emptyK[s]);
    }
    commit_if(lead, &B->drain[0]);
    mbar_wait(&B->drain[0], 0, kWaitNs);
    __syncwarp();
  } else if (warp == 16) {
    // ---- products of the output: O and Oc (once those of the last chunk are read) ----
    const uint32_t lead = (tid & 31) == 0;
    constexpr uint32_t id_x = idesc_bf16(128, kV, false, true);
    const uint64_t dQ0 = desc_sw128(smem_u32(sm + G::kQo), 16, 1024);
    const uint64_t dX = desc_sw128(smem_u32(sm + G::kXo), 16, 1024);
    const uint64_t dV0 = desc_sw128(smem_u32(sm + G::kVo), 16, 1024);
#pragma unroll 1
    for (int it = 0; it < nit && !kStates; ++it) {
      const int s = it % NS;
      const uint32_t full = (it / NS) & 1, ph = it & 1;
      if (it > 0 && !all_wait(&B->ofree, ph ^ 1)) break;
      if (!all_wait(&B->x, ph) || !all_wait(&B->fullQ[s], full)) break;
      fence_after_sync();
      const uint64_t dQ = dQ0 + s * (G::QT >> 4);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk)
        mma_ss(lead, tm + cC, dQ + ((kk >> 2) * 1024 + (kk & 3) * 2), dX + 128 * kk, id_x, kk > 0);
      commit_if(lead, &B->xfree);
      commit_if(lead, &B->emptyQ[s]);
      if (!all_wait(&B->p, ph) || !all_wait(&B->fullV[s], full)) break;
      fence_after_sync();
      const uint64_t dV = dV0 + s * (G::VT >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts(lead, tm + cO, tm + cP + 8 * kk, dV + 128 * kk, id_x, kk > 0);
      commit_if(lead, &B->o);
      commit_if(lead, &B->emptyV[s]);
    }
    commit_if(lead, &B->drain[2]);
    mbar_wait(&B->drain[2], 0, kWaitNs);
    __syncwarp();
  } else if (warp == 18) {
    // ---- products of the state: U, the parts side by side (3 x 64 columns) ----
    const uint32_t lead = (tid & 31) == 0;
    constexpr uint32_t id_u = idesc_bf16(128, 3 * kV, true, true);
    const uint64_t dK0 = desc_sw128(smem_u32(sm + G::kKo), 16384, 1024);
    const uint64_t dW0 = desc_sw128(smem_u32(sm + G::kWo), G::WP, 1024);
#pragma unroll 1
    for (int it = 0; it < nit; ++it) {
      const int s = it % NS;
      if (!all_wait(&B->fullK[s], (it / NS) & 1)) break;
      if (ragged(chunk(it)) && !all_wait(&B->fix, 0)) break;
      bool go = true;
#pragma unroll 1
      for (int piece = 0; piece < 4; ++piece) {
        const int wb = piece % NW;
        go = go && all_wait(&B->w[wb], (it * (4 / NW) + piece / NW) & 1);
        if (!go) break;
        fence_after_sync();
        // (two accumulators in turn in a states walk, which has the columns: the
        // first pieces come before the last U is read)
        const uint32_t u0 = kStates ? (it & 1) * 192 : cU;
        const uint64_t dK = dK0 + (s * (G::QT >> 4) + piece * (kPiece * 8));
        const uint64_t dW = dW0 + wb * (3 * G::WP >> 4);
#pragma unroll
        for (int kk = 0; kk < kPiece / 16; ++kk)
          mma_ss(lead, tm + u0, dK + 128 * kk, dW + 128 * kk, id_u, piece + kk > 0);
        commit_if(lead, &B->wfree[wb]);
      }
      if (!go) break;
      commit_if(lead, &B->u);
      commit_if(lead, &B->emptyK[s]);
      commit_if(lead, &B->emptyV[s]);
    }
    commit_if(lead, &B->drain[1]);
    mbar_wait(&B->drain[1], 0, kWaitNs);
    __syncwarp();
  } else if (warp < 8) {
    // ---- P and o: thread = row i of the chunk and every second 32 columns ----
    const int row = tid & 127, il = row & 31, ib = warp & 3, hf = warp >> 2;
    const uint32_t lane_base = (uint32_t)(ib * 32) << 16;
    if (kStates) {  // the first two pieces of w o V
#pragma unroll 1
      for (int it = 0; it < nit; ++it) {
        if (!all_wait(&B->fullV[it % NS], (it / NS) & 1)) break;
        if (ragged(chunk(it)) && !all_wait(&B->fix, 0)) break;
        if (!pieces(it, 0, 2, tid)) break;
      }
    }
    // per turn: o of chunk it - 1 out of TMEM, P of chunk it, then the stores of
    // that o.  (After a wait that gave up the warps still meet at their barriers,
    // without touching the data.)
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it <= nit && !kStates && nit > 0; ++it) {
      uint32_t y[kF32 ? 32 : 16];  // this thread's 32 columns of o, bf16 in pairs or fp32
      if (it > 0) {
        ok = __all_sync(0xffffffffu, ok && wait(&B->o, (it - 1) & 1, B));
        fence_after_sync();
        const int n = valid(chunk(it - 1));
        const float lead =
            row < n ? p.s_carry * bars.pw[(p.reverse ? n - 1 - row : row) + p.off] : 0.f;
        const float2 l2 = make_float2(lead, lead);
        if (ok) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float u[16], w[16];
            tmem_ld16(tm + cO + lane_base + hf * 32 + z * 16, u);
            tmem_ld16(tm + cC + lane_base + hf * 32 + z * 16, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 a = fma2(l2, make_float2(w[j], w[j + 1]), make_float2(u[j], u[j + 1]));
              if (kF32) {
                y[(kF32 ? 16 * z : 0) + j] = __float_as_uint(a.x);
                y[(kF32 ? 16 * z : 0) + j + 1] = __float_as_uint(a.y);
              } else {
                y[8 * z + j / 2] = pack_bf16(a.x, a.y);
              }
            }
          }
          if (n < kQ && row >= n) {
#pragma unroll
            for (int j = 0; j < (kF32 ? 32 : 16); ++j) y[j] = 0;
          }
          fence_before_sync();
          warp_arrive(&B->ofree);
        }
      }
      if (it < nit) {
        const int c = chunk(it);
        if (ragged(c)) {
          const int s = it % NS;
          const uint32_t full = (it / NS) & 1;
          ok = __all_sync(0xffffffffu, ok && wait(&B->fullK[s], full, B) &&
                                           wait(&B->fullV[s], full, B) &&
                                           wait(&B->fullQ[s], full, B));
          if (ok) {
            if (row >= valid(c)) clear_row(s, row, hf);
            fence_async_smem();
            warp_arrive(&B->fix);
          }
        }
        ok = __all_sync(0xffffffffu, ok && wait(&B->s, it & 1, B));
        fence_after_sync();
        // a^{|i-j|}: on the diagonal from the table; elsewhere the steps between the
        // blocks' facing edges, split into a factor of the row and one of the
        // column.  Blocks of later steps are zero.  (The product that read the last
        // P is over: its o was waited for.)
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int jb = 2 * x + hf, dist = p.reverse ? jb - ib : ib - jb;
          uint32_t r[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = 0;
          if (ok && dist >= 0) {
            float v[32];
            tmem_ld32(tm + cS + lane_base + jb * 32, v);
            tmem_wait_ld();
            if (dist == 0) {
              const float* g = diag + il * kDiagRow;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 e = *(const float4*)(g + 4 * j);
                const float2 a0 = mul2(make_float2(v[4 * j], v[4 * j + 1]), make_float2(e.x, e.y));
                const float2 a1 = mul2(make_float2(v[4 * j + 2], v[4 * j + 3]), make_float2(e.z, e.w));
                r[2 * j] = pack_bf16(a0.x, a0.y);
                r[2 * j + 1] = pack_bf16(a1.x, a1.y);
              }
            } else {
              const float f = p.s_intra * bars.pw[(p.reverse ? 32 - il : il + 1) + 32 * (dist - 1)];
              const float2 f2 = make_float2(f, f);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 g = *(const float4*)&bars.col[4 * j];
                const float2 a0 = mul2(mul2(make_float2(v[4 * j], v[4 * j + 1]), f2), make_float2(g.x, g.y));
                const float2 a1 = mul2(mul2(make_float2(v[4 * j + 2], v[4 * j + 3]), f2), make_float2(g.z, g.w));
                r[2 * j] = pack_bf16(a0.x, a0.y);
                r[2 * j + 1] = pack_bf16(a1.x, a1.y);
              }
            }
          }
          if (ok) {
            tmem_st16(tm + cP + lane_base + jb * 16, r);
            if (x == 1) {
              tmem_wait_st();
              fence_before_sync();
              warp_arrive(&B->sfree);
              if ((tid & 31) == 0) mbar_arrive(&B->p);
            }
          }
        }
      }
      if (it == 0) continue;
      // o, staged in 128-byte rows: 64 columns of bf16 (both halves of the threads),
      // or 32 of fp32 (one half; one after the other where there is one buffer)
#pragma unroll 1
      for (int x = 0; x < (kF32 && G::NB == 1 ? 2 : 1); ++x) {
        uint8_t* st = sm + G::kSo + (kF32 && G::NB == 2 ? hf : 0) * 16384;
        if (tid == 0) bulk_wait_read0();
        named_sync(1, 256);
        if (ok && (!kF32 || G::NB == 2 || x == hf)) {
#pragma unroll
          for (int j = 0; j < (kF32 ? 8 : 4); ++j)
            *(uint4*)(st + sw128(row, (kF32 ? 0 : hf * 4) + j)) =
                make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
        fence_async_smem();
        named_sync(1, 256);
        if (tid == 0 && ok) {
          // (a box that starts past the width would start out of range)
          const int x0 = v0 + x * 32, t0 = chunk(it - 1) * kQ;
          if (x0 < p.dv) tma_store_4d(&maps.o, sm + G::kSo, x0, h, t0, b);
          if (kF32 && G::NB == 2 && x0 + 32 < p.dv)
            tma_store_4d(&maps.o, sm + G::kSo + 16384, x0 + 32, h, t0, b);
          bulk_commit();
        }
      }
    }
    if (!kStates && tid == 0) bulk_wait0();
  } else if (warp < 16) {
    // ---- w o V: thread = row of a piece and a 16-byte chunk; X: thread = row k of
    // the state and 32 columns ----
    const int t = tid - 256, k = t & 127, hf = t >> 7;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    float X[32];  // columns v0 + 32 hf + i
#pragma unroll
    for (int i = 0; i < 32; ++i) X[i] = 0.f;
    const size_t sbase = (((size_t)seg * p.B + b) * p.H + h) * p.dk * p.dv;
    const int vx = v0 + hf * 32;
    if (!kStates && p.first && k < p.dk) {
      const float* f = p.first + sbase;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (vx + i < p.dv)
          X[i] = f[p.first_swapped ? (size_t)k * p.dv + vx + i : (size_t)(vx + i) * p.dk + k];
    }
#pragma unroll 1
    for (int it = 0; it < nit; ++it) {
      const int c = chunk(it), n = valid(c), s = it % NS;
      const uint32_t full = (it / NS) & 1;
      if (!all_wait(&B->fullV[s], full)) break;
      if (ragged(c)) {
        if (kStates) {  // (where warps 0-7 do not follow K's loads)
          if (!all_wait(&B->fullK[s], full)) break;
          if (k >= n) clear_row(s, k, hf);
          fence_async_smem();
          warp_arrive(&B->fix);
        }
        if (!all_wait(&B->fix, 0)) break;
      }
      // (in a states walk warps 0-7 form the first two pieces)
      if (!pieces(it, kStates ? 2 : 0, 4, t)) break;
      if (!kStates) {  // X before this chunk, for its Oc
        if (it > 0 && !all_wait(&B->xfree, (it - 1) & 1)) break;
        if (k < DK)
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *(uint4*)(sm + G::kXo + sw128(k, hf * 4 + i / 8)) = pack8(X + i);
        fence_async_smem();
        warp_arrive(&B->x);
      }
      if (!all_wait(&B->u, it & 1)) break;
      fence_after_sync();
      const float an = bars.pw[n];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t at = tm + (kStates ? (it & 1) * 192 : cU) + lane_base + hf * 32 + x * 8;
        float v[8], m[8], l[8];
        tmem_ld8(at, v);
        tmem_ld8(at + 64, m);
        tmem_ld8(at + 128, l);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 y = add2(make_float2(v[i], v[i + 1]),
                                add2(make_float2(m[i], m[i + 1]), make_float2(l[i], l[i + 1])));
          const float2 z = fma2(make_float2(an, an), make_float2(X[8 * x + i], X[8 * x + i + 1]), y);
          X[8 * x + i] = z.x;
          X[8 * x + i + 1] = z.y;
        }
      }
      fence_before_sync();
    }
    if (p.last && k < p.dk) {
      float* l = p.last + sbase;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (vx + i < p.dv)
          l[!kStates && p.first_swapped ? (size_t)k * p.dv + vx + i : (size_t)(vx + i) * p.dk + k] = X[i];
    }
  }
  if (!kStates) {
    // whole chunks of the segment past the row's end
    const int z0 = max(c1, c0) * kQ, z1 = min((c0 + p.seg_chunks) * kQ, p.T);
    const int esz = kF32 ? 4 : 2, at = (tid & 31) * 16, row = min(kV, p.dv - v0) * esz;
    uint8_t* o = (uint8_t*)p.o + (((size_t)b * p.T * p.H + h) * p.dv + v0) * esz + at;
    if (at < row)
#pragma unroll 1
      for (int t = z0 + warp; t < z1; t += kThreads / 32)
        *(uint4*)(o + (size_t)t * p.H * p.dv * esz) = make_uint4(0, 0, 0, 0);
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
  // what follows on the stream has to find the kernel before this one finished too
  if (p.beside && tid == 0) grid_dep_wait();
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

template <int DK, bool kStates, bool kF32>
cudaError_t launch(const Maps& m, const TcWalk& p, cudaStream_t s) {
  constexpr size_t smem = Geom<DK, kStates>::smem;
  static_assert(smem + sizeof(Bars) + 1024 <= 232448, "shared memory of a CTA");
  auto kernel = k_la_walk_tc<DK, kStates, kF32>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "linattn_states" : p.reverse ? "linattn_walk_back" : "linattn_walk", s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.H * ((p.dv + kV - 1) / kV), p.B, p.nseg);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, m, p);
}

template <bool kStates, bool kF32>
cudaError_t launch_d(const Maps& m, const TcWalk& p, cudaStream_t s) {
  return p.dk <= 64 ? launch<64, kStates, kF32>(m, p, s) : launch<128, kStates, kF32>(m, p, s);
}

}  // namespace

// one CTA an SM
static int la_tc_segments(int B, int H, int T, int dv) {
  return la_segments((long long)B * H * ((dv + kV - 1) / kV), (T + kQ - 1) / kQ, 152);
}

size_t la_tc_scratch_floats(int B, int H, int T, int dk, int dv) {
  // (the walks of a backward pass have dk and dv in either order)
  const int a = la_tc_segments(B, H, T, dv), b = la_tc_segments(B, H, T, dk), n = a > b ? a : b;
  return n > 1 ? (size_t)n * B * H * dk * dv : 0;
}

cudaError_t la_walk_tc(const LaWalk& w, bool beside, float* scratch, cudaStream_t s) {
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
  p.s_intra = w.s_intra;
  p.s_carry = w.s_carry;
  p.s_inject = w.s_inject;
  p.off = w.off;
  p.reverse = w.reverse;
  const int nc = (w.T + kQ - 1) / kQ;
  int n = la_tc_segments(w.B, w.H, w.T, w.dv);
  p.seg_chunks = (nc + n - 1) / n;
  n = (nc + p.seg_chunks - 1) / p.seg_chunks;
  p.nseg = n;
  p.first = w.first;
  p.last = w.last;
  p.first_swapped = w.first_swapped;
  if (n > 1) {
    p.last = scratch;
    cudaError_t e = launch_d<true, false>(m, p, s);
    if (e != cudaSuccess) return e;
    const LaSegments g = {w.B, w.H, w.T, w.dk, w.dv, n, p.seg_chunks * kQ, w.log_decay, w.lens,
                          scratch, w.first, w.last, w.first_swapped, w.reverse};
    if ((e = la_segment_states(g, s)) != cudaSuccess) return e;
    p.first = scratch;
    p.first_swapped = 0;
    p.last = nullptr;
  } else {
    p.beside = beside;
  }
  return w.o_f32 ? launch_d<false, true>(m, p, s) : launch_d<false, false>(m, p, s);
}

cudaError_t la_read_and_clear_error(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_la_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_la_error, &zero, sizeof(unsigned int));
}

}  // namespace ssd
