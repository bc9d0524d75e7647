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
// second product) and X once as an operand; the output is bf16 itself.  Together
// 0.0023 of the outputs' root mean square, 0.0017 from the last rounding alone;
// a second part of P and of X would double the products of O and Oc.  The
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
// Measured: 2.5 us a chunk at dk = 128, of which 1.6 us remain with the work
// taken out, the hand-overs between the warps; 45 us for 4 x 2048 steps of 32
// heads 128/64 (68 % of the copy rate, 128 CTAs on 152 SMs), 87 % for 4 x 8192
// steps of 38 heads.
//
// Rows past the end of a batch row (its length, or T) take part as zeros: TMA
// fills what lies past T; between a shorter row's end and T warps 0-7 clear
// the tile's rows before any product reads them.
#include <cuda.h>
#include <cuda_bf16.h>

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
  CUtensorMap q, k, v, o, hist;
};

// What of a walk a kernel needs.
struct TcWalk {
  int B, T, H, dk, dv;
  int qs, ks, vs;  // heads that share an operand's head
  int nseg, seg_chunks;
  const float* log_decay;
  const float* first;  // state before the row (nseg == 1) or before each segment
  float* last;         // state after it; after each segment alone in a states walk
  const int* lens;
  void* o;
  float s_intra, s_carry, s_inject;
  int off, reverse;
  int hist;    // X before every chunk goes to maps.hist (see Hist)
  int beside;  // launched beside the kernel before it, whose end it waits for last
  int early;   // the kernel launched after it is such a one and may start with it
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
// (64 columns, as many rows as the map's box has)
__device__ __forceinline__ void tma_store_rows(const void* tmap, const void* src, long long row) {
  tma_store_2d(tmap, src, 0, (int)row);
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
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// NS: stages of the loads; NW: buffers of a piece's three parts.  The sums
// stay below the 227 KB of a CTA.
template <int DK, bool kStates>
struct Geom {
  static constexpr int NS = kStates || DK == 64 ? 3 : 2;
  static constexpr int NW = kStates || DK == 64 ? 4 : 2;
  static constexpr int QT = DK * 256, VT = kV * 256;  // bytes of 128 rows
  static constexpr int WP = kPiece * 128;              // one part of a piece
  static constexpr int kQo = 0;
  static constexpr int kKo = kStates ? 0 : NS * QT;
  static constexpr int kVo = kKo + NS * QT;
  static constexpr int kWo = kVo + NS * VT;
  static constexpr int kXo = kWo + NW * 3 * WP;
  static constexpr int kSo = kXo + DK * kV * 2;
  static constexpr int kDo = kSo + (kStates ? 0 : 16384);  // (o is staged at kSo)
  static constexpr int kBytes = kDo + (kStates ? 0 : 32 * kDiagRow * 4);  // kDiagRow floats a row
  static constexpr size_t smem = kBytes + 1024;
};

// States before every chunk, bf16: [B][chunks][H][blocks of 64 columns of v][DK]
// rows of 64 (DK: dk rounded up to 64 or 128).
__host__ __device__ inline long long hist_row(int B, int nc, int H, int vblocks, int DK, int b, int c,
                                              int h, int vb) {
  return ((((long long)b * nc + c) * H + h) * vblocks + vb) * DK;
}

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
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitClocks) {
      *abort = 1;
      atomicOr(&g_la_error, 1u);
      return false;
    }
  }
}
template <typename B>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, B* bars) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, &bars->abort);
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

// kStates: only the states (K, V, U, X); each segment from zero, or with a
// history to be written from the state before it.
template <int DK, bool kStates>
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
  // (only where the kernel behind it is known to need nothing of this one: a
  // kernel of another call may read what this one writes)
  if (p.early) grid_dep_launch();
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
  auto history = [&](int it) {  // row of the state before chunk `it` of the walk
    return hist_row(p.B, (p.T + kQ - 1) / kQ, p.H, vblocks, DK, b, chunk(it), h, v0 / kV);
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
      if (!all_wait(&B->x, ph)) break;
      if (p.hist && lead) {
        tma_store_rows(&maps.hist, sm + G::kXo, history(it));
        bulk_commit();
      }
      __syncwarp();
      if (!all_wait(&B->fullQ[s], full)) break;
      fence_after_sync();
      const uint64_t dQ = dQ0 + s * (G::QT >> 4);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk)
        mma_ss(lead, tm + cC, dQ + ((kk >> 2) * 1024 + (kk & 3) * 2), dX + 128 * kk, id_x, kk > 0);
      if (p.hist && lead) bulk_wait_read0();
      __syncwarp();
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
    if (kStates && p.hist)  // the states of a states walk, which forms no Oc
#pragma unroll 1
      for (int it = 0; it < nit; ++it) {
        if (!all_wait(&B->x, it & 1)) break;
        if (lead) {
          tma_store_rows(&maps.hist, sm + G::kXo, history(it));
          bulk_commit();
          bulk_wait_read0();
          mbar_arrive(&B->xfree);
        }
        __syncwarp();
      }
    if (p.hist && lead) bulk_wait0();
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
      uint32_t y[16];  // this thread's 32 columns of o, bf16 in pairs
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
              y[8 * z + j / 2] = pack_bf16(a.x, a.y);
            }
          }
          if (n < kQ && row >= n) {
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = 0;
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
      // o, staged as 128 rows of 64 columns (both halves of the threads)
      uint8_t* st = sm + G::kSo;
      if (tid == 0) bulk_wait_read0();
      named_sync(1, 256);
      if (ok)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(uint4*)(st + sw128(row, hf * 4 + j)) =
              make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      fence_async_smem();
      named_sync(1, 256);
      if (tid == 0 && ok) {
        tma_store_4d(&maps.o, st, v0, h, chunk(it - 1) * kQ, b);
        bulk_commit();
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
    if ((!kStates || p.hist) && p.first && k < p.dk) {
      const float* f = p.first + sbase;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (vx + i < p.dv)
          X[i] = f[(size_t)(vx + i) * p.dk + k];
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
      if (!kStates || p.hist) {  // X before this chunk, for its Oc and the history
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
          l[(size_t)(vx + i) * p.dk + k] = X[i];
    }
  }
  if (!kStates) {
    // whole chunks of the segment past the row's end
    const int z0 = max(c1, c0) * kQ, z1 = min((c0 + p.seg_chunks) * kQ, p.T);
    const int at = (tid & 31) * 16, row = min(kV, p.dv - v0) * 2;
    uint8_t* o = (uint8_t*)p.o + (((size_t)b * p.T * p.H + h) * p.dv + v0) * 2 + at;
    if (at < row)
#pragma unroll 1
      for (int t = z0 + warp; t < z1; t += kThreads / 32)
        *(uint4*)(o + (size_t)t * p.H * p.dv * 2) = make_uint4(0, 0, 0, 0);
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


// ---- dq and dk ------------------------------------------------------------------
//
// dq (and with exchanged roles dk) of a group is a sum over its heads, of which
// there may be one; with the states before every chunk at hand the chunks are
// independent, and the sum is formed where the products accumulate:
//   out = sum over heads  P_h C + (lead_h o A_h) X_h^T,   P_h = mask_h(A_h B_h^T)
// with dq: A = do, B = v, C = k, X = the forward's states, mask i >= j;
//      dk: A = v, B = do, C = q, X = the backward's states, mask i <= j
// (the states' rows are k, so X_h^T has the width of C).  A unit is a (group,
// row, chunk, gradient); its items are the heads and 64-column blocks of v.  out
// stays in TMEM until the last of them and is rounded once.  A walk of every head
// would write its part in fp32 for a second kernel to add up: 2 x 537 MB written
// and read for 2 x 8192 steps, 64 heads in 8 groups.
//
// Precision: P is rounded to bf16 once, X once (in the history); lead o A is
// carried in two bf16 parts.
//
// One CTA an SM goes over units (the two gradients of a chunk are neighbours and
// share v and do in L2).  Warps as in the walk: 0-7 turn T = A B^T into P, in
// place, 8-15 form lead o A and write out of the unit before, one each loads,
// forms T and accumulates; two stages of items, two of C and two of out keep them
// apart.  Per item 48 KB are loaded and 1430 cycles of products issued.  Measured
// (128/64): 89 us for 4 x 2048 steps, 32 heads of their own q and k, of 165 for
// all gradients (three walks: 183); 233 us for 2 x 8192 steps, 64 heads in 8
// groups, of 473 (walks of every head with a kernel for the sums: 876).
struct Grad {
  int B, T, H, dk, dv, share, nc;  // heads of a group, chunks of a row
  const float* log_decay;
  const int* lens;
  struct Role {
    void* out;              // [B][T][H / share][dk]
    float s_intra, s_carry;
    int off, reverse;
  } role[2];
};
struct GradMaps {
  struct Role {
    CUtensorMap a, b, c, x, out;
  } role[2];
};

template <int DK>
struct GradGeom {
  static constexpr int VT = kV * 256, CT = DK * 256, XT = DK * 128;
  static constexpr int kCo = 0;                      // two stages of C
  static constexpr int kSto = kCo + 2 * CT;          // two stages of A, B, X
  static constexpr int kStage = 2 * VT + XT;
  static constexpr int kHo = kSto + 2 * kStage;      // lead o A: two parts
  static constexpr int kOo = kHo + 2 * VT;           // out is staged here
  static constexpr int kBytes = kOo + CT;
  static constexpr size_t smem = kBytes + 1024;
};
constexpr int gT = 0, gOut = 256;  // TMEM: two of 128 columns each

struct GradBars {
  uint64_t full[2], empty[2], c[2], cempty[2], t[2], half[2], p[2], pfree[2], hat, hatfree, out[2], outfree[2],
      fix[2], drain[2];
  uint32_t tmem;
  volatile int abort;
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
k_la_grad_tc(const __grid_constant__ GradMaps maps, const __grid_constant__ Grad g) {
  using G = GradGeom<DK>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = align1024(raw);
  __shared__ GradBars bars;
  GradBars* B = &bars;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int vblocks = (g.dv + kV - 1) / kV, items = g.share * vblocks, groups = g.H / g.share;
  const int units = 2 * g.nc * g.B * groups;
  const uint32_t lead = (tid & 31) == 0;
  auto all_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity, B)) != 0;
  };
  struct Unit {
    int role, c, grp, b, n;  // n: steps of the chunk that the row has (<= 0: none)
    bool ragged;             // rows past the row's end, not past T
  };
  auto unit = [&](int w) {
    Unit u;
    u.role = w & 1;
    u.c = (w >> 1) % g.nc;
    const int rg = (w >> 1) / g.nc;
    u.grp = rg % groups;
    u.b = rg / groups;
    int len = g.T;
    if (g.lens) len = __shfl_sync(__activemask(), min(max(g.lens[u.b], 0), g.T), 0);
    u.n = min(kQ, len - u.c * kQ);
    u.ragged = u.n < kQ && len < g.T;
    return u;
  };
  // Every role goes over the same units and items; `it` counts the items and
  // `w` the units that have steps.
  if (tid == 19 * 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
      mbar_init(&B->c[i], 1);
      mbar_init(&B->cempty[i], 1);
      mbar_init(&B->t[i], 1);
      mbar_init(&B->half[i], 4);
      mbar_init(&B->p[i], 8);
      mbar_init(&B->pfree[i], 1);
      mbar_init(&B->out[i], 1);
      mbar_init(&B->outfree[i], 8);
      mbar_init(&B->fix[i], 8);
      mbar_init(&B->drain[i], 1);
    }
    mbar_init(&B->hat, 8);
    mbar_init(&B->hatfree, 1);
    B->abort = 0;
    fence_mbar_init();
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
    int it = 0, w = 0;
    bool go = true;
#pragma unroll 1
    for (int x = blockIdx.x; go && x < units; x += gridDim.x) {
      const Unit u = unit(x);
      if (u.n <= 0) continue;
      const GradMaps::Role& m = maps.role[u.role];
      const int ws = w & 1, t0 = u.c * kQ;
      go = all_wait(&B->cempty[ws], ((w >> 1) & 1) ^ 1);
      if (!go) break;
      if (lead) {
        mbar_expect_tx(&B->c[ws], G::CT);
        for (int d = 0; d < DK; d += 64)
          tma_load_4d(sm + G::kCo + ws * G::CT + d * 256, &m.c, d, u.grp, t0, u.b, &B->c[ws]);
      }
      ++w;
#pragma unroll 1
      for (int i = 0; i < items; ++i, ++it) {
        const int s = it & 1, h = u.grp * g.share + i / vblocks, vb = i % vblocks;
        go = all_wait(&B->empty[s], ((it >> 1) & 1) ^ 1);
        if (!go) break;
        if (lead) {
          uint8_t* d = sm + G::kSto + s * G::kStage;
          mbar_expect_tx(&B->full[s], G::kStage);
          tma_load_4d(d, &m.a, vb * kV, h, t0, u.b, &B->full[s]);
          tma_load_4d(d + G::VT, &m.b, vb * kV, h, t0, u.b, &B->full[s]);
          tma_load_2d(d + 2 * G::VT, &m.x, 0,
                      (int)hist_row(g.B, g.nc, g.H, vblocks, DK, u.b, u.c, h, vb), &B->full[s]);
        }
        __syncwarp();
      }
    }
    if (B->abort) {  // no copy may be in flight when the CTA ends
      const uint64_t lim = 50000000ull;
      for (int j = max(it - 2, 0); j < it; ++j) mbar_wait(&B->full[j & 1], (j >> 1) & 1, lim);
      for (int j = max(w - 2, 0); j < w; ++j) mbar_wait(&B->c[j & 1], (j >> 1) & 1, lim);
    }
    __syncwarp();
  } else if (warp == 17) {
    // ---- T = A B^T ----
    constexpr uint32_t id_t = idesc_bf16(128, 128, false, false);
    const uint64_t dA0 = desc_sw128(smem_u32(sm + G::kSto), 16, 1024);
    int it = 0;
    uint32_t fixes = 0;
    bool go = true;
#pragma unroll 1
    for (int x = blockIdx.x; go && x < units; x += gridDim.x) {
      const Unit u = unit(x);
      if (u.n <= 0) continue;
#pragma unroll 1
      for (int i = 0; i < items; ++i, ++it) {
        const int s = it & 1;
        const uint32_t ph = (it >> 1) & 1;
        go = all_wait(&B->full[s], ph);
        if (go && u.ragged) {
          go = all_wait(&B->fix[s], (fixes >> s) & 1);
          fixes ^= 1u << s;
        }
        // (the P that was formed in place of T two items ago has been used)
        if (go && it > 1) go = all_wait(&B->pfree[s], ph ^ 1);
        if (!go) break;
        fence_after_sync();
        const uint64_t dA = dA0 + s * (G::kStage >> 4), dB = dA + (G::VT >> 4);
#pragma unroll
        for (int kk = 0; kk < kV / 16; ++kk)
          mma_ss(lead, tm + gT + s * 128, dA + 2 * kk, dB + 2 * kk, id_t, kk > 0);
        commit_if(lead, &B->t[s]);
      }
    }
    commit_if(lead, &B->drain[0]);
    mbar_wait(&B->drain[0], 0, kWaitNs);
    __syncwarp();
  } else if (warp == 18) {
    // ---- out += (lead o A) X^T + P C ----
    constexpr uint32_t id_c = idesc_bf16(128, DK, false, true), id_x = idesc_bf16(128, DK, false, false);
    const uint64_t dC0 = desc_sw128(smem_u32(sm + G::kCo), 16384, 1024);
    const uint64_t dX0 = desc_sw128(smem_u32(sm + G::kSto + 2 * G::VT), 16, 1024);
    const uint64_t dH = desc_sw128(smem_u32(sm + G::kHo), 16, 1024);
    int it = 0, w = 0;
    bool go = true;
#pragma unroll 1
    for (int x = blockIdx.x; go && x < units; x += gridDim.x) {
      const Unit u = unit(x);
      if (u.n <= 0) continue;
      const int ws = w & 1;
      const uint32_t pw = (w >> 1) & 1, tO = tm + gOut + ws * 128;
      go = all_wait(&B->c[ws], pw) && (w < 2 || all_wait(&B->outfree[ws], pw ^ 1));
      if (!go) break;
      const uint64_t dC = dC0 + ws * (G::CT >> 4);
#pragma unroll 1
      for (int i = 0; i < items; ++i, ++it) {
        const int s = it & 1;
        const uint32_t ph = (it >> 1) & 1;
        go = all_wait(&B->hat, it & 1) && all_wait(&B->full[s], ph);
        if (!go) break;
        fence_after_sync();
        const uint64_t dX = dX0 + s * (G::kStage >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < kV / 16; ++kk)
            mma_ss(lead, tO, dH + part * (G::VT >> 4) + 2 * kk, dX + 2 * kk, id_x, i > 0 || part + kk > 0);
        commit_if(lead, &B->hatfree);
        go = all_wait(&B->p[s], ph);
        if (!go) break;
        fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(lead, tO, tm + gT + s * 128 + 8 * kk, dC + 128 * kk, id_c, 1);
        commit_if(lead, &B->pfree[s]);
        commit_if(lead, &B->empty[s]);
      }
      if (!go) break;
      commit_if(lead, &B->out[ws]);
      commit_if(lead, &B->cempty[ws]);
      ++w;
    }
    commit_if(lead, &B->drain[1]);
    mbar_wait(&B->drain[1], 0, kWaitNs);
    __syncwarp();
  } else if (warp < 8) {
    // ---- P: thread = row i and half of the columns ----
    const int row = tid & 127, il = row & 31, ib = warp & 3, hf = warp >> 2;
    const uint32_t lane_base = (uint32_t)(ib * 32) << 16;
    int it = 0, w = 0;
    uint32_t wph = 0;
    bool ok = true;
#pragma unroll 1
    for (int x = blockIdx.x; x < units; x += gridDim.x) {
      const Unit u = unit(x);
      const Grad::Role& r = g.role[u.role];
      if (u.n <= 0) {  // a chunk past the row's end
        const int row16 = g.dk / 8, rows = min(kQ, g.T - u.c * kQ);
        uint8_t* o = (uint8_t*)r.out + (((size_t)u.b * g.T + u.c * kQ) * groups + u.grp) * g.dk * 2;
#pragma unroll 1
        for (int i = tid; i < rows * row16; i += 256)
          *(uint4*)(o + (size_t)(i / row16) * groups * g.dk * 2 + (i % row16) * 16) = make_uint4(0, 0, 0, 0);
        continue;
      }
      // zeros into the rows past the row's end: of C once, of A and B of every item
      auto clear = [&](uint8_t* tile, int tiles) {
        if (row >= u.n)
#pragma unroll 1
          for (int y = 0; y < tiles * 4; ++y)
            *(uint4*)(tile + (y >> 2) * 16384 + row * 128 + hf * 64 + (y & 3) * 16) = make_uint4(0, 0, 0, 0);
      };
      const int ws = w & 1;
      wph = (w >> 1) & 1;
      ++w;
      if (u.ragged) {
        ok = __all_sync(0xffffffffu, ok && wait(&B->c[ws], wph, B));
        if (ok) clear(sm + G::kCo + ws * G::CT, DK / 64);
      }
#pragma unroll 1
      for (int i = 0; i < items; ++i, ++it) {
        const int s = it & 1;
        const uint32_t ph = (it >> 1) & 1;
        if (u.ragged) {
          ok = __all_sync(0xffffffffu, ok && wait(&B->full[s], ph, B));
          if (ok) {
            clear(sm + G::kSto + s * G::kStage, 2);
            fence_async_smem();
            warp_arrive(&B->fix[s]);
          }
        }
        // a^{|i-j|} = 2^{(i-j) la2}, la2 of the mask's sign (a decay below 2^-1e30
        // counts as that: its powers are 0 but for the power 0)
        const float la = g.log_decay[u.grp * g.share + i / vblocks];
        const float la2 = fmaxf(la * 1.4426950408889634f, -1e30f) * (r.reverse ? -1.f : 1.f);
        ok = __all_sync(0xffffffffu, ok && wait(&B->t[s], ph, B));
        fence_after_sync();
        // (P takes T's columns: a half overwrites T of its own blocks, or of block 1,
        // which the first half reads before the second half writes)
#pragma unroll 1
        for (int y = 0; y < 2; ++y) {
          const int jb = 2 * hf + y, dist = r.reverse ? jb - ib : ib - jb;
          uint32_t q[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) q[j] = 0;
          float v[32];
          if (ok && dist >= 0) {
            tmem_ld32(tm + gT + s * 128 + lane_base + jb * 32, v);
            tmem_wait_ld();
          }
          if (hf == 0 && y == 1 && ok) {
            fence_before_sync();
            warp_arrive(&B->half[s]);
          } else if (hf == 1 && y == 0) {
            ok = __all_sync(0xffffffffu, ok && wait(&B->half[s], ph, B));
            fence_after_sync();
          }
          if (ok && dist >= 0) {
            float d0 = (float)(32 * (ib - jb) + il);
            asm volatile("" : "+f"(d0));
            // (on the diagonal a later step has no part in this row, whatever its
            // product is)
            const uint32_t in = dist > 0 ? 0xffffffffu : r.reverse ? 0xffffffffu << il : 0xffffffffu >> (31 - il);
            const float si = r.s_intra;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float f = si * ex2((d0 - (float)j) * la2);
              v[j] = (in >> j) & 1 ? v[j] * f : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) q[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          }
          if (ok) tmem_st16(tm + gT + s * 128 + lane_base + jb * 16, q);
        }
        if (ok) {
          tmem_wait_st();
          fence_before_sync();
          warp_arrive(&B->p[s]);
        }
      }
    }
  } else if (warp < 16) {
    // ---- lead o A in two parts (thread = row of A and four of its eight chunks);
    // out of the unit before (thread = row and half of the columns) ----
    const int t = tid - 256, row = t & 127, hf = t >> 7;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    int it = 0, w = 0;
    uint32_t fixes = 0;
    bool ok = true;  // (after a wait that gave up the warps still meet at their barriers)
    Unit last = {};
    // out of unit number v, in 64-column tiles
    auto finish = [&](int v, const Unit& u) {
      const int ws = v & 1;
      ok = __all_sync(0xffffffffu, ok && wait(&B->out[ws], (v >> 1) & 1, B));
      fence_after_sync();
      if (t == 0) bulk_wait_read0();
      named_sync(3, 256);
      if (ok) {
#pragma unroll 1
        for (int z = 0; z < DK / 32; ++z) {  // 16 of this thread's columns at a time
          const int col = (z >> 1) * 64 + hf * 32 + (z & 1) * 16;
          float f[16];
          tmem_ld16(tm + gOut + ws * 128 + lane_base + col, f);
          tmem_wait_ld();
          if (row >= u.n)
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.f;
          uint8_t* st = sm + G::kOo + (z >> 1) * 16384;
          *(uint4*)(st + sw128(row, (col & 63) / 8)) = pack8(f);
          *(uint4*)(st + sw128(row, (col & 63) / 8 + 1)) = pack8(f + 8);
        }
        fence_before_sync();
        fence_async_smem();
        warp_arrive(&B->outfree[ws]);
      }
      named_sync(3, 256);
      if (t == 0 && ok) {
        for (int d = 0; d < g.dk; d += 64)
          tma_store_4d(&maps.role[u.role].out, sm + G::kOo + (d >> 6) * 16384, d, u.grp, u.c * kQ, u.b);
        bulk_commit();
      }
    };
#pragma unroll 1
    for (int x = blockIdx.x; x < units; x += gridDim.x) {
      const Unit u = unit(x);
      if (u.n <= 0) continue;
      const Grad::Role& r = g.role[u.role];
#pragma unroll 1
      for (int i = 0; i < items; ++i, ++it) {
        const int s = it & 1;
        const uint32_t ph = (it >> 1) & 1;
        const float la = g.log_decay[u.grp * g.share + i / vblocks];
        const float wt =
            row < u.n ? r.s_carry * decay_pow(la, (float)((r.reverse ? u.n - 1 - row : row) + r.off)) : 0.f;
        const float2 w2 = make_float2(wt, wt);
        bool in = ok && wait(&B->full[s], ph, B);
        if (u.ragged) {
          in = in && wait(&B->fix[s], (fixes >> s) & 1, B);
          fixes ^= 1u << s;
        }
        ok = __all_sync(0xffffffffu, in && (it == 0 || wait(&B->hatfree, (it - 1) & 1, B)));
        if (ok) {
          const uint8_t* src = sm + G::kSto + s * G::kStage;
          uint8_t* dst = sm + G::kHo;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t at = sw128(row, hf * 4 + q);
            float2 f[4], e[4];
            unpack8(*(const uint4*)(src + at), (float*)f);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], w2);
            const uint4 hi = pack8((const float*)f);
            unpack8(hi, (float*)e);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = fma2(e[j], make_float2(-1.f, -1.f), f[j]);
            *(uint4*)(dst + at) = hi;
            *(uint4*)(dst + G::VT + at) = pack8((const float*)f);
          }
          fence_async_smem();
          warp_arrive(&B->hat);
        }
        if (i == 0 && w > 0) finish(w - 1, last);
      }
      last = u;
      ++w;
    }
    if (w > 0) finish(w - 1, last);
    if (t == 0) bulk_wait0();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
}

// ---- host --------------------------------------------------------------------------

// [B][T][heads][D] with {128 bytes of D, one head, 128 steps, one row} boxes.
bool map_4d(CUtensorMap* m, const void* base, int D, int heads, int T, int B,
            long long step, long long batch) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = 2;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {D * e, (cuuint64_t)step * e, (cuuint64_t)batch * e};
  cuuint32_t box[4] = {64, 1, kQ, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of 64 bf16 with {64, box_rows} boxes
bool map_rows(CUtensorMap* m, const void* base, long long rows, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || rows > (1ll << 31) - 1) return false;
  cuuint64_t dims[2] = {64, (cuuint64_t)rows};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, bool kStates>
cudaError_t launch(const Maps& m, const TcWalk& p, cudaStream_t s) {
  constexpr size_t smem = Geom<DK, kStates>::smem;
  static_assert(smem + sizeof(Bars) + 1024 <= 232448, "shared memory of a CTA");
  auto kernel = k_la_walk_tc<DK, kStates>;
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

template <bool kStates>
cudaError_t launch_d(const Maps& m, const TcWalk& p, cudaStream_t s) {
  return p.dk <= 64 ? launch<64, kStates>(m, p, s) : launch<128, kStates>(m, p, s);
}

}  // namespace

// one CTA an SM
static int la_tc_segments(int B, int H, int T, int dv) {
  return la_segments((long long)B * H * ((dv + kV - 1) / kV), (T + kQ - 1) / kQ, kLaSms);
}

size_t la_tc_scratch_floats(int B, int H, int T, int dk, int dv) {
  const int n = la_tc_segments(B, H, T, dv);
  return n > 1 ? (size_t)n * B * H * dk * dv : 0;
}

long long la_tc_hist_rows(int B, int H, int T, int dk, int dv) {
  const int DK = dk <= 64 ? 64 : 128;
  return hist_row(B, (T + kQ - 1) / kQ, H, (dv + kV - 1) / kV, DK, B, 0, 0, 0);
}

cudaError_t la_grads_tc(const LaGrads& d, cudaStream_t s) {
  GradMaps m;
  Grad g = {};
  g.B = d.B;
  g.T = d.T;
  g.H = d.H;
  g.dk = d.dk;
  g.dv = d.dv;
  g.share = d.q.share;
  g.nc = (d.T + kQ - 1) / kQ;
  g.log_decay = d.log_decay;
  g.lens = d.lens;
  g.role[0] = {d.dq, d.scale, d.scale, 1, 0};
  g.role[1] = {d.dk_out, d.scale, 1.f, 0, 1};
  const LaOperand* a[2] = {&d.dout, &d.v};
  const LaOperand* b[2] = {&d.v, &d.dout};
  const LaOperand* c[2] = {&d.k, &d.q};
  const void* x[2] = {d.hist_s, d.hist_g};
  const int G = d.H / g.share, DK = d.dk <= 64 ? 64 : 128;
  const long long rows = la_tc_hist_rows(d.B, d.H, d.T, d.dk, d.dv);
  for (int i = 0; i < 2; ++i) {
    GradMaps::Role& r = m.role[i];
    if (!map_4d(&r.a, a[i]->p, d.dv, d.H, d.T, d.B, a[i]->step, a[i]->batch) ||
        !map_4d(&r.b, b[i]->p, d.dv, d.H, d.T, d.B, b[i]->step, b[i]->batch) ||
        !map_4d(&r.c, c[i]->p, d.dk, G, d.T, d.B, c[i]->step, c[i]->batch) ||
        !map_4d(&r.out, g.role[i].out, d.dk, G, d.T, d.B, (long long)G * d.dk,
                (long long)d.T * G * d.dk) ||
        !map_rows(&r.x, x[i], rows, DK))
      return cudaErrorNotSupported;
  }
  auto go = [&](auto kernel, size_t smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    LaunchScope ls("linattn_grads", s);
    const long long units = 2ll * g.nc * d.B * G;
    kernel<<<(unsigned)(units < kLaSms ? units : kLaSms), kThreads, smem, s>>>(m, g);
    return cudaGetLastError();
  };
  static_assert(GradGeom<128>::smem + 1024 <= 232448, "shared memory of a CTA");
  return DK == 64 ? go(k_la_grad_tc<64>, GradGeom<64>::smem) : go(k_la_grad_tc<128>, GradGeom<128>::smem);
}

cudaError_t la_walk_tc(const LaWalk& w, bool beside, float* scratch, cudaStream_t s) {
  Maps m;
  if (!map_4d(&m.q, w.q.p, w.dk, w.H / w.q.share, w.T, w.B, w.q.step, w.q.batch) ||
      !map_4d(&m.k, w.k.p, w.dk, w.H / w.k.share, w.T, w.B, w.k.step, w.k.batch) ||
      !map_4d(&m.v, w.v.p, w.dv, w.H / w.v.share, w.T, w.B, w.v.step, w.v.batch) ||
      (w.o && !map_4d(&m.o, w.o, w.dv, w.H, w.T, w.B, (long long)w.H * w.dv,
                      (long long)w.T * w.H * w.dv)))
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
  if (n > 1) {
    p.last = scratch;
    cudaError_t e = launch_d<true>(m, p, s);
    if (e != cudaSuccess) return e;
    const LaSegments g = {w.B, w.H, w.T, w.dk, w.dv, n, p.seg_chunks * kQ, w.log_decay, w.lens,
                          scratch, w.first, w.last, false, w.reverse};
    if ((e = la_segment_states(g, s)) != cudaSuccess) return e;
    p.first = scratch;
    p.last = nullptr;
  } else {
    p.beside = beside;
    p.early = w.followed;
  }
  if (w.hist) {
    const int DK = w.dk <= 64 ? 64 : 128;
    if (!map_rows(&m.hist, w.hist, la_tc_hist_rows(w.B, w.H, w.T, w.dk, w.dv), DK))
      return cudaErrorNotSupported;
    p.hist = 1;
    if (!w.o) return launch_d<true>(m, p, s);  // the states alone
  }
  return launch_d<false>(m, p, s);
}

// Two warps wait on a barrier that nothing arrives on: one gives up after
// kWaitClocks and sets the error word, the other follows it by the abort word.
static __global__ void k_la_selftest_wait() {
  __shared__ struct {
    uint64_t bar;
    volatile int abort;
  } w;
  if (threadIdx.x == 0) {
    mbar_init(&w.bar, 1);
    w.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  (void)wait(&w.bar, 0, &w);
}

cudaError_t la_selftest_timeout(cudaStream_t s) {
  LaunchScope ls("linattn_selftest_wait", s);
  k_la_selftest_wait<<<1, 64, 0, s>>>();
  return cudaGetLastError();
}

cudaError_t la_read_and_clear_error(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_la_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_la_error, &zero, sizeof(unsigned int));
}

}  // namespace ssd
