// Linear attention with a decay for each head: the walk over the steps of a
// row (forward, and with exchanged roles the gradients), the sum over a
// group's heads, and the step of one token.
//
// With a = e^{log_decay_h} and chunks of C steps, S the state before a chunk
// and positions i, j inside it,
//   o_i = s sum_{j <= i} a^{i-j} (q_i . k_j) v_j + s a^{i+1} S q_i
//   S  <- a^C S + sum_j a^{C-1-j} v_j k_j^T
// which is the recurrence S_t = a S_{t-1} + v_t k_t^T, o_t = s S_t q_t
// regrouped.  The gradients of L = sum(do . o) + sum(dS . S_T) are
//   dq_i = s sum_{j <= i} a^{i-j} (do_i . v_j) k_j + s a^{i+1} S0^T do_i
//   dk_j = s sum_{i >= j} a^{i-j} (v_j . do_i) q_i + a^{T-1-j} dS^T v_j
//   dv_j = s sum_{i >= j} a^{i-j} (k_j . q_i) do_i + a^{T-1-j} dS k_j
//   dS0  = a^T dS + s sum_i a^{i+1} do_i q_i^T
// i.e. the same walk with the operands' roles exchanged, the last three from
// the last step back (off = 0: the incoming dS belongs to the last step
// itself, not to the one before the first).
#include "f32x2.cuh"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

// a^e for e >= 0 from log a; a^0 = 1 also where a = 0 (log a = -inf)
__device__ __forceinline__ float decay_pow(float la, float e) { return e == 0.f ? 1.f : expf(la * e); }

// ---- the walk in fp32 -----------------------------------------------------------
//
// One CTA per (h, 32 columns of v, b, segment of the row), chunks of 64 steps,
// eight warps.  Of rows 16 w ... 16 w + 15 of a chunk, two warps form
//   u = Q X,  S = Q K^T,  P = mask(S),  o = lead u + P V
// each for every other eight columns of S and 16 columns of u, and add up the
// halves of P V; and of the state's rows k a quarter, 16 columns of v each, of X =
// a^n X + K^T w V, which stays in registers.  P does too: the layout in which the
// matrix instructions leave S is the one in which they take P as a left operand,
// with the steps j of eight taken in the order that ja, jb below give.  Columns
// that the mask empties for all of a warp's rows are left out; a scheduler's two
// warps have rows w and 3 - w, with as many such columns together.
//
// Precision: the operands have 24 significant bits and the matrix instructions
// take 11 (tf32), so each operand x is hi + lo, hi = x rounded to 11 bits, lo the
// exact rest, of which the 11 leading bits count; x y is lo_x hi_y + hi_x lo_y +
// hi_x hi_y in fp32, with an error of a few 2^-22 of the product at most.  (An
// infinity, or a number that rounds to one in 11 bits, has no such parts and gives
// NaN; below 2^-102 or so lo loses bits to fp32's smallest numbers.)
//
// Why not on the CUDA cores: their operands come from shared memory for every
// 4 x 4 block of products that a thread's registers hold, 16 bytes a lane and so
// four cycles of the SM's 128 bytes each, and that bounded them: 271 us on
// 8 x 1024 steps, 24 heads of 64/64, and 247 with two products an instruction.
// A matrix instruction's operands are spread over the warp, an eighth of those
// bytes: 170 us.  No one unit bounds it now: taking operands apart is half of the
// instructions (they fill 58 % of the issue slots), the matrix pipes are 43 %
// busy, and 384 CTAs put three on some SMs and two on others.  Four warps a CTA
// that form whole rows took 168 us, but 346 us instead of 310 for heads of
// 128/64, where fewer CTAs fit an SM, and 18.5 instead of 14.6 for 4 x 1000
// steps of 3 heads of 32/32.
//
// Rows of shared memory are 8 floats apart in the banks (K, Q, X: two floats a
// lane of rows 0-3 and 4-7; V and K read across rows t, or ja and jb, and
// eight columns), so that no access conflicts.
constexpr int kC = 64;         // steps of a chunk
constexpr int kB = 32;         // columns of v of a CTA
constexpr int kThreads = 256;

template <int DK, bool kStates>
struct Walk32 {
  static constexpr int LK = DK + 8;
  static constexpr int LV = kB + 8;
  static constexpr int kFloats = kC * LK + kC * LV + (kStates ? 0 : kC * LK + kB * LK);
  static constexpr size_t smem = kFloats * sizeof(float);
};

struct Walk32Args {
  LaWalk w;
  int nseg, span;  // steps of a segment
};

// 16 bytes, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// N operands of a lane as hi + lo
template <int N>
struct Parts {
  uint32_t hi[N], lo[N];
  __device__ __forceinline__ void set(int i, float x) {
    hi[i] = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo[i] = __float_as_uint(x - __uint_as_float(hi[i]));
  }
};

// d = a b + c
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2],
                                         float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(c1),
        "f"(c2), "f"(c3));
}
// c[i] += a b[i] for N tiles, 16 x 8 times 8 x 8.  With g = lane / 4, t = lane %
// 4: a holds rows g, g + 8 of terms t, then of terms t + 4; b terms t, t + 4 of
// column g; c row g, columns 2 t and 2 t + 1, then row g + 8.  The tiles take
// turns, since an instruction waits for the one before it on the same sum.
//
// The instructions round their sums toward zero, which over a long sum adds up
// (2.6e-6 of the outputs after 1024 steps, where the plain form has 3e-7), so
// theirs start from zero, the small terms first, and are added to c outside.
template <int N>
__device__ __forceinline__ void mma_fp32(float (*c)[4], const Parts<4>& a, const Parts<2> (&b)[N]) {
  float d[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i) mma_tf32(d[i], a.lo, b[i].hi, 0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) mma_tf32(d[i], a.hi, b[i].lo, d[i][0], d[i][1], d[i][2], d[i][3]);
#pragma unroll
  for (int i = 0; i < N; ++i) mma_tf32(d[i], a.hi, b[i].hi, d[i][0], d[i][1], d[i][2], d[i][3]);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 f = add2(make_float2(c[i][e], c[i][e + 1]), make_float2(d[i][e], d[i][e + 1]));
      c[i][e] = f.x;
      c[i][e + 1] = f.y;
    }
}
// the same with the right operands of N tiles `step` floats apart at p: terms 2 t
// and 2 t + 1 of a row
template <int N>
__device__ __forceinline__ void mma_rows(float (*c)[4], const Parts<4>& a, const float* p, int step) {
  Parts<2> b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = *(const float2*)(p + i * step);
    b[i].set(0, f.x);
    b[i].set(1, f.y);
  }
  mma_fp32<N>(c, a, b);
}

// kStates: only the state, each segment from zero, into w.last
// [nseg][B][H][dv][dk].
template <int DK, bool kStates>
__global__ void __launch_bounds__(kThreads, DK == 64 ? 3 : 2)
k_la_walk(const __grid_constant__ Walk32Args args) {
  using G = Walk32<DK, kStates>;
  constexpr int LK = G::LK, LV = G::LV;
  constexpr int NX = DK / 32;  // eights of rows k of a warp
  constexpr int LE = 24;
  const LaWalk& w = args.w;
  extern __shared__ __align__(16) float sm[];
  float* K = sm;
  float* V = K + kC * LK;
  float* Q = V + kC * LV;
  float* X = Q + kC * LK;  // [v][k]
  __shared__ float pw[kC + 2];
  const int vblocks = (w.dv + kB - 1) / kB;
  const int h = blockIdx.x / vblocks, v0 = (blockIdx.x % vblocks) * kB;
  const int b = blockIdx.y, seg = blockIdx.z, t = threadIdx.x;
  const int half = t >> 7, wp = half ? 3 - (t >> 5 & 3) : t >> 5;
  const int g = (t & 31) >> 2, t4 = t & 3;
  const int ja = 2 * t4 + (t4 >> 1), jb = 2 * t4 + 1 - (t4 >> 1);  // columns 2 t, 2 t + 1 of S
  const int jg = g ^ (g >> 2);                                     // column g of S
  const float la = w.log_decay[h];
  int len = w.T;
  if (w.lens) len = min(max(w.lens[b], 0), w.T);
  if (t < kC + 2) pw[t] = decay_pow(la, (float)t);
  const int dv = min(kB, w.dv - v0);
  const size_t sbase = (((size_t)seg * w.B + b) * w.H + h) * w.dv * w.dk;
  // state element (k, v)
  auto state_at = [&](int k, int v) {
    return sbase + (!kStates && w.first_swapped ? (size_t)k * w.dv + v0 + v : (size_t)(v0 + v) * w.dk + k);
  };
  // x[i][c]: v = vx (+ 8 for c >= 2), k = kx + 8 i (+ 1 for odd c)
  const int vx = 16 * half + g, kx = wp * (DK / 4) + 2 * t4;
  float x[NX][4];
#pragma unroll
  for (int i = 0; i < NX; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int v = vx + 8 * (c >> 1), k = kx + 8 * i + (c & 1);
      x[i][c] = !kStates && w.first && k < w.dk && v < dv ? w.first[state_at(k, v)] : 0.f;
    }
  const float* qp = (const float*)w.q.p + b * w.q.batch + (long long)(h / w.q.share) * w.dk;
  const float* kp = (const float*)w.k.p + b * w.k.batch + (long long)(h / w.k.share) * w.dk;
  const float* vp = (const float*)w.v.p + b * w.v.batch + (long long)(h / w.v.share) * w.dv + v0;
  float* op = (float*)w.o + ((long long)b * w.T * w.H + h) * w.dv + v0;
  const int s0 = seg * args.span, s1 = min(s0 + args.span, len);  // the segment's steps
  const int nc = s1 > s0 ? (s1 - s0 + kC - 1) / kC : 0;
  for (int ci = 0; ci < nc; ++ci) {
    const int t0 = s0 + (w.reverse ? nc - 1 - ci : ci) * kC, n = min(kC, s1 - t0);
    __syncthreads();
#pragma unroll 4
    for (int i = t; i < kC * (DK / 4); i += kThreads) {
      const int r = i / (DK / 4), d = i % (DK / 4) * 4;
      const bool in = r < n && d < w.dk;
      if (!kStates) copy16(Q + r * LK + d, in ? qp + (long long)(t0 + r) * w.q.step + d : qp, in);
      copy16(K + r * LK + d, in ? kp + (long long)(t0 + r) * w.k.step + d : kp, in);
    }
#pragma unroll
    for (int i = t; i < kC * (kB / 4); i += kThreads) {
      const int r = i / (kB / 4), d = i % (kB / 4) * 4;
      const bool in = r < n && d < dv;
      copy16(V + r * LV + d, in ? vp + (long long)(t0 + r) * w.v.step + d : vp, in);
    }
    if (!kStates)
#pragma unroll
      for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *(float2*)(X + (vx + 8 * u) * LK + kx + 8 * i) = make_float2(x[i][2 * u], x[i][2 * u + 1]);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!kStates) {
      // o[0], o[1]: columns 16 half ... of o, which this warp writes; o[2], o[3]:
      // the other half's.  s[j]: columns 16 j + 8 half ... of S
      float o[4][4], s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] = s[i][c] = 0.f;
      // columns 16 j ... of S are needed by this warp
      auto needed = [&](int j) { return w.reverse ? j >= wp : j <= wp; };
      const float* qr = Q + (16 * wp + g) * LK + 2 * t4;
#pragma unroll 2
      for (int d = 0; d < DK; d += 8) {
        const float2 q0 = *(const float2*)(qr + d), q1 = *(const float2*)(qr + 8 * LK + d);
        Parts<4> a;
        a.set(0, q0.x);
        a.set(1, q1.x);
        a.set(2, q0.y);
        a.set(3, q1.y);
        mma_rows<2>(o, a, X + vx * LK + d + 2 * t4, 8 * LK);
        const float* kr = K + (8 * half + jg) * LK + d + 2 * t4;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          if (needed(j) && needed(j + 1)) mma_rows<2>(s + j, a, kr + 16 * j * LK, 16 * LK);
          else if (needed(j)) mma_rows<1>(s + j, a, kr + 16 * j * LK, 0);
          else if (needed(j + 1)) mma_rows<1>(s + j + 1, a, kr + 16 * (j + 1) * LK, 0);
        }
      }
      const int i0 = 16 * wp + g;  // this lane's rows: i0, i0 + 8
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = min(i0 + 8 * u, n - 1);  // (a row past the end is not written)
        const float lead = w.s_carry * pw[(w.reverse ? n - 1 - i : i) + w.off];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          o[e][2 * u] *= lead;
          o[e][2 * u + 1] *= lead;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (needed(j)) {
          const int j0 = 16 * j + 8 * half;
          Parts<4> a;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = i0 + 8 * (c >> 1), col = j0 + (c & 1 ? jb : ja);
            const int d = w.reverse ? col - i : i - col;
            a.set((c >> 1) + 2 * (c & 1), d >= 0 ? w.s_intra * pw[d] * s[j][c] : 0.f);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int v = 16 * (u ? 1 - half : half) + g;
            const float *va = V + (j0 + ja) * LV + v, *vb = V + (j0 + jb) * LV + v;
            Parts<2> p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              p[e].set(0, va[8 * e]);
              p[e].set(1, vb[8 * e]);
            }
            mma_fp32<2>(o + 2 * u, a, p);
          }
        }
      // the halves' sums, exchanged in place of the rows of Q (the two warps')
      float* E = Q + 16 * wp * LK + g * LE + 2 * t4;
      auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + wp) : "memory"); };
      pair_sync();
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *(float2*)(E + (16 * half + 8 * u) * LE + 8 * e) = make_float2(o[2 + e][2 * u], o[2 + e][2 * u + 1]);
      pair_sync();
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (i0 + 8 * u < n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (16 * half + 8 * e < dv) {
              const float2 f = *(const float2*)(E + (16 * (1 - half) + 8 * u) * LE + 8 * e);
              *(float2*)(op + (long long)(t0 + i0 + 8 * u) * w.H * w.dv + 16 * half + 8 * e + 2 * t4) =
                  make_float2(o[e][2 * u] + f.x, o[e][2 * u + 1] + f.y);
            }
    }
    const float an = pw[n];
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i][c] *= an;
#pragma unroll 2
    for (int j = 0; j < n; j += 8) {  // (rows past n are zero)
      Parts<4> a;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = j + t4 + 4 * u;
        const float f = w.s_inject * pw[max(w.reverse ? r : n - 1 - r, 0) + 1 - w.off];
        const float* vr = V + r * LV + vx;
        a.set(2 * u, f * vr[0]);
        a.set(2 * u + 1, f * vr[8]);
      }
      const float* kr = K + (j + t4) * LK + wp * (DK / 4) + g;
      Parts<2> k[NX];
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        k[i].set(0, kr[8 * i]);
        k[i].set(1, kr[4 * LK + 8 * i]);
      }
      mma_fp32<NX>(x, a, k);
    }
  }
  if (!kStates) {  // past the row's end
    const int z0 = max(s0, min(len, s0 + args.span)), z1 = min(s0 + args.span, w.T);
    const int d = t % (kB / 4) * 4;
    if (d < dv)
      for (int r = z0 + t / (kB / 4); r < z1; r += kThreads / (kB / 4))
        *(float4*)(op + (long long)r * w.H * w.dv + d) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (w.last)
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int v = vx + 8 * (c >> 1), k = kx + 8 * i + (c & 1);
        if (k < w.dk && v < dv) w.last[state_at(k, v)] = x[i][c];
      }
}

// The states before each segment from the segments' own: in walk order
//   X_0 = first, X_{s+1} = a^{steps of s} X_s + local_s;  last = X_nseg.
// seg [nseg][B][H][dv][dk], overwritten in place.
__global__ void __launch_bounds__(256) k_la_segments(const LaSegments p) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int i = blockIdx.x * 256 + threadIdx.x, n = p.dk * p.dv;
  if (i >= n) return;
  const float la = p.log_decay[h];
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const size_t row = ((size_t)b * p.H + h) * n, stride = (size_t)p.B * p.H * n;
  const size_t at = row + (p.swapped ? (size_t)(i % p.dk) * p.dv + i / p.dk : (size_t)i);
  float x = p.first ? p.first[at] : 0.f;
  for (int j0 = 0; j0 < p.nseg; j0 += 8) {
    float local[8];  // read ahead: the loads do not wait for one another
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int s = p.reverse ? p.nseg - 1 - j0 - u : j0 + u;
      local[u] = j0 + u < p.nseg ? p.seg[s * stride + row + i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + u >= p.nseg) break;
      const int s = p.reverse ? p.nseg - 1 - j0 - u : j0 + u;
      const int steps = min(max(len - s * p.span, 0), p.span);
      p.seg[s * stride + row + i] = x;
      x = fmaf(decay_pow(la, (float)steps), x, local[u]);
    }
  }
  if (p.last) p.last[at] = x;
}

template <int DK, bool kStates>
cudaError_t walk_t(const Walk32Args& a, cudaStream_t s) {
  constexpr int smem = (int)Walk32<DK, kStates>::smem;
  cudaError_t e = cudaFuncSetAttribute(k_la_walk<DK, kStates>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls(kStates ? "linattn_states" : a.w.reverse ? "linattn_walk_back" : "linattn_walk", s);
  const int vblocks = (a.w.dv + kB - 1) / kB;
  k_la_walk<DK, kStates><<<dim3(a.w.H * vblocks, a.w.B, a.nseg), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

// part [rows][G][share][D] -> out [rows][G][D]
__global__ void k_la_group_sum(long long n, int share, int D, const float* __restrict__ part,
                               float* __restrict__ out) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const float* p = part + i / D * share * D + i % D;
    float s = 0.f;
    for (int j = 0; j < share; ++j) s += p[(long long)j * D];
    out[i] = s;
  }
}

// One token: S' = a S + v k^T, o = s S' q.  A row of the state (dk floats) is
// held by LPR lanes, four floats each; a warp takes NR rows a lane at once, so
// that as many 16-byte loads are in flight, and adds the NR dot products up
// together: while a lane holds several, each exchange halves them (lanes of one
// half keep one half of the values), nine exchanges for eight sums over 32
// lanes instead of forty.
//
// Bound by the states' bytes, read and written once.  Measured on 256 rows of
// 64 heads, 128 x 64 (1.08 GB): 191 us with one row a lane at a time and sixteen
// rows a CTA, 160 us with eight.
constexpr int kStepWarps = 4;

// four consecutive operands of a lane
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

template <typename T, int LPR, int NR>
__global__ void __launch_bounds__(kStepWarps * 32) k_la_step(const LaStep p) {
  constexpr int RPW = 32 / LPR;                  // rows of a warp side by side
  constexpr int kRows = kStepWarps * RPW * NR;   // rows of a CTA
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
  const float a = decay_pow(p.log_decay[b * p.decay_batch + h], 1.f);
  float q[4] = {0.f, 0.f, 0.f, 0.f}, k[4] = {0.f, 0.f, 0.f, 0.f};
  if (kin) {
    load4((const T*)p.q + b * p.q_batch + (long long)g * p.dk + k0, q);
    load4((const T*)p.k + b * p.k_batch + (long long)g * p.dk + k0, k);
  }
  const T* vp = (const T*)p.v + b * p.v_batch + (long long)h * p.dv;
  float o[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int v = vb + i * RPW;
    const float x = v < p.dv ? to_f32(vp[v]) : 0.f;
    s[i].x = fmaf(a, s[i].x, x * k[0]);
    s[i].y = fmaf(a, s[i].y, x * k[1]);
    s[i].z = fmaf(a, s[i].z, x * k[2]);
    s[i].w = fmaf(a, s[i].w, x * k[3]);
    if (kin && row >= 0 && v < p.dv) *(float4*)(p.state_out + at + (long long)i * RPW * p.dk) = s[i];
    o[i] = fmaf(s[i].x, q[0], fmaf(s[i].y, q[1], fmaf(s[i].z, q[2], s[i].w * q[3])));
  }
  int n = NR, first = 0;  // this lane holds the sums first ... first + n - 1
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) {
    if (n > 1) {
      const bool up = (sub & d) != 0;
      n /= 2;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i)
        if (i < n) {
          const float send = up ? o[i] : o[i + n], keep = up ? o[i + n] : o[i];
          o[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
      if (up) first += n;
    } else {
      o[0] += __shfl_xor_sync(0xffffffffu, o[0], d);
    }
  }
  // lanes that differ below the exchanges that halved hold the same sums
  if (sub % (LPR * n / NR > 1 ? LPR * n / NR : 1) == 0)
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i < n && vb + (first + i) * RPW < p.dv)
        ((T*)p.o)[((long long)b * p.H + h) * p.dv + vb + (first + i) * RPW] =
            from_f32<T>(row >= 0 ? p.scale * o[i] : 0.f);
}

template <typename T, int LPR>
cudaError_t step_l(const LaStep& p, cudaStream_t s) {
  LaunchScope ls("linattn_step", s);
  constexpr int rows = kStepWarps * (32 / LPR);
  // eight rows a lane once that leaves work for every SM (with fewer rows the
  // latency of one counts: 32 heads of one row ran in 8.1 us with two a lane)
  if ((long long)p.B * p.H * ((p.dv + 8 * rows - 1) / (8 * rows)) >= 2 * kLaSms)
    k_la_step<T, LPR, 8><<<dim3((p.dv + 8 * rows - 1) / (8 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  else
    k_la_step<T, LPR, 2><<<dim3((p.dv + 2 * rows - 1) / (2 * rows), p.H, p.B), kStepWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const LaStep& p, cudaStream_t s) {
  const int lanes = p.dk / 4;
  if (lanes <= 4) return step_l<T, 4>(p, s);
  if (lanes <= 8) return step_l<T, 8>(p, s);
  if (lanes <= 16) return step_l<T, 16>(p, s);
  return step_l<T, 32>(p, s);
}

}  // namespace

int la_segments(long long rows, long long chunks, long long slots) {
  // A row's chunks go to one CTA unless that leaves SMs idle.  Splitting a row
  // costs a pass for the segments' states (about half a walk) and two more
  // launches, and every wave of CTAs its start (about two chunks), so it has to
  // pay for that.  At most 32 segments: more were not measured.
  auto waves = [&](long long n) { return (rows * n + slots - 1) / slots; };
  double best = (double)(waves(1) * (chunks + 2));
  int at = 1;
  for (int n = 2; n <= chunks && n <= 32; ++n) {
    const long long per = (chunks + n - 1) / n;
    const double cost = 1.5 * (double)(waves(n) * (per + 2)) + 4.0 + 0.25 * n;
    if (cost < best) {
      best = cost;
      at = n;
    }
  }
  return at;
}

cudaError_t la_segment_states(const LaSegments& p, cudaStream_t s) {
  LaunchScope ls("linattn_segments", s);
  k_la_segments<<<dim3((p.dk * p.dv + 255) / 256, p.H, p.B), 256, 0, s>>>(p);
  return cudaGetLastError();
}

// CTAs of the fp32 walk that run at once (three an SM, or two for dk > 64)
static int segments32(int B, int H, int T, int dk, int dv) {
  return la_segments((long long)B * H * ((dv + kB - 1) / kB), (T + kC - 1) / kC,
                     (dk <= 64 ? 3 : 2) * kLaSms);
}

size_t la_scratch_floats(int B, int H, int T, int dk, int dv, bool bf16) {
  if (bf16) return la_tc_scratch_floats(B, H, T, dk, dv);
  // (the walks of a backward pass have dk and dv in either order)
  const int a = segments32(B, H, T, dk, dv), b = segments32(B, H, T, dv, dk), n = a > b ? a : b;
  return n > 1 ? (size_t)n * B * H * dk * dv : 0;
}

cudaError_t la_walk(const LaWalk& w, bool bf16, bool beside, float* scratch, cudaStream_t s) {
  if (bf16) return la_walk_tc(w, beside, scratch, s);
  Walk32Args a;
  a.w = w;
  const int nc = (w.T + kC - 1) / kC;
  int n = segments32(w.B, w.H, w.T, w.dk, w.dv);
  a.span = (nc + n - 1) / n * kC;
  n = (w.T + a.span - 1) / a.span;
  a.nseg = n;
  if (n > 1) {
    a.w.last = scratch;
    cudaError_t e = w.dk <= 64 ? walk_t<64, true>(a, s) : walk_t<128, true>(a, s);
    if (e != cudaSuccess) return e;
    const LaSegments g = {w.B, w.H, w.T, w.dk, w.dv, n, a.span, w.log_decay, w.lens, scratch,
                          w.first, w.last, w.first_swapped, w.reverse};
    if ((e = la_segment_states(g, s)) != cudaSuccess) return e;
    a.w.first = scratch;
    a.w.first_swapped = false;
    a.w.last = nullptr;
  }
  return w.dk <= 64 ? walk_t<64, false>(a, s) : walk_t<128, false>(a, s);
}

cudaError_t la_group_sum(long long rows, int G, int share, int D, const float* part, float* out,
                         cudaStream_t s) {
  const long long n = rows * G * D;
  const long long want = (n + 255) / 256;
  LaunchScope ls("linattn_group_sum", s);
  k_la_group_sum<<<(int)(want < 8192 ? want : 8192), 256, 0, s>>>(n, share, D, part, out);
  return cudaGetLastError();
}

cudaError_t la_step(const LaStep& p, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace ssd
