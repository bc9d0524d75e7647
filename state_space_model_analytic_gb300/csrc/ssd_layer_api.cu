// C ABI of the layer operators (linear attention, the gated delta rule, norms
// around a block, layer norm, gradient clipping): argument validation, workspace carve-up and the launches of each
// call.  Declarations and contracts: include/ssd.h.
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/ssd.h"
#include "ssd_internal.h"
#include "ssd_layer_internal.h"

namespace ssd {
namespace {

int refuse(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return code;
}

int cuda_refuse(cudaError_t e, const char* who) {
  return refuse(SSD_ERR_CUDA, "%s: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Named {
  const char* name;
  const void* p;
};

// Required pointers are there, and every given pointer is 16-byte aligned.
int check_pointers(const char* who, const Named* need, int n_need, const Named* may, int n_may) {
  for (int i = 0; i < n_need; ++i)
    if (!need[i].p) return refuse(SSD_ERR_INVALID_ARG, "%s: %s is NULL", who, need[i].name);
  for (int i = 0; i < n_need + n_may; ++i) {
    const Named& q = i < n_need ? need[i] : may[i - n_need];
    if (q.p && ((uintptr_t)q.p & 15u))
      return refuse(SSD_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", who, q.name);
  }
  return SSD_OK;
}

// Arrays of fp32 or int32 that are read element by element.
int check_words(const char* who, const Named* words, int n) {
  for (int i = 0; i < n; ++i)
    if ((uintptr_t)words[i].p & 3u)
      return refuse(SSD_ERR_ALIGNMENT, "%s: %s is not 4-byte aligned", who, words[i].name);
  return SSD_OK;
}

// ---- linear attention ------------------------------------------------------

int la_check(const char* who, const ssd_linattn_dims* d) {
  if (!d) return refuse(SSD_ERR_INVALID_ARG, "%s: dims is NULL", who);
  if (d->batch < 1 || d->seqlen < 1 || d->nheads < 1 || d->ngroups < 1)
    return refuse(SSD_ERR_INVALID_ARG, "%s: every dimension must be >= 1", who);
  if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
    return refuse(SSD_ERR_INVALID_ARG, "%s: dtype %d is not SSD_F32 or SSD_BF16", who, (int)d->dtype);
  if (d->nheads % d->ngroups)
    return refuse(SSD_ERR_INVALID_ARG, "%s: nheads %lld is not a multiple of ngroups %lld", who,
                  (long long)d->nheads, (long long)d->ngroups);
  if (d->dk < 8 || d->dk > 128 || d->dk % 8 || d->dv < 8 || d->dv > 128 || d->dv % 8)
    return refuse(SSD_ERR_UNSUPPORTED, "%s: dk and dv must be multiples of 8 in [8, 128]", who);
  if (d->batch > 65535 || d->nheads > 65535)
    return refuse(SSD_ERR_UNSUPPORTED, "%s: batch and nheads must be at most 65535", who);
  if (d->seqlen > (1ll << 30))
    return refuse(SSD_ERR_UNSUPPORTED, "%s: seqlen must be at most 2^30", who);
  if ((double)d->batch * (double)d->seqlen * (double)d->nheads > 4.0e10)
    return refuse(SSD_ERR_UNSUPPORTED, "%s: problem too large", who);
  return SSD_OK;
}

// An operand with its strides; an extent of 1 takes the dense stride.
int la_operand(const char* who, const char* name, const ssd_linattn_dims* d, const void* p,
               int64_t batch, int64_t step, int64_t heads, int64_t dim, bool one_step, LaOperand* o) {
  if (d->seqlen == 1 || one_step) step = heads * dim;
  if (d->batch == 1) batch = step * d->seqlen;
  const int64_t unit = d->dtype == SSD_BF16 ? 8 : 4;
  if (step <= 0 || batch <= 0 || step % unit || batch % unit)
    return refuse(SSD_ERR_INVALID_ARG, "%s: the strides of %s must be positive multiples of 16 bytes",
                  who, name);
  if (step > (1ll << 36) || batch > (1ll << 36))
    return refuse(SSD_ERR_UNSUPPORTED, "%s: a stride of %s is too large", who, name);
  o->p = p;
  o->batch = batch;
  o->step = step;
  o->share = (int)(d->nheads / heads);
  return SSD_OK;
}

LaWalk la_base(const ssd_linattn_dims* d, const float* log_decay, const int32_t* lens) {
  LaWalk w = {};
  w.B = (int)d->batch;
  w.T = (int)d->seqlen;
  w.H = (int)d->nheads;
  w.log_decay = log_decay;
  w.lens = lens;
  return w;
}

size_t la_scratch_bytes(const ssd_linattn_dims* d) {
  return up256(sizeof(float) * la_scratch_floats((int)d->batch, (int)d->nheads, (int)d->seqlen,
                                                 (int)d->dk, (int)d->dv, d->dtype == SSD_BF16));
}

// One state history.
size_t la_hist_bytes(const ssd_linattn_dims* d) {
  return up256((size_t)128 * la_tc_hist_rows((int)d->batch, (int)d->nheads, (int)d->seqlen,
                                             (int)d->dk, (int)d->dv));
}

// What the backward keeps between its kernels, beside the walks' scratch.
size_t la_part_bytes(const ssd_linattn_dims* d, int which) {
  if (which == 0) return 0;
  if (d->dtype == SSD_BF16) return 2 * la_hist_bytes(d);  // the states before every chunk
  if (d->nheads == d->ngroups) return 0;
  // dq's, then dk's part of every head
  return up256(sizeof(float) * (size_t)d->batch * d->seqlen * d->nheads * d->dk);
}

// ---- the gated delta rule ------------------------------------------------------

// What the backward keeps between its kernels, in this order: the states before
// every chunk and the gradients of those after it, E and y, and where heads share q
// and k their own dq and dk.
struct DeltaKept {
  size_t state, steps, part;
  size_t total() const { return 2 * state + 2 * steps + part; }
};
DeltaKept delta_kept(const ssd_linattn_dims* d) {
  const size_t c = (size_t)delta_chunk(d->dtype == SSD_BF16);
  const size_t units = (size_t)d->batch * d->nheads * (((size_t)d->seqlen + c - 1) / c);
  DeltaKept k;
  k.state = up256(sizeof(float) * units * d->dv * d->dk);
  k.steps = up256(sizeof(float) * units * c * d->dv);
  k.part = d->nheads == d->ngroups
               ? 0
               : up256(2 * sizeof(float) * (size_t)d->batch * d->seqlen * d->nheads * d->dk);
  return k;
}

// log_decay and beta are given and aligned
int gates_check(const char* who, const float* log_decay, const float* beta, const int32_t* ints,
                const char* ints_name) {
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  if (!beta) return refuse(SSD_ERR_INVALID_ARG, "%s: beta is NULL", who);
  const Named words[] = {{"log_decay", log_decay}, {"beta", beta}, {ints_name, ints}};
  return check_words(who, words, 3);
}

// (256 bytes stand for none)
int workspace_check(const char* who, const void* workspace, size_t bytes, size_t need) {
  if (!workspace && need == 256) return SSD_OK;
  if (!workspace) return refuse(SSD_ERR_INVALID_ARG, "%s: workspace is NULL", who);
  if ((uintptr_t)workspace & 255u)
    return refuse(SSD_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", who);
  if (bytes < need)
    return refuse(SSD_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, bytes, need);
  return SSD_OK;
}

// ---- norms around a block, gradient clipping -----------------------------------

// A pointer to elements of a type, aligned to their own size.
struct Sized {
  const char* name;
  const void* p;
  int dtype;
};
int check_sized(const char* who, const Sized* need, int n_need, const Sized* may, int n_may) {
  for (int i = 0; i < n_need; ++i)
    if (!need[i].p) return refuse(SSD_ERR_INVALID_ARG, "%s: %s is NULL", who, need[i].name);
  for (int i = 0; i < n_need + n_may; ++i) {
    const Sized& q = i < n_need ? need[i] : may[i - n_need];
    if ((uintptr_t)q.p & (q.dtype == SSD_BF16 ? 1u : 3u))
      return refuse(SSD_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, q.name);
  }
  return SSD_OK;
}

int norm_check(const char* who, int64_t rows, int64_t width, int32_t dtype, int32_t res_dtype,
               int64_t y_stride, int64_t z_stride, float eps) {
  if (rows < 1) return refuse(SSD_ERR_INVALID_ARG, "%s: rows must be >= 1", who);
  if (dtype != SSD_F32 && dtype != SSD_BF16)
    return refuse(SSD_ERR_INVALID_ARG, "%s: dtype %d is not SSD_F32 or SSD_BF16", who, (int)dtype);
  if (res_dtype != SSD_F32 && res_dtype != dtype)
    return refuse(SSD_ERR_INVALID_ARG, "%s: res_dtype must be dtype or SSD_F32", who);
  if (width < 1 || width > 8192)
    return refuse(SSD_ERR_UNSUPPORTED, "%s: width %lld must be in [1, 8192]", who, (long long)width);
  if (y_stride < width || z_stride < width)
    return refuse(SSD_ERR_INVALID_ARG, "%s: a row stride is smaller than the width", who);
  if (!(eps >= 0.f)) return refuse(SSD_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  return SSD_OK;
}

// *used: tensors with elements, *bytes: of all of them
int clip_check(const char* who, const ssd_clip_tensor* t, int64_t count, int* used, long long* bytes) {
  if (count < 0 || count > (1 << 24) || (count && !t))
    return refuse(SSD_ERR_INVALID_ARG, "%s: count must be in [0, 2^24] and tensors not NULL", who);
  *used = 0;
  *bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    const ssd_clip_tensor& x = t[i];
    if (x.numel < 0 || x.numel > (1ll << 40) || x.reserved != 0 ||
        (x.dtype != SSD_F32 && x.dtype != SSD_BF16))
      return refuse(SSD_ERR_INVALID_ARG, "%s: tensor %lld: bad numel, dtype or reserved", who,
                    (long long)i);
    if (!x.numel) continue;
    if (!x.g || !x.out)
      return refuse(SSD_ERR_INVALID_ARG, "%s: tensor %lld: NULL pointer", who, (long long)i);
    if ((((uintptr_t)x.g | (uintptr_t)x.out) & (x.dtype == SSD_BF16 ? 1u : 3u)) != 0)
      return refuse(SSD_ERR_ALIGNMENT, "%s: tensor %lld is not aligned to its elements", who,
                    (long long)i);
    *used += 1;
    *bytes += x.numel * (x.dtype == SSD_BF16 ? 2 : 4);
  }
  return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_linattn_workspace_bytes(const ssd_linattn_dims* d, int which) {
  set_last_error("");
  if (la_check("ssd_linattn_workspace_bytes", d)) return 0;
  if (which != 0 && which != 1) {
    refuse(SSD_ERR_INVALID_ARG, "ssd_linattn_workspace_bytes: which must be 0 or 1");
    return 0;
  }
  return 256 + la_part_bytes(d, which) + la_scratch_bytes(d);
}

int ssd_linattn_forward(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                        const float* log_decay, const float* state0, const int32_t* lens, void* o,
                        float* state, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_linattn_forward";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  const Named need[] = {{"q", q}, {"k", k}, {"v", v}, {"o", o}};
  const Named may[] = {{"state0", state0}, {"state", state}};
  if ((rc = check_pointers(who, need, 4, may, 2))) return rc;
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  const Named words[] = {{"log_decay", log_decay}, {"lens", lens}};
  if ((rc = check_words(who, words, 2))) return rc;
  if ((rc = workspace_check(who, workspace, workspace_bytes, ssd_linattn_workspace_bytes(d, 0))))
    return rc;
  LaWalk w = la_base(d, log_decay, lens);
  w.dk = (int)d->dk;
  w.dv = (int)d->dv;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, d->q_step, d->ngroups, d->dk, false, &w.q)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, d->k_step, d->ngroups, d->dk, false, &w.k)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, d->v_step, d->nheads, d->dv, false, &w.v)))
    return rc;
  w.first = state0;
  w.last = state;
  w.o = o;
  w.s_intra = w.s_carry = d->scale;
  w.s_inject = 1.f;
  w.off = 1;
  const cudaError_t e = la_walk(w, d->dtype == SSD_BF16, false, (float*)workspace, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

int ssd_linattn_backward(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                         const float* log_decay, const float* state0, const void* dout,
                         const float* dstate, const int32_t* lens, void* dq, void* dk, void* dv,
                         float* dstate0, void* workspace, size_t workspace_bytes,
                         void* cuda_stream) {
  const char* who = "ssd_linattn_backward";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  const Named need[] = {{"q", q},   {"k", k},   {"v", v},   {"dout", dout},
                        {"dq", dq}, {"dk", dk}, {"dv", dv}};
  const Named may[] = {{"state0", state0}, {"dstate", dstate}, {"dstate0", dstate0}};
  if ((rc = check_pointers(who, need, 7, may, 3))) return rc;
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  const Named words[] = {{"log_decay", log_decay}, {"lens", lens}};
  if ((rc = check_words(who, words, 2))) return rc;
  if ((rc = workspace_check(who, workspace, workspace_bytes, ssd_linattn_workspace_bytes(d, 1))))
    return rc;
  LaOperand oq, ok, ov, og;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, d->q_step, d->ngroups, d->dk, false, &oq)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, d->k_step, d->ngroups, d->dk, false, &ok)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, d->v_step, d->nheads, d->dv, false, &ov)) ||
      (rc = la_operand(who, "dout", d, dout, d->dout_batch, d->dout_step, d->nheads, d->dv, false,
                       &og)))
    return rc;
  const bool bf16 = d->dtype == SSD_BF16;
  const int share = (int)(d->nheads / d->ngroups);
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  float* scratch = (float*)workspace;
  char* rest = (char*)workspace + la_scratch_bytes(d);
  // dv, dstate0: backwards over (k, q, do)
  LaWalk w = la_base(d, log_decay, lens);
  w.dk = (int)d->dk;
  w.dv = (int)d->dv;
  w.q = ok;
  w.k = oq;
  w.v = og;
  w.first = dstate;
  w.last = dstate0;
  w.o = dv;
  w.s_intra = w.s_inject = d->scale;
  w.s_carry = 1.f;
  w.reverse = true;
  if (bf16) {
    // with the states before every chunk, backward and forward, dq and dk are
    // sums over chunks and a group's heads that need no walk
    w.hist = rest + la_hist_bytes(d);
    w.followed = true;
    LaWalk f = la_base(d, log_decay, lens);
    f.dk = (int)d->dk;
    f.dv = (int)d->dv;
    f.q = oq;  // (not read)
    f.k = ok;
    f.v = ov;
    f.first = state0;
    f.s_inject = 1.f;
    f.off = 1;
    f.hist = rest;
    const LaGrads x = {w.B, w.T, w.H, w.dk, w.dv, oq, ok, ov, og, log_decay, lens, f.hist, w.hist,
                       dq, dk, d->scale};
    cudaError_t e = la_walk(w, true, false, scratch, s);
    if (e == cudaSuccess) e = la_walk(f, true, true, scratch, s);
    if (e == cudaSuccess) e = la_grads_tc(x, s);
    return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
  }
  cudaError_t e = la_walk(w, false, false, scratch, s);
  if (e != cudaSuccess) return cuda_refuse(e, who);
  // dq: forward over (do, v, k), from the transposed state; dk: backwards over
  // (v, do, q), from the transposed gradient of the state
  for (int i = 0; i < 2; ++i) {
    LaWalk y = la_base(d, log_decay, lens);
    y.dk = (int)d->dv;
    y.dv = (int)d->dk;
    y.q = i ? ov : og;
    y.k = i ? og : ov;
    y.v = i ? oq : ok;
    y.first = i ? dstate : state0;
    y.first_swapped = true;
    y.s_intra = d->scale;
    y.s_carry = i ? 1.f : d->scale;
    y.s_inject = i ? d->scale : 1.f;
    y.off = i ? 0 : 1;
    y.reverse = i == 1;
    float* out = (float*)(i ? dk : dq);
    y.o = share > 1 ? (float*)rest : out;
    if ((e = la_walk(y, false, false, scratch, s)) != cudaSuccess) return cuda_refuse(e, who);
    if (share == 1) continue;
    e = la_group_sum(d->batch * d->seqlen, (int)d->ngroups, share, (int)d->dk, (const float*)y.o,
                     out, s);
    if (e != cudaSuccess) return cuda_refuse(e, who);
  }
  return SSD_OK;
}

int ssd_linattn_step(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                     const float* log_decay, int64_t decay_batch, const float* state_in,
                     float* state_out, const int32_t* slots, int64_t nslots, void* o,
                     void* cuda_stream) {
  const char* who = "ssd_linattn_step";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  if (d->seqlen != 1) return refuse(SSD_ERR_INVALID_ARG, "%s: seqlen must be 1", who);
  const Named need[] = {{"q", q}, {"k", k}, {"v", v}, {"state_in", state_in},
                        {"state_out", state_out}, {"o", o}};
  if ((rc = check_pointers(who, need, 6, nullptr, 0))) return rc;
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  const Named words[] = {{"log_decay", log_decay}, {"slots", slots}};
  if ((rc = check_words(who, words, 2))) return rc;
  if (decay_batch != 0 && decay_batch != d->nheads)
    return refuse(SSD_ERR_INVALID_ARG, "%s: decay_batch must be 0 or nheads", who);
  if (nslots < 1 || (!slots && nslots < d->batch) || nslots > (1ll << 31))
    return refuse(SSD_ERR_INVALID_ARG, "%s: nslots must be in [1, 2^31], and at least batch without slots", who);
  LaOperand oq, ok, ov;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, 0, d->ngroups, d->dk, true, &oq)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, 0, d->ngroups, d->dk, true, &ok)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, 0, d->nheads, d->dv, true, &ov)))
    return rc;
  LaStep p = {};
  p.B = (int)d->batch;
  p.H = (int)d->nheads;
  p.G = (int)d->ngroups;
  p.dk = (int)d->dk;
  p.dv = (int)d->dv;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_batch = oq.batch;
  p.k_batch = ok.batch;
  p.v_batch = ov.batch;
  p.log_decay = log_decay;
  p.decay_batch = decay_batch;
  p.state_in = state_in;
  p.state_out = state_out;
  p.slots = slots;
  p.nslots = nslots;
  p.o = o;
  p.scale = d->scale;
  const cudaError_t e = la_step(p, d->dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

// ---- the gated delta rule ------------------------------------------------------

size_t ssd_delta_rule_workspace_bytes(const ssd_linattn_dims* d, int which) {
  set_last_error("");
  if (la_check("ssd_delta_rule_workspace_bytes", d)) return 0;
  if (which != 0 && which != 1) {
    refuse(SSD_ERR_INVALID_ARG, "ssd_delta_rule_workspace_bytes: which must be 0 or 1");
    return 0;
  }
  return 256 + (which ? delta_kept(d).total() : 0);
}

int ssd_delta_rule_forward(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                           const float* log_decay, const float* beta, const float* state0,
                           const int32_t* lens, void* o, float* state, void* workspace,
                           size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_delta_rule_forward";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  const Named need[] = {{"q", q}, {"k", k}, {"v", v}, {"o", o}};
  const Named may[] = {{"state0", state0}, {"state", state}};
  if ((rc = check_pointers(who, need, 4, may, 2))) return rc;
  if ((rc = gates_check(who, log_decay, beta, lens, "lens"))) return rc;
  if ((rc = workspace_check(who, workspace, workspace_bytes, ssd_delta_rule_workspace_bytes(d, 0))))
    return rc;
  DeltaWalk w = {};
  w.B = (int)d->batch;
  w.T = (int)d->seqlen;
  w.H = (int)d->nheads;
  w.dk = (int)d->dk;
  w.dv = (int)d->dv;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, d->q_step, d->ngroups, d->dk, false, &w.q)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, d->k_step, d->ngroups, d->dk, false, &w.k)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, d->v_step, d->nheads, d->dv, false, &w.v)))
    return rc;
  w.log_decay = log_decay;
  w.beta = beta;
  w.first = state0;
  w.last = state;
  w.lens = lens;
  w.o = o;
  w.scale = d->scale;
  const cudaError_t e = delta_walk(w, d->dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

int ssd_delta_rule_backward(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                            const float* log_decay, const float* beta, const float* state0,
                            const void* dout, const float* dstate, const int32_t* lens, void* dq,
                            void* dk, void* dv, float* dlog_decay, float* dbeta, float* dstate0,
                            void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_delta_rule_backward";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  const Named need[] = {{"q", q},   {"k", k},   {"v", v},   {"dout", dout},
                        {"dq", dq}, {"dk", dk}, {"dv", dv}};
  const Named may[] = {{"state0", state0}, {"dstate", dstate}, {"dstate0", dstate0}};
  if ((rc = check_pointers(who, need, 7, may, 3))) return rc;
  if ((rc = gates_check(who, log_decay, beta, lens, "lens"))) return rc;
  if (!dlog_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: dlog_decay is NULL", who);
  if (!dbeta) return refuse(SSD_ERR_INVALID_ARG, "%s: dbeta is NULL", who);
  const Named words[] = {{"dlog_decay", dlog_decay}, {"dbeta", dbeta}};
  if ((rc = check_words(who, words, 2))) return rc;
  if ((rc = workspace_check(who, workspace, workspace_bytes, ssd_delta_rule_workspace_bytes(d, 1))))
    return rc;
  LaOperand oq, ok, ov, og;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, d->q_step, d->ngroups, d->dk, false, &oq)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, d->k_step, d->ngroups, d->dk, false, &ok)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, d->v_step, d->nheads, d->dv, false, &ov)) ||
      (rc = la_operand(who, "dout", d, dout, d->dout_batch, d->dout_step, d->nheads, d->dv, false,
                       &og)))
    return rc;
  const bool bf16 = d->dtype == SSD_BF16;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const DeltaKept kept = delta_kept(d);
  char* at = (char*)workspace;
  float* hist_s = (float*)at;
  float* hist_d = (float*)(at += kept.state);
  float* err = (float*)(at += kept.state);
  float* y = (float*)(at += kept.steps);
  float* part = (float*)(at += kept.steps);
  const int B = (int)d->batch, T = (int)d->seqlen, H = (int)d->nheads, G = (int)d->ngroups;
  const int K = (int)d->dk, V = (int)d->dv;
  const DeltaWalk w = {B, T, H, K, V, oq, ok, ov, log_decay, beta, state0, nullptr, lens, nullptr,
                       hist_s, err, d->scale};
  cudaError_t e = delta_walk(w, bf16, s);
  const DeltaBack r = {B, T, H, K, V, oq, ok, og, log_decay, beta, dstate, dstate0, lens, dv,
                       hist_d, y, d->scale};
  if (e == cudaSuccess) e = delta_back(r, bf16, s);
  const DeltaGrads x = {B, T, H, G, K, V, oq, ok, og, log_decay, beta, lens, hist_s, hist_d, err, y,
                        dq, dk, dlog_decay, dbeta, d->scale};
  if (e == cudaSuccess) e = delta_grads(x, part, bf16, s);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

int ssd_delta_rule_step(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                        const float* log_decay, const float* beta, const float* state_in,
                        float* state_out, const int32_t* slots, int64_t nslots, void* o,
                        void* cuda_stream) {
  const char* who = "ssd_delta_rule_step";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  if (d->seqlen != 1) return refuse(SSD_ERR_INVALID_ARG, "%s: seqlen must be 1", who);
  const Named need[] = {{"q", q}, {"k", k}, {"v", v}, {"state_in", state_in},
                        {"state_out", state_out}, {"o", o}};
  if ((rc = check_pointers(who, need, 6, nullptr, 0))) return rc;
  if ((rc = gates_check(who, log_decay, beta, slots, "slots"))) return rc;
  if (nslots < 1 || (!slots && nslots < d->batch) || nslots > (1ll << 31))
    return refuse(SSD_ERR_INVALID_ARG, "%s: nslots must be in [1, 2^31], and at least batch without slots", who);
  LaOperand oq, ok, ov;
  if ((rc = la_operand(who, "q", d, q, d->q_batch, 0, d->ngroups, d->dk, true, &oq)) ||
      (rc = la_operand(who, "k", d, k, d->k_batch, 0, d->ngroups, d->dk, true, &ok)) ||
      (rc = la_operand(who, "v", d, v, d->v_batch, 0, d->nheads, d->dv, true, &ov)))
    return rc;
  const DeltaStep p = {(int)d->batch, (int)d->nheads, (int)d->ngroups, (int)d->dk, (int)d->dv,
                       q, k, v, oq.batch, ok.batch, ov.batch, log_decay, beta, state_in, state_out,
                       slots, nslots, o, d->scale};
  const cudaError_t e = delta_step(p, d->dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

// ---- norms around a block ------------------------------------------------------

size_t ssd_block_norm_workspace_bytes(int64_t rows, int64_t width) {
  set_last_error("");
  if (rows < 1 || width < 1 || width > 8192) {
    refuse(SSD_ERR_INVALID_ARG, "ssd_block_norm_workspace_bytes: rows >= 1 and width in [1, 8192]");
    return 0;
  }
  return up256((size_t)kBlockNormMaxCtas * 2 * width * sizeof(float));
}

int ssd_block_norm_forward(int64_t rows, int64_t width, int32_t dtype, int32_t res_dtype,
                           const void* residual, const void* y, int64_t y_stride, const void* z,
                           int64_t z_stride, const float* w_post, const float* res_scale,
                           const float* w_pre, float eps, void* new_residual, void* x,
                           float* stats, void* cuda_stream) {
  const char* who = "ssd_block_norm_forward";
  set_last_error("");
  int rc = norm_check(who, rows, width, dtype, res_dtype, y_stride, z ? z_stride : width, eps);
  if (rc) return rc;
  const Sized need[] = {{"residual", residual, res_dtype}, {"y", y, dtype}, {"w_post", w_post, 0},
                        {"w_pre", w_pre, 0}, {"new_residual", new_residual, res_dtype},
                        {"x", x, dtype}};
  const Sized may[] = {{"z", z, dtype}, {"res_scale", res_scale, 0}};
  if ((rc = check_sized(who, need, 6, may, 2))) return rc;
  if (stats && ((uintptr_t)stats & 7u))
    return refuse(SSD_ERR_ALIGNMENT, "%s: stats is not 8-byte aligned", who);
  BlockNorm p = {};
  p.rows = rows;
  p.width = (int)width;
  p.y_stride = y_stride;
  p.z_stride = z_stride;
  p.eps = eps;
  p.residual = residual;
  p.y = y;
  p.z = z;
  p.w_post = w_post;
  p.res_scale = res_scale;
  p.w_pre = w_pre;
  p.new_residual = new_residual;
  p.x = x;
  p.stats = stats;
  const cudaError_t e =
      block_norm_forward(p, dtype == SSD_BF16, res_dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

int ssd_block_norm_backward(int64_t rows, int64_t width, int32_t dtype, int32_t res_dtype,
                            const void* new_residual, const void* y, int64_t y_stride,
                            const void* z, int64_t z_stride, const float* w_post,
                            const float* res_scale, const float* w_pre, float eps,
                            const float* stats, const void* dx, const void* dnew, void* dresidual,
                            void* dy, void* dz, float* dw_post, float* dres_scale, float* dw_pre,
                            void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_block_norm_backward";
  set_last_error("");
  int rc = norm_check(who, rows, width, dtype, res_dtype, y_stride, z ? z_stride : width, eps);
  if (rc) return rc;
  const Sized need[] = {{"new_residual", new_residual, res_dtype}, {"y", y, dtype},
                        {"w_post", w_post, 0}, {"w_pre", w_pre, 0}, {"dx", dx, dtype},
                        {"dresidual", dresidual, res_dtype}, {"dy", dy, dtype},
                        {"dw_post", dw_post, 0}, {"dw_pre", dw_pre, 0}};
  const Sized may[] = {{"z", z, dtype}, {"res_scale", res_scale, 0}, {"dnew", dnew, res_dtype},
                       {"dz", dz, dtype}, {"dres_scale", dres_scale, 0}};
  if ((rc = check_sized(who, need, 9, may, 5))) return rc;
  if (z && !dz) return refuse(SSD_ERR_INVALID_ARG, "%s: dz is NULL", who);
  if (stats && ((uintptr_t)stats & 7u))
    return refuse(SSD_ERR_ALIGNMENT, "%s: stats is not 8-byte aligned", who);
  if ((rc = workspace_check(who, workspace, workspace_bytes,
                            ssd_block_norm_workspace_bytes(rows, width))))
    return rc;
  BlockNorm p = {};
  p.rows = rows;
  p.width = (int)width;
  p.y_stride = y_stride;
  p.z_stride = z_stride;
  p.eps = eps;
  p.residual = new_residual;
  p.y = y;
  p.z = z;
  p.w_post = w_post;
  p.res_scale = res_scale;
  p.w_pre = w_pre;
  p.stats = const_cast<float*>(stats);
  p.dx = dx;
  p.dnew = dnew;
  p.dresidual = dresidual;
  p.dy = dy;
  p.dz = dz;
  p.dw_post = dw_post;
  p.dres_scale = dres_scale;
  p.dw_pre = dw_pre;
  p.part = (float*)workspace;
  const cudaError_t e =
      block_norm_backward(p, dtype == SSD_BF16, res_dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

// ---- layer norm ------------------------------------------------------------------

size_t ssd_layer_norm_workspace_bytes(int64_t rows, int64_t width) {
  set_last_error("");
  if (rows < 1 || width < 1 || width > 8192) {
    refuse(SSD_ERR_INVALID_ARG, "ssd_layer_norm_workspace_bytes: rows >= 1 and width in [1, 8192]");
    return 0;
  }
  return up256((size_t)kLayerNormMaxCtas * 2 * width * sizeof(float));
}

int ssd_layer_norm_forward(int64_t rows, int64_t width, int32_t dtype, const void* x,
                           int64_t x_stride, const float* weight, const float* bias, float eps,
                           void* y, float* stats, void* cuda_stream) {
  const char* who = "ssd_layer_norm_forward";
  set_last_error("");
  int rc = norm_check(who, rows, width, dtype, dtype, x_stride, width, eps);
  if (rc) return rc;
  const Sized need[] = {{"x", x, dtype}, {"y", y, dtype}};
  const Sized may[] = {{"weight", weight, SSD_F32}, {"bias", bias, SSD_F32}};
  if ((rc = check_sized(who, need, 2, may, 2))) return rc;
  if (stats && ((uintptr_t)stats & 7u))
    return refuse(SSD_ERR_ALIGNMENT, "%s: stats is not 8-byte aligned", who);
  LayerNorm p = {};
  p.rows = rows;
  p.width = (int)width;
  p.x_stride = x_stride;
  p.eps = eps;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.y = y;
  p.stats = stats;
  const cudaError_t e = layer_norm_forward(p, dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

int ssd_layer_norm_backward(int64_t rows, int64_t width, int32_t dtype, const void* x,
                            int64_t x_stride, const float* weight, float eps, const float* stats,
                            const void* dy, void* dx, float* dweight, float* dbias,
                            void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_layer_norm_backward";
  set_last_error("");
  int rc = norm_check(who, rows, width, dtype, dtype, x_stride, width, eps);
  if (rc) return rc;
  const Sized need[] = {{"x", x, dtype}, {"dy", dy, dtype}, {"dx", dx, dtype}};
  const Sized may[] = {{"weight", weight, SSD_F32}, {"dweight", dweight, SSD_F32},
                       {"dbias", dbias, SSD_F32}};
  if ((rc = check_sized(who, need, 3, may, 3))) return rc;
  if (stats && ((uintptr_t)stats & 7u))
    return refuse(SSD_ERR_ALIGNMENT, "%s: stats is not 8-byte aligned", who);
  if ((rc = workspace_check(who, workspace, workspace_bytes,
                            ssd_layer_norm_workspace_bytes(rows, width))))
    return rc;
  LayerNorm p = {};
  p.rows = rows;
  p.width = (int)width;
  p.x_stride = x_stride;
  p.eps = eps;
  p.x = x;
  p.weight = weight;
  p.stats = const_cast<float*>(stats);
  p.dy = dy;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.part = (float*)workspace;
  const cudaError_t e = layer_norm_backward(p, dtype == SSD_BF16, (cudaStream_t)cuda_stream);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
}

// ---- gradient clipping -----------------------------------------------------------

size_t ssd_clip_workspace_bytes(const ssd_clip_tensor* tensors, int64_t count) {
  set_last_error("");
  int used = 0;
  long long bytes = 0;
  if (clip_check("ssd_clip_workspace_bytes", tensors, count, &used, &bytes)) return 0;
  const size_t launches = ((size_t)used + kClipTable - 1) / kClipTable;
  return up256((launches ? launches : 1) * kClipMaxCtas * sizeof(double));
}

int ssd_clip_grad_norm(const ssd_clip_tensor* tensors, int64_t count, float max_norm, float eps,
                       float* norm, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_clip_grad_norm";
  set_last_error("");
  int used = 0;
  long long bytes = 0;
  int rc = clip_check(who, tensors, count, &used, &bytes);
  if (rc) return rc;
  if (!norm) return refuse(SSD_ERR_INVALID_ARG, "%s: norm is NULL", who);
  if ((uintptr_t)norm & 3u) return refuse(SSD_ERR_ALIGNMENT, "%s: norm is not 4-byte aligned", who);
  if (!(max_norm >= 0.f) || !(eps >= 0.f))
    return refuse(SSD_ERR_INVALID_ARG, "%s: max_norm and eps must be >= 0", who);
  if ((rc = workspace_check(who, workspace, workspace_bytes,
                            ssd_clip_workspace_bytes(tensors, count))))
    return rc;
  ClipEntry few[64];
  ClipEntry* e = used <= 64 ? few : new (std::nothrow) ClipEntry[used];
  if (!e) return refuse(SSD_ERR_INVALID_ARG, "%s: no host memory for %d tensors", who, used);
  int n = 0;
  for (int64_t i = 0; i < count; ++i)
    if (tensors[i].numel)
      e[n++] = ClipEntry{tensors[i].g, tensors[i].out, (long long)tensors[i].numel, 0,
                         tensors[i].dtype == SSD_BF16};
  // chunks: the least power of two from 4 KB up that makes at most four of
  // them a CTA; a launch's chunk count stays an int
  int shift = 12;
  while ((bytes >> shift) > 4ll * kClipMaxCtas) ++shift;
  const cudaError_t err = clip_grad_norm(e, used, shift, (double*)workspace, max_norm, eps, norm,
                                         (cudaStream_t)cuda_stream);
  if (e != few) delete[] e;
  return err == cudaSuccess ? SSD_OK : cuda_refuse(err, who);
}

}  // extern "C"
