// C ABI of the layer operators (linear attention): argument validation,
// workspace carve-up and the launches of each call.  Declarations and
// contracts: include/ssd.h.
#include <cstdarg>
#include <cstdio>

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
  if (step < 0 || batch < 0 || step % unit || batch % unit)
    return refuse(SSD_ERR_INVALID_ARG, "%s: the strides of %s must be non-negative multiples of 16 bytes",
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

size_t la_part_bytes(const ssd_linattn_dims* d, int which) {
  if (which == 0 || d->nheads == d->ngroups) return 0;
  return up256(sizeof(float) * (size_t)d->batch * d->seqlen * d->nheads * d->dk);
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
  return 256 + la_part_bytes(d, which);
}

int ssd_linattn_forward(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                        const float* log_decay, const float* state0, const int32_t* lens, void* o,
                        float* state, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const char* who = "ssd_linattn_forward";
  set_last_error("");
  int rc = la_check(who, d);
  if (rc) return rc;
  const Named need[] = {{"q", q}, {"k", k}, {"v", v}, {"o", o}, {"workspace", workspace}};
  const Named may[] = {{"state0", state0}, {"state", state}};
  if ((rc = check_pointers(who, need, 5, may, 2))) return rc;
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  if (workspace_bytes < ssd_linattn_workspace_bytes(d, 0))
    return refuse(SSD_ERR_INVALID_ARG, "%s: workspace too small", who);
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
  const cudaError_t e = la_walk(w, d->dtype == SSD_BF16, (cudaStream_t)cuda_stream);
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
                        {"dq", dq}, {"dk", dk}, {"dv", dv}, {"workspace", workspace}};
  const Named may[] = {{"state0", state0}, {"dstate", dstate}, {"dstate0", dstate0}};
  if ((rc = check_pointers(who, need, 8, may, 3))) return rc;
  if (!log_decay) return refuse(SSD_ERR_INVALID_ARG, "%s: log_decay is NULL", who);
  if (workspace_bytes < ssd_linattn_workspace_bytes(d, 1))
    return refuse(SSD_ERR_INVALID_ARG, "%s: workspace too small", who);
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
  float* part = share > 1 ? (float*)workspace : nullptr;
  // dq: forward over (do, v, k), from the transposed state
  LaWalk w = la_base(d, log_decay, lens);
  w.dk = (int)d->dv;
  w.dv = (int)d->dk;
  w.q = og;
  w.k = ov;
  w.v = ok;
  w.first = state0;
  w.first_swapped = true;
  w.o = part ? (void*)part : dq;
  w.o_f32 = part != nullptr;
  w.s_intra = w.s_carry = d->scale;
  w.s_inject = 1.f;
  w.off = 1;
  cudaError_t e = la_walk(w, bf16, s);
  if (e != cudaSuccess) return cuda_refuse(e, who);
  if (part) {
    e = la_group_sum(d->batch * d->seqlen, (int)d->ngroups, share, (int)d->dk, bf16, part, dq, s);
    if (e != cudaSuccess) return cuda_refuse(e, who);
  }
  // dk: backwards over (v, do, q), from the transposed gradient of the state
  w.q = ov;
  w.k = og;
  w.v = oq;
  w.first = dstate;
  w.o = part ? (void*)part : dk;
  w.s_carry = 1.f;
  w.s_inject = d->scale;
  w.off = 0;
  w.reverse = true;
  e = la_walk(w, bf16, s);
  if (e != cudaSuccess) return cuda_refuse(e, who);
  if (part) {
    e = la_group_sum(d->batch * d->seqlen, (int)d->ngroups, share, (int)d->dk, bf16, part, dk, s);
    if (e != cudaSuccess) return cuda_refuse(e, who);
  }
  // dv, dstate0: backwards over (k, q, do)
  w.dk = (int)d->dk;
  w.dv = (int)d->dv;
  w.q = ok;
  w.k = oq;
  w.v = og;
  w.first_swapped = false;
  w.last = dstate0;
  w.o = dv;
  w.o_f32 = false;
  e = la_walk(w, bf16, s);
  return e == cudaSuccess ? SSD_OK : cuda_refuse(e, who);
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

}  // extern "C"
