// ssd_delta_api.cu -- the C ABI of the gated delta rule: argument validation,
// workspace planning and the launch sequences.
#include <string.h>

#include "delta_internal.cuh"

namespace ssd {
namespace {

constexpr size_t kStatusBytes = 256;  // the device status word's place in the workspaces

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
bool misaligned(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

int make_delta_plan(const ssd_delta_problem* pr, DeltaPlan* p) {
  if (!pr) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->batch < 1 || pr->seqlen < 1 || pr->nheads < 1 || pr->headdim < 1 || pr->dstate < 1 || pr->ngroups < 1)
    return SSD_ERR_INVALID_ARGUMENT;
  if (pr->nheads % pr->ngroups != 0) return SSD_ERR_INVALID_ARGUMENT;
  if ((pr->dtype != SSD_F32 && pr->dtype != SSD_BF16) || (pr->state_dtype != SSD_F32 && pr->state_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARGUMENT;
  if (pr->flags & ~(SSD_HAS_INIT | SSD_HAS_SEQ_IDX | SSD_HAS_DFINAL | SSD_WANT_DINIT)) return SSD_ERR_INVALID_ARGUMENT;
  if (!(pr->scale >= -3.402823466e38f && pr->scale <= 3.402823466e38f)) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->headdim > 256 || pr->dstate > 256) return SSD_ERR_UNSUPPORTED;
  if (pr->nheads > (1 << 20) || pr->batch > (1 << 20) || pr->seqlen > (1LL << 30)) return SSD_ERR_UNSUPPORTED;
  const int64_t qk = pr->ngroups * pr->dstate, vv = pr->nheads * pr->headdim;
  const int64_t qs = pr->q_stride ? pr->q_stride : qk, ks = pr->k_stride ? pr->k_stride : qk;
  const int64_t vs = pr->v_stride ? pr->v_stride : vv;
  if (qs < qk || ks < qk || vs < vv) return SSD_ERR_INVALID_ARGUMENT;
  // 2^40 elements per tensor, 2^31 - 1 CTAs of any launch (the recurrent kernels' 16-column tiles, the
  // chunk kernels' 32-token chunks)
  int64_t wide = qs > ks ? qs : ks;
  wide = vs > wide ? vs : wide;
  const double tokens = (double)pr->batch * (double)pr->seqlen;
  const double cap = (double)(1LL << 40);
  if (tokens * (double)wide >= cap || (double)pr->batch * (double)vv * (double)pr->dstate >= cap)
    return SSD_ERR_UNSUPPORTED;
  const double chunks = (double)pr->batch * (double)((pr->seqlen + 31) / 32);
  if (chunks * (double)vv * (double)pr->dstate >= cap || chunks * (double)pr->nheads >= 2147483648.0 ||
      (double)pr->batch * (double)pr->nheads * 16.0 >= 2147483648.0)
    return SSD_ERR_UNSUPPORTED;

  memset(p, 0, sizeof(*p));
  p->b = (int)pr->batch;
  p->L = (int)pr->seqlen;
  p->H = (int)pr->nheads;
  p->P = (int)pr->headdim;
  p->N = (int)pr->dstate;
  p->G = (int)pr->ngroups;
  p->hpg = p->H / p->G;
  p->qs = qs;
  p->ks = ks;
  p->vs = vs;
  p->scale = pr->scale;
  p->bf16 = pr->dtype == SSD_BF16;
  p->st_bf16 = pr->state_dtype == SSD_BF16;
  p->tc = p->bf16 && p->P % 64 == 0 && (p->N == 64 || p->N == 128) && qs % 8 == 0 && ks % 8 == 0 && vs % 8 == 0;
  p->C = p->tc ? kDeltaChunk : kDeltaChunkF32;
  p->nc = (p->L + p->C - 1) / p->C;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  const size_t bh = (size_t)p->b * p->H, states = bh * p->nc * p->P * p->N, rows = bh * p->L * p->P;
  if (p->tc) {
    const size_t units = bh * p->nc, cc = (size_t)p->C * p->C * 2;
    p->sv_S = take(states * 2);
    p->sv_w = take(units * p->C * p->P * 2);
    p->sv_T = take(units * cc);
    p->sv_A = take(units * cc);
    p->sv_e = take(units * kGateRows * p->C * 4);
    p->saved_bytes = off;
    off = kStatusBytes;
    p->wf_T = take(units * cc);
    p->wf_A = take(units * cc);
    p->wf_e = take(units * kGateRows * p->C * 4);
    p->fwd_bytes = off;
    off = kStatusBytes;
    p->wb_D = take(states * 2);
    p->bwd_bytes = off;
    return SSD_OK;
  }
  const size_t units = bh * p->nc, cc = (size_t)p->C * p->C * 4;
  p->sv_S = take(states * 4);
  p->sv_w = take(rows * 4);
  p->sv_T = take(units * cc);
  p->sv_A = take(units * cc);
  p->sv_e = take(units * 2 * p->C * 4);
  p->saved_bytes = off;
  off = kStatusBytes;
  p->wf_T = take(units * cc);
  p->wf_A = take(units * cc);
  p->wf_e = take(units * 2 * p->C * 4);
  p->fwd_bytes = off;
  off = kStatusBytes;
  p->wb_D = take(states * 4);
  p->wb_r = take(rows * 4);
  p->bwd_bytes = off;
  return SSD_OK;
}

#define DELTA_LAUNCH(expr)                      \
  do {                                          \
    prof_before(s);                             \
    cudaError_t e_ = (expr);                    \
    prof_after(s);                              \
    if (e_ != cudaSuccess) return SSD_ERR_CUDA; \
  } while (0)

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_delta_fwd_workspace_bytes(const ssd_delta_problem* prob) {
  DeltaPlan p;
  return make_delta_plan(prob, &p) == SSD_OK ? p.fwd_bytes : 0;
}
size_t ssd_delta_bwd_workspace_bytes(const ssd_delta_problem* prob) {
  DeltaPlan p;
  return make_delta_plan(prob, &p) == SSD_OK ? p.bwd_bytes : 0;
}
size_t ssd_delta_saved_bytes(const ssd_delta_problem* prob) {
  DeltaPlan p;
  return make_delta_plan(prob, &p) == SSD_OK ? p.saved_bytes : 0;
}

int ssd_delta_fwd(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                  const void* beta, const void* initial_states, const int32_t* seq_idx, void* y, void* final_states,
                  void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes, ssd_stream_t stream) {
  DeltaPlan p;
  int rc = make_delta_plan(prob, &p);
  if (rc != SSD_OK) return rc;
  if (prob->flags & (SSD_HAS_DFINAL | SSD_WANT_DINIT)) return SSD_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !g || !beta || !y || !workspace) return SSD_ERR_INVALID_ARGUMENT;
  if (((prob->flags & SSD_HAS_INIT) != 0) != (initial_states != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (((prob->flags & SSD_HAS_SEQ_IDX) != 0) != (seq_idx != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, k, v, g, beta, initial_states, seq_idx, y, final_states, saved, workspace};
  for (const void* ptr : ptrs)
    if (misaligned(ptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < p.fwd_bytes || (saved && saved_bytes < p.saved_bytes)) return SSD_ERR_WORKSPACE_TOO_SMALL;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  DeltaBufs f;
  memset(&f, 0, sizeof(f));
  f.q = q; f.k = k; f.v = v; f.g = g; f.beta = beta;
  f.init = initial_states; f.seq = seq_idx; f.y = y; f.fin = final_states;
  char* sv = static_cast<char*>(saved);
  if (sv) {
    f.S = sv + p.sv_S;
    f.w = sv + p.sv_w;
  }
  char* ws = static_cast<char*>(workspace);
  f.status = reinterpret_cast<int*>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  f.T = sv ? sv + p.sv_T : ws + p.wf_T;
  f.A = sv ? sv + p.sv_A : ws + p.wf_A;
  f.e = sv ? sv + p.sv_e : ws + p.wf_e;
  if (p.tc) {
    DELTA_LAUNCH(launch_delta_prep(p, f, s));
    DELTA_LAUNCH(launch_delta_chain_fwd(p, f, s));
  } else {
    DELTA_LAUNCH(launch_delta_prep_simt(p, f, s));
    DELTA_LAUNCH(launch_delta_chain_simt(p, f, false, s));
  }
  return SSD_OK;
}

int ssd_delta_bwd(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                  const void* beta, const int32_t* seq_idx, const void* dy, const void* dfinal_states, void* dq,
                  void* dk, void* dv, void* dg, void* dbeta, void* dinitial_states, const void* saved,
                  size_t saved_bytes, void* workspace, size_t workspace_bytes, ssd_stream_t stream) {
  DeltaPlan p;
  int rc = make_delta_plan(prob, &p);
  if (rc != SSD_OK) return rc;
  if (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta || !saved || !workspace)
    return SSD_ERR_INVALID_ARGUMENT;
  if (((prob->flags & SSD_HAS_SEQ_IDX) != 0) != (seq_idx != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (((prob->flags & SSD_HAS_DFINAL) != 0) != (dfinal_states != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (((prob->flags & SSD_WANT_DINIT) != 0) != (dinitial_states != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q,  k,  v,  g,  beta,  seq_idx,         dy,    dfinal_states,
                        dq, dk, dv, dg, dbeta, dinitial_states, saved, workspace};
  for (const void* ptr : ptrs)
    if (misaligned(ptr)) return SSD_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < p.bwd_bytes || saved_bytes < p.saved_bytes) return SSD_ERR_WORKSPACE_TOO_SMALL;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  DeltaBufs f;
  memset(&f, 0, sizeof(f));
  f.q = q; f.k = k; f.v = v; f.g = g; f.beta = beta; f.seq = seq_idx;
  f.dy = dy; f.dfin = dfinal_states;
  f.dq = dq; f.dk = dk; f.dv = dv; f.dg = dg; f.dbeta = dbeta; f.dinit = dinitial_states;
  char* sv = static_cast<char*>(const_cast<void*>(saved));
  char* ws = static_cast<char*>(workspace);
  f.S = sv + p.sv_S;
  f.w = sv + p.sv_w;
  f.D = ws + p.wb_D;
  f.r = ws + p.wb_r;
  f.status = reinterpret_cast<int*>(ws);
  f.T = sv + p.sv_T;
  f.A = sv + p.sv_A;
  f.e = sv + p.sv_e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.tc) {
    if (cudaMemsetAsync(f.status, 0, sizeof(int), s) != cudaSuccess) return SSD_ERR_CUDA;
    DELTA_LAUNCH(launch_delta_chain_bwd(p, f, s));
    DELTA_LAUNCH(launch_delta_grad_tc(p, f, s));
  } else {
    DELTA_LAUNCH(launch_delta_chain_simt(p, f, true, s));
    DELTA_LAUNCH(launch_delta_grad(p, f, s));
  }
  return SSD_OK;
}

int ssd_delta_step(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                   const void* beta, int64_t nslots, const float* states_in, float* states_out, const int32_t* slots,
                   const int32_t* lengths, void* y, ssd_stream_t stream) {
  DeltaPlan p;
  int rc = make_delta_plan(prob, &p);
  if (rc != SSD_OK) return rc;
  if (prob->flags != 0 || prob->state_dtype != SSD_F32) return SSD_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !g || !beta || !states_in || (!y && !states_out)) return SSD_ERR_INVALID_ARGUMENT;
  if (nslots < 1 || (!slots && nslots < prob->batch)) return SSD_ERR_INVALID_ARGUMENT;
  if ((double)nslots * (double)prob->nheads * (double)prob->headdim * (double)prob->dstate >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v, g, beta, states_in, states_out, slots, lengths, y};
  for (const void* ptr : ptrs)
    if (misaligned(ptr)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  DeltaBufs f;
  memset(&f, 0, sizeof(f));
  f.q = q; f.k = k; f.v = v; f.g = g; f.beta = beta; f.y = y;
  const DeltaStep st = {states_in, states_out, slots, lengths, nslots};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DELTA_LAUNCH(launch_delta_step(p, f, st, s));
  return SSD_OK;
}

}  // extern "C"
