// delta_internal.cuh -- plan of one gated-delta-rule problem, shared by the
// host entry points (ssd_delta_api.cu) and the kernels.
//
// The algebra of a chunk of C tokens, used by every kernel.  With gam the
// cumulative log decay inside the chunk (inclusive), S0 the state entering it
// (headdim x dstate; written here as dstate x headdim so that a token's key
// multiplies from the left), E_ij = exp(gam_i - gam_j) for j <= i in one
// sequence (else 0), e_i = exp(gam_i) while the entering state's sequence
// lasts (else 0), o_j = E_{C-1,j}:
//
//   w_i  = v_i - e_i k_i S0 - sum_{j<i} E_ij (k_i.k_j) beta_j w_j    (u_i = beta_i w_i)
//   y_i  = scale (e_i q_i S0 + sum_{j<=i} E_ij (q_i.k_j) beta_j w_j)
//   S1   = e_{C-1} S0 + sum_j o_j beta_j k_j^T w_j
//
// and its reverse, given D1 = dL/dS1 (r_i = dL/dv_i):
//
//   r_j  = beta_j (scale sum_{i>=j} E_ij (q_i.k_j) dy_i + o_j k_j D1
//                  - sum_{i>j} E_ij (k_i.k_j) r_i)
//   D0   = e_{C-1} D1 + sum_i e_i (scale q_i^T dy_i - k_i^T r_i)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd_internal.cuh"

namespace ssd {

struct DeltaPlan {
  int b, L, H, P, N, G, hpg;
  long long qs, ks, vs;  // elements from token to token
  float scale;
  int bf16, st_bf16;     // dtype, state_dtype
  int tc;                // the tensor-core kernels run this problem
  int C, nc;             // chunk length of the saved states, chunks per row
  // byte offsets in `saved`
  size_t sv_S, sv_w, sv_T, sv_A, sv_e, saved_bytes;
  // forward workspace (T, A and e when there is no `saved`), backward workspace
  size_t wf_T, wf_A, wf_e, fwd_bytes;
  size_t wb_D, wb_r, bwd_bytes;
};

// Device pointers of one call, passed by value to every kernel.
struct DeltaBufs {
  const void *q, *k, *v, *g, *beta;
  const void* init;
  const int32_t* seq;
  void* y;
  void* fin;
  const void *dy, *dfin;
  void *dq, *dk, *dv, *dg, *dbeta, *dinit;
  // fp32 kernels: S (b,H,nc,P,N) states entering each chunk, w (b,L,H,P),
  // D (b,H,nc,P,N) gradients of the state after each chunk, r (b,L,H,P),
  // T = (I + M)^-1 and A (b,H,nc,C,C), e (b,H,nc,2,C).  Tensor-core kernels:
  // bf16 S, D (b,H,nc,P,N), w transposed (b,H,nc,P,C), T and A (b,H,nc,C,C; see
  // k_delta_prep.cu), and fp32 gate records e (b,H,nc,kGateRows,C); r is dv.
  void *S, *w, *T, *A, *e, *D, *r;
  int* status;  // device status word, at the start of the workspace
};

// Pool arguments of the recurrent step.
struct DeltaStep {
  const float* in;
  float* out;
  const int32_t* slots;
  const int32_t* lengths;
  long long nslots;
};

__device__ __forceinline__ float ld_state(const void* p, long long i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void st_state(void* p, long long i, int bf16, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// A log decay below this counts as -inf: exp of it is no normal fp32 number,
// and sums that held such a term would lose the digits of the others.
constexpr float kForget = -100.0f;

// The decays' running sum over a chunk of the fp32 kernels, a token a lane, in
// two parts: differences of it are taken before it is rounded.  (31 decays may sum
// to -3000, which fp32 holds to 2e-4, while the pairs behind them differ by 1e-2.)
// starts becomes the number of sequence starts up to the lane.
struct GateSum {
  float hi, lo;
};
__device__ __forceinline__ GateSum gate_sum(float g, int& starts, int lane) {
  double sum = g;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double ug = __shfl_up_sync(0xffffffffu, sum, o);
    const int us = __shfl_up_sync(0xffffffffu, starts, o);
    if (lane >= o) {
      sum += ug;
      starts += us;
    }
  }
  const float hi = (float)sum;
  return {hi, (float)(sum - hi)};
}

constexpr int kDeltaChunk = 64;  // tokens per chunk of the tensor-core kernels
// Rows of a chunk's gate record (fp32): e_i; o_j beta_j; gam_i log2(e); beta;
// o_j; the decay between token 32 and the token (of the second half's rows
// from it, of the first half's columns to it; 0 across a sequence start); and
// the number of sequence starts up to the token (an int).
enum { kGateE, kGateOB, kGateGam, kGateBeta, kGateO, kGateHalf, kGateSeg, kGateRows };

constexpr int kDeltaChunkF32 = 32;  // and of the fp32 kernels

cudaError_t launch_delta_step(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep& st, cudaStream_t s);
// the fp32 kernels
cudaError_t launch_delta_prep_simt(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);
cudaError_t launch_delta_chain_simt(const DeltaPlan& p, const DeltaBufs& f, bool reverse, cudaStream_t s);
cudaError_t launch_delta_grad(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);

// the tensor-core kernels
cudaError_t launch_delta_prep(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);
cudaError_t launch_delta_chain_fwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);
cudaError_t launch_delta_chain_bwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);
cudaError_t launch_delta_grad_tc(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s);

int device_check();

}  // namespace ssd
