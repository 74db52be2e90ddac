// k_delta_step.cu -- the recurrent form of the gated delta rule: the tokens of
// a serving batch (one, or a few drafted ones) on a pool of fp32 states.
//
// The columns of the state (the headdim values p of S) evolve independently:
//   S'[p,:] = a S[p,:];  w = v_p - S'[p,:].k;  S[p,:] = S'[p,:] + beta w k;
//   y_p = scale S[p,:].q
// so a thread group of eight lanes keeps one column's dstate values in fp32
// registers.  Both dot products are taken of the state before the token, in
// one pass (S.q = a S_old.q + (q.k) beta w).  A single token is bound by the
// state's bytes (each read and written once, 16-byte accesses, whole 128-byte
// lines per group).
// Several tokens follow each other through the same registers; their operands
// are staged four tokens at a time, the next four on their way meanwhile.
// (Taking four tokens against one state, with the products that they owe each
// other from tables, costs more for up to eight tokens than it saves: 11.9 us
// against 9.8 at 4 sequences of 5 tokens, 48 heads of 64 x 16.)
// Measured with 64 sequences of one token, 64 heads of 64 x 128: 46 us for 269 MB
// of states, in and out (5.8 TB/s).
#include "delta_internal.cuh"

namespace ssd {
namespace {

constexpr int kLanes = 8;                    // lanes per state column
constexpr int kThreads = 128;
constexpr int kCols = kThreads / kLanes;     // columns per CTA

__device__ __forceinline__ float group_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// The dstate index of a lane's element i: four consecutive values out of
// every 32, so that a group's accesses are contiguous.
__device__ __forceinline__ int elem_n(int lane, int i) { return (i >> 2) * (4 * kLanes) + lane * 4 + (i & 3); }

template <int NR>
__device__ __forceinline__ void load_col(float (&S)[NR], const float* row, int lane, int N) {
#pragma unroll
  for (int i = 0; i < NR; i += 4) {
    const int n = elem_n(lane, i);
    if ((N & 3) == 0) {
      const float4 v = n < N ? __ldcs(reinterpret_cast<const float4*>(row + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i] = v.x; S[i + 1] = v.y; S[i + 2] = v.z; S[i + 3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i + j] = n + j < N ? row[n + j] : 0.f;
    }
  }
}
template <int NR>
__device__ __forceinline__ void store_col(const float (&S)[NR], float* row, int lane, int N) {
#pragma unroll
  for (int i = 0; i < NR; i += 4) {
    const int n = elem_n(lane, i);
    if ((N & 3) == 0) {
      if (n < N) __stcs(reinterpret_cast<float4*>(row + n), make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < N) row[n + j] = S[i + j];
    }
  }
}

// TOK tokens in shared memory, as fp32.
template <int NR, int TOK>
struct Stage {
  float q[TOK][NR * kLanes], k[TOK][NR * kLanes];
  float v[TOK][kCols];  // v of this CTA's columns
  float a[TOK], beta[TOK];
};

// A thread's part of TOK tokens on their way to shared memory: loaded ahead,
// written when the stage is free.  Tokens past n are zeros with decay 1.
template <typename T, int NR, int TOK>
struct Ahead {
  static constexpr int E = (TOK * NR * kLanes + kThreads - 1) / kThreads;
  T q[E], k[E], v, g, beta;
  __device__ __forceinline__ void load(const DeltaPlan& p, const DeltaBufs& f, int bi, int h, int p0, int t0, int n) {
    const int grp = h / p.hpg;
    const long long tok0 = (long long)bi * p.L + t0;
    const T zero = from_f<T>(0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int x = threadIdx.x + i * kThreads, t = x / (NR * kLanes), e = x % (NR * kLanes);
      q[i] = k[i] = zero;
      if (t < n && e < p.N) {
        q[i] = static_cast<const T*>(f.q)[(tok0 + t) * p.qs + (long long)grp * p.N + e];
        k[i] = static_cast<const T*>(f.k)[(tok0 + t) * p.ks + (long long)grp * p.N + e];
      }
    }
    v = g = beta = zero;
    const int t = threadIdx.x / kCols, c = threadIdx.x % kCols;
    if (t < n && p0 + c < p.P) v = static_cast<const T*>(f.v)[(tok0 + t) * p.vs + (long long)h * p.P + p0 + c];
    if (threadIdx.x < n) {
      const long long i = (tok0 + threadIdx.x) * p.H + h;
      g = static_cast<const T*>(f.g)[i];
      beta = static_cast<const T*>(f.beta)[i];
    }
  }
  __device__ __forceinline__ void put(Stage<NR, TOK>& sm) const {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int x = threadIdx.x + i * kThreads;
      if (x >= TOK * NR * kLanes) break;
      (&sm.q[0][0])[x] = to_f(q[i]);
      (&sm.k[0][0])[x] = to_f(k[i]);
    }
    if (threadIdx.x < TOK * kCols) (&sm.v[0][0])[threadIdx.x] = to_f(v);
    if (threadIdx.x < TOK) {
      sm.a[threadIdx.x] = to_f(g) < kForget ? 0.f : expf(to_f(g));  // 0: the state is forgotten
      sm.beta[threadIdx.x] = to_f(beta);
    }
  }
};

// TOK = 1 for single tokens, 4 for more.  Eight CTAs of single tokens to an
// SM: 64 KB of states in flight there.
template <typename T, int NR, int TOK>
__global__ void __launch_bounds__(kThreads, TOK == 1 && NR <= 16 ? 8 : 1)
    delta_step_kernel(DeltaPlan p, DeltaBufs f, DeltaStep st) {
  __shared__ Stage<NR, TOK> sm;
  const int ptiles = (p.P + kCols - 1) / kCols;
  const int p0 = (int)(blockIdx.x % ptiles) * kCols;
  const int h = (int)((blockIdx.x / ptiles) % p.H);
  const int bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int lane = threadIdx.x % kLanes, c = threadIdx.x / kLanes, col = p0 + c;
  const bool live = col < p.P;
  const long long slot = st.slots ? st.slots[bi] : bi;
  const bool pad = slot < 0 || slot >= st.nslots;  // no sequence: y is zero, no state is touched
  const long long row = ((slot * p.H + h) * p.P + col) * p.N;
  Ahead<T, NR, TOK> ahead;
  ahead.load(p, f, bi, h, p0, 0, min(TOK, p.L));
  float S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) S[i] = 0.f;
  if (live && !pad) load_col<NR>(S, st.in + row, lane, p.N);
  // the state after this many tokens is the one that is kept
  const int keep = st.lengths ? min(max(st.lengths[bi], 0), p.L) : p.L;
  const bool put = st.out && live && !pad;
  if (put && keep == 0 && st.out != st.in) store_col<NR>(S, st.out + row, lane, p.N);
  // without y the tokens past the last kept one are not needed
  const int last = f.y ? p.L : keep;
  for (int t0 = 0; t0 < last; t0 += TOK) {
    const int n = min(TOK, last - t0);
    if (t0) __syncthreads();
    ahead.put(sm);
    __syncthreads();
    const long long o = (((long long)bi * p.L + t0) * p.H + h) * p.P + col;
    if (t0 + TOK < last) ahead.load(p, f, bi, h, p0, t0 + TOK, min(TOK, last - t0 - TOK));
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t >= n) break;
      const float a = sm.a[t];
      if (a == 0.f) {  // whatever it holds
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = 0.f;
      }
      float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f}, kk[NR];
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[t][elem_n(lane, i)]);
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[t][elem_n(lane, i)]);
        kk[i] = k4.x; kk[i + 1] = k4.y; kk[i + 2] = k4.z; kk[i + 3] = k4.w;
        sk[0] += k4.x * S[i]; sk[1] += k4.y * S[i + 1]; sk[2] += k4.z * S[i + 2]; sk[3] += k4.w * S[i + 3];
        sq[0] += q4.x * S[i]; sq[1] += q4.y * S[i + 1]; sq[2] += q4.z * S[i + 2]; sq[3] += q4.w * S[i + 3];
        d[0] += k4.x * q4.x; d[1] += k4.y * q4.y; d[2] += k4.z * q4.z; d[3] += k4.w * q4.w;
      }
      const float dk = group_sum((sk[0] + sk[1]) + (sk[2] + sk[3]));
      const float dq = group_sum((sq[0] + sq[1]) + (sq[2] + sq[3]));
      const float qk = group_sum((d[0] + d[1]) + (d[2] + d[3]));
      const float u = sm.beta[t] * (sm.v[t][c] - a * dk);
#pragma unroll
      for (int i = 0; i < NR; ++i) S[i] = a * S[i] + kk[i] * u;
      if (live && lane == 0 && f.y)
        static_cast<T*>(f.y)[o + (long long)t * p.H * p.P] = from_f<T>(pad ? 0.f : p.scale * (a * dq + qk * u));
      if (put && t0 + t + 1 == keep) store_col<NR>(S, st.out + row, lane, p.N);
    }
  }
}

template <typename T, int NR>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep& st, cudaStream_t s) {
  const long long grid = (long long)((p.P + kCols - 1) / kCols) * p.H * p.b;
  set_kernel_name("delta_step");
  if (p.L == 1)
    delta_step_kernel<T, NR, 1><<<(unsigned)grid, kThreads, 0, s>>>(p, f, st);
  else
    delta_step_kernel<T, NR, 4><<<(unsigned)grid, kThreads, 0, s>>>(p, f, st);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_n(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep& st, cudaStream_t s) {
  if (p.N <= 32) return launch_t<T, 4>(p, f, st, s);
  if (p.N <= 64) return launch_t<T, 8>(p, f, st, s);
  if (p.N <= 128) return launch_t<T, 16>(p, f, st, s);
  return launch_t<T, 32>(p, f, st, s);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep& st, cudaStream_t s) {
  return p.bf16 ? launch_n<__nv_bfloat16>(p, f, st, s) : launch_n<float>(p, f, st, s);
}

}  // namespace ssd
