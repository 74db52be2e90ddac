// k_delta_recurrent.cu -- the gated delta rule token by token: the recurrent
// step on a pool of states, the forward of fp32 problems and of head sizes
// outside the tensor-core set, and the reverse recurrence of their gradient.
//
// The columns of the state (the headdim values p of S) evolve independently:
//   S'[p,:] = a S[p,:];  w = v_p - S'[p,:].k;  S[p,:] = S'[p,:] + beta w k;
//   y_p = scale S[p,:].q
// so a thread group of eight lanes keeps one column's dstate values in fp32
// registers and walks the tokens.  Both dot products are taken of the old
// state in one pass (S.q = a S_old.q + (q.k) beta w), so that a token costs
// one round of three shuffles; the next tokens are on their way meanwhile.  A single token is bound by the state's bytes
// (each read and written once, 16-byte accesses, whole 128-byte lines per
// group); a long sequence by the latency of one token's chain.
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
__device__ __forceinline__ void load_col(float (&S)[NR], const void* base, long long row, int lane, int N, int bf16) {
#pragma unroll
  for (int i = 0; i < NR; i += 4) {
    const int n = elem_n(lane, i);
    if (!bf16 && (N & 3) == 0) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n < N) v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row + n);
      S[i] = v.x; S[i + 1] = v.y; S[i + 2] = v.z; S[i + 3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i + j] = n + j < N ? ld_state(base, row + n + j, bf16) : 0.f;
    }
  }
}
template <int NR>
__device__ __forceinline__ void store_col(const float (&S)[NR], void* base, long long row, int lane, int N, int bf16) {
#pragma unroll
  for (int i = 0; i < NR; i += 4) {
    const int n = elem_n(lane, i);
    if (!bf16 && (N & 3) == 0) {
      if (n < N)
        *reinterpret_cast<float4*>(static_cast<float*>(base) + row + n) =
            make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < N) st_state(base, row + n + j, bf16, S[i + j]);
    }
  }
}

// TOK tokens in shared memory, as fp32
template <int NR, int TOK>
struct Stage {
  float q[TOK][NR * kLanes];
  float k[TOK][NR * kLanes];
  float v[TOK][kCols];   // v of this CTA's columns (the reverse pass: dy)
  float a[TOK], beta[TOK];
  int reset[TOK];
};

// A thread's part of TOK tokens on their way to shared memory: loaded ahead,
// written when the stage is free.
template <typename T, int NR, int TOK>
struct Ahead {
  static constexpr int E = (TOK * NR * kLanes + kThreads - 1) / kThreads;  // q and k values
  static constexpr int EV = (TOK * kCols + kThreads - 1) / kThreads;
  T q[E], k[E], v[EV];
  T g, beta;
  int reset;
  __device__ __forceinline__ void load(const DeltaPlan& p, const DeltaBufs& f, const void* vals, long long vstride,
                                       int bi, int h, int p0, int t0, int n) {
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
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      const int x = threadIdx.x + i * kThreads, t = x / kCols, c = x % kCols;
      v[i] = zero;
      if (t < n && p0 + c < p.P)
        v[i] = static_cast<const T*>(vals)[(tok0 + t) * vstride + (long long)h * p.P + p0 + c];
    }
    g = beta = zero;
    reset = 0;
    if (threadIdx.x < n) {
      const long long i = (tok0 + threadIdx.x) * p.H + h;
      g = static_cast<const T*>(f.g)[i];
      beta = static_cast<const T*>(f.beta)[i];
      reset = f.seq != nullptr && t0 + threadIdx.x > 0 && f.seq[tok0 + threadIdx.x] != f.seq[tok0 + threadIdx.x - 1];
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
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      const int x = threadIdx.x + i * kThreads;
      if (x < TOK * kCols) (&sm.v[0][0])[x] = to_f(v[i]);
    }
    if (threadIdx.x < TOK) {
      sm.a[threadIdx.x] = expf(to_f(g));
      sm.beta[threadIdx.x] = to_f(beta);
      sm.reset[threadIdx.x] = reset;
    }
  }
};

// Forward: kStep takes its states from a pool, else from init; f.S and f.w,
// when given, get the states entering each chunk of p.C tokens and every w.
template <typename T, int NR, int TOK, bool kStep>
__global__ void __launch_bounds__(kThreads, kStep && TOK == 1 && NR <= 16 ? 8 : 1) delta_recurrent_kernel(DeltaPlan p, DeltaBufs f, DeltaStep st) {
  __shared__ Stage<NR, TOK> sm;
  const int ptiles = (p.P + kCols - 1) / kCols;
  const int p0 = (int)(blockIdx.x % ptiles) * kCols;
  const int h = (int)((blockIdx.x / ptiles) % p.H);
  const int bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int lane = threadIdx.x % kLanes, c = threadIdx.x / kLanes;
  const int col = p0 + c;
  const bool live = col < p.P;
  if (!kStep && blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
  float S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) S[i] = 0.f;
  Ahead<T, NR, TOK> ahead;
  ahead.load(p, f, f.v, p.vs, bi, h, p0, 0, min(TOK, p.L));
  int keep = p.L;  // the state after this many tokens is the one that is kept
  long long slot = bi;
  bool pad = false;
  if (kStep) {
    if (st.slots) slot = st.slots[bi];
    pad = slot < 0 || slot >= st.nslots;
    if (st.lengths) keep = min(max(st.lengths[bi], 0), p.L);
    if (live && !pad) load_col<NR>(S, st.in, ((slot * p.H + h) * p.P + col) * p.N, lane, p.N, 0);
  } else if (f.init && live) {
    load_col<NR>(S, f.init, (((long long)bi * p.H + h) * p.P + col) * p.N, lane, p.N, p.st_bf16);
  }
  const long long out_row = ((slot * p.H + h) * p.P + col) * p.N;
  if (kStep && keep == 0 && st.out && live && !pad && st.out != st.in)
    store_col<NR>(S, st.out, out_row, lane, p.N, 0);
  // without y the tokens past the last kept one are not needed
  const int last = kStep && !f.y ? keep : p.L;
  for (int t0 = 0; t0 < last; t0 += TOK) {
    const int n = min(TOK, last - t0);
    if (t0) __syncthreads();
    ahead.put(sm);
    // (no token of this stage starts a sequence: the usual case has no branch)
    const bool resets = __syncthreads_or(ahead.reset);
    if (t0 + TOK < last) ahead.load(p, f, f.v, p.vs, bi, h, p0, t0 + TOK, min(TOK, last - t0 - TOK));
    // (the stages divide the chunks, so that only their first tokens begin one)
    if (!kStep && f.S && t0 % p.C == 0) {
      if (sm.reset[0]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = 0.f;
      }
      if (live)
        store_col<NR>(S, f.S, ((((long long)bi * p.H + h) * p.nc + t0 / p.C) * p.P + col) * p.N, lane, p.N, 0);
    }
    long long o = (((long long)bi * p.L + t0) * p.H + h) * p.P + col;
    auto token = [&](int t, bool checked) {
      if (checked && sm.reset[t]) {
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
      const float a = sm.a[t];
      const float dk = group_sum((sk[0] + sk[1]) + (sk[2] + sk[3]));
      const float dq = group_sum((sq[0] + sq[1]) + (sq[2] + sq[3]));
      const float qk = group_sum((d[0] + d[1]) + (d[2] + d[3]));
      const float w = sm.v[t][c] - a * dk;
      const float u = sm.beta[t] * w;
#pragma unroll
      for (int i = 0; i < NR; ++i) S[i] = a * S[i] + kk[i] * u;
      if (live && lane == 0) {
        if (f.y) {
          const float y = pad ? 0.f : p.scale * (a * dq + qk * u);
          static_cast<T*>(f.y)[o] = from_f<T>(y);
        }
        if (!kStep && f.w) static_cast<float*>(f.w)[o] = w;
      }
      o += (long long)p.H * p.P;
      if (kStep && t0 + t + 1 == keep && st.out && live && !pad) store_col<NR>(S, st.out, out_row, lane, p.N, 0);
    };
    if (resets) {
      for (int t = 0; t < n; ++t) token(t, true);
    } else if (n == TOK) {
#pragma unroll(TOK > 4 ? 4 : TOK)
      for (int t = 0; t < TOK; ++t) token(t, false);
    } else {
      for (int t = 0; t < n; ++t) token(t, false);
    }
  }
  if (!kStep && f.fin && live)
    store_col<NR>(S, f.fin, (((long long)bi * p.H + h) * p.P + col) * p.N, lane, p.N, p.st_bf16);
}

// Reverse: D, the gradient of the state, in the same layout; per token, last
// first, D += scale dy_p q; r = beta k.D; D = a (D - r k).  Writes r (as dv,
// and in fp32 for the gradient kernel) and D after each chunk of p.C tokens.
template <typename T, int NR, int TOK>
__global__ void __launch_bounds__(kThreads) delta_reverse_kernel(DeltaPlan p, DeltaBufs f) {
  __shared__ Stage<NR, TOK> sm;
  const int ptiles = (p.P + kCols - 1) / kCols;
  const int p0 = (int)(blockIdx.x % ptiles) * kCols;
  const int h = (int)((blockIdx.x / ptiles) % p.H);
  const int bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int lane = threadIdx.x % kLanes, c = threadIdx.x / kLanes;
  const int col = p0 + c;
  const bool live = col < p.P;
  const long long state_row = (((long long)bi * p.H + h) * p.P + col) * p.N;
  if (blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
  float D[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) D[i] = 0.f;
  const int first = (p.L - 1) / TOK * TOK;
  const long long dys = (long long)p.H * p.P;
  Ahead<T, NR, TOK> ahead;
  ahead.load(p, f, f.dy, dys, bi, h, p0, first, p.L - first);
  if (f.dfin && live) load_col<NR>(D, f.dfin, state_row, lane, p.N, p.st_bf16);
  for (int t0 = first; t0 >= 0; t0 -= TOK) {
    const int n = min(TOK, p.L - t0);
    __syncthreads();
    ahead.put(sm);
    const bool resets = __syncthreads_or(ahead.reset);
    if (t0 > 0) ahead.load(p, f, f.dy, dys, bi, h, p0, t0 - TOK, TOK);
    // the stages divide the chunks, so that only their last tokens end one
    if (((t0 + n) % p.C == 0 || t0 + n == p.L) && live)
      store_col<NR>(D, f.D, ((((long long)bi * p.H + h) * p.nc + (t0 + n - 1) / p.C) * p.P + col) * p.N, lane, p.N, 0);
    long long o = (((long long)bi * p.L + t0 + n - 1) * p.H + h) * p.P + col;
    auto token = [&](int t, bool checked) {
      const float dy = p.scale * sm.v[t][c];
      float dk[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f}, kk[NR], qq[NR];
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[t][elem_n(lane, i)]);
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[t][elem_n(lane, i)]);
        kk[i] = k4.x; kk[i + 1] = k4.y; kk[i + 2] = k4.z; kk[i + 3] = k4.w;
        qq[i] = q4.x; qq[i + 1] = q4.y; qq[i + 2] = q4.z; qq[i + 3] = q4.w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dk[j] += kk[i + j] * D[i + j];
          d[j] += kk[i + j] * qq[i + j];
        }
      }
      const float kd = group_sum((dk[0] + dk[1]) + (dk[2] + dk[3]));
      const float qk = group_sum((d[0] + d[1]) + (d[2] + d[3]));
      const float r = sm.beta[t] * (kd + qk * dy);
      const float a = sm.a[t];
      if (checked && sm.reset[t]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) D[i] = 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) D[i] = a * (D[i] + qq[i] * dy - kk[i] * r);
      }
      if (live && lane == 0) {
        static_cast<T*>(f.dv)[o] = from_f<T>(r);
        static_cast<float*>(f.r)[o] = r;
      }
      o -= dys;
    };
    if (resets) {
      for (int t = n - 1; t >= 0; --t) token(t, true);
    } else if (n == TOK) {
#pragma unroll 4
      for (int t = TOK - 1; t >= 0; --t) token(t, false);
    } else {
      for (int t = n - 1; t >= 0; --t) token(t, false);
    }
  }
  if (f.dinit && live) store_col<NR>(D, f.dinit, state_row, lane, p.N, p.st_bf16);
}

template <typename T, int NR>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep* st, bool reverse, cudaStream_t s) {
  const long long grid = (long long)((p.P + kCols - 1) / kCols) * p.H * p.b;
  const DeltaStep none = {nullptr, nullptr, nullptr, nullptr, 0};
  constexpr int kTok = NR > 16 ? 8 : 16;  // tokens staged at a time; they divide a chunk of 32
  if (reverse) {
    set_kernel_name("delta_reverse");
    delta_reverse_kernel<T, NR, kTok><<<(unsigned)grid, kThreads, 0, s>>>(p, f);
  } else if (st) {
    set_kernel_name("delta_step");
    if (p.L == 1)  // no shared memory for tokens that are not there
      delta_recurrent_kernel<T, NR, 1, true><<<(unsigned)grid, kThreads, 0, s>>>(p, f, *st);
    else
      delta_recurrent_kernel<T, NR, 4, true><<<(unsigned)grid, kThreads, 0, s>>>(p, f, *st);
  } else {
    set_kernel_name("delta_recurrent");
    delta_recurrent_kernel<T, NR, kTok, false><<<(unsigned)grid, kThreads, 0, s>>>(p, f, none);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_n(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep* st, bool reverse, cudaStream_t s) {
  if (p.N <= 32) return launch_t<T, 4>(p, f, st, reverse, s);
  if (p.N <= 64) return launch_t<T, 8>(p, f, st, reverse, s);
  if (p.N <= 128) return launch_t<T, 16>(p, f, st, reverse, s);
  return launch_t<T, 32>(p, f, st, reverse, s);
}

cudaError_t launch_any(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep* st, bool reverse, cudaStream_t s) {
  return p.bf16 ? launch_n<__nv_bfloat16>(p, f, st, reverse, s) : launch_n<float>(p, f, st, reverse, s);
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return launch_any(p, f, nullptr, false, s);
}
cudaError_t launch_delta_step(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep& st, cudaStream_t s) {
  return launch_any(p, f, &st, false, s);
}
cudaError_t launch_delta_reverse(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return launch_any(p, f, nullptr, true, s);
}

}  // namespace ssd
