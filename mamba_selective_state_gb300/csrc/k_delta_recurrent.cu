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
// one round of three shuffles.  A single token is bound by the state's bytes
// (each read and written once, 16-byte accesses, whole 128-byte lines per
// group); a long sequence by the latency of one token's chain.
#include "delta_internal.cuh"

namespace ssd {
namespace {

constexpr int kLanes = 8;                    // lanes per state column
constexpr int kThreads = 128;
constexpr int kCols = kThreads / kLanes;     // columns per CTA
constexpr int kTok = 16;                     // tokens staged at a time

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

template <int NR>
struct Stage {
  float q[kTok][NR * kLanes];
  float k[kTok][NR * kLanes];
  float v[kTok][kCols];   // v of this CTA's columns (the reverse pass: dy)
  float a[kTok], beta[kTok], qk[kTok];
  int reset[kTok];
};

// One chunk of tokens [t0, t0 + n) into shared memory, as fp32.
template <typename T, int NR>
__device__ __forceinline__ void stage_tokens(Stage<NR>& sm, const DeltaPlan& p, const DeltaBufs& f, const void* vals,
                                             long long vstride, int bi, int h, int p0, int t0, int n) {
  const int grp = h / p.hpg;
  const long long tok0 = (long long)bi * p.L + t0;
  const T* q = static_cast<const T*>(f.q);
  const T* k = static_cast<const T*>(f.k);
  for (int i = threadIdx.x; i < n * NR * kLanes; i += kThreads) {
    const int t = i / (NR * kLanes), e = i % (NR * kLanes);
    float qv = 0.f, kv = 0.f;
    if (e < p.N) {
      qv = to_f(q[(tok0 + t) * p.qs + (long long)grp * p.N + e]);
      kv = to_f(k[(tok0 + t) * p.ks + (long long)grp * p.N + e]);
    }
    sm.q[t][e] = qv;
    sm.k[t][e] = kv;
  }
  for (int i = threadIdx.x; i < n * kCols; i += kThreads) {
    const int t = i / kCols, c = i % kCols;
    sm.v[t][c] = p0 + c < p.P ? to_f(static_cast<const T*>(vals)[(tok0 + t) * vstride + (long long)h * p.P + p0 + c])
                              : 0.f;
  }
  if (threadIdx.x < n) {
    const int t = threadIdx.x;
    const long long i = (tok0 + t) * p.H + h;
    sm.a[t] = expf(to_f(static_cast<const T*>(f.g)[i]));
    sm.beta[t] = to_f(static_cast<const T*>(f.beta)[i]);
    sm.reset[t] = f.seq != nullptr && t0 + t > 0 && f.seq[tok0 + t] != f.seq[tok0 + t - 1];
  }
}

// q.k of every staged token, one warp at a time over the tokens.
template <int NR>
__device__ __forceinline__ void token_dots(Stage<NR>& sm, int n) {
  const int lane = threadIdx.x & 31;
  for (int t = threadIdx.x >> 5; t < n; t += kThreads / 32) {
    float d = 0.f;
    for (int e = lane; e < NR * kLanes; e += 32) d += sm.q[t][e] * sm.k[t][e];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) sm.qk[t] = d;
  }
}

// Forward: kStep takes its states from a pool, else from init; f.S and f.w,
// when given, get the states entering each chunk of p.C tokens and every w.
template <typename T, int NR, bool kStep>
__global__ void __launch_bounds__(kThreads) delta_recurrent_kernel(DeltaPlan p, DeltaBufs f, DeltaStep st) {
  __shared__ Stage<NR> sm;
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
  for (int t0 = 0; t0 < last; t0 += kTok) {
    const int n = min(kTok, last - t0);
    if (t0) __syncthreads();
    stage_tokens<T, NR>(sm, p, f, f.v, p.vs, bi, h, p0, t0, n);
    __syncthreads();
    token_dots<NR>(sm, n);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      if (sm.reset[t]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = 0.f;
      }
      if (!kStep && f.S && (t0 + t) % p.C == 0 && live)
        store_col<NR>(S, f.S, ((((long long)bi * p.H + h) * p.nc + (t0 + t) / p.C) * p.P + col) * p.N, lane, p.N, 0);
      float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, kk[NR];
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[t][elem_n(lane, i)]);
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[t][elem_n(lane, i)]);
        kk[i] = k4.x; kk[i + 1] = k4.y; kk[i + 2] = k4.z; kk[i + 3] = k4.w;
        sk[0] += k4.x * S[i]; sk[1] += k4.y * S[i + 1]; sk[2] += k4.z * S[i + 2]; sk[3] += k4.w * S[i + 3];
        sq[0] += q4.x * S[i]; sq[1] += q4.y * S[i + 1]; sq[2] += q4.z * S[i + 2]; sq[3] += q4.w * S[i + 3];
      }
      const float a = sm.a[t];
      const float dk = group_sum((sk[0] + sk[1]) + (sk[2] + sk[3]));
      const float dq = group_sum((sq[0] + sq[1]) + (sq[2] + sq[3]));
      const float w = sm.v[t][c] - a * dk;
      const float u = sm.beta[t] * w;
#pragma unroll
      for (int i = 0; i < NR; ++i) S[i] = a * S[i] + kk[i] * u;
      if (live && lane == 0) {
        const long long o = (((long long)bi * p.L + t0 + t) * p.H + h) * p.P + col;
        if (f.y) {
          const float y = pad ? 0.f : p.scale * (a * dq + sm.qk[t] * u);
          static_cast<T*>(f.y)[o] = from_f<T>(y);
        }
        if (!kStep && f.w) static_cast<float*>(f.w)[o] = w;
      }
      if (kStep && t0 + t + 1 == keep && st.out && live && !pad) store_col<NR>(S, st.out, out_row, lane, p.N, 0);
    }
  }
  if (!kStep && f.fin && live)
    store_col<NR>(S, f.fin, (((long long)bi * p.H + h) * p.P + col) * p.N, lane, p.N, p.st_bf16);
}

// Reverse: D, the gradient of the state, in the same layout; per token, last
// first, D += scale dy_p q; r = beta k.D; D = a (D - r k).  Writes r (as dv,
// and in fp32 for the gradient kernel) and D after each chunk of p.C tokens.
template <typename T, int NR>
__global__ void __launch_bounds__(kThreads) delta_reverse_kernel(DeltaPlan p, DeltaBufs f) {
  __shared__ Stage<NR> sm;
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
  if (f.dfin && live) load_col<NR>(D, f.dfin, state_row, lane, p.N, p.st_bf16);
  for (int t0 = (p.L - 1) / kTok * kTok; t0 >= 0; t0 -= kTok) {
    const int n = min(kTok, p.L - t0);
    __syncthreads();
    stage_tokens<T, NR>(sm, p, f, f.dy, (long long)p.H * p.P, bi, h, p0, t0, n);
    __syncthreads();
    token_dots<NR>(sm, n);
    __syncthreads();
    for (int t = n - 1; t >= 0; --t) {
      const int tt = t0 + t;
      if (((tt + 1) % p.C == 0 || tt + 1 == p.L) && live)
        store_col<NR>(D, f.D, ((((long long)bi * p.H + h) * p.nc + tt / p.C) * p.P + col) * p.N, lane, p.N, 0);
      const float dy = p.scale * sm.v[t][c];
      float dk[4] = {0.f, 0.f, 0.f, 0.f}, kk[NR], qq[NR];
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[t][elem_n(lane, i)]);
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[t][elem_n(lane, i)]);
        kk[i] = k4.x; kk[i + 1] = k4.y; kk[i + 2] = k4.z; kk[i + 3] = k4.w;
        qq[i] = q4.x; qq[i + 1] = q4.y; qq[i + 2] = q4.z; qq[i + 3] = q4.w;
#pragma unroll
        for (int j = 0; j < 4; ++j) dk[j] += kk[i + j] * D[i + j];
      }
      const float kd = group_sum((dk[0] + dk[1]) + (dk[2] + dk[3]));
      const float r = sm.beta[t] * (kd + sm.qk[t] * dy);
      const float a = sm.reset[t] ? 0.f : sm.a[t];
      if (sm.reset[t]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) D[i] = 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) D[i] = a * (D[i] + qq[i] * dy - kk[i] * r);
      }
      if (live && lane == 0) {
        const long long o = (((long long)bi * p.L + tt) * p.H + h) * p.P + col;
        static_cast<T*>(f.dv)[o] = from_f<T>(r);
        static_cast<float*>(f.r)[o] = r;
      }
    }
  }
  if (f.dinit && live) store_col<NR>(D, f.dinit, state_row, lane, p.N, p.st_bf16);
}

template <typename T, int NR>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, const DeltaStep* st, bool reverse, cudaStream_t s) {
  const long long grid = (long long)((p.P + kCols - 1) / kCols) * p.H * p.b;
  const DeltaStep none = {nullptr, nullptr, nullptr, nullptr, 0};
  if (reverse) {
    set_kernel_name("delta_reverse");
    delta_reverse_kernel<T, NR><<<(unsigned)grid, kThreads, 0, s>>>(p, f);
  } else if (st) {
    set_kernel_name("delta_step");
    delta_recurrent_kernel<T, NR, true><<<(unsigned)grid, kThreads, 0, s>>>(p, f, *st);
  } else {
    set_kernel_name("delta_recurrent");
    delta_recurrent_kernel<T, NR, false><<<(unsigned)grid, kThreads, 0, s>>>(p, f, none);
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
