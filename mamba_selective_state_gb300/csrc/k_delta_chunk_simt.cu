// k_delta_chunk_simt.cu -- the gated delta rule in fp32, by chunks of 32
// tokens, for fp32 problems and for head sizes outside the tensor-core set:
// the chunks' preparation, and the state's way through them, forward and
// reverse (the formulas of delta_internal.cuh).
//
// Token by token the chain is 110 cycles of latency and 80 instructions a warp
// for each token; by chunks it is a few products of 32 rows whose terms are
// independent.  The preparation (everything that does not depend on the state,
// the inverse of the triangular system among it) runs for all chunks at once;
// a chain's CTA keeps 16 columns of its head's state in shared memory and does
// four products a chunk, four columns and one token (or state row) a thread,
// with the next chunk's operands on their way to registers.  Measured: 102 us
// forward and 105 reverse for 32 chunks of 12 heads of 40 x 56 (36 CTAs), 5,900
// cycles and 1,970 instructions a warp for a chunk.  Bound by shared memory's
// pipe (2.9 passes for each of 250 loads a warp) and the latency of the products
// it feeds: four more warps that take the loads, the outputs and Q S off the
// chain did not help (100 and 107 us, and 690 instead of 478 us where the SMs
// are full), nor did longer unrolled loops; two warps a sub-partition with half
// the columns each took 2.5 times as long.
#include "delta_internal.cuh"

namespace ssd {
namespace {

constexpr int kC = kDeltaChunkF32;
constexpr int kPrep = 256;     // threads of the preparation
constexpr int kThreads = 128;  // of a chain: 32 tokens (or state rows) x 4 quadruples of columns
constexpr int kCols = 16;      // headdim columns per CTA
constexpr int kSs = 20;        // row stride of the 16-column tiles
constexpr int kTs = kC + 4;    // row stride of the 32 x 32 tiles
constexpr int kRec = 2 * kC;   // a chunk's gates: e_i, o_j beta_j

__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void sts4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void fma4(float4& a, float x, float4 y) {
  a.x += x * y.x;
  a.y += x * y.y;
  a.z += x * y.z;
  a.w += x * y.w;
}
__device__ __forceinline__ float4 mul4(float x, float4 y) { return make_float4(x * y.x, x * y.y, x * y.z, x * y.w); }
// x y, and zero where x is, whatever y holds
__device__ __forceinline__ float4 scaled(float x, float4 y) {
  return x == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : mul4(x, y);
}
__device__ __forceinline__ float part(float4 v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// T = (I + M)^-1, A and the gates of every chunk; a warp per head.
template <typename T>
__global__ void __launch_bounds__(kPrep) delta_prep_simt_kernel(DeltaPlan p, DeltaBufs f, int heads_per_cta) {
  extern __shared__ float sh[];
  const int np = (p.N + 3) & ~3, ks = np + 4;
  float* q_s = sh;                        // [kC][ks]
  float* k_s = q_s + kC * ks;
  float* qk_s = k_s + kC * ks;            // [kC][kTs]
  float* kk_s = qk_s + kC * kTs;
  float* M_s = kk_s + kC * kTs;           // [8][kC][kTs] by warp
  float* g_s = M_s + 8 * kC * kTs;        // [8][3][kC]: gam in two parts, beta
  int* s_s = reinterpret_cast<int*>(g_s + 8 * 3 * kC);  // [8][kC]
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int nsplit = (p.hpg + heads_per_cta - 1) / heads_per_cta;
  long long idx = blockIdx.x;
  const int sp = (int)(idx % nsplit);
  idx /= nsplit;
  const int c = (int)(idx % p.nc);
  idx /= p.nc;
  const int grp = (int)(idx % p.G), bi = (int)(idx / p.G);
  const int t0 = c * kC, n = min(kC, p.L - t0);
  const long long tok0 = (long long)bi * p.L + t0;
  if (blockIdx.x == 0 && tid == 0) *f.status = 0;
  for (int i = tid; i < kC * np; i += kPrep) {
    const int t = i / np, e = i % np;
    float q = 0.f, k = 0.f;
    if (t < n && e < p.N) {
      q = to_f(static_cast<const T*>(f.q)[(tok0 + t) * p.qs + (long long)grp * p.N + e]);
      k = to_f(static_cast<const T*>(f.k)[(tok0 + t) * p.ks + (long long)grp * p.N + e]);
    }
    q_s[t * ks + e] = q;
    k_s[t * ks + e] = k;
  }
  __syncthreads();
  {
    const int i = tid >> 3, j0 = tid & 7;
    float kk[4] = {0.f, 0.f, 0.f, 0.f}, qk[4] = {0.f, 0.f, 0.f, 0.f};
    for (int e = 0; e < np; e += 4) {
      const float4 k = lds4(k_s + i * ks + e), q = lds4(q_s + i * ks + e);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float4 x = lds4(k_s + (j0 + 8 * m) * ks + e);
        kk[m] += k.x * x.x + k.y * x.y + k.z * x.z + k.w * x.w;
        qk[m] += q.x * x.x + q.y * x.y + q.z * x.z + q.w * x.w;
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      qk_s[i * kTs + j0 + 8 * m] = qk[m];
      kk_s[i * kTs + j0 + 8 * m] = kk[m];
    }
  }
  __syncthreads();
  const int h0 = grp * p.hpg + sp * heads_per_cta, h1 = min(h0 + heads_per_cta, (grp + 1) * p.hpg);
  float* M = M_s + w * kC * kTs;
  float* gam = g_s + w * 3 * kC;
  float* gam_lo = gam + kC;
  float* bet = gam_lo + kC;
  int* seg = s_s + w * kC;
  for (int h = h0 + w; h < h1; h += kPrep / 32) {
    const long long unit = ((long long)bi * p.H + h) * p.nc + c;
    float g = 0.f, be = 0.f;
    int rs = 0;
    if (lane < n) {
      const long long o = (tok0 + lane) * p.H + h;
      g = to_f(static_cast<const T*>(f.g)[o]);
      be = to_f(static_cast<const T*>(f.beta)[o]);
      rs = (f.seq != nullptr && t0 + lane > 0 && f.seq[tok0 + lane] != f.seq[tok0 + lane - 1]) || g < kForget;
      if (rs) g = 0.f;
    }
    const GateSum sum = gate_sum(g, rs, lane);
    const float hi = sum.hi, lo = sum.lo, hi_last = __shfl_sync(0xffffffffu, hi, 31),
                lo_last = __shfl_sync(0xffffffffu, lo, 31);
    const int slast = __shfl_sync(0xffffffffu, rs, 31);
    __syncwarp();
    gam[lane] = hi;
    gam_lo[lane] = lo;
    bet[lane] = be;
    seg[lane] = rs;
    float* rec = static_cast<float*>(f.e) + unit * kRec;
    rec[lane] = rs == 0 ? expf(hi) : 0.f;
    rec[kC + lane] = rs == slast ? expf((hi_last - hi) + (lo_last - lo)) * be : 0.f;
    __syncwarp();
    // column `lane` of M and A
    float* A = static_cast<float*>(f.A) + unit * kC * kC;
    for (int i = 0; i < kC; ++i) {
      const float E = (lane <= i) & (seg[i] == rs) ? expf((gam[i] - hi) + (gam_lo[i] - lo)) * be : 0.f;
      M[i * kTs + lane] = lane < i ? E * kk_s[i * kTs + lane] : 0.f;
      A[i * kC + lane] = p.scale * E * qk_s[i * kTs + lane];
    }
    __syncwarp();
    // column `lane` of the inverse by forward substitution, four known values at a time
    float x[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
    for (int jb = 0; jb < kC; jb += 4)
#pragma unroll
      for (int i = jb + 1; i < kC; ++i) {
        const float4 m = lds4(M + i * kTs + jb);  // zeros from the diagonal on
        x[i] -= m.x * x[jb];
        if (i > jb + 1) x[i] -= m.y * x[jb + 1];
        if (i > jb + 2) x[i] -= m.z * x[jb + 2];
        if (i > jb + 3) x[i] -= m.w * x[jb + 3];
      }
    float* Tg = static_cast<float*>(f.T) + unit * kC * kC;
#pragma unroll
    for (int i = 0; i < kC; ++i) Tg[i * kC + lane] = x[i];
  }
}

// A thread's part of a chunk's operands on their way to shared memory.
template <typename T, int NP>
struct ChunkAhead {
  static constexpr int E = kC * NP / kThreads, V = kC * kCols / kThreads, R = kC * kC / kThreads;
  T q[E], k[E], v[V];
  float tt[R], aa[R], rec;
  __device__ __forceinline__ void load(const DeltaPlan& p, const DeltaBufs& f, const void* vals, long long vstride,
                                       int bi, int h, int p0, int c) {
    const int grp = h / p.hpg, t0 = c * kC, n = min(kC, p.L - t0);
    const long long tok0 = (long long)bi * p.L + t0, unit = ((long long)bi * p.H + h) * p.nc + c;
    const T zero = from_f<T>(0.f);
    const int e = threadIdx.x % NP, t1 = threadIdx.x / NP;
    constexpr int dt = kThreads >= NP ? kThreads / NP : 1;  // tokens a round (NP = 256: two rounds a token)
    const T* qp = static_cast<const T*>(f.q) + tok0 * p.qs + (long long)grp * p.N;
    const T* kp = static_cast<const T*>(f.k) + tok0 * p.ks + (long long)grp * p.N;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int t = NP > kThreads ? i / (NP / kThreads) : t1 + i * dt;
      const int ee = NP > kThreads ? threadIdx.x + (i % (NP / kThreads)) * kThreads : e;
      q[i] = k[i] = zero;
      if (t < n && ee < p.N) {
        q[i] = qp[t * p.qs + ee];
        k[i] = kp[t * p.ks + ee];
      }
    }
    const int col = threadIdx.x % kCols;
    const T* vp = static_cast<const T*>(vals) + tok0 * vstride + (long long)h * p.P + p0 + col;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int t = threadIdx.x / kCols + i * (kThreads / kCols);
      v[i] = t < n && p0 + col < p.P ? vp[t * vstride] : zero;
    }
    const float* tp = static_cast<const float*>(f.T) + unit * kC * kC + threadIdx.x;
    const float* ap = static_cast<const float*>(f.A) + unit * kC * kC + threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      tt[i] = tp[i * kThreads];
      aa[i] = ap[i * kThreads];
    }
    rec = threadIdx.x < kRec ? static_cast<const float*>(f.e)[unit * kRec + threadIdx.x] : 0.f;
  }
};

template <int NP>
struct ChunkSmem {
  static constexpr int ks = NP + 4;
  float q[kC][ks], k[kC][ks];
  float S[NP][kSs];
  float T[kC][kTs], A[kC][kTs];  // the reverse chain: their transposes
  float v[kC][kSs];              // v; the reverse chain: dy, then scale e dy
  float R[kC][kSs];              // the right-hand side; forward: then o beta w
  float w[kC][kSs];              // w; the reverse chain: -e r
  float e[kRec];
};

template <typename T, int NP, bool kReverse>
__device__ __forceinline__ void put_chunk(ChunkSmem<NP>& sm, const ChunkAhead<T, NP>& a) {
#pragma unroll
  for (int i = 0; i < ChunkAhead<T, NP>::E; ++i) {
    const int x = threadIdx.x + i * kThreads;
    sm.q[x / NP][x % NP] = to_f(a.q[i]);
    sm.k[x / NP][x % NP] = to_f(a.k[i]);
  }
#pragma unroll
  for (int i = 0; i < ChunkAhead<T, NP>::V; ++i) {
    const int x = threadIdx.x + i * kThreads;
    sm.v[x / kCols][x % kCols] = to_f(a.v[i]);
  }
#pragma unroll
  for (int i = 0; i < ChunkAhead<T, NP>::R; ++i) {
    const int x = threadIdx.x + i * kThreads, r = x / kC, col = x % kC;
    if (kReverse) {
      sm.T[col][r] = a.tt[i];
      sm.A[col][r] = a.aa[i];
    } else {
      sm.T[r][col] = a.tt[i];
      sm.A[r][col] = a.aa[i];
    }
  }
  if (threadIdx.x < kRec) sm.e[threadIdx.x] = a.rec;
}

// acc += columns j0 .. j1 of a triangle's row X times Y (bounds of the warp's
// rows: what lies above the diagonal is zero)
__device__ __forceinline__ void tri(float4& acc, const float* X, const float (*Y)[kSs], int j0, int j1, int pp) {
#pragma unroll 2
  for (int j = j0; j < j1; j += 4) {
    const float4 x = lds4(X + j);
    fma4(acc, x.x, lds4(&Y[j][pp]));
    fma4(acc, x.y, lds4(&Y[j + 1][pp]));
    fma4(acc, x.z, lds4(&Y[j + 2][pp]));
    fma4(acc, x.w, lds4(&Y[j + 3][pp]));
  }
}

// The CTA's columns of a state: global (P, N) <-> shared [n][column]
template <int NP>
__device__ __forceinline__ void read_state(ChunkSmem<NP>& sm, const DeltaPlan& p, const void* src, long long base,
                                           int p0) {
  for (int x = threadIdx.x; x < NP * kCols; x += kThreads) {
    const int col = x / NP, n = x % NP;
    sm.S[n][col] = src && n < p.N && p0 + col < p.P ? ld_state(src, base + (long long)col * p.N + n, p.st_bf16) : 0.f;
  }
}
// (four values of a column to a thread: two threads fill a 32-byte sector; zeros
// for a state that nobody sees)
template <int NP>
__device__ __forceinline__ void write_state(const ChunkSmem<NP>& sm, const DeltaPlan& p, void* dst, long long base,
                                            int p0, int bf16, bool seen = true) {
  const int col = threadIdx.x % kCols;
  if (p0 + col >= p.P) return;
  const long long row = base + (long long)col * p.N;
  for (int n = threadIdx.x / kCols * 4; n < p.N; n += kThreads / kCols * 4) {
    const float4 v = seen ? make_float4(sm.S[n][col], sm.S[n + 1][col], sm.S[n + 2][col], sm.S[n + 3][col])
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    if (!bf16 && (p.N & 3) == 0) {
      *reinterpret_cast<float4*>(static_cast<float*>(dst) + row + n) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < p.N) st_state(dst, row + n + j, bf16, part(v, j));
    }
  }
}
// A token's four columns of a (b, L, H, P) tensor
template <typename O>
__device__ __forceinline__ void put_row(const DeltaPlan& p, void* dst, long long o, int col, float4 v) {
  O* d = static_cast<O*>(dst) + o;
  if (sizeof(O) == 4 && (p.P & 3) == 0 && col + 4 <= p.P) {
    *reinterpret_cast<float4*>(d) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < p.P) d[j] = from_f<O>(part(v, j));
}

__device__ __forceinline__ bool finite4(float4 v) {
  return (v.x - v.x) + (v.y - v.y) + (v.z - v.z) + (v.w - v.w) == 0.f;
}

// A chunk token by token, by the definition alone.  The chunk's products
// multiply what a token must not see by zero, which does not hide an infinity or
// a NaN from it: a chunk whose solve gives one is done again here, so that such
// a value reaches what it reaches by definition -- not the tokens before it, nor
// the next sequence of a packed row.  Eight threads walk a column; columns do
// not meet.
constexpr int kWalkers = kThreads / kCols;
__device__ __forceinline__ float walk_sum(float v) {
#pragma unroll
  for (int o = kWalkers / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
struct WalkGate {
  float a, beta;
  bool starts;  // the token does not see the state before it
};
template <typename T>
__device__ __forceinline__ WalkGate walk_gate(const DeltaPlan& p, const DeltaBufs& f, int bi, int h, int t) {
  const long long tok = (long long)bi * p.L + t;
  const float g = to_f(static_cast<const T*>(f.g)[tok * p.H + h]);
  const bool cut = f.seq != nullptr && t > 0 && f.seq[tok] != f.seq[tok - 1];
  return {expf(g), to_f(static_cast<const T*>(f.beta)[tok * p.H + h]), cut || g < kForget};
}

// Forward: S from the state before chunk c to the one after it; y and w
template <typename T, int NP>
__device__ __noinline__ void walk_fwd(ChunkSmem<NP>& sm, const DeltaPlan& p, const DeltaBufs& f, int bi, int h, int p0,
                                      int c) {
  const int col = threadIdx.x / kWalkers, l = threadIdx.x % kWalkers;
  for (int i = 0; i < kC && c * kC + i < p.L; ++i) {
    const int t = c * kC + i;
    const WalkGate x = walk_gate<T>(p, f, bi, h, t);
    float d = 0.f, y = 0.f;
    for (int n = l; n < p.N; n += kWalkers) {
      const float s = x.starts ? 0.f : x.a * sm.S[n][col];
      sm.S[n][col] = s;
      d += s * sm.k[i][n];
    }
    const float w = sm.v[i][col] - walk_sum(d), u = x.beta * w;
    for (int n = l; n < p.N; n += kWalkers) {
      const float s = sm.S[n][col] + u * sm.k[i][n];
      sm.S[n][col] = s;
      y += s * sm.q[i][n];
    }
    y = walk_sum(y);
    if (l == 0 && p0 + col < p.P) {
      const long long o = (((long long)bi * p.L + t) * p.H + h) * p.P + p0 + col;
      static_cast<T*>(f.y)[o] = from_f<T>(p.scale * y);
      if (f.w) static_cast<float*>(f.w)[o] = w;
    }
  }
}
// Reverse: S holds the gradient of the state after chunk c, then of the one before it; r
template <typename T, int NP>
__device__ __noinline__ void walk_bwd(ChunkSmem<NP>& sm, const DeltaPlan& p, const DeltaBufs& f, int bi, int h, int p0,
                                      int c) {
  const int col = threadIdx.x / kWalkers, l = threadIdx.x % kWalkers;
  for (int i = min(kC, p.L - c * kC) - 1; i >= 0; --i) {
    const int t = c * kC + i;
    const WalkGate x = walk_gate<T>(p, f, bi, h, t);
    const long long o = (((long long)bi * p.L + t) * p.H + h) * p.P + p0 + col;
    const bool live = p0 + col < p.P;
    const float dy = live ? p.scale * to_f(static_cast<const T*>(f.dy)[o]) : 0.f;
    float d = 0.f;
    for (int n = l; n < p.N; n += kWalkers) {
      const float s = sm.S[n][col] + dy * sm.q[i][n];
      sm.S[n][col] = s;
      d += s * sm.k[i][n];
    }
    const float r = x.beta * walk_sum(d);
    for (int n = l; n < p.N; n += kWalkers)
      sm.S[n][col] = x.starts ? 0.f : x.a * (sm.S[n][col] - r * sm.k[i][n]);
    if (l == 0 && live) {
      static_cast<T*>(f.dv)[o] = from_f<T>(r);
      static_cast<float*>(f.r)[o] = r;
    }
  }
}

template <typename T, int NP>
__global__ void __launch_bounds__(kThreads) delta_chain_simt_fwd_kernel(DeltaPlan p, DeltaBufs f) {
  extern __shared__ __align__(16) unsigned char raw[];
  ChunkSmem<NP>& sm = *reinterpret_cast<ChunkSmem<NP>*>(raw);
  const int ptiles = (p.P + kCols - 1) / kCols;
  const int p0 = (int)(blockIdx.x % ptiles) * kCols;
  const int h = (int)((blockIdx.x / ptiles) % p.H), bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int i = threadIdx.x >> 2, pp = (threadIdx.x & 3) * 4, w_rows = (i & ~7) + 8;
  const long long bh = (long long)bi * p.H + h;
  constexpr bool kPrefetch = NP <= 128;  // beyond that the operands do not fit the registers
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  ChunkAhead<T, NP> ahead;
  if (kPrefetch) ahead.load(p, f, f.v, p.vs, bi, h, p0, 0);
  read_state(sm, p, f.init, (bh * p.P + p0) * p.N, p0);
  for (int c = 0; c < p.nc; ++c) {
    if (!kPrefetch) ahead.load(p, f, f.v, p.vs, bi, h, p0, c);
    __syncthreads();
    put_chunk<T, NP, false>(sm, ahead);
    __syncthreads();
    if (kPrefetch && c + 1 < p.nc) ahead.load(p, f, f.v, p.vs, bi, h, p0, c + 1);
    if (f.S) write_state(sm, p, f.S, ((bh * p.nc + c) * p.P + p0) * p.N, p0, 0, sm.e[0] != 0.f);
    // K S and Q S
    float4 x = zero, y = zero;
#pragma unroll 4
    for (int n = 0; n < NP; n += 4) {
      const float4 k = lds4(&sm.k[i][n]), q = lds4(&sm.q[i][n]);
      const float4 s0 = lds4(&sm.S[n][pp]), s1 = lds4(&sm.S[n + 1][pp]), s2 = lds4(&sm.S[n + 2][pp]),
                   s3 = lds4(&sm.S[n + 3][pp]);
      fma4(x, k.x, s0); fma4(y, q.x, s0);
      fma4(x, k.y, s1); fma4(y, q.y, s1);
      fma4(x, k.z, s2); fma4(y, q.z, s2);
      fma4(x, k.w, s3); fma4(y, q.w, s3);
    }
    // (a sequence that starts here does not read the state, whatever it holds)
    const float e = sm.e[i];
    float4 r = lds4(&sm.v[i][pp]);
    fma4(r, -1.f, scaled(e, x));
    y = scaled(p.scale * e, y);
    sts4(&sm.R[i][pp], r);
    __syncthreads();
    float4 w = zero;
    tri(w, sm.T[i], sm.R, 0, w_rows, pp);
    sts4(&sm.w[i][pp], w);
    if (__syncthreads_or(!finite4(w))) {
      walk_fwd<T, NP>(sm, p, f, bi, h, p0, c);
      continue;
    }
    sts4(&sm.R[i][pp], mul4(sm.e[kC + i], w));
    tri(y, sm.A[i], sm.w, 0, w_rows, pp);
    const int t = c * kC + i;
    if (t < p.L) {
      const long long o = (((long long)bi * p.L + t) * p.H + h) * p.P + p0 + pp;
      put_row<T>(p, f.y, o, p0 + pp, y);
      if (f.w) put_row<float>(p, f.w, o, p0 + pp, w);
    }
    __syncthreads();
    // S = e_last S + K^T (o beta w)
    const float last = sm.e[kC - 1];
    float4 s[NP / 32];
#pragma unroll
    for (int m = 0; m < NP / 32; ++m) s[m] = scaled(last, lds4(&sm.S[i + 32 * m][pp]));
#pragma unroll 4
    for (int j = 0; j < kC; ++j) {
      const float4 u = lds4(&sm.R[j][pp]);
#pragma unroll
      for (int m = 0; m < NP / 32; ++m) fma4(s[m], sm.k[j][i + 32 * m], u);
    }
#pragma unroll
    for (int m = 0; m < NP / 32; ++m) sts4(&sm.S[i + 32 * m][pp], s[m]);
  }
  if (f.fin) {
    __syncthreads();
    write_state(sm, p, f.fin, (bh * p.P + p0) * p.N, p0, p.st_bf16);
  }
}

template <typename T, int NP>
__global__ void __launch_bounds__(kThreads) delta_chain_simt_bwd_kernel(DeltaPlan p, DeltaBufs f) {
  extern __shared__ __align__(16) unsigned char raw[];
  ChunkSmem<NP>& sm = *reinterpret_cast<ChunkSmem<NP>*>(raw);  // S holds the state's gradient D
  const int ptiles = (p.P + kCols - 1) / kCols;
  const int p0 = (int)(blockIdx.x % ptiles) * kCols;
  const int h = (int)((blockIdx.x / ptiles) % p.H), bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int i = threadIdx.x >> 2, pp = (threadIdx.x & 3) * 4, w_row = i & ~7;
  const long long bh = (long long)bi * p.H + h, dys = (long long)p.H * p.P;
  constexpr bool kPrefetch = NP <= 128;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
  ChunkAhead<T, NP> ahead;
  if (kPrefetch) ahead.load(p, f, f.dy, dys, bi, h, p0, p.nc - 1);
  read_state(sm, p, f.dfin, (bh * p.P + p0) * p.N, p0);
  for (int c = p.nc - 1; c >= 0; --c) {
    if (!kPrefetch) ahead.load(p, f, f.dy, dys, bi, h, p0, c);
    __syncthreads();
    put_chunk<T, NP, true>(sm, ahead);
    __syncthreads();
    if (kPrefetch && c > 0) ahead.load(p, f, f.dy, dys, bi, h, p0, c - 1);
    write_state(sm, p, f.D, ((bh * p.nc + c) * p.P + p0) * p.N, p0, 0);
    // R = o beta (K D) + A^T dY
    float4 x = zero, x2 = zero;
#pragma unroll 4
    for (int n = 0; n < NP; n += 4) {
      const float4 k = lds4(&sm.k[i][n]);
      fma4(x, k.x, lds4(&sm.S[n][pp]));
      fma4(x2, k.y, lds4(&sm.S[n + 1][pp]));
      fma4(x, k.z, lds4(&sm.S[n + 2][pp]));
      fma4(x2, k.w, lds4(&sm.S[n + 3][pp]));
    }
    fma4(x, 1.f, x2);
    const float e = sm.e[i], last = sm.e[kC - 1];
    x = scaled(sm.e[kC + i], x);
    tri(x, sm.A[i], sm.v, w_row, kC, pp);
    sts4(&sm.R[i][pp], x);
    __syncthreads();
    float4 r = zero;
    tri(r, sm.T[i], sm.R, w_row, kC, pp);
    // (v has been read before the barrier: its own element becomes scale e dy)
    sts4(&sm.w[i][pp], mul4(-e, r));
    sts4(&sm.v[i][pp], mul4(p.scale * e, lds4(&sm.v[i][pp])));
    const int t = c * kC + i;
    if (t < p.L) {
      const long long o = (((long long)bi * p.L + t) * p.H + h) * p.P + p0 + pp;
      put_row<T>(p, f.dv, o, p0 + pp, r);
      put_row<float>(p, f.r, o, p0 + pp, r);
    }
    if (__syncthreads_or(!finite4(r))) {
      walk_bwd<T, NP>(sm, p, f, bi, h, p0, c);  // writes the chunk's r anew
      continue;
    }
    // D = e_last D + Q^T (scale e dY) - K^T (e r); none passes a sequence's first token
    float4 s[NP / 32];
#pragma unroll
    for (int m = 0; m < NP / 32; ++m) s[m] = scaled(last, lds4(&sm.S[i + 32 * m][pp]));
#pragma unroll 4
    for (int j = 0; j < kC; ++j) {
      const float4 u = lds4(&sm.w[j][pp]), y = lds4(&sm.v[j][pp]);
#pragma unroll
      for (int m = 0; m < NP / 32; ++m) {
        fma4(s[m], sm.k[j][i + 32 * m], u);
        fma4(s[m], sm.q[j][i + 32 * m], y);
      }
    }
#pragma unroll
    for (int m = 0; m < NP / 32; ++m) sts4(&sm.S[i + 32 * m][pp], sm.e[0] == 0.f ? zero : s[m]);
  }
  if (f.dinit) {
    __syncthreads();
    write_state(sm, p, f.dinit, (bh * p.P + p0) * p.N, p0, p.st_bf16);
  }
}

template <typename T>
cudaError_t launch_prep_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  const int np = (p.N + 3) & ~3;
  const size_t smem = sizeof(float) * (2 * kC * (np + 4) + 10 * kC * kTs + 8 * 4 * kC);
  auto kern = delta_prep_simt_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int heads = p.hpg < 8 ? p.hpg : 8;  // one a warp
  const long long grid = (long long)p.b * p.G * p.nc * ((p.hpg + heads - 1) / heads);
  set_kernel_name("delta_prep_simt");
  kern<<<(unsigned)grid, kPrep, smem, s>>>(p, f, heads);
  return cudaGetLastError();
}

template <typename T, int NP>
cudaError_t launch_chain_t(const DeltaPlan& p, const DeltaBufs& f, bool reverse, cudaStream_t s) {
  auto kern = reverse ? delta_chain_simt_bwd_kernel<T, NP> : delta_chain_simt_fwd_kernel<T, NP>;
  const int smem = (int)sizeof(ChunkSmem<NP>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name(reverse ? "delta_chain_simt_bwd" : "delta_chain_simt_fwd");
  kern<<<(unsigned)((long long)((p.P + kCols - 1) / kCols) * p.H * p.b), kThreads, smem, s>>>(p, f);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_chain_n(const DeltaPlan& p, const DeltaBufs& f, bool reverse, cudaStream_t s) {
  if (p.N <= 32) return launch_chain_t<T, 32>(p, f, reverse, s);
  if (p.N <= 64) return launch_chain_t<T, 64>(p, f, reverse, s);
  if (p.N <= 128) return launch_chain_t<T, 128>(p, f, reverse, s);
  return launch_chain_t<T, 256>(p, f, reverse, s);
}

}  // namespace

cudaError_t launch_delta_prep_simt(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return p.bf16 ? launch_prep_t<__nv_bfloat16>(p, f, s) : launch_prep_t<float>(p, f, s);
}
cudaError_t launch_delta_chain_simt(const DeltaPlan& p, const DeltaBufs& f, bool reverse, cudaStream_t s) {
  return p.bf16 ? launch_chain_n<__nv_bfloat16>(p, f, reverse, s) : launch_chain_n<float>(p, f, reverse, s);
}

}  // namespace ssd
