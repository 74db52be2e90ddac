// k_delta_chain.cu -- the state's way through the chunks of the gated delta
// rule (see delta_internal.cuh for the formulas, k_delta_prep.cu for T, A, e
// and o), one CTA per (batch row, head, 64 or 32 columns of headdim): the
// columns of the state are independent, so a chain can be split over CTAs.
//
// Forward, eight chain warps per chunk:
//   R = V - e (K S0)  ->  w = T R  ->  S = e_last S + K^T (o beta w)
// with S in fp32 accumulators (each warp 16 of its dstate rows) and bf16
// copies of S, R and w in shared memory as the next product's operands.
// Four output warps follow a chunk behind the solve, off the chain's critical
// path: y = scale e (Q S0) + A w; they also write S0 and w for the backward.
//
// Reverse, given D = dL/dS after the chunk:
//   R = o beta (K D) + A^T dY  ->  r = T^T R (= dv)
//   D = e_last D + Q^T (scale e dY) - K^T (e r)
#include "delta_internal.cuh"
#include "mma_common.cuh"

namespace ssd {
namespace {

using namespace mm;

constexpr int kC = kDeltaChunk;
constexpr int kChain = 256;          // threads of the chain warps
constexpr int kOut = 128;            // threads of the output warps
constexpr int kAll = kChain + kOut;
// named barriers: the chain's own, then "w of the chunk is written" and "the
// output warps are done with it" for even and odd chunks
constexpr int kBarChain = 1, kBarOut = 2, kBarReady = 3, kBarFree = 5;

// The fp32 state rows of one warp: n0.. (16 rows) x NT 8-column tiles from
// column p0w of this CTA's PT columns.
template <int N, int PT>
struct Split {
  static constexpr int NT = N == 128 ? PT / 8 : PT / 16;
  __device__ static int n0(int w) { return N == 128 ? 16 * w : 16 * (w & 3); }
  __device__ static int p0(int w) { return N == 128 ? 0 : (w >> 2) * (PT / 2); }
};

template <int N, int PT>
__device__ __forceinline__ void load_state(float (&S)[Split<N, PT>::NT][4], const void* src, long long base, int n0,
                                           int p0, int lane, int bf16) {
#pragma unroll
  for (int i = 0; i < Split<N, PT>::NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + (lane >> 2) + (j >> 1) * 8, pp = p0 + i * 8 + 2 * (lane & 3) + (j & 1);
      S[i][j] = src ? ld_state(src, base + (long long)pp * N + n, bf16) : 0.f;
    }
}
template <int N, int PT>
__device__ __forceinline__ void store_state(const float (&S)[Split<N, PT>::NT][4], void* dst, long long base, int n0,
                                            int p0, int lane, int bf16) {
#pragma unroll
  for (int i = 0; i < Split<N, PT>::NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + (lane >> 2) + (j >> 1) * 8, pp = p0 + i * 8 + 2 * (lane & 3) + (j & 1);
      st_state(dst, base + (long long)pp * N + n, bf16, S[i][j]);
    }
}
// the bf16 copy of the state, [n][p]
template <int N, int PT>
__device__ __forceinline__ void publish_state(const float (&S)[Split<N, PT>::NT][4], uint32_t dst, int n0, int p0,
                                              int lane) {
#pragma unroll
  for (int i = 0; i < Split<N, PT>::NT; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      sts32(dst + elem_off<PT / 8>(n0 + (lane >> 2) + 8 * r, p0 + i * 8 + 2 * (lane & 3)),
            pack2(S[i][2 * r], S[i][2 * r + 1]));
}

template <int N, int PT>
struct FwdSmem {
  static constexpr int kK = kC * N * 2, kV = kC * PT * 2, kT = kC * kC * 2, kS = N * PT * 2;
  // two stages of K, V, T, e; two of Q, A, e; S0 and w for two chunks; R; o beta w
  static constexpr int oK = 0, oT = oK + 2 * kK, oV = oT + 2 * kT, oQ = oV + 2 * kV, oA = oQ + 2 * kK,
                       oS = oA + 2 * kT, oW = oS + 2 * kS, oR = oW + 2 * kV, oU = oR + kV, oE = oU + kV,
                       bytes = oE + 4 * 2 * kC * 4;
};

template <int N, int PT>
__global__ void __launch_bounds__(kAll, 1) delta_chain_fwd_kernel(DeltaPlan p, DeltaBufs f) {
  using L = FwdSmem<N, PT>;
  using Sp = Split<N, PT>;
  constexpr int UN = N / 8, UP = PT / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sm = smem_u32(raw);
  const int ptiles = p.P / PT;
  const int p0 = (int)(blockIdx.x % ptiles) * PT;
  const int h = (int)((blockIdx.x / ptiles) % p.H), bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int grp = h / p.hpg;
  const long long row0 = (long long)bi * p.L;
  const long long unit0 = ((long long)bi * p.H + h) * p.nc;
  const long long state0 = (((long long)bi * p.H + h) * p.P + p0) * N;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const __nv_bfloat16* T = static_cast<const __nv_bfloat16*>(f.T) + unit0 * kC * kC;
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(f.A) + unit0 * kC * kC;
  const float* eg = static_cast<const float*>(f.e) + unit0 * 2 * kC;

  if (threadIdx.x < kChain) {
    const int tid = threadIdx.x, w = tid >> 5;
    const __nv_bfloat16* kg = static_cast<const __nv_bfloat16*>(f.k) + row0 * p.ks + (long long)grp * N;
    const __nv_bfloat16* vg = static_cast<const __nv_bfloat16*>(f.v) + row0 * p.vs + (long long)h * p.P + p0;
    auto load = [&](int c) {
      const int st = c & 1, n = min(kC, p.L - c * kC);
      cp_tile<kC, UN>(sm + L::oK + st * L::kK, kg + (long long)c * kC * p.ks, p.ks, n, tid, kChain);
      cp_tile<kC, 8>(sm + L::oT + st * L::kT, T + (long long)c * kC * kC, kC, kC, tid, kChain);
      cp_tile<kC, UP>(sm + L::oV + st * L::kV, vg + (long long)c * kC * p.vs, p.vs, n, tid, kChain);
      if (tid < 32) cp16(sm + L::oE + st * 2 * kC * 4 + tid * 16, eg + (long long)c * 2 * kC + tid * 4, true);
      cp_commit();
    };
    load(0);
    const int n0 = Sp::n0(w), pw = Sp::p0(w);
    float S[Sp::NT][4];
    load_state<N, PT>(S, f.init, state0, n0, pw, lane, p.st_bf16);
    publish_state<N, PT>(S, sm + L::oS, n0, pw, lane);
    constexpr int NH = PT / 16;  // 8-column tiles of half the columns
    // the two warps of a sub-partition take a long and a short row of the triangle
    const int ch = w >> 2, rb = ch ? 3 - (w & 3) : (w & 3), c0 = ch * (PT / 2);
    for (int c = 0; c < p.nc; ++c) {
      const int st = c & 1;
      cp_wait<0>();
      bar_sync(kBarChain, kChain);  // this chunk's tiles and state are in place; the last chunk's have been read
      if (c + 1 < p.nc) load(c + 1);
      const float* e = reinterpret_cast<const float*>(raw + L::oE + st * 2 * kC * 4);
      const uint32_t Ks = sm + L::oK + st * L::kK, Vs = sm + L::oV + st * L::kV, Ts = sm + L::oT + st * L::kT;
      const uint32_t Ss = sm + L::oS + st * L::kS, Ws = sm + L::oW + st * L::kV;
      float x[NH][4] = {};
#pragma unroll
      for (int ks = 0; ks < N; ks += 16) {
        uint32_t a[4], b[4];
        load_a<UN>(a, Ks, 16 * rb, ks, lane);
#pragma unroll
        for (int j = 0; j < NH; j += 2) {
          load_bt<UP>(b, Ss, c0 + j * 8, ks, lane);
          mma(x[j], a, b[0], b[1]);
          mma(x[j + 1], a, b[2], b[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < NH; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * rb + g + 8 * r, col = c0 + j * 8 + 2 * t;
          const float2 v = unpack2(lds32(Vs + elem_off<UP>(i, col)));
          // a sequence that starts here does not read the state, whatever it holds
          x[j][2 * r] = e[i] != 0.f ? v.x - e[i] * x[j][2 * r] : v.x;
          x[j][2 * r + 1] = e[i] != 0.f ? v.y - e[i] * x[j][2 * r + 1] : v.y;
          sts32(sm + L::oR + elem_off<UP>(i, col), pack2(x[j][2 * r], x[j][2 * r + 1]));
        }
      bar_sync(kBarChain, kChain);
      // w = R + (T - I) R: the unit diagonal takes R as it is, in fp32
      for (int ks = 0; ks <= rb; ++ks) {
        uint32_t a[4], b[4];
        load_a<8>(a, Ts, 16 * rb, 16 * ks, lane);
#pragma unroll
        for (int j = 0; j < NH; j += 2) {
          load_bt<UP>(b, sm + L::oR, c0 + j * 8, 16 * ks, lane);
          mma(x[j], a, b[0], b[1]);
          mma(x[j + 1], a, b[2], b[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < NH; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * rb + g + 8 * r, col = c0 + j * 8 + 2 * t;
          const float o = e[kC + i];
          sts32(Ws + elem_off<UP>(i, col), pack2(x[j][2 * r], x[j][2 * r + 1]));
          sts32(sm + L::oU + elem_off<UP>(i, col), pack2(o * x[j][2 * r], o * x[j][2 * r + 1]));
        }
      bar_arrive(kBarReady + st, kAll);
      bar_sync(kBarChain, kChain);
      const float last = e[kC - 1];
#pragma unroll
      for (int i = 0; i < Sp::NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = last == 0.f ? 0.f : S[i][j] * last;
#pragma unroll
      for (int ks = 0; ks < kC; ks += 16) {
        uint32_t a[4], b[4];
        load_at<UN>(a, Ks, n0, ks, lane);
#pragma unroll
        for (int j = 0; j < Sp::NT; j += 2) {
          load_bt<UP>(b, sm + L::oU, pw + j * 8, ks, lane);
          mma(S[j], a, b[0], b[1]);
          mma(S[j + 1], a, b[2], b[3]);
        }
      }
      if (c + 1 < p.nc) {
        // the output warps are done with chunk c - 1: its state and w make room
        if (c >= 1) bar_sync(kBarFree + (st ^ 1), kAll);
        publish_state<N, PT>(S, sm + L::oS + (st ^ 1) * L::kS, n0, pw, lane);
      }
    }
    if (f.fin) store_state<N, PT>(S, f.fin, state0, n0, pw, lane, p.st_bf16);
  } else {
    const int tid = threadIdx.x - kChain, w = tid >> 5;
    const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(f.q) + row0 * p.qs + (long long)grp * N;
    __nv_bfloat16* yg = static_cast<__nv_bfloat16*>(f.y) + (row0 * p.H + h) * p.P + p0;
    auto load = [&](int c) {
      const int st = c & 1, n = min(kC, p.L - c * kC);
      cp_tile<kC, UN>(sm + L::oQ + st * L::kK, qg + (long long)c * kC * p.qs, p.qs, n, tid, kOut);
      cp_tile<kC, 8>(sm + L::oA + st * L::kT, A + (long long)c * kC * kC, kC, kC, tid, kOut);
      if (tid < 32) cp16(sm + L::oE + (2 + st) * 2 * kC * 4 + tid * 16, eg + (long long)c * 2 * kC + tid * 4, true);
      cp_commit();
    };
    load(0);
    constexpr int NT = PT / 8;
    for (int c = 0; c < p.nc; ++c) {
      const int st = c & 1;
      cp_wait<0>();
      bar_sync(kBarOut, kOut);
      if (c + 1 < p.nc) load(c + 1);
      const float* e = reinterpret_cast<const float*>(raw + L::oE + (2 + st) * 2 * kC * 4);
      const uint32_t Qs = sm + L::oQ + st * L::kK, As = sm + L::oA + st * L::kT;
      const uint32_t Ss = sm + L::oS + st * L::kS, Ws = sm + L::oW + st * L::kV;
      bar_sync(kBarReady + st, kAll);
      float y[NT][4] = {};
#pragma unroll
      for (int ks = 0; ks < N; ks += 16) {
        uint32_t a[4], b[4];
        load_a<UN>(a, Qs, 16 * w, ks, lane);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          load_bt<UP>(b, Ss, j * 8, ks, lane);
          mma(y[j], a, b[0], b[1]);
          mma(y[j + 1], a, b[2], b[3]);
        }
      }
      const float e0 = p.scale * e[16 * w + g], e1 = p.scale * e[16 * w + g + 8];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        y[j][0] = e0 == 0.f ? 0.f : y[j][0] * e0;
        y[j][1] = e0 == 0.f ? 0.f : y[j][1] * e0;
        y[j][2] = e1 == 0.f ? 0.f : y[j][2] * e1;
        y[j][3] = e1 == 0.f ? 0.f : y[j][3] * e1;
      }
      for (int ks = 0; ks <= w; ++ks) {
        uint32_t a[4], b[4];
        load_a<8>(a, As, 16 * w, 16 * ks, lane);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          load_bt<UP>(b, Ws, j * 8, 16 * ks, lane);
          mma(y[j], a, b[0], b[1]);
          mma(y[j + 1], a, b[2], b[3]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = 16 * w + g + 8 * r;
        if (c * kC + i < p.L) {
          __nv_bfloat16* dst = yg + (long long)(c * kC + i) * p.H * p.P + 2 * t;
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<uint32_t*>(dst + j * 8) = pack2(y[j][2 * r], y[j][2 * r + 1]);
        }
      }
      if (f.S) {
        __nv_bfloat16* Sg = static_cast<__nv_bfloat16*>(f.S) + (unit0 + c) * N * p.P + p0;
        __nv_bfloat16* Wg = static_cast<__nv_bfloat16*>(f.w) + (unit0 + c) * kC * p.P + p0;
#pragma unroll 4
        for (int i = tid; i < N * UP; i += kOut)
          *reinterpret_cast<uint4*>(Sg + (long long)(i / UP) * p.P + (i % UP) * 8) = lds128(Ss + tile_off<UP>(i / UP, i % UP));
#pragma unroll 4
        for (int i = tid; i < kC * UP; i += kOut)
          *reinterpret_cast<uint4*>(Wg + (long long)(i / UP) * p.P + (i % UP) * 8) = lds128(Ws + tile_off<UP>(i / UP, i % UP));
      }
      // nobody waits for the last two chunks' buffers
      if (c + 2 < p.nc) bar_arrive(kBarFree + st, kAll);
    }
  }
}

template <int N, int PT>
struct RevSmem {
  static constexpr int kK = kC * N * 2, kV = kC * PT * 2, kT = kC * kC * 2;
  // two stages of K, Q, T, A, dY, e; D; R; -e r; scale e dY
  static constexpr int oK = 0, oQ = oK + 2 * kK, oT = oQ + 2 * kK, oA = oT + 2 * kT, oY = oA + 2 * kT,
                       oD = oY + 2 * kV, oR = oD + N * PT * 2, oU = oR + kV, oP = oU + kV, oE = oP + kV,
                       bytes = oE + 2 * 2 * kC * 4;
};

template <int N, int PT>
__global__ void __launch_bounds__(kChain, 1) delta_chain_bwd_kernel(DeltaPlan p, DeltaBufs f) {
  using L = RevSmem<N, PT>;
  using Sp = Split<N, PT>;
  constexpr int UN = N / 8, UP = PT / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sm = smem_u32(raw);
  const int ptiles = p.P / PT;
  const int p0 = (int)(blockIdx.x % ptiles) * PT;
  const int h = (int)((blockIdx.x / ptiles) % p.H), bi = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int grp = h / p.hpg;
  const long long row0 = (long long)bi * p.L;
  const long long unit0 = ((long long)bi * p.H + h) * p.nc;
  const long long state0 = (((long long)bi * p.H + h) * p.P + p0) * N;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3, w = tid >> 5;
  const __nv_bfloat16* T = static_cast<const __nv_bfloat16*>(f.T) + unit0 * kC * kC;
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(f.A) + unit0 * kC * kC;
  const float* eg = static_cast<const float*>(f.e) + unit0 * 2 * kC;
  const __nv_bfloat16* kg = static_cast<const __nv_bfloat16*>(f.k) + row0 * p.ks + (long long)grp * N;
  const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(f.q) + row0 * p.qs + (long long)grp * N;
  const long long vs = (long long)p.H * p.P, v0 = row0 * vs + (long long)h * p.P + p0;
  const __nv_bfloat16* yg = static_cast<const __nv_bfloat16*>(f.dy) + v0;
  __nv_bfloat16* dvg = static_cast<__nv_bfloat16*>(f.dv) + v0;
  auto load = [&](int c) {
    const int st = c & 1, n = min(kC, p.L - c * kC);
    cp_tile<kC, UN>(sm + L::oK + st * L::kK, kg + (long long)c * kC * p.ks, p.ks, n, tid, kChain);
    cp_tile<kC, UN>(sm + L::oQ + st * L::kK, qg + (long long)c * kC * p.qs, p.qs, n, tid, kChain);
    cp_tile<kC, 8>(sm + L::oT + st * L::kT, T + (long long)c * kC * kC, kC, kC, tid, kChain);
    cp_tile<kC, 8>(sm + L::oA + st * L::kT, A + (long long)c * kC * kC, kC, kC, tid, kChain);
    cp_tile<kC, UP>(sm + L::oY + st * L::kV, yg + (long long)c * kC * vs, vs, n, tid, kChain);
    if (tid < 32) cp16(sm + L::oE + st * 2 * kC * 4 + tid * 16, eg + (long long)c * 2 * kC + tid * 4, true);
    cp_commit();
  };
  load(p.nc - 1);
  const int n0 = Sp::n0(w), pw = Sp::p0(w);
  float D[Sp::NT][4];
  load_state<N, PT>(D, f.dfin, state0, n0, pw, lane, p.st_bf16);
  publish_state<N, PT>(D, sm + L::oD, n0, pw, lane);
  constexpr int NH = PT / 16;
  const int ch = w >> 2, rb = ch ? 3 - (w & 3) : (w & 3), c0 = ch * (PT / 2);
  for (int c = p.nc - 1; c >= 0; --c) {
    const int st = c & 1;
    cp_wait<0>();
    __syncthreads();
    if (c > 0) load(c - 1);
    const float* e = reinterpret_cast<const float*>(raw + L::oE + st * 2 * kC * 4);
    const uint32_t Ks = sm + L::oK + st * L::kK, Qs = sm + L::oQ + st * L::kK, Ys = sm + L::oY + st * L::kV;
    const uint32_t Ts = sm + L::oT + st * L::kT, As = sm + L::oA + st * L::kT, Ds = sm + L::oD;
    __nv_bfloat16* Dg = static_cast<__nv_bfloat16*>(f.D) + (unit0 + c) * N * p.P + p0;
#pragma unroll 4
    for (int i = tid; i < N * UP; i += kChain)
      *reinterpret_cast<uint4*>(Dg + (long long)(i / UP) * p.P + (i % UP) * 8) = lds128(Ds + tile_off<UP>(i / UP, i % UP));
    for (int i = tid; i < kC * PT / 2; i += kChain) {
      const int r = i / (PT / 2), col = 2 * (i % (PT / 2));
      const float2 v = unpack2(lds32(Ys + elem_off<UP>(r, col)));
      const float s = p.scale * e[r];
      sts32(sm + L::oP + elem_off<UP>(r, col), pack2(s * v.x, s * v.y));
    }
    float x[NH][4] = {};
#pragma unroll
    for (int ks = 0; ks < N; ks += 16) {
      uint32_t a[4], b[4];
      load_a<UN>(a, Ks, 16 * rb, ks, lane);
#pragma unroll
      for (int j = 0; j < NH; j += 2) {
        load_bt<UP>(b, Ds, c0 + j * 8, ks, lane);
        mma(x[j], a, b[0], b[1]);
        mma(x[j + 1], a, b[2], b[3]);
      }
    }
    const float o0 = e[kC + 16 * rb + g], o1 = e[kC + 16 * rb + g + 8];
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      x[j][0] = o0 == 0.f ? 0.f : x[j][0] * o0;
      x[j][1] = o0 == 0.f ? 0.f : x[j][1] * o0;
      x[j][2] = o1 == 0.f ? 0.f : x[j][2] * o1;
      x[j][3] = o1 == 0.f ? 0.f : x[j][3] * o1;
    }
    for (int ks = rb; ks < 4; ++ks) {
      uint32_t a[4], b[4];
      load_at<8>(a, As, 16 * rb, 16 * ks, lane);
#pragma unroll
      for (int j = 0; j < NH; j += 2) {
        load_bt<UP>(b, Ys, c0 + j * 8, 16 * ks, lane);
        mma(x[j], a, b[0], b[1]);
        mma(x[j + 1], a, b[2], b[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < NH; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        sts32(sm + L::oR + elem_off<UP>(16 * rb + g + 8 * r, c0 + j * 8 + 2 * t), pack2(x[j][2 * r], x[j][2 * r + 1]));
    __syncthreads();
    // r = R + (T - I)^T R, the unit diagonal in fp32
    for (int ks = rb; ks < 4; ++ks) {
      uint32_t a[4], b[4];
      load_at<8>(a, Ts, 16 * rb, 16 * ks, lane);
#pragma unroll
      for (int j = 0; j < NH; j += 2) {
        load_bt<UP>(b, sm + L::oR, c0 + j * 8, 16 * ks, lane);
        mma(x[j], a, b[0], b[1]);
        mma(x[j + 1], a, b[2], b[3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 16 * rb + g + 8 * r;
      const float s = -e[i];
      const bool in = c * kC + i < p.L;
      __nv_bfloat16* dst = dvg + (long long)(c * kC + i) * vs + c0 + 2 * t;
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        if (in) *reinterpret_cast<uint32_t*>(dst + j * 8) = pack2(x[j][2 * r], x[j][2 * r + 1]);
        sts32(sm + L::oU + elem_off<UP>(i, c0 + j * 8 + 2 * t), pack2(s * x[j][2 * r], s * x[j][2 * r + 1]));
      }
    }
    __syncthreads();
    const float last = e[kC - 1];
#pragma unroll
    for (int i = 0; i < Sp::NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) D[i][j] = last == 0.f ? 0.f : D[i][j] * last;
#pragma unroll
    for (int ks = 0; ks < kC; ks += 16) {
      uint32_t a[4], b[4], aq[4];
      load_at<UN>(aq, Qs, n0, ks, lane);
      load_at<UN>(a, Ks, n0, ks, lane);
#pragma unroll
      for (int j = 0; j < Sp::NT; j += 2) {
        load_bt<UP>(b, sm + L::oP, pw + j * 8, ks, lane);
        mma(D[j], aq, b[0], b[1]);
        mma(D[j + 1], aq, b[2], b[3]);
        load_bt<UP>(b, sm + L::oU, pw + j * 8, ks, lane);
        mma(D[j], a, b[0], b[1]);
        mma(D[j + 1], a, b[2], b[3]);
      }
    }
    publish_state<N, PT>(D, Ds, n0, pw, lane);
  }
  if (f.dinit) store_state<N, PT>(D, f.dinit, state0, n0, pw, lane, p.st_bf16);
}

// 32 columns a CTA when 64 would leave SMs idle, else 64
int chain_cols(const DeltaPlan& p) {
  return p.P % 64 != 0 || (long long)p.b * p.H * (p.P / 64) * 2 <= device_sm_count() ? 32 : 64;
}

template <int N, int PT>
cudaError_t launch_fwd_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  auto kern = delta_chain_fwd_kernel<N, PT>;
  constexpr int smem = FwdSmem<N, PT>::bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("delta_chain_fwd");
  kern<<<(unsigned)((long long)(p.P / PT) * p.H * p.b), kAll, smem, s>>>(p, f);
  return cudaGetLastError();
}

template <int N, int PT>
cudaError_t launch_bwd_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  auto kern = delta_chain_bwd_kernel<N, PT>;
  constexpr int smem = RevSmem<N, PT>::bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("delta_chain_bwd");
  kern<<<(unsigned)((long long)(p.P / PT) * p.H * p.b), kChain, smem, s>>>(p, f);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain_bwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  if (chain_cols(p) == 64) return p.N == 128 ? launch_bwd_t<128, 64>(p, f, s) : launch_bwd_t<64, 64>(p, f, s);
  return p.N == 128 ? launch_bwd_t<128, 32>(p, f, s) : launch_bwd_t<64, 32>(p, f, s);
}

cudaError_t launch_delta_chain_fwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  if (chain_cols(p) == 64) return p.N == 128 ? launch_fwd_t<128, 64>(p, f, s) : launch_fwd_t<64, 64>(p, f, s);
  return p.N == 128 ? launch_fwd_t<128, 32>(p, f, s) : launch_fwd_t<64, 32>(p, f, s);
}

}  // namespace ssd
