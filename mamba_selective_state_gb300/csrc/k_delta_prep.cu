// k_delta_prep.cu -- the parts of the gated delta rule's chunks that do not
// depend on the state, for every chunk of 64 tokens at once:
//
//   T = (I + M)^-1, M_ij = E_ij (k_i.k_j) beta_j (j < i)
//   A_ij = scale E_ij (q_i.k_j) beta_j (j <= i)
//   the gates' records: e_i, o_j beta_j, ...   (see delta_internal.cuh)
//
// One CTA takes a chunk of a group: k k^T and q k^T do not depend on the head
// and stay in registers while the CTA walks its heads.  The triangular
// inverse is by blocks of 16: the four diagonal blocks by forward
// substitution in fp32 (one warp each, a lane per column), the others by
// T_ij = -sum_k (T_ii M_ik) T_kj on the tensor cores.  Those products round
// their operands to 10 mantissa bits; T - I is rounded to bf16 (8 bits) once,
// when it is written as the operand of the chains' products (which add the
// unit diagonal in fp32).  A warp owns 16 rows of M, A and T, so that only
// the blocks T_kj cross warps: four barriers a head.
// Powers of M would need fewer steps, but they overflow where keys repeat
// (k.k = 1 along a chunk gives binomial coefficients up to 1e18).
#include "delta_internal.cuh"
#include "mma_common.cuh"

namespace ssd {
namespace {

using namespace mm;

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 128;
constexpr int kMs = 68;  // row stride of the fp32 tiles: the right operands' reads (rows 2t, columns g)
constexpr int kTs = kMs; // fall into different banks

// acc (16 x 16) += a * Y (16 x 16, row stride ys).  The left operand's column
// 2t + x of each 8 is its fragment's column t + 4x: the order in which a
// product's result holds its columns, so that a result is an operand as it is.
__device__ __forceinline__ void block_mul(float (&acc)[2][4], const uint32_t (&a)[2][4], const float* Y, int ys,
                                          int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma_tf32(acc[n], a[k], tf32(Y[(8 * k + 2 * t) * ys + n * 8 + g]), tf32(Y[(8 * k + 2 * t + 1) * ys + n * 8 + g]));
}

template <int N>
struct PrepSmem {
  static constexpr int kQK = 2 * kC * N * 2;                   // q and k tiles, then in the same place
  static constexpr int kMT = (kC * kMs + kC * kTs) * 4;        // M and T
  static constexpr int oA = kQK > kMT ? kQK : kMT;             // [64][64] bf16
  static constexpr int oGate = oA + kC * kC * 2;               // gam, beta of four heads
  static constexpr int oSeg = oGate + 4 * 2 * kC * 4, bytes = oSeg + 4 * kC * 4;
};

template <int N>
__global__ void __launch_bounds__(kThreads, 4) delta_prep_kernel(DeltaPlan p, DeltaBufs f, int heads_per_cta) {
  using L = PrepSmem<N>;
  constexpr int U = N / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t k_s = smem_u32(raw), q_s = k_s + kC * N * 2, A_s = k_s + L::oA;
  float* M_s = reinterpret_cast<float*>(raw);
  float* T_s = M_s + kC * kMs;

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int nsplit = (p.hpg + heads_per_cta - 1) / heads_per_cta;
  long long idx = blockIdx.x;
  const int sp = (int)(idx % nsplit);
  idx /= nsplit;
  const int c = (int)(idx % p.nc);
  idx /= p.nc;
  const int grp = (int)(idx % p.G);
  const int bi = (int)(idx / p.G);
  const int t0 = c * kC, n = min(kC, p.L - t0);
  const long long tok0 = (long long)bi * p.L + t0;
  if (blockIdx.x == 0 && tid == 0) *f.status = 0;
  const int h0 = grp * p.hpg + sp * heads_per_cta;
  const int h1 = min(h0 + heads_per_cta, (grp + 1) * p.hpg);

  // gam, beta and sequence starts of head h into slot h & 3, e and o beta to
  // global, by one warp with two tokens a lane
  auto gates = [&](int h) {
    float* gam = reinterpret_cast<float*>(raw + L::oGate) + (h & 3) * 2 * kC;
    int* seg = reinterpret_cast<int*>(raw + L::oSeg) + (h & 3) * kC;
    float gv[2], be[2];
    int rs[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * lane + j;
      gv[j] = be[j] = 0.f;
      rs[j] = 0;
      if (i < n) {
        const long long o = (tok0 + i) * p.H + h;
        gv[j] = to_f(static_cast<const __nv_bfloat16*>(f.g)[o]);
        be[j] = to_f(static_cast<const __nv_bfloat16*>(f.beta)[o]);
        rs[j] = (f.seq != nullptr && t0 + i > 0 && f.seq[tok0 + i] != f.seq[tok0 + i - 1]) || gv[j] < kForget;
        if (rs[j]) gv[j] = 0.f;
      }
    }
    float sum = gv[0] + gv[1];
    int cnt = rs[0] + rs[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float us = __shfl_up_sync(0xffffffffu, sum, o);
      const int uc = __shfl_up_sync(0xffffffffu, cnt, o);
      if (lane >= o) {
        sum += us;
        cnt += uc;
      }
    }
    const float last = __shfl_sync(0xffffffffu, sum, 31);
    const int slast = __shfl_sync(0xffffffffu, cnt, 31);
    const float ga[2] = {sum - gv[1], sum};
    const int sg[2] = {cnt - rs[1], cnt};
    *reinterpret_cast<float2*>(gam + 2 * lane) = make_float2(ga[0], ga[1]);
    *reinterpret_cast<float2*>(gam + kC + 2 * lane) = make_float2(be[0], be[1]);
    *reinterpret_cast<int2*>(seg + 2 * lane) = make_int2(sg[0], sg[1]);
    float* eg = static_cast<float*>(f.e) + (((long long)bi * p.H + h) * p.nc + c) * kGateRows * kC + 2 * lane;
    float e[2], o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      e[j] = sg[j] == 0 ? expf(ga[j]) : 0.f;
      o[j] = sg[j] == slast ? expf(last - ga[j]) : 0.f;
    }
    *reinterpret_cast<float2*>(eg) = make_float2(e[0], e[1]);
    *reinterpret_cast<float2*>(eg + kC) = make_float2(o[0] * be[0], o[1] * be[1]);
    *reinterpret_cast<float2*>(eg + 2 * kC) = make_float2(ga[0], ga[1]);
    *reinterpret_cast<float2*>(eg + 3 * kC) = make_float2(be[0], be[1]);
    *reinterpret_cast<float2*>(eg + 4 * kC) = make_float2(o[0], o[1]);
    *reinterpret_cast<int2*>(eg + 5 * kC) = make_int2(sg[0], sg[1]);
  };

  cp_tile<kC, U>(k_s, static_cast<const __nv_bfloat16*>(f.k) + tok0 * p.ks + (long long)grp * N, p.ks, n, tid, kThreads);
  cp_tile<kC, U>(q_s, static_cast<const __nv_bfloat16*>(f.q) + tok0 * p.qs + (long long)grp * N, p.qs, n, tid, kThreads);
  cp_commit();
  // head h's gates sit in slot h & 3: warp w takes the head of its slot
  for (int h = h0; h < min(h0 + 4, h1); ++h)
    if ((h & 3) == w) gates(h);
  cp_wait<0>();
  __syncthreads();
  // rows 16w.. of k k^T and q k^T, columns up to the diagonal block
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < N; ks += 16) {
    uint32_t ka[4], qa[4], b[4];
    load_a<U>(ka, k_s, 16 * w, ks, lane);
    load_a<U>(qa, q_s, 16 * w, ks, lane);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      if (nb <= w) {
        load_b<U>(b, k_s, 16 * nb, ks, lane);
        mma(kk[2 * nb], ka, b[0], b[1]);
        mma(kk[2 * nb + 1], ka, b[2], b[3]);
        mma(qk[2 * nb], qa, b[0], b[1]);
        mma(qk[2 * nb + 1], qa, b[2], b[3]);
      }
  }
  float* Mw = M_s + 16 * w * kMs;  // this warp's rows
  float* Tw = T_s + 16 * w * kTs;
  for (int h = h0; h < h1; ++h) {
    __syncthreads();  // the tiles (first head) or the last head's T and gates have been read
    const long long unit = ((long long)bi * p.H + h) * p.nc + c;
    const float* gam = reinterpret_cast<const float*>(raw + L::oGate) + (h & 3) * 2 * kC;
    const float* bet = gam + kC;
    const int* seg = reinterpret_cast<const int*>(raw + L::oSeg) + (h & 3) * kC;
    // M (fp32) and A (bf16), zeros above the diagonal
    const int i0 = 16 * w + g;
    const float gi[2] = {gam[i0], gam[i0 + 8]};
    const int si[2] = {seg[i0], seg[i0 + 8]};
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const int j = nt * 8 + 2 * t;
      if (nt <= 2 * w + 1) {
        const float2 gj = *reinterpret_cast<const float2*>(gam + j), bj = *reinterpret_cast<const float2*>(bet + j);
        const int2 sj = *reinterpret_cast<const int2*>(seg + j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = i0 + 8 * r;
          // (no branches: the exponentials' latencies overlap)
          const float e0 = __expf(gi[r] - gj.x) * bj.x, e1 = __expf(gi[r] - gj.y) * bj.y;
          const float E0 = (j <= i) & (sj.x == si[r]) ? e0 : 0.f;
          const float E1 = (j + 1 <= i) & (sj.y == si[r]) ? e1 : 0.f;
          *reinterpret_cast<float2*>(&M_s[i * kMs + j]) =
              make_float2(j < i ? E0 * kk[nt][2 * r] : 0.f, j + 1 < i ? E1 * kk[nt][2 * r + 1] : 0.f);
          sts32(A_s + elem_off<8>(i, j), pack2(p.scale * E0 * qk[nt][2 * r], p.scale * E1 * qk[nt][2 * r + 1]));
        }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) sts32(A_s + elem_off<8>(i0 + 8 * r, j), 0u);
      }
    }
    __syncwarp();
    {
      // the diagonal block: column `col` of (I + M_ww)^-1 by forward
      // substitution, four known values at a time
      const int col = lane & 15;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
      for (int jb = 0; jb < 16; jb += 4)
#pragma unroll
        for (int i = jb + 1; i < 16; ++i) {
          const float4 m = *reinterpret_cast<const float4*>(&Mw[i * kMs + 16 * w + jb]);  // zeros from the diagonal on
          x[i] -= m.x * x[jb];
          if (i > jb + 1) x[i] -= m.y * x[jb + 1];
          if (i > jb + 2) x[i] -= m.z * x[jb + 2];
          if (i > jb + 3) x[i] -= m.w * x[jb + 3];
        }
      if (lane < 16)
#pragma unroll
        for (int i = 0; i < 16; ++i) Tw[i * kTs + 16 * w + col] = x[i];
    }
    __syncwarp();
    // P_k = -T_ww M_wk
    uint32_t P[3][2][4];
    if (w > 0) {
      uint32_t a[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          a[k][x] = tf32(Tw[(g + 8 * (x & 1)) * kTs + 16 * w + 8 * k + 2 * t + (x >> 1)]);
#pragma unroll
      for (int bk = 0; bk < 3; ++bk)
        if (bk < w) {
          float acc[2][4] = {};
          block_mul(acc, a, Mw + 16 * bk, kMs, lane);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            P[bk][nt][0] = tf32(-acc[nt][0]);
            P[bk][nt][1] = tf32(-acc[nt][2]);
            P[bk][nt][2] = tf32(-acc[nt][1]);
            P[bk][nt][3] = tf32(-acc[nt][3]);
          }
        }
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {  // the block d to the left of the diagonal
      __syncthreads();
      if (w >= d) {
        const int bj = w - d;
        float acc[2][4] = {};
#pragma unroll
        for (int bk = 0; bk < 3; ++bk)
          if (bk >= bj && bk < w) block_mul(acc, P[bk], T_s + 16 * bk * kTs + 16 * bj, kTs, lane);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(&Tw[(g + 8 * r) * kTs + 16 * bj + nt * 8 + 2 * t]) =
                make_float2(acc[nt][2 * r], acc[nt][2 * r + 1]);
      }
    }
    __syncwarp();
    uint4* Tg = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.T) + unit * kC * kC);
    uint4* Ag = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.A) + unit * kC * kC);
#pragma unroll
    for (int i = lane; i < 16 * 8; i += 32) {
      const int r = i >> 3, u = i & 7;
      uint4 v = make_uint4(0, 0, 0, 0);
      if ((u >> 1) <= w) {
        float4 a = *reinterpret_cast<const float4*>(&Tw[r * kTs + u * 8]);
        float4 b = *reinterpret_cast<const float4*>(&Tw[r * kTs + u * 8 + 4]);
        const int d = 16 * w + r - u * 8;  // the diagonal's place among the eight
        if (d == 0) a.x = 0.f;
        if (d == 1) a.y = 0.f;
        if (d == 2) a.z = 0.f;
        if (d == 3) a.w = 0.f;
        if (d == 4) b.x = 0.f;
        if (d == 5) b.y = 0.f;
        if (d == 6) b.z = 0.f;
        if (d == 7) b.w = 0.f;
        v = make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
      }
      Tg[16 * 8 * w + i] = v;
      Ag[16 * 8 * w + i] = lds128(A_s + tile_off<8>(16 * w + r, u));
    }
    // the next heads' gates: slot w is free once its head is done
    const int next = (h & ~3) + 4 + w;
    if ((h & 3) == 3 && h + 1 < h1) {
      __syncthreads();
      if (next < h1) gates(next);
    }
  }
}

template <int N>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  const int smem = PrepSmem<N>::bytes;
  auto kern = delta_prep_kernel<N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // a group's heads share one CTA's products of q and k, unless that leaves SMs without work
  const long long units = (long long)p.b * p.G * p.nc;
  int heads = p.hpg;
  while (heads > 1 && units * ((p.hpg + heads - 1) / heads) < 4LL * device_sm_count()) heads = (heads + 1) / 2;
  const long long grid = units * ((p.hpg + heads - 1) / heads);
  set_kernel_name("delta_prep");
  kern<<<(unsigned)grid, kThreads, smem, s>>>(p, f, heads);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return p.N == 128 ? launch_t<128>(p, f, s) : launch_t<64>(p, f, s);
}

}  // namespace ssd
