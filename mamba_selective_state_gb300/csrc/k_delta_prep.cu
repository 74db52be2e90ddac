// k_delta_prep.cu -- the parts of the gated delta rule's chunks that do not
// depend on the state, for every chunk of 64 tokens at once:
//
//   T = (I + M)^-1, M_ij = E_ij (k_i.k_j) beta_j (j < i)
//   A_ij = scale E_ij (q_i.k_j) beta_j (j <= i)
//   e_i, and o_j beta_j            (see delta_internal.cuh)
//
// One CTA takes a chunk of a group: k k^T and q k^T do not depend on the head
// and stay in registers while the CTA walks its heads.  The triangular
// inverse is by blocks of 16: the four diagonal blocks by forward
// substitution in fp32 (one warp each, a lane per column), the others by
// T_ij = -T_ii sum_k M_ik T_kj, three levels of 16 x 16 products.  Those
// round their operands to 10 mantissa bits; T itself is rounded to bf16 (8
// bits) once, when it is written as the operand of the chains' products.
// Powers of M would need fewer steps, but they overflow where keys repeat
// (k.k = 1 along a chunk gives binomial coefficients up to 1e18).
#include "delta_internal.cuh"
#include "mma_common.cuh"

namespace ssd {
namespace {

using namespace mm;

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 128;
constexpr int kMs = 68;  // row strides of the fp32 tiles: 68 keeps the left
constexpr int kTs = 72;  // operand's fragments off each other's banks, 72 the right's

// acc (16 x 16) += X (16 x 16, row stride xs) * Y (16 x 16, row stride ys)
__device__ __forceinline__ void block_mul(float (&acc)[2][4], const float* X, int xs, const float* Y, int ys,
                                          int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int k = 0; k < 16; k += 8) {
    const uint32_t a[4] = {tf32(X[g * xs + k + t]), tf32(X[(g + 8) * xs + k + t]), tf32(X[g * xs + k + t + 4]),
                           tf32(X[(g + 8) * xs + k + t + 4])};
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma_tf32(acc[n], a, tf32(Y[(k + t) * ys + n * 8 + g]), tf32(Y[(k + t + 4) * ys + n * 8 + g]));
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(DeltaPlan p, DeltaBufs f, int heads_per_cta) {
  constexpr int U = N / 8;
  constexpr int kQK = 2 * kC * N * 2;                        // q and k tiles
  constexpr int kMT = (kC * kMs + kC * kTs + 3 * 16 * kTs) * 4;  // M, T, scratch: the same memory later
  constexpr int kBytes = kQK > kMT ? kQK : kMT;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t k_s = smem_u32(raw), q_s = k_s + kC * N * 2;
  float* M_s = reinterpret_cast<float*>(raw);
  float* T_s = M_s + kC * kMs;
  float* X_s = T_s + kC * kTs;  // [3][16][kTs]
  float* gam = reinterpret_cast<float*>(raw + kBytes);
  float* bet = gam + kC;
  int* seg = reinterpret_cast<int*>(bet + kC);
  const uint32_t A_s = smem_u32(seg + kC);  // [64][64] bf16

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

  cp_tile<kC, U>(k_s, static_cast<const __nv_bfloat16*>(f.k) + tok0 * p.ks + (long long)grp * N, p.ks, n, tid, kThreads);
  cp_tile<kC, U>(q_s, static_cast<const __nv_bfloat16*>(f.q) + tok0 * p.qs + (long long)grp * N, p.qs, n, tid, kThreads);
  cp_commit();
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
  const int h0 = grp * p.hpg + sp * heads_per_cta;
  const int h1 = min(h0 + heads_per_cta, (grp + 1) * p.hpg);
  for (int h = h0; h < h1; ++h) {
    __syncthreads();  // the tiles (first head) or the last head's T have been read
    const long long unit = ((long long)bi * p.H + h) * p.nc + c;
    if (w == 0) {
      // cumulative decay and sequence starts, two tokens a lane
      float gv[2];
      int rs[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        gv[j] = 0.f;
        rs[j] = 0;
        float be = 0.f;
        if (i < n) {
          const long long o = (tok0 + i) * p.H + h;
          gv[j] = to_f(static_cast<const __nv_bfloat16*>(f.g)[o]);
          be = to_f(static_cast<const __nv_bfloat16*>(f.beta)[o]);
          rs[j] = (f.seq != nullptr && t0 + i > 0 && f.seq[tok0 + i] != f.seq[tok0 + i - 1]) || gv[j] < kForget;
          if (rs[j]) gv[j] = 0.f;
        }
        bet[i] = be;
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
      gam[2 * lane] = sum - gv[1];
      gam[2 * lane + 1] = sum;
      seg[2 * lane] = cnt - rs[1];
      seg[2 * lane + 1] = cnt;
    }
    __syncthreads();
    if (tid < kC) {
      const float e = seg[tid] == 0 ? expf(gam[tid]) : 0.f;
      const float o = seg[tid] == seg[kC - 1] ? expf(gam[kC - 1] - gam[tid]) * bet[tid] : 0.f;
      static_cast<float*>(f.e)[unit * 2 * kC + tid] = e;
      static_cast<float*>(f.e)[unit * 2 * kC + kC + tid] = o;
    }
    // M (fp32, zeros above and on the diagonal) and A (bf16)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 16 * w + g + 8 * r;
      const float gi = gam[i];
      const int si = seg[i];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const int j = nt * 8 + 2 * t;
        float m[2] = {0.f, 0.f}, a[2] = {0.f, 0.f};
        if (nt <= 2 * w + 1) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (j + x <= i && seg[j + x] == si) {
              const float E = __expf(gi - gam[j + x]) * bet[j + x];
              a[x] = p.scale * E * qk[nt][2 * r + x];
              if (j + x < i) m[x] = E * kk[nt][2 * r + x];
            }
        }
        *reinterpret_cast<float2*>(&M_s[i * kMs + j]) = make_float2(m[0], m[1]);
        sts32(A_s + elem_off<8>(i, j), pack2(a[0], a[1]));
      }
    }
    __syncthreads();
    {
      // the diagonal block: column `col` of (I + M_ww)^-1 by forward substitution
      const int col = lane & 15;
      const float* Mw = M_s + 16 * w * kMs + 16 * w;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == col ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s -= Mw[i * kMs + j] * x[j];
        x[i] = s;
      }
      if (lane < 16)
#pragma unroll
        for (int i = 0; i < 16; ++i) T_s[(16 * w + i) * kTs + 16 * w + col] = x[i];
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {  // blocks (j + d, j)
      __syncthreads();
      if (w < 4 - d) {
        const int bj = w, bi2 = w + d;
        float acc[2][4] = {};
        for (int bk = bj; bk < bi2; ++bk)
          block_mul(acc, M_s + 16 * bi2 * kMs + 16 * bk, kMs, T_s + 16 * bk * kTs + 16 * bj, kTs, lane);
        float* X = X_s + w * 16 * kTs;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(&X[(g + 8 * r) * kTs + nt * 8 + 2 * t]) =
                make_float2(-acc[nt][2 * r], -acc[nt][2 * r + 1]);
        __syncwarp();
        float out[2][4] = {};
        block_mul(out, T_s + 16 * bi2 * kTs + 16 * bi2, kTs, X, kTs, lane);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(&T_s[(16 * bi2 + g + 8 * r) * kTs + 16 * bj + nt * 8 + 2 * t]) =
                make_float2(out[nt][2 * r], out[nt][2 * r + 1]);
      }
    }
    __syncthreads();
    uint4* Tg = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.T) + unit * kC * kC);
    uint4* Ag = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.A) + unit * kC * kC);
#pragma unroll
    for (int i = tid; i < kC * 8; i += kThreads) {
      const int r = i >> 3, u = i & 7;
      uint4 v = make_uint4(0, 0, 0, 0);
      if ((u >> 1) <= (r >> 4)) {
        const float4 a = *reinterpret_cast<const float4*>(&T_s[r * kTs + u * 8]);
        const float4 b = *reinterpret_cast<const float4*>(&T_s[r * kTs + u * 8 + 4]);
        v = make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
      }
      Tg[i] = v;
      Ag[i] = lds128(A_s + tile_off<8>(r, u));
    }
  }
}

template <int N>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  constexpr int kQK = 2 * kC * N * 2;
  constexpr int kMT = (kC * kMs + kC * kTs + 3 * 16 * kTs) * 4;
  const int smem = (kQK > kMT ? kQK : kMT) + 3 * kC * 4 + kC * kC * 2;
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
