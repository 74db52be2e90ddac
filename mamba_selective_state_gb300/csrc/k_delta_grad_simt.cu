// k_delta_grad_simt.cu -- dq, dk, dg and dbeta of the gated delta rule in
// fp32, chunk by chunk, from the states entering each chunk, the gradients of
// the states leaving it, and every token's w and r (see delta_internal.cuh).
//
// With Z_ij = scale E_ij beta_j (dy_i.w_j) (j <= i) and M_ij = -(r_i.w_j) E_ij
// beta_j (j < i):
//   dq_i    = sum_h scale e_i S0 dy_i + sum_j Z_ij k_j
//   dk_i    = sum_h -e_i S0 r_i + o_i beta_i D1 w_i
//                   + sum_j Z_ji q_j + M_ij k_j + M_ji k_j
//   dbeta_j = o_j k_j.(D1 w_j) + sum_i Z_ij (q_i.k_j)/beta_j + M_ij (k_i.k_j)/beta_j
//   dgam    : row i gains, column j loses every pair's Z_ij (q_i.k_j) + M_ij (k_i.k_j);
//             row i gains scale e_i q_i.(S0 dy_i) - e_i k_i.(S0 r_i); the last token gains
//             and token j loses o_j beta_j k_j.(D1 w_j); the last gains e_{C-1} <S0, D1>
// and dg is the reverse cumulative sum of dgam.  One CTA per (chunk, group,
// row) adds its heads in order, so dq and dk need no atomics.
#include "delta_internal.cuh"

namespace ssd {
namespace {

constexpr int kC = kDeltaChunkF32;
constexpr int kTp = 16;       // headdim columns staged at a time
constexpr int kThreads = 256; // 16 pairs of rows x 16 columns

__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int NJ>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(DeltaPlan p, DeltaBufs f) {
  extern __shared__ float sh[];
  constexpr int NP = NJ * 16;  // padded dstate
  float* q_s = sh;                       // [kC][NP + 1]
  float* k_s = q_s + kC * (NP + 1);      // [kC][NP + 1]
  float* S_s = k_s + kC * (NP + 1);      // [kTp][NP]
  float* D_s = S_s + kTp * NP;           // [kTp][NP]
  float* dy_s = D_s + kTp * NP;          // [kC][kTp + 1] x 3
  float* w_s = dy_s + kC * (kTp + 1);
  float* r_s = w_s + kC * (kTp + 1);
  float* qk_s = r_s + kC * (kTp + 1);    // [kC][kC + 1] x 4
  float* kk_s = qk_s + kC * (kC + 1);
  float* Z_s = kk_s + kC * (kC + 1);
  float* M_s = Z_s + kC * (kC + 1);
  float* gam = M_s + kC * (kC + 1);      // [kC] each
  float* gam_lo = gam + kC;              // the cumulative decay in two parts
  float* bet = gam_lo + kC;
  float* drow = bet + kC;                // what row i's decay gains
  float* dout = drow + kC;               // beta_j o_j k_j.(D1 w_j)
  float* dbo = dout + kC;                // the same without beta_j
  float* red = dbo + kC;                 // [8] <S0, D1> by warp
  int* seg = reinterpret_cast<int*>(red + 8);  // [kC] sequence starts up to the token

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = ty * 2;
  const int nchunk = p.nc;
  const int c = (int)(blockIdx.x % nchunk);
  const int grp = (int)((blockIdx.x / nchunk) % p.G);
  const int bi = (int)(blockIdx.x / ((long long)nchunk * p.G));
  const int t0 = c * kC;
  const int n = min(kC, p.L - t0);
  const long long tok0 = (long long)bi * p.L + t0;

  for (int i = threadIdx.x; i < kC * NP; i += kThreads) {
    const int t = i / NP, e = i % NP;
    float qv = 0.f, kv = 0.f;
    if (t < n && e < p.N) {
      qv = to_f(static_cast<const T*>(f.q)[(tok0 + t) * p.qs + (long long)grp * p.N + e]);
      kv = to_f(static_cast<const T*>(f.k)[(tok0 + t) * p.ks + (long long)grp * p.N + e]);
    }
    q_s[t * (NP + 1) + e] = qv;
    k_s[t * (NP + 1) + e] = kv;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kC * kC; i += kThreads) {
    const int a = i / kC, b2 = i % kC;
    float d = 0.f, e = 0.f;
    for (int m = 0; m < p.N; ++m) {
      const float kb = k_s[b2 * (NP + 1) + m];
      d += q_s[a * (NP + 1) + m] * kb;
      e += k_s[a * (NP + 1) + m] * kb;
    }
    qk_s[a * (kC + 1) + b2] = d;
    kk_s[a * (kC + 1) + b2] = e;
  }
  float dq[2][NJ], dk[2][NJ];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int j = 0; j < NJ; ++j) dq[a][j] = dk[a][j] = 0.f;

  for (int hh = 0; hh < p.hpg; ++hh) {
    const int h = grp * p.hpg + hh;
    __syncthreads();
    if (threadIdx.x < kC) {  // one warp: cumulative decay and sequence starts
      const int t = threadIdx.x;
      float g = 0.f, be = 0.f;
      int rs = 0;
      if (t < n) {
        g = to_f(static_cast<const T*>(f.g)[(tok0 + t) * p.H + h]);
        be = to_f(static_cast<const T*>(f.beta)[(tok0 + t) * p.H + h]);
        rs = f.seq != nullptr && t0 + t > 0 && f.seq[tok0 + t] != f.seq[tok0 + t - 1];
        if (g < kForget) { rs = 1; }
      }
      const GateSum sum = gate_sum(rs ? 0.f : g, rs, t);
      gam[t] = sum.hi;
      gam_lo[t] = sum.lo;
      bet[t] = be;
      seg[t] = rs;
    }
    float x1[2][NJ], x2[2][NJ], x3[2][NJ], m1[2][2], m2[2][2], sd = 0.f;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) x1[a][j] = x2[a][j] = x3[a][j] = 0.f;
      m1[a][0] = m1[a][1] = m2[a][0] = m2[a][1] = 0.f;
    }
    const long long st = (((long long)bi * p.H + h) * p.nc + c) * p.P;
    for (int p0 = 0; p0 < p.P; p0 += kTp) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTp * NP; i += kThreads) {
        const int pp = i / NP, e = i % NP;
        const bool in = p0 + pp < p.P && e < p.N;
        const float sv = in ? static_cast<const float*>(f.S)[(st + p0 + pp) * p.N + e] : 0.f;
        const float dv = in ? static_cast<const float*>(f.D)[(st + p0 + pp) * p.N + e] : 0.f;
        S_s[i] = sv;
        D_s[i] = dv;
        sd += sv * dv;
      }
      for (int i = threadIdx.x; i < kC * kTp; i += kThreads) {
        const int t = i / kTp, pp = i % kTp;
        const bool in = t < n && p0 + pp < p.P;
        const long long o = ((tok0 + t) * p.H + h) * p.P + p0 + pp;
        dy_s[t * (kTp + 1) + pp] = in ? to_f(static_cast<const T*>(f.dy)[o]) : 0.f;
        w_s[t * (kTp + 1) + pp] = in ? static_cast<const float*>(f.w)[o] : 0.f;
        r_s[t * (kTp + 1) + pp] = in ? static_cast<const float*>(f.r)[o] : 0.f;
      }
      __syncthreads();
      for (int pp = 0; pp < kTp; ++pp) {
        const float dy0 = dy_s[i0 * (kTp + 1) + pp], dy1 = dy_s[(i0 + 1) * (kTp + 1) + pp];
        const float w0 = w_s[i0 * (kTp + 1) + pp], w1 = w_s[(i0 + 1) * (kTp + 1) + pp];
        const float r0 = r_s[i0 * (kTp + 1) + pp], r1 = r_s[(i0 + 1) * (kTp + 1) + pp];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float s0 = S_s[pp * NP + j * 16 + tx], d1 = D_s[pp * NP + j * 16 + tx];
          x1[0][j] += dy0 * s0;
          x1[1][j] += dy1 * s0;
          x2[0][j] += r0 * s0;
          x2[1][j] += r1 * s0;
          x3[0][j] += w0 * d1;
          x3[1][j] += w1 * d1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float wj = w_s[(j * 16 + tx) * (kTp + 1) + pp];
          m1[0][j] += dy0 * wj;
          m1[1][j] += dy1 * wj;
          m2[0][j] += r0 * wj;
          m2[1][j] += r1 * wj;
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sd;
    const float glast = gam[kC - 1], glast_lo = gam_lo[kC - 1];
    const int slast = seg[kC - 1];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int i = i0 + a;
      const float e = seg[i] == 0 ? expf(gam[i]) : 0.f;
      const float o = seg[i] == slast ? expf((glast - gam[i]) + (glast_lo - gam_lo[i])) : 0.f;
      float row = 0.f, out = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float qn = q_s[i * (NP + 1) + j * 16 + tx], kn = k_s[i * (NP + 1) + j * 16 + tx];
        const float a1 = p.scale * e * x1[a][j], a2 = e * x2[a][j], a3 = o * x3[a][j];
        row += qn * a1 - kn * a2;
        out += kn * a3;
        dq[a][j] += a1;
        dk[a][j] += bet[i] * a3 - a2;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int jj = j * 16 + tx;
        const float E =
            jj <= i && seg[i] == seg[jj] ? expf((gam[i] - gam[jj]) + (gam_lo[i] - gam_lo[jj])) : 0.f;
        Z_s[i * (kC + 1) + jj] = p.scale * E * m1[a][j];
        M_s[i * (kC + 1) + jj] = jj < i ? -E * m2[a][j] : 0.f;
      }
      row = half_warp_sum(row);
      out = half_warp_sum(out);
      if (tx == 0) {
        drow[i] = row;
        dbo[i] = out;
        dout[i] = bet[i] * out;
      }
    }
    __syncthreads();
    // Z and M hold everything but beta_j until here: dbeta and the pairs' part of dgam
    if (threadIdx.x < kC) {
      const int t = threadIdx.x;
      float db = dbo[t], row = drow[t], col = 0.f;
      for (int i = 0; i < kC; ++i) {
        const float down = Z_s[i * (kC + 1) + t] * qk_s[i * (kC + 1) + t] + M_s[i * (kC + 1) + t] * kk_s[i * (kC + 1) + t];
        db += down;
        if (i != t) {
          col += bet[t] * down;
          row += bet[i] * (Z_s[t * (kC + 1) + i] * qk_s[t * (kC + 1) + i] + M_s[t * (kC + 1) + i] * kk_s[t * (kC + 1) + i]);
        }
      }
      float all = dout[t];
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      float sdot = 0.f;
      for (int i = 0; i < 8; ++i) sdot += red[i];
      float d = row - col - dout[t];
      if (t == kC - 1) d += all + (seg[t] == 0 ? expf(gam[t]) * sdot : 0.f);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float dn = __shfl_down_sync(0xffffffffu, d, o);
        if (t + o < 32) d += dn;
      }
      if (t < n) {
        // a token that forgets the state does not depend on its decay
        const bool starts = t > 0 ? seg[t] != seg[t - 1] : seg[0] != 0;
        static_cast<T*>(f.dg)[(tok0 + t) * p.H + h] = from_f<T>(starts ? 0.f : d);
        static_cast<T*>(f.dbeta)[(tok0 + t) * p.H + h] = from_f<T>(db);
      }
    }
    // the pairs' part of dq and dk
    for (int m = 0; m < kC; ++m) {
      const float z0 = Z_s[i0 * (kC + 1) + m] * bet[m], z1 = Z_s[(i0 + 1) * (kC + 1) + m] * bet[m];
      const float zt0 = Z_s[m * (kC + 1) + i0] * bet[i0], zt1 = Z_s[m * (kC + 1) + i0 + 1] * bet[i0 + 1];
      const float mm0 = M_s[i0 * (kC + 1) + m] * bet[m] + M_s[m * (kC + 1) + i0] * bet[i0];
      const float mm1 = M_s[(i0 + 1) * (kC + 1) + m] * bet[m] + M_s[m * (kC + 1) + i0 + 1] * bet[i0 + 1];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float kn = k_s[m * (NP + 1) + j * 16 + tx], qn = q_s[m * (NP + 1) + j * 16 + tx];
        dq[0][j] += z0 * kn;
        dq[1][j] += z1 * kn;
        dk[0][j] += zt0 * qn + mm0 * kn;
        dk[1][j] += zt1 * qn + mm1 * kn;
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 2; ++a)
    if (i0 + a < n)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = j * 16 + tx;
        if (e < p.N) {
          const long long o = ((tok0 + i0 + a) * p.G + grp) * p.N + e;
          static_cast<T*>(f.dq)[o] = from_f<T>(dq[a][j]);
          static_cast<T*>(f.dk)[o] = from_f<T>(dk[a][j]);
        }
      }
}

template <typename T, int NJ>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  constexpr int NP = NJ * 16;
  const size_t smem = sizeof(float) * (2 * kC * (NP + 1) + 2 * kTp * NP + 3 * kC * (kTp + 1) + 4 * kC * (kC + 1) +
                                       7 * kC + 8);
  auto kern = delta_grad_kernel<T, NJ>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("delta_grad");
  kern<<<(unsigned)((long long)p.nc * p.G * p.b), kThreads, smem, s>>>(p, f);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_n(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  if (p.N <= 32) return launch_t<T, 2>(p, f, s);
  if (p.N <= 64) return launch_t<T, 4>(p, f, s);
  if (p.N <= 128) return launch_t<T, 8>(p, f, s);
  return launch_t<T, 16>(p, f, s);
}

}  // namespace

cudaError_t launch_delta_grad(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return p.bf16 ? launch_n<__nv_bfloat16>(p, f, s) : launch_n<float>(p, f, s);
}

}  // namespace ssd
