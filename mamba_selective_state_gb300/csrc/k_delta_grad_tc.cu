// k_delta_grad_tc.cu -- dq, dk, dg and dbeta of the gated delta rule on the
// tensor cores, chunk by chunk: the formulas at the head of
// k_delta_grad_simt.cu, with bf16 S0, D1, w and r = dv from the chains.
//
// One CTA takes a chunk of a group and walks its heads, so that q k^T, k k^T
// and the sums over heads stay on chip: dq and dk accumulate in registers, and
// of the pairs' part only Z and M are summed per head, their products with k
// and q taken once per group.  Per head the tensor cores form dY S0^T, r S0^T,
// w D1^T (64 x dstate) and dY w^T, r w^T (64 x 64) from a double-buffered
// stage.  The pairs' contributions to dgam are formed once in fp32 and summed
// by rows and by columns, so that what cancels in their running difference
// cancels exactly.
#include "delta_internal.cuh"
#include "mma_common.cuh"

namespace ssd {
namespace {

using namespace mm;

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 256;
constexpr int kPs = 72;     // row stride of the fp32 q k^T and k k^T
constexpr int kGate = 8;    // heads whose gates are prepared together, one a warp

template <int N, int PC>
struct GradSmem {
  static constexpr int kK = kC * N * 2, kS = N * PC * 2, kV = kC * PC * 2;
  static constexpr int stage = 2 * kS + 3 * kV;  // S0, D1, w, r, dY
  static constexpr int pair = kC * kPs * 4;
  static constexpr int oK = 0, oQ = oK + kK, oSt = oQ + kK, oQK = oSt + 2 * stage, oKK = oQK + pair,
                       oGate = oKK + pair,                       // gam, beta, e, o of kGate heads
                       oSeg = oGate + kGate * 4 * kC * 4, oCol = oSeg + kGate * kC * 4,  // [4][64]
                       oRow = oCol + 4 * kC * 4, oOut = oRow + 2 * kC * 4, oDiag = oOut + 2 * kC * 4, oRed = oDiag + kC * 4,
                       bytes = oRed + 8 * 4;
  static_assert(2 * stage >= 2 * kC * kC * 2, "Z and M reuse the stage");
};

template <int N, int PC>
__global__ void __launch_bounds__(kThreads, 1) delta_grad_tc_kernel(DeltaPlan p, DeltaBufs f) {
  using L = GradSmem<N, PC>;
  constexpr int UN = N / 8, UP = PC / 8;
  constexpr int NT = N / 16;  // 8-column tiles of half of dstate
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sm = smem_u32(raw);
  float* qk_s = reinterpret_cast<float*>(raw + L::oQK);
  float* kk_s = reinterpret_cast<float*>(raw + L::oKK);
  float* colp = reinterpret_cast<float*>(raw + L::oCol);
  float* rowp = reinterpret_cast<float*>(raw + L::oRow);
  float* outp = reinterpret_cast<float*>(raw + L::oOut);
  float* diag = reinterpret_cast<float*>(raw + L::oDiag);
  float* red = reinterpret_cast<float*>(raw + L::oRed);
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3, w = tid >> 5;
  const int rb = w & 3, ch = w >> 2, i0 = 16 * rb + g;
  const int c = (int)(blockIdx.x % p.nc);
  const int grp = (int)((blockIdx.x / p.nc) % p.G);
  const int bi = (int)(blockIdx.x / ((long long)p.nc * p.G));
  const int t0 = c * kC, n = min(kC, p.L - t0);
  const long long tok0 = (long long)bi * p.L + t0;
  const int npc = p.P / PC, steps = p.hpg * npc;
  const long long vs = (long long)p.H * p.P;

  auto load = [&](int s) {
    const int h = grp * p.hpg + s / npc, p0 = (s % npc) * PC;
    const uint32_t st = sm + L::oSt + (s & 1) * L::stage;
    const long long unit = ((long long)bi * p.H + h) * p.nc + c;
    cp_tile<N, UP>(st, static_cast<const __nv_bfloat16*>(f.S) + unit * N * p.P + p0, p.P, N, tid, kThreads);
    cp_tile<N, UP>(st + L::kS, static_cast<const __nv_bfloat16*>(f.D) + unit * N * p.P + p0, p.P, N, tid, kThreads);
    cp_tile<kC, UP>(st + 2 * L::kS, static_cast<const __nv_bfloat16*>(f.w) + unit * kC * p.P + p0, p.P, kC, tid, kThreads);
    const long long o = tok0 * vs + (long long)h * p.P + p0;
    cp_tile<kC, UP>(st + 2 * L::kS + L::kV, static_cast<const __nv_bfloat16*>(f.dv) + o, vs, n, tid, kThreads);
    cp_tile<kC, UP>(st + 2 * L::kS + 2 * L::kV, static_cast<const __nv_bfloat16*>(f.dy) + o, vs, n, tid, kThreads);
    cp_commit();
  };
  // gam, beta, e, o and the sequence starts of head hh, by one warp
  auto gates = [&](int hh) {
    float* ga = reinterpret_cast<float*>(raw + L::oGate) + (hh % kGate) * 4 * kC;
    int* sg = reinterpret_cast<int*>(raw + L::oSeg) + (hh % kGate) * kC;
    const int h = grp * p.hpg + hh;
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
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * lane + j;
      const float gam = j ? sum : sum - gv[1];
      const int s = j ? cnt : cnt - rs[1];
      ga[i] = gam;
      ga[kC + i] = be[j];
      ga[2 * kC + i] = s == 0 ? expf(gam) : 0.f;
      ga[3 * kC + i] = s == slast ? expf(last - gam) : 0.f;
      sg[i] = s;
    }
  };

  cp_tile<kC, UN>(sm + L::oK, static_cast<const __nv_bfloat16*>(f.k) + tok0 * p.ks + (long long)grp * N, p.ks, n, tid, kThreads);
  cp_tile<kC, UN>(sm + L::oQ, static_cast<const __nv_bfloat16*>(f.q) + tok0 * p.qs + (long long)grp * N, p.qs, n, tid, kThreads);
  cp_commit();
  load(0);
  if (w < p.hpg) gates(w);
  cp_wait<1>();
  __syncthreads();
  {
    float a1[4][4] = {}, a2[4][4] = {};
#pragma unroll 2
    for (int ks = 0; ks < N; ks += 16) {
      uint32_t ka[4], qa[4], b[4];
      load_a<UN>(ka, sm + L::oK, 16 * rb, ks, lane);
      load_a<UN>(qa, sm + L::oQ, 16 * rb, ks, lane);
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        load_b<UN>(b, sm + L::oK, 32 * ch + j * 8, ks, lane);
        mma(a1[j], qa, b[0], b[1]);
        mma(a1[j + 1], qa, b[2], b[3]);
        mma(a2[j], ka, b[0], b[1]);
        mma(a2[j + 1], ka, b[2], b[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int o = (i0 + 8 * r) * kPs + 32 * ch + j * 8 + 2 * t;
        *reinterpret_cast<float2*>(&qk_s[o]) = make_float2(a1[j][2 * r], a1[j][2 * r + 1]);
        *reinterpret_cast<float2*>(&kk_s[o]) = make_float2(a2[j][2 * r], a2[j][2 * r + 1]);
      }
  }
  float dq[NT][4] = {}, dk[NT][4] = {}, Z[4][4] = {}, M[4][4] = {};
  float m1[4][4], m2[4][4], row[2], out[2], sd;
  for (int s = 0; s < steps; ++s) {
    const int hh = s / npc, pc = s % npc;
    cp_wait<0>();
    __syncthreads();
    if (s + 1 < steps) load(s + 1);
    const float* ga = reinterpret_cast<const float*>(raw + L::oGate) + (hh % kGate) * 4 * kC;
    const int* sg = reinterpret_cast<const int*>(raw + L::oSeg) + (hh % kGate) * kC;
    const uint32_t Ss = sm + L::oSt + (s & 1) * L::stage, Ds = Ss + L::kS, Ws = Ss + 2 * L::kS, Rs = Ws + L::kV,
                   Ys = Rs + L::kV;
    if (pc == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) m1[j][x] = m2[j][x] = 0.f;
      row[0] = row[1] = out[0] = out[1] = sd = 0.f;
    }
    for (int i = tid; i < N * UP; i += kThreads) {
      const uint4 a = lds128(Ss + i * 16), b = lds128(Ds + i * 16);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = unpack2(av[j]), v = unpack2(bv[j]);
        sd += u.x * v.x + u.y * v.y;
      }
    }
    // which: 0 dY S0^T, 1 r S0^T, 2 w D1^T; the first two also against w
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const uint32_t As = which == 0 ? Ys : which == 1 ? Rs : Ws, Bs = which == 2 ? Ds : Ss;
      float x[NT][4] = {};
#pragma unroll
      for (int ks = 0; ks < PC; ks += 16) {
        uint32_t a[4], b[4];
        load_a<UP>(a, As, 16 * rb, ks, lane);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          load_b<UP>(b, Bs, ch * (N / 2) + j * 8, ks, lane);
          mma(x[j], a, b[0], b[1]);
          mma(x[j + 1], a, b[2], b[3]);
        }
        if (which < 2) {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            load_b<UP>(b, Ws, 32 * ch + j * 8, ks, lane);
            if (which == 0) {
              mma(m1[j], a, b[0], b[1]);
              mma(m1[j + 1], a, b[2], b[3]);
            } else {
              mma(m2[j], a, b[0], b[1]);
              mma(m2[j + 1], a, b[2], b[3]);
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = i0 + 8 * r;
        const float fac = which == 0 ? p.scale * ga[2 * kC + i] : which == 1 ? -ga[2 * kC + i] : ga[3 * kC + i];
        const float be = ga[kC + i];
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = ch * (N / 2) + j * 8 + 2 * t;
          const float2 v = unpack2(lds32(sm + (which == 0 ? L::oQ : L::oK) + elem_off<UN>(i, col)));
          const float x0 = fac == 0.f ? 0.f : fac * x[j][2 * r], x1 = fac == 0.f ? 0.f : fac * x[j][2 * r + 1];
          dot += v.x * x0 + v.y * x1;
          if (which == 0) {
            dq[j][2 * r] += x0;
            dq[j][2 * r + 1] += x1;
          } else {
            dk[j][2 * r] += which == 2 ? be * x0 : x0;
            dk[j][2 * r + 1] += which == 2 ? be * x1 : x1;
          }
        }
        if (which == 2) out[r] += dot; else row[r] += dot;
      }
    }
    if (pc + 1 < npc) continue;
    // the pairs of this head
    float col[4][2] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = i0 + 8 * r;
      const float gi = ga[i];
      const int si = sg[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int jj = 32 * ch + j * 8 + 2 * t;
        const float2 qk = *reinterpret_cast<const float2*>(&qk_s[i * kPs + jj]);
        const float2 kk = *reinterpret_cast<const float2*>(&kk_s[i * kPs + jj]);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (jj + x <= i && sg[jj + x] == si) {
            const float E = __expf(gi - ga[jj + x]), be = ga[kC + jj + x];
            const float z = p.scale * E * m1[j][2 * r + x];
            const float m = jj + x < i ? -E * m2[j][2 * r + x] : 0.f;
            const float both = z * (x ? qk.y : qk.x) + m * (x ? kk.y : kk.x);
            if (jj + x < i) {
              col[j][x] += both;
              row[r] += be * both;
            } else {
              diag[i] = both;  // a token's own pair does not depend on the decays
            }
            Z[j][2 * r + x] += be * z;
            M[j][2 * r + x] += be * m;
          }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = col[j][x];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (g == 0) colp[rb * kC + 32 * ch + j * 8 + 2 * t + x] = v;
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v = row[r], o = out[r];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      o += __shfl_xor_sync(0xffffffffu, o, 1);
      o += __shfl_xor_sync(0xffffffffu, o, 2);
      if (t == 0) {
        rowp[ch * kC + i0 + 8 * r] = v;
        outp[ch * kC + i0 + 8 * r] = o;
      }
    }
    float v = sd;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[w] = v;
    __syncthreads();
    if (w == (hh & 7)) {
      // this head's dbeta, and dg as the reverse cumulative sum of dgam
      float d[2], all = 0.f, sdot = 0.f;
      for (int i = 0; i < 8; ++i) sdot += red[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        const float o = outp[i] + outp[kC + i], be = ga[kC + i];
        const float cs = (colp[i] + colp[kC + i]) + (colp[2 * kC + i] + colp[3 * kC + i]);
        d[j] = rowp[i] + rowp[kC + i] - be * (cs + o);
        all += be * o;
        if (i < n) static_cast<__nv_bfloat16*>(f.dbeta)[(tok0 + i) * p.H + grp * p.hpg + hh] = __float2bfloat16_rn(cs + diag[i] + o);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      const float el = ga[2 * kC + kC - 1];
      if (lane == 31) d[1] += all + (el == 0.f ? 0.f : el * sdot);
      float sum = d[0] + d[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float dn = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += dn;
      }
      // `sum` runs from this lane's first token to the end
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        const bool starts = i > 0 ? sg[i] != sg[i - 1] : sg[0] != 0;
        const float v2 = starts ? 0.f : j ? sum - d[0] : sum;
        if (i < n) static_cast<__nv_bfloat16*>(f.dg)[(tok0 + i) * p.H + grp * p.hpg + hh] = __float2bfloat16_rn(v2);
      }
    }
    if ((hh + 1) % kGate == 0 && hh + 1 < p.hpg) {
      __syncthreads();  // the gates of these heads have been read
      if (hh + 1 + w < p.hpg) gates(hh + 1 + w);
    }
  }
  // the pairs' part of dq and dk, once for all heads
  __syncthreads();
  const uint32_t Zs = sm + L::oSt, Ms = Zs + kC * kC * 2;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t o = elem_off<8>(i0 + 8 * r, 32 * ch + j * 8 + 2 * t);
      sts32(Zs + o, pack2(Z[j][2 * r], Z[j][2 * r + 1]));
      sts32(Ms + o, pack2(M[j][2 * r], M[j][2 * r + 1]));
    }
  __syncthreads();
#pragma unroll
  for (int ks = 0; ks < kC; ks += 16) {
    uint32_t a[4], b[4], bq[4], am[4], amt[4], azt[4];
    const bool lower = ks <= 16 * rb, upper = ks >= 16 * rb;
    if (lower) {
      load_a<8>(a, Zs, 16 * rb, ks, lane);
      load_a<8>(am, Ms, 16 * rb, ks, lane);
    }
    if (upper) {
      load_at<8>(azt, Zs, 16 * rb, ks, lane);
      load_at<8>(amt, Ms, 16 * rb, ks, lane);
    }
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      load_bt<UN>(b, sm + L::oK, ch * (N / 2) + j * 8, ks, lane);
      if (lower) {
        mma(dq[j], a, b[0], b[1]);
        mma(dq[j + 1], a, b[2], b[3]);
        mma(dk[j], am, b[0], b[1]);
        mma(dk[j + 1], am, b[2], b[3]);
      }
      if (upper) {
        load_bt<UN>(bq, sm + L::oQ, ch * (N / 2) + j * 8, ks, lane);
        mma(dk[j], azt, bq[0], bq[1]);
        mma(dk[j + 1], azt, bq[2], bq[3]);
        mma(dk[j], amt, b[0], b[1]);
        mma(dk[j + 1], amt, b[2], b[3]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = i0 + 8 * r;
    if (i < n) {
      const long long o = ((tok0 + i) * p.G + grp) * N + ch * (N / 2) + 2 * t;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(f.dq) + o + j * 8) = pack2(dq[j][2 * r], dq[j][2 * r + 1]);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(f.dk) + o + j * 8) = pack2(dk[j][2 * r], dk[j][2 * r + 1]);
      }
    }
  }
}

template <int N, int PC>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  auto kern = delta_grad_tc_kernel<N, PC>;
  constexpr int smem = GradSmem<N, PC>::bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("delta_grad_tc");
  kern<<<(unsigned)((long long)p.nc * p.G * p.b), kThreads, smem, s>>>(p, f);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grad_tc(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  if (p.P % 64 == 0) return p.N == 128 ? launch_t<128, 64>(p, f, s) : launch_t<64, 64>(p, f, s);
  return p.N == 128 ? launch_t<128, 32>(p, f, s) : launch_t<64, 32>(p, f, s);
}

}  // namespace ssd
