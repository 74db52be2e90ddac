// k_delta_prep.cu -- the parts of the gated delta rule's chunks that do not
// depend on the state, for every chunk of 64 tokens at once:
//
//   M_ij = E_ij (k_i.k_j) beta_j (j < i),  A_ij = scale E_ij (q_i.k_j) beta_j (j <= i)
//   the gates' records                     (see delta_internal.cuh)
//
// The chains solve (I + M) w = R by blocks of 16 tokens; T holds what they
// need for it: -M below the diagonal blocks, and (I + M_ii)^-1 - I in them.
// Those four inverses are taken by forward substitution in fp32, a lane per
// column.  (Powers of M would need fewer steps, but they overflow where keys
// repeat; and the whole inverse of 64 x 64 costs this kernel three times as
// much as its four blocks while it saves the chains' solve 6 % of their time.)
//
// One CTA takes a chunk of up to eight heads of a group: k k^T and q k^T do
// not depend on the head and stay in registers, four warps with 16 rows of
// k k^T (T) and four with q k^T (A).  A warp's rows depend on no other warp's.
// M, the inverses and A are formed in fp32 and rounded to bf16 once, as operands of
// the chains' products (see k_delta_chain.cu).
// Bound by the instructions of the pairs' decays and of the substitution: 110 us
// at batch 2, L = 8192, 64 heads in 8 groups, where it writes 0.30 GB.
#include "delta_internal.cuh"
#include "mma_common.cuh"

namespace ssd {
namespace {

using namespace mm;

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 256;
constexpr int kHeads = 8;  // heads a CTA takes at most: their gates are prepared together, one a warp
constexpr int kDs = 20;  // row stride of the fp32 diagonal blocks

template <int N>
struct PrepSmem {
  // q and k tiles, then in the same place T, A and the diagonal blocks
  static constexpr int kQK = 2 * kC * N * 2 > 2 * kC * kC * 2 + 4 * 16 * kDs * 4 ? 2 * kC * N * 2
                                                                                 : 2 * kC * kC * 2 + 4 * 16 * kDs * 4;
  static constexpr int kTile = kC * kC * 2;                    // T and A, bf16
  static constexpr int oA = kTile, oDg = 2 * kTile;            // fp32 diagonal blocks of M
  static constexpr int oGate = kQK;                            // gam, beta by head
  static constexpr int oSeg = oGate + kHeads * 2 * kC * 4;
  static constexpr int oTab = oSeg + kHeads * kC * 4;          // decay factors by warp
  static constexpr int bytes = oTab + 8 * kC * 4;
};

template <int N>
__global__ void __launch_bounds__(kThreads, 3) delta_prep_kernel(DeltaPlan p, DeltaBufs f, int heads_per_cta) {
  using L = PrepSmem<N>;
  constexpr int U = N / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t k_s = smem_u32(raw), q_s = k_s + kC * N * 2, A_s = k_s + L::oA, T_s = k_s;

  const int tid = threadIdx.x, lane = tid & 31, w = (tid >> 5) & 3;
  const bool forms_a = tid >= 128;
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

  // gam, beta and sequence starts of head h into its slot, its record to
  // global, by one warp with two tokens a lane.  (gam is one fp32 sum of at most 64
  // decays of -100: it rounds a pair's decay by up to 2e-4 of it, a tenth of the
  // bf16 rounding of the products that take it.)
  auto gates = [&](int h) {
    float* gam = reinterpret_cast<float*>(raw + L::oGate) + (h - h0) * 2 * kC;
    int* seg = reinterpret_cast<int*>(raw + L::oSeg) + (h - h0) * kC;
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
    *reinterpret_cast<float2*>(eg + kGateOB * kC) = make_float2(o[0] * be[0], o[1] * be[1]);
    const float mid = __shfl_sync(0xffffffffu, ga[0], 16);
    const int smid = __shfl_sync(0xffffffffu, sg[0], 16);
    const float dir = lane < 16 ? -1.f : 1.f;
    constexpr float kLog2e = 1.4426950408889634f;
    *reinterpret_cast<float2*>(eg + kGateGam * kC) = make_float2(kLog2e * ga[0], kLog2e * ga[1]);
    *reinterpret_cast<float2*>(eg + kGateBeta * kC) = make_float2(be[0], be[1]);
    *reinterpret_cast<float2*>(eg + kGateO * kC) = make_float2(o[0], o[1]);
    *reinterpret_cast<float2*>(eg + kGateHalf * kC) = make_float2(sg[0] == smid ? expf(dir * (ga[0] - mid)) : 0.f,
                                                                  sg[1] == smid ? expf(dir * (ga[1] - mid)) : 0.f);
    *reinterpret_cast<int2*>(eg + kGateSeg * kC) = make_int2(sg[0], sg[1]);
  };

  cp_tile<kC, U>(k_s, static_cast<const __nv_bfloat16*>(f.k) + tok0 * p.ks + (long long)grp * N, p.ks, n, tid, kThreads);
  cp_tile<kC, U>(q_s, static_cast<const __nv_bfloat16*>(f.q) + tok0 * p.qs + (long long)grp * N, p.qs, n, tid, kThreads);
  cp_commit();
  if (h0 + (tid >> 5) < h1) gates(h0 + (tid >> 5));
  cp_wait<0>();
  __syncthreads();
  // rows 16w.. of k k^T or of q k^T, columns up to the diagonal block
  float prod[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) prod[i][j] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < N; ks += 16) {
    uint32_t a[4], b[4];
    load_a<U>(a, forms_a ? q_s : k_s, 16 * w, ks, lane);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      if (nb <= w) {
        load_b<U>(b, k_s, 16 * nb, ks, lane);
        mma(prod[2 * nb], a, b[0], b[1]);
        mma(prod[2 * nb + 1], a, b[2], b[3]);
      }
  }
  __syncthreads();  // the tiles have been read
  const int i0 = 16 * w + g;
  // Left of the diagonal block the decay from column j to row i is the product
  // of those to and from the block's first token: two exponentials a lane
  // instead of one a pair.
  float* tab = reinterpret_cast<float*>(raw + L::oTab) + (tid >> 5) * kC;
  float* Dg = reinterpret_cast<float*>(raw + L::oDg) + w * 16 * kDs;
  struct Head {
    const float *gam, *bet;
    const int* seg;
    float gi[2], rf[2];
    int si[2];
  };
  auto head = [&](int h) {
    Head x;
    x.gam = reinterpret_cast<const float*>(raw + L::oGate) + (h - h0) * 2 * kC;
    x.bet = x.gam + kC;
    x.seg = reinterpret_cast<const int*>(raw + L::oSeg) + (h - h0) * kC;
    const float gr = x.gam[16 * w];
    const int sr = x.seg[16 * w];
    __syncwarp();
    for (int j = lane; j < 16 * w; j += 32) tab[j] = x.seg[j] == sr ? __expf(gr - x.gam[j]) * x.bet[j] : 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      x.gi[r] = x.gam[i0 + 8 * r];
      x.si[r] = x.seg[i0 + 8 * r];
      x.rf[r] = x.si[r] == sr ? __expf(x.gi[r] - gr) : 0.f;
    }
    __syncwarp();
    return x;
  };
  // E_ij beta_j of the columns j, j + 1 of the diagonal block (no branches:
  // the exponentials' latencies overlap)
  auto near = [&](const Head& x, int r, int j) {
    const float2 gj = *reinterpret_cast<const float2*>(x.gam + j), bj = *reinterpret_cast<const float2*>(x.bet + j);
    const int2 sj = *reinterpret_cast<const int2*>(x.seg + j);
    const int i = i0 + 8 * r;
    const float e0 = __expf(x.gi[r] - gj.x) * bj.x, e1 = __expf(x.gi[r] - gj.y) * bj.y;
    return make_float2((j <= i) & (sj.x == x.si[r]) ? e0 : 0.f, (j + 1 <= i) & (sj.y == x.si[r]) ? e1 : 0.f);
  };
  if (forms_a) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (nt > 2 * w + 1)
          sts32(A_s + elem_off<8>(i0 + 8 * r, nt * 8 + 2 * t), 0u);  // above the diagonal block, once
        else
          prod[nt][2 * r] *= p.scale, prod[nt][2 * r + 1] *= p.scale;
    for (int h = h0; h < h1; ++h) {
      const long long unit = ((long long)bi * p.H + h) * p.nc + c;
      const Head x = head(h);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const int j = nt * 8 + 2 * t;
        if (nt < 2 * w) {
          const float2 cf = *reinterpret_cast<const float2*>(tab + j);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sts32(A_s + elem_off<8>(i0 + 8 * r, j),
                  pack2(x.rf[r] * cf.x * prod[nt][2 * r], x.rf[r] * cf.y * prod[nt][2 * r + 1]));
        } else if (nt <= 2 * w + 1) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 E = near(x, r, j);
            sts32(A_s + elem_off<8>(i0 + 8 * r, j), pack2(E.x * prod[nt][2 * r], E.y * prod[nt][2 * r + 1]));
          }
        }
      }
      __syncwarp();
      uint4* Ag = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.A) + unit * kC * kC) + 16 * 8 * w;
#pragma unroll
      for (int i = lane; i < 16 * 8; i += 32) Ag[i] = lds128(A_s + tile_off<8>(16 * w + (i >> 3), i & 7));
    }
    return;
  }
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (nt > 2 * w + 1) sts32(T_s + elem_off<8>(i0 + 8 * r, nt * 8 + 2 * t), 0u);
  for (int h = h0; h < h1; ++h) {
    const long long unit = ((long long)bi * p.H + h) * p.nc + c;
    const Head x = head(h);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const int j = nt * 8 + 2 * t;
      if (nt < 2 * w) {
        const float2 cf = *reinterpret_cast<const float2*>(tab + j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sts32(T_s + elem_off<8>(i0 + 8 * r, j),
                pack2(-x.rf[r] * cf.x * prod[nt][2 * r], -x.rf[r] * cf.y * prod[nt][2 * r + 1]));
        }
      } else if (nt <= 2 * w + 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 E = near(x, r, j);
          const int i = i0 + 8 * r;
          *reinterpret_cast<float2*>(&Dg[(g + 8 * r) * kDs + j - 16 * w]) =
              make_float2(j < i ? E.x * prod[nt][2 * r] : 0.f, j + 1 < i ? E.y * prod[nt][2 * r + 1] : 0.f);
        }
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
          const float4 m = *reinterpret_cast<const float4*>(&Dg[i * kDs + jb]);  // zeros from the diagonal on
          x[i] -= m.x * x[jb];
          if (i > jb + 1) x[i] -= m.y * x[jb + 1];
          if (i > jb + 2) x[i] -= m.z * x[jb + 2];
          if (i > jb + 3) x[i] -= m.w * x[jb + 3];
        }
      if (lane < 16)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat16 v = __float2bfloat16_rn(i == col ? 0.f : x[i]);
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(T_s + elem_off<8>(16 * w + i, 16 * w + col)),
                       "h"(*reinterpret_cast<const uint16_t*>(&v))
                       : "memory");
        }
    }
    __syncwarp();
    uint4* Tg = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.T) + unit * kC * kC) + 16 * 8 * w;
#pragma unroll
    for (int i = lane; i < 16 * 8; i += 32) Tg[i] = lds128(T_s + tile_off<8>(16 * w + (i >> 3), i & 7));
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
  int heads = p.hpg < kHeads ? p.hpg : kHeads;
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
