// k_delta_grad_tc.cu -- dq, dk, dg and dbeta of the gated delta rule on the
// tensor cores, chunk by chunk: the formulas at the head of
// k_delta_grad_simt.cu, with bf16 S0, D1, w and r = dv from the chains.
//
// One CTA takes a chunk of a group and walks its heads.  Per head, with the
// tokens of dY and of r as the 128 rows of one left operand,
//
//   [dY ; r] [S0 | w']  ->  dY S0, r S0 (64 x dstate) and dY w', r w' (64 x 64)
//   [.. ; w]  D1        ->  w D1
//
// come from tcgen05 products into tensor memory (S0, D1 and w' are stored with
// headdim as rows, as the chains write them, and enter as MN-major operands).
// Sixteen warps read them back: a thread owns one token's row -- of dY and dq
// in the lower 64 lanes, of r, w and dk in the upper -- and a quarter of the
// columns, so the dot products with q and k and the sums over heads stay in
// its registers.  q k^T and k k^T do not depend on the head, and the pairs'
// part of dq and dk is summed over the heads before its products with k and
// q: both are one more product of 128 rows per group.  The pairs'
// contributions to dgam are formed once in fp32 and summed by rows and by
// columns, so that what cancels in their running difference cancels exactly.
#include "delta_internal.cuh"
#include "mma_common.cuh"
#include "tma_host.h"

namespace ssd {
namespace {

using namespace mm;
using namespace tc;

constexpr int kC = kDeltaChunk;
constexpr int kWarps = 16;                    // epilogue warps
constexpr int kEpi = kWarps * 32;
constexpr int kThreads = kEpi + 128;          // and the control warp with three idle ones: registers
                                              // are handed over by groups of four warps
// Registers a thread: 640 threads are launched with 96; the control warps keep
// 32 and the epilogue warps take 112 (4 x 112 + 32 = 5 x 96).  Without that
// the epilogue spills, and the ring leaves the L1 cache too small for it.
// named barriers: the epilogue's own; a head's sums are written (by parity), and have been used
constexpr int kBarSums = 2, kBarFree = 4;
constexpr int kSums = kEpi + 64;  // the epilogue, the warp of <S0, D1> and the one that uses the sums
constexpr int kRegsEpi = 112, kRegsCtl = 32;
constexpr uint32_t kTile = 8192;              // [64][64] bf16, 128-byte swizzle
constexpr int kGate = kGateRows * kC * 4;

struct GradMaps {
  CUtensorMap q, k, S, D, w, dv, dy;
};

template <int N>
struct GradSmem {
  static constexpr int NB = N / 64;
  // per head and 64 columns of headdim: dY, r, S0, w, D1
  static constexpr int stage = (2 + 2 * NB + 1) * (int)kTile;
  static constexpr int kStages = N == 128 ? 3 : 4;
  // q and k: for each 64 columns of dstate the tile of q above that of k
  static constexpr int oQK = 0, oSt = NB * 2 * (int)kTile, oGate = oSt + kStages * stage,  // four gate records
                       oCol = oGate + 4 * kGate,       // [2][4][64] column sums by lane quarter
                       oRow = oCol + 2 * 4 * kC * 4,   // [2][4][128] row sums by column quarter
                       oOut = oRow + 2 * 4 * 128 * 4,  // [2][4][64] k.(D1 w)
                       oDiag = oOut + 2 * 4 * kC * 4, oRed = oDiag + 2 * kC * 4, oBar = oRed + 16,
                       bytes = oBar + 256 + 1024;
  static_assert(kStages * stage >= 4 * (int)kTile, "the pairs' operand reuses the ring");
};

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Sum over the warp's lanes of v[0..15]: lane l returns the total of v[l >> 1].
__device__ __forceinline__ float sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    const bool up = lane & (2 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half];
      const float keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * half);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    delta_grad_tc_kernel(DeltaPlan p, DeltaBufs f, const __grid_constant__ GradMaps m) {
  using L = GradSmem<N>;
  constexpr int NB = L::NB, NC = N / 4;        // columns of dstate per thread
  constexpr uint32_t kX = N + 64;              // columns of [dY ; r] [S0 | w']
  constexpr uint32_t kX3 = 2 * kX;             // tensor-memory column of w D1
  constexpr uint32_t kCols = 512;
  extern __shared__ unsigned char raw_[];
  unsigned char* raw = raw_ + ((1024 - (smem_u32(raw_) & 1023)) & 1023);
  const uint32_t sm = smem_u32(raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(raw + L::oBar);
  uint64_t *s_full = bars, *s_free = bars + 4, *g_full = bars + 8, *g_free = bars + 12, *x_full = bars + 16,
           *x_free = bars + 18, *x3_free = bars + 20, *qk_full = bars + 21, *qk_done = bars + 22, *z_done = bars + 23;
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(bars + 24);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int c = (int)(blockIdx.x % p.nc);
  const int grp = (int)((blockIdx.x / p.nc) % p.G);
  const int bi = (int)(blockIdx.x / ((long long)p.nc * p.G));
  const int t0 = c * kC, n = min(kC, p.L - t0);
  const long long tok0 = (long long)bi * p.L + t0;
  const int npc = p.P / 64, h0 = grp * p.hpg;

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(g_full + i, 1);
      mbar_init(g_free + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(x_full + i, 1);
      mbar_init(x_free + i, kWarps);
    }
    mbar_init(x3_free, kWarps);
    mbar_init(qk_full, 1);
    mbar_init(qk_done, 1);
    mbar_init(z_done, 1);
    mbar_fence_init();
  }
  if (w == kWarps) tmem_alloc(tm_slot, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tm_slot;
  bool ok = true;

  if (w >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (w == kWarps && lane == 0) {
      const int steps = p.hpg * npc;
      auto load = [&](int s) {
        const int hh = s / npc, pc = s % npc, st = s % L::kStages, use = s / L::kStages;
        const int h = h0 + hh, bh = bi * p.H + h;
        if (pc == 0) {
          // four records: this runs up to three heads ahead of the products
          const int gb = hh & 3;
          if (hh >= 4) mbar_wait_flag(g_free + gb, ((hh >> 2) - 1) & 1, ok);
          mbar_expect_tx(g_full + gb, kGate);
          bulk_load(raw + L::oGate + gb * kGate,
                    static_cast<const float*>(f.e) + ((long long)bh * p.nc + c) * kGateRows * kC, kGate, g_full + gb);
        }
        if (use > 0) mbar_wait_flag(s_free + st, (use - 1) & 1, ok);
        unsigned char* d = raw + L::oSt + st * L::stage;
        mbar_expect_tx(s_full + st, L::stage);
        tma_load_4d(d, &m.dy, s_full + st, 64 * pc, h, t0, bi);
        tma_load_4d(d + kTile, &m.dv, s_full + st, 64 * pc, h, t0, bi);
        for (int j = 0; j < NB; ++j) tma_load_4d(d + (2 + j) * kTile, &m.S, s_full + st, 64 * j, 64 * pc, c, bh);
        tma_load_4d(d + (2 + NB) * kTile, &m.w, s_full + st, 0, 64 * pc, c, bh);
        for (int j = 0; j < NB; ++j) tma_load_4d(d + (3 + NB + j) * kTile, &m.D, s_full + st, 64 * j, 64 * pc, c, bh);
      };
      mbar_expect_tx(qk_full, NB * 2 * kTile);
      for (int j = 0; j < NB; ++j) {
        tma_load_4d(raw + L::oQK + 2 * j * kTile, &m.q, qk_full, 64 * j, grp, t0, bi);
        tma_load_4d(raw + L::oQK + (2 * j + 1) * kTile, &m.k, qk_full, 64 * j, grp, t0, bi);
      }
      int loaded = 0;
      for (; loaded < L::kStages - 1 && loaded < steps; ++loaded) load(loaded);
      // [q ; k] k^T into the first columns
      mbar_wait_flag(qk_full, 0, ok);
      tc_fence_after();
      for (int ks = 0; ks < N / 16; ++ks) {
        const uint32_t a = sm + L::oQK + (ks >> 2) * 2 * kTile + (ks & 3) * 32;
        mma_bf16(tm, smem_desc(a, 16, 1024, kSwz128), smem_desc(a + kTile, 16, 1024, kSwz128),
                 idesc_bf16(128, 64, 0, 0), ks > 0);
      }
      mma_commit(qk_done);
      for (int s = 0; s < steps; ++s) {
        const int hh = s / npc, pc = s % npc, st = s % L::kStages, use = s / L::kStages, buf = hh & 1;
        if (loaded < steps) load(loaded++);
        mbar_wait_flag(s_full + st, use & 1, ok);
        if (pc == 0) {
          // the buffer's last head has been read (the first head's: q k^T)
          if (hh >= 2) mbar_wait_flag(x_free + buf, ((hh >> 1) - 1) & 1, ok);
          if (hh == 0) mbar_wait_flag(z_done, 0, ok);
        }
        tc_fence_after();
        const uint32_t base = sm + L::oSt + st * L::stage, S0 = base + 2 * kTile, D1 = base + (3 + NB) * kTile;
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16(tm + buf * kX, smem_desc(base + ks * 32, 16, 1024, kSwz128),
                   smem_desc(S0 + ks * 2048, kTile, 1024, kSwz128), idesc_bf16(128, N + 64, 0, 1), pc > 0 || ks > 0);
        if (pc == 0 && hh >= 1) {
          mbar_wait_flag(x3_free, (hh - 1) & 1, ok);
          tc_fence_after();
        }
        // rows 64.. are w: the tile before it only fills the product's 128 rows
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16(tm + kX3, smem_desc(S0 + (NB - 1) * kTile + ks * 2048, kTile, 1024, kSwz128),
                   smem_desc(D1 + ks * 2048, kTile, 1024, kSwz128), idesc_bf16(128, N, 1, 1), pc > 0 || ks > 0);
        mma_commit(s_free + st);
        if (pc == npc - 1) mma_commit(x_full + buf);
      }
      // the pairs' part, once its operand is in place (the epilogue's arrivals on qk_full)
      mbar_wait_flag(qk_full, 1, ok);
      tc_fence_after();
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t a = sm + L::oSt + (ks >> 2) * 2 * kTile + (ks & 3) * 32;
        mma_bf16(tm, smem_desc(a, 16, 1024, kSwz128), smem_desc(sm + L::oQK + ks * 2048, 2 * kTile, 1024, kSwz128),
                 idesc_bf16(128, N, 0, 1), ks > 0);
      }
      mma_commit(qk_done);
    }
    __syncwarp();
    if (w == kWarps + 1 || w == kWarps + 2) {
      // the even or the odd heads' sums over a chunk, beside the next head's epilogue
      for (int hh = w - kWarps - 1; hh < p.hpg; hh += 2) {
        const int buf = hh & 1;
        const float* ga = reinterpret_cast<const float*>(raw + L::oGate + (hh & 3) * kGate);
        const int* sg = reinterpret_cast<const int*>(ga + kGateSeg * kC);
        const float* colp = reinterpret_cast<const float*>(raw + L::oCol) + buf * 4 * kC;
        const float* rowp = reinterpret_cast<const float*>(raw + L::oRow) + buf * 4 * 128;
        const float* outp = reinterpret_cast<const float*>(raw + L::oOut) + buf * 4 * kC;
        const float* diag = reinterpret_cast<const float*>(raw + L::oDiag) + buf * kC;
        mbar_wait_flag(g_full + (hh & 3), (hh >> 2) & 1, ok);
        bar_sync(kBarSums + buf, kSums);
        // this head's dbeta, and dg as the reverse cumulative sum of dgam
        float d[2], all = 0.f;
        const float sdot = reinterpret_cast<const float*>(raw + L::oRed)[buf];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int a = 2 * lane + j;
          const float o = (outp[a] + outp[kC + a]) + (outp[2 * kC + a] + outp[3 * kC + a]);
          const float cj = (colp[a] + colp[kC + a]) + (colp[2 * kC + a] + colp[3 * kC + a]);
          float r = 0.f;
#pragma unroll
          for (int x2 = 0; x2 < 4; ++x2) r += rowp[x2 * 128 + a] + rowp[x2 * 128 + 64 + a];
          const float b2 = ga[kGateBeta * kC + a];
          d[j] = r - b2 * (cj + o);
          all += b2 * o;
          if (a < n)
            static_cast<__nv_bfloat16*>(f.dbeta)[(tok0 + a) * p.H + h0 + hh] = __float2bfloat16_rn(cj + diag[a] + o);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const float el = ga[kC - 1];
        if (lane == 31) d[1] += all + (el == 0.f ? 0.f : el * sdot);
        float sum = d[0] + d[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float dn = __shfl_down_sync(0xffffffffu, sum, o);
          if (lane + o < 32) sum += dn;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int a = 2 * lane + j;
          const bool starts = a > 0 ? sg[a] != sg[a - 1] : sg[0] != 0;
          const float v = starts ? 0.f : j ? sum - d[0] : sum;
          if (a < n) static_cast<__nv_bfloat16*>(f.dg)[(tok0 + a) * p.H + h0 + hh] = __float2bfloat16_rn(v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(g_free + (hh & 3));
        if (hh + 2 < p.hpg) bar_arrive(kBarFree + buf, kSums);
      }
    } else if (w == kWarps + 3) {
      // <S0, D1> of every head: the diagonal of 16 x 8 products
      const int g = lane >> 2, t = lane & 3;
      for (int hh = 0; hh < p.hpg; ++hh) {
        float sd = 0.f;
        for (int pc = 0; pc < npc; ++pc) {
          const int s = hh * npc + pc, st = s % L::kStages;
          mbar_wait_flag(s_full + st, (s / L::kStages) & 1, ok);
          const uint32_t S0 = sm + L::oSt + st * L::stage + 2 * kTile, D1 = S0 + (NB + 1) * kTile;
          for (int r = 0; r < 64; r += 16) {
            float x0[4] = {}, x1[4] = {};
#pragma unroll
            for (int k = 0; k < N; k += 16) {
              uint32_t a[4], b[4];
              load_a<8>(a, S0 + (k >> 6) * kTile, r, k & 63, lane);
              load_b<8>(b, D1 + (k >> 6) * kTile, r, k & 63, lane);
              mm::mma(x0, a, b[0], b[1]);
              mm::mma(x1, a, b[2], b[3]);
            }
            if (t == (g >> 1)) sd += (g & 1) ? x0[1] + x1[3] : x0[0] + x1[2];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + st);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
        if (hh >= 2) bar_sync(kBarFree + (hh & 1), kSums);
        if (lane == 0) reinterpret_cast<float*>(raw + L::oRed)[hh & 1] = sd;
        __syncwarp();
        bar_arrive(kBarSums + (hh & 1), kSums);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int quarter = w & 3, cq = w >> 2;          // tensor-memory lanes, columns
    const int row = 32 * quarter + lane, i = row & 63;
    const bool lower = quarter < 2;                  // dY, dq, q k^T; else r, w, dk, k k^T
    const uint32_t tlane = tmem_addr(tm, 32 * quarter, 0);
    float acc[NC], pair[16], qk[16];
    // acc[j0 ..] += fac x over 16 columns of a product; returns the dot product with this row of q or k
    const uint32_t own = sm + L::oQK + ((cq * NC) >> 6) * 2 * kTile + (lower ? 0 : kTile);
    auto add16 = [&](float (&a)[NC], int j0, uint32_t col, float fac) {
      float x[16], dot = 0.f;
      tmem_ld16(col, x);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 v4 = lds128(own + tile_off<8>(i, (((cq * NC) & 63) + j0) / 8 + u));
        const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = unpack2(v[j]);
          const float x0 = x[8 * u + 2 * j], x1 = x[8 * u + 2 * j + 1];
          a[j0 + 8 * u + 2 * j] += fac * x0;
          a[j0 + 8 * u + 2 * j + 1] += fac * x1;
          dot += y.x * x0 + y.y * x1;
        }
      }
      return dot;
    };
    // the pairs (i, 16 cq + j): all of them, none, or those around the diagonal
    const bool none = !(quarter & 1) && cq >= 2, all = (quarter & 1) && cq < 2;
    const float sign = lower ? p.scale : -1.f;
    float qk_own = 0.f, pair_own = 0.f;
    {
      mbar_wait_flag(qk_full, 0, ok);
      mbar_wait_flag(qk_done, 0, ok);
      tc_fence_after();
      tmem_ld16(tlane + cq * 16, qk);
      tc_fence_before();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        qk[j] *= sign;
        qk_own = 16 * cq + j == i ? qk[j] : qk_own;
      }
      for (int x = tid; x < 2 * 4 * kC; x += kEpi) reinterpret_cast<float*>(raw + L::oCol)[x] = 0.f;
      // every warp has read q k^T before the first head's product takes its place
      bar_sync(1, kEpi);
      if (tid == 0) mbar_arrive(z_done);
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) pair[j] = 0.f;
    for (int hh = 0; hh < p.hpg; ++hh) {
      const int buf = hh & 1;
      const float* ga = reinterpret_cast<const float*>(raw + L::oGate + (hh & 3) * kGate);
      const int* sg = reinterpret_cast<const int*>(ga + kGateSeg * kC);
      float* colp = reinterpret_cast<float*>(raw + L::oCol) + buf * 4 * kC;
      float* rowp = reinterpret_cast<float*>(raw + L::oRow) + buf * 4 * 128;
      float* outp = reinterpret_cast<float*>(raw + L::oOut) + buf * 4 * kC;
      float* diag = reinterpret_cast<float*>(raw + L::oDiag) + buf * kC;
      if (hh >= 2) bar_sync(kBarFree + buf, kSums);  // head hh - 2's sums have been used
      mbar_wait_flag(g_full + (hh & 3), (hh >> 2) & 1, ok);
      const float ei = ga[i], be = ga[kGateBeta * kC + i], oi = ga[kGateO * kC + i];
      mbar_wait_flag(x_full + buf, (hh >> 1) & 1, ok);
      tc_fence_after();
      if (!lower) {  // w D1: dk_i += o_i beta_i D1 w_i
        float dot = 0.f;
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += 16) dot += add16(acc, j0, tlane + kX3 + cq * NC + j0, oi * be);
        outp[cq * kC + i] = oi * dot;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x3_free);
      // dY S0 or r S0: dq_i += scale e_i ..., dk_i -= e_i ...
      const float fac = lower ? p.scale * ei : -ei;
      float rsum = 0.f;
#pragma unroll
      for (int j0 = 0; j0 < NC; j0 += 16) rsum += add16(acc, j0, tlane + buf * kX + cq * NC + j0, fac);
      rsum *= fac;
      float x[16];
      if (!none) tmem_ld16(tlane + buf * kX + N + cq * 16, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_free + buf);
      if (all) {
        // below the diagonal the decay is that from token 32 times that to it
        const float ri = ga[kGateHalf * kC + i];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j0 = 16 * cq + 4 * u;
          const float4 c4 = *reinterpret_cast<const float4*>(ga + kGateHalf * kC + j0);
          const float4 b4 = *reinterpret_cast<const float4*>(ga + kGateBeta * kC + j0);
          const float cj[4] = {c4.x, c4.y, c4.z, c4.w}, bj[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int j = 4 * u + v;
            const float z = x[j] * ri * cj[v];
            pair[j] += bj[v] * z;
            x[j] = z * qk[j];
            rsum += bj[v] * x[j];
          }
        }
      } else if (!none) {
        const float gi = ga[kGateGam * kC + i];
        const int si = sg[i];
        if (lower) {  // a token's own pair: it does not depend on the decays
          float own_x = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) own_x = 16 * cq + j == i ? x[j] : own_x;
          pair_own += be * own_x;
          if ((i >> 4) == cq) diag[i] = own_x * qk_own;
        }
        // (no branches: each pair's chain of loads and exponential has its latency, and sixteen overlap)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j0 = 16 * cq + 4 * u;
          const float4 g4 = *reinterpret_cast<const float4*>(ga + kGateGam * kC + j0);
          const float4 b4 = *reinterpret_cast<const float4*>(ga + kGateBeta * kC + j0);
          const int4 s4 = *reinterpret_cast<const int4*>(sg + j0);
          const float gj[4] = {g4.x, g4.y, g4.z, g4.w}, bj[4] = {b4.x, b4.y, b4.z, b4.w};
          const int sj[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int j = 4 * u + v;
            const float Ex = exp2_fast(gi - gj[v]) * x[j];
            const float z = (j0 + v < i) & (sj[v] == si) ? Ex : 0.f;
            pair[j] += bj[v] * z;
            x[j] = z * qk[j];
            rsum += bj[v] * x[j];
          }
        }
      }
      rowp[cq * 128 + row] = rsum;
      if (!none) {
        const float cs = sum16(x, lane);
        if ((lane & 1) == 0) colp[quarter * kC + 16 * cq + (lane >> 1)] = cs;
      }
      __syncwarp();
      bar_arrive(kBarSums + buf, kSums);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) pair[j] = sign * (lower && 16 * cq + j == i ? pair_own : pair[j]);
    // The pairs' part for all heads: rows of [0 | Z ; Z^T | M + M^T] against
    // [q ; k], Z (i, j) and M (i, j) summed over the heads.  All of the ring's
    // products are done: the last head's x_full followed them.
    bar_sync(1, kEpi);
    const uint32_t Zb = sm + L::oSt;  // 128 rows x 64 columns of q's tokens, then of k's
    if (lower) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(Zb + tile_off<8>(i, 2 * cq + u)), "r"(0), "r"(0),
                     "r"(0), "r"(0)
                     : "memory");
#pragma unroll
      for (int u = 0; u < 2; ++u)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(Zb + 2 * kTile + tile_off<8>(i, 2 * cq + u)),
                     "r"(pack2(pair[8 * u], pair[8 * u + 1])), "r"(pack2(pair[8 * u + 2], pair[8 * u + 3])),
                     "r"(pack2(pair[8 * u + 4], pair[8 * u + 5])), "r"(pack2(pair[8 * u + 6], pair[8 * u + 7]))
                     : "memory");
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int jj = 16 * cq + j;
      const __nv_bfloat16 v = __float2bfloat16_rn(pair[j]);
      const uint16_t b = *reinterpret_cast<const uint16_t*>(&v);
      if (lower) {  // Z^T below the zeros
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(Zb + elem_off<8>(64 + jj, i)), "h"(b) : "memory");
      } else if (jj <= i) {  // M is zero on its diagonal
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(Zb + 2 * kTile + elem_off<8>(64 + i, jj)), "h"(b) : "memory");
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(Zb + 2 * kTile + elem_off<8>(64 + jj, i)), "h"(b) : "memory");
      }
    }
    fence_async_smem();
    bar_sync(1, kEpi);
    if (tid == 0) mbar_arrive(qk_full);
    mbar_wait_flag(qk_done, 1, ok);
    tc_fence_after();
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(lower ? f.dq : f.dk) + ((tok0 + i) * p.G + grp) * N + cq * NC;
#pragma unroll
    for (int j0 = 0; j0 < NC; j0 += 16) {
      float x[16];
      tmem_ld16(tlane + cq * NC + j0, x);
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = pack2(acc[j0 + 2 * j] + x[2 * j], acc[j0 + 2 * j + 1] + x[2 * j + 1]);
      if (i < n) {
        reinterpret_cast<uint4*>(dst + j0)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(dst + j0)[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
  if (!ok) atomicOr(f.status, kDevTimeout);
  tc_fence_before();
  __syncthreads();
  if (w == kWarps) tmem_dealloc(tm, kCols);
}

template <int N>
cudaError_t launch_t(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  const uint64_t P = p.P, H = p.H, G = p.G, Ln = p.L, b = p.b, nc = p.nc, e = 2;
  GradMaps m = {};
  auto tokens = [&](CUtensorMap* t, const void* base, uint64_t width, uint64_t heads, uint64_t stride) {
    const uint64_t d[4] = {width, heads, Ln, b}, st[3] = {width * e, stride * e, Ln * stride * e};
    const uint32_t box[4] = {64, 1, (uint32_t)kC, 1};
    return encode_tmap_bf16_4d(t, base, d, st, box, 128);
  };
  auto chunks = [&](CUtensorMap* t, const void* base, uint64_t width) {
    const uint64_t d[4] = {width, P, nc, b * H}, st[3] = {width * e, P * width * e, nc * P * width * e};
    const uint32_t box[4] = {64, 64, 1, 1};
    return encode_tmap_bf16_4d(t, base, d, st, box, 128);
  };
  if (!tokens(&m.q, f.q, N, G, p.qs) || !tokens(&m.k, f.k, N, G, p.ks) || !tokens(&m.dy, f.dy, P, H, H * P) ||
      !tokens(&m.dv, f.dv, P, H, H * P) || !chunks(&m.S, f.S, N) || !chunks(&m.D, f.D, N) || !chunks(&m.w, f.w, 64))
    return cudaErrorInvalidValue;
  auto kern = delta_grad_tc_kernel<N>;
  constexpr int smem = GradSmem<N>::bytes;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  set_kernel_name("delta_grad_tc");
  kern<<<(unsigned)((long long)p.nc * p.G * p.b), kThreads, smem, s>>>(p, f, m);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grad_tc(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return p.N == 128 ? launch_t<128>(p, f, s) : launch_t<64>(p, f, s);
}

}  // namespace ssd
