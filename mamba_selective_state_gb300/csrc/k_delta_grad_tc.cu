// k_delta_grad_tc.cu -- dq, dk, dg and dbeta of the gated delta rule on the
// tensor cores, chunk by chunk: the formulas at the head of
// k_delta_grad_simt.cu, with bf16 S0, D1, w and r = dv from the chains (operands of
// bf16 products, and half the bytes of what is saved; so is the pairs' part summed
// over the heads, Z and M, before its product with k and q).
//
// One CTA takes a chunk of a group and walks its heads.  Per head, with the
// tokens of dY and of r as the 128 rows of one left operand,
//
//   [dY ; r] [S0 | w']  ->  dY S0, r S0 (64 x dstate) and dY w', r w' (64 x 64)
//   [w ; w]  D1         ->  w D1, twice: each half of the warps takes half its columns
//
// come from tcgen05 products into tensor memory (S0, D1 and w' are stored with
// headdim as rows, as the chains write them, and enter as MN-major operands).
// Sixteen warps read them back: a thread owns one token's row -- of dY and dq
// in the lower 64 lanes, of r and dk in the upper -- and a quarter of the
// columns, so the dot products with q and k and the sums over heads stay in
// its registers (as pairs, for the two-value fp32 multiply-add).  q k^T and
// k k^T do not depend on the head, and the pairs' part of dq and dk is summed
// over the heads before its products with k and q: both are one more product
// of 128 rows per group.  The pairs' contributions to dgam are formed once in
// fp32 and summed by rows and by columns, so that what cancels in their running
// difference cancels exactly.
//
// Measured: 363 us at batch 2, L = 8192, 64 heads in 8 groups, headdim 64 and
// dstate 128, where it reads 0.95 GB (2.7 TB/s).  The sixteen warps' epilogue
// bounds it: of 60,000 cycles for eight heads it takes 40,000, the first loads
// 7,500, and waiting for products 9,200.  A third stage of the ring, prefetches
// into L2 and a kernel that also accumulates dq and dk in tensor memory (from
// left operands that are scaled and written back) did not shorten it: 359 to
// 394 us.  Nor did evening out the warps' work, with w D1 only for those of the
// earlier tokens, which have few pairs (399 us): a warp's own chain of reads
// counts, not the number of instructions.
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
constexpr int kThreads = kEpi + 128;          // and a warp of copies and products, two of sums, one of
                                              // <S0, D1>; registers are handed over by groups of four warps
// Registers a thread: 640 threads are launched with 96; the other warps keep
// 64 and the epilogue warps take 104 (4 x 104 + 64 = 5 x 96).  Where the
// epilogue spills, it waits: the ring leaves the L1 cache too small for that.
constexpr int kRegsEpi = 104, kRegsCtl = 64;
constexpr int kPairThreads = 12 * 32;         // of the warps that have pairs at all
constexpr uint32_t kTile = 8192;              // [64][64] bf16, 128-byte swizzle
constexpr int kGate = kGateRows * kC * 4;

struct GradMaps {
  CUtensorMap q, k, S, D, w, dv, dy;
};

template <int N>
struct GradSmem {
  static constexpr int NB = N / 64;
  // per head and 64 columns of headdim: dY, r, S0, w, w, D1
  static constexpr int stage = (2 + 2 * NB + 2) * (int)kTile;
  static constexpr int kStages = N == 128 ? 2 : 3;
  // q and k: for each 64 columns of dstate the tile of q above that of k
  static constexpr int oQK = 0, oSt = NB * 2 * (int)kTile, oGate = oSt + kStages * stage,  // four gate records
                       oCol = oGate + 4 * kGate,       // [2][4][64] column sums by lane quarter
                       oRow = oCol + 2 * 4 * kC * 4,   // [2][4][128] row sums by column quarter
                       oOut = oRow + 2 * 4 * 128 * 4,  // [2][8][64] k.(D1 w) by columns
                       oDiag = oOut + 2 * 8 * kC * 4, oRed = oDiag + 2 * kC * 4,
                       oPair = oRed + 16,                    // q k^T or k k^T by pair of columns and thread
                       oHalf = oPair + 8 * kPairThreads * 8, // the lower lanes' half of w D1, likewise
                       oBar = oHalf + N / 16 * (kEpi / 2) * 8,
                       bytes = oBar + 256 + 1024;
  static_assert(kStages * stage >= 4 * (int)kTile, "the pairs' operand reuses the ring");
};

// Two fp32 values in one register pair
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) { return fma2(b, pair2(-1.f, -1.f), a); }

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
           *x_free = bars + 18, *x3_free = bars + 20, *qk_full = bars + 21, *qk_done = bars + 22, *z_done = bars + 23,
           *sums = bars + 24, *used = bars + 26;  // a head's sums are written, and have been used
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(bars + 28);
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
      mbar_init(sums + i, kWarps + 1);
      mbar_init(used + i, 1);
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
        for (int j = 0; j < 2; ++j) tma_load_4d(d + (2 + NB + j) * kTile, &m.w, s_full + st, 0, 64 * pc, c, bh);
        for (int j = 0; j < NB; ++j) tma_load_4d(d + (4 + NB + j) * kTile, &m.D, s_full + st, 64 * j, 64 * pc, c, bh);
      };
      mbar_expect_tx(qk_full, NB * 2 * kTile);
      for (int j = 0; j < NB; ++j) {
        tma_load_4d(raw + L::oQK + 2 * j * kTile, &m.q, qk_full, 64 * j, grp, t0, bi);
        tma_load_4d(raw + L::oQK + (2 * j + 1) * kTile, &m.k, qk_full, 64 * j, grp, t0, bi);
      }
      int loaded = 0;
      for (; loaded < L::kStages && loaded < steps; ++loaded) load(loaded);
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
        // the stage of the step before: its products and <S0, D1> were taken during the last head's epilogue
        if (s >= 1 && loaded < steps) load(loaded++);
        mbar_wait_flag(s_full + st, use & 1, ok);
        if (pc == 0) {
          // the buffer's last head has been read (the first head's: q k^T)
          if (hh >= 2) mbar_wait_flag(x_free + buf, ((hh >> 1) - 1) & 1, ok);
          if (hh == 0) mbar_wait_flag(z_done, 0, ok);
        }
        tc_fence_after();
        const uint32_t base = sm + L::oSt + st * L::stage, S0 = base + 2 * kTile, D1 = base + (4 + NB) * kTile;
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16(tm + buf * kX, smem_desc(base + ks * 32, 16, 1024, kSwz128),
                   smem_desc(S0 + ks * 2048, kTile, 1024, kSwz128), idesc_bf16(128, N + 64, 0, 1), pc > 0 || ks > 0);
        if (pc == 0 && hh >= 1) {
          mbar_wait_flag(x3_free, (hh - 1) & 1, ok);
          tc_fence_after();
        }
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16(tm + kX3, smem_desc(S0 + NB * kTile + ks * 2048, kTile, 1024, kSwz128),
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
        const float* outp = reinterpret_cast<const float*>(raw + L::oOut) + buf * 8 * kC;
        const float* diag = reinterpret_cast<const float*>(raw + L::oDiag) + buf * kC;
        mbar_wait_flag(g_full + (hh & 3), (hh >> 2) & 1, ok);
        mbar_wait_flag(sums + buf, (hh >> 1) & 1, ok);
        // this head's dbeta, and dg as the reverse cumulative sum of dgam
        float d[2], all = 0.f;
        const float sdot = reinterpret_cast<const float*>(raw + L::oRed)[buf];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int a = 2 * lane + j;
          float o = 0.f;
#pragma unroll
          for (int x2 = 0; x2 < 8; ++x2) o += outp[x2 * kC + a];
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
        if (lane == 0) {
          mbar_arrive(g_free + (hh & 3));
          mbar_arrive(used + buf);
        }
      }
    } else if (w == kWarps + 3) {
      // <S0, D1> of every head: the diagonal of 16 x 8 products
      const int g = lane >> 2, t = lane & 3;
      for (int hh = 0; hh < p.hpg; ++hh) {
        float sd = 0.f;
        for (int pc = 0; pc < npc; ++pc) {
          const int s = hh * npc + pc, st = s % L::kStages;
          mbar_wait_flag(s_full + st, (s / L::kStages) & 1, ok);
          const uint32_t S0 = sm + L::oSt + st * L::stage + 2 * kTile, D1 = S0 + (NB + 2) * kTile;
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
        if (hh >= 2) mbar_wait_flag(used + (hh & 1), ((hh >> 1) - 1) & 1, ok);
        if (lane == 0) {
          reinterpret_cast<float*>(raw + L::oRed)[hh & 1] = sd;
          mbar_arrive(sums + (hh & 1));
        }
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int quarter = w & 3, cq = w >> 2;          // tensor-memory lanes, columns
    const int row = 32 * quarter + lane, i = row & 63;
    const bool lower = quarter < 2;                  // dY, dq, q k^T; else r, w, dk, k k^T
    const uint32_t tlane = tmem_addr(tm, 32 * quarter, 0);
    // sums over heads: this row of dq or dk, the pairs, and in shared memory (registers are short) the lower lanes'
    // half of w D1
    f2 acc[NC / 2], pair[8];
    f2* acc3 = reinterpret_cast<f2*>(raw + L::oHalf) + (cq * 64 + row);  // [NC / 4][256], the lower lanes' only
    // this thread's 16 products of q or k and k, scaled
    f2* qk = reinterpret_cast<f2*>(raw + L::oPair) + ((cq < 2 ? w : 8 + 2 * (cq - 2) + (quarter >> 1)) * 32 + lane);
    // Column pairs c0.. of a product: a[] += fac x; returns the dot product with the row of q or k at `own`
    const uint32_t own_k = sm + L::oQK + ((cq * NC) >> 6) * 2 * kTile + kTile, own = lower ? own_k - kTile : own_k;
    auto add8 = [&](f2* a, const float* x, uint32_t row_at, int col, f2 fac, f2 dot) {
      const uint4 v4 = lds128(row_at + tile_off<8>(i, (((cq * NC) & 63) + col) / 8));
      const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 x2 = pair2(x[2 * j], x[2 * j + 1]);
        a[j] = fma2(fac, x2, a[j]);
        dot = fma2(pair2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xffff0000u)), x2, dot);
      }
      return dot;
    };
    const f2 zero2 = pair2(0.f, 0.f);
    // the pairs (i, 16 cq + j): all of them, none, or those around the diagonal
    const bool none = !(quarter & 1) && cq >= 2, all = (quarter & 1) && cq < 2;
    const float sign = lower ? p.scale : -1.f;
    float qk_own = 0.f, pair_own = 0.f;
    {
      mbar_wait_flag(qk_full, 0, ok);
      mbar_wait_flag(qk_done, 0, ok);
      tc_fence_after();
      float q16[16];
      tmem_ld16(tlane + cq * 16, q16);
      tc_fence_before();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        q16[j] *= sign;
        qk_own = 16 * cq + j == i ? q16[j] : qk_own;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!none) qk[j * kPairThreads] = pair2(q16[2 * j], q16[2 * j + 1]);
      for (int x = tid; x < 2 * 4 * kC; x += kEpi) reinterpret_cast<float*>(raw + L::oCol)[x] = 0.f;
      // every warp has read q k^T before the first head's product takes its place
      bar_sync(1, kEpi);
      if (tid == 0) mbar_arrive(z_done);
    }
#pragma unroll
    for (int j = 0; j < NC / 2; ++j) acc[j] = zero2;
#pragma unroll
    for (int j = 0; j < NC / 4; ++j)
      if (lower) acc3[j * (kEpi / 2)] = zero2;
#pragma unroll
    for (int j = 0; j < 8; ++j) pair[j] = zero2;
    for (int hh = 0; hh < p.hpg; ++hh) {
      const int buf = hh & 1;
      const float* ga = reinterpret_cast<const float*>(raw + L::oGate + (hh & 3) * kGate);
      const int* sg = reinterpret_cast<const int*>(ga + kGateSeg * kC);
      float* colp = reinterpret_cast<float*>(raw + L::oCol) + buf * 4 * kC;
      float* rowp = reinterpret_cast<float*>(raw + L::oRow) + buf * 4 * 128;
      float* outp = reinterpret_cast<float*>(raw + L::oOut) + buf * 8 * kC;
      float* diag = reinterpret_cast<float*>(raw + L::oDiag) + buf * kC;
      if (hh >= 2) mbar_wait_flag(used + buf, ((hh >> 1) - 1) & 1, ok);  // head hh - 2's sums
      mbar_wait_flag(g_full + (hh & 3), (hh >> 2) & 1, ok);
      const float ei = ga[i], be = ga[kGateBeta * kC + i], oi = ga[kGateO * kC + i];
      mbar_wait_flag(x_full + buf, (hh >> 1) & 1, ok);
      tc_fence_after();
      {  // w D1: dk_i += o_i beta_i D1 w_i, the lower lanes the first half of this quarter's columns
        constexpr int H3 = NC / 2;
        float x3[16];
        tmem_ld16(tlane + kX3 + cq * NC + (NC == 32 && !lower ? 16 : 0), x3);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(x3_free);
        const f2 fac = pair2(oi * be, oi * be);
        f2 dot = zero2;
#pragma unroll
        for (int u = 0; u < H3 / 8; ++u) {
          if (lower) {
            f2 t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = acc3[(4 * u + j) * (kEpi / 2)];
            dot = add8(t, x3 + 8 * u, own_k, 8 * u, fac, dot);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc3[(4 * u + j) * (kEpi / 2)] = t[j];
          } else
            dot = add8(acc + H3 / 2 + 4 * u, x3 + (NC == 32 ? 0 : H3) + 8 * u, own_k, H3 + 8 * u, fac, dot);
        }
        const float2 d = both2(dot);
        outp[((lower ? 0 : 4) + cq) * kC + i] = oi * (d.x + d.y);
      }
      // dY S0 or r S0: dq_i += scale e_i ..., dk_i -= e_i ...
      const float fac1 = lower ? p.scale * ei : -ei;
      f2 rsum2 = zero2;
#pragma unroll
      for (int j0 = 0; j0 < NC; j0 += 16) {
        float x[16];
        tmem_ld16(tlane + buf * kX + cq * NC + j0, x);
        const f2 fac = pair2(fac1, fac1);
#pragma unroll
        for (int u = 0; u < 2; ++u) rsum2 = add8(acc + j0 / 2 + 4 * u, x + 8 * u, own, j0 + 8 * u, fac, rsum2);
      }
      rsum2 = mul2(rsum2, pair2(fac1, fac1));
      float x[16];
      if (!none) tmem_ld16(tlane + buf * kX + N + cq * 16, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_free + buf);
      if (all) {
        // below the diagonal the decay is that from token 32 times that to it
        const float ri = ga[kGateHalf * kC + i];
        const f2 ri2 = pair2(ri, ri);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(ga + kGateHalf * kC + 16 * cq + 4 * u);
          const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(ga + kGateBeta * kC + 16 * cq + 4 * u);
          const f2 cj[2] = {c4.x, c4.y}, bj[2] = {b4.x, b4.y};
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int j = 2 * u + v;
            const f2 z = mul2(pair2(x[2 * j], x[2 * j + 1]), mul2(ri2, cj[v]));
            pair[j] = fma2(bj[v], z, pair[j]);
            const f2 both = mul2(z, qk[j * kPairThreads]);
            rsum2 = fma2(bj[v], both, rsum2);
            const float2 bb = both2(both);
            x[2 * j] = bb.x;
            x[2 * j + 1] = bb.y;
          }
        }
      } else if (!none) {
        const float gi = ga[kGateGam * kC + i];
        const int si = sg[i];
        const f2 gi2 = pair2(gi, gi);
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
          const ulonglong2 g4 = *reinterpret_cast<const ulonglong2*>(ga + kGateGam * kC + j0);
          const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(ga + kGateBeta * kC + j0);
          const int4 s4 = *reinterpret_cast<const int4*>(sg + j0);
          const f2 gj[2] = {g4.x, g4.y}, bj[2] = {b4.x, b4.y};
          const int sj[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int j = 2 * u + v, jj = j0 + 2 * v;
            const float2 a = both2(sub2(gi2, gj[v]));
            const float z0 = exp2_fast(a.x) * x[2 * j], z1 = exp2_fast(a.y) * x[2 * j + 1];
            const f2 z = pair2((jj < i) & (sj[2 * v] == si) ? z0 : 0.f, (jj + 1 < i) & (sj[2 * v + 1] == si) ? z1 : 0.f);
            pair[j] = fma2(bj[v], z, pair[j]);
            const f2 both = mul2(z, qk[j * kPairThreads]);
            rsum2 = fma2(bj[v], both, rsum2);
            const float2 bb = both2(both);
            x[2 * j] = bb.x;
            x[2 * j + 1] = bb.y;
          }
        }
      }
      const float2 rs = both2(rsum2);
      rowp[cq * 128 + row] = rs.x + rs.y;
      if (!none) {
        const float cs = sum16(x, lane);
        if ((lane & 1) == 0) colp[quarter * kC + 16 * cq + (lane >> 1)] = cs;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sums + buf);
    }
    float z16[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = both2(pair[j]);
      z16[2 * j] = sign * (lower && 16 * cq + 2 * j == i ? pair_own : v.x);
      z16[2 * j + 1] = sign * (lower && 16 * cq + 2 * j + 1 == i ? pair_own : v.y);
    }
    // The pairs' part for all heads: rows of [0 | Z ; Z^T | M + M^T] against
    // [q ; k], Z (i, j) and M (i, j) summed over the heads.  Their operand takes
    // the ring's place once the products and the warp of <S0, D1> have left it.
    const int steps = p.hpg * npc;
    for (int s = steps > L::kStages ? steps - L::kStages : 0; s < steps; ++s)
      mbar_wait_flag(s_free + s % L::kStages, (s / L::kStages) & 1, ok);
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
                     "r"(pack2(z16[8 * u], z16[8 * u + 1])), "r"(pack2(z16[8 * u + 2], z16[8 * u + 3])),
                     "r"(pack2(z16[8 * u + 4], z16[8 * u + 5])), "r"(pack2(z16[8 * u + 6], z16[8 * u + 7]))
                     : "memory");
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int jj = 16 * cq + j;
      const __nv_bfloat16 v = __float2bfloat16_rn(z16[j]);
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
      for (int j = 0; j < 8; ++j) {
        const float2 v = both2(acc[j0 / 2 + j]);
        const int col = j0 + 2 * j;
        // (the lower lanes' half of w D1 belongs to the same token's row of dk)
        const float2 more = !lower && col < NC / 2 ? both2(acc3[col / 2 * (kEpi / 2) - 64]) : make_float2(0.f, 0.f);
        o[j] = pack2(v.x + x[2 * j] + more.x, v.y + x[2 * j + 1] + more.y);
      }
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
