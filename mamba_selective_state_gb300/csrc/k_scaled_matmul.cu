// k_scaled_matmul.cu -- the product of 8-bit codes (int8 or e4m3) with a scale
// for each token and for each channel, and its C ABI.
//
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n]
//
// This chip's integer tensor rate is a small part of its fp16 rate, so int8
// codes are multiplied as fp16, which holds them and their products' factors
// exactly; sums are fp32.  e4m3 codes go to the tensor cores as they are.
//
// Few tokens (m <= 64): bound by the weights' bytes.  Warps read 16 channels'
// codes in 16-byte pieces, turn them into fp16 in registers and multiply them
// with the tokens' by warp-level products; the order of k inside a product is
// free, so a lane's 16 neighbouring codes serve four products as they lie.
//
// More tokens: tensor-memory products of 256 x 256 outputs by pairs of CTAs,
// persistent, fed by TMA through a ring of stages, the epilogue of one tile
// under the products of the next.  int8 codes are first written out as fp16.
#include <cuda_fp16.h>
#include <string.h>

#include "codes.cuh"
#include "ssd_internal.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace ssd {

int device_check();

namespace {

constexpr int kFewTokens = 64;

struct MatmulArgs {
  const uint8_t *a, *w;
  const float *as, *ws, *bias;
  void* out;
  int* status;
  long long m, n, k;  // k: codes in a row as the kernel reads it
};

// ---- codes to fp16 ----------------------------------------------------------
// Four int8: as 0x6400 | (x + 128) they are 1024 + (x + 128), from which 1152 is taken
__device__ __forceinline__ void int8_to_half(uint32_t x, uint32_t& lo, uint32_t& hi) {
  x ^= 0x80808080u;
  const uint32_t k = 0x64646464u, off = 0x64806480u;
  lo = __byte_perm(x, k, 0x4140);
  hi = __byte_perm(x, k, 0x4342);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(off));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(off));
}
__device__ __forceinline__ void e4m3_to_half(uint32_t x, uint32_t& lo, uint32_t& hi) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3),
                    b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3);
  lo = (uint32_t)a.x | (uint32_t)a.y << 16;
  hi = (uint32_t)b.x | (uint32_t)b.y << 16;
}
template <bool kFp8>
__device__ __forceinline__ void to_half(const uint4& u, uint32_t (&h)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kFp8) e4m3_to_half(w[i], h[2 * i], h[2 * i + 1]);
    else int8_to_half(w[i], h[2 * i], h[2 * i + 1]);
  }
}

// ---- rows written out with a whole number of vectors -----------------------
// as fp16 (kHalf) or as they are, zeros behind the k-th code
struct PackArgs {
  const uint8_t *src[2];
  uint8_t* dst[2];
  long long groups[2];  // 16-code groups in all
  long long bytes[2];   // of the source
  int k, per_row;       // groups to a row
  int* status;
};

// 16 codes from any address: words where they are whole, else bytes
__device__ __forceinline__ uint4 load16(const uint8_t* base, long long at, int count, long long bytes) {
  if (count == 16 && (at & 15) == 0) return *reinterpret_cast<const uint4*>(base + at);
  uint32_t w[5];
  const long long a0 = at & ~3LL;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const long long p = a0 + 4 * i;
    w[i] = 0;
    if (p >= at + count) continue;
    if (p + 4 <= bytes) {
      w[i] = *reinterpret_cast<const uint32_t*>(base + p);
    } else {
      for (int j = 0; j < 4 && p + j < bytes; ++j) w[i] |= (uint32_t)base[p + j] << (8 * j);
    }
  }
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = __funnelshift_r(w[i], w[i + 1], (unsigned)(at & 3) * 8);
    const int left = count - 4 * i;  // codes of this word
    if (left < 4) r[i] = left <= 0 ? 0u : r[i] & ((1u << (8 * left)) - 1u);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool kHalf>
__global__ void __launch_bounds__(256) pack_rows_kernel(PackArgs p) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const long long total = p.groups[0] + p.groups[1];
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int which = i >= p.groups[0];
    const long long g = which ? i - p.groups[0] : i;
    const long long row = g / p.per_row;
    const int c = (int)(g - row * p.per_row) * 16, count = min(max(p.k - c, 0), 16);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (count) u = load16(p.src[which], row * p.k + c, count, p.bytes[which]);
    uint4* to = reinterpret_cast<uint4*>(p.dst[which]);
    if constexpr (kHalf) {
      uint32_t h[8];
      to_half<false>(u, h);
      to[2 * g] = make_uint4(h[0], h[1], h[2], h[3]);
      to[2 * g + 1] = make_uint4(h[4], h[5], h[6], h[7]);
    } else {
      to[g] = u;
    }
  }
}

// ---- few tokens -------------------------------------------------------------
__device__ __forceinline__ void mma_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kSkWarps = 8;

// CT: tiles of 16 channels to a CTA; MT: groups of 8 tokens.  The warps split k,
// 64 codes at a time; k is a multiple of 16.
template <bool kFp8, typename O, int CT, int MT>
__global__ void __launch_bounds__(kSkWarps * 32) skinny_kernel(MatmulArgs p) {
  constexpr int kCh = CT * 16, kTok = MT * 8, kPitch = kCh + 1;
  extern __shared__ float part[];  // [warp][token][channel]
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const long long n0 = (long long)blockIdx.x * kCh;
  const uint8_t* wrow[CT][2];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (rows past the last channel are read from it and not written)
      long long r = n0 + c * 16 + h * 8 + g;
      r = r < p.n ? r : p.n - 1;
      wrow[c][h] = p.w + r * p.k + q * 16;
    }
  float acc[CT][MT][4] = {};
  constexpr int kAhead = CT * MT >= 8 ? 2 : 4;
  const int k = (int)p.k;
  for (int k0 = warp * 64; k0 < k; k0 += kSkWarps * 64 * kAhead) {
    uint4 w[kAhead][CT][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int kk = k0 + u * kSkWarps * 64;
      const bool in = kk + q * 16 < k;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[u][c][h] = in ? __ldcs(reinterpret_cast<const uint4*>(wrow[c][h] + kk)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int kk = k0 + u * kSkWarps * 64;
      const bool in = kk + q * 16 < k;
      uint32_t wh[CT][2][8];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        to_half<kFp8>(w[u][c][0], wh[c][0]);
        to_half<kFp8>(w[u][c][1], wh[c][1]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int tok = t * 8 + g;
        uint4 a = make_uint4(0, 0, 0, 0);
        if (in && tok < p.m) a = __ldg(reinterpret_cast<const uint4*>(p.a + tok * p.k + kk + q * 16));
        uint32_t ah[8];
        to_half<kFp8>(a, ah);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            mma_half(acc[c][t], wh[c][0][2 * j], wh[c][1][2 * j], wh[c][0][2 * j + 1], wh[c][1][2 * j + 1], ah[2 * j],
                     ah[2 * j + 1]);
      }
    }
  }
  float* mine = part + warp * kTok * kPitch;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(t * 8 + 2 * q + (i & 1)) * kPitch + c * 16 + (i >> 1) * 8 + g] = acc[c][t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kCh * kTok; i += kSkWarps * 32) {
    const int tok = i / kCh, ch = i % kCh;
    const long long n = n0 + ch;
    if (tok >= p.m || n >= p.n) continue;
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < kSkWarps; ++x) s += part[(x * kTok + tok) * kPitch + ch];
    s = s * p.as[tok] * p.ws[n];
    static_cast<O*>(p.out)[tok * p.n + n] = from_f<O>(p.bias ? s + p.bias[n] : s);
  }
}

template <bool kFp8, typename O, int CT, int MT>
cudaError_t launch_skinny_t(const MatmulArgs& p, cudaStream_t s) {
  constexpr int smem = kSkWarps * MT * 8 * (CT * 16 + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(skinny_kernel<kFp8, O, CT, MT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  set_kernel_name("scaled_matmul_few");
  skinny_kernel<kFp8, O, CT, MT><<<(unsigned)((p.n + CT * 16 - 1) / (CT * 16)), kSkWarps * 32, smem, s>>>(p);
  return cudaGetLastError();
}
template <bool kFp8, typename O>
cudaError_t launch_skinny(const MatmulArgs& p, cudaStream_t s) {
  if (p.m <= 8) return launch_skinny_t<kFp8, O, 1, 1>(p, s);
  if (p.m <= 16) return launch_skinny_t<kFp8, O, 1, 2>(p, s);
  if (p.m <= 32) return launch_skinny_t<kFp8, O, 2, 4>(p, s);
  return launch_skinny_t<kFp8, O, 2, 8>(p, s);
}

// ---- many tokens: tensor-memory products by pairs of CTAs -------------------
//
// A pair computes 256 tokens x BN channels: each CTA holds 128 tokens' rows and
// half of the channels' rows of every stage (128 bytes of k: 64 fp16 or 128
// e4m3), and 128 rows of the result in its own tensor memory, twice.  The
// leader (even rank) issues the products for both; its `full` barriers take the
// bytes of both CTAs' copies.  Commits arrive in both CTAs.
constexpr int kStages = 6;
constexpr int kRowsA = 128;
constexpr int kTcThreads = 192;  // warp 0 copies, warp 1 products, warps 2-5 epilogue

template <int BN>
struct TcSmem {
  static constexpr int kA = kRowsA * 128, kB = BN / 2 * 128;
  static constexpr int kStageBytes = kA + kB;
  static constexpr int kBytes = kStages * kStageBytes + 1024 + 256;
};

__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A box into this CTA's shared memory, its bytes counted by a barrier of the pair
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
template <bool kFp8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs once this thread's products are done
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The tile-th pair of (token, channel) tiles: bands of 8 token tiles, channel by
// channel, so that a wave of pairs reads few rows of either operand.
__device__ __forceinline__ void tile_of(long long tile, int mt, int nt, int& tm, int& tn) {
  constexpr int kBand = 8;
  const long long per = (long long)kBand * nt;
  const int band = (int)(tile / per), rows = min(kBand, mt - band * kBand);
  const int in = (int)(tile - band * per);
  tm = band * kBand + in % rows;
  tn = in / rows;
}

struct TcArgs {
  const float *as, *ws, *bias;
  void* out;
  int* status;
  long long m, n;
  int mt, nt, kb;  // tiles of tokens and channels; 128-byte blocks of k
};

template <bool kFp8, typename O, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads)
    pair_matmul_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap, TcArgs p) {
  using S = TcSmem<BN>;
  extern __shared__ uint8_t raw[];
  const uint32_t smem = (tc::smem_u32(raw) + 1023u) & ~1023u;
  __shared__ uint64_t full[kStages], empty[kStages], done[2], drained[2];
  __shared__ uint32_t tmem_s;
  const uint32_t rank = cta_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&done[i], 1);
      tc::mbar_init(&drained[i], 8);  // four epilogue warps of both CTAs
    }
    tc::mbar_fence_init();
  }
  constexpr uint32_t kCols = BN * 2 < 32 ? 32 : BN * 2;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&tmem_s)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_s;
  const long long tiles = (long long)p.mt * p.nt, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      tc::prefetch_tmap(&amap);
      tc::prefetch_tmap(&wmap);
      int st = 0;
      uint32_t ph = 0;
      for (long long t = pair; t < tiles; t += pairs) {
        int tm, tn;
        tile_of(t, p.mt, p.nt, tm, tn);
        const int ya = tm * 256 + (int)rank * 128, yw = tn * BN + (int)rank * (BN / 2);
        for (int b = 0; b < p.kb; ++b) {
          tc::mbar_wait_flag(&empty[st], ph ^ 1, ok);
          if (rank == 0) tc::mbar_expect_tx(&full[st], 2 * S::kStageBytes);
          const uint32_t bar = at_rank(tc::smem_u32(&full[st]), 0), to = smem + st * S::kStageBytes;
          pair_load(to, &amap, bar, b * 128, ya);
          pair_load(to + S::kA, &wmap, bar, b * 128, yw);
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // M = 256, N = BN, fp32 sums of fp16 (kind::f16) or e4m3 (kind::f8f6f4): both formats are number 0
      constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | (16u << 24);
      int st = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (long long t = pair; t < tiles; t += pairs) {
        tc::mbar_wait_flag(&drained[acc], aph ^ 1, ok);
        tc::tc_fence_after();
        for (int b = 0; b < p.kb; ++b) {
          tc::mbar_wait_flag(&full[st], ph, ok);
          tc::tc_fence_after();
          const uint32_t a = smem + st * S::kStageBytes, w = a + S::kA;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            pair_mma<kFp8>(tmem + acc * BN, tc::smem_desc(a + j * 32, 16, 1024, tc::kSwz128),
                           tc::smem_desc(w + j * 32, 16, 1024, tc::kSwz128), idesc, b | j);
          pair_commit(tc::smem_u32(&empty[st]));
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
        pair_commit(tc::smem_u32(&done[acc]));
        acc ^= 1;
        if (acc == 0) aph ^= 1;
      }
    }
  } else {
    const int quarter = warp & 3;  // the lanes of tensor memory that this warp may read
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const bool vec = p.n % (16 / (int)sizeof(O)) == 0;
    int acc = 0;
    uint32_t aph = 0;
    for (long long t = pair; t < tiles; t += pairs) {
      int tm, tn;
      tile_of(t, p.mt, p.nt, tm, tn);
      const long long row = (long long)tm * 256 + rank * 128 + quarter * 32 + lane, n0 = (long long)tn * BN;
      const bool in = row < p.m;
      const float as = in ? __ldg(p.as + row) : 0.f;
      O* out = static_cast<O*>(p.out) + row * p.n + n0;
      tc::mbar_wait_flag(&done[acc], aph, ok);
      tc::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BN && n0 + c < p.n; c += 32) {
        float v[32];
        {
          float x[16], y[16];
          tc::tmem_ld16x2(lanes + acc * BN + c, lanes + acc * BN + c + 16, x, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = x[i];
            v[16 + i] = y[i];
          }
        }
        if (n0 + c + 32 <= p.n) {
          if ((p.n & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 s = __ldg(reinterpret_cast<const float4*>(p.ws + n0 + c + i));
              v[i] *= as * s.x; v[i + 1] *= as * s.y; v[i + 2] *= as * s.z; v[i + 3] *= as * s.w;
            }
            if (p.bias) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 s = __ldg(reinterpret_cast<const float4*>(p.bias + n0 + c + i));
                v[i] += s.x; v[i + 1] += s.y; v[i + 2] += s.z; v[i + 3] += s.w;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] *= as * __ldg(p.ws + n0 + c + i);
              if (p.bias) v[i] += __ldg(p.bias + n0 + c + i);
            }
          }
          if (in && vec) {
            if constexpr (sizeof(O) == 2) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                  h[j] = *reinterpret_cast<const uint32_t*>(&b);
                }
                *reinterpret_cast<uint4*>(out + c + i) = make_uint4(h[0], h[1], h[2], h[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(out + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          } else if (in) {
#pragma unroll
            for (int i = 0; i < 32; ++i) out[c + i] = from_f<O>(v[i]);
          }
        } else if (in) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (n0 + c + i < p.n) {
              v[i] *= as * __ldg(p.ws + n0 + c + i);
              out[c + i] = from_f<O>(p.bias ? v[i] + __ldg(p.bias + n0 + c + i) : v[i]);
            }
        }
        __syncwarp();  // (the next load is the whole warp's)
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(at_rank(tc::smem_u32(&drained[acc]), 0));
      acc ^= 1;
      if (acc == 0) aph ^= 1;
    }
  }
  if (!ok) atomicOr(p.status, kDevTimeout);
  __syncwarp();
  tc::tc_fence_before();
  cluster_sync_all();  // the other CTA's barriers and tensor memory are in use until here
  tc::tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

template <bool kFp8, typename O, int BN>
cudaError_t launch_pairs_t(const MatmulArgs& p, const void* a, const void* w, uint64_t row_bytes, uint64_t stride,
                           cudaStream_t s) {
  CUtensorMap am, wm;
  if (!encode_tmap_rows(&am, a, row_bytes, (uint64_t)p.m, stride, kRowsA) ||
      !encode_tmap_rows(&wm, w, row_bytes, (uint64_t)p.n, stride, BN / 2))
    return cudaErrorInvalidValue;
  TcArgs t = {p.as, p.ws, p.bias, p.out, p.status, p.m, p.n, (int)((p.m + 255) / 256), (int)((p.n + BN - 1) / BN),
              (int)((row_bytes + 127) / 128)};
  const long long tiles = (long long)t.mt * t.nt;
  const int pairs = device_sm_count() / 2;
  const unsigned grid = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
  constexpr int smem = TcSmem<BN>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(pair_matmul_kernel<kFp8, O, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("scaled_matmul_pairs");
  pair_matmul_kernel<kFp8, O, BN><<<grid, kTcThreads, smem, s>>>(am, wm, t);
  return cudaGetLastError();
}
template <bool kFp8, typename O>
cudaError_t launch_pairs(const MatmulArgs& p, const void* a, const void* w, uint64_t row_bytes, uint64_t stride,
                         cudaStream_t s) {
  const long long mt = (p.m + 255) / 256;
  const int pairs = device_sm_count() / 2;
  if (mt * ((p.n + 255) / 256) >= pairs) return launch_pairs_t<kFp8, O, 256>(p, a, w, row_bytes, stride, s);
  if (mt * ((p.n + 127) / 128) >= pairs) return launch_pairs_t<kFp8, O, 128>(p, a, w, row_bytes, stride, s);
  return launch_pairs_t<kFp8, O, 64>(p, a, w, row_bytes, stride, s);
}

// ---- plan -------------------------------------------------------------------
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct MatmulPlan {
  bool few, pack, half;   // which kernel; rows written out first; as fp16
  long long pitch;        // bytes of a written row
  size_t off_a, off_w, bytes;
};

int check(const ssd_matmul_problem* pr, MatmulPlan* p) {
  if (!pr || pr->m < 1 || pr->n < 1 || pr->k < 1 || pr->flags != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->format != SSD_CACHE_INT8 && pr->format != SSD_CACHE_E4M3) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->out_dtype != SSD_F32 && pr->out_dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
  // 2^40 elements per tensor; rows and tiles in 32 bits
  const int64_t cap = 1LL << 22;
  if (pr->m > cap || pr->n > cap || pr->k > cap || (double)pr->m * (double)pr->n >= (double)(1LL << 40) ||
      (double)pr->m * (double)pr->k >= (double)(1LL << 40) || (double)pr->n * (double)pr->k >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  p->few = pr->m <= kFewTokens;
  p->half = !p->few && pr->format == SSD_CACHE_INT8;
  p->pack = p->half || pr->k % 16 != 0;
  p->pitch = p->half ? (pr->k + 63) / 64 * 128 : (pr->k + 15) / 16 * 16;
  p->off_a = p->off_w = 256;
  p->bytes = 256;
  if (p->pack) {
    p->off_w = 256 + align256((size_t)pr->m * p->pitch);
    p->bytes = p->off_w + align256((size_t)pr->n * p->pitch);
  }
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

template <bool kFp8, typename O>
cudaError_t launch_product(const MatmulPlan& pl, const MatmulArgs& p, const void* a, const void* w, cudaStream_t s) {
  if (pl.few) return launch_skinny<kFp8, O>(p, s);
  return launch_pairs<kFp8, O>(p, a, w, pl.half ? (uint64_t)pl.pitch : (uint64_t)p.k, pl.pack ? pl.pitch : p.k, s);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_scaled_matmul_workspace_bytes(const ssd_matmul_problem* pr) {
  MatmulPlan pl;
  return check(pr, &pl) == SSD_OK ? pl.bytes : 0;
}

int ssd_scaled_matmul(const ssd_matmul_problem* pr, const void* a, const float* a_scales, const void* w,
                      const float* w_scales, const float* bias, void* out, void* workspace, size_t workspace_bytes,
                      ssd_stream_t stream) {
  MatmulPlan pl;
  int rc = check(pr, &pl);
  if (rc != SSD_OK) return rc;
  if (!a || !a_scales || !w || !w_scales || !out || !workspace) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {a, a_scales, w, w_scales, bias, out, workspace};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < pl.bytes) return SSD_ERR_WORKSPACE_TOO_SMALL;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MatmulArgs p = {static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(w), a_scales, w_scales, bias, out,
                  reinterpret_cast<int*>(ws), pr->m, pr->n, pr->k};
  cudaError_t e;
  if (pl.pack) {
    PackArgs q;
    memset(&q, 0, sizeof(q));
    q.src[0] = p.a; q.src[1] = p.w;
    q.dst[0] = ws + pl.off_a; q.dst[1] = ws + pl.off_w;
    q.k = (int)pr->k;
    q.per_row = (int)(pl.half ? pl.pitch / 32 : pl.pitch / 16);
    q.groups[0] = pr->m * q.per_row; q.groups[1] = pr->n * q.per_row;
    q.bytes[0] = pr->m * pr->k; q.bytes[1] = pr->n * pr->k;
    q.status = p.status;
    long long grid = (q.groups[0] + q.groups[1] + 255) / 256;
    const long long most = (long long)device_sm_count() * 16;
    if (grid > most) grid = most;
    set_kernel_name("scaled_matmul_pack");
    prof_before(s);
    if (pl.half) pack_rows_kernel<true><<<(unsigned)grid, 256, 0, s>>>(q);
    else pack_rows_kernel<false><<<(unsigned)grid, 256, 0, s>>>(q);
    e = cudaGetLastError();
    prof_after(s);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
    p.a = ws + pl.off_a;
    p.w = ws + pl.off_w;
    if (!pl.half) p.k = pl.pitch;
  } else if (!pl.few) {
    if (cudaMemsetAsync(p.status, 0, sizeof(int), s) != cudaSuccess) return SSD_ERR_CUDA;
  }
  const bool fp8 = pr->format == SSD_CACHE_E4M3, b16 = pr->out_dtype == SSD_BF16;
  prof_before(s);
  e = fp8 ? (b16 ? launch_product<true, __nv_bfloat16>(pl, p, p.a, p.w, s) : launch_product<true, float>(pl, p, p.a, p.w, s))
          : (b16 ? launch_product<false, __nv_bfloat16>(pl, p, p.a, p.w, s)
                 : launch_product<false, float>(pl, p, p.a, p.w, s));
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
