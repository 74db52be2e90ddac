// k_scaled_matmul.cu -- the product of 8-bit codes (int8 or e4m3) with a scale
// for each token and for each channel, and its C ABI.
//
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n]
//
// This chip's integer tensor rate is a small part of its fp16 rate, so int8
// codes are multiplied as fp16, which holds them and their products' factors
// exactly; sums are fp32.  e4m3 codes go to the tensor cores as they are.
//
// Three kernels, by the number of tokens:
//  * up to 16 (e4m3) or 24 (int8): bound by the weights' bytes.  Warps read 16
//    channels' codes in 16-byte pieces, turn them into fp16 in registers and
//    multiply them with the tokens' by warp-level products; the order of k inside
//    a product is free, so a lane's 16 neighbouring codes serve four products as
//    they lie.  One token, 10304 x 4096 int8: 10 us (4.2 TB/s), 7.7 with the weights in L2.
//  * some hundreds: tensor-memory products of 128 tokens x up to 256 channels, k
//    shared by the CTAs of a cluster.  An instruction with 128 rows takes about 136
//    cycles whether it has 32 columns or 256, so the weights are the columns.  int8
//    codes stay int8 up to shared memory; warps turn them into fp16 there, and the
//    chain of copy, turn and product bounds it.  61 tokens: int8 20 us, e4m3 14.7 (17 and 11
//    with the weights in L2); from 129 tokens on the weights are read and turned again
//    for every 128: int8 22 us at 128, 37 at 129, 69 at 512.
//  * more: products of 256 tokens x up to 256 channels by pairs of CTAs,
//    persistent, the epilogue of one tile under the products of the next, bound by
//    the tensor cores.  16,384 tokens: int8 0.83 ms (1,650 TFLOP/s, 1,790 without
//    writing the codes out), e4m3 0.43 ms (3,230).
// A launch before them writes out what they cannot read as it is: int8 codes as
// fp16 for the last one, rows that are not whole 16-byte vectors for all.
#include <cuda_fp16.h>
#include <string.h>

#include "codes.cuh"
#include "ssd_internal.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace ssd {

int device_check();

namespace {

constexpr int kFewTokens[2] = {24, 16};  // of int8, e4m3: what the first kernel takes

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

// ---- rows written out -------------------------------------------------------
// as fp16 or as they are, with rows of whole 16-byte vectors and zeros behind
// the k-th code
struct PackPart {
  const uint8_t* src;
  uint8_t* dst;
  long long groups, bytes;  // groups of 16 codes in all; bytes of the source
  int per_row, half;        // groups to a row; as fp16
};
struct PackArgs {
  PackPart part[2];
  int k;
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

__global__ void __launch_bounds__(256) pack_rows_kernel(PackArgs p) {
  // (the pairs' launch may come up; it waits for this one's end before it reads)
  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const long long total = p.part[0].groups + p.part[1].groups;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int which = i >= p.part[0].groups;
    const PackPart& t = p.part[which];
    const long long g = which ? i - p.part[0].groups : i, row = g / t.per_row;
    const int c = (int)(g - row * t.per_row) * 16, count = min(max(p.k - c, 0), 16);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (count) u = load16(t.src, row * p.k + c, count, t.bytes);
    uint4* to = reinterpret_cast<uint4*>(t.dst);
    if (t.half) {
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
__global__ void __launch_bounds__(kSkWarps * 32, MT == 1 ? 5 : MT == 2 ? 4 : 2) skinny_kernel(MatmulArgs p) {
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
  constexpr int kAhead = 2;
  const int k = (int)p.k;
  // (a warp's kAhead pieces of a row are neighbours: whole lines of memory)
  for (int k0 = warp * 64 * kAhead; k0 < k; k0 += kSkWarps * 64 * kAhead) {
    uint4 w[kAhead][CT][2], tok_codes[kAhead][MT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int kk = k0 + u * 64;
      const bool in = kk + q * 16 < k;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[u][c][h] = in ? __ldcs(reinterpret_cast<const uint4*>(wrow[c][h] + kk)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        tok_codes[u][t] = in && t * 8 + g < p.m
                              ? __ldg(reinterpret_cast<const uint4*>(p.a + (t * 8 + g) * p.k + kk + q * 16))
                              : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      uint32_t wh[CT][2][8];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        to_half<kFp8>(w[u][c][0], wh[c][0]);
        to_half<kFp8>(w[u][c][1], wh[c][1]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t ah[8];
        to_half<kFp8>(tok_codes[u][t], ah);
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
  if constexpr (!kFp8) return launch_skinny_t<kFp8, O, 2, 3>(p, s);
  return cudaErrorInvalidValue;  // (more e4m3 tokens than check() sends here)
}

// D (+)= A B^T of a pair of CTAs, or of one (e4m3), from shared memory
template <bool kFp8, bool kPair>
__device__ __forceinline__ void block_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  static_assert(kPair || kFp8, "one CTA's fp16 products take A from tensor memory");
#define SSD_MMA(group, kind)                                              \
  asm volatile(                                                           \
      "{\n\t.reg .pred p;\n\t"                                            \
      "setp.ne.b32 p, %4, 0;\n\t"                                         \
      "tcgen05.mma." group "." kind " [%0], %1, %2, %3, p;\n\t}\n" ::"r"( \
          d),                                                             \
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                         \
      : "memory")
  if constexpr (kPair && kFp8) SSD_MMA("cta_group::2", "kind::f8f6f4");
  else if constexpr (kPair) SSD_MMA("cta_group::2", "kind::f16");
  else SSD_MMA("cta_group::1", "kind::f8f6f4");
#undef SSD_MMA
}
// fp32 sums of fp16 (kind::f16) or e4m3 (kind::f8f6f4): both formats are number 0
constexpr uint32_t idesc_of(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

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
// tc::mbar_wait_flag for barriers at which another CTA's threads arrive
__device__ __forceinline__ void wait_cluster(uint64_t* bar, uint32_t parity, bool& ok) {
  const long long c0 = clock64();
  for (uint32_t outer = 0; outer < (ok ? 1u << 14 : 64u); ++outer) {
    for (int i = 0; i < 64; ++i) {
      uint32_t hit;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}\n"
          : "=r"(hit)
          : "r"(tc::smem_u32(bar)), "r"(parity)
          : "memory");
      if (hit) return;
    }
    if (clock64() - c0 > (1ll << 31)) break;
  }
  ok = false;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ---- some tokens ------------------------------------------------------------
// A CTA multiplies 128 tokens' rows with up to 256 channels over its share of k,
// 128 codes to a stage.  e4m3: the products take both from the stage.  int8: two
// groups of eight warps turn the weights into fp16, each 64 codes of every stage,
// in a place of its own, so that one group writes under the other's products (one
// group for both places: 2100 cycles a stage, two: 1700); four warps turn the
// tokens, a lane to a row, and put them into tensor memory.  The CTAs of a cluster
// share k; they leave their sums in shared memory and each joins and writes some
// of the tokens, in the order of the shares.
constexpr int kRows = 128;                                  // tokens of a CTA
constexpr int kWide = 256;                                  // channels of a CTA, at most
constexpr int kGroup = 8, kTurners = 2 * kGroup, kTokTurners = 4;
constexpr int kSomeThreads = (kTurners + kTokTurners + 2) * 32;

template <bool kFp8>
struct SomeShape {
  // The stages: as many of (ch + box) 128-byte rows as there is room for
  static constexpr int kRing = kFp8 ? 196608 : 147456, kStages = 8;
  // behind them two places of 64 codes as fp16, or the rows up to the 128th that products of the last stage's tokens read
  // (whatever they hold; their sums are not written)
  static constexpr int kTurned = kFp8 ? kRows * 128 : 2 * kWide * 128;
  static constexpr int kBytes = kRing + kTurned + 1024;
  static constexpr int kPlaces = 4;                           // of the tokens in tensor memory, 64 columns each
  static constexpr uint32_t kCols = kFp8 ? kWide : kWide + 64 * kPlaces;
  static_assert(kRows * kWide * 4 <= kRing && 3 * (kWide + kRows) * 128 <= kRing, "the sums, and three stages, fit into the ring");
};

struct SomeArgs {
  MatmulArgs p;
  int ch, kb, per;  // channels of a CTA (a multiple of 16); stages of k in all; of a CTA
  int nt;           // tiles of channels
  int box;          // rows of a tile's tokens that are copied (a multiple of 8)
  int clear;        // no launch before this one has cleared the status word
};

// 32 columns of a lane's row of tensor memory
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (+)= A B^T with A in tensor memory: lane i is row i, a column two neighbouring k
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint4 shared_load(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
  return u;
}
__device__ __forceinline__ void shared_store(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// A place in a ring of n, and the parity of the round that it is in
struct Ring {
  int n, at = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ explicit Ring(int places) : n(places) {}
  __device__ __forceinline__ void next() {
    if (++at == n) {
      at = 0;
      ph ^= 1;
    }
  }
};

template <bool kFp8, typename O>
__global__ void __launch_bounds__(kSomeThreads)
    some_tokens_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap, SomeArgs s) {
  using S = SomeShape<kFp8>;
  constexpr int kStages = S::kStages, kPlaces = S::kPlaces;
  extern __shared__ uint8_t raw[];
  const MatmulArgs& p = s.p;
  const uint32_t pad = (1024u - (tc::smem_u32(raw) & 1023u)) & 1023u, smem = tc::smem_u32(raw) + pad;
  const uint32_t wbuf = smem + S::kRing, w_bytes = s.ch * 128, stage_bytes = w_bytes + s.box * 128;
  const int stages = min(S::kRing / (int)stage_bytes, kStages);
  __shared__ uint64_t full[kStages], empty[kStages], wfull[2], wempty[2], turned[kPlaces], taken[kPlaces], done;
  __shared__ uint32_t tmem_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  uint32_t ncta;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const int tile = (int)(blockIdx.x / ncta);
  const long long n0 = (long long)(tile % s.nt) * s.ch;
  const int m0 = tile / s.nt * kRows, rows = (int)min(p.m - m0, (long long)kRows);
  const int quarters = (rows + 31) / 32;  // lane quarters that hold tokens
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], kFp8 ? 1 : kTurners + quarters);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&wfull[i], kGroup);
      tc::mbar_init(&wempty[i], 1);
    }
    for (int i = 0; i < kPlaces; ++i) {
      tc::mbar_init(&turned[i], quarters);
      tc::mbar_init(&taken[i], 1);
    }
    tc::mbar_init(&done, 1);
    tc::mbar_fence_init();
    if (s.clear && blockIdx.x == 0) *p.status = 0;  // (a wait that expires does so a second later)
  }
  constexpr int kMmaWarp = kTurners + kTokTurners, kCopyWarp = kMmaWarp + 1;
  if (warp == kCopyWarp && lane == 0) {
    tc::prefetch_tmap(&amap);
    tc::prefetch_tmap(&wmap);
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_s, S::kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_s;
  const int b0 = (int)rank * s.per, nb = min(s.per, s.kb - b0);
  bool ok = true;

  if (warp == kCopyWarp) {
    if (lane == 0) {
      Ring st(stages);
      for (int b = 0; b < nb; ++b, st.next()) {
        tc::mbar_wait_flag(&empty[st.at], st.ph ^ 1, ok);
        const uint32_t to = smem + st.at * stage_bytes;
        tc::mbar_expect_tx(&full[st.at], stage_bytes);
        box_load(to, &wmap, &full[st.at], (b0 + b) * 128, (int)n0);
        box_load(to + w_bytes, &amap, &full[st.at], (b0 + b) * 128, m0);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const uint32_t idesc = idesc_of(kRows, s.ch);
      Ring st(stages);
      Ring pl(kPlaces);
      for (int b = 0; b < nb; ++b) {
        if constexpr (kFp8) {
          tc::mbar_wait_flag(&full[st.at], st.ph, ok);
          tc::tc_fence_after();
          const uint32_t w = smem + st.at * stage_bytes, a = w + w_bytes;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            block_mma<true, false>(tmem, tc::smem_desc(a + j * 32, 16, 1024, tc::kSwz128),
                                   tc::smem_desc(w + j * 32, 16, 1024, tc::kSwz128), idesc, b | j);
          tc::mma_commit(&empty[st.at]);
          st.next();
        } else {
          tc::mbar_wait_flag(&turned[pl.at], pl.ph, ok);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc::mbar_wait_flag(&wfull[h], (uint32_t)b & 1u, ok);
            tc::tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_from_tmem(tmem, tmem + kWide + pl.at * 64 + h * 32 + j * 8,
                            tc::smem_desc(wbuf + h * (kWide * 128) + j * 32, 16, 1024, tc::kSwz128), idesc, b | h | j);
            tc::mma_commit(&wempty[h]);
          }
          tc::mma_commit(&taken[pl.at]);
          pl.next();
        }
      }
      tc::mma_commit(&done);
    }
  } else if (!kFp8 && warp < kTurners) {
    // A unit is 16 codes of a channel, 32 bytes as fp16.  Eight lanes read the
    // units of rows x and x ^ 5, so that neither their reads nor their writes meet in
    // a bank.
    const int unit = lane & 3, g = lane >> 2, x = (g >> 1) ^ (g & 1 ? 5 : 0);
    const int half = warp / kGroup, row0 = (warp % kGroup) * 8 + x;
    const uint32_t from = row0 * 128, read0 = from + (((half * 4 + unit) ^ x) << 4);
    const uint32_t put0 = wbuf + half * (kWide * 128) + from + ((2 * unit ^ x) << 4),
                   put1 = wbuf + half * (kWide * 128) + from + (((2 * unit + 1) ^ x) << 4);
    const int units = (s.ch - row0 + 63) / 64;  // rows row0, row0 + 64, ... of this tile (at most four)
    Ring st(stages);
    for (int b = 0; b < nb; ++b, st.next()) {
      tc::mbar_wait_flag(&full[st.at], st.ph, ok);
      uint32_t v[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < units) to_half<false>(shared_load(smem + st.at * stage_bytes + read0 + i * 64 * 128), v[i]);
      tc::fence_async_smem();  // read here, written by a copy
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[st.at]);
      tc::mbar_wait_flag(&wempty[half], (uint32_t)(b & 1) ^ 1u, ok);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < units) {
          shared_store(put0 + i * 64 * 128, v[i][0], v[i][1], v[i][2], v[i][3]);
          shared_store(put1 + i * 64 * 128, v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      tc::fence_async_smem();  // written here, read by the products
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&wfull[half]);
    }
  } else if (!kFp8 && warp - kTurners < quarters) {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    Ring st(stages);
    Ring pl(kPlaces);
    for (int b = 0; b < nb; ++b) {
      tc::mbar_wait_flag(&full[st.at], st.ph, ok);
      const uint32_t row = smem + st.at * stage_bytes + w_bytes + r * 128;
      uint32_t h[2][32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v[8];
        to_half<false>(shared_load(row + ((j ^ (r & 7)) << 4)), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j >> 2][(j & 3) * 8 + i] = v[i];
      }
      tc::fence_async_smem();  // read here, written by a copy
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[st.at]);
      tc::mbar_wait_flag(&taken[pl.at], pl.ph ^ 1, ok);
      tc::tc_fence_after();
      __syncwarp();
      const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + kWide + pl.at * 64;
      tmem_store32(to, h[0]);
      tmem_store32(to + 32, h[1]);
      tmem_store_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&turned[pl.at]);
      st.next();
      pl.next();
    }
  }
  __syncwarp();
  // Every product is done: the stages become the sums, a row of kWide fp32 to a
  // token, whose 16-byte pieces are swapped by the row, so that neither a column's
  // writes nor a row's reads meet in a bank.
  tc::mbar_wait_flag(&done, 0, ok);
  tc::tc_fence_after();
  __syncwarp();
  if (warp < kMmaWarp && (warp & 3) < quarters) {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    for (int c = (warp >> 2) * 16; c < s.ch; c += (kMmaWarp / 4) * 16) {
      float v[16];
      tc::tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        shared_store(smem + r * (kWide * 4) + (((c / 4 + i) ^ (r & 7)) << 4), __float_as_uint(v[4 * i]),
                     __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    }
  }
  tc::tc_fence_before();
  __syncwarp();
  if (ncta > 1) cluster_sync_all();
  else __syncthreads();
  tc::tc_fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, S::kCols);
  const int share = (rows + (int)ncta - 1) / (int)ncta, lo = (int)rank * share, hi = min(lo + share, rows);
  const int pieces = s.ch / 4;
  for (int i = lo * pieces + (int)threadIdx.x; i < hi * pieces; i += kSomeThreads) {
    const int t = i / pieces, c = i - t * pieces;
    const long long n = n0 + c * 4;
    if (n >= p.n) continue;
    const int cols = (int)min(p.n - n, 4LL);
    const uint32_t at = smem + t * (kWide * 4) + ((c ^ (t & 7)) << 4);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t r = 0; r < ncta; ++r) {
      float x[4];
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                   : "r"(at_rank(at, r))
                   : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += x[j];
    }
    const float as = __ldg(p.as + m0 + t);
    O* out = static_cast<O*>(p.out) + (m0 + t) * p.n + n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cols) {
        v[j] = v[j] * as * __ldg(p.ws + n + j);
        if (p.bias) v[j] += __ldg(p.bias + n + j);
      }
    if (p.n % 4 == 0) {  // (then there are four)
      if constexpr (sizeof(O) == 2) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]), y = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(out) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      } else {
        *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) out[j] = from_f<O>(v[j]);
    }
  }
  if (!ok) atomicOr(p.status, kDevTimeout);
  __syncwarp();
  if (ncta > 1) cluster_sync_all();  // other CTAs read this one's sums until here
}

// Clusters of 1 .. 8 CTAs that this chip holds at once, one CTA to an SM (they only
// decide how the work is shared out).
constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

// Channels to a CTA and CTAs to a cluster: what costs least by the cycles of a
// stage (measured: about 1500 and one for each channel with int8, 800 with e4m3),
// the stages of a share, the waves of clusters, and what a CTA takes beside its
// stages.  Few channels make no stage shorter, so they are as many as leave no
// wave more.  Returns the cycles.
double share_out(bool fp8, int64_t m, int64_t n, int64_t k, SomeArgs* a, int* split) {
  a->kb = (int)((k + 127) / 128);
  const long long mt = (m + kRows - 1) / kRows, wide = (n + kWide - 1) / kWide;
  double best = 0;
  for (int x = 1; x <= 8 && x <= a->kb; ++x) {
    const int per = (a->kb + x - 1) / x;
    if ((long long)per * (x - 1) >= a->kb) continue;  // a share without a stage
    const long long waves = (wide * mt + kClusters[x] - 1) / kClusters[x], tiles = waves * kClusters[x] / mt;
    const int ch = (int)((n + tiles - 1) / tiles + 15) / 16 * 16;
    if (waves * kClusters[x] * x > (1LL << 30)) continue;  // (CTAs of a grid)
    const double cost = (double)waves * (1.15 * (per * ((fp8 ? 800.0 : 1500.0) + ch) + 7000 + (x > 1 ? 2000 : 0)));
    if (best == 0 || cost < best) {
      best = cost;
      a->ch = ch < 32 ? 32 : ch;
      a->per = per;
      *split = x;
    }
  }
  if (best > 0) a->nt = (int)((n + a->ch - 1) / a->ch);
  return best;  // (0: too many)
}

// a, w: rows as the copies read them, of bytes in all and in memory
struct Rows {
  const void* at;
  uint64_t bytes, pitch;
};

template <bool kFp8, typename O>
cudaError_t launch_some(const MatmulArgs& p, const Rows& ra, const Rows& rw, cudaStream_t s, bool clear) {
  auto kernel = some_tokens_kernel<kFp8, O>;
  constexpr int smem = SomeShape<kFp8>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  SomeArgs a;
  memset(&a, 0, sizeof(a));
  a.p = p;
  a.clear = clear;
  int split = 1;
  share_out(kFp8, p.m, p.n, p.k, &a, &split);
  // (the rows behind the tokens' last are whatever shared memory holds: their sums are not written)
  a.box = p.m < kRows ? (int)(p.m + 7) / 8 * 8 : kRows;
  CUtensorMap am, wm;
  if (!encode_tmap_rows(&am, ra.at, ra.bytes, (uint64_t)p.m, ra.pitch, (uint32_t)a.box) ||
      !encode_tmap_rows(&wm, rw.at, rw.bytes, (uint64_t)p.n, rw.pitch, (uint32_t)a.ch))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.nt * ((p.m + kRows - 1) / kRows) * split));
  cfg.blockDim = dim3(kSomeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  set_kernel_name("scaled_matmul_some");
  return cudaLaunchKernelEx(&cfg, kernel, am, wm, a);
}

// ---- many tokens: tensor-memory products by pairs of CTAs -------------------
//
// A pair computes 256 tokens x BN channels: each CTA holds 128 tokens' rows and
// half of the channels' rows of every stage, and 128 rows of the result in its
// own tensor memory, twice.  The leader (even rank) issues the products for
// both; its `full` barriers take the bytes of both CTAs' copies.  Commits arrive
// in both CTAs.
constexpr int kStages = 6;
constexpr int kRowsA = 128;  // tokens of one of its CTAs

template <int BN>
struct PairSmem {
  static constexpr int kA = kRowsA * 128, kB = BN / 2 * 128;
  static constexpr int kStageBytes = kA + kB;
  static constexpr int kOut = 4 * 32 * 128;  // 32 rows of 128 bytes for each epilogue warp
  static constexpr int kBytes = kStages * kStageBytes + kOut + 1024;
};

// A box into this CTA's shared memory, its bytes counted by a barrier of the pair
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrives on the barrier at this place in both CTAs once this thread's products are done
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
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

struct PairArgs {
  MatmulArgs p;
  int mt, nt, kb;  // tiles of tokens and channels; blocks of k
  int clear;       // no launch before this one has cleared the status word
};

// 32 rows of 128 bytes of results from an epilogue warp, a row to a lane, through
// shared memory, so that eight lanes write a row's 128 bytes together.
template <typename O>
__device__ __forceinline__ void write_rows(uint32_t buf, const uint4 (&mine)[8], O* out, long long row0, long long col0,
                                           const MatmulArgs& p, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((j ^ (lane & 7)) << 4)),
                 "r"(mine[j].x), "r"(mine[j].y), "r"(mine[j].z), "r"(mine[j].w)
                 : "memory");
  __syncwarp();
  constexpr int n = 16 / sizeof(O);
  if (p.n % n == 0) {
    const int piece = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      uint4 u;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "r"(buf + r * 128 + ((piece ^ (r & 7)) << 4))
                   : "memory");
      if (row0 + r < p.m && col0 + piece * n < p.n)
        *reinterpret_cast<uint4*>(out + (row0 + r) * p.n + col0 + piece * n) = u;
    }
  } else {
    for (int r = 0; r < 32 && row0 + r < p.m; ++r)
#pragma unroll
      for (int i = 0; i < 128 / (int)sizeof(O) / 32; ++i) {
        const int c = i * 32 + lane, at = c * (int)sizeof(O);
        const uint32_t from = buf + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15);
        if (col0 + c < p.n) {
          if constexpr (sizeof(O) == 2) {
            unsigned short h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(from) : "memory");
            out[(row0 + r) * p.n + col0 + c] = __ushort_as_bfloat16(h);
          } else {
            float f;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(from) : "memory");
            out[(row0 + r) * p.n + col0 + c] = f;
          }
        }
      }
  }
  __syncwarp();
}

// One warp issues copies, one the products, four write results.
constexpr int kPairThreads = 192;
template <bool kFp8, typename O, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
    pair_matmul_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap, PairArgs s) {
  using S = PairSmem<BN>;
  extern __shared__ uint8_t raw[];
  const MatmulArgs& p = s.p;
  const uint32_t smem = (tc::smem_u32(raw) + 1023u) & ~1023u;
  __shared__ uint64_t full[kStages], empty[kStages], done[2], drained[2];
  __shared__ alignas(16) float scale_s[2][2][BN];  // the channels' scales and biases of a tile
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
    if (s.clear && blockIdx.x == 0) *p.status = 0;  // (a wait that expires does so a second later)
  }
  constexpr uint32_t kCols = BN * 2;
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
  const long long tiles = (long long)s.mt * s.nt, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      tc::prefetch_tmap(&amap);
      tc::prefetch_tmap(&wmap);
      asm volatile("griddepcontrol.wait;" ::: "memory");  // what the launch before this one has written is there
      int st = 0;
      uint32_t ph = 0;
      for (long long t = pair; t < tiles; t += pairs) {
        int tm, tn;
        tile_of(t, s.mt, s.nt, tm, tn);
        const int ya = tm * 256 + (int)rank * 128, yw = tn * BN + (int)rank * (BN / 2);
        for (int b = 0; b < s.kb; ++b) {
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
      int st = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (long long t = pair; t < tiles; t += pairs) {
        wait_cluster(&drained[acc], aph ^ 1, ok);
        tc::tc_fence_after();
        for (int b = 0; b < s.kb; ++b) {
          wait_cluster(&full[st], ph, ok);
          tc::tc_fence_after();
          const uint32_t a = smem + st * S::kStageBytes, w = a + S::kA;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            block_mma<kFp8, true>(tmem + acc * BN, tc::smem_desc(a + j * 32, 16, 1024, tc::kSwz128),
                                  tc::smem_desc(w + j * 32, 16, 1024, tc::kSwz128), idesc_of(256, BN), b | j);
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
    const int et = (warp - 2) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t buf = smem + kStages * S::kStageBytes + (uint32_t)quarter * 4096;
    constexpr int CH = 128 / sizeof(O);  // columns at a time: 128 bytes of a row
    int acc = 0;
    uint32_t aph = 0;
    for (long long t = pair; t < tiles; t += pairs) {
      int tm, tn;
      tile_of(t, s.mt, s.nt, tm, tn);
      const long long row0 = (long long)tm * 256 + rank * 128 + quarter * 32, n0 = (long long)tn * BN;
      const float as = row0 + lane < p.m ? __ldg(p.as + row0 + lane) : 0.f;
      for (int i = et; i < BN; i += 128) {
        const bool in = n0 + i < p.n;
        scale_s[acc][0][i] = in ? __ldg(p.ws + n0 + i) : 0.f;
        scale_s[acc][1][i] = in && p.bias ? __ldg(p.bias + n0 + i) : 0.f;
      }
      // (a buffer is written again two tiles on: every warp has passed this barrier of the tile between)
      asm volatile("bar.sync 1, 128;" ::: "memory");
      tc::mbar_wait_flag(&done[acc], aph, ok);
      tc::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BN && n0 + c < p.n; c += CH) {
        uint4 mine[8];
        uint32_t* word = reinterpret_cast<uint32_t*>(mine);
#pragma unroll
        for (int h = 0; h < CH; h += 32) {
          float x[16], y[16];
          tc::tmem_ld16x2(lanes + acc * BN + c + h, lanes + acc * BN + c + h + 16, x, y);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float u = i < 16 ? x[i] : y[i - 16], v = i < 16 ? x[i + 1] : y[i - 15];
            const float2 sc = *reinterpret_cast<const float2*>(&scale_s[acc][0][c + h + i]);
            u = u * as * sc.x;
            v = v * as * sc.y;
            if (p.bias) {
              const float2 bi = *reinterpret_cast<const float2*>(&scale_s[acc][1][c + h + i]);
              u += bi.x;
              v += bi.y;
            }
            if constexpr (sizeof(O) == 2) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(u, v);
              word[(h + i) / 2] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
              word[i] = __float_as_uint(u);
              word[i + 1] = __float_as_uint(v);
            }
          }
        }
        write_rows<O>(buf, mine, static_cast<O*>(p.out), row0, n0 + c, p, lane);
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
cudaError_t launch_pairs_t(const MatmulArgs& p, const Rows& ra, const Rows& rw, cudaStream_t s, bool clear) {
  CUtensorMap am, wm;
  if (!encode_tmap_rows(&am, ra.at, ra.bytes, (uint64_t)p.m, ra.pitch, kRowsA) ||
      !encode_tmap_rows(&wm, rw.at, rw.bytes, (uint64_t)p.n, rw.pitch, BN / 2))
    return cudaErrorInvalidValue;
  PairArgs t = {p, (int)((p.m + 255) / 256), (int)((p.n + BN - 1) / BN), (int)((ra.bytes + 127) / 128), clear};
  const long long tiles = (long long)t.mt * t.nt;
  const int pairs = device_sm_count() / 2;
  const unsigned grid = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
  constexpr int smem = PairSmem<BN>::kBytes;
  auto kernel = pair_matmul_kernel<kFp8, O, BN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  set_kernel_name("scaled_matmul_pairs");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  // Behind the launch that writes out the rows this one comes up early, and waits for it before its first copy.
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = clear ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, am, wm, t);
}
// Waves of tiles of the pairs' products with tiles of bn channels (by this chip's 76
// pairs of SMs: they only choose the plan, without a device at hand), and whether
// narrow tiles take no wave more: their products take as long as the wide ones',
// but their ends are shorter.
long long pair_waves(int64_t m, int64_t n, int bn) { return ((m + 255) / 256 * ((n + bn - 1) / bn) + 75) / 76; }
bool narrow_pairs(int64_t m, int64_t n) { return pair_waves(m, n, 128) <= pair_waves(m, n, 256); }

template <bool kFp8, typename O>
cudaError_t launch_pairs(const MatmulArgs& p, const Rows& ra, const Rows& rw, cudaStream_t s, bool clear) {
  if (narrow_pairs(p.m, p.n)) return launch_pairs_t<kFp8, O, 128>(p, ra, rw, s, clear);
  return launch_pairs_t<kFp8, O, 256>(p, ra, rw, s, clear);
}

// The cycles of the products of few tokens: a short launch, and the weights at so
// many bytes a cycle (e4m3 codes become fp16 at a lower rate).  One token, 10304 x
// 4096, weights in L2: int8 8.7 us, by the next kernel 17; e4m3 11.6 and 10; 2048 x
// 4096: 5.6 and 7.7.
double few_cost(bool fp8, int64_t m, int64_t n, int64_t k) {
  const double rate = fp8 ? (m <= 8 ? 2000 : 1500) : m <= 8 ? 2900 : m <= 16 ? 2100 : 1600;
  return 5000 + (double)n * (double)k / rate;
}

// The cycles of the products by pairs: waves of tiles by the stages of 128 bytes
// (four products of about 175 cycles), what writing int8 codes out as fp16 takes at
// 2600 bytes a cycle, and a tile's beginning and end.
double pairs_cost(bool fp8, int64_t m, int64_t n, int64_t k) {
  return (double)pair_waves(m, n, 256) * (double)((k * (fp8 ? 1 : 2) + 127) / 128) * 700 + 12000 +
         (fp8 ? 0 : (double)(m + n) * (double)k * 3 / 2600);
}

// ---- plan -------------------------------------------------------------------
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct MatmulPlan {
  bool few, some;
  // which operand is written out first (as fp16), with what pitch, and where
  bool out_a, out_w, half_a, half_w;
  long long pitch_a, pitch_w;
  size_t off_a, off_w, bytes;
};

int check(const ssd_matmul_problem* pr, MatmulPlan* pl) {
  if (!pr || pr->m < 1 || pr->n < 1 || pr->k < 1 || pr->flags != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->format != SSD_CACHE_INT8 && pr->format != SSD_CACHE_E4M3) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->out_dtype != SSD_F32 && pr->out_dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
  // 2^40 elements per tensor; rows and tiles in 32 bits
  const int64_t cap = 1LL << 22;
  if (pr->m > cap || pr->n > cap || pr->k > (1LL << 20) || (double)pr->m * (double)pr->n >= (double)(1LL << 40) ||
      (double)pr->m * (double)pr->k >= (double)(1LL << 40) || (double)pr->n * (double)pr->k >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  const bool whole = pr->k % 16 == 0, int8 = pr->format == SSD_CACHE_INT8;
  SomeArgs share;
  int split;
  const double some = share_out(!int8, pr->m, pr->n, pr->k, &share, &split);  // (0: too many CTAs)
  pl->few = pr->m <= kFewTokens[!int8] && (some == 0 || few_cost(!int8, pr->m, pr->n, pr->k) <= some);
  pl->some = !pl->few && some > 0 && some <= pairs_cost(!int8, pr->m, pr->n, pr->k);
  pl->half_a = pl->half_w = int8 && !pl->few && !pl->some;
  pl->out_a = pl->half_a || !whole;
  pl->out_w = pl->half_w || !whole;
  const long long codes = (pr->k + 15) / 16 * 16;
  pl->pitch_a = codes << pl->half_a;
  pl->pitch_w = codes << pl->half_w;
  pl->off_a = 256;
  pl->off_w = 256 + (pl->out_a ? align256((size_t)pr->m * pl->pitch_a) : 0);
  pl->bytes = pl->off_w + (pl->out_w ? align256((size_t)pr->n * pl->pitch_w) : 0);
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

template <bool kFp8, typename O>
cudaError_t launch_product(const MatmulPlan& pl, MatmulArgs p, const Rows& ra, const Rows& rw, cudaStream_t s) {
  const bool clear = !pl.out_a && !pl.out_w;
  if (pl.few) {
    p.a = static_cast<const uint8_t*>(ra.at);
    p.w = static_cast<const uint8_t*>(rw.at);
    p.k = (long long)ra.pitch;  // (zeros behind the last code)
    return launch_skinny<kFp8, O>(p, s);
  }
  if (pl.some) return launch_some<kFp8, O>(p, ra, rw, s, clear);
  return launch_pairs<kFp8, O>(p, ra, rw, s, clear);
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
  const MatmulArgs p = {static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(w), a_scales, w_scales, bias, out,
                        reinterpret_cast<int*>(ws), pr->m, pr->n, pr->k};
  const Rows ra = {pl.out_a ? ws + pl.off_a : a, (uint64_t)pr->k << pl.half_a,
                   (uint64_t)(pl.out_a ? pl.pitch_a : pr->k)},
             rw = {pl.out_w ? ws + pl.off_w : w, (uint64_t)pr->k << pl.half_w,
                   (uint64_t)(pl.out_w ? pl.pitch_w : pr->k)};
  cudaError_t e;
  if (pl.out_a || pl.out_w) {
    PackArgs q;
    memset(&q, 0, sizeof(q));
    q.k = (int)pr->k;
    q.status = p.status;
    const int per_row = (int)((pr->k + 15) / 16);
    if (pl.out_a) q.part[0] = {p.a, ws + pl.off_a, pr->m * per_row, pr->m * pr->k, per_row, pl.half_a};
    if (pl.out_w) q.part[1] = {p.w, ws + pl.off_w, pr->n * per_row, pr->n * pr->k, per_row, pl.half_w};
    long long grid = (q.part[0].groups + q.part[1].groups + 255) / 256;
    const long long most = (long long)device_sm_count() * 16;
    if (grid > most) grid = most;
    set_kernel_name("scaled_matmul_pack");
    prof_before(s);
    pack_rows_kernel<<<(unsigned)grid, 256, 0, s>>>(q);
    e = cudaGetLastError();
    prof_after(s);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
  }
  const bool fp8 = pr->format == SSD_CACHE_E4M3, b16 = pr->out_dtype == SSD_BF16;
  prof_before(s);
  e = fp8 ? (b16 ? launch_product<true, __nv_bfloat16>(pl, p, ra, rw, s) : launch_product<true, float>(pl, p, ra, rw, s))
          : (b16 ? launch_product<false, __nv_bfloat16>(pl, p, ra, rw, s)
                 : launch_product<false, float>(pl, p, ra, rw, s));
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
