// k_delta_chain.cu -- the state's way through the chunks of the gated delta
// rule (see delta_internal.cuh for the formulas, k_delta_prep.cu for T, A and
// the gates).
//
// The columns of the state (values of headdim) are independent of each other,
// and everything a column's chain needs besides its own v is shared: so one
// warp keeps 16 columns, transposed, as the fp32 accumulators of a product
// with 16 rows, and walks the chunks by itself.  Written transposed, every
// product of the chain takes the last one's result as its left operand
// straight from registers (an accumulator's layout is a left operand's
// layout), and its right operand -- K, T, Q or A -- from shared memory:
//
//   forward   R' = V' - e (S' K')    w' = R' (I + M)'^-1    S' = e_last S' + (o beta w)' K
//             y' = scale e (S' Q') + w' A'
//   reverse   R' = o beta (D' K') + dY' A    r' = R' (I + M)^-1
//             D' = e_last D' + (scale e dY)' Q - (e r)' K
//
// The solves go by blocks of 16 tokens: each block takes the earlier (reverse:
// later) ones' share of M, then its own inverse; T holds -M and those inverses
// less their unit diagonals, which pass the accumulators through in fp32.
// The state's update and the next chunk's product with it are one stream of
// products, state tile by state tile, so that neither waits for the other's
// end.
//
// There is no barrier between warps on a chain and no state in shared memory.
// The forward hands each chunk's S' and w' (bf16) to a second warp, which
// forms y' off the chain's critical path; from the same tiles they leave for
// the backward.  One more warp issues the TMA copies of the next chunks.  (Output
// warps that take 32 columns of every other chunk read Q and A half as often, and
// were not faster: 232 us instead of 231 below, 236 instead of 227 packed.)
// Every operand of a product is rounded to bf16 on its way into it -- T and A, S',
// w', (o beta w)', D', r', (scale e dY)' -- because the tensor cores take no more:
// both halves of an operand would be three products for one, and twice the shared
// memory, on chains bound by both.  The accumulators, S and D among them, are fp32
// from the first chunk to the last, so the roundings do not add up along a row: y is
// 3.5e-3 off float64 in the 2-norm, where rounding y itself is 1.7e-3.
// Bound by a warp's own sequence of products (148 of 16 x 8 x 16 a chunk on one
// sub-partition's tensor pipe, 8 cycles each, between the solve's waits) and, with
// four column warps, by shared-memory reads of the right operands (about 70 KB
// per 16 columns and chunk; that pipe is busy for 73 % of the forward's cycles and
// 67 % of the reverse's, the tensor pipe for 62 and 65 %).  Measured at dstate 128:
// 1.69 us a chunk for 64 columns (batch 2, L = 8192, 64 heads: 217 us forward, 233
// with what the backward needs, 219 reverse), 1.24 for 32 and 1.18 for 16.
#include "delta_internal.cuh"
#include "mma_common.cuh"
#include "tma_host.h"

#include <type_traits>

namespace ssd {
namespace {

using namespace mm;
using namespace tc;

constexpr int kC = kDeltaChunk;
constexpr uint32_t kTile = kC * 128;  // a [64][64] bf16 tile, 128-byte swizzle
constexpr int kGateBytes = 2 * kC * 4;  // the chains read e and o beta

// Right operands from [64][64] tiles of a [64][64 * blocks] matrix.
__device__ __forceinline__ void ld_b(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
  load_b<8>(r, base + (uint32_t)(k0 >> 6) * kTile, n0, k0 & 63, lane);
}
__device__ __forceinline__ void ld_bt(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
  load_bt<8>(r, base + (uint32_t)(n0 >> 6) * kTile, n0 & 63, k0, lane);
}
// The left operand of rows k0.. from two accumulators
__device__ __forceinline__ void as_left(uint32_t (&a)[4], const float (&lo)[4], const float (&hi)[4]) {
  a[0] = pack2(lo[0], lo[1]);
  a[1] = pack2(lo[2], lo[3]);
  a[2] = pack2(hi[0], hi[1]);
  a[3] = pack2(hi[2], hi[3]);
}
// A [16][64 * blocks] bf16 tile (blocks of [16][64], 128-byte swizzle) in
// shared memory: where the fragment of columns k0.. goes
__device__ __forceinline__ uint32_t frag_at(uint32_t base, int k0, int lane) {
  return base + (uint32_t)(k0 >> 6) * 2048u + tile_off<8>(lane & 15, ((k0 & 63) >> 3) + (lane >> 4));
}
// Where the transposed fragment of 16 tokens from tok0 goes in a [64][16]
// tile of 32-byte rows
__device__ __forceinline__ uint32_t token_at(uint32_t base, int tok0, int lane) {
  return base + (uint32_t)(tok0 + ((lane >> 4) << 3) + (lane & 7)) * 32u + (uint32_t)((lane >> 3) & 1) * 16u;
}

template <int N>
__device__ __forceinline__ void load_state(float (&S)[N / 8][4], const void* src, long long base, int lane, int bf16) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      S[i][j] = src ? ld_state(src, base + (long long)((lane >> 2) + (j >> 1) * 8) * N + i * 8 + 2 * (lane & 3) + (j & 1), bf16)
                    : 0.f;
}
template <int N>
__device__ __forceinline__ void store_state(const float (&S)[N / 8][4], void* dst, long long base, int lane, int bf16) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const long long o = base + (long long)((lane >> 2) + 8 * r) * N + i * 8 + 2 * (lane & 3);
      if (bf16)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(dst) + o) = pack2(S[i][2 * r], S[i][2 * r + 1]);
      else
        *reinterpret_cast<float2*>(static_cast<float*>(dst) + o) = make_float2(S[i][2 * r], S[i][2 * r + 1]);
    }
}

// A chunk token by token, by the definition alone.  The chunk's products
// multiply what a token must not see by zero, which does not hide an infinity or
// a NaN from it.  In a chunk without a sequence's start that stays in the
// sequence and in the chunk; where one starts (no state passes through), and the
// result is not finite, the chunk is done again here, one warp's 16 columns as
// in the products' accumulators, from the operands in global memory.
template <int M>
__device__ __forceinline__ bool all_finite(const float (&v)[M][4]) {
  bool fine = true;
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) fine &= fabsf(v[i][j]) <= 3.402823466e38f;
  return __all_sync(0xffffffffu, fine);
}
// the same of a [64][16] bf16 tile
__device__ __forceinline__ bool all_finite_tile(uint32_t tile, int lane) {
  bool fine = true;
  for (int i = lane; i < kC * 2; i += 32) {
    const uint4 v = lds128(tile + i * 16);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) fine &= (u[j] & 0x7f80u) != 0x7f80u && (u[j] & 0x7f800000u) != 0x7f800000u;
  }
  return __all_sync(0xffffffffu, fine);
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ void sts16(uint32_t addr, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&b)) : "memory");
}
// Since such a chunk is rare, and the tests for it would cost every chain a
// tenth of its time, they are left to a second pass over the chain's chunks, made
// where the first one gave a value that is not finite and met a sequence's start.
enum { kNotFinite = 1, kExpired = 2 };
// seen += x 0, a product like the others: NaN from the first x on that is not finite
__device__ __forceinline__ void watch(float (&seen)[4], const uint32_t (&x)[4]) { mma(seen, x, 0u, 0u); }
__device__ __forceinline__ bool met_not_finite(const float (&seen)[4]) {
  return __any_sync(0xffffffffu, !(seen[0] + seen[1] + seen[2] + seen[3] == 0.f));
}
// Whether a sequence begins in one of n chunks, or the state is forgotten there (e: the first one's gate record)
__device__ __forceinline__ bool any_start(const float* e, int n, int lane) {
  bool cut = false;
  for (int c = lane; c < n; c += 32)
    cut |= reinterpret_cast<const int*>(e + ((long long)c * kGateRows + kGateSeg) * kC)[kC - 1] != 0;
  return __any_sync(0xffffffffu, cut);
}
struct Walk {
  const DeltaPlan& p;
  const DeltaBufs& f;
  int bi, h, c, col, lane;  // col: the warp's first column of headdim
  struct Gate {
    float a, beta;
    bool starts;  // the token does not see the state before it
  };
  __device__ __forceinline__ long long token(int i) const { return (long long)bi * p.L + c * kC + i; }
  __device__ __forceinline__ int tokens() const { return min(kC, p.L - c * kC); }
  __device__ __forceinline__ Gate gate(int i) const {
    const long long tok = token(i), o = tok * p.H + h;
    const float g = to_f(static_cast<const __nv_bfloat16*>(f.g)[o]);
    const bool cut = f.seq != nullptr && c * kC + i > 0 && f.seq[tok] != f.seq[tok - 1];
    return {expf(g), to_f(static_cast<const __nv_bfloat16*>(f.beta)[o]), cut || g < kForget};
  }
  // this lane's values of a row of q or k, eight columns apart
  __device__ __forceinline__ const uint32_t* row(const void* x, long long stride, int N, int i) const {
    return reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(x) + token(i) * stride +
                                             (long long)(h / p.hpg) * N) + (lane & 3);
  }
  // and of v or dy: columns lane / 4 and eight further
  __device__ __forceinline__ float2 column(const void* x, long long stride, int i) const {
    const __nv_bfloat16* v =
        static_cast<const __nv_bfloat16*>(x) + token(i) * stride + (long long)h * p.P + col + (lane >> 2);
    return make_float2(to_f(v[0]), to_f(v[8]));
  }
  template <int N>
  __device__ __forceinline__ void state_from(float (&S)[N / 8][4], uint32_t tile) const {
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks) {
      uint32_t a[4];
      ldsm4(a, frag_at(tile, 16 * ks, lane));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2(a[j]);
        S[2 * ks + (j >> 1)][2 * (j & 1)] = v.x;
        S[2 * ks + (j >> 1)][2 * (j & 1) + 1] = v.y;
      }
    }
  }
  // S'x for the two columns: the row's products over dstate
  template <int N>
  __device__ __forceinline__ float2 dot(const float (&S)[N / 8][4], const uint32_t* x) const {
    float2 d = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
      const float2 v = unpack2(x[4 * j]);
      d.x += S[j][0] * v.x + S[j][1] * v.y;
      d.y += S[j][2] * v.x + S[j][3] * v.y;
    }
    return make_float2(quad_sum(d.x), quad_sum(d.y));
  }
  template <int N>
  __device__ __forceinline__ void add(float (&S)[N / 8][4], float2 u, const uint32_t* x) const {
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
      const float2 v = unpack2(x[4 * j]);
      S[j][0] += u.x * v.x;
      S[j][1] += u.x * v.y;
      S[j][2] += u.y * v.x;
      S[j][3] += u.y * v.y;
    }
  }
  template <int N>
  __device__ __forceinline__ void decay(float (&S)[N / 8][4], const Gate& x) const {
#pragma unroll
    for (int j = 0; j < N / 8; ++j)
#pragma unroll
      for (int m = 0; m < 4; ++m) S[j][m] = x.starts ? 0.f : x.a * S[j][m];
  }
  // Forward from the state in `tile`: the state S after the chunk and, with kOut,
  // y into a [64][16] tile
  template <int N, bool kOut>
  __device__ __forceinline__ void forward(float (&S)[N / 8][4], uint32_t tile, uint32_t out) const {
    state_from<N>(S, tile);
    const int n = tokens();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const Gate x = gate(i);
      const uint32_t* k = row(f.k, p.ks, N, i);
      const float2 v = column(f.v, p.vs, i);
      decay<N>(S, x);
      const float2 d = dot<N>(S, k);
      add<N>(S, make_float2(x.beta * (v.x - d.x), x.beta * (v.y - d.y)), k);
      if (kOut) {
        const float2 y = dot<N>(S, row(f.q, p.qs, N, i));
        if ((lane & 3) == 0) {
          sts16(out + i * 32 + (lane >> 2) * 2, p.scale * y.x);
          sts16(out + i * 32 + (lane >> 2) * 2 + 16, p.scale * y.y);
        }
      }
    }
  }
  // Reverse from the gradient of the state after the chunk (in `tile`, or zeros):
  // the gradient D of the one before it, and r into a [64][16] tile
  template <int N>
  __device__ __forceinline__ void reverse(float (&D)[N / 8][4], uint32_t tile, bool zeros, uint32_t out) const {
    state_from<N>(D, tile);
#pragma unroll
    for (int j = 0; j < N / 8; ++j)
#pragma unroll
      for (int m = 0; m < 4; ++m) D[j][m] = zeros ? 0.f : D[j][m];
#pragma unroll 1
    for (int i = tokens() - 1; i >= 0; --i) {
      const Gate x = gate(i);
      const uint32_t* k = row(f.k, p.ks, N, i);
      const float2 y = column(f.dy, (long long)p.H * p.P, i);
      add<N>(D, make_float2(p.scale * y.x, p.scale * y.y), row(f.q, p.qs, N, i));
      const float2 d = dot<N>(D, k), r = make_float2(x.beta * d.x, x.beta * d.y);
      add<N>(D, make_float2(-r.x, -r.y), k);
      decay<N>(D, x);
      if ((lane & 3) == 0) {
        sts16(out + i * 32 + (lane >> 2) * 2, r.x);
        sts16(out + i * 32 + (lane >> 2) * 2 + 16, r.y);
      }
    }
  }
};

struct ChainMaps {
  CUtensorMap q, k, v, T, A, y, S, w;  // reverse: v is dy, y is dv, S is D
};

// A packed row's chain in pieces.  Where a sequence begins inside a chunk (a
// cut), the state that leaves the chunk does not depend on the one that enters
// it, nor the gradient that leaves it to the left on the one from the right.  So
// piece z begins at the cut nearest to z / pieces of the chunks, from zeros, and
// goes through the next piece's first chunk; what that chunk's columns give is
// written by the one of the two pieces that enters it with its neighbour's state
// (or gradient).
//
// The host cannot see the cuts.  A CTA that takes a piece has twice the columns
// that it would have of a whole chain (see chain_shape), and where a row's cuts
// leave one piece nearly the whole chain, that is a loss: then the row's first two
// CTAs take the whole chain, half of the column warps each, and the others end.
struct Piece {
  int first, next;  // its first chunk, and the next piece's (or nc)
  int z;            // its number; 0 where it begins with the row
  int warp0, warps; // the column warps at work
  __device__ __forceinline__ bool has(int w) const { return w >= warp0 && w < warp0 + warps; }
};
// The cut nearest to chunk `mid`, or nc; e: the gate records.  (128 chunks to
// either side at a time: a row without cuts is searched to its ends.)
__device__ __forceinline__ int near_cut(const float* e, int mid, int nc, int lane) {
  // (the segment of a chunk's last token, counted from the chunk's start)
  auto cut = [&](int c) {
    const bool in = c >= 0 && c < nc;
    return in && reinterpret_cast<const int*>(e + ((long long)c * kGateRows + kGateSeg) * kC)[kC - 1] != 0;
  };
  for (int d0 = 0; d0 < nc; d0 += 128) {
    bool below[4], above[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      below[u] = cut(mid - d0 - 32 * u - lane);
      above[u] = cut(mid + d0 + 32 * u + lane);
    }
    for (int u = 0; u < 4; ++u) {
      const unsigned lo = __ballot_sync(0xffffffffu, below[u]), hi = __ballot_sync(0xffffffffu, above[u]);
      if (lo | hi) {
        const int l = __ffs(lo | hi) - 1, d = d0 + 32 * u + l;
        return lo >> l & 1 ? mid - d : mid + d;
      }
    }
  }
  return nc;
}
template <int NW>
__device__ __forceinline__ Piece find_piece(const float* e, int z, int pieces, int nc, int lane) {
  auto cut = [&](int i) {
    return i <= 0 ? 0 : i < pieces ? near_cut(e, (int)((long long)i * nc / pieces), nc, lane) : nc;
  };
  if (NW > 1) {  // two or three pieces
    const int c1 = cut(1), c2 = cut(2);
    const int largest = max(max(min(c1 + 1, nc), min(c2 + 1, nc) - c1), nc - c2);
    // (a chunk of 64 columns takes 1.37 times as long as one of 32, one of 32 1.05 times as long as one of 16)
    if (NW == 4 ? largest * 4 > nc * 3 : largest * 16 > nc * 15) return {0, nc, 0, z * (NW / 2), z < 2 ? NW / 2 : 0};
    return {z == 0 ? 0 : z == 1 ? c1 : c2, z == 0 ? c1 : z == 1 ? c2 : nc, z, 0, NW};
  }
  return {cut(z), cut(z + 1), z, 0, NW};
}

// NW column warps: 16 NW columns a CTA
template <int N, int NW>
struct FwdSmem {
  static constexpr int kK = kC * N * 2, kV = kC * NW * 32;
  // the chain's ring: K, T, V, gates, three deep (a chunk's K is in use until
  // the next one's has been); the output warps': Q, A, gates, two deep
  static constexpr int chain = kK + (int)kTile + kV, out = kK + (int)kTile;
  static constexpr int oChain = 0, oOut = oChain + 3 * chain, oS = oOut + 2 * out,  // S' by warp, two each
                       oW = oS + NW * 2 * N * 32, oY = oW + NW * 2 * 2048, oE = oY + NW * 2 * 2048,
                       oBar = oE + 5 * kGateBytes, oPlace = oBar + (10 + 4 * NW) * 8, bytes = oPlace + 64 + 1024;
};

// Column, output and copying warps.  Nine warps would leave each 168 registers
// (three on one sub-partition), which the chain's loads need more than:
// registers are handed over by groups of four warps, so three idle ones join
// the copying warp (launched with 168 each: 240 + 208 + 40 <= 3 x 168).
constexpr int fwd_threads(int nw) { return nw == 4 ? 384 : (2 * nw + 1) * 32; }
// The column warp whose outputs warp w forms: not one of its own sub-partition, so
// that half of the column warps and their output warps have all four.
__device__ __forceinline__ int output_columns(int w, int nw) { return (w - nw) ^ (nw / 2); }

// A forward chain's CTA: its columns and its chunks
struct FwdPlace {
  int bi, h, p0, z, first, nch;
  bool last_of_row;
};
template <int N, int NW>
struct FwdChain {
  using L = FwdSmem<N, NW>;
  const DeltaPlan& p;
  const DeltaBufs& f;
  unsigned char* raw;
  uint32_t sm;
  uint64_t* bars;
  int w, lane;
  bool ok;
  int bi, h, p0, z, first, nch, bh;
  bool last_of_row;
  __device__ __forceinline__ FwdChain(const DeltaPlan& p, const DeltaBufs& f, unsigned char* raw, const FwdPlace& at)
      : p(p), f(f), raw(raw), sm(smem_u32(raw)), bars(reinterpret_cast<uint64_t*>(raw + L::oBar)),
        w(threadIdx.x >> 5), lane(threadIdx.x & 31), ok(true), bi(at.bi), h(at.h), p0(at.p0), z(at.z), first(at.first),
        nch(at.nch), bh(at.bi * p.H + at.h), last_of_row(at.last_of_row) {}
  __device__ __forceinline__ const float* gates() const {
    return static_cast<const float*>(f.e) + (long long)bh * p.nc * kGateRows * kC;
  }

  // The column warps' part; kGuard: the second pass
  template <bool kGuard>
  __device__ __forceinline__ void columns() {
    uint64_t *c_full = bars, *c_free = bars + 3, *h_full = bars + 10, *h_free = h_full + 2 * NW;
    const int t = lane & 3;
    const bool saves = f.S != nullptr;
    const long long state0 = ((long long)bh * p.P + p0 + 16 * w) * N;
    float S[N / 8][4], x[8][4];
    load_state<N>(S, z ? nullptr : f.init, state0, lane, p.st_bf16);
    int cs = 0, cph = 0;
    // S' K' for one 16-row step of K; the step's bf16 copy stays in `half` until
    // the products are under way (a store to shared memory would hold back
    // the loads of the next step's operands)
    uint32_t half[N / 16][4];
    auto state_product = [&](int ks, uint32_t Ks) {
      uint32_t b[4];
      as_left(half[ks], S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        ld_b(b, Ks, 8 * j, 16 * ks, lane);
        mma(x[j], half[ks], b[0], b[1]);
        mma(x[j + 1], half[ks], b[2], b[3]);
      }
    };
    auto put_state = [&](uint32_t Sd) {
#pragma unroll
      for (int ks = 0; ks < N / 16; ++ks)
        stsm4(frag_at(Sd, 16 * ks, lane), half[ks][0], half[ks][1], half[ks][2], half[ks][3]);
    };
    auto zero = [](float(&v)[8][4]) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
    };
    mbar_wait_flag(c_full, 0, ok);
    zero(x);
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks) state_product(ks, sm + L::oChain);
    put_state(sm + L::oS + 2 * w * N * 32);
    // from x = S' K' of a chunk its w', handed to the output warp, and (o beta w)' as left operands
    uint32_t left[4][4];
    auto solve = [&](int c) {
      const int st = c & 1;
      const uint32_t Ts = sm + L::oChain + cs * L::chain + L::kK, Vs = Ts + kTile;
      const uint32_t Wd = sm + L::oW + (2 * w + st) * 2048;
      const float* e = reinterpret_cast<const float*>(raw + L::oE + cs * kGateBytes) + 2 * t;
      // all the operands before the first product that waits for another
      uint32_t v[4][4], tb[10][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        load_at<2 * NW>(v[k], Vs, 16 * w, 16 * k, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k <= i; ++k) ld_b(tb[i * (i + 1) / 2 + k], Ts, 16 * i, 16 * k, lane);
      // R' = V' - e (S' K')
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 ej = *reinterpret_cast<const float2*>(e + 16 * k + 8 * j);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 vv = unpack2(v[k][2 * j + r]);
            float(&xx)[4] = x[2 * k + j];
            xx[2 * r] = vv.x - ej.x * xx[2 * r];
            xx[2 * r + 1] = vv.y - ej.y * xx[2 * r + 1];
          }
        }
      // w' block by block: its own inverse, then its share of the later blocks
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t(&d)[4] = tb[k * (k + 1) / 2 + k];
        as_left(left[k], x[2 * k], x[2 * k + 1]);
        mma(x[2 * k], left[k], d[0], d[1]);
        mma(x[2 * k + 1], left[k], d[2], d[3]);
        as_left(left[k], x[2 * k], x[2 * k + 1]);
#pragma unroll
        for (int i = k + 1; i < 4; ++i) {
          const uint32_t(&b)[4] = tb[i * (i + 1) / 2 + k];
          mma(x[2 * i], left[k], b[0], b[1]);
          mma(x[2 * i + 1], left[k], b[2], b[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        stsm4(frag_at(Wd, 16 * k, lane), left[k][0], left[k][1], left[k][2], left[k][3]);
      if (saves) fence_async_smem();  // the tiles also leave through TMA
      __syncwarp();
      if (lane == 0) mbar_arrive(h_full + 2 * w + st);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 o = *reinterpret_cast<const float2*>(e + kGateOB * kC + 16 * k + 8 * j);
          float(&xx)[4] = x[2 * k + j];
          xx[0] *= o.x;
          xx[1] *= o.y;
          xx[2] *= o.x;
          xx[3] *= o.y;
        }
        as_left(left[k], x[2 * k], x[2 * k + 1]);
      }
    };
    auto update = [&](int i, uint32_t Ks, float last) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[2 * i][j] *= last;
        S[2 * i + 1][j] *= last;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t b[4];
        ld_bt(b, Ks, 16 * i, 16 * k, lane);
        mma(S[2 * i], left[k], b[0], b[1]);
        mma(S[2 * i + 1], left[k], b[2], b[3]);
      }
    };
    // chunk c again token by token, from the state that the output warp also has
    auto walk = [&](int c) {
      Walk{p, f, bi, h, first + c, p0 + 16 * w, lane}.template forward<N, false>(
          S, sm + L::oS + (2 * w + (c & 1)) * N * 32, 0);
    };
    for (int c = 0; c + 1 < nch; ++c) {
      const int st = c & 1, ns = cs == 2 ? 0 : cs + 1;
      const uint32_t Ks = sm + L::oChain + cs * L::chain;
      const uint32_t Kn = sm + L::oChain + ns * L::chain, Sn = sm + L::oS + (2 * w + (st ^ 1)) * N * 32;
      solve(c);
      const float last = reinterpret_cast<const float*>(raw + L::oE + cs * kGateBytes)[kC - 1];
      mbar_wait_flag(c_full + ns, ns ? cph : cph ^ 1, ok);
      if (c >= 1) mbar_wait_flag(h_free + 2 * w + (st ^ 1), ((c - 1) >> 1) & 1, ok);
      // S' = e_last S' + (o beta w)' K, each pair of tiles followed by the
      // next chunk's product with the pair before
      zero(x);
      update(0, Ks, last);
#pragma unroll
      for (int i = 1; i < N / 16; ++i) {
        update(i, Ks, last);
        state_product(i - 1, Kn);
      }
      state_product(N / 16 - 1, Kn);
      if (*reinterpret_cast<const float*>(raw + L::oE + ns * kGateBytes) == 0.f) {
        // the next chunk starts a sequence: it does not read the state, whatever that holds
        zero(x);
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) S[i][j] = 0.f;
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) half[ks][0] = half[ks][1] = half[ks][2] = half[ks][3] = 0u;
      } else if (kGuard && last == 0.f && !all_finite(S)) {
        walk(c);
        zero(x);
#pragma unroll
        for (int i = 0; i < N / 16; ++i) state_product(i, Kn);
      }
      put_state(Sn);
      __syncwarp();
      if (lane == 0) mbar_arrive(c_free + cs);
      cs = ns;
      if (ns == 0) cph ^= 1;
    }
    solve(nch - 1);
    const bool last_piece = last_of_row;
    if (f.fin && last_piece) {
      const float last = reinterpret_cast<const float*>(raw + L::oE + cs * kGateBytes)[kC - 1];
#pragma unroll
      for (int i = 0; i < N / 16; ++i) update(i, sm + L::oChain + cs * L::chain, last);
      if (kGuard && last == 0.f && !all_finite(S)) walk(nch - 1);
    }
    if (f.fin && last_piece) store_state<N>(S, f.fin, state0, lane, p.st_bf16);
  }

  // The output warps' part (warp cw's columns); true where an output was not
  // finite and a sequence begins
  template <bool kGuard>
  __device__ __forceinline__ bool outputs(const ChainMaps& m, int cw) {
    uint64_t *o_full = bars + 6, *o_free = bars + 8, *h_full = bars + 10, *h_free = h_full + 2 * NW;
    const int t = lane & 3;
    const bool saves = f.S != nullptr;
    const float scale = p.scale;
    float seen[4] = {};  // NaN once an output was not finite
    for (int k = 0; k < nch; ++k) {
      const int st = k & 1, c = first + k;
      const bool write = k > 0 || z == 0;
      const uint32_t Qs = sm + L::oOut + st * L::out, As = Qs + L::kK;
      const uint32_t Sd = sm + L::oS + (2 * cw + st) * N * 32, Wd = sm + L::oW + (2 * cw + st) * 2048;
      const uint32_t Yd = sm + L::oY + (2 * cw + st) * 2048;
      const float* e = reinterpret_cast<const float*>(raw + L::oE + (3 + st) * kGateBytes) + 2 * t;
      mbar_wait_flag(o_full + st, (k >> 1) & 1, ok);
      mbar_wait_flag(h_full + 2 * cw + st, (k >> 1) & 1, ok);
      if (saves && write && lane == 0) {
        for (int j = 0; j < N / 64; ++j)
          tma_store_4d(&m.S, raw + (Sd - sm) + j * 2048, 64 * j, p0 + 16 * cw, c, bh);
        tma_store_4d(&m.w, raw + (Wd - sm), 0, p0 + 16 * cw, c, bh);
        bulk_commit();
      }
      float y[8][4] = {};
#pragma unroll
      for (int ks = 0; ks < N / 16; ++ks) {
        uint32_t a[4], b[4];
        ldsm4(a, frag_at(Sd, 16 * ks, lane));
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          ld_b(b, Qs, 8 * j, 16 * ks, lane);
          mma(y[j], a, b[0], b[1]);
          mma(y[j + 1], a, b[2], b[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 ej = *reinterpret_cast<const float2*>(e + 8 * j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          y[j][2 * r] *= scale * ej.x;
          y[j][2 * r + 1] *= scale * ej.y;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4], b[4];
        ldsm4(a, frag_at(Wd, 16 * k, lane));
#pragma unroll
        for (int i = k; i < 4; ++i) {
          ld_b(b, As, 16 * i, 16 * k, lane);
          mma(y[2 * i], a, b[0], b[1]);
          mma(y[2 * i + 1], a, b[2], b[3]);
        }
      }
      const bool cut = kGuard && e[kC - 1 - 2 * t] == 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free + st);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4];
        as_left(a, y[2 * k], y[2 * k + 1]);
        if (!kGuard) watch(seen, a);
        stsm4t(token_at(Yd, 16 * k, lane), a[0], a[1], a[2], a[3]);
      }
      if (cut) {
        __syncwarp();
        if (!all_finite_tile(Yd, lane)) {
          float S[N / 8][4];
          Walk{p, f, bi, h, c, p0 + 16 * cw, lane}.template forward<N, true>(S, Sd, Yd);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (write) tma_store_4d(&m.y, raw + (Yd - sm), p0 + 16 * cw, h, c * kC, bi);
        bulk_commit();
        bulk_wait_read<1>();  // all but this chunk's y have been read: its S', w' and the last y's tile are free
        mbar_arrive(h_free + 2 * cw + st);
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    return !kGuard && met_not_finite(seen) && any_start(gates() + (long long)first * kGateRows * kC, nch, lane);
  }
};
// The second pass, as calls that need nothing but the CTA's place in shared
// memory (batch 2, L = 8192, 64 heads: 217 us for the first pass so, 213 without
// a second one, 229 inlined, and 239 to 265 with the tests and walks in one pass
// for all).
__device__ __forceinline__ unsigned char* chain_smem() {
  extern __shared__ unsigned char raw_[];
  return raw_ + ((1024 - (smem_u32(raw_) & 1023)) & 1023);
}
template <int N, int NW>
__device__ __noinline__ bool columns_again(const DeltaPlan& p, const DeltaBufs& f) {
  unsigned char* raw = chain_smem();
  FwdChain<N, NW> x(p, f, raw, *reinterpret_cast<const FwdPlace*>(raw + FwdSmem<N, NW>::oPlace));
  x.template columns<true>();
  return x.ok;
}
template <int N, int NW>
__device__ __noinline__ bool outputs_again(const DeltaPlan& p, const DeltaBufs& f, const ChainMaps& m) {
  unsigned char* raw = chain_smem();
  FwdChain<N, NW> x(p, f, raw, *reinterpret_cast<const FwdPlace*>(raw + FwdSmem<N, NW>::oPlace));
  x.template outputs<true>(m, output_columns(x.w, NW));
  return x.ok;
}

// By every warp of a CTA at its first pass's end (redo: what they found): whether
// there is a second one, with the barriers as at the start
template <typename Init>
__device__ __forceinline__ bool chain_again(int& redo, bool ok, uint64_t* bars, int nbars, int threads, Init init) {
  if (!ok) atomicOr(&redo, kExpired);
  bar_sync(0, threads);
  const bool again = redo == kNotFinite;
  if (again) {
    if (threadIdx.x == threads - 1) {
      for (int i = 0; i < nbars; ++i) mbar_inval(bars + i);
      init();
    }
    bar_sync(0, threads);
  }
  return again;
}

template <int N, int NW, bool kPieces>
__global__ void __launch_bounds__(fwd_threads(NW), 1)
    delta_chain_fwd_kernel(const __grid_constant__ DeltaPlan p, const __grid_constant__ DeltaBufs f, int pieces,
                           const __grid_constant__ ChainMaps m) {
  using L = FwdSmem<N, NW>;
  constexpr bool kHandOver = NW == 4;
  extern __shared__ unsigned char raw_[];
  unsigned char* raw = raw_ + ((1024 - (smem_u32(raw_) & 1023)) & 1023);
  const uint32_t sm = smem_u32(raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(raw + L::oBar);
  uint64_t *c_full = bars, *c_free = bars + 3, *o_full = bars + 6, *o_free = bars + 8;
  uint64_t *h_full = bars + 10, *h_free = h_full + 2 * NW;  // [warp][2]
  constexpr int kThreads = fwd_threads(NW), kBars = 10 + 4 * NW;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ptiles = p.P / (16 * NW);
  const int p0 = (int)(blockIdx.x % ptiles) * 16 * NW;
  const int h = (int)((blockIdx.x / ptiles) % p.H), row = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int bi = kPieces ? row % p.b : row;
  const int grp = h / p.hpg, bh = bi * p.H + h;
  const float* gates = static_cast<const float*>(f.e) + (long long)bh * p.nc * kGateRows * kC;
  __shared__ Piece piece_s;
  if (kPieces && w == 0) {
    const Piece found = find_piece<NW>(gates, row / p.b, pieces, p.nc, lane);
    if (lane == 0) piece_s = found;
  }
  __shared__ int redo_s;
  auto init_bars = [&]() {
    for (int i = 0; i < 3; ++i) {
      mbar_init(c_full + i, 1);
      mbar_init(c_free + i, kPieces ? max(piece_s.warps, 1) : NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(o_full + i, 1);
      mbar_init(o_free + i, kPieces ? max(piece_s.warps, 1) : NW);
    }
    for (int i = 0; i < 2 * NW; ++i) {
      mbar_init(h_full + i, 1);
      mbar_init(h_free + i, 1);
    }
    mbar_fence_init();
  };
  if (threadIdx.x == 0) {
    init_bars();
    redo_s = 0;
  }
  __syncthreads();
  const Piece piece = kPieces ? piece_s : Piece{0, p.nc, 0, 0, NW};
  const int z = piece.z;
  if ((z && piece.first >= piece.next) || piece.warps == 0) return;  // no cut of its own, or nothing left
  // its chunks; a later piece gives no outputs for its first one
  const int first = piece.first, nch = min(piece.next + 1, p.nc) - first;
  const FwdPlace here = {bi, h, p0, z, first, nch, piece.next == p.nc};
  if (threadIdx.x == 0) *reinterpret_cast<FwdPlace*>(raw + L::oPlace) = here;
  FwdChain<N, NW> x(p, f, raw, here);
  bool& ok = x.ok;
  // Every warp has ended its first pass: whether there is to be a second one
  auto again = [&]() { return chain_again(redo_s, ok, bars, kBars, kThreads, init_bars); };
  if (w >= 2 * NW) {
    if (kHandOver) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    auto copies = [&]() {
      int cs = 0, cph = 0;  // the chain's ring position and phase
      for (int k = 0; k < nch; ++k) {
        const int st = k & 1, c = first + k;
        if (k >= 3) mbar_wait_flag(c_free + cs, cph ^ 1, ok);
        unsigned char* d = raw + L::oChain + cs * L::chain;
        mbar_expect_tx(c_full + cs, L::chain + kGateBytes);
        tma_load_4d(d, &m.k, c_full + cs, 0, c * kC, grp * (N / 64), bi);
        tma_load_4d(d + L::kK, &m.T, c_full + cs, 0, 0, c, bh);
        tma_load_4d(d + L::kK + kTile, &m.v, c_full + cs, p0, h, c * kC, bi);
        bulk_load(raw + L::oE + cs * kGateBytes, gates + (long long)c * kGateRows * kC, kGateBytes, c_full + cs);
        if (++cs == 3) cs = 0, cph ^= 1;
        if (k >= 2) mbar_wait_flag(o_free + st, ((k >> 1) - 1) & 1, ok);
        d = raw + L::oOut + st * L::out;
        mbar_expect_tx(o_full + st, L::out + kGateBytes);
        tma_load_4d(d, &m.q, o_full + st, 0, c * kC, grp * (N / 64), bi);
        tma_load_4d(d + L::kK, &m.A, o_full + st, 0, 0, c, bh);
        bulk_load(raw + L::oE + (3 + st) * kGateBytes, gates + (long long)c * kGateRows * kC, kGateBytes, o_full + st);
      }
    };
    const bool copies_here = w == 2 * NW && lane == 0;
    if (copies_here) copies();
    __syncwarp();
    if (again() && copies_here) copies();
  } else if (w < NW) {
    if (kHandOver) asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    const bool live = !kPieces || piece.has(w);
    if (live) x.template columns<false>();
    if (again() && live) ok = columns_again<N, NW>(p, f);
  } else {
    if (kHandOver) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int cw = output_columns(w, NW);
    const bool live = !kPieces || piece.has(cw);
    if (live && x.template outputs<false>(m, cw)) atomicOr(&redo_s, kNotFinite);
    __syncwarp();
    if (again() && live) ok = outputs_again<N, NW>(p, f, m);
  }
  if (!ok) atomicOr(f.status, kDevTimeout);
}

template <int N, int NW>
struct RevSmem {
  static constexpr int kK = kC * N * 2, kV = kC * NW * 32;
  // a ring three deep of K, Q, T, A, dY, gates; D' and r by warp
  static constexpr int stage = 2 * kK + 2 * (int)kTile + kV;
  static constexpr int oSt = 0, oD = oSt + 3 * stage, oR = oD + NW * N * 32, oE = oR + NW * 2048,
                       oBar = oE + 3 * kGateBytes, oPlace = oBar + 6 * 8, bytes = oPlace + 64 + 1024;
};


// A reverse chain's CTA: its columns and its chunks, `right` the first of them
struct RevPlace {
  int bi, h, p0, z, right, nch;
  bool inner;
};
template <int N, int NW>
struct RevChain {
  using L = RevSmem<N, NW>;
  const DeltaPlan& p;
  const DeltaBufs& f;
  unsigned char* raw;
  uint32_t sm;
  int w, lane;
  bool ok;
  int bi, h, p0, z, right, nch, bh;
  bool inner;
  __device__ __forceinline__ RevChain(const DeltaPlan& p, const DeltaBufs& f, unsigned char* raw, const RevPlace& at)
      : p(p), f(f), raw(raw), sm(smem_u32(raw)), w(threadIdx.x >> 5), lane(threadIdx.x & 31), ok(true), bi(at.bi),
        h(at.h), p0(at.p0), z(at.z), right(at.right), nch(at.nch), bh(at.bi * p.H + at.h), inner(at.inner) {}
  __device__ __forceinline__ const float* gates() const {
    return static_cast<const float*>(f.e) + (long long)bh * p.nc * kGateRows * kC;
  }

  // The column warps' part (kGuard: the second pass); true where a value was not
  // finite and a sequence begins
  template <bool kGuard>
  __device__ __forceinline__ bool columns(const ChainMaps& m) {
    uint64_t *full = reinterpret_cast<uint64_t*>(raw + L::oBar), *empty = full + 3;
    const int t = lane & 3;
    const float scale = p.scale;
    // Whether a value was not finite: an r that is not leaves no column of D finite,
    // and D stays so up to a chunk whose first token starts a sequence, or to the end
    bool bad = false;
    const long long state0 = ((long long)bh * p.P + p0 + 16 * w) * N;
    float D[N / 8][4], x[8][4];
    load_state<N>(D, inner ? nullptr : f.dfin, state0, lane, p.st_bf16);
    // one 16-row step of D' K'; the step's bf16 copy for the gradient kernel stays in `half`
    uint32_t half[N / 16][4];
    auto state_product = [&](int ks, uint32_t Ks) {
      uint32_t b[4];
      as_left(half[ks], D[2 * ks], D[2 * ks + 1]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        ld_b(b, Ks, 8 * j, 16 * ks, lane);
        mma(x[j], half[ks], b[0], b[1]);
        mma(x[j + 1], half[ks], b[2], b[3]);
      }
    };
    auto zero = [](float(&v)[8][4]) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
    };
    // r' of chunk c (but for the first call) and D' after chunk c - 1 leave through TMA
    const uint32_t Dd = sm + L::oD + w * N * 32, Rd = sm + L::oR + w * 2048;
    uint32_t rk[4][4];
    auto put_r = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k) stsm4t(token_at(Rd, 16 * k, lane), rk[k][0], rk[k][1], rk[k][2], rk[k][3]);
    };
    auto put = [&](int c, bool with_r, bool with_d, bool walked = false) {
      if (lane == 0) bulk_wait_read<0>();  // the tiles' last contents have been read
      __syncwarp();
      if (with_r && !walked) put_r();
      if (with_d)
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks)
          stsm4(frag_at(Dd, 16 * ks, lane), half[ks][0], half[ks][1], half[ks][2], half[ks][3]);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (with_r) tma_store_4d(&m.y, raw + (Rd - sm), p0 + 16 * w, h, c * kC, bi);
        if (with_d)
          for (int j = 0; j < N / 64; ++j)
            tma_store_4d(&m.S, raw + (Dd - sm) + j * 2048, 64 * j, p0 + 16 * w, c - 1, bh);
        bulk_commit();
      }
    };
    int st = 0, ph = 0;
    mbar_wait_flag(full, 0, ok);
    zero(x);
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks) state_product(ks, sm + L::oSt);
    if (!inner) put(p.nc, false, true);
    // from x = D' K' of a chunk its r' (rk), its gradient's part of D', and (-e r)' as left operands
    uint32_t left[4][4];
    auto solve = [&]() {
      const uint32_t Qs = sm + L::oSt + st * L::stage + L::kK, Ts = Qs + L::kK, As = Ts + kTile, Ys = As + kTile;
      const float* e = reinterpret_cast<const float*>(raw + L::oE + st * kGateBytes) + 2 * t;
      const float last = e[kC - 1 - 2 * t];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 o = *reinterpret_cast<const float2*>(e + kGateOB * kC + 8 * j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[j][2 * r] *= o.x;
          x[j][2 * r + 1] *= o.y;
        }
      }
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) D[i][j] *= last;
      // R' += dY' A, and the part of D' that does not wait for r: (scale e dY)' Q
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        uint32_t y[4], b[4];
        load_at<2 * NW>(y, Ys, 16 * w, 16 * i, lane);
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          load_bt<8>(b, As, 16 * j, 16 * i, lane);
          mma(x[2 * j], y, b[0], b[1]);
          mma(x[2 * j + 1], y, b[2], b[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 ej = *reinterpret_cast<const float2*>(e + 16 * i + 8 * j);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 v = unpack2(y[2 * j + r]);
            y[2 * j + r] = pack2(scale * ej.x * v.x, scale * ej.y * v.y);
          }
        }
#pragma unroll
        for (int n = 0; n < N / 8; n += 2) {
          ld_bt(b, Qs, 8 * n, 16 * i, lane);
          mma(D[n], y, b[0], b[1]);
          mma(D[n + 1], y, b[2], b[3]);
        }
      }
      // r' block by block from the last
      uint32_t tb[10][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) load_bt<8>(tb[i * (i + 1) / 2 + j], Ts, 16 * j, 16 * i, lane);
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const uint32_t(&d)[4] = tb[i * (i + 1) / 2 + i];
        as_left(rk[i], x[2 * i], x[2 * i + 1]);
        mma(x[2 * i], rk[i], d[0], d[1]);
        mma(x[2 * i + 1], rk[i], d[2], d[3]);
        as_left(rk[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int j = i - 1; j >= 0; --j) {
          const uint32_t(&b)[4] = tb[i * (i + 1) / 2 + j];
          mma(x[2 * j], rk[i], b[0], b[1]);
          mma(x[2 * j + 1], rk[i], b[2], b[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 ej = *reinterpret_cast<const float2*>(e + 16 * k + 8 * j);
          float(&xx)[4] = x[2 * k + j];
          xx[0] *= -ej.x;
          xx[1] *= -ej.y;
          xx[2] *= -ej.x;
          xx[3] *= -ej.y;
        }
        as_left(left[k], x[2 * k], x[2 * k + 1]);
      }
    };
    auto update = [&](int i, uint32_t Ks) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t b[4];
        ld_bt(b, Ks, 16 * i, 16 * k, lane);
        mma(D[2 * i], left[k], b[0], b[1]);
        mma(D[2 * i + 1], left[k], b[2], b[3]);
      }
    };
    // a chunk whose first token starts a sequence has no gradient to pass on, whatever its values
    auto starts = [&]() { return *reinterpret_cast<const float*>(raw + L::oE + st * kGateBytes) == 0.f; };
    auto zero_state = [&]() {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) D[i][j] = 0.f;
    };
    // whether step k0's chunk was walked: r is in its tile and D is the gradient before the chunk
    auto walked_at = [&](int k0) {
      if (!kGuard || reinterpret_cast<const float*>(raw + L::oE + st * kGateBytes)[kC - 1] != 0.f ||
          (all_finite(x) && all_finite(D)))
        return false;
      if (lane == 0) bulk_wait_read<0>();  // the last r has been read
      __syncwarp();
      Walk{p, f, bi, h, right - k0, p0 + 16 * w, lane}.template reverse<N>(D, Dd, inner && k0 == 0, Rd);
      return true;
    };
    for (int k0 = 0; k0 + 1 < nch; ++k0) {
      const int c = right - k0, ns = st == 2 ? 0 : st + 1;
      const uint32_t Ks = sm + L::oSt + st * L::stage, Kn = sm + L::oSt + ns * L::stage;
      solve();
      const bool walked = walked_at(k0);
      mbar_wait_flag(full + ns, ns ? ph : ph ^ 1, ok);
      // D' += (-e r)' K, each pair of tiles followed by the next chunk's product with the pair before
      zero(x);
      if (walked) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) state_product(i, Kn);
      } else {
        update(0, Ks);
#pragma unroll
        for (int i = 1; i < N / 16; ++i) {
          update(i, Ks);
          state_product(i - 1, Kn);
        }
        state_product(N / 16 - 1, Kn);
      }
      if (starts()) {
        if (!kGuard) bad |= !all_finite(D);
        zero(x);
        zero_state();
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) half[ks][0] = half[ks][1] = half[ks][2] = half[ks][3] = 0u;
      }
      put(c, k0 > 0 || !inner, true, walked);
      if (lane == 0) mbar_arrive(empty + st);
      st = ns;
      if (ns == 0) ph ^= 1;
    }
    solve();
    if (!kGuard) bad |= !all_finite(x) || !all_finite(D);
    const bool walked = walked_at(nch - 1);
    if (nch > 1 || !inner) put(right + 1 - nch, true, false, walked);
    if (f.dinit && z == 0) {
      if (!walked)
#pragma unroll
        for (int i = 0; i < N / 16; ++i) update(i, sm + L::oSt + st * L::stage);
      if (starts()) zero_state();
    }
    if (f.dinit && z == 0) store_state<N>(D, f.dinit, state0, lane, p.st_bf16);
    if (lane == 0) bulk_wait_all();
    const float* e = gates() + (long long)(right + 1 - nch) * kGateRows * kC;
    return bad && any_start(e, nch, lane);
  }
};
template <int N, int NW>
__device__ __noinline__ bool reverse_again(const DeltaPlan& p, const DeltaBufs& f, const ChainMaps& m) {
  unsigned char* raw = chain_smem();
  RevChain<N, NW> x(p, f, raw, *reinterpret_cast<const RevPlace*>(raw + RevSmem<N, NW>::oPlace));
  x.template columns<true>(m);
  return x.ok;
}

template <int N, int NW, bool kPieces>
__global__ void __launch_bounds__((NW + 1) * 32, 1)
    delta_chain_bwd_kernel(const __grid_constant__ DeltaPlan p, const __grid_constant__ DeltaBufs f, int pieces,
                           const __grid_constant__ ChainMaps m) {
  using L = RevSmem<N, NW>;
  extern __shared__ unsigned char raw_[];
  unsigned char* raw = raw_ + ((1024 - (smem_u32(raw_) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + L::oBar);
  uint64_t* empty = full + 3;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ptiles = p.P / (16 * NW);
  const int p0 = (int)(blockIdx.x % ptiles) * 16 * NW;
  const int h = (int)((blockIdx.x / ptiles) % p.H), row = (int)(blockIdx.x / ((long long)ptiles * p.H));
  const int bi = kPieces ? row % p.b : row;
  const int grp = h / p.hpg, bh = bi * p.H + h;
  const float* gates = static_cast<const float*>(f.e) + (long long)bh * p.nc * kGateRows * kC;
  __shared__ Piece piece_s;
  if (kPieces && w == 0) {
    const Piece found = find_piece<NW>(gates, row / p.b, pieces, p.nc, lane);
    if (lane == 0) piece_s = found;
  }
  __shared__ int redo_s;
  auto init_bars = [&]() {
    for (int i = 0; i < 3; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kPieces ? max(piece_s.warps, 1) : NW);
    }
    mbar_fence_init();
  };
  if (threadIdx.x == 0) {
    init_bars();
    redo_s = 0;
  }
  __syncthreads();
  const Piece piece = kPieces ? piece_s : Piece{0, p.nc, 0, 0, NW};
  const int z = piece.z;
  if ((z && piece.first >= piece.next) || piece.warps == 0) return;  // no cut of its own, or nothing left
  // its chunks, from the right; an earlier piece gives no outputs for its first one (which is the next piece's too)
  const bool inner = piece.next < p.nc;
  const int right = inner ? piece.next : p.nc - 1, nch = right + 1 - piece.first;
  const RevPlace here = {bi, h, p0, z, right, nch, inner};
  if (threadIdx.x == 0) *reinterpret_cast<RevPlace*>(raw + L::oPlace) = here;
  RevChain<N, NW> x(p, f, raw, here);
  bool& ok = x.ok;
  // Every warp has ended its first pass: whether there is to be a second one
  auto again = [&]() { return chain_again(redo_s, ok, full, 6, (NW + 1) * 32, init_bars); };
  if (w == NW) {
    auto copies = [&]() {
      int st = 0, ph = 0;
      for (int k = 0; k < nch; ++k) {
        const int c = right - k;
        if (k >= 3) mbar_wait_flag(empty + st, ph ^ 1, ok);
        unsigned char* d = raw + L::oSt + st * L::stage;
        mbar_expect_tx(full + st, L::stage + kGateBytes);
        tma_load_4d(d, &m.k, full + st, 0, c * kC, grp * (N / 64), bi);
        tma_load_4d(d + L::kK, &m.q, full + st, 0, c * kC, grp * (N / 64), bi);
        d += 2 * L::kK;
        tma_load_4d(d, &m.T, full + st, 0, 0, c, bh);
        tma_load_4d(d + kTile, &m.A, full + st, 0, 0, c, bh);
        tma_load_4d(d + 2 * kTile, &m.v, full + st, p0, h, c * kC, bi);
        bulk_load(raw + L::oE + st * kGateBytes, gates + (long long)c * kGateRows * kC, kGateBytes, full + st);
        if (++st == 3) st = 0, ph ^= 1;
      }
    };
    if (lane == 0) copies();
    __syncwarp();
    if (again() && lane == 0) copies();
  } else {
    const bool live = !kPieces || piece.has(w);
    if (live && x.template columns<false>(m)) atomicOr(&redo_s, kNotFinite);
    __syncwarp();
    if (again() && live) ok = reverse_again<N, NW>(p, f, m);
  }
  if (!ok) atomicOr(f.status, kDevTimeout);
}

// Columns a CTA: 64, or 32 or 16 while every CTA still has an SM of its own --
// fewer warps share an SM's shared memory, but each CTA copies the chunks'
// operands for itself (one row of 4001 tokens, 32 heads of 64 x 128, forward:
// 78 us by 32 columns, 75 by 16; 8192 tokens: reverse 197 and 186).  Packed rows
// have their chains in as many pieces as there are SMs for, and rather twice the
// columns than one piece (one row of 20,011 tokens in 16 sequences, 64 heads of 64 x
// 64: forward 229 us instead of 292, reverse 216 instead of 338; where one sequence
// leaves one piece, and two CTAs share its columns, 289 and 362).
struct ChainShape {
  int warps, pieces;  // of 16 columns
};
ChainShape chain_shape(const DeltaPlan& p, const DeltaBufs& f) {
  const long long sms = device_sm_count(), wide = (long long)p.b * p.H * (p.P / 64);
  auto warps = [&](int pieces) { return wide * 4 * pieces <= sms ? 1 : wide * 2 * pieces <= sms ? 2 : 4; };
  ChainShape c = {warps(1), 1};
  if (f.seq && wide * 2 <= sms && p.nc >= 8) {
    c.warps = warps(2);
    const long long fit = sms / (wide * (4 / c.warps));
    c.pieces = (int)(fit < p.nc / 4 ? fit : p.nc / 4);
  }
  return c;
}

bool chain_maps(const DeltaPlan& p, const DeltaBufs& f, bool reverse, int nw, ChainMaps* m) {
  const uint64_t N = p.N, P = p.P, H = p.H, G = p.G, Ln = p.L, b = p.b, nc = p.nc, e = 2;
  auto tokens = [&](CUtensorMap* t, const void* base, uint64_t width, uint64_t heads, uint64_t stride, uint32_t cols,
                    int swizzle) {
    const uint64_t d[4] = {width, heads, Ln, b}, s[3] = {width * e, stride * e, Ln * stride * e};
    const uint32_t box[4] = {cols, 1, (uint32_t)kC, 1};
    return encode_tmap_bf16_4d(t, base, d, s, box, swizzle);
  };
  auto chunks = [&](CUtensorMap* t, const void* base, uint64_t width, uint64_t rows, uint32_t box_rows) {
    const uint64_t d[4] = {width, rows, nc, b * H}, s[3] = {width * e, rows * width * e, nc * rows * width * e};
    const uint32_t box[4] = {64, box_rows, 1, 1};
    return encode_tmap_bf16_4d(t, base, d, s, box, 128);
  };
  const uint32_t cols = 16 * nw;
  // q and k: all dstate columns of a group in one copy, 64-column blocks of [token][64] one after the other
  auto groups = [&](CUtensorMap* t, const void* base, uint64_t stride) {
    const uint64_t d[4] = {64, Ln, G * N / 64, b}, s[3] = {stride * e, 128, Ln * stride * e};
    const uint32_t box[4] = {64, (uint32_t)kC, (uint32_t)N / 64, 1};
    return encode_tmap_bf16_4d(t, base, d, s, box, 128);
  };
  bool good = groups(&m->q, f.q, p.qs) && groups(&m->k, f.k, p.ks) &&
              tokens(&m->v, reverse ? f.dy : f.v, P, H, reverse ? H * P : p.vs, cols, (int)cols * 2) &&
              tokens(&m->y, reverse ? f.dv : f.y, P, H, H * P, 16, 0) && chunks(&m->T, f.T, 64, 64, 64) &&
              chunks(&m->A, f.A, 64, 64, 64);
  if (good && (reverse || f.S)) good = chunks(&m->S, reverse ? f.D : f.S, N, P, 16);
  if (good && !reverse && f.S) good = chunks(&m->w, f.w, 64, P, 16);
  return good;
}

template <int N, int NW, bool kPieces>
cudaError_t launch_chain_t(const DeltaPlan& p, const DeltaBufs& f, int pieces, bool reverse, cudaStream_t s) {
  ChainMaps m = {};
  if (!chain_maps(p, f, reverse, NW, &m)) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)((long long)(p.P / (16 * NW)) * p.H * p.b * pieces);
  if (reverse) {
    auto kern = delta_chain_bwd_kernel<N, NW, kPieces>;
    constexpr int smem = RevSmem<N, NW>::bytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set_kernel_name("delta_chain_bwd");
    kern<<<grid, (NW + 1) * 32, smem, s>>>(p, f, pieces, m);
  } else {
    auto kern = delta_chain_fwd_kernel<N, NW, kPieces>;
    constexpr int smem = FwdSmem<N, NW>::bytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set_kernel_name("delta_chain_fwd");
    kern<<<grid, fwd_threads(NW), smem, s>>>(p, f, pieces, m);
  }
  return cudaGetLastError();
}

cudaError_t launch_chain(const DeltaPlan& p, const DeltaBufs& f, bool reverse, cudaStream_t s) {
  const ChainShape c = chain_shape(p, f);
  auto go = [&](auto cut) {
    constexpr bool kPieces = decltype(cut)::value;
    auto shaped = [&](auto n) {
      constexpr int N = decltype(n)::value;
      return c.warps == 4   ? launch_chain_t<N, 4, kPieces>(p, f, c.pieces, reverse, s)
             : c.warps == 2 ? launch_chain_t<N, 2, kPieces>(p, f, c.pieces, reverse, s)
                            : launch_chain_t<N, 1, kPieces>(p, f, c.pieces, reverse, s);
    };
    return p.N == 128 ? shaped(std::integral_constant<int, 128>()) : shaped(std::integral_constant<int, 64>());
  };
  return c.pieces > 1 ? go(std::true_type()) : go(std::false_type());
}

}  // namespace

cudaError_t launch_delta_chain_fwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return launch_chain(p, f, false, s);
}
cudaError_t launch_delta_chain_bwd(const DeltaPlan& p, const DeltaBufs& f, cudaStream_t s) {
  return launch_chain(p, f, true, s);
}

}  // namespace ssd
