// k_add_norm.cu -- the norm that takes in the residual, forward (output in the
// type, or in 8 bits with a scale for each row) and backward, and its C ABI.
//
//   h = x + residual, in the residual's type          v = h in fp32
//   r = 1 / sqrt(mean v^2 + eps)                      out = v r weight
//   backward, with g = dout weight and n = v r:
//   dx = dresidual = dh + r (g - n mean(g n))         dweight = sum over rows of dout n
//
// The norm reads h as it is stored: the backward, which has only h, then sees
// the forward's own values.  Everything but the stored tensors is fp32.
//
// Bound by HBM; each tensor is read and written once.  A CTA takes a row, a
// thread 8 neighbouring columns at a time (one 16-byte access in bf16), which
// stay in registers from the sum to the store, with the CTA's next row on its way;
// in the backward they stay the thread's own from row to row, so that it also
// holds their dweight.  The CTAs' dweights are joined by a second kernel in a
// fixed order.  16,384 rows of 4096 bf16: with a bf16 stream to e4m3 77 us (6.1
// TB/s); on an fp32 stream to bf16 132 us (6.1), its backward 179 us (6.0).
#include <string.h>

#include "codes.cuh"
#include "ssd_internal.cuh"

namespace ssd {

int device_check();

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxDim = kMaxThreads * 8 * 4;
constexpr int kMaxSlices = 1216;  // CTAs of the backward, each with a row of partial dweights

struct AddNormArgs {
  const void *x, *res;
  const float* w;
  void *h, *out;
  float* scales;
  const void *dout, *dh;
  void *dx, *dres;
  float* part;
  long long rows, xs;  // xs: elements from row to row of x
  int dim, codes;      // codes: 0 none, 1 int8, 2 e4m3
  float inv_dim, eps;
};

// Which eight values of a row a thread takes at a time.
enum How {
  kApart,   // columns a CTA's width apart, one by one
  kWhole,   // neighbours: rows are whole 16-byte vectors
  kAligned  // neighbours in memory's vectors, in which a row of dense tensors begins `shift` values late; a row's first and
            // last vectors are shared with other rows: they are read whole but at the tensor's end, what is another row's
            // is masked, and their own values are written one by one
};

// Eight values of a row.  They are fetched as they lie and turned into fp32 when
// they are wanted, so that a row ahead costs few registers.
template <typename T, How kHow>
struct Cols {
  struct Raw {
    uint4 u[sizeof(T) / 2];
  };
  static __device__ __forceinline__ int col(int i, int j, int shift) {
    return kHow == kApart ? (i * 8 + j) * (int)blockDim.x + (int)threadIdx.x
                          : (i * (int)blockDim.x + (int)threadIdx.x) * 8 + j - (kHow == kAligned ? shift : 0);
  }
  // whether the eight are a vector of this row
  static __device__ __forceinline__ bool whole(int c, int dim) {
    return kHow == kWhole ? c < dim : kHow == kAligned && c >= 0 && c + 8 <= dim;
  }
  static __device__ __forceinline__ bool inside(int c, int dim) { return (kHow != kAligned || c >= 0) && c < dim; }
  // reach: how many values of the tensor there are from the row's first on, or 8 past the row if there are more.  (Before
  // it there are `shift`, for the tensor begins with a whole vector.)
  static __device__ __forceinline__ void fetch(const T* row, int i, int dim, int shift, int reach, Raw& r) {
    const int c = col(i, 0, shift);
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) r.u[j] = make_uint4(0, 0, 0, 0);
    if (kHow == kAligned ? c < dim && c + 8 <= reach : whole(c, dim)) {
#pragma unroll
      for (int j = 0; j < (int)sizeof(T) / 2; ++j) r.u[j] = __ldcs(reinterpret_cast<const uint4*>(row + c) + j);
    } else if (kHow == kApart || (kHow == kAligned && c < dim)) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = 0;
        if (inside(col(i, j, shift), dim)) {
          if constexpr (sizeof(T) == 2) w[j] = __ldcs(reinterpret_cast<const unsigned short*>(row) + col(i, j, shift));
          else w[j] = __ldcs(reinterpret_cast<const uint32_t*>(row) + col(i, j, shift));
        }
      }
      if constexpr (sizeof(T) == 2) {
        r.u[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
      } else {
        r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        r.u[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      const uint4 x = r.u[sizeof(T) / 2 - 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]);
      v[4] = __uint_as_float(x.x); v[5] = __uint_as_float(x.y);
      v[6] = __uint_as_float(x.z); v[7] = __uint_as_float(x.w);
    }
  }
  // Nothing of other rows' values
  static __device__ __forceinline__ void mask(int i, int dim, int shift, float (&v)[8]) {
    if constexpr (kHow == kAligned) {
      if (whole(col(i, 0, shift), dim)) return;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!inside(col(i, j, shift), dim)) v[j] = 0.f;
    }
  }
  static __device__ __forceinline__ void store(T* row, int i, int dim, int shift, const float (&v)[8]) {
    const int c = col(i, 0, shift);
    if (whole(c, dim)) {
      if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
        __stcs(reinterpret_cast<uint4*>(row + c), make_uint4(w[0], w[1], w[2], w[3]));
      } else {
        __stcs(reinterpret_cast<float4*>(row + c), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(row + c) + 1, make_float4(v[4], v[5], v[6], v[7]));
      }
    } else if (kHow != kWhole) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (inside(col(i, j, shift), dim)) row[col(i, j, shift)] = from_f<T>(v[j]);
    }
  }
};

// The weight's values stay in the caches: every row reads them.
template <How kHow>
__device__ __forceinline__ void load_weight(const float* w, int i, int dim, int shift, float (&v)[8]) {
  using C = Cols<float, kHow>;
  const int c = C::col(i, 0, shift), c4 = c & ~3;
  if (kHow == kWhole && c < dim) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + c)), b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else if (kHow == kAligned && c >= 0 && c4 + 12 <= dim) {
    // three vectors hold them, from the same place on for the whole row
    float x[12];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(w + c4) + j);
      x[4 * j] = q.x; x[4 * j + 1] = q.y; x[4 * j + 2] = q.z; x[4 * j + 3] = q.w;
    }
    const int late = -shift & 3;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = late == 0 ? x[j] : late == 1 ? x[j + 1] : late == 2 ? x[j + 2] : x[j + 3];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = kHow != kWhole && C::inside(C::col(i, j, shift), dim) ? __ldg(w + C::col(i, j, shift)) : 0.f;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the CTA, the same for every thread, in a fixed order.  red: a value
// for each warp, not in use by an earlier call that some warp may still be in.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += red[i];
  return v;
}

template <bool kFp8, How kHow>
__device__ __forceinline__ void store_codes(uint8_t* row, int i, int dim, int shift, const float (&v)[8], float inv,
                                            bool zero) {
  using C = Cols<float, kHow>;
  const int c = C::col(i, 0, shift);
  if (C::whole(c, dim)) {
    uint2 u = make_uint2(0, 0);
    if (!zero)
      u = make_uint2(encode4<kFp8>(make_float4(v[0], v[1], v[2], v[3]), inv),
                     encode4<kFp8>(make_float4(v[4], v[5], v[6], v[7]), inv));
    *reinterpret_cast<uint2*>(row + c) = u;
  } else if (kHow != kWhole) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (C::inside(C::col(i, j, shift), dim)) row[C::col(i, j, shift)] = zero ? 0 : encode<kFp8>(v[j] * inv);
  }
}

// NP: pieces of 8 columns to a thread.  The next row of a CTA is on its way
// while this one is summed, rounded and written.
template <typename T, typename R, int NP, How kHow>
__global__ void __launch_bounds__(kMaxThreads) add_norm_fwd_kernel(AddNormArgs a) {
  using X = Cols<T, kHow>;
  using H = Cols<R, kHow>;
  __shared__ float red[2][kMaxThreads / 32], big_s[2][kMaxThreads / 32];
  typename X::Raw x[NP];
  typename H::Raw y[NP];
  auto shift_of = [&](long long row) { return kHow == kAligned ? (int)((row * a.dim) & 7) : 0; };
  auto fetch = [&](long long row) {
    const int shift = shift_of(row);
    const int reach = a.dim + (int)min((a.rows - 1 - row) * a.dim, 8LL);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      X::fetch(static_cast<const T*>(a.x) + row * a.xs, i, a.dim, shift, reach, x[i]);
      if (a.res) H::fetch(static_cast<const R*>(a.res) + row * a.dim, i, a.dim, shift, reach, y[i]);
    }
  };
  fetch(blockIdx.x);
  float w0[8];  // the weight of a single piece stays in registers
  if (NP == 1 && kHow != kAligned) load_weight<kHow>(a.w, 0, a.dim, 0, w0);
  int par = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    float v[NP][8];
    float ss = 0.f;
    const int shift = shift_of(row);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      X::values(x[i], v[i]);
      if (a.res) {
        float u[8];
        H::values(y[i], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = to_f(from_f<R>(v[i][j] + u[j]));
      }
      X::mask(i, a.dim, shift, v[i]);
    }
    if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (a.h) H::store(static_cast<R*>(a.h) + row * a.dim, i, a.dim, shift, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    const float r = rsqrtf(cta_sum(ss, red[par]) * a.inv_dim + a.eps);
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float w[8];
      if (NP > 1 || kHow == kAligned) load_weight<kHow>(a.w, i, a.dim, shift, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = v[i][j] * r * (NP == 1 && kHow != kAligned ? w0[j] : w[j]);
        // what is not finite makes the row's largest an infinity
        big = fmaxf(big, fabsf(v[i][j]) <= 3.402823466e38f ? fabsf(v[i][j]) : __int_as_float(0x7f800000));
      }
    }
    if (a.codes == 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) X::store(static_cast<T*>(a.out) + row * a.dim, i, a.dim, shift, v[i]);
      continue;
    }
    // (values that are not negative order as integers)
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
    if (blockDim.x > 32) {
      if ((threadIdx.x & 31) == 0) big_s[par][threadIdx.x >> 5] = big;
      __syncthreads();
      for (int i = 0; i < (int)(blockDim.x >> 5); ++i) big = fmaxf(big, big_s[par][i]);
    }
    const bool bad = big == __int_as_float(0x7f800000), zero = bad || !(big >= kTiny);
    const bool fp8 = a.codes == 2;
    const float inv = zero ? 0.f : fp8 ? factor_of<true>(big) : factor_of<false>(big);
    uint8_t* to = static_cast<uint8_t*>(a.out) + row * a.dim;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (fp8) store_codes<true, kHow>(to, i, a.dim, shift, v[i], inv, zero);
      else store_codes<false, kHow>(to, i, a.dim, shift, v[i], inv, zero);
    }
    if (threadIdx.x == 0)
      a.scales[row] = bad ? __int_as_float(0x7fc00000) : zero ? 0.f : fp8 ? scale_of<true>(big) : scale_of<false>(big);
  }
}

template <typename T, typename R, int NP, How kHow>
__global__ void __launch_bounds__(kMaxThreads) add_norm_bwd_kernel(AddNormArgs a) {
  using X = Cols<T, kHow>;
  using H = Cols<R, kHow>;
  __shared__ float red[2][2][kMaxThreads / 32];
  float dw[NP][8];
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  typename H::Raw h[NP], dh[NP];
  typename X::Raw dout[NP];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      H::fetch(static_cast<const R*>(a.h) + row * a.dim, i, a.dim, 0, a.dim, h[i]);
      X::fetch(static_cast<const T*>(a.dout) + row * a.dim, i, a.dim, 0, a.dim, dout[i]);
    }
  };
  constexpr bool kNext = NP <= 2;  // (four pieces leave no registers for another row)
  if (kNext) fetch(blockIdx.x);
  int par = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    float v[NP][8], d[NP][8];
    float ss = 0.f, sg = 0.f;
    if (!kNext) fetch(row);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (a.dh && kNext) H::fetch(static_cast<const R*>(a.dh) + row * a.dim, i, a.dim, 0, a.dim, dh[i]);
      H::values(h[i], v[i]);
      X::values(dout[i], d[i]);
    }
    if (kNext && row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float w[8];
      load_weight<kHow>(a.w, i, a.dim, 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(v[i][j], v[i][j], ss);
        sg = fmaf(d[i][j] * w[j], v[i][j], sg);
      }
    }
    ss = warp_sum(ss);
    sg = warp_sum(sg);
    if (blockDim.x > 32) {
      if ((threadIdx.x & 31) == 0) {
        red[par][0][threadIdx.x >> 5] = ss;
        red[par][1][threadIdx.x >> 5] = sg;
      }
      __syncthreads();
      ss = sg = 0.f;
      for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
        ss += red[par][0][i];
        sg += red[par][1][i];
      }
    }
    const float r = rsqrtf(ss * a.inv_dim + a.eps);
    const float proj = sg * r * a.inv_dim;  // mean(g n)
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float w[8], u[8];
      load_weight<kHow>(a.w, i, a.dim, 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = 0.f;
      if (a.dh) {
        if (!kNext) H::fetch(static_cast<const R*>(a.dh) + row * a.dim, i, a.dim, 0, a.dim, dh[i]);
        H::values(dh[i], u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i][j] * r;
        dw[i][j] = fmaf(d[i][j], n, dw[i][j]);
        u[j] += r * (d[i][j] * w[j] - n * proj);
      }
      X::store(static_cast<T*>(a.dx) + row * a.dim, i, a.dim, 0, u);
      if (a.dres) H::store(static_cast<R*>(a.dres) + row * a.dim, i, a.dim, 0, u);
    }
  }
  // (the launch that joins the partial sums comes up while the last of them are written)
  asm volatile("griddepcontrol.launch_dependents;");
  float* part = a.part + (long long)blockIdx.x * a.dim;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (X::col(i, j, 0) < a.dim) part[X::col(i, j, 0)] = dw[i][j];
}

// dweight[c] = sum of the slices' partials: 32 columns to a CTA, each warp a
// run of slices, then the warps in order.
constexpr int kFoldWarps = 16;
__global__ void __launch_bounds__(kFoldWarps * 32) add_norm_fold_kernel(const float* part, float* dweight, int slices,
                                                                        int dim) {
  __shared__ float sums[kFoldWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int per = (slices + kFoldWarps - 1) / kFoldWarps;
  float s = 0.f;
  if (c < dim) {
    const int hi = min((warp + 1) * per, slices);
#pragma unroll 8
    for (int i = warp * per; i < hi; ++i) s += part[(long long)i * dim + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kFoldWarps; ++i) s += sums[i][lane];
    dweight[c] = s;
  }
}

// Threads to a row and pieces to a thread.  Few rows: as many threads as there
// are pieces, for the shortest way through one row (1001 rows of 1237 fp32: 4.4 us
// with one piece, 5.9 with two).  Many rows: two pieces to a thread (16,384 rows of
// 4096 bf16 to e4m3: 77 us, with one piece 96), four where 512 threads of two would
// not hold the row.
struct Shape {
  int threads, np;
};
Shape shape_of(int dim, long long rows, int sms, How how) {
  const int pieces = how == kAligned ? (dim + 7) / 8 + 1 : (dim + 7) / 8;
  int np = rows > 8 * sms && pieces >= 64 ? 2 : 1;
  while (pieces > np * kMaxThreads) np *= 2;
  const int t = ((pieces + np - 1) / np + 31) / 32 * 32;
  return {t, np};
}
// CTAs: those that are resident at once, with 64 registers to a thread, and in
// the backward 128 (16,384 x 4096 on an fp32 stream: 179 us; three CTAs to an SM
// without the next row in registers 197).
long long grid_of(long long rows, int threads, int sms, bool bwd) {
  int per = (bwd ? 512 : 1024) / threads;
  if (per > 8 && bwd) per = 8;
  if (per < 1) per = 1;
  long long grid = (long long)sms * per;
  if (grid > rows) grid = rows;
  return bwd && grid > kMaxSlices ? kMaxSlices : grid;
}

template <typename T, typename R, int NP>
cudaError_t launch_np(const AddNormArgs& a, int threads, unsigned grid, How how, bool bwd, cudaStream_t s) {
  if (bwd) {
    set_kernel_name("add_norm_bwd");
    if (how == kWhole) add_norm_bwd_kernel<T, R, NP, kWhole><<<grid, threads, 0, s>>>(a);
    else add_norm_bwd_kernel<T, R, NP, kApart><<<grid, threads, 0, s>>>(a);
  } else {
    set_kernel_name("add_norm_fwd");
    if (how == kWhole) add_norm_fwd_kernel<T, R, NP, kWhole><<<grid, threads, 0, s>>>(a);
    else if (sizeof(T) == 2 && how == kAligned)
      add_norm_fwd_kernel<T, R, NP, sizeof(T) == 2 ? kAligned : kApart><<<grid, threads, 0, s>>>(a);
    else add_norm_fwd_kernel<T, R, NP, kApart><<<grid, threads, 0, s>>>(a);
  }
  return cudaGetLastError();
}
template <typename T, typename R>
cudaError_t launch_t(const AddNormArgs& a, const Shape& sh, How how, unsigned grid, bool bwd, cudaStream_t s) {
  if (sh.np == 1) return launch_np<T, R, 1>(a, sh.threads, grid, how, bwd, s);
  if (sh.np == 2) return launch_np<T, R, 2>(a, sh.threads, grid, how, bwd, s);
  return launch_np<T, R, 4>(a, sh.threads, grid, how, bwd, s);
}
cudaError_t launch(const ssd_add_norm_problem& pr, const AddNormArgs& a, const Shape& sh, How how, unsigned grid,
                   bool bwd, cudaStream_t s) {
  if (pr.dtype == SSD_F32) return launch_t<float, float>(a, sh, how, grid, bwd, s);
  if (pr.residual_dtype == SSD_F32) return launch_t<__nv_bfloat16, float>(a, sh, how, grid, bwd, s);
  return launch_t<__nv_bfloat16, __nv_bfloat16>(a, sh, how, grid, bwd, s);
}
// The forward of many dense odd rows of bf16 goes by memory's vectors, of which a
// row may touch one more than it fills (16,384 x 4095 to e4m3: 126 us, column by
// column 267; fp32 rows are no faster so, few rows slower).  No byte is read twice;
// 1.4 times the instructions of 4096 columns bound it: edges, masks, the weight's
// shift.  The backward's threads keep their columns' dweight, which a row's
// shift would move (16,384 x 4095 bf16: 264 us column by column, 4096: 103).
How how_of(int dim, long long xs, long long rows, bool bf16, bool bwd, int sms) {
  if (dim % 8 == 0 && xs % 8 == 0) return kWhole;
  return !bwd && bf16 && xs == dim && rows > 8 * sms && dim / 8 + 2 <= kMaxThreads * 4 ? kAligned : kApart;
}

int check(const ssd_add_norm_problem* pr) {
  if (!pr || pr->rows < 1 || pr->dim < 1 || pr->x_stride < 0 || (pr->x_stride && pr->x_stride < pr->dim))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!(pr->eps > 0.f && pr->eps <= 3.402823466e38f)) return SSD_ERR_INVALID_ARGUMENT;
  if ((pr->dtype != SSD_F32 && pr->dtype != SSD_BF16) || (pr->residual_dtype != SSD_F32 && pr->residual_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARGUMENT;
  if (pr->out_format < SSD_OUT_PLAIN || pr->out_format > SSD_OUT_E4M3) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->flags & ~SSD_NORM_HAS_RESIDUAL) return SSD_ERR_INVALID_ARGUMENT;
  // without a residual there is nothing of another type to add to
  if (!(pr->flags & SSD_NORM_HAS_RESIDUAL) && pr->residual_dtype != pr->dtype) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->dtype == SSD_F32 && pr->residual_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  const int64_t xs = pr->x_stride ? pr->x_stride : pr->dim;
  if (pr->dim > kMaxDim || xs > (1LL << 30) || pr->rows > (1LL << 40) || (double)pr->rows * (double)xs >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_add_rmsnorm_fwd(const ssd_add_norm_problem* pr, const void* x, const void* residual, const float* weight,
                        void* h, void* out, float* scales, ssd_stream_t stream) {
  int rc = check(pr);
  if (rc != SSD_OK) return rc;
  if (!x || !weight || !out) return SSD_ERR_INVALID_ARGUMENT;
  if (((pr->flags & SSD_NORM_HAS_RESIDUAL) != 0) != (residual != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if ((pr->out_format != SSD_OUT_PLAIN) != (scales != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {x, residual, weight, h, out, scales};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  AddNormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.res = residual; a.w = weight; a.h = h; a.out = out; a.scales = scales;
  a.rows = pr->rows;
  a.xs = pr->x_stride ? pr->x_stride : pr->dim;
  a.dim = (int)pr->dim;
  a.codes = pr->out_format;
  a.inv_dim = 1.f / (float)pr->dim;
  a.eps = pr->eps;
  const int sms = device_sm_count();
  const How how = how_of(a.dim, a.xs, a.rows, pr->dtype == SSD_BF16, false, sms);
  const Shape sh = shape_of(a.dim, a.rows, sms, how);
  const long long grid = grid_of(a.rows, sh.threads, sms, false);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = launch(*pr, a, sh, how, (unsigned)grid, false, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_add_rmsnorm_bwd_workspace_bytes(const ssd_add_norm_problem* pr) {
  if (check(pr) != SSD_OK) return 0;
  const int64_t slices = pr->rows < kMaxSlices ? pr->rows : kMaxSlices;
  return ((size_t)slices * (size_t)pr->dim * sizeof(float) + 255) & ~(size_t)255;
}

int ssd_add_rmsnorm_bwd(const ssd_add_norm_problem* pr, const void* h, const float* weight, const void* dout,
                        const void* dh, void* dx, void* dresidual, float* dweight, void* workspace,
                        size_t workspace_bytes, ssd_stream_t stream) {
  int rc = check(pr);
  if (rc != SSD_OK) return rc;
  if (!h || !weight || !dout || !dx || !dweight || !workspace) return SSD_ERR_INVALID_ARGUMENT;
  if (dresidual && !(pr->flags & SSD_NORM_HAS_RESIDUAL)) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {h, weight, dout, dh, dx, dresidual, dweight, workspace};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < ssd_add_rmsnorm_bwd_workspace_bytes(pr)) return SSD_ERR_WORKSPACE_TOO_SMALL;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  AddNormArgs a;
  memset(&a, 0, sizeof(a));
  a.h = const_cast<void*>(h);
  a.w = weight; a.dout = dout; a.dh = dh; a.dx = dx; a.dres = dresidual;
  a.part = static_cast<float*>(workspace);
  a.rows = pr->rows;
  a.dim = (int)pr->dim;
  a.inv_dim = 1.f / (float)pr->dim;
  a.eps = pr->eps;
  const int sms = device_sm_count();
  const How how = how_of(a.dim, a.dim, a.rows, false, true, sms);
  const Shape sh = shape_of(a.dim, a.rows, sms, how);
  const long long grid = grid_of(a.rows, sh.threads, sms, true);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  cudaError_t e = launch(*pr, a, sh, how, (unsigned)grid, true, s);
  prof_after(s);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  prof_before(s);
  set_kernel_name("add_norm_fold");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.dim + 31) / 32));
  cfg.blockDim = dim3(kFoldWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, add_norm_fold_kernel, static_cast<const float*>(a.part), dweight, (int)grid, a.dim);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
