// k_scaled_matmul.cu -- the product of 8-bit codes (int8 or e4m3) with a scale
// for each token and for each channel, and its C ABI.
//
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n]
#include <string.h>

#include "codes.cuh"
#include "ssd_internal.cuh"

namespace ssd {

int device_check();

namespace {

struct MatmulArgs {
  const uint8_t *a, *w;
  const float *as, *ws, *bias;
  void* out;
  int* status;
  long long m, n, k;
};

// 64 tokens x 64 channels to a CTA of 16 x 16 threads, 32 codes of each row at
// a time, decoded to fp32 in shared memory.
template <bool kFp8, typename O>
__global__ void __launch_bounds__(256) scaled_matmul_simt_kernel(MatmulArgs p) {
  __shared__ float sa[32][65], sw[32][65];
  const long long m0 = (long long)blockIdx.y * 64, n0 = (long long)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
  float acc[4][4] = {};
  for (long long k0 = 0; k0 < p.k; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int row = i >> 5, c = i & 31;
      const bool in = k0 + c < p.k;
      sa[c][row] = in && m0 + row < p.m ? decode<kFp8>(p.a[(m0 + row) * p.k + k0 + c]) : 0.f;
      sw[c][row] = in && n0 + row < p.n ? decode<kFp8>(p.w[(n0 + row) * p.k + k0 + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int c = 0; c < 32; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty + 16 * i], sw[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < p.m && n < p.n) {
        const float v = acc[i][j] * p.as[m] * p.ws[n];
        static_cast<O*>(p.out)[m * p.n + n] = from_f<O>(p.bias ? v + p.bias[n] : v);
      }
    }
}

template <bool kFp8, typename O>
cudaError_t launch_simt(const MatmulArgs& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.n + 63) / 64), (unsigned)((p.m + 63) / 64));
  set_kernel_name("scaled_matmul_simt");
  scaled_matmul_simt_kernel<kFp8, O><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

int check(const ssd_matmul_problem* pr) {
  if (!pr || pr->m < 1 || pr->n < 1 || pr->k < 1 || pr->flags != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->format != SSD_CACHE_INT8 && pr->format != SSD_CACHE_E4M3) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->out_dtype != SSD_F32 && pr->out_dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
  // 2^40 elements per tensor; rows and tiles in 32 bits
  const int64_t cap = 1LL << 22;
  if (pr->m > cap || pr->n > cap || pr->k > cap || (double)pr->m * (double)pr->n >= (double)(1LL << 40) ||
      (double)pr->m * (double)pr->k >= (double)(1LL << 40) || (double)pr->n * (double)pr->k >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_scaled_matmul_workspace_bytes(const ssd_matmul_problem* pr) {
  return check(pr) == SSD_OK ? 256 : 0;
}

int ssd_scaled_matmul(const ssd_matmul_problem* pr, const void* a, const float* a_scales, const void* w,
                      const float* w_scales, const float* bias, void* out, void* workspace, size_t workspace_bytes,
                      ssd_stream_t stream) {
  int rc = check(pr);
  if (rc != SSD_OK) return rc;
  if (!a || !a_scales || !w || !w_scales || !out || !workspace) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {a, a_scales, w, w_scales, bias, out, workspace};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < ssd_scaled_matmul_workspace_bytes(pr)) return SSD_ERR_WORKSPACE_TOO_SMALL;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  const MatmulArgs p = {static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(w), a_scales, w_scales, bias, out, static_cast<int*>(workspace),
                        pr->m, pr->n, pr->k};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = pr->format == SSD_CACHE_E4M3, b16 = pr->out_dtype == SSD_BF16;
  prof_before(s);
  const cudaError_t e = fp8 ? (b16 ? launch_simt<true, __nv_bfloat16>(p, s) : launch_simt<true, float>(p, s))
                            : (b16 ? launch_simt<false, __nv_bfloat16>(p, s) : launch_simt<false, float>(p, s));
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
