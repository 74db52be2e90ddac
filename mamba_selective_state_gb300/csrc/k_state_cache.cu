// k_state_cache.cu -- recurrent states put away in 8 bits and read back.
//
// One row of dstate values has one scale.  A warp takes a row: its values
// stay in registers between the maximum and the rounding, so the states are
// read once; both directions are bound by HBM (5 bytes per value, 4 of them
// the fp32 state).
#include <cuda_fp8.h>

#include "ssd_internal.cuh"

namespace ssd {

int device_check();

namespace {

constexpr int kThreads = 256;
constexpr int kMaxVals = 8;  // values per lane: dstate <= 256

struct CacheArgs {
  const float* in;
  float* out;
  uint8_t* vals;
  float* scales;
  const int32_t* slots;
  long long rows, nslots;  // rows of one call
  int hp, N;               // rows per state, values per row
};

// Below this largest value top / amax is not finite: the row is zeros.
constexpr float kTiny = 3.009265538105056e-36f;  // 2^-118

template <bool kFp8>
__device__ __forceinline__ uint8_t encode(float y) {
  if (kFp8) return (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(y, -127.f), 127.f));
}
template <bool kFp8>
__device__ __forceinline__ float decode(uint8_t v) {
  if (kFp8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return (float)(int8_t)v;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads) cache_store_kernel(CacheArgs a) {
  const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 31;
  const long long bi = row / a.hp;
  const long long slot = a.slots ? a.slots[bi] : bi;
  if (slot < 0 || slot >= a.nslots) return;
  const float* x = a.in + row * a.N;
  float v[kMaxVals], big = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kMaxVals; ++i) {
    const int n = i * 32 + lane;
    v[i] = n < a.N ? x[n] : 0.f;
    big = fmaxf(big, fabsf(v[i]));
    bad |= !(fabsf(v[i]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  bad = __any_sync(0xffffffffu, bad);
  const float top = kFp8 ? 448.f : 127.f;
  const bool empty = bad || !(big >= kTiny);
  const float inv = empty ? 0.f : top / big;
  const long long to = slot * a.hp + row % a.hp;
#pragma unroll
  for (int i = 0; i < kMaxVals; ++i) {
    const int n = i * 32 + lane;
    if (n < a.N) a.vals[to * a.N + n] = empty ? 0 : encode<kFp8>(v[i] * inv);
  }
  if (lane == 0) a.scales[to] = bad ? __int_as_float(0x7fc00000) : empty ? 0.f : big / top;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads) cache_load_kernel(CacheArgs a) {
  const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 31;
  const long long bi = row / a.hp;
  const long long slot = a.slots ? a.slots[bi] : bi;
  const bool in = slot >= 0 && slot < a.nslots;
  const long long from = slot * a.hp + row % a.hp;
  const float sc = in ? a.scales[from] : 0.f;
#pragma unroll
  for (int i = 0; i < kMaxVals; ++i) {
    const int n = i * 32 + lane;
    if (n < a.N) a.out[row * a.N + n] = in ? decode<kFp8>(a.vals[from * a.N + n]) * sc : 0.f;
  }
}

bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

int run_cache(const ssd_cache_problem* pr, const float* in, float* out, const void* vals, const float* scales,
              const int32_t* slots, bool store, ssd_stream_t stream) {
  if (!pr || pr->batch < 1 || pr->nheads < 1 || pr->headdim < 1 || pr->dstate < 1 || pr->nslots < 1 || pr->flags != 0)
    return SSD_ERR_INVALID_ARGUMENT;
  if (pr->format != SSD_CACHE_INT8 && pr->format != SSD_CACHE_E4M3) return SSD_ERR_INVALID_ARGUMENT;
  if (!vals || !scales || (store ? !in : !out)) return SSD_ERR_INVALID_ARGUMENT;
  if (!slots && pr->nslots < pr->batch) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {in, out, vals, scales, slots};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->dstate > 32 * kMaxVals) return SSD_ERR_UNSUPPORTED;
  const double most = (double)(pr->batch > pr->nslots ? pr->batch : pr->nslots);
  if ((double)pr->nheads * (double)pr->headdim >= 2147483648.0 ||
      most * (double)pr->nheads * (double)pr->headdim * (double)pr->dstate >= (double)(1LL << 40) ||
      (double)pr->batch * (double)pr->nheads * (double)pr->headdim >= (double)(1LL << 33))
    return SSD_ERR_UNSUPPORTED;
  const int rc = device_check();
  if (rc != SSD_OK) return rc;
  CacheArgs a = {in,
                 out,
                 static_cast<uint8_t*>(const_cast<void*>(vals)),
                 const_cast<float*>(scales),
                 slots,
                 (long long)pr->batch * pr->nheads * pr->headdim,
                 pr->nslots,
                 (int)(pr->nheads * pr->headdim),
                 (int)pr->dstate};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)((a.rows + kThreads / 32 - 1) / (kThreads / 32));
  const bool fp8 = pr->format == SSD_CACHE_E4M3;
  prof_before(s);
  set_kernel_name(store ? "state_cache_store" : "state_cache_load");
  if (store) {
    if (fp8) cache_store_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else cache_store_kernel<false><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (fp8) cache_load_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else cache_load_kernel<false><<<grid, kThreads, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_state_cache_store(const ssd_cache_problem* prob, const float* states, const int32_t* slots, void* cache,
                          float* scales, ssd_stream_t stream) {
  return run_cache(prob, states, nullptr, cache, scales, slots, true, stream);
}

int ssd_state_cache_load(const ssd_cache_problem* prob, const void* cache, const float* scales, const int32_t* slots,
                         float* states, ssd_stream_t stream) {
  return run_cache(prob, nullptr, states, cache, scales, slots, false, stream);
}

}  // extern "C"
