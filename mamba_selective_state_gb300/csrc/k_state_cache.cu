// k_state_cache.cu -- recurrent states put away in 8 bits and read back.
//
// One row of dstate values has one scale.  Its values stay in registers
// between the maximum and the rounding, so the states are read once; both
// directions are bound by HBM (5 bytes per value, 4 of them the fp32 state).
// Rows of a multiple of four values take four to a lane, in 16-byte accesses,
// as few lanes to a row as hold it, and four rows to a lane at a time; other
// rows take a warp and single values.  Measured with 64 states of 64 heads x 64 x
// 128 (169 MB each way): store 42 us (4.0 TB/s), load 31 us (5.4 TB/s).  The store
// also waits for each row's maximum between its loads and its rounding.
#include "codes.cuh"
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
  const bool empty = bad || !(big >= kTiny);
  const float inv = empty ? 0.f : factor_of<kFp8>(big);
  const long long to = slot * a.hp + row % a.hp;
#pragma unroll
  for (int i = 0; i < kMaxVals; ++i) {
    const int n = i * 32 + lane;
    if (n < a.N) a.vals[to * a.N + n] = empty ? 0 : encode<kFp8>(v[i] * inv);
  }
  if (lane == 0) a.scales[to] = bad ? __int_as_float(0x7fc00000) : empty ? 0.f : scale_of<kFp8>(big);
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

constexpr int kRows = 4;  // rows of a lane in flight

// The largest of the row's lanes (values that are not negative order as integers)
template <int LR>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LR == 32) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
  } else {
#pragma unroll
    for (int o = LR / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

// LR lanes to a row (a power of two), V vectors of four values to a lane.
template <bool kFp8, int LR, int V>
__global__ void __launch_bounds__(kThreads) cache_store4_kernel(CacheArgs a) {
  const int lane = threadIdx.x % LR;
  const long long row0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / LR;
  const long long step = (long long)gridDim.x * kThreads / LR;
  const int n4 = a.N / 4;
  float4 v[kRows][V];
  long long to[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const long long row = row0 + r * step;
    to[r] = -1;
    if (row < a.rows) {
      const long long bi = row / a.hp, slot = a.slots ? a.slots[bi] : bi;
      if (slot >= 0 && slot < a.nslots) to[r] = slot * a.hp + (row - bi * a.hp);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int n = i * LR + lane;
      v[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (to[r] >= 0 && n < n4) v[r][i] = __ldcs(reinterpret_cast<const float4*>(a.in) + row * n4 + n);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float4 x = v[r][i];
      // infinities show in the maximum, a NaN in the differences, which are zero for every other value
      const float nan = (x.x - x.x) + (x.y - x.y) + (x.z - x.z) + (x.w - x.w);
      big = fmaxf(fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
      big = nan == 0.f ? big : __int_as_float(0x7f800000);
    }
    big = row_max<LR>(big);
    if (to[r] < 0) continue;
    const bool any = big == __int_as_float(0x7f800000), empty = any || !(big >= kTiny);
    const float inv = empty ? 0.f : factor_of<kFp8>(big);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int n = i * LR + lane;
      if (n < n4) reinterpret_cast<uint32_t*>(a.vals)[to[r] * n4 + n] = empty ? 0u : encode4<kFp8>(v[r][i], inv);
    }
    if (lane == 0) a.scales[to[r]] = any ? __int_as_float(0x7fc00000) : empty ? 0.f : scale_of<kFp8>(big);
  }
}

template <bool kFp8, int LR, int V>
__global__ void __launch_bounds__(kThreads) cache_load4_kernel(CacheArgs a) {
  const int lane = threadIdx.x % LR;
  const long long row0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / LR;
  const long long step = (long long)gridDim.x * kThreads / LR;
  const int n4 = a.N / 4;
  uint32_t v[kRows][V];
  float sc[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const long long row = row0 + r * step;
    sc[r] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) v[r][i] = 0u;
    if (row < a.rows) {
      const long long bi = row / a.hp, slot = a.slots ? a.slots[bi] : bi;
      if (slot >= 0 && slot < a.nslots) {
        const long long from = slot * a.hp + (row - bi * a.hp);
        sc[r] = a.scales[from];
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i * LR + lane < n4) v[r][i] = reinterpret_cast<const uint32_t*>(a.vals)[from * n4 + i * LR + lane];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const long long row = row0 + r * step;
    if (row >= a.rows) break;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int n = i * LR + lane;
      const uint32_t x = v[r][i];
      if (n < n4)
        __stcs(reinterpret_cast<float4*>(a.out) + row * n4 + n,
               make_float4(decode<kFp8>(x & 255) * sc[r], decode<kFp8>((x >> 8) & 255) * sc[r],
                           decode<kFp8>((x >> 16) & 255) * sc[r], decode<kFp8>(x >> 24) * sc[r]));
    }
  }
}

template <bool kFp8, int LR, int V>
void launch4(const CacheArgs& a, bool store, cudaStream_t s) {
  const long long per = kThreads / LR * kRows;
  const unsigned grid = (unsigned)((a.rows + per - 1) / per);
  if (store)
    cache_store4_kernel<kFp8, LR, V><<<grid, kThreads, 0, s>>>(a);
  else
    cache_load4_kernel<kFp8, LR, V><<<grid, kThreads, 0, s>>>(a);
}

template <bool kFp8>
void launch_cache(const CacheArgs& a, bool store, cudaStream_t s) {
  if (a.N % 4 == 0) {
    const int n4 = a.N / 4;
    if (n4 <= 4) launch4<kFp8, 4, 1>(a, store, s);
    else if (n4 <= 8) launch4<kFp8, 8, 1>(a, store, s);
    else if (n4 <= 16) launch4<kFp8, 16, 1>(a, store, s);
    else if (n4 <= 32) launch4<kFp8, 32, 1>(a, store, s);
    else launch4<kFp8, 32, 2>(a, store, s);
    return;
  }
  const unsigned grid = (unsigned)((a.rows + kThreads / 32 - 1) / (kThreads / 32));
  if (store)
    cache_store_kernel<kFp8><<<grid, kThreads, 0, s>>>(a);
  else
    cache_load_kernel<kFp8><<<grid, kThreads, 0, s>>>(a);
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
  prof_before(s);
  set_kernel_name(store ? "state_cache_store" : "state_cache_load");
  if (pr->format == SSD_CACHE_E4M3)
    launch_cache<true>(a, store, s);
  else
    launch_cache<false>(a, store, s);
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
