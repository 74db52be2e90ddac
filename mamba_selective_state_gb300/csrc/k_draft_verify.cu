// k_draft_verify.cu -- verification of drafted tokens: how many of a
// sequence's drafted tokens the target keeps, and the token after them.
//
// The kept number comes from a few gathered probabilities; the next token is
// the argmax over the vocabulary of w(v) / noise(v), a race of exponentials
// whose winner is distributed as w.  Only the row of the first refused token
// is read.  One cluster of CTAs per sequence splits the vocabulary and joins
// its winners through distributed shared memory, so there is no workspace, no
// atomic and no second launch; the join takes the largest of (ratio, lowest
// index) keys, which does not depend on the order.
//
// Bound by the dependent reads before the row (the drafted tokens, their
// probabilities) and the first touch of rows that lie megabytes apart: 4 us to
// the first words and 10 to the fourth 16 KB of each CTA, after which they come
// at 7 TB/s.  batch 4 of 32,000 words: 11 us; batch 128 of 100,003 (102 MB):
// 38 us, 2.7 TB/s.  A ring of bulk copies instead of the loads into registers
// took 35 us there and 29 instead of 28 at batch 64 of 128,000 fp32 words.
#include <cooperative_groups.h>

#include "ssd_internal.cuh"

namespace ssd {

int device_check();

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;

struct VerifyArgs {
  const void *p, *q;
  const int32_t* tok;
  const int32_t* lengths;
  const float *uniform, *noise;
  int32_t *out, *accepted;
  long long V;
  int K;
};

// Larger ratio first, then lower index; key 0 means none.
__device__ __forceinline__ unsigned long long race_key(float s, unsigned v) {
  return s > 0.f ? ((unsigned long long)__float_as_uint(s) << 32) | (0xffffffffu - v) : 0ull;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1) verify_draft_kernel(VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned ncta = cluster.num_blocks(), rank = cluster.block_rank();
  const long long b = blockIdx.x / ncta;
  __shared__ int kept_s, len_s;
  __shared__ unsigned long long warp_best[kThreads / 32];
  __shared__ unsigned long long cta_best[2][kMaxCluster];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.K) : a.K;
    int kept = len;
    for (int i0 = 0; i0 < len && kept == len; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < a.K) {
        // (loads that do not wait for the sequence's length)
        const long long x = a.tok[b * a.K + i];
        const float u = a.uniform[b * a.K + i];
        ok = i >= len;
        if (!ok && x >= 0 && x < a.V) {
          const float pv = to_f(static_cast<const T*>(a.p)[(b * (a.K + 1) + i) * a.V + x]);
          const float qv = a.q ? to_f(static_cast<const T*>(a.q)[(b * a.K + i) * a.V + x]) : 1.f;
          ok = u * qv < pv;
        }
      }
      const unsigned bad = __ballot_sync(0xffffffffu, !ok);
      if (bad) kept = i0 + __ffs(bad) - 1;
    }
    if (lane == 0) {
      kept_s = kept;
      len_s = len;
    }
  }
  __syncthreads();
  const int kept = kept_s;
  const bool refused = kept < len_s;
  const T* p = static_cast<const T*>(a.p) + (b * (a.K + 1) + kept) * a.V;
  const T* q = refused && a.q ? static_cast<const T*>(a.q) + (b * a.K + kept) * a.V : nullptr;
  const int one = refused && !a.q ? a.tok[b * a.K + kept] : -1;
  const float* noise = a.noise + b * a.V;
  // (a row's words are counted in 32 bits)
  const unsigned V = (unsigned)a.V, per = (V + ncta - 1) / ncta;
  const unsigned lo = min(rank * per, V), hi = min(lo + per, V);
  // round 0: the residual weights; round 1, only where none was positive: p
  unsigned long long best = 0;
  for (int round = 0; round < 2; ++round) {
    // A thread meets its words in ascending order, so the first of equal ratios
    // stays.  A ratio is divided out only where an estimate of it (off by a few
    // units of 2^-23, where divisor and ratio are neither huge nor tiny) says
    // that it may be the largest yet; ratios that are not above zero, or are
    // NaN, never are.
    float top = 0.f, bar = 0.f;
    unsigned at = 0;
    constexpr int kAhead = 8;
    for (unsigned v0 = lo + threadIdx.x; v0 < hi; v0 += kAhead * kThreads) {
      // (unconditional loads, past the end of the last word: all are in flight before the first is used)
      float w[kAhead], r[kAhead];
      T pv[kAhead], qv[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned v = min(v0 + i * kThreads, hi - 1);
        pv[i] = p[v];
        r[i] = noise[v];
      }
      if (round == 0 && q) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) qv[i] = q[min(v0 + i * kThreads, hi - 1)];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = to_f(pv[i]) - to_f(qv[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = to_f(pv[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) w[i] = v0 + i * kThreads < hi ? w[i] : 0.f;
      if (round == 0 && one >= 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] -= v0 + i * kThreads == one ? 1.f : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned v = v0 + i * kThreads;
        if (w[i] > 0.f && (!(__fdividef(w[i], r[i]) < bar) || r[i] > 8e37f)) {
          const float s = w[i] / r[i];
          if (s > top) {
            top = s;
            at = v;
            bar = s > 1e-37f ? s * 0.999f : 0.f;
          }
        }
      }
    }
    unsigned long long key = race_key(top, at);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
      key = k > key ? k : key;
    }
    if (lane == 0) warp_best[threadIdx.x >> 5] = key;
    __syncthreads();
    if (threadIdx.x < 32) {
      key = lane < kThreads / 32 ? warp_best[lane] : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
      }
      // every CTA of the cluster gets every other's winner
      if (lane < ncta) *cluster.map_shared_rank(&cta_best[round][rank], lane) = key;
    }
    cluster.sync();
    best = 0;
    for (unsigned i = 0; i < ncta; ++i) best = cta_best[round][i] > best ? cta_best[round][i] : best;
    if (best != 0 || !refused) break;
  }
  if (rank == 0) {
    const int next = best ? (int)(0xffffffffu - (unsigned)best) : 0;
    for (int i = threadIdx.x; i <= a.K; i += kThreads)
      a.out[b * (a.K + 1) + i] = i < kept ? a.tok[b * a.K + i] : i == kept ? next : -1;
    if (threadIdx.x == 0) a.accepted[b] = kept;
  }
}

template <typename T, int kThreads>
cudaError_t launch_verify_t(const VerifyArgs& a, int64_t batch, int ncta, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(batch * ncta));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ncta;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  set_kernel_name("verify_draft");
  return cudaLaunchKernelEx(&cfg, verify_draft_kernel<T, kThreads>, a);
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs& a, int64_t batch, cudaStream_t s) {
  // CTAs per sequence: one for each 2048 words of the vocabulary, in powers of two up to the portable cluster size,
  // but no more than are resident at once, four narrow ones to an SM: every wave has the dependent reads before its
  // row anew (batch 128, 100,003 words: 38 us in one wave, 41 in two).  Wide CTAs while each has an SM of its own
  // (batch 4, 32,000 words: 11 us, with narrow ones 12; batch 128 of 5,000: 19 and 12).
  const int sms = device_sm_count();
  int ncta = 1;
  while (ncta < kMaxCluster && (long long)ncta * 2048 < a.V && batch * ncta * 2 <= 4 * sms) ncta *= 2;
  return batch * ncta <= sms ? launch_verify_t<T, 512>(a, batch, ncta, s)
                                           : launch_verify_t<T, 256>(a, batch, ncta, s);
}

bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" int ssd_verify_draft(const ssd_verify_problem* pr, const void* target_probs, const void* draft_probs,
                                const int32_t* draft_tokens, const int32_t* lengths, const float* uniform,
                                const float* noise, int32_t* out_tokens, int32_t* accepted, ssd_stream_t stream) {
  if (!pr || pr->batch < 1 || pr->ndraft < 0 || pr->vocab < 1 || pr->flags != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->dtype != SSD_F32 && pr->dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
  // 32-bit indices into a row, positions and grid; 2^40 elements per tensor
  if (pr->vocab >= (1LL << 31) || pr->ndraft >= (1 << 20) || pr->batch >= (1 << 24) ||
      (double)pr->batch * (double)(pr->ndraft + 1) * (double)pr->vocab >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  if (!target_probs || !noise || !out_tokens || !accepted) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->ndraft > 0 && (!draft_tokens || !uniform)) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {target_probs, draft_probs, draft_tokens, lengths, uniform, noise, out_tokens, accepted};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  const int rc = device_check();
  if (rc != SSD_OK) return rc;
  VerifyArgs a = {target_probs, draft_probs, draft_tokens, lengths, uniform, noise,
                  out_tokens,   accepted,    pr->vocab,    (int)pr->ndraft};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = pr->dtype == SSD_BF16 ? launch_verify<__nv_bfloat16>(a, pr->batch, s)
                                              : launch_verify<float>(a, pr->batch, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
