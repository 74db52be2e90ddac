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
// the first words and 10 to the fourth 16 KB of each CTA.  batch 4 of 32,000 fp32
// words: 10 us; batch 128 of 100,003 bf16 words (102 MB): 28 to 30 us, 3.5 TB/s.  Words
// whose bounds were checked one by one, with a best ratio of each thread's own,
// took 48 instructions each and 38 us there.
#include <cooperative_groups.h>

#include "ssd_internal.cuh"

#include <type_traits>

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

// What one thread has met of the race, in ascending order of the words, so
// that the first of equal ratios stays.  A ratio is divided out only where an
// estimate of it (off by a few units of 2^-23, where divisor and ratio are
// neither huge nor tiny) says that it may be the largest that the warp has met
// yet; ratios that are not above zero, or are NaN, never are.
struct Race {
  float top = 0.f, bar = 0.f;
  unsigned at = 0;
  __device__ __forceinline__ bool may_win(float w, float r) const {
    return w > 0.f && (!(__fdividef(w, r) < bar) || r > 8e37f);
  }
  // K words, a step apart; the warp's lanes come together
  template <int K>
  __device__ __forceinline__ void meet(const float (&w)[K], const float (&r)[K], unsigned v, unsigned step) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < K; ++i) any |= may_win(w[i], r[i]);
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (may_win(w[i], r[i])) {
          const float s = w[i] / r[i];
          if (s > top) {
            top = s;
            at = v + i * step;
          }
        }
      const float s = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      bar = s > 1e-37f ? s * 0.999f : 0.f;
    }
  }
};

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1) verify_draft_kernel(VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  // Another CTA's shared memory may be written only once that CTA is known to
  // have started: each says so here, and the wait comes before the first such
  // write, long after the others have arrived.
  cluster.barrier_arrive();
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
    Race race;
    // A CTA's words in tiles of eight to a thread: unconditional loads, all in
    // flight before the first is used; whole tiles need no bounds, in the last
    // one what lies past the end is read from the last word and weighs nothing
    constexpr int kAhead = 8;
    const bool minus = round == 0 && q;
    const int gone = round == 0 ? one : -1;
    auto tile = [&](unsigned u0, auto whole) {
      const unsigned v0 = u0 + threadIdx.x;
      const T *pt = p + v0, *qt = q + v0;
      const float* rt = noise + v0;
      float w[kAhead], r[kAhead];
      T pv[kAhead], qv[kAhead];
      auto at = [&](int i) { return decltype(whole)::value ? i * kThreads : (int)(min(v0 + i * kThreads, hi - 1) - v0); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        pv[i] = pt[at(i)];
        r[i] = rt[at(i)];
      }
      if (minus) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) qv[i] = qt[at(i)];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = to_f(pv[i]) - to_f(qv[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = to_f(pv[i]);
      }
      if (gone >= 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] -= v0 + i * kThreads == gone ? 1.f : 0.f;
      }
      if (!decltype(whole)::value) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = v0 + i * kThreads < hi ? w[i] : 0.f;
      }
      race.meet(w, r, v0, kThreads);
    };
    constexpr unsigned kTile = kAhead * kThreads;
    unsigned u0 = lo;
    for (; u0 < hi && hi - u0 >= kTile; u0 += kTile) tile(u0, std::true_type());
    if (u0 < hi) tile(u0, std::false_type());
    unsigned long long key = race_key(race.top, race.at);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
      key = k > key ? k : key;
    }
    if (lane == 0) warp_best[threadIdx.x >> 5] = key;
    __syncthreads();
    if (round == 0) cluster.barrier_wait();
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
  // row anew (batch 128, 100,003 words, before other savings: 38 us in one wave, 41 in two).  Wide CTAs while each has
  // an SM of its own (batch 4, 32,000 words: 11 us, with narrow ones 12; batch 128 of 5,000: 19 and 12).
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
