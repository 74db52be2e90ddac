// k_token_logprobs.cu -- log probabilities of given tokens with the entropy and
// the top alternatives of their distributions, the gradient to the logits, and
// their C ABI.
//
//   z = scale logits     lse = log sum exp z      logprob = z[token] - lse
//   entropy = -sum p log p = ln s - t / s   with  s = sum e^(z - m),  t = sum e^(z - m) (z - m)
//   dlogits = scale (dlogprob (1[token] - p) - dentropy p (log p + entropy))
//
// Forward: one pass over the logits, bound by HBM where there are many rows.  A
// CTA, or a cluster of up to eight where rows are few, takes a row; each thread
// keeps the largest logit that it has met and the two sums relative to it, in
// units of log 2, and they are joined in a fixed order.
//
// Alternatives.  The k-th largest of the maxima of 64 groups of threads is at
// most the row's k-th largest logit: every alternative is at or above that
// bound, so only threads whose maximum is have any.  Their words are read once
// more (one vector to a lane), what reaches the bound is put on a list, and
// counting who is ahead of whom sorts the list.  A list that overflows (many
// equal logits) is replaced by k passes over the words that find the next
// largest each.
#include <cooperative_groups.h>

#include "ssd_internal.cuh"

#include <type_traits>

namespace ssd {

int device_check();

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroups = 64;      // groups of threads whose maxima give the bound
constexpr int kMaxTop = 32;      // alternatives
constexpr int kMaxCluster = 8;
constexpr int kList = 512;       // words that may reach the bound
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

struct LogpArgs {
  const void* logits;
  const int32_t* tokens;
  float *logprobs, *entropy, *lse;
  int32_t* top_tok;
  float* top_lp;
  const float *lse_in, *ent_in, *dlogp, *dent;
  void* dlogits;
  long long rows, V, stride, gstride;
  float scale, c2;  // c2 = scale log2(e)
  int ntop;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A difference of exponents, kept where the exponential is zero and its product
// with the exponent too; a NaN stays one.
__device__ __forceinline__ float floored(float d) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(d), "f"(-200.f));
  return y;
}

// Exponents are (x - m) c2: fma(x, c2, -rn(m c2)) saves the difference's own
// operation.  It is off by off_of(m), the same for every word met under m, which
// the joins take back; from 2^10 on, where that would no longer be little, the
// difference is formed.
__device__ __forceinline__ bool by_product(float mc) { return fabsf(mc) < 1024.f; }
__device__ __forceinline__ float off_of(float m, float c2) {
  const float mc = __fmul_rn(m, c2);
  return by_product(mc) ? fmaf(m, c2, -mc) : 0.f;
}
// The factor's exponent from sums under a to sums under b
__device__ __forceinline__ float apart(float a, float b, float c2) {
  return fmaf(a - b, c2, off_of(b, c2) - off_of(a, c2));
}

// What has been met of a row: the largest logit m, and the sums of 2^d and of
// 2^d d over its words, d = (x - m) c2.
struct Sums {
  float m = kNegInf, s = 0.f, t = 0.f;
  __device__ __forceinline__ void rebase(float m2, float c2) {
    if (m == kNegInf) return;  // (s may be a NaN: it stays)
    const float d = floored(apart(m, m2, c2)), f = ex2(d);
    t = f * (t + s * d);
    s = f * s;
    m = m2;
  }
  __device__ __forceinline__ void join(float m2, float s2, float t2, float c2) {
    Sums o;
    o.m = m2; o.s = s2; o.t = t2;
    const float top = fmaxf(m, m2);
    if (top > m) rebase(top, c2);
    if (top > m2) o.rebase(top, c2);
    m = top;
    s += o.s;
    t += o.t;
  }
  template <int K>
  __device__ __forceinline__ void meet(const float (&x)[K], float c2) {
    float b = x[0];
#pragma unroll
    for (int i = 1; i < K; ++i) b = fmaxf(b, x[i]);
    if (b > m) {
      rebase(b, c2);
      m = b;
    }
    if (m == kNegInf) {  // nothing but excluded words, or NaN
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (x[i] != x[i]) s = x[i];
      return;
    }
    const float mc = __fmul_rn(m, c2);
    if (by_product(mc)) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float d = floored(fmaf(x[i], c2, -mc)), e = ex2(d);
        s += e;
        t = fmaf(e, d, t);
      }
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float d = floored((x[i] - m) * c2), e = ex2(d);
        s += e;
        t = fmaf(e, d, t);
      }
    }
  }
};

// A row seen as 16-byte vectors of memory: its first and last words may share
// theirs with other rows and are taken one by one.
template <typename T>
struct Row {
  static constexpr int n = 16 / sizeof(T);
  const T* base;      // the row's first word
  const uint4* vec;   // the first whole vector
  unsigned V, head, nvec, tail;
  __device__ __forceinline__ Row(const void* p, long long row, long long stride, long long words) {
    base = static_cast<const T*>(p) + row * stride;
    V = (unsigned)words;
    const unsigned off = (unsigned)((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
    head = min(off ? n - off : 0u, V);
    vec = reinterpret_cast<const uint4*>(base + head);
    nvec = (V - head) / n;
    tail = V - head - nvec * n;
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
};

// Larger logit first, then lower index; key 0 means none.
__device__ __forceinline__ unsigned long long word_key(float x, unsigned v) {
  const unsigned b = __float_as_uint(x + 0.f);
  return (unsigned long long)(b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u)) << 32 | (0xffffffffu - v);
}
__device__ __forceinline__ float key_logit(unsigned long long k) {
  const unsigned b = (unsigned)(k >> 32);
  return __uint_as_float(b ^ ((int)b < 0 ? 0x80000000u : 0xffffffffu));
}

struct TopShared {
  float group[kGroups];
  unsigned long long list[kList];
  unsigned long long warp[kWarps];
  int count;
};

// The words of thread `of` of this CTA, one vector to a lane at a time: f(logit, index)
template <typename T, typename F>
__device__ __forceinline__ void words_of(const Row<T>& r, unsigned lo, unsigned hi, bool first, int of, int lane, F f) {
  constexpr int n = Row<T>::n;
  for (unsigned v = lo + of + lane * kThreads; v < hi; v += 32 * kThreads) {
    float x[n];
    Row<T>::unpack(r.vec[v], x);
#pragma unroll
    for (int i = 0; i < n; ++i) f(x[i], r.head + v * n + i);
  }
  if (first && of == 0 && (unsigned)lane < r.head) f(to_f(r.base[lane]), (unsigned)lane);
  if (first && of == 1 && (unsigned)lane < r.tail) f(to_f(r.base[r.V - r.tail + lane]), r.V - r.tail + lane);
}

// This CTA's k largest words, in order, to `to` (0 where there is none)
template <typename T>
__device__ void cta_top(const Row<T>& r, unsigned lo, unsigned hi, bool first, float mine, int k, TopShared& sh,
                        unsigned long long* to) {
  const int lane = threadIdx.x & 31;
  float g = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((threadIdx.x & 3) == 0) sh.group[threadIdx.x >> 2] = g;
  if (threadIdx.x == 0) sh.count = 0;
  if (threadIdx.x < kMaxTop) to[threadIdx.x] = 0;
  __syncthreads();
  // (every warp finds the bound for itself)
  const float a = sh.group[lane], b = sh.group[lane + 32];
  int ra = 0, rb = 0;
#pragma unroll 16
  for (int i = 0; i < kGroups; ++i) {
    const float o = sh.group[i];
    ra += o > a || (o == a && i < lane);
    rb += o > b || (o == b && i < lane + 32);
  }
  const unsigned ha = __ballot_sync(0xffffffffu, ra == k - 1), hb = __ballot_sync(0xffffffffu, rb == k - 1);
  const float bound = ha ? __shfl_sync(0xffffffffu, a, __ffs(ha) - 1) : __shfl_sync(0xffffffffu, b, __ffs(hb) - 1);
  for (unsigned has = __ballot_sync(0xffffffffu, mine >= bound && mine > kNegInf); has; has &= has - 1)
    words_of(r, lo, hi, first, (int)(threadIdx.x & ~31u) + __ffs(has) - 1, lane, [&](float x, unsigned v) {
      if (x >= bound && x > kNegInf) {
        const int at = atomicAdd(&sh.count, 1);  // (the list's order does not matter)
        if (at < kList) sh.list[at] = word_key(x, v);
      }
    });
  __syncthreads();
  const int count = sh.count;
  if (count <= kList) {
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const unsigned long long key = sh.list[i];
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += sh.list[j] > key;
      if (rank < k) to[rank] = key;
    }
  } else {
    unsigned long long last = ~0ull;
    for (int i = 0; i < k && last; ++i) {
      unsigned long long best = 0;
      for (int of = (int)(threadIdx.x & ~31u), end = of + 32; of < end; ++of)
        words_of(r, lo, hi, first, of, lane, [&](float x, unsigned v) {
          if (x >= bound && x > kNegInf) {
            const unsigned long long key = word_key(x, v);
            if (key < last && key > best) best = key;
          }
        });
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
      }
      if (lane == 0) sh.warp[threadIdx.x >> 5] = best;
      __syncthreads();
      best = 0;
      for (int w = 0; w < kWarps; ++w) best = sh.warp[w] > best ? sh.warp[w] : best;
      if (threadIdx.x == 0) to[i] = best;
      last = best;
      __syncthreads();
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(LogpArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  // Another CTA's shared memory may be written only once that CTA is known to
  // have started: each says so here, and the wait comes before the first such write.
  cluster.barrier_arrive();
  const unsigned ncta = cluster.num_blocks(), rank = cluster.block_rank();
  const long long row = blockIdx.x / ncta;
  __shared__ TopShared sh;
  __shared__ float warp_sums[kWarps][3], cta_sums[kMaxCluster][3];
  __shared__ unsigned long long mine[kMaxTop], all[kMaxCluster * kMaxTop];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int n = Row<T>::n, kAhead = 4;
  const Row<T> r(a.logits, row, a.stride, a.V);
  const bool first = rank == 0;
  const int tok = a.tokens ? a.tokens[row] : -1;
  const bool known = tok >= 0 && tok < a.V;
  float tok_x = 0.f;
  if (first && known) tok_x = to_f(r.base[tok]);
  const unsigned per = (r.nvec + ncta - 1) / ncta, lo = min(rank * per, r.nvec), hi = min(lo + per, r.nvec);
  Sums sum;
  float top = kNegInf;
  auto tile = [&](unsigned v0, auto whole) {
    uint4 u[kAhead];
    const uint4* at = r.vec + v0 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (decltype(whole)::value || v0 + threadIdx.x + i * kThreads < hi) {
        u[i] = __ldg(at + i * kThreads);
      } else {  // nothing there: excluded words
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        u[i] = make_uint4(none, none, none, none);
      }
    }
    float x[kAhead * n];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) Row<T>::unpack(u[i], x + i * n);
    sum.meet(x, a.c2);
  };
  constexpr unsigned kTile = kAhead * kThreads;
  unsigned v0 = lo;
  for (; v0 < hi && hi - v0 >= kTile; v0 += kTile) tile(v0, std::true_type());
  if (v0 < hi) tile(v0, std::false_type());
  if (first && threadIdx.x < 2) {
    const unsigned cnt = threadIdx.x == 0 ? r.head : r.tail, from = threadIdx.x == 0 ? 0 : r.V - r.tail;
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = (unsigned)i < cnt ? to_f(r.base[from + i]) : kNegInf;
    sum.meet(x, a.c2);
  }
  top = sum.m;
#pragma unroll
  for (int o = 16; o; o >>= 1)
    sum.join(__shfl_down_sync(0xffffffffu, sum.m, o), __shfl_down_sync(0xffffffffu, sum.s, o),
             __shfl_down_sync(0xffffffffu, sum.t, o), a.c2);
  if (lane == 0) {
    warp_sums[warp][0] = sum.m;
    warp_sums[warp][1] = sum.s;
    warp_sums[warp][2] = sum.t;
  }
  if (a.ntop) cta_top<T>(r, lo, hi, first, top, a.ntop, sh, mine);
  else __syncthreads();
  cluster.barrier_wait();
  if (threadIdx.x == 0) {
    Sums c;
    for (int w = 0; w < kWarps; ++w) c.join(warp_sums[w][0], warp_sums[w][1], warp_sums[w][2], a.c2);
    float* to = cluster.map_shared_rank(&cta_sums[rank][0], 0);
    to[0] = c.m;
    to[1] = c.s;
    to[2] = c.t;
  }
  if ((int)threadIdx.x < a.ntop) *cluster.map_shared_rank(&all[rank * a.ntop + threadIdx.x], 0) = mine[threadIdx.x];
  cluster.sync();
  if (!first) return;
  Sums c;
  for (unsigned w = 0; w < ncta; ++w) c.join(cta_sums[w][0], cta_sums[w][1], cta_sums[w][2], a.c2);
  const bool nothing = c.m == kNegInf && c.s == 0.f;  // every word is excluded
  const float ln_s = logf(c.s) - off_of(c.m, a.c2) * kLn2;  // ln sum e^(z - m)
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[row] = nothing ? kNegInf : fmaf(c.m, a.scale, ln_s);
    if (a.entropy) a.entropy[row] = nothing ? 0.f : logf(c.s) - kLn2 * (c.t / c.s);
    if (a.logprobs) a.logprobs[row] = !known ? 0.f : nothing ? kNegInf : (tok_x - c.m) * a.scale - ln_s;
  }
  const int have = (int)ncta * a.ntop;
  for (int i = threadIdx.x; i < have; i += kThreads) {
    const unsigned long long key = all[i];
    int at = 0;
    if (ncta > 1) {
      for (int j = 0; j < have; ++j) at += all[j] > key || (all[j] == key && j < i);
    } else {
      at = i;
    }
    if (at < a.ntop) {
      const long long o = row * a.ntop + at;
      a.top_tok[o] = key ? (int)(0xffffffffu - (unsigned)key) : -1;
      a.top_lp[o] = key ? (key_logit(key) - c.m) * a.scale - ln_s : kNegInf;
    }
  }
}

// One CTA to a row's run of vectors.  kSame: the gradient's rows lie in their
// vectors as the logits' do.
template <typename T, bool kSame>
__global__ void __launch_bounds__(kThreads) token_logprobs_bwd_kernel(LogpArgs a, unsigned per) {
  const long long row = blockIdx.x;
  constexpr int n = Row<T>::n, kAhead = 4;
  const Row<T> r(a.logits, row, a.stride, a.V);
  T* out = static_cast<T*>(a.dlogits) + row * a.gstride;
  const float lse = a.lse_in[row], H = a.ent_in ? a.ent_in[row] : 0.f;
  const int t = a.tokens ? a.tokens[row] : -1;
  const unsigned tok = t >= 0 && t < a.V ? (unsigned)t : 0xffffffffu;
  const float dl = tok != 0xffffffffu && a.dlogp ? a.dlogp[row] : 0.f, dH = a.dent ? a.dent[row] : 0.f;
  const bool nothing = lse == kNegInf;
  // p (-dl - dH (log p + H)) with log p = z - lse
  auto grad = [&](float x, unsigned v) {
    const float lp = floored(fmaf(x, a.scale, -lse)), p = ex2(lp * kLog2e);
    float g = -p * fmaf(dH, lp + H, dl);
    if (v == tok) g += dl;
    return nothing ? 0.f : g * a.scale;
  };
  auto one = [&](unsigned v) { out[v] = from_f<T>(grad(to_f(r.base[v]), v)); };
  if (blockIdx.y == 0) {
    if (threadIdx.x < r.head) one(threadIdx.x);
    if (threadIdx.x < r.tail) one(r.V - r.tail + threadIdx.x);
  }
  for (unsigned b = blockIdx.y * per; b < r.nvec; b += gridDim.y * per) {
    const unsigned hi = min(b + per, r.nvec);
    for (unsigned v0 = b + threadIdx.x; v0 < hi; v0 += kAhead * kThreads) {
      uint4 u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (v0 + i * kThreads < hi) u[i] = r.vec[v0 + i * kThreads];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned v = v0 + i * kThreads;
        if (v >= hi) break;
        float x[n];
        Row<T>::unpack(u[i], x);
        const unsigned w = r.head + v * n;
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = grad(x[j], w + j);
        if (!kSame) {
#pragma unroll
          for (int j = 0; j < n; ++j) out[w + j] = from_f<T>(x[j]);
        } else if constexpr (sizeof(T) == 2) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            q[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          __stcs(reinterpret_cast<uint4*>(out + w), make_uint4(q[0], q[1], q[2], q[3]));
        } else {
          __stcs(reinterpret_cast<float4*>(out + w), make_float4(x[0], x[1], x[2], x[3]));
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_fwd(const LogpArgs& a, cudaStream_t s) {
  // CTAs to a row: more, in powers of two up to the portable cluster size, while all of them are resident at once and
  // each has more than 2048 words.
  const int sms = device_sm_count();
  int ncta = 1;
  while (ncta < kMaxCluster && (long long)ncta * 2048 < a.V && a.rows * ncta * 2 <= 4 * sms) ncta *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * ncta));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ncta;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  set_kernel_name("token_logprobs");
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a);
}

template <typename T>
cudaError_t launch_bwd(const LogpArgs& a, cudaStream_t s) {
  // runs of 4 tiles where there are rows enough, else of one
  const long long vecs = (a.V * (long long)sizeof(T) + 15) / 16;
  const unsigned per = 4 * kThreads * (a.rows >= 4 * device_sm_count() ? 4 : 1);
  long long runs = (vecs + per - 1) / per;
  if (runs < 1) runs = 1;
  if (runs > 65535) runs = 65535;
  const bool same = ((reinterpret_cast<uintptr_t>(a.dlogits) - reinterpret_cast<uintptr_t>(a.logits)) & 15u) == 0 &&
                    ((a.stride - a.gstride) * (long long)sizeof(T)) % 16 == 0;
  const dim3 grid((unsigned)a.rows, (unsigned)runs);
  set_kernel_name("token_logprobs_bwd");
  if (same) token_logprobs_bwd_kernel<T, true><<<grid, kThreads, 0, s>>>(a, per);
  else token_logprobs_bwd_kernel<T, false><<<grid, kThreads, 0, s>>>(a, per);
  return cudaGetLastError();
}

int check(const ssd_logprob_problem* pr, LogpArgs* a) {
  if (!pr || pr->rows < 1 || pr->vocab < 1 || pr->flags != 0) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->dtype != SSD_F32 && pr->dtype != SSD_BF16) return SSD_ERR_INVALID_ARGUMENT;
  if (pr->ntop < 0 || !(pr->scale > 0.f && pr->scale <= 3.402823466e38f)) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t ls = pr->logit_stride ? pr->logit_stride : pr->vocab, gs = pr->grad_stride ? pr->grad_stride : pr->vocab;
  if (ls < pr->vocab || gs < pr->vocab) return SSD_ERR_INVALID_ARGUMENT;
  // 32-bit indices into a row and CTAs of a grid; 2^40 elements per tensor
  const int64_t wide = ls > gs ? ls : gs;
  if (pr->ntop > kMaxTop || pr->vocab >= (1LL << 31) || pr->rows >= (1LL << 28) ||
      (double)pr->rows * (double)wide >= (double)(1LL << 40))
    return SSD_ERR_UNSUPPORTED;
  *a = LogpArgs();
  a->rows = pr->rows;
  a->V = pr->vocab;
  a->stride = ls;
  a->gstride = gs;
  a->scale = pr->scale;
  a->c2 = pr->scale * kLog2e;
  a->ntop = pr->ntop;
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_token_logprobs(const ssd_logprob_problem* pr, const void* logits, const int32_t* tokens, float* logprobs,
                       float* entropy, float* lse, int32_t* top_tokens, float* top_logprobs, ssd_stream_t stream) {
  LogpArgs a;
  int rc = check(pr, &a);
  if (rc != SSD_OK) return rc;
  if (!logits || (logprobs != nullptr) != (tokens != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if ((pr->ntop > 0) != (top_tokens != nullptr) || (pr->ntop > 0) != (top_logprobs != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!logprobs && !entropy && !lse && !top_tokens) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {logits, tokens, logprobs, entropy, lse, top_tokens, top_logprobs};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  a.logits = logits; a.tokens = tokens; a.logprobs = logprobs; a.entropy = entropy; a.lse = lse;
  a.top_tok = top_tokens; a.top_lp = top_logprobs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = pr->dtype == SSD_BF16 ? launch_fwd<__nv_bfloat16>(a, s) : launch_fwd<float>(a, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_token_logprobs_bwd(const ssd_logprob_problem* pr, const void* logits, const int32_t* tokens, const float* lse,
                           const float* entropy, const float* dlogprobs, const float* dentropy, void* dlogits,
                           ssd_stream_t stream) {
  LogpArgs a;
  int rc = check(pr, &a);
  if (rc != SSD_OK) return rc;
  if (!logits || !lse || !dlogits || (!dlogprobs && !dentropy)) return SSD_ERR_INVALID_ARGUMENT;
  if ((dlogprobs != nullptr) != (tokens != nullptr) || (dentropy != nullptr) != (entropy != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (dlogits == logits && a.stride != a.gstride) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {logits, tokens, lse, entropy, dlogprobs, dentropy, dlogits};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  a.logits = logits; a.tokens = tokens; a.lse_in = lse; a.ent_in = entropy; a.dlogp = dlogprobs; a.dent = dentropy;
  a.dlogits = dlogits;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = pr->dtype == SSD_BF16 ? launch_bwd<__nv_bfloat16>(a, s) : launch_bwd<float>(a, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
