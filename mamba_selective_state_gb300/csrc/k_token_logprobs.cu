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
// units of log 2, and they are joined in a fixed order.  A CTA goes on to its
// next row while the joins of the last one are under way: the first vectors of
// that row are in flight by then.  4096 rows of 100,003 bf16 words: 137 us (6.0
// TB/s), with 20 alternatives 163.  The gradient reads and writes once: 4096 rows
// of 32,000 words 81 us (6.5 TB/s).
//
// Alternatives.  The k-th largest of the maxima of 64 groups of threads is at
// most the row's k-th largest logit: every alternative is at or above that
// bound.  Each thread also keeps the largest logit of every run of its vectors
// in shared memory, so only the runs that reach the bound (about k of them) are
// read once more, all at a time; what reaches the bound is put on a list, and
// counting who is ahead of whom sorts the list.  A list that overflows
// (many equal logits) is replaced by k passes over those words that find the
// next largest each.
#include <cooperative_groups.h>

#include "ssd_internal.cuh"

#include <type_traits>

namespace ssd {

int device_check();

namespace {

namespace cg = cooperative_groups;

constexpr int kBwdThreads = 256;
constexpr int kAhead = 4;        // 16-byte vectors of a thread in flight
constexpr int kGroups = 64;      // groups of threads whose maxima give the bound
constexpr int kMaxTop = 32;      // alternatives
constexpr int kMaxCluster = 8;
constexpr int kList = 512;       // words that may reach the bound
constexpr int kLong = 96;        // a list that is shortened first
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeastScale = 7.52316385e-37f;  // 2^-120: 2^128 of it is an exponent of 256
constexpr float kNegInf = -__builtin_huge_valf();

struct LogpArgs {
  const void* logits;
  const int32_t* tokens;
  float *logprobs, *entropy, *lse;
  float2* stats;
  int32_t* top_tok;
  float* top_lp;
  const float2* stats_in;
  const float *ent_in, *dlogp, *dent;
  void* dlogits;
  long long rows, V, stride, gstride;
  float scale, c2;  // c2 = scale log2(e), rounded:
  float c2_less;    // by this part of itself it is too small, times ln 2
  int ntop;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two values at a time (4096 rows of 100,003 bf16 words: 137 us, one at a time 146)
__device__ __forceinline__ unsigned long long two(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 apart2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// scale (x - m), also of values that are farther apart than fp32's largest
__device__ __forceinline__ float below(float x, float m, float scale) {
  const float d = x - m;
  return fabsf(d) <= 3.402823466e38f ? d * scale : (0.5f * x - 0.5f * m) * scale * 2.f;
}

// What has been met of a row: the largest logit m, and the sums of 2^d and of
// 2^d d over its words, d = (x - m) c2.  Those are added up from sums of a batch
// of words each, which keeps the chains of roundings short.
//
// A row that is nearly all one word has log probabilities and an entropy that are
// as small as what the other words leave, which a sum with that word's 1 would
// round away.  So the batch that holds the first m is kept out of s, in q; a row
// whose sum comes out below 1.5 reads that batch once more and leaves s without
// the word itself (q = kAlone).
constexpr float kAlone = -1.f;
struct Sums {
  float m = kNegInf, s = 0.f, q = 0.f, t = 0.f;
  // q as a sum: the word alone has 2^off
  __device__ __forceinline__ float batch(float c2) const {
    return q == kAlone ? fmaf(off_of(m, c2), kLn2, 1.f) : q;
  }
  __device__ __forceinline__ void rebase(float m2, float c2) {
    if (m == kNegInf) return;  // (s may be a NaN: it stays)
    const float d = floored(apart(m, m2, c2)), f = ex2(d), all = s + batch(c2);
    t = f * (t + all * d);
    s = f * all;
    q = 0.f;
    m = m2;
  }
  __device__ __forceinline__ void join(float m2, float s2, float t2, float q2, float c2) {
    Sums o;
    o.m = m2; o.s = s2; o.t = t2; o.q = q2;
    const float top = fmaxf(m, m2);
    if (top > m) rebase(top, c2);
    if (top > m2) o.rebase(top, c2);
    m = top;
    s += o.s;
    t += o.t;
    if (q == 0.f) q = o.q;
    else if (o.q != 0.f) s += o.batch(c2);
  }
  // A batch's sums; fresh: it holds the first m
  __device__ __forceinline__ void take(bool fresh, float es, float et) {
    if (fresh) q = es;
    else s += es;
    t += et;
  }
  // words of which none is above m; kNear: by_product(m c2)
  template <bool kNear, int K>
  __device__ __forceinline__ void add(const float (&x)[K], float mc, float c2, float& es, float& et) const {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float d = floored(kNear ? fmaf(x[i], c2, -mc) : (x[i] - m) * c2), e = ex2(d);
      es += e;
      et = fmaf(e, d, et);
    }
  }
  // the same two words at a time, near ones
  template <int K>
  __device__ __forceinline__ void add_pairs(const float (&x)[K], unsigned long long mc, unsigned long long c2,
                                            unsigned long long& es, unsigned long long& et) const {
#pragma unroll
    for (int i = 0; i < K; i += 2) {
      const float2 v = apart2(fma2(two(x[i], x[i + 1]), c2, mc));
      const float dx = floored(v.x), dy = floored(v.y);
      const unsigned long long e = two(ex2(dx), ex2(dy));
      es = add2(es, e);
      et = fma2(e, two(dx, dy), et);
    }
  }
  // nothing but excluded words so far: is one a NaN?
  template <int K>
  __device__ __forceinline__ void add_none(const float (&x)[K], float& es) const {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (x[i] != x[i]) es = x[i];
  }
};

// A row seen as 16-byte vectors of memory: its first and last words may share
// theirs with other rows and are taken one by one.
template <typename T>
struct Row {
  static constexpr int n = 16 / sizeof(T);
  const T* base;      // the row's first word
  unsigned V, head, nvec, tail;
  __device__ __forceinline__ Row(const void* p, long long row, long long stride, long long words) {
    base = static_cast<const T*>(p) + row * stride;
    V = (unsigned)words;
    const unsigned off = (unsigned)((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
    head = min(off ? n - off : 0u, V);
    nvec = (V - head) / n;
    tail = V - head - nvec * n;
  }
  __device__ __forceinline__ Row() {}
  // the first whole vector
  __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(base + head); }
  // The largest word of some vectors (NaN passed over)
  template <int K>
  static __device__ __forceinline__ float largest(const uint4 (&u)[K]) {
    if constexpr (sizeof(T) == 2) {
      uint32_t b = u[0].x;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("max.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(w[j]));
      }
      return fmaxf(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    } else {
      float b = kNegInf;
#pragma unroll
      for (int i = 0; i < K; ++i)
        b = fmaxf(fmaxf(fmaxf(b, __uint_as_float(u[i].x)), fmaxf(__uint_as_float(u[i].y), __uint_as_float(u[i].z))),
                  __uint_as_float(u[i].w));
      return b;
    }
  }
  template <int K>
  static __device__ __forceinline__ float meet(Sums& sum, const uint4 (&u)[K], float c2, unsigned here, unsigned& at) {
    const float b = largest(u);
    const bool fresh = b > sum.m;
    if (fresh) {
      sum.rebase(b, c2);
      sum.m = b;
      at = here;
    }
    const float mc = __fmul_rn(sum.m, c2);
    float es = 0.f, et = 0.f;
    if (by_product(mc)) {
      unsigned long long es2 = 0, et2 = 0;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float x[n];
        unpack(u[i], x);
        sum.add_pairs(x, two(-mc, -mc), two(c2, c2), es2, et2);
      }
      const float2 p = apart2(es2), q = apart2(et2);
      es = p.x + p.y;
      et = q.x + q.y;
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float x[n];
        unpack(u[i], x);
        if (sum.m == kNegInf) sum.add_none(x, es);
        else sum.template add<false>(x, mc, c2, es, et);
      }
    }
    sum.take(fresh, es, et);
    return b;
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

template <int kThreads>
struct Shared {
  static constexpr int kRuns = kThreads > 256 ? 8 : 16;  // runs of a thread's vectors
  alignas(16) float group[kGroups];  // (read four at a time)
  float warp[kThreads / 32][4];     // m, s, t, q of the warps
  float all[4];                     // of the CTA
  float alone;                      // s without the largest word, where it is wanted
  int first;                        // the warp whose q is the CTA's
  float cta[kMaxCluster][4];        // of the cluster's CTAs
  unsigned long long best[kThreads / 32];
  alignas(16) unsigned long long list[kList];
  alignas(16) unsigned long long list2[kList];
  alignas(16) unsigned long long part[kGroups];
  unsigned long long near;
  unsigned long long top[kMaxCluster * kMaxTop];
  float run[kRuns][kThreads];       // the largest of each thread's runs
  unsigned short owner[kRuns * kThreads];  // runs that have an alternative
  float bound;
  int owners, count, kept;         // lengths: of owner, of list, of list2
};

// Sums of a warp's first `lanes` lanes (a power of two), in every one of them.
// Returns the lane whose q is theirs, -1 if there is none.
template <int lanes>
__device__ __forceinline__ int join_lanes(Sums& sum, float c2) {
  const unsigned b = __float_as_uint(sum.m);
  const unsigned key = __reduce_max_sync(0xffffffffu, b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u));
  const float m = __uint_as_float(key ^ ((int)key < 0 ? 0x80000000u : 0xffffffffu));
  if (m > sum.m) sum.rebase(m, c2);
  sum.m = m;
  const int first = __ffs(__ballot_sync(0xffffffffu, sum.q != 0.f)) - 1;
  if ((int)(threadIdx.x & 31) != first) sum.s += sum.q;
  sum.q = first < 0 ? 0.f : __shfl_sync(0xffffffffu, sum.q, first);
#pragma unroll
  for (int o = lanes / 2; o; o >>= 1) {
    sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
    sum.t += __shfl_xor_sync(0xffffffffu, sum.t, o);
  }
  return first;
}

// CTAs to an SM: 80 registers to a thread (with 64 what is kept across a row is
// spilled: 4096 rows of 32,000 bf16 words 62 us instead of 51)
constexpr int resident(int threads) { return threads > 256 ? 1 : 768 / threads; }

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, resident(kThreads)) token_logprobs_kernel(LogpArgs a) {
  constexpr int n = Row<T>::n, kWarps = kThreads / 32, kTile = kAhead * kThreads, kRuns = Shared<kThreads>::kRuns;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned ncta = cluster.num_blocks(), rank = cluster.block_rank();
  // Another CTA's shared memory may be written only once that CTA is known to
  // have started: each says so here, and the wait comes before the first such write.
  if (ncta > 1) cluster.barrier_arrive();
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = rank == 0;
  const long long step = gridDim.x / ncta;
  unsigned lo = 0, hi = 0;
  auto take = [&](long long row) {
    const Row<T> r(a.logits, row, a.stride, a.V);
    const unsigned per = (r.nvec + ncta - 1) / ncta;
    lo = min(rank * per, r.nvec);
    hi = min(lo + per, r.nvec);
    return r;
  };
  uint4 u[kAhead];
  auto fetch = [&](const Row<T>& r, unsigned v0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // nothing there: excluded words
      constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
      u[i] = make_uint4(none, none, none, none);
      if (v0 + i * kThreads + tid < hi) u[i] = __ldg(r.vec() + v0 + i * kThreads + tid);
    }
  };
  Row<T> r = take(blockIdx.x / ncta);
  fetch(r, lo);
  for (long long row = blockIdx.x / ncta; row < a.rows; row += step) {
    const int tok = a.tokens ? a.tokens[row] : -1;
    const bool known = tok >= 0 && tok < a.V;
    float tok_x = 0.f;
    if (known) tok_x = to_f(r.base[tok]);
    const Row<T> now = r;
    const unsigned from = lo, to = hi;
    Sums sum;
    constexpr unsigned kEdge = ~0u;
    unsigned at = 0;     // the first vector of the batch in q, or kEdge
    unsigned shift = 0;  // tiles to a run: 1 << shift
    while ((to - from) > ((unsigned)(kRuns * kTile) << shift)) ++shift;
    float run = kNegInf;
    unsigned tile = 0;
#pragma unroll 1
    for (unsigned v0 = from; v0 < to; v0 += kTile, ++tile) {
      uint4 w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) w[i] = u[i];
      if (v0 + kTile < to) fetch(now, v0 + kTile);
      const float b = Row<T>::meet(sum, w, a.c2, v0, at);
      if (a.ntop) {
        run = (tile & ((1u << shift) - 1)) == 0 ? b : fmaxf(run, b);
        sh.run[tile >> shift][tid] = run;
      }
    }
    const unsigned runs = (tile + (1u << shift) - 1) >> shift;
    if (row + step < a.rows) {
      r = take(row + step);
      fetch(r, lo);
    }
    // the words before (0) and behind (1) the whole vectors
    auto edge = [&](int which, float (&x)[n]) {
      const unsigned cnt = which == 0 ? now.head : now.tail, off = which == 0 ? 0 : now.V - now.tail;
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = (unsigned)i < cnt ? to_f(now.base[off + i]) : kNegInf;
    };
    if (first && tid < 2) {
      float x[n], b = kNegInf;
      edge(tid, x);
#pragma unroll
      for (int i = 0; i < n; ++i) b = fmaxf(b, x[i]);
      const bool fresh = b > sum.m;
      if (fresh) {
        sum.rebase(b, a.c2);
        sum.m = b;
        at = kEdge;
      }
      const float mc = __fmul_rn(sum.m, a.c2);
      float es = 0.f, et = 0.f;
      if (sum.m == kNegInf) sum.add_none(x, es);
      else if (by_product(mc)) sum.template add<true>(x, mc, a.c2, es, et);
      else sum.template add<false>(x, mc, a.c2, es, et);
      sum.take(fresh, es, et);
    }
    const float top = sum.m;
    if (a.ntop) {
      float g = top;
#pragma unroll
      for (int o = 1; o < kThreads / kGroups; o *= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (tid % (kThreads / kGroups) == 0) sh.group[tid / (kThreads / kGroups)] = g;
      if (tid == 0) sh.owners = sh.count = sh.kept = 0;
    }
    const int holder = join_lanes<32>(sum, a.c2);
    if (lane == 0) {
      sh.warp[warp][0] = sum.m;
      sh.warp[warp][1] = sum.s;
      sh.warp[warp][2] = sum.t;
      sh.warp[warp][3] = sum.q;
    }
    __syncthreads();
    if (warp == 0) {
      Sums c;
      if (lane < kWarps) {
        c.m = sh.warp[lane][0];
        c.s = sh.warp[lane][1];
        c.t = sh.warp[lane][2];
        c.q = sh.warp[lane][3];
      }
      const int w = join_lanes<kWarps>(c, a.c2);
      if (lane == 0) {
        sh.all[0] = c.m;
        sh.all[1] = c.s;
        sh.all[2] = c.t;
        sh.all[3] = c.q;
        sh.first = w;
      }
    } else if (warp == 1 && a.ntop) {
      // the ntop-th largest of the groups' maxima
      const float x = sh.group[lane], y = sh.group[lane + 32];
      int rx = 0, ry = 0;
#pragma unroll 4
      for (int i = 0; i < kGroups; i += 4) {
        const float4 o = *reinterpret_cast<const float4*>(&sh.group[i]);
        const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rx += v[j] > x || (v[j] == x && i + j < lane);
          ry += v[j] > y || (v[j] == y && i + j < lane + 32);
        }
      }
      if (rx == a.ntop - 1) sh.bound = x;
      if (ry == a.ntop - 1) sh.bound = y;
    }
    __syncthreads();
    const bool alone = sh.all[1] + sh.all[3] < 1.5f && sh.all[3] > 0.f;
    if (alone && warp == sh.first) {
      // that batch again, a vector to a lane, without the first of its words that is m
      const float m = sh.all[0], mc = __fmul_rn(m, a.c2);
      const unsigned v0 = __shfl_sync(0xffffffffu, at, holder);
      float x[n];
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = kNegInf;
      if (v0 == kEdge) {
        if (lane == 0) edge(holder, x);
      } else if (lane < kAhead) {
        const unsigned v = v0 + lane * kThreads + warp * 32 + holder;
        if (v < to) Row<T>::unpack(__ldg(now.vec() + v), x);
      }
      bool is = false;
#pragma unroll
      for (int i = 0; i < n; ++i) is |= x[i] == m;
      bool skip = lane == __ffs(__ballot_sync(0xffffffffu, is)) - 1;
      float es = 0.f;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float d = by_product(mc) ? fmaf(x[i], a.c2, -mc) : (x[i] - m) * a.c2;
        if (skip && x[i] == m) skip = false;
        else es += ex2(floored(d));
      }
#pragma unroll
      for (int o = kAhead / 2; o; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
      if (lane == 0) sh.alone = sh.all[1] + es;
    }
    if (alone && !a.ntop) __syncthreads();  // (with alternatives there are others before it is read)
    if (a.ntop) {
      const float bound = sh.bound;
      auto in = [&](float x) { return x >= bound && x > kNegInf; };
      if (in(top))
        for (unsigned i = 0; i < runs; ++i)  // (their order does not matter)
          if (in(sh.run[i][tid])) sh.owner[atomicAdd(&sh.owners, 1)] = (unsigned short)(i * kThreads + tid);
      __syncthreads();
      const unsigned all = (unsigned)sh.owners * kAhead << shift;
      // every word of those runs: f(logit, index)
      auto scan = [&](auto f) {
        constexpr int kScan = 2;
#pragma unroll 1
        for (unsigned i0 = tid; i0 < all; i0 += kScan * kThreads) {
          uint4 w[kScan];
          unsigned at[kScan];
#pragma unroll
          for (int i = 0; i < kScan; ++i) {
            const unsigned j = i0 + i * kThreads;
            at[i] = to;
            if (j < all) {
              const unsigned o = sh.owner[j / kAhead >> shift], in_run = j & ((kAhead << shift) - 1);
              at[i] = from + (((o / kThreads) << shift) * kAhead + in_run) * kThreads + o % kThreads;
            }
            if (at[i] < to) w[i] = __ldg(now.vec() + at[i]);
          }
#pragma unroll
          for (int i = 0; i < kScan; ++i) {
            if (at[i] >= to) continue;
            float x[n];
            Row<T>::unpack(w[i], x);
#pragma unroll
            for (int j = 0; j < n; ++j) f(x[j], now.head + at[i] * n + j);
          }
        }
        if (first && (unsigned)tid < now.head) f(to_f(now.base[tid]), (unsigned)tid);
        if (first && (unsigned)tid < now.tail) f(to_f(now.base[now.V - now.tail + tid]), now.V - now.tail + tid);
      };
      scan([&](float x, unsigned v) {
        if (in(x)) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kList) sh.list[at] = word_key(x, v);
        }
      });
      if (tid < a.ntop) sh.top[tid] = 0;
      __syncthreads();
      int count = sh.count;
      if (count <= kList) {
        const unsigned long long* list = sh.list;
        if (count > kLong) {
          // a nearer bound: the ntop-th largest of the maxima of 64 parts of the list
          for (int g = tid; g < kGroups; g += kThreads) {
            unsigned long long best = 0;
            for (int i = g; i < count; i += kGroups) best = sh.list[i] > best ? sh.list[i] : best;
            sh.part[g] = best;
          }
          __syncthreads();
          for (int g = tid; g < kGroups; g += kThreads) {
            const unsigned long long key = sh.part[g];
            int ahead = 0;
#pragma unroll 8
            for (int j = 0; j < kGroups; j += 2) {
              const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.part[j]);
              ahead += (o.x > key) + (o.y > key);
            }
            if (ahead == a.ntop - 1) sh.near = key;  // (the keys are all different)
          }
          __syncthreads();
          const unsigned long long near = sh.near;
          for (int i = tid; i < count; i += kThreads)
            if (sh.list[i] >= near) sh.list2[atomicAdd(&sh.kept, 1)] = sh.list[i];
          __syncthreads();
          count = sh.kept;
          list = sh.list2;
        }
        if (tid == 0 && (count & 1)) const_cast<unsigned long long*>(list)[count] = 0;  // (they are compared in pairs)
        __syncthreads();
        for (int i = tid; i < count; i += kThreads) {
          const unsigned long long key = list[i];
          int ahead = 0;
#pragma unroll 4
          for (int j = 0; j < count; j += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&list[j]);
            ahead += (o.x > key) + (o.y > key);
          }
          if (ahead < a.ntop) sh.top[ahead] = key;
        }
      } else {
        unsigned long long last = ~0ull;
        for (int i = 0; i < a.ntop && last; ++i) {
          unsigned long long best = 0;
          scan([&](float x, unsigned v) {
            if (in(x)) {
              const unsigned long long key = word_key(x, v);
              if (key < last && key > best) best = key;
            }
          });
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
            best = other > best ? other : best;
          }
          if (lane == 0) sh.best[warp] = best;
          __syncthreads();
          best = 0;
          for (int w = 0; w < kWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
          if (tid == 0) sh.top[i] = best;
          last = best;
          __syncthreads();
        }
      }
      __syncthreads();
    }
    Sums c;
    c.m = sh.all[0];
    c.s = alone ? sh.alone : sh.all[1];
    c.t = sh.all[2];
    c.q = alone ? kAlone : sh.all[3];
    if (ncta > 1) {
      cluster.barrier_wait();
      if (tid < 4) *cluster.map_shared_rank(&sh.cta[rank][tid], 0) = tid == 0 ? c.m : tid == 1 ? c.s : tid == 2 ? c.t : c.q;
      if (!first && tid < a.ntop) *cluster.map_shared_rank(&sh.top[rank * a.ntop + tid], 0) = sh.top[tid];
      cluster.sync();
      if (!first) return;
      c = Sums();
      for (unsigned w = 0; w < ncta; ++w) c.join(sh.cta[w][0], sh.cta[w][1], sh.cta[w][2], sh.cta[w][3], a.c2);
    }
    const bool nothing = c.m == kNegInf && c.s == 0.f;  // every word is excluded
    const float off = off_of(c.m, a.c2);
    // ln of such a sum, under m itself
    auto ln_of = [&](float s) {
      return c.q == kAlone ? log1pf(fmaf(s, -off * kLn2, s)) : logf(s + c.q) - off * kLn2;
    };
    // ln sum e^(z - scale m): c2's rounding, to first order
    const float ln_s = ln_of(fmaf(c.t, a.c2_less, c.s));
    if (tid == 0) {
      if (a.stats) a.stats[row] = make_float2(c.m, nothing ? kNegInf : ln_s);
      if (a.lse) a.lse[row] = nothing ? kNegInf : fmaf(c.m, a.scale, ln_s);
      if (a.entropy) {
        const float all = c.s + c.batch(a.c2);
        a.entropy[row] = nothing ? 0.f : ln_of(c.s) - kLn2 * (fmaf(-off, all, c.t) / all);
      }
      if (a.logprobs) a.logprobs[row] = !known ? 0.f : nothing ? kNegInf : below(tok_x, c.m, a.scale) - ln_s;
    }
    const int have = (int)ncta * a.ntop;
    for (int i = tid; i < have; i += kThreads) {
      const unsigned long long key = sh.top[i];
      int at = i;
      if (ncta > 1) {
        at = 0;
        for (int j = 0; j < have; ++j) at += sh.top[j] > key || (sh.top[j] == key && j < i);
      }
      if (at < a.ntop) {
        const long long o = row * a.ntop + at;
        a.top_tok[o] = key ? (int)(0xffffffffu - (unsigned)key) : -1;
        a.top_lp[o] = key ? below(key_logit(key), c.m, a.scale) - ln_s : kNegInf;
      }
    }
    __syncthreads();  // the next row writes over what this one has read
  }
}

// One CTA to a row's run of vectors.  kSame: the gradient's rows lie in their
// vectors as the logits' do.
template <typename T, bool kSame>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_bwd_kernel(LogpArgs a, unsigned per) {
  const long long row = blockIdx.x;
  constexpr int n = Row<T>::n;
  const Row<T> r(a.logits, row, a.stride, a.V);
  T* out = static_cast<T*>(a.dlogits) + row * a.gstride;
  const float2 st = a.stats_in[row];  // the largest logit m, and ln sum e^(z - scale m)
  const float m = st.x, ln_s = st.y, H = a.ent_in ? a.ent_in[row] : 0.f;
  const int t = a.tokens ? a.tokens[row] : -1;
  const unsigned tok = t >= 0 && t < a.V ? (unsigned)t : 0xffffffffu;
  const float dl = tok != 0xffffffffu && a.dlogp ? a.dlogp[row] : 0.f, dH = a.dent ? a.dent[row] : 0.f;
  // every word is excluded, or nothing comes in (padding): zeros, whatever the row holds
  const bool nothing = ln_s == kNegInf || (tok == 0xffffffffu && dH == 0.f);
  // p (-dl - dH (log p + H)) with log p = scale (x - m) - ln_s: the difference keeps
  // its digits where the logits are large
  auto grad = [&](float x) {
    const float lp = floored(fmaf(x - m, a.scale, -ln_s)), p = ex2(lp * kLog2e);
    const float g = -p * fmaf(dH, lp + H, dl);
    return nothing ? 0.f : g * a.scale;
  };
  // the token's, with 1 - p whole however near p is to 1
  auto chosen = [&](float x) {
    const float lp = floored(fmaf(x - m, a.scale, -ln_s)), p = ex2(lp * kLog2e);
    const float g = -p * dH * (lp + H) - dl * expm1f(lp);
    return nothing ? 0.f : g * a.scale;
  };
  auto one = [&](unsigned v) { out[v] = from_f<T>(v == tok ? chosen(to_f(r.base[v])) : grad(to_f(r.base[v]))); };
  if (blockIdx.y == 0) {
    if (threadIdx.x < r.head) one(threadIdx.x);
    if (threadIdx.x < r.tail) one(r.V - r.tail + threadIdx.x);
  }
  for (unsigned b = blockIdx.y * per; b < r.nvec; b += gridDim.y * per) {
    const unsigned hi = min(b + per, r.nvec);
    for (unsigned v0 = b + threadIdx.x; v0 < hi; v0 += kAhead * kBwdThreads) {
      uint4 u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (v0 + i * kBwdThreads < hi) u[i] = r.vec()[v0 + i * kBwdThreads];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const unsigned v = v0 + i * kBwdThreads;
        if (v >= hi) break;
        float x[n];
        Row<T>::unpack(u[i], x);
        const unsigned w = r.head + v * n;
#pragma unroll
        for (int j = 0; j < n; ++j) x[j] = grad(x[j]);
        if (tok - w < n) {
          float y[n], c = 0.f;
          Row<T>::unpack(u[i], y);
#pragma unroll
          for (int j = 0; j < n; ++j)
            if (w + j == tok) c = y[j];
          c = chosen(c);
#pragma unroll
          for (int j = 0; j < n; ++j)
            if (w + j == tok) x[j] = c;
        }
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

template <typename T, int kThreads>
cudaError_t launch_fwd_t(const LogpArgs& a, int ncta, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const long long most = (long long)device_sm_count() * resident(kThreads);
  cfg.gridDim = dim3((unsigned)(ncta > 1 ? a.rows * ncta : a.rows < most ? a.rows : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ncta;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ncta > 1 ? 1 : 0;
  set_kernel_name("token_logprobs");
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, kThreads>, a);
}
template <typename T>
cudaError_t launch_fwd(const LogpArgs& a, cudaStream_t s) {
  // CTAs to a row: more, in powers of two up to the portable cluster size, while each has an SM of its own and more than
  // 2048 words; they are wide, for the shortest way through the row.
  const int sms = device_sm_count();
  int ncta = 1;
  while (ncta < kMaxCluster && (long long)ncta * 2048 < a.V && a.rows * ncta * 2 <= sms) ncta *= 2;
  if (ncta > 1) return launch_fwd_t<T, 512>(a, ncta, s);
  // Else narrow ones, whose joins leave the SM to others (4096 rows of 32,000 bf16 words: 51 us with 128 threads, 62 with
  // 256, 56 with 64), the narrowest for rows of up to 8 vectors to each of their threads (rows of 300 with 20
  // alternatives: 25 us with 64 threads, 40 with 128).
  // Between 77 and some 900 rows they leave an SM little in flight: rows of 128,000 fp32 words take 12 us at 76 rows
  // (two CTAs to a row), 45 at 77, 50 at 256 and 76 at 912, where HBM takes 69.
  if (a.V * (long long)sizeof(T) <= 64 * 8 * 16) return launch_fwd_t<T, 64>(a, 1, s);
  return launch_fwd_t<T, 128>(a, 1, s);
}

template <typename T>
cudaError_t launch_bwd(const LogpArgs& a, cudaStream_t s) {
  // runs of 4 tiles where there are rows enough, else of one
  const long long vecs = (a.V * (long long)sizeof(T) + 15) / 16;
  const unsigned per = 4 * kBwdThreads * (a.rows >= 4 * device_sm_count() ? 4 : 1);
  long long runs = (vecs + per - 1) / per;
  if (runs < 1) runs = 1;
  if (runs > 65535) runs = 65535;
  const bool same = ((reinterpret_cast<uintptr_t>(a.dlogits) - reinterpret_cast<uintptr_t>(a.logits)) & 15u) == 0 &&
                    ((a.stride - a.gstride) * (long long)sizeof(T)) % 16 == 0;
  const dim3 grid((unsigned)a.rows, (unsigned)runs);
  set_kernel_name("token_logprobs_bwd");
  if (same) token_logprobs_bwd_kernel<T, true><<<grid, kBwdThreads, 0, s>>>(a, per);
  else token_logprobs_bwd_kernel<T, false><<<grid, kBwdThreads, 0, s>>>(a, per);
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
  // exponents' factors are finite; a difference of logits that is not has the exponential 0
  if (!(pr->scale * kLog2e <= 3.402823466e38f) || pr->scale < kLeastScale) return SSD_ERR_UNSUPPORTED;
  *a = LogpArgs();
  a->rows = pr->rows;
  a->V = pr->vocab;
  a->stride = ls;
  a->gstride = gs;
  a->scale = pr->scale;
  a->c2 = pr->scale * kLog2e;
  const double less = (double)pr->scale * 1.4426950408889634 / (double)a->c2 - 1.0;
  a->c2_less = less > -1e-6 && less < 1e-6 ? (float)(less * 0.6931471805599453) : 0.f;
  a->ntop = pr->ntop;
  return SSD_OK;
}
bool misaligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15u); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_token_logprobs(const ssd_logprob_problem* pr, const void* logits, const int32_t* tokens, float* logprobs,
                       float* entropy, float* lse, float* stats, int32_t* top_tokens, float* top_logprobs,
                       ssd_stream_t stream) {
  LogpArgs a;
  int rc = check(pr, &a);
  if (rc != SSD_OK) return rc;
  if (!logits || (logprobs != nullptr) != (tokens != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  if ((pr->ntop > 0) != (top_tokens != nullptr) || (pr->ntop > 0) != (top_logprobs != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!logprobs && !entropy && !lse && !stats && !top_tokens) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {logits, tokens, logprobs, entropy, lse, stats, top_tokens, top_logprobs};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  a.logits = logits; a.tokens = tokens; a.logprobs = logprobs; a.entropy = entropy; a.lse = lse;
  a.stats = reinterpret_cast<float2*>(stats);
  a.top_tok = top_tokens; a.top_lp = top_logprobs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = pr->dtype == SSD_BF16 ? launch_fwd<__nv_bfloat16>(a, s) : launch_fwd<float>(a, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_token_logprobs_bwd(const ssd_logprob_problem* pr, const void* logits, const int32_t* tokens,
                           const float* stats, const float* entropy, const float* dlogprobs, const float* dentropy, void* dlogits,
                           ssd_stream_t stream) {
  LogpArgs a;
  int rc = check(pr, &a);
  if (rc != SSD_OK) return rc;
  if (!logits || !stats || !dlogits || (!dlogprobs && !dentropy)) return SSD_ERR_INVALID_ARGUMENT;
  if ((dlogprobs != nullptr) != (tokens != nullptr) || (dentropy != nullptr) != (entropy != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (dlogits == logits && a.stride != a.gstride) return SSD_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {logits, tokens, stats, entropy, dlogprobs, dentropy, dlogits};
  for (const void* q : ptrs)
    if (misaligned16(q)) return SSD_ERR_INVALID_ARGUMENT;
  rc = device_check();
  if (rc != SSD_OK) return rc;
  a.logits = logits; a.tokens = tokens; a.stats_in = reinterpret_cast<const float2*>(stats); a.ent_in = entropy; a.dlogp = dlogprobs; a.dent = dentropy;
  a.dlogits = dlogits;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_before(s);
  const cudaError_t e = pr->dtype == SSD_BF16 ? launch_bwd<__nv_bfloat16>(a, s) : launch_bwd<float>(a, s);
  prof_after(s);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
