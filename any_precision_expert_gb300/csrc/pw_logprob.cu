// Log probabilities of given tokens, entropies and the best alternatives of
// rows of logits x, in one pass.  With a_i = (x_i - m) log2 e about a maximum m,
//   l = sum 2^a,  t = sum 2^a a,
//   ln p_i = (x_i - m) - ln l,  H = ln l - ln 2 t / l.
// Partial (m, l, t) join like the sums of a softmax; H's two terms have the
// same sign, so nothing cancels.
//
// Bound: every logit is read once, HBM for long prompts, the chain of loads,
// maxima and joins for a few rows.  Measured: 2047 rows of 131072 bf16 logits
// with 8 alternatives, 537 MB, in 106 us (5.0 TB/s; a tenth less without
// alternatives), where it issues 69 million instructions, 55 us of issue slots;
// 8 rows of 32000 in 7.2 us.  A thread holds kVecs 16-byte vectors of a round in
// registers, so that their loads are in flight together (with 2 / 4 / 6 in the
// place of 8 it took 30 / 3 / 5 % longer); a cluster of CTAs shares a row only
// where rows are few.
//
// Alternatives: a thread notes its vectors' maxima.  After kEpoch rounds the n-th
// largest of 32 sets' maxima so far (the threads of a lane number) is a bound
// that n logits reach, and hardly more than n do: the few vectors that reach it
// are read again, from the L2, and their logits that do go to a list, whose
// best n by (value, lowest index) are found by counting.  Where more than kList
// have reached it, the n are searched one after another instead, each with a
// read of the row: rows of equal or rising logits, and with 32 alternatives, of
// which about 130 places go in the first look and 130 / k in the k-th, ordinary
// ones of large vocabularies (of normal fp32 logits by one CTA a row 1 % of the
// rows at 131072, 10 to 15 % at 262144, nine in ten at a million; none of them
// with 20 alternatives).
#include <cooperative_groups.h>
#include <math_constants.h>

#include <utility>

#include "pw_heads.cuh"
#include "pw_mma.cuh"
#include "pw_serve.h"

namespace pw {

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kVecs = 8;       // 16-byte vectors a thread and round
constexpr int kThreads = 128;
constexpr int kCtas = 6;       // an SM
constexpr int kEpoch = 4;      // rounds between two looks for alternatives: 32 vectors a thread, one a lane that looks at them
constexpr int kList = 512;    // alternatives a CTA lists
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays one
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A vector's values as fp32, and the larger of two vectors, value by value (what is no number gives way).
template <typename E>
struct Vec {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = __is_same(E, __half) ? 0xfc00fc00u : 0xff80ff80u;
  static __device__ __forceinline__ void up(const uint4& r, float (&x)[N]) { unpack8<E>(r, x); }
  static __device__ __forceinline__ float one(const E* p) { return (float)*p; }
  // Values from a low number up, so that a weight of 0 meets no infinity; what is no number stays that.  About a maximum
  // of at most kSafe that number weighs 0.
  static constexpr float kSafe = __is_same(E, __half) ? 6e4f : 1e6f;
  static __device__ __forceinline__ uint4 finite_below(const uint4& r) {
    constexpr uint32_t kLow = __is_same(E, __half) ? 0xfbfffbffu : 0xfe96fe96u;  // -65504, -1e38
    const uint32_t low = kLow;
    auto f = [&](uint32_t a) {
      using V = typename Pair<E>::V;
      const V m = __hmax2_nan(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&low));
      return *reinterpret_cast<const uint32_t*>(&m);
    };
    return make_uint4(f(r.x), f(r.y), f(r.z), f(r.w));
  }
  static __device__ __forceinline__ uint32_t more(uint32_t a, uint32_t b) {
    using V = typename Pair<E>::V;
    const V m = __hmax2(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float top(uint32_t a) {
    const float2 f = Pair<E>::up(*reinterpret_cast<const typename Pair<E>::V*>(&a));
    return fmaxf(fmaxf(f.x, f.y), -CUDART_INF_F);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void up(const uint4& r, float (&x)[N]) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static constexpr float kSafe = 1e6f;
  static __device__ __forceinline__ uint4 finite_below(const uint4& r) {
    auto f = [](uint32_t a) { return __float_as_uint(max_nan(__uint_as_float(a), -1e38f)); };
    return make_uint4(f(r.x), f(r.y), f(r.z), f(r.w));
  }
  static __device__ __forceinline__ uint32_t more(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float top(uint32_t a) { return fmaxf(__uint_as_float(a), -CUDART_INF_F); }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

struct Sums {
  float m, l, t;
  __device__ __forceinline__ void join(float om, float ol, float ot) {
    const float mm = fmaxf(m, om);
    if (mm == -CUDART_INF_F) {  // nothing on either side, or no numbers
      l += ol, t += ot;
      return;
    }
    const float da = max_nan((m - mm) * kLog2e, -1e30f), db = max_nan((om - mm) * kLog2e, -1e30f);  // an empty side weighs 0
    const float fa = ex2(da), fb = ex2(db);
    t = fa * fmaf(da, l, t) + fb * fmaf(db, ol, ot);
    l = fa * l + fb * ol;
    m = mm;
  }
  __device__ __forceinline__ void warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o), __shfl_xor_sync(0xffffffffu, t, o));
  }
};

struct Alt {
  float v;
  int i;
  __device__ __forceinline__ bool before(const Alt& o) const { return v > o.v || (v == o.v && i < o.i); }
};
constexpr int kNoToken = 0x7fffffff;

// What the CTAs of a cluster hand to the first of them.
struct Handed {
  Sums sums[kMaxCluster];
  Alt best[kMaxCluster][kMaxTop];
};

template <typename E>
__global__ void __launch_bounds__(kThreads, kCtas) logprob_kernel(const LogprobParams P) {
  using V = Vec<E>;
  constexpr int N = V::N, WARPS = kThreads / 32;
  __shared__ Handed handed;
  __shared__ Alt list[kList];
  __shared__ uint32_t vec_max[kEpoch * kVecs][kThreads + 1];
  __shared__ Sums warp_sums[WARPS];
  __shared__ float set_max[2][WARPS][32];
  __shared__ Alt best[kMaxTop];
  __shared__ Alt warp_best[WARPS];
  __shared__ int s_count;
  behind_the_stream();
  let_next_start();
  const cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // every CTA runs before another one writes to its shared memory
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int row = blockIdx.x / parts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = P.n_top;
  const E* x = static_cast<const E*>(P.logits) + (long long)row * P.row_stride;
  // whole vectors between the values in front of the first 16-byte boundary and those behind the last
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(E), P.V);
  const int vecs = (P.V - head) / N, tail = P.V - head - vecs * N;
  const int share = (vecs + parts - 1) / parts, lo = min(part * share, vecs), hi = min(lo + share, vecs);
  // the odd ones: one a thread, the first CTA's in front, the last one's behind
  int odd_at = -1;
  if (part == 0 && tid < head) odd_at = tid;
  if (part == parts - 1 && tid >= 32 && tid - 32 < tail) odd_at = head + vecs * N + tid - 32;
  const float odd = odd_at >= 0 ? V::one(x + odd_at) : -CUDART_INF_F;
  if (tid == 0) s_count = 0;
  Sums sums;
  const uint4* body = reinterpret_cast<const uint4*>(x + head);
  constexpr int STEP = kVecs * kThreads;
  uint4 raw[kVecs];
  const uint4* mine = body + lo + tid;
  auto load = [&](int v0) {
    if (v0 + STEP <= hi) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) raw[u] = __ldcs(mine + v0 - lo + u * kThreads);
    } else {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        raw[u] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
        if (v0 + u * kThreads + tid < hi) raw[u] = __ldcs(mine + v0 - lo + u * kThreads);
      }
    }
  };
  load(lo);
  float seen = odd, epoch_top = -CUDART_INF_F;  // the largest so far, and since the last look
  uint64_t l2 = 0, t2 = 0;
  // a = (x - m) log2 e in one operation: x log2 e - rn(m log2 e), off by the rounding of the latter in all of a thread's
  // terms alike, which the sums make good when m changes and at the end.  Not for an m beyond kSafe.
  auto large = [](float m) { return !(fabsf(m) <= V::kSafe); };
  auto rounded = [&](float m) {  // the power of two that makes it good
    return large(m) ? 0.f : -fmaf(m, kLog2e, -(m * kLog2e));
  };
#pragma unroll 1
  for (int v0 = lo, round = 0; v0 < hi || round == 0; v0 += STEP, ++round) {
    uint32_t w = V::kNone;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t y = V::more(V::more(raw[u].x, raw[u].y), V::more(raw[u].z, raw[u].w));
      if (n > 0) vec_max[(round % kEpoch) * kVecs + u][tid] = y;
      w = V::more(w, y);
    }
    const float was = seen, top = V::top(w);
    seen = fmaxf(seen, top);
    epoch_top = fmaxf(round % kEpoch == 0 ? -CUDART_INF_F : epoch_top, top);
    // this round's sums, about the largest so far
    const float ref = seen == -CUDART_INF_F ? 0.f : seen;
    if (round > 0 && was != -CUDART_INF_F && seen > was) {
      const float d = max_nan((was - seen) * kLog2e, -1e30f) + rounded(was) - rounded(seen), f = ex2(d);
      t2 = mul2(pack(f, f), fma2(pack(d, d), l2, t2));
      l2 = mul2(pack(f, f), l2);
    }
    if (!large(ref)) {
      const float off = -(ref * kLog2e);
      const uint64_t off2 = pack(off, off), unit = pack(kLog2e, kLog2e);
      auto add = [&](float x, float y) {
        const uint64_t a = fma2(pack(x, y), unit, off2);
        const float2 f = unpack(a);
        const uint64_t e = pack(ex2(f.x), ex2(f.y));
        l2 = add2(l2, e);
        t2 = fma2(e, a, t2);
      };
      if (round == 0 && odd_at >= 0) add(max_nan(odd, -1e38f), -1e38f);  // and one of no weight
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        float f[N];
        V::up(V::finite_below(raw[u]), f);
#pragma unroll
        for (int k = 0; k < N; k += 2) add(f[k], f[k + 1]);
      }
    } else {
      auto add = [&](float x) {
        const float a = max_nan((x - ref) * kLog2e, -1e30f), e = ex2(a);
        l2 = add2(l2, pack(e, 0.f));
        t2 = fma2(pack(e, 0.f), pack(a, 0.f), t2);
      };
      if (round == 0 && odd_at >= 0) add(odd);
#pragma unroll 1
      for (int v = v0 + tid; v < min(v0 + STEP, hi); v += kThreads) {
        float f[N];
        V::up(body[v], f);
#pragma unroll
        for (int k = 0; k < N; ++k) add(f[k]);
      }
    }
    if (v0 + STEP < hi) load(v0 + STEP);
    if (n > 0 && (round % kEpoch == kEpoch - 1 || v0 + kVecs * kThreads >= hi)) {
      // every warp finds the bound for itself; a set's places are written again two looks later
      float (&sets)[WARPS][32] = set_max[round / kEpoch & 1];
      sets[warp][lane] = seen;
      __syncthreads();
      float top_set = sets[0][lane];
#pragma unroll
      for (int k = 1; k < WARPS; ++k) top_set = fmaxf(top_set, sets[k][lane]);
      int rank = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const float other = __shfl_sync(0xffffffffu, top_set, o);
        rank += other > top_set || (other == top_set && o < lane);
      }
      const float bar = __shfl_sync(0xffffffffu, top_set, __ffs(__ballot_sync(0xffffffffu, rank == n - 1)) - 1);
      auto put = [&](float v, int i) {
        if (v >= bar && v > -CUDART_INF_F) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kList) list[at] = {v, i};
        }
      };
      if (round < kEpoch && odd_at >= 0) put(odd, odd_at);
      // the threads with a vector that reaches it, one after another: a lane a vector, then a lane a logit
      unsigned threads = __ballot_sync(0xffffffffu, epoch_top >= bar && epoch_top > -CUDART_INF_F);
#pragma unroll 1
      for (; threads; threads &= threads - 1) {
        const int who = warp * 32 + __ffs(threads) - 1;
        const bool noted = lane / kVecs <= round % kEpoch;
        const float most = noted ? V::top(vec_max[lane][who]) : -CUDART_INF_F;
        unsigned vectors = __ballot_sync(0xffffffffu, most >= bar && most > -CUDART_INF_F);
#pragma unroll 1
        for (; vectors; vectors &= vectors - 1) {
          const int v = lo + ((round - round % kEpoch) * kVecs + __ffs(vectors) - 1) * kThreads + who;
          if (lane < N) put(V::one(x + head + (long long)v * N + lane), head + v * N + lane);
        }
      }
    }
  }
  {
    const float2 l = unpack(l2), t = unpack(t2);
    const float c = seen == -CUDART_INF_F ? 0.f : rounded(seen), f = ex2(c);
    sums = {seen, f * (l.x + l.y), f * fmaf(c, l.x + l.y, t.x + t.y)};
  }
  sums.warp();
  if (lane == 0) warp_sums[warp] = sums;
  __syncthreads();
  if (n > 0) {  // this CTA's n best
    if (tid < n) best[tid] = {-CUDART_INF_F, kNoToken};
    __syncthreads();
    const int count = s_count;
    if (count <= kList) {
      for (int i = tid; i < count; i += kThreads) {
        const Alt mine = list[i];
        int rank = 0;
        for (int j = 0; j < count && rank < n; ++j) rank += list[j].before(mine);
        if (rank < n) best[rank] = mine;
      }
    } else {
      Alt last = {CUDART_INF_F, -1};  // before everything
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        Alt a = {-CUDART_INF_F, kNoToken};
        auto look = [&](float v, int i) {
          const Alt c = {v, i};
          if (v > -CUDART_INF_F && last.before(c) && c.before(a)) a = c;
        };
        if (odd_at >= 0) look(odd, odd_at);
        for (int v = lo + tid; v < hi; v += kThreads) {
          float f[N];
          V::up(body[v], f);
#pragma unroll
          for (int j = 0; j < N; ++j) look(f[j], head + v * N + j);
        }
        auto reduce = [&]() {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const Alt c = {__shfl_xor_sync(0xffffffffu, a.v, o), __shfl_xor_sync(0xffffffffu, a.i, o)};
            if (c.before(a)) a = c;
          }
        };
        reduce();
        if (lane == 0) warp_best[warp] = a;
        __syncthreads();
        a = lane < WARPS ? warp_best[lane] : Alt{-CUDART_INF_F, kNoToken};
        reduce();
        if (tid == 0) best[k] = a;
        last = a;
        __syncthreads();
        if (a.i == kNoToken) break;
      }
    }
    __syncthreads();
  }
  cluster.barrier_wait(std::move(started));
  if (warp == 0) {
    sums = lane < WARPS ? warp_sums[lane] : Sums{-CUDART_INF_F, 0.f, 0.f};
    sums.warp();
    Handed* to = cluster.map_shared_rank(&handed, 0);
    if (lane == 0) to->sums[part] = sums;
    if (lane < n) to->best[part][lane] = best[lane];
  }
  cluster.sync();
  if (part != 0) return;
  Sums all = handed.sums[0];
  for (int i = 1; i < parts; ++i) all.join(handed.sums[i].m, handed.sums[i].l, handed.sums[i].t);
  // a row of nothing but -infinity has no distribution: every log probability is -infinity, the entropy 0
  const bool none = all.l == 0.f;
  const float log_l = none ? 0.f : logf(all.l);
  auto log_p = [&](float v) { return none || (v == -CUDART_INF_F && all.l == all.l) ? -CUDART_INF_F : (v - all.m) - log_l; };
  if (tid == 0) {
    const int tok = P.tokens[row];
    float lp = 0.f;  // a negative token: none
    if (tok >= P.V) {
      lp = CUDART_NAN_F;
      if (P.err) atomicExch(P.err, kErrToken);
    } else if (tok >= 0) {
      lp = log_p(V::one(x + tok));
    }
    P.logprob[row] = lp;
    if (P.entropy) P.entropy[row] = none ? 0.f : log_l - all.t / all.l * kLn2;
  }
  for (int i = tid; i < parts * n; i += kThreads) {
    const Alt mine = handed.best[i / n][i % n];
    int rank = 0;
    for (int j = 0; j < parts * n; ++j) {
      const Alt o = handed.best[j / n][j % n];
      rank += o.before(mine) || (o.v == mine.v && o.i == mine.i && j < i);  // places without a token count in order
    }
    if (rank < n) {
      const bool some = mine.i != kNoToken;
      P.top_ids[(long long)row * n + rank] = some ? mine.i : -1;
      P.top_logprobs[(long long)row * n + rank] = some ? log_p(mine.v) : -CUDART_INF_F;
    }
  }
}

template <typename E>
cudaError_t launch_typed(const LogprobParams& P, cudaStream_t s) {
  // CTAs a row: more than one only while the rows leave places for CTAs idle and every thread keeps a vector.  A CTA's
  // fixed times weigh more than uneven ends: 2047 rows of 131072 took 8 / 24 / 76 % longer with 2 / 4 / 8 than with 1.
  int parts = 1;
  while (parts < kMaxCluster && (long long)P.T * parts < kCtas * sm_count() && P.V > parts * kThreads * Vec<E>::N) parts *= 2;
  const Launch at(dim3(P.T * parts), kThreads, 0, s, parts);
  return cudaLaunchKernelEx(&at.cfg, logprob_kernel<E>, P);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& P, int dtype, cudaStream_t s) {
  return dtype == PW_F32 ? launch_typed<float>(P, s) : dtype == PW_F16 ? launch_typed<__half>(P, s) : launch_typed<__nv_bfloat16>(P, s);
}

}  // namespace pw
