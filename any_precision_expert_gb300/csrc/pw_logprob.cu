// Log probabilities of given tokens, entropies and the best alternatives of
// rows of logits x, in one pass:
//   m = max x,  l = sum e^(x - m),  t = sum e^(x - m) (x - m),
//   ln p_i = (x_i - m) - ln l,  H = ln l - t / l.
// Partial (m, l, t) join like the sums of a softmax; H's two terms have the
// same sign, so nothing cancels.
//
// Bound: every logit is read once, HBM for long prompts, the chain of loads,
// maxima and joins for a few rows.  A thread holds kVecs 16-byte vectors of a
// round in registers, so that all its loads are in flight together and the
// alternatives are picked without a second read; a cluster of CTAs shares a row.
//
// Alternatives: a round's threads fall into 32 sets (by lane); the n-th largest
// of the sets' maxima is a bound that n logits reach, and hardly more than n
// do.  Those go to a list, whose best n by (value, lowest index) are found by
// counting.  Where too many reach the bound (rows of equal logits), the n are
// searched one after another instead.
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
constexpr int kThreads = 256;
constexpr int kList = 1024;    // alternatives a CTA lists
constexpr float kLog2e = 1.4426950408889634f;

// A vector's values as fp32.
template <typename E>
struct Vec {
  static constexpr int N = 8;
  static __device__ __forceinline__ void up(const uint4& r, float (&x)[N]) { unpack8<E>(r, x); }
  static __device__ __forceinline__ float one(const E* p) { return (float)*p; }
  static __device__ __forceinline__ uint32_t none() { return sizeof(E) == 2 && __is_same(E, __half) ? 0xfc00fc00u : 0xff80ff80u; }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void up(const uint4& r, float (&x)[N]) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ uint32_t none() { return 0xff800000u; }
};

struct Sums {
  float m, l, t;
  __device__ __forceinline__ void join(float om, float ol, float ot) {
    const float mm = fmaxf(m, om);
    if (mm == -CUDART_INF_F) {  // nothing on either side, or no numbers
      l += ol, t += ot;
      return;
    }
    const float da = fmaxf(m - mm, -1e30f), db = fmaxf(om - mm, -1e30f);  // of an empty side: a weight of 0
    const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
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
__global__ void __launch_bounds__(kThreads, 3) logprob_kernel(const LogprobParams P) {
  using V = Vec<E>;
  constexpr int N = V::N, WARPS = kThreads / 32;
  __shared__ Handed handed;
  __shared__ Alt list[kList];
  __shared__ Sums warp_sums[WARPS];
  __shared__ float set_max[WARPS][32];
  __shared__ Alt best[kMaxTop];
  __shared__ Alt warp_best[WARPS];
  __shared__ int s_count;
  __shared__ float s_bar;
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
  if (tid == 0) s_count = 0, s_bar = -CUDART_INF_F;
  Sums sums = {-CUDART_INF_F, 0.f, 0.f};
  const uint4* body = reinterpret_cast<const uint4*>(x + head);
  bool first = true;
#pragma unroll 1
  for (int v0 = lo; v0 < hi || first; v0 += kVecs * kThreads) {
    uint4 raw[kVecs];
    int most = 0;  // vectors of this thread
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int v = v0 + u * kThreads + tid;
      raw[u] = make_uint4(V::none(), V::none(), V::none(), V::none());
      if (v < hi) raw[u] = __ldcs(body + v), most = u + 1;
    }
    float top = first ? fmaxf(odd, -CUDART_INF_F) : -CUDART_INF_F;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float f[N];
      V::up(raw[u], f);
#pragma unroll
      for (int k = 0; k < N; ++k) top = fmaxf(top, f[k]);
    }
    if (n > 0) {
      set_max[warp][lane] = top;
      __syncthreads();
      if (warp == 0) {
        float mine = set_max[0][lane];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) mine = fmaxf(mine, set_max[w][lane]);
        int rank = 0;
#pragma unroll
        for (int o = 0; o < 32; ++o) {
          const float other = __shfl_sync(0xffffffffu, mine, o);
          rank += other > mine || (other == mine && o < lane);
        }
        if (rank == n - 1) s_bar = fmaxf(s_bar, mine);
      }
      __syncthreads();
      const float bar = s_bar;
      if (top >= bar && top > -CUDART_INF_F) {
        auto put = [&](float v, int i) {
          if (v >= bar && v > -CUDART_INF_F) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kList) list[at] = {v, i};
          }
        };
        if (first && odd_at >= 0) put(odd, odd_at);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          float f[N];
          V::up(raw[u], f);
#pragma unroll
          for (int k = 0; k < N; ++k) put(f[k], head + (v0 + u * kThreads + tid) * N + k);
        }
      }
    }
    // this round's sums, about the larger of its own and the earlier maximum
    const float mm = fmaxf(sums.m, top), ref = mm == -CUDART_INF_F ? 0.f : mm;
    if (sums.m != -CUDART_INF_F && mm > sums.m) {
      const float d = fmaxf(sums.m - mm, -1e30f), f = ex2(d * kLog2e);
      sums.t = f * fmaf(d, sums.l, sums.t);
      sums.l *= f;
    }
    sums.m = mm;
    auto add = [&](float v) {
      const float d = v - ref, e = ex2(d * kLog2e);
      sums.l += e;
      sums.t = fmaf(e, fmaxf(d, -1e30f), sums.t);  // 0 for a logit of -infinity
    };
    if (first && odd_at >= 0) add(odd);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      if (u < most) {
        float f[N];
        V::up(raw[u], f);
#pragma unroll
        for (int k = 0; k < N; ++k) add(f[k]);
      }
    }
    first = false;
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
    if (P.entropy) P.entropy[row] = none ? 0.f : log_l - all.t / all.l;
  }
  if (tid < parts * n) {
    const Alt mine = handed.best[tid / n][tid % n];
    int rank = 0;
    for (int j = 0; j < parts * n; ++j) {
      const Alt o = handed.best[j / n][j % n];
      rank += o.before(mine) || (o.v == mine.v && o.i == mine.i && j < tid);  // places without a token count in order
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
  constexpr int kRound = kVecs * kThreads * Vec<E>::N;
  // CTAs a row: as many as hold it in one round, more while the rows alone leave SMs idle and every thread has a vector
  int parts = 1;
  while (parts < kMaxCluster && ((long long)parts * kRound < P.V ||
                                 ((long long)P.T * parts < 2 * sm_count() && P.V > parts * kThreads * Vec<E>::N)))
    parts *= 2;
  const Launch at(dim3(P.T * parts), kThreads, 0, s, parts);
  return cudaLaunchKernelEx(&at.cfg, logprob_kernel<E>, P);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& P, int dtype, cudaStream_t s) {
  return dtype == PW_F32 ? launch_typed<float>(P, s) : dtype == PW_F16 ? launch_typed<__half>(P, s) : launch_typed<__nv_bfloat16>(P, s);
}

}  // namespace pw
