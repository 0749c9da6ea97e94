// Verification of drafted tokens: acceptance, then a draw from the residual
// distribution as the largest quotient r / e over the vocabulary.
//
// Bound: one row each of the target's probabilities, the noise and, where a
// draft was refused, the draft's probabilities, read once: HBM for a large
// batch, the chain draft count -> token -> its probabilities -> row for a
// small one.  A cluster of CTAs shares a sequence's vocabulary and joins its
// maxima through shared memory: one launch, no workspace, and the largest
// (quotient, lowest index) does not depend on any order.  Measured: 256
// sequences over 131072 tokens, half of them refused a draft, 336 MB in 52 us
// (6.4 TB/s; 108 us when every index was divided); 4 over 32000 4.7 us.
#include <cooperative_groups.h>

#include "pw_serve.h"

namespace pw {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;

// The largest quotient so far and its index; the lower index wins among equal ones.
struct Best {
  float v;
  int i;
  __device__ __forceinline__ void take(float ov, int oi) {
    if (ov > v || (ov == v && oi < i)) v = ov, i = oi;
  }
  __device__ __forceinline__ void warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) take(__shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, i, o));
  }
};

// A quotient costs some twenty instructions and almost none is the largest, so an index is first held against the
// CTA's best so far, t: fl(r / e) >= t needs r >= t e (1 - 2^-24), and bar = t (1 - 2^-20) leaves room for the rounding
// of both products.  Below 1e-30 (where they could round to subnormals) everything is a candidate; an infinite t is
// taken as the largest number, so that other infinite quotients still are.
__device__ __forceinline__ float bar_of(float t) {
  return t > 1e-30f ? fminf(t, 3.402823466e38f) * (1.f - 9.5367431640625e-7f) : 0.f;
}

__device__ __forceinline__ void weigh(Best& best, int* cta_best, float r, float e, int i) {
  if (!(r > 0.f)) return;  // 0, or not a number
  const float v = r / e;
  if (v > best.v) {        // NaN does not; equal ones keep the lower index
    best.v = v, best.i = i;
    atomicMax(cta_best, __float_as_int(v));  // numbers above 0 order like their bits
  }
}

template <bool VEC>
__device__ __forceinline__ void scan(Best& best, float& most, int* cta_best, const float* p, const float* q,
                                     const float* e, int lo, int hi) {
  constexpr int N = VEC ? 4 : 1, UN = VEC ? 1 : 4;  // values a load, loads of an array in flight
  for (int i0 = lo + N * threadIdx.x; i0 < hi; i0 += N * UN * kVerifyThreads) {
    float r[UN][N], c[UN][N];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int i = i0 + N * u * kVerifyThreads;
#pragma unroll
      for (int k = 0; k < N; ++k) r[u][k] = 0.f, c[u][k] = 1.f;
      if (i >= hi) continue;
      if constexpr (VEC) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p + i)), d = __ldcs(reinterpret_cast<const float4*>(e + i));
        r[u][0] = a.x, r[u][1] = a.y, r[u][2] = a.z, r[u][3] = a.w;
        c[u][0] = d.x, c[u][1] = d.y, c[u][2] = d.z, c[u][3] = d.w;
        if (q) {
          const float4 b = __ldcs(reinterpret_cast<const float4*>(q + i));
          r[u][0] -= b.x, r[u][1] -= b.y, r[u][2] -= b.z, r[u][3] -= b.w;
        }
      } else {
        r[u][0] = __ldcs(p + i);
        c[u][0] = __ldcs(e + i);
        if (q) r[u][0] -= __ldcs(q + i);
      }
    }
    const float bar = bar_of(__int_as_float(*reinterpret_cast<volatile int*>(cta_best)));
    bool some = false;
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        most = fmaxf(most, r[u][k]);
        some |= r[u][k] >= bar * c[u][k];
      }
    if (some) {
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (r[u][k] >= bar * c[u][k]) weigh(best, cta_best, r[u][k], c[u][k], i0 + N * u * kVerifyThreads + k);
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2048 / kVerifyThreads) verify_kernel(const VerifyParams P) {
  __shared__ Best warp_best[kVerifyWarps];
  __shared__ Best all_best[2][kMaxCluster];   // [pass][CTA of the cluster], written by all of them
  __shared__ int all_any[2][kMaxCluster];
  __shared__ int s_any, s_best, s_kept, s_n;
  behind_the_stream();
  let_next_start();
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int b = blockIdx.x / parts, tid = threadIdx.x, lane = tid & 31, K = P.K, V = P.V;
  if (tid == 0) s_any = s_best = 0;
  if (tid < 32) {
    int n = 0, kept = 0;
    if (K > 0) {
      const int given = P.n_draft[b];
      n = min(max(given, 0), K);
      if (given != n && lane == 0 && P.err) atomicExch(P.err, kErrToken);
      kept = n;
      for (int i0 = 0; i0 < K; i0 += 32) {  // the drafts side by side; the first refusal ends the kept ones
        const int i = i0 + lane;
        bool ok = true, bad = false;
        if (i < K) {  // read whether or not it counts: the count is on its way too
          const int x = P.tokens[(size_t)b * K + i];
          bad = x < 0 || x >= V;
          ok = !bad;
          if (ok) {
            const float uq = P.u[(size_t)b * K + i] * P.q[((size_t)b * K + i) * V + x];
            ok = uq < P.p[((size_t)b * (K + 1) + i) * V + x];
          }
        }
        const unsigned no = __ballot_sync(0xffffffffu, !ok && i < n), wrong = __ballot_sync(0xffffffffu, bad);
        if (no) {
          kept = i0 + __ffs(no) - 1;
          if (lane == 0 && P.err && (wrong >> (kept - i0) & 1)) atomicExch(P.err, kErrToken);
          break;
        }
      }
    }
    if (lane == 0) s_kept = kept, s_n = n;
  }
  __syncthreads();
  const int kept = s_kept;
  const float* p = P.p + ((size_t)b * (K + 1) + kept) * V;
  const float* q = kept < s_n ? P.q + ((size_t)b * K + kept) * V : nullptr;
  const float* e = P.noise + (size_t)b * V;
  const int share = ((V + parts - 1) / parts + 3) & ~3, lo = min(part * share, V), hi = min(lo + share, V);
  int next = 0;
  for (int pass = 0; pass < 2; ++pass) {  // the second only where the residual has no positive entry
    Best best = {0.f, lo < V ? lo : 0x7fffffff};  // quotients of 0: the lowest index
    float most = 0.f;
    scan<VEC>(best, most, &s_best, p, q, e, lo, hi);
    best.warp();
    if (lane == 0) warp_best[tid >> 5] = best;
    if (most > 0.f) s_any = 1;
    __syncthreads();
    if (tid < 32) {
      best = lane < kVerifyWarps ? warp_best[lane] : Best{0.f, 0x7fffffff};
      best.warp();
      if (lane < parts) {
        *cluster.map_shared_rank(&all_best[pass][part], lane) = best;
        *cluster.map_shared_rank(&all_any[pass][part], lane) = s_any;
      }
    }
    cluster.sync();
    int found = 0;
    Best all = {0.f, 0x7fffffff};
    for (int i = 0; i < parts; ++i) {
      found |= all_any[pass][i];
      all.take(all_best[pass][i].v, all_best[pass][i].i);
    }
    next = all.i;
    if (found || !q) break;
    q = nullptr;
  }
  if (part != 0) return;
  for (int i = tid; i <= K; i += kVerifyThreads)
    P.out[(size_t)b * (K + 1) + i] = i < kept ? P.tokens[(size_t)b * K + i] : i == kept ? next : -1;
  if (tid == 0) P.accepted[b] = kept;
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& P, cudaStream_t s) {
  // Shares of at least one step of every thread; eight CTAs a sequence, four where those fill the GPU twice over
  // (measured: 256 sequences of 131072 54 us with four, 57 with eight; 4 of 32000 8.2 and 6.3 us).
  const int most = 4 * P.B >= 2 * sm_count() ? 4 : kMaxCluster;
  int parts = 1;
  while (parts < most && P.V > 4 * kVerifyThreads * parts) parts *= 2;
  const bool vec = P.V % 4 == 0 && ((reinterpret_cast<uintptr_t>(P.p) | reinterpret_cast<uintptr_t>(P.q) |
                                     reinterpret_cast<uintptr_t>(P.noise)) & 15) == 0;
  const Launch at(dim3(P.B * parts), kVerifyThreads, 0, s, parts);
  return vec ? cudaLaunchKernelEx(&at.cfg, verify_kernel<true>, P) : cudaLaunchKernelEx(&at.cfg, verify_kernel<false>, P);
}

}  // namespace pw
