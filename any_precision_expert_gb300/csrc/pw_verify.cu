// Verification of drafted tokens: acceptance, then a draw from the residual
// distribution as the largest quotient r / e over the vocabulary.
//
// Bound: one row each of the target's probabilities, the noise and, where a
// draft was refused, the draft's probabilities, read once: HBM for a large
// batch, the chain draft count -> token -> its probabilities -> row for a
// small one.  A cluster of CTAs shares a sequence's vocabulary and joins its
// maxima through shared memory of its first CTA: one launch, no workspace, and
// the largest (quotient, lowest index) does not depend on any order.
#include <cooperative_groups.h>

#include "pw_serve.h"

namespace pw {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
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

// One index of the vocabulary (in ascending order within a thread).
__device__ __forceinline__ void weigh(Best& best, bool& any, float r, float e, int i) {
  r = fmaxf(r, 0.f);  // NaN counts as 0
  any |= r > 0.f;
  const float v = r / e;
  if (v > best.v) best.v = v, best.i = i;  // NaN does not; equal ones keep the lower index
}

template <bool VEC>
__device__ __forceinline__ void scan(Best& best, bool& any, const float* p, const float* q, const float* e, int lo,
                                     int hi) {
  if constexpr (VEC) {
    constexpr int UN = 2;
    for (int i0 = lo + 4 * threadIdx.x; i0 < hi; i0 += 4 * UN * kVerifyThreads) {
      float4 a[UN], b[UN], c[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + 4 * u * kVerifyThreads;
        if (i < hi) {
          a[u] = __ldcs(reinterpret_cast<const float4*>(p + i));
          c[u] = __ldcs(reinterpret_cast<const float4*>(e + i));
          b[u] = q ? __ldcs(reinterpret_cast<const float4*>(q + i)) : make_float4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + 4 * u * kVerifyThreads;
        if (i < hi) {
          weigh(best, any, a[u].x - b[u].x, c[u].x, i);
          weigh(best, any, a[u].y - b[u].y, c[u].y, i + 1);
          weigh(best, any, a[u].z - b[u].z, c[u].z, i + 2);
          weigh(best, any, a[u].w - b[u].w, c[u].w, i + 3);
        }
      }
    }
  } else {
    constexpr int UN = 4;
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += UN * kVerifyThreads) {
      float a[UN], b[UN], c[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * kVerifyThreads;
        if (i < hi) {
          a[u] = __ldcs(p + i);
          c[u] = __ldcs(e + i);
          b[u] = q ? __ldcs(q + i) : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u)
        if (i0 + u * kVerifyThreads < hi) weigh(best, any, a[u] - b[u], c[u], i0 + u * kVerifyThreads);
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams P) {
  __shared__ Best warp_best[kVerifyWarps];
  __shared__ Best cta_best[kMaxCluster];   // the first CTA's copy is used
  __shared__ int cta_any[kMaxCluster];
  __shared__ int s_any, s_kept, s_n;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int b = blockIdx.x / parts, tid = threadIdx.x, lane = tid & 31, K = P.K, V = P.V;
  if (tid == 0) s_any = 0;
  if (tid < 32) {
    int n = 0;
    if (K > 0) {
      n = P.n_draft[b];
      if (n < 0 || n > K) {
        if (lane == 0 && P.err) atomicExch(P.err, kErrToken);
        n = n < 0 ? 0 : K;
      }
    }
    int kept = n;
    for (int i0 = 0; i0 < n; i0 += 32) {  // the drafts side by side; the first refusal ends the kept ones
      const int i = i0 + lane;
      bool ok = true, bad = false;
      if (i < n) {
        const int x = P.tokens[(size_t)b * K + i];
        bad = x < 0 || x >= V;
        ok = !bad;
        if (ok) {
          const float uq = P.u[(size_t)b * K + i] * P.q[((size_t)b * K + i) * V + x];
          ok = uq < P.p[((size_t)b * (K + 1) + i) * V + x];
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok), wrong = __ballot_sync(0xffffffffu, bad);
      if (no) {
        kept = i0 + __ffs(no) - 1;
        if (lane == 0 && P.err && (wrong >> (kept - i0) & 1)) atomicExch(P.err, kErrToken);
        break;
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
    Best best = {0.f, lo < V ? lo : 0x7fffffff};  // quotients of 0 and below: the lowest index
    bool any = false;
    scan<VEC>(best, any, p, q, e, lo, hi);
    best.warp();
    if (lane == 0) warp_best[tid >> 5] = best;
    if (any) s_any = 1;
    __syncthreads();
    if (tid < 32) {
      best = lane < kVerifyWarps ? warp_best[lane] : Best{0.f, 0x7fffffff};
      best.warp();
      if (lane == 0) {
        *cluster.map_shared_rank(&cta_best[part], 0) = best;
        *cluster.map_shared_rank(&cta_any[part], 0) = s_any;
      }
    }
    cluster.sync();
    int found = 0;
    Best all = {0.f, 0x7fffffff};
    for (int i = 0; i < parts; ++i) {
      found |= *cluster.map_shared_rank(&cta_any[i], 0);
      const Best* o = cluster.map_shared_rank(&cta_best[i], 0);
      all.take(o->v, o->i);
    }
    next = all.i;
    cluster.sync();  // every CTA has read the first one's shared memory
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
  // a share of at least one step of every thread, and at most eight CTAs a sequence
  int parts = 1;
  while (parts < kMaxCluster && P.V > 4 * kVerifyThreads * parts) parts *= 2;
  const bool vec = P.V % 4 == 0 && ((reinterpret_cast<uintptr_t>(P.p) | reinterpret_cast<uintptr_t>(P.q) |
                                     reinterpret_cast<uintptr_t>(P.noise)) & 15) == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.B * parts);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return vec ? cudaLaunchKernelEx(&cfg, verify_kernel<true>, P) : cudaLaunchKernelEx(&cfg, verify_kernel<false>, P);
}

}  // namespace pw
