// Verification of drafted tokens: acceptance, then a draw from the residual
// distribution as the largest quotient r / e over the vocabulary.
//
// Bound: one row each of the target's probabilities, the noise and, where a
// draft was refused, the draft's probabilities, read once: HBM for a large
// batch, the chain draft count -> token -> its probabilities -> row for a
// small one.  A cluster of CTAs shares a sequence's vocabulary and joins its
// maxima through shared memory: one launch, no workspace, and the largest
// (quotient, lowest index) does not depend on any order.  Measured: 256
// sequences over 131072 tokens, half of them refused a draft, 336 MB in 54.5
// us (6.2 TB/s; 108 us when every index was divided); 4 over 32000 4.9 us.
#include <cooperative_groups.h>

#include <utility>

#include "pw_serve.h"

namespace pw {

namespace {

namespace cg = cooperative_groups;

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

// N x UN values of each array in flight a thread: all loads of a step go out before anything waits for one.
template <int N, int UN, bool Q>
__device__ __forceinline__ void scan_step(Best& best, float& most, int* cta_best, const float* p, const float* q,
                                          const float* e, int i0, int step) {
  float r[UN][N], c[UN][N], d[UN][N];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int i = i0 + u * step;
    if constexpr (N == 4) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(p + i)), y = __ldcs(reinterpret_cast<const float4*>(e + i));
      r[u][0] = x.x, r[u][1] = x.y, r[u][2] = x.z, r[u][3] = x.w;
      c[u][0] = y.x, c[u][1] = y.y, c[u][2] = y.z, c[u][3] = y.w;
      if constexpr (Q) {
        const float4 z = __ldcs(reinterpret_cast<const float4*>(q + i));
        d[u][0] = z.x, d[u][1] = z.y, d[u][2] = z.z, d[u][3] = z.w;
      }
    } else {
      r[u][0] = __ldcs(p + i);
      c[u][0] = __ldcs(e + i);
      if constexpr (Q) d[u][0] = __ldcs(q + i);
    }
  }
  const float bar = bar_of(__int_as_float(*reinterpret_cast<volatile int*>(cta_best)));
  bool some = false;
#pragma unroll
  for (int u = 0; u < UN; ++u)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (Q) r[u][k] -= d[u][k];
      most = fmaxf(most, r[u][k]);
      some |= r[u][k] >= bar * c[u][k];
    }
  if (some) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (r[u][k] >= bar * c[u][k]) weigh(best, cta_best, r[u][k], c[u][k], i0 + u * step + k);
  }
}

template <bool VEC, int NT, bool Q>
__device__ __forceinline__ void scan(Best& best, float& most, int* cta_best, const float* p, const float* q,
                                     const float* e, int lo, int hi) {
  constexpr int N = VEC ? 4 : 1, UN = VEC ? 1 : 4, STEP = N * NT;
  int i = lo + N * threadIdx.x;
#pragma unroll 1
  for (; i + (UN - 1) * STEP < hi; i += UN * STEP) scan_step<N, UN, Q>(best, most, cta_best, p, q, e, i, STEP);
  if constexpr (UN > 1) {
#pragma unroll 1
    for (; i < hi; i += STEP) scan_step<N, 1, Q>(best, most, cta_best, p, q, e, i, STEP);
  }
}

template <bool VEC, int NT>
__global__ void __launch_bounds__(NT, 2048 / NT) verify_kernel(const VerifyParams P) {
  __shared__ Best warp_best[(NT / 32)];
  __shared__ Best all_best[2][kMaxCluster];   // [pass][CTA of the cluster], written by all of them
  __shared__ int all_any[2][kMaxCluster];
  __shared__ int s_any, s_best, s_kept, s_n;
  behind_the_stream();
  let_next_start();
  const cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // every CTA runs before another one writes to its shared memory
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
        bool ok = true;
        if (i < K) {  // read whether or not it counts: the count is on its way too
          const int x = P.tokens[(size_t)b * K + i];
          ok = x >= 0 && x < V;
          if (ok) {
            const float uq = P.u[(size_t)b * K + i] * P.q[((size_t)b * K + i) * V + x];
            ok = uq < P.p[((size_t)b * (K + 1) + i) * V + x];
          }
        }
        const unsigned no = __ballot_sync(0xffffffffu, !ok && i < n);
        if (no) {
          kept = i0 + __ffs(no) - 1;
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
    if (q)
      scan<VEC, NT, true>(best, most, &s_best, p, q, e, lo, hi);
    else
      scan<VEC, NT, false>(best, most, &s_best, p, q, e, lo, hi);
    best.warp();
    if (lane == 0) warp_best[tid >> 5] = best;
    if (most > 0.f) s_any = 1;
    __syncthreads();
    if (pass == 0) cluster.barrier_wait(std::move(started));
    if (tid < 32) {
      best = lane < (NT / 32) ? warp_best[lane] : Best{0.f, 0x7fffffff};
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
  for (int i = tid; i <= K; i += NT) {
    const int x = i < K ? P.tokens[(size_t)b * K + i] : 0;
    P.out[(size_t)b * (K + 1) + i] = i < kept ? x : i == kept ? next : -1;
    if ((x < 0 || x >= V) && i < s_n && P.err) atomicExch(P.err, kErrToken);  // behind a refusal too
  }
  if (tid == 0) P.accepted[b] = kept;
}

}  // namespace

namespace {
template <int NT>
cudaError_t launch_shape(const VerifyParams& P, bool vec, int parts, cudaStream_t s) {
  const Launch at(dim3(P.B * parts), NT, 0, s, parts);
  return vec ? cudaLaunchKernelEx(&at.cfg, verify_kernel<true, NT>, P) : cudaLaunchKernelEx(&at.cfg, verify_kernel<false, NT>, P);
}
}  // namespace

cudaError_t launch_verify(const VerifyParams& P, cudaStream_t s) {
  const bool vec = P.V % 4 == 0 && ((reinterpret_cast<uintptr_t>(P.p) | reinterpret_cast<uintptr_t>(P.q) |
                                     reinterpret_cast<uintptr_t>(P.noise)) & 15) == 0;
  // Eight CTAs a sequence and at least a step of every thread, four where those alone are many (256 sequences of 131072 50.7
  // us with four, 52.6 with eight); CTAs of 512 threads while two of 256 on every SM would not be filled (14 sequences of
  // 131072 9.8 and 14.1 us, 91 of 94207 23.1 and 21.6).
  const int most = 4 * P.B >= 1000 ? 4 : kMaxCluster;
  int parts = 1;
  while (parts < most && P.V > 1024 * parts) parts *= 2;
  return (long long)P.B * parts > 2 * sm_count() ? launch_shape<256>(P, vec, parts, s) : launch_shape<512>(P, vec, parts, s);
}

}  // namespace pw
