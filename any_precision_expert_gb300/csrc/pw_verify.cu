// Verification of drafted tokens: acceptance, then a draw from the residual
// distribution as the largest quotient r / e over the vocabulary.
#include <math_constants.h>

#include "pw_serve.h"

namespace pw {

namespace {

constexpr int kVerifyThreads = 1024;

// A quotient and its index as one word that orders by quotient, then by the
// lower index.  Quotients are >= 0 (or +inf), so their bits order like they do.
__device__ __forceinline__ unsigned long long score_key(float r, float e, int i) {
  float v = r / e;
  if (!(v >= 0.f)) v = 0.f;
  v += 0.f;  // -0 -> +0
  return ((unsigned long long)__float_as_uint(v) << 32) | (0xffffffffu - (unsigned)i);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, k, o);
    if (y > k) k = y;
  }
  return k;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams P) {
  __shared__ unsigned long long best[32];
  __shared__ int positive;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, K = P.K, V = P.V;
  int n = 0;
  if (K > 0) {
    n = P.n_draft[b];
    if (n < 0 || n > K) {
      if (tid == 0 && P.err) atomicExch(P.err, kErrToken);
      n = n < 0 ? 0 : K;
    }
  }
  int kept = 0;
  for (int i = 0; i < n; ++i) {
    const int x = P.tokens[(size_t)b * K + i];
    if (x < 0 || x >= V) {
      if (tid == 0 && P.err) atomicExch(P.err, kErrToken);
      break;
    }
    const float uq = P.u[(size_t)b * K + i] * P.q[((size_t)b * K + i) * V + x];
    if (!(uq < P.p[((size_t)b * (K + 1) + i) * V + x])) break;
    kept = i + 1;
  }
  const float* p = P.p + ((size_t)b * (K + 1) + kept) * V;
  const float* q = kept < n ? P.q + ((size_t)b * K + kept) * V : nullptr;
  const float* e = P.noise + (size_t)b * V;
  if (tid == 0) positive = 0;
  unsigned long long top = 0;
  for (int pass = 0; pass < 2; ++pass) {  // the second only where the residual has no positive entry
    __syncthreads();
    bool any = false;
    top = 0;
    for (int i = tid; i < V; i += kVerifyThreads) {
      const float r = fmaxf(q ? p[i] - q[i] : p[i], 0.f);
      any |= r > 0.f;
      const unsigned long long k = score_key(r, e[i], i);
      if (k > top) top = k;
    }
    if (any) positive = 1;
    top = warp_max(top);
    if (lane == 0) best[tid >> 5] = top;
    __syncthreads();
    if (positive || !q) break;
    q = nullptr;
  }
  if (tid < 32) top = warp_max(best[lane]);
  for (int i = tid; i <= K; i += kVerifyThreads) {
    if (i == kept) continue;
    P.out[(size_t)b * (K + 1) + i] = i < kept ? P.tokens[(size_t)b * K + i] : -1;
  }
  if (tid == 0) {
    P.out[(size_t)b * (K + 1) + kept] = (int)(0xffffffffu - (unsigned)top);
    P.accepted[b] = kept;
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& P, cudaStream_t s) {
  verify_kernel<<<P.B, kVerifyThreads, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace pw
