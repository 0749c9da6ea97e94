// Attention of a decode batch over the paged cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// o = sum e^(s - m) v and l = sum e^(s - m) are rescaled when m grows, and
// partial (m, l, o) of disjoint key sets join exactly the same way.
#include <math_constants.h>

#include "pw_heads.cuh"
#include "pw_serve.h"

namespace pw {

namespace {

constexpr int kSimpleWarps = 4;

// Length of a table row's sequence, clamped to what its pages can hold.
__device__ __forceinline__ int clamp_len(int len, int stride, int page_shift, int* err) {
  const int most = stride << page_shift;
  if (len >= 0 && len <= most) return len;
  atomicExch(err, kErrLength);
  return len < 0 ? 0 : most;
}

// One CTA a (query token, head); its warps take every fourth key.
template <typename E, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32) attend_simple_kernel(const AttendParams P) {
  constexpr int PER = D / 32;
  __shared__ float sm[kSimpleWarps], sl[kSimpleWarps], so[kSimpleWarps][D];
  const int row = blockIdx.x, b = row / P.ql, j = row % P.ql, h = blockIdx.y, hk = h / P.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const KvView& kv = P.kv;
  int g = -1, lo = P.group_offsets ? 0 : -1;
  for (int i = 0; i <= P.n_groups && P.n_groups > 0; ++i) {  // bounds clamped to ascending values in [0, B]
    const int raw = P.group_offsets ? P.group_offsets[i] : i ? P.B : 0, hi = min(max(raw, max(lo, 0)), P.B);
    if (hi != raw) atomicExch(kv.err, kErrLength);
    if (i > 0 && b >= lo && b < hi) g = i - 1;
    lo = hi;
  }
  const int plen = g < 0 ? 0 : clamp_len(P.prefix_lens[g], P.prefix_stride, kv.page_shift, kv.err);
  const int slen = clamp_len(P.lens[b], P.table_stride, kv.page_shift, kv.err);
  const int vis = max(0, slen - P.ql + 1 + j);
  float q[PER], o[PER], m = -CUDART_INF_F, l = 0.f;
  const E* qp = static_cast<const E*>(P.q.ptr) + row * P.q.token_stride + h * P.q.head_stride;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = (float)qp[lane * PER + i];
    o[i] = 0.f;
  }
  for (int n = warp; n < plen + vis; n += kSimpleWarps) {
    const int at = n < plen ? n : n - plen;
    const int* tab = n < plen ? P.prefix_table + (size_t)g * P.prefix_stride : P.table + (size_t)b * P.table_stride;
    const int page = tab[at >> kv.page_shift];
    const bool in = page >= 0 && page < kv.n_pages;
    if (!in && lane == 0) atomicExch(kv.err, kErrPage);
    const size_t off = in ? page * kv.page_stride + hk * kv.head_stride +
                                (at & ((1 << kv.page_shift) - 1)) * kv.token_stride
                          : 0;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      s += in ? q[i] * (float)reinterpret_cast<const E*>(kv.k)[off + lane * PER + i] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= P.scale;
    const float mn = fmaxf(m, s), keep = m == -CUDART_INF_F ? 0.f : expf(m - mn), w = expf(s - mn);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      o[i] = o[i] * keep + (in ? w * (float)reinterpret_cast<const E*>(kv.v)[off + lane * PER + i] : 0.f);
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < PER; ++i) so[warp][lane * PER + i] = o[i];
  __syncthreads();
  float top = -CUDART_INF_F, sum = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kSimpleWarps; ++w) sum += sl[w] > 0.f ? sl[w] * expf(sm[w] - top) : 0.f;
  if (threadIdx.x < D) {
    float v = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) v += sl[w] > 0.f ? so[w][threadIdx.x] * expf(sm[w] - top) : 0.f;
    static_cast<E*>(P.out.ptr)[row * P.out.token_stride + h * P.out.head_stride + threadIdx.x] =
        (E)(sum > 0.f ? v / sum : 0.f);
  }
  if (threadIdx.x == 0 && P.lse) P.lse[(size_t)row * kv.hq + h] = sum > 0.f ? top + logf(sum) : -CUDART_INF_F;
}

template <typename E>
cudaError_t launch_typed(const AttendParams& P, cudaStream_t s) {
  const dim3 grid(P.B * P.ql, P.kv.hq);
  if (P.kv.d == 128)
    attend_simple_kernel<E, 128><<<grid, kSimpleWarps * 32, 0, s>>>(P);
  else
    attend_simple_kernel<E, 64><<<grid, kSimpleWarps * 32, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace

size_t attend_ws_bytes(const KvView&, int, int, int) { return 256; }

cudaError_t launch_attend(const AttendParams& P, void*, cudaStream_t s) {
  return P.kv.dtype == PW_F16 ? launch_typed<__half>(P, s) : launch_typed<__nv_bfloat16>(P, s);
}

}  // namespace pw
