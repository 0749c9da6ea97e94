// Eviction from the paged cache by accumulated attention weight: the weights
// of a step's queries added up by key (weigh), the choice of the tokens that
// stay (select), and their move into the first slots of a page table (move).
#include <math_constants.h>

#include "pw_heads.cuh"
#include "pw_mma.cuh"
#include "pw_serve.h"

namespace pw {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---- weigh --------------------------------------------------------------------
//
// out[i] = decay mass[i] + sum over rows r of e^(scale q_r . k_i - lse_r).
// The rows' statistics are given, so a key's sum needs no other key: a CTA
// takes kKeys keys of one sequence and all key heads, and adds up in a fixed
// order.  Bound by reading the keys once.  A lane reads 16 bytes of a key row
// at a time, straight into the fragments of the product: the order of the
// products inside a head does not matter as long as queries and keys share it.

constexpr int kWeighWarps = 8;
constexpr int kKeys = 64;            // keys a CTA

template <typename E, int D>
__global__ void __launch_bounds__(kWeighWarps * 32) weigh_kernel(const WeighParams P) {
  __shared__ float part[kWeighWarps][kKeys];
  behind_the_stream();
  let_next_start();
  const int b = blockIdx.y, key0 = blockIdx.x * kKeys, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int cap = (int)min((long long)P.table_stride << P.kv.page_shift, (long long)P.mass_stride), given = P.lens[b];
  const int len = min(max(given, 0), cap);
  if (given != len && blockIdx.x == 0 && tid == 0) atomicExch(P.kv.err, kErrLength);
  if (key0 >= len) return;
  for (int i = tid; i < kWeighWarps * kKeys; i += kWeighWarps * 32) part[i / kKeys][i % kKeys] = 0.f;
  __syncthreads();
  const int* table = P.table + (long long)b * P.table_stride;
  const int rows = P.ql * P.G, sure = len - P.ql + 1;  // keys below this are seen by every row
  // units: (key head, 16 keys) pairs, the heads' keys side by side, so that a warp keeps its queries
  constexpr int GROUPS = kKeys / 16;
  const int units = P.kv.hkv * GROUPS, per = (units + kWeighWarps - 1) / kWeighWarps;
  const float scale2 = P.scale * kLog2e;
#pragma unroll 1
  for (int row0 = 0; row0 < rows; row0 += 16) {
    int head = -1;
    uint32_t qf[D / 16][4];
    float ref[2];
    int vis[2];
#pragma unroll 1
    for (int u = warp * per; u < min(units, (warp + 1) * per); ++u) {
      const int h = u / GROUPS, first = key0 + (u % GROUPS) * 16;
      if (first >= len) continue;
      if (h != head) {
        head = h;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = row0 + g + 8 * i;
          const bool in = r < rows;
          const int tok = in ? r / P.G : 0, hd = in ? h * P.G + r - tok * P.G : 0;
          const long long at = (long long)b * P.ql + tok;
          const E* src = static_cast<const E*>(P.q.ptr) + at * P.q.token_stride + hd * P.q.head_stride + 8 * t4;
#pragma unroll
          for (int s = 0; s < D / 32; ++s) {
            const uint4 v = in ? *reinterpret_cast<const uint4*>(src + 32 * s) : make_uint4(0, 0, 0, 0);
            qf[2 * s][i] = v.x, qf[2 * s][2 + i] = v.y;
            qf[2 * s + 1][i] = v.z, qf[2 * s + 1][2 + i] = v.w;
          }
          const float lse = in ? P.lse[at * P.kv.hq + hd] : -CUDART_INF_F;
          vis[i] = !in || lse == -CUDART_INF_F ? 0 : sure + tok;  // a row that saw nothing weighs nothing
          ref[i] = lse * kLog2e;
        }
      }
      uint4 kr[2][D / 32];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int key = first + 8 * n;  // eight keys lie in one page
        const int page = key < len ? table[key >> P.kv.page_shift] : -1;
        const bool in = key < len && page >= 0 && page < P.kv.n_pages;
        if (key < len && !in && lane == 0) atomicExch(P.kv.err, kErrPage);
        const E* src = reinterpret_cast<const E*>(P.kv.k) + page * P.kv.page_stride + h * P.kv.head_stride +
                       ((key & ((1 << P.kv.page_shift) - 1)) + g) * P.kv.token_stride + 8 * t4;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) kr[n][s] = in ? __ldcs(reinterpret_cast<const uint4*>(src + 32 * s)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          mma16816<E>(s, qf[2 * c], kr[n][c].x, kr[n][c].y);
          mma16816<E>(s, qf[2 * c + 1], kr[n][c].z, kr[n][c].w);
        }
        float w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int key = first + 8 * n + 2 * t4 + k;
          w[k] = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) w[k] += key < vis[i] ? ex2(fmaf(s[2 * i + k], scale2, -ref[i])) : 0.f;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) w[k] += __shfl_xor_sync(0xffffffffu, w[k], o);
          if (g == 0) part[warp][key - key0] += w[k];
        }
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < kKeys && key0 + i < len; i += kWeighWarps * 32) {
    float w = 0.f;
#pragma unroll
    for (int k = 0; k < kWeighWarps; ++k) w += part[k][i];
    const long long at = (long long)b * P.mass_stride + key0 + i;
    P.out[at] = fmaf(P.decay, P.mass[at], w);
  }
}

// ---- select -------------------------------------------------------------------
//
// A CTA a sequence.  Of the n - recent older tokens the budget - recent of the
// largest masses stay: a radix search over the masses as ordered integers
// finds the smallest that stays and how many of its equals do (the first
// ones), and a scan in token order numbers them.

constexpr int kSelectThreads = 1024;

// Order of masses as unsigned integers: larger is heavier; -0 is 0, what is no number is lightest.
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams P) {
  __shared__ unsigned hist[256];
  __shared__ unsigned s_prefix, s_left;
  __shared__ int2 warp_sum[kSelectThreads / 32];
  behind_the_stream();
  let_next_start();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long old_cap = (long long)P.table_stride << P.kv.page_shift, new_cap = (long long)P.new_stride << P.kv.page_shift;
  const int cap = (int)min(old_cap, (long long)P.mass_stride), given = P.lens[b], n = min(max(given, 0), cap);
  if (given != n && tid == 0) atomicExch(P.kv.err, kErrLength);
  const int left = (int)min((long long)min(n, P.budget), new_cap);  // tokens that stay
  const int recent = min(P.recent, left), older = n - recent, need = left - recent;
  const float* mass = P.mass + (long long)b * P.mass_stride;
  int* kept = P.ws_kept + (long long)b * P.budget;
  float* held = P.ws_mass + (long long)b * P.budget;
  // the smallest key that stays (`bar`), and how many tokens of it
  unsigned bar = 0;
  int equal = older;
  if (need < older) {
    if (tid == 0) s_prefix = 0, s_left = need;
    __syncthreads();
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const unsigned prefix = s_prefix;
      for (int i = tid; i < older; i += kSelectThreads) {
        const unsigned k = mass_key(mass[i]);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[k >> shift & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // the digit that holds the s_left-th largest
        unsigned mine[8], sum = 0;  // lane 0 holds the largest digits
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += mine[k] = hist[255 - 8 * lane - k];
        unsigned scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, scan, o);
          if (lane >= o) scan += y;
        }
        unsigned before = scan - sum;
        const unsigned want = s_left;
        __syncwarp();
        // want = 0 (only the recent stay) ends on the largest digit, with none of it
        if ((before < want || (want == 0 && lane == 0)) && (scan >= want)) {
          int k = 0;
          while (k < 7 && before + mine[k] < want) before += mine[k++];
          s_prefix = prefix << 8 | (255 - 8 * lane - k);
          s_left = want - before;
        }
      }
      __syncthreads();
    }
    bar = s_prefix;
    equal = s_left;
  }
  // a run of tokens a thread, numbered in order
  const int per = (older + kSelectThreads - 1) / kSelectThreads, i0 = min(tid * per, older), i1 = min(i0 + per, older);
  const bool all = need >= older;
  int more = 0, same = 0;
  for (int i = i0; i < i1; ++i) {
    const unsigned k = all ? 1u : mass_key(mass[i]);
    more += k > bar;
    same += k == bar;
  }
  int2 scan = make_int2(more, same);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan.x, o), y = __shfl_up_sync(0xffffffffu, scan.y, o);
    if (lane >= o) scan.x += x, scan.y += y;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int at_more = scan.x - more, at_same = scan.y - same;
  for (int w = 0; w < warp; ++w) at_more += warp_sum[w].x, at_same += warp_sum[w].y;
  int at = at_more + min(at_same, equal);
  for (int i = i0; i < i1; ++i) {
    const float x = mass[i];
    const unsigned k = all ? 1u : mass_key(x);
    const bool stays = k > bar || (k == bar && at_same < equal);
    at_same += k == bar;
    if (stays) {
      kept[at] = i;
      held[at++] = x;
    }
  }
  for (int i = tid; i < recent; i += kSelectThreads) {
    kept[need + i] = older + i;
    held[need + i] = mass[older + i];
  }
  __syncthreads();  // the new masses may lie in the old ones' place
  float* out = P.new_mass + (long long)b * P.mass_stride;
  for (int i = tid; i < P.mass_stride; i += kSelectThreads) out[i] = i < left ? held[i] : 0.f;
  if (P.kept)
    for (int i = tid; i < P.budget; i += kSelectThreads) P.kept[(long long)b * P.budget + i] = i < left ? kept[i] : -1;
  if (tid == 0) P.new_lens[b] = left, P.ws_left[b] = left;
}

// ---- move ---------------------------------------------------------------------
//
// Kept token j goes to slot j.  j is never above the token's old place, so a
// CTA that goes through a row of places in order, and reads each step's rows
// before any of the step is written, may move them inside the same pages.  The
// rows of the next step are on their way meanwhile.  A CTA takes the keys or
// the values of one head (or a 64-byte column of them, where the rows alone
// would leave SMs idle).

constexpr int kMoveThreads = 256;

template <int LPR>  // lanes a row: 16 bytes each
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams P, int columns) {
  constexpr int U = 4, RPS = kMoveThreads / LPR, STEP = U * RPS;
  behind_the_stream();
  let_next_start();
  const int b = blockIdx.y, tid = threadIdx.x, sub = tid / LPR;
  int c = blockIdx.x;
  const int col = c % columns;
  c /= columns;
  char* cache = (c & 1) ? P.kv.v : P.kv.k;
  const long long base = (c >> 1) * P.kv.head_stride + (col * LPR + tid % LPR) * 8;
  const int left = P.ws_left[b], shift = P.kv.page_shift, mask = (1 << shift) - 1;
  const int* kept = P.ws_kept + (long long)b * P.budget;
  const int* from = P.table + (long long)b * P.table_stride;
  const int* to = P.new_table + (long long)b * P.new_stride;
  auto place = [&](const int* table, int i) -> uint4* {  // null outside the cache
    const int page = table[i >> shift];
    if (page < 0 || page >= P.kv.n_pages) return nullptr;
    return reinterpret_cast<uint4*>(cache + 2 * (page * P.kv.page_stride + (i & mask) * P.kv.token_stride + base));
  };
  uint4 row[U], next[U];
  uint4 *src[U], *dst[U], *next_dst[U];
  auto load = [&](int j0, uint4 (&r)[U], uint4* (&d)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * RPS + sub;
      src[u] = d[u] = nullptr;
      if (j < left) {
        src[u] = place(from, kept[j]);
        d[u] = place(to, j);
        if (!src[u] || !d[u]) atomicExch(P.kv.err, kErrPage);
        if (src[u] == d[u]) d[u] = nullptr;  // there already
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = make_uint4(0, 0, 0, 0);  // a page outside the cache reads as zeros
      if (src[u] && d[u]) r[u] = *src[u];
    }
  };
  load(0, row, dst);
#pragma unroll 1
  for (int j0 = 0; j0 < left; j0 += STEP) {
    load(j0 + STEP, next, next_dst);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u]) *dst[u] = row[u];
      row[u] = next[u];
      dst[u] = next_dst[u];
    }
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& P, cudaStream_t s) {
  const long long cap = min((long long)P.table_stride << P.kv.page_shift, (long long)P.mass_stride);
  const unsigned tiles = (unsigned)((cap + kKeys - 1) / kKeys);
  // without keys a CTA a sequence still looks at its length
  const Launch at(dim3(tiles ? tiles : 1, P.B), kWeighWarps * 32, 0, s);
  if (P.kv.dtype == PW_F16)
    return P.kv.d == 128 ? cudaLaunchKernelEx(&at.cfg, weigh_kernel<__half, 128>, P) : cudaLaunchKernelEx(&at.cfg, weigh_kernel<__half, 64>, P);
  return P.kv.d == 128 ? cudaLaunchKernelEx(&at.cfg, weigh_kernel<__nv_bfloat16, 128>, P)
                       : cudaLaunchKernelEx(&at.cfg, weigh_kernel<__nv_bfloat16, 64>, P);
}

cudaError_t launch_evict(const EvictParams& P, cudaStream_t s) {
  const Launch sel(dim3(P.B), kSelectThreads, 0, s);
  const cudaError_t e = cudaLaunchKernelEx(&sel.cfg, select_kernel, P);
  if (e != cudaSuccess || P.budget == 0) return e;
  const long long ctas = (long long)P.B * P.kv.hkv * 2;
  const bool split = ctas < 2 * sm_count();
  const int lpr = split ? 4 : P.kv.d / 8, columns = P.kv.d / 8 / lpr;
  const Launch at(dim3(P.kv.hkv * 2 * columns, P.B), kMoveThreads, 0, s);
  switch (lpr) {
    case 4: return cudaLaunchKernelEx(&at.cfg, move_kernel<4>, P, columns);
    case 8: return cudaLaunchKernelEx(&at.cfg, move_kernel<8>, P, columns);
    default: return cudaLaunchKernelEx(&at.cfg, move_kernel<16>, P, columns);
  }
}

}  // namespace pw
