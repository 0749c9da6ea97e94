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
// Measured: 64 sequences to 4095, 8 heads of 128, 270 MB in 49.6 us (5.4 TB/s).
// The grid goes by the tables' and masses' width, and a CTA past a sequence's
// length reads that and leaves: behind rows of 32768 / 131072 / 2^20 positions
// the same call takes 58 / 86 / 526 us, 64 sequences to 200 20 / 68 / 526
// instead of 15.  More than 16 rows a key head read the keys once for every 16.

// CTAs of kWeighWarps warps take kKeys keys: 64 by 8 where there are few, so that more SMs share them, 128 by 4 where
// there are many, so that a CTA's start weighs less (5 sequences to 1500 took 1.8 times as long in the
// second shape, 64 to 4095 9 % longer in the first).
template <typename E, int D, int kKeys, int kWeighWarps>
__global__ void __launch_bounds__(kWeighWarps * 32, 16 / kWeighWarps) weigh_kernel(const WeighParams P) {
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
    const int u1 = min(units, (warp + 1) * per);
    auto next = [&](int u) {  // the next unit with keys
      while (u < u1 && key0 + (u % GROUPS) * 16 >= len) ++u;
      return u;
    };
    auto load = [&](int u, uint4 (&kr)[2][D / 32]) {
      const int h = u / GROUPS, first = key0 + (u % GROUPS) * 16;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int key = first + 8 * n;  // eight keys lie in one page
        const int page = u < u1 && key < len ? table[key >> P.kv.page_shift] : -1;
        const bool in = page >= 0 && page < P.kv.n_pages;
        if (u < u1 && key < len && !in && lane == 0) atomicExch(P.kv.err, kErrPage);
        const E* src = reinterpret_cast<const E*>(P.kv.k) + page * P.kv.page_stride + h * P.kv.head_stride +
                       ((key & ((1 << P.kv.page_shift) - 1)) + g) * P.kv.token_stride + 8 * t4;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) kr[n][s] = in ? __ldcs(reinterpret_cast<const uint4*>(src + 32 * s)) : make_uint4(0, 0, 0, 0);
      }
    };
    auto weigh = [&](int u, const uint4 (&kr)[2][D / 32]) {
      const int h = u / GROUPS, first = key0 + (u % GROUPS) * 16;
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
    };
    // two units' keys in registers: one on its way while the other is weighed
    uint4 ka[2][D / 32], kb[2][D / 32];
    int u = next(warp * per);
    load(u, ka);
#pragma unroll 1
    while (u < u1) {
      const int v = next(u + 1);
      load(v, kb);
      weigh(u, ka);
      if (v >= u1) break;
      u = next(v + 1);
      load(u, ka);
      weigh(v, kb);
    }
  }
  __syncthreads();
  for (int i = tid; i < kKeys && key0 + i < len; i += kWeighWarps * 32) {
    float w = 0.f;
#pragma unroll
    for (int k = 0; k < kWeighWarps; ++k) w += part[k][i];
    const long long at = (long long)b * P.mass_stride + key0 + i;
    P.out[at] = P.decay == 0.f ? w : fmaf(P.decay, P.mass[at], w);
  }
}

// ---- select -------------------------------------------------------------------
//
// A CTA a sequence.  Of the n - recent older tokens the budget - recent of the
// largest masses stay: a radix search over the masses as ordered integers finds
// the smallest that stays and how many of its equals do (the first ones), and a
// scan in token order numbers them.  Latency bounds it (64 sequences to 8190
// 16 us); masses of up to kSpan tokens stay in registers over its passes.

constexpr int kSelectThreads = 1024;
constexpr int kOwn = 8;                          // masses a thread holds
constexpr int kSpan = kOwn * kSelectThreads;

// Order of masses as unsigned integers: larger is heavier; -0 is 0, what is no number is lightest.
__device__ __forceinline__ unsigned mass_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The cache slot of position i of a page table's row; -1 outside the cache.
__device__ __forceinline__ int slot_of(const KvView& kv, const int* table, int i) {
  const int page = table[i >> kv.page_shift];
  return page < 0 || page >= kv.n_pages ? -1 : (page << kv.page_shift) + (i & ((1 << kv.page_shift) - 1));
}

constexpr int kBins = 2048;                      // of a digit of the search: 11, 11 and 10 bits

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams P) {
  __shared__ unsigned hist[kBins];
  __shared__ unsigned s_prefix, s_left;
  __shared__ unsigned count[kOwn * 32];            // of 1024 tokens by warp: heavier ones, and equal ones << 16; then their sums
  __shared__ unsigned s_all;
  behind_the_stream();
  let_next_start();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long old_cap = (long long)P.table_stride << P.kv.page_shift, new_cap = (long long)P.new_stride << P.kv.page_shift;
  const int cap = (int)min(old_cap, (long long)P.mass_stride), given = P.lens[b], n = min(max(given, 0), cap);
  if (given != n && tid == 0) atomicExch(P.kv.err, kErrLength);
  const int left = (int)min((long long)min(n, P.budget), new_cap);  // tokens that stay
  const int recent = min(P.recent, left), older = n - recent, need = left - recent;
  const float* mass = P.mass + (long long)b * P.mass_stride;
  const int *from = P.table + (long long)b * P.table_stride, *to = P.new_table + (long long)b * P.new_stride;
  const long long row = (long long)b * P.budget;
  int2* moves = P.ws_moves + row;
  float* out = P.new_mass + (long long)b * P.mass_stride;
  float own[kOwn];
  // positions are unsigned: a span's first may pass 2^31 where it ends the walk, and a span's last does before that
  const unsigned candidates = older;
  auto load = [&](unsigned first) {
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const unsigned i = first + k * kSelectThreads + tid;
      own[k] = i < candidates ? mass[i] : 0.f;
    }
  };
  // Token i stays, as number `at`.  Masses may go to their own place: `at` is never above i, and what a span's tokens
  // write was read before (the span's own masses ahead of the barriers in it).
  auto keep = [&](int at, int i, float x) {
    const int src = slot_of(P.kv, from, i), dst = slot_of(P.kv, to, at);
    if (src < 0 || dst < 0) atomicExch(P.kv.err, kErrPage);
    moves[at] = make_int2(src, src == dst ? -1 : dst);
    out[at] = x;
    if (P.kept) P.kept[row + at] = i;
  };
  load(0);
  const bool all = need >= older;
  // the smallest key that stays (`bar`), and how many tokens of it
  unsigned bar = 0, equal = 0;
  if (!all) {
    if (tid == 0) s_prefix = 0, s_left = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      const unsigned prefix = s_prefix, want = s_left;
#pragma unroll 1
      for (unsigned first = 0; first < candidates; first += kSpan) {
        if (older > kSpan) load(first);
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          if (first + k * kSelectThreads + tid >= candidates) break;
          const unsigned key = mass_key(own[k]);
          if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1u);
        }
      }
      __syncthreads();
      // the digit that holds the want-th largest; thread 0 has the two largest
      const unsigned high = hist[kBins - 1 - 2 * tid], low = hist[kBins - 2 - 2 * tid];
      unsigned scan = high + low;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      if (lane == 31) count[warp] = scan;
      __syncthreads();
      unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? count[lane] : 0u);  // in the warps in front
      before += scan - high - low;
      // want = 0 (only the recent stay) ends on the largest digit, with none of it
      if ((before < want && want <= before + high) || (want == 0 && tid == 0)) {
        s_prefix = prefix << bits | (kBins - 1 - 2 * tid & ((1u << bits) - 1));
        s_left = want - before;
      } else if (before + high < want && want <= before + high + low) {
        s_prefix = prefix << bits | (kBins - 2 - 2 * tid & ((1u << bits) - 1));
        s_left = want - before - high;
      }
      __syncthreads();
    }
    bar = s_prefix;
    equal = s_left;
  }
  unsigned more_before = 0, same_before = 0;  // in the spans before
#pragma unroll 1
  for (unsigned first = 0; first < candidates; first += kSpan) {
    if (older > kSpan) load(first);
    unsigned at[kOwn];  // heavier and equal tokens of the warp's 32 in front of this thread's, with its own flags
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const bool in = first + k * kSelectThreads + tid < candidates;
      const unsigned key = mass_key(own[k]);
      const unsigned more = __ballot_sync(0xffffffffu, in && (all || key > bar));
      const unsigned same = __ballot_sync(0xffffffffu, in && !all && key == bar);
      const unsigned front = (1u << lane) - 1;
      at[k] = __popc(more & front) | __popc(same & front) << 8 | (more >> lane & 1) << 16 | (same >> lane & 1) << 17;
      if (lane == 0) count[k * 32 + warp] = __popc(more) | __popc(same) << 16;
    }
    __syncthreads();
    if (warp == 0) {  // sums in front of every group of 32: of at most kSpan tokens, so both fit 16 bits
      unsigned mine[kOwn], sum = 0;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) sum += mine[k] = count[lane * kOwn + k];
      unsigned scan = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      if (lane == 31) s_all = scan;
      scan -= sum;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        count[lane * kOwn + k] = scan;
        scan += mine[k];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const unsigned sums = count[k * 32 + warp];
      const unsigned more = more_before + (sums & 0xffff) + (at[k] & 255), same = same_before + (sums >> 16) + (at[k] >> 8 & 255);
      const bool stays = (at[k] >> 16 & 1) || ((at[k] >> 17 & 1) && same < equal);
      if (stays) keep(more + min(same, equal), first + k * kSelectThreads + tid, own[k]);
    }
    more_before += s_all & 0xffff, same_before += s_all >> 16;
    __syncthreads();
  }
  // the recent ones, a step's masses read before any of it is written, then zeros behind them
#pragma unroll 1
  for (int i = tid; i - tid < recent; i += kSelectThreads) {
    const float x = i < recent ? mass[older + i] : 0.f;
    __syncthreads();
    if (i < recent) keep(need + i, older + i, x);
  }
  __syncthreads();
  for (int i = left + tid; i < P.mass_stride; i += kSelectThreads) out[i] = 0.f;
  if (P.kept)
    for (int i = left + tid; i < P.budget; i += kSelectThreads) P.kept[row + i] = -1;
  if (tid == 0) P.new_lens[b] = left, P.ws_left[b] = left;
}

// ---- move ---------------------------------------------------------------------
//
// Kept token j goes to slot j.  j is never above the token's old place, so a
// CTA that goes through a row of places in order, and has each step's rows in
// registers before any of the step is written, may move them inside the same
// pages; the next step's rows and the slots of the one after are on their way
// meanwhile.  A CTA takes the keys or the values of one head (or a 64-byte
// column of them, where whole rows would leave SMs idle).  Bound by HBM: 64
// sequences to 2048 tokens of 8 heads of 128, 1.03 GB in 156 us (6.3 TB/s read
// and written); bulk copies of a row each go out one in 12 cycles an SM, 176 us.

constexpr int kMoveThreads = 128;

template <int LPR>  // lanes a row: 16 bytes each
__global__ void __launch_bounds__(kMoveThreads, 8) move_kernel(const EvictParams P, int columns) {
  constexpr int U = 4, RPS = kMoveThreads / LPR, STEP = U * RPS;
  behind_the_stream();
  let_next_start();
  const int b = blockIdx.y, tid = threadIdx.x, sub = tid / LPR, c = blockIdx.x / columns, col = blockIdx.x % columns;
  char* cache = ((c & 1) ? P.kv.v : P.kv.k) + 2 * (c >> 1) * P.kv.head_stride + (col * LPR + tid % LPR) * 16;
  const int left = P.ws_left[b], shift = P.kv.page_shift, mask = (1 << shift) - 1;
  const int2* moves = P.ws_moves + (long long)b * P.budget;
  auto place = [&](int slot) {
    return reinterpret_cast<uint4*>(cache + 2 * ((slot >> shift) * P.kv.page_stride + (slot & mask) * P.kv.token_stride));
  };
  int2 slots[U];
  uint4 row[U], next[U];
  int dst[U], next_dst[U];
  auto look = [&](int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * RPS + sub;
      slots[u] = j < left ? moves[j] : make_int2(-1, -1);
    }
  };
  auto load = [&](uint4 (&r)[U], int (&d)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = make_uint4(0, 0, 0, 0);  // a page outside the cache reads as zeros
      d[u] = slots[u].y;
      if (slots[u].x >= 0 && slots[u].y >= 0) r[u] = *place(slots[u].x);
    }
  };
  look(0);
  load(row, dst);
  look(STEP);
#pragma unroll 1
  for (int j0 = 0; j0 < left; j0 += STEP) {
    load(next, next_dst);
    look(j0 + 2 * STEP);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] >= 0) *place(dst[u]) = row[u];
      row[u] = next[u];
      dst[u] = next_dst[u];
    }
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& P, cudaStream_t s) {
  const long long cap = min((long long)P.table_stride << P.kv.page_shift, (long long)P.mass_stride);
  const bool many = P.B * (cap / 64) > 16 * sm_count();
  const int keys = many ? 128 : 64;
  const unsigned tiles = (unsigned)((cap + keys - 1) / keys);
  // without keys a CTA a sequence still looks at its length
  const Launch at(dim3(tiles ? tiles : 1, P.B), many ? 128 : 256, 0, s);
  auto go = [&](auto few, auto lots) { return many ? cudaLaunchKernelEx(&at.cfg, lots, P) : cudaLaunchKernelEx(&at.cfg, few, P); };
  if (P.kv.dtype == PW_F16)
    return P.kv.d == 128 ? go(weigh_kernel<__half, 128, 64, 8>, weigh_kernel<__half, 128, 128, 4>)
                         : go(weigh_kernel<__half, 64, 64, 8>, weigh_kernel<__half, 64, 128, 4>);
  return P.kv.d == 128 ? go(weigh_kernel<__nv_bfloat16, 128, 64, 8>, weigh_kernel<__nv_bfloat16, 128, 128, 4>)
                       : go(weigh_kernel<__nv_bfloat16, 64, 64, 8>, weigh_kernel<__nv_bfloat16, 64, 128, 4>);
}

cudaError_t launch_evict(const EvictParams& P, cudaStream_t s) {
  const Launch sel(dim3(P.B), kSelectThreads, 0, s);
  const cudaError_t e = cudaLaunchKernelEx(&sel.cfg, select_kernel, P);
  if (e != cudaSuccess) return e;
  // 64-byte columns where whole rows leave SMs idle (see move_kernel)
  const bool split = (long long)P.B * P.kv.hkv * 2 < 2 * sm_count();
  const int row = 2 * P.kv.d, columns = split ? row / 64 : 1;
  const Launch at(dim3(P.kv.hkv * 2 * columns, P.B), kMoveThreads, 0, s);
  switch (row / columns) {
    case 64: return cudaLaunchKernelEx(&at.cfg, move_kernel<4>, P, columns);
    case 128: return cudaLaunchKernelEx(&at.cfg, move_kernel<8>, P, columns);
    default: return cudaLaunchKernelEx(&at.cfg, move_kernel<16>, P, columns);
  }
}

}  // namespace pw
