// RMS norm of query and key heads, the position rotation, and the append of
// keys and values to the paged cache, in one pass.
//
// A head row of D values lies in D / 8 lanes of a warp, eight values a lane,
// placed so that a lane holds both values of every pair it turns: for the
// half-split rotation four values i .. i + 3 and their partners i + rot / 2
// .., for the interleaved one eight consecutive values.  So a rotation needs
// no exchange, four cosines and four sines serve a lane, and the row's mean of
// squares is a few shuffles.  All arithmetic is fp32; an output is rounded
// once.
//
// Bound: every row is read and written once and little is computed, so HBM
// for long prompts, launch and load latency for a decode step.  A warp takes U
// steps of rows of one token and kind (query, key or value), so that its loads
// are in flight together and its cosines, sines and weights are loaded once.
// Measured: 16384 tokens of 40 heads of 128 in 55 us, 6.3 TB/s (one row a warp
// in flight 100 us, eight 76; with partners exchanged by shuffles 169); one
// token 2.3 us, the launch.
#include "pw_heads.cuh"
#include "pw_serve.h"

namespace pw {

namespace {

constexpr int kRopeThreads = 128;  // smaller CTAs, so that the ends of some overlap the loads of others

// Row chunks of a token: queries, keys, values.
struct Chunks {
  int q, k, v;
  __host__ __device__ Chunks(const RopeParams& P, int rows)
      : q((P.hq + rows - 1) / rows), k((P.hk + rows - 1) / rows), v((P.hv + rows - 1) / rows) {}
  __host__ __device__ int all() const { return q + k + v; }
};

template <typename E>
__device__ __forceinline__ void load_pair(const E* p, int a0, int a1, uint4& r) {
  const uint2 lo = *reinterpret_cast<const uint2*>(p + a0), hi = *reinterpret_cast<const uint2*>(p + a1);
  r = make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// The same of a row that is read once: its lines are the first to leave the L2.
template <typename E>
__device__ __forceinline__ void stream_pair(const E* p, int a0, int a1, uint4& r) {
  const uint2 lo = __ldcs(reinterpret_cast<const uint2*>(p + a0)), hi = __ldcs(reinterpret_cast<const uint2*>(p + a1));
  r = make_uint4(lo.x, lo.y, hi.x, hi.y);
}

template <typename E, int D, int U, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams P) {
  behind_the_stream();
  let_next_start();
  constexpr int LPR = D / 8;          // lanes a row
  constexpr int RPW = 32 / LPR;       // rows a warp holds side by side
  constexpr int ROWS = RPW * U;       // rows of a unit
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const Chunks ch(P, ROWS);
  const unsigned per = ch.all(), unit = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const unsigned t = unit / per;
  if (t >= (unsigned)P.T) return;
  int c = unit - t * per;
  const int kind = c < ch.q ? 0 : c < ch.q + ch.k ? 1 : 2;
  c -= kind == 0 ? 0 : kind == 1 ? ch.q : ch.q + ch.k;
  const int nrows = kind == 0 ? P.hq : kind == 1 ? P.hk : P.hv, h0 = c * ROWS + sub;
  // this lane's values: a0 .. a0 + 3 and a1 .. a1 + 3 of the row
  const bool turns = kind < 2 && 8 * l < P.rot;
  int a0 = 8 * l, a1 = 8 * l + 4;
  if (!INTER && turns) a0 = 4 * l, a1 = (P.rot >> 1) + 4 * l;
  const pw_rows in = kind == 0 ? P.q : kind == 1 ? P.k : P.v;
  const E* src = static_cast<const E*>(in.ptr) + t * in.token_stride;
  uint4 raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * RPW;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (h < nrows) stream_pair(src + h * in.head_stride, a0, a1, raw[i]);
  }
  E* dst;
  long long dst_stride;
  if (kind == 0 || !P.slots) {
    const pw_rows& o = kind == 0 ? P.q_out : P.k_out;
    dst = static_cast<E*>(o.ptr) + t * o.token_stride;
    dst_stride = o.head_stride;
  } else {
    const int slot = P.slots[t];
    if (slot < 0) return;
    if ((slot >> P.kv.page_shift) >= P.kv.n_pages) {
      if (lane == 0) atomicExch(P.err, kErrSlot);
      return;
    }
    dst = reinterpret_cast<E*>(kind == 1 ? P.kv.k : P.kv.v) + (slot >> P.kv.page_shift) * P.kv.page_stride +
          (slot & ((1 << P.kv.page_shift) - 1)) * P.kv.token_stride;
    dst_stride = P.kv.head_stride;
  }
  if (kind < 2 && (P.rot > 0 || (kind == 0 ? P.qw : P.kw))) {  // else the bits are copied
    float4 cs = make_float4(1, 1, 1, 1), sn = make_float4(0, 0, 0, 0);
    if (turns) {
      int pos = P.positions[t];
      if (pos < 0 || pos >= P.max_pos) {
        if (l == 0 && P.err) atomicExch(P.err, kErrPosition);
        pos = pos < 0 ? 0 : P.max_pos - 1;
      }
      const float* row = P.cos_sin + (long long)pos * P.rot + 4 * l;
      cs = *reinterpret_cast<const float4*>(row);
      sn = *reinterpret_cast<const float4*>(row + (P.rot >> 1));
    }
    const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
    const void* w = kind == 0 ? P.qw : P.kw;
    float g[8];
    if (w) {
      uint4 gr;
      load_pair(static_cast<const E*>(w), a0, a1, gr);
      unpack8<E>(gr, g);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float x[8];
      unpack8<E>(raw[i], x);
      if (w) {
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float inv = rsqrtf(sq * (1.f / D) + P.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j];
      }
      if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float& a = x[INTER ? 2 * j : j];
          float& b = x[INTER ? 2 * j + 1 : 4 + j];
          const float ta = a * cv[j] - b * sv[j];
          b = b * cv[j] + a * sv[j];
          a = ta;
        }
      }
      raw[i] = pack8<E>(x);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * RPW;
    if (h >= nrows) continue;
    E* to = dst + h * dst_stride;
    __stcs(reinterpret_cast<uint2*>(to + a0), make_uint2(raw[i].x, raw[i].y));
    __stcs(reinterpret_cast<uint2*>(to + a1), make_uint2(raw[i].z, raw[i].w));
  }
}

template <typename E, int D, int U>
cudaError_t launch_one(const RopeParams& P, cudaStream_t s) {
  const long long units = (long long)P.T * Chunks(P, 32 / (D / 8) * U).all();
  const long long blocks = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 0x7fffffffll || units > 0xffffff00ll) return cudaErrorInvalidConfiguration;
  const Launch at(dim3((unsigned)blocks), kRopeThreads, 0, s);
  return P.interleaved ? cudaLaunchKernelEx(&at.cfg, rope_kernel<E, D, U, true>, P)
                       : cudaLaunchKernelEx(&at.cfg, rope_kernel<E, D, U, false>, P);
}

template <typename E>
cudaError_t launch_typed(const RopeParams& P, int d, cudaStream_t s) {
  // Below 2^20 values one row step a warp, so that there are more warps (append of 128 tokens of 48 heads of 128: 2.26 us,
  // 2.61 with four; of 256: 3.01 and 2.89; of 1024: 8.0 and 6.2).
  const bool few = (long long)P.T * (P.hq + P.hk + P.hv) * d < (1 << 20);
  if (d == 128) return few ? launch_one<E, 128, 1>(P, s) : launch_one<E, 128, 4>(P, s);
  return few ? launch_one<E, 64, 1>(P, s) : launch_one<E, 64, 4>(P, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& P, int dtype, int d, cudaStream_t s) {
  return dtype == PW_F16 ? launch_typed<__half>(P, d, s) : launch_typed<__nv_bfloat16>(P, d, s);
}

}  // namespace pw
