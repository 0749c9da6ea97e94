// RMS norm of query and key heads, the position rotation, and the append of
// keys and values to the paged cache, in one pass.
//
// A head row of D values lies in D / 8 lanes of a warp, 16 bytes a lane, so a
// row's mean of squares is a few shuffles and the partner of a half-split
// rotation (value i turns with i + rot / 2) sits rot / 16 lanes away.  All
// arithmetic is fp32 and an output is rounded once.
//
// Bound: every row is read and written once and little is computed, so HBM
// for long prompts, launch and load latency for a decode step.
#include "pw_heads.cuh"
#include "pw_serve.h"

namespace pw {

namespace {

constexpr int kRopeThreads = 256;

template <typename E, int D, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams P) {
  constexpr int LPR = D / 8;          // lanes a row
  constexpr int RPW = 32 / LPR;       // rows a warp holds side by side
  constexpr int ROWS = RPW * U;       // rows of a unit
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int nrows = P.hq + P.hk + P.hv;
  const int per = (nrows + ROWS - 1) / ROWS;
  const long long units = (long long)P.T * per;
  const int half = P.rot >> 1;
  for (long long unit = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); unit < units;
       unit += (long long)gridDim.x * (kRopeThreads / 32)) {
    const int t = (int)(unit / per), r0 = (int)(unit % per) * ROWS;
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * RPW + sub;
      if (r >= nrows) continue;
      const bool isq = r < P.hq, isk = !isq && r < P.hq + P.hk;
      const pw_rows& in = isq ? P.q : isk ? P.k : P.v;
      const int h = isq ? r : isk ? r - P.hq : r - P.hq - P.hk;
      raw[i] = *reinterpret_cast<const uint4*>(static_cast<const E*>(in.ptr) + t * in.token_stride +
                                               h * in.head_stride + 8 * l);
    }
    // this lane's cosines and sines: values 8 l .. 8 l + 7 of the row
    float c[8], s[8];
    const bool turns = 8 * l < P.rot;
    if (turns) {
      int pos = P.positions[t];
      if (pos < 0 || pos >= P.max_pos) {
        if (lane == 0 && P.err) atomicExch(P.err, kErrPosition);
        pos = pos < 0 ? 0 : P.max_pos - 1;
      }
      const float* cs = P.cos_sin + (long long)pos * P.rot;
      if (P.interleaved) {
        const float4 cc = *reinterpret_cast<const float4*>(cs + 4 * l);
        const float4 ss = *reinterpret_cast<const float4*>(cs + half + 4 * l);
        c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
        s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
      } else {
        const int at = 8 * l < half ? 8 * l : 8 * l - half;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const float4 cc = *reinterpret_cast<const float4*>(cs + at + j);
          const float4 ss = *reinterpret_cast<const float4*>(cs + half + at + j);
          c[j] = cc.x, c[j + 1] = cc.y, c[j + 2] = cc.z, c[j + 3] = cc.w;
          s[j] = ss.x, s[j + 1] = ss.y, s[j + 2] = ss.z, s[j + 3] = ss.w;
        }
        if (8 * l < half) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = -s[j];
        }
      }
    }
    const int partner = P.interleaved || !turns ? lane : 8 * l < half ? lane + half / 8 : lane - half / 8;
    int slot = -1;
    if (P.slots) {
      slot = P.slots[t];
      if (slot >= 0 && (slot >> P.kv.page_shift) >= P.kv.n_pages) {
        if (lane == 0) atomicExch(P.err, kErrSlot);
        slot = -1;
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * RPW + sub;
      const bool live = r < nrows;
      const bool isq = r < P.hq, isk = !isq && r < P.hq + P.hk;
      const int h = isq ? r : isk ? r - P.hq : r - P.hq - P.hk;
      uint4 res = raw[i];
      float x[8];
      unpack8<E>(live ? raw[i] : make_uint4(0, 0, 0, 0), x);
      const void* w = isq ? P.qw : isk ? P.kw : nullptr;
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (w) {
        float g[8];
        unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const E*>(w) + 8 * l), g);
        const float inv = rsqrtf(sq * (1.f / D) + P.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j];
      }
      if (P.rot > 0) {
        if (P.interleaved) {
          if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = x[2 * j], b = x[2 * j + 1];
              x[2 * j] = a * c[j] - b * s[j];
              x[2 * j + 1] = b * c[j] + a * s[j];
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = __shfl_sync(0xffffffffu, x[j], partner);
            if (turns) x[j] = x[j] * c[j] + y * s[j];
          }
        }
      }
      if (!live) continue;
      if (isq || isk) res = pack8<E>(x);  // values are copied bit for bit
      E* dst;
      if (isq) {
        dst = static_cast<E*>(P.q_out.ptr) + t * P.q_out.token_stride + h * P.q_out.head_stride;
      } else if (!P.slots) {
        dst = static_cast<E*>(P.k_out.ptr) + t * P.k_out.token_stride + h * P.k_out.head_stride;
      } else {
        if (slot < 0) continue;
        dst = reinterpret_cast<E*>(isk ? P.kv.k : P.kv.v) + (slot >> P.kv.page_shift) * P.kv.page_stride +
              h * P.kv.head_stride + (slot & ((1 << P.kv.page_shift) - 1)) * P.kv.token_stride;
      }
      *reinterpret_cast<uint4*>(dst + 8 * l) = res;
    }
  }
}

template <typename E, int D, int U>
cudaError_t launch_one(const RopeParams& P, cudaStream_t s) {
  constexpr int ROWS = 32 / (D / 8) * U;
  const long long units = (long long)P.T * ((P.hq + P.hk + P.hv + ROWS - 1) / ROWS);
  const long long blocks = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  rope_kernel<E, D, U><<<(unsigned)(blocks < 0x7fffffffll ? blocks : 0x7fffffffll), kRopeThreads, 0, s>>>(P);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_typed(const RopeParams& P, int d, cudaStream_t s) {
  return d == 128 ? launch_one<E, 128, 1>(P, s) : launch_one<E, 64, 1>(P, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& P, int dtype, int d, cudaStream_t s) {
  return dtype == PW_F16 ? launch_typed<__half>(P, d, s) : launch_typed<__nv_bfloat16>(P, d, s);
}

}  // namespace pw
