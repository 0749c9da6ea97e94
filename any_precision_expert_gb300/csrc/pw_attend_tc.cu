// Attention of many query rows on one key head: tcgen05 products.
//
// A prefix shared by B sequences meets B q_len G query rows a key head, and
// from about 280 rows a key byte on the products, not the loads, are the
// floor.  A CTA takes 256 rows (two 128-row tiles) of a segment past its
// 128-key tiles: S = Q K^T and O += P V are tcgen05.mma with accumulators in
// tensor memory (S of both tiles, O of both tiles: all 512 columns); P takes
// the place of S, two 16-bit weights a column, and is read from there as the
// A operand.
//
// Warps: two softmax warpgroups (one a row tile, one row a thread, so row
// maxima and sums need no exchange), a TMA producer and one MMA thread.  While
// one tile's softmax runs, the tensor cores work on the other tile:
//   PV0(n) QK0(n+1) PV1(n) QK1(n+1) PV0(n+1) ...
// O is rescaled only when a row's maximum has grown by more than 2^kGrow since
// the last time; until then the weights may reach 2^(kShift + kGrow), which
// fp16 still holds, and nothing is lost: the reference cancels in o / l.
#include <math_constants.h>

#include "pw_attend.cuh"
#include "pw_heads.cuh"
#include "pw_tc.cuh"

namespace pw {

namespace {

constexpr int kTile = 128;           // keys a tile
constexpr int kThreads = 384;
// Registers: launched with 168 a thread; the softmax warpgroups, a row of 128 scores a thread, take what the third
// warpgroup gives up (256 * 208 + 128 * 88 = 384 * 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kSegmentCost = 2;      // a segment's fixed cost, in key tiles
constexpr float kGrow = 8.f;

template <int D>
struct Cfg {
  static constexpr int NH = D / 64;
  static constexpr int HALF = kTile * 128;                 // 64-value column block of 128 rows
  static constexpr int SLOT = NH * HALF;                   // keys or values of a tile
  static constexpr int Q_AT = 0;                           // two row tiles
  static constexpr int RING_AT = 2 * SLOT;
  static constexpr int SLOTS = (226 * 1024 - RING_AT) / SLOT;
  static constexpr int BAR_AT = RING_AT + SLOTS * SLOT;
  static constexpr int PIECE_AT = BAR_AT + 16 * SLOTS + 16 * kPieces + 96;
  static constexpr int SCRATCH_AT = PIECE_AT + kPieces * (int)sizeof(Piece);
  static constexpr int SMEM = SCRATCH_AT + 144;
  static constexpr int S_COL = 0, O_COL = 256;             // tensor-memory columns: S0 S1 O0 O1, 128 each
};

using Walk = AttendWalk<kTcRows, kTile, kSegmentCost, 1>;

__device__ __forceinline__ bool active(const Piece& pc, int i) { return i == 0 || pc.row0 + 128 < pc.nrows; }

// The key tiles of a CTA's pieces as one sequence.
struct Tiles {
  Piece pc;
  int t = 0;
  bool first = false;   // first tile of its piece
  __device__ __forceinline__ bool next(PieceRing& ring) {
    first = false;
    if (++t < pc.tile1) return true;
    if (!ring.take<false>(pc)) return false;
    t = pc.tile0;
    first = true;
    return true;
  }
};

template <typename E>
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_outer) {
  const uint32_t type = __is_same(E, __half) ? 0u : 1u;
  return idesc_f16(128, n) | (type << 7) | (type << 10) | ((b_outer ? 1u : 0u) << 16);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 32 bytes: a whole sector a lane.
__device__ __forceinline__ void store8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const AttendParams P, const AttendWork W, const __grid_constant__ KvMaps maps) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t full = base + C::BAR_AT, empty = full + 8 * C::SLOTS, bars = empty + 8 * C::SLOTS + 16 * kPieces;
  // p_full: two halves (64 keys) of each row tile's weights
  const uint32_t q_full = bars, s_full = bars + 16, p_full = bars + 32, o_done = bars + 64;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::PIECE_AT - 16);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::PIECE_AT - 8);
  int* err = P.kv.err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (base & 1023) {
    if (tid == 0) atomicExch(err, kErrLayout);
    return;
  }
  PieceRing ring;
  ring.full = empty + 8 * C::SLOTS;
  ring.empty = ring.full + 8 * kPieces;
  ring.at = reinterpret_cast<Piece*>(smem + C::PIECE_AT);
  ring.abort_flag = abort_flag;
  ring.err = err;
  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(ring.full + 8 * i, 1);
      mbar_init(ring.empty + 8 * i, 9);  // eight softmax warps and the MMA thread
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 128);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(p_full + 16 + 8 * i, 128);
      mbar_init(o_done + 8 * i, 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 0) tmem_alloc((uint32_t)__cvta_generic_to_shared(tmem_at), 512);
  Walk walk;
  walk.start(P, W, reinterpret_cast<unsigned*>(smem + C::SCRATCH_AT));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: warpgroup i holds row tile i, one row a thread ----
    const int i = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + C::S_COL + i * 128, to = tmem + lanes + C::O_COL + i * 128;
    // a negative scale turns the queries around, a scale of 0 takes them away
    const uint32_t flip = P.scale < 0.f ? 0x80008000u : 0u, keep = P.scale == 0.f ? 0u : 0xffffffffu;
    const float scale2 = P.scale == 0.f ? 1.f : fabsf(P.scale) * 1.4426950408889634f;
    const uint32_t q_at = base + C::Q_AT + i * C::SLOT + r * 128;
    Piece pc = {};
    auto load_q = [&]() {
      const int row = pc.row0 + 128 * i + r;
      const bool in = row < pc.nrows;
      const int tok = in ? row / P.G : 0, hd = in ? pc.head * P.G + row - tok * P.G : 0;
      const E* src = static_cast<const E*>(P.q.ptr) + (pc.tok0 + tok) * P.q.token_stride + hd * P.q.head_stride;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint4 v = in ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0, 0, 0, 0);
        v = make_uint4((v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep, (v.w ^ flip) & keep);
        sts128(q_at + (c / 8) * C::HALF + (((c & 7) ^ (r & 7)) << 4), v);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full + 8 * i);
    };
    unsigned n = 0;     // tiles of this warpgroup so far
    unsigned flat = 0;  // tiles of the CTA so far
    bool ok = true;
    auto advance = [&]() {  // to the next piece with rows of this tile
      while (ring.take<true>(pc)) {
        if (active(pc, i)) return true;
        flat += pc.tile1 - pc.tile0;
      }
      return false;
    };
    bool have = advance();
    if (have) load_q();
    while (have && ok) {
      const Piece cur = pc;
      const int row = cur.row0 + 128 * i + r;
      const int tok = min(row, cur.nrows - 1) / P.G;
      const int vis = cur.causal ? cur.len - P.ql + 1 + tok : cur.len;  // keys this row sees
      float m = -CUDART_INF_F;
      float2 l = make_float2(0.f, 0.f);
      for (int t = cur.tile0; t < cur.tile1; ++t, ++n, ++flat) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * i, n & 1, abort_flag, err));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_load128(ts, s);
        const int see = vis - t * kTile;
        const bool edge = __any_sync(0xffffffffu, see < kTile);
        float top = -CUDART_INF_F;
        if (edge) {
          // what a row does not see counts as -infinity: a weight of 0
#pragma unroll
          for (int k = 0; k < 128; ++k) {
            if (k >= see) s[k] = 0xff800000u;
            top = fmaxf(top, __uint_as_float(s[k]));
          }
        } else {
          float t1 = -CUDART_INF_F, t2 = t1, t3 = t1;
#pragma unroll
          for (int k = 0; k < 128; k += 8) {
            top = fmaxf(fmaxf(top, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
            t1 = fmaxf(fmaxf(t1, __uint_as_float(s[k + 2])), __uint_as_float(s[k + 3]));
            t2 = fmaxf(fmaxf(t2, __uint_as_float(s[k + 4])), __uint_as_float(s[k + 5]));
            t3 = fmaxf(fmaxf(t3, __uint_as_float(s[k + 6])), __uint_as_float(s[k + 7]));
          }
          top = fmaxf(fmaxf(top, t1), fmaxf(t2, t3));
        }
        top = top == -CUDART_INF_F ? top : top * scale2 - kShift;
        if (t == cur.tile0) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kGrow)) {
          const float mm = fmaxf(m, top), f = mm == -CUDART_INF_F ? 1.f : ex2(m - mm);
          m = mm;
          l.x *= f, l.y *= f;
          ok = __all_sync(0xffffffffu, mbar_wait(o_done + 8 * i, (n - 1) & 1, abort_flag, err));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_load32(to + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_store32(to + c, o);
          }
        }
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        const float2 sc = make_float2(scale2, scale2), off = make_float2(-ref, -ref);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 64 keys: 32 columns
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const int at = 64 * h + k;
            float2 a = fma2(make_float2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), sc, off);
            a.x = ex2(a.x), a.y = ex2(a.y);
            l = add2(l, a);
            p[k / 2] = pack2<E>(a.x, a.y);
          }
          tmem_store32(ts + 32 * h, p);
          if (h == 0 && i == 0 && cur.len - t * kTile < kTile) {
            // values past the length may be anything: 0 instead (one key a thread)
            const unsigned slot = 2 * flat + 1;
            ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * (slot % C::SLOTS), (slot / C::SLOTS) & 1, abort_flag, err));
            if (!ok) break;
            if (r >= cur.len - t * kTile) {
              const uint32_t at = base + C::RING_AT + (slot % C::SLOTS) * C::SLOT + r * 128;
#pragma unroll
              for (int b = 0; b < C::NH; ++b)
#pragma unroll
                for (int c = 0; c < 8; ++c) sts128(at + b * C::HALF + 16 * c, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
          }
          tmem_store_wait();
          tc_fence_before();
          mbar_arrive(p_full + 16 * i + 8 * h);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // the last S is out of the queries' way: the next piece's queries go in before this one's sums come out
      have = advance();
      if (have) load_q();
      ok = __all_sync(0xffffffffu, mbar_wait(o_done + 8 * i, (n - 1) & 1, abort_flag, err));
      if (!ok) break;
      tc_fence_after();
      const AttendPieces& dst = cur.prefix ? W.prefix : W.suffix;
      const bool in = row < cur.nrows;
      const long long grow = (long long)(cur.tok0 + tok) * P.kv.hq + cur.head * P.G + row - tok * P.G;
      const long long crow = (long long)blockIdx.x * kTcRows + 128 * i + r;
      float* out = cur.first ? dst.row_o + grow * D : dst.cta_o + crow * D;
      if (in) {
        if (cur.first)
          dst.row_ml[grow] = make_float4(m, l.x + l.y, __int_as_float((int)blockIdx.x), __int_as_float(cur.last_cta));
        else
          dst.cta_ml[crow] = make_float2(m, l.x + l.y);
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_load32(to + c, o);
        if (in) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) store8(out + c + k, o + k);
        }
      }
      tc_fence_before();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---- producer: keys and values of a tile take one ring slot each; one lane a page ----
      const int shift = P.kv.page_shift, box = min(1 << shift, kBoxTokens);
      unsigned x = 0;  // slots filled so far
      bool ok = true;
      Piece pc;
      const int* table;
      while (ok) {
        const bool more = walk.next(P, pc, table);
        ok = __all_sync(0xffffffffu, lane != 0 || ring.put(pc));
        if (!more) break;
        for (int t = pc.tile0; ok && t < pc.tile1; ++t) {
          const int keys = min(kTile, pc.len - t * kTile), boxes = (keys + box - 1) / box;
          const int at = t * kTile + lane * box, tok = at & ((1 << shift) - 1);
          int page = 0;
          if (lane < boxes) {
            page = table[at >> shift];
            if (page < 0 || page >= P.kv.n_pages) atomicExch(err, kErrPage);  // reads as zeros
          }
          for (int v = 0; v < 2; ++v, ++x) {
            const unsigned slot = x % C::SLOTS, round = x / C::SLOTS;
            ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, (round & 1) ^ 1, abort_flag, err));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full + 8 * slot, (uint32_t)(boxes * box * D * 2));
            __syncwarp();
            if (lane < boxes) {
              const uint32_t dst = base + C::RING_AT + slot * C::SLOT + lane * box * 128;
  #pragma unroll
              for (int h = 0; h < C::NH; ++h)
                tma_load_page(dst + h * C::HALF, v ? &maps.v : &maps.k, 64 * h, tok, pc.head, page, full + 8 * slot);
            }
            __syncwarp();
          }
        }
      }
      // copies in flight land before the shared memory goes away (after a normal end all have)
      for (int i = 0; i < C::SLOTS; ++i) {
        const unsigned fills = (x + C::SLOTS - 1 - i) / C::SLOTS;
        for (int k = 0; fills > 0 && k < (1 << 16) && !mbar_try_wait(full + 8 * i, (fills - 1) & 1); ++k) {
        }
      }
    } else if (warp == 9) {
      if (lane == 0) {
        // ---- MMA ----
        constexpr uint32_t id_qk = idesc_of<E>(kTile, false), id_pv = idesc_of<E>(D, true);
        unsigned qn[2] = {0, 0}, pn[2] = {0, 0};  // phases of q_full and p_full waited for so far
        unsigned x = 0;                           // tiles whose keys have been multiplied
        bool ok = true;
        Tiles it;
        it.pc.tile1 = 0;
        auto landed = [&](unsigned s) {
          return mbar_wait(full + 8 * (s % C::SLOTS), (s / C::SLOTS) & 1, abort_flag, err);
        };
        auto qk = [&](int i, unsigned tile) {     // S_i = Q_i K^T
          const uint64_t q = sw128_desc(base + C::Q_AT + i * C::SLOT);
          const uint64_t k = sw128_desc(base + C::RING_AT + (2 * tile % C::SLOTS) * C::SLOT);
  #pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t at = (c / 4) * (C::HALF >> 4) + 2 * (c % 4);
            umma_f16(tmem + C::S_COL + i * 128, q + at, k + at, id_qk, c != 0);
          }
          umma_commit(s_full + 8 * i);
        };
        auto pv = [&](int i, unsigned tile, bool first) {  // O_i (+)= P_i V, as the halves of P come
          const uint64_t v = sw128_desc_outer(base + C::RING_AT + ((2 * tile + 1) % C::SLOTS) * C::SLOT, C::HALF);
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(p_full + 16 * i + 8 * h, pn[i] & 1, abort_flag, err)) return false;
            if (h == 0 && i == 0 && !landed(2 * tile + 1)) return false;
            tc_fence_after();
  #pragma unroll
            for (int c = 0; c < 4; ++c)
              umma_ts(tmem + C::O_COL + i * 128, tmem + C::S_COL + i * 128 + 32 * h + 8 * c, v + 512 * h + 128 * c, id_pv,
                      !first || h + c != 0);
          }
          ++pn[i];
          umma_commit(o_done + 8 * i);
          return true;
        };
        bool have = it.next(ring);
        if (have) {
          for (int i = 0; i < 2 && ok; ++i) {
            if (!active(it.pc, i)) continue;
            ok = mbar_wait(q_full + 8 * i, qn[i]++ & 1, abort_flag, err) && landed(0);
            tc_fence_after();
            if (ok) qk(i, 0);
          }
          umma_commit(empty);
        }
        while (ok && have) {
          const bool second = active(it.pc, 1), first = it.first;
          const unsigned tile = x++;
          have = it.next(ring);
          for (int i = 0; i < 2 && ok; ++i) {
            if (i == 0 || second) ok = pv(i, tile, first);
            if (ok && have && active(it.pc, i)) {
              if (it.first) ok = mbar_wait(q_full + 8 * i, qn[i]++ & 1, abort_flag, err);
              ok = ok && (i > 0 || landed(2 * x));
              tc_fence_after();
              if (ok) qk(i, x);
            }
          }
          umma_commit(empty + 8 * ((2 * tile + 1) % C::SLOTS));
          if (have) umma_commit(empty + 8 * (2 * x % C::SLOTS));
        }
      }
      __syncwarp();
    }
  }
  // ---- teardown: every MMA has completed or the wait for it has run out ----
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && warp == 9 && lane == 0) {
    umma_commit(q_full);  // arrives when the products issued so far are done
    const long long t0 = clock64();
    while (clock64() - t0 < 1000000) {
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

template <typename E, int D>
cudaError_t launch_typed(const AttendParams& P, const AttendWork& W, const KvMaps& maps, int ctas, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(attend_tc_kernel<E, D>);
  cudaError_t e = ensure_smem(fn, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  attend_tc_kernel<E, D><<<ctas, kThreads, Cfg<D>::SMEM, s>>>(P, W, maps);
  return cudaGetLastError();
}

}  // namespace

int attend_tc_ctas() { return sm_count(); }

cudaError_t launch_attend_tc(const AttendParams& P, const AttendWork& W, const KvMaps& maps, int ctas, cudaStream_t s) {
  if (P.kv.dtype == PW_F16)
    return P.kv.d == 128 ? launch_typed<__half, 128>(P, W, maps, ctas, s) : launch_typed<__half, 64>(P, W, maps, ctas, s);
  return P.kv.d == 128 ? launch_typed<__nv_bfloat16, 128>(P, W, maps, ctas, s)
                       : launch_typed<__nv_bfloat16, 64>(P, W, maps, ctas, s);
}

}  // namespace pw
