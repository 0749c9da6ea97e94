// Attention of many query rows on one key head: tcgen05 products.
//
// A prefix shared by B sequences meets B q_len G query rows a key head, and
// from about 280 rows a key byte on the products, not the loads, are the
// floor.  A CTA takes 256 rows (two 128-row tiles) of a segment past its
// 128-key tiles: S = Q K^T and O += P V are tcgen05.mma with accumulators in
// tensor memory (S of both tiles, O of both tiles: all 512 columns); P takes
// the place of S, two 16-bit weights a column, and is read from there as the
// A operand, which leaves shared memory to K, V and Q.
//
// Warps: a softmax warpgroup a row tile (one row a thread, so row maxima and
// sums need no exchange), a TMA producer and one MMA warp a row tile.  While
// one tile's softmax runs, the tensor cores work on the other:
//   PV0(n) QK0(n+1) | PV1(n) QK1(n+1) | PV0(n+1) ...
// O is rescaled only when a row's maximum has grown by more than 2^kGrow since
// the last time; until then the weights may reach 2^(kShift + kGrow), which
// fp16 still holds, and nothing is lost: the reference cancels in o / l.
//
// Measured (heads of 128, 1.9 GHz): 2850-2950 cycles a tile pair whose MMAs
// take 2048, so 70% of their rate once it runs; what is left is the chain
// scores -> softmax (1.2-1.4 k cycles) -> weights -> products of one row tile,
// as P and S share their columns.  256 sequences of 4 rows a head on 32768
// keys: 98-104 us, 1320-1400 TFLOP/s, of which 6 us pass before a CTA's first scores
// and 3 after its last.  Tried: one MMA warp for both row tiles 3600 cycles,
// half a row a softmax thread 3070-3250, weights in 4 parts 3190, in one part
// 3010, the warpgroups not in turns 3450-4030, the first half's weights taken
// before the tile's maximum is known 3720, a branch for the scale's sign in
// every tile 3150.
#include <math_constants.h>

#include "pw_attend.cuh"
#include "pw_heads.cuh"
#include "pw_tc.cuh"

namespace pw {

namespace {

constexpr int kTile = 128;           // keys a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
// Registers: launched with 168 a thread; the softmax warps, a row of 128 scores a thread, take what the other four give
// up (256 * 208 + 128 * 88 = 384 * 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kParts = 2;            // a tile's weights are handed over in halves: P V starts on the first
constexpr int kSegmentCost = 2;      // a segment's fixed cost, in key tiles
// Tiles a CTA takes at least: fewer CTAs leave SMs to the streaming kernel and write fewer partial sums, more share the
// work (the call with 2 / 3 / 6 / 10: 24 sequences of 20 rows behind 8191 tokens 52.2 / 52.1 / 52.1 / 59.7 us, four groups
// of 132 rows behind up to 6000 25.7 / 25.7 / 28.0 / 33.0).
constexpr int kLeastUnits = 3;
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
  static constexpr int PIECE_AT = BAR_AT + 16 * SLOTS + 16 * kPieces + 192;
  static constexpr int SCRATCH_AT = PIECE_AT + kPieces * (int)sizeof(Piece);
  static constexpr int SMEM = SCRATCH_AT + 144;
  static constexpr int S_COL = 0, O_COL = 256;             // tensor-memory columns: S0 S1 O0 O1, 128 each
};

using Walk = AttendWalk<kTcRows, kTile, kSegmentCost, 1, kLeastUnits>;

__device__ __forceinline__ bool active(const Piece& pc, int i) { return i == 0 || pc.row0 + 128 < pc.nrows; }

// The key tiles of a CTA's pieces as one sequence.
struct Tiles {
  Piece pc;
  int t = 0;
  bool first = false;   // first tile of its piece
  __device__ __forceinline__ bool next(PieceRing& ring) {
    first = false;
    if (++t < pc.tile1) return true;
    if (!ring.take(pc)) return false;
    t = pc.tile0;
    first = true;
    return true;
  }
};

// The MMA warp of row tile I.  One warp a row tile, so that neither tile waits for the other's weights and the cost of
// issuing is shared (an instruction of 128 x 128 x 16 takes the tensor cores 64 cycles, about what issuing one takes).
// The whole warp walks, one lane issues: what the instructions take is then the same in every lane.
template <typename E, int D, int I>
__device__ __forceinline__ void mma_role(PieceRing ring, uint32_t base, uint32_t full, uint32_t empty, uint32_t bars,
                                         uint32_t tmem, volatile int* abort_flag, int* err) {
  using C = Cfg<D>;
  constexpr uint32_t id_qk = idesc_of<E>(kTile, false), id_pv = idesc_of<E>(D, true);
  const uint32_t q_full = bars + 8 * I, s_full = bars + 16 + 8 * I, o_done = bars + 32 + 8 * I,
                 p_full = bars + 64 + 8 * kParts * I;
  const uint32_t ts = tmem + C::S_COL + I * 128, to = tmem + C::O_COL + I * 128;
  const uint64_t q = sw128_desc(base + C::Q_AT + I * C::SLOT), k0 = sw128_desc(base + C::RING_AT);
  const uint64_t v0 = sw128_desc_outer(base + C::RING_AT, C::HALF);
  const uint32_t q_lo = (uint32_t)q, k_hi = (uint32_t)(k0 >> 32), v_hi = (uint32_t)(v0 >> 32);
  const bool leader = elect_one();
  unsigned qn = 0, pn = 0;     // phases of q_full and p_full waited for so far
  unsigned slot = 0, par = 0;  // ring slot of the next keys or values, and its phase
  Tiles it;
  it.pc.tile1 = 0;
  auto wait = [&](uint32_t bar, unsigned parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, abort_flag, err)) != 0;
  };
  bool have = it.next(ring), act = false, first = false;
  unsigned vs = 0, vp = 0;     // the current tile's values
  bool run = false;            // a tile is waiting for its weights
  while (have || run) {
    const bool k_act = have && active(it.pc, I);
    const unsigned ks = slot, kp = par;
    if (have) {
      if (++slot == C::SLOTS) slot = 0, par ^= 1;
      if (!wait(full + 8 * ks, kp)) return;   // also of keys that this tile has no use for: an arrival belongs to their phase
    }
    if (run) {
      if (!wait(full + 8 * vs, vp)) return;
      if (act) {  // O (+)= P V
        const uint32_t v_lo = (uint32_t)v0 + vs * (C::SLOT >> 4);
#pragma unroll
        for (int h = 0; h < kParts; ++h) {  // as the parts of P come
          if (!wait(p_full + 8 * h, pn)) return;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int c = 8 / kParts * h; c < 8 / kParts * (h + 1); ++c)
              umma_ts_lo(to, ts + 8 * c, v_lo + 128 * c, v_hi, id_pv, c > 0 || !first);
          }
          __syncwarp();
        }
        ++pn;
      }
    }
    // a piece's queries come once the sums of the one before are out, so not before its last product is issued
    if (run && act && (!have || it.first)) {
      if (leader) umma_commit(o_done);
      __syncwarp();
    }
    if (k_act && it.first && !wait(q_full, qn++)) return;
    tc_fence_after();
    if (leader) {
      if (k_act) {  // S = Q K^T; in order behind the product that reads the weights in its place
        const uint32_t k_lo = (uint32_t)k0 + ks * (C::SLOT >> 4);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t step = (c / 4) * (C::HALF >> 4) + 2 * (c % 4);
          umma_f16_lo(ts, q_lo + step, k_hi, k_lo + step, k_hi, id_qk, c != 0);
        }
        umma_commit(s_full);
      }
      if (run) umma_commit(empty + 8 * vs);
      if (have) umma_commit(empty + 8 * ks);
    }
    __syncwarp();
    run = have;
    act = k_act;
    first = it.first;
    if (have) {
      vs = slot, vp = par;
      if (++slot == C::SLOTS) slot = 0, par ^= 1;
      have = it.next(ring);
    }
  }
}

// Adds to 32 of a row's sums the values that are no numbers, of the piece's keys from lo on that the row sees.
template <typename E>
__device__ __forceinline__ void add_odd(const AttendParams& P, const Piece& pc, int lo, int vis, int col, uint32_t (&o)[32]) {
  const int* table = P.table + (long long)(pc.item - P.n_groups) * P.table_stride;
#pragma unroll 1
  for (int t = pc.tile0; t < pc.tile1; ++t) {
    const int at = key_tile<kTile>(pc, t) * kTile;
#pragma unroll 1
    for (int key = max(max(lo, 0), at); key < min(vis, at + kTile); ++key) {
      const int page = table[key >> P.kv.page_shift];
      if (page < 0 || page >= P.kv.n_pages) continue;
      const E* src = reinterpret_cast<const E*>(P.kv.v) + page * P.kv.page_stride + pc.head * P.kv.head_stride +
                     (key & ((1 << P.kv.page_shift) - 1)) * P.kv.token_stride + col;
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        float x[8];
        unpack8<E>(*reinterpret_cast<const uint4*>(src + c), x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!isfinite(x[k])) o[c + k] = __float_as_uint(__uint_as_float(o[c + k]) + x[k]);
      }
    }
  }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const AttendParams P, const AttendWork W, const __grid_constant__ KvMaps maps) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t full = base + C::BAR_AT, empty = full + 8 * C::SLOTS, bars = empty + 8 * C::SLOTS + 16 * kPieces;
  const uint32_t q_full = bars, s_full = bars + 16, o_done = bars + 32, turn = bars + 48, p_full = bars + 64;  // p_full: [row tile][part]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::PIECE_AT - 16);
  volatile int* odd_seen = reinterpret_cast<volatile int*>(smem + C::PIECE_AT - 12);  // values that are no numbers were taken out
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::PIECE_AT - 8);
  int* err = P.kv.err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (base & 1023) {
    if (tid == 0) atomicExch(err, kErrLayout);
    return;
  }
  behind_the_stream();
  let_next_start();
  const Walk::Mine mine = Walk::mine(P, W);
  PieceRing ring;
  ring.full = empty + 8 * C::SLOTS;
  ring.empty = ring.full + 8 * kPieces;
  ring.at = reinterpret_cast<Piece*>(smem + C::PIECE_AT);
  ring.abort_flag = abort_flag;
  ring.err = err;
  {
    // the barriers lie side by side, one thread each: ring slots (full, empty), pieces (full, empty), then by row tile
    // queries, scores, sums, turns and the parts of the weights
    constexpr int kNear = 2 * C::SLOTS + 2 * kPieces, kAll = kNear + 8 + 2 * kParts;
    if (tid < kAll) {
      const int k = tid - kNear;
      const int count = tid < C::SLOTS ? 1 : tid < 2 * C::SLOTS ? 2 : tid < 2 * C::SLOTS + kPieces ? 1
                        : k < 0 ? kSoftmaxWarps + 2 : k < 2 ? 128 : k < 6 ? 1 : 128;
      mbar_init(full + 8 * tid, count);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) *abort_flag = *odd_seen = 0;
  }
  if (warp == kSoftmaxWarps + 3) tmem_alloc((uint32_t)__cvta_generic_to_shared(tmem_at), 512);
  Walk walk;
  walk.start(P, W, mine, reinterpret_cast<unsigned*>(smem + C::SCRATCH_AT));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: warpgroup i holds row tile i, one row a thread ----
    const int i = warp >> 2, w4 = warp & 3, r = tid & 127;
    const uint32_t lanes = (uint32_t)w4 << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + C::S_COL + i * 128, to = tmem + lanes + C::O_COL + i * 128;
    const bool plain_q = P.scale > 0.f;  // a negative scale turns the queries around, a scale of 0 takes them away
    const float scale2 = P.scale == 0.f ? 1.f : fabsf(P.scale) * 1.4426950408889634f;
    Piece pc = {};
    // Queries: a warp brings its 32 rows, whole lines at a time.
    constexpr int LPR = D / 8, RPS = 32 / LPR, STEPS = 32 / RPS;  // lanes a row, rows a step, steps
    const int q_row = 32 * w4, q_sub = lane / LPR, q_col = lane % LPR;
    const uint32_t q_base = base + C::Q_AT + i * C::SLOT;
    // The lane's rows, RPS apart: f(k, source or null past the rows).
    auto each_row = [&](auto f) {
      const int row0 = pc.row0 + 128 * i + q_row + q_sub, tok = row0 / P.G;
      int hd = row0 - tok * P.G, left = pc.nrows - row0;
      const E* src = static_cast<const E*>(P.q.ptr) + (pc.tok0 + tok) * P.q.token_stride +
                     (pc.head * P.G + hd) * P.q.head_stride + 8 * q_col;
      const long long turn_over = P.q.token_stride - P.G * P.q.head_stride;
#pragma unroll 4
      for (int k = 0; k < STEPS; ++k) {
        f(k, left > 0 ? src : nullptr);
        left -= RPS;
        hd += RPS;
        src += RPS * P.q.head_stride;
        while (hd >= P.G) hd -= P.G, src += turn_over;
      }
    };
    auto place_q = [&]() {
      each_row([&](int k, const E* src) {
        const int at = q_row + k * RPS + q_sub;
        const uint32_t dst = q_base + (q_col / 8) * C::HALF + at * 128 + (((q_col & 7) ^ (at & 7)) << 4);
        if (src && plain_q) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        } else {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (src && P.scale < 0.f) {
            v = *reinterpret_cast<const uint4*>(src);
            v = make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
          }
          sts128(dst, v);
        }
      });
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(q_full + 8 * i);
    };
    unsigned n = 0;     // tiles of this row tile so far
    unsigned flat = 0;  // tiles of the CTA so far
    unsigned turns = 0, done = 0;  // turns taken, pieces finished
    bool ok = true;
    auto advance = [&]() {  // to the next piece with rows of this tile
      while (ring.take(pc)) {
        if (active(pc, i)) return true;
        flat += pc.tile1 - pc.tile0;
      }
      return false;
    };
    bool have = advance();
    if (have) place_q();
    while (have && ok) {
      const Piece cur = pc;
      const int row = cur.row0 + 128 * i + r;
      const int tok = min(row, cur.nrows - 1) / P.G;
      const int vis = cur.causal ? cur.len - P.ql + 1 + tok : cur.len;  // keys this row sees
      const int sure = cur.causal ? cur.len - P.ql + 1 : cur.len;  // keys that every row sees
      const bool both = active(cur, 1);
      float m = -CUDART_INF_F;
      float2 l = make_float2(0.f, 0.f);
      const int key_tiles = (cur.len + kTile - 1) / kTile;
      int kt = key_tile<kTile>(cur, cur.tile0);
      for (int t = cur.tile0; t < cur.tile1; ++t, ++n, ++flat, kt = kt + 1 == key_tiles ? 0 : kt + 1) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * i, n & 1, abort_flag, err));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_load128(ts, s);
        if (both) {  // the warpgroups take turns, so that one's softmax meets the other's products
          ok = __all_sync(0xffffffffu, mbar_wait(turn + 8 * i, (turns & 1) ^ (i ^ 1), abort_flag, err));
          if (!ok) break;
          ++turns;
        }
        const int see = vis - kt * kTile;
        float top = -CUDART_INF_F;
        if ((kt + 1) * kTile > sure) {
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
            top = max3(top, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
            t1 = max3(t1, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
            t2 = max3(t2, __uint_as_float(s[k + 4]), __uint_as_float(s[k + 5]));
            t3 = max3(t3, __uint_as_float(s[k + 6]), __uint_as_float(s[k + 7]));
          }
          top = fmaxf(max3(top, t1, t2), t3);
        }
        top = top == -CUDART_INF_F ? top : top * scale2 - kShift;
        if (t == cur.tile0) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kGrow)) {
          const float mm = fmaxf(m, top), f = mm == -CUDART_INF_F ? 1.f : ex2(m - mm);
          m = mm;
          l.x *= f, l.y *= f;
          // these scores were issued behind the last product into O: it is done
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_load16(to + c, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_store16(to + c, o);
          }
        }
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        const float2 sc = make_float2(scale2, scale2), off = make_float2(-ref, -ref);
        if (i == 0 && (kt + 1) * kTile > sure) {
          // values past the length may be anything: 0 instead (one key a thread; the other row tile's turn comes after
          // this); so for those that are no numbers and that some rows do not see, which the others get at the end
          const unsigned slot = 2 * flat + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * (slot % C::SLOTS), (slot / C::SLOTS) & 1, abort_flag, err));
          if (!ok) break;
          const uint32_t at = base + C::RING_AT + (slot % C::SLOTS) * C::SLOT + r * 128;
          const int key = kt * kTile + r;
          if (key >= sure && key < cur.len) {
#pragma unroll 1
            for (int c = 0; c < 8 * C::NH; ++c) {
              const uint32_t to = at + (c >> 3) * C::HALF + 16 * (c & 7);
              const uint4 v = shared16(to);
              if (!all_finite<E>(v)) {
                sts128(to, make_uint4(v.x & finite_bits<E>(v.x), v.y & finite_bits<E>(v.y), v.z & finite_bits<E>(v.z),
                                      v.w & finite_bits<E>(v.w)));
                *odd_seen = 1;
              }
            }
          }
          if (key >= cur.len) {
#pragma unroll
            for (int b = 0; b < C::NH; ++b)
#pragma unroll
              for (int c = 0; c < 8; ++c) sts128(at + b * C::HALF + 16 * c, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          constexpr int N = kTile / kParts;  // keys of a part, two a column
          uint32_t p[N / 2];
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const int at = N * h + k;
            float2 a = fma2(make_float2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), sc, off);
            a.x = ex2(a.x), a.y = ex2(a.y);
            l = add2(l, a);
            p[k / 2] = pack2<E>(a.x, a.y);
          }
#pragma unroll
          for (int k = 0; k < N / 2; k += 16) tmem_store16(ts + N / 2 * h + k, p + k);
          tmem_store_wait();
          tc_fence_before();
          mbar_arrive(p_full + 8 * (kParts * i + h));
          if (h == 0 && both) mbar_arrive(turn + 8 * (i ^ 1));
        }
      }
      if (!ok) break;
      // the last S is out of the queries' way: the next piece's go in before this one's sums come out
      have = advance();
      if (have) place_q();
      ok = __all_sync(0xffffffffu, mbar_wait(o_done + 8 * i, done++ & 1, abort_flag, err));
      if (!ok) break;
      tc_fence_after();
      // the wait is over already: it makes what any thread of the first row tile has seen known here
      const bool odd = sure < cur.len && mbar_wait(p_full + 8 * (kParts * i + kParts - 1), (n - 1) & 1, abort_flag, err) && *odd_seen;
      const AttendPieces& dst = cur.prefix ? W.prefix : W.suffix;
      const bool in = row < cur.nrows;
      const long long grow = (long long)(cur.tok0 + tok) * P.kv.hq + cur.head * P.G + row - tok * P.G;
      const int crow = blockIdx.x * kTcRows + 128 * i + r;
      if (in) {
        const float sum = l.x + l.y;
        if (cur.first)
          dst.row_ml[grow] = make_float4(m, sum, __int_as_float((int)blockIdx.x), __int_as_float(cur.last_cta));
        else
          dst.cta_ml[crow] = make_float2(m, sum);
      }
      // blocks of 8-value columns; a suffix's first pieces, which would leave most of a block empty, in plain rows
      const bool plain = cur.first && !cur.prefix;
      const int column = plain ? 8 : kTcRows * 8;
      float* out = plain       ? dst.row_o + grow * D
                   : cur.first ? dst.row_o + tc_block(cur.tok0, P.G, cur.item, cur.row0 / kTcRows, P.kv.hkv, cur.head) * kTcRows * D +
                                     (128 * i + r) * 8
                               : dst.cta_o + (long long)blockIdx.x * kTcRows * D + (128 * i + r) * 8;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_load32(to + c, o);
        if (odd && in) add_odd<E>(P, cur, sure, vis, c, o);
        if (in) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) store8(out + (c + k) / 8 * column, o + k);
        }
      }
      tc_fence_before();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps) {
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
          const int kt = key_tile<kTile>(pc, t);
          const int keys = min(kTile, pc.len - kt * kTile), boxes = (keys + box - 1) / box;
          const int at = kt * kTile + lane * box, tok = at & ((1 << shift) - 1);
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
    } else if (warp == kSoftmaxWarps + 1) {
      mma_role<E, D, 0>(ring, base, full, empty, bars, tmem, abort_flag, err);
    } else if (warp == kSoftmaxWarps + 2) {
      mma_role<E, D, 1>(ring, base, full, empty, bars, tmem, abort_flag, err);
    }
  }
  // ---- teardown: every MMA has completed or the wait for it has run out ----
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {  // products issued before the wait ran out end well within this time
    const long long t0 = clock64();
    while (clock64() - t0 < 1000000) {
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftmaxWarps + 3) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

template <typename E, int D>
cudaError_t launch_typed(const AttendParams& P, const AttendWork& W, const KvMaps& maps, int ctas, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(attend_tc_kernel<E, D>);
  cudaError_t e = ensure_smem(fn, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const Launch at(dim3(ctas), kThreads, Cfg<D>::SMEM, s);
  return cudaLaunchKernelEx(&at.cfg, attend_tc_kernel<E, D>, P, W, maps);
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
