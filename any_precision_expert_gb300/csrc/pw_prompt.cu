// Causal attention of packed prompts over their own keys: tcgen05 products.
//
// The G heads that share keys lie side by side: row r of a row tile is token r /
// G, head r % G, and a row tile holds the floor(128 / G) whole tokens that fit
// its 128 rows, so that one tensor copy brings its queries and it ends within
// 128 / G keys of its diagonal.  A CTA takes two row tiles past the 128-key
// tiles that they see, as attend_tc_kernel does (pw_attend_tc.cu, which explains
// the parts): S = Q K^T and O += P V with accumulators in tensor memory, P in
// the place of S, a softmax warpgroup and an MMA warp a row tile.  Nothing is
// split: a row's keys stay in one CTA, and its sums are divided and rounded on
// their way out.
//
// Values at keys that only some rows see would bring an infinity or NaN into
// the others' sums (0 times it): a warp looks the tiles on the diagonal through
// before they go to the products, takes such values out and the rows that see
// them get them back at the end.
//
// Weights are one number of the heads' type each, which the product wants: two,
// as the 4-bit kernel takes, would double that product, half of what bounds
// heads of 128.  Their rounding makes the errors 1.2 to 1.35 times those of
// rounding the output alone.
//
// Measured: one sequence of 8191 tokens, 32 heads of 128 on 8, 379 to 413 us as
// the SM clock goes (1450 to 1330 TFLOP/s of what its rows see): 2750 cycles a
// tile pair, whose MMAs take 2048, and some 6 k cycles a piece for its first
// scores, last sums and their way out.  24 sequences of up to 1111 tokens, 44
// heads of 64 on 4: 147 us; there a piece has 3.4 key tiles on average, so those
// times are half of it, and no pipe is full (tensor 25 %, exponentials 25 %, 1.5
// instructions a cycle).
//
// Work grows with a tile's place in its sequence, so the CTAs take the tiles by
// falling place (a counting sort over the sequences' lengths, which every CTA
// does for itself), to and fro: CTA c takes c, 2 P - 1 - c, 2 P + c, ...
#include <cuda.h>
#include <math_constants.h>

#include "pw_attend.cuh"
#include "pw_heads.cuh"
#include "pw_tc.cuh"

namespace pw {

namespace {

constexpr int kTile = 128;           // keys a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
// Registers: launched with 168 a thread; the softmax warps take what the other four give up (256 * 216 + 128 * 72 = 384 * 168;
// with 208 and 88 a document of 8191 tokens took 1 % longer).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
// Parts in which a tile's weights are handed over: with 2 / 4 the document took 4 / 17 % longer, 24 prompts 6 / 19 %.
constexpr int kParts = 1;
constexpr float kGrow = 8.f;         // sums are rescaled when a row's maximum has grown by 2^kGrow
constexpr int kBuckets = 512;
// The softmax of heads of 128 meets the other row tile's products if the warpgroups take turns; with heads of 64, whose
// products are half as long, the two do better side by side (24 prompts of up to 1111 tokens took 15 % longer with turns, a
// document with heads of 128 19 % longer without).
template <int D>
constexpr bool kTurns = D == 128;

template <int D>
struct Cfg {
  static constexpr int NH = D / 64;
  static constexpr int HALF = kTile * 128;                 // 64-value column block of 128 rows
  static constexpr int SLOT = NH * HALF;                   // keys or values of a tile
  static constexpr int Q_AT = 0;                           // two row tiles
  static constexpr int RING_AT = 2 * SLOT;
  static constexpr int SORT = (3 * kBuckets + 4) * 4;
  static constexpr int FIT = (226 * 1024 - RING_AT - SORT - 1024) / SLOT;
  static constexpr int SLOTS = FIT < 8 ? FIT / 2 * 2 : 8;  // even: keys, then values
  static constexpr int BAR_AT = RING_AT + SLOTS * SLOT;
  static constexpr int PIECE_AT = BAR_AT + 16 * SLOTS + 16 * kPieces + 192;
  static constexpr int SORT_AT = PIECE_AT + kPieces * (int)sizeof(Piece);
  static constexpr int SMEM = SORT_AT + SORT;
  static constexpr int S_COL = 0, O_COL = 256;             // tensor-memory columns: S0 S1 O0 O1, 128 each
};

struct PromptMaps {
  CUtensorMap q, k, v;
};

__device__ int prompt_err;  // the error word of calls without one, read by pw_prompt_check_device

// Tokens of a sequence, inside the call's.
struct Span {
  int lo, n;
};
__device__ __forceinline__ Span span_of(const PromptParams& P, int b, int* err) {
  const int lo = P.offsets[b], hi = P.offsets[b + 1];
  const int l = min(max(lo, 0), P.T), h = min(max(hi, l), P.T);
  if (err && (l != lo || h != hi)) atomicExch(err, kErrOffsets);
  return {l, h - l};
}
// Tokens of a row tile, and a sequence's tiles of two of them.
__host__ __device__ __forceinline__ int tile_tokens(const PromptParams& P) { return 128 / P.G; }
__host__ __device__ __forceinline__ int row_tiles(const PromptParams& P, int n) {
  return (n + 2 * tile_tokens(P) - 1) / (2 * tile_tokens(P));
}

// Row tiles in falling order of their place in the sequence.  Places are sorted into buckets of 2^shift.
struct PromptWalk {
  int* full;    // [kBuckets] sequences whose last, partial bucket this is; then what they hold of it
  int* rest;
  int* start;   // [kBuckets] row tiles in the buckets above; [kBuckets]: all row tiles
  int shift, turn, bucket, b0, before;

  __device__ __forceinline__ unsigned& held() { return reinterpret_cast<unsigned*>(start)[kBuckets + 1]; }  // tokens of all sequences
  __device__ __forceinline__ void clear(int tid) {
    for (int i = tid; i < kBuckets; i += kThreads) full[i] = rest[i] = 0;
    if (tid == 0) held() = 0;
  }
  __device__ __forceinline__ void count(const PromptParams& P, int tid, int* err) {
    int tokens = 0;  // of this thread's sequences, at most 11 of 2^20
    for (int b = tid; b < P.B; b += kThreads) {
      const Span s = span_of(P, b, blockIdx.x == 0 ? err : nullptr);
      const int tiles = row_tiles(P, s.n);
      tokens += s.n;
      if (tiles > 0) {
        atomicAdd(&full[tiles >> shift], 1);
        atomicAdd(&rest[tiles >> shift], tiles & ((1 << shift) - 1));
      }
    }
    if (tokens > 0) atomicAdd(&held(), (unsigned)min(tokens, P.T + 1));  // kThreads of them stay below 2^32
  }
  // Sequences that hold more than the call's tokens overlap: descending offsets could ask for 4096 times a call's work,
  // more row tiles than the ranks count in 32 bits.  Nothing of such a call runs.
  __device__ __forceinline__ bool overlap(const PromptParams& P) { return held() > (unsigned)P.T; }
  // One warp; lane 0 holds the highest buckets.
  __device__ __forceinline__ void sort(const PromptParams& P, int lane) {
    if (overlap(P)) {
      for (int i = lane; i <= kBuckets; i += 32) start[i] = 0;
      return;
    }
    constexpr int PER = kBuckets / 32;
    auto scan = [&](int sum) {  // what the lanes before this one hold
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      return x - sum;
    };
    const int top = kBuckets - 1 - lane * PER;
    int sum = 0;
    for (int i = 0; i < PER; ++i) sum += full[top - i];
    const int above = scan(sum);  // sequences that reach past this lane's buckets
    int a = above;
    sum = 0;
    for (int i = 0; i < PER; ++i) {
      sum += (a << shift) + rest[top - i];
      a += full[top - i];
    }
    int at = scan(sum);
    a = above;
    for (int i = 0; i < PER; ++i) {
      start[top - i] = at;
      at += (a << shift) + rest[top - i];
      a += full[top - i];
    }
    if (lane == 31) start[kBuckets] = at;
  }
  __device__ __forceinline__ void begin() { turn = 0, bucket = -1, b0 = before = 0; }

  // One warp: the CTA's next row tile; false (and a piece without tiles) at the end.
  __device__ __forceinline__ bool next(const PromptParams& P, Piece& p, int lane) {
    p.tile1 = 0;
    const unsigned grid = gridDim.x;
    const unsigned rank = turn * grid + ((turn & 1) ? grid - 1 - blockIdx.x : blockIdx.x);
    ++turn;
    const int unit = rank / P.hkv;
    if (unit >= start[kBuckets]) return false;
    int lo = 0, hi = kBuckets - 1;  // the lowest bucket that does not begin behind the tile
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= unit) hi = mid;
      else lo = mid + 1;
    }
    if (lo != bucket) bucket = lo, b0 = before = 0;
    const int want = unit - start[bucket], first = bucket << shift;
#pragma unroll 1
    for (; b0 < P.B; b0 += 32) {
      const int b = b0 + lane;
      Span s = {0, 0};
      if (b < P.B) s = span_of(P, b, nullptr);
      const int mine = min(max(row_tiles(P, s.n) - first, 0), 1 << shift);
      int scan = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + scan > want);
      if (hit) {
        const int at = __ffs(hit) - 1;
        const int tile = first + want - before - __shfl_sync(0xffffffffu, scan - mine, at);
        p.tok0 = __shfl_sync(0xffffffffu, s.lo, at);
        p.nrows = __shfl_sync(0xffffffffu, s.n, at);         // tokens here
        p.head = rank - unit * P.hkv;
        const int tokens = tile_tokens(P);
        p.row0 = tile * 2 * tokens;                          // the first row tile's first token
        // the keys that each of the two row tiles sees, in tiles
        p.tile0 = (min(p.row0 + tokens, p.nrows) + kTile - 1) / kTile;
        p.len = min(p.row0 + 2 * tokens, p.nrows);
        p.tile1 = (p.len + kTile - 1) / kTile;
        return true;
      }
      before += __shfl_sync(0xffffffffu, scan, 31);
    }
    return false;
  }
};

__device__ __forceinline__ bool active(const Piece& pc, int i, int tokens) { return i == 0 || pc.row0 + tokens < pc.nrows; }
// Key tiles of row tile i.
__device__ __forceinline__ int tiles_of(const Piece& pc, int i, int tokens) {
  return i == 0 ? pc.tile0 : active(pc, 1, tokens) ? pc.tile1 : 0;
}

// The key tiles of a CTA's pieces as one sequence.
struct Tiles {
  Piece pc;
  int t = 0;
  __device__ __forceinline__ bool next(PieceRing& ring) {
    if (++t < pc.tile1) return true;
    if (!ring.take(pc)) return false;
    t = 0;
    return true;
  }
};

// The MMA warp of row tile I: the whole warp walks, one lane issues.  PV(n) goes out behind QK(n + 1)'s keys have come and
// before QK(n + 1), whose scores take the place of the weights.
template <typename E, int D, int I>
__device__ __forceinline__ void mma_role(PieceRing ring, uint32_t base, uint32_t full, uint32_t empty, uint32_t bars,
                                         uint32_t clean, uint32_t tmem, int tokens, bool negative, volatile int* abort_flag, int* err) {
  using C = Cfg<D>;
  const uint32_t id_qk = idesc_of<E>(kTile, false) | (negative ? 1u << 13 : 0u);  // -Q K^T
  constexpr uint32_t id_pv = idesc_of<E>(D, true);
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
  bool have = it.next(ring), act = false, first = false, last = false;
  unsigned vs = 0, vp = 0;     // the current tile's values
  bool run = false;            // a tile is waiting for its weights
  while (have || run) {
    const bool k_act = have && it.t < tiles_of(it.pc, I, tokens), k_last = k_act && it.t + 1 == tiles_of(it.pc, I, tokens);
    const unsigned ks = slot, kp = par;
    if (have) {
      if (++slot == C::SLOTS) slot = 0, par ^= 1;
      if (!wait(full + 8 * ks, kp)) return;   // also of keys that this tile has no use for: an arrival belongs to their phase
    }
    if (run) {
      if (!wait(clean + 8 * vs, vp)) return;
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
    if (run && last) {
      if (leader) umma_commit(o_done);
      __syncwarp();
    }
    const bool k_first = k_act && it.t == 0;
    if (k_first && !wait(q_full, qn++)) return;
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
    first = k_first;
    last = k_last;
    if (have) {
      vs = slot, vp = par;
      if (++slot == C::SLOTS) slot = 0, par ^= 1;
      have = it.next(ring);
    }
  }
}

// Adds to 32 of a row's sums the values that are no numbers, of the keys lo .. vis - 1.
template <typename E>
__device__ __forceinline__ void add_odd(const PromptParams& P, const Piece& pc, int lo, int vis, int col, uint32_t (&o)[32]) {
#pragma unroll 1
  for (int key = lo; key < vis; ++key) {
    const E* src = static_cast<const E*>(P.v.ptr) + (pc.tok0 + key) * P.v.token_stride + pc.head * P.v.head_stride + col;
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

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PromptParams P, int shift, const __grid_constant__ PromptMaps maps) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t full = base + C::BAR_AT, empty = full + 8 * C::SLOTS, bars = empty + 8 * C::SLOTS + 16 * kPieces;
  const uint32_t q_full = bars, s_full = bars + 16, o_done = bars + 32, turn = bars + 48, p_full = bars + 64;  // p_full: [row tile][part]
  const uint32_t clean = p_full + 16 * kParts;  // [ring slot], of values: looked through
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::PIECE_AT - 16);
  volatile int* odd_seen = reinterpret_cast<volatile int*>(smem + C::PIECE_AT - 12);  // values that are no numbers were taken out
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::PIECE_AT - 8);
  int* err = P.err ? P.err : &prompt_err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tokens = tile_tokens(P);
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
  {
    // the barriers lie side by side, one thread each: ring slots (full, empty), pieces (full, empty), then by row tile
    // queries, scores, sums, turns and the parts of the weights, then by slot values looked through
    constexpr int kNear = 2 * C::SLOTS + 2 * kPieces, kAll = kNear + 8 + 2 * kParts + C::SLOTS;
    if (tid < kAll) {
      const int k = tid - kNear;
      const int count = tid < C::SLOTS ? 1 : tid < 2 * C::SLOTS ? 2 : tid < 2 * C::SLOTS + kPieces ? 1
                        : k < 0 ? kSoftmaxWarps + 3 : k < 6 ? 1 : k < 8 + 2 * kParts ? 128 : 1;
      mbar_init(full + 8 * tid, count);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) *abort_flag = *odd_seen = 0;
  }
  PromptWalk walk;
  walk.full = reinterpret_cast<int*>(smem + C::SORT_AT);
  walk.rest = walk.full + kBuckets;
  walk.start = walk.rest + kBuckets;
  walk.shift = shift;
  walk.clear(tid);
  if (warp == kSoftmaxWarps + 3) tmem_alloc((uint32_t)__cvta_generic_to_shared(tmem_at), 512);
  __syncthreads();
  behind_the_stream();
  let_next_start();
  walk.count(P, tid, err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  if (tid == 0 && blockIdx.x == 0 && walk.overlap(P)) atomicExch(err, kErrOffsets);

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: warpgroup i holds row tile i, one row a thread ----
    const int i = warp >> 2, w4 = warp & 3, r = tid & 127;
    const uint32_t lanes = (uint32_t)w4 << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + C::S_COL + i * 128, to = tmem + lanes + C::O_COL + i * 128;
    // a negative scale turns the products around; for one of 0 a number that leaves -infinity what it is
    const float scale2 = P.scale == 0.f ? 1.17549435e-38f : fabsf(P.scale) * 1.4426950408889634f;
    Piece pc = {};
    // Queries: a box of whole tokens, called by one thread once the last product with the ones before is done.
    auto call_q = [&]() {
      if (r == 0) {
        mbar_arrive_expect_tx(q_full + 8 * i, (uint32_t)(tokens * P.G * D * 2));
#pragma unroll
        for (int h = 0; h < C::NH; ++h)
          tma_load_3d(base + C::Q_AT + i * C::SLOT + h * C::HALF, &maps.q, 64 * h, pc.head * P.G, pc.tok0 + pc.row0 + i * tokens,
                      q_full + 8 * i);
      }
    };
    // A row's token in the tile and head of its group; rows past the whole tokens are nobody's.
    const int row_tok = r / P.G, row_head = r - row_tok * P.G;
    // whole sectors a lane where rows lie on them, halves else
    const bool sectors = (((uintptr_t)P.out.ptr & 31) | (P.out.token_stride & 15) | (P.out.head_stride & 15)) == 0;
    unsigned n = 0;     // tiles of this row tile so far
    unsigned flat = 0;  // tiles of the CTA before the current piece
    unsigned turns = 0, done = 0;  // turns taken, pieces finished
    bool ok = true;
    auto advance = [&]() {  // to the next piece with rows of this tile
      while (ring.take(pc)) {
        if (active(pc, i, tokens)) return true;
        flat += pc.tile1;
      }
      return false;
    };
    bool have = advance();
    if (have) call_q();
    while (have && ok) {
      const Piece cur = pc;
      const int first = cur.row0 + i * tokens;        // the row tile's first token
      const int tok = min(first + row_tok, cur.nrows - 1);
      const int vis = tok + 1;                        // keys this row sees
      const int sure0 = cur.row0 + 1;                 // keys that every row of the piece sees
      const int sure = first + 1;                     // ... of the row tile
      const int tiles = tiles_of(cur, i, tokens);
      const bool two = active(cur, 1, tokens), in = row_tok < tokens && first + row_tok < cur.nrows;
      bool odd = false;
      float m = -CUDART_INF_F;
      float2 l = make_float2(0.f, 0.f);
      for (int t = 0; t < tiles; ++t, ++n) {
        const bool both = kTurns<D> && two && t < cur.tile0;
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
        const int see = vis - t * kTile;
        if ((t + 1) * kTile > sure) {
          // what a row does not see counts as -infinity: a weight of 0
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= see) s[k] = 0xff800000u;
        }
        float top = -CUDART_INF_F, t1 = top, t2 = top, t3 = top;
#pragma unroll
        for (int k = 0; k < 128; k += 8) {
          top = max3(top, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
          t1 = max3(t1, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
          t2 = max3(t2, __uint_as_float(s[k + 4]), __uint_as_float(s[k + 5]));
          t3 = max3(t3, __uint_as_float(s[k + 6]), __uint_as_float(s[k + 7]));
        }
        top = fmaxf(max3(top, t1, t2), t3);
        top = top == -CUDART_INF_F ? top : top * scale2 - kShift;
        // A row's reference moves with its own maximum alone: rows of the warp that see other keys, belong to the next
        // sequence or to nobody (whose queries are what shared memory holds) leave its bits as they are.
        const bool grew = in && top > m + kGrow;
        if (t == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, grew)) {
          const float f = grew ? ex2(m - top) : 1.f;
          if (grew) m = top;
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
        if (t + 1 == tiles) {
          // whether values that are no numbers were taken out of this piece's is known once its last ones have been looked
          // through, and to be asked while they are still there
          const unsigned slot = 2 * (flat + t) + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(clean + 8 * (slot % C::SLOTS), (slot / C::SLOTS) & 1, abort_flag, err));
          if (!ok) break;
          odd = *odd_seen;
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
      // The queries of the next piece with rows of this tile are called in before this one's sums come out.  Not before its
      // last weights are handed over: that piece may be several ahead, and is announced only as the products go on.
      flat += cur.tile1;
      have = advance();
      if (have) call_q();
      ok = __all_sync(0xffffffffu, mbar_wait(o_done + 8 * i, done++ & 1, abort_flag, err));
      if (!ok) break;
      tc_fence_after();
      const float sum = l.x + l.y, inv = sum == 0.f ? 0.f : __frcp_rn(sum);
      E* row = static_cast<E*>(P.out.ptr) + (long long)(cur.tok0 + tok) * P.out.token_stride +
               (long long)(cur.head * P.G + row_head) * P.out.head_stride;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t all[2][32];
        tmem_load64(to + c0, all[0], all[1]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t (&o)[32] = all[b];
          if (odd && in) add_odd<E>(P, cur, sure0, vis, c0 + 32 * b, o);
          if (in) {
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j] = pack2<E>(__uint_as_float(o[k + 2 * j]) * inv, __uint_as_float(o[k + 2 * j + 1]) * inv);
              E* to = row + c0 + 32 * b + k;
              if (sectors) {
                store8(reinterpret_cast<float*>(to), w);
              } else {
                reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
      }
      if (in && P.lse)
        P.lse[(long long)(cur.tok0 + tok) * P.hq + cur.head * P.G + row_head] =
            sum == 0.f ? -CUDART_INF_F : (m + log2f(sum)) * 0.6931471805599453f;
      tc_fence_before();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps) {
      // ---- producer: keys and values of a tile take one ring slot each ----
      walk.sort(P, lane);
      __syncwarp();
      walk.begin();
      unsigned x = 0;  // slots filled so far
      // pieces are announced before the loads of the one in front of them
      Piece pc = {}, ahead = {};
      bool more = walk.next(P, ahead, lane);
      bool ok = __all_sync(0xffffffffu, lane != 0 || ring.put(ahead));
      while (ok && more) {
        pc = ahead;
        more = walk.next(P, ahead, lane);
        ok = __all_sync(0xffffffffu, lane != 0 || ring.put(ahead));
        for (int t = 0; ok && t < pc.tile1; ++t) {
          for (int v = 0; v < 2; ++v, ++x) {
            const unsigned slot = x % C::SLOTS, round = x / C::SLOTS;
            ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, (round & 1) ^ 1, abort_flag, err));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full + 8 * slot, C::SLOT);
            __syncwarp();
            if (lane < C::NH)
              tma_load_3d(base + C::RING_AT + slot * C::SLOT + lane * C::HALF, v ? &maps.v : &maps.k, 64 * lane, pc.head,
                          pc.tok0 + t * kTile, full + 8 * slot);
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
      mma_role<E, D, 0>(ring, base, full, empty, bars, clean, tmem, tokens, P.scale < 0.f, abort_flag, err);
    } else if (warp == kSoftmaxWarps + 2) {
      mma_role<E, D, 1>(ring, base, full, empty, bars, clean, tmem, tokens, P.scale < 0.f, abort_flag, err);
    } else {
      // ---- values are looked through on their way to the products: those at keys that no row of the piece sees may be
      // anything, and those that are no numbers, at keys that only some rows see, come back to these rows at the end ----
      unsigned slot = 1, par = 0;
      Tiles it;
      it.pc.tile1 = 0;
      while (it.next(ring)) {
        if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * slot, par, abort_flag, err))) break;
        const int sure = it.pc.row0 + 1, key0 = it.t * kTile;
        const uint32_t at = base + C::RING_AT + slot * C::SLOT;
        const int c0 = max(sure - key0, 0) * 8 * C::NH + lane, c1 = kTile * 8 * C::NH;  // 16 bytes each
        auto place = [&](int c) { return at + (c / 8 % C::NH) * C::HALF + c / (8 * C::NH) * 128 + 16 * (c & 7); };
        // 0 times a value adds up to what is no number as soon as one is none
        using V = typename Pair<E>::V;
        uint32_t sum[4] = {0, 0, 0, 0};
        const uint32_t zero = 0;
        auto add = [&](uint32_t& to, uint32_t x) {
          const V y = __hfma2(*reinterpret_cast<const V*>(&x), *reinterpret_cast<const V*>(&zero), *reinterpret_cast<const V*>(&to));
          to = *reinterpret_cast<const uint32_t*>(&y);
        };
#pragma unroll 8
        for (int c = c0; c < c1; c += 32) {
          const uint4 v = shared16(place(c));
          add(sum[0], v.x), add(sum[1], v.y), add(sum[2], v.z), add(sum[3], v.w);
        }
        if (!all_finite<E>(make_uint4(sum[0], sum[1], sum[2], sum[3]))) {
#pragma unroll 1
          for (int c = c0; c < c1; c += 32) {
            const uint4 v = shared16(place(c));
            if (all_finite<E>(v)) continue;
            const bool seen = key0 + c / (8 * C::NH) < it.pc.len;
            sts128(place(c), seen ? make_uint4(v.x & finite_bits<E>(v.x), v.y & finite_bits<E>(v.y), v.z & finite_bits<E>(v.z),
                                               v.w & finite_bits<E>(v.w))
                                  : make_uint4(0, 0, 0, 0));
            if (seen) *odd_seen = 1;
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(clean + 8 * slot);
        slot += 2;
        if (slot > C::SLOTS) slot = 1, par ^= 1;
      }
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

// Boxes of 64 values x `heads_in` heads x `tokens_in` tokens, a row tile's queries, or of kTile tokens of one head.
cudaError_t encode(const pw_rows& r, int T, int heads, int dtype, int d, int heads_in, int tokens_in, CUtensorMap* map) {
  using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const auto enc = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  // the stride of a dimension of one does not matter to the caller, but has to be a stride
  const cuuint64_t dim[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t stride[2] = {(cuuint64_t)(heads > 1 ? r.head_stride : d) * 2, (cuuint64_t)(T > 1 ? r.token_stride : d) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_in, (cuuint32_t)tokens_in}, step[3] = {1, 1, 1};
  return enc(map, dtype == PW_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.ptr, dim, stride, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename E, int D>
cudaError_t launch_typed(const PromptParams& P, const PromptMaps& maps, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(prompt_kernel<E, D>);
  cudaError_t e = ensure_smem(fn, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be row tiles
  const long long most = ((long long)P.T / (2 * tile_tokens(P)) + P.B) * P.hkv;
  int shift = 0;
  while ((row_tiles(P, P.T) >> shift) >= kBuckets) ++shift;
  const Launch at(dim3(most < sm_count() ? (unsigned)most : sm_count()), kThreads, Cfg<D>::SMEM, s);
  return cudaLaunchKernelEx(&at.cfg, prompt_kernel<E, D>, P, shift, maps);
}

}  // namespace

cudaError_t prompt_error_word(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), prompt_err); }

cudaError_t launch_prompt(const PromptParams& P, int dtype, int d, cudaStream_t s) {
  PromptMaps maps;
  cudaError_t e = encode(P.k, P.T, P.hkv, dtype, d, 1, kTile, &maps.k);
  if (e == cudaSuccess) e = encode(P.v, P.T, P.hkv, dtype, d, 1, kTile, &maps.v);
  if (e == cudaSuccess) e = encode(P.q, P.T, P.hq, dtype, d, P.G, tile_tokens(P), &maps.q);
  if (e != cudaSuccess) return e;
  if (dtype == PW_F16) return d == 128 ? launch_typed<__half, 128>(P, maps, s) : launch_typed<__half, 64>(P, maps, s);
  return d == 128 ? launch_typed<__nv_bfloat16, 128>(P, maps, s) : launch_typed<__nv_bfloat16, 64>(P, maps, s);
}

}  // namespace pw
