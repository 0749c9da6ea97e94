// Attention of a decode batch over the paged cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// o = sum e^(s - m) v and l = sum e^(s - m) are rescaled when m grows, and
// partial (m, l, o) of disjoint key sets join exactly the same way, so the
// keys of one row may be split among CTAs (pw_attend.cuh) and joined at the
// end.  Exponents are taken in log2 units: e^s = 2^(s log2 e).
//
// attend_kernel streams keys and values once for up to 64 query rows: a
// producer warp issues TMA boxes of whole pages into a ring of 32 KB stages,
// four warps multiply them with mma.sync.  A stage holds 64 / HB keys of HB
// key heads; a warp takes one head (or, with fewer heads a stage, a row tile
// or a share of the keys), so with four heads a stage no warp ever waits for
// another.  With R rows a key head it does R products a key byte; up to 64 of
// them the legacy tensor path keeps up with HBM, so the loads bound it.  Items
// with more rows go to the tcgen05 kernel (pw_attend_tc.cu).  Measured: 64
// sequences with suffixes of 2048 tokens on average, 8 key heads of 128, 537
// MB in 88 us (6.1 TB/s); a call of one piece a CTA takes about 4 us from its
// first instruction (lengths, page, keys and products one after another).
#include <math_constants.h>

#include "pw_attend.cuh"
#include "pw_heads.cuh"
#include "pw_tc.cuh"

namespace pw {

namespace {

constexpr int kStageKeys = 64;             // keys x heads a stage
constexpr int kComputeWarps = 4;
constexpr int kThreads = (kComputeWarps + 1) * 32;

template <int D>
struct Cfg {
  static constexpr int HALF = kStageKeys * 128;         // one 64-value column block of a stage, 128-byte rows
  static constexpr int NH = D / 64;
  static constexpr int STAGE = 2 * NH * HALF;           // keys, then values
  static constexpr int STAGES = 98304 / STAGE;
  static constexpr int JOIN = 2 * (D / 8) * 512;        // accumulators of two warps
  static constexpr int JOIN_AT = STAGES * STAGE;
  static constexpr int ML_AT = JOIN_AT + JOIN;          // (m, l) of two warps' rows
  static constexpr int PIECE_AT = ML_AT + 2 * 128;
  static constexpr int BAR_AT = PIECE_AT + kPieces * (int)sizeof(Piece);
  static constexpr int SMEM = BAR_AT + 16 * STAGES + 16 * kPieces + 16;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(E) == 2 && __is_same(E, __half))
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kComputeWarps * 32) : "memory"); }
// The same, and whether it holds in all of them.
__device__ __forceinline__ bool compute_all(bool mine) {
  uint32_t all;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbar.red.and.pred p, 1, %2, q;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(all)
      : "r"((uint32_t)mine), "n"(kComputeWarps * 32)
      : "memory");
  return all != 0;
}

// Which keys of a tile each of a thread's two fragment words may hold: words
// whose key is at or past `n` (relative to the fragment's first key) become 0.
__device__ __forceinline__ uint32_t keep_keys(uint32_t w, int k, int n) {
  return k + 1 < n ? w : k < n ? (w & 0xffffu) : 0u;
}

// MT row tiles of 16, HB heads a stage; KS warps share the keys of a (row tile, head).
template <typename E, int D, int MT, int HB>
__global__ void __launch_bounds__(kThreads, 2)
    attend_kernel(const AttendParams P, const AttendWork W, const __grid_constant__ KvMaps maps) {
  using C = Cfg<D>;
  constexpr int ROWS = 16 * MT, KS = kComputeWarps / (MT * HB), TILE = kStageKeys / HB, KPW = TILE / KS;
  constexpr int HEAD = TILE * 128;  // bytes of one head's rows in a column block
  // a segment's fixed cost and a CTA's least work: about a 64-key tile's time
  using Walk = AttendWalk<ROWS, TILE, HB, HB, HB>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t full = base + C::BAR_AT, empty = full + 8 * C::STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::BAR_AT + 16 * C::STAGES + 16 * kPieces);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (base & 1023) {
    if (tid == 0) atomicExch(P.kv.err, kErrLayout);
    return;
  }
  // behind the tcgen05 kernel of the same call there is nothing to wait for here, only before the end
  if (W.behind) behind_the_stream();
  const typename Walk::Mine mine = Walk::mine(P, W);
  PieceRing ring;
  ring.full = empty + 8 * C::STAGES;
  ring.empty = ring.full + 8 * kPieces;
  ring.at = reinterpret_cast<Piece*>(smem + C::PIECE_AT);
  ring.abort_flag = abort_flag;
  ring.err = P.kv.err;
  if (tid < 2 * (C::STAGES + kPieces)) {  // one thread a barrier: stages (full, empty), pieces (full, empty)
    const bool one = tid < C::STAGES || (tid >= 2 * C::STAGES && tid < 2 * C::STAGES + kPieces);
    mbar_init(full + 8 * tid, one ? 1 : kComputeWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) *abort_flag = 0;
  Walk walk;
  walk.start(P, W, mine, reinterpret_cast<unsigned*>(smem + C::JOIN_AT));
  Piece pc;
  int stage = 0, phase = 0;

  if (warp == kComputeWarps) {
    // ---- producer: one lane a page ----
    const int shift = P.kv.page_shift;
    const int box = min(1 << shift, TILE);  // tokens of a box
    const int* table;
    bool ok = true;
    // a suffix is read once: its lines are the first to leave the L2, and the partial sums stay
    uint64_t once, normal, policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    while (ok) {
      const bool more = walk.next(P, pc, table);
      ok = __all_sync(0xffffffffu, lane != 0 || ring.put(pc));
      if (!more) break;
      policy = pc.prefix ? normal : once;
      for (int t = pc.tile0; ok && t < pc.tile1; ++t) {
        const int kt = key_tile<TILE>(pc, t), keys = min(TILE, pc.len - kt * TILE), boxes = (keys + box - 1) / box;
        const int at = kt * TILE + lane * box;
        int page = 0;
        if (lane < boxes) {
          page = table[at >> shift];
          if (page < 0 || page >= P.kv.n_pages) atomicExch(P.kv.err, kErrPage);  // reads as zeros
        }
        ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * stage, phase ^ 1, abort_flag, P.kv.err));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * stage, (uint32_t)(boxes * box * HB * D * 4));
        __syncwarp();
        if (lane < boxes) {
          // HB heads of a box that is shorter than the tile: one load a head, else one load for all
          const uint32_t dst = base + stage * C::STAGE + lane * box * 128;
          const int tok = at & ((1 << shift) - 1);
#pragma unroll
          for (int h = 0; h < C::NH; ++h) {
            if (HB == 1 || box == TILE) {
              tma_load_page(dst + h * C::HALF, &maps.k, 64 * h, tok, pc.head, page, full + 8 * stage, policy);
              tma_load_page(dst + (C::NH + h) * C::HALF, &maps.v, 64 * h, tok, pc.head, page, full + 8 * stage, policy);
            } else {
#pragma unroll
              for (int g = 0; g < HB; ++g) {
                tma_load_page(dst + h * C::HALF + g * HEAD, &maps.k, 64 * h, tok, pc.head + g, page, full + 8 * stage,
                              policy);
                tma_load_page(dst + (C::NH + h) * C::HALF + g * HEAD, &maps.v, 64 * h, tok, pc.head + g, page,
                              full + 8 * stage, policy);
              }
            }
          }
        }
        __syncwarp();
        if (++stage == C::STAGES) stage = 0, phase ^= 1;
      }
    }
    let_next_start();  // the join may take its place beside the last pieces
    if (!W.behind) behind_the_stream();
    // Copies in flight land before the shared memory goes away: the compute warps have waited for all of them, unless a
    // wait has given up, in any warp and at any time.
    for (int i = 0; i < C::STAGES; ++i)
      for (int k = 0; k < (1 << 16) && !mbar_try_wait(full + 8 * i, phase ^ (i < stage ? 0 : 1)); ++k) {
      }
    return;
  }

  // ---- compute warps ----
  const int g = lane >> 2, t4 = lane & 3;
  const int mt = warp % MT, hb = (warp / MT) % HB, ks = warp / (MT * HB), k0 = ks * KPW;
  const float scale2 = P.scale * 1.4426950408889634f;
  // ldmatrix row addresses inside a 128-byte-row block: lane l supplies row l % 8 of matrix l / 8
  const int mrow = lane & 7, msel = lane >> 3;
  uint32_t qf[D / 16][4];
  auto load_q = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = pc.row0 + mt * 16 + g + 8 * i;
      const bool in = r < pc.nrows;
      const int tok = in ? r / P.G : 0, hd = in ? (pc.head + hb) * P.G + r - tok * P.G : 0;
      const E* src = static_cast<const E*>(P.q.ptr) + (pc.tok0 + tok) * P.q.token_stride + hd * P.q.head_stride;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][i] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * t4) : 0u;
        qf[s][2 + i] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * t4) : 0u;
      }
    }
  };
  bool have = ring.take(pc);
  if (have) load_q();
  // Warps that share keys meet at barriers in every piece.  Where the wait for a piece gives up it may do so in some of
  // them only, so they go on together or not at all.
  if constexpr (KS > 1) have = compute_all(have);
  while (have) {
    const Piece cur = pc;
    const int ra = cur.row0 + mt * 16 + g;
    int vis[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      vis[i] = cur.causal && ra + 8 * i < cur.nrows ? cur.len - P.ql + 1 + (ra + 8 * i) / P.G : cur.len;
    const int sure = cur.causal ? cur.len - P.ql + 1 : cur.len;  // keys below this are seen by every row
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    bool odd_seen = false;
    for (int t = cur.tile0; t < cur.tile1; ++t) {
      // a wait that gives up leaves the sums as they are; the walk goes on, so that every barrier is met
      const bool landed = __all_sync(0xffffffffu, mbar_wait(full + 8 * stage, phase, abort_flag, P.kv.err));
      const int first = key_tile<TILE>(cur, t) * TILE + k0;  // this warp's first key
      if (landed && first < cur.len) {
        const uint32_t kb = base + stage * C::STAGE + hb * HEAD, vb = kb + C::NH * C::HALF;
        float s[KPW / 8][4];
#pragma unroll
        for (int n = 0; n < KPW / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        // matrices of a load: keys 0-7 / 8-15 (msel >> 1), values 0-7 / 8-15 (msel & 1)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
#pragma unroll
          for (int n = 0; n < KPW / 16; ++n) {
            const int row = k0 + 16 * n + 8 * (msel >> 1) + mrow, chunk = (2 * c + (msel & 1)) & 7;
            uint32_t b[4];
            ldsm4(kb + (c / 4) * C::HALF + row * 128 + ((chunk ^ mrow) << 4), b);
            mma16816<E>(s[2 * n], qf[c], b[0], b[1]);
            mma16816<E>(s[2 * n + 1], qf[c], b[2], b[3]);
          }
        }
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
        const bool edge = first + KPW > sure;
#pragma unroll
        for (int n = 0; n < KPW / 8; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[n][i] *= scale2;
            if (edge && first + 8 * n + 2 * t4 + (i & 1) >= vis[i >> 1]) s[n][i] = -CUDART_INF_F;
            top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
          }
        }
        float ref[2];
        bool grew = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
          top[i] = fmaxf(top[i] - kShift, m[i]);
          ref[i] = top[i] == -CUDART_INF_F ? 0.f : top[i];
          grew |= top[i] > m[i];
        }
        if (__any_sync(0xffffffffu, grew)) {
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f[i] = ex2(m[i] - ref[i]);  // 0 while m is -inf
            l[i] *= f[i];
            m[i] = top[i];
          }
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][0] *= f[0], o[d][1] *= f[0];
            o[d][2] *= f[1], o[d][3] *= f[1];
          }
        }
        uint32_t pf[KPW / 16][4];
#pragma unroll
        for (int n = 0; n < KPW / 8; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[n][i] = ex2(s[n][i] - ref[i >> 1]);
            l[i >> 1] += s[n][i];
          }
          pf[n / 2][2 * (n & 1)] = pack2<E>(s[n][0], s[n][1]);
          pf[n / 2][2 * (n & 1) + 1] = pack2<E>(s[n][2], s[n][3]);
        }
        bool odd = false;  // some value that is no number, at a key that some rows do not see
        if (first + KPW > sure && sure < cur.len) {
          const int lo = max(sure - first, 0), hi = min(cur.len - first, KPW);
          for (int k = 8 * C::NH * lo + lane; k < 8 * C::NH * hi; k += 32)
            odd |= !all_finite<E>(shared16(vb + (k & (C::NH - 1)) * C::HALF + (k0 + k / (8 * C::NH)) * 128 +
                                           16 * (k / C::NH & 7)));
          odd = __any_sync(0xffffffffu, odd);
          odd_seen |= odd;
        }
        const bool tail = first + KPW > cur.len;  // values past the length may be anything: 0 instead
#pragma unroll
        for (int n = 0; n < KPW / 16; ++n) {
          const int left = cur.len - first - 16 * n;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            // matrices: keys 0-7 / 8-15 (msel & 1), values 0-7 / 8-15 (msel >> 1)
            const int row = k0 + 16 * n + 8 * (msel & 1) + mrow, chunk = (2 * d + (msel >> 1)) & 7;
            uint32_t b[4];
            ldsm4t(vb + (d / 4) * C::HALF + row * 128 + ((chunk ^ mrow) << 4), b);
            if (tail) {
              b[0] = keep_keys(b[0], 2 * t4, left), b[1] = keep_keys(b[1], 2 * t4 + 8, left);
              b[2] = keep_keys(b[2], 2 * t4, left), b[3] = keep_keys(b[3], 2 * t4 + 8, left);
            }
            if (odd) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                b[i] = finite_bits<E>(b[i]) & b[i] | keep_keys(b[i], 2 * t4 + 8 * (i & 1), sure - first - 16 * n);
            }
            mma16816<E>(o[2 * d], pf[n], b[0], b[1]);
            mma16816<E>(o[2 * d + 1], pf[n], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage);
      if (++stage == C::STAGES) stage = 0, phase ^= 1;
    }

    if (odd_seen) {  // the rows that see them get them here
      const int* table = P.table + (long long)(cur.item - P.n_groups) * P.table_stride;
#pragma unroll 1
      for (int t = cur.tile0; t < cur.tile1; ++t) {
        const int at = key_tile<TILE>(cur, t) * TILE + k0;
#pragma unroll 1
        for (int key = max(max(sure, 0), at); key < min(cur.len, at + KPW); ++key) {
          const int page = table[key >> P.kv.page_shift];
          if (page < 0 || page >= P.kv.n_pages) continue;
          const E* src = reinterpret_cast<const E*>(P.kv.v) + page * P.kv.page_stride + (cur.head + hb) * P.kv.head_stride +
                         (key & ((1 << P.kv.page_shift) - 1)) * P.kv.token_stride + 2 * t4;
#pragma unroll
          for (int d = 0; d < D / 8; ++d)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 x = Pair<E>::up(*reinterpret_cast<const typename Pair<E>::V*>(src + 8 * d));
              if (key < vis[i]) {
                if (!isfinite(x.x)) o[d][2 * i] += x.x;
                if (!isfinite(x.y)) o[d][2 * i + 1] += x.y;
              }
            }
        }
      }
    }
    have = ring.take(pc);
    if (have) load_q();  // on their way while this piece's sums are stored

    // ---- join the warps that share keys: the upper half hands its sums to the lower one, in halving steps ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
#pragma unroll
    for (int step = KS / 2; step > 0; step >>= 1) {
      if (step == KS / 2)
        have = compute_all(have);
      else
        compute_sync();
      // the buffer is free
      if (ks >= step && ks < 2 * step) {
        const int slot = ((ks - step) * HB + hb) * MT + mt;
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          *reinterpret_cast<float4*>(smem + C::JOIN_AT + (slot * (D / 8) + d) * 512 + lane * 16) =
              make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
        if (t4 == 0)
          *reinterpret_cast<float4*>(smem + C::ML_AT + slot * 128 + g * 16) = make_float4(m[0], l[0], m[1], l[1]);
      }
      compute_sync();
      if (ks < step) {
        const int slot = (ks * HB + hb) * MT + mt;
        const float4 y = *reinterpret_cast<const float4*>(smem + C::ML_AT + slot * 128 + g * 16);
        const float ym[2] = {y.x, y.z}, yl[2] = {y.y, y.w};
        float fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mm = fmaxf(m[i], ym[i]), rr = mm == -CUDART_INF_F ? 0.f : mm;
          fa[i] = ex2(m[i] - rr);
          fb[i] = ex2(ym[i] - rr);
          l[i] = l[i] * fa[i] + yl[i] * fb[i];
          m[i] = mm;
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          const float4 v =
              *reinterpret_cast<const float4*>(smem + C::JOIN_AT + (slot * (D / 8) + d) * 512 + lane * 16);
          o[d][0] = o[d][0] * fa[0] + v.x * fb[0];
          o[d][1] = o[d][1] * fa[0] + v.y * fb[0];
          o[d][2] = o[d][2] * fa[1] + v.z * fb[1];
          o[d][3] = o[d][3] * fa[1] + v.w * fb[1];
        }
      }
    }
    if (ks == 0) {
      const AttendPieces& to = cur.prefix ? W.prefix : W.suffix;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = ra + 8 * i;
        if (r >= cur.nrows) continue;
        float* dst;
        if (cur.first) {
          const int tok = r / P.G;
          const long long row = (long long)(cur.tok0 + tok) * P.kv.hq + (cur.head + hb) * P.G + r - tok * P.G;
          dst = to.row_o + row * D;
          if (t4 == 0)
            to.row_ml[row] = make_float4(m[i], l[i], __int_as_float((int)blockIdx.x), __int_as_float(cur.last_cta));
        } else {
          const int row = (blockIdx.x * HB + hb) * ROWS + mt * 16 + g + 8 * i;
          dst = to.cta_o + (long long)row * D;
          if (t4 == 0) to.cta_ml[row] = make_float2(m[i], l[i]);
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          *reinterpret_cast<float2*>(dst + 8 * d + 2 * t4) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
      }
    }
  }
}

// How the prefix and the suffix kernel cut rows: rows and heads of a segment, CTAs, and whether it is the tcgen05 one.
struct JoinShape {
  int rows[2], heads[2], ctas[2], tc[2];
  int split;  // warps that share four rows
};

// Warps that share four rows' pieces, by the number of rows (query tokens x heads), 16 up to four rows an SM: a lone
// sequence on a long prefix has a piece from every CTA (measured: 20 rows of 300 pieces, the call 41 us with 4 warps, 31
// with 16), many rows fill the GPU by themselves (8192 rows: the call 136 us with 1, 142 with 4).
constexpr int kJoinWarps = 4;         // a CTA's, but for
constexpr int kJoinMost = 16;
constexpr int kJoinFlight = 4;        // pieces of a row that a warp has in flight
inline int join_split(long long rows, long long keys) {
  return rows <= 4 * sm_count() && keys > 64 * 32 ? kJoinMost : rows <= 4096 ? kJoinWarps : 1;
}

// With fewer segments than this every one is split among many CTAs: stages of one head then, whose four warps join their
// keys in the CTA, leave a quarter of the pieces (measured: one sequence of 4 key heads on 19327 tokens 31 -> 21 us; at
// 64 segments and more four heads a stage are as good or better).
constexpr int kFewSegments = 16;

// A row's pieces of one kind, as one lane of the join sees them.
struct Pieces {
  float2 first;        // m and l of the first, in the row's own place
  const float* row_o;  // this lane's values of it
  const float2* ml;    // of piece p >= 1: ml[p * step], o[p * step * D], in the slots of the CTAs after the first's
  const float* o;
  int count, step, far;  // far: from a lane's first 8 values to its second
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

// Joins the pieces of the rows.  A warp takes four adjacent rows of a key head (the tcgen05 blocks' lines hold 8 values
// of four rows), eight lanes a row, 8 values at a time, and goes through the pieces of the prefix and then of the suffix
// in their order, four in flight.  No exchange between lanes, and little code: its instructions are as cold as its data.
// With few rows several warps share them: each takes its four of every 4 x split pieces, and the first adds up.
template <typename E, int D>
__global__ void __launch_bounds__(kJoinMost * 32) join_kernel(const AttendParams P, const AttendWork W,
                                                               const JoinShape shape) {
  constexpr int NC = D / 64;  // times 8 values a lane
  const int lane = threadIdx.x & 31, hk = blockIdx.y, c8 = lane >> 2;
  const int warp = threadIdx.x >> 5, part = warp & (shape.split - 1);
  const int rows = P.B * P.ql * P.G;  // (query token, head of the group)
  const int mine = (blockIdx.x * (blockDim.x / 32 / shape.split) + warp / shape.split) * 4 + (lane & 3);
  const bool live = mine < rows;
  if (shape.split == 1 && !live) return;
  const int r = live ? mine : 0, n = r / P.G, h = hk * P.G + r - n * P.G, b = n / P.ql;
  int grp = P.n_groups - 1, tok0 = 0;  // the group of the sequence: the last that begins at or before it
  if (P.group_offsets && P.n_groups > 0) {
    int lo = 0, hi = P.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (P.group_offsets[mid] <= b) lo = mid;
      else hi = mid - 1;
    }
    const int first = min(max(P.group_offsets[lo], 0), P.B), last = min(max(P.group_offsets[lo + 1], first), P.B);
    grp = b >= first && b < last ? lo : -1;
    tok0 = first * P.ql;
  }
  const bool has[2] = {grp >= 0 && min(P.prefix_lens[grp], P.prefix_stride << P.kv.page_shift) > 0,
                       min(P.lens[b], P.table_stride << P.kv.page_shift) > 0};
  // What comes before this line reads the call's inputs only: this kernel starts once every CTA of the one before it in
  // the call has waited for the stream itself.
  behind_the_stream();
  let_next_start();
  const long long row = (long long)n * P.kv.hq + h;
  Pieces pc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const AttendPieces& from = i ? W.suffix : W.prefix;
    const float4 rec = has[i] ? from.row_ml[row] : make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
    // CTAs inside the slots whatever a kernel that gave up on a wait has left there
    const int c0 = min(max(__float_as_int(rec.z), 0), shape.ctas[i] - 1);
    const int c1 = min(max(__float_as_int(rec.w), c0), shape.ctas[i] - 1);
    const int item_row = r - (i ? b * P.ql : tok0) * P.G, in_tile = item_row & (shape.rows[i] - 1);
    const int slot = (c0 * shape.heads[i] + (hk & (shape.heads[i] - 1))) * shape.rows[i] + in_tile;
    pc[i].first = make_float2(rec.x, rec.y);
    pc[i].count = has[i] ? c1 - c0 + 1 : 0;
    pc[i].step = shape.heads[i] * shape.rows[i];
    pc[i].ml = from.cta_ml + slot;
    pc[i].far = shape.tc[i] ? 8 * kTcRows * 8 : 64;
    const int column = c8 * 8 * (shape.tc[i] ? kTcRows : 1);
    pc[i].o = from.cta_o + (shape.tc[i] ? (long long)c0 * kTcRows * D + in_tile * 8 : (long long)slot * D) + column;
    pc[i].row_o = from.row_o + row * D + c8 * 8;
    if (shape.tc[i] && i == 0)
      pc[i].row_o = from.row_o + tc_block(tok0, P.G, grp, item_row / kTcRows, P.kv.hkv, hk) * kTcRows * D + in_tile * 8 + column;
  }
  float m = -CUDART_INF_F, l = 0.f, o[NC * 8];
#pragma unroll
  for (int k = 0; k < NC * 8; ++k) o[k] = 0.f;
  const int all = pc[0].count + pc[1].count;
#pragma unroll 1
  for (int p0 = kJoinFlight * part; p0 < all; p0 += kJoinFlight * shape.split) {
    float2 ml[kJoinFlight];
    float v[kJoinFlight][NC][8];
#pragma unroll
    for (int j = 0; j < kJoinFlight; ++j) {
      const bool suf = p0 + j >= pc[0].count;
      const int p = p0 + j - (suf ? pc[0].count : 0), step = suf ? pc[1].step : pc[0].step;
      ml[j] = make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][c][k] = 0.f;
      if (p0 + j >= all) continue;
      const float* src = suf ? pc[1].row_o : pc[0].row_o;
      int far = suf ? 64 : pc[0].far;  // a suffix's first piece is a plain row
      if (p == 0) {
        ml[j] = suf ? pc[1].first : pc[0].first;
      } else {
        ml[j] = (suf ? pc[1].ml : pc[0].ml)[p * step];
        src = (suf ? pc[1].o : pc[0].o) + (long long)p * step * D;
        far = suf ? pc[1].far : pc[0].far;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) load8(src + c * far, v[j][c]);
    }
    float mm = m;
#pragma unroll
    for (int j = 0; j < kJoinFlight; ++j) mm = fmaxf(mm, ml[j].x);
    const float rr = mm == -CUDART_INF_F ? 0.f : mm, keep = ex2(m - rr);
    m = mm;
    l *= keep;
#pragma unroll
    for (int k = 0; k < NC * 8; ++k) o[k] *= keep;
#pragma unroll
    for (int j = 0; j < kJoinFlight; ++j) {
      const float w = ex2(ml[j].x - rr);
      l = fmaf(ml[j].y, w, l);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) o[c * 8 + k] = fmaf(v[j][c][k], w, o[c * 8 + k]);
    }
  }
  if (shape.split > 1) {
    __shared__ float2 other_ml[kJoinMost][32];
    __shared__ float4 other_o[kJoinMost][NC * 2][32];
    if (part != 0) {
      other_ml[warp][lane] = make_float2(m, l);
#pragma unroll
      for (int k = 0; k < NC * 2; ++k)
        other_o[warp][k][lane] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    }
    __syncthreads();
    if (part != 0 || !live) return;
#pragma unroll 1
    for (int w = warp + 1; w < warp + shape.split; ++w) {
      const float2 y = other_ml[w][lane];
      const float mm = fmaxf(m, y.x), rr = mm == -CUDART_INF_F ? 0.f : mm, fa = ex2(m - rr), fb = ex2(y.x - rr);
      m = mm;
      l = l * fa + y.y * fb;
#pragma unroll
      for (int k = 0; k < NC * 2; ++k) {
        const float4 v = other_o[w][k][lane];
        o[4 * k] = o[4 * k] * fa + v.x * fb;
        o[4 * k + 1] = o[4 * k + 1] * fa + v.y * fb;
        o[4 * k + 2] = o[4 * k + 2] * fa + v.z * fb;
        o[4 * k + 3] = o[4 * k + 3] * fa + v.w * fb;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  E* out = static_cast<E*>(P.out.ptr) + n * P.out.token_stride + h * P.out.head_stride + c8 * 8;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = o[c * 8 + k] * inv;
    *reinterpret_cast<uint4*>(out + c * 64) = pack8<E>(v);
  }
  if (c8 == 0 && P.lse) P.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

int stream_ctas() { return 2 * sm_count(); }

// A prefix of little work (rows x keys x key heads, by what its table can hold) goes through the streaming kernel with
// the suffixes: its own launch would cost more (12 sequences of 25 rows behind 3 tokens 16.1 -> 10.5 us, 23 of 11 behind
// 1289 16.8 -> 11.7; 100 of 55 rows behind 320 48.8 -> 53.1 at 2.2e6, 70 of 25 behind 1116 24.9 -> 32.4 at 7.8e6).  Where
// long suffixes keep that kernel waiting for HBM it takes eight times as much along (64 sequences of 4 rows, suffixes to
// 1000: 35.5 -> 29.2 us at 2.1e6, to 4095: 95.2 -> 89.4 at 4.2e6; 32 of 4, to 4000: 62 -> 56 at 8.2e6).
// The host knows the tables' widths, not the lengths: with tables much wider than their sequences the rule sees more work
// than there is, and such a call costs up to what its other side measured (calls like the first two 12.1 -> 16.6 and 12.3 ->
// 16.3 us with a table for 32768 prefix tokens; 64 sequences of 4 rows behind 2048 tokens, suffixes to 100, with a table for
// 32768 suffix tokens 23.3 -> 26.5).
constexpr double kLittlePrefix = 2e6, kLongSuffix = 262144;  // the latter in keys x key heads of the whole batch

// Which kernel takes which items.  Up to 64 rows a key head the streaming
// kernel is bound by its loads; beyond, its products are.
struct Plan {
  bool tc_prefix, tc_suffix;
  int stream_rows;     // rows of the streaming kernel's tiles, 0 when it has no items
  int heads;           // key heads of its stages
  // prefix_keys, suffix_keys: what a row of the prefix's and of the suffix's table can hold
  Plan(int G, int hkv, int B, int ql, int n_groups, long long prefix_keys, long long suffix_keys) {
    const long long own = (long long)ql * G, shared = n_groups > 0 ? (B * own + n_groups - 1) / n_groups : 0;
    const double work = (double)B * own * hkv * prefix_keys;
    const bool waits = own <= 16 && (double)B * hkv * suffix_keys >= kLongSuffix;
    const bool little = work <= (waits ? 8 : 1) * kLittlePrefix;
    tc_suffix = own > 64;
    tc_prefix = n_groups > 0 && ((shared > 64 && !little) || tc_suffix);
    const long long rows = !tc_suffix && !tc_prefix && shared > own && shared <= 64 ? shared : own;
    stream_rows = tc_suffix ? 0 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    heads = stream_rows == 16 ? 4 : stream_rows == 32 ? 2 : 1;
    while (hkv % heads || (heads > 1 && (long long)(B + (tc_prefix ? 0 : n_groups)) * (hkv / heads) < kFewSegments)) heads /= 2;
  }
  bool tc() const { return tc_prefix || tc_suffix; }
};

struct Layout {
  size_t row_o[2], row_ml[2], cta_o[2], cta_ml[2], total;  // [prefix, suffix], [streaming, tcgen05]
  Layout(const Plan& plan, int hq, int hkv, int d, int B, int ql, int n_groups) {
    const size_t rows = (size_t)B * ql * hq;
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t was = at;
      at += (n + 255) & ~(size_t)255;
      return was;
    };
    for (int i = 0; i < 2; ++i) {
      const size_t blocks = tc_block((long long)B * ql, hq / hkv, n_groups, 0, hkv, 0) + hkv;
      row_o[i] = take(i == 1 ? rows * d * 4 : n_groups == 0 ? 0 : (plan.tc_prefix ? blocks * kTcRows : rows) * d * 4);
      row_ml[i] = take(rows * 16);
      const size_t most = i ? (plan.tc() ? (size_t)attend_tc_ctas() * kTcRows : 0) : (size_t)stream_ctas() * plan.stream_rows * plan.heads;
      cta_o[i] = take(most * d * 4);
      cta_ml[i] = take(most * 8);
    }
    total = at + 256;
  }
};

template <typename E, int D, int MT, int HB>
cudaError_t launch_stream(const AttendParams& P, const AttendWork& W, const KvMapSet& maps, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(attend_kernel<E, D, MT, HB>);
  const cudaError_t e = ensure_smem(fn, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  // boxes of several heads only where a page holds a whole tile
  const bool whole = (1 << P.kv.page_shift) >= kStageKeys / HB;
  const KvMaps& m = HB == 4 && whole ? maps.heads4 : HB == 2 && whole ? maps.heads2 : maps.heads1;
  const Launch at(dim3(stream_ctas()), kThreads, Cfg<D>::SMEM, s);
  return cudaLaunchKernelEx(&at.cfg, attend_kernel<E, D, MT, HB>, P, W, m);
}

template <typename E, int D>
cudaError_t launch_typed(const AttendParams& P, const KvMapSet& maps, void* ws, cudaStream_t s) {
  const Plan plan(P.G, P.kv.hkv, P.B, P.ql, P.n_groups, (long long)P.prefix_stride << P.kv.page_shift,
                  (long long)P.table_stride << P.kv.page_shift);
  const Layout L(plan, P.kv.hq, P.kv.hkv, D, P.B, P.ql, P.n_groups);
  char* w = static_cast<char*>(ws);
  auto pieces = [&](bool suffix, bool tc) {
    AttendPieces p;
    p.row_o = reinterpret_cast<float*>(w + L.row_o[suffix]);
    p.row_ml = reinterpret_cast<float4*>(w + L.row_ml[suffix]);
    p.cta_o = reinterpret_cast<float*>(w + L.cta_o[tc]);
    p.cta_ml = reinterpret_cast<float2*>(w + L.cta_ml[tc]);
    return p;
  };
  AttendWork W = {};
  W.prefix = pieces(false, plan.tc_prefix);
  W.suffix = pieces(true, plan.tc_suffix);
  cudaError_t e = cudaSuccess;
  if (plan.tc()) {
    W.behind = true;
    W.first = 0;
    W.count = P.n_groups + (plan.tc_suffix ? P.B : 0);
    e = launch_attend_tc(P, W, maps.heads1, attend_tc_ctas(), s);
    if (e != cudaSuccess) return e;
  }
  if (plan.stream_rows) {
    W.behind = !plan.tc();
    W.first = plan.tc_prefix ? P.n_groups : 0;
    W.count = P.n_groups + P.B - W.first;
    switch (plan.stream_rows * 8 + plan.heads) {
      case 16 * 8 + 4: e = launch_stream<E, D, 1, 4>(P, W, maps, s); break;
      case 16 * 8 + 2: e = launch_stream<E, D, 1, 2>(P, W, maps, s); break;
      case 16 * 8 + 1: e = launch_stream<E, D, 1, 1>(P, W, maps, s); break;
      case 32 * 8 + 2: e = launch_stream<E, D, 2, 2>(P, W, maps, s); break;
      case 32 * 8 + 1: e = launch_stream<E, D, 2, 1>(P, W, maps, s); break;
      default: e = launch_stream<E, D, 4, 1>(P, W, maps, s);
    }
    if (e != cudaSuccess) return e;
  }
  JoinShape shape;
  for (int i = 0; i < 2; ++i) {
    const bool tc = i ? plan.tc_suffix : plan.tc_prefix;
    shape.rows[i] = tc ? kTcRows : plan.stream_rows;
    shape.heads[i] = tc ? 1 : plan.heads;
    shape.tc[i] = tc;
    shape.ctas[i] = tc ? attend_tc_ctas() : stream_ctas();
  }
  const int join_rows = P.B * P.ql * P.G;
  shape.split = join_split((long long)join_rows * P.kv.hkv,
                           (long long)(P.table_stride + (P.n_groups ? P.prefix_stride : 0)) << P.kv.page_shift);
  const int warps = shape.split > kJoinWarps ? shape.split : kJoinWarps, cta_rows = 4 * warps / shape.split;
  const Launch at(dim3((join_rows + cta_rows - 1) / cta_rows, P.kv.hkv), warps * 32, 0, s);
  return cudaLaunchKernelEx(&at.cfg, join_kernel<E, D>, P, W, shape);
}

}  // namespace

cudaError_t encode_kv_maps(const KvView& kv, KvMapSet* maps) {
  using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const auto enc = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  const int pt = 1 << kv.page_shift;
  const cuuint64_t dim[4] = {(cuuint64_t)kv.d, (cuuint64_t)pt, (cuuint64_t)kv.hkv, (cuuint64_t)kv.n_pages};
  const cuuint64_t stride[3] = {(cuuint64_t)kv.token_stride * 2, (cuuint64_t)kv.head_stride * 2,
                                (cuuint64_t)kv.page_stride * 2};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const auto type = kv.dtype == PW_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  for (int heads = 1; heads <= 4; heads *= 2) {
    const int tokens = kBoxTokens / heads;
    if (heads > 1 && (kv.hkv % heads || pt < tokens)) continue;  // never asked for
    KvMaps* m = heads == 1 ? &maps->heads1 : heads == 2 ? &maps->heads2 : &maps->heads4;
    const cuuint32_t box[4] = {64, (cuuint32_t)(pt < tokens ? pt : tokens), (cuuint32_t)heads, 1};
    for (int i = 0; i < 2; ++i)
      if (enc(i ? &m->v : &m->k, type, 4, i ? kv.v : kv.k, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

size_t attend_ws_bytes(const KvView& kv, int B, int ql, int n_groups) {
  size_t most = 0;  // whichever kernel a call's prefix table leads to
  for (long long keys : {0ll, 1ll << 40}) {
    const size_t n = Layout(Plan(kv.hq / kv.hkv, kv.hkv, B, ql, n_groups, keys, 0), kv.hq, kv.hkv, kv.d, B, ql, n_groups).total;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_attend(const AttendParams& P, const KvMapSet& maps, void* ws, cudaStream_t s) {
  if (P.kv.dtype == PW_F16)
    return P.kv.d == 128 ? launch_typed<__half, 128>(P, maps, ws, s) : launch_typed<__half, 64>(P, maps, ws, s);
  return P.kv.d == 128 ? launch_typed<__nv_bfloat16, 128>(P, maps, ws, s)
                       : launch_typed<__nv_bfloat16, 64>(P, maps, ws, s);
}

}  // namespace pw
