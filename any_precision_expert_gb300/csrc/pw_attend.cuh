// How an attention call is cut into pieces, shared by its kernels.
//
// Items are the prefix groups (all query rows of the group against the
// prefix) and the sequences (their own rows against their suffix).  Rows of an
// item are flat: row r is query token r / G, head r % G of the key head's
// group.  An item is cut into segments (key head, row tile), a segment into
// key tiles.  All key tiles of a launch, plus a fixed cost in tiles for every
// segment, form one line that is divided evenly among the CTAs, so ragged
// lengths and few long sequences load every SM alike, and the host never
// needs the lengths.  A CTA's range covers at most one segment that began
// before it (its result goes to the CTA's own slot) and any number that begin
// in it (their results go to the rows' slots); a merge kernel joins the pieces
// of a row in a fixed order.
#pragma once

#include <cuda.h>

#include "pw_mma.cuh"
#include "pw_serve.h"
#include "pw_tc.cuh"

namespace pw {

// Where the pieces of a launch go.  Values are sums relative to the piece's
// reference m: o = sum 2^(s - m) v, l = sum 2^(s - m), s in log2 units.
// The streaming kernel writes plain rows: a first piece's in the row's place
// (query token, head), a further one's in slots [cta][HB][ROWS].  The tcgen05
// kernel, whose threads hold a row each, writes blocks of 256 rows in 8-value
// columns [D / 8][256][8], so that a warp's stores are whole lines: a prefix's
// first piece in block (row tile, key head), a further piece in block [cta];
// first pieces of suffixes are plain rows here too.
struct AttendPieces {
  float* row_o;      // segments' first pieces
  float4* row_ml;    // [rows]: m, l, and the CTAs that hold the further pieces: (first, last] as int bits
  float* cta_o;      // pieces that continue a segment
  float2* cta_ml;    // their m and l
};

// Block of an item's row tile: items' tiles numbered without gaps larger than one.
__host__ __device__ inline long long tc_block(long long tok0, int G, int item, int tile, int hkv, int head) {
  return (tok0 * G / 256 + item + tile) * hkv + head;
}

struct AttendWork {
  int first, count;       // items of this launch: 0 .. n_groups - 1 prefixes, then the sequences
  bool behind;            // the call's first kernel: waits for what comes before it in the stream
  AttendPieces prefix, suffix;
};

struct Item {
  int tok0, nrows, len;   // first query token, rows (tokens * G), keys
  const int* table;
  bool causal;
};

__device__ __forceinline__ Item attend_item(const AttendParams& P, int i, bool flag) {
  Item it;
  bool bad;
  if (i < P.n_groups) {
    const int lo = P.group_offsets ? P.group_offsets[i] : 0, hi = P.group_offsets ? P.group_offsets[i + 1] : P.B;
    const int l = min(max(lo, 0), P.B), h = min(max(hi, l), P.B);
    const int len = P.prefix_lens[i], most = P.prefix_stride << P.kv.page_shift;
    it.tok0 = l * P.ql;
    it.nrows = (h - l) * P.ql * P.G;
    it.len = min(max(len, 0), most);
    it.table = P.prefix_table + (long long)i * P.prefix_stride;
    it.causal = false;
    bad = l != lo || h != hi || it.len != len;
  } else {
    const int b = i - P.n_groups, len = P.lens[b], most = P.table_stride << P.kv.page_shift;
    it.tok0 = b * P.ql;
    it.nrows = P.ql * P.G;
    it.len = min(max(len, 0), most);
    it.table = P.table + (long long)b * P.table_stride;
    it.causal = true;
    bad = it.len != len;
  }
  if (flag && bad) atomicExch(P.kv.err, kErrLength);
  return it;
}

// One piece of work, as the producer hands it to the CTA's other warps.
struct __align__(16) Piece {
  int tok0, nrows, len, causal;   // the item
  int head, row0;                 // first key head, first row of the row tile
  int tile0, tile1;               // key tiles; none (tile1 = 0) ends the CTA's range
  int first;                      // holds the segment's first tile
  int last_cta;                   // CTA that holds its last one
  int prefix, item;
  int turn, pad[3];               // tile t of the piece is key tile t - turn, or that + tiles of the segment where negative
};

constexpr int kPieces = 4;        // pieces announced ahead

// The key tile that a piece's tile t stands for.
template <int TILE>
__device__ __forceinline__ int key_tile(const Piece& p, int t) {
  const int k = t - p.turn;
  return k < 0 ? k + (p.len + TILE - 1) / TILE : k;
}

// Shared-memory ring of pieces: the producer writes, every reader warp takes each.
struct PieceRing {
  uint32_t full, empty;           // mbarriers (kPieces each)
  Piece* at;
  volatile int* abort_flag;
  int* err;
  unsigned n = 0;                 // pieces written or taken so far

  // Producer, one lane.
  __device__ __forceinline__ bool put(const Piece& p) {
    const unsigned i = n % kPieces;
    if (!mbar_wait(empty + 8 * i, ((n / kPieces) & 1) ^ 1, abort_flag, err)) return false;
    at[i] = p;
    mbar_arrive(full + 8 * i);
    ++n;
    return true;
  }
  // Reader, whole warp.
  __device__ __forceinline__ bool take(Piece& p) {
    const unsigned i = n % kPieces;
    if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * i, (n / kPieces) & 1, abort_flag, err))) return false;
    p = at[i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * i);
    ++n;
    return p.tile1 > 0;
  }
};

// A CTA's walk over its range of the line.  Segments hold HB key heads and cost COST tiles beside their own; a CTA gets
// LEAST units or none, so that its fixed costs and the partial sums of a split stay in proportion.
template <int ROWS, int TILE, int COST, int HB, int LEAST>
struct AttendWalk {
  int item;             // current item
  unsigned off;         // units of the item before the current position
  unsigned left;        // units of the range not walked yet
  unsigned pos;         // position on the line
  unsigned share, more; // CTAs 0 .. more - 1 take share + 1 units, the others share

  static __device__ __forceinline__ unsigned units(const AttendParams& P, const Item& it) {
    if (it.len == 0 || it.nrows == 0) return 0;
    return (unsigned)((it.len + TILE - 1) / TILE + COST) * ((it.nrows + ROWS - 1) / ROWS) * (P.kv.hkv / HB);
  }

  // Each thread's share of the items, read at the kernel's start so that the reads overlap the set-up.
  struct Mine {
    int i0, i1;
    unsigned sum;
  };
  static __device__ __forceinline__ Mine mine(const AttendParams& P, const AttendWork& W) {
    const int per = (W.count + blockDim.x - 1) / blockDim.x;
    Mine m;
    m.i0 = min((int)threadIdx.x * per, W.count);
    m.i1 = min(m.i0 + per, W.count);
    m.sum = 0;
#pragma unroll 1
    for (int i = m.i0; i < m.i1; ++i) m.sum += units(P, attend_item(P, W.first + i, blockIdx.x == 0));
    return m;
  }

  // Whole CTA: finds the CTA's range.  scratch: 34 words of shared memory.
  __device__ __forceinline__ void start(const AttendParams& P, const AttendWork& W, const Mine& my, unsigned* scratch) {
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned sum = my.sum;
    unsigned scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    if (lane == 31) scratch[warp] = scan;
    if (tid == 0) scratch[32] = scratch[33] = 0;
    __syncthreads();
    unsigned before = scan - sum, total = 0;
#pragma unroll 1
    for (int w = 0; w < nt / 32; ++w) {
      if (w < warp) before += scratch[w];
      total += scratch[w];
    }
    const unsigned ctas = min((unsigned)gridDim.x, max(1u, total / LEAST)), c = blockIdx.x;
    share = total / ctas;
    more = total - share * ctas;
    pos = c * share + min(c, more);
    left = c < ctas ? share + (c < more) : 0;
    if (left > 0 && pos >= before && pos < before + sum) {  // one thread's items hold the start
      unsigned at = before, n = sum;
      int i = my.i0;
#pragma unroll 1
      for (; my.i1 - my.i0 > 1 && i < my.i1; ++i) {
        n = units(P, attend_item(P, W.first + i, false));
        if (pos < at + n) break;
        at += n;
      }
      scratch[32] = W.first + i;
      scratch[33] = pos - at;
    }
    __syncthreads();
    item = (int)scratch[32];
    off = scratch[33];
  }

  // The CTA whose range holds position x.
  __device__ __forceinline__ int owner(unsigned x) const {
    const unsigned big = more * (share + 1);
    return (int)(x < big ? x / (share + 1) : more + (x - big) / share);
  }

  // The next piece with tiles in it and its item's page table; false (and a piece without tiles) at the end of the range.
  __device__ __forceinline__ bool next(const AttendParams& P, Piece& p, const int*& table) {
    p.tile1 = 0;
#pragma unroll 1
    while (left > 0) {
      const Item it = attend_item(P, item, false);
      const unsigned n = units(P, it);
      if (off >= n) {
        ++item;
        off = 0;
        continue;
      }
      const int kt = (it.len + TILE - 1) / TILE, rt = (it.nrows + ROWS - 1) / ROWS;
      const unsigned su = kt + COST, seg = off / su, within = off - seg * su;
      const unsigned take = min(su - within, left), end = within + take;
      const unsigned seg_last = pos - within + su - 1;  // the segment's last unit
      off += take;
      pos += take;
      left -= take;
      if (end <= COST) continue;
      p.tok0 = it.tok0;
      p.nrows = it.nrows;
      p.len = it.len;
      p.causal = it.causal;
      p.head = rt == 1 ? seg : seg / rt;
      p.row0 = (seg - p.head * rt) * ROWS;
      p.head *= HB;
      p.tile0 = within > COST ? within - COST : 0;
      p.tile1 = end - COST;
      p.first = within <= COST;
      p.last_cta = owner(seg_last);
      p.prefix = item < P.n_groups;
      p.item = item;
      // Row tiles of the same keys begin at the same key tile in the first CTA that begins in them, so that these CTAs
      // go through the keys side by side and find each other's lines in the L2.
      p.turn = 0;
      if (rt > 1) {
        const unsigned begin = seg_last + 1 - su, c = owner(begin), at = c * share + min(c, more);
        const unsigned ahead = at == begin ? 0 : at + share + (c < more) - begin;  // units up to the next CTA's start
        if (ahead > COST && ahead - COST < (unsigned)kt) p.turn = ahead - COST;
      }
      table = it.table;
      return true;
    }
    return false;
  }
};

// Weights are kept as 2^(s - max + kShift): fp16 weights down to 2^-(14 + kShift) of the largest stay normal numbers.
constexpr float kShift = 6.f;

__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int x, int tok, int head, int page,
                                              uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(tok), "r"(head), "r"(page), "r"(mbar)
      : "memory");
}
// The same with an L2 policy.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int x, int tok, int head, int page,
                                              uint32_t mbar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(map), "r"(x), "r"(tok), "r"(head), "r"(page), "r"(mbar), "l"(policy)
      : "memory");
}

// A query's weight for a key that it does not see is 0, but 0 times an infinity or NaN is NaN.  Values at keys that only
// some rows of a sequence see (the last q_len - 1) are therefore looked at, and those that are no numbers kept from the
// other rows.
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// Ones where the two 16-bit values of a word are finite.
template <typename E>
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7c00u : 0x7f80u;
  return ((w & kExp) == kExp ? 0u : 0xffffu) | ((w >> 16 & kExp) == kExp ? 0u : 0xffff0000u);
}
template <typename E>
__device__ __forceinline__ bool all_finite(const uint4& v) {
  return (finite_bits<E>(v.x) & finite_bits<E>(v.y) & finite_bits<E>(v.z) & finite_bits<E>(v.w)) == 0xffffffffu;
}

// Where the join finds the pieces of prefixes [0] and suffixes [1]: rows and key heads of the slots, CTAs that wrote them,
// whether the tcgen05 kernel did.
struct JoinShape {
  int rows[2], heads[2], ctas[2], tc[2];
  int split;  // warps that share four rows; the launch sets it
};
cudaError_t launch_join(const AttendParams& P, const AttendWork& W, JoinShape shape, cudaStream_t s);

// The tensor-core kernel for prefix groups with many rows (pw_attend_tc.cu).
constexpr int kTcRows = 256;
cudaError_t launch_attend_tc(const AttendParams& P, const AttendWork& W, const KvMaps& maps, int ctas, cudaStream_t s);
int attend_tc_ctas();

}  // namespace pw
