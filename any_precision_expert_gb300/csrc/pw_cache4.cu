// The paged cache held in 4 bits: append, load and attention.
//
// A head row is cut into groups of 32 values.  A group keeps its least value
// and a step of the heads' type and 32 codes c in 0..15; a value stands for
// least + c step.  The order of a row's codes is that of the products, so that
// a lane's share of a row is one aligned piece and a mask turns it into
// operands:
// * keys: word t D / 32 + i (i < D / 32, t < 4) holds values 32 i + 8 t .. + 7,
//   what lane t of four multiplies, in the order 0 4 2 6 1 5 3 7 from the lowest
//   nibble on: values (0, 1) and (2, 3) are the operand pairs of an even product
//   step, (4, 5) and (6, 7) of the odd one, and a pair lies 16 bits apart;
// * values: in order, D / 8 for each of eight lanes; heads of 128 with the
//   row's halves exchanged where bit 2 of the token is set, so that the rows
//   a warp reads at once lie in different banks (value_word).
#include <math_constants.h>

#include "pw_attend.cuh"
#include "pw_heads.cuh"
#include "pw_mma.cuh"

namespace pw {

namespace {

template <int D>
__device__ __forceinline__ int value_word(int l, int token) {
  return D == 128 ? l ^ ((token & 4) << 1) : l;
}

template <typename E>
__device__ __forceinline__ float to_f32(uint16_t bits) {
  E e;
  memcpy(&e, &bits, 2);
  return (float)e;
}
template <typename E>
__device__ __forceinline__ uint16_t from_f32(float x) {
  E e;
  if constexpr (__is_same(E, __half)) e = __float2half_rn(x);
  else e = __float2bfloat16_rn(x);
  uint16_t bits;
  memcpy(&bits, &e, 2);
  return bits;
}

// ---- append and load ------------------------------------------------------------
//
// Eight values a lane: a row is D / 8 lanes, a group four of them, a lane's
// codes one word.  Bound by HBM for long prompts, by one chain of loads else; a
// warp has U steps of rows in flight (one while there are few).  Quotients are
// products with the step's reciprocal, off by less than 2^-17, and exact
// divisions where one falls that near to a half.  Measured: 8191 tokens of 16
// heads of 128, append 37 us in bf16 (some 265 instructions a lane and eight
// values issued; 32 us in fp16, where halves are rarer), load 21 (4.2 TB/s; 147).

constexpr int kRowThreads = 128;

struct Row4 {
  uint32_t* codes;   // this lane's word
  uint32_t* step;    // its group's least value and step
};

template <int D>
__device__ __forceinline__ Row4 row4(const Kv4View& kv, int value, long long row, int l) {
  uint32_t* codes = reinterpret_cast<uint32_t*>(value ? kv.v : kv.k) + row * (D / 8);
  uint32_t* steps = reinterpret_cast<uint32_t*>(value ? kv.vs : kv.ks) + row * (D / 32);
  return {codes + (value ? value_word<D>(l, (int)row) : (l & 3) * (D / 32) + (l >> 2)), steps + (l >> 2)};
}

// The row of a slot and head; negative where nothing is written or read.
__device__ __forceinline__ long long row_of(const Kv4View& kv, int slot, int head, bool flag) {
  if (slot < 0) return -1;
  const int page = slot >> kv.page_shift;
  if (page >= kv.n_pages) {
    if (flag) atomicExch(kv.err, kErrSlot);
    return -1;
  }
  return (((long long)page * kv.hkv + head) << kv.page_shift) + (slot & ((1 << kv.page_shift) - 1));
}

template <typename E>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // of two values each; what is no number stays
  using V = typename Pair<E>::V;
  const V m = __hmin2_nan(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The codes of eight values of a group as a word (all of its lanes call), and its least value and step, given the values of its other lanes.
template <typename E>
__device__ __forceinline__ uint2 quantise8(const uint4& raw, bool value) {
  // the group's least value and largest, the latter as the least of the negatives
  constexpr uint32_t kSign = 0x80008000u;
  const uint32_t lo2 = min2<E>(min2<E>(raw.x, raw.y), min2<E>(raw.z, raw.w));
  const uint32_t hi2 = min2<E>(min2<E>(raw.x ^ kSign, raw.y ^ kSign), min2<E>(raw.z ^ kSign, raw.w ^ kSign));
  uint32_t ends = min2<E>(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
  ends = min2<E>(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
  ends = min2<E>(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
  const float lo = to_f32<E>(ends & 0xffff), hi = -to_f32<E>(ends >> 16), range = hi - lo;
  // The step is the rounding of a quotient.  A product is within 2^-23 of it: where the numbers 2^-22 around round alike,
  // so does the quotient.
  const float about = range * (1.f / 15.f);
  const uint32_t around = pack2<E>(about * (1.f - 2.384185791015625e-7f), about * (1.f + 2.384185791015625e-7f));
  uint32_t step_bits = around & 0xffff;
  if (around >> 16 != step_bits) step_bits = from_f32<E>(range / 15.f);
  float step = to_f32<E>(step_bits);
  // A top code that would stand for an infinity (of a value near the type's largest, and a step rounded up) takes the next
  // lower step.  That is enough: rounding moved the step by half a last place, so 15 of the lower one stay below the largest.
  constexpr float kOver = __is_same(E, __half) ? 65520.f : 3.39617752923046e38f;  // the least that rounds to infinity
  if (fmaf(15.f, step, lo) >= kOver && step < CUDART_INF_F) step = to_f32<E>(--step_bits);
  float x[8];
  unpack8<E>(raw, x);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  constexpr float kRound = 12582912.f;  // 1.5 2^23: a sum with it is rounded to a whole number, in its low bits
  float far = 0.f;                      // the largest distance from a whole number
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = fminf((x[k] - lo) * inv, 15.f), r = q + kRound;
    far = fmaxf(far, fabsf(q - (r - kRound)));
    w += (__float_as_uint(r) - __float_as_uint(kRound)) << 4 * k;
  }
  constexpr float kNear = 0.5f - 7.62939453125e-6f;
  if (far > kNear || !(inv < CUDART_INF_F)) {
    // halves themselves are common where the type has few bits: a value less half-and-codes of steps is then 0, exactly.
    // Past 14.5 a half stays the 15 that it was cut to: 15.5 comes of a step that lost a thirty-first, and is even at 16.
    far = 0.f;
    w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = x[k] - lo, q = fminf(d * inv, 15.f), half = fminf(floorf(q), 14.f) + 0.5f;
      const bool tie = fmaf(-half, step, d) == 0.f;
      const float r = (tie ? half : q) + kRound;
      far = fmaxf(far, tie ? 0.f : fabsf(q - (r - kRound)));
      w += (__float_as_uint(r) - __float_as_uint(kRound)) << 4 * k;
    }
    if (far > kNear || !(inv < CUDART_INF_F)) {
      w = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) w |= (uint32_t)min(max(__float2int_rn((x[k] - lo) / step), 0), 15) << 4 * k;
    }
  }
  if (!(step > 0.f)) w = 0;
  if (!value) {  // keys: in the order 0 4 2 6 1 5 3 7
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    w = __byte_perm(even | even >> 12, odd | odd >> 12, 0x5410);
  }
  if (!isfinite(lo) || !isfinite(hi) || !isfinite(step)) return make_uint2(0, 0x7fff7fff);  // the group holds what is no number
  return make_uint2(w, (ends & 0xffff) | step_bits << 16);
}

template <typename E>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t st, bool value) {
  const float least = to_f32<E>(st & 0xffff), step = to_f32<E>(st >> 16);
  if (!value) {  // back to the order of the values
    const uint32_t even = w & 0xffffu, odd = w >> 16;
    w = ((even | even << 12) & 0x0f0f0f0fu) | ((odd | odd << 12) & 0x0f0f0f0fu) << 4;
  }
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float c = __uint_as_float((w >> 4 * k & 15) | 0x4b000000u) - 8388608.f;  // 2^23 + c, less 2^23
    x[k] = fmaf(c, step, least);
  }
  return pack8<E>(x);
}

template <typename E, int D, bool LOAD, int U>
__global__ void __launch_bounds__(kRowThreads) row4_kernel(const Row4Params P) {
  behind_the_stream();
  let_next_start();
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const unsigned per = 2 * P.kv.hkv;  // rows a token: keys, then values
  const unsigned unit = (blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * (RPW * U) + lane / LPR;
  unsigned t = unit / per, h = unit - t * per;
  E* at[U];
  int slot[U], head[U];
  uint4 raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    head[i] = h;
    slot[i] = -1;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (t < (unsigned)P.T) {
      slot[i] = P.slots[t];
      const bool value = h >= (unsigned)P.kv.hkv;
      const long long ts = value ? P.v.token_stride : P.k.token_stride, hs = value ? P.v.head_stride : P.k.head_stride;
      at[i] = static_cast<E*>(value ? P.v.ptr : P.k.ptr) + t * ts + (value ? h - P.kv.hkv : h) * hs + 8 * l;
      if (!LOAD) raw[i] = __ldcs(reinterpret_cast<const uint4*>(at[i]));
    }
    h += RPW;
    while (h >= per) h -= per, ++t;
  }
  uint32_t w[U], st[U];
  Row4 place[U];
  bool live[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int value = head[i] >= P.kv.hkv;
    const long long row = row_of(P.kv, slot[i], value ? head[i] - P.kv.hkv : head[i], l == 0);
    live[i] = row >= 0;
    place[i] = row4<D>(P.kv, value, live[i] ? row : 0, l);
    if (LOAD && live[i]) w[i] = *place[i].codes, st[i] = *place[i].step;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const bool value = head[i] >= P.kv.hkv;
    if constexpr (LOAD) {
      if (live[i]) __stcs(reinterpret_cast<uint4*>(at[i]), values8<E>(w[i], st[i], value));
    } else {
      const uint2 r = quantise8<E>(raw[i], value);
      if (live[i]) {
        *place[i].codes = r.x;
        if ((l & 3) == 0) *place[i].step = r.y;
      }
    }
  }
}

template <typename E, int D, int U>
cudaError_t launch_unrolled(const Row4Params& P, bool load, cudaStream_t s) {
  constexpr int kRows = kRowThreads / 32 * (32 / (D / 8)) * U;
  const unsigned blocks = (unsigned)(((long long)P.T * 2 * P.kv.hkv + kRows - 1) / kRows);
  const Launch at(dim3(blocks), kRowThreads, 0, s);
  return load ? cudaLaunchKernelEx(&at.cfg, row4_kernel<E, D, true, U>, P) : cudaLaunchKernelEx(&at.cfg, row4_kernel<E, D, false, U>, P);
}
template <typename E, int D>
cudaError_t launch_rows(const Row4Params& P, bool load, cudaStream_t s) {
  // One step a warp below 2^20 values, four from there (append / load, us): of 2^18 values 1.6 / 1.5 and 2.9 / 2.0, of 2^20
  // 3.25 / 2.4 and 3.3 / 2.3, of 2^22 6.0 / 4.5 and 6.5 / 5.6, of 2^24 20.1 / 16.8 and 22.7 / 11.2, of 2^25 39.7 / 33.2 and
  // 37.1 / 21.0.
  const bool few = (long long)P.T * 2 * P.kv.hkv * D < (1 << 20);
  if (few) return launch_unrolled<E, D, 1>(P, load, s);
  // rows are counted in 32 bits: as many tokens a launch as stay below that
  const int most = (int)(0xfff00000u / (2u * P.kv.hkv));
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < P.T && e == cudaSuccess; t += most) {
    Row4Params Q = P;
    Q.T = P.T - t < most ? P.T - t : most;
    Q.slots += t;
    Q.k.ptr = static_cast<E*>(P.k.ptr) + t * P.k.token_stride;
    Q.v.ptr = static_cast<E*>(P.v.ptr) + t * P.v.token_stride;
    e = launch_unrolled<E, D, 4>(Q, load, s);
  }
  return e;
}

// ---- attention ------------------------------------------------------------------
//
// The streaming kernel of pw_attend.cu on codes.  Scores take the keys exactly:
//   q . k = sum over groups g of  step_g (q_g . c_g) + least_g sum(q_g),
// the first from products of fp16 queries with codes as fp16 numbers (c 2^-24:
// the bits of a code are a subnormal number; a code 4 bits up is 16 of it,
// which the queries of odd steps make up for), the second from one more product
// with sum(q_g) cut into three numbers of the heads' type.  For the range of
// the codes' products the queries are brought to a largest value of 2^8 .. 2^9
// a row by a power of two: that is exact but for values of less than 2^-18 of
// the row's largest, which are off by at most 2^-29 of it.  Values are turned
// into the heads' type, one rounding each.
//
// Both products have the cache as their first operand, 16 keys (or 16 of a
// head's values) by 8 query rows, so that up to eight rows a key head, which is
// what decode steps have, leave nothing idle and take 32 sums a lane; scores
// become the second product's operand by transposing 8 x 8 blocks of weights.
// A warp brings its own keys and values, 32 of a tile, by asynchronous copies
// of 16 bytes a lane into a ring of its own, one block ahead (tensor copies of
// small pages cost a producer warp more instructions than this costs all four).
// Bound by the instructions that turn codes into operands, ahead of the loads:
// 64 sequences of up to 8190 tokens, 8 key heads of 128, 337 MB in 95 to 99 us
// (3.5 TB/s), some 430 instructions for 16 keys and values (8 % less with the
// weights as one number, and errors of 1.5 times those of rounding the output
// alone, not 1.2 to 1.4).

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;                                // keys a tile
constexpr int kBlock = 32;                                // of them a warp has at a time
constexpr float kGrow = 8.f;

template <int D, int NT>
struct Cfg {
  static constexpr int CTAS = NT == 1 ? 4 : D == 64 ? 3 : 2;  // an SM
  static constexpr int CODES = kBlock * (D / 2), STEPS = kBlock * (D / 8);
  static constexpr int K_AT = 0, V_AT = CODES, KS_AT = 2 * CODES, VS_AT = KS_AT + STEPS;
  static constexpr int STAGE = 2 * (CODES + STEPS);       // of a warp
  static constexpr int STAGES = 2;
  static constexpr int JOIN_AT = kWarps * STAGES * STAGE;
  static constexpr int JOIN = NT * (D / 16) * 512;        // half the accumulators of two warps
  static constexpr int ML_AT = JOIN_AT + JOIN;
  static constexpr int SMEM = ML_AT + 2 * NT * 64;
};

__device__ __forceinline__ void compute_sync() { __syncthreads(); }

// N bytes of a lane, or zeros.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const char* from, bool live) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(N), "r"(live ? N : 0) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(const unsigned char* at, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}
__device__ __forceinline__ uint32_t lds32(const unsigned char* at) { return *reinterpret_cast<const uint32_t*>(at); }

// Rows and columns of an 8 x 8 block of 16-bit values exchanged (a row a group of four lanes).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t more) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(more));
  return d;
}

// The code pair at bits 4 n and 4 n + 16 of w as numbers, times step, plus least, rounded once.
template <typename E>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int n, uint32_t step2, uint32_t least2) {
  if constexpr (__is_same(E, __half)) {
    const uint32_t bits = and_or(n & 2 ? w >> 8 : w, n & 1 ? 0x00f000f0u : 0x000f000fu, 0x64006400u);  // 1024 + c (or 16 c)
    __half2 c = *reinterpret_cast<const __half2*>(&bits);
    c = n & 1 ? __hfma2(c, __float2half2_rn(0.0625f), __float2half2_rn(-64.f)) : __hadd2(c, __float2half2_rn(-1024.f));
    const __half2 r = __hfma2(c, *reinterpret_cast<const __half2*>(&step2), *reinterpret_cast<const __half2*>(&least2));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const uint32_t bits = and_or(w >> 4 * n, 0x000f000fu, 0x43004300u);  // 128 + c
    __nv_bfloat162 c = *reinterpret_cast<const __nv_bfloat162*>(&bits);
    c = __hadd2(c, __float2bfloat162_rn(-128.f));
    const __nv_bfloat162 r =
        __hfma2(c, *reinterpret_cast<const __nv_bfloat162*>(&step2), *reinterpret_cast<const __nv_bfloat162*>(&least2));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// NT row tiles of 8 a warp, MT such sets of rows; KS warps share the keys of a set.
template <typename E, int D, int NT, int MT>
__global__ void __launch_bounds__(kThreads, (Cfg<D, NT>::CTAS))
    attend4_kernel(const AttendParams P, const Kv4View kv, const AttendWork W) {
  using C = Cfg<D, NT>;
  constexpr int SET = 8 * NT, ROWS = SET * MT, KS = kWarps / MT, KPW = kTile / KS, NG = D / 32, VW = D / 64, MV = D / 16;
  using Walk = AttendWalk<ROWS, kTile, 1, 1, 2>;  // with 1 / 3 / 5 tiles a CTA at least one sequence of 19327 tokens took 8 / 0 / 10 % longer
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  behind_the_stream();
  const typename Walk::Mine mine = Walk::mine(P, W);
  Walk walk;
  walk.start(P, W, mine, reinterpret_cast<unsigned*>(smem + C::JOIN_AT));
  const int mt = warp % MT, ks = warp / MT, k0 = ks * KPW;

  // ---- the warp's blocks of 32 keys as one sequence, two ahead of the products: the pages of one, the copies of another.
  // A page's rows of codes are page_bytes, a head's among them head_bytes from its start; steps take a quarter. ----
  Walk ahead = walk;
  Piece lp = {};
  const int* table = nullptr;
  const int shift = P.kv.page_shift, mask = (1 << shift) - 1;
  const uint32_t page_bytes = (uint32_t)(P.kv.hkv << shift) * (D / 2);
  uint32_t head_bytes = 0;
  int lt = 0, lb = KPW, page = -1, first = 0;
  bool more = true;
  lp.tile1 = 0;
  auto look = [&]() {  // finds the next block with keys and reads its pages, a key a lane
    do {
      lb += kBlock;
      if (lb >= KPW) {
        lb = 0;
        if (++lt >= lp.tile1) {
          more = ahead.next(P, lp, table);
          if (!more) return;
          lt = lp.tile0;
          head_bytes = (uint32_t)(lp.head << shift) * (D / 2);
        }
      }
      first = key_tile<kTile>(lp, lt) * kTile + k0 + lb;
    } while (first >= lp.len);
    page = -1;
    if (first + lane < lp.len) {
      page = table[(first + lane) >> shift];
      if ((unsigned)page >= (unsigned)P.kv.n_pages) {
        atomicExch(P.kv.err, kErrPage);  // reads as zeros
        page = -1;
      }
    }
  };
  const uint32_t ring = base + warp * C::STAGES * C::STAGE;
  auto fetch = [&](int stage) {  // the copies of the block found last
    if (more) {
      const uint32_t to = ring + stage * C::STAGE;
      constexpr int PARTS = D / 32;  // 16 bytes of a row's codes each
#pragma unroll
      for (int j = 0; j < PARTS; ++j) {
        const int r = 32 / PARTS * j + lane / PARTS, pg = __shfl_sync(0xffffffffu, page, r);
        const uint64_t at = (uint64_t)(uint32_t)max(pg, 0) * page_bytes +
                            (head_bytes + ((first + r) & mask) * (D / 2) + 16 * (lane % PARTS));
        copy_async<16>(to + C::K_AT + 512 * j + 16 * lane, kv.k + at, pg >= 0);
        copy_async<16>(to + C::V_AT + 512 * j + 16 * lane, kv.v + at, pg >= 0);
      }
      const uint64_t at = (uint64_t)(uint32_t)max(page, 0) * (page_bytes / 4) + (head_bytes / 4 + ((first + lane) & mask) * (D / 8));
      copy_async<D / 8>(to + C::KS_AT + lane * (D / 8), kv.ks + at, page >= 0);
      copy_async<D / 8>(to + C::VS_AT + lane * (D / 8), kv.vs + at, page >= 0);
      look();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look();
  fetch(0);
  int stage = 0;
  Piece pc;
  const int* unused;

  // ---- compute warps ----
  const int g = lane >> 2, t4 = lane & 3;
  // Row m of eight keys is key order(m): the rows 2 t (and 2 t + 1) of values, which lanes t read at once, then lie in
  // different banks, and so do the keys that lanes g and g + 1 read.
  auto order = [](int m) { return m ^ (m >> 1 & 1); };
  const int key_g = order(g), val_a = order(2 * t4), val_b = order(2 * t4 + 1);
  uint32_t qf[NT][2 * NG][2], qs[NT][2];
  float rs[NT][2];  // the score of row 2 t4 + k in log2 units is rs times its product
  auto load_q = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = pc.row0 + mt * SET + 8 * j + g;
      const bool in = r < pc.nrows;
      const int tok = in ? r / P.G : 0, hd = in ? pc.head * P.G + r - tok * P.G : 0;
      const E* src = static_cast<const E*>(P.q.ptr) + (pc.tok0 + tok) * P.q.token_stride + hd * P.q.head_stride + 8 * t4;
      float x[NG][8], most = 0.f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        unpack8<E>(in ? *reinterpret_cast<const uint4*>(src + 32 * n) : make_uint4(0, 0, 0, 0), x[n]);
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(x[n][k]));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // a power of two that brings the largest to 2^8 .. 2^9, in two factors that are numbers
      const int e = most > 0.f && most < CUDART_INF_F ? 8 - ilogbf(most) : 0, e1 = e / 2, e2 = e - e1;
      const float f1 = ldexpf(1.f, e1), f2 = ldexpf(1.f, e2);
      const float mine_rs = ldexpf(ldexpf(P.scale * 1.4426950408889634f, -e1), -e2);
      rs[j][0] = __shfl_sync(0xffffffffu, mine_rs, 8 * t4);
      rs[j][1] = __shfl_sync(0xffffffffu, mine_rs, 8 * t4 + 4);
      float mine = 0.f;  // of the group t4
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[n][k] = x[n][k] * f1 * f2;
          sum += x[n][k];
        }
        qf[j][2 * n][0] = pack2<__half>(x[n][0], x[n][1]);
        qf[j][2 * n][1] = pack2<__half>(x[n][2], x[n][3]);
        qf[j][2 * n + 1][0] = pack2<__half>(x[n][4] * 0.0625f, x[n][5] * 0.0625f);
        qf[j][2 * n + 1][1] = pack2<__half>(x[n][6] * 0.0625f, x[n][7] * 0.0625f);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (n == t4) mine = sum;
      }
      // three parts of the heads' type; their products with the least values are exact
      const float a = to_f32<E>(from_f32<E>(mine)), b = to_f32<E>(from_f32<E>(mine - a)), c = mine - a - b;
      qs[j][0] = pack2<E>(a, b);
      qs[j][1] = pack2<E>(c, 0.f);
    }
  };
  bool have = walk.next(P, pc, unused);
  if (have) load_q();
  while (have) {
    const Piece cur = pc;
    const int ra = cur.row0 + mt * SET + 2 * t4;  // this lane's first row of a tile
    int vis[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) vis[j][k] = ra + 8 * j + k < cur.nrows ? cur.len - P.ql + 1 + (ra + 8 * j + k) / P.G : cur.len;
    const int sure = cur.len - P.ql + 1;  // keys below this are seen by every row
    float m[NT][2], l[NT][2], o[NT][MV][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m[j][0] = m[j][1] = -CUDART_INF_F, l[j][0] = l[j][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MV; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
    }

    for (int t = cur.tile0; t < cur.tile1; ++t) {
      const int tile_first = key_tile<kTile>(cur, t) * kTile + k0;
#pragma unroll 1
      for (int blk = 0; blk < KPW; blk += kBlock) {
        const int first = tile_first + blk;  // this warp's next 32 keys
        if (first >= cur.len) break;
        fetch(stage ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const unsigned char* at = smem + warp * C::STAGES * C::STAGE + stage * C::STAGE;
        stage ^= 1;
        float s[NT][2][4];                   // [row tile][16 keys]: keys order(g), + 8; rows 2 t4, + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int krow = 16 * h;
          uint32_t ka[NG], kb[NG], sa[NG], sb[NG];
          lds_words<NG>(at + C::K_AT + (krow + key_g) * (D / 2) + t4 * (NG * 4), ka);
          lds_words<NG>(at + C::K_AT + (krow + 8 + key_g) * (D / 2) + t4 * (NG * 4), kb);
          lds_words<NG>(at + C::KS_AT + (krow + key_g) * (D / 8), sa);
          lds_words<NG>(at + C::KS_AT + (krow + 8 + key_g) * (D / 8), sb);
          float p[NT][4];
#pragma unroll
          for (int j = 0; j < NT; ++j) p[j][0] = p[j][1] = p[j][2] = p[j][3] = 0.f;
          // least values of the group t4
          const uint32_t la = t4 < NG ? lds32(at + C::KS_AT + (krow + key_g) * (D / 8) + 4 * t4) : 0u;
          const uint32_t lb = t4 < NG ? lds32(at + C::KS_AT + (krow + 8 + key_g) * (D / 8) + 4 * t4) : 0u;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const uint32_t wa = ka[i], wb = kb[i], wa8 = wa >> 8, wb8 = wb >> 8;
            const uint32_t even[4] = {wa & 0x000f000fu, wb & 0x000f000fu, wa8 & 0x000f000fu, wb8 & 0x000f000fu};
            const uint32_t odd[4] = {wa & 0x00f000f0u, wb & 0x00f000f0u, wa8 & 0x00f000f0u, wb8 & 0x00f000f0u};
            const float fa = to_f32<E>(sa[i] >> 16), fb = to_f32<E>(sb[i] >> 16);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float acc[4];
              mma16816_first<__half>(acc, even, qf[j][2 * i][0], qf[j][2 * i][1]);
              mma16816<__half>(acc, odd, qf[j][2 * i + 1][0], qf[j][2 * i + 1][1]);
              p[j][0] = fmaf(fa, acc[0], p[j][0]);
              p[j][1] = fmaf(fa, acc[1], p[j][1]);
              p[j][2] = fmaf(fb, acc[2], p[j][2]);
              p[j][3] = fmaf(fb, acc[3], p[j][3]);
            }
          }
          const uint32_t least[4] = {__byte_perm(la, la, 0x1010), __byte_perm(lb, lb, 0x1010), la & 0xffffu, lb & 0xffffu};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816_first<E>(s[j][h], least, qs[j][0], qs[j][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][h][i] = fmaf(p[j][i], 16777216.f, s[j][h][i]);
          }
        }
        const bool edge = first + 32 > sure;
        // Weights as the second operand: keys 2 t4, + 1 (and + 8) of 16, row g.  Their rounding would add to the values' own,
        // so what a first number leaves of a weight goes into a second one and a second product.
        constexpr int TERMS = 2;
        uint32_t pf[NT][2][2][TERMS];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[j][h][i] *= rs[j][i & 1];
              if (edge && first + 16 * h + 8 * (i >> 1) + key_g >= vis[j][i & 1]) s[j][h][i] = -CUDART_INF_F;
              top[i & 1] = fmaxf(top[i & 1], s[j][h][i]);
            }
          // the sums' reference moves when a lane's maximum has passed it by 2^kGrow (weights stay below 2^(kShift + kGrow),
          // which fp16 holds, and nothing is lost: it cancels in o / l), and then to the row's maximum; rows that have not
          // grown stay, so that a query's bits do not go by keys that only the later ones beside it see
          float ref[2];
          bool grew = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            grew |= top[k] - kShift > m[j][k] + kGrow;
            ref[k] = m[j][k] == -CUDART_INF_F ? 0.f : m[j][k];
          }
          if (__any_sync(0xffffffffu, grew)) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], x));
              top[k] -= kShift;
              f[k] = 1.f;
              if (top[k] > m[j][k] + kGrow) {
                f[k] = ex2(m[j][k] - top[k]);
                m[j][k] = ref[k] = top[k];
              }
              l[j][k] *= f[k];
            }
#pragma unroll
            for (int i = 0; i < MV; ++i) {
              o[j][i][0] *= f[0], o[j][i][1] *= f[1];
              o[j][i][2] *= f[0], o[j][i][3] *= f[1];
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[j][h][i] = ex2(s[j][h][i] - ref[i & 1]);
              l[j][i & 1] += s[j][h][i];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float u = s[j][h][2 * b], v = s[j][h][2 * b + 1];
#pragma unroll
              for (int x = 0; x < TERMS; ++x) {
                const uint32_t w = pack2<E>(u, v);
                pf[j][h][b][x] = transpose8(w);
                if (x + 1 < TERMS) {
                  const float2 f = Pair<E>::up(*reinterpret_cast<const typename Pair<E>::V*>(&w));
                  u -= f.x, v -= f.y;
                }
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t vw[4][VW], vs[4];  // keys order(2 t4), order(2 t4 + 1), and those + 8
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int in8 = k & 1 ? val_b : val_a, row = 16 * h + 8 * (k >> 1) + in8;
            lds_words<VW>(at + C::V_AT + row * (D / 2) + value_word<D>(g * VW, in8) * 4, vw[k]);
            vs[k] = lds32(at + C::VS_AT + row * (D / 8) + (g * NG / 8) * 4);
            // nothing past the length counts, nor (of what only some rows see) what is no number: those rows get it below
            if (edge) {
              const int key = first + 16 * h + 8 * (k >> 1) + in8;
              if (key >= cur.len || (key >= sure && finite_bits<E>(vs[k]) != 0xffffffffu)) vs[k] = 0;
            }
          }
          const uint32_t least01 = __byte_perm(vs[0], vs[1], 0x5410), step01 = __byte_perm(vs[0], vs[1], 0x7632);
          const uint32_t least23 = __byte_perm(vs[2], vs[3], 0x5410), step23 = __byte_perm(vs[2], vs[3], 0x7632);
#pragma unroll
          for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t pick = half ? 0x7632 : 0x5410;
              const uint32_t x = __byte_perm(vw[0][w], vw[1][w], pick), y = __byte_perm(vw[2][w], vw[3][w], pick);
#pragma unroll
              for (int n = 0; n < 4; n += 2) {
                const uint32_t a[4] = {value_pair<E>(x, n, step01, least01), value_pair<E>(x, n + 1, step01, least01),
                                       value_pair<E>(y, n, step23, least23), value_pair<E>(y, n + 1, step23, least23)};
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int x = 0; x < TERMS; ++x) mma16816<E>(o[j][4 * w + 2 * half + n / 2], a, pf[j][h][0][x], pf[j][h][1][x]);
              }
            }
        }
        if (edge && P.ql > 1) {
#pragma unroll 1
          for (int key = max(sure, first); key < min(cur.len, first + 32); ++key) {
            // this lane's values of a row lie in one group
            if (finite_bits<E>(lds32(at + C::VS_AT + (key - first) * (D / 8) + (g * NG / 8) * 4)) == 0xffffffffu)
              continue;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (key < vis[j][k]) {
#pragma unroll
                  for (int i = 0; i < MV; ++i) o[j][i][k] = o[j][i][2 + k] = CUDART_NAN_F;
                }
          }
        }
        __syncwarp();  // the block's place is free
      }
    }

    have = walk.next(P, pc, unused);
    if (have) load_q();  // on their way while this piece's sums are stored

    // ---- join the warps that share keys, in halving steps ----
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[j][k] += __shfl_xor_sync(0xffffffffu, l[j][k], x);
#pragma unroll
    for (int step = KS / 2; step > 0; step >>= 1) {
      float fa[NT][2], fb[NT][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        compute_sync();  // the buffer is free
        if (ks >= step && ks < 2 * step) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int slot = ((ks - step) * MT + mt) * NT + j;
#pragma unroll
            for (int i = 0; i < MV / 2; ++i) {
              const float(&v)[4] = o[j][half * (MV / 2) + i];
              *reinterpret_cast<float4*>(smem + C::JOIN_AT + (slot * (MV / 2) + i) * 512 + lane * 16) = make_float4(v[0], v[1], v[2], v[3]);
            }
            if (half == 0 && g == 0)
              *reinterpret_cast<float4*>(smem + C::ML_AT + slot * 64 + t4 * 16) = make_float4(m[j][0], l[j][0], m[j][1], l[j][1]);
          }
        }
        compute_sync();
        if (ks < step) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int slot = (ks * MT + mt) * NT + j;
            if (half == 0) {
              const float4 y = *reinterpret_cast<const float4*>(smem + C::ML_AT + slot * 64 + t4 * 16);
              const float ym[2] = {y.x, y.z}, yl[2] = {y.y, y.w};
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float mm = fmaxf(m[j][k], ym[k]), rr = mm == -CUDART_INF_F ? 0.f : mm;
                fa[j][k] = ex2(m[j][k] - rr);
                fb[j][k] = ex2(ym[k] - rr);
                l[j][k] = l[j][k] * fa[j][k] + yl[k] * fb[j][k];
                m[j][k] = mm;
              }
            }
#pragma unroll
            for (int i = 0; i < MV / 2; ++i) {
              const float4 v = *reinterpret_cast<const float4*>(smem + C::JOIN_AT + (slot * (MV / 2) + i) * 512 + lane * 16);
              float(&x)[4] = o[j][half * (MV / 2) + i];
              x[0] = x[0] * fa[j][0] + v.x * fb[j][0];
              x[1] = x[1] * fa[j][1] + v.y * fb[j][1];
              x[2] = x[2] * fa[j][0] + v.z * fb[j][0];
              x[3] = x[3] * fa[j][1] + v.w * fb[j][1];
            }
          }
        }
      }
    }
    if (ks == 0) {
      const AttendPieces& to = W.suffix;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = ra + 8 * j + k;
          if (r >= cur.nrows) continue;
          float* dst;
          if (cur.first) {
            const int tok = r / P.G;
            const long long row = (long long)(cur.tok0 + tok) * P.kv.hq + cur.head * P.G + r - tok * P.G;
            dst = to.row_o + row * D;
            if (g == 0) to.row_ml[row] = make_float4(m[j][k], l[j][k], __int_as_float((int)blockIdx.x), __int_as_float(cur.last_cta));
          } else {
            const int slot = blockIdx.x * ROWS + r - cur.row0;
            dst = to.cta_o + (long long)slot * D;
            if (g == 0) to.cta_ml[slot] = make_float2(m[j][k], l[j][k]);
          }
          // rows g and g + 8 of the sums' tile i are values g D / 8 + 2 i and + 1
#pragma unroll
          for (int i = 0; i < MV; i += 2)
            *reinterpret_cast<float4*>(dst + g * (D / 8) + 2 * i) =
                make_float4(o[j][i][k], o[j][i][2 + k], o[j][i + 1][k], o[j][i + 1][2 + k]);
        }
    }
  }
  let_next_start();
}

// Rows of a tile: 8 or 16 where a key head has no more, else 32 or 64.
int attend4_rows(int G, int ql) {
  const long long rows = (long long)G * ql;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
int attend4_ctas(int rows, int d) {
  return sm_count() * (d == 64 ? rows == 8 ? Cfg<64, 1>::CTAS : Cfg<64, 2>::CTAS : rows == 8 ? Cfg<128, 1>::CTAS : Cfg<128, 2>::CTAS);
}

struct Layout4 {
  size_t row_o, row_ml, cta_o, cta_ml, total;
  Layout4(const KvView& kv, int B, int ql) {
    const int tile = attend4_rows(kv.hq / kv.hkv, ql);
    const size_t rows = (size_t)B * ql * kv.hq, slots = (size_t)attend4_ctas(tile, kv.d) * tile;
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t was = at;
      at += (n + 255) & ~(size_t)255;
      return was;
    };
    row_o = take(rows * kv.d * 4);
    row_ml = take(rows * 16);
    cta_o = take(slots * kv.d * 4);
    cta_ml = take(slots * 8);
    total = at;
  }
};

template <typename E, int D, int NT, int MT>
cudaError_t launch_stream(const AttendParams& P, const Kv4View& kv, const AttendWork& W, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const void* fn = reinterpret_cast<const void*>(attend4_kernel<E, D, NT, MT>);
  const cudaError_t e = ensure_smem(fn, C::SMEM);
  if (e != cudaSuccess) return e;
  const Launch at(dim3(attend4_ctas(8 * NT * MT, D)), kThreads, C::SMEM, s);
  return cudaLaunchKernelEx(&at.cfg, attend4_kernel<E, D, NT, MT>, P, kv, W);
}

template <typename E, int D>
cudaError_t launch_typed(const AttendParams& P, const Kv4View& kv, void* ws, cudaStream_t s) {
  const Layout4 L(P.kv, P.B, P.ql);
  char* w = static_cast<char*>(ws);
  AttendWork W = {};
  W.first = 0;
  W.count = P.B;
  W.behind = true;
  W.suffix.row_o = reinterpret_cast<float*>(w + L.row_o);
  W.suffix.row_ml = reinterpret_cast<float4*>(w + L.row_ml);
  W.suffix.cta_o = reinterpret_cast<float*>(w + L.cta_o);
  W.suffix.cta_ml = reinterpret_cast<float2*>(w + L.cta_ml);
  const int rows = attend4_rows(P.G, P.ql);
  const cudaError_t e = rows == 8    ? launch_stream<E, D, 1, 1>(P, kv, W, s)
                        : rows == 16 ? launch_stream<E, D, 2, 1>(P, kv, W, s)
                        : rows == 32 ? launch_stream<E, D, 2, 2>(P, kv, W, s)
                                     : launch_stream<E, D, 2, 4>(P, kv, W, s);
  if (e != cudaSuccess) return e;
  JoinShape shape = {};
  shape.rows[0] = shape.rows[1] = rows;
  shape.heads[0] = shape.heads[1] = 1;
  shape.ctas[0] = shape.ctas[1] = attend4_ctas(rows, D);
  return launch_join(P, W, shape, s);
}

}  // namespace

cudaError_t launch_rows4(const Row4Params& P, bool load, cudaStream_t s) {
  if (P.kv.dtype == PW_F16) return P.kv.d == 128 ? launch_rows<__half, 128>(P, load, s) : launch_rows<__half, 64>(P, load, s);
  return P.kv.d == 128 ? launch_rows<__nv_bfloat16, 128>(P, load, s) : launch_rows<__nv_bfloat16, 64>(P, load, s);
}

size_t attend4_ws_bytes(const KvView& kv, int B, int ql) { return B == 0 ? 0 : Layout4(kv, B, ql).total; }

cudaError_t launch_attend4(const AttendParams& P, const Kv4View& kv, void* ws, cudaStream_t s) {
  if (P.kv.dtype == PW_F16) return P.kv.d == 128 ? launch_typed<__half, 128>(P, kv, ws, s) : launch_typed<__half, 64>(P, kv, ws, s);
  return P.kv.d == 128 ? launch_typed<__nv_bfloat16, 128>(P, kv, ws, s) : launch_typed<__nv_bfloat16, 64>(P, kv, ws, s);
}

}  // namespace pw
