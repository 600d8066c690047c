// Attention over a paged cache for requests with many rows (prompts' chunks):
// 16-bit types, tensor cores with accumulators in tensor memory.
//
// The G query heads of a KV head are rows of the same tile, (token, head) pairs
// in that order: a tile holds 256 rows, 256 / G tokens, as two halves of 128
// that read the same keys.  Blocks of 128 keys and values pass through a ring
// of shared-memory stages, one TMA box a page and 64-column panel.  Per block
// and half
//   S = Q K^T        (tcgen05.mma, 128 x 128 fp32 in tensor memory)
//   P = 2^(S c - m)  (a thread a row: no exchange between threads)
//   O += P V         (tcgen05.mma with P read from tensor memory, where it has
//                     taken the place of S; O stays in tensor memory)
// One warp issues all products, one all loads, and a group of four warps does
// the softmax of each half.  The halves alternate: while one group works on its
// S, the tensor cores do the other half's two products.  They need 2 x 512
// cycles a half and block at head dim 128, the exponentials 1024 a half: both
// units are the bound, about equally.  Measured, 4K bf16 tokens over 12K (32 query
// heads on 8 of 128): 0.82 ms in a single call, list and joining included, 0.79 ms
// (1.22 PFLOP/s) this kernel's launch alone, the tensor cores busy 64% of the
// cycles; 0.80 to 0.90 ms one call after the other, as the card's power limit lowers
// the clock.  What is left is the chain of a half's block, whose parts cannot overlap
// for want of tensor memory: S is ready, softmax (1900 cycles of one warp a
// scheduler), the rest of P V and the next S.
//
// The running maximum is lazy (it moves when a score exceeds it by more than 8
// in base 2), so that O is rarely read back and rescaled; the sums use the
// weights before they are rounded to the values' type for the second product.
// That rounding, at most half a step a weight, is what the tensor cores' operand
// costs: a remainder as a second operand would make P V twice as long.  The error
// against 64 bits is 1.4 times that of fp32 weights (4K tokens above: 2.3e-3 and
// 1.7e-3 of the outputs, most of it the outputs' own rounding to bf16).  Keys that a
// row does not see have weight exactly 0; values behind a request's last token are
// zeroed in shared memory, and a row whose result is not finite is looked at again
// (mend_rows), since a value that it does not see may have been infinite or NaN.
#include <cudaTypedefs.h>

#include <cstring>
#include <type_traits>

#include "paged_work.cuh"
#include "stream_common.cuh"

namespace mp {
namespace paged {

constexpr int kHalf = 128;                         // rows of a half (MMA M)
constexpr int kKeys = kTilesBlock;                 // keys a block (MMA N, then K)
constexpr int kTilesThreads = 384;                 // 2 x 4 softmax warps, MMA, load, two idle
constexpr int kSoftRegs = 208, kRestRegs = 88;     // 256 * 208 + 128 * 88 <= 384 * 168
constexpr int kItems = 4;                          // items on their way from the loading warp to the others

struct Tiles {
  CUtensorMap tmQ, tmK, tmV;
  Attend a;
  Work w;
  int tile;                                        // tokens a tile
  int box;                                         // tokens a K or V box
};

template <int D>
struct TilesCfg {
  static constexpr int KT = D / 64;                                   // 64-column panels
  static constexpr int PANEL = kKeys * 128;                           // bytes of a panel of 128 rows
  static constexpr int STAGE = KT * PANEL;
  static constexpr int QB = D == 64 ? 2 : 1;                          // tiles of Q: the next item's where there is room
  static constexpr int NS = (224 * 1024 - 2 * QB * STAGE) / STAGE;
  static constexpr int OFF_Q = 0;                                     // [QB][2 halves][KT][128 rows][128 B]
  static constexpr int OFF_KV = 2 * QB * STAGE;                       // [NS][KT][128 rows][128 B]
  static constexpr int OFF_BAR = OFF_KV + NS * STAGE;
  static constexpr int BARS = 2 * NS + 9 + 2 * QB + 2 * kItems;
  static constexpr int OFF_ITEM = (OFF_BAR + BARS * 8 + 8 + 15) / 16 * 16;   // [kItems][16] words
  static constexpr int USED = OFF_ITEM + kItems * 64;
  static constexpr int SMEM = USED + 1024;
  static_assert(SMEM <= 232448, "shared memory of a block");
};

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
// Shared-memory descriptors, 128-byte swizzle, version 1.  K-major (Q, K): rows
// of 128 bytes, groups of 8 rows 1024 bytes apart; 16 elements along K are 32
// bytes.  MN-major (V as [keys][columns]): groups of 8 keys 1024 bytes apart,
// the next 64 columns a panel further; 16 keys are 2048 bytes.
// A descriptor is a constant high word and a low word that holds the address,
// so that stepping through an operand is one addition.
__device__ __forceinline__ uint32_t desc_hi(int stride) { return (uint32_t)(stride >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, int leading) {
  return (addr >> 4) | ((uint32_t)(leading >> 4) << 16);
}
template <typename T>
__device__ __forceinline__ uint32_t idesc(int n, bool v_major) {
  const uint32_t f = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | (v_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kHalf >> 4) << 24);
}
// Products and commits are issued by the one lane whose `one` is set, inside
// control flow that the whole warp shares: operands then stay in uniform
// registers (4K tokens over 12K: 1.38 M cycles, 1.50 M in a branch of one lane).
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
      " setp.ne.b32 q, %6, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d), "r"(a_lo),
      "r"(b_lo), "r"(hi), "r"(id), "n"(ADD ? 1 : 0), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t ta, uint32_t b_lo, uint32_t hi, uint32_t id,
                                       uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d), "r"(ta), "r"(b_lo), "r"(hi), "r"(id),
      "r"(add), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one;
}
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
// 32 columns of this thread's lane; the values are there after tmem_ld_wait
__device__ __forceinline__ void tmem_ld(uint32_t at, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// waits for this warp's loads; 32 loaded values pass through, so that no use of them can move before it
__device__ __forceinline__ void tmem_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tma_kv(uint32_t dst, const CUtensorMap* tm, int row, int panel, int head, int page,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(panel), "r"(head),
      "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* tm, int col, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(head), "r"(row), "r"(bar)
      : "memory");
}

// One look at a barrier's phase, without the suspension that mbar_try asks for
// (waking from it costs more than the usual wait here).
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits last two seconds at most, and longer only while rows are summed again
// (`turns` counts up then), which takes as long as they have keys.
__device__ __forceinline__ bool stuck(const int* turns, int& seen, int32_t* err) {
  const int now = *reinterpret_cast<const volatile int*>(turns);
  const bool same = now == seen;
  seen = now;
  if (same) set_error(err, E_TIMEOUT);
  return same;
}
__device__ __forceinline__ bool poll_long(uint32_t bar, uint32_t parity, const int* turns, int32_t* err) {
  long long end = sc::gtimer() + 2000000000LL;
  int seen = *reinterpret_cast<const volatile int*>(turns);
  for (uint32_t n = 1; !poll(bar, parity); ++n)
    if ((n & 255u) == 0u && sc::gtimer() > end) {
      if (stuck(turns, seen, err)) return false;
      end = sc::gtimer() + 2000000000LL;
    }
  return true;
}
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, const int* turns, int32_t* err) {
  int seen = *reinterpret_cast<const volatile int*>(turns);
  while (!sc::mbar_wait(bar, parity, sc::gtimer() + 2000000000LL))
    if (stuck(turns, seen, err)) return false;
  return true;
}

// ---------------------------------------------------------------------------
// A block's items: the units, or parts of units, of its share
// ---------------------------------------------------------------------------
struct Item {
  int b, h, i0;                        // request, KV head, first token of the tile in the request
  Request r;
  int key0, nb;                        // first key, blocks
  int from[2], to[2];                  // blocks that each half's rows can see ([0, 0): none)
  int lo, hi;                          // keys that any of its rows sees (the loading warp's alone)
  bool whole, head;                    // the unit is not cut; the share begins with this item
  int64_t next;
};

struct Walk {
  int64_t x, x1, start;
  int e;
};

// The keys [lo, hi) that the rows [i0, i1) of a request see together.  All lanes of a warp together.
__device__ __forceinline__ void seen_by(const Attend& a, const Request& r, int prefix, int i0, int i1, int& lo, int& hi) {
  lo = INT32_MAX;
  hi = 0;
  for (int i = i0 + (threadIdx.x & 31); i < i1; i += 32) {
    const Interval v = interval_of(a, r, prefix, i);
    if (v.hi > v.lo) {
      lo = min(lo, v.lo);
      hi = max(hi, v.hi);
    }
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
}

// The next item, or false at the share's end.  All lanes of a warp together.
__device__ __forceinline__ bool next_item(const Tiles& f, Walk& w, Item& it) {
  if (w.x >= w.x1) return false;
  const Attend& a = f.a;
  while (f.w.before[w.e + 1] * a.H <= w.x) ++w.e;
  const int64_t first = f.w.before[w.e] * a.H, n = f.w.before[w.e + 1] - f.w.before[w.e];
  const Entry en = f.w.entry[w.e];
  it.b = en.b;
  it.h = (int)((w.x - first) / n);
  const int64_t u0 = first + it.h * n, u1 = u0 + n, end = min(w.x1, u1);
  it.i0 = en.tile * f.tile;
  it.r = request_of(a, en.b);
  it.key0 = en.k0 + (int)(w.x - u0) * kKeys;
  it.nb = (int)(end - w.x);
  it.whole = w.x == u0 && end == u1;
  it.head = w.x == w.start;
  const int prefix = prefix_of(a, en.b);
  it.lo = INT32_MAX;
  it.hi = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int i0 = it.i0 + g * (f.tile / 2);
    int lo, hi;
    seen_by(a, it.r, prefix, i0, min(it.r.n, i0 + f.tile / 2), lo, hi);
    it.lo = min(it.lo, lo);
    it.hi = max(it.hi, hi);
    it.from[g] = hi > lo ? max(0, min(it.nb, (lo - it.key0) >> 7)) : 0;
    it.to[g] = hi > lo ? max(0, min(it.nb, (hi - it.key0 + kKeys - 1) >> 7)) : 0;
    if (it.to[g] <= it.from[g]) it.from[g] = it.to[g] = 0;
  }
  w.x = end;
  return true;
}

// A warp's rows whose sum is not NaN and whose numerator is not finite (mend_rows),
// out of line: they are rare and need registers.  `rows`: the lanes of such rows; i,
// hq, m, l: this lane's row; the keys [k0, k1) went into the products.  `slot`, `num`:
// the partial results' maximum and numerator of this warp's first row, or slot null.
template <typename T, int D>
__device__ __noinline__ void rows_again(const Attend& a, int b, const Request r, int tile0, int tile, uint32_t rows, int i,
                                        int hq, float m, float l, int k0, int k1, float* slot, float* num, int* turns) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, prefix = prefix_of(a, b), h = __shfl_sync(kFull, hq, __ffs(rows) - 1) / a.G;
  int low, high, common[E] = {};
  seen_by(a, r, prefix, tile0, min(r.n, tile0 + tile), low, high);
  // the keys that all of these rows see
  const bool mine = (rows >> lane & 1u) && l > 0.f;
  const Interval v = interval_of(a, r, prefix, mine ? i : 0);
  const int c0 = __reduce_max_sync(kFull, mine ? max(v.lo, k0) : k0),
            c1 = max(c0, __reduce_min_sync(kFull, mine ? min(v.hi, k1) : k1));
  if (__any_sync(kFull, mine)) odd_values<T, D>(a, b, h, c0, c1, low, high, common, turns);
  const uint32_t none = __ballot_sync(kFull, l == 0.f);
  auto result = [&](int hr, int ir) {
    return reinterpret_cast<T*>(a.O + (int64_t)(r.row0 + ir) * a.o_row_b + (int64_t)hr * a.o_head_b) + lane * E;
  };
  for (uint32_t x = rows & none; x; x &= x - 1) {          // zeros (a part that saw nothing: its numerator is not used)
    const int src = __ffs(x) - 1, ri = __shfl_sync(kFull, i, src), rh = __shfl_sync(kFull, hq, src);
    if (!slot)
#pragma unroll
      for (int e = 0; e < E; ++e) result(rh, ri)[e] = from_f32<T>(0.f);
  }
  rows &= ~none;
  while (rows) {
    Rows4 four;
    int src[4];
    float s[4][E] = {};
    four.n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!rows) continue;
      src[k] = __ffs(rows) - 1;
      rows &= rows - 1;
      four.i[k] = __shfl_sync(kFull, i, src[k]);
      four.hq[k] = __shfl_sync(kFull, hq, src[k]);
      four.base[k] = __shfl_sync(kFull, m + log2f(l), src[k]);
      four.n = k + 1;
#pragma unroll
      for (int e = 0; e < E; ++e)
        s[k][e] = slot ? num[src[k] * D + lane * E + e] : to_f32(result(four.hq[k], four.i[k])[e]);
    }
    const uint32_t again = mend_rows<T, D>(a, b, r, four, k0, k1, low, high, c0, c1, common, s, turns);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= four.n) continue;
      if (slot && (again >> k & 1u) && lane == 0) {
        slot[src[k]] = four.base[k];
        slot[2 * kHalf + src[k]] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (slot) num[src[k] * D + lane * E + e] = s[k][e];
        else result(four.hq[k], four.i[k])[e] = from_f32<T>(s[k][e]);
    }
  }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t*>(&d))
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return d;
}
// 2^x for x <= 127 by arithmetic: x = n + f with n the nearest integer (what
// adding 1.5 * 2^23 leaves in the low bits) and |f| <= 1/2, 2^f by the polynomial
// of degree 5 whose relative error is least on that interval (Remez exchange),
// 2^-22 with its roundings: the weights enter the row's sum, and with it the lse,
// before they are rounded to the values' type, so they are as good as the
// exponential unit's whatever that type is.  Below -126.5, minus infinity
// included, the result is 0; a NaN stays one.
__device__ __forceinline__ float2 exp2_pair(float2 x) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));   // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
  const float2 magic = make_float2(12582912.f, 12582912.f), back = make_float2(-12582912.f, -12582912.f);
  const float2 r = add2(x, magic), f = fma2(add2(r, back), make_float2(-1.f, -1.f), x);
  auto c = [](float v) { return make_float2(v, v); };
  float2 p = fma2(c(0.0013276472454890609f), f, c(0.009675540961325169f));
  p = fma2(p, f, c(0.05550713092088699f));
  p = fma2(p, f, c(0.24022120237350464f));
  p = fma2(p, f, c(0.6931469440460205f));
  p = fma2(p, f, c(1.0000001192092896f));
  const float2 scale = make_float2(__int_as_float((__float_as_int(r.x) << 23) + 0x3f800000),
                                   __int_as_float((__float_as_int(r.y) << 23) + 0x3f800000));
  return mul2(p, scale);
}
// cap_of for two scores in half the instructions: the loop around it has to stay in the instruction cache.
__device__ __forceinline__ float2 cap_pair(const Attend& a, float2 z) {
  auto c = [](float v) { return make_float2(v, v); };
  const float2 u = mul2(z, c(a.to_u)), x = mul2(u, u), e = mul2(u, c(2.f * kLog2e));
  float2 y = c(kTanh[5]);
#pragma unroll
  for (int q = 4; q >= 0; --q) y = fma2(y, x, c(kTanh[q]));
  const float2 near = mul2(mul2(z, c(a.to_z)), y), d = add2(make_float2(sc::ex2(e.x), sc::ex2(e.y)), c(1.f)),
               far = fma2(c(-2.f * a.cap2), make_float2(rcp(d.x), rcp(d.y)), c(a.cap2));
  return make_float2(select_near(u.x, near.x, far.x), select_near(u.y, near.y, far.y));
}
// kTanh's like on |u| <= 5/16, 2^-26: two terms fewer (odd chunks and decode
// tokens, scores capped at 30 over a window: 6% less time; where every |u| passes
// 3/4, the extra look costs 1.5%).
__device__ constexpr float kTanhNear[4] = {1.0f, -0.33332863450050354f, 0.1330905258655548f, -0.04992058873176575f};
template <int N>
__device__ __forceinline__ float top_of(const float* v) {
  float t[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int k = 4; k + 8 <= N; k += 8)
#pragma unroll
    for (int q = 0; q < 4; ++q) t[q] = max3(t[q], v[k + 2 * q], v[k + 2 * q + 1]);
#pragma unroll
  for (int k = (N - 4) / 8 * 8 + 4; k < N; ++k) t[k & 3] = fmaxf(t[k & 3], v[k]);
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

template <typename T>
__device__ __forceinline__ uint32_t to_pair(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return sc::pack_bf16(lo, hi);
  }
}

// CAP, BIAS: scores are capped, biased (or the scale is negative): the exponent is
// formed first, and its factor is 1.  A kernel for each, as their loops have to
// stay in the instruction cache.
template <typename T, int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kTilesThreads, 1) tiles_kernel(const __grid_constant__ Tiles f) {
  using C = TilesCfg<D>;
  constexpr int NS = C::NS, KT = C::KT;
  constexpr bool GEN = CAP || BIAS;
  const Attend& a = f.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (sc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = sc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t kv_full = sb + C::OFF_BAR, kv_empty = kv_full + 8 * NS, q_full = kv_empty + 8 * NS, q_empty = q_full + 8 * C::QB,
                 s_full = q_empty + 8 * C::QB, p_full = s_full + 16, o_full = p_full + 32, drain = o_full + 16,
                 item_full = drain + 8, item_empty = item_full + 8 * kItems;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + C::BARS * 8);
  int* turns = reinterpret_cast<int*>(tmem_slot + 1);    // counts up while rows are done again

  if (threadIdx.x == 0) {
    *turns = 0;
    for (int s = 0; s < NS; ++s) {
      sc::mbar_init(kv_full + 8 * s, 1);
      sc::mbar_init(kv_empty + 8 * s, 1);
    }
    for (int k = 0; k < C::QB; ++k) {
      sc::mbar_init(q_full + 8 * k, 1);
      sc::mbar_init(q_empty + 8 * k, 1);
    }
    sc::mbar_init(drain, 1);
    for (int k = 0; k < kItems; ++k) {
      sc::mbar_init(item_full + 8 * k, 1);
      sc::mbar_init(item_empty + 8 * k, 9);              // the softmax warps' and the issuing warp's
    }
    for (int g = 0; g < 2; ++g) {
      sc::mbar_init(s_full + 8 * g, 1);
      sc::mbar_init(p_full + 16 * g, 4);                 // the first 64 keys' weights, the last's
      sc::mbar_init(p_full + 16 * g + 8, 4);
      sc::mbar_init(o_full + 8 * g, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sc::smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int part = blockIdx.x;
  Item it;
  bool ok = true;
  auto wait_one = [&](uint32_t bar, uint32_t parity) {   // this thread alone
    return poll(bar, parity) || poll_long(bar, parity, turns, a.err);
  };
  auto wait = [&](uint32_t bar, uint32_t parity) {       // a warp together; after one failure at once
    ok = ok && (sc::mbar_try(bar, parity) || wait_long(bar, parity, turns, a.err));
    return ok = __all_sync(kFull, ok);
  };

  // the n-th item, as the loading warp has written it; false behind the last
  auto take = [&](uint32_t n) {
    const uint32_t k = n % kItems;
    if (!wait(item_full + 8 * k, (n / kItems) & 1u)) return false;
    const int4* p = reinterpret_cast<const int4*>(smem + C::OFF_ITEM + k * 64);
    const int4 x = p[0], y = p[1], z = p[2];
    const int flags = reinterpret_cast<const int*>(p)[12];
    it.b = x.x; it.h = x.y; it.i0 = x.z; it.key0 = x.w;
    it.r.row0 = y.x; it.r.n = y.y; it.r.len = y.z; it.nb = y.w;
    it.from[0] = z.x; it.to[0] = z.y; it.from[1] = z.z; it.to[1] = z.w;
    it.whole = flags & 1;
    it.head = flags & 2;
    __syncwarp();
    if (lane == 0) sc::mbar_arrive(item_empty + 8 * k);
    return (flags & 4) == 0;
  };

  if (warp < 8) {
    // ================= softmax: a thread a row =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    const int g = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + 128 * g + lanes, tO = tmem + 256 + 128 * g + lanes;
    const float c = a.to_z;
    const bool straight = !a.full && !a.prefix;          // no row sees a key behind its own
    uint32_t n_s = 0, n_o = 0, n_kv = 0;                 // phases of s_full and o_full, tiles that have passed the ring
    for (uint32_t n_item = 0; take(n_item); ++n_item) {
      // capped scores as s times a polynomial of s^2 (cap_of's), its coefficients made for the raw score, while no s^2 and
      // no coefficient passes fp32's range; cap_of otherwise
      float capped[6], near[4];
      {
        float by = a.to_z;
        asm volatile("" : "+f"(by));     // (made anew for each item: kept over all of them they cost registers elsewhere)
#pragma unroll
        for (int q = 0; q < 6; ++q, by *= a.to_u * a.to_u) {
          capped[q] = kTanh[q] * by;
          if (q < 4) near[q] = kTanhNear[q] * by;
        }
      }
      const float most = isfinite(capped[5]) ? kTanhMost : -1.f;
      const int i = it.i0 + g * (f.tile / 2) + row / a.G, hq = it.h * a.G + row % a.G;
      const bool valid = i < it.r.n;
      Interval v{0, INT32_MAX, 0};
      if (valid) v = interval_of(a, it.r, prefix_of(a, it.b), i);
      const float slope = BIAS && a.slopes ? __ldg(a.slopes + hq) * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int j = it.from[g]; j < it.to[g]; ++j) {
        if (!wait(s_full + 8 * g, n_s++ & 1u)) break;
        tc_after();
        const int kb = it.key0 + j * kKeys, lo = v.lo - kb, hi = v.hi - kb;
        const bool cut = __any_sync(kFull, v.lo > kb || v.hi < kb + kKeys);
        const float say = valid ? INFINITY : 0.f;
        // which of the 32 columns from 32 k on this row sees
        auto seen = [&](int k) {
          const int from = min(max(lo - 32 * k, 0), 32), to = min(max(hi - 32 * k, 0), 32);
          return (to == 32 ? ~0u : (1u << to) - 1u) & (from == 32 ? 0u : ~0u << from);
        };
        // values behind the last token become zeros before a product reads them (the second half's follows the first's)
        auto clear_tail = [&]() {
          if (kb + kKeys <= it.r.len || (g == 1 && j >= it.from[0] && j < it.to[0])) return true;
          const uint32_t at = n_kv + 2 * j + 1, st = at % NS;
          if (!wait(kv_full + 8 * st, (at / NS) & 1u)) return false;
          for (int x = max(0, it.r.len - kb) * 8 + row; x < kKeys * 8; x += 128)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
              *reinterpret_cast<uint4*>(smem + C::OFF_KV + st * C::STAGE + kt * C::PANEL + x * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          sc::fence_proxy_async();
          return true;
        };
        // the running maximum, in base 2, and with it the numerator, whose last product has ended with this S (a warp's
        // rows together: those that are none, whose scores come of anything, have no say)
        auto raise = [&](float mx) {
          if (!__any_sync(kFull, valid && mx > m + 8.f)) return;
          const float nm = fmaxf(m, mx), keep = m == -INFINITY ? 0.f : sc::ex2(m - nm);
          m = nm;
          l *= keep;
          if (j == it.from[g]) return;
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            float o[32];
            tmem_ld(tO + k, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] *= keep;
            tmem_st(tO + k, reinterpret_cast<const uint32_t*>(o));
          }
        };
        // 32 columns of P to columns [16 k, 16 k + 16) in the place of S; the product may begin with half of them
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](const float* z, int k, float2 mul, float2 sub) {
          uint32_t p[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float2 x = fma2(make_float2(z[2 * q], z[2 * q + 1]), mul, sub);
            // every fourth pair by arithmetic: the exponential unit alone needs 1024 cycles a half, as long as the
            // products (none: 846 us for 4K tokens over 12K in a single call, every eighth 837, fourth 817, third 950)
            const float2 w = (q & 3) == 3 ? exp2_pair(x) : make_float2(sc::ex2(x.x), sc::ex2(x.y));
            sum[q & 1] = add2(sum[q & 1], w);
            p[q] = to_pair<T>(w.x, w.y);
          }
          tmem_st16(tS + 16 * k, p);
        };
        auto hand_over = [&](int part_of_p) {
          tmem_st_wait();
          tc_before();
          __syncwarp();
          if (lane == 0) sc::mbar_arrive(p_full + 16 * g + 8 * part_of_p);
        };
        if constexpr (!GEN) {
          float s[128];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld(tS + 32 * k, s + 32 * k);
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld_wait(s + 32 * k);
          if (cut) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t keys = seen(k);
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (!(keys & 1u << q)) s[32 * k + q] = -INFINITY;
            }
          }
          raise(top_of<128>(s) * c);
          const float base = m == -INFINITY ? 0.f : -(m - kLift<T>);
          const float2 mul = make_float2(c, c), sub = make_float2(base, base);
          if (!clear_tail()) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            weigh(s + 32 * k, k, mul, sub);
            if (k & 1) hand_over(k >> 1);
          }
        } else {
          // 32 columns at a time: everything unrolled does not stay in the instruction cache and takes half as long
          // again.  The exponents go back to where the scores were.
          float mx = -INFINITY;
          const float ahead = (float)(v.pos - kb);
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            float z[32];
            tmem_ld(tS + 32 * k, z);
            tmem_ld_wait(z);
            if constexpr (CAP) {
              // the exponential (two results of a unit that the weights need too) only where some |u| of the warp's 32
              // columns is above 3/4; what memory happened to hold behind the last token has no say, nor has a row that is none
              const int held = it.r.len - kb - 32 * k;
              if (held < 32) {
#pragma unroll
                for (int q = 0; q < 32; ++q)
                  if (q >= held) z[q] = 0.f;
              }
              float t[4] = {};
#pragma unroll
              for (int q = 0; q < 32; q += 2) t[q / 2 & 3] = max3(t[q / 2 & 3], fabsf(z[q]), fabsf(z[q + 1]));
              const float top = fminf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), say),
                          far = top <= 0x1p60f ? top * fabsf(a.to_u) : 1.f;
              if (__all_sync(kFull, far <= fminf(most, 0.3125f))) {
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                  auto c = [](float w) { return make_float2(w, w); };
                  const float2 u = make_float2(z[q], z[q + 1]), x = mul2(u, u);
                  float2 y = fma2(c(near[3]), x, c(near[2]));
                  y = fma2(fma2(y, x, c(near[1])), x, c(near[0]));
                  y = mul2(y, u);
                  z[q] = y.x;
                  z[q + 1] = y.y;
                }
              } else if (__any_sync(kFull, far > most)) {
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                  const float2 y = cap_pair(a, make_float2(z[q], z[q + 1]));
                  z[q] = y.x;
                  z[q + 1] = y.y;
                }
              } else {
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                  auto c = [](float w) { return make_float2(w, w); };
                  const float2 u = make_float2(z[q], z[q + 1]), x = mul2(u, u);
                  float2 y = fma2(c(capped[5]), x, c(capped[4]));
#pragma unroll
                  for (int t = 3; t >= 0; --t) y = fma2(y, x, c(capped[t]));
                  y = mul2(y, u);
                  z[q] = y.x;
                  z[q + 1] = y.y;
                }
              }
            } else {
#pragma unroll
              for (int q = 0; q < 32; q += 2) {
                const float2 y = mul2(make_float2(z[q], z[q + 1]), make_float2(c, c));
                z[q] = y.x;
                z[q + 1] = y.y;
              }
            }
            if (BIAS && a.slopes) {
              const float d = ahead - (float)(32 * k);
              if (__all_sync(kFull, straight || d >= 31.f)) {    // no key behind a row, or none that it sees
                const float2 at = make_float2(-slope * d, -slope * d), by = make_float2(slope, slope);
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                  const float2 y = add2(make_float2(z[q], z[q + 1]), fma2(make_float2((float)q, (float)(q + 1)), by, at));
                  z[q] = y.x;
                  z[q + 1] = y.y;
                }
              } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) z[q] = fmaf(-slope, fabsf(d - (float)q), z[q]);
              }
            }
            if (cut) {
              const uint32_t keys = seen(k);
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (!(keys & 1u << q)) z[q] = -INFINITY;
            }
            mx = fmaxf(mx, top_of<32>(z));
            tmem_st(tS + 32 * k, reinterpret_cast<const uint32_t*>(z));
          }
          tmem_st_wait();
          raise(mx);
          const float base = m == -INFINITY ? 0.f : -(m - kLift<T>);
          const float2 mul = make_float2(1.f, 1.f), sub = make_float2(base, base);
          if (!clear_tail()) break;
          float z0[32], z1[32];
          tmem_ld(tS, z0);
#pragma unroll 1
          for (int k = 0; k < 4; k += 2) {
            tmem_ld_wait(z0);
            tmem_ld(tS + 32 * k + 32, z1);
            weigh(z0, k, mul, sub);
            tmem_ld_wait(z1);
            if (k == 0) tmem_ld(tS + 64, z0);
            weigh(z1, k + 1, mul, sub);
            hand_over(k >> 1);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // --- the half's result
      const bool none = it.to[g] == it.from[g];
      float* slot = f.w.part + (2 * (int64_t)part + (it.head ? 0 : 1)) * (int64_t)(2 * kHalf) * (2 + D);
      const int cell = g * kHalf + row;
      float* num = slot + 2 * (2 * kHalf) + (int64_t)cell * D;
      T* out = reinterpret_cast<T*>(a.O + (int64_t)(it.r.row0 + i) * a.o_row_b + (int64_t)hq * a.o_head_b);
      if (!none) {
        if (!wait(o_full + 8 * g, n_o++ & 1u)) break;
        tc_after();
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      bool finite = true;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        __syncwarp();
        if (none) {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0.f;
        } else {
          tmem_ld(tO + k, o);
          tmem_ld_wait(o);
        }
#pragma unroll
        for (int q = 0; q < 32; ++q) finite &= fabsf(o[q]) <= 3.4028235e38f;
        if (!valid) continue;
        if (it.whole) {
#pragma unroll
          for (int q = 0; q < 32; q += 8) {
            uint4 w;
            w.x = to_pair<T>(o[q] * inv, o[q + 1] * inv);
            w.y = to_pair<T>(o[q + 2] * inv, o[q + 3] * inv);
            w.z = to_pair<T>(o[q + 4] * inv, o[q + 5] * inv);
            w.w = to_pair<T>(o[q + 6] * inv, o[q + 7] * inv);
            *reinterpret_cast<uint4*>(out + k + q) = w;
          }
        } else {
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(num + k + q) = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
        }
      }
      tc_before();
      if (valid) {
        if (it.whole) {
          if (a.lse)
            a.lse[(int64_t)(it.r.row0 + i) * a.H * a.G + hq] = l == 0.f ? -INFINITY : (m - kLift<T> + log2f(l)) / kLog2e;
        } else {
          slot[cell] = l == 0.f ? -INFINITY : m - kLift<T>;
          slot[2 * kHalf + cell] = l;
        }
      }
      const uint32_t again = __ballot_sync(kFull, valid && !finite && l == l);       // (not where the sum is NaN)
      __syncwarp();                    // what the rows' own threads have written is there before another overwrites it
      if (again)
        rows_again<T, D>(a, it.b, it.r, it.i0, f.tile, again, i, hq, m - kLift<T>, l, it.key0 + it.from[g] * kKeys,
                         it.key0 + it.to[g] * kKeys, it.whole ? nullptr : slot + cell - lane, num - (int64_t)lane * D, turns);
      if (it.to[0] > it.from[0] || it.to[1] > it.from[1]) n_kv += 2 * it.nb;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRestRegs));
    if (warp == 8) {
      // ================= products (one thread) =================
      // This thread must not fall behind: the tensor cores' queue is short, and what it spends on waits and addresses
      // beyond a product's own time they spend idle (with votes of the warp at each wait and descriptors made
      // anew it took 4000 cycles a block, of which the products are 2048).
      const uint32_t one = elect_one();
      const uint32_t hi = desc_hi(1024), id_s = idesc<T>(kKeys, false), id_o = idesc<T>(D, true);
      const uint32_t q_lo = desc_lo(sb + C::OFF_Q, 16), k_lo = desc_lo(sb + C::OFF_KV, 16),
                     v_lo = desc_lo(sb + C::OFF_KV, C::PANEL);
      const uint32_t acc = __shfl_sync(kFull, tmem, 0);
      uint32_t n_q = 0, n_p0 = 0, n_p1 = 0;
      uint32_t ks = 0, kp = 0;                           // stage and phase of the next K; its V is the next tile
      for (uint32_t n_item = 0; take(n_item); ++n_item) {
        if (it.to[0] == it.from[0] && it.to[1] == it.from[1]) continue;
        const int from0 = __shfl_sync(kFull, it.from[0], 0), to0 = __shfl_sync(kFull, it.to[0], 0),
                  from1 = __shfl_sync(kFull, it.from[1], 0), to1 = __shfl_sync(kFull, it.to[1], 0),
                  nb = __shfl_sync(kFull, it.nb, 0);
        uint32_t vs = 0, vp = 0;                         // of the V whose products come next
        const uint32_t qb = n_q % C::QB;
        auto scores = [&](uint32_t g) {                  // S = Q K^T
          tc_after();
          const uint32_t q = q_lo + (2 * qb + g) * (C::STAGE >> 4), k = k_lo + ks * (C::STAGE >> 4);
          mma_ss<false>(one, acc + 128 * g, q, k, hi, id_s);
#pragma unroll
          for (int i = 1; i < D / 16; ++i)
            mma_ss<true>(one, acc + 128 * g, q + (i >> 2) * (C::PANEL >> 4) + (i & 3) * 2,
                         k + (i >> 2) * (C::PANEL >> 4) + (i & 3) * 2, hi, id_s);
          commit(one, s_full + 8 * g);
        };
        auto output = [&](uint32_t g, uint32_t& n, bool first, bool last) {  // O += P V
          const uint32_t v = v_lo + vs * (C::STAGE >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait_one(p_full + 16 * g + 8 * h, n & 1u)) return false;
            tc_after();
#pragma unroll
            for (int i = h * (kKeys / 32); i < (h + 1) * (kKeys / 32); ++i)
              mma_ts(one, acc + 256 + 128 * g, acc + 128 * g + 8 * i, v + i * (2048 >> 4), hi, id_o, !first || i > 0);
          }
          ++n;
          if (last) commit(one, o_full + 8 * g);
          return true;
        };
        ok = wait_one(q_full + 8 * qb, (n_q / C::QB) & 1u);
        for (int j = 0; j <= nb && ok; ++j) {
          // a stage is waited for as late and released as early as its products allow
          if (j > 0 && !(ok = wait_one(kv_full + 8 * vs, vp))) break;
          if (j > from0 && j <= to0 && !(ok = output(0, n_p0, j - 1 == from0, j == to0))) break;
          if (j < nb && !(ok = wait_one(kv_full + 8 * ks, kp))) break;
          if (j >= from0 && j < to0) scores(0);
          if (j > from1 && j <= to1 && !(ok = output(1, n_p1, j - 1 == from1, j == to1))) break;
          if (j > 0) commit(one, kv_empty + 8 * vs);
          if (j >= from1 && j < to1) scores(1);
          if (j < nb) {
            commit(one, kv_empty + 8 * ks);
            vs = ks + 1;
            vp = kp;
            if (vs == NS) { vs = 0; vp ^= 1u; }
            ks = vs + 1;
            kp = vp;
            if (ks == NS) { ks = 0; kp ^= 1u; }
          } else {
            commit(one, q_empty + 8 * qb);
          }
        }
        ++n_q;
        ok = __all_sync(kFull, ok);
      }
      if (!ok) {                                         // gave up: products under way end before the memory is freed
        commit(one, drain);
        sc::mbar_wait(drain, 0, sc::gtimer() + 200000000LL);
      }
    } else if (warp == 9) {
      // ================= loads =================
      // It runs ahead of the others and finds the items for them: the chain of loads that this takes would
      // otherwise lie between two items of each.
      uint32_t n_kv = 0, n_q = 0, issued = 0;
      const int pg = 1 << a.page_shift, boxes = kKeys / f.box;
      Walk walk;
      walk.x = walk.start = f.w.edge[part];
      walk.x1 = f.w.edge[part + 1];
      walk.e = f.w.edge_entry[part];
      uint32_t n_item = 0;
      auto publish = [&](Item& x) {                      // finds the next item and hands it on
        const uint32_t slot = n_item % kItems;
        const bool more = next_item(f, walk, x);
        if (n_item >= kItems && !wait(item_empty + 8 * slot, (n_item / kItems - 1) & 1u)) return false;
        ++n_item;
        if (lane == 0) {
          int4* p = reinterpret_cast<int4*>(smem + C::OFF_ITEM + slot * 64);
          if (more) {
            p[0] = make_int4(x.b, x.h, x.i0, x.key0);
            p[1] = make_int4(x.r.row0, x.r.n, x.r.len, x.nb);
            p[2] = make_int4(x.from[0], x.to[0], x.from[1], x.to[1]);
          }
          p[3].x = more ? (x.whole ? 1 : 0) | (x.head ? 2 : 0) : 4;
          sc::mbar_arrive(item_full + 8 * slot);
        }
        __syncwarp();
        return more;
      };
      for (bool more = publish(it); more && ok;) {
        const bool used[2] = {it.to[0] > it.from[0], it.to[1] > it.from[1]};
        if (!used[0] && !used[1]) {
          more = publish(it);
          continue;
        }
        const uint32_t qb = n_q % C::QB;
        if (n_q >= C::QB && !wait(q_empty + 8 * qb, (n_q / C::QB - 1) & 1u)) break;
        ++n_q;
        if (lane == 0) {
          sc::mbar_arrive_tx(q_full + 8 * qb, (used[0] ? C::STAGE : 0) + (used[1] ? C::STAGE : 0));
          for (int g = 0; g < 2; ++g)
            for (int k = 0; k < KT && used[g]; ++k)
              tma_q(sb + C::OFF_Q + (2 * qb + g) * C::STAGE + k * C::PANEL, &f.tmQ, 64 * k, it.h * a.G,
                    it.r.row0 + it.i0 + g * (f.tile / 2), q_full + 8 * qb);
        }
        for (int j = 0; j < it.nb && ok; ++j) {
          // a lane a box: its keys' page (a page behind the pool's last, which reads as zeros, in the place of a bad one,
          // so that nothing of another request is read; a neighbour that is seen in the place of one that is not, whose
          // table entry need not be valid any more)
          const int key = it.key0 + j * kKeys + lane * f.box;
          const bool mine = lane < boxes && key < it.r.len;
          const int known = min(max(key, it.lo), it.hi - 1);
          int page = mine ? page_of(a, it.b, known) : 0;
          if (page < 0) page = a.num_pages;
          const uint32_t bytes = __popc(__ballot_sync(kFull, mine)) * (uint32_t)f.box * D * 2;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t t = n_kv + 2 * j + kv, s = t % NS;
            if (t >= NS && !wait(kv_empty + 8 * s, (t / NS - 1) & 1u)) break;
            if (lane == 0) sc::mbar_arrive_tx(kv_full + 8 * s, bytes);
            __syncwarp();
            issued = t + 1;
            if (mine) {
              const uint32_t dst = sb + C::OFF_KV + s * C::STAGE + lane * f.box * 128;
              for (int k = 0; k < (f.box == kKeys ? 1 : KT); ++k)
                tma_kv(dst + k * C::PANEL, kv ? &f.tmV : &f.tmK, key & (pg - 1), k, it.h, page, kv_full + 8 * s);
            }
          }
        }
        if (!ok) break;
        n_kv += 2 * it.nb;
        more = publish(it);
      }
      // copies under way land before the block ends (only after a wait that gave up are there any left)
      if (!ok)
        for (uint32_t t = issued > NS ? issued - NS : 0; t < issued; ++t)
          if (!sc::mbar_wait(kv_full + 8 * (t % NS), (t / NS) & 1u, sc::gtimer() + 200000000LL)) break;
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 8) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename T, int D, bool CAP, bool BIAS>
static cudaError_t launch_tiles_t(const Tiles& f, cudaStream_t st) {
  using C = TilesCfg<D>;
  auto kern = tiles_kernel<T, D, CAP, BIAS>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)f.w.parts);
  cfg.blockDim = dim3(kTilesThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> allowed{0};
  return launch_large(kern, cfg, f, f.a.device, allowed, C::SMEM);
}

template <typename T, int D>
static cudaError_t launch_tiles(const Tiles& f, cudaStream_t st) {
  if (f.a.cap > 0.f) return f.a.slopes ? launch_tiles_t<T, D, true, true>(f, st) : launch_tiles_t<T, D, true, false>(f, st);
  return f.a.slopes || f.a.scale < 0.f ? launch_tiles_t<T, D, false, true>(f, st) : launch_tiles_t<T, D, false, false>(f, st);
}

// Q as [row][head][d]: a box is one KV head's query heads of kHalf / G rows, 64
// columns.  Rows past the tensor's end read as zeros.
static bool encode_q(CUtensorMap* tm, const Attend& a, int dtype, int D) {
  auto fn = map_encoder();
  if (!fn) return false;
  cuuint64_t gdim[3] = {(cuuint64_t)D, (cuuint64_t)a.H * a.G, (cuuint64_t)a.rows};
  cuuint64_t gstride[2] = {(cuuint64_t)a.q_head_b, (cuuint64_t)a.q_row_b};
  cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)(kHalf / a.G)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, dtype == MP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<char*>(a.Q), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t attend_tiles(const Attend& a, const mp_paged_cache& c, const Work& w, cudaStream_t st) {
  Tiles f{};
  const int D = c.cfg.head_dim;
  memcpy(&f.tmK, c.maps + 16 * MAP_KPAGE, sizeof(CUtensorMap));
  memcpy(&f.tmV, c.maps + 16 * MAP_VPAGE, sizeof(CUtensorMap));
  if (!encode_q(&f.tmQ, a, c.cfg.dtype, D)) return cudaErrorNotSupported;
  f.a = a;
  f.w = w;
  f.tile = tiles_tokens(a.G);
  f.box = c.cfg.page_tokens < kKeys ? c.cfg.page_tokens : kKeys;
  cudaError_t e = launch_work(a, w, f.tile, kKeys, st);
  if (e != cudaSuccess) return e;
  if (c.cfg.dtype == MP_F16) e = D == 128 ? launch_tiles<__half, 128>(f, st) : launch_tiles<__half, 64>(f, st);
  else e = D == 128 ? launch_tiles<__nv_bfloat16, 128>(f, st) : launch_tiles<__nv_bfloat16, 64>(f, st);
  if (e != cudaSuccess) return e;
  return launch_join(a, w, c.cfg.dtype, D, f.tile, 2 * kHalf, false, st);
}

}  // namespace paged
}  // namespace mp
