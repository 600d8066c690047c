// The work list of a split attention call and its share-out.
//
// An entry is a tile of one request's rows; its cost is the number of key
// blocks that its rows can see.  With H heads, the units (entry, head) laid
// end to end, blocks inside, are one line of W blocks, of which part c of N
// gets [c W / N, (c + 1) W / N): equal shares whatever the requests' lengths,
// most units whole, and those of up to kWholeBlocks blocks always (an edge inside
// one moves to its nearer end).  A unit cut between parts leaves a partial result
// in each (two at most a part: the unit its share begins inside of, and the one it
// ends inside of), and a second kernel joins them in the parts' order, so the
// result does not depend on timing.
#pragma once

#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "paged_common.cuh"
#include "stream_common.cuh"

namespace mp {
namespace paged {

struct Entry {
  int32_t b, tile, k0, n;            // request, tile of its rows, first key (a block's), blocks
};

struct Work {
  int32_t* count;                    // entries; 8 bytes on, as 64 bits: blocks of all, for one head
  int64_t* before;                   // [entries + 1] blocks of the entries before, for one head
  Entry* entry;                      // [entries]
  int64_t* edge;                     // [parts + 1] where each part begins (the list kernel's)
  int32_t* edge_entry;               // [parts + 1] and in which entry
  float* part;                       // [2 parts][rows (2 + D)]: maxima, sums, numerators
  int32_t parts;                     // parts launched
  int32_t least;                     // blocks a part gets at least, as far as there are that many
};

__device__ __forceinline__ int64_t share(int64_t W, int N, int c) { return W * c / N; }
// parts in use: as many as launched, fewer when shares would be smaller than `least`
__device__ __forceinline__ int parts_used(const Work& w, int64_t W) {
  const int64_t n = (W + w.least - 1) / w.least;
  return (int)(n < w.parts ? (n < 1 ? 1 : n) : w.parts);
}
// the last part whose share begins at or before block x
__device__ __forceinline__ int part_of(int64_t W, int N, int64_t x) {
  int c = (int)(x * N / W);
  while (c + 1 < N && share(W, N, c + 1) <= x) ++c;
  while (c > 0 && share(W, N, c) > x) --c;
  return c;
}
constexpr int kWholeBlocks = 4;      // two joined parts of a unit cost more than so many blocks
// the entry that block x of the line belongs to
__device__ __forceinline__ int entry_of(const int64_t* before, int E, int H, int64_t x) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] * H <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// the same by the lanes of a warp together, 32 places a round
__device__ __forceinline__ int entry_of_warp(const int64_t* before, int E, int H, int64_t x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = E;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const int hits = __popc(__ballot_sync(kFull, lane * step < n && before[at] * H <= x));
    lo += (hits - 1) * step;
    n = min(step, n - (hits - 1) * step);
  }
  return lo;
}

// An entry's blocks from the keys [lo, hi) that its rows see together.  Rows
// that see nothing cost a block: their zeros are written.
__device__ __forceinline__ void set_span(Entry& x, int lo, int hi, int block) {
  x.k0 = hi > lo ? lo / block * block : 0;
  x.n = hi > lo ? (hi - x.k0 + block - 1) / block : 1;
}
__device__ __forceinline__ void span_of(const Attend& a, const Request& r, int b, int i0, int i1, int block, Entry& x) {
  const int prefix = prefix_of(a, b);
  int lo = INT32_MAX, hi = 0;
  if (a.first_key) {                   // in any order: every row counts
    for (int i = i0; i < i1; ++i) {
      const Interval v = interval_of(a, r, prefix, i);
      if (v.hi > v.lo) { lo = min(lo, v.lo); hi = max(hi, v.hi); }
    }
  } else if (i0 < i1) {                // the ends move with the rows
    const Interval v = interval_of(a, r, prefix, i0), z = interval_of(a, r, prefix, i1 - 1);
    lo = min(v.lo, z.lo);
    hi = max(v.hi, z.hi);
  }
  set_span(x, lo, hi, block);
}

// The end of a block's work on a unit whose keys its warps have shared out: the
// warps' states (ml: [warps][2][ROWS] maxima and sums; num: numerators, PITCH
// floats a row, `stride` floats a warp) become the result, a partial result in
// the scratch, or, in a cluster that shares the unit, the cluster's result.
struct Settle {
  int b, h, i0, cells, key0, key1;     // request, KV head, first token, (token, head) rows, keys
  Request r;
  int cluster, part;                   // blocks of the cluster (0: none), this block's place
  bool whole;                          // the unit is this block's alone
  float* slot;                         // of a partial result
};
// Shared words that settle needs: rows to be looked at again, and the keys that the
// unit's rows see together (written before its keys are worked on: there they cost
// no registers).
template <int ROWS>
struct Again {
  int bad[ROWS], low, high;
};
// The factor of a part with maximum mp where all have m: never 0 for a part that saw
// keys, so that its infinities and NaN stay (of finite numerators less than 2^-21 is
// left then).
__device__ __forceinline__ float part_factor(float mp, float m) {
  return mp == -INFINITY ? 0.f : fmaxf(exp2f(mp - m), 0x1p-149f);
}
template <typename T>
__device__ __forceinline__ void settle_final(const Attend& a, const Settle& s, int row, int c, float m, float l, float v) {
  const bool none = l == 0.f;
  const int64_t t = s.r.row0 + s.i0 + row / a.G, hq = s.h * a.G + row % a.G;
  reinterpret_cast<T*>(a.O + t * a.o_row_b + hq * a.o_head_b)[c] = from_f32<T>(none ? 0.f : v / l);
  if (a.lse && c == 0) a.lse[t * a.H * a.G + hq] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
}
template <typename T, int D, int ROWS, int PITCH>
__device__ __forceinline__ void settle_put(const Attend& a, const Settle& s, float* num, float* unit, int row, int c, float m,
                                           float l, float v) {
  if (s.cluster) {                     // warp 0's numerators are replaced, each by the thread that read it
    num[row * PITCH + c] = v;
    if (c == 0) { unit[row] = m; unit[ROWS + row] = l; }
  } else if (s.whole) {
    settle_final<T>(a, s, row, c, m, l, v);
  } else {
    s.slot[2 * ROWS + row * D + c] = v;
    if (c == 0) { s.slot[row] = m; s.slot[ROWS + row] = l; }
  }
}
// Rows with a finite sum and a numerator that is not (mend_rows): out of line, for the registers' sake.
template <typename T, int D, int ROWS, int PITCH, int WARPS>
__device__ __noinline__ void settle_again(const Attend& a, const Settle& s, const float* ml, float* num, int stride,
                                          float* unit, const Again<ROWS>* again) {
  constexpr int E = D / 32;
  const int* bad = again->bad;
  const int low = again->low, high = again->high;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, prefix = prefix_of(a, s.b);
  // the keys that all of this warp's rows see
  int c0 = s.key0, c1 = s.key1, common[E] = {};
  bool any = false;
  for (int row = warp; row < s.cells; row += WARPS)
    if (bad[row]) {
      const Interval v = interval_of(a, s.r, prefix, s.i0 + row / a.G);
      c0 = max(c0, v.lo);
      c1 = min(c1, v.hi);
      any = true;
    }
  if (!any) return;
  c1 = max(c0, c1);
  odd_values<T, D>(a, s.b, s.h, c0, c1, low, high, common, nullptr);
  for (int next = warp; next < s.cells;) {
    Rows4 rows;
    int row[4];
    float m[4], l[4], v[4][E] = {};
    rows.n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      while (next < s.cells && !bad[next]) next += WARPS;
      if (next >= s.cells) continue;
      row[k] = next;
      m[k] = -INFINITY;
      l[k] = 0.f;
      for (int w = 0; w < WARPS; ++w) m[k] = fmaxf(m[k], ml[(w * 2) * ROWS + next]);
      for (int w = 0; w < WARPS; ++w) {
        const float mw = ml[(w * 2) * ROWS + next], f = mw == -INFINITY ? 0.f : exp2f(mw - m[k]);
        l[k] = fmaf(f, ml[(w * 2 + 1) * ROWS + next], l[k]);
#pragma unroll
        for (int e = 0; e < E; ++e)    // (in a cluster the first warp's have been replaced by the sum)
          if (!s.cluster) v[k][e] = fmaf(f, num[w * stride + next * PITCH + lane * E + e], v[k][e]);
          else if (w == 0) v[k][e] = num[next * PITCH + lane * E + e];
      }
      rows.i[k] = s.i0 + next / a.G;
      rows.hq[k] = s.h * a.G + next % a.G;
      rows.base[k] = m[k] + log2f(l[k]);
      rows.n = k + 1;
      next += WARPS;
    }
    if (rows.n == 0) break;
    const uint32_t summed = mend_rows<T, D>(a, s.b, s.r, rows, s.key0, s.key1, low, high, c0, c1, common, v, nullptr);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= rows.n) continue;
      const bool one = summed >> k & 1u;
#pragma unroll
      for (int e = 0; e < E; ++e)
        settle_put<T, D, ROWS, PITCH>(a, s, num, unit, row[k], lane * E + e, one ? rows.base[k] : m[k], one ? 1.f : l[k],
                                      v[k][e]);
    }
  }
}
template <typename T, int D, int ROWS, int PITCH, int WARPS>
__device__ void settle(const Attend& a, const Settle& s, const float* ml, float* num, int stride, float* unit,
                       Again<ROWS>* again) {
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x;
  if (tid < ROWS) again->bad[tid] = 0;
  __syncthreads();
  bool mine = false;
  for (int row = tid / D; row < s.cells; row += WARPS * 32 / D) {
    const int c = tid % D;
    float m = -INFINITY, l = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, ml[(w * 2) * ROWS + row]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float mw = ml[(w * 2) * ROWS + row], k = mw == -INFINITY ? 0.f : exp2f(mw - m);
      l = fmaf(k, ml[(w * 2 + 1) * ROWS + row], l);
      v = fmaf(k, num[w * stride + row * PITCH + c], v);
    }
    if (!isfinite(v) && isfinite(l) && l > 0.f) {
      again->bad[row] = 1;
      mine = true;
    }
    settle_put<T, D, ROWS, PITCH>(a, s, num, unit, row, c, m, l, v);
  }
  if (__syncthreads_or(mine)) settle_again<T, D, ROWS, PITCH, WARPS>(a, s, ml, num, stride, unit, again);
  if (!s.cluster) return;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int cell = s.part * (WARPS * 32) + tid; cell < s.cells * D; cell += s.cluster * WARPS * 32) {
    const int row = cell / D, c = cell % D;
    float m = -INFINITY, l = 0.f, v = 0.f;
    for (int p = 0; p < s.cluster; ++p) m = fmaxf(m, cl.map_shared_rank(unit, p)[row]);
    for (int p = 0; p < s.cluster; ++p) {
      const float mp = cl.map_shared_rank(unit, p)[row], k = part_factor(mp, m);
      l = fmaf(k, cl.map_shared_rank(unit, p)[ROWS + row], l);
      if (k != 0.f) v = fmaf(k, cl.map_shared_rank(num, p)[row * PITCH + c], v);
    }
    settle_final<T>(a, s, row, c, m, l, v);
  }
  cl.sync();                           // no block leaves while its state is read
}

// where part c begins
__device__ __forceinline__ int64_t edge(const int64_t* before, int E, int H, int64_t W, int N, int c) {
  const int64_t x = share(W, N, c);
  if (x <= 0 || x >= W) return x;
  const int e = entry_of(before, E, H, x);
  const int64_t n = before[e + 1] - before[e];
  if (n > kWholeBlocks) return x;
  const int64_t in = (x - before[e] * H) % n;
  return 2 * in < n ? x - in : x - in + n;
}

// Makes the list: tiles of `tile` rows (tokens), blocks of `block` keys.
cudaError_t launch_work(const Attend& a, const Work& w, int tile, int block, cudaStream_t st);
// Joins the partial results of cut units: `rows` (token, head) rows a unit, of `tile` tokens.
// own: the parts' blocks made the list, not the list kernel.
cudaError_t launch_join(const Attend& a, const Work& w, int dtype, int D, int tile, int rows, bool own, cudaStream_t st);

// The cap of scores, cap tanh(u) with u = scale q.k / cap, in the exponent's base
// 2.  Up to |u| = 3/4 it is the score times a polynomial of u^2, above that
// cap - 2 cap / (1 + e^(2 u)): that form is off by a few 2^-24 of the cap, far too
// much where the score is far below it.
//
// tanh(u) / u = sum of kTanh[i] u^(2 i) on |u| <= 3/4: the polynomial of its
// degree with the least relative error there, 2^-25 (Remez exchange).
__device__ constexpr float kTanh[6] = {1.0f, -0.33332958817481995f, 0.1332540661096573f, -0.05334442853927612f,
                                       0.01958290860056877f, -0.004716257099062204f};
constexpr float kTanhMost = 0.75f;
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// near's form for |u| <= 3/4, else far's: as a branch, rows with scores on both sides took twice the time
__device__ __forceinline__ float select_near(float u, float near, float far) {
  float r;
  asm("{\n .reg .pred p;\n setp.le.f32 p, %1, %2;\n selp.f32 %0, %3, %4, p;\n}\n"
      : "=f"(r)
      : "f"(fabsf(u)), "f"(kTanhMost), "f"(near), "f"(far));
  return r;
}
__device__ __forceinline__ float cap_of(const Attend& a, float z) {
  const float u = z * a.to_u, x = u * u;
  float y = kTanh[5];
#pragma unroll
  for (int q = 4; q >= 0; --q) y = fmaf(y, x, kTanh[q]);
  return select_near(u, z * a.to_z * y, fmaf(-2.f * a.cap2, rcp(1.f + sc::ex2(u * (2.f * kLog2e))), a.cap2));
}

// Weights that a product takes in the values' type are 2^(z - m + kLift): fp16's
// smallest step is 2^-24, so that of 64K keys whose weights lie just below half of
// it all would vanish from the numerator (0.2% of the largest weight together) and
// stay in the sum.  7 lifts the largest, 2^8 by the lazy maximum, to 2^15 of
// fp16's 65504, and what rounding can lose of a weight to 2^-32 of the largest.
// bf16 has fp32's range.  A state's maximum is then m - kLift, which its sum and
// numerator count from.
template <typename T> constexpr float kLift = 0.f;
template <> constexpr float kLift<__half> = 7.f;

// Few rows (paged_rows.cu): `cells` (token, head) rows a unit at most.  cluster
// > 0: that many blocks share a unit and no list or scratch is needed.
constexpr int kFewBlock = 64;                      // keys a block of the share-out
inline int few_rows(int cells) { return cells <= 8 ? 8 : cells <= 16 ? 16 : 32; }
cudaError_t attend_few(const Attend& a, const mp_paged_cache& c, Work w, int cells, int cluster, cudaStream_t st);

// fp32 (paged_f32.cu): `rows` of 4, 8, 16 or 64 (token, head) rows a tile of `tile` tokens.
constexpr int kF32ManyRows = 64;
inline int f32_rows(int64_t cells) { return cells <= 4 ? 4 : cells <= 8 ? 8 : cells <= 16 ? 16 : kF32ManyRows; }
cudaError_t attend_f32(const Attend& a, const mp_paged_cache& c, const Work& w, int rows, int tile, int cluster,
                       cudaStream_t st);

// Many rows (paged_tiles.cu).
constexpr int kTilesBlock = 128;                   // keys a block of the share-out
constexpr int kTilesRows = 256;                    // (token, head) rows a unit
inline int tiles_tokens(int G) { return kTilesRows / G; }
cudaError_t attend_tiles(const Attend& a, const mp_paged_cache& c, const Work& w, cudaStream_t st);

// Launches a kernel that needs more shared memory than the default.  The
// permission costs about as much as a launch and stays with the device's
// context, so it is asked for once a device, and again if a launch is refused
// (the context may be a new one).  It is for the most that any call of the kernel
// needs (`most`), so that calls from several threads do not take it from another.
template <typename Kernel, typename Args>
inline cudaError_t launch_large(Kernel* kernel, const cudaLaunchConfig_t& cfg, const Args& args, int device,
                                std::atomic<uint64_t>& done, size_t most) {
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  const bool had = (done.load(std::memory_order_relaxed) & bit) != 0;
  for (int turn = had ? 1 : 0;; ++turn) {
    if (turn != 1 || !had) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_relaxed);
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    if (e != cudaErrorInvalidValue || turn != 1 || !had) return e;
    cudaGetLastError();
  }
}

// cuTensorMapEncodeTiled, or null (paged.cu).
PFN_cuTensorMapEncodeTiled_v12000 map_encoder();

}  // namespace paged
}  // namespace mp
