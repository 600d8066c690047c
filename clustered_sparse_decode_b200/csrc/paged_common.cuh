// Definitions shared by the paged-cache operators: the arguments of an
// attention call, a row's visible keys, and what the kernels do about a row into
// which a key that it does not see may have got.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "mp_internal.cuh"

namespace mp {

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

namespace paged {

// Tensor maps of a cache handle (mp_paged_cache::maps), 16 words each: 16-bit
// dtypes only.
enum Map { MAP_K16 = 0, MAP_V16, MAP_KPAGE, MAP_VPAGE };

struct Attend {
  const char* K;
  const char* V;
  int64_t page_b, head_b, tok_b;       // strides in bytes
  int32_t num_pages, page_shift;
  int32_t H, G;
  const int32_t* table;
  int32_t table_pages, table_stride;
  const int32_t* lens;
  const int32_t* cu;
  int32_t batch, rows, max_new;
  const char* Q;
  char* O;
  int64_t q_row_b, q_head_b, o_row_b, o_head_b;
  float scale;                         // of q.k
  float cap;                           // 0: none
  float to_z, to_u, cap2;              // scale in the exponent's base 2; scale / cap; cap in base 2
  int32_t window;                      // 0: none, at most 2^30
  int32_t full;
  const float* slopes;
  const int32_t* prefix;
  const int32_t* first_key;
  float* lse;
  int32_t* err;
  int32_t device;
};

// A request's rows and length, clamped to what the tensors hold: a bad offset
// or length sets the error word and cannot lead out of range.
struct Request {
  int32_t row0, n, len;
};
__device__ __forceinline__ Request request_of(const Attend& a, int b) {
  Request r;
  const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.lens + b);
  const int64_t most = (int64_t)a.table_pages << a.page_shift;
  r.row0 = min(max(c0, 0), a.rows);
  r.n = min(max(c1, r.row0), a.rows) - r.row0;
  r.len = (int32_t)min((int64_t)max(len, 0), most);
  if (r.row0 != c0 || r.row0 + r.n != c1 || r.len != len) set_error(a.err, E_BAD_OFFSET);
  if (r.n > a.max_new) {
    r.n = a.max_new;
    set_error(a.err, E_CAPACITY);
  }
  return r;
}

// The keys [lo, hi) that the request's i-th row sees, and its position.
struct Interval {
  int32_t lo, hi, pos;
};
__device__ __forceinline__ Interval interval_of(const Attend& a, const Request& r, int prefix, int i) {
  Interval v;
  v.pos = r.len - r.n + i;
  v.hi = a.full ? r.len : max(v.pos + 1, min(prefix, r.len));
  v.lo = a.window > 0 ? max(0, v.pos - a.window + 1) : 0;
  if (a.first_key) v.lo = max(v.lo, __ldg(a.first_key + r.row0 + i));
  return v;
}
__device__ __forceinline__ int prefix_of(const Attend& a, int b) { return a.prefix ? __ldg(a.prefix + b) : 0; }

// The page of key j of request b, or -1 (error word set).
__device__ __forceinline__ int page_of(const Attend& a, int b, int j) {
  const int p = __ldg(a.table + (int64_t)b * a.table_stride + (j >> a.page_shift));
  if ((unsigned)p >= (unsigned)a.num_pages) {
    set_error(a.err, E_BAD_OFFSET);
    return -1;
  }
  return p;
}

// The score in the exponent's base 2 from the raw dot product.
__device__ __forceinline__ float score2(const Attend& a, float dot, float slope, int away) {
  float z = dot * a.scale;
  if (a.cap > 0.f) z = a.cap * tanhf(z / a.cap);
  return (z - slope * (float)abs(away)) * kLog2e;
}

// A key that a row does not see has weight 0, but 0 times an infinite or NaN
// value is NaN: only so, and only through a product that takes whole tiles of
// keys, can it reach the row's numerator (its score is replaced, so never the
// sum).  A row with a finite sum and a numerator that is not finite is therefore
// looked at again (mend_rows), column by column.  Where the row itself sees
// infinities or NaN in a column, these alone are the result: no key has to be
// multiplied again, so that one bad value among a request's keys does not cost all
// later tokens a second pass.  Any other column that is not finite (a value that
// the row does not see, or large values that overflowed beside weights of up to
// 2^8) needs row_sums, over the keys that the row sees and with weights that add up
// to 1.
enum { V_NAN = 1, V_UP = 2, V_DOWN = 4 };

// A lane's E elements of a row.
template <typename T, int E>
struct alignas(sizeof(T) * E) Slice {
  T v[E];
};

// What lane l's elements [l * D/32, (l + 1) * D/32) of the values of the keys
// [k0, k1) hold, or-ed into `odd`.  Keys outside [low, high), what the tile's rows
// see together, stand on the page of the nearest one inside, as where a kernel
// loads them.  A warp together, 16 keys in flight; `turns`, if given, counts up.
template <typename T, int D>
__device__ __noinline__ void odd_values(const Attend& a, int b, int h, int k0, int k1, int low, int high,
                                        int (&result)[D / 32], int* turns) {
  constexpr int E = D / 32, U = 16;
  int odd[E] = {};                     // (in registers: the result's address could be any that the loads read)
  const int lane = threadIdx.x & 31, mask = (1 << a.page_shift) - 1;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
#pragma unroll 1
  for (int j0 = k0; j0 < k1; j0 += U) {
    Slice<T, E> x[U];
    bool held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u, k1 - 1), page = __ldg(table + (min(max(j, low), high - 1) >> a.page_shift));
      held[u] = (unsigned)page < (unsigned)a.num_pages;
      x[u] = *reinterpret_cast<const Slice<T, E>*>(a.V + (held[u] ? page : 0) * a.page_b + h * a.head_b +
                                                   (j & mask) * a.tok_b + lane * sizeof(x[u]));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float f = to_f32(x[u].v[e]);
        if (held[u] && !isfinite(f)) odd[e] |= f != f ? V_NAN : f > 0.f ? V_UP : V_DOWN;
      }
    if (turns && lane == 0) atomicAdd(turns, 1);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) result[e] |= odd[e];
}

// Up to four rows of query heads of one KV head.
struct Rows4 {
  int n, i[4], hq[4];                  // tokens of the request, query heads
  float base[4];                       // maximum + log2 of the sum
};

// The sums 2^(z - base) v of the rows over the keys of [k0, k1) that each sees, by
// one warp, eight keys at a time; no other key is used.  Lane l gets the elements
// [l * D/32, (l + 1) * D/32).  The 32 products of four rows and eight keys are
// added up so that lane 8 r + u ends with row r's score of key u.
template <typename T, int D>
__device__ __noinline__ void row_sums(const Attend& a, int b, const Request& r, const Rows4& rows, int k0, int k1,
                                      float (&result)[4][D / 32], int* turns) {
  constexpr int E = D / 32, U = 8;
  const int lane = threadIdx.x & 31, shift = a.page_shift, mask = (1 << shift) - 1, pages = a.num_pages, h = rows.hq[0] / a.G;
  const int64_t page_b = a.page_b, tok_b = a.tok_b;
  const char *K = a.K + h * a.head_b, *V = a.V + h * a.head_b;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  float q[4][E], acc[4][E];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = k < rows.n ? k : 0;
    const Slice<T, E> x = *reinterpret_cast<const Slice<T, E>*>(a.Q + (int64_t)(r.row0 + rows.i[t]) * a.q_row_b +
                                                                (int64_t)rows.hq[t] * a.q_head_b + lane * sizeof(x));
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[k][e] = to_f32(x.v[e]);
      acc[k][e] = 0.f;
    }
  }
  const int own = lane >> 3;           // the row whose scores this lane gets
  Interval v{0, 0, 0};
  float base = 0.f, slope = 0.f;
  if (own < rows.n) {
    v = interval_of(a, r, prefix_of(a, b), rows.i[own]);
    base = rows.base[own];
    if (a.slopes) slope = __ldg(a.slopes + rows.hq[own]);
  }
  const int lo = max(k0, v.lo), hi = min(k1, v.hi);
  const int from = __reduce_min_sync(kFull, hi > lo ? lo : INT32_MAX), to = __reduce_max_sync(kFull, hi > lo ? hi : 0);
  bool bad = false;
#pragma unroll 1
  for (int j0 = from; j0 < to; j0 += U) {
    Slice<T, E> kx[U], vx[U];
    uint32_t held = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u, to - 1), page = __ldg(table + (j >> shift));
      const bool in = (unsigned)page < (unsigned)pages;
      bad |= !in;
      held |= in ? 1u << u : 0u;
      const int64_t off = (in ? page : 0) * page_b + (j & mask) * tok_b + lane * sizeof(kx[u]);
      kx[u] = *reinterpret_cast<const Slice<T, E>*>(K + off);
      vx[u] = *reinterpret_cast<const Slice<T, E>*>(V + off);
    }
    float dot[4 * U];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[k * U + u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) dot[k * U + u] = fmaf(q[k][e], to_f32(kx[u].v[e]), dot[k * U + u]);
      }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int x = 0; x < o; ++x) {
        const float send = lane & o ? dot[x] : dot[x + o], keep = lane & o ? dot[x + o] : dot[x];
        dot[x] = keep + __shfl_xor_sync(kFull, send, o);
      }
    const int j = j0 + (lane & 7);
    const bool sees = j >= lo && j < hi && (held >> (lane & 7) & 1u);
    const float w = exp2f(score2(a, dot[0], slope, v.pos - j) - base);
    const uint32_t seen = __ballot_sync(kFull, sees);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wk = __shfl_sync(kFull, w, k * U + u);
        if (seen >> (k * U + u) & 1u)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[k][e] = fmaf(wk, to_f32(vx[u].v[e]), acc[k][e]);
      }
    if (turns && lane == 0) atomicAdd(turns, 1);
  }
  if (bad) set_error(a.err, E_BAD_OFFSET);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) result[k][e] = acc[k][e];
}

// Rows' numerators, val, put right: the keys [k0, k1) went into them, those of
// [c0, c1) all of them see and their odd_values are known.  Returns which of them
// now go with weights that add up to 1.
template <typename T, int D>
__device__ __forceinline__ uint32_t mend_rows(const Attend& a, int b, const Request& r, const Rows4& rows, int k0, int k1,
                                              int low, int high, int c0, int c1, const int (&common)[D / 32],
                                              float (&val)[4][D / 32], int* turns) {
  constexpr int E = D / 32;
  const int h = rows.hq[0] / a.G, prefix = prefix_of(a, b);
  int odd[4][E];
  uint32_t again = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= rows.n) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) odd[k][e] = common[e];
    const Interval v = interval_of(a, r, prefix, rows.i[k]);
    const int from = max(k0, v.lo), to = min(k1, v.hi);
    odd_values<T, D>(a, b, h, from, min(c0, to), low, high, odd[k], turns);
    odd_values<T, D>(a, b, h, max(c1, from), to, low, high, odd[k], turns);
    bool sum = false;
#pragma unroll
    for (int e = 0; e < E; ++e) sum |= odd[k][e] == 0 && !isfinite(val[k][e]);
    if (__any_sync(kFull, sum)) again |= 1u << k;
  }
  if (again) {
    float sums[4][E];
    row_sums<T, D>(a, b, r, rows, k0, k1, sums, turns);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (again >> k & 1u) val[k][e] = sums[k][e];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= rows.n) continue;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (odd[k][e]) val[k][e] = odd[k][e] == V_UP ? INFINITY : odd[k][e] == V_DOWN ? -INFINITY : NAN;
  }
  return again;
}

}  // namespace paged

mp_status paged_attend_impl(const mp_paged_cache& c, const mp_paged_attend_args& p, void* scratch,
                            size_t scratch_bytes, cudaStream_t st);
size_t paged_attend_scratch_bytes(const mp_paged_cache& c, const mp_paged_attend_args& p);

}  // namespace mp
