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
// looked at again.  Only a NaN that it sees itself explains the result: then it
// stands, so that one NaN among a request's keys does not cost all later tokens a
// second pass.  Otherwise (a NaN that it does not see; infinities, which rounded
// weights and remainders can turn into NaN; no such value at all, where large
// values have overflowed beside weights of up to 2^8) row_sum sums over the keys
// that the row sees, with weights that add up to 1.
enum { V_NAN = 1, V_INF = 2 };
// whether such a row has to be summed again: `any` of all keys that went in, `unseen` of those that it does not see
__device__ __forceinline__ bool sum_again(int any, bool inf, int unseen) {
  return any != V_NAN || inf || unseen != 0;
}

// Which of V_NAN and V_INF the keys of [k0, k1) outside [lo, hi) hold.
// [low, high): what the tile's rows see together; keys beyond it stand on the
// page of the nearest one inside, as where a kernel loads them.  A warp together,
// 4 KB in flight; `turns`, if given, counts up meanwhile.
template <typename T, int D>
__device__ __noinline__ int odd_values(const Attend& a, int b, int h, int lo, int hi, int k0, int k1, int low, int high,
                                       int* turns) {
  constexpr int VEC = D * (int)sizeof(T) / 16, KEYS = 32 / VEC, U = 8;
  const int lane = threadIdx.x & 31, mask = (1 << a.page_shift) - 1;
  int odd = 0;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int from = side ? max(hi, k0) : k0, to = side ? k1 : min(lo, k1);
#pragma unroll 1
    for (int j0 = from; j0 < to; j0 += KEYS * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * KEYS + lane / VEC;
        if (j >= to) continue;
        const int page = page_of(a, b, min(max(j, low), high - 1));
        if (page < 0) continue;
        const uint4 x = *reinterpret_cast<const uint4*>(a.V + page * a.page_b + h * a.head_b + (j & mask) * a.tok_b +
                                                        lane % VEC * 16);
        const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
        for (int i = 0; i < 16 / (int)sizeof(T); ++i) {
          const float f = to_f32(e[i]);
          odd |= f != f ? V_NAN : isfinite(f) ? 0 : V_INF;
        }
      }
      if (turns && lane == 0) atomicAdd(turns, 1);
      if (__any_sync(kFull, odd & V_INF)) return V_INF;
    }
  }
  return __reduce_or_sync(kFull, odd);
}

// The sum 2^(z - m) v of one row of one query head over the keys of [k0, k1) that
// it sees, by one warp; no other key is read.  Lane l gets the elements
// [l * D/32, (l + 1) * D/32).  From the last key backwards, until nothing but NaN
// is left: values that went bad at some token mostly stay so behind it.
template <typename T, int D>
__device__ __noinline__ void row_sum(const Attend& a, int b, const Request& r, int i, int hq, int k0, int k1, float m,
                                       float (&acc)[D / 32], int* turns) {
  constexpr int E = D / 32, U = 8;
  const int lane = threadIdx.x & 31, h = hq / a.G, mask = (1 << a.page_shift) - 1;
  const Interval v = interval_of(a, r, prefix_of(a, b), i);
  const T* q = reinterpret_cast<const T*>(a.Q + (int64_t)(r.row0 + i) * a.q_row_b + (int64_t)hq * a.q_head_b) + lane * E;
  float qf[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qf[e] = to_f32(q[e]);
  const float slope = a.slopes ? __ldg(a.slopes + hq) : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int from = max(k0, v.lo), to = min(k1, v.hi);
#pragma unroll 1
  for (int j0 = to - 1; j0 >= from; j0 -= U) {
    float dot[U], val[U][E];
    bool held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 - u, page = j >= from ? page_of(a, b, j) : -1;
      held[u] = page >= 0;
      const int64_t off = (held[u] ? page : 0) * a.page_b + h * a.head_b + (held[u] ? j & mask : 0) * a.tok_b;
      dot[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (held[u]) dot[u] = fmaf(qf[e], to_f32(reinterpret_cast<const T*>(a.K + off)[lane * E + e]), dot[u]);
        val[u][e] = held[u] ? to_f32(reinterpret_cast<const T*>(a.V + off)[lane * E + e]) : 0.f;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(kFull, dot[u], o);
    bool gone = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = held[u] ? exp2f(score2(a, dot[u], slope, v.pos - (j0 - u)) - m) : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, val[u][e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) gone = gone && acc[e] != acc[e];
    if (turns && lane == 0) atomicAdd(turns, 1);
    if (__all_sync(kFull, gone)) return;
  }
}

}  // namespace paged

mp_status paged_attend_impl(const mp_paged_cache& c, const mp_paged_attend_args& p, void* scratch,
                            size_t scratch_bytes, cudaStream_t st);
size_t paged_attend_scratch_bytes(const mp_paged_cache& c, const mp_paged_attend_args& p);

}  // namespace mp
