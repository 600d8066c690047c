// Definitions shared by the paged-cache operators: the arguments of an
// attention call, a row's visible keys, and the exact row kernel body that the
// fast kernels fall back on.
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

// One row of one query head over the keys [k0, k1) that it sees, by one warp,
// one key at a time, so that a key it does not see is not even read.  The
// running maximum m is in base-2 units; lane l holds the elements
// [l * D/32, (l + 1) * D/32) of the numerator.
template <typename T, int D>
struct RowState {
  float m, l, acc[D / 32];
};
template <typename T, int D>
__device__ void attend_row(const Attend& a, int b, const Request& r, int i, int hq, int k0, int k1, RowState<T, D>& s) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, h = hq / a.G;
  const Interval v = interval_of(a, r, prefix_of(a, b), i);
  const T* q = reinterpret_cast<const T*>(a.Q + (int64_t)(r.row0 + i) * a.q_row_b + (int64_t)hq * a.q_head_b) + lane * E;
  float qf[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qf[e] = to_f32(q[e]);
  const float slope = a.slopes ? __ldg(a.slopes + hq) : 0.f;
  s.m = -INFINITY;
  s.l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) s.acc[e] = 0.f;
  for (int j = max(k0, v.lo); j < min(k1, v.hi); ++j) {
    const int page = page_of(a, b, j);
    if (page < 0) continue;
    const int64_t off = page * a.page_b + h * a.head_b + (j & ((1 << a.page_shift) - 1)) * a.tok_b;
    const T* kr = reinterpret_cast<const T*>(a.K + off) + lane * E;
    const T* vr = reinterpret_cast<const T*>(a.V + off) + lane * E;
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(qf[e], to_f32(kr[e]), dot);
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    const float z = score2(a, dot, slope, v.pos - j);
    const float m = fmaxf(s.m, z), keep = s.m == -INFINITY ? 0.f : exp2f(s.m - m);
    const float w = z == -INFINITY ? 0.f : exp2f(z - m);
    s.l = s.l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) s.acc[e] = s.acc[e] * keep + w * to_f32(vr[e]);
    s.m = m;
  }
  if (s.l != s.l) s.m = s.l;         // a NaN among the keys seen must not pass for "nothing seen"
}

}  // namespace paged

mp_status paged_attend_impl(const mp_paged_cache& c, const mp_paged_attend_args& p, void* scratch,
                            size_t scratch_bytes, cudaStream_t st);
size_t paged_attend_scratch_bytes(const mp_paged_cache& c, const mp_paged_attend_args& p);

}  // namespace mp
