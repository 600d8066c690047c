// Work list of a split attention call, and the joining of its partial results.
#include <type_traits>

#include "paged_work.cuh"

namespace mp {
namespace paged {

constexpr int kListThreads = 1024;

// One block: first the requests' tiles are counted (their sums are the
// entries' places), then a thread makes each entry and the costs are summed.
__global__ void __launch_bounds__(kListThreads) list_kernel(const Attend a, const Work w, int tile, int block) {
  __shared__ int64_t wsum[32];
  __shared__ int64_t carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // exclusive sum over the block's threads of x, on top of `carry`
  auto scan = [&](int64_t x) {
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int64_t base = carry;
    for (int i = 0; i < warp; ++i) base += wsum[i];
    __syncthreads();
    if (tid == kListThreads - 1) carry = base + s;
    __syncthreads();
    return base + s - x;
  };
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < a.batch; b0 += kListThreads) {
    const int b = b0 + tid;
    int tiles = 0;
    if (b < a.batch) {
      const Request r = request_of(a, b);
      tiles = (r.n + tile - 1) / tile;
    }
    const int64_t at = scan(tiles);
    // tiles past the rows that Q has can only come from offsets that overlap: not followed
    for (int i = 0; i < tiles; ++i)
      if (at + i < (int64_t)a.rows / tile + a.batch) {
        w.entry[at + i].b = b;
        w.entry[at + i].tile = i;
      } else {
        set_error(a.err, E_BAD_OFFSET);
      }
  }
  const int E = (int)min(carry, (int64_t)a.rows / tile + a.batch);
  __syncthreads();
  if (tid == 0) { carry = 0; w.count[0] = E; }
  __syncthreads();
  if (a.first_key) {                           // every row counts: a warp an entry
    for (int e = warp; e < E; e += kListThreads / 32) {
      Entry x = w.entry[e];
      const Request r = request_of(a, x.b);
      const int prefix = prefix_of(a, x.b), i1 = min(r.n, (x.tile + 1) * tile);
      int lo = INT32_MAX, hi = 0;
      for (int i = x.tile * tile + lane; i < i1; i += 32) {
        const Interval v = interval_of(a, r, prefix, i);
        if (v.hi > v.lo) { lo = min(lo, v.lo); hi = max(hi, v.hi); }
      }
      lo = __reduce_min_sync(kFull, lo);
      hi = __reduce_max_sync(kFull, hi);
      set_span(x, lo, hi, block);
      if (lane == 0) w.entry[e] = x;
    }
    __syncthreads();
  }
  for (int e0 = 0; e0 < E; e0 += kListThreads) {
    const int e = e0 + tid;
    int n = 0;
    if (e < E) {
      Entry x = w.entry[e];
      if (!a.first_key) {
        const Request r = request_of(a, x.b);
        span_of(a, r, x.b, x.tile * tile, min(r.n, (x.tile + 1) * tile), block, x);
        w.entry[e] = x;
      }
      n = x.n;
    }
    const int64_t at = scan(n);
    if (e < E) w.before[e] = at;
  }
  if (tid == 0) w.before[E] = carry;
}

// Joins the units that were cut.  Each is found at the first boundary between
// parts that lies inside it (blockIdx.x: the part behind the boundary); a warp
// takes a row: its lanes hold 32 parts' maxima and sums at a time, then every
// lane adds up its columns, eight parts' loads in flight.
constexpr int kJoinWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Attend a, const Work w, int tile, int rows) {
  constexpr int E = D / 32;                    // columns a lane
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int count = w.count[0], c = blockIdx.x + 1;
  const int64_t W = count > 0 ? w.before[count] * a.H : 0;
  if (W == 0) return;
  const int N = parts_used(w, W);
  if (c >= N) return;
  const int64_t x = share(W, N, c), before = share(W, N, c - 1);
  const int e = entry_of_warp(w.before, count, a.H, x);
  const int64_t first = w.before[e] * a.H, n = w.before[e + 1] - w.before[e];
  const int h = (int)((x - first) / n);
  const int64_t u0 = first + h * n, u1 = u0 + n;
  if (x == u0 || before > u0) return;          // a boundary between units, or not this unit's first
  const int c1 = part_of(W, N, u1 - 1), np = c1 - c + 2;
  const Entry en = w.entry[e];
  const Request r = request_of(a, en.b);
  const int cells = min(tile, r.n - en.tile * tile) * a.G, lane = threadIdx.x & 31;
  const int64_t size = (int64_t)rows * (2 + D);
  // part c - 1 holds the unit as its first item or as its last; later parts begin inside it
  const float* p0 = w.part + (2 * (int64_t)(c - 1) + (before < u0 ? 1 : 0)) * size;
  const float* p1 = w.part + 2 * (int64_t)c * size;
  auto slot = [&](int i) { return i == 0 ? p0 : p1 + 2 * (int64_t)(i - 1) * size; };
  for (int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < cells; row += gridDim.y * kJoinWarps) {
    float m = -INFINITY;
    for (int i = lane; i < np; i += 32) m = fmaxf(m, slot(i)[row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float l = 0.f, acc[E];
#pragma unroll
    for (int q = 0; q < E; ++q) acc[q] = 0.f;
    for (int i0 = 0; i0 < np; i0 += 32) {
      float f = 0.f;
      if (i0 + lane < np) {
        const float mi = slot(i0 + lane)[row];
        f = mi == -INFINITY ? 0.f : exp2f(mi - m);
        l = fmaf(f, slot(i0 + lane)[rows + row], l);
      }
      for (int k0 = 0; k0 < min(32, np - i0); k0 += 8) {
        Vec v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = *reinterpret_cast<const Vec*>(slot(min(i0 + k0 + k, np - 1)) + 2 * rows + (int64_t)row * D + lane * E);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float fk = __shfl_sync(kFull, f, k0 + k);          // 0 behind the last part
          const float* vk = reinterpret_cast<const float*>(&v[k]);
          if (fk != 0.f)                       // a part that saw nothing holds no numerator
#pragma unroll
            for (int q = 0; q < E; ++q) acc[q] = fmaf(fk, vk[q], acc[q]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    const int t = r.row0 + en.tile * tile + row / a.G, hq = h * a.G + row % a.G;
    T* dst = reinterpret_cast<T*>(a.O + (int64_t)t * a.o_row_b + (int64_t)hq * a.o_head_b) + lane * E;
#pragma unroll
    for (int q = 0; q < E; ++q) dst[q] = from_f32<T>(l == 0.f ? 0.f : acc[q] / l);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.H * a.G + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) / kLog2e;
  }
}

cudaError_t launch_work(const Attend& a, const Work& w, int tile, int block, cudaStream_t st) {
  list_kernel<<<1, kListThreads, 0, st>>>(a, w, tile, block);
  return cudaGetLastError();
}

cudaError_t launch_join(const Attend& a, const Work& w, int dtype, int D, int tile, int rows, cudaStream_t st) {
  if (w.parts < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  // four rows a warp of a large unit, one of a small
  cfg.gridDim = dim3((unsigned)(w.parts - 1), (unsigned)(rows <= 32 ? (rows + kJoinWarps - 1) / kJoinWarps : rows / 16));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a, w, tile, rows); };
  if (dtype == MP_F32) return D == 128 ? go(join_kernel<float, 128>) : go(join_kernel<float, 64>);
  if (dtype == MP_F16) return D == 128 ? go(join_kernel<__half, 128>) : go(join_kernel<__half, 64>);
  return D == 128 ? go(join_kernel<__nv_bfloat16, 128>) : go(join_kernel<__nv_bfloat16, 64>);
}

}  // namespace paged
}  // namespace mp
