// Work list of a split attention call, and the joining of its partial results.
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
  for (int e0 = 0; e0 < E; e0 += kListThreads) {
    const int e = e0 + tid;
    int n = 0;
    if (e < E) {
      Entry x = w.entry[e];
      const Request r = request_of(a, x.b);
      span_of(a, r, x.b, x.tile * tile, min(r.n, (x.tile + 1) * tile), block, x);
      n = x.n;
      w.entry[e] = x;
    }
    const int64_t at = scan(n);
    if (e < E) w.before[e] = at;
  }
  if (tid == 0) w.before[E] = carry;
}

// A block joins one row of one unit: first all parts' maxima and sums side by
// side, then thread c adds up its column c, eight parts' loads in flight (one
// after the other they took three times as long: 16.8 us against 5 for the 38
// parts of 64K tokens on 8 heads).
template <typename T, int D>
__global__ void __launch_bounds__(D) join_kernel(const Attend a, const Work w, int tile, int rows) {
  __shared__ float weight[kMostParts];
  __shared__ float red[2][D / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int E = w.count[0], e = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  if (e >= E) return;
  const int64_t W = w.before[E] * a.H, n = w.before[e + 1] - w.before[e], u0 = w.before[e] * a.H + h * n, u1 = u0 + n;
  if (n == 0) return;                          // a request without rows
  const Entry x = w.entry[e];
  const int N = parts_used(w, W), c0 = part_of(W, N, u0), c1 = part_of(W, N, u1 - 1), np = c1 - c0 + 1;
  if (np == 1) return;                         // the part wrote the result itself
  const Request r = request_of(a, x.b);
  const int cells = min(tile, r.n - x.tile * tile) * a.G;
  const bool inside = share(W, N, c0) < u0;    // part c0 began with another unit
  const int64_t size = (int64_t)rows * (2 + D);
  const float* p0 = w.part + (2 * (int64_t)c0 + (inside ? 1 : 0)) * size;
  const float* p1 = w.part + 2 * (int64_t)(c0 + 1) * size;             // parts behind c0 begin inside the unit
  auto slot = [&](int i) { return i == 0 ? p0 : p1 + 2 * (int64_t)(i - 1) * size; };
  for (int row = blockIdx.y; row < cells; row += gridDim.y) {
    float m = -INFINITY;
    for (int i = tid; i < np; i += D) {
      weight[i] = slot(i)[row];
      m = fmaxf(m, weight[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if ((tid & 31) == 0) red[0][tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < D / 32; ++i) m = fmaxf(m, red[0][i]);
    float l = 0.f;
    for (int i = tid; i < np; i += D) {
      const float f = weight[i] == -INFINITY ? 0.f : exp2f(weight[i] - m);
      weight[i] = f;
      l = fmaf(f, slot(i)[rows + row], l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    if ((tid & 31) == 0) red[1][tid >> 5] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) l += red[1][i];
    float o = 0.f;
    int i = 0;
    for (; i + 8 <= np; i += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = slot(i + k)[2 * rows + row * D + tid];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (weight[i + k] != 0.f) o = fmaf(weight[i + k], v[k], o);    // a part that saw nothing holds no numerator
    }
    for (; i < np; ++i) {
      const float v = slot(i)[2 * rows + row * D + tid];
      if (weight[i] != 0.f) o = fmaf(weight[i], v, o);
    }
    const bool none = l == 0.f;
    const int t = r.row0 + x.tile * tile + row / a.G, hq = h * a.G + row % a.G;
    T* dst = reinterpret_cast<T*>(a.O + (int64_t)t * a.o_row_b + (int64_t)hq * a.o_head_b);
    dst[tid] = from_f32<T>(none ? 0.f : o / l);
    if (a.lse && tid == 0)
      a.lse[(int64_t)t * a.H * a.G + hq] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
    __syncthreads();
  }
}

cudaError_t launch_work(const Attend& a, const Work& w, int tile, int block, cudaStream_t st) {
  list_kernel<<<1, kListThreads, 0, st>>>(a, w, tile, block);
  return cudaGetLastError();
}

cudaError_t launch_join(const Attend& a, const Work& w, int dtype, int D, int tile, int rows, int max_entries,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  // rows of a unit over the grid's second axis, as many as keep the grid at a few blocks an SM
  int y = 1;
  while (y * 2 <= rows && (int64_t)max_entries * a.H * y < 1184) y *= 2;
  cfg.gridDim = dim3((unsigned)(max_entries * a.H), (unsigned)y);
  cfg.blockDim = dim3(D);
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
