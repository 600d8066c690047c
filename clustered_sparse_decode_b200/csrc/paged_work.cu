// Work list of a split attention call, and the joining of its partial results.
#include <type_traits>

#include "paged_work.cuh"

namespace mp {
namespace paged {

constexpr int kListThreads = 1024;

// One block.  Requests are taken 1024 at a time: their tiles are counted and
// summed, then a thread makes each entry, finding its request by bisection in
// shared memory (a warp an entry where every row has its own first key), and
// the costs are summed.  A chain of loads and barriers: 4 us for a few requests.
__global__ void __launch_bounds__(kListThreads) list_kernel(const Attend a, const Work w, int tile, int block) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int64_t sums[2][32];
  __shared__ int32_t first[kListThreads + 1];            // entries before each request of the round
  __shared__ int32_t spans[2][kListThreads];             // of the round's entries: first key, blocks (first_key only)
  __shared__ int64_t sums_of[kListThreads + 1];          // w.before, if it is short
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  // exclusive sum of x over the block's threads, and their total; consecutive calls use different halves of `sums`
  auto scan = [&](int64_t x, int64_t& total) {
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) sums[turn][warp] = s;
    __syncthreads();
    int64_t all = sums[turn][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, all, o);
      if (lane >= o) all += y;
    }
    total = __shfl_sync(kFull, all, 31);
    const int64_t base = __shfl_sync(kFull, all, max(0, warp - 1));
    turn ^= 1;
    return (warp ? base : 0) + s - x;
  };
  // entries past the rows that Q has can only come from offsets that overlap: they are not followed
  const int64_t most = (int64_t)a.rows / tile + a.batch;
  int64_t entries = 0, blocks = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kListThreads) {
    int tiles = 0;
    if (b0 + tid < a.batch) tiles = (request_of(a, b0 + tid).n + tile - 1) / tile;
    int64_t round;
    const int64_t at = scan(tiles, round);
    if (entries + round > most) {
      round = most - entries;
      if (tid == 0) set_error(a.err, E_BAD_OFFSET);
    }
    first[tid] = (int32_t)min(at, round);
    if (tid == 0) first[kListThreads] = (int32_t)round;
    __syncthreads();
    const int requests = min(kListThreads, a.batch - b0);
    auto entry_at = [&](int e) {                         // the last request whose first entry is at or before e
      int lo = 0, hi = requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= e) lo = mid;
        else hi = mid;
      }
      return Entry{b0 + lo, e - first[lo], 0, 0};
    };
    for (int e0 = 0; e0 < round; e0 += kListThreads) {
      if (a.first_key) {                                 // every row counts: a warp an entry
        for (int k = warp; k < kListThreads && e0 + k < round; k += kListThreads / 32) {
          Entry x = entry_at(e0 + k);
          const Request r = request_of(a, x.b);
          const int prefix = prefix_of(a, x.b), i1 = min(r.n, (x.tile + 1) * tile);
          int lo = INT32_MAX, hi = 0;
#pragma unroll 8
          for (int u = 0; u < (tile + 31) / 32; ++u) {
            const int i = x.tile * tile + 32 * u + lane;
            const Interval v = interval_of(a, r, prefix, min(i, i1 - 1));
            if (i < i1 && v.hi > v.lo) { lo = min(lo, v.lo); hi = max(hi, v.hi); }
          }
          set_span(x, __reduce_min_sync(kFull, lo), __reduce_max_sync(kFull, hi), block);
          if (lane == 0) { spans[0][k] = x.k0; spans[1][k] = x.n; }
        }
        __syncthreads();
      }
      Entry x{0, 0, 0, 0};
      if (e0 + tid < round) {
        x = entry_at(e0 + tid);
        if (a.first_key) {
          x.k0 = spans[0][tid];
          x.n = spans[1][tid];
        } else {
          const Request r = request_of(a, x.b);
          span_of(a, r, x.b, x.tile * tile, min(r.n, (x.tile + 1) * tile), block, x);
        }
      }
      int64_t cost;
      const int64_t before = scan(x.n, cost);
      if (e0 + tid < round) {
        w.entry[entries + e0 + tid] = x;
        w.before[entries + e0 + tid] = blocks + before;
        if (entries + e0 + tid < kListThreads) sums_of[entries + e0 + tid] = blocks + before;
      }
      blocks += cost;
      if (a.first_key) __syncthreads();                  // spans are read
    }
    entries += round;
    __syncthreads();                                     // first is read
  }
  if (tid == 0) {
    w.before[entries] = blocks;
    w.count[0] = (int32_t)entries;
    *reinterpret_cast<int64_t*>(w.count + 2) = blocks;
    if (entries <= kListThreads) sums_of[entries] = blocks;
  }
  __syncthreads();
  // where the parts begin, found here once (a dozen dependent loads in each of their blocks otherwise)
  const int64_t W = blocks * a.H;
  const int E = (int)entries, N = W > 0 ? parts_used(w, W) : 0;
  const int64_t* before = entries <= kListThreads ? sums_of : w.before;
  for (int c = tid; c <= w.parts; c += kListThreads) {
    const int64_t x = c < N ? edge(before, E, a.H, W, N, c) : W;
    w.edge[c] = x;
    w.edge_entry[c] = x < W ? entry_of(before, E, a.H, x) : 0;
  }
}

// Joins the units that were cut.  Each is found at the first boundary between
// parts that lies inside it (blockIdx.x: the part behind the boundary).  A warp
// takes R rows at once: lane (32 / R) r + k holds row r's maximum and sum of part
// k (32 / R parts a round), then every lane adds up its columns of the rows, eight
// loads in flight.  Large units are cut in two or three (R = 4), small ones in
// many parts (R = 1: the 38 parts of 64K tokens on 8 heads take 10 us less).
constexpr int kJoinWarps = 4;

template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Attend a, const Work w, int tile, int rows, int own) {
  constexpr int E = D / 32;                    // columns a lane
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int count = w.count[0], c = blockIdx.x + 1;
  const int64_t W = *reinterpret_cast<const int64_t*>(w.count + 2) * a.H;
  if (W == 0) return;
  const int N = parts_used(w, W);
  if (c >= N) return;
  const int64_t x = share(W, N, c);
  const int e = entry_of_warp(w.before, count, a.H, x);
  const int64_t first = w.before[e] * a.H, n = w.before[e + 1] - w.before[e];
  const Entry en = w.entry[e];
  const int h = (int)((x - first) / n);
  const int64_t u0 = first + h * n, u1 = u0 + n;
  // an edge between units, of a unit that is not cut, or not the first inside its unit
  if (x == u0 || n <= kWholeBlocks || share(W, N, c - 1) > u0) return;
  const int64_t before = own ? edge(w.before, count, a.H, W, N, c - 1) : w.edge[c - 1];
  const int c1 = part_of(W, N, u1 - 1), np = c1 - c + 2;
  const Request r = request_of(a, en.b);
  const int cells = min(tile, r.n - en.tile * tile) * a.G, lane = threadIdx.x & 31;
  const int64_t size = (int64_t)rows * (2 + D);
  // part c - 1 holds the unit as its first item or as its last; later parts begin inside it
  const float* p0 = w.part + (2 * (int64_t)(c - 1) + (before < u0 ? 1 : 0)) * size;
  const float* p1 = w.part + 2 * (int64_t)c * size;
  auto slot = [&](int i) { return i == 0 ? p0 : p1 + 2 * (int64_t)(i - 1) * size; };
  for (int row0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * R; row0 < cells;
       row0 += gridDim.y * kJoinWarps * R) {
    constexpr int K = 32 / R, S = 8 / R;         // parts a round, parts whose loads are in flight
    const int row = row0 + lane / K, k = lane % K;
    float m = -INFINITY;
    for (int i = k; i < np; i += K)
      if (row < cells) m = fmaxf(m, slot(i)[row]);
#pragma unroll
    for (int o = K / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float l = 0.f, acc[R][E];
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int d = 0; d < E; ++d) acc[q][d] = 0.f;
    for (int i0 = 0; i0 < np; i0 += K) {
      float f = 0.f;
      if (i0 + k < np && row < cells) {
        const float mi = slot(i0 + k)[row];
        f = part_factor(mi, m);
        l = fmaf(f, slot(i0 + k)[rows + row], l);
      }
      for (int k0 = 0; k0 < min(K, np - i0); k0 += S) {
        Vec v[S][R];
#pragma unroll
        for (int t = 0; t < S; ++t)
#pragma unroll
          for (int q = 0; q < R; ++q)
            v[t][q] = *reinterpret_cast<const Vec*>(slot(min(i0 + k0 + t, np - 1)) + 2 * rows +
                                                    (int64_t)min(row0 + q, cells - 1) * D + lane * E);
#pragma unroll
        for (int t = 0; t < S; ++t)
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const float fk = __shfl_sync(kFull, f, K * q + ((k0 + t) & (K - 1)));
            const float* vk = reinterpret_cast<const float*>(&v[t][q]);
            if (fk != 0.f && i0 + k0 + t < np)           // a part that saw nothing holds no numerator
#pragma unroll
              for (int d = 0; d < E; ++d) acc[q][d] = fmaf(fk, vk[d], acc[q][d]);
          }
      }
    }
#pragma unroll
    for (int o = K / 2; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float lq = __shfl_sync(kFull, l, K * q), mq = __shfl_sync(kFull, m, K * q);
      if (row0 + q >= cells) continue;
      const int t = r.row0 + en.tile * tile + (row0 + q) / a.G, hq = h * a.G + (row0 + q) % a.G;
      T* dst = reinterpret_cast<T*>(a.O + (int64_t)t * a.o_row_b + (int64_t)hq * a.o_head_b) + lane * E;
#pragma unroll
      for (int d = 0; d < E; ++d) dst[d] = from_f32<T>(lq == 0.f ? 0.f : acc[q][d] / lq);
      if (a.lse && lane == 0) a.lse[(int64_t)t * a.H * a.G + hq] = lq == 0.f ? -INFINITY : (mq + log2f(lq)) / kLog2e;
    }
  }
}

cudaError_t launch_work(const Attend& a, const Work& w, int tile, int block, cudaStream_t st) {
  list_kernel<<<1, kListThreads, 0, st>>>(a, w, tile, block);
  return cudaGetLastError();
}

template <int R>
static cudaError_t launch_join_r(const Attend& a, const Work& w, int dtype, int D, int tile, int rows, int own,
                                 cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(w.parts - 1), (unsigned)((rows + kJoinWarps * R - 1) / (kJoinWarps * R)));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a, w, tile, rows, own); };
  if (dtype == MP_F32) return D == 128 ? go(join_kernel<float, 128, R>) : go(join_kernel<float, 64, R>);
  if (dtype == MP_F16) return D == 128 ? go(join_kernel<__half, 128, R>) : go(join_kernel<__half, 64, R>);
  return D == 128 ? go(join_kernel<__nv_bfloat16, 128, R>) : go(join_kernel<__nv_bfloat16, 64, R>);
}

cudaError_t launch_join(const Attend& a, const Work& w, int dtype, int D, int tile, int rows, bool own, cudaStream_t st) {
  if (w.parts < 2) return cudaSuccess;
  return rows <= 32 ? launch_join_r<1>(a, w, dtype, D, tile, rows, own, st)
                    : launch_join_r<4>(a, w, dtype, D, tile, rows, own, st);
}

}  // namespace paged
}  // namespace mp
