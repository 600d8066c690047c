// Attention of new tokens over a paged cache: the choice of kernel, its scratch,
// and the row-by-row kernel.
#include <algorithm>

#include "paged_work.cuh"

namespace mp {
namespace paged {

// One warp a (row, query head): the operator as its definition reads.
constexpr int kRowWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32) rows_plain(const Attend a) {
  const int Hq = a.H * a.G, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  // every request's offsets and length are looked at, those without rows too
  for (int64_t b = w; b < a.batch; b += (int64_t)gridDim.x * kRowWarps)
    if (lane == 0) request_of(a, (int)b);
  if (w >= (int64_t)a.rows * Hq) return;
  const int t = (int)(w / Hq), hq = (int)(w % Hq);
  if (t >= min(__ldg(a.cu + a.batch), a.rows)) return;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const Request r = request_of(a, lo);
  const int i = t - r.row0;
  if (i < 0 || i >= r.n) return;
  RowState<T, D> s;
  attend_row<T, D>(a, lo, r, i, hq, 0, r.len, s);
  T* o = reinterpret_cast<T*>(a.O + (int64_t)t * a.o_row_b + (int64_t)hq * a.o_head_b) + lane * (D / 32);
  const bool none = s.l == 0.f;
  const float inv = none ? 0.f : 1.f / s.l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = from_f32<T>(s.acc[e] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)t * Hq + hq] = none ? -INFINITY : (s.m + log2f(s.l)) / kLog2e;
}

static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

static Attend args_of(const mp_paged_cache& c, const mp_paged_attend_args& p) {
  Attend a{};
  const mp_paged_config& g = c.cfg;
  const int es = g.dtype == MP_F32 ? 4 : 2;
  a.K = static_cast<const char*>(c.K);
  a.V = static_cast<const char*>(c.V);
  a.page_b = g.page_stride * es;
  a.head_b = g.head_stride * es;
  a.tok_b = g.token_stride * es;
  a.num_pages = g.num_pages;
  a.page_shift = log2_of(g.page_tokens);
  a.H = g.kv_heads;
  a.G = p.q_heads / g.kv_heads;
  a.table = p.table;
  a.table_pages = p.table_pages;
  a.table_stride = p.table_stride;
  a.lens = p.lens;
  a.cu = p.cu;
  a.batch = p.batch;
  a.rows = p.rows;
  a.max_new = p.max_new ? p.max_new : p.rows;
  a.Q = static_cast<const char*>(p.Q);
  a.O = static_cast<char*>(p.O);
  a.q_row_b = p.q_row_stride * es;
  a.q_head_b = p.q_head_stride * es;
  a.o_row_b = p.o_row_stride * es;
  a.o_head_b = p.o_head_stride * es;
  a.scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)g.head_dim);
  a.cap = p.softcap;
  a.window = std::min(p.window, 1 << 30);
  a.full = (p.flags & MP_ATTEND_FULL) != 0;
  a.slopes = p.slopes;
  a.prefix = p.prefix;
  a.first_key = p.first_key;
  a.lse = p.lse;
  a.err = c.err;
  return a;
}

template <typename T>
static void launch_plain(const Attend& a, int D, cudaStream_t st) {
  const unsigned grid = (unsigned)(((int64_t)a.rows * a.H * a.G + kRowWarps - 1) / kRowWarps);
  if (D == 128) rows_plain<T, 128><<<grid, kRowWarps * 32, 0, st>>>(a);
  else rows_plain<T, 64><<<grid, kRowWarps * 32, 0, st>>>(a);
}

// How a call is done.  Few (token, head) rows a KV head: paged_rows.cu, blocks
// in clusters of one unit (one launch) while a block's part of the longest
// request that the table can hold stays short, shares over all SMs otherwise
// (two or three launches, the same time whatever the lengths).  More rows:
// paged_tiles.cu.  fp32: row by row.
constexpr int kFewCells = 32;          // rows that the few-rows kernel takes
constexpr int kFewParts = kMostParts;  // two blocks an SM
constexpr int kTilesParts = 148;       // one
constexpr int kClusterBlocks = 16;     // blocks of keys of a clustered block at most

struct Way {
  bool few, tiles;
  int cells, cluster, entries, rows, parts;
};

static Way way_of(const mp_paged_cache& c, const mp_paged_attend_args& p) {
  Way w{};
  const int G = p.q_heads / c.cfg.kv_heads, max_new = p.max_new ? p.max_new : p.rows;
  if (c.cfg.dtype == MP_F32) return w;
  if ((int64_t)max_new * G > kFewCells) {
    w.tiles = true;
    w.entries = p.rows / tiles_tokens(G) + p.batch;
    w.rows = kTilesRows;
    w.parts = kTilesParts;
    return w;
  }
  w.few = true;
  w.cells = max_new * G;
  const int64_t units = (int64_t)p.batch * c.cfg.kv_heads;
  const int64_t blocks = ((int64_t)p.table_pages * c.cfg.page_tokens + kFewBlock - 1) / kFewBlock;
  int k = 1;
  while (k < 8 && units * k < kFewParts) k *= 2;
  if (blocks <= (int64_t)kClusterBlocks * k && units * k <= (1 << 30)) {
    w.cluster = k;
    return w;
  }
  w.entries = p.rows / max_new + p.batch;
  w.rows = few_rows(w.cells);
  w.parts = kFewParts;
  return w;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The scratch of a split call: count, sums, entries, partial results.
static size_t lay_work(const Way& w, int D, void* base, Work* out) {
  if (w.entries == 0) return 0;
  size_t at = 256;
  const size_t before = at;
  at = align256(at + (size_t)(w.entries + 1) * sizeof(int64_t));
  const size_t entry = at;
  at = align256(at + (size_t)w.entries * sizeof(Entry));
  const size_t part = at;
  at = align256(at + (size_t)2 * w.parts * w.rows * (2 + D) * sizeof(float));
  if (out) {
    char* s = static_cast<char*>(base);
    out->count = reinterpret_cast<int32_t*>(s);
    out->before = reinterpret_cast<int64_t*>(s + before);
    out->entry = reinterpret_cast<Entry*>(s + entry);
    out->part = reinterpret_cast<float*>(s + part);
    out->parts = w.parts;
  }
  return at;
}

}  // namespace paged

size_t paged_attend_scratch_bytes(const mp_paged_cache& c, const mp_paged_attend_args& p) {
  if (p.batch == 0 || p.rows == 0) return 0;
  return paged::lay_work(paged::way_of(c, p), c.cfg.head_dim, nullptr, nullptr);
}

mp_status paged_attend_impl(const mp_paged_cache& c, const mp_paged_attend_args& p, void* scratch, size_t,
                            cudaStream_t st) {
  const paged::Attend a = paged::args_of(c, p);
  const paged::Way w = paged::way_of(c, p);
  cudaError_t e = cudaSuccess;
  paged::Work work{};
  paged::lay_work(w, c.cfg.head_dim, scratch, &work);
  if (w.few) {
    work.least = 4;
    e = paged::attend_few(a, c, work, w.cells, w.cluster, st);
  } else if (w.tiles) {
    work.least = 4;
    e = paged::attend_tiles(a, c, work, w.entries, st);
  } else {
    paged::launch_plain<float>(a, c.cfg.head_dim, st);
  }
  if (e == cudaSuccess) return cudaGetLastError() == cudaSuccess ? MP_OK : MP_ECUDA;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? MP_EUNSUPPORTED : MP_ECUDA;
}

}  // namespace mp
