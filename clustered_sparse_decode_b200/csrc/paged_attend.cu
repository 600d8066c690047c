// Attention of new tokens over a paged cache: the choice of kernel and its
// scratch.
#include <algorithm>

#include "paged_work.cuh"

namespace mp {
namespace paged {

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
  const int64_t row = (int64_t)p.q_heads * g.head_dim * es;    // in the place of strides that mean nothing
  if (p.rows == 1) a.q_row_b = a.o_row_b = row;
  if (p.q_heads == 1) a.q_head_b = a.o_head_b = row;
  a.scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)g.head_dim);
  a.cap = p.softcap;
  a.to_z = a.scale * kLog2e;
  const float huge = 0x1p126f;         // for caps and ratios that fp32 cannot hold: 0 times them stays 0
  a.to_u = a.cap > 0.f ? std::min(std::max(a.scale / a.cap, -huge), huge) : 0.f;
  a.cap2 = std::min(a.cap * kLog2e, huge);
  a.window = std::min(p.window, 1 << 30);
  a.full = (p.flags & MP_ATTEND_FULL) != 0;
  a.slopes = p.slopes;
  a.prefix = p.prefix;
  a.first_key = p.first_key;
  a.lse = p.lse;
  a.err = c.err;
  a.device = c.device;
  return a;
}

// How a call is done.  16-bit types with few (token, head) rows a KV head:
// paged_rows.cu; with more: paged_tiles.cu; fp32: paged_f32.cu, which has a kernel
// for up to 16 rows and one for more.  Few rows run as clusters of one unit (one
// launch, no scratch) while a block's part of the longest request that the table
// can hold stays short, otherwise with shares over all SMs (two or three launches,
// the same time whatever the lengths).
constexpr int kFewCells = 32;          // rows that the few-rows kernel takes
constexpr int kClusterBlocks = 16;     // blocks of keys of a clustered block at most

struct Way {
  enum { FEW, TILES, F32 } kind;
  int cells, cluster, entries, rows, tile, parts, least;
  bool pack;                           // Q is copied to the scratch first
};

// The many-rows kernel reads Q through a tensor map, whose strides are not 0: an
// expanded Q (rows or heads that stand on one another) is laid out in the scratch
// for it, 16 bytes a thread and turn.
__global__ void __launch_bounds__(256) pack_kernel(const Attend a, char* out, int vectors) {
  const int64_t heads = (int64_t)a.H * a.G, total = a.rows * heads * vectors;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += (int64_t)gridDim.x * 256) {
    const int64_t th = x / vectors, t = th / heads, h = th - t * heads;
    reinterpret_cast<uint4*>(out)[x] =
        *reinterpret_cast<const uint4*>(a.Q + t * a.q_row_b + h * a.q_head_b + (x - th * vectors) * 16);
  }
}

static Way way_of(const mp_paged_cache& c, const mp_paged_attend_args& p) {
  Way w{};
  const int G = p.q_heads / c.cfg.kv_heads, max_new = p.max_new ? p.max_new : p.rows;
  const int64_t cells = (int64_t)max_new * G;
  w.least = 1;
  if (c.cfg.dtype != MP_F32 && cells > kFewCells) {
    w.kind = Way::TILES;
    w.pack = (p.rows > 1 && p.q_row_stride == 0) || (p.q_heads > 1 && p.q_head_stride == 0);
    w.rows = kTilesRows;
    w.tile = tiles_tokens(G);
    w.parts = c.sms;                   // one block an SM
  } else {
    const bool f32 = c.cfg.dtype == MP_F32;
    w.kind = f32 ? Way::F32 : Way::FEW;
    w.cells = (int)(cells < 32 ? cells : 32);
    w.rows = f32 ? f32_rows(w.cells) : few_rows(w.cells);
    w.tile = f32 ? w.rows / G : max_new;
    const bool many = f32 && w.rows == kF32ManyRows;
    const int blocks_sm = f32 && !many ? 1 : 2;
    const int64_t units = (int64_t)p.batch * c.cfg.kv_heads * ((max_new + w.tile - 1) / w.tile);
    const int64_t blocks = ((int64_t)p.table_pages * c.cfg.page_tokens + kFewBlock - 1) / kFewBlock;
    int k = 1;
    while (k < 8 && units * k < blocks_sm * c.sms) k *= 2;
    if (!many && blocks <= (int64_t)kClusterBlocks * k && units * k <= (1 << 30)) {
      w.cluster = k;
      return w;
    }
    w.parts = blocks_sm * c.sms;
  }
  w.entries = p.rows / w.tile + p.batch;
  return w;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The scratch of a split call: count, sums, entries, partial results, queries (16-bit, q_rows of head dim D).
static size_t lay_work(const Way& w, int D, int64_t q_rows, void* base, Work* out, char** q) {
  if (w.entries == 0) return 0;
  size_t at = 256;
  const size_t before = at;
  at = align256(at + (size_t)(w.entries + 1) * sizeof(int64_t));
  const size_t entry = at;
  at = align256(at + (size_t)w.entries * sizeof(Entry));
  const size_t edge = at;
  at = align256(at + (size_t)(w.parts + 1) * sizeof(int64_t));
  const size_t edge_entry = at;
  at = align256(at + (size_t)(w.parts + 1) * sizeof(int32_t));
  const size_t part = at;
  at = align256(at + (size_t)2 * w.parts * w.rows * (2 + D) * sizeof(float));
  const size_t packed = at;
  if (w.pack) at = align256(at + (size_t)q_rows * D * 2);
  if (out) {
    char* s = static_cast<char*>(base);
    out->count = reinterpret_cast<int32_t*>(s);
    out->before = reinterpret_cast<int64_t*>(s + before);
    out->entry = reinterpret_cast<Entry*>(s + entry);
    out->edge = reinterpret_cast<int64_t*>(s + edge);
    out->edge_entry = reinterpret_cast<int32_t*>(s + edge_entry);
    out->part = reinterpret_cast<float*>(s + part);
    out->parts = w.parts;
    *q = s + packed;
  }
  return at;
}

}  // namespace paged

size_t paged_attend_scratch_bytes(const mp_paged_cache& c, const mp_paged_attend_args& p) {
  if (p.batch == 0 || p.rows == 0) return 0;
  return paged::lay_work(paged::way_of(c, p), c.cfg.head_dim, (int64_t)p.rows * p.q_heads, nullptr, nullptr, nullptr);
}

mp_status paged_attend_impl(const mp_paged_cache& c, const mp_paged_attend_args& p, void* scratch, size_t,
                            cudaStream_t st) {
  paged::Attend a = paged::args_of(c, p);
  const paged::Way w = paged::way_of(c, p);
  const int D = c.cfg.head_dim;
  cudaError_t e;
  paged::Work work{};
  char* q = nullptr;
  paged::lay_work(w, D, (int64_t)p.rows * p.q_heads, scratch, &work, &q);
  work.least = w.least;
  if (w.pack) {
    const int vectors = D * 2 / 16;
    const int64_t blocks = ((int64_t)p.rows * p.q_heads * vectors + 255) / 256;
    paged::pack_kernel<<<(unsigned)std::min<int64_t>(blocks, (int64_t)c.sms * 8), 256, 0, st>>>(a, q, vectors);
    if (cudaGetLastError() != cudaSuccess) return MP_ECUDA;
    a.Q = q;
    a.q_head_b = D * 2;
    a.q_row_b = a.q_head_b * p.q_heads;
  }
  if (w.kind == paged::Way::FEW) e = paged::attend_few(a, c, work, w.cells, w.cluster, st);
  else if (w.kind == paged::Way::TILES) e = paged::attend_tiles(a, c, work, st);
  else e = paged::attend_f32(a, c, work, w.rows, w.tile, w.cluster, st);
  if (e == cudaSuccess) return cudaGetLastError() == cudaSuccess ? MP_OK : MP_ECUDA;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? MP_EUNSUPPORTED : MP_ECUDA;
}

}  // namespace mp
