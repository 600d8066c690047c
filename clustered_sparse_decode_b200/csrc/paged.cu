// Paged cache: handle, step addresses, appending, gathering (attention in
// paged_attend.cu).
#include <cooperative_groups.h>
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <utility>

#include "paged_work.cuh"

namespace cg = cooperative_groups;

namespace mp {
namespace paged {

static inline int elem_bytes16(int dtype) { return dtype == MP_F32 ? 4 : 2; }

// ---------------------------------------------------------------------------
// Step addresses
// ---------------------------------------------------------------------------
// Every block repeats the scan over the requests (their new tokens and new
// pages), keeps its sums in shared memory, and then fills its share of the
// rows, each finding its request by bisection: no block waits for another's
// results.  A new page's id is written to the table by the row that starts it
// and computed, not read back, by all others.  In one cluster (as long as the
// rows are few, and whenever lengths or count are updated in place) a cluster
// barrier lies between the blocks' reads of the lengths and the writes of the
// new ones, so that in and out may be the same memory.  The work is a chain of
// loads and barriers, not bytes: 4.7 us for 16 requests of a token, 8.4 us for 256
// prompts of 250,000 tokens (3 MB of slots and positions).
constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;
constexpr int kPlanBatch = 8192;

struct Plan {
  mp_paged_plan_args p;
  int32_t page_shift, num_pages, clustered;
  int32_t* err;
};

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const Plan a) {
  extern __shared__ int32_t sm[];
  const int B = a.p.batch, P = 1 << a.page_shift;
  int32_t* cu = sm;                      // [B + 1] first row
  int32_t* pg = cu + B + 1;              // [B] new pages of the requests before
  int32_t* ln = pg + B;                  // [B] cached tokens
  __shared__ int64_t wsum[2][32];
  __shared__ int bad_any;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) bad_any = 0;
  const int count = __ldcg(a.p.free_count);
  int64_t rows0 = 0, pages0 = 0;         // of the requests of earlier rounds
  __syncthreads();
  for (int base = 0; base < B; base += blockDim.x) {
    const int b = base + tid;
    int len = 0, n = 0, need = 0;
    bool bad = false;
    if (b < B) {
      len = __ldcg(a.p.lens + b);
      n = __ldg(a.p.new_tokens + b);
      bad = len < 0 || n < 0 || (int64_t)len + n > (int64_t)a.p.table_pages * P || (int64_t)len + n > INT32_MAX;
      if (bad) len = n = 0;
      need = (int)(((int64_t)len + n + P - 1) >> a.page_shift) - (int)(((int64_t)len + P - 1) >> a.page_shift);
    }
    if (bad) bad_any = 1;
    int64_t sr = n, sp = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t r = __shfl_up_sync(kFull, sr, o), p = __shfl_up_sync(kFull, sp, o);
      if (lane >= o) { sr += r; sp += p; }
    }
    if (lane == 31) { wsum[0][warp] = sr; wsum[1][warp] = sp; }
    __syncthreads();
    int64_t br = rows0, bp = pages0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) { br += wsum[0][w]; bp += wsum[1][w]; }
      rows0 += wsum[0][w];
      pages0 += wsum[1][w];
    }
    if (b < B) {
      // sums past the tensors' ends are not used: the step is then refused below
      cu[b] = (int32_t)min(br + sr - n, (int64_t)INT32_MAX);
      pg[b] = (int32_t)min(bp + sp - need, (int64_t)INT32_MAX);
      ln[b] = len;
    }
    __syncthreads();
  }
  const bool fits = !bad_any && rows0 <= a.p.rows && count >= 0 && count <= a.p.free_capacity && pages0 <= count;
  const int total = fits ? (int)rows0 : 0;
  if (tid == 0) cu[B] = total;
  if (a.clustered) cg::this_cluster().sync();      // every block has read lengths and count
  else __syncthreads();

  if (blockIdx.x == 0) {
    for (int b = tid; b <= B; b += blockDim.x) {
      a.p.cu_out[b] = fits ? cu[b] : 0;
      if (b < B) {
        // on a refused step the lengths stay as they are, whatever they hold
        if (fits) a.p.lens_out[b] = ln[b] + cu[b + 1] - cu[b];
        else if (a.p.lens_out != a.p.lens) a.p.lens_out[b] = __ldcg(a.p.lens + b);
      }
    }
    if (tid == 0) {
      a.p.free_count_out[0] = fits ? count - (int)pages0 : count;
      if (!fits) set_error(a.err, E_CAPACITY);
    }
  }
  for (int t = blockIdx.x * blockDim.x + tid; t < a.p.rows; t += gridDim.x * blockDim.x) {
    int64_t slot = -1;
    int pos = 0;
    if (t < total) {
      int lo = 0, hi = B;                // the last request whose first row is at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      pos = ln[lo] + t - cu[lo];
      const int col = pos >> a.page_shift, held = (ln[lo] + P - 1) >> a.page_shift;
      const bool fresh = col >= held;
      int32_t* entry = a.p.table + (int64_t)lo * a.p.table_stride + col;
      int id = fresh ? __ldg(a.p.free_pages + (count - 1 - (pg[lo] + col - held))) : __ldcg(entry);
      if ((unsigned)id >= (unsigned)a.num_pages) {
        set_error(a.err, E_BAD_OFFSET);
        id = -1;
      }
      if (fresh && (pos & (P - 1)) == 0) *entry = id;
      if (id >= 0) slot = ((int64_t)id << a.page_shift) + (pos & (P - 1));
    }
    a.p.slots_out[t] = slot;
    a.p.positions_out[t] = pos;
  }
}

// ---------------------------------------------------------------------------
// Appending: rows [T, H, d] to their slots
// ---------------------------------------------------------------------------
// A copy by 16-byte vectors: consecutive threads take consecutive vectors of a
// row, `kCopies` loads of K and V in flight before the first store.  Bound by the
// memory, each byte read and written once: 16K tokens (8 heads of 128, bf16) to
// pages of 16, 134 MB, take 26.6 us, 5.0 TB/s; one, two or four copies in flight and
// more blocks make no difference of a microsecond.
constexpr int kCopyThreads = 256;
constexpr int kCopies = 4;

struct Append {
  const char* k;
  const char* v;
  char* K;
  char* V;
  int64_t row_b, in_head_b, page_b, head_b, tok_b;
  const int64_t* slots;
  int64_t total, limit;                  // vectors in all, slots in all
  int32_t H, vshift, page_shift;         // 2^vshift vectors of a head's row
  int32_t* err;
};

__device__ __forceinline__ uint4 ld_stream(const char* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kCopyThreads) append_kernel(const Append a) {
  const int64_t step = (int64_t)gridDim.x * kCopyThreads;
  for (int64_t x0 = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; x0 < a.total; x0 += step * kCopies) {
    uint4 k[kCopies], v[kCopies];
    int64_t dst[kCopies];
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int64_t x = x0 + c * step;
      dst[c] = -1;
      if (x >= a.total) continue;
      const int64_t rh = x >> a.vshift;
      const int64_t t = (uint64_t)rh <= 0xffffffffu ? (uint32_t)rh / (uint32_t)a.H : rh / a.H;
      const int h = (int)(rh - t * a.H);
      const int64_t vec = (x & ((1 << a.vshift) - 1)) * 16;
      const int64_t slot = __ldg(a.slots + t);
      if (slot < 0) continue;
      if (slot >= a.limit) {
        set_error(a.err, E_BAD_OFFSET);
        continue;
      }
      const int64_t src = t * a.row_b + h * a.in_head_b + vec;
      k[c] = ld_stream(a.k + src);
      v[c] = ld_stream(a.v + src);
      dst[c] = (slot >> a.page_shift) * a.page_b + h * a.head_b + (slot & ((1 << a.page_shift) - 1)) * a.tok_b + vec;
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      if (dst[c] < 0) continue;
      *reinterpret_cast<uint4*>(a.K + dst[c]) = k[c];
      *reinterpret_cast<uint4*>(a.V + dst[c]) = v[c];
    }
  }
}

// ---------------------------------------------------------------------------
// Gathering: requests' first n tokens as [B, H, n, d]
// ---------------------------------------------------------------------------
// A block copies kGatherRows tokens of one (request, head), K and V, by
// 16-byte vectors, `kCopies` rows of each thread in flight: 16 requests of 32K
// tokens, 4.3 GB, in 653 us, 6.57 TB/s, the rate of a plain copy.
constexpr int kGatherRows = 128;

struct Gather {
  const char* K;
  const char* V;
  char* Ko;
  char* Vo;
  int64_t page_b, head_b, tok_b;
  const int32_t* table;
  const int32_t* lens;
  int32_t table_pages, table_stride, num_pages, page_shift, H, n, vshift, chunks;
  int32_t least;                         // tokens that a request has to hold
  int32_t* err;
};

__global__ void __launch_bounds__(kCopyThreads) gather_kernel(const Gather a) {
  const int chunk = (int)(blockIdx.x % (unsigned)a.chunks), bh = (int)(blockIdx.x / (unsigned)a.chunks);
  const int b = bh / a.H, h = bh - b * a.H;
  const int held = __ldg(a.lens + b), len = min((int64_t)max(held, 0), (int64_t)a.table_pages << a.page_shift);
  if ((len != held || held < a.least) && threadIdx.x == 0) set_error(a.err, E_BAD_OFFSET);
  const int vec = threadIdx.x & ((1 << a.vshift) - 1), r0 = threadIdx.x >> a.vshift, dr = kCopyThreads >> a.vshift;
  const int end = min(a.n, (chunk + 1) * kGatherRows);
  const int64_t out0 = (int64_t)bh * a.n;
  for (int j0 = chunk * kGatherRows + r0; j0 < end; j0 += dr * kCopies) {
    uint4 k[kCopies], v[kCopies];
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int j = j0 + c * dr;
      k[c] = v[c] = make_uint4(0u, 0u, 0u, 0u);
      if (j >= end || j >= len) continue;
      const int page = __ldg(a.table + (int64_t)b * a.table_stride + (j >> a.page_shift));
      if ((unsigned)page >= (unsigned)a.num_pages) {
        set_error(a.err, E_BAD_OFFSET);
        continue;
      }
      const int64_t src = page * a.page_b + h * a.head_b + (j & ((1 << a.page_shift) - 1)) * a.tok_b + vec * 16;
      k[c] = ld_stream(a.K + src);
      v[c] = ld_stream(a.V + src);
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int j = j0 + c * dr;
      if (j >= end) continue;
      const int64_t dst = (((out0 + j) << a.vshift) + vec) * 16;
      *reinterpret_cast<uint4*>(a.Ko + dst) = k[c];
      *reinterpret_cast<uint4*>(a.Vo + dst) = v[c];
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// K or V as [page][head][64-column panel][token][64 columns], 128-byte
// swizzle; a box is `rows` tokens of one head's page, one panel or all.
static bool encode_pages(uint64_t* out, const mp_paged_cache& c, void* base, int rows, int panels) {
  auto fn = map_encoder();
  if (!fn) return false;
  const mp_paged_config& g = c.cfg;
  CUtensorMap tm;
  static_assert(sizeof(tm) == 16 * sizeof(uint64_t), "tensor map size");
  cuuint64_t gdim[5] = {64, (cuuint64_t)g.page_tokens, (cuuint64_t)(g.head_dim / 64), (cuuint64_t)g.kv_heads,
                        (cuuint64_t)g.num_pages};
  cuuint64_t gstride[4] = {(cuuint64_t)g.token_stride * 2, 128, (cuuint64_t)g.head_stride * 2,
                           (cuuint64_t)g.page_stride * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)panels, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const bool ok = fn(&tm, g.dtype == MP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base,
                     gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  std::memcpy(out, &tm, sizeof(tm));
  return ok;
}

static mp_status check_cache(const mp_paged_cache* c) {
  if (!c || !c->K || !c->V || !c->err) return MP_EINVAL;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return MP_ECUDA;
  return dev == c->device ? MP_OK : MP_EINVAL;
}

static mp_status launched() {
  return cudaGetLastError() == cudaSuccess ? MP_OK : MP_ECUDA;
}

}  // namespace paged
}  // namespace mp

using namespace mp;
using namespace mp::paged;

extern "C" {

mp_status mp_paged_init(const mp_paged_config* cfg, void* K, void* V, int32_t* d_err, mp_paged_cache* out) {
  if (!cfg || !K || !V || !d_err || !out) return MP_EINVAL;
  mp_paged_config g = *cfg;
  if (g.kv_heads < 1 || g.head_dim < 1 || g.num_pages < 1 || g.page_tokens < 1 || g.reserved != 0) return MP_EINVAL;
  if (g.dtype != MP_F32 && g.dtype != MP_BF16 && g.dtype != MP_F16) return MP_EINVAL;
  const int es = elem_bytes16(g.dtype);
  if (g.page_stride == 0 && g.head_stride == 0 && g.token_stride == 0) {
    g.token_stride = g.head_dim;
    g.head_stride = (int64_t)g.page_tokens * g.head_dim;
    g.page_stride = g.head_stride * g.kv_heads;
  }
  const int64_t st[3] = {g.page_stride, g.head_stride, g.token_stride};
  for (int64_t s : st)
    if (s < g.head_dim || (s * es) % 16 != 0) return MP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(d_err) % 4 != 0)
    return MP_EINVAL;
  if ((g.head_dim != 64 && g.head_dim != 128) || g.page_tokens < 16 || g.page_tokens > 256 ||
      (g.page_tokens & (g.page_tokens - 1)) != 0 || g.kv_heads > 65535)
    return MP_EUNSUPPORTED;
  // a pool of up to 2^40 bytes between neighbours along an axis is what a tensor map can address
  for (int64_t s : st)
    if (s >= ((int64_t)1 << 40) / es) return MP_EUNSUPPORTED;
  mp_paged_cache c;
  std::memset(&c, 0, sizeof(c));
  c.cfg = g;
  c.K = K;
  c.V = V;
  c.err = d_err;
  if (cudaGetDevice(&c.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, c.device) != cudaSuccess) {
    cudaGetLastError();
    return MP_ECUDA;
  }
  if (g.dtype != MP_F32) {
    const int panels = g.head_dim / 64, rows = std::min(g.page_tokens, 128);
    if (!encode_pages(c.maps + 16 * MAP_K16, c, K, 16, panels) || !encode_pages(c.maps + 16 * MAP_V16, c, V, 16, panels) ||
        !encode_pages(c.maps + 16 * MAP_KPAGE, c, K, rows, rows == 128 ? panels : 1) ||
        !encode_pages(c.maps + 16 * MAP_VPAGE, c, V, rows, rows == 128 ? panels : 1))
      return MP_ECUDA;
  }
  *out = c;
  return MP_OK;
}

mp_status mp_paged_plan(const mp_paged_cache* c, const mp_paged_plan_args* p, void* stream) {
  if (!c || !p) return MP_EINVAL;
  if (p->batch < 0 || p->table_pages < 0 || p->table_stride < p->table_pages || p->rows < 0 || p->free_capacity < 0 ||
      p->reserved != 0)
    return MP_EINVAL;
  if (!p->free_count || !p->free_count_out || !p->cu_out) return MP_EINVAL;
  if (p->batch > 0 && (!p->lens || !p->new_tokens || !p->lens_out)) return MP_EINVAL;
  if (p->rows > 0 && (!p->slots_out || !p->positions_out)) return MP_EINVAL;
  if (p->batch > 0 && p->table_pages > 0 && !p->table) return MP_EINVAL;
  if (p->free_capacity > 0 && !p->free_pages) return MP_EINVAL;
  if (p->batch > kPlanBatch) return MP_EUNSUPPORTED;
  mp_status s = check_cache(c);
  if (s != MP_OK) return s;
  Plan a{};
  a.p = *p;
  a.page_shift = log2_of(c->cfg.page_tokens);
  a.num_pages = c->cfg.num_pages;
  a.err = c->err;
  const int threads = std::max(p->batch, p->rows) <= 256 ? 256 : kPlanThreads;
  const int blocks = std::max(1, (int)(((int64_t)p->rows + threads - 1) / threads));
  const bool in_place = p->lens == p->lens_out || p->free_count == p->free_count_out;
  a.clustered = blocks <= kPlanCluster || in_place;
  const size_t smem = (size_t)(3 * p->batch + 1) * 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(std::min(blocks, a.clustered ? kPlanCluster : c->sms));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.clustered ? 1 : 0;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = smem > 40 * 1024
                            ? launch_large(plan_kernel, cfg, a, c->device, allowed, (size_t)(3 * kPlanBatch + 1) * 4)
                            : cudaLaunchKernelEx(&cfg, plan_kernel, (const Plan)a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MP_ECUDA;
  }
  return MP_OK;
}

mp_status mp_paged_append(const mp_paged_cache* c, const void* K_new, const void* V_new, int64_t row_stride,
                          int64_t head_stride, const int64_t* slots, int32_t rows, void* stream) {
  if (!c || rows < 0) return MP_EINVAL;
  if (rows > 0 && (!K_new || !V_new || !slots)) return MP_EINVAL;
  const int es = elem_bytes16(c->cfg.dtype);
  if (rows <= 1) row_stride = 0;                   // the stride of an axis of length 1 means nothing
  if (c->cfg.kv_heads == 1) head_stride = 0;
  if (row_stride < 0 || head_stride < 0 || (row_stride * es) % 16 != 0 || (head_stride * es) % 16 != 0 ||
      (reinterpret_cast<uintptr_t>(K_new) | reinterpret_cast<uintptr_t>(V_new)) % 16 != 0)
    return MP_EINVAL;
  mp_status s = check_cache(c);
  if (s != MP_OK) return s;
  if (rows == 0) return MP_OK;
  Append a{};
  a.k = static_cast<const char*>(K_new);
  a.v = static_cast<const char*>(V_new);
  a.K = static_cast<char*>(c->K);
  a.V = static_cast<char*>(c->V);
  a.row_b = row_stride * es;
  a.in_head_b = head_stride * es;
  a.page_b = c->cfg.page_stride * es;
  a.head_b = c->cfg.head_stride * es;
  a.tok_b = c->cfg.token_stride * es;
  a.slots = slots;
  a.H = c->cfg.kv_heads;
  a.vshift = log2_of(c->cfg.head_dim * es / 16);
  a.total = ((int64_t)rows * a.H) << a.vshift;
  a.page_shift = log2_of(c->cfg.page_tokens);
  a.limit = (int64_t)c->cfg.num_pages * c->cfg.page_tokens;
  a.err = c->err;
  const int64_t blocks = (a.total + kCopyThreads - 1) / kCopyThreads;
  const int grid = (int)std::min<int64_t>(blocks, (int64_t)c->sms * 8);
  append_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

static mp_status gather(const mp_paged_cache* c, int32_t batch, const int32_t* table, int32_t table_pages,
                        int32_t table_stride, const int32_t* lens, int32_t n, int32_t least, void* K_out, void* V_out,
                        void* stream) {
  if (!c || batch < 0 || n < 0 || table_pages < 0 || table_stride < table_pages) return MP_EINVAL;
  if (n > (int64_t)table_pages * c->cfg.page_tokens) return MP_EINVAL;
  if (batch > 0 && n > 0 && (!table || !lens || !K_out || !V_out)) return MP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(K_out) | reinterpret_cast<uintptr_t>(V_out)) % 16 != 0) return MP_EINVAL;
  mp_status s = check_cache(c);
  if (s != MP_OK) return s;
  if (batch == 0 || n == 0) return MP_OK;
  const int es = elem_bytes16(c->cfg.dtype);
  Gather a{};
  a.K = static_cast<const char*>(c->K);
  a.V = static_cast<const char*>(c->V);
  a.Ko = static_cast<char*>(K_out);
  a.Vo = static_cast<char*>(V_out);
  a.page_b = c->cfg.page_stride * es;
  a.head_b = c->cfg.head_stride * es;
  a.tok_b = c->cfg.token_stride * es;
  a.table = table;
  a.lens = lens;
  a.table_pages = table_pages;
  a.table_stride = table_stride;
  a.num_pages = c->cfg.num_pages;
  a.page_shift = log2_of(c->cfg.page_tokens);
  a.H = c->cfg.kv_heads;
  a.n = n;
  a.vshift = log2_of(c->cfg.head_dim * es / 16);
  a.chunks = (n - 1) / kGatherRows + 1;
  a.least = least;
  a.err = c->err;
  const int64_t grid = (int64_t)batch * a.H * a.chunks;
  if (grid > INT32_MAX) return MP_EUNSUPPORTED;
  gather_kernel<<<(unsigned)grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

mp_status mp_paged_gather(const mp_paged_cache* c, int32_t batch, const int32_t* table, int32_t table_pages,
                          int32_t table_stride, const int32_t* lens, int32_t n, void* K_out, void* V_out, void* stream) {
  return gather(c, batch, table, table_pages, table_stride, lens, n, 0, K_out, V_out, stream);
}

mp_status mp_paged_gather_whole(const mp_paged_cache* c, int32_t batch, const int32_t* table, int32_t table_pages,
                                int32_t table_stride, const int32_t* lens, int32_t n, void* K_out, void* V_out,
                                void* stream) {
  return gather(c, batch, table, table_pages, table_stride, lens, n, n, K_out, V_out, stream);
}

// Whether two of the d-element rows at i row + j head, |i| < rows, |j| < heads, can
// be less than d elements apart, the second set `shift` elements behind the first
// (0: one set, and a row is not compared with itself).
static bool rows_meet(int64_t shift, int64_t rows, int64_t heads, int64_t row, int64_t head, int64_t d) {
  using wide = __int128;
  if (rows == 1) row = 0;
  if (heads == 1) head = 0;
  if (shift == 0 && (row >= (wide)(heads - 1) * head + d || rows == 1) && (head >= d || heads == 1)) return false;
  if (shift == 0 && (head >= (wide)(rows - 1) * row + d || heads == 1) && (row >= d || rows == 1)) return false;
  // where one axis steps over all of the other, few pairs can be near; otherwise the shorter is gone through
  const bool over = row >= (wide)(heads - 1) * head + d, under = head >= (wide)(rows - 1) * row + d;
  if (!over && (under || heads < rows)) {
    std::swap(rows, heads);
    std::swap(row, head);
  }
  int64_t i0 = 1 - rows, i1 = rows;
  if (over || under) {
    const wide q = -(wide)shift / row;
    i0 = (int64_t)std::max<wide>(i0, q - 1);
    i1 = (int64_t)std::min<wide>(i1, q + 2);
  }
  for (int64_t i = i0; i < i1; ++i) {
    const wide at = (wide)shift + (wide)i * row;
    const wide near = head > 0 ? -at / head : 0;         // the j that brings the two rows nearest, or its neighbour
    for (wide j = near - 1; j <= near + 1; ++j) {
      if (j <= -heads || j >= heads || (shift == 0 && i == 0 && j == 0)) continue;
      const wide apart = at + j * head;
      if (apart < d && apart > -d) return true;
    }
  }
  return false;
}

// Whether O's rows meet Q's.  Rows of unlike strides in one another's span count as meeting.
static bool output_meets_input(const mp_paged_attend_args& p, int d, int es) {
  const int64_t qr = p.rows > 1 ? p.q_row_stride : 0, qh = p.q_heads > 1 ? p.q_head_stride : 0;
  const int64_t orow = p.rows > 1 ? p.o_row_stride : 0, oh = p.q_heads > 1 ? p.o_head_stride : 0;
  const __int128 q0 = reinterpret_cast<uintptr_t>(p.Q), o0 = reinterpret_cast<uintptr_t>(p.O), t = p.rows - 1, h = p.q_heads - 1;
  if (q0 + (t * qr + h * qh + d) * es <= o0 || o0 + (t * orow + h * oh + d) * es <= q0) return false;
  if (qr != orow || qh != oh || o0 == q0) return true;
  return rows_meet((int64_t)(o0 - q0) / es, p.rows, p.q_heads, qr, qh, d);
}

static mp_status check_attend(const mp_paged_cache* c, const mp_paged_attend_args* p) {
  if (!c || !p) return MP_EINVAL;
  const mp_paged_config& g = c->cfg;
  if (p->batch < 0 || p->rows < 0 || p->max_new < 0 || p->max_new > p->rows || p->table_pages < 0 ||
      p->table_stride < p->table_pages || p->q_heads < 1 || g.kv_heads < 1 || p->q_heads % g.kv_heads != 0)
    return MP_EINVAL;
  if (p->batch > 0 && p->rows > 0 && (!p->lens || !p->cu || !p->Q || !p->O || (p->table_pages > 0 && !p->table)))
    return MP_EINVAL;
  const int es = elem_bytes16(g.dtype);
  // (the stride of an axis of length 1 means nothing)
  const int64_t rows_st[2] = {p->q_row_stride, p->o_row_stride}, heads_st[2] = {p->q_head_stride, p->o_head_stride};
  for (int i = 0; i < 2; ++i) {
    if (p->rows > 1 && (rows_st[i] < 0 || (rows_st[i] * es) % 16 != 0)) return MP_EINVAL;
    if (p->q_heads > 1 && (heads_st[i] < 0 || (heads_st[i] * es) % 16 != 0)) return MP_EINVAL;
  }
  if ((reinterpret_cast<uintptr_t>(p->Q) | reinterpret_cast<uintptr_t>(p->O)) % 16 != 0) return MP_EINVAL;
  if ((p->rows > 1 && p->o_row_stride < g.head_dim) || (p->q_heads > 1 && p->o_head_stride < g.head_dim)) return MP_EINVAL;
  if (!std::isfinite(p->scale) || !std::isfinite(p->softcap) || p->softcap < 0.f || p->window < 0 ||
      (p->flags & ~MP_ATTEND_FULL) != 0)
    return MP_EINVAL;
  const int G = p->q_heads / g.kv_heads;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || p->batch > 65535 || p->rows > (1 << 24) ||
      (int64_t)p->table_pages * g.page_tokens > (1 << 30))
    return MP_EUNSUPPORTED;
  // rows of O that fall on one another would be written by several blocks
  if (p->batch > 0 && p->rows > 0 && rows_meet(0, p->rows, p->q_heads, p->o_row_stride, p->o_head_stride, g.head_dim))
    return MP_EINVAL;
  return MP_OK;
}

mp_status mp_paged_attend_scratch(const mp_paged_cache* c, const mp_paged_attend_args* p, size_t* bytes) {
  if (!bytes) return MP_EINVAL;
  mp_status s = check_attend(c, p);
  if (s != MP_OK) return s;
  *bytes = paged_attend_scratch_bytes(*c, *p);
  return MP_OK;
}

mp_status mp_paged_attend(const mp_paged_cache* c, const mp_paged_attend_args* p, void* d_scratch,
                          size_t scratch_bytes, void* stream) {
  mp_status s = check_attend(c, p);
  if (s != MP_OK) return s;
  if (reinterpret_cast<uintptr_t>(d_scratch) % 256 != 0) return MP_EINVAL;
  // (a row that is done again reads its queries after other rows' results are written)
  if (p->batch > 0 && p->rows > 0 && output_meets_input(*p, c->cfg.head_dim, elem_bytes16(c->cfg.dtype))) return MP_EINVAL;
  if ((s = check_cache(c)) != MP_OK) return s;
  if (p->batch == 0 || p->rows == 0) return MP_OK;
  const size_t need = paged_attend_scratch_bytes(*c, *p);
  if (need > 0 && !d_scratch) return MP_EINVAL;
  if (scratch_bytes < need) return MP_ENOSPC;
  return paged_attend_impl(*c, *p, d_scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}

mp_status mp_paged_check_error(const mp_paged_cache* c, int32_t* code, void* stream) {
  mp_status s = check_cache(c);
  if (s != MP_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t h = 0;
  if (cudaMemcpyAsync(&h, c->err, sizeof(h), cudaMemcpyDeviceToHost, st) != cudaSuccess) return MP_ECUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MP_ECUDA;
  if (code) *code = h;
  if (h == 0) return MP_OK;
  if (cudaMemsetAsync(c->err, 0, sizeof(h), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return MP_ECUDA;
  return MP_EDEVICE;
}

}  // extern "C"
