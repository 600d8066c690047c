// Attention over a paged cache in fp32, any number of rows.
//
// fp32 products have no fast matrix instruction that keeps their precision, so
// both products run on the ordinary multiply-add units.  A block's 4 warps take
// every fourth 16-key tile of its share; each streams its tiles through its own
// ring of shared-memory stages with cp.async (rows behind the last token are
// filled with zeros).  Scores: lane l computes key l % 16 against half of the
// tile's rows (4, 8 or 16 (token, head) rows in all), keys from rows padded by 16
// bytes so that 8 lanes' vector loads fall into different banks, queries
// broadcast.  Output: lane l owns columns [l D/32, (l + 1) D/32) of all rows, the
// weights come back from shared memory.  Single tokens are bound by reading the
// cache once; 16 rows by the multiply-adds and their shared-memory reads (one
// vector read a 4 multiply-adds a lane).  The tiny cache (1 head of 64, 4 query
// heads, 2048 tokens) takes 12.3 us, of which 8 are left with 16 tokens: the launch
// and the chain of first loads.
#include <type_traits>

#include "paged_work.cuh"
#include "stream_common.cuh"

namespace mp {
namespace paged {

constexpr int kF32Warps = 4;
constexpr int kF32Tile = 16;                       // keys a tile
static_assert(kFewBlock == kF32Warps * kF32Tile, "a block of the share-out is a tile a warp");

struct F32 {
  Attend a;
  Work w;
  int tile;                                        // tokens a tile
  int cluster;                                     // > 0: that many blocks share a unit
};

template <int D, int RH>                           // RH rows a half warp
struct F32Cfg {
  static constexpr int ROWS = 2 * RH;
  static constexpr int KP = D + 4;                                    // floats between rows of keys
  static constexpr int STAGE = kF32Tile * (KP + D) * 4;
  static constexpr int NS = 3;
  static constexpr int WARP = NS * STAGE + kF32Tile * ROWS * 4;       // ring and weights
  static constexpr int PITCH = D + 8;
  static constexpr int OFF_Q = kF32Warps * WARP;                      // [ROWS][D]
  static constexpr int OFF_ML = OFF_Q + ROWS * D * 4;
  static constexpr int OFF_UNIT = OFF_ML + kF32Warps * 2 * ROWS * 4;
  static constexpr int OFF_BAD = OFF_UNIT + 2 * ROWS * 4;
  static constexpr int SMEM = OFF_BAD + (int)sizeof(Again<ROWS>);
  static_assert(ROWS * PITCH * 4 <= NS * STAGE, "a warp's numerators fit its ring");
  static_assert(SMEM <= 227 * 1024 && WARP % 16 == 0 && STAGE % 16 == 0, "shared memory");
};

template <int D, int RH>
__global__ void __launch_bounds__(kF32Warps * 32) f32_kernel(const F32 f) {
  using C = F32Cfg<D, RH>;
  constexpr int ROWS = C::ROWS, NS = C::NS, E = D / 32;
  const Attend& a = f.a;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, key = lane & 15;
  float* ring = reinterpret_cast<float*>(smem + warp * C::WARP);
  float* pw = reinterpret_cast<float*>(smem + warp * C::WARP + NS * C::STAGE);     // [16 keys][ROWS]
  float* q = reinterpret_cast<float*>(smem + C::OFF_Q);
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
  Again<ROWS>* again = reinterpret_cast<Again<ROWS>*>(smem + C::OFF_BAD);
  const uint32_t ring_s = sc::smem_u32(ring);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int64_t x = 0, x1 = 1;
  int e = 0;
  const int part = f.cluster ? (int)(blockIdx.x % f.cluster) : (int)blockIdx.x;
  if (!f.cluster) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    x = f.w.edge[part];
    x1 = f.w.edge[part + 1];
    if (x >= x1) return;
    e = f.w.edge_entry[part];
  }
  const int64_t start = x;

  while (x < x1) {
    Settle st;
    int blk0, blk1, k0;
    int64_t u0 = 0, u1 = 1;
    Entry en;
    if (f.cluster) {
      const int u = blockIdx.x / f.cluster, tiles = (a.max_new + f.tile - 1) / f.tile;
      en.tile = u % tiles;
      st.h = u / tiles % a.H;
      en.b = u / tiles / a.H;
    } else {
      while (f.w.before[e + 1] * a.H <= x) ++e;
      const int64_t n = f.w.before[e + 1] - f.w.before[e], first = f.w.before[e] * a.H;
      en = f.w.entry[e];
      st.h = (int)((x - first) / n);
      u0 = first + st.h * n;
      u1 = u0 + n;
    }
    st.b = en.b;
    st.r = request_of(a, en.b);
    st.i0 = en.tile * f.tile;
    st.cells = max(0, min(st.r.n - st.i0, f.tile)) * a.G;
    const int prefix = prefix_of(a, en.b);
    if (f.cluster) span_of(a, st.r, en.b, st.i0, min(st.r.n, st.i0 + f.tile), kFewBlock, en);
    k0 = en.k0;
    blk0 = f.cluster ? (int)((int64_t)en.n * part / f.cluster) : (int)(x - u0);
    blk1 = f.cluster ? (int)((int64_t)en.n * (part + 1) / f.cluster) : (int)(min(x1, u1) - u0);
    // this lane's rows
    int lo[RH], hi[RH], pos[RH], low = INT32_MAX, top = 0;
    float slope[RH];
#pragma unroll
    for (int k = 0; k < RH; ++k) {
      const int row = half * RH + k;
      lo[k] = 0;
      hi[k] = 0;
      pos[k] = 0;
      slope[k] = 0.f;
      if (row >= st.cells) continue;
      const Interval v = interval_of(a, st.r, prefix, st.i0 + row / a.G);
      lo[k] = v.lo;
      hi[k] = v.hi;
      pos[k] = v.pos;
      if (a.slopes) slope[k] = __ldg(a.slopes + st.h * a.G + row % a.G);
      if (v.hi > v.lo) {
        low = min(low, v.lo);
        top = max(top, v.hi);
      }
    }
    low = __reduce_min_sync(kFull, low);
    top = __reduce_max_sync(kFull, top);
    st.key0 = k0 + blk0 * kFewBlock;
    st.key1 = min(k0 + blk1 * kFewBlock, top);
    if (tid == 0) {
      again->low = low;
      again->high = top;
    }
    for (int c = tid; c < ROWS * D / 4; c += kF32Warps * 32) {
      const int row = c / (D / 4), d = c % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < st.cells)
        v = *reinterpret_cast<const float4*>(a.Q + (int64_t)(st.r.row0 + st.i0 + row / a.G) * a.q_row_b +
                                             (int64_t)(st.h * a.G + row % a.G) * a.q_head_b + d * 16);
      reinterpret_cast<float4*>(q)[c] = v;
    }
    __syncthreads();

    // --- this warp's tiles: keys key0 + 16 (warp + 4 i)
    const int first = st.key0 + warp * kF32Tile;
    const int tiles = st.key1 > first ? (st.key1 - first + kFewBlock - 1) / kFewBlock : 0;
    int pages = -1;                    // lane l: the page of tile 32 (i / 32) + l
    uint32_t void_stages = 0;
    auto fetch = [&](int i) {          // always one group, empty behind the last tile
      if (i < tiles) {
        if ((i & 31) == 0) pages = i + lane < tiles && first + (i + lane) * kFewBlock + kF32Tile > low    // unseen: maybe no page
                                      ? page_of(a, en.b, first + (i + lane) * kFewBlock) : -1;
        const int page = __shfl_sync(kFull, pages, i & 31), j = first + i * kFewBlock, s = i % NS;
        void_stages = page < 0 ? void_stages | 1u << s : void_stages & ~(1u << s);
        if (page >= 0) {
          const int64_t off = page * a.page_b + st.h * a.head_b + (j & ((1 << a.page_shift) - 1)) * a.tok_b;
#pragma unroll 4
          for (int c = lane; c < kF32Tile * D / 4; c += 32) {
            const int row = c / (D / 4), d = c % (D / 4);
            const bool in = j + row < st.r.len;
            const int64_t at = off + (in ? row * a.tok_b : 0) + d * 16;
            sc::cp16(ring_s + s * C::STAGE + (row * C::KP + d * 4) * 4, a.K + at, in);
            sc::cp16(ring_s + s * C::STAGE + (kF32Tile * C::KP + row * D + d * 4) * 4, a.V + at, in);
          }
        }
      }
      sc::cp_commit();
    };
    float acc[ROWS][E], m[RH], l[RH];
#pragma unroll
    for (int k = 0; k < RH; ++k) { m[k] = -INFINITY; l[k] = 0.f; }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < E; ++c) acc[r][c] = 0.f;
    for (int i = 0; i < NS - 1; ++i) fetch(i);
    for (int i = 0; i < tiles; ++i) {
      fetch(i + NS - 1);
      asm volatile("cp.async.wait_group %0;\n" ::"n"(NS - 1) : "memory");
      __syncwarp();
      const int s = i % NS, j = first + i * kFewBlock + key;
      if (!(void_stages >> s & 1u)) {
        const float* kr = ring + s * (C::STAGE / 4) + key * C::KP;
        const float* vr = ring + s * (C::STAGE / 4) + kF32Tile * C::KP + lane * E;
        float z[RH];
#pragma unroll
        for (int k = 0; k < RH; ++k) z[k] = 0.f;
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
          const float4 kv = *reinterpret_cast<const float4*>(kr + d);
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const float4 qv = *reinterpret_cast<const float4*>(q + (half * RH + k) * D + d);
            z[k] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, z[k]))));
          }
        }
        bool grow = false;
#pragma unroll
        for (int k = 0; k < RH; ++k) {
          z[k] = j < lo[k] || j >= hi[k] ? -INFINITY : score2(a, z[k], slope[k], pos[k] - j);
          grow |= z[k] > m[k] + 8.f;
        }
        if (__any_sync(kFull, grow)) {
          float keep[RH];
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            float t = z[k];
#pragma unroll
            for (int o = 8; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
            const float nm = fmaxf(m[k], t);
            keep[k] = m[k] == -INFINITY ? 0.f : exp2f(m[k] - nm);
            m[k] = nm;
            l[k] *= keep[k];
          }
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const float kp = __shfl_sync(kFull, keep[r % RH], r < RH ? 0 : 16);
#pragma unroll
            for (int c = 0; c < E; ++c) acc[r][c] *= kp;
          }
        }
#pragma unroll
        for (int k = 0; k < RH; ++k) {
          const float p = exp2f(z[k] - (m[k] == -INFINITY ? 0.f : m[k]));
          l[k] += p;
          pw[key * ROWS + half * RH + k] = p;
        }
        __syncwarp();
#pragma unroll 4
        for (int t = 0; t < kF32Tile; ++t) {
          float v[E], p[ROWS];
#pragma unroll
          for (int c = 0; c < E; c += 2) *reinterpret_cast<float2*>(v + c) = *reinterpret_cast<const float2*>(vr + t * D + c);
#pragma unroll
          for (int r = 0; r < ROWS; r += 4) *reinterpret_cast<float4*>(p + r) = *reinterpret_cast<const float4*>(pw + t * ROWS + r);
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int c = 0; c < E; ++c) acc[r][c] = fmaf(p[r], v[c], acc[r][c]);
        }
      }
      __syncwarp();                    // all lanes have read the stage and the weights
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int k = 0; k < RH; ++k) {
      float s = l[k];
#pragma unroll
      for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      if (key == 0) {
        const int row = half * RH + k;
        ml[(warp * 2) * ROWS + row] = s != s ? s : m[k];
        ml[(warp * 2 + 1) * ROWS + row] = s;
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < E; ++c) ring[r * C::PITCH + lane * E + c] = acc[r][c];
    st.cluster = f.cluster;
    st.part = part;
    st.whole = !f.cluster && x == u0 && min(x1, u1) == u1;
    st.slot = f.cluster ? nullptr : f.w.part + (2 * (int64_t)part + (x == start ? 0 : 1)) * (int64_t)ROWS * (2 + D);
    settle<float, D, ROWS, C::PITCH, kF32Warps>(a, st, ml, reinterpret_cast<float*>(smem), C::WARP / 4,
                                                reinterpret_cast<float*>(smem + C::OFF_UNIT),
                                                again);
    if (f.cluster) return;
    __syncthreads();
    x = min(x1, u1);
  }
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
// More rows than a warp can hold share a block: 8 warps of 8 rows read the same
// 32-key tiles, which all threads load (cp.async, two stages).  Lane l computes
// key l against its warp's rows, then owns D / 32 columns of their outputs; no
// warp needs another's results.  Two blocks an SM, 16 warps to hide the latency
// of the multiply-adds: three prompts of up to 1164 tokens (32 query heads on 8 of
// 128) take 0.54 ms, 16 TFLOP/s of useful operations; the key-sharing kernel above,
// 4 warps an SM, took 1.39.
constexpr int kManyWarps = 8;
constexpr int kManyHeld = 8;                       // rows a warp
constexpr int kManyRows = kManyWarps * kManyHeld;
constexpr int kManyTile = 32;                      // keys a tile
static_assert(kManyRows == kF32ManyRows && kFewBlock % kManyTile == 0, "rows of a unit, tiles of a block");

template <int D>
struct ManyCfg {
  static constexpr int KP = D + 4;
  static constexpr int STAGE = kManyTile * (KP + D) * 4;
  static constexpr int OFF_Q = 2 * STAGE;                             // [64 rows][D]
  static constexpr int OFF_P = OFF_Q + kManyRows * D * 4;             // [warps][32 keys][8 rows]
  static constexpr int OFF_ROW = OFF_P + kManyWarps * kManyTile * kManyHeld * 4;   // [64 rows] first key, end, position, slope
  static constexpr int SMEM = OFF_ROW + kManyRows * 16;
  static_assert(2 * SMEM <= 225 * 1024, "two blocks an SM");
};

// A warp's row of a unit: its result, or its state for the joining.  Lane l holds
// the elements [l * D/32, (l + 1) * D/32).
template <int D>
struct ManyPut {
  int row0, h;                         // the unit's first row of Q, KV head
  float* slot;                         // of a partial result; null: the unit is whole
  __device__ __forceinline__ void operator()(const Attend& a, int row, float top, float sum, const float* v) const {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, hq = h * a.G + row % a.G;
    const int64_t t = row0 + row / a.G;
    const bool none = sum == 0.f;
    if (!slot) {
      float* o = reinterpret_cast<float*>(a.O + t * a.o_row_b + (int64_t)hq * a.o_head_b) + lane * E;
#pragma unroll
      for (int c = 0; c < E; ++c) o[c] = none ? 0.f : v[c] / sum;
      if (a.lse && lane == 0) a.lse[t * a.H * a.G + hq] = none ? -INFINITY : (top + log2f(sum)) / kLog2e;
    } else {
#pragma unroll
      for (int c = 0; c < E; ++c) slot[2 * kManyRows + row * D + lane * E + c] = v[c];
      if (lane == 0) {
        slot[row] = none ? -INFINITY : top;
        slot[kManyRows + row] = sum;
      }
    }
  }
};

// Rows with a finite sum and a numerator that is not (mend_rows), `again` of this
// warp's: ml holds their maxima and sums, num their numerators.
template <int D>
__device__ __noinline__ void many_again(const Attend& a, int b, const Request r, int i0, int h, int cells, int key0, int key1,
                                        int low, int high, uint32_t again, const float* ml, const float* num,
                                        const ManyPut<D> put) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, prefix = prefix_of(a, b);
  const int rows = min(kManyHeld, cells - warp * kManyHeld);
  again &= rows > 0 ? (1u << rows) - 1 : 0u;
  if (again == 0) return;
  int c0 = key0, c1 = min(key1, r.len), common[E] = {};     // the keys that all of them see
  for (uint32_t x = again; x; x &= x - 1) {
    const Interval v = interval_of(a, r, prefix, i0 + (warp * kManyHeld + __ffs(x) - 1) / a.G);
    c0 = max(c0, v.lo);
    c1 = min(c1, v.hi);
  }
  c1 = max(c0, c1);
  odd_values<float, D>(a, b, h, c0, c1, low, high, common, nullptr);
  while (again) {
    Rows4 rows;
    int at[4];
    float v[4][E] = {};
    rows.n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!again) continue;
      at[k] = __ffs(again) - 1;
      again &= again - 1;
      const int row = warp * kManyHeld + at[k];
      rows.i[k] = i0 + row / a.G;
      rows.hq[k] = h * a.G + row % a.G;
      rows.base[k] = ml[at[k]] + log2f(ml[kManyHeld + at[k]]);
      rows.n = k + 1;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = num[at[k] * D + lane * E + e];
    }
    const uint32_t done = mend_rows<float, D>(a, b, r, rows, key0, key1, low, high, c0, c1, common, v, nullptr);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= rows.n) continue;
      const bool one = done >> k & 1u;
      put(a, warp * kManyHeld + at[k], one ? rows.base[k] : ml[at[k]], one ? 1.f : ml[kManyHeld + at[k]], v[k]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kManyWarps * 32, 2) f32_many_kernel(const F32 f) {
  using C = ManyCfg<D>;
  constexpr int E = D / 32, RW = kManyHeld;
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  const Attend& a = f.a;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* q = reinterpret_cast<float*>(smem + C::OFF_Q) + warp * RW * D;
  float* pw = reinterpret_cast<float*>(smem + C::OFF_P) + warp * kManyTile * RW;
  int4* rows = reinterpret_cast<int4*>(smem + C::OFF_ROW) + warp * RW;
  const uint32_t base = sc::smem_u32(smem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int part = blockIdx.x;
  const int64_t start = f.w.edge[part], x1 = f.w.edge[part + 1];
  int64_t x = start;
  if (x >= x1) return;
  int e = f.w.edge_entry[part];

  while (x < x1) {
    while (f.w.before[e + 1] * a.H <= x) ++e;
    const int64_t n = f.w.before[e + 1] - f.w.before[e], first = f.w.before[e] * a.H;
    const Entry en = f.w.entry[e];
    const int h = (int)((x - first) / n);
    const int64_t u0 = first + h * n, u1 = u0 + n, end = min(x1, u1);
    const Request r = request_of(a, en.b);
    const int i0 = en.tile * f.tile, cells = min(r.n - i0, f.tile) * a.G, prefix = prefix_of(a, en.b);
    const int key0 = en.k0 + (int)(x - u0) * kFewBlock;
    // the warp's rows, and the keys they see together
    int from = INT32_MAX, to = 0;
    if (lane < RW) {
      const int row = warp * RW + lane;
      int4 x4 = make_int4(0, 0, 0, 0);
      if (row < cells) {
        const Interval v = interval_of(a, r, prefix, i0 + row / a.G);
        x4 = make_int4(v.lo, v.hi, v.pos, a.slopes ? __float_as_int(__ldg(a.slopes + h * a.G + row % a.G)) : 0);
        if (v.hi > v.lo) {
          from = v.lo;
          to = v.hi;
        }
      }
      rows[lane] = x4;
    }
    from = __reduce_min_sync(kFull, from);
    to = __reduce_max_sync(kFull, to);
    int low = INT32_MAX, top = 0;      // keys that any row of the block sees
    for (int row = lane; row < cells; row += 32) {
      const Interval v = interval_of(a, r, prefix, i0 + row / a.G);
      if (v.hi > v.lo) {
        low = min(low, v.lo);
        top = max(top, v.hi);
      }
    }
    low = __reduce_min_sync(kFull, low);
    top = __reduce_max_sync(kFull, top);
    for (int c = tid; c < kManyRows * D / 4; c += kManyWarps * 32) {
      const int row = c / (D / 4), d = c % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < cells)
        v = *reinterpret_cast<const float4*>(a.Q + (int64_t)(r.row0 + i0 + row / a.G) * a.q_row_b +
                                             (int64_t)(h * a.G + row % a.G) * a.q_head_b + d * 16);
      reinterpret_cast<float4*>(smem + C::OFF_Q)[c] = v;
    }
    const int tiles = (int)(end - x) * (kFewBlock / kManyTile);
    uint32_t empty = 0;                // halves of the stages' tiles whose page is bad: nothing of them is used
    // a tile lies in one page or in two of 16 tokens; their numbers are asked for a tile ahead of its loads
    const int32_t* table = a.table + (int64_t)en.b * a.table_stride;
    // (one that no row sees counts as empty: its table entry need not be valid any more)
    constexpr int kUnseen = INT32_MIN;
    int page0 = kUnseen, page1 = kUnseen;
    auto look_up = [&](int t) {
      const int j = key0 + t * kManyTile;
      const bool see0 = t < tiles && j < top && j + 16 > low, see1 = t < tiles && j + 16 < top && j + 32 > low;
      page0 = see0 ? __ldg(table + (j >> a.page_shift)) : kUnseen;
      page1 = see1 ? __ldg(table + ((j + 16) >> a.page_shift)) : kUnseen;
    };
    auto fetch = [&](int t) {          // always one group
      if (t < tiles) {
        const int j0 = key0 + t * kManyTile, s = t & 1, mask = (1 << a.page_shift) - 1;
        const bool bad0 = (unsigned)page0 >= (unsigned)a.num_pages, bad1 = (unsigned)page1 >= (unsigned)a.num_pages;
        if ((bad0 && page0 != kUnseen) || (bad1 && page1 != kUnseen)) set_error(a.err, E_BAD_OFFSET);
        empty = (empty & ~(3u << (2 * s))) | (bad0 ? 1u << (2 * s) : 0u) | (bad1 ? 2u << (2 * s) : 0u);
        const int64_t at0 = (bad0 ? 0 : page0) * a.page_b + h * a.head_b + (j0 & mask) * a.tok_b,
                      at1 = (bad1 ? 0 : page1) * a.page_b + h * a.head_b + ((j0 + 16) & mask) * a.tok_b;
#pragma unroll
        for (int c = tid; c < kManyTile * D / 4; c += kManyWarps * 32) {
          const int row = c / (D / 4), d = c % (D / 4);
          const bool in = !(row < 16 ? bad0 : bad1) && j0 + row < r.len;
          const int64_t src = in ? (row < 16 ? at0 : at1) + (row & 15) * a.tok_b + d * 16 : 0;
          sc::cp16(base + s * C::STAGE + (row * C::KP + d * 4) * 4, a.K + src, in);
          sc::cp16(base + s * C::STAGE + (kManyTile * C::KP + row * D + d * 4) * 4, a.V + src, in);
        }
      }
      sc::cp_commit();
      look_up(t + 1);
    };
    float acc[RW][E], m[RW], l[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) acc[k][c] = 0.f;
    }
    look_up(0);
    fetch(0);
    for (int t = 0; t < tiles; ++t) {
      fetch(t + 1);
      asm volatile("cp.async.wait_group 1;\n" ::: "memory");
      __syncthreads();
      const int j0 = key0 + t * kManyTile, s = t & 1, j = j0 + lane;
      if (j0 < to && j0 + kManyTile > from) {
        const float* kr = reinterpret_cast<const float*>(smem + s * C::STAGE) + lane * C::KP;
        const float* vr = reinterpret_cast<const float*>(smem + s * C::STAGE) + kManyTile * C::KP + lane * E;
        const bool held = !(empty >> (2 * s + (lane >> 4)) & 1u);
        float z[RW];
#pragma unroll
        for (int k = 0; k < RW; ++k) z[k] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          const float4 kv = *reinterpret_cast<const float4*>(kr + d);
#pragma unroll
          for (int k = 0; k < RW; ++k) {
            const float4 qv = *reinterpret_cast<const float4*>(q + k * D + d);
            z[k] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, z[k]))));
          }
        }
        bool grow = false;
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const int4 v = rows[k];
          z[k] = !held || j < v.x || j >= v.y ? -INFINITY : score2(a, z[k], __int_as_float(v.w), v.z - j);
          grow |= z[k] > m[k] + 8.f;
        }
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int k = 0; k < RW; ++k) {
            float top = z[k];
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            const float nm = fmaxf(m[k], top), keep = m[k] == -INFINITY ? 0.f : exp2f(m[k] - nm);
            m[k] = nm;
            l[k] *= keep;
#pragma unroll
            for (int c = 0; c < E; ++c) acc[k][c] *= keep;
          }
        }
        float p[RW];
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          p[k] = exp2f(z[k] - (m[k] == -INFINITY ? 0.f : m[k]));
          l[k] += p[k];
        }
        *reinterpret_cast<float4*>(pw + lane * RW) = make_float4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<float4*>(pw + lane * RW + 4) = make_float4(p[4], p[5], p[6], p[7]);
        __syncwarp();
#pragma unroll 4
        for (int u = 0; u < kManyTile; ++u) {
          const Vec v = *reinterpret_cast<const Vec*>(vr + u * D);
          const float* ve = reinterpret_cast<const float*>(&v);
          const float4 w0 = *reinterpret_cast<const float4*>(pw + u * RW), w1 = *reinterpret_cast<const float4*>(pw + u * RW + 4);
          const float w[RW] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < RW; ++k)
#pragma unroll
            for (int c = 0; c < E; ++c) acc[k][c] = fmaf(w[k], ve[c], acc[k][c]);
        }
      }
      __syncthreads();                 // the stage is read
    }
    ManyPut<D> put{r.row0 + i0, h, nullptr};
    if (x != u0 || end != u1) put.slot = f.w.part + (2 * (int64_t)part + (x == start ? 0 : 1)) * (int64_t)kManyRows * (2 + D);
    uint32_t again = 0;                // rows to look at again
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      float sum = l[k];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      bool fine = true;
#pragma unroll
      for (int c = 0; c < E; ++c) fine = fine && isfinite(acc[k][c]);
      fine = fine || !isfinite(sum) || sum == 0.f;
      again |= __all_sync(kFull, fine) ? 0u : 1u << k;
      if (warp * RW + k < cells) put(a, warp * RW + k, m[k], sum, acc[k]);
      l[k] = sum;
    }
    if (again) {                       // (the queries and weights in shared memory are this warp's own)
#pragma unroll
      for (int k = 0; k < RW; ++k) {
#pragma unroll
        for (int c = 0; c < E; ++c) q[k * D + lane * E + c] = acc[k][c];
        if (lane == 0) {
          pw[k] = m[k];
          pw[RW + k] = l[k];
        }
      }
      __syncwarp();
      many_again<D>(a, en.b, r, i0, h, cells, key0, key0 + tiles * kManyTile, low, top, again, pw, q, put);
    }
    __syncthreads();
    x = end;
  }
}

template <int D, int RH>
static cudaError_t launch_f32_t(const F32& f, int units, cudaStream_t st) {
  using C = F32Cfg<D, RH>;
  auto kern = f32_kernel<D, RH>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(f.cluster ? units * f.cluster : f.w.parts));
  cfg.blockDim = dim3(kF32Warps * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (f.cluster) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = f.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  } else {                             // the list kernel lies before it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> allowed{0};
  return launch_large(kern, cfg, f, f.a.device, allowed, C::SMEM);
}

template <int D>
static cudaError_t launch_f32(const F32& f, int rows, int units, cudaStream_t st) {
  if (rows == 4) return launch_f32_t<D, 2>(f, units, st);
  if (rows == 8) return launch_f32_t<D, 4>(f, units, st);
  return launch_f32_t<D, 8>(f, units, st);
}

template <int D>
static cudaError_t launch_many(const F32& f, cudaStream_t st) {
  using C = ManyCfg<D>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)f.w.parts);
  cfg.blockDim = dim3(kManyWarps * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> allowed{0};
  return launch_large(f32_many_kernel<D>, cfg, f, f.a.device, allowed, C::SMEM);
}

cudaError_t attend_f32(const Attend& a, const mp_paged_cache& c, const Work& w, int rows, int tile, int cluster,
                       cudaStream_t st) {
  F32 f{a, w, tile, cluster};
  const int D = c.cfg.head_dim, units = cluster ? a.batch * a.H * ((a.max_new + tile - 1) / tile) : 0;
  cudaError_t e = cluster ? cudaSuccess : launch_work(a, w, tile, kFewBlock, st);
  if (e != cudaSuccess) return e;
  if (rows == kF32ManyRows) e = D == 128 ? launch_many<128>(f, st) : launch_many<64>(f, st);
  else e = D == 128 ? launch_f32<128>(f, rows, units, st) : launch_f32<64>(f, rows, units, st);
  if (e != cudaSuccess || cluster) return e;
  return launch_join(a, w, MP_F32, D, tile, rows, false, st);
}

}  // namespace paged
}  // namespace mp
