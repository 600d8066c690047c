// Attention over a paged cache for requests with few rows (single tokens and
// drafts of a few): 16-bit types, at most 32 (token, head) rows a KV head.
//
// Bound by reading each key and value once: about 2 rows operations a byte, far
// below what the tensor cores need, so everything is built around bytes in
// flight.  A block has 4 warps; a warp takes every fourth 16-key tile of its
// block's share and owns a ring of shared-memory stages that its own TMA loads
// fill (one box of 16 tokens by head_dim of keys, one of values; no two warps
// wait for each other until the share ends).  Two blocks lie on an SM, 12
// stages of 8 KB (head dim 128) each: 192 KB in flight, and one block's ends of
// shares fall into the other's stream.  Measured: 16 requests of 16K to 32K tokens
// (32 query heads on 8 of 128, bf16, pages of 16) 277 to 283 us, 6.0 to 6.2 TB/s, 92
// to 94% of a copy's rate; drafts of 8 tokens on them (32 rows a KV head) 307 us; one
// request of 64K, fp16, 62 us, 4.3 TB/s: 41 us of bytes, the rest the blocks' first
// loads (lengths, table, keys, one after the other) and the joining of 37 parts.
//
// Rows are the M of mma.sync m16n8k16 (S = Q K^T with 16 keys as N, O += P V
// with 16 keys as K), so the P that comes out of S is already the operand that
// P V takes.  With at most 8 rows the other 8 are the same rows again, whose
// lanes pass the remainder p - round(p) into P V: the weights keep twice the
// type's bits at no cost (fp16's down to its smallest step).  Above that, weights
// are rounded once to the values' type, off by at most half a step each, as the
// matrix instruction has no operand of more bits.  The running maximum is lazy: it
// moves when a score exceeds it by more than 8 (base 2), so weights stay below 256
// and the numerator is rarely rescaled.  Statistics and numerators are fp32.
#include <cstring>
#include <type_traits>

#include "paged_work.cuh"
#include "stream_common.cuh"

namespace mp {
namespace paged {

constexpr int kFewWarps = 4;
constexpr int kTile = 16;                          // keys a tile
static_assert(kFewBlock == kFewWarps * kTile, "a block of the share-out is a tile a warp");
constexpr int kRing = 24 * 1024;                   // bytes of a warp's ring
constexpr float kLazyLimit = 8.f;

struct Few {
  CUtensorMap tmK, tmV;
  Attend a;
  Work w;
  int cluster;                                     // > 0: that many blocks share a unit and join in shared memory
};
// Up to this many requests every block makes the list itself, in shared memory
// (a list kernel before it costs 5 us and a chain of dependent loads).
constexpr int kOwnList = 512;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    sc::mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return sc::pack_bf16(lo, hi);
  }
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else return make_float2(sc::bf16_lo(v), sc::bf16_hi(v));
}
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* tm, int row, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4, "
      "%5}], [%6];\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
// Waits for a phase, two seconds at most.
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity) {
  return sc::mbar_try(bar, parity) || sc::mbar_wait(bar, parity, sc::gtimer() + 2000000000LL);
}

// MT tiles of 16 rows; DUP: at most 8 rows, held twice.
template <typename T, int D, int MT, bool DUP>
struct FewCfg {
  static constexpr int STAGE = 2 * kTile * D * 2;                     // keys and values of a tile
  static constexpr int NS = kRing / STAGE;
  static constexpr int ROWS = DUP ? 8 : 16 * MT;
  static constexpr int PITCH = D + 8;                                 // floats between the rows of a warp's numerators
  static constexpr int OFF_BAR = kFewWarps * kRing;                   // [warps][NS] barriers
  static constexpr int OFF_ML = OFF_BAR + kFewWarps * NS * 8;         // [warps][2][ROWS] maxima, sums
  static constexpr int OFF_UNIT = OFF_ML + kFewWarps * 2 * ROWS * 4;  // [2][ROWS] maxima, sums of the block
  static constexpr int OFF_BAD = OFF_UNIT + 2 * ROWS * 4;             // rows to be looked at again
  static constexpr int OFF_LIST = (OFF_BAD + (int)sizeof(Again<ROWS>) + 7) / 8 * 8;   // [kOwnList + 1] blocks before each request
  static constexpr int OFF_KEY = OFF_LIST + (kOwnList + 1) * 8;       // [kOwnList] first keys
  static constexpr int OFF_SUM = OFF_KEY + kOwnList * 4;              // [warps] sums
  static constexpr int OFF_ROW = (OFF_SUM + kFewWarps * 8 + 15) / 16 * 16;   // [warps][ROWS] first key, end, position, slope
  static constexpr int USED = OFF_ROW + kFewWarps * ROWS * 16;
  static constexpr int SMEM = USED + 1024;                            // room to align
  static_assert(ROWS * PITCH * 4 <= kRing, "a warp's numerators fit its ring");
  static_assert(2 * SMEM <= 227 * 1024, "two blocks an SM");
};

template <typename T, int D, int MT, bool DUP>
__global__ void __launch_bounds__(kFewWarps * 32, 2) few_kernel(const __grid_constant__ Few f) {
  using C = FewCfg<T, D, MT, DUP>;
  constexpr int KS = D / 16, NT = D / 8, NS = C::NS, ROWS = C::ROWS;
  const Attend& a = f.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (sc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = sc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = sb + warp * kRing, bars = sb + C::OFF_BAR + warp * NS * 8;
  float* num = reinterpret_cast<float*>(smem + warp * kRing);         // this warp's numerators, at a share's end
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* unit_m = reinterpret_cast<float*>(smem + C::OFF_UNIT);
  Again<ROWS>* again = reinterpret_cast<Again<ROWS>*>(smem + C::OFF_BAD);
  int4* mine = reinterpret_cast<int4*>(smem + C::OFF_ROW) + warp * ROWS;

  if (lane == 0)
    for (int s = 0; s < NS; ++s) sc::mbar_init(bars + 8 * s, 1);
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // this block's share of the line of blocks
  int64_t W = 0, x = 0, x1 = 0;
  int E = 0, N = 1, e = 0;
  const int part = f.cluster ? (int)(blockIdx.x % f.cluster) : (int)blockIdx.x;
  const bool own = a.batch <= kOwnList;
  const int64_t* before = own ? reinterpret_cast<const int64_t*>(smem + C::OFF_LIST) : f.w.before;
  const int32_t* own_k0 = reinterpret_cast<const int32_t*>(smem + C::OFF_KEY);
  if (!f.cluster) {
    if (own) {
      int64_t* sum = reinterpret_cast<int64_t*>(smem + C::OFF_SUM);
      int64_t done = 0;
      for (int b0 = 0; b0 < a.batch; b0 += kFewWarps * 32) {
        const int b = b0 + tid;
        Entry en{b, 0, 0, 0};
        if (b < a.batch) {
          const Request r = request_of(a, b);
          if (r.n > 0) span_of(a, r, b, 0, r.n, kFewBlock, en);
        }
        int64_t s = en.n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(kFull, s, o);
          if (lane >= o) s += y;
        }
        if (lane == 31) sum[warp] = s;
        __syncthreads();
        int64_t at = done;
        for (int w = 0; w < kFewWarps; ++w) {
          if (w < warp) at += sum[w];
          done += sum[w];
        }
        if (b < a.batch) {
          const_cast<int64_t*>(before)[b] = at + s - en.n;
          const_cast<int32_t*>(own_k0)[b] = en.k0;
          if (part == 0) {             // for the joining kernel
            f.w.before[b] = at + s - en.n;
            f.w.entry[b] = en;
          }
        }
        __syncthreads();
      }
      if (tid == 0) {
        const_cast<int64_t*>(before)[a.batch] = done;
        if (part == 0) {
          f.w.before[a.batch] = done;
          f.w.count[0] = a.batch;
          *reinterpret_cast<int64_t*>(f.w.count + 2) = done;
        }
      }
      __syncthreads();
    }
    E = own ? a.batch : f.w.count[0];
    W = (own ? before[E] : *reinterpret_cast<const int64_t*>(f.w.count + 2)) * a.H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (W == 0) return;
    N = parts_used(f.w, W);
    if (part >= N) return;
    x = own ? edge(before, E, a.H, W, N, part) : f.w.edge[part];
    x1 = own ? edge(before, E, a.H, W, N, part + 1) : f.w.edge[part + 1];
    if (x >= x1) return;
    e = own ? entry_of(before, E, a.H, x) : f.w.edge_entry[part];
  } else {
    x1 = 1;
  }
  const int64_t start = x;
  uint32_t fills = 0;                  // tiles that this warp has asked for: stage and phase
  bool ok = true;

  while (x < x1) {
    // --- the unit: a request's rows and a KV head; this block's keys of it
    int b, h, blk0, blk1, k0;
    int64_t u0 = 0, u1 = 0;
    if (f.cluster) {
      const int u = blockIdx.x / f.cluster;
      b = u / a.H;
      h = u - b * a.H;
    } else {
      while (before[e + 1] * a.H <= x) ++e;      // requests without rows have no blocks
      const int64_t n = before[e + 1] - before[e], first = before[e] * a.H;
      b = own ? e : f.w.entry[e].b;
      h = (int)((x - first) / n);
      u0 = first + h * n;
      u1 = u0 + n;
      blk0 = (int)(x - u0);
      blk1 = (int)(min(x1, u1) - u0);
      k0 = own ? own_k0[e] : f.w.entry[e].k0;
    }
    const Request r = request_of(a, b);
    const int prefix = prefix_of(a, b), cells = r.n * a.G;
    // this lane's rows (g and g + 8 of each tile) and what the rows see together; a row's own keys, position and slope
    // are kept in shared memory (in registers they cost those that the two tiles of 17 to 32 rows lack)
    int lo_min = INT32_MAX, lo_max = 0, hi_min = INT32_MAX, hi_max = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = DUP ? g : mt * 16 + s * 8 + g;
        if (row >= cells) {
          if (t4 == 0) mine[row] = make_int4(0, 0, 0, 0);
          continue;
        }
        const Interval v = interval_of(a, r, prefix, row / a.G);
        if (t4 == 0)
          mine[row] = make_int4(v.lo, v.hi, v.pos,
                                a.slopes ? __float_as_int(__ldg(a.slopes + h * a.G + row % a.G) * kLog2e) : 0);
        lo_max = max(lo_max, v.lo);
        hi_min = min(hi_min, v.hi);
        if (v.hi > v.lo) {
          lo_min = min(lo_min, v.lo);
          hi_max = max(hi_max, v.hi);
        }
      }
    __syncwarp();
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      lo_min = min(lo_min, __shfl_xor_sync(kFull, lo_min, o));
      hi_min = min(hi_min, __shfl_xor_sync(kFull, hi_min, o));
      lo_max = max(lo_max, __shfl_xor_sync(kFull, lo_max, o));
      hi_max = max(hi_max, __shfl_xor_sync(kFull, hi_max, o));
    }
    if (f.cluster) {
      k0 = hi_max > lo_min ? lo_min / kFewBlock * kFewBlock : 0;
      const int n = hi_max > lo_min ? (hi_max - k0 + kFewBlock - 1) / kFewBlock : 0;
      blk0 = (int)((int64_t)n * part / f.cluster);
      blk1 = (int)((int64_t)n * (part + 1) / f.cluster);
    }
    const int key0 = k0 + blk0 * kFewBlock, key1 = min(k0 + blk1 * kFewBlock, hi_max);
    if (tid == 0) {
      again->low = lo_min;
      again->high = hi_max;
    }

    uint32_t qf[MT][KS][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = DUP ? g : mt * 16 + s * 8 + g;
        const char* q = a.Q + (int64_t)(r.row0 + row / a.G) * a.q_row_b + (int64_t)(h * a.G + row % a.G) * a.q_head_b + 4 * t4;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[mt][ks][s] = row < cells ? *reinterpret_cast<const uint32_t*>(q + ks * 32) : 0u;
          qf[mt][ks][s + 2] = row < cells ? *reinterpret_cast<const uint32_t*>(q + ks * 32 + 16) : 0u;
        }
      }

    // --- this warp's tiles: keys key0 + 16 (warp + 4 i)
    const int first = key0 + warp * kTile;
    const int tiles = key1 > first ? (key1 - first + kFewBlock - 1) / kFewBlock : 0;
    int pages = -1;                    // lane l: the page of tile 32 (i / 32) + l
    uint32_t void_stages = 0;          // stages whose tile has no page
    auto fetch = [&](int i) {
      if ((i & 31) == 0) {
        const int j = first + (i + lane) * kFewBlock;    // a tile that no row sees may have no page any more
        pages = i + lane < tiles && j + kTile > lo_min ? page_of(a, b, j) : -1;
      }
      const int page = __shfl_sync(kFull, pages, i & 31), j = first + i * kFewBlock;
      const uint32_t s = fills % NS;
      ++fills;
      if (page < 0 || !ok) {
        void_stages |= 1u << s;
        if (lane == 0) sc::mbar_arrive(bars + 8 * s);
      } else {
        void_stages &= ~(1u << s);
        if (lane == 0) {
          const int row = j & ((1 << a.page_shift) - 1);
          sc::mbar_arrive_tx(bars + 8 * s, C::STAGE);
          tma_5d(ring + s * C::STAGE, &f.tmK, row, h, page, bars + 8 * s);
          tma_5d(ring + s * C::STAGE + C::STAGE / 2, &f.tmV, row, h, page, bars + 8 * s);
        }
      }
    };
    float acc[MT][NT][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
    }
    const uint32_t fill0 = fills;
    for (int i = 0; i < min(tiles, NS); ++i) fetch(i);

    for (int i = 0; i < tiles; ++i) {
      const uint32_t at = fill0 + i, s = at % NS;
      if (ok && !wait_limited(bars + 8 * s, (at / NS) & 1u)) {
        ok = false;
        set_error(a.err, E_TIMEOUT);
      }
      ok = __all_sync(kFull, ok);
      const int j0 = first + i * kFewBlock;
      if (ok && !(void_stages >> s & 1u)) {
        const uint32_t kb = ring + s * C::STAGE, vb = kb + C::STAGE / 2;
        if (j0 + kTile > r.len) {      // what lies behind the last token is not the request's: no value of it may count
          unsigned char* v = smem + (vb - sb);
          for (int c = lane; c < kTile * D / 8; c += 32) {
            const int row = (c >> 3) & 15;          // [panel][16 rows][8 chunks]: the swizzle moves chunks inside rows
            if (j0 + row >= r.len) reinterpret_cast<uint4*>(v)[c] = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // scores: [2 halves of 8 keys]
        float z[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nh = 0; nh < 2; ++nh) z[mt][nh][0] = z[mt][nh][1] = z[mt][nh][2] = z[mt][nh][3] = 0.f;
        {
          const int key = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t k0r, k1r, k2r, k3r;
            sc::ldsm4(kb + sc::tswz<16>(key, 2 * ks + odd), k0r, k1r, k2r, k3r);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<T>(z[mt][0], qf[mt][ks], k0r, k1r);
              mma<T>(z[mt][1], qf[mt][ks], k2r, k3r);
            }
          }
        }
        const bool whole = j0 >= lo_max && j0 + kTile <= hi_min;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float& v = z[mt][c >> 2][c & 3];
            v = a.cap > 0.f ? cap_of(a, v) : v * a.to_z;
          }
        if (!whole || a.slopes) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
              const int4 x = mine[DUP ? g : mt * 16 + hrow * 8 + g];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float& v = z[mt][k >> 1][2 * hrow + (k & 1)];
                const int j = j0 + (k >> 1) * 8 + 2 * t4 + (k & 1);
                if (a.slopes) v -= __int_as_float(x.w) * (float)abs(x.z - j);
                if (j < x.x || j >= x.y) v = -INFINITY;
              }
            }
        }
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 8; ++c) grow |= z[mt][c >> 2][c & 3] > m[mt][(c & 3) >> 1] + kLazyLimit;
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
              float top = fmaxf(fmaxf(z[mt][0][2 * hrow], z[mt][0][2 * hrow + 1]),
                                fmaxf(z[mt][1][2 * hrow], z[mt][1][2 * hrow + 1]));
              top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
              top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
              const float nm = fmaxf(m[mt][hrow], top);
              const float keep = m[mt][hrow] == -INFINITY ? 0.f : sc::ex2(m[mt][hrow] - nm);
              m[mt][hrow] = nm;
              l[mt][hrow] *= keep;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                acc[mt][nt][2 * hrow] *= keep;
                acc[mt][nt][2 * hrow + 1] *= keep;
              }
            }
        }
        uint32_t pf[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int hrow = 0; hrow < 2; ++hrow) {
            if (DUP && hrow == 1) continue;
            const float base = m[mt][hrow] == -INFINITY ? 0.f : m[mt][hrow] - kLift<T>;
#pragma unroll
            for (int nh = 0; nh < 2; ++nh) {
              const float p0 = sc::ex2(z[mt][nh][2 * hrow] - base), p1 = sc::ex2(z[mt][nh][2 * hrow + 1] - base);
              l[mt][hrow] += p0 + p1;
              const uint32_t w = pack2<T>(p0, p1);
              pf[mt][2 * nh + hrow] = w;
              if (DUP) {
                const float2 back = unpack2<T>(w);
                pf[mt][2 * nh + 1] = pack2<T>(p0 - back.x, p1 - back.y);
              }
            }
          }
        }
        {
          const int key = (lane & 7) + (((lane >> 3) & 1) << 3), odd = lane >> 4;
#pragma unroll
          for (int n2 = 0; n2 < NT / 2; ++n2) {
            uint32_t v0, v1, v2, v3;
            sc::ldsm4t(vb + sc::tswz<16>(key, 2 * n2 + odd), v0, v1, v2, v3);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<T>(acc[mt][2 * n2], pf[mt], v0, v1);
              mma<T>(acc[mt][2 * n2 + 1], pf[mt], v2, v3);
            }
          }
        }
        if (j0 + kTile > r.len) sc::fence_proxy_async();   // the zeros are written before a load takes the stage again
      }
      __syncwarp();                    // all lanes have read the stage
      if (i + NS < tiles) fetch(i + NS);
    }

    if (!ok)                           // gave up: the loads still under way, within the limit, before their stages are reused
      for (uint32_t at = fills - min((uint32_t)NS, fills - fill0); at != fills; ++at)
        if (!wait_limited(bars + 8 * (at % NS), (at / NS) & 1u)) break;

    // --- the warps' states meet in shared memory
    __syncwarp();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hrow = 0; hrow < (DUP ? 1 : 2); ++hrow) {
        float s = l[mt][hrow];
        s += __shfl_xor_sync(kFull, s, 1);
        s += __shfl_xor_sync(kFull, s, 2);
        const int row = mt * 16 + hrow * 8 + g;
        if (t4 == 0) {
          ml[(warp * 2) * ROWS + row] = s != s ? s : m[mt][hrow] - kLift<T>;   // a NaN must not pass for "nothing seen"
          ml[(warp * 2 + 1) * ROWS + row] = s;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float2 v = make_float2(acc[mt][nt][2 * hrow], acc[mt][nt][2 * hrow + 1]);
          if (DUP) { v.x += acc[mt][nt][2]; v.y += acc[mt][nt][3]; }
          *reinterpret_cast<float2*>(num + row * C::PITCH + nt * 8 + 2 * t4) = v;
        }
      }
    Settle st;
    st.b = b;
    st.h = h;
    st.r = r;
    st.i0 = 0;
    st.cells = min(cells, ROWS);
    st.key0 = key0;
    st.key1 = key1;
    st.cluster = f.cluster;
    st.part = part;
    st.whole = !f.cluster && x == u0 && min(x1, u1) == u1;
    st.slot = f.cluster ? nullptr : f.w.part + (2 * (int64_t)part + (x == start ? 0 : 1)) * (int64_t)ROWS * (2 + D);
    settle<T, D, ROWS, C::PITCH, kFewWarps>(a, st, ml, reinterpret_cast<float*>(smem), kRing / 4, unit_m, again);
    if (f.cluster) return;
    sc::fence_proxy_async();           // the numerators were written where the next loads go
    __syncthreads();
    x = min(x1, u1);
  }
}

template <typename T, int D, int MT, bool DUP>
static cudaError_t launch_few_t(Few& f, int units, cudaStream_t st) {
  using C = FewCfg<T, D, MT, DUP>;
  auto kern = few_kernel<T, D, MT, DUP>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(f.cluster ? units * f.cluster : f.w.parts));
  cfg.blockDim = dim3(kFewWarps * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (f.cluster) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = f.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  } else if (f.a.batch > kOwnList) {   // the list kernel lies before it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = f.cluster || f.a.batch > kOwnList ? 1 : 0;
  static std::atomic<uint64_t> allowed{0};
  return launch_large(kern, cfg, f, f.a.device, allowed, C::SMEM);
}

template <typename T, int D>
static cudaError_t launch_few_d(Few& f, int cells, int units, cudaStream_t st) {
  if (cells <= 8) return launch_few_t<T, D, 1, true>(f, units, st);
  if (cells <= 16) return launch_few_t<T, D, 1, false>(f, units, st);
  return launch_few_t<T, D, 2, false>(f, units, st);
}

static cudaError_t launch_few(Few& f, int dtype, int D, int cells, int units, cudaStream_t st) {
  if (dtype == MP_F16)
    return D == 128 ? launch_few_d<__half, 128>(f, cells, units, st) : launch_few_d<__half, 64>(f, cells, units, st);
  return D == 128 ? launch_few_d<__nv_bfloat16, 128>(f, cells, units, st)
                  : launch_few_d<__nv_bfloat16, 64>(f, cells, units, st);
}

// The whole call: shares over all SMs, or a cluster a unit.
cudaError_t attend_few(const Attend& a, const mp_paged_cache& c, Work w, int cells, int cluster, cudaStream_t st) {
  Few f{};
  static_assert(sizeof(CUtensorMap) == 128, "tensor map size");
  memcpy(&f.tmK, c.maps + 16 * MAP_K16, sizeof(CUtensorMap));
  memcpy(&f.tmV, c.maps + 16 * MAP_V16, sizeof(CUtensorMap));
  f.a = a;
  f.cluster = cluster;
  const int D = c.cfg.head_dim;
  if (cluster) return launch_few(f, c.cfg.dtype, D, cells, a.batch * a.H, st);
  f.w = w;
  cudaError_t e = a.batch > kOwnList ? launch_work(a, w, a.max_new, kFewBlock, st) : cudaSuccess;
  if (e == cudaSuccess) e = launch_few(f, c.cfg.dtype, D, cells, a.batch * a.H, st);
  if (e == cudaSuccess) e = launch_join(a, w, c.cfg.dtype, D, a.max_new, few_rows(cells), a.batch <= kOwnList, st);
  return e;
}

}  // namespace paged
}  // namespace mp
