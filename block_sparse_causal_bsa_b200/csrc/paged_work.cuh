// Work of the paged attention kernels: items, the split of their key tiles over CTAs, and the
// rows of an item.
//
// An item is a set of query rows that read the same keys:
//   whole cache  (slot, KV head, row tile): rows r of the G * ql (head of the group, token) pairs
//                of the slot, RT at a time, r = g * ql + t
//   page lists   (slot, KV head, token): the G heads of the group
// Its keys come in tiles of 64. All items' tiles are laid end to end (those of row tiles of 256 with more
// than 128 rows count twice: they take about twice as long) and every CTA takes an equal, contiguous
// share of them, so ragged lengths balance without the host knowing them. A share may
// begin or end inside an item: such segments leave a partial result (running maximum, sum,
// unnormalised output) in one of the CTA's two slots of the workspace, 0 for a segment that starts
// inside its item, 1 for one that starts with it. The CTA that arrives last at an item's counter joins its
// parts, in their order along the keys whichever CTA that is: the split depends on lengths alone, and
// results repeat bit for bit. (A second kernel for the joins took 28 us behind 354 us of attention for
// wide trees and 7 to 12 us behind small calls, most of it spent on finding the split again.)
// A small kernel zeroes the counters first. The attention kernel starts beside it (programmatic
// serialization) and waits for it only before its first arrival.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace bsa {

constexpr int kTileKeys = 64;

struct PagedArgs {
  CacheGeom g;
  int Hq, G;                        // query heads, heads per KV head
  int words;                        // mask words per token
  const uint16_t* q;
  const uint16_t* v;                // the pool again: repair of non-finite drafted values
  const unsigned long long* mask;   // null: chain
  const int32_t* kv_idx;            // page lists (null: the whole cache)
  const int32_t* kv_cnt;
  int W;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_o;                    // [2 * n_cta][RT][d]
  float* part_ml;                   // [2 * n_cta][RT][2]
  int32_t* part_flag;               // [2 * n_cta], two each on tcgen05 (a group's rows)
  int32_t* arrived;                 // [n_cta], two each on tcgen05: parts of the item that ends in the CTA's share
  int n_arrived;
  int32_t* dev_status;
  int n_cta;
};

__host__ __device__ inline int ceil_div_i(int a, int b) { return (a + b - 1) / b; }

// One item, and where a walk stands in it.
struct Item {
  int b, h;
  int base, ql;                     // the slot's tokens
  int row0, rows;                   // whole cache: first row and number of rows (<= RT)
  int t;                            // page lists: the token
  int n_tiles;                      // tiles of the item (page lists: of a full list)
  int weight;                       // what a tile counts in the whole order
  long long first;                  // the item's first place there
  __device__ int units() const { return n_tiles * weight; }
  // Tiles of the places [x, xe) of the item: a tile belongs to the share that holds its first place.
  __device__ void tiles_of(long long x, long long xe, int& ta, int& tb) const {
    ta = (int)(x - first);
    tb = (int)(xe - first);
    if (weight == 2) {
      ta = (ta + 1) / 2;
      tb = (tb + 1) / 2;
    }
  }
};

// How far a share may shrink: below this many tiles per CTA the arrival and the join cost more time
// than the shorter share saves (one user, eight lists of 64 tiles: 4 tiles 14.6 us, 2 tiles 16.7, 6 tiles 17.3;
// eight drafts over 1003 tokens on tcgen05: 2 tiles 18.8 us, 1 tile 20.9).
template <int RT>
constexpr int kMinTiles = RT == 256 ? 2 : 4;

template <bool LIST, int RT>
struct Walk {
  long long total;                  // weighted tiles of all items
  long long per;                    // ... per CTA (the last ones may have fewer, or none)
  // lane b (whole cache): slot b's tiles and tokens
  long long tiles;
  int base, ql;

  __device__ static int slot_items(const PagedArgs& a, int ql) {
    return a.g.Hkv * ceil_div_i(a.G * ql, RT);
  }
  __device__ static int tile_weight(const PagedArgs& a, int ql) { return RT == 256 && a.G * ql > 128 ? 2 : 1; }
  __device__ static long long slot_tiles(const PagedArgs& a, int base, int ql) {
    return ql ? (long long)slot_items(a, ql) * ceil_div_i(base + ql, kTileKeys) * tile_weight(a, ql) : 0;
  }
  __device__ static int list_tiles(const PagedArgs& a) {
    return (int)(((long long)a.W * a.g.page + kTileKeys - 1) / kTileKeys);
  }
  // (64-bit divisions are slow)
  __device__ static long long divide(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
  }
  // slot b0 + lane
  __device__ static void load(const PagedArgs& a, int b0, long long& tiles, int& base, int& ql) {
    const int b = b0 + threadIdx.x % 32;
    base = ql = 0;
    if (b < a.g.slots) query_span(a.g, b, base, ql);
    tiles = slot_tiles(a, base, ql);
  }

  // Whole warp.
  __device__ void init(const PagedArgs& a) {
    if (LIST) {
      total = (long long)a.g.slots * a.g.Hkv * a.g.T * list_tiles(a);
    } else {
      long long s = 0;
      for (int b0 = (a.g.slots - 1) / 32 * 32; b0 >= 0; b0 -= 32) {    // (the first slots stay loaded)
        load(a, b0, tiles, base, ql);
        s += tiles;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      total = s;
    }
    per = max(divide(total + a.n_cta - 1, a.n_cta), (long long)kMinTiles<RT>);
  }
  __device__ long long start(int c) const { return min(c * per, total); }
  // the CTA whose share holds tile x
  __device__ int owner(long long x) const { return (int)divide(x, per); }

  __device__ void set_list_item(const PagedArgs& a, long long item, Item& it) const {
    it.n_tiles = list_tiles(a);
    it.weight = 1;
    it.first = item * it.n_tiles;
    it.t = (int)item % a.g.T;                        // (slots * Hq * T is below 2^31)
    const int bh = (int)item / a.g.T;
    it.h = bh % a.g.Hkv;
    it.b = bh / a.g.Hkv;
    query_span(a.g, it.b, it.base, it.ql);
    it.row0 = 0;
    it.rows = a.G;
  }
  // it.b, it.base and it.ql are set
  __device__ void set_slot_item(const PagedArgs& a, long long slot_first, int item, Item& it) const {
    it.n_tiles = ceil_div_i(it.base + it.ql, kTileKeys);
    it.weight = tile_weight(a, it.ql);
    it.first = slot_first + (long long)item * it.units();
    const int M = a.G * it.ql, mts = ceil_div_i(M, RT);
    it.h = mts == 1 ? item : item / mts;
    it.row0 = (item - it.h * mts) * RT;
    it.rows = min(RT, M - it.row0);
    it.t = 0;
  }

  // The item of tile x (0 <= x < total). Whole warp.
  __device__ void locate(const PagedArgs& a, long long x, Item& it) const {
    if (LIST) {
      set_list_item(a, divide(x, list_tiles(a)), it);
      return;
    }
    const int lane = threadIdx.x % 32;
    long long before = 0;
    long long lt = tiles;                           // (locals: the members stay the first slots')
    int lb = base, lq = ql;
    for (int b0 = 0; b0 < a.g.slots; b0 += 32) {
      if (b0) load(a, b0, lt, lb, lq);
      long long p = lt;                             // inclusive prefix
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += y;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + p > x);
      if (m) {
        const int l = __ffs(m) - 1;
        const long long first = before + __shfl_sync(0xffffffffu, p - lt, l);
        it.b = b0 + l;
        it.base = __shfl_sync(0xffffffffu, lb, l);
        it.ql = __shfl_sync(0xffffffffu, lq, l);
        set_slot_item(a, first, (int)divide(x - first, ceil_div_i(it.base + it.ql, kTileKeys) * tile_weight(a, it.ql)), it);
        return;
      }
      before += __shfl_sync(0xffffffffu, p, 31);
    }
  }
  // The item after it (there is one: it ends before total).
  __device__ void next(const PagedArgs& a, Item& it) const {
    const long long x = it.first + it.units();
    if (LIST) {
      set_list_item(a, ((long long)it.b * a.g.Hkv + it.h) * a.g.T + it.t + 1, it);
      return;
    }
    const int mts = ceil_div_i(a.G * it.ql, RT);
    const int item = it.h * mts + it.row0 / RT + 1;
    if (item < a.g.Hkv * mts) {
      set_slot_item(a, it.first - (long long)(item - 1) * it.units(), item, it);
      return;
    }
    do {
      ++it.b;
      query_span(a.g, it.b, it.base, it.ql);
    } while (it.ql == 0);
    set_slot_item(a, x, 0, it);
  }
};

// Tiles of the item that hold keys: for a page list, those up to its count.
template <bool LIST>
__device__ __forceinline__ int item_live_tiles(const PagedArgs& a, const Item& it, int& cnt, bool& bad) {
  bad = false;
  cnt = 0;
  if (!LIST) return it.n_tiles;
  if (it.t >= it.ql) return 0;
  cnt = a.kv_cnt[((size_t)it.b * a.g.Hkv + it.h) * a.g.T + it.t];
  if (cnt < 0 || cnt > a.W) {
    bad = true;
    cnt = cnt < 0 ? 0 : a.W;
  }
  return (int)(((long long)cnt * a.g.page + kTileKeys - 1) / kTileKeys);
}

// Row r of an item: query head and token.
template <bool LIST>
__device__ __forceinline__ void row_of(const PagedArgs& a, const Item& it, int r, int& head, int& t) {
  if (LIST) {
    head = it.h * a.G + r;
    t = it.t;
  } else {
    const int x = it.row0 + r;
    head = it.h * a.G + x / it.ql;
    t = x % it.ql;
  }
}

// Does token t see drafted token j of its slot?
__device__ __forceinline__ bool sees_draft(const PagedArgs& a, int b, int t, int j) {
  if (!a.mask) return j <= t;
  return (a.mask[((size_t)b * a.g.T + t) * a.words + (j >> 6)] >> (j & 63)) & 1ull;
}

template <bool F16>
__device__ __forceinline__ float cvt_f32(uint16_t x) {
  if (F16) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(x));
    return f;
  }
  return bf16_to_f32(x);
}
template <bool F16>
__device__ __forceinline__ uint16_t cvt_16(float x) {
  if (F16) {
    uint16_t h;
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
  }
  return f32_to_bf16_rn(x);
}
// (lo, hi) rounded to two 16-bit floats in one register
template <bool F16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Clears the non-finite halves of a packed pair; true if there was one.
template <bool F16>
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w) {
  const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  const bool lo = (w & e) == e, hi = ((w >> 16) & e) == e;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

// The kernels take non-finite values of drafted tokens as zero (a weight of zero times NaN or infinity
// would reach rows that do not see them). Where a tile had some, the rows that do see them get them
// here, after their result is stored: channels [d0, d1) of output row `row` (token t), whose sum of such
// values is NaN or infinite, get it added.
template <bool F16>
__device__ __noinline__ void store_nonfinite(const PagedArgs& a, const Item& it, int t, size_t row, int d0, int d1) {
  for (int d = d0; d < d1; ++d) {
    float s = 0.f;
    for (int j = 0; j < it.ql; ++j) {
      if (!sees_draft(a, it.b, t, j)) continue;
      const int pos = it.base + j;
      const int pg = a.g.table[(size_t)it.b * a.g.max_pages + pos / a.g.page];
      if (pg < 0 || pg >= a.g.n_pages) continue;
      const float x = cvt_f32<F16>(a.v[(((size_t)pg * a.g.Hkv + it.h) * a.g.page + pos % a.g.page) * a.g.d + d]);
      if (!isfinite(x)) s += x;
    }
    uint16_t* o = a.out + row * a.g.d + d;
    if (!isfinite(s)) *o = cvt_16<F16>(cvt_f32<F16>(*o) + s);
  }
}

// Reads from L2 of what other SMs wrote in this kernel. (volatile: they stay behind the barrier or
// the atomic that says it is there.)
__device__ __forceinline__ float4 read_l2(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float2 read_l2(const float2* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int read_l2(const int32_t* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// What waits for the preparing kernel (counters and *dev_status are set when it returns).
__device__ __forceinline__ void wait_prepared() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The parts of a split item: CTAs c0 .. c1, and the slot of the part of CTA c0 + i.
template <bool LIST, int RT>
struct Parts {
  int c0, n, c1;
  __device__ Parts(const Walk<LIST, RT>& w, const Item& it) {
    c0 = w.owner(it.first);
    c1 = w.owner(it.first + it.units() - 1);
    n = c1 - c0 + 1;
  }
  __device__ size_t slot(int i) const { return 2 * (size_t)(c0 + i) + (i == 0 ? 1 : 0); }
};

// One thread, behind a barrier that the CTA's writes of its part precede: counts the part in; true
// for the last one, whose CTA joins them (behind another barrier).
__device__ __forceinline__ bool arrive_part(int32_t* counter, int n) {
  wait_prepared();
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old == n - 1;
}

// Zeroes the counters and sets *dev_status to what the lengths say.
cudaError_t launch_paged_prepare(const PagedArgs& a, cudaStream_t st);

// Launch attributes of a kernel that may start beside the one before it.
inline cudaLaunchConfig_t beside(cudaLaunchAttribute* at, unsigned grid, unsigned block, size_t smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

// Attention on warp-level MMAs (row tiles of 8 or 16).
cudaError_t launch_paged_attend_mma(const bsa_cache_shape& s, PagedArgs a, const void* k, const void* v,
                                    cudaStream_t st);

// The same on tcgen05 (row tiles of 256, whole cache only).
cudaError_t launch_paged_attend_tc(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                                   cudaStream_t st);

// Shares per SM of the kernel on warp-level MMAs: the CTAs that fit.
constexpr int kMmaSharesPerSm = 2;

// Query rows per KV head up to which a call runs on warp-level MMAs (of the call's T: lengths are on the device).
// Both kernels at 8 KV heads, bf16, graph replays in us, warp-level MMAs against tcgen05 (above 16 rows the former
// takes 16 at a time):
//                              4 rows      8 rows      16 rows     20 rows      32 rows      64 rows
//   d 128, 1 x 1000 tokens     14 : 18     17 : 18     21 : 19     22 : 19      23 : 18      24 : 21
//   d 128, 1 x 64000           58 : 68     63 : 69     81 : 69     91 : 69     101 : 68     183 : 74
//   d 128, 16 x 64000         613 : 616   616 : 688   640 : 677  1260 : 620   1242 : 692   2454 : 755
//   d 64, 1 x 64000            43 : 71     44 : 65     51 : 61     66 : 62      68 : 60     104 : 60
//   d 64, 16 x 64000          327 : 552   328 : 552   325 : 552   624 : 579    677 : 555   1329 : 552
constexpr int kMaxMmaRows = 16;

}  // namespace bsa
