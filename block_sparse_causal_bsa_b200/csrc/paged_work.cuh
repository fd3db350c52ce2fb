// Work of the paged attention kernels: items, the split of their key tiles over CTAs, and the
// rows of an item.
//
// An item is a set of query rows that read the same keys:
//   whole cache  (slot, KV head, row tile): rows r of the G * ql (head of the group, token) pairs
//                of the slot, RT at a time, r = g * ql + t
//   page lists   (slot, KV head, token): the G heads of the group
// Its keys come in tiles of 64. All items' tiles are laid end to end and every CTA takes an equal,
// contiguous share of them, so ragged lengths balance without the host knowing them. A share may
// begin or end inside an item: such segments leave a partial result (running maximum, sum,
// unnormalised output) in one of the CTA's two slots of the workspace, 0 for a segment that starts
// inside its item, 1 for one that starts with it, and a second kernel joins them. The split depends on
// lengths alone, so results repeat bit for bit.
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
  int32_t* part_flag;               // [2 * n_cta]
  int32_t* cta_status;              // [n_cta]
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
  long long first;                  // its first tile in the whole order
};

template <bool LIST, int RT>
struct Walk {
  long long total;                  // tiles of all items
  long long per;                    // tiles per CTA (the last ones may have fewer, or none)

  __device__ static int slot_items(const PagedArgs& a, int ql) {
    return a.g.Hkv * ceil_div_i(a.G * ql, RT);
  }
  // tiles of all items of slot b
  __device__ static long long slot_tiles(const PagedArgs& a, int b) {
    int base, ql;
    query_span(a.g, b, base, ql);
    return ql ? (long long)slot_items(a, ql) * ceil_div_i(base + ql, kTileKeys) : 0;
  }
  __device__ static int list_tiles(const PagedArgs& a) {
    return (int)(((long long)a.W * a.g.page + kTileKeys - 1) / kTileKeys);
  }

  // Whole warp.
  __device__ void init(const PagedArgs& a) {
    if (LIST) {
      total = (long long)a.g.slots * a.g.Hkv * a.g.T * list_tiles(a);
    } else {
      const int lane = threadIdx.x % 32;
      long long s = 0;
      for (int b = lane; b < a.g.slots; b += 32) s += slot_tiles(a, b);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      total = s;
    }
    const long long n = total + a.n_cta - 1;         // (64-bit divisions are slow)
    per = n >> 32 ? n / a.n_cta : (long long)((uint32_t)n / (uint32_t)a.n_cta);
  }
  __device__ long long start(int c) const { return min(c * per, total); }
  // the CTA whose share holds tile x
  __device__ int owner(long long x) const {
    return x >> 32 || per >> 32 ? (int)(x / per) : (int)((uint32_t)x / (uint32_t)per);
  }

  __device__ void set_list_item(const PagedArgs& a, long long item, Item& it) const {
    it.n_tiles = list_tiles(a);
    it.first = item * it.n_tiles;
    it.t = (int)item % a.g.T;                        // (slots * Hq * T is below 2^31)
    const int bh = (int)item / a.g.T;
    it.h = bh % a.g.Hkv;
    it.b = bh / a.g.Hkv;
    query_span(a.g, it.b, it.base, it.ql);
    it.row0 = 0;
    it.rows = a.G;
  }
  __device__ void set_slot_item(const PagedArgs& a, int b, long long slot_first, int item, Item& it) const {
    query_span(a.g, b, it.base, it.ql);
    it.b = b;
    it.n_tiles = ceil_div_i(it.base + it.ql, kTileKeys);
    it.first = slot_first + (long long)item * it.n_tiles;
    const int M = a.G * it.ql, mts = ceil_div_i(M, RT);
    it.h = item / mts;
    it.row0 = (item % mts) * RT;
    it.rows = min(RT, M - it.row0);
    it.t = 0;
  }

  // The item of tile x (0 <= x < total). Whole warp.
  __device__ void locate(const PagedArgs& a, long long x, Item& it) const {
    if (LIST) {
      const int n = list_tiles(a);
      set_list_item(a, x >> 32 ? x / n : (long long)((uint32_t)x / (uint32_t)n), it);
      return;
    }
    const int lane = threadIdx.x % 32;
    long long before = 0;
    for (int b0 = 0; b0 < a.g.slots; b0 += 32) {
      const int b = b0 + lane;
      const long long w = b < a.g.slots ? slot_tiles(a, b) : 0;
      long long p = w;                              // inclusive prefix
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += y;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + p > x);
      if (m) {
        const int l = __ffs(m) - 1;
        const long long first = before + __shfl_sync(0xffffffffu, p - w, l);
        int base, ql;
        query_span(a.g, b0 + l, base, ql);
        const long long off = x - first;
        const int nt = ceil_div_i(base + ql, kTileKeys);
        set_slot_item(a, b0 + l, first, off >> 32 ? (int)(off / nt) : (int)((uint32_t)off / (uint32_t)nt), it);
        return;
      }
      before += __shfl_sync(0xffffffffu, p, 31);
    }
  }
  // The item after it (there is one: it ends before total).
  __device__ void next(const PagedArgs& a, Item& it) const {
    const long long x = it.first + it.n_tiles;
    if (LIST) {
      set_list_item(a, ((long long)it.b * a.g.Hkv + it.h) * a.g.T + it.t + 1, it);
      return;
    }
    const int mts = ceil_div_i(a.G * it.ql, RT);
    const int item = it.h * mts + it.row0 / RT + 1;
    if (item < a.g.Hkv * mts) {
      set_slot_item(a, it.b, it.first - (long long)(item - 1) * it.n_tiles, item, it);
      return;
    }
    int b = it.b + 1;
    while (slot_tiles(a, b) == 0) ++b;
    set_slot_item(a, b, x, 0, it);
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

// The kernel launched behind this one (with programmatic serialization) may start its blocks as
// room appears; it waits for the end of this one itself before it reads results.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// The sum of the non-finite drafted values of channel d that token t sees: the kernels take such
// values as zero (a weight of zero times NaN or infinity would reach rows that do not see them)
// and the rows that do see them get them here.
template <bool F16>
__device__ __noinline__ float nonfinite_drafts(const PagedArgs& a, const Item& it, int t, int d) {
  float s = 0.f;
  for (int j = 0; j < it.ql; ++j) {
    if (!sees_draft(a, it.b, t, j)) continue;
    const int pos = it.base + j;
    const int pg = a.g.table[(size_t)it.b * a.g.max_pages + pos / a.g.page];
    if (pg < 0 || pg >= a.g.n_pages) continue;
    const float x = cvt_f32<F16>(
        a.v[(((size_t)pg * a.g.Hkv + it.h) * a.g.page + pos % a.g.page) * a.g.d + d]);
    if (!isfinite(x)) s += x;
  }
  return s;
}

// Joins the partial results of the items that are split over CTAs (a warp per row), and gathers
// the status words. The scale of fp16 weights cancels, but for the lse: shift is its exponent.
cudaError_t launch_paged_join(const PagedArgs& a, int rt, bool list, bool f16, cudaStream_t st);

// Attention on warp-level MMAs (row tiles of 8 or 16).
cudaError_t launch_paged_attend_mma(const bsa_cache_shape& s, PagedArgs a, const void* k, const void* v,
                                    cudaStream_t st);

// The same on tcgen05 (row tiles of 128, whole cache only; a.n_cta: two per SM).
cudaError_t launch_paged_attend_tc(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                                   cudaStream_t st);

// Query rows per KV head up to which a call runs on warp-level MMAs.
constexpr int kMaxMmaRows = 16;

}  // namespace bsa
