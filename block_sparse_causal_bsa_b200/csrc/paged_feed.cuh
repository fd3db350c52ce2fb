// The producer of the paged attention kernels: one warp that brings the tiles of one operand (K or
// V) of a CTA's share into a ring of shared-memory stages.
#pragma once

#include <limits.h>

#include "paged_work.cuh"
#include "tc_common.cuh"

namespace bsa {

template <int D>
struct Feed {
  const CUtensorMap* map;
  uint8_t* stage0;                  // 64 rows x 128 bytes per 64-column half, 128-byte swizzled
  uint32_t stage_bytes;             // from stage to stage
  uint64_t* full;                   // [stages]: an arrival and the bytes per operand
  uint64_t* empty;
  unsigned long long* vmask;        // [ring], by tile: rows that are keys (null: the other operand's warp says)
};

// A lane holds one box (a page, or half a page of 128) of a batch of up to 32 tiles, and lanes issue
// their boxes in parallel: a TMA load costs the issuing warp some 80 cycles, so 16-row pages made
// a single producer of both operands the slowest part of the kernels (1340 cycles a tile at d = 64).
// The table entries of the next batch and the list entries of the one after are read while a batch
// is issued. Pages without a visible row are not read. Returns the tiles issued; the whole warp.
template <bool LIST, int RT, int D, int STAGES, int RING>
__device__ __noinline__ int feed_share(const PagedArgs& a, Walk<LIST, RT> w, long long x0, long long x1,
                                       const Feed<D> f, volatile int* abort_flag, int32_t* status) {
  constexpr uint32_t kHalf = kTileKeys * 128;
  const int lane = threadIdx.x % 32;
  // (copies of what is read behind the ordered statements below)
  const int page = a.g.page, n_pages = a.g.n_pages, Hkv = a.g.Hkv, W = a.W;
  const int rpb = page < kTileKeys ? page : kTileKeys, npt = kTileKeys / rpb, per_load = 32 / npt;
  const int my_tile = lane / npt, my_row = (lane % npt) * rpb;     // of the batch; of the tile
  if (lane == 0) tc::prefetch_tmap(f.map);
  if (x0 >= x1) return 0;
  Item it;
  w.locate(a, x0, it);
  int n = 0, s = 0;
  uint32_t parity = 1;
  bool bad = false;
  for (long long x = x0; x < x1;) {
    const long long xe = min(x1, it.first + it.units());
    int cnt;
    bool bad_count;
    const int live = item_live_tiles<LIST>(a, it, cnt, bad_count);
    bad |= bad_count;
    int ta, tb;
    it.tiles_of(x, xe, ta, tb);
    tb = min(tb, live);
    const int h = it.h;
    const int32_t* table = a.g.table + (size_t)it.b * a.g.max_pages;
    const int32_t* list = LIST ? a.kv_idx + (((size_t)it.b * Hkv + h) * a.g.T + it.t) * W : nullptr;
    // positions below it are keys
    const int limit = LIST ? (it.t < it.ql ? it.base + it.t + 1 : 0) : it.base + it.ql;
    // this lane's box of the batch from t0 on: the page's number within the sequence (-1: no such page,
    // INT_MIN: no box), and its page of the pool
    auto entry = [&](int t0) -> int {
      const int tile = t0 + my_tile;
      if (!LIST && tile >= tb) return INT_MIN;
      const int e = (tile * kTileKeys + my_row) / page;
      if (!LIST) return e * page < limit ? e : INT_MIN;
      if (e >= W) return INT_MIN;
      const int j = __ldg(list + e);             // (within the row of W entries; not behind the count's read)
      return tile < tb && e < cnt ? max(j, -1) : INT_MIN;
    };
    auto held = [&](int j) -> int { return j >= 0 && (long long)j * page < limit ? __ldg(table + j) : -1; };
    int j_now = entry(ta), pg_now = held(j_now), j_next = entry(ta + per_load);
    for (int t0 = ta; t0 < tb; t0 += per_load) {
      const int pg_next = held(j_next), j_next2 = entry(t0 + 2 * per_load);
      int rows = 0, y = 0;
      if (j_now != INT_MIN) {
        const int off = ((t0 + my_tile) * kTileKeys + my_row) % page;
        if (j_now < 0 || (long long)j_now * page >= limit) {
          bad = true;                            // a list entry past the token's page
        } else {
          rows = min(max(limit - (j_now * page + off), 0), rpb);
          if (rows > 0 && (pg_now < 0 || pg_now >= n_pages)) {
            bad = true;
            rows = 0;
          }
          y = (int)(((long long)pg_now * Hkv + h) * page) + off;
        }
      }
      const int n_here = min(per_load, tb - t0);
      const bool whole = __all_sync(0xffffffffu, my_tile >= n_here || rows == rpb);
      const unsigned long long bits = rows == 0 ? 0 : (rows == 64 ? ~0ull : (1ull << rows) - 1) << my_row;
      for (int i = 0; i < n_here; ++i) {
        const bool mine = my_tile == i && rows > 0;
        unsigned long long keys = ~0ull;
        uint32_t bytes = kTileKeys * D * 2u;
        if (!whole) {
          bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * rpb) * D * 2u;
          const unsigned lo = __reduce_or_sync(0xffffffffu, mine ? (unsigned)bits : 0u);
          const unsigned hi = __reduce_or_sync(0xffffffffu, mine ? (unsigned)(bits >> 32) : 0u);
          keys = ((unsigned long long)hi << 32) | lo;
        }
        if (n >= STAGES && !__all_sync(0xffffffffu, tc::mbar_wait(f.empty + s, parity, abort_flag, status))) return n;
        if (lane == 0) {
          if (f.vmask) f.vmask[n % RING] = keys;
          tc::mbar_arrive_expect_tx(f.full + s, bytes);
        }
        __syncwarp();
        if (mine) {
          uint8_t* dst = f.stage0 + s * f.stage_bytes + my_row * 128;
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh) tc::tma_load_2d(dst + hh * kHalf, f.map, hh * 64, y, f.full + s);
        }
        ++n;
        if (++s == STAGES) {
          s = 0;
          parity ^= 1;
        }
      }
      j_now = j_next;
      pg_now = pg_next;
      j_next = j_next2;
    }
    x = xe;
    if (x < x1) w.next(a, it);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, BSA_DEV_BAD_INDEX);
  return n;
}

// After the other warps are done: no copy of the warp's own is still landing (the last phase issued
// on every stage; earlier phases completed before it). One lane.
template <int STAGES>
__device__ __forceinline__ void feed_drain(uint64_t* full, int issued) {
  for (int t = max(0, issued - STAGES); t < issued; ++t) tc::mbar_wait_timed(full + t % STAGES, (t / STAGES) & 1);
}

}  // namespace bsa
