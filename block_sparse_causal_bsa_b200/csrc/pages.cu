// Pages of a KV cache: forking sequences, growing / shrinking them, copying pages, appending
// rows and compacting the accepted rows of a draft; ancestor masks of a tree of drafts.
//
// The pool and its bookkeeping (page table, lengths, reference counts) live in device memory,
// so that a whole serving step (resize, append, attend, compact) can sit in one CUDA graph. A
// page is free when its reference count is 0, and free pages are taken lowest first: the state
// after a call depends on the state before it alone, not on the order in which threads ran.
//
//   fork     table row and length of the parent copied, one reference more per page
//   resize   shrinking slots give up pages; growing slots then take free ones, and a partly
//            filled last page that other sequences hold too is replaced by a fresh page (the
//            (old, new) pair is returned for the copy of its contents, layer by layer)
//   copy     K, V and bounds of page old -> new
//   append   rows of new tokens into their pages, and those pages' channel bounds
//   compact  rows base + keep[i] -> base + i, and the touched pages' bounds recomputed
//
// All of them move bytes and compute nothing but minima and maxima: the copies are bound by
// memory bandwidth, the bookkeeping by latency (one CTA, a handful of barriers).
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.h"

namespace bsa {

namespace {

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// packed minimum / maximum of two 16-bit floats, NaN if either is NaN

template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Channel bounds of eight channels per thread, over the rows a thread has seen.
template <bool F16>
struct Bounds8 {
  uint32_t lo[4], hi[4];
  __device__ void reset() {
    const uint32_t pinf = F16 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) { lo[i] = pinf; hi[i] = pinf | 0x80008000u; }
  }
  __device__ void add(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { lo[i] = min2<F16>(lo[i], w[i]); hi[i] = max2<F16>(hi[i], w[i]); }
  }
  __device__ void merge(const uint4& l, const uint4& h) {
    const uint32_t a[4] = {l.x, l.y, l.z, l.w}, b[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { lo[i] = min2<F16>(lo[i], a[i]); hi[i] = max2<F16>(hi[i], b[i]); }
  }
  __device__ uint4 vlo() const { return make_uint4(lo[0], lo[1], lo[2], lo[3]); }
  __device__ uint4 vhi() const { return make_uint4(hi[0], hi[1], hi[2], hi[3]); }
};

// Bounds of a block of threads: vectors of a row on consecutive threads (vpr of them), groups
// of vpr threads on different rows. sh holds 2 uint4 per thread. On return, threads < vpr hold
// the bounds over every group. All threads call it.
template <bool F16>
__device__ void reduce_bounds(Bounds8<F16>& b, uint4* sh, int vpr, int groups) {
  sh[2 * threadIdx.x] = b.vlo();
  sh[2 * threadIdx.x + 1] = b.vhi();
  __syncthreads();
  if ((int)threadIdx.x < vpr) {
    for (int g = 1; g < groups; ++g) b.merge(sh[2 * (threadIdx.x + g * vpr)], sh[2 * (threadIdx.x + g * vpr) + 1]);
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// fork: one CTA per slot

__global__ void __launch_bounds__(256) pages_fork_kernel(int slots, int max_pages, int n_pages, int page,
                                                         int32_t* __restrict__ table, int32_t* seq_len,
                                                         int32_t* refs, const int32_t* __restrict__ parent,
                                                         int32_t* dev_status) {
  const int c = blockIdx.x;
  const int p = parent[c];
  if (p < 0) return;
  // a parent is not a child of the same call (its row and length are then not written here),
  // and a child starts empty
  bool ok = p < slots && p != c;
  ok = ok && parent[p] < 0 && seq_len[c] == 0;
  const int len = ok ? seq_len[p] : 0;
  ok = ok && len >= 0 && (long long)len <= (long long)max_pages * page;
  __syncthreads();                       // every thread has read seq_len[c]
  if (!ok) {
    if (threadIdx.x == 0) set_status(dev_status, BSA_DEV_BAD_INDEX);
    return;
  }
  const int n = ceil_div(len, page);
  for (int j = threadIdx.x; j < max_pages; j += blockDim.x) {
    int e = -1;
    if (j < n) {
      e = table[(size_t)p * max_pages + j];
      if (e >= 0 && e < n_pages) {
        atomicAdd(refs + e, 1);
      } else {
        e = -1;
        set_status(dev_status, BSA_DEV_BAD_INDEX);
      }
    }
    table[(size_t)c * max_pages + j] = e;
  }
  if (threadIdx.x == 0) seq_len[c] = len;
}

// ---------------------------------------------------------------------------
// resize: one CTA

constexpr int kResizeThreads = 1024;

struct __align__(16) ResizeSmem {
  int tail[kMaxSlots];                   // shared last page of a growing slot, or -1 (read four at a time)
  int first[kMaxSlots + 1];              // exclusive prefix of the pages given up, then of the pages needed
  int len[kMaxSlots], want[kMaxSlots];   // before and after (want = len: left as it is)
  uint8_t flags[kMaxSlots];              // 1 grows, 2 copy on write, 4 keeps a shared page, 8 granted
  int warp_sum[32];
  int status;
  int taken;                             // pages given out
};

// Exclusive prefix of one value per thread; *total gets the sum. All threads call it.
__device__ int block_exclusive(int v, int* warp_sum, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int r = x - v + (warp ? warp_sum[warp - 1] : 0);
  *total = warp_sum[31];
  __syncthreads();
  return r;
}

// Prefix of per-slot counts count(t) into s.first, in slot order; returns the total. All threads.
template <class F>
__device__ int slot_prefix(ResizeSmem& s, int slots, F count) {
  const int per = ceil_div(slots, kResizeThreads);
  const int t0 = min((int)threadIdx.x * per, slots), t1 = min(t0 + per, slots);
  int mine = 0;
  for (int t = t0; t < t1; ++t) {
    const int c = count(t);
    s.first[t] = c;
    mine += c;
  }
  int total;
  int at = block_exclusive(mine, s.warp_sum, &total);
  for (int t = t0; t < t1; ++t) {
    const int c = s.first[t];
    s.first[t] = at;
    at += c;
  }
  if (threadIdx.x == 0) s.first[slots] = total;
  __syncthreads();
  return total;
}

// The slot whose range of s.first holds i.
__device__ __forceinline__ int slot_of(const ResizeSmem& s, int slots, int i) {
  int lo = 0, hi = slots;                // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (s.first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Everything per slot sits in shared memory after one coalesced read, and every loop over pages runs
// one page per thread, whatever slot it belongs to: the kernel is a chain of some ten barriers and
// five memory latencies. (A warp per slot took 35 us to free 504 slots of up to 47 pages each, now 25: one SM's
// rate of scattered atomics. Growing them takes 16.)
__global__ void __launch_bounds__(kResizeThreads) pages_resize_kernel(
    int slots, int max_pages, int n_pages, int page, int32_t* table, int32_t* seq_len, int32_t* refs,
    const int32_t* __restrict__ new_len, int32_t* __restrict__ pairs, int32_t* n_free, int32_t* dev_status) {
  extern __shared__ __align__(16) uint8_t raw[];
  ResizeSmem& s = *reinterpret_cast<ResizeSmem*>(raw);
  const int tid = threadIdx.x;
  const long long max_len = (long long)max_pages * page;
  if (tid == 0) s.status = s.taken = 0;
  __syncthreads();
  for (int t = tid; t < slots; t += kResizeThreads) {
    const int L = seq_len[t], n = new_len[t];
    const bool ok = L >= 0 && L <= max_len && n <= max_len;
    if (!ok) atomicOr(&s.status, BSA_DEV_BAD_INDEX);
    s.len[t] = ok ? L : 0;
    s.want[t] = ok ? (n < 0 ? L : n) : 0;
    s.flags[t] = ok && n > L ? 1 : 0;
  }
  __syncthreads();

  // 1. shrinking slots give up pages
  const int dropped = slot_prefix(s, slots, [&](int t) {
    return max(ceil_div(s.len[t], page) - ceil_div(s.want[t], page), 0);
  });
  constexpr int kU = 4;                  // pages of a thread in flight
  for (int i0 = tid; i0 < dropped; i0 += kU * kResizeThreads) {
    int32_t* e[kU];
    int pg[kU], held[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kResizeThreads;
      e[u] = nullptr;
      if (i < dropped) {
        const int t = slot_of(s, slots, i);
        e[u] = table + (size_t)t * max_pages + ceil_div(s.want[t], page) + i - s.first[t];
      }
      pg[u] = e[u] ? *e[u] : 0;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      held[u] = 1;
      if (!e[u]) continue;
      *e[u] = -1;
      if (pg[u] < 0 || pg[u] >= n_pages) atomicOr(&s.status, BSA_DEV_BAD_INDEX);
      else held[u] = atomicSub(refs + pg[u], 1);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (held[u] > 0) continue;
      atomicAdd(refs + pg[u], 1);        // was not held: leave the count as it was
      atomicOr(&s.status, BSA_DEV_BAD_INDEX);
    }
  }
  __threadfence();
  __syncthreads();

  // 2. growing slots whose partly filled last page has other holders (shrinking slots set their length)
  for (int t = tid; t < kMaxSlots; t += kResizeThreads) {
    int tail = -1;
    if (t < slots) {
      const int L = s.len[t];
      if (s.want[t] < L) seq_len[t] = s.want[t];
      if ((s.flags[t] & 1) && L % page) {
        const int pg = table[(size_t)t * max_pages + L / page];
        if (pg < 0 || pg >= n_pages) {
          atomicOr(&s.status, BSA_DEV_BAD_INDEX);
          s.flags[t] = 0;                // not grown
        } else if (__ldcg(refs + pg) > 1) {
          tail = pg;
        }
      }
    }
    s.tail[t] = tail;
  }
  __syncthreads();
  // When every holder of such a page grows, the last of them keeps it and the others copy;
  // else all of them copy. (The pages go to a prefix of the slots, so if the keeper is
  // granted its own, every other holder has left.)
  for (int t = tid; t < slots; t += kResizeThreads) {
    const int pg = s.tail[t];
    if (pg < 0) continue;
    int holders = 0, last = 0;
    for (int u = 0; u < slots; u += 4) {           // (tail is -1 past the slots)
      const int4 v = *reinterpret_cast<const int4*>(s.tail + u);
      holders += (v.x == pg) + (v.y == pg) + (v.z == pg) + (v.w == pg);
      if (v.x == pg) last = u;
      if (v.y == pg) last = u + 1;
      if (v.z == pg) last = u + 2;
      if (v.w == pg) last = u + 3;
    }
    s.flags[t] |= (holders == __ldcg(refs + pg) && last == t) ? 4 : 2;
  }
  __syncthreads();

  // 3. pages needed per slot, in slot order
  const int total = slot_prefix(s, slots, [&](int t) {
    return s.flags[t] & 1 ? ceil_div(s.want[t], page) - ceil_div(s.len[t], page) + ((s.flags[t] >> 1) & 1) : 0;
  });

  // 4. free pages: a contiguous range of the pool per thread (rounded to a multiple of four,
  // so that it is read 16 bytes at a time), counted, then given out lowest first
  const int seg = ceil_div(ceil_div(n_pages, kResizeThreads), 4) * 4;
  const int p0 = (int)min((long long)tid * seg, (long long)n_pages), p1 = min(p0 + seg, n_pages);
  auto counts = [&](int p) {             // of pages p .. p + 3; 1 past the end
    if (p + 4 <= p1) return __ldcg(reinterpret_cast<const int4*>(refs + p));
    int4 r = make_int4(1, 1, 1, 1);
    if (p < p1) r.x = __ldcg(refs + p);
    if (p + 1 < p1) r.y = __ldcg(refs + p + 1);
    if (p + 2 < p1) r.z = __ldcg(refs + p + 2);
    return r;
  };
  int free_here = 0;
#pragma unroll 4
  for (int p = p0; p < p1; p += 4) {
    const int4 r = counts(p);
    free_here += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  int avail;
  int rank = block_exclusive(free_here, s.warp_sum, &avail);
  for (int t = tid; t < slots; t += kResizeThreads) {
    if (!(s.flags[t] & 1)) continue;
    const int need = s.first[t + 1] - s.first[t];
    if ((need == 0 && !(s.flags[t] & 4)) || s.first[t + 1] <= avail) {
      s.flags[t] |= 8;
      if (need) atomicAdd(&s.taken, need);
    } else {
      atomicOr(&s.status, BSA_DEV_NO_PAGES);
    }
  }
  __syncthreads();
  for (int p = p0; p < p1 && rank < total; p += 4) {
    const int4 r4 = counts(p);
    const int c4[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c4[k] != 0 || rank >= total) continue;
      const int r = rank++, pg = p + k;
      const int t = slot_of(s, slots, r);          // (the last slot with first <= r: it needs pages)
      if (!(s.flags[t] & 8)) continue;
      const int i = r - s.first[t], cow = (s.flags[t] >> 1) & 1, L = s.len[t];
      refs[pg] = 1;
      if (cow && i == 0) {
        pairs[2 * t] = s.tail[t];
        pairs[2 * t + 1] = pg;
        atomicSub(refs + s.tail[t], 1);            // stays above 0: another holder keeps the page
        table[(size_t)t * max_pages + L / page] = pg;
      } else {
        table[(size_t)t * max_pages + ceil_div(L, page) + i - cow] = pg;
      }
    }
  }
  for (int t = tid; t < slots; t += kResizeThreads) {
    if (s.flags[t] & 8) seq_len[t] = s.want[t];
    if ((s.flags[t] & 10) != 10) pairs[2 * t] = pairs[2 * t + 1] = -1;
  }
  if (tid == 0) {
    if (n_free) *n_free = avail - s.taken;
    if (dev_status) *dev_status = s.status;
  }
}

// ---------------------------------------------------------------------------
// copy: one CTA per (pair, head, K or V). The reads of the page are on their way while the pair is
// checked against the others, and sources stay in L2, since several pairs may read one (448 copies of
// 56 pages of 512 KB: 67 us with reads behind the check and past L2, now 42, that is 6.3 TB/s).

__global__ void __launch_bounds__(256) pages_copy_kernel(uint4* __restrict__ k, uint4* __restrict__ v,
                                                         uint4* __restrict__ bounds,
                                                         const int2* __restrict__ pairs, int n_pairs,
                                                         int n_pages, int Hkv, int vec_page, int vec_bounds,
                                                         int32_t* dev_status) {
  const int i = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
  const int2 pr = pairs[i];
  if (pr.x < 0 && pr.y < 0) return;
  bool bad = pr.x < 0 || pr.x >= n_pages || pr.y < 0 || pr.y >= n_pages;     // (the same for all threads)
  const size_t src = ((size_t)(bad ? 0 : pr.x) * Hkv + h), dst = ((size_t)(bad ? 0 : pr.y) * Hkv + h);
  const uint4* from = (blockIdx.y ? v : k) + src * vec_page;
  uint4* to = (blockIdx.y ? v : k) + dst * vec_page;
  constexpr int U = 8;                           // 128 rows of 128 channels in one go
  uint4 a[U];
  auto load = [&](int e) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e + u * 256 < vec_page) a[u] = __ldcg(from + e + u * 256);
  };
  if (!bad) load(threadIdx.x);
  // the destination must be no page that another pair reads, nor one that an earlier pair
  // writes: the copies run in any order
  for (int j = threadIdx.x; j < n_pairs; j += 256) {
    const int2 o = pairs[j];
    bad |= o.x == pr.y || (o.y == pr.y && j < i);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(dev_status, BSA_DEV_BAD_INDEX);
    return;
  }
  for (int e = threadIdx.x; e < vec_page; e += U * 256) {
    if (e >= U * 256) load(e);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e + u * 256 < vec_page) __stcs(to + e + u * 256, a[u]);
  }
  if (bounds && blockIdx.y == 0)
    for (int e = threadIdx.x; e < vec_bounds; e += 256) bounds[dst * vec_bounds + e] = bounds[src * vec_bounds + e];
}

// ---------------------------------------------------------------------------
// Checks of append and compact that one CTA makes for the whole call (the others skip what
// they may not touch without a word): lengths, and the table entries of the call's tokens.
__device__ int check_spans(const CacheGeom& g) {
  int st = 0;
  for (int b = threadIdx.x; b < g.slots; b += blockDim.x) {
    int base, ql;
    if (!query_span(g, b, base, ql)) st |= BSA_DEV_BAD_INDEX;
    if (ql == 0) continue;
    for (int j = base / g.page; j <= (base + ql - 1) / g.page; ++j) {
      const int pg = g.table[(size_t)b * g.max_pages + j];
      if (pg < 0 || pg >= g.n_pages) st |= BSA_DEV_BAD_INDEX;
    }
  }
  return st;
}

// append: one CTA per (slot, head, touched page), and one that checks. Bound by memory; the rows' reads go
// out with the table's entry (behind it, 32 chunks of 513 to 1024 rows took 39 us; now 37, 5.4 TB/s). The first page's
// earlier rows are read as well, for its bounds (64 users' rows, replayed: 4.5 us without them, 6.4 with).

constexpr int kAppendThreads = 128;

template <bool F16>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(
    CacheGeom g, int touch, const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
    uint4* __restrict__ k, uint4* __restrict__ v, uint4* __restrict__ bounds, int32_t* dev_status) {
  __shared__ uint4 sh[2 * kAppendThreads];
  if (blockIdx.x == gridDim.x - 1) {
    const int st = __syncthreads_or(check_spans(g));
    if (threadIdx.x == 0) *dev_status = st ? BSA_DEV_BAD_INDEX : 0;
    return;
  }
  int x = blockIdx.x;
  const int ti = x % touch;
  x /= touch;
  const int h = x % g.Hkv, b = x / g.Hkv;
  int base, ql;
  if (!query_span(g, b, base, ql) || ql == 0) return;
  const int j = base / g.page + ti;
  const int lo = max(base, j * g.page), hi = min(base + ql, (j + 1) * g.page);   // positions
  if (lo >= hi) return;
  const int vpr = g.d / 8, groups = kAppendThreads / vpr, n = hi - lo;
  const int vec = threadIdx.x % vpr, row = threadIdx.x / vpr;
  const size_t src = (((size_t)b * g.Hkv + h) * g.T + (lo - base)) * vpr + vec;
  // (the first rows are on their way with the table's entry)
  constexpr int U = 4;
  uint4 a[U], c[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * groups;
      if (r < n) {
        a[u] = __ldcs(k_new + src + (size_t)r * vpr);
        c[u] = __ldcs(v_new + src + (size_t)r * vpr);
      }
    }
  };
  load(row);
  const int pg = g.table[(size_t)b * g.max_pages + j];
  if (pg < 0 || pg >= g.n_pages) return;
  const size_t dst = (((size_t)pg * g.Hkv + h) * g.page + (lo - j * g.page)) * vpr + vec;
  Bounds8<F16> bd;
  bd.reset();
  // The page's rows before the call are read again: the bounds kept with it may be those of more rows, since
  // dropped by a resize, or of another slot's rows, where the page was copied.
  const int before = bounds ? lo - j * g.page : 0;
  const uint4* const old = k + ((size_t)pg * g.Hkv + h) * g.page * vpr + vec;
  uint4 o[U];                            // (twice as many: 121 registers, 48 drafts compacted 14.6 us for 12.6)
  auto load_old = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u * groups < before) o[u] = old[(size_t)(r0 + u * groups) * vpr];
  };
  load_old(row);                         // (on their way while the new rows are written)
  for (int r0 = row; r0 < n; r0 += U * groups) {
    if (r0 != row) load(r0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * groups;
      if (r < n) {
        k[dst + (size_t)r * vpr] = a[u];
        v[dst + (size_t)r * vpr] = c[u];
        bd.add(a[u]);
      }
    }
  }
  for (int r0 = row; r0 < before; r0 += U * groups) {
    if (r0 != row) load_old(r0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u * groups < before) bd.add(o[u]);
  }
  if (!bounds) return;
  reduce_bounds<F16>(bd, sh, vpr, groups);
  if ((int)threadIdx.x < vpr) {
    uint4* bp = bounds + ((size_t)pg * g.Hkv + h) * 2 * vpr + threadIdx.x;
    bp[0] = bd.vlo();
    bp[vpr] = bd.vhi();
  }
}

// compact: one CTA per (slot, head), and one that checks

constexpr int kCompactThreads = 256;

// Whether this thread's share (i0, i0 + step, ...) of a keep list breaks the rule: ascending,
// and within the call's tokens.
__device__ __forceinline__ bool keep_bad(const int32_t* keep, int nk, int ql, int i0, int step) {
  bool bad = nk < 0 || nk > ql;
  if (!bad)
    for (int i = i0; i < nk; i += step) bad |= keep[i] < 0 || keep[i] >= ql || (i > 0 && keep[i] <= keep[i - 1]);
  return bad;
}

template <bool F16>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(
    CacheGeom g, const int32_t* __restrict__ keep, const int32_t* __restrict__ n_keep, uint4* k, uint4* v,
    uint4* __restrict__ bounds, int32_t* dev_status) {
  __shared__ uint4 sh[2 * kCompactThreads];
  if (blockIdx.x == gridDim.x - 1) {
    int st = check_spans(g);
    for (int b = threadIdx.x / 32; b < g.slots; b += kCompactThreads / 32) {
      int base, ql;
      query_span(g, b, base, ql);
      if (ql > 0 && keep_bad(keep + (size_t)b * g.T, n_keep[b], ql, threadIdx.x % 32, 32)) st |= BSA_DEV_BAD_INDEX;
    }
    st = __syncthreads_or(st);
    if (threadIdx.x == 0) *dev_status = st ? BSA_DEV_BAD_INDEX : 0;
    return;
  }
  const int b = blockIdx.x / g.Hkv, h = blockIdx.x % g.Hkv;
  int base, ql;
  if (!query_span(g, b, base, ql) || ql == 0) return;
  const int32_t* kp = keep + (size_t)b * g.T;
  const int32_t* tb = g.table + (size_t)b * g.max_pages;
  const int nk = n_keep[b];
  bool bad = false;
  for (int j = base / g.page + threadIdx.x; j <= (base + ql - 1) / g.page; j += blockDim.x)
    bad |= tb[j] < 0 || tb[j] >= g.n_pages;
  bad |= keep_bad(kp, nk, ql, threadIdx.x, blockDim.x);
  if (__syncthreads_or(bad)) return;

  const int vpr = g.d / 8, groups = kCompactThreads / vpr;
  const int vec = threadIdx.x % vpr, row = threadIdx.x / vpr;
  auto at = [&](int pos) {
    return (((size_t)tb[pos / g.page] * g.Hkv + h) * g.page + pos % g.page) * vpr + vec;
  };
  // Chunks of rows in ascending order, each read whole before it is written: row i goes to
  // base + i <= base + keep[i], so no chunk overwrites a row that a later one reads.
  for (int c0 = 0; c0 < nk; c0 += groups) {
    const int i = c0 + row;
    const int from = i < nk ? kp[i] : i;
    uint4 a, c;
    size_t to = 0;
    if (from != i) {
      const size_t src = at(base + from);
      to = at(base + i);
      a = k[src];
      c = v[src];
    }
    __syncthreads();
    if (from != i) {
      k[to] = a;
      v[to] = c;
    }
    __syncthreads();
  }
  if (!bounds) return;
  const int end = base + nk;
  for (int j = base / g.page; j * g.page < end; ++j) {
    Bounds8<F16> bd;
    bd.reset();
    for (int p = j * g.page + row; p < min(end, (j + 1) * g.page); p += groups) bd.add(k[at(p)]);
    reduce_bounds<F16>(bd, sh, vpr, groups);
    if ((int)threadIdx.x < vpr) {
      uint4* bp = bounds + ((size_t)tb[j] * g.Hkv + h) * 2 * vpr + threadIdx.x;
      bp[0] = bd.vlo();
      bp[vpr] = bd.vhi();
    }
  }
}

// ---------------------------------------------------------------------------
// tree masks: bit j of row t is set when j is t or an ancestor of t. One CTA per sequence. A
// parent comes before its token, so a walk up the tree passes the 64-token blocks in descending
// order. First every token walks to the end of its own block and leaves the bits it met and the token
// it came out at; then a thread per mask word hops from block to block: at most 64 + 16 steps
// where a plain walk per word took up to 1024 (a chain of 1024 tokens: 1134 -> 45 us).

__global__ void __launch_bounds__(256) tree_mask_kernel(int T, int words, const int32_t* __restrict__ parents,
                                                        const int32_t* __restrict__ q_len,
                                                        unsigned long long* __restrict__ mask,
                                                        int32_t* dev_status) {
  __shared__ int16_t par[kMaxQueryTokens], out_at[kMaxQueryTokens];
  __shared__ unsigned long long met[kMaxQueryTokens];
  const int b = blockIdx.x;
  int ql = q_len ? q_len[b] : T;
  bool bad = ql < 0 || ql > T;
  if (bad) ql = 0;
  for (int t = threadIdx.x; t < ql; t += blockDim.x) {
    const int p = parents[(size_t)b * T + t];
    const bool ok = p >= -1 && p < t;                  // parents come first: the walk ends
    bad |= !ok;
    par[t] = ok ? (int16_t)p : (int16_t)-1;
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) set_status(dev_status, BSA_DEV_BAD_INDEX);
  for (int t = threadIdx.x; t < ql; t += blockDim.x) {
    const int first = t & ~63;
    unsigned long long bits = 0;
    int x = t;
    for (; x >= first; x = par[x]) bits |= 1ull << (x & 63);
    met[t] = bits;
    out_at[t] = (int16_t)x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * words; i += blockDim.x) {
    const int t = i / words, w = i % words;
    unsigned long long bits = 0;
    if (t < ql) {
      int x = t;
      while (x >= 64 * (w + 1)) x = out_at[x];
      if (x >= 64 * w) bits = met[x];
    }
    mask[(size_t)b * T * words + i] = bits;
  }
}

}  // namespace

cudaError_t launch_pages_fork(int slots, int max_pages, int n_pages, int page, int32_t* table,
                              int32_t* seq_len, int32_t* refs, const int32_t* parent, int32_t* dev_status,
                              cudaStream_t st) {
  pages_fork_kernel<<<slots, 256, 0, st>>>(slots, max_pages, n_pages, page, table, seq_len, refs, parent,
                                           dev_status);
  return cudaGetLastError();
}

cudaError_t launch_pages_resize(int slots, int max_pages, int n_pages, int page, int32_t* table,
                                int32_t* seq_len, int32_t* refs, const int32_t* new_len, int32_t* pairs,
                                int32_t* n_free, int32_t* dev_status, cudaStream_t st) {
  static SmemSet set;
  cudaError_t e = allow_smem((const void*)pages_resize_kernel, sizeof(ResizeSmem), set);
  if (e != cudaSuccess) return e;
  pages_resize_kernel<<<1, kResizeThreads, sizeof(ResizeSmem), st>>>(
      slots, max_pages, n_pages, page, table, seq_len, refs, new_len, pairs, n_free, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const bsa_cache_shape& s, void* k, void* v, void* bounds, const int32_t* pairs,
                              int n_pairs, int32_t* dev_status, cudaStream_t st) {
  const int vpr = s.d / 8;
  pages_copy_kernel<<<dim3((unsigned)((long long)n_pairs * s.Hkv), 2), 256, 0, st>>>(
      (uint4*)k, (uint4*)v, (uint4*)bounds, (const int2*)pairs, n_pairs, s.n_pages, s.Hkv, s.page * vpr,
      2 * vpr, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const bsa_cache_shape& s, const CacheGeom& g, const void* k_new,
                                const void* v_new, void* k, void* v, void* bounds, int32_t* dev_status,
                                cudaStream_t st) {
  const int touch = (g.T + g.page - 2) / g.page + 1;   // pages that T consecutive positions can touch
  const unsigned grid = (unsigned)((long long)g.slots * g.Hkv * touch + 1);
  auto kern = s.dtype == BSA_F16 ? cache_append_kernel<true> : cache_append_kernel<false>;
  kern<<<grid, kAppendThreads, 0, st>>>(g, touch, (const uint4*)k_new, (const uint4*)v_new, (uint4*)k,
                                        (uint4*)v, (uint4*)bounds, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const bsa_cache_shape& s, const CacheGeom& g, const int32_t* keep,
                                 const int32_t* n_keep, void* k, void* v, void* bounds, int32_t* dev_status,
                                 cudaStream_t st) {
  const unsigned grid = (unsigned)((long long)g.slots * g.Hkv + 1);
  auto kern = s.dtype == BSA_F16 ? cache_compact_kernel<true> : cache_compact_kernel<false>;
  kern<<<grid, kCompactThreads, 0, st>>>(g, keep, n_keep, (uint4*)k, (uint4*)v, (uint4*)bounds, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_tree_mask(int B, int T, const int32_t* parents, const int32_t* q_len,
                             unsigned long long* mask, int32_t* dev_status, cudaStream_t st) {
  tree_mask_kernel<<<B, 256, 0, st>>>(T, (T + 63) / 64, parents, q_len, mask, dev_status);
  return cudaGetLastError();
}

}  // namespace bsa
