// Attention over a paged cache on tcgen05: trees and chains of drafted tokens, up to 128 query
// rows (heads of a KV group x tokens) per item.
//
//   O = sum softmax(scale q.k) v over the positions a token sees
//
// 128 rows against a key cost 4 * 128 * d flops for the 4 d bytes of its K and V: with full tiles the
// tensor cores and the exponentials bound the kernel, with few rows the HBM reads of the cache.
// Two CTAs per SM (192 threads, 256 TMEM columns, ~100 KB of shared memory each), each
// walking its share of all key tiles (paged_work.cuh), so that one's softmax overlaps the other's
// products and loads:
//   warp 0     producer: page numbers in its lanes' registers, then per tile one TMA box per page and
//              64-column half, K and V in separate stages
//   warp 1     one thread issues S_n = Q K_n^T into one of two TMEM buffers, S_{n+1} before the value product of
//              tile n, and O += P_n V_n with P read from TMEM
//   warps 2-5  a thread per row: Q of the item into shared memory (128-byte swizzle, as TMA would write
//              it), then per tile S from TMEM, the mask where the tile needs one, the online
//              softmax (O rescaled in TMEM only when the maximum grew by more than 2^8), P in 16
//              bits over the S just read; O / l or the partial result at the end of a segment. Warps whose
//              rows are all past the item's skip the arithmetic.
// P is rounded to 16 bits, a relative 2^-9 (bf16) or 2^-12 (fp16) per weight, within the rounding of the
// output; sums and maxima are fp32. For fp16, weights carry a factor 2^7: with the maximum up to 2^8
// stale they stay below 2^15, and weights down to 2^-31 of the largest still count.
// Rows that are no keys, and non-finite values of drafted rows, are treated as in paged_attend.cu:
// the softmax warps mend the V tile in shared memory before they release P.
#include <math.h>

#include "paged_work.cuh"
#include "tc_common.cuh"

namespace bsa {

namespace {

constexpr int kThreads = 192;
constexpr int RT = 128;
constexpr int kMaskRing = 16;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColO = 0;                   // O accumulator
constexpr uint32_t kColS = 128;                 // S buffers at 128 and 192

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQHalf = RT * 128;
  static constexpr uint32_t kHalf = kTileKeys * 128;
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr int NS = D == 128 ? 2 : 4;
  static constexpr size_t kQ = 0, kK = kHalves * kQHalf, kV = kK + NS * kTile, kCtrl = kV + NS * kTile;
};

struct __align__(16) Ctrl {
  uint64_t q_full;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2];
  uint64_t p_full, o_ready, done;
  unsigned long long vmask[kMaskRing];          // by tile: rows that are keys
  uint32_t tmem;
  int abort_flag;
  int32_t status;
  int flag[2];                                  // by segment parity: non-finite drafts taken out
  int last;                                     // this CTA joins the item's parts
};

template <int D>
constexpr size_t smem_bytes() { return Cfg<D>::kCtrl + sizeof(Ctrl) + 1024; }

__device__ __forceinline__ bool warp_all(bool x) { return __all_sync(0xffffffffu, x); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Keys of the tile that starts dj positions after the slot's first token (dj may be negative) that
// token t sees: bit i for key i.
__device__ __forceinline__ uint64_t draft_window(const PagedArgs& a, int b, int t, int dj) {
  if (!a.mask) {
    const int n = t - dj + 1;
    return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1);
  }
  const unsigned long long* m = a.mask + ((size_t)b * a.g.T + t) * a.words;
  if (dj < 0) return dj <= -64 ? ~0ull : (m[0] << -dj) | ((1ull << -dj) - 1);
  const int w = dj >> 6, s = dj & 63;
  if (w >= a.words) return 0ull;
  uint64_t x = m[w] >> s;
  if (s && w + 1 < a.words) x |= m[w + 1] << (64 - s);
  return x;
}

// Parts lie transposed, [D / 4][RT] of four floats: a warp's rows are then neighbours both when a
// part is written (a thread per row) and when parts are joined.
__device__ __forceinline__ float4* part4(const PagedArgs& a, size_t slot, int D, int d4, int r) {
  return reinterpret_cast<float4*>(a.part_o) + (slot * (D / 4) + d4) * RT + r;
}

// Joins the parts of an item, the four softmax warps: 128 / R threads per row, R the rows rounded up
// to whole warps; eight reads of 16 bytes in flight per thread.
template <int D, bool F16>
__device__ __noinline__ void join_rows(const PagedArgs& a, const Item& it, const Parts<false, RT>& parts, int tid,
                                       bool ok) {
  constexpr float kShift = F16 ? 7.f : 0.f;
  constexpr int kU = 8;
  const int np = parts.n, R = (it.rows + 31) / 32 * 32;
  const int groups = 128 / R, r = tid % R, dg = tid / R;       // (R = 96: one group, 32 threads idle)
  if (dg >= groups || r >= it.rows) return;
  float mx = -INFINITY, ls = 0.f;
  int flag = 0;
#pragma unroll 8
  for (int i = 0; i < np; ++i) {
    mx = fmaxf(mx, __ldcg(a.part_ml + (parts.slot(i) * RT + r) * 2));
    flag |= __ldcg(a.part_flag + parts.slot(i));
  }
  int head, t;
  row_of<false>(a, it, r, head, t);
  const size_t row = ((size_t)it.b * a.Hq + head) * a.g.T + t;
  for (int d0 = dg; d0 < D / 4; d0 += groups * kU) {
    float4 acc[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    ls = 0.f;
#pragma unroll 2
    for (int i = 0; i < np; ++i) {
      const size_t slot = parts.slot(i);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (slot * RT + r) * 2));
      float4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d0 + u * groups < D / 4) v[u] = __ldcg(part4(a, slot, D, d0 + u * groups, r));
      }
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
      ls += ml.y * f;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        acc[u].x = fmaf(v[u].x, f, acc[u].x);
        acc[u].y = fmaf(v[u].y, f, acc[u].y);
        acc[u].z = fmaf(v[u].z, f, acc[u].z);
        acc[u].w = fmaf(v[u].w, f, acc[u].w);
      }
    }
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int d4 = d0 + u * groups;
      if (d4 >= D / 4) break;
      float y[4] = {acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv};
      if (flag) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += nonfinite_drafts<F16>(a, it, t, 4 * d4 + e);
      }
      if (ok)
        *reinterpret_cast<uint2*>(a.out + row * D + 4 * d4) =
            make_uint2(pack_16<F16>(y[0], y[1]), pack_16<F16>(y[2], y[3]));
    }
  }
  if (ok && dg == 0 && a.lse) a.lse[row] = ls == 0.f ? -INFINITY : (mx - kShift + log2f(ls)) * 0.69314718055994531f;
}

}  // namespace

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2) paged_attend_tc_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
    const __grid_constant__ PagedArgs a) {
  using C = Cfg<D>;
  constexpr int NS = C::NS;
  constexpr float kShift = F16 ? 7.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl& c = *reinterpret_cast<Ctrl*>(sm + C::kCtrl);
  const uint32_t sQ = tc::smem_u32(sm + C::kQ), sK = tc::smem_u32(sm + C::kK), sV = tc::smem_u32(sm + C::kV);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    tc::mbar_init(&c.q_full, 4);
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&c.k_full[s], 1);
      tc::mbar_init(&c.k_empty[s], 1);
      tc::mbar_init(&c.v_full[s], 1);
      tc::mbar_init(&c.v_empty[s], 1);
    }
    // the issuing thread arrives itself, too: what it saw (the tile's mask) is then visible to
    // the softmax warps
    tc::mbar_init(&c.s_full[0], 2);
    tc::mbar_init(&c.s_full[1], 2);
    tc::mbar_init(&c.p_full, 4);
    tc::mbar_init(&c.o_ready, 1);
    tc::mbar_init(&c.done, 1);
    c.abort_flag = 0;
    c.status = 0;
    c.flag[0] = c.flag[1] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&c.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort_flag = &c.abort_flag;
  int32_t* status = &c.status;

  Walk<false, RT> w;
  w.init(a);
  const long long x0 = w.start(blockIdx.x), x1 = w.start(blockIdx.x + 1);
  Item it;
  if (x0 < x1) w.locate(a, x0, it);
  int k_issued = 0, v_issued = 0;
  bool mma_issued = false;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0) {
      tc::prefetch_tmap(&tmk);
      tc::prefetch_tmap(&tmv);
    }
    const int page = a.g.page, rpb = page < kTileKeys ? page : kTileKeys, npt = kTileKeys / rpb;
    const int per_load = 32 / npt;
    int n = 0;
    bool ok = true;
    for (long long x = x0; ok && x < x1;) {
      const long long xe = min(x1, it.first + it.n_tiles);
      const int ta = (int)(x - it.first), tb = (int)(xe - it.first);
      const int32_t* table = a.g.table + (size_t)it.b * a.g.max_pages;
      const int limit = it.base + it.ql;
      bool bad = false;
      for (int t0 = ta; ok && t0 < tb; t0 += per_load) {
        // lane i: box (i % npt) of tile t0 + i / npt
        const int tile = t0 + lane / npt;
        const int pos = tile * kTileKeys + (lane % npt) * rpb;
        int rows = tile < tb ? min(max(limit - pos, 0), rpb) : 0, y = 0;
        if (rows > 0) {
          const int pg = table[pos / page];
          if (pg < 0 || pg >= a.g.n_pages) {
            bad = true;
            rows = 0;
          }
          y = (int)(((long long)pg * a.g.Hkv + it.h) * page) + pos % page;
        }
        const unsigned long long bits =
            rows == 0 ? 0 : (rows == 64 ? ~0ull : (1ull << rows) - 1) << ((lane % npt) * rpb);
        const int n_here = min(per_load, tb - t0);
        for (int i = 0; i < n_here; ++i) {
          const int s = n % NS;
          const bool mine = lane / npt == i;
          const unsigned boxes = __ballot_sync(0xffffffffu, mine && rows > 0);
          const unsigned lo = __reduce_or_sync(0xffffffffu, mine ? (unsigned)bits : 0u);
          const unsigned hi = __reduce_or_sync(0xffffffffu, mine ? (unsigned)(bits >> 32) : 0u);
          const uint32_t bytes = (uint32_t)(__popc(boxes) * rpb) * D * 2u;
          const uint32_t row_off = (uint32_t)((lane % npt) * rpb) * 128u;
          if (n >= NS) ok = warp_all(tc::mbar_wait(&c.k_empty[s], ((n / NS) - 1) & 1, abort_flag, status));
          if (!ok) break;
          if (lane == 0) {
            c.vmask[n % kMaskRing] = ((unsigned long long)hi << 32) | lo;
            tc::mbar_arrive_expect_tx(&c.k_full[s], bytes);
          }
          __syncwarp();
          if (mine && rows > 0) {
#pragma unroll
            for (int hh = 0; hh < C::kHalves; ++hh)
              tc::tma_load_2d(sm + C::kK + s * C::kTile + hh * C::kHalf + row_off, &tmk, hh * 64, y, &c.k_full[s]);
          }
          k_issued = n + 1;
          if (n >= NS) ok = warp_all(tc::mbar_wait(&c.v_empty[s], ((n / NS) - 1) & 1, abort_flag, status));
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(&c.v_full[s], bytes);
          __syncwarp();
          if (mine && rows > 0) {
#pragma unroll
            for (int hh = 0; hh < C::kHalves; ++hh)
              tc::tma_load_2d(sm + C::kV + s * C::kTile + hh * C::kHalf + row_off, &tmv, hh * 64, y, &c.v_full[s]);
          }
          v_issued = n + 1;
          ++n;
        }
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, BSA_DEV_BAD_INDEX);
      x = xe;
      if (x < x1) w.next(a, it);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // (the walk is the whole warp's; one lane waits and issues)
    constexpr uint32_t idS = F16 ? tc::idesc_f16_f32(128, 64, false, false) : tc::idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idPV = F16 ? tc::idesc_f16_f32(128, D, false, true) : tc::idesc_bf16_f32(128, D, false, true);
    int n = 0, seg = 0;
    bool ok = true;
    for (long long x = x0; x < x1; ++seg) {
      const long long xe = min(x1, it.first + it.n_tiles);
      const int L = (int)(xe - x);
      if (lane == 0 && ok) {
        auto issue_s = [&](int j) {
          const uint32_t kb = sK + (j % NS) * C::kTile;
          const uint32_t d = tmem + kColS + (j % 2) * 64;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qoff = (kk >> 2) * C::kQHalf + (kk & 3) * 32;
            const uint32_t koff = (kk >> 2) * C::kHalf + (kk & 3) * 32;
            tc::umma_bf16(d, tc::sdesc_sw128(sQ + qoff, 16, 1024), tc::sdesc_sw128(kb + koff, 16, 1024), idS, kk > 0);
          }
          tc::mbar_arrive(&c.s_full[j % 2]);
          tc::umma_commit(&c.s_full[j % 2]);
          tc::umma_commit(&c.k_empty[j % NS]);
        };
        ok = tc::mbar_wait(&c.q_full, seg & 1, abort_flag, status) &&
             tc::mbar_wait(&c.k_full[n % NS], (n / NS) & 1, abort_flag, status);
        if (ok) {
          tc::tc_fence_after();
          issue_s(n);
          mma_issued = true;
        }
        for (int i = 0; ok && i < L; ++i) {
          const int j = n + i, jn = j + 1;
          if (i + 1 < L) {
            // S(jn) overwrites the buffer whose P the value product of tile jn - 2 reads
            ok = tc::mbar_wait(&c.k_full[jn % NS], (jn / NS) & 1, abort_flag, status) &&
                 (jn < 2 || tc::mbar_wait(&c.o_ready, (jn - 2) & 1, abort_flag, status));
            if (!ok) break;
            tc::tc_fence_after();
            issue_s(jn);
          }
          ok = tc::mbar_wait(&c.v_full[j % NS], (j / NS) & 1, abort_flag, status) &&
               tc::mbar_wait(&c.p_full, j & 1, abort_flag, status);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t vb = sV + (j % NS) * C::kTile;
          const uint32_t pa = tmem + kColS + (j % 2) * 64;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::umma_bf16_ts(tmem + kColO, pa + kk * 8, tc::sdesc_sw128(vb + kk * 2048, C::kHalf, 1024), idPV,
                             (i > 0 || kk > 0) ? 1u : 0u);
          tc::umma_commit(&c.o_ready);
          tc::umma_commit(&c.v_empty[j % NS]);
        }
      }
      __syncwarp();
      n += L;
      x = xe;
      if (x < x1) w.next(a, it);
    }
  } else {
    // ---------------- softmax warps ----------------
    const int quarter = warp & 3;                        // TMEM lane quarter of this warp
    const int r = quarter * 32 + lane;                   // row of the item
    const int tid = threadIdx.x - 64;                    // 0..127
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const float scale_log2 = a.scale_log2;
    int n = 0, seg = 0;
    bool ok = true;
    for (long long x = x0; x < x1; ++seg) {
      const long long xe = min(x1, it.first + it.n_tiles);
      const int ta = (int)(x - it.first), tb = (int)(xe - it.first);
      const bool live = quarter * 32 < it.rows;          // the warp has rows
      int head, t;
      row_of<false>(a, it, r < it.rows ? r : 0, head, t);
      const size_t grow = ((size_t)it.b * a.Hq + head) * a.g.T + t;
      {
        // every product that read the previous Q has completed: its S was read below
        const uint4* qr = reinterpret_cast<const uint4*>(a.q + grow * D);
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = r < it.rows ? __ldg(qr + ch) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(sm + C::kQ + (ch >> 3) * C::kQHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&c.q_full);
      }
      float m_used = -INFINITY, l = 0.f;
      for (int tile = ta; tile < tb; ++tile, ++n) {
        if (ok) ok = warp_all(tc::mbar_wait(&c.s_full[n % 2], (n / 2) & 1, abort_flag, status));
        if (!ok) continue;
        tc::tc_fence_after();
        const int pos0 = tile * kTileKeys;
        const uint64_t vm = c.vmask[n % kMaskRing];
        const bool drafts = pos0 + kTileKeys > it.base;
        if (vm != ~0ull || (drafts && (a.mask || it.ql > 1))) {
          // mend the V tile: rows that are no keys become 0, non-finite drafted values are taken out
          ok = warp_all(tc::mbar_wait(&c.v_full[n % NS], (n / NS) & 1, abort_flag, status));
          if (!ok) continue;
          const int row = tid / 2;
          const bool key = (vm >> row) & 1;
          if (!key || (drafts && pos0 + row >= it.base)) {
            bool found = false;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const int ch = (tid & 1) * (D / 16) + i;
              uint4* p = reinterpret_cast<uint4*>(sm + C::kV + (n % NS) * C::kTile + (ch >> 3) * C::kHalf + row * 128 +
                                                  (((ch & 7) ^ (row & 7)) << 4));
              uint4 v = make_uint4(0, 0, 0, 0);
              if (key) {
                v = *p;
                found |= clear_nonfinite<F16>(v.x) | clear_nonfinite<F16>(v.y) | clear_nonfinite<F16>(v.z) |
                         clear_nonfinite<F16>(v.w);
              }
              *p = v;
            }
            if (found) atomicOr(&c.flag[seg & 1], 1);
          }
          tc::fence_proxy_async_smem();
        }
        float alpha = 1.f;
        uint32_t pk[32];
        if (live) {
          float s[64];
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t v[32];
            tc::tmem_ld32(tl + kColS + (n % 2) * 64 + cc * 32, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[cc * 32 + i] = __uint_as_float(v[i]);
          }
          float mx8[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) mx8[u] = -INFINITY;
          if (vm != ~0ull || drafts) {
            const uint64_t keep = vm & (drafts ? draft_window(a, it.b, t, pos0 - it.base) : ~0ull);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              s[i] = ((keep >> i) & 1ull) ? s[i] : -INFINITY;
              mx8[i & 7] = fmaxf(mx8[i & 7], s[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) mx8[i & 7] = fmaxf(mx8[i & 7], s[i]);
          }
          const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          const float m_tile = mx * scale_log2;
          if (m_tile > m_used + 8.0f) {                  // also taken when m_used is -inf
            alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_tile);
            m_used = m_tile;
          }
          const float z = kShift - ((m_used == -INFINITY) ? 0.f : m_used);
          float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f, sum3 = 0.f;
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float p0 = ex2(fmaf(s[i], scale_log2, z));
            const float p1 = ex2(fmaf(s[i + 1], scale_log2, z));
            const float p2 = ex2(fmaf(s[i + 2], scale_log2, z));
            const float p3 = ex2(fmaf(s[i + 3], scale_log2, z));
            pk[i / 2] = pack_16<F16>(p0, p1);
            pk[i / 2 + 1] = pack_16<F16>(p2, p3);
            add2(sum0, sum1, p0, p1);
            add2(sum2, sum3, p2, p3);
          }
          l = l * alpha + ((sum0 + sum1) + (sum2 + sum3));
        }
        if (n > 0) {
          // the previous value product has landed: O may be rescaled, and the arrival below is
          // for phase n
          ok = warp_all(tc::mbar_wait(&c.o_ready, (n - 1) & 1, abort_flag, status));
          if (!ok) continue;
          tc::tc_fence_after();
        }
        if (live) {
          if (tile > ta && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t v[32];
              tc::tmem_ld32(tl + kColO + cc * 32, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tc::tmem_st32(tl + kColO + cc * 32, v);
            }
          }
          tc::tmem_st32(tl + kColS + (n % 2) * 64, pk);  // P over the S just read
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&c.p_full);
      }
      // ---- result, or partial result ----
      if (ok) ok = warp_all(tc::mbar_wait(&c.o_ready, (n - 1) & 1, abort_flag, status));
      softmax_sync();                                    // the flag is complete
      const int fixup = *(volatile int*)&c.flag[seg & 1];
      const bool whole = ta == 0 && tb == it.n_tiles;
      const size_t slot = 2 * (size_t)blockIdx.x + (ta == 0 ? 1 : 0);
      if (ok && live) {
        tc::tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t v[32];
          __syncwarp();
          tc::tmem_ld32(tl + kColO + cc * 32, v);
          if (r < it.rows && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[i + e]) * inv;
              if (fixup) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += nonfinite_drafts<F16>(a, it, t, cc * 32 + i + e);
              }
              *reinterpret_cast<uint4*>(a.out + grow * D + cc * 32 + i) =
                  make_uint4(pack_16<F16>(y[0], y[1]), pack_16<F16>(y[2], y[3]), pack_16<F16>(y[4], y[5]),
                             pack_16<F16>(y[6], y[7]));
            }
          } else if (r < it.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(part4(a, slot, D, cc * 8 + i, r)) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (r < it.rows) {
          if (whole) {
            if (a.lse)
              a.lse[grow] = l == 0.f ? -INFINITY : (m_used - kShift + log2f(l)) * 0.69314718055994531f;
          } else {
            *reinterpret_cast<float2*>(a.part_ml + (slot * RT + r) * 2) = make_float2(m_used, l);
          }
        }
        __syncwarp();
        tc::tc_fence_before();
      }
      if (!whole) {
        // ---- arrival; the last CTA joins the parts ----
        if (tid == 0) a.part_flag[slot] = fixup;
        softmax_sync();
        const Parts<false, RT> parts(w, it);
        if (tid == 0) c.last = arrive_part(a.arrived + parts.c1, parts.n);
        softmax_sync();
        if (c.last) join_rows<D, F16>(a, it, parts, tid, ok);
      }
      softmax_sync();
      if (tid == 0) c.flag[seg & 1] = 0;                 // next used two segments on, behind barriers
      x = xe;
      if (x < x1) w.next(a, it);
    }
  }

  // ---------------- teardown ----------------
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int j = max(0, k_issued - NS); j < k_issued; ++j) tc::mbar_wait_timed(&c.k_full[j % NS], (j / NS) & 1);
    for (int j = max(0, v_issued - NS); j < v_issued; ++j) tc::mbar_wait_timed(&c.v_full[j % NS], (j / NS) & 1);
    wait_prepared();                             // in every CTA: this kernel's end is that one's, too
    if (c.status) atomicOr(a.dev_status, c.status);
  }
  if (warp == 1) {
    if (lane == 0 && mma_issued) {
      tc::umma_commit(&c.done);
      tc::mbar_wait_timed(&c.done, 0);
    }
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool F16>
static cudaError_t attend_tc_t(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                               cudaStream_t st) {
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)s.n_pages * s.Hkv * s.page;
  const uint32_t box = s.page < kTileKeys ? s.page : kTileKeys;
  if (!make_tmap_bf16_2d(&mk, k, rows, D, 64, box) || !make_tmap_bf16_2d(&mv, v, rows, D, 64, box))
    return cudaErrorInvalidValue;
  auto kern = paged_attend_tc_kernel<D, F16>;
  constexpr size_t smem = smem_bytes<D>();
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_paged_prepare(a, st);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = beside(at, a.n_cta, kThreads, smem, st);
  return cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
}

cudaError_t launch_paged_attend_tc(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                                   cudaStream_t st) {
  const bool f16 = s.dtype == BSA_F16;
  if (s.d == 128) return f16 ? attend_tc_t<128, true>(s, a, k, v, st) : attend_tc_t<128, false>(s, a, k, v, st);
  return f16 ? attend_tc_t<64, true>(s, a, k, v, st) : attend_tc_t<64, false>(s, a, k, v, st);
}

}  // namespace bsa
