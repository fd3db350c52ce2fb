// Attention over a paged cache on tcgen05: trees and chains of drafted tokens, up to 256 query
// rows (heads of a KV group x tokens) per item.
//
//   O = sum softmax(scale q.k) v over the positions a token sees
//
// A key costs 4 d flops per row for the 4 d bytes of its K and V: from some 250 rows on the products
// bound the kernel, below that the HBM reads of the cache, and between them the exponentials (one
// per row and key, 16 a clock and SM) are never far behind. So every K and V tile is read once for up to
// 256 rows, and two independent chains of products and softmax share it. One CTA per SM, 384
// threads, all 512 columns of TMEM, walking its share of all key tiles (paged_work.cuh):
//   warps 0, 3  producers of K and of V (paged_feed.cuh), separate stages
//   warps 1, 2  one thread each issues the products of group 0 and of group 1: S_j = Q K_j^T into one of
//               two TMEM buffers, S of the group's next tile before the value product of this one,
//               and O += P_j V_j with P read from TMEM
//   warps 4-7, 8-11  softmax of groups 0 and 1, a thread per row: Q of the item into shared memory
//               (128-byte swizzle, as TMA would write it), then per tile S from TMEM, the mask where
//               the tile needs one, the online softmax (O rescaled in TMEM only when the maximum grew
//               by more than 2^8), P in 16 bits over the S just read; O / l or the partial result at the end
//               of a segment. Warps whose rows are all past the item's skip the arithmetic.
// Items of more than 128 rows: group 1 takes rows 128 and up, both groups every tile; the warps of the two
// groups that share a scheduler take turns at the exponentials (64 of them keep its unit busy for 512
// cycles; both groups at once, then both waiting for products: 340 us below, 303 with turns). Items of up to
// 128 rows: both groups take the same rows and every other tile, and at the end of a segment each adds
// up the two states for half the channels (a row sits in the same TMEM lane in both groups, so a warp
// reads the other group's output where it is).
// P is rounded to 16 bits, at most a relative 2^-8 (bf16) or 2^-11 (fp16) per weight, as the output is
// (its error against 64 bits, random values in bf16: 0.0021 relative rms, where rounding the exact output alone
// gives 0.0017); sums and maxima are fp32. For fp16, weights carry a factor 2^7: with the maximum up to 2^8
// stale they stay below 2^15, and weights down to 2^-31 of the largest still count.
// Measured: 8 users with 64 drafts (256 rows per KV head) over 32768 tokens, 300 us, 916 TFLOP/s, in a few dozen replays
// at 1965 MHz; from half a second on the 1000 W limit leaves 1545 MHz, 345 to 355 us. 24 users with 9 to 33 drafts, d = 64:
// 92 us (1965 MHz throughout). Of the 2070 cycles of a tile of 256 rows, its products take 1270 when nothing
// else runs (S of 64 columns is bound by the reads of Q from shared memory, 418 cycles for 256 of
// products) and its exponentials 1024. Tried: S of 128 keys at once (one buffer then, or two rewritten
// together, so that S cannot run ahead of the value products: 462 and 369 us), two threads per row (850 us:
// 96 registers each).
// Rows that are no keys, and non-finite values of drafted rows, are treated as in paged_attend.cu:
// the softmax warps mend the V tile in shared memory before they release P.
#include <math.h>

#include "paged_feed.cuh"

namespace bsa {

namespace {

constexpr int kThreads = 384;
constexpr int RT = 256;
constexpr int GR = 128;                         // rows of a group
constexpr int kMaskRing = 16;
constexpr uint32_t kTmemCols = 512;             // group g: O at 256 g, S buffers at 256 g + 128 and + 192
constexpr uint32_t kColS = 128;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQHalf = GR * 128;
  static constexpr uint32_t kQTile = kHalves * kQHalf;
  static constexpr uint32_t kHalf = kTileKeys * 128;
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr int NS = D == 128 ? 4 : 8;     // even: a stage's tiles are one group's where they take turns
  static constexpr size_t kQ = 0, kK = 2 * kQTile, kV = kK + NS * kTile, kCtrl = kV + NS * kTile;
};
constexpr int kMaxStages = 8;
static_assert(kMaskRing > kMaxStages, "the producer is at most a ring ahead of the softmax");

struct Group {                                  // barriers of one group
  uint64_t q_full;
  uint64_t s_full[2];
  uint64_t p_full, o_ready, done;
};
struct __align__(16) Ctrl {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  Group g[2];
  unsigned long long vmask[kMaskRing];          // by tile: rows that are keys
  uint32_t tmem;
  int abort_flag;
  int32_t status;
  int flag[2][2];                               // [group][segment parity]: non-finite drafts taken out
  int last[2];                                  // [group]: this CTA joins the item's parts
  float2 ml[2][GR];                             // [group]: maxima and sums of shared segments
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
// x = x f + z, twice
__device__ __forceinline__ void fma2(float& x0, float& x1, float f, float z) {
  asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %2};\n\tmov.b64 rc, {%3, %3};\n\t"
      "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(z));
}
// the four softmax warps of a group; both groups
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ void both_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }
// Turns at the exponentials: two warps, one of each group, that share a scheduler.
__device__ __forceinline__ void turn_wait(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void turn_pass(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

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

// Of a segment's tiles (the CTA's n-th and up) group g takes the one at this place and, where the groups take turns,
// every other one after it. At or past the segment's end: the group has no tile there, and its Q is neither
// brought in nor waited for. (Were q_full counted there too, the softmax warps, held back by the
// other group alone, could complete it twice before this group's issuer looks once, which then never sees it.)
__device__ __forceinline__ int first_tile(bool share, int n, int g) { return share ? (n ^ g) & 1 : 0; }

// What the state of a row (maximum m, sum l) counts in a join with the maximum mx. An empty state has no weights,
// l = 0, and counts nothing. Where every score was NaN, m is still -inf (maxima pass NaN by) but l is NaN, which
// the result has to be, too.
__device__ __forceinline__ float state_weight(float m, float l, float mx) {
  return l == 0.f ? 0.f : (l != l ? l : ex2(m - mx));
}

// Parts lie transposed, [D / 4][RT] of four floats: a warp's rows are then neighbours both when a
// part is written (a thread per row) and when parts are joined.
__device__ __forceinline__ float4* part4(float* part_o, size_t slot, int D, int d4, int r) {
  return reinterpret_cast<float4*>(part_o) + (slot * (D / 4) + d4) * RT + r;
}
// Joins the parts of the rows [r0, r0 + rows) of an item, channels 4 d0 .. 4 d1, one group: 128 / R
// threads per row, R the rows rounded up to whole warps, each a run of channels; four quads of channels of
// three parts are read at once. (One user's eight drafts 20.8 -> 18.8 us against eight quads of two parts, of which
// a short run has half; four parts take registers that the main loop then spills.)
template <int D, bool F16>
__device__ __noinline__ void join_rows(const PagedArgs& a, const Item& it, const Parts<false, RT>& parts, int r0,
                                       int rows, int d0, int d1, int flag_at, int tid, bool ok) {
  constexpr float kShift = F16 ? 7.f : 0.f;
  constexpr int kU = 4, kP = 3;
  // (copies: behind the ordered reads below, what the references name would be read again each time)
  float* const part_o = a.part_o;
  const float2* const part_ml = reinterpret_cast<const float2*>(a.part_ml);
  const int32_t* const part_flag = a.part_flag;
  const Parts<false, RT> pt = parts;
  const int np = pt.n, R = (rows + 31) / 32 * 32;
  const int groups = 128 / R, dg = tid / R;                    // (R = 96: one group, 32 threads idle)
  if (dg >= groups || tid % R >= rows) return;
  const int r = r0 + tid % R;
  const int per = (d1 - d0 + groups - 1) / groups;
  const int da = d0 + dg * per, db = min(da + per, d1);
  auto ml_of = [&](int i) { return part_ml + pt.slot(i) * RT + r; };
  float mx = -INFINITY, ls = 0.f;
  int flag = 0;
#pragma unroll 4
  for (int i = 0; i < np; ++i) {
    mx = fmaxf(mx, read_l2(ml_of(i)).x);
    flag |= read_l2(part_flag + 2 * pt.slot(i) + flag_at);
  }
  int head, t;
  row_of<false>(a, it, r, head, t);
  const size_t row = ((size_t)it.b * a.Hq + head) * a.g.T + t;
  uint16_t* const out = a.out + row * D;
  for (int dc = da; dc < db; dc += kU) {
    float4 acc[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    ls = 0.f;
    for (int i = 0; i < np; i += kP) {
      float2 ml[kP];
      float4 v[kP][kU];
#pragma unroll
      for (int k = 0; k < kP; ++k) {
        const size_t at = pt.slot(min(i + k, np - 1));         // (past the last: a weight of 0 below)
        ml[k] = read_l2(part_ml + at * RT + r);
#pragma unroll
        for (int u = 0; u < kU; ++u) v[k][u] = read_l2(part4(part_o, at, D, min(dc + u, db - 1), r));
      }
#pragma unroll
      for (int k = 0; k < kP; ++k) {
        if (i + k >= np || ml[k].y == 0.f) continue;           // (must not meet what an empty part holds)
        const float f = state_weight(ml[k].x, ml[k].y, mx);
        ls += ml[k].y * f;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          acc[u].x = fmaf(v[k][u].x, f, acc[u].x);
          acc[u].y = fmaf(v[k][u].y, f, acc[u].y);
          acc[u].z = fmaf(v[k][u].z, f, acc[u].z);
          acc[u].w = fmaf(v[k][u].w, f, acc[u].w);
        }
      }
    }
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    // (runs are even: 16 bytes a store)
#pragma unroll
    for (int u = 0; u < kU; u += 2) {
      if (dc + u >= db) break;
      if (ok)
        *reinterpret_cast<uint4*>(out + 4 * (dc + u)) =
            make_uint4(pack_16<F16>(acc[u].x * inv, acc[u].y * inv), pack_16<F16>(acc[u].z * inv, acc[u].w * inv),
                       pack_16<F16>(acc[u + 1].x * inv, acc[u + 1].y * inv),
                       pack_16<F16>(acc[u + 1].z * inv, acc[u + 1].w * inv));
    }
  }
  if (flag && ok) store_nonfinite<F16>(a, it, t, row, 4 * da, 4 * db);
  if (ok && da == 0 && a.lse) a.lse[row] = ls == 0.f ? -INFINITY : (mx - kShift + log2f(ls)) * 0.69314718055994531f;
}

}  // namespace

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_tc_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
    const __grid_constant__ PagedArgs a) {
  using C = Cfg<D>;
  constexpr int NS = C::NS;
  constexpr float kShift = F16 ? 7.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl& c = *reinterpret_cast<Ctrl*>(sm + C::kCtrl);
  const uint32_t sQ = tc::smem_u32(sm + C::kQ), sK = tc::smem_u32(sm + C::kK), sV = tc::smem_u32(sm + C::kV);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&c.k_full[s], 1);
      tc::mbar_init(&c.v_full[s], 1);
      tc::mbar_init(&c.k_empty[s], 2);          // both issuers, or twice the one whose tile it was
      tc::mbar_init(&c.v_empty[s], 2);
    }
    for (int g = 0; g < 2; ++g) {
      tc::mbar_init(&c.g[g].q_full, 4);
      // the issuing thread arrives itself, too: what it saw (the tile's mask) is then visible to
      // the softmax warps
      tc::mbar_init(&c.g[g].s_full[0], 2);
      tc::mbar_init(&c.g[g].s_full[1], 2);
      tc::mbar_init(&c.g[g].p_full, 4);
      tc::mbar_init(&c.g[g].o_ready, 1);
      tc::mbar_init(&c.g[g].done, 1);
      c.flag[g][0] = c.flag[g][1] = 0;
    }
    c.abort_flag = 0;
    c.status = 0;
    tc::fence_mbar_init();
  }
  if (warp == 3) {
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
  int issued = 0;
  bool mma_issued = false;

  if (warp == 0 || warp == 3) {
    // ---------------- producers: K, V ----------------
    const bool is_k = warp == 0;
    const Feed<D> f{is_k ? &tmk : &tmv, sm + (is_k ? C::kK : C::kV), C::kTile, is_k ? c.k_full : c.v_full,
                    is_k ? c.k_empty : c.v_empty, is_k ? c.vmask : nullptr};
    issued = feed_share<false, RT, D, NS, kMaskRing>(a, w, x0, x1, f, abort_flag, status);
  } else if (warp <= 2) {
    // ---------------- MMA issuers ----------------
    // The whole warp walks, waits and computes descriptors, one elected lane issues: with the products
    // inside a branch of one lane their operands would have to be moved to uniform registers one by one.
    constexpr uint32_t idS = F16 ? tc::idesc_f16_f32(128, 64, false, false) : tc::idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idPV = F16 ? tc::idesc_f16_f32(128, D, false, true) : tc::idesc_bf16_f32(128, D, false, true);
    const int g = warp - 1;
    Group& b = c.g[g];
    const uint32_t tg = tmem + g * 256;
    const uint64_t descQ = tc::sdesc_sw128(sQ + g * C::kQTile, 16, 1024);
    const uint64_t descK = tc::sdesc_sw128(sK, 16, 1024), descV = tc::sdesc_sw128(sV, C::kHalf, 1024);
    int n = 0, nq = 0, js = 0, jv = 0;           // tiles of the CTA; Qs and products of this group
    bool ok = true;
    for (long long x = x0; ok && x < x1;) {
      const long long xe = min(x1, it.first + it.units());
      int ta, tb;
      it.tiles_of(x, xe, ta, tb);
      const int L = tb - ta;
      const bool share = it.rows <= GR;          // the groups take the tiles in turn
      const int step = share ? 2 : 1, i0 = first_tile(share, n, g);
      int si = i0;                               // the group's next tile of the segment to get its S
      auto next_s = [&]() {
        if (si >= L) return;
        const int s = (n + si) % NS;
        ok = tc::mbar_wait(&c.k_full[s], ((n + si) / NS) & 1, abort_flag, status);
        // S overwrites the buffer whose P the value product of two tiles ago read. (For the first of
        // a segment every product has landed, as Q's arrival says; the parity of two ago would
        // wait for the next one.)
        if (ok && js >= 2 && si != i0) ok = tc::mbar_wait(&b.o_ready, js & 1, abort_flag, status);
        ok = warp_all(ok);
        if (!ok) return;
        tc::tc_fence_after();
        const uint32_t d = tg + kColS + (js % 2) * 64;
        const uint64_t kd = descK + (uint64_t)(s * (C::kTile >> 4));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::umma_bf16(d, descQ + (((kk >> 2) * C::kQHalf + (kk & 3) * 32) >> 4),
                          kd + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), idS, kk > 0);
          tc::mbar_arrive(&b.s_full[js % 2]);
          tc::umma_commit(&b.s_full[js % 2]);
          tc::umma_commit(&c.k_empty[s]);
          if (share) tc::umma_commit(&c.k_empty[s]);
        }
        __syncwarp();
        mma_issued = true;
        ++js;
        si += step;
      };
      if (i0 < L) {
        ok = warp_all(tc::mbar_wait(&b.q_full, nq & 1, abort_flag, status));
        ++nq;
        if (ok) next_s();
      }
      uint32_t add = 0;
      for (int i = i0; ok && i < L; i += step) {
        const int s = (n + i) % NS;
        next_s();
        if (!ok) break;
        ok = warp_all(tc::mbar_wait(&c.v_full[s], ((n + i) / NS) & 1, abort_flag, status) &&
                      tc::mbar_wait(&b.p_full, jv & 1, abort_flag, status));
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t pa = tg + kColS + (jv % 2) * 64;
        const uint64_t vd = descV + (uint64_t)(s * (C::kTile >> 4));
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::umma_bf16_ts(tg, pa + kk * 8, vd + kk * (2048 >> 4), idPV, kk > 0 ? 1u : add);
          tc::umma_commit(&b.o_ready);
          tc::umma_commit(&c.v_empty[s]);
          if (share) tc::umma_commit(&c.v_empty[s]);
        }
        __syncwarp();
        add = 1;
        ++jv;
      }
      n += L;
      x = xe;
      if (x < x1) w.next(a, it);
    }
    // what the elected lane has in flight completes before the teardown
    if (mma_issued) {
      if (tc::elect_one()) tc::umma_commit(&b.done);
      __syncwarp();
      if (lane == 0) tc::mbar_wait_timed(&b.done, 0);
    }
  } else if (warp >= 4) {
    // ---------------- softmax warps ----------------
    const int g = (warp - 4) / 4;
    Group& b = c.g[g];
    const int quarter = warp & 3;                        // TMEM lane quarter of this warp
    const int tid = (threadIdx.x - 128) % 128;           // thread of the group
    const int rt = quarter * 32 + lane;                  // row of the group's tile
    const uint32_t tl = tmem + g * 256 + ((uint32_t)(quarter * 32) << 16);
    const float scale_log2 = a.scale_log2;
    // This thread's row of an item: output row and token. r0, rows: the group's rows.
    struct Row {
      int r0, rows, t;
      bool ok;
      size_t row;
    };
    auto row_in = [&](const Item& i) {
      Row o;
      o.r0 = i.rows <= GR ? 0 : g * GR;
      o.rows = min(GR, i.rows - o.r0);
      o.ok = rt < o.rows;
      int head;
      row_of<false>(a, i, o.ok ? o.r0 + rt : 0, head, o.t);
      o.row = ((size_t)i.b * a.Hq + head) * a.g.T + o.t;
      return o;
    };
    // Q of an item: the copies start, and (later) have landed. No product that reads the previous Q is
    // left when they start.
    uint8_t* const qs = sm + C::kQ + g * C::kQTile + rt * 128;
    auto load_q = [&](const Row& o) {
      const uint4* qr = reinterpret_cast<const uint4*>(a.q + o.row * D);
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch) {
        uint8_t* dst = qs + (ch >> 3) * C::kQHalf + (((ch & 7) ^ (rt & 7)) << 4);
        if (o.ok) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(qr + ch) : "memory");
        else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
    };
    auto q_landed = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&b.q_full);
    };
    // Does the group have a tile in the segment that starts at place x of item i, the CTA's n-th tile?
    auto has_tile = [&](const Item& i, long long x, int n) {
      int ta, tb;
      i.tiles_of(x, min(x1, i.first + i.units()), ta, tb);
      return first_tile(i.rows <= GR, n, g) < tb - ta;
    };
    const int my_turn = 4 + 4 * g + quarter, other_turn = 4 + 4 * (1 - g) + quarter;
    if (g == 1) turn_pass(other_turn);
    int n = 0, seg = 0, j = 0;                           // j: tiles of this group
    bool ok = true;
    Row me{};
    if (x0 < x1) {
      me = row_in(it);
      if (has_tile(it, x0, 0)) {
        load_q(me);
        q_landed();
      }
    }
    for (long long x = x0; x < x1; ++seg) {
      const long long xe = min(x1, it.first + it.units());
      int ta, tb;
      it.tiles_of(x, xe, ta, tb);
      const bool share = it.rows <= GR;
      const int r0 = me.r0, rows = me.rows, t = me.t, r = r0 + rt;
      const bool row_ok = me.ok;
      const bool live = quarter * 32 < rows;             // the warp has rows
      const bool turns = !share;                         // both groups: every tile
      const size_t grow = me.row;
      float m_used = -INFINITY, l = 0.f;
      bool first = true;                                 // no tile of the group in this segment yet
      for (int tile = ta; tile < tb; ++tile, ++n) {
        if (share && (n & 1) != g) continue;
        if (ok) ok = warp_all(tc::mbar_wait(&b.s_full[j % 2], (j / 2) & 1, abort_flag, status));
        if (!ok) {
          if (turns) {
            turn_wait(my_turn);
            turn_pass(other_turn);
          }
          continue;
        }
        tc::tc_fence_after();
        const int pos0 = tile * kTileKeys;
        const uint64_t vm = c.vmask[n % kMaskRing];
        const bool drafts = pos0 + kTileKeys > it.base;
        if (vm != ~0ull || (drafts && (a.mask || it.ql > 1))) {
          // mend the V tile: rows that are no keys become 0, non-finite drafted values are taken out
          // (by both groups, alike, where both use the tile)
          ok = warp_all(tc::mbar_wait(&c.v_full[n % NS], (n / NS) & 1, abort_flag, status));
          if (!ok) {
            if (turns) {
              turn_wait(my_turn);
              turn_pass(other_turn);
            }
            continue;
          }
          const int row = tid / 2;
          const bool key = (vm >> row) & 1;
          if (!key || (drafts && pos0 + row >= it.base)) {
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              const int ch = (tid & 1) * (D / 16) + i;
              uint4* p = reinterpret_cast<uint4*>(sm + C::kV + (n % NS) * C::kTile + (ch >> 3) * C::kHalf + row * 128 +
                                                  (((ch & 7) ^ (row & 7)) << 4));
              uint4 v = make_uint4(0, 0, 0, 0);
              if (key) {
                v = *p;
                if (clear_nonfinite<F16>(v.x) | clear_nonfinite<F16>(v.y) | clear_nonfinite<F16>(v.z) |
                    clear_nonfinite<F16>(v.w)) {
                  // before the value goes: who finds it gone finds the flags set
                  atomicOr(&c.flag[0][seg & 1], 1);
                  atomicOr(&c.flag[1][seg & 1], 1);
                  __threadfence_block();
                }
              }
              *p = v;
            }
          }
          tc::fence_proxy_async_smem();
        }
        float alpha = 1.f;
        uint32_t pk[32];
        if (live) {
          float s[64];
          {
            uint32_t v[64];
            tc::tmem_ld64(tl + kColS + (j % 2) * 64, v);
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(v[i]);
          }
          if (vm != ~0ull || drafts) {
            const uint64_t keep = vm & (drafts ? draft_window(a, it.b, t, pos0 - it.base) : ~0ull);
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = ((keep >> i) & 1ull) ? s[i] : -INFINITY;
          }
          float mx4[4];                                  // (three-operand maxima)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx4[u] = fmaxf(s[u], s[u + 4]);
#pragma unroll
          for (int i = 8; i < 64; i += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx4[u] = fmaxf(fmaxf(mx4[u], s[i + u]), s[i + u + 4]);
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const float m_tile = mx * scale_log2;
          if (m_tile > m_used + 8.0f) {                  // also taken when m_used is -inf
            alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_tile);
            m_used = m_tile;
          }
          float z = kShift - ((m_used == -INFINITY) ? 0.f : m_used);
          if (turns) {
            turn_wait(my_turn);
            asm volatile("" : "+f"(z));
          }
          float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f, sum3 = 0.f;
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            fma2(s[i], s[i + 1], scale_log2, z);
            fma2(s[i + 2], s[i + 3], scale_log2, z);
            const float p0 = ex2(s[i]), p1 = ex2(s[i + 1]), p2 = ex2(s[i + 2]), p3 = ex2(s[i + 3]);
            pk[i / 2] = pack_16<F16>(p0, p1);
            pk[i / 2 + 1] = pack_16<F16>(p2, p3);
            add2(sum0, sum1, p0, p1);
            add2(sum2, sum3, p2, p3);
          }
          l = l * alpha + ((sum0 + sum1) + (sum2 + sum3));
          if (turns) turn_pass(other_turn);
        } else if (turns) {
          turn_wait(my_turn);
          turn_pass(other_turn);
        }
        if (j > 0) {
          // the previous value product has landed: O may be rescaled, and the arrival below is
          // for phase j
          ok = warp_all(tc::mbar_wait(&b.o_ready, (j - 1) & 1, abort_flag, status));
          if (!ok) continue;
          tc::tc_fence_after();
        }
        if (live) {
          if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t v[32];
              tc::tmem_ld32(tl + cc * 32, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tc::tmem_st32(tl + cc * 32, v);
            }
          }
          tc::tmem_st32(tl + kColS + (j % 2) * 64, pk);  // P over the S just read
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&b.p_full);
        first = false;
        ++j;
      }
      // ---- result, or partial result ----
      if (ok && j > 0) ok = warp_all(tc::mbar_wait(&b.o_ready, (j - 1) & 1, abort_flag, status));
      tc::tc_fence_after();
      // the next item's Q is on its way while this one's result is written
      Item nx = it;
      bool q_next = false;
      if (xe < x1) {
        w.next(a, nx);
        me = row_in(nx);
        q_next = has_tile(nx, xe, n);
        if (q_next) load_q(me);
      }
      const bool whole = x == it.first && xe == it.first + it.units();
      const size_t slot = 2 * (size_t)blockIdx.x + (x == it.first ? 1 : 0);
      constexpr int kCh = D / 32;                        // pieces of 32 channels
      const int c0 = share ? g * (kCh / 2) : 0, c1 = share ? c0 + kCh / 2 : kCh;     // the group's
      auto tail_sync = [&]() {
        if (share) both_sync();
        else group_sync(g);
      };
      float f0 = 1.f, f1 = 0.f;                          // weights of the group's state and of the other's
      bool some0 = !first, some1 = false;                // ... and whether there is one (else O holds anything)
      if (share) c.ml[g][rt] = make_float2(m_used, l);
      tc::tc_fence_before();
      // the flags and states are there (and no group is more than a segment ahead, whose flags are the
      // other pair's)
      both_sync();
      tc::tc_fence_after();
      const uint32_t other = tl - g * 256 + (1 - g) * 256;
      if (share) {
        const float2 o = c.ml[1 - g][rt];
        const float m = fmaxf(m_used, o.x);
        f0 = state_weight(m_used, l, m);
        f1 = state_weight(o.x, o.y, m);
        some0 = l != 0.f;
        some1 = o.y != 0.f;
        l = l * f0 + o.y * f1;
        m_used = m;
      }
      const int fixup = *(volatile int*)&c.flag[g][seg & 1];
      if (ok && live) {
        const float inv = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
#pragma unroll 1
        for (int cc = c0; cc < c1; ++cc) {
          uint32_t v[32];
          __syncwarp();
          tc::tmem_ld32(tl + cc * 32, v);
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = some0 ? __uint_as_float(v[i]) * (f0 * inv) : 0.f;
          if (share) {
            tc::tmem_ld32(other + cc * 32, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (some1) y[i] = fmaf(__uint_as_float(v[i]), f1 * inv, y[i]);
          }
          if (row_ok && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(a.out + grow * D + cc * 32 + i) =
                  make_uint4(pack_16<F16>(y[i], y[i + 1]), pack_16<F16>(y[i + 2], y[i + 3]),
                             pack_16<F16>(y[i + 4], y[i + 5]), pack_16<F16>(y[i + 6], y[i + 7]));
          } else if (row_ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *part4(a.part_o, slot, D, cc * 8 + i, r) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
        if (fixup && whole && row_ok) store_nonfinite<F16>(a, it, t, grow, c0 * 32, c1 * 32);
        if (row_ok && c0 == 0) {
          if (whole) {
            if (a.lse) a.lse[grow] = l == 0.f ? -INFINITY : (m_used - kShift + log2f(l)) * 0.69314718055994531f;
          } else {
            *reinterpret_cast<float2*>(a.part_ml + (slot * RT + r) * 2) = make_float2(m_used, l);
          }
        }
        __syncwarp();
        tc::tc_fence_before();
      }
      if (q_next) q_landed();                            // S of its first tile may start
      if (!whole) {
        // ---- arrival; the last CTA joins the parts ----
        const int at = share ? 0 : g;
        const bool lead = tid == 0 && (!share || g == 0);
        if (lead) a.part_flag[2 * slot + at] = fixup;
        tail_sync();
        const Parts<false, RT> parts(w, it);
        if (lead) c.last[at] = arrive_part(a.arrived + 2 * parts.c1 + at, parts.n);
        tail_sync();
        if (c.last[at]) join_rows<D, F16>(a, it, parts, r0, rows, c0 * 8, c1 * 8, at, tid, ok);
      }
      tail_sync();                                       // O, the states and the flags may be written again
      if (tid == 0) c.flag[g][seg & 1] = 0;              // next used two segments on, behind barriers
      x = xe;
      it = nx;
    }
    if (g == 0) turn_wait(my_turn);
  }

  // ---------------- teardown ----------------
  tc::tc_fence_before();
  __syncthreads();
  if (issued > 0 && lane == 0) feed_drain<NS>(warp == 0 ? c.k_full : c.v_full, issued);
  if (threadIdx.x == 0) {
    wait_prepared();                             // in every CTA: this kernel's end is that one's, too
    if (c.status) atomicOr(a.dev_status, c.status);
  }
  if (warp == 3) {
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
  static_assert(smem <= 227 * 1024, "paged attend shared memory");
  static SmemSet set;
  cudaError_t e = allow_smem((const void*)kern, smem, set);
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
