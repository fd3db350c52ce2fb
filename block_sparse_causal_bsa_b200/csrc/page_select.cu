// Selection of cache pages for single query tokens by the K-min/K-max bound of their keys.
//
//   s(t, j) = max over the heads of a KV group of sum_c max(q_c kmin_jc, q_c kmax_jc)
//
// The lists that come out are compared for equality, so the scores that decide must not depend on
// the order of a sum: every product of two 16-bit floats is exact in fp64, and a sum of at most 128
// of them is exact or off by a few 2^-53, so its fp32 rounding is the definition's. Computing all
// scores that way is bound by the integer pipe that moves the bits into place (47 us for 16 users
// at 64k tokens, against 11 us for reading the bounds), so the scores are screened first:
//
// page_screen_kernel (scores not asked for): max(q a, q b) = max(q, 0) b + min(q, 0) a for a <= b, so
//   the score is a product of [min(q,0), max(q,0)] with a page's [kmin, kmax], 2 d long: warp-level MMAs
//   with fp32 sums, 16 rows (heads x tokens) against 8 pages, the bounds going from global memory
//   straight into the B fragments (the sum over channels may run in any order, so a lane takes the
//   channels of its 16-byte loads). One pass over the bounds for up to 16 rows; bound by HBM
//   (10 of its 14 us for 16 users at 64k tokens). Also the largest magnitude among a page's bounds, for the
//   margin.
// page_list_kernel: one CTA per (slot, KV head, token), a dozen barriers (11 us there). The m-th largest
//   score theta: of exact scores by radix selection over keys in shared memory, of the screen's to within
//   a few delta by one or two histograms. An MMA sum is off by at most delta = 2^-14 sum|q| max|k|: 273
//   additions and roundings of 2^-23 each, at least single precision's, come to 2^-14.9; the rest covers the roundings of
//   sum|q|, of theta +- 2 delta and of the exact score to fp32. At least m pages score
//   theta - delta or more, so pages below theta - 2 delta are out; pages above theta + 2 delta are in, since
//   what scores as high as they do lies above theta. Those between (a few) are computed in fp64, a
//   warp per page, and ranked by (fp32 rounding desc, index asc).
// page_score_kernel (scores asked for): every score in fp64. A 16-bit float becomes a double by
//   shifting its bits into place (the exponent is then too small by a constant, which q carries as a
//   factor), and the sign of q_c picks kmax or kmin: one DFMA and one select per channel and head.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "paged.h"

namespace bsa {

namespace {

constexpr int kScoreThreads = 256;
// inverse of score_key (0 and -0 share a key, and give 0)
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

constexpr uint32_t kNoPage = 0x7fffffffu;       // score of a page the table does not hold (a NaN)
constexpr uint32_t kBadScore = 0x7fc00000u;     // ... with a non-finite operand

// High word of the double x * 2^-896 (bf16) or x * 2^-1008 (fp16), low word 0, from the 16 bits of x
// in the high half of w (the low half is ignored): the sign stays, exponent and mantissa move
// down by the difference of the exponents' widths. Exact for zeros and subnormals too.
template <bool F16>
__device__ __forceinline__ uint32_t dbl_hi(uint32_t w) {
  constexpr int sh = F16 ? 6 : 3;
  constexpr uint32_t keep = 0x80000000u | (0x7fff0000u >> sh);
  return (uint32_t)((int32_t)w >> sh) & keep;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Any NaN or infinity among the eight 16-bit floats of a and b?
template <bool F16>
__device__ __forceinline__ bool nonfinite8(const uint2& a, const uint2& b) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  const uint32_t m = max_u16x2(max_u16x2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu),
                               max_u16x2(b.x & 0x7fff7fffu, b.y & 0x7fff7fffu));
  return (m & 0xffffu) >= e || (m >> 16) >= e;
}

template <bool F16>
__device__ __forceinline__ double q_scaled(uint16_t x) {
  // x * 2^896 or x * 2^1008 (the product with dbl_hi's value is then x * k); NaN if not finite
  const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  if ((x & e) == e) return __longlong_as_double(0x7ff8000000000000ll);
  const double d = __hiloint2double((int)dbl_hi<F16>((uint32_t)x << 16), 0);
  constexpr double up = F16 ? 0x1p1008 : 0x1p896;
  return d * up * up;
}

// a where the mask is 0, b where it is all ones
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t mask) { return (a & ~mask) | (b & mask); }

template <int D, int G>
struct ScoreCfg {
  static constexpr int LPP = D / 4;             // lanes per page, four channels each
  static constexpr int PPW = 32 / LPP;          // pages a warp reads side by side
  static constexpr int U = G >= 8 ? 1 : 8 / G;  // pages a lane has in hand
  static constexpr int NV = U * G;              // sums per lane
  static constexpr int kGroup = PPW * U;        // pages of a warp's step
  static constexpr int kStep = (kScoreThreads / 32) * kGroup;
};

template <int D, int G, bool F16>
__global__ void __launch_bounds__(kScoreThreads, G <= 4 ? 2 : 1) page_score_kernel(
    CacheGeom g, int G_real, int chunk, int n_chunks, const uint16_t* __restrict__ q,
    const uint16_t* __restrict__ bounds, float* __restrict__ scores, int32_t* dev_status) {
  using C = ScoreCfg<D, G>;
  constexpr int LPP = C::LPP, PPW = C::PPW, U = C::U, NV = C::NV;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) *dev_status = 0;   // the list kernel reports
  const int row = blockIdx.x / n_chunks;
  const int j0 = (blockIdx.x % n_chunks) * chunk;
  const int t = row % g.T, bh = row / g.T;
  const int h = bh % g.Hkv, b = bh / g.Hkv;
  int base, ql;
  query_span(g, b, base, ql);
  const int vis = t < ql ? (base + t) / g.page + 1 : 0;      // pages 0 .. own page
  const int j1 = min(j0 + chunk, g.max_pages);
  float* out = scores + (size_t)row * g.max_pages;
  for (int j = max(j0, vis) + threadIdx.x; j < j1; j += kScoreThreads) out[j] = -INFINITY;
  const int je = min(j1, vis);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int jw = j0 + warp * C::kGroup;
  if (jw >= je) return;                         // (the whole warp)

  const int sub = lane / LPP, ch = (lane % LPP) * 4;
  const int32_t* table = g.table + (size_t)b * g.max_pages;
  // page number of page jw + lane (lane < kGroup), -1 where there is none
  auto page_ids = [&](int jg) {
    int pg = lane < C::kGroup && jg + lane < je ? __ldg(table + jg + lane) : -1;
    return pg >= 0 && pg < g.n_pages ? pg : -1;
  };
  // bounds of this lane's channels of pages jw + u * PPW + sub
  auto load = [&](int ids, uint2 (&lo)[U], uint2 (&hi)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pg = __shfl_sync(0xffffffffu, ids, u * PPW + sub);
      lo[u] = hi[u] = make_uint2(0, 0);
      if (pg >= 0) {
        const uint2* bp = reinterpret_cast<const uint2*>(bounds + (((size_t)pg * g.Hkv + h) * 2) * D + ch);
        lo[u] = __ldg(bp);
        hi[u] = __ldg(bp + D / 4);
      }
    }
  };
  uint2 lo[U], hi[U];
  int ids = page_ids(jw);
  load(ids, lo, hi);
  int ids_next = page_ids(jw + C::kStep);

  double qd[G][4];
  uint32_t neg[G][4];                           // all ones where q < 0: kmin is picked
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const uint16_t* qr = q + ((((size_t)b * g.Hkv + h) * G_real + min(i, G_real - 1)) * g.T + t) * D + ch;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(qr));
    const uint16_t x[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      qd[i][c] = q_scaled<F16>(x[c]);
      neg[i][c] = (x[c] & 0x8000u) ? 0xffffffffu : 0u;
    }
  }
  for (; jw < je; jw += C::kStep) {
    // the next step's bounds and the one after's page numbers are on their way meanwhile
    uint2 lo_n[U], hi_n[U];
    load(ids_next, lo_n, hi_n);
    const int ids_next2 = page_ids(jw + 2 * C::kStep);
    double s[NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kl[4] = {dbl_hi<F16>(lo[u].x << 16), dbl_hi<F16>(lo[u].x), dbl_hi<F16>(lo[u].y << 16),
                              dbl_hi<F16>(lo[u].y)};
      const uint32_t kh[4] = {dbl_hi<F16>(hi[u].x << 16), dbl_hi<F16>(hi[u].x), dbl_hi<F16>(hi[u].y << 16),
                              dbl_hi<F16>(hi[u].y)};
      const double z = nonfinite8<F16>(lo[u], hi[u]) ? __longlong_as_double(0x7ff8000000000000ll) : 0.0;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        double acc = z;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc = fma(qd[i][c], __hiloint2double((int)pick(kh[c], kl[c], neg[i][c]), 0), acc);
        s[u * G + i] = acc;
      }
    }
    // sums over the LPP lanes, halving the values: after the step with distance o, a lane keeps
    // the half that bit o of its number names
    int n = NV;
    int v0 = 0;                                 // value number of this lane's s[0]
#pragma unroll
    for (int o = LPP / 2; o > 0; o >>= 1) {
      if (n > 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
          if (i < n / 2) {
            const double give = up ? s[i] : s[i + n / 2];
            const double keep = up ? s[i + n / 2] : s[i];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        n /= 2;
        if (up) v0 += n;
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
      }
    }
    // s[0 .. n) are the sums of values v0 ..: the maximum over the G heads of a page. NaN stays.
    float r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = i < n ? (float)s[i] : 0.f;
    auto maxn = [](float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); };
    constexpr int kSteps = LPP == 32 ? 5 : 4;
    constexpr int kLeft = NV >> kSteps ? NV >> kSteps : 1;     // sums per lane now
    if (kLeft >= G) {
#pragma unroll
      for (int p = 0; p < kLeft / G; ++p) {
        float m = r[p * G];
#pragma unroll
        for (int i = 1; i < G; ++i) m = maxn(m, r[p * G + i]);
        r[p] = m;
      }
    } else {
#pragma unroll
      for (int i = 1; i < kLeft; ++i) r[0] = maxn(r[0], r[i]);
      // the other heads of the page sit on the lanes whose value number differs below G: those are
      // the last halvings, distances kDist, 2 kDist, ...
      constexpr int kHalvings = (NV >= 32 ? 5 : NV >= 16 ? 4 : NV >= 8 ? 3 : NV >= 4 ? 2 : NV >= 2 ? 1 : 0);
      constexpr int kUsed = kHalvings < kSteps ? kHalvings : kSteps;
      constexpr int kDist = (LPP >> kUsed);                   // distance of the last halving
      constexpr int kHeads = G / kLeft;                       // lanes that share a page
#pragma unroll
      for (int x = 1; x < kHeads; x <<= 1) r[0] = maxn(r[0], __shfl_xor_sync(0xffffffffu, r[0], kDist * x));
    }
    constexpr int kPages = kLeft >= G ? kLeft / G : 1;
#pragma unroll
    for (int p = 0; p < kPages; ++p) {
      const int u = v0 / G + p;
      const int j = jw + u * PPW + sub;
      const bool held = __shfl_sync(0xffffffffu, ids, u * PPW + sub) >= 0;
      if (j < je) out[j] = held ? (r[p] != r[p] ? __uint_as_float(kBadScore) : r[p]) : __uint_as_float(kNoPage);
    }
    ids = ids_next;
    ids_next = ids_next2;
#pragma unroll
    for (int u = 0; u < U; ++u) { lo[u] = lo_n[u]; hi[u] = hi_n[u]; }
  }
}

// ---------------------------------------------------------------------------
// screen

// c += a (16x16, row) * b (16x8, col)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The halves of a packed pair that are below zero (neg) or not, the others 0.
__device__ __forceinline__ uint32_t keep_sign(uint32_t w, bool neg) {
  const uint32_t lo = (w & 0x8000u) ? 0xffffu : 0u, hi = (w & 0x80000000u) ? 0xffff0000u : 0u;
  return neg ? w & (lo | hi) : w & ~(lo | hi);
}

// GP: heads of a group, rounded up to a power of two; rows = 16 / GP tokens x GP heads.
template <int D, int GP, bool F16>
__global__ void __launch_bounds__(kScoreThreads, 2) page_screen_kernel(
    CacheGeom g, int G, int chunk, int n_chunks, const uint16_t* __restrict__ q,
    const uint16_t* __restrict__ bounds, float* __restrict__ scores, float* __restrict__ kmax_abs,
    int32_t* dev_status) {
  constexpr int TPT = 16 / GP;                  // tokens per row tile
  constexpr int NL = 2 * D / 32;                // 16-byte loads per lane and page; two k16 steps each
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) *dev_status = 0;   // the list kernel reports
  const int n_tt = (g.T + TPT - 1) / TPT;
  int x = blockIdx.x;
  const int ck = x % n_chunks;
  x /= n_chunks;
  const int t0 = (x % n_tt) * TPT, bh = x / n_tt;
  const int h = bh % g.Hkv, b = bh / g.Hkv;
  int base, ql;
  query_span(g, b, base, ql);
  if (t0 >= ql) return;
  const int t_last = min(t0 + TPT, ql) - 1;
  const int je = min((ck + 1) * chunk, (base + t_last) / g.page + 1);   // pages up to the last token's own
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int jw = ck * chunk + warp * 8;
  const int g8 = lane >> 2, tig = lane & 3;
  constexpr int kStep = (kScoreThreads / 32) * 8;
  const int32_t* table = g.table + (size_t)b * g.max_pages;
  auto page_of = [&](int j) {
    const int pg = j < je ? __ldg(table + j) : -1;
    return pg >= 0 && pg < g.n_pages ? pg : -1;
  };
  auto load = [&](int pg, uint4 (&v)[NL]) {
    const uint4* bp = reinterpret_cast<const uint4*>(bounds + ((size_t)max(pg, 0) * g.Hkv + h) * 2 * D) + tig;
#pragma unroll
    for (int l = 0; l < NL; ++l) v[l] = pg >= 0 ? __ldg(bp + 4 * l) : make_uint4(0, 0, 0, 0);
  };
  // B column n = page jw + lane / 4; the next step's bounds and the one after's page numbers are on
  // their way while a step is computed
  int pg = page_of(jw + g8), pg_next = page_of(jw + kStep + g8);

  // A: rows g8 and g8 + 8 of [min(q,0), max(q,0)], in fragments. Load l, lane tig of a page row: channels
  // 32 l + 8 tig + (0..7) of [kmin, kmax]; its words 0, 1 are the B fragment of one k16 step, words 2, 3 of
  // the next, and A takes the same channels. A warp builds the steps of its share of the loads.
  __shared__ uint4 af[2 * NL][32];
  for (int l = warp; l < NL / 2; l += kScoreThreads / 32) {
    uint4 w[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g8 + 8 * half;
      const int t = min(t0 + r / GP, ql - 1), head = min(r % GP, G - 1);
      w[half] = __ldg(reinterpret_cast<const uint4*>(q + ((((size_t)b * g.Hkv + h) * G + head) * g.T + t) * D) +
                      4 * l + tig);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {               // kmin part (q < 0), kmax part
      const int st = 2 * (l + s * (NL / 2));
      af[st][lane] = make_uint4(keep_sign(w[0].x, s == 0), keep_sign(w[1].x, s == 0), keep_sign(w[0].y, s == 0),
                                keep_sign(w[1].y, s == 0));
      af[st + 1][lane] = make_uint4(keep_sign(w[0].z, s == 0), keep_sign(w[1].z, s == 0), keep_sign(w[0].w, s == 0),
                                    keep_sign(w[1].w, s == 0));
    }
  }
  uint4 v[NL], v_next[NL];
  load(pg, v);
  __syncthreads();
  float* out = scores + ((size_t)bh * g.T + t0) * g.max_pages;
#pragma unroll 1
  for (; jw < je; jw += kStep) {
    const bool held = pg >= 0;
    load(pg_next, v_next);
    pg = pg_next;
    pg_next = page_of(jw + 2 * kStep + g8);
    float c[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[0][i] = c[1][i] = 0.f;
    uint32_t mx = 0;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const uint4 a0 = af[2 * l][lane], a1 = af[2 * l + 1][lane];
      mma16816<F16>(c[0], a0, v[l].x, v[l].y);
      mma16816<F16>(c[1], a1, v[l].z, v[l].w);
      mx = max_u16x2(mx, max_u16x2(max_u16x2(v[l].x & 0x7fff7fffu, v[l].y & 0x7fff7fffu),
                                   max_u16x2(v[l].z & 0x7fff7fffu, v[l].w & 0x7fff7fffu)));
    }
    // largest magnitude of the page's bounds, for its four lanes
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (tig == 0 && jw + g8 < je) {              // (every token tile writes the same)
      float m;
      if (F16) asm("cvt.f32.f16 %0, %1;" : "=f"(m) : "h"((uint16_t)mx));
      else m = __uint_as_float(mx << 16);
      // (a NaN that was converted may have any bits, those of kNoPage too)
      kmax_abs[(size_t)bh * g.max_pages + jw + g8] =
          __uint_as_float(!held ? kNoPage : m < INFINITY ? __float_as_uint(m) : kBadScore);
    }
    // rows g8 (r[0], r[1]) and g8 + 8 (r[2], r[3]) of pages jw + 2 tig (+1): maximum over the heads
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = c[0][i] + c[1][i];
    auto maxn = [](float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); };
#pragma unroll
    for (int o = 1; o < (GP < 8 ? GP : 8); o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = maxn(r[i], __shfl_xor_sync(0xffffffffu, r[i], 4 * o));
    if (GP == 16) {
      r[0] = maxn(r[0], r[2]);
      r[1] = maxn(r[1], r[3]);
    }
    if (g8 % (GP < 8 ? GP : 8) == 0) {
#pragma unroll
      for (int half = 0; half < (GP == 16 ? 1 : 2); ++half) {
        const int tl = (g8 + 8 * half) / GP;
        if (t0 + tl > t_last) continue;
        float* o = out + (size_t)tl * g.max_pages + jw + 2 * tig;
        if (jw + 2 * tig < je) o[0] = r[2 * half];
        if (jw + 2 * tig + 1 < je) o[1] = r[2 * half + 1];
      }
    }
#pragma unroll
    for (int l = 0; l < NL; ++l) v[l] = v_next[l];
  }
}

// ---------------------------------------------------------------------------

constexpr int kListThreads = 512;
constexpr int kBins = 2048;                     // of the screen's histogram, four per thread
constexpr int kListWarps = kListThreads / 32;
constexpr int kWindow = 256;                    // pages near the threshold that are ranked pairwise

struct __align__(16) ListSmem {
  unsigned hist[kBins];
  unsigned red[kListWarps], red2[kListWarps];
  float fred[kListWarps];
  unsigned digit, above;                        // the bin that holds the threshold, keys in bins above it
  int status;
  int n_win;                                    // pages near the threshold
  int win[kWindow];
  uint32_t wkey[kWindow];
  double qd[16 * 128];                          // the heads' queries, scaled
};

// What a threshold of the m-th largest of keys[0, n) (m < n) says: in are the keys with (key &
// mask) > thr, and of those equal the first `left` by index.
struct Cut {
  unsigned thr, mask;
  int left;
};

// Radix selection: digits of up to eight bits from the highest bit in which keys differ down; mn, mx
// the least and the largest key. All threads call it; keys are visible to all.
__device__ __noinline__ Cut radix_cut(const uint32_t* keys, int n, int m, unsigned mn, unsigned mx, ListSmem& s) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  Cut c{mx, 0xffffffffu, m};
  if (mn == mx) return c;
  int top = 32 - __clz(mn ^ mx);                // bits [0, top) differ
  c.mask = top == 32 ? 0u : ~((1u << top) - 1u);
  c.thr = mx & c.mask;
  while (top > 0) {
    const int sh = max(top - 8, 0), width = top - sh;
    if (tid < 256) s.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kListThreads) {
      const unsigned key = keys[i];
      if ((key & c.mask) == c.thr) atomicAdd(&s.hist[(key >> sh) & ((1u << width) - 1u)], 1u);
    }
    __syncthreads();
    // thread tid: keys in digits above d, a suffix sum from the top digit down
    const int d = 255 - tid;
    const unsigned mine = d >= 0 ? s.hist[d] : 0u;
    unsigned x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s.red[warp] = x;
    __syncthreads();
    unsigned above = x - mine;
    for (int i = 0; i < warp; ++i) above += s.red[i];
    if (above < (unsigned)c.left && above + mine >= (unsigned)c.left) { s.digit = d; s.above = above; }
    __syncthreads();
    c.thr |= s.digit << sh;
    c.mask |= ((1u << width) - 1u) << sh;
    c.left -= s.above;
    top = sh;
    if (s.hist[s.digit] == (unsigned)c.left) break;   // the whole digit is in: thr is a lower bound
    __syncthreads();
  }
  return c;
}

// s(t, j) in fp64, rounded to fp32, of one page: the whole warp. qd: the heads' scaled queries.
template <bool F16>
__device__ __noinline__ float exact_score(const uint16_t* bp, const double* qd, int G, int d) {
  const int lane = threadIdx.x % 32;
  float best = -INFINITY;
  bool nan = false;
  // lane: channels 4 lane .. (d = 128), or of d = 64 the lower 16 lanes
  const bool on = lane * 4 < d;
  const uint2 lo = on ? __ldg(reinterpret_cast<const uint2*>(bp) + lane) : make_uint2(0, 0);
  const uint2 hi = on ? __ldg(reinterpret_cast<const uint2*>(bp + d) + lane) : make_uint2(0, 0);
  const uint32_t kl[4] = {dbl_hi<F16>(lo.x << 16), dbl_hi<F16>(lo.x), dbl_hi<F16>(lo.y << 16), dbl_hi<F16>(lo.y)};
  const uint32_t kh[4] = {dbl_hi<F16>(hi.x << 16), dbl_hi<F16>(hi.x), dbl_hi<F16>(hi.y << 16), dbl_hi<F16>(hi.y)};
  for (int i0 = 0; i0 < G; i0 += 4) {            // four heads' sums at a time hide their latencies
    double sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] = 0.0;
      if (on) {
        const double* x = qd + min(i0 + i, G - 1) * d + lane * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sum[i] = fma(x[c], __hiloint2double((int)(__double2hiint(x[c]) < 0 ? kl[c] : kh[c]), 0), sum[i]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = (float)sum[i];
      nan |= f != f;
      best = fmaxf(best, f);
    }
  }
  return nan ? __uint_as_float(kBadScore) : best;
}

// SCREEN: scores are the screen's, kmax_abs the pages' largest magnitudes; else they are exact.
template <bool SCREEN, bool F16>
__global__ void __launch_bounds__(kListThreads) page_list_kernel(
    CacheGeom g, bsa_page_select_params p, int G, const uint16_t* __restrict__ q,
    const uint16_t* __restrict__ bounds, const float* __restrict__ scores, const float* __restrict__ kmax_abs,
    int32_t* __restrict__ kv_idx, int32_t* __restrict__ kv_cnt, int32_t* dev_status) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ ListSmem s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int row = blockIdx.x, t = row % g.T, bh = row / g.T, b = bh / g.Hkv, h = bh % g.Hkv;
  int base, ql;
  const bool fits = query_span(g, b, base, ql);
  const int vis = t < ql ? (base + t) / g.page + 1 : 0;
  const int cnt = min(vis, p.k);
  const int n = vis - p.n_first - p.n_last, m = p.k - p.n_first - p.n_last;    // candidates, slots
  const bool ranked = vis > p.k && m > 0;
  float q1 = 0.f;                               // the largest sum |q_c| over the heads
  if (tid == 0) {
    s.status = 0;
    s.n_win = 0;
  }
  for (int i = tid; SCREEN && i < kBins; i += kListThreads) s.hist[i] = 0;
  if (SCREEN && ranked) {
    // a warp per head: the scaled query, and the sum of magnitudes (0 stands in for what is not
    // finite: such a query makes every score NaN, which the screen shows)
    for (int i = warp; i < G; i += kListWarps) {
      const uint16_t* qr = q + (((size_t)bh * G + i) * g.T + t) * g.d;
      float sum = 0.f;
      for (int c = lane; c < g.d; c += 32) {
        const uint16_t w = __ldg(qr + c);
        s.qd[i * g.d + c] = q_scaled<F16>(w);
        float f;
        if (F16) asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(w));
        else f = bf16_to_f32(w);
        sum += fabsf(f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      q1 = fmaxf(q1, sum < INFINITY ? sum : INFINITY);
    }
    if (lane == 0) s.fred[warp] = q1;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t* out = kv_idx + (size_t)row * p.k;
  for (int i = cnt + tid; i < p.k; i += kListThreads) out[i] = -1;
  if (tid == 0) {
    kv_cnt[row] = cnt;
    if (!fits && t == 0) set_status(dev_status, BSA_DEV_BAD_INDEX);
  }
  if (vis <= p.k) {
    for (int i = tid; i < vis; i += kListThreads) out[i] = i;
    return;
  }
  for (int i = tid; i < p.n_first; i += kListThreads) out[i] = i;
  for (int i = tid; i < p.n_last; i += kListThreads) out[p.k - p.n_last + i] = vis - p.n_last + i;
  if (m == 0) return;

  // keys, their least and largest, what is not finite, and the largest magnitude of the bounds
  __syncthreads();
  const float* sc = scores + (size_t)row * g.max_pages + p.n_first;
  const float* ka = SCREEN ? kmax_abs + (size_t)bh * g.max_pages + p.n_first : nullptr;
  unsigned mn = 0xffffffffu, mx = 0;
  int st = 0;
  float kabs = 0.f;
#pragma unroll 4
  for (int i = tid; i < n; i += kListThreads) {
    const float v = __ldcg(sc + i);
    const uint32_t u = SCREEN ? __float_as_uint(__ldcg(ka + i)) : __float_as_uint(v);
    uint32_t key = score_key(v);
    if ((u & 0x7f800000u) == 0x7f800000u) {
      st |= u == kNoPage ? BSA_DEV_BAD_INDEX : BSA_DEV_BAD_SCORE;
      key = 0;                                  // ranks last
    } else if (SCREEN) {
      // (where an estimate is not finite, none is used: see the margin below)
      const bool over = !(fabsf(v) < INFINITY);
      kabs = fmaxf(kabs, over ? INFINITY : __uint_as_float(u));
      if (over) key = 1;
    }
    keys[i] = key;
    if (!SCREEN || key > 1) {                   // (bad pages take no part in the range of the screen's scores)
      mn = min(mn, key);
      mx = max(mx, key);
    }
  }
  if (st) atomicOr(&s.status, st);
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  q1 = 0.f;
  if (SCREEN) {
#pragma unroll
    for (int i = 0; i < kListWarps; ++i) q1 = fmaxf(q1, s.fred[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kabs = fmaxf(kabs, __shfl_xor_sync(0xffffffffu, kabs, o));
  }
  __syncthreads();                              // fred is read
  if (lane == 0) {
    s.red[warp] = mn;
    s.red2[warp] = mx;
    s.fred[warp] = kabs;
  }
  __syncthreads();
  mn = s.red[0];
  mx = s.red2[0];
#pragma unroll
  for (int i = 1; i < kListWarps; ++i) { mn = min(mn, s.red[i]); mx = max(mx, s.red2[i]); }
#pragma unroll
  for (int i = 0; i < kListWarps; ++i) kabs = fmaxf(kabs, s.fred[i]);
  __syncthreads();                              // red is read
  Cut c{0u, 0u, 0};
  if (!SCREEN) c = radix_cut(keys, n, m, mn, mx, s);

  if (SCREEN) {
    // Below 2^127 no sum of the screen overflows, in any head, and estimates are off by delta at most. Above (or with a
    // query that is not finite) they say nothing: every page that is not known to be bad is computed, and ranked with
    // those that are.
    const float span = q1 * kabs;
    const bool usable = span < 0x1p127f;
    // 2^-14 for the sums; what 16-bit subnormals could lose if an MMA flushed them
    const float delta = 0x1p-14f * span + (F16 ? 0x1p-13f : 0x1p-100f) * (q1 + g.d * kabs);
    // The threshold, to within a few delta: a histogram of equal ranges of the finite scores' keys. Where a bin is wider
    // (scores of both signs: their keys lie far apart) a second one of its keys; a bin of that is at most 2^10 keys,
    // 2^-13 of its scores, that is 2 delta. (One histogram over all keys, bad pages' among them, left windows of hundreds of
    // pages: selection at 128k tokens with one page missing 420 us, now 16; sixteen users at 64k with scores around zero
    // 37, now 25.)
    unsigned klo = mn, khi = mx, rank = (unsigned)m, finite = 0;
    float th_lo = 0.f, th_hi = 0.f;
    for (int level = 0; usable; ++level) {
      const int sh = max(0, 21 - __clz((khi - klo) | 1u));
#pragma unroll 4
      for (int i = tid; i < n; i += kListThreads) {
        const unsigned key = keys[i];
        if (key - klo <= khi - klo) atomicAdd(&s.hist[(key - klo) >> sh], 1u);
      }
      __syncthreads();
      // thread tid: the bins 4 d .. 4 d + 3 and the keys above them, from the top down
      const int d = kBins / 4 - 1 - tid;
      const uint4 h4 = *reinterpret_cast<const uint4*>(&s.hist[4 * d]);
      const unsigned mine = h4.x + h4.y + h4.z + h4.w;
      unsigned x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s.red[warp] = x;
      __syncthreads();
      const unsigned part = lane < kListWarps ? s.red[lane] : 0u;
      const unsigned above = x - mine + __reduce_add_sync(0xffffffffu, lane < warp ? part : 0u);
      const unsigned all = __reduce_add_sync(0xffffffffu, part);
      if (level == 0) finite = all;
      if (all < rank) break;                    // fewer finite scores than places
      if (above < rank && above + mine >= rank) {
        unsigned at = above, bin = 4 * d + 3;
        if (at + h4.w < rank) { at += h4.w; --bin;
          if (at + h4.z < rank) { at += h4.z; --bin;
            if (at + h4.y < rank) { at += h4.y; --bin; } } }
        s.digit = bin;
        s.above = at;
      }
      __syncthreads();
      klo += s.digit << sh;
      khi = min(khi, klo + ((1u << sh) - 1u));
      rank -= s.above;
      th_lo = key_score(klo);
      th_hi = key_score(khi);
      if (level || !(th_hi - th_lo > 8.f * delta)) break;
      *reinterpret_cast<uint4*>(&s.hist[4 * d]) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    const bool few = finite < (unsigned)m;
    const float lo = usable ? th_lo - 2.f * delta : -INFINITY, hi = usable ? th_hi + 2.f * delta : INFINITY;
    const unsigned sure = hi < INFINITY ? score_key(hi) : 0xfffffffeu;      // keys above it are in
    int in = 0;
    for (int i = tid; i < n; i += kListThreads) {
      const unsigned key = keys[i];
      in += key > sure;
      if (key <= sure && key != 0 && !(key_score(key) < lo)) {
        const int at = atomicAdd(&s.n_win, 1);
        if (at < kWindow) s.win[at] = i;
      }
    }
    in = __reduce_add_sync(0xffffffffu, in);
    if (lane == 0) s.red2[warp] = in;
    __syncthreads();
    in = 0;
#pragma unroll
    for (int i = 0; i < kListWarps; ++i) in += s.red2[i];
    const int nw = s.n_win, need = m - in;
    const int32_t* table = g.table + (size_t)b * g.max_pages + p.n_first;
    const uint16_t* bh_bounds = bounds + (size_t)h * 2 * g.d;
    const size_t page_stride = (size_t)g.Hkv * 2 * g.d;
    if (usable && few) {
      c = Cut{0u, 0xffffffffu, m - (int)finite};   // every page that is not bad, and the first bad ones
    } else if (usable && nw <= kWindow) {
      c = Cut{sure, 0xffffffffu, 0};
      if (nw > need) {
        // exact scores of the window, a warp per page, then ranks within it
        for (int w = warp; w < nw; w += kListWarps) {
          const float e = exact_score<F16>(bh_bounds + __ldg(table + s.win[w]) * page_stride, s.qd, G, g.d);
          if (lane == 0) {
            if (!(fabsf(e) < INFINITY)) atomicOr(&s.status, BSA_DEV_BAD_SCORE);
            s.wkey[w] = fabsf(e) < INFINITY ? score_key(e) : 0u;
          }
        }
        __syncthreads();
      }
      if (tid < nw) {
        const int i = s.win[tid];
        int better = 0;
        if (nw > need) {
          const uint32_t key = s.wkey[tid];
          for (int w = 0; w < nw; ++w) better += s.wkey[w] > key || (s.wkey[w] == key && s.win[w] < i);
        }
        if (better < need) keys[i] = 0xffffffffu;
      }
    } else {
      // a large window (copies of pages), or estimates that say nothing: exact keys, and another selection
      for (int i = warp; i < n; i += kListWarps) {
        const unsigned key = keys[i];
        unsigned exact = key > sure ? 0xffffffffu : 0u;
        if (key <= sure && key != 0 && !(key_score(key) < lo)) {
          const float e = exact_score<F16>(bh_bounds + __ldg(table + i) * page_stride, s.qd, G, g.d);
          if (fabsf(e) < INFINITY) exact = score_key(e);
          else if (lane == 0) atomicOr(&s.status, BSA_DEV_BAD_SCORE);
        }
        __syncwarp();
        if (lane == 0) keys[i] = exact;
      }
      __syncthreads();
      c = radix_cut(keys, n, m, 0u, 0xffffffffu, s);
    }
    __syncthreads();
  }
  if (tid == 0 && s.status) set_status(dev_status, s.status);
  // in: (key & mask) > thr, or equal and among the first `left` of those. A warp takes a
  // contiguous range; counts first, then the places.
  __syncthreads();
  const int per = (n + kListWarps - 1) / kListWarps;
  const int i0 = min(warp * per, n), i1 = min(i0 + per, n);
  unsigned gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const unsigned k = keys[i] & c.mask;
    gt += k > c.thr;
    eq += k == c.thr;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) { s.red[warp] = gt; s.red2[warp] = eq; }
  __syncthreads();
  unsigned at_gt = 0, at_eq = 0;
  for (int i = 0; i < warp; ++i) { at_gt += s.red[i]; at_eq += s.red2[i]; }
  const unsigned below = (1u << lane) - 1u;
  for (int ib = i0; ib < i1; ib += 32) {
    const int i = ib + lane;
    const unsigned k = i < i1 ? keys[i] & c.mask : 0u;
    const bool is_gt = i < i1 && k > c.thr, is_eq = i < i1 && k == c.thr;
    const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const unsigned eq_rank = at_eq + __popc(be & below);
    if (is_gt || (is_eq && eq_rank < (unsigned)c.left))
      out[p.n_first + at_gt + __popc(bg & below) + min(eq_rank, (unsigned)c.left)] = p.n_first + i;
    at_gt += __popc(bg);
    at_eq += __popc(be);
  }
}

// Pages per CTA of the scoring kernels, in whole steps of their warps: equal chunks of the table, as many as
// run at once (two CTAs per SM) one, two, three or four times over, whichever is shortest; a CTA's start counts
// as two steps. (Chunks of all pages / 296, 384 CTAs of which 88 ran in a second wave: 16 users at 64k tokens
// 26.0 us for the selection, now 24.8.)
int pages_per_cta(long long rows, int max_pages, int step) {
  const long long ctas = 2ll * sm_count();
  long long best = 0;
  int per = 0;
  for (int k = 1; k <= 4; ++k) {
    const int chunks = (int)std::max(1ll, k * ctas / rows);
    const int p = ((max_pages + chunks - 1) / chunks + step - 1) / step * step;
    const long long n = (max_pages + p - 1) / p, time = (rows * n + ctas - 1) / ctas * (p + 2 * step);
    if (per == 0 || time < best) {
      best = time;
      per = p;
    }
  }
  return per;
}

template <int D, int G>
cudaError_t score_g(const CacheGeom& g, bool f16, int G_real, const void* q, const void* bounds, float* scores,
                    int32_t* dev_status, cudaStream_t st) {
  const long long rows = (long long)g.slots * g.Hkv * g.T;
  const int chunk = pages_per_cta(rows, g.max_pages, ScoreCfg<D, G>::kStep);
  const int n_chunks = (g.max_pages + chunk - 1) / chunk;
  auto kern = f16 ? page_score_kernel<D, G, true> : page_score_kernel<D, G, false>;
  kern<<<(unsigned)(rows * n_chunks), kScoreThreads, 0, st>>>(g, G_real, chunk, n_chunks, (const uint16_t*)q,
                                                            (const uint16_t*)bounds, scores, dev_status);
  return cudaGetLastError();
}

template <int D, int GP>
cudaError_t screen_g(const CacheGeom& g, bool f16, int G, const void* q, const void* bounds, float* scores,
                     float* kmax_abs, int32_t* dev_status, cudaStream_t st) {
  const long long rows = (long long)g.slots * g.Hkv * ((g.T + 16 / GP - 1) / (16 / GP));
  const int chunk = pages_per_cta(rows, g.max_pages, kScoreThreads / 32 * 8);
  const int n_chunks = (g.max_pages + chunk - 1) / chunk;
  auto kern = f16 ? page_screen_kernel<D, GP, true> : page_screen_kernel<D, GP, false>;
  kern<<<(unsigned)(rows * n_chunks), kScoreThreads, 0, st>>>(g, G, chunk, n_chunks, (const uint16_t*)q,
                                                            (const uint16_t*)bounds, scores, kmax_abs, dev_status);
  return cudaGetLastError();
}

// kmax_abs null: exact scores; else the screen
template <int D, int GP>
cudaError_t any_g(const CacheGeom& g, bool f16, int G, const void* q, const void* bounds, float* scores,
                  float* kmax_abs, int32_t* dev_status, cudaStream_t st) {
  return kmax_abs ? screen_g<D, GP>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st)
                  : score_g<D, GP>(g, f16, G, q, bounds, scores, dev_status, st);
}

template <int D>
cudaError_t any_d(const CacheGeom& g, bool f16, int G, const void* q, const void* bounds, float* scores,
                  float* kmax_abs, int32_t* dev_status, cudaStream_t st) {
  if (G == 1) return any_g<D, 1>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
  if (G == 2) return any_g<D, 2>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
  if (G <= 4) return any_g<D, 4>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
  if (G <= 8) return any_g<D, 8>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
  return any_g<D, 16>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
}

}  // namespace

cudaError_t launch_select_pages(const bsa_cache_shape& s, const CacheGeom& g, const bsa_page_select_params& p,
                                int Hq, const void* q, const void* bounds, float* scores, float* kmax_abs,
                                int32_t* kv_idx, int32_t* kv_cnt, int32_t* dev_status, cudaStream_t st) {
  const int G = Hq / g.Hkv;
  const bool f16 = s.dtype == BSA_F16;
  cudaError_t e = s.d == 128 ? any_d<128>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st)
                             : any_d<64>(g, f16, G, q, bounds, scores, kmax_abs, dev_status, st);
  if (e != cudaSuccess) return e;
  auto kern = kmax_abs ? (f16 ? page_list_kernel<true, true> : page_list_kernel<true, false>)
                       : (f16 ? page_list_kernel<false, true> : page_list_kernel<false, false>);
  const size_t smem = (size_t)g.max_pages * 4;
  static SmemSet sets[4];                       // (the most that any table needs)
  e = allow_smem((const void*)kern, kMaxTablePages * 4, sets[(kmax_abs ? 2 : 0) + f16]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)g.slots * g.Hkv * g.T));
  cfg.blockDim = dim3(kListThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, g, p, G, (const uint16_t*)q, (const uint16_t*)bounds, (const float*)scores,
                            (const float*)kmax_abs, kv_idx, kv_cnt, dev_status);
}

}  // namespace bsa
