// Selection of cache pages for single query tokens by the K-min/K-max bound of their keys.
//
//   s(t, j) = max over the heads of a KV group of sum_c max(q_c kmin_jc, q_c kmax_jc)
//
// The list that comes out is compared for equality, so the scores must not depend on the order of
// a sum: every product of two 16-bit floats is exact in fp64, and a sum of at most 128 of them is
// exact or off by a few 2^-53, so its fp32 rounding is the definition's. What that costs: one DFMA
// per channel and head. A 16-bit float becomes a double by shifting its bits into place (the
// exponent is then too small by a constant, which q carries as a factor), and q_c >= 0 picks kmax,
// q_c < 0 picks kmin, a choice per channel and head of the high word alone.
//
// page_score_kernel: one pass over the bounds (4 d bytes per page and head, the bound of the
// kernel: at four heads per group 16 DFMAs and as many selects a lane for 16 bytes read). d / 4
// lanes share a page, four channels each; a warp takes U pages at a time and adds the U * G sums
// over its lanes by halving (each step exchanges half the values), which needs 1 + 2 + 4 + 8 (+ 1)
// exchanges for 16 sums instead of 5 each.
// page_list_kernel: one CTA per (slot, KV head, token): keys in shared memory, the m-th largest by
// radix selection over the bits in which the row's keys differ, ties by ascending index, and the
// list written in ascending order.
#include <math.h>

#include "common.cuh"
#include "paged.h"

namespace bsa {

namespace {

constexpr int kScoreThreads = 256;
constexpr uint32_t kNoPage = 0x7fffffffu;       // score of a page the table does not hold (a NaN)
constexpr uint32_t kBadScore = 0x7fc00000u;     // ... with a non-finite operand

// High word of the double x * 2^-896 (bf16) or x * 2^-1008 (fp16), low word 0, from the 16 bits
// of x in the low half of w. Exact for zeros and subnormals too.
template <bool F16>
__device__ __forceinline__ uint32_t dbl_hi(uint32_t w) {
  return ((w & 0x7fffu) << (F16 ? 10 : 13)) | ((w & 0x8000u) << 16);
}

template <bool F16>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

template <bool F16>
__device__ __forceinline__ double q_scaled(uint16_t x) {
  // x * 2^896 or x * 2^1008 (the product with dbl_hi's value is then x * k); NaN if not finite
  const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  if ((x & e) == e) return __longlong_as_double(0x7ff8000000000000ll);
  const double d = __hiloint2double((int)dbl_hi<F16>(x), 0);
  constexpr double half = F16 ? 0x1p1008 : 0x1p896;
  return d * half * half;
}

template <int D, int G, bool F16>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(
    CacheGeom g, int G_real, int chunk, int n_chunks, const uint16_t* __restrict__ q,
    const uint16_t* __restrict__ bounds, float* __restrict__ scores, int fill, int32_t* dev_status) {
  constexpr int LPP = D / 4;                    // lanes per page
  constexpr int PPW = 32 / LPP;                 // pages a warp reads side by side
  constexpr int U = G >= 16 ? 1 : (G * 8 <= 16 ? 8 : 16 / G);
  constexpr int NV = U * G;                     // sums per lane
  if (blockIdx.x == 0 && threadIdx.x == 0 && dev_status) *dev_status = 0;   // the list kernel reports
  const long long row = blockIdx.x / n_chunks;
  const int j0 = (int)(blockIdx.x % n_chunks) * chunk;
  const int t = (int)(row % g.T);
  const int h = (int)((row / g.T) % g.Hkv), b = (int)(row / g.T / g.Hkv);
  int base, ql;
  query_span(g, b, base, ql);
  const int vis = t < ql ? (base + t) / g.page + 1 : 0;      // pages 0 .. own page
  const int j1 = min(j0 + chunk, g.max_pages);
  float* out = scores + row * g.max_pages;
  if (fill)
    for (int j = max(j0, vis) + threadIdx.x; j < j1; j += kScoreThreads) out[j] = -INFINITY;
  const int je = min(j1, vis);
  if (j0 >= je) return;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = lane / LPP, ch = (lane % LPP) * 4;
  double qd[G][4];
  bool pos[G][4];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const uint16_t* qr = q + ((((size_t)b * g.Hkv + h) * G_real + min(i, G_real - 1)) * g.T + t) * D + ch;
    const uint2 w = *reinterpret_cast<const uint2*>(qr);
    const uint16_t x[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      qd[i][c] = q_scaled<F16>(x[c]);
      pos[i][c] = !(x[c] & 0x8000u);
    }
  }
  const int32_t* table = g.table + (size_t)b * g.max_pages;
  constexpr int kStep = (kScoreThreads / 32) * PPW * U;
  for (int jw = j0 + warp * PPW * U; jw < je; jw += kStep) {
    // pages jw + u * PPW + sub
    uint2 lo[U], hi[U];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = jw + u * PPW + sub;
      const int pg = j < je ? table[j] : -1;
      have[u] = pg >= 0 && pg < g.n_pages;
      const uint2* bp = reinterpret_cast<const uint2*>(
          bounds + (((size_t)(have[u] ? pg : 0) * g.Hkv + h) * 2) * D + ch);
      lo[u] = have[u] ? __ldg(bp) : make_uint2(0, 0);
      hi[u] = have[u] ? __ldg(bp + D / 4) : make_uint2(0, 0);
    }
    double s[NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kl[4] = {dbl_hi<F16>(lo[u].x), dbl_hi<F16>(lo[u].x >> 16), dbl_hi<F16>(lo[u].y),
                              dbl_hi<F16>(lo[u].y >> 16)};
      const uint32_t kh[4] = {dbl_hi<F16>(hi[u].x), dbl_hi<F16>(hi[u].x >> 16), dbl_hi<F16>(hi[u].y),
                              dbl_hi<F16>(hi[u].y >> 16)};
      const bool bad = nonfinite2<F16>(lo[u].x) || nonfinite2<F16>(lo[u].y) || nonfinite2<F16>(hi[u].x) ||
                       nonfinite2<F16>(hi[u].y);
      const double z = bad ? __longlong_as_double(0x7ff8000000000000ll) : 0.0;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        double acc = z;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc = fma(qd[i][c], __hiloint2double((int)(pos[i][c] ? kh[c] : kl[c]), 0), acc);
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
      if (j < je) {
        const int pg = table[j];
        const bool held = pg >= 0 && pg < g.n_pages;
        out[j] = held ? (r[p] != r[p] ? __uint_as_float(kBadScore) : r[p]) : __uint_as_float(kNoPage);
      }
    }
  }
}

// ---------------------------------------------------------------------------

constexpr int kListThreads = 256;
constexpr int kListWarps = kListThreads / 32;

struct ListSmem {
  unsigned hist[256];
  unsigned red[kListWarps], red2[kListWarps];
  unsigned digit, above;
  int status;
};

__global__ void __launch_bounds__(kListThreads) page_list_kernel(CacheGeom g, bsa_page_select_params p,
                                                                 const float* __restrict__ scores,
                                                                 int32_t* __restrict__ kv_idx,
                                                                 int32_t* __restrict__ kv_cnt,
                                                                 int32_t* dev_status) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ ListSmem s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long row = blockIdx.x;
  const int t = (int)(row % g.T), b = (int)(row / g.T / g.Hkv);
  int base, ql;
  const bool fits = query_span(g, b, base, ql);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t* out = kv_idx + row * p.k;
  if (t >= ql) {
    for (int i = tid; i < p.k; i += kListThreads) out[i] = -1;
    if (tid == 0) {
      kv_cnt[row] = 0;
      if (!fits) set_status(dev_status, BSA_DEV_BAD_INDEX);
    }
    return;
  }
  const int vis = (base + t) / g.page + 1;
  const int cnt = min(vis, p.k);
  for (int i = cnt + tid; i < p.k; i += kListThreads) out[i] = -1;
  if (tid == 0) kv_cnt[row] = cnt;
  if (vis <= p.k) {
    for (int i = tid; i < vis; i += kListThreads) out[i] = i;
    return;
  }
  const int n = vis - p.n_first - p.n_last, m = p.k - p.n_first - p.n_last;    // candidates, slots; n > m
  for (int i = tid; i < p.n_first; i += kListThreads) out[i] = i;
  for (int i = tid; i < p.n_last; i += kListThreads) out[p.k - p.n_last + i] = vis - p.n_last + i;
  if (m == 0) return;

  // keys, their minimum and maximum, and what is not finite
  if (tid == 0) s.status = 0;
  __syncthreads();
  const uint32_t* sc = reinterpret_cast<const uint32_t*>(scores + row * g.max_pages + p.n_first);
  unsigned mn = 0xffffffffu, mx = 0;
  int st = 0;
  for (int i = tid; i < n; i += kListThreads) {
    const uint32_t u = sc[i];
    uint32_t key = score_key(__uint_as_float(u));
    if ((u & 0x7f800000u) == 0x7f800000u) {
      st |= u == kNoPage ? BSA_DEV_BAD_INDEX : BSA_DEV_BAD_SCORE;
      key = 0;
    }
    keys[i] = key;
    mn = min(mn, key);
    mx = max(mx, key);
  }
  if (st) atomicOr(&s.status, st);
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) { s.red[warp] = mn; s.red2[warp] = mx; }
  __syncthreads();
  mn = s.red[0];
  mx = s.red2[0];
#pragma unroll
  for (int i = 1; i < kListWarps; ++i) { mn = min(mn, s.red[i]); mx = max(mx, s.red2[i]); }
  if (tid == 0 && s.status) set_status(dev_status, s.status);

  // Threshold: every key above it is in, and `left` of those equal to it. Digits of up to eight
  // bits from the highest bit in which keys differ down; `thr` holds the digits found, `mask` where.
  unsigned thr = mx, mask = 0xffffffffu;
  int left = m;
  if (mn != mx) {
    int top = 32 - __clz(mn ^ mx);              // bits [0, top) differ
    mask = top == 32 ? 0u : ~((1u << top) - 1u);
    thr = mx & mask;
    while (top > 0) {
      const int sh = max(top - 8, 0), width = top - sh;
      for (int i = tid; i < 256; i += kListThreads) s.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kListThreads) {
        const unsigned key = keys[i];
        if ((key & mask) == thr) atomicAdd(&s.hist[(key >> sh) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      // thread d: keys in digits above d (a suffix sum), from the top digit down
      const int d = 255 - tid;
      const unsigned mine = s.hist[d];
      unsigned x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();                          // red is free again
      if (lane == 31) s.red[warp] = x;
      __syncthreads();
      unsigned above = x - mine;
      for (int i = 0; i < warp; ++i) above += s.red[i];
      if (above < (unsigned)left && above + mine >= (unsigned)left) { s.digit = d; s.above = above; }
      __syncthreads();
      thr |= s.digit << sh;
      mask |= ((1u << width) - 1u) << sh;
      left -= s.above;
      top = sh;
      if (s.hist[s.digit] == (unsigned)left) break;   // the whole digit is in: thr is a lower bound
      __syncthreads();
    }
  }
  // in: (key & mask) > thr, or equal and among the first `left` of those. A warp takes a
  // contiguous range; counts first, then the places.
  __syncthreads();
  const int per = (n + kListWarps - 1) / kListWarps;
  const int i0 = min(warp * per, n), i1 = min(i0 + per, n);
  unsigned gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const unsigned k = keys[i] & mask;
    gt += k > thr;
    eq += k == thr;
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
    const unsigned k = i < i1 ? keys[i] & mask : 0u;
    const bool is_gt = i < i1 && k > thr, is_eq = i < i1 && k == thr;
    const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const unsigned eq_rank = at_eq + __popc(be & below);
    if (is_gt || (is_eq && eq_rank < (unsigned)left))
      out[p.n_first + at_gt + __popc(bg & below) + min(eq_rank, (unsigned)left)] = p.n_first + i;
    at_gt += __popc(bg);
    at_eq += __popc(be);
  }
}

template <int D, int G>
cudaError_t score_g(const CacheGeom& g, bool f16, int G_real, int chunk, int n_chunks, unsigned grid, const void* q,
                    const void* bounds, float* scores, int fill, int32_t* dev_status, cudaStream_t st) {
  auto kern = f16 ? page_score_kernel<D, G, true> : page_score_kernel<D, G, false>;
  kern<<<grid, kScoreThreads, 0, st>>>(g, G_real, chunk, n_chunks, (const uint16_t*)q, (const uint16_t*)bounds,
                                       scores, fill, dev_status);
  return cudaGetLastError();
}

template <int D>
cudaError_t score_d(const CacheGeom& g, bool f16, int G, int chunk, int n_chunks, unsigned grid, const void* q,
                    const void* bounds, float* scores, int fill, int32_t* dev_status, cudaStream_t st) {
  if (G == 1) return score_g<D, 1>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
  if (G == 2) return score_g<D, 2>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
  if (G <= 4) return score_g<D, 4>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
  if (G <= 8) return score_g<D, 8>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
  return score_g<D, 16>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
}

}  // namespace

cudaError_t launch_select_pages(const bsa_cache_shape& s, const CacheGeom& g, const bsa_page_select_params& p,
                                int Hq, const void* q, const void* bounds, float* scores, bool fill,
                                int32_t* kv_idx, int32_t* kv_cnt, int32_t* dev_status, cudaStream_t st) {
  const long long rows = (long long)g.slots * g.Hkv * g.T;
  const int chunk = 128;
  const int n_chunks = (g.max_pages + chunk - 1) / chunk;
  const unsigned grid = (unsigned)(rows * n_chunks);
  const int G = Hq / g.Hkv;
  const bool f16 = s.dtype == BSA_F16;
  cudaError_t e = s.d == 128 ? score_d<128>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st)
                             : score_d<64>(g, f16, G, chunk, n_chunks, grid, q, bounds, scores, fill, dev_status, st);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)g.max_pages * 4;
  e = cudaFuncSetAttribute(page_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rows);
  cfg.blockDim = dim3(kListThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_list_kernel, g, p, (const float*)scores, kv_idx, kv_cnt, dev_status);
}

}  // namespace bsa
