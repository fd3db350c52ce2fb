// Attention over a paged cache on warp-level tensor-core MMAs: few query rows per KV head
// (decode, small trees of drafts), or a list of pages per token.
//
//   O = sum softmax(scale q.k) v over the positions a token sees
//
// The rows of an item (at most RT = 8 or 16) meet every key of a long cache: 4 d RT flops for 4 d
// bytes of K and V per key, so the kernel is bound by the HBM reads of the cache. What it does about
// it: a CTA streams its equal share of all key tiles (paged_work.cuh) through a ring of
// TMA-fed stages that never drains between items, and the MMAs, exponentials and shared-memory
// reads of a tile are spread over four warps so that they stay under the time its bytes take. Two
// CTAs share an SM: one streams while the other starts, writes a partial result or joins (one CTA of
// twice the size: 16 sequences of 64k tokens 638 us, now 629, that is 6.8 TB/s; 12 drafted chains over
// page lists 29 us, now 23). More, shorter shares than fit at once cost more starts than they even out
// (16 x 8 lists of 64 pages: 55 us, with twice the shares 62).
//
// 192 threads:
//   warps 0, 5 producers of K and of V (paged_feed.cuh)
//   warps 1-4  a warp owns 16 keys of every tile and keeps its own online softmax over them (maximum
//              m, sum l, unnormalised O):
//                S = K Q^T (A = K rows by ldmatrix, B = Q in registers), P = 2^(S scale log2 e - m),
//                O^T += V^T P^T (A = V^T by ldmatrix.trans, B = P^T from S by movmatrix)
//              P goes into the product as two 16-bit terms (value and rounding remainder), so O carries
//              no rounding of P: the second MMA is free here, the tensor pipe idles anyway. At the end of
//              a segment the four states are joined in shared memory.
// For fp16, weights are scaled by 2^14: fp16's smallest value is 2^-24, and many small weights
// would be lost below it.
// Rows that are no keys (the tail of the last page, missing pages) have their S masked and their
// V rows zeroed in shared memory, and non-finite values of drafted tokens are taken out of the
// tile and given back only to rows that see them.
#include <math.h>

#include <atomic>

#include "paged_feed.cuh"

namespace bsa {

namespace {

constexpr int kWarps = 4;                       // compute warps
constexpr int kThreads = 32 * (kWarps + 2);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the compute warps
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, int RT>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kHalf = kTileKeys * 128;          // 64 rows x 128 bytes
  static constexpr uint32_t kTile = kHalves * kHalf;          // K or V of a tile
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kPasses = D * RT > 1024 ? 2 : 1;       // of the join of the warps' states
  static constexpr int kDP = D / kPasses;                     // channels of a pass
};

// Column of channel d in row r of a dumped output: the rows 2 tig of a fragment's store fall eight
// banks apart, and four neighbouring channels stay together.
__device__ __forceinline__ int dump_col(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }

template <int D, int RT>
struct __align__(16) Ctrl {
  uint64_t full[Cfg<D, RT>::kStages], empty[Cfg<D, RT>::kStages];
  unsigned long long vmask[Cfg<D, RT>::kStages];    // rows of the stage that are keys of its item
  int abort_flag;
  int32_t status;
  int flag[2];                                  // by segment parity: non-finite drafts taken out
  int last;                                     // this CTA joins the item's parts
  float m[kWarps][RT], l[kWarps][RT];
  union {
    alignas(16) float o[kWarps][RT][Cfg<D, RT>::kDP];      // the warps' unnormalised outputs
    float2 ml[kWarps * RT * Cfg<D, RT>::kDP / 2];             // maxima and sums of an item's parts
  };
};

template <int D, int RT>
constexpr size_t smem_bytes() { return Cfg<D, RT>::kStages * Cfg<D, RT>::kStage + sizeof(Ctrl<D, RT>); }

// Four values of a row, final: normalised, rounded and stored, then the non-finite drafted values.
template <int D, bool F16, bool LIST>
__device__ __forceinline__ void store_row4(const PagedArgs& a, const Item& it, int r, int d4, float4 v, float mx,
                                           float ls, bool fixup) {
  constexpr float kShift = F16 ? 14.f : 0.f;
  int head, t;
  row_of<LIST>(a, it, r, head, t);
  const size_t row = ((size_t)it.b * a.Hq + head) * a.g.T + t;
  const float inv = ls == 0.f ? 0.f : 1.f / ls;
  *reinterpret_cast<uint2*>(a.out + row * D + d4) =
      make_uint2(pack_16<F16>(v.x * inv, v.y * inv), pack_16<F16>(v.z * inv, v.w * inv));
  if (!LIST && fixup) store_nonfinite<F16>(a, it, t, row, d4, d4 + 4);
  if (d4 == 0 && a.lse) a.lse[row] = ls == 0.f ? -INFINITY : (mx - kShift + log2f(ls)) * 0.69314718055994531f;
}

__device__ __forceinline__ void add4(float4& acc, const float4& v, float f) {
  acc.x = fmaf(v.x, f, acc.x);
  acc.y = fmaf(v.y, f, acc.y);
  acc.z = fmaf(v.z, f, acc.z);
  acc.w = fmaf(v.w, f, acc.w);
}

// Joins the parts of an item, the threads of the compute warps: four values of a row at a time. Parts come in
// chunks whose maxima and sums fit in shared memory (one chunk nearly always); the first reads of a chunk's
// outputs are on their way with those of its maxima and sums.
template <int D, int RT, bool F16, bool LIST>
__device__ __noinline__ void join_rows(const PagedArgs& a, const Item& it, const Parts<LIST, RT>& parts,
                                       Ctrl<D, RT>& c, int tid, bool ok) {
  constexpr int kU = 8;                          // reads in flight
  constexpr int kThr = 32 * kWarps;
  constexpr int kNI = RT * (D / 4) / kThr;       // quads of values per thread
  constexpr int kChunk = sizeof(c.ml) / (RT * sizeof(float2));
  // (copies: behind the ordered reads below, what the references name would be read again each time)
  const float* const part_o = a.part_o;
  const float2* const part_ml = reinterpret_cast<const float2*>(a.part_ml);
  const int32_t* const part_flag = a.part_flag;
  const Parts<LIST, RT> pt = parts;
  const int np = pt.n, quads = it.rows * (D / 4);
  if (!LIST)
    for (int i = tid; i < np; i += kThr)
      if (read_l2(part_flag + pt.slot(i))) atomicOr(&c.last, 2);
  float4 acc[kNI];
  float mx[kNI], ls[kNI];
#pragma unroll
  for (int k = 0; k < kNI; ++k) {
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    mx[k] = -INFINITY;
    ls[k] = 0.f;
  }
  for (int c0 = 0; c0 < np; c0 += kChunk) {
    const int nc = min(np - c0, kChunk);
    if (c0) compute_sync();                      // the chunk before has been used
    for (int i = tid; i < nc * RT; i += kThr) c.ml[i] = read_l2(part_ml + pt.slot(c0 + i / RT) * RT + i % RT);
    float4 v[kU];
    auto read = [&](int i, int p0) {
      const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p0 + u < nc && i < quads)
          v[u] = read_l2(reinterpret_cast<const float4*>(part_o + (pt.slot(c0 + p0 + u) * RT + r) * D + d4));
      }
    };
    read(tid, 0);
    compute_sync();
#pragma unroll
    for (int k = 0; k < kNI; ++k) {
      const int i = tid + k * kThr, r = i / (D / 4);
      if (i >= quads) continue;
      if (k) read(i, 0);
      float m = mx[k];
      for (int p = 0; p < nc; ++p) m = fmaxf(m, c.ml[p * RT + r].x);
      if (c0) {
        const float f = mx[k] == -INFINITY ? 0.f : ex2(mx[k] - m);
        ls[k] *= f;
        acc[k] = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
      }
      mx[k] = m;
      for (int p0 = 0; p0 < nc; p0 += kU) {
        if (p0) read(i, p0);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (p0 + u < nc) {
            const float2 ml = c.ml[(p0 + u) * RT + r];
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
            ls[k] += ml.y * f;
            add4(acc[k], v[u], f);
          }
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kNI; ++k) {
    const int i = tid + k * kThr;
    if (ok && i < quads) store_row4<D, F16, LIST>(a, it, i / (D / 4), (i % (D / 4)) * 4, acc[k], mx[k], ls[k], c.last & 2);
  }
}

}  // namespace

template <int D, int RT, bool F16, bool LIST>
__global__ void __launch_bounds__(kThreads, 2) paged_attend_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
    const __grid_constant__ PagedArgs a) {
  using C = Cfg<D, RT>;
  constexpr int NT = RT / 8;                    // MMA column tiles of the rows
  constexpr int DM = D / 16;                    // MMA row tiles of the head dim
  constexpr float kShift = F16 ? 14.f : 0.f;      // (store_row4 takes it back)
  extern __shared__ __align__(1024) uint8_t sm[];   // (the kernel has no other shared memory)
  Ctrl<D, RT>& c = *reinterpret_cast<Ctrl<D, RT>*>(sm + C::kStages * C::kStage);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::mbar_init(&c.full[s], 2);             // both producers
      tc::mbar_init(&c.empty[s], kWarps);
    }
    c.abort_flag = 0;
    c.status = 0;
    c.flag[0] = c.flag[1] = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort_flag = &c.abort_flag;

  Walk<LIST, RT> w;
  w.init(a);
  const long long x0 = w.start(blockIdx.x), x1 = w.start(blockIdx.x + 1);
  int issued = 0;

  if (warp == 0 || warp == kWarps + 1) {
    // ---------------- producers: K, V ----------------
    const bool is_k = warp == 0;
    const Feed<D> f{is_k ? &tmk : &tmv, sm + (is_k ? 0 : C::kTile), C::kStage, c.full, c.empty,
                    is_k ? c.vmask : nullptr};
    issued = feed_share<LIST, RT, D, C::kStages, C::kStages>(a, w, x0, x1, f, abort_flag, &c.status);
  } else {
    // ---------------- compute ----------------
    const int kw = warp - 1;
    const int g8 = lane >> 2, tig = lane & 3;
    const uint32_t sStages = tc::smem_u32(sm);
    const uint32_t rowK = (uint32_t)(16 * kw + (lane & 7) + ((lane >> 3) & 1) * 8) * 128u;
    const uint32_t rowV = (uint32_t)(16 * kw + (lane & 7) + (lane >> 4) * 8) * 128u;
    const uint32_t selK = (uint32_t)(lane >> 4), selV = (uint32_t)((lane >> 3) & 1);
    const uint32_t sw = (uint32_t)(lane & 7);
    const float sl2 = a.scale_log2;
    int n = 0, seg = 0;
    bool ok = true;
    Item it;
    if (x0 < x1) w.locate(a, x0, it);
    for (long long x = x0; x < x1; ++seg) {
      const long long xe = min(x1, it.first + it.units());
      int cnt;
      bool bad;
      const int live = item_live_tiles<LIST>(a, it, cnt, bad);
      const int ta = (int)(x - it.first), tend = (int)(xe - it.first), tb = min(tend, live);
      if (!LIST || it.t < it.ql) {
        // Q as the B operand: column = row of the item, k = head dim
        uint32_t qf[D / 16][NT][2];
        int tq[NT][2];                           // tokens of this thread's columns 8 nt + 2 tig (+1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = 8 * nt + g8;
          int head, t;
          row_of<LIST>(a, it, r < it.rows ? r : 0, head, t);
          const uint32_t* qr = reinterpret_cast<const uint32_t*>(
              a.q + (((size_t)it.b * a.Hq + head) * a.g.T + t) * D);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j) qf[kk][nt][j] = r < it.rows ? qr[8 * kk + 4 * j + tig] : 0u;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int rc = 8 * nt + 2 * tig + j;
            int hd;
            row_of<LIST>(a, it, rc < it.rows ? rc : 0, hd, tq[nt][j]);
          }
        }
        float o[DM][NT][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
          for (int dm = 0; dm < DM; ++dm)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[dm][nt][i] = 0.f;
        }

        for (int tile = ta; tile < tb; ++tile, ++n) {
          const int s = n % C::kStages;
          if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&c.full[s], (n / C::kStages) & 1, abort_flag, &c.status));
          if (!ok) continue;                     // still joins the barriers below
          const uint32_t kb = sStages + s * C::kStage, vb = kb + C::kTile;
          const unsigned vm = (unsigned)(c.vmask[s] >> (16 * kw)) & 0xffffu;      // this warp's keys
          const int pos0 = tile * kTileKeys + 16 * kw;                            // whole cache only
          const bool drafts = !LIST && pos0 + 16 > it.base;
          if (vm != 0xffffu || (drafts && (a.mask || it.ql > 1))) {
            // rows that are no keys get V = 0; non-finite values of drafted rows are taken out
            bool found = false;
            for (int r = 0; r < 16; ++r) {
              const bool key = (vm >> r) & 1;
              if (key && !(drafts && pos0 + r >= it.base)) continue;
              for (int ch = lane; ch < D / 8; ch += 32) {
                uint4* p = reinterpret_cast<uint4*>(sm + (vb - sStages) + (ch >> 3) * C::kHalf + (16 * kw + r) * 128 +
                                                    (((ch & 7) ^ (r & 7)) << 4));
                uint4 v = make_uint4(0, 0, 0, 0);
                if (key) {
                  v = *p;
                  found |= clear_nonfinite<F16>(v.x) | clear_nonfinite<F16>(v.y) |
                           clear_nonfinite<F16>(v.z) | clear_nonfinite<F16>(v.w);
                }
                *p = v;
              }
            }
            if (found) atomicOr(&c.flag[seg & 1], 1);
            tc::fence_proxy_async_smem();        // the stage is written by TMA next
            __syncwarp();
          }
          // S = K Q^T, two accumulator chains per column tile
          float sc[2][NT][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) sc[j][nt][i] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t af[4];
            const uint32_t chunk = (uint32_t)(2 * (kk & 3)) + selK;
            ldsm4(kb + (uint32_t)(kk >> 2) * C::kHalf + rowK + ((chunk ^ sw) << 4), af);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<F16>(sc[kk & 1][nt], af, qf[kk][nt][0], qf[kk][nt][1]);
          }
          // sv[nt][i]: key g8 (i < 2) or g8 + 8, columns 8 nt + 2 tig + (i & 1)
          float sv[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sv[nt][i] = sc[0][nt][i] + sc[1][nt][i];
          if (vm != 0xffffu || drafts) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kr = g8 + 8 * (i >> 1);
              const bool key = (vm >> kr) & 1;
              const int dj = pos0 + kr - it.base;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                bool see = key;
                if (!LIST && see && dj >= 0) see = sees_draft(a, it.b, tq[nt][i & 1], dj);
                if (!see) sv[nt][i] = -INFINITY;
              }
            }
          }
          // the maximum is exact, and reduced over the warp only when some score passes it
          float al[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float b0 = fmaxf(sv[nt][0], sv[nt][2]), b1 = fmaxf(sv[nt][1], sv[nt][3]);
            al[nt][0] = al[nt][1] = 1.f;
            if (__any_sync(0xffffffffu, b0 * sl2 > m[nt][0] || b1 * sl2 > m[nt][1])) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, off));
                b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, off));
              }
              const float t0 = b0 * sl2, t1 = b1 * sl2;
              if (t0 > m[nt][0]) { al[nt][0] = m[nt][0] == -INFINITY ? 0.f : ex2(m[nt][0] - t0); m[nt][0] = t0; }
              if (t1 > m[nt][1]) { al[nt][1] = m[nt][1] == -INFINITY ? 0.f : ex2(m[nt][1] - t1); m[nt][1] = t1; }
              if (al[nt][0] != 1.f || al[nt][1] != 1.f) {
#pragma unroll
                for (int dm = 0; dm < DM; ++dm) {
                  o[dm][nt][0] *= al[nt][0]; o[dm][nt][1] *= al[nt][1];
                  o[dm][nt][2] *= al[nt][0]; o[dm][nt][3] *= al[nt][1];
                }
              }
            }
          }
          // P = hi + lo in 16 bits each, as the B operand of O^T += V^T P^T
          uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float z0 = kShift - (m[nt][0] == -INFINITY ? 0.f : m[nt][0]);
            const float z1 = kShift - (m[nt][1] == -INFINITY ? 0.f : m[nt][1]);
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(sv[nt][i], sl2, (i & 1) ? z1 : z0));
            l[nt][0] = fmaf(l[nt][0], al[nt][0], p[0] + p[2]);
            l[nt][1] = fmaf(l[nt][1], al[nt][1], p[1] + p[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t h = pack_16<F16>(p[2 * u], p[2 * u + 1]);
              const uint32_t r = pack_16<F16>(p[2 * u] - cvt_f32<F16>((uint16_t)h),
                                              p[2 * u + 1] - cvt_f32<F16>((uint16_t)(h >> 16)));
              ph[nt][u] = movm_t(h);
              pl[nt][u] = movm_t(r);
            }
          }
#pragma unroll
          for (int dm = 0; dm < DM; ++dm) {
            uint32_t af[4];
            const uint32_t chunk = (uint32_t)(2 * (dm & 3)) + selV;
            ldsm4_t(vb + (uint32_t)(dm >> 2) * C::kHalf + rowV + ((chunk ^ sw) << 4), af);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<F16>(o[dm][nt], af, ph[nt][0], ph[nt][1]);
              mma16816<F16>(o[dm][nt], af, pl[nt][0], pl[nt][1]);
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&c.empty[s]);
        }

        // ---- join the warps' states: every warp leaves its own, then a thread adds up four values ----
        const int tid = threadIdx.x - 32;
        const bool whole = ta == 0 && tend == it.n_tiles;
        const size_t slot = 2 * (size_t)blockIdx.x + (ta == 0 ? 1 : 0);
        int fixup = 0;
#pragma unroll
        for (int pass = 0; pass < C::kPasses; ++pass) {
          if (pass) compute_sync();              // the pass before has been read
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = 8 * nt + 2 * tig + j;
#pragma unroll
              for (int dm = 0; dm < DM / C::kPasses; ++dm) {
                const int dd = pass * (DM / C::kPasses) + dm;
                c.o[kw][r][dump_col(r, 16 * dm + g8)] = o[dd][nt][j];
                c.o[kw][r][dump_col(r, 16 * dm + g8 + 8)] = o[dd][nt][2 + j];
              }
              if (pass) continue;
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
              if (g8 == 0) {
                c.m[kw][r] = m[nt][j];
                c.l[kw][r] = l[nt][j];
              }
            }
          compute_sync();
          fixup = *(volatile int*)&c.flag[seg & 1];
          for (int i = tid; i < it.rows * (C::kDP / 4); i += 32 * kWarps) {
            const int r = i / (C::kDP / 4), dp = (i % (C::kDP / 4)) * 4, d4 = pass * C::kDP + dp;
            float mw[kWarps], mx = -INFINITY, ls = 0.f;
#pragma unroll
            for (int u = 0; u < kWarps; ++u) {
              mw[u] = c.m[u][r];
              mx = fmaxf(mx, mw[u]);
            }
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < kWarps; ++u) {
              const float f = mw[u] == -INFINITY ? 0.f : ex2(mw[u] - mx);
              ls += c.l[u][r] * f;
              add4(v, *reinterpret_cast<const float4*>(&c.o[u][r][dump_col(r, dp)]), f);
            }
            if (whole) {
              if (ok) store_row4<D, F16, LIST>(a, it, r, d4, v, mx, ls, fixup);
            } else {
              *reinterpret_cast<float4*>(a.part_o + (slot * RT + r) * D + d4) = v;
              if (d4 == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * RT + r) * 2) = make_float2(mx, ls);
            }
          }
        }
        if (!whole) {
          // ---- arrival; the last CTA joins the parts ----
          if (tid == 0) a.part_flag[slot] = fixup;
          compute_sync();
          const Parts<LIST, RT> parts(w, it);
          if (tid == 0) c.last = arrive_part(a.arrived + parts.c1, parts.n);
          compute_sync();
          if (c.last) join_rows<D, RT, F16, LIST>(a, it, parts, c, tid, ok);
        }
        compute_sync();
        if (tid == 0) c.flag[seg & 1] = 0;       // next used two segments on, behind barriers
      }
      x = xe;
      if (x < x1) w.next(a, it);
    }
  }

  // ---------------- teardown ----------------
  __syncthreads();
  if (issued > 0 && lane == 0) feed_drain<C::kStages>(c.full, issued);
  if (threadIdx.x == 0) {
    wait_prepared();                             // in every CTA: this kernel's end is that one's, too
    if (c.status) atomicOr(a.dev_status, c.status);
  }
}

// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(256) paged_prepare_kernel(CacheGeom g, int n, int32_t* arrived,
                                                            int32_t* dev_status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < n; i += blockDim.x) arrived[i] = 0;
  bool bad = false;
  for (int b = threadIdx.x; b < g.slots; b += blockDim.x) {
    int base, ql;
    bad |= !query_span(g, b, base, ql);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *dev_status = bad ? BSA_DEV_BAD_INDEX : 0;
}

// ---------------------------------------------------------------------------
// host

int sm_count() {
  static std::atomic<int> count[256];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 256) return 148;
  n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaError_t allow_smem(const void* kernel, size_t bytes, SmemSet& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev < 256;
  unsigned long long* word = &set.done[(dev & 255) / 64];
  const unsigned long long bit = 1ull << (dev & 63);
  if (known && (__atomic_load_n(word, __ATOMIC_RELAXED) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && known) __atomic_fetch_or(word, bit, __ATOMIC_RELAXED);
  return e;
}

cudaError_t launch_paged_prepare(const PagedArgs& a, cudaStream_t st) {
  paged_prepare_kernel<<<1, 256, 0, st>>>(a.g, a.n_arrived, a.arrived, a.dev_status);
  return cudaGetLastError();
}

template <int D, int RT, bool F16, bool LIST>
static cudaError_t attend_t(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                            cudaStream_t st) {
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)s.n_pages * s.Hkv * s.page;
  const uint32_t box = s.page < kTileKeys ? s.page : kTileKeys;
  if (!make_tmap_bf16_2d(&mk, k, rows, D, 64, box) || !make_tmap_bf16_2d(&mv, v, rows, D, 64, box))
    return cudaErrorInvalidValue;
  auto kern = paged_attend_kernel<D, RT, F16, LIST>;
  constexpr size_t smem = smem_bytes<D, RT>();
  static_assert(smem <= 113 * 1024, "two CTAs per SM");
  static SmemSet set;
  cudaError_t e = allow_smem((const void*)kern, smem, set);
  if (e != cudaSuccess) return e;
  e = launch_paged_prepare(a, st);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = beside(at, a.n_cta, kThreads, smem, st);
  return cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
}

template <int D, int RT>
static cudaError_t attend_d(const bsa_cache_shape& s, const PagedArgs& a, const void* k, const void* v,
                            cudaStream_t st) {
  const bool f16 = s.dtype == BSA_F16;
  if (a.kv_idx)
    return f16 ? attend_t<D, RT, true, true>(s, a, k, v, st) : attend_t<D, RT, false, true>(s, a, k, v, st);
  return f16 ? attend_t<D, RT, true, false>(s, a, k, v, st) : attend_t<D, RT, false, false>(s, a, k, v, st);
}

cudaError_t launch_paged_attend_mma(const bsa_cache_shape& s, PagedArgs a, const void* k, const void* v,
                                    cudaStream_t st) {
  const int rows = a.kv_idx ? a.G : a.G * a.g.T;
  if (s.d == 128)
    return rows <= 8 ? attend_d<128, 8>(s, a, k, v, st) : attend_d<128, 16>(s, a, k, v, st);
  return rows <= 8 ? attend_d<64, 8>(s, a, k, v, st) : attend_d<64, 16>(s, a, k, v, st);
}

}  // namespace bsa
