// C ABI of the paged-cache calls: argument validation, workspace layout and dispatch.
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "kernels.h"
#include "paged_work.cuh"

namespace {

template <class... A>
bsa_status fail(bsa_status st, const char* fmt, A... args) {
  bsa::set_last_error(fmt, args...);
  return st;
}
bsa_status fail(bsa_status st, const char* msg) {
  bsa::set_last_error("%s", msg);
  return st;
}
bsa_status done(cudaError_t e, const char* where) {
  if (e != cudaSuccess) return fail(BSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  bsa::set_last_error("%s", "");
  return BSA_OK;
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bsa_status check_table(int slots, int max_pages, int n_pages, int page) {
  if (slots < 1 || max_pages < 1 || n_pages < 1)
    return fail(BSA_ERR_INVALID_ARG, "slots, max_pages and n_pages must be >= 1");
  if (page != 16 && page != 32 && page != 64 && page != 128)
    return fail(BSA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128");
  if (slots > bsa::kMaxSlots) return fail(BSA_ERR_UNSUPPORTED, "more than %d slots", bsa::kMaxSlots);
  if (max_pages > bsa::kMaxTablePages)
    return fail(BSA_ERR_UNSUPPORTED, "more than %d pages per slot", bsa::kMaxTablePages);
  if ((long long)n_pages * page >= (1ll << 31)) return fail(BSA_ERR_UNSUPPORTED, "n_pages * page must be below 2^31");
  return BSA_OK;
}

bsa_status check_cache(const bsa_cache_shape* s) {
  if (!s) return fail(BSA_ERR_INVALID_ARG, "shape is NULL");
  if (s->n_pages < 1 || s->Hkv < 1) return fail(BSA_ERR_INVALID_ARG, "n_pages and Hkv must be >= 1");
  if (s->d != 64 && s->d != 128) return fail(BSA_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (s->page != 16 && s->page != 32 && s->page != 64 && s->page != 128)
    return fail(BSA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128");
  if (s->dtype != BSA_BF16 && s->dtype != BSA_F16)
    return fail(BSA_ERR_UNSUPPORTED, "the paged cache takes bf16 and fp16");
  if ((long long)s->n_pages * s->Hkv * s->page >= (1ll << 31))
    return fail(BSA_ERR_UNSUPPORTED, "n_pages * Hkv * page must be below 2^31 (cache rows are int32 coordinates)");
  return BSA_OK;
}

// Shape, table and token count of the calls that read or write the cache for a step's tokens.
bsa_status check_step(const bsa_cache_shape* s, int slots, int max_pages, int T) {
  bsa_status st = check_cache(s);
  if (st != BSA_OK) return st;
  st = check_table(slots, max_pages, s->n_pages, s->page);
  if (st != BSA_OK) return st;
  if (T < 1) return fail(BSA_ERR_INVALID_ARG, "T must be >= 1");
  if (T > bsa::kMaxQueryTokens) return fail(BSA_ERR_UNSUPPORTED, "T must be at most %d", bsa::kMaxQueryTokens);
  if ((long long)slots * s->Hkv * ((T + s->page - 2) / s->page + 1) >= (1ll << 31) - 1)
    return fail(BSA_ERR_UNSUPPORTED, "too many slots * Hkv * T");
  return BSA_OK;
}

bsa_status check_heads(const bsa_cache_shape* s, int slots, int Hq, int T) {
  if (Hq < 1 || Hq % s->Hkv) return fail(BSA_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (Hq / s->Hkv > 16) return fail(BSA_ERR_UNSUPPORTED, "Hq/Hkv must be at most 16");
  if ((long long)slots * Hq * T >= (1ll << 31)) return fail(BSA_ERR_UNSUPPORTED, "slots * Hq * T must be below 2^31");
  return BSA_OK;
}

bsa::CacheGeom geom(const bsa_cache_shape* s, int slots, int max_pages, int T, const int32_t* table,
                    const int32_t* seq_len, const int32_t* q_len) {
  bsa::CacheGeom g{};
  g.n_pages = s->n_pages;
  g.Hkv = s->Hkv;
  g.page = s->page;
  g.d = s->d;
  g.slots = slots;
  g.max_pages = max_pages;
  g.table = table;
  g.seq_len = seq_len;
  g.q_len = q_len;
  g.T = T;
  return g;
}

struct AttendWs {
  float* part_o;
  float* part_ml;
  int32_t* part_flag;
  int32_t* arrived;
  int n_cta, n_arrived;
  bool tc;
  size_t bytes;
};

AttendWs attend_ws(const bsa_cache_shape& s, int Hq, int T, bool list, void* base) {
  AttendWs w{};
  const int rows = (Hq / s.Hkv) * (list ? 1 : T);
  const bool tc = rows > bsa::kMaxMmaRows;
  const int rt = tc ? 256 : (rows <= 8 ? 8 : 16);
  w.n_cta = bsa::sm_count() * (tc ? 1 : bsa::kMmaSharesPerSm);
  w.n_arrived = (tc ? 2 : 1) * w.n_cta;
  w.tc = tc;
  const size_t slots = 2 * (size_t)w.n_cta;
  char* p = (char*)base;
  size_t off = 0;
  w.part_o = (float*)(p + off); off += align256(slots * rt * s.d * 4);
  w.part_ml = (float*)(p + off); off += align256(slots * rt * 2 * 4);
  w.part_flag = (int32_t*)(p + off); off += align256(2 * slots * 4);
  w.arrived = (int32_t*)(p + off); off += align256((size_t)w.n_arrived * 4);
  w.bytes = off;
  return w;
}

struct SelectWs {
  float* scores;                     // [slots*Hkv*T][max_pages]
  float* kmax_abs;                   // [slots*Hkv][max_pages]
  size_t bytes;
};

SelectWs select_ws(const bsa_cache_shape& s, int slots, int max_pages, int T, void* base) {
  SelectWs w{};
  char* p = (char*)base;
  size_t off = 0;
  w.scores = (float*)(p + off); off += align256((size_t)slots * s.Hkv * T * max_pages * 4);
  w.kmax_abs = (float*)(p + off); off += align256((size_t)slots * s.Hkv * max_pages * 4);
  w.bytes = off;
  return w;
}

bsa_status attend(const bsa_cache_shape* s, int slots, int max_pages, int Hq, int T, const void* q,
                  const void* k, const void* v, const int32_t* table, const int32_t* seq_len,
                  const int32_t* q_len, const uint64_t* mask, const int32_t* kv_idx, const int32_t* kv_cnt,
                  int W, float scale, void* out, float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                  void* stream) {
  if (!q || !k || !v || !table || !seq_len || !out || !dev_status || !ws)
    return fail(BSA_ERR_INVALID_ARG, "NULL q, pages, page_table, seq_len, out, dev_status or workspace");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return fail(BSA_ERR_INVALID_ARG, "q/pages/out need 16-byte alignment");
  if (!aligned(ws, 256)) return fail(BSA_ERR_INVALID_ARG, "workspace needs 256-byte alignment");
  if (mask && !aligned(mask, 8)) return fail(BSA_ERR_INVALID_ARG, "mask needs 8-byte alignment");
  if (!(scale > 0.0f) || !(scale < INFINITY)) return fail(BSA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  AttendWs w = attend_ws(*s, Hq, T, kv_idx != nullptr, ws);
  if (ws_bytes < w.bytes)
    return fail(BSA_ERR_INVALID_ARG, "workspace too small (%zu < %zu)", ws_bytes, w.bytes);
  bsa::PagedArgs a{};
  a.g = geom(s, slots, max_pages, T, table, seq_len, q_len);
  a.Hq = Hq;
  a.G = Hq / s->Hkv;
  a.words = (T + 63) / 64;
  a.q = (const uint16_t*)q;
  a.v = (const uint16_t*)v;
  a.mask = (const unsigned long long*)mask;
  a.kv_idx = kv_idx;
  a.kv_cnt = kv_cnt;
  a.W = W;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.part_o = w.part_o;
  a.part_ml = w.part_ml;
  a.part_flag = w.part_flag;
  a.arrived = w.arrived;
  a.n_arrived = w.n_arrived;
  a.dev_status = dev_status;
  a.n_cta = w.n_cta;
  cudaStream_t cs = (cudaStream_t)stream;
  if (w.tc) return done(bsa::launch_paged_attend_tc(*s, a, k, v, cs), "paged attend (tcgen05)");
  return done(bsa::launch_paged_attend_mma(*s, a, k, v, cs), "paged attend");
}

}  // namespace

extern "C" {

bsa_status bsa_pages_fork(int slots, int max_pages, int n_pages, int page, int32_t* page_table,
                          int32_t* seq_len, int32_t* refs, const int32_t* parent, int32_t* dev_status,
                          void* stream) {
  bsa_status st = check_table(slots, max_pages, n_pages, page);
  if (st != BSA_OK) return st;
  if (!page_table || !seq_len || !refs || !parent || !dev_status)
    return fail(BSA_ERR_INVALID_ARG, "NULL page_table, seq_len, refs, parent or dev_status");
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(dev_status, 0, sizeof(int32_t), cs);
  if (e != cudaSuccess) return done(e, "clear dev_status");
  return done(bsa::launch_pages_fork(slots, max_pages, n_pages, page, page_table, seq_len, refs, parent,
                                     dev_status, cs), "pages fork");
}

bsa_status bsa_pages_resize(int slots, int max_pages, int n_pages, int page, int32_t* page_table,
                            int32_t* seq_len, int32_t* refs, const int32_t* new_len, int32_t* pairs,
                            int32_t* n_free, int32_t* dev_status, void* stream) {
  bsa_status st = check_table(slots, max_pages, n_pages, page);
  if (st != BSA_OK) return st;
  if (!page_table || !seq_len || !refs || !new_len || !pairs || !dev_status)
    return fail(BSA_ERR_INVALID_ARG, "NULL page_table, seq_len, refs, new_len, pairs or dev_status");
  if (!aligned(refs, 16)) return fail(BSA_ERR_INVALID_ARG, "refs needs 16-byte alignment");
  return done(bsa::launch_pages_resize(slots, max_pages, n_pages, page, page_table, seq_len, refs, new_len,
                                       pairs, n_free, dev_status, (cudaStream_t)stream), "pages resize");
}

bsa_status bsa_pages_copy(const bsa_cache_shape* s, void* k, void* v, void* bounds, const int32_t* pairs,
                          int n_pairs, int32_t* dev_status, void* stream) {
  bsa_status st = check_cache(s);
  if (st != BSA_OK) return st;
  if (!k || !v || !pairs || !dev_status) return fail(BSA_ERR_INVALID_ARG, "NULL pages, pairs or dev_status");
  if (n_pairs < 0) return fail(BSA_ERR_INVALID_ARG, "n_pairs must be >= 0");
  if ((long long)n_pairs * s->Hkv >= (1ll << 31)) return fail(BSA_ERR_UNSUPPORTED, "n_pairs * Hkv must be below 2^31");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(bounds, 16) || !aligned(pairs, 8))
    return fail(BSA_ERR_INVALID_ARG, "pages and bounds need 16-byte, pairs 8-byte alignment");
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(dev_status, 0, sizeof(int32_t), cs);
  if (e != cudaSuccess) return done(e, "clear dev_status");
  if (n_pairs == 0) return done(cudaSuccess, "");
  return done(bsa::launch_pages_copy(*s, k, v, bounds, pairs, n_pairs, dev_status, cs), "pages copy");
}

bsa_status bsa_cache_append(const bsa_cache_shape* s, int slots, int max_pages, int T, const void* k_new,
                            const void* v_new, void* k, void* v, void* bounds, const int32_t* page_table,
                            const int32_t* seq_len, const int32_t* q_len, int32_t* dev_status, void* stream) {
  bsa_status st = check_step(s, slots, max_pages, T);
  if (st != BSA_OK) return st;
  if (!k_new || !v_new || !k || !v || !page_table || !seq_len || !dev_status)
    return fail(BSA_ERR_INVALID_ARG, "NULL k_new, v_new, pages, page_table, seq_len or dev_status");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(bounds, 16))
    return fail(BSA_ERR_INVALID_ARG, "k_new/v_new/pages/bounds need 16-byte alignment");
  return done(bsa::launch_cache_append(*s, geom(s, slots, max_pages, T, page_table, seq_len, q_len), k_new,
                                       v_new, k, v, bounds, dev_status, (cudaStream_t)stream), "cache append");
}

bsa_status bsa_cache_compact(const bsa_cache_shape* s, int slots, int max_pages, int T, const int32_t* keep,
                             const int32_t* n_keep, void* k, void* v, void* bounds,
                             const int32_t* page_table, const int32_t* seq_len, const int32_t* q_len,
                             int32_t* dev_status, void* stream) {
  bsa_status st = check_step(s, slots, max_pages, T);
  if (st != BSA_OK) return st;
  if (!keep || !n_keep || !k || !v || !page_table || !seq_len || !dev_status)
    return fail(BSA_ERR_INVALID_ARG, "NULL keep, n_keep, pages, page_table, seq_len or dev_status");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(bounds, 16))
    return fail(BSA_ERR_INVALID_ARG, "pages/bounds need 16-byte alignment");
  return done(bsa::launch_cache_compact(*s, geom(s, slots, max_pages, T, page_table, seq_len, q_len), keep,
                                        n_keep, k, v, bounds, dev_status, (cudaStream_t)stream), "cache compact");
}

bsa_status bsa_tree_mask(int B, int T, const int32_t* parents, const int32_t* q_len, uint64_t* mask,
                         int32_t* dev_status, void* stream) {
  if (B < 1 || T < 1) return fail(BSA_ERR_INVALID_ARG, "B and T must be >= 1");
  if (T > bsa::kMaxQueryTokens) return fail(BSA_ERR_UNSUPPORTED, "T must be at most %d", bsa::kMaxQueryTokens);
  if (!parents || !mask || !dev_status) return fail(BSA_ERR_INVALID_ARG, "NULL parents, mask or dev_status");
  if (!aligned(mask, 8)) return fail(BSA_ERR_INVALID_ARG, "mask needs 8-byte alignment");
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(dev_status, 0, sizeof(int32_t), cs);
  if (e != cudaSuccess) return done(e, "clear dev_status");
  return done(bsa::launch_tree_mask(B, T, parents, q_len, (unsigned long long*)mask, dev_status, cs), "tree mask");
}

size_t bsa_attend_paged_workspace_bytes(const bsa_cache_shape* s, int slots, int max_pages, int Hq, int T) {
  if (check_step(s, slots, max_pages, T) != BSA_OK || check_heads(s, slots, Hq, T) != BSA_OK) return 0;
  // the larger of the two calls
  const size_t tree = attend_ws(*s, Hq, T, false, nullptr).bytes, list = attend_ws(*s, Hq, T, true, nullptr).bytes;
  return tree > list ? tree : list;
}

bsa_status bsa_attend_tree(const bsa_cache_shape* s, int slots, int max_pages, int Hq, int T, const void* q,
                           const void* k, const void* v, const int32_t* page_table, const int32_t* seq_len,
                           const int32_t* q_len, const uint64_t* mask, float scale, void* out, float* lse,
                           int32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  bsa_status st = check_step(s, slots, max_pages, T);
  if (st == BSA_OK) st = check_heads(s, slots, Hq, T);
  if (st != BSA_OK) return st;
  return attend(s, slots, max_pages, Hq, T, q, k, v, page_table, seq_len, q_len, mask, nullptr, nullptr, 0,
                scale, out, lse, dev_status, ws, ws_bytes, stream);
}

bsa_status bsa_attend_pages(const bsa_cache_shape* s, int slots, int max_pages, int Hq, int T, const void* q,
                            const void* k, const void* v, const int32_t* page_table, const int32_t* seq_len,
                            const int32_t* q_len, const int32_t* kv_idx, const int32_t* kv_cnt, int W,
                            float scale, void* out, float* lse, int32_t* dev_status, void* ws,
                            size_t ws_bytes, void* stream) {
  bsa_status st = check_step(s, slots, max_pages, T);
  if (st == BSA_OK) st = check_heads(s, slots, Hq, T);
  if (st != BSA_OK) return st;
  if (!kv_idx || !kv_cnt) return fail(BSA_ERR_INVALID_ARG, "NULL kv_idx or kv_cnt");
  if (W < 1) return fail(BSA_ERR_INVALID_ARG, "W must be >= 1");
  if (W > bsa::kMaxTablePages) return fail(BSA_ERR_UNSUPPORTED, "W must be at most %d", bsa::kMaxTablePages);
  return attend(s, slots, max_pages, Hq, T, q, k, v, page_table, seq_len, q_len, nullptr, kv_idx, kv_cnt, W,
                scale, out, lse, dev_status, ws, ws_bytes, stream);
}

size_t bsa_select_pages_workspace_bytes(const bsa_cache_shape* s, int slots, int max_pages, int Hq, int T) {
  if (check_step(s, slots, max_pages, T) != BSA_OK || check_heads(s, slots, Hq, T) != BSA_OK) return 0;
  return select_ws(*s, slots, max_pages, T, nullptr).bytes;
}

bsa_status bsa_select_pages(const bsa_cache_shape* s, const bsa_page_select_params* p, int slots, int max_pages,
                            int Hq, int T, const void* q, const void* bounds, const int32_t* page_table,
                            const int32_t* seq_len, const int32_t* q_len, int32_t* kv_idx, int32_t* kv_cnt,
                            float* scores, int32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  bsa_status st = check_step(s, slots, max_pages, T);
  if (st == BSA_OK) st = check_heads(s, slots, Hq, T);
  if (st != BSA_OK) return st;
  if (!p) return fail(BSA_ERR_INVALID_ARG, "params is NULL");
  if (p->n_first < 0 || p->n_last < 1 || p->n_first > p->k || p->n_last > p->k - p->n_first)
    return fail(BSA_ERR_INVALID_ARG, "need n_first >= 0, n_last >= 1, n_first + n_last <= k");
  if (p->k > bsa::kMaxTablePages) return fail(BSA_ERR_UNSUPPORTED, "k must be at most %d", bsa::kMaxTablePages);
  if (!q || !bounds || !page_table || !seq_len || !kv_idx || !kv_cnt || !dev_status)
    return fail(BSA_ERR_INVALID_ARG, "NULL q, bounds, page_table, seq_len, kv_idx, kv_cnt or dev_status");
  if (!aligned(q, 16) || !aligned(bounds, 16)) return fail(BSA_ERR_INVALID_ARG, "q and bounds need 16-byte alignment");
  if ((long long)slots * s->Hkv * T * ((max_pages + 7) / 8) >= (1ll << 31))
    return fail(BSA_ERR_UNSUPPORTED, "slots * Hkv * T * max_pages / 8 must be below 2^31");
  SelectWs w{};
  if (!scores) {
    if (!ws) return fail(BSA_ERR_INVALID_ARG, "NULL workspace without scores");
    if (!aligned(ws, 256)) return fail(BSA_ERR_INVALID_ARG, "workspace needs 256-byte alignment");
    w = select_ws(*s, slots, max_pages, T, ws);
    if (ws_bytes < w.bytes) return fail(BSA_ERR_INVALID_ARG, "workspace too small (%zu < %zu)", ws_bytes, w.bytes);
  }
  return done(bsa::launch_select_pages(*s, geom(s, slots, max_pages, T, page_table, seq_len, q_len), *p, Hq, q,
                                       bounds, scores ? scores : w.scores, w.kmax_abs, kv_idx, kv_cnt, dev_status,
                                       (cudaStream_t)stream), "select pages");
}

}  // extern "C"
