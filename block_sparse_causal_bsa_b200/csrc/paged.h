// Internal launchers of the paged-cache operators (host side). Pools: K, V
// [n_pages, Hkv, page, d], key bounds [n_pages, Hkv, 2, d] (per-channel minimum, maximum),
// page table [slots, max_pages] int32 (-1: no page).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/bsa.h"

namespace bsa {

constexpr int kMaxSlots = 4096;        // sequences of a table (resize keeps per-slot state in shared memory)
constexpr int kMaxTablePages = 32768;  // pages per sequence (a selection row is ranked in shared memory)
constexpr int kMaxQueryTokens = 1024;  // T

struct CacheGeom {
  int n_pages, Hkv, page, d;
  int slots, max_pages;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* q_len;                // null: T for every sequence
  int T;
};

// The tokens of slot b in this call: positions [base, base + ql). False (and ql = 0) when the
// lengths do not fit each other or the table.
__host__ __device__ inline bool query_span(const CacheGeom& g, int b, int& base, int& ql) {
  const int len = g.seq_len[b];
  ql = g.q_len ? g.q_len[b] : g.T;
  base = 0;
  if (ql == 0) return true;
  // (each compared by itself: a difference of wild lengths could overflow to one that fits)
  if (ql < 0 || ql > g.T || len < ql || (long long)len > (long long)g.max_pages * g.page) {
    ql = 0;
    return false;
  }
  base = len - ql;
  return true;
}

cudaError_t launch_pages_fork(int slots, int max_pages, int n_pages, int page, int32_t* table,
                              int32_t* seq_len, int32_t* refs, const int32_t* parent, int32_t* dev_status,
                              cudaStream_t st);
cudaError_t launch_pages_resize(int slots, int max_pages, int n_pages, int page, int32_t* table,
                                int32_t* seq_len, int32_t* refs, const int32_t* new_len, int32_t* pairs,
                                int32_t* n_free, int32_t* dev_status, cudaStream_t st);
cudaError_t launch_pages_copy(const bsa_cache_shape& s, void* k, void* v, void* bounds, const int32_t* pairs,
                              int n_pairs, int32_t* dev_status, cudaStream_t st);
cudaError_t launch_cache_append(const bsa_cache_shape& s, const CacheGeom& g, const void* k_new,
                                const void* v_new, void* k, void* v, void* bounds, int32_t* dev_status,
                                cudaStream_t st);
cudaError_t launch_cache_compact(const bsa_cache_shape& s, const CacheGeom& g, const int32_t* keep,
                                 const int32_t* n_keep, void* k, void* v, void* bounds, int32_t* dev_status,
                                 cudaStream_t st);
cudaError_t launch_tree_mask(int B, int T, const int32_t* parents, const int32_t* q_len,
                             unsigned long long* mask, int32_t* dev_status, cudaStream_t st);

}  // namespace bsa

namespace bsa {

// Of the current device; both are asked once per device (a step makes many of these calls).
int sm_count();
struct SmemSet {                       // one per kernel, static
  unsigned long long done[4] = {};
};
cudaError_t allow_smem(const void* kernel, size_t bytes, SmemSet& set);

// Page scores into scores [slots*Hkv*T][max_pages], then the lists. kmax_abs [slots*Hkv][max_pages]
// (workspace): the scores are fp32 estimates, and what they leave open is decided in fp64; null: the
// scores are exact, -inf past the visible pages.
cudaError_t launch_select_pages(const bsa_cache_shape& s, const CacheGeom& g, const bsa_page_select_params& p,
                                int Hq, const void* q, const void* bounds, float* scores, float* kmax_abs,
                                int32_t* kv_idx, int32_t* kv_cnt, int32_t* dev_status, cudaStream_t st);

}  // namespace bsa
