// Internal launchers of the page operators of the cache (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/smla.h"

namespace smla {

struct CachePages {
  uint8_t* kv;
  int32_t L, B, stride, log2_page;
  int32_t row_bytes;     // bytes of a slot's row; index keys: 128 (codes), scales apart
  int32_t index_keys;    // SMLA_CACHE_INDEX_KEYS: a page is P x 128 codes, then P fp32 scales
  int64_t page_bytes, num_pages, layer_stride;
  int32_t* err;          // device error word or NULL
};

cudaError_t launch_cache_copy_pages(const CachePages& c, const int32_t* src, const int32_t* dst, int64_t n, int sms,
                                    cudaStream_t s);
cudaError_t launch_cache_compact(const CachePages& c, const int32_t* page_table, const int32_t* starts,
                                 const int32_t* cu_keep, const int32_t* keep, int64_t n_keep, int32_t* new_lens, int sms,
                                 cudaStream_t s);

// The tables of smla_cache_fork and smla_cache_resize.
struct CacheTables {
  int32_t* page_table;
  int32_t* lens;
  int32_t* refs;
  int32_t* free_list;
  int32_t* free_count;
};
// Rows of the page table at most: a call marks each in a few bits of shared memory.
constexpr int kCacheMaxRequests = 1 << 16;
cudaError_t launch_cache_fork(const CachePages& c, const CacheTables& t, const int32_t* src_req, const int32_t* dst_req,
                              int32_t n, int32_t* fork_pages, int sms, cudaStream_t s);
cudaError_t launch_cache_resize(const CachePages& c, const CacheTables& t, const int32_t* req, const int32_t* new_lens,
                                int32_t n, int32_t* work, int sms, cudaStream_t s);

}  // namespace smla
