// Page operators of the paged cache: copying pages, compacting kept rows in place, forking
// requests with shared pages, and growing or shrinking requests over a free list of pages.
// All of them move bytes or whole numbers: nothing is computed, every result is exact, and
// none depends on the order in which threads run.
#include "cache_pages.h"
#include "common.cuh"
#include "tcgen05.cuh"

namespace smla {
namespace {

__device__ __forceinline__ void flag(int32_t* err, int32_t bit) {
  if (err) atomicOr(err, bit);
}

// ---------------------------------------------------------------- copying pages

// Pages src[i] -> dst[i] in every layer. One CTA takes a piece of U x 4 KB of one page of one
// layer: U 16-byte loads a thread in flight, then U stores. Bound: HBM, 2 bytes moved for each
// byte of a page.
template <int U>
__global__ void __launch_bounds__(256) cache_copy_kernel(const CachePages c, const int32_t* src,
                                                         const int32_t* dst, int64_t n, int pieces) {
  const int64_t b = blockIdx.x;
  const int piece = static_cast<int>(b % pieces);
  const int64_t li = b / pieces, i = li % n, layer = li / n;
  pdl_wait();
  const int32_t s = src[i], d = dst[i];
  if (s == -1 || d == -1 || s == d) return;
  if (s < 0 || d < 0 || s >= c.num_pages || d >= c.num_pages) {
    if (piece == 0 && layer == 0 && threadIdx.x == 0) flag(c.err, SMLA_DEVERR_PAGE);
    return;
  }
  const uint8_t* a = c.kv + layer * c.layer_stride + int64_t(s) * c.page_bytes;
  uint8_t* o = c.kv + layer * c.layer_stride + int64_t(d) * c.page_bytes;
  const int64_t off = (int64_t(piece) * U * 256 + threadIdx.x) * 16;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (off + u * 4096 < c.page_bytes) v[u] = *reinterpret_cast<const uint4*>(a + off + u * 4096);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (off + u * 4096 < c.page_bytes) *reinterpret_cast<uint4*>(o + off + u * 4096) = v[u];
}

// ---------------------------------------------------------------- compacting rows

constexpr int kCpThreads = 256;

// Row starts[r] + keep[k] -> row starts[r] + k for each kept row k of request r, in place, in
// every layer. One CTA takes one (layer, request, range of 16-byte columns) and walks the kept
// rows in ascending chunks: it loads a chunk's pieces into registers, the whole CTA meets, and they are
// stored. With keep strictly ascending, keep[k] >= k, so row k of the result is a source of
// rows <= k only: those of earlier chunks, already loaded, and of this one, loaded before the
// barrier. No row that a later chunk reads is written early, and no other CTA touches these
// columns of this request. Bound: HBM, every moved row read and written once; what it reaches is set by how many CTAs an
// SM holds and by the chunks that follow one another: half of 16 contexts of 4k-16k slots kept, 656-byte rows, 4 layers,
// 437 MB, 116 us (3.8 TB/s; 128 with the places found in the chunk before, 182 with pieces staged in
// shared memory by cp.async, four chunks ahead); half of 4 contexts of 4k slots, 32 layers, 86 us (4.0 TB/s).
template <int kCpItems>  // 16-byte pieces a thread holds
__global__ void __launch_bounds__(kCpThreads, kCpItems == 4 ? 4 : 3) cache_compact_kernel(
    const CachePages c, const int32_t* page_table, const int32_t* starts,
    const int32_t* cu_keep, const int32_t* keep, int64_t n_keep, int32_t* new_lens, int columns,
    int slices, int group) {
  // byte offsets of the rows' old and new places, -1: not moved. Three chunks' worth: a chunk's are found
  // while others still store the one before the last.
  constexpr int kCpRows = kCpThreads / 4 * kCpItems;  // rows of a chunk at most: four columns a CTA at least
  __shared__ longlong2 s_row[3][kCpRows];
  const int tid = threadIdx.x;
  const int slice = blockIdx.x % slices;
  const int64_t rest = blockIdx.x / slices;
  const int r = static_cast<int>(rest % c.B), layer0 = static_cast<int>(rest / c.B) * group;
  const int layer1 = min(c.L, layer0 + group);
  bool first = slice == 0 && layer0 == 0;  // this CTA reports errors (once: for its first layer)
  pdl_wait();
  const int32_t start = starts[r], a = cu_keep[r], b = cu_keep[r + 1];
  if (start < 0 || a < 0 || b < a || b > n_keep || int64_t(start) + (b - a) > 0x7fffffff) {
    if (first && tid == 0) flag(c.err, SMLA_DEVERR_INDEX);
    return;
  }
  const int count = b - a;
  if (first && tid == 0 && new_lens) new_lens[r] = start + count;
  const int c0 = int(int64_t(columns) * slice / slices), c1 = int(int64_t(columns) * (slice + 1) / slices);
  const int cols = c1 - c0;
  // thread tid: column tid % cols of rows tid / cols + j (256 / cols) of a chunk
  const int step = kCpThreads / cols, my = tid / cols, col = c0 + tid - my * cols;
  const int rows = step * kCpItems;
  const int32_t* pt = page_table + int64_t(r) * c.stride;
  const int P = 1 << c.log2_page;
  // byte offset of a slot's row (index keys: of its codes), -1 where the slot has no page; `in`: the table has an
  // entry for it, `page`
  auto row_at = [&](int64_t slot, bool in, int32_t page) -> int64_t {
    if (!in || page < 0 || page >= c.num_pages) {
      if (first) flag(c.err, in ? SMLA_DEVERR_PAGE : SMLA_DEVERR_INDEX);
      return -1;
    }
    return int64_t(page) * c.page_bytes + (slot & (P - 1)) * c.row_bytes;
  };
  // the scale of an index key, from the offset of its codes
  auto scale_at = [&](int64_t off) -> int64_t {
    const int64_t page = off / c.page_bytes, in = off - page * c.page_bytes;
    return page * c.page_bytes + int64_t(P) * 128 + (in >> 7) * 4;
  };
  const int chunks = (count + rows - 1) / rows;
  // The places of a chunk's rows, kMine a thread, in three steps a chunk apart, so that no load is waited for: the kept
  // offsets, the pages of their slots and of where they go, the byte offsets. (All in one chunk: 183 us where this
  // takes 151, one request of 64k slots.)
  constexpr int kMine = (kCpRows + kCpThreads - 1) / kCpThreads;
  int32_t kept[kMine], prior[kMine], from[kMine], page0[kMine], page1[kMine];
  auto offsets = [&](int ch) {
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int i = tid + x * kCpThreads;
      const int64_t k = int64_t(ch) * rows + i;
      const bool in = i < rows && k < count;
      kept[x] = in ? keep[a + k] : -1;
      prior[x] = in && k ? keep[a + k - 1] : -1;
    }
  };
  auto pages = [&](int ch) {
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int i = tid + x * kCpThreads;
      const int64_t k = int64_t(ch) * rows + i;
      from[x] = -1;  // not moved
      if (i >= rows || k >= count) continue;
      if (kept[x] < k || kept[x] <= prior[x]) {
        if (first) flag(c.err, SMLA_DEVERR_INDEX);
      } else if (kept[x] != k) {
        from[x] = kept[x];
        const int64_t s0 = (int64_t(start) + kept[x]) >> c.log2_page, s1 = (int64_t(start) + k) >> c.log2_page;
        page0[x] = s0 < c.stride ? pt[s0] : -1;
        page1[x] = s1 < c.stride ? pt[s1] : -1;
      }
    }
  };
  auto places = [&](int ch) {
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int i = tid + x * kCpThreads;
      const int64_t k = int64_t(ch) * rows + i;
      if (i >= rows || k >= count) continue;
      longlong2 v = make_longlong2(-1, -1);
      if (from[x] >= 0) {
        const int64_t s0 = int64_t(start) + from[x], s1 = int64_t(start) + k;
        v.x = row_at(s0, (s0 >> c.log2_page) < c.stride, page0[x]);
        v.y = row_at(s1, (s1 >> c.log2_page) < c.stride, page1[x]);
        if (v.y < 0) v.x = -1;
      }
      s_row[ch % 3][i] = v;
    }
  };
  auto begin = [&] {  // the first chunk's, and what the next ones need
    offsets(0);
    pages(0);
    offsets(1);
    places(0);
    pages(1);
    offsets(2);
  };
  auto get = [&](uint4& v, const uint8_t* base, int64_t so) {
    if (c.index_keys && col == 8)
      v.x = *reinterpret_cast<const uint32_t*>(base + scale_at(so));
    else
      v = *reinterpret_cast<const uint4*>(base + so + 16 * col);
  };
  auto put = [&](const uint4& v, uint8_t* base, int64_t dp) {
    if (c.index_keys && col == 8)
      *reinterpret_cast<uint32_t*>(base + scale_at(dp)) = v.x;
    else
      *reinterpret_cast<uint4*>(base + dp + 16 * col) = v;
  };
  uint4 v[kCpItems];
  if (chunks <= 1) {
    // Few rows (an accepted path): their places are found once, and as many layers as fit are loaded
    // together.
    if (count == 0) return;
    begin();
    __syncthreads();
    const int each = (count + step - 1) / step, together = kCpItems / each;  // items of a layer; layers at once
    for (int l0 = layer0; l0 < layer1; l0 += together) {
#pragma unroll
      for (int j = 0; j < kCpItems; ++j) {
        const int l = j / each, i = my + (j - l * each) * step;
        if (my >= step || i >= count || l >= together || l0 + l >= layer1 || s_row[0][i].x < 0) continue;
        get(v[j], c.kv + int64_t(l0 + l) * c.layer_stride, s_row[0][i].x);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kCpItems; ++j) {
        const int l = j / each, i = my + (j - l * each) * step;
        if (my >= step || i >= count || l >= together || l0 + l >= layer1 || s_row[0][i].x < 0) continue;
        put(v[j], c.kv + int64_t(l0 + l) * c.layer_stride, s_row[0][i].y);
      }
    }
    return;
  }
  for (int layer = layer0; layer < layer1; ++layer) {
    uint8_t* base = c.kv + int64_t(layer) * c.layer_stride;
    begin();
    __syncthreads();
    for (int ch = 0; ch < chunks; ++ch) {
      const int m = min(rows, count - ch * rows);
#pragma unroll
      for (int j = 0; j < kCpItems; ++j) {
        const int i = my + j * step;
        if (my < step && i < m && s_row[ch % 3][i].x >= 0) get(v[j], base, s_row[ch % 3][i].x);
      }
      places(ch + 1);  // behind this chunk's loads
      pages(ch + 2);
      offsets(ch + 3);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kCpItems; ++j) {
        const int i = my + j * step;
        if (my < step && i < m && s_row[ch % 3][i].x >= 0) put(v[j], base, s_row[ch % 3][i].y);
      }
    }
    first = false;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- forking and resizing

constexpr int kListThreads = 1024;

// Inclusive sum of v over the CTA's threads (1024); `total` gets the sum. One call's result is
// read before the next call starts.
__device__ __forceinline__ int64_t block_sum_scan(int64_t v, int64_t* s_warp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[31];
  return v + (warp ? s_warp[warp - 1] : 0);
}

__device__ __forceinline__ int64_t pages_of(int64_t len, int log2_page) {
  return (len + (int64_t(1) << log2_page) - 1) >> log2_page;
}
// The free pages a list can hold, whatever its count says.
__device__ __forceinline__ int64_t clamp_count(int64_t v, int64_t num_pages, int32_t* err, bool say) {
  if (v >= 0 && v <= num_pages) return v;
  if (say) flag(err, SMLA_DEVERR_PAGE);
  return v < 0 ? 0 : num_pages;
}

// First step of a fork: which forks are taken, and the page of each partly filled last page.
// One CTA. A fork is refused (SMLA_DEVERR_INDEX) when a request is out of range, when its
// target is listed twice as a target or at all as a source, or still holds slots; and
// (SMLA_DEVERR_PAGE) when its source's partly filled last page is no page, when fewer free pages are left than
// it and those before it need, or when the one it would take is no page.
// fork_pages[i]: the page taken, -1 where none was needed, -2 for a refused fork.
__global__ void __launch_bounds__(kListThreads) cache_fork_plan_kernel(const CachePages c, const CacheTables t,
                                                                       const int32_t* src_req,
                                                                       const int32_t* dst_req, int32_t n,
                                                                       int32_t* fork_pages) {
  extern __shared__ uint32_t bits[];  // targets seen, targets seen twice, sources: a bit a request
  __shared__ int64_t s_warp[32];
  const int tid = threadIdx.x, words = (c.B + 31) >> 5;
  for (int i = tid; i < 3 * words; i += kListThreads) bits[i] = 0;
  pdl_wait();
  pdl_trigger();  // (the copies read lengths and tables before they wait for this kernel)
  const int64_t count = clamp_count(*t.free_count, c.num_pages, c.err, tid == 0);
  __syncthreads();
  for (int i = tid; i < n; i += kListThreads) {
    const int32_t d = dst_req[i], s = src_req[i];
    if (d >= 0 && d < c.B) {
      const uint32_t m = 1u << (d & 31);
      if (atomicOr(&bits[d >> 5], m) & m) atomicOr(&bits[words + (d >> 5)], m);
    }
    if (s >= 0 && s < c.B) atomicOr(&bits[2 * words + (s >> 5)], 1u << (s & 31));
  }
  __syncthreads();
  int64_t used = 0;
  for (int i0 = 0; i0 < n; i0 += kListThreads) {
    const int i = i0 + tid;
    bool ok = false, need = false, lost = false;  // lost: rows to copy, and no page that holds them
    int32_t s = 0, d = 0;
    int64_t len = 0;
    if (i < n) {
      s = src_req[i];
      d = dst_req[i];
      ok = s >= 0 && s < c.B && d >= 0 && d < c.B;
      if (ok) {
        const uint32_t m = 1u << (d & 31);
        len = t.lens[s];
        ok = !(bits[words + (d >> 5)] & m) && !(bits[2 * words + (d >> 5)] & m) && t.lens[d] == 0 && len >= 0 &&
             len <= (int64_t(c.stride) << c.log2_page);
      }
      if (!ok) flag(c.err, SMLA_DEVERR_INDEX);
      if (ok && (len & ((1 << c.log2_page) - 1)) != 0) {
        const int32_t last = t.page_table[int64_t(s) * c.stride + (len >> c.log2_page)];
        need = last >= 0 && last < c.num_pages;
        lost = !need;
      }
    }
    int64_t total;
    const int64_t at = used + block_sum_scan(need ? 1 : 0, s_warp, total);  // needs up to this one
    used += total;
    if (i < n) {
      int32_t got = ok && !lost ? -1 : -2;
      if (lost) flag(c.err, SMLA_DEVERR_PAGE);
      if (need) {
        got = -2;
        if (at <= count) {
          const int64_t pos = count - at;
          const int32_t page = t.free_list[pos];
          t.free_list[pos] = -1;
          if (page >= 0 && page < c.num_pages) {
            got = page;
            t.refs[page] = 1;
            t.page_table[int64_t(d) * c.stride + (len >> c.log2_page)] = page;
          }
        }
        if (got == -2) flag(c.err, SMLA_DEVERR_PAGE);
      }
      fork_pages[i] = got;
      if (got != -2) t.lens[d] = static_cast<int32_t>(len);
    }
  }
  if (tid == 0) *t.free_count = static_cast<int32_t>(count - (used < count ? used : count));
}

// Second step: the full pages are shared, and the used rows of the last page are copied in every
// layer. CTA (i, y) of a fork takes every y-th group of table entries and piece of rows.
__global__ void __launch_bounds__(256) cache_fork_kernel(const CachePages c, const CacheTables t,
                                                         const int32_t* src_req,
                                                         const int32_t* dst_req,
                                                         const int32_t* fork_pages) {
  const int i = blockIdx.x, y = blockIdx.y, ny = gridDim.y, tid = threadIdx.x;
  // the sources' lengths and table rows are not touched by the first step: they are read while it runs
  const int32_t s = src_req[i], d = dst_req[i];
  const bool in = s >= 0 && s < c.B;
  const int64_t cap = int64_t(c.stride) << c.log2_page, len = in ? min(max(int64_t(t.lens[s]), int64_t(0)), cap) : 0;
  const int full = static_cast<int>(len >> c.log2_page);
  const int part = static_cast<int>(len & ((1 << c.log2_page) - 1));
  const int32_t* from = t.page_table + int64_t(in ? s : 0) * c.stride;
  const int32_t last = part ? from[full] : -1;
  pdl_wait();
  const int32_t got = __ldcg(fork_pages + i);
  if (got == -2) return;
  int32_t* to = t.page_table + int64_t(d) * c.stride;
  for (int k = y * 256 + tid; k < full; k += ny * 256) {
    const int32_t page = from[k];
    to[k] = page;
    if (page >= 0 && page < c.num_pages)
      atomicAdd(t.refs + page, 1);
    else
      flag(c.err, SMLA_DEVERR_PAGE);
  }
  if (part == 0) return;  // (a fork whose last page is no page has been refused)
  const int64_t bytes = int64_t(part) * c.row_bytes;
  const int pieces = static_cast<int>((bytes + 8191) / 8192);
  for (int w = y; w < pieces * c.L; w += ny) {
    const int layer = w / pieces, piece = w - layer * pieces;
    const uint8_t* a = c.kv + layer * c.layer_stride + int64_t(last) * c.page_bytes;
    uint8_t* o = c.kv + layer * c.layer_stride + int64_t(got) * c.page_bytes;
    const int64_t off = int64_t(piece) * 8192 + tid * 16;
    uint4 v0, v1;
    if (off < bytes) v0 = *reinterpret_cast<const uint4*>(a + off);
    if (off + 4096 < bytes) v1 = *reinterpret_cast<const uint4*>(a + off + 4096);
    if (off < bytes) *reinterpret_cast<uint4*>(o + off) = v0;
    if (off + 4096 < bytes) *reinterpret_cast<uint4*>(o + off + 4096) = v1;
    if (c.index_keys && piece == 0) {  // and the scales of those slots
      const int64_t so = int64_t(128) << c.log2_page;
      if (tid < part)
        reinterpret_cast<uint32_t*>(o + so)[tid] = reinterpret_cast<const uint32_t*>(a + so)[tid];
    }
  }
}

// A page whose last holder has let go carries this bit until the push step lists it.
constexpr int32_t kRefFreed = 1 << 30;

// Whether entry i of a resize list is valid by itself; its request's old and new page counts. (A request that is listed
// twice is refused both times: that the callers find out.)
struct Resize {
  bool ok;
  int32_t r;
  int64_t old_pages, new_pages;
};
__device__ __forceinline__ Resize resize_entry(const CachePages& c, const CacheTables& t, const int32_t* req,
                                               const int32_t* new_lens, int i) {
  Resize e;
  e.r = req[i];
  e.old_pages = e.new_pages = 0;
  e.ok = e.r >= 0 && e.r < c.B;
  if (e.ok) {
    const int64_t cap = int64_t(c.stride) << c.log2_page;
    const int64_t a = __ldcg(t.lens + e.r), b = new_lens[i];
    e.ok = a >= 0 && a <= cap && b >= 0 && b <= cap;
    e.old_pages = pages_of(a, c.log2_page);
    e.new_pages = pages_of(b, c.log2_page);
  }
  return e;
}

constexpr int kPushCtas = 8;
constexpr int kMarkWords = 1536;  // words of marks a CTA and round
constexpr int64_t kResizeOneLaunch = 1 << 16;  // table entries

// The pages of entry e beyond its new length leave the table and lose a holder; threads `at`, at + step, ...
__device__ __forceinline__ void release_pages(const CachePages& c, const CacheTables& t, const Resize& e, int64_t at, int64_t step) {
  int32_t* row = t.page_table + int64_t(e.r) * c.stride;
  for (int64_t k = e.new_pages + at; k < e.old_pages; k += step) {
    const int32_t page = row[k];
    row[k] = -1;
    if (page < 0 || page >= c.num_pages) {
      flag(c.err, SMLA_DEVERR_PAGE);
      continue;
    }
    // Sums only, so that every order of several releases ends the same: a count of holders before is 1 .. 2^29 - 1,
    // and what one release too many finds is 0, negative or near the mark.
    const int32_t had = atomicSub(t.refs + page, 1);
    if (had == 1) {
      atomicAdd(t.refs + page, kRefFreed);
    } else if (had <= 0 || had >= kRefFreed / 2) {  // more holders let go than there were
      atomicAdd(t.refs + page, 1);
      flag(c.err, SMLA_DEVERR_PAGE);
    }
  }
}

// A growing request takes its pages off the list, the last one first.
__device__ __forceinline__ void pop_pages(const CachePages& c, const CacheTables& t, int32_t r, int64_t pos, int64_t old_pages,
                                          int64_t new_pages, int64_t at, int64_t step) {
  int32_t* row = t.page_table + int64_t(r) * c.stride;
  for (int64_t k = old_pages + at; k < new_pages; k += step) {
    const int64_t from = pos - (k - old_pages);
    const int32_t page = __ldcg(t.free_list + from);
    t.free_list[from] = -1;
    const bool ok = page >= 0 && page < c.num_pages;
    row[k] = ok ? page : -1;
    if (ok)
      t.refs[page] = 1;
    else
      flag(c.err, SMLA_DEVERR_PAGE);
  }
}

// First step of a resize: the releases. CTA (i, y) takes every y-th group of request i's entries.
__global__ void __launch_bounds__(256) cache_release_kernel(const CachePages c, const CacheTables t,
                                                            const int32_t* req,
                                                            const int32_t* new_lens, int32_t n) {
  const int i = blockIdx.x;
  pdl_wait();
  pdl_trigger();  // (the next step reads the lists and lengths before it waits for this kernel)
  const Resize e = resize_entry(c, t, req, new_lens, i);
  int twice = 0;
  for (int j = threadIdx.x; j < n; j += 256) twice |= j != i && req[j] == e.r;
  twice = __syncthreads_or(twice);
  if (!e.ok || twice) {
    if (threadIdx.x == 0) flag(c.err, SMLA_DEVERR_INDEX);
    return;
  }
  release_pages(c, t, e, blockIdx.y * 256 + threadIdx.x, int64_t(gridDim.y) * 256);
}

// Lists the freed pages behind the `count` pages of the free list, in ascending order, and clears their marks;
// returns how many. All CTAs of a cluster of kPushCtas call it, 1024 threads each; marks: 2 kMarkWords
// words of shared memory. Their pushes are visible to one another after the next cluster barrier.
__device__ __forceinline__ int64_t push_freed(const CachePages& c, const CacheTables& t, uint32_t* marks, int64_t* s_warp,
                                              int64_t* s_sum, int rank, int64_t count) {
  const int tid = threadIdx.x, lane = tid & 31;
  int64_t freed = 0;
  // The marks of a range of pages, an eighth a CTA, a bit a page, go to shared memory in one pass; then each
  // warp lists the pages of a word, so that its stores are next to one another.
  int32_t* before = reinterpret_cast<int32_t*>(marks + kMarkWords);  // marks of the CTA's words before
  constexpr int64_t kRound = 32 * int64_t(kMarkWords) * kPushCtas;  // pages a round: 393,216
  int64_t at = count;
  for (int64_t r0 = 0; r0 < c.num_pages; r0 += kRound) {
    const int64_t r1 = min(c.num_pages, r0 + kRound), per = ((r1 - r0 + kPushCtas - 1) / kPushCtas + 31) & ~int64_t(31);
    const int64_t a = min(r1, r0 + per * rank), b = min(r1, a + per);
    const int nw = static_cast<int>((b - a + 31) >> 5);
    constexpr int kAhead = 16, kW = kListThreads / 32;  // words a warp loads at once
    for (int w = tid >> 5; w < nw; w += kAhead * kW) {
      int32_t v[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {  // (past the end: the last page again, so that no load hangs on a branch)
        const int64_t p = a + 32 * int64_t(w + x * kW) + lane;
        v[x] = __ldcg(t.refs + min(p, b - 1));
        if (p >= b) v[x] = 0;
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const uint32_t m = __ballot_sync(0xffffffffu, (v[x] & kRefFreed) != 0);
        if (lane == 0 && w + x * kW < nw) marks[w + x * kW] = m;
      }
    }
    __syncthreads();
    const int each = (nw + kListThreads - 1) / kListThreads, w0 = min(nw, tid * each), w1 = min(nw, w0 + each);
    int64_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(marks[w]);
    int64_t total;
    int64_t upto = block_sum_scan(mine, s_warp, total) - mine;
    for (int w = w0; w < w1; ++w) {
      before[w] = static_cast<int32_t>(upto);
      upto += __popc(marks[w]);
    }
    if (tid == 0) *s_sum = total;
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    int64_t from = at, sum = 0;
    for (int k = 0; k < kPushCtas; ++k) {
      int64_t v;
      asm volatile("ld.shared::cluster.b64 %0, [%1];"
                   : "=l"(v)
                   : "r"(tc::mapa(static_cast<uint32_t>(__cvta_generic_to_shared(s_sum)), k)));
      if (k < rank) from += v;
      sum += v;
    }
    at += sum;
    freed += sum;
    for (int w = tid >> 5; w < nw; w += kListThreads / 32) {
      const uint32_t m = marks[w];
      if (!((m >> lane) & 1)) continue;
      const int64_t p = a + 32 * int64_t(w) + lane, pos = from + before[w] + __popc(m & ((1u << lane) - 1));
      t.refs[p] = 0;
      if (pos < c.num_pages)
        t.free_list[pos] = static_cast<int32_t>(p);
      else
        flag(c.err, SMLA_DEVERR_PAGE);
    }
    if (r0 + kRound < c.num_pages) {  // the counts and the marks are rewritten
      tc::cluster_arrive();
      tc::cluster_wait();
    }
  }
  return freed;
}

// A list of up to 1024 requests in one launch, one cluster of eight CTAs. Every CTA looks at the whole list, a
// thread a request. The cluster's threads then form teams of 32 to 1024, about one a request, that take the
// released pages out of the tables; the freed ones are listed; every CTA gives the growing requests their
// places in the list, in the order of the call (a request is refused, SMLA_DEVERR_PAGE, when fewer pages
// are free than it and those before it ask for); the teams take the pages.
__global__ void __cluster_dims__(kPushCtas, 1, 1) __launch_bounds__(kListThreads)
    cache_resize_kernel(const CachePages c, const CacheTables t, const int32_t* req,
                        const int32_t* new_lens, int32_t n) {
  extern __shared__ uint32_t bits[];  // requests listed, requests listed twice; marks
  __shared__ int64_t s_warp[32], s_sum;
  __shared__ int3 s_entry[kListThreads];  // (request or -1, old pages, new pages)
  __shared__ int32_t s_pos[kListThreads];
  const int tid = threadIdx.x, rank = blockIdx.x, words = (c.B + 31) >> 5;
  Resize e;
  e.ok = false;
  e.r = -1;
  e.old_pages = e.new_pages = 0;
  pdl_wait();
  if (tid < n) e = resize_entry(c, t, req, new_lens, tid);
  const int64_t count = clamp_count(__ldcg(t.free_count), c.num_pages, c.err, rank == 0 && tid == 0);
  for (int i = tid; i < 2 * words; i += kListThreads) bits[i] = 0;
  __syncthreads();
  const bool in = tid < n && e.r >= 0 && e.r < c.B;
  if (in) {
    const uint32_t m = 1u << (e.r & 31);
    if (atomicOr(&bits[e.r >> 5], m) & m) atomicOr(&bits[words + (e.r >> 5)], m);
  }
  __syncthreads();
  if (in && ((bits[words + (e.r >> 5)] >> (e.r & 31)) & 1)) e.ok = false;
  if (tid < n && !e.ok && rank == 0) flag(c.err, SMLA_DEVERR_INDEX);
  if (tid < n) s_entry[tid] = make_int3(e.ok ? e.r : -1, static_cast<int>(e.old_pages), static_cast<int>(e.new_pages));
  const int64_t need = e.ok && e.new_pages > e.old_pages ? e.new_pages - e.old_pages : 0;
  const int any = __syncthreads_or(e.ok && e.new_pages < e.old_pages);
  int64_t total;
  const int64_t upto = block_sum_scan(need, s_warp, total);
  int team = kListThreads;
  while (team > 32 && int64_t(team) * n > kPushCtas * kListThreads) team >>= 1;
  const int teams = kPushCtas * kListThreads / team, at = tid & (team - 1);
  const int first = rank * (kListThreads / team) + tid / team;
  tc::cluster_arrive();  // the old lengths and the count have been read
  int64_t freed = 0;
  if (any) {
    for (int i = first; i < n; i += teams) {
      const int3 x = s_entry[i];
      if (x.x < 0) continue;
      Resize y;
      y.ok = true;
      y.r = x.x;
      y.old_pages = x.y;
      y.new_pages = x.z;
      release_pages(c, t, y, at, team);
    }
    tc::cluster_wait();
    tc::cluster_arrive();
    tc::cluster_wait();  // all releases are visible
    freed = push_freed(c, t, bits + 2 * words, s_warp, &s_sum, rank, count);
    tc::cluster_arrive();
    tc::cluster_wait();
  }
  const int64_t avail = min(c.num_pages, count + freed);
  const bool fits = need == 0 || upto <= avail;
  int64_t given;
  block_sum_scan(fits ? need : 0, s_warp, given);
  if (tid < n) s_pos[tid] = need != 0 && fits ? static_cast<int32_t>(avail - 1 - (upto - need)) : -1;
  if (rank == 0 && !fits) flag(c.err, SMLA_DEVERR_PAGE);
  __syncthreads();
  for (int i = first; i < n; i += teams) {
    const int64_t pos = s_pos[i];
    if (pos >= 0) pop_pages(c, t, s_entry[i].x, pos, s_entry[i].y, s_entry[i].z, at, team);
  }
  if (!any) tc::cluster_wait();
  if (rank == 0) {
    if (e.ok && fits) t.lens[e.r] = new_lens[tid];
    if (tid == 0) *t.free_count = static_cast<int32_t>(avail - given);
  }
}

// Longer lists and tables, in three launches. The second step, one cluster of eight CTAs: the freed pages are
// listed, then the first CTA gives the growing requests their places as above. work[2i]: the list position
// of the request's first page, -1 where it takes none; work[2i+1]: its old page count.
__global__ void __cluster_dims__(kPushCtas, 1, 1) __launch_bounds__(kListThreads)
    cache_push_kernel(const CachePages c, const CacheTables t, const int32_t* req,
                      const int32_t* new_lens, int32_t n, int32_t* work) {
  extern __shared__ uint32_t bits[];  // requests listed, requests listed twice; marks
  __shared__ int64_t s_warp[32], s_sum;
  pdl_trigger();
  const int tid = threadIdx.x, rank = blockIdx.x, words = (c.B + 31) >> 5;
  for (int i = tid; i < 2 * words; i += kListThreads) bits[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kListThreads) {
    const int32_t r = req[i];
    if (r >= 0 && r < c.B) {
      const uint32_t m = 1u << (r & 31);
      if (atomicOr(&bits[r >> 5], m) & m) atomicOr(&bits[words + (r >> 5)], m);
    }
  }
  __syncthreads();
  auto entry = [&](int i) {
    Resize e = resize_entry(c, t, req, new_lens, i);
    if (e.ok && (bits[words + (e.r >> 5)] >> (e.r & 31)) & 1) e.ok = false;
    return e;
  };
  // nothing is released when no listed request shrinks
  int any = 0;
  for (int i = tid; i < n; i += kListThreads) {
    const Resize e = entry(i);
    any |= e.ok && e.new_pages < e.old_pages;
  }
  any = __syncthreads_or(any);
  pdl_wait();  // the releases have been made
  const int64_t count = clamp_count(__ldcg(t.free_count), c.num_pages, c.err, rank == 0 && tid == 0);
  const int64_t freed = any ? push_freed(c, t, bits + 2 * words, s_warp, &s_sum, rank, count) : 0;
  // every CTA has read the count, and no other CTA's counts are read any more
  tc::cluster_arrive();
  tc::cluster_wait();
  if (rank != 0) return;
  const int64_t avail = min(c.num_pages, count + freed);
  int64_t asked = 0, given = 0;
  for (int i0 = 0; i0 < n; i0 += kListThreads) {
    const int i = i0 + tid;
    Resize e;
    e.ok = false;
    e.r = 0;
    e.old_pages = e.new_pages = 0;
    if (i < n) e = entry(i);
    const int64_t need = e.ok && e.new_pages > e.old_pages ? e.new_pages - e.old_pages : 0;
    int64_t total;
    const int64_t upto = asked + block_sum_scan(need, s_warp, total);
    asked += total;
    const bool fits = need == 0 || upto <= avail;
    int64_t took;
    block_sum_scan(fits ? need : 0, s_warp, took);
    given += took;
    if (i < n) {
      work[2 * i] = need != 0 && fits ? static_cast<int32_t>(avail - 1 - (upto - need)) : -1;
      work[2 * i + 1] = static_cast<int32_t>(e.old_pages);
      if (!fits) flag(c.err, SMLA_DEVERR_PAGE);
      if (e.ok && fits) t.lens[e.r] = new_lens[i];
    }
  }
  if (tid == 0) *t.free_count = static_cast<int32_t>(avail - given);
}

// Third step: the growing requests' pages.
__global__ void __launch_bounds__(256) cache_pop_kernel(const CachePages c, const CacheTables t,
                                                        const int32_t* req,
                                                        const int32_t* new_lens, const int32_t* work) {
  const int i = blockIdx.x;
  pdl_wait();
  const int64_t pos = __ldcg(work + 2 * i);
  if (pos < 0) return;
  pop_pages(c, t, req[i], pos, __ldcg(work + 2 * i + 1), pages_of(new_lens[i], c.log2_page), blockIdx.y * 256 + threadIdx.x,
            int64_t(gridDim.y) * 256);
}

// A kernel that starts up while the one before it on the stream ends, and waits for it itself (pdl_wait). What
// another kernel may have written is read after that, by plain or L2 loads.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_cache_copy_pages(const CachePages& c, const int32_t* src, const int32_t* dst, int64_t n, int sms,
                                    cudaStream_t s) {
  // four pieces a thread in flight once that still leaves every SM a few CTAs
  const bool wide = n * c.L * c.page_bytes >= int64_t(sms) * 8 * 16384;
  const int piece = wide ? 16384 : 4096;
  const int64_t pieces = (c.page_bytes + piece - 1) / piece;
  const int64_t blocks = pieces * n * c.L;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (wide)
    return launch_behind(cache_copy_kernel<4>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, c, src, dst, n, static_cast<int>(pieces));
  return launch_behind(cache_copy_kernel<1>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, c, src, dst, n, static_cast<int>(pieces));
}

cudaError_t launch_cache_compact(const CachePages& c, const int32_t* page_table, const int32_t* starts,
                                 const int32_t* cu_keep, const int32_t* keep, int64_t n_keep, int32_t* new_lens, int sms,
                                 cudaStream_t s) {
  const int columns = c.index_keys ? 9 : c.row_bytes / 16;
  // enough CTAs for eight an SM, where the requests and layers alone are fewer
  const int64_t pairs = int64_t(c.B) * c.L;
  int64_t slices = (int64_t(sms) * 8 + pairs - 1) / pairs;
  if (slices > columns / 4) slices = columns / 4;
  if (slices < 1) slices = 1;
  // a few layers a CTA where there are more than four CTAs an SM
  int64_t group = pairs * slices / (int64_t(sms) * 4);
  if (group > 8) group = 8;
  if (group < 1) group = 1;
  const int64_t blocks = c.B * ((c.L + group - 1) / group) * slices;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  const int nc = columns, ns = static_cast<int>(slices), ng = static_cast<int>(group);
  // Short lists: fewer registers, four CTAs an SM instead of three. 64 requests, 32 layers, 16 kept rows each: 8.5 us
  // against 9.3; 24: 10.6 against 11.8; 28: 17.3 against 12.8.
  if (n_keep <= int64_t(c.B) * 24)
    return launch_behind(cache_compact_kernel<4>, grid, kCpThreads, 0, s, c, page_table, starts, cu_keep, keep, n_keep, new_lens, nc, ns, ng);
  return launch_behind(cache_compact_kernel<7>, grid, kCpThreads, 0, s, c, page_table, starts, cu_keep, keep, n_keep, new_lens, nc, ns, ng);
}

cudaError_t launch_cache_fork(const CachePages& c, const CacheTables& t, const int32_t* src_req, const int32_t* dst_req,
                              int32_t n, int32_t* fork_pages, int sms, cudaStream_t s) {
  const size_t smem = size_t(3) * ((c.B + 31) / 32) * 4;
  const cudaError_t e = launch_behind(cache_fork_plan_kernel, dim3(1), kListThreads, smem, s, c, t, src_req, dst_req, n, fork_pages);
  if (e != cudaSuccess) return e;
  const int64_t pieces = ((c.page_bytes + 8191) / 8192) * c.L;
  int64_t y = (int64_t(sms) * 8 + n - 1) / n;
  if (y > pieces) y = pieces;
  if (y > 65535) y = 65535;
  return launch_behind(cache_fork_kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(y)), 256, 0, s, c, t, src_req,
                       dst_req, (const int32_t*)fork_pages);
}

cudaError_t launch_cache_resize(const CachePages& c, const CacheTables& t, const int32_t* req, const int32_t* new_lens,
                                int32_t n, int32_t* work, int sms, cudaStream_t s) {
  const size_t smem = size_t(2) * ((c.B + 31) / 32) * 4 + 2 * kMarkWords * 4;
  // One launch while the cluster has few table entries to walk (the lengths are known on the device only: all
  // of the listed rows count). Two calls, one launch each against three: at 32,000 entries growing 14.4 us
  // against 20.8, freeing everything and taking it again 20.4 against 20.5; at 128,000 15.4 against 24.3 and 29.3
  // against 26.3.
  if (n <= kListThreads && int64_t(n) * c.stride <= kResizeOneLaunch) {
    return launch_behind(cache_resize_kernel, dim3(kPushCtas), kListThreads, smem, s, c, t, req, new_lens, n);
  }
  int64_t y = (int64_t(sms) * 4 + n - 1) / n;
  if (y > (c.stride + 255) / 256) y = (c.stride + 255) / 256;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(y));
  cudaError_t e = launch_behind(cache_release_kernel, grid, 256, 0, s, c, t, req, new_lens, n);
  if (e == cudaSuccess) e = launch_behind(cache_push_kernel, dim3(kPushCtas), kListThreads, smem, s, c, t, req, new_lens, n, work);
  if (e == cudaSuccess) e = launch_behind(cache_pop_kernel, grid, 256, 0, s, c, t, req, new_lens, (const int32_t*)work);
  return e;
}

}  // namespace smla
