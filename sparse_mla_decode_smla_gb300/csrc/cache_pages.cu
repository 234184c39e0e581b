// Page operators of the paged cache: copying pages, compacting kept rows in place, forking
// requests with shared pages, and growing or shrinking requests over a free list of pages.
// All of them move bytes or whole numbers: nothing is computed, every result is exact, and
// none depends on the order in which threads run.
#include "cache_pages.h"
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
__global__ void __launch_bounds__(256) cache_copy_kernel(const CachePages c, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, int64_t n, int pieces) {
  const int64_t b = blockIdx.x;
  const int piece = static_cast<int>(b % pieces);
  const int64_t li = b / pieces, i = li % n, layer = li / n;
  const int32_t s = __ldg(src + i), d = __ldg(dst + i);
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
constexpr int kCpItems = 8;                          // 16-byte pieces a thread holds
constexpr int kCpRows = 512;                         // rows of a chunk at most
constexpr int kCpPieces = kCpThreads * kCpItems;     // pieces of a chunk at most

// Row starts[r] + keep[k] -> row starts[r] + k for each kept row k of request r, in place, in
// every layer. One CTA takes one (layer, request, range of 16-byte columns) and walks the kept
// rows in ascending chunks: it loads a chunk's pieces into registers, waits for the whole CTA,
// then stores them. With keep strictly ascending, keep[k] >= k, so row k of the result is a
// source of rows <= k only: those of earlier chunks, already loaded, and of this one, loaded
// before the barrier. No row that a later chunk reads is written early, and no other CTA
// touches these columns of this request.
__global__ void __launch_bounds__(kCpThreads) cache_compact_kernel(
    const CachePages c, const int32_t* __restrict__ page_table, const int32_t* __restrict__ starts,
    const int32_t* __restrict__ cu_keep, const int32_t* __restrict__ keep, int64_t n_keep, int32_t* new_lens, int columns,
    int slices) {
  __shared__ int64_t s_src[kCpRows], s_dst[kCpRows];  // byte offsets of the rows; -1: not moved
  const int tid = threadIdx.x;
  const int slice = blockIdx.x % slices;
  const int64_t rest = blockIdx.x / slices;
  const int r = static_cast<int>(rest % c.B), layer = static_cast<int>(rest / c.B);
  const bool first = slice == 0 && layer == 0;
  const int32_t start = __ldg(starts + r), a = __ldg(cu_keep + r), b = __ldg(cu_keep + r + 1);
  if (start < 0 || a < 0 || b < a || b > n_keep) {
    if (first && tid == 0) flag(c.err, SMLA_DEVERR_INDEX);
    return;
  }
  const int count = b - a;
  if (first && tid == 0 && new_lens) new_lens[r] = start + count;
  const int c0 = int(int64_t(columns) * slice / slices), c1 = int(int64_t(columns) * (slice + 1) / slices);
  const int cols = c1 - c0;
  const int rows = min(kCpRows, kCpPieces / cols);
  uint8_t* base = c.kv + int64_t(layer) * c.layer_stride;
  const int32_t* pt = page_table + int64_t(r) * c.stride;
  const int P = 1 << c.log2_page;
  // byte offset of a slot's row (index keys: of its codes), -1 where the slot has no page
  auto row_at = [&](int64_t slot) -> int64_t {
    const int64_t k = slot >> c.log2_page;
    if (k >= c.stride) {
      if (first) flag(c.err, SMLA_DEVERR_INDEX);
      return -1;
    }
    const int32_t page = __ldg(pt + k);
    if (page < 0 || page >= c.num_pages) {
      if (first) flag(c.err, SMLA_DEVERR_PAGE);
      return -1;
    }
    return int64_t(page) * c.page_bytes + (slot & (P - 1)) * c.row_bytes;
  };
  // the scale of an index key, from the offset of its codes
  auto scale_at = [&](int64_t off) -> int64_t {
    const int64_t page = off / c.page_bytes, in = off - page * c.page_bytes;
    return page * c.page_bytes + int64_t(P) * 128 + (in >> 7) * 4;
  };
  for (int k0 = 0; k0 < count; k0 += rows) {
    const int m = min(rows, count - k0);
    for (int i = tid; i < m; i += kCpThreads) {
      const int k = k0 + i;
      const int32_t from = __ldg(keep + a + k);
      const int32_t before = k ? __ldg(keep + a + k - 1) : -1;
      int64_t so = -1, dp = -1;
      if (from < k || from <= before) {
        if (first) flag(c.err, SMLA_DEVERR_INDEX);
      } else if (from != k) {
        so = row_at(int64_t(start) + from);
        dp = row_at(int64_t(start) + k);
        if (dp < 0) so = -1;
      }
      s_src[i] = so;
      s_dst[i] = dp;
    }
    __syncthreads();
    uint4 v[kCpItems];
    const int items = m * cols;
#pragma unroll
    for (int j = 0; j < kCpItems; ++j) {
      const int it = tid + j * kCpThreads;
      if (it >= items) continue;
      const int i = it / cols, col = c0 + it - i * cols;
      const int64_t so = s_src[i];
      if (so < 0) continue;
      if (c.index_keys && col == 8)
        v[j].x = *reinterpret_cast<const uint32_t*>(base + scale_at(so));
      else
        v[j] = *reinterpret_cast<const uint4*>(base + so + 16 * col);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCpItems; ++j) {
      const int it = tid + j * kCpThreads;
      if (it >= items) continue;
      const int i = it / cols, col = c0 + it - i * cols;
      if (s_src[i] < 0) continue;
      const int64_t dp = s_dst[i];
      if (c.index_keys && col == 8)
        *reinterpret_cast<uint32_t*>(base + scale_at(dp)) = v[j].x;
      else
        *reinterpret_cast<uint4*>(base + dp + 16 * col) = v[j];
    }
    __syncthreads();  // s_src and s_dst are rewritten
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
// (SMLA_DEVERR_PAGE) when fewer free pages are left than it and those before it need.
// fork_pages[i]: the page taken, -1 where none was needed, -2 for a refused fork.
__global__ void __launch_bounds__(kListThreads) cache_fork_plan_kernel(const CachePages c, const CacheTables t,
                                                                       const int32_t* __restrict__ src_req,
                                                                       const int32_t* __restrict__ dst_req, int32_t n,
                                                                       int32_t* fork_pages) {
  extern __shared__ uint32_t bits[];  // targets seen, targets seen twice, sources: a bit a request
  __shared__ int64_t s_warp[32];
  const int tid = threadIdx.x, words = (c.B + 31) >> 5;
  for (int i = tid; i < 3 * words; i += kListThreads) bits[i] = 0;
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
    bool ok = false, need = false;
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
      need = ok && (len & ((1 << c.log2_page) - 1)) != 0;
    }
    int64_t total;
    const int64_t at = used + block_sum_scan(need ? 1 : 0, s_warp, total);  // needs up to this one
    used += total;
    if (i < n) {
      int32_t got = ok ? -1 : -2;
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
                                                         const int32_t* __restrict__ src_req,
                                                         const int32_t* __restrict__ dst_req,
                                                         const int32_t* __restrict__ fork_pages) {
  const int i = blockIdx.x, y = blockIdx.y, ny = gridDim.y, tid = threadIdx.x;
  const int32_t got = fork_pages[i];
  if (got == -2) return;
  const int32_t s = src_req[i], d = dst_req[i];
  const int64_t len = t.lens[s];
  const int full = static_cast<int>(len >> c.log2_page);
  const int part = static_cast<int>(len & ((1 << c.log2_page) - 1));
  const int32_t* from = t.page_table + int64_t(s) * c.stride;
  int32_t* to = t.page_table + int64_t(d) * c.stride;
  for (int k = y * 256 + tid; k < full; k += ny * 256) {
    const int32_t page = from[k];
    to[k] = page;
    if (page >= 0 && page < c.num_pages)
      atomicAdd(t.refs + page, 1);
    else
      flag(c.err, SMLA_DEVERR_PAGE);
  }
  if (part == 0) return;
  const int32_t last = from[full];
  if (last < 0 || last >= c.num_pages) {
    if (y == 0 && tid == 0) flag(c.err, SMLA_DEVERR_PAGE);
    return;
  }
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

// Whether entry i of a resize list is valid; its request's old and new page counts. Uniform over
// the CTA. A request listed twice is refused both times.
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

// First step of a resize: the pages beyond the new length leave the table and lose a holder.
// CTA (i, y) takes every y-th group of request i's entries.
__global__ void __launch_bounds__(256) cache_release_kernel(const CachePages c, const CacheTables t,
                                                            const int32_t* __restrict__ req,
                                                            const int32_t* __restrict__ new_lens, int32_t n) {
  const int i = blockIdx.x;
  const Resize e = resize_entry(c, t, req, new_lens, i);
  int twice = 0;
  for (int j = threadIdx.x; j < n; j += 256) twice |= j != i && req[j] == e.r;
  twice = __syncthreads_or(twice);
  if (!e.ok || twice) {
    if (threadIdx.x == 0) flag(c.err, SMLA_DEVERR_INDEX);
    return;
  }
  int32_t* row = t.page_table + int64_t(e.r) * c.stride;
  for (int64_t k = e.new_pages + blockIdx.y * 256 + threadIdx.x; k < e.old_pages; k += int64_t(gridDim.y) * 256) {
    const int32_t page = row[k];
    row[k] = -1;
    if (page < 0 || page >= c.num_pages) {
      flag(c.err, SMLA_DEVERR_PAGE);
      continue;
    }
    const int32_t had = atomicSub(t.refs + page, 1);
    if (had == 1) {
      atomicOr(t.refs + page, kRefFreed);
    } else if ((had & ~kRefFreed) <= 0) {  // more holders let go than there were
      atomicAdd(t.refs + page, 1);
      flag(c.err, SMLA_DEVERR_PAGE);
    }
  }
}

constexpr int kPushCtas = 8;

// Second step, one cluster of eight CTAs: the freed pages go to the end of the free list in
// ascending order (each CTA counts its range of pages, the counts meet over distributed shared
// memory), then the first CTA gives each growing request its place in the list, in the order of
// the call. A request is refused (SMLA_DEVERR_PAGE) when fewer pages are free than it and those
// before it ask for. work[2i]: the list position of the request's first page, -1 where it takes
// none; work[2i+1]: its old page count.
__global__ void __cluster_dims__(kPushCtas, 1, 1) __launch_bounds__(kListThreads)
    cache_push_kernel(const CachePages c, const CacheTables t, const int32_t* __restrict__ req,
                      const int32_t* __restrict__ new_lens, int32_t n, int32_t* work) {
  extern __shared__ uint32_t bits[];  // requests listed, requests listed twice
  __shared__ int64_t s_warp[32];
  __shared__ int64_t s_mine;
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
  // nothing was released when no listed request shrinks
  int any = 0;
  for (int i = tid; i < n; i += kListThreads) {
    const Resize e = entry(i);
    any |= e.ok && e.new_pages < e.old_pages;
  }
  any = __syncthreads_or(any);
  const int64_t count = clamp_count(*t.free_count, c.num_pages, c.err, rank == 0 && tid == 0);
  int64_t freed = 0;
  if (any) {
    const int64_t per = ((c.num_pages + kPushCtas - 1) / kPushCtas + 3) & ~int64_t(3);
    const int64_t lo = min(c.num_pages, per * rank), hi = min(c.num_pages, lo + per);
    int64_t mine = 0;
    for (int64_t p = lo + tid; p < hi; p += kListThreads) mine += (__ldcg(t.refs + p) & kRefFreed) != 0;
    int64_t total;
    block_sum_scan(mine, s_warp, total);
    if (tid == 0) s_mine = total;
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    int64_t at = count;
    for (int k = 0; k < kPushCtas; ++k) {
      int64_t v;
      asm volatile("ld.shared::cluster.b64 %0, [%1];"
                   : "=l"(v)
                   : "r"(tc::mapa(static_cast<uint32_t>(__cvta_generic_to_shared(&s_mine)), k)));
      freed += v;
      if (k < rank) at += v;
    }
    for (int64_t p0 = lo; p0 < hi; p0 += kListThreads) {
      const int64_t p = p0 + tid;
      const int32_t v = p < hi ? __ldcg(t.refs + p) : 0;
      const bool f = (v & kRefFreed) != 0;
      const int64_t before = at + block_sum_scan(f ? 1 : 0, s_warp, total) - 1;
      at += total;
      if (f) {
        t.refs[p] = v & ~kRefFreed;
        if (before < c.num_pages)
          t.free_list[before] = static_cast<int32_t>(p);
        else
          flag(c.err, SMLA_DEVERR_PAGE);
      }
    }
  }
  // every CTA has read the others' counts and the old lengths, and its pushes are visible
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

// Third step: each growing request takes its pages off the list, the last one first.
__global__ void __launch_bounds__(256) cache_pop_kernel(const CachePages c, const CacheTables t,
                                                        const int32_t* __restrict__ req,
                                                        const int32_t* __restrict__ new_lens,
                                                        const int32_t* __restrict__ work) {
  const int i = blockIdx.x;
  const int64_t pos = work[2 * i];
  if (pos < 0) return;
  const int64_t old_pages = work[2 * i + 1], new_pages = pages_of(new_lens[i], c.log2_page);
  int32_t* row = t.page_table + int64_t(req[i]) * c.stride;
  for (int64_t k = old_pages + blockIdx.y * 256 + threadIdx.x; k < new_pages; k += int64_t(gridDim.y) * 256) {
    const int64_t at = pos - (k - old_pages);
    const int32_t page = t.free_list[at];
    t.free_list[at] = -1;
    row[k] = page;
    if (page >= 0 && page < c.num_pages)
      t.refs[page] = 1;
    else
      flag(c.err, SMLA_DEVERR_PAGE);
  }
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
    cache_copy_kernel<4><<<static_cast<unsigned>(blocks), 256, 0, s>>>(c, src, dst, n, static_cast<int>(pieces));
  else
    cache_copy_kernel<1><<<static_cast<unsigned>(blocks), 256, 0, s>>>(c, src, dst, n, static_cast<int>(pieces));
  return cudaGetLastError();
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
  const int64_t blocks = pairs * slices;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cache_compact_kernel<<<static_cast<unsigned>(blocks), kCpThreads, 0, s>>>(
      c, page_table, starts, cu_keep, keep, n_keep, new_lens, columns, static_cast<int>(slices));
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CachePages& c, const CacheTables& t, const int32_t* src_req, const int32_t* dst_req,
                              int32_t n, int32_t* fork_pages, int sms, cudaStream_t s) {
  const size_t smem = size_t(3) * ((c.B + 31) / 32) * 4;
  cache_fork_plan_kernel<<<1, kListThreads, smem, s>>>(c, t, src_req, dst_req, n, fork_pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t pieces = ((c.page_bytes + 8191) / 8192) * c.L;
  int64_t y = (int64_t(sms) * 8 + n - 1) / n;
  if (y > pieces) y = pieces;
  if (y > 65535) y = 65535;
  cache_fork_kernel<<<dim3(static_cast<unsigned>(n), static_cast<unsigned>(y)), 256, 0, s>>>(c, t, src_req, dst_req,
                                                                                           fork_pages);
  return cudaGetLastError();
}

cudaError_t launch_cache_resize(const CachePages& c, const CacheTables& t, const int32_t* req, const int32_t* new_lens,
                                int32_t n, int32_t* work, int sms, cudaStream_t s) {
  int64_t y = (int64_t(sms) * 4 + n - 1) / n;
  if (y > (c.stride + 255) / 256) y = (c.stride + 255) / 256;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(y));
  cache_release_kernel<<<grid, 256, 0, s>>>(c, t, req, new_lens, n);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t smem = size_t(2) * ((c.B + 31) / 32) * 4;
  cache_push_kernel<<<kPushCtas, kListThreads, smem, s>>>(c, t, req, new_lens, n, work);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_pop_kernel<<<grid, 256, 0, s>>>(c, t, req, new_lens, work);
  return cudaGetLastError();
}

}  // namespace smla
