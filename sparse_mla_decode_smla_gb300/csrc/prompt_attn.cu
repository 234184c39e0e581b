// Attention of packed prompts over per-head keys and values (smla_prompt_attention), on the 5th-generation tensor cores.
//
//   s_ij = sm_scale (<q_i[0:128], k_j> + <q_i[128:192], k_rope_j>),  x_ij = [cap tanh](s_ij) - slope |p_i - j|,
//   out_i = sum_j e^{x_ij} v_j / (sum_j e^{x_ij} + e^{sink}) over the keys j < lim_i:
// every mask here (the other documents, the future, a visible prefix, a shorter context) leaves a row the first lim_i
// keys of its request, so that a number a row is all that the kernel knows of masks.
//
// Work. An item is 256 rows of one request and kv head, in two row tiles of 128: consecutive tokens, with as many query
// heads of the kv head as a power of two allows beside one another (a single token's grouped heads share a tile). Its
// keys come in tiles of 128. The CTAs, one an SM, share the items in one of two ways, from the lengths on the device:
//  * items that are short beside an SM's share are taken off a counter, a request's last rows (most keys) first, heads
//    whose keys fit L2 together at a time;
//  * else the key tiles of all items, in order, are cut into equal runs, one a CTA. An item that a run's end cuts leaves its
//    parts in the workspace, two a CTA at most; the piece that ends last joins them, in the order of the keys.
// Up to 32 requests are laid out by a warp of every CTA, more by a small kernel before.
//
// A key tile on one SM: S = Q K^T (12 MMAs of 128 x 128 x 16 a row tile), the weights P = 2^(x - m) in BF16 written over
// S in tensor memory, O += P V (8 MMAs, P from tensor memory). The two row tiles alternate: one's softmax runs while the
// tensor cores work for the other. m moves only when a row's maximum grows by more than 2^16 (in a lone row tile whenever it
// grows), so O is rescaled rarely, by the softmax threads themselves; by the time S of a tile is there, PV of the tile before
// is complete.
//
// What bounds it: one 8191-token prompt of 32 heads takes 468 to 483 us from GPU to GPU, 1,420 to 1,470 TFLOP/s and 75 to 77 % of
// the measured matrix rate, the tensor pipe busy for 67 % of the time. A row tile's chain is scores, softmax, P, then PV and the next
// scores; tensor memory (two S, two O) has no room for a third row tile's, so a tile's softmax, about 2,500 clocks, is longer than
// the 1,280 that the other's MMAs cover. With a cap the chain is longer still (2 x 1024 tokens over 12k keys, 16 heads, where the
// MMAs' rate would allow 96 us: 183 us with scores small beside the cap, 303 with ones on both sides of 0.6 of it), and no pipe
// is full either: issue slots 40 %, FMA 36 %, XU 17 %, tensor 43 %. Single tokens are bound by memory: 32 of them over 0.7k to
// 16k keys, 8 kv heads: 159 us, 90 % of the bandwidth; 250 to 265 us with scores past 0.6 of a cap.
//
// P in BF16 is off by 2^-8 of each weight at most, independently of the others; the sums of weights are of the fp32 values.
//
// What is hidden never counts: its score is replaced, and in tiles that not all rows see whole, value rows past the last
// key become zeros and a value row with a non-finite element does too and is remembered, so that the rows that see it
// become NaN and the others never meet it.
//
// Per CTA (384 threads): warps 0-3 and 4-7 softmax and epilogue of a row tile each (a thread a row), 8 MMA issue, 9 items
// and TMA loads, 10-11 the check of value tiles. Q takes 96 KB, 16 KB units of keys and values share a ring of eight.
// Every wait is bounded in time; one that gives up sets SMLA_DEVERR_TIMEOUT.
#include <math_constants.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "prompt.h"
#include "tcgen05.cuh"

namespace smla {
namespace {

constexpr int kPaM = 128, kPaN = 128;      // rows of a row tile, keys of a key tile
constexpr int kPaRows = 2 * kPaM;          // rows of an item
constexpr int kPaUnit = 16384;             // bytes of a ring unit: 128 keys x 64 dims, or 64 values x 128 dims
constexpr int kPaThreads = 384;
constexpr int kPaMmaWarp = 8, kPaLoadWarp = 9, kPaGuardWarp = 10, kPaGuards = 2;
constexpr int kPaTiles = 4;                // key (value) tiles in the ring at most: 3
// m moves when a row's maximum exceeds it by more than this (log2 units): weights stay below 2^16, which neither BF16 nor the
// fp32 sums notice, and with a bias, where scores grow from tile to tile, it moves less often than with 2^8
constexpr float kPaRescale = 16.f;
// With a bias m moves this far beyond the maximum, so that it moves less often (8191 tokens of 32 heads: 1.7 % less than with 0);
// weights around 2^-40 are as exact as others.
constexpr float kPaAhead = 40.f;
constexpr int kPaMinTiles = 8;             // key tiles of a run, and of a piece but the odd one, at least
constexpr int kPaItemCost = 3;             // an item's own work, in key tiles
constexpr int kPaSlotFloats = kPaRows * 128 + kPaRows * 2;  // a piece's part: O, then (m, l) of each row

struct PaItem {
  int q0;       // row of q of the request's first token
  int nq, nk;   // tokens and keys of the request
  int k0;       // row of k of the request's first key
  int tok0;     // first token of the item
  int head0;    // first query head
  int kvh;      // kv head
  int kt0;      // first key tile of this piece
  int n[2];     // key tiles of this piece that each row tile sees
  int prefix;   // keys that every token sees
  int pieces;   // pieces of the item (1: not cut)
  int cta0;     // the CTA of the first one: the others follow it
  int piece;
  int last;     // no more items
  int paired;   // one row tile: the key tiles alternate between the two halves of the CTA
};

template <int ROPE>
struct PaLay {
  static constexpr int qk_units = 2 + ROPE / 64;  // units of a key tile and of a row tile of q
  static constexpr int ring = ROPE ? 8 : 10;
  static constexpr size_t q = 0;
  static constexpr size_t units = q + 2 * qk_units * size_t(kPaUnit);
  static constexpr size_t item = units + ring * size_t(kPaUnit);
  static constexpr size_t ml = item + 2 * sizeof(PaItem);  // (m, l) of a paired item's rows, from either half
  static constexpr size_t bad = ml + 2 * kPaM * 8;
  static constexpr size_t flag = bad + 8;
  static constexpr size_t tmem = flag + 8;
  static constexpr size_t bars = tmem + 16;
  static constexpr size_t bytes = bars + 48 * 8;
  static_assert(bytes <= 232448 && bars % 8 == 0 && units % 1024 == 0, "shared memory");
};
enum {
  A_UFREE = 0,             // [unit]
  A_QFULL = A_UFREE + 10,  // [row tile], and so the next ones
  A_QFREE = A_QFULL + 2,
  A_S = A_QFREE + 2,
  A_P = A_S + 2,           // [row tile][half of the keys]
  A_O = A_P + 4,
  A_ITEM = A_O + 2,        // [item parity]
  A_TAKEN = A_ITEM + 2,
  A_KFULL = A_TAKEN + 2,   // [tile % kPaTiles]: keys, values, values that the guards look at, those after they have
  A_VFULL = A_KFULL + kPaTiles,
  A_GFULL = A_VFULL + kPaTiles,
  A_READY = A_GFULL + kPaTiles,
  A_HALF = A_READY + kPaTiles,  // [row tile]: its four warps meet, where an item is cut
  A_PAIR = A_HALF + 2,          // the eight softmax warps meet, in paired items
  A_DRAIN,
  A_COUNT
};
static_assert(A_COUNT <= 48, "barriers");

// ---------------------------------------------------------------- the plan

struct PaReq {
  int q0, nq, k0, nk, prefix, blocks;
};

// 1: a request with tokens, 0: without, -1: one that does not fit the description
__device__ __forceinline__ int pa_request(const PromptArgs& p, int r, PaReq& q) {
  const int64_t a = p.cu_q[r], b = p.cu_q[r + 1], c = p.cu_k[r], d = p.cu_k[r + 1];
  q = PaReq{};
  if (a < 0 || b < a || b > p.T || c < 0 || d < c || d > p.N) return -1;
  q.q0 = static_cast<int>(a);
  q.nq = static_cast<int>(b - a);
  q.k0 = static_cast<int>(c);
  q.nk = static_cast<int>(d - c);
  q.prefix = p.prefix ? min(max(p.prefix[r], 0), q.nk) : 0;
  const int tb = kPaRows >> p.log2_pack;
  q.blocks = (q.nq + tb - 1) / tb;
  return q.nq > 0;
}
// the keys that token i of a request sees
__device__ __forceinline__ int pa_lim(int causal, int nq, int nk, int prefix, int i) {
  return causal ? min(max(nk - nq + i + 1, prefix), nk) : nk;
}
__device__ __forceinline__ int pa_tiles(const PromptArgs& p, const PaReq& q, int token) {
  return (max(pa_lim(p.causal, q.nq, q.nk, q.prefix, token), 0) + kPaN - 1) / kPaN;
}

struct PaHead {  // the start of the workspace
  int32_t err, claim, done, longest;  // device error word; next item; CTAs that have ended; key tiles of the longest item
};
struct PaTab {  // key tiles and items before a request, of all its heads; [B] holds the totals
  int64_t tiles;
  int32_t items, pad;
};
__device__ __forceinline__ PaTab* pa_table(const PromptArgs& p) { return reinterpret_cast<PaTab*>(p.table); }

constexpr int kPlanThreads = 256;
constexpr int kPlanWarp = 32;  // requests that a warp lays out itself

// The key tiles of every lane's request over all its blocks of rows, for one group of heads beside one another (by a whole
// warp; a request without tokens has no blocks). Requests of many blocks are added up by all lanes together.
__device__ __forceinline__ int64_t pa_sum(const PromptArgs& p, const PaReq& mine) {
  const int tb = kPaRows >> p.log2_pack, lane = threadIdx.x & 31;
  int64_t n = 0;
  const bool many = mine.blocks > 32;
  if (!many)
    for (int b = 0; b < mine.blocks; ++b) n += pa_tiles(p, mine, min((b + 1) * tb, mine.nq) - 1);
  for (uint32_t left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
    const int r = __ffs(left) - 1;
    PaReq q = {};
    q.nq = __shfl_sync(0xffffffffu, mine.nq, r);
    q.nk = __shfl_sync(0xffffffffu, mine.nk, r);
    q.prefix = __shfl_sync(0xffffffffu, mine.prefix, r);
    q.blocks = __shfl_sync(0xffffffffu, mine.blocks, r);
    int64_t sum = 0;
    for (int b = lane; b < q.blocks; b += 32) sum += pa_tiles(p, q, static_cast<int>(min(int64_t(b + 1) * tb, int64_t(q.nq))) - 1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == r) n = sum;
  }
  return n;
}

// A request that starts before the last token of an earlier one would write its rows too, in no order (and offsets that go to and fro
// would ask for work without bound): it is left out. By a whole warp, a request with its `ok` of pa_request a lane: the largest end of
// the requests with tokens before the lane's, and of all of them.
__device__ __forceinline__ int pa_ends(const PaReq& q, int ok, int& all) {
  int x = ok > 0 ? q.q0 + q.nq : 0;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int a = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x = max(x, a);
  }
  all = __shfl_sync(0xffffffffu, x, 31);
  x = __shfl_up_sync(0xffffffffu, x, 1);
  return threadIdx.x & 31 ? x : 0;
}

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptArgs p) {
  __shared__ PaTab scan[kPlanThreads / 32];
  __shared__ int ends[kPlanThreads / 32];
  __shared__ int most[kPlanThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, G = p.H >> p.log2_pack;
  PaHead* head = reinterpret_cast<PaHead*>(p.ws);
  PaTab before = {0, 0, 0};  // of the requests before this round's
  int longest = 0, end = 0;
  for (int r0 = 0; r0 < p.B; r0 += kPlanThreads) {
    const int r = r0 + tid;
    PaTab v = {0, 0, 0};
    PaReq q = {};
    int ok = r < p.B ? pa_request(p, r, q) : 0, all;
    const int in_warp = pa_ends(q, ok, all);
    if (lane == 0) ends[tid >> 5] = all;
    __syncthreads();
    int taken = end;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < (tid >> 5)) taken = max(taken, ends[i]);
      end = max(end, ends[i]);
    }
    if (ok > 0 && q.q0 < max(taken, in_warp)) {
      ok = -1;
      q = PaReq{};
    }
    if (ok < 0) atomicOr(&head->err, SMLA_DEVERR_INDEX);
    const int64_t tiles = pa_sum(p, q);
    if (ok > 0) {
      v.tiles = tiles * G;
      v.items = q.blocks * G;
      longest = max(longest, pa_tiles(p, q, q.nq - 1));
    }
    PaTab x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t a = __shfl_up_sync(0xffffffffu, x.tiles, o);
      const int b = __shfl_up_sync(0xffffffffu, x.items, o);
      if (lane >= o) {
        x.tiles += a;
        x.items += b;
      }
    }
    __syncthreads();
    if (lane == 31) scan[tid >> 5] = x;
    __syncthreads();
    PaTab mine = before;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < (tid >> 5)) {
        mine.tiles += scan[i].tiles;
        mine.items += scan[i].items;
      }
      before.tiles += scan[i].tiles;
      before.items += scan[i].items;
    }
    if (r < p.B) pa_table(p)[r] = PaTab{mine.tiles + x.tiles - v.tiles, mine.items + x.items - v.items, 0};
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) most[tid >> 5] = longest;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kPlanThreads / 32; ++i) longest = max(longest, most[i]);
    head->longest = longest;
    pa_table(p)[p.B] = before;
  }
}

// What a warp knows of the batch, and its CTA's way through it. Lane r holds request r's line where there are few.
struct PaWalk {
  PaTab tab;       // few requests: this lane's line
  PaTab total;
  int64_t per;     // runs: their length; 0: items come off the counter
  int cost;        // an item's own, in key tiles
  // runs: the next item, how much of it is done, and where the run ends
  int64_t x;       // the item's start
  int r, hg, block, from;
  int64_t x_end;   // start of the item that the run ends in
  int end;         // key tiles of that item that belong to the run
  int cta;
};
constexpr int kPaAll = 0x7fffffff;

__device__ __forceinline__ PaTab pa_line(const PromptArgs& p, const PaWalk& w, int r) {
  PaTab t;
  if (p.B <= kPlanWarp) {
    t.tiles = __shfl_sync(0xffffffffu, w.tab.tiles, r);
    t.items = __shfl_sync(0xffffffffu, w.tab.items, r);
  } else {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(pa_table(p) + r));
    t.tiles = int64_t(uint32_t(v.x)) | int64_t(v.y) << 32;
    t.items = v.z;
  }
  return t;
}
// The last request whose tiles * a + items * b before it are no more than x.
__device__ __forceinline__ int pa_find(const PromptArgs& p, const PaWalk& w, int a, int b, int64_t x) {
  const int lane = threadIdx.x & 31;
  if (p.B <= kPlanWarp) {
    const uint32_t le = __ballot_sync(0xffffffffu, lane < p.B && w.tab.tiles * a + int64_t(w.tab.items) * b <= x);
    return 31 - __clz(le);
  }
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    bool ok = false;
    if (at < hi) {
      const int4 v = __ldcg(reinterpret_cast<const int4*>(pa_table(p) + at));
      ok = (int64_t(uint32_t(v.x)) | int64_t(v.y) << 32) * a + int64_t(v.z) * b <= x;
    }
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, ok));  // lane 0 holds
    hi = min(hi, lo + (k + 1) * step);
    lo += k * step;
  }
  return lo;
}
// How many of an item's n key tiles lie before a cut at offset o of its n + cost: short pieces at the ends are avoided.
__device__ __forceinline__ int pa_cut(int n, int cost, int o) {
  if (n < 2 * kPaMinTiles) return 2 * o < n + cost ? 0 : kPaAll;
  if (o < kPaMinTiles) return o < kPaMinTiles / 2 ? 0 : kPaMinTiles;
  if (o > n - kPaMinTiles) return o > n - kPaMinTiles / 2 ? kPaAll : n - kPaMinTiles;
  return o;
}
__device__ __forceinline__ int pa_block_tiles(const PromptArgs& p, const PaReq& q, int block) {
  return pa_tiles(p, q, min((block + 1) * (kPaRows >> p.log2_pack), q.nq) - 1);
}
// The item that x lies in (its request, heads and block), its start, and the cut there.
__device__ __forceinline__ int pa_locate(const PromptArgs& p, const PaWalk& w, int64_t x, int& r, int& hg, int& block, int64_t& start) {
  const int lane = threadIdx.x & 31, G = p.H >> p.log2_pack;
  r = pa_find(p, w, 1, w.cost, x);
  const PaTab t = pa_line(p, w, r);
  const PaTab next = r + 1 < p.B ? pa_line(p, w, r + 1) : w.total;
  PaReq q;
  pa_request(p, r, q);
  const int64_t head = (next.tiles - t.tiles + int64_t(next.items - t.items) * w.cost) / G;  // one group of heads
  int64_t at = x - t.tiles - int64_t(t.items) * w.cost;
  hg = static_cast<int>(at / head);
  at -= hg * head;
  start = x - at;
  for (int b0 = 0;; b0 += 32) {  // blocks, 32 at a time
    const int b = b0 + lane, v = b < q.blocks ? pa_block_tiles(p, q, b) + w.cost : 0;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    if (at < all) {
      const int k = __ffs(__ballot_sync(0xffffffffu, sum > at)) - 1;
      const int mine = __shfl_sync(0xffffffffu, sum - v, k), n = __shfl_sync(0xffffffffu, v, k) - w.cost;
      block = b0 + k;
      start += mine;
      return pa_cut(n, w.cost, static_cast<int>(at) - mine);
    }
    at -= all;
    start += all;
    if (b0 + 32 >= q.blocks) break;  // not reached
  }
  block = 0;
  return kPaAll;
}
__device__ __forceinline__ void pa_next(const PromptArgs& p, PaWalk& w, const PaReq& q) {  // the item behind this one
  w.x += pa_block_tiles(p, q, w.block) + w.cost;
  w.from = 0;
  if (++w.block < q.blocks) return;
  w.block = 0;
  if (++w.hg < (p.H >> p.log2_pack)) return;
  w.hg = 0;
  do ++w.r;  // past requests without items
  while (w.r < p.B && pa_line(p, w, w.r).items == (w.r + 1 < p.B ? pa_line(p, w, w.r + 1) : w.total).items);
}

// Lays the batch out: by a whole warp.
__device__ __forceinline__ void pa_plan(const PromptArgs& p, PaWalk& w) {
  const int lane = threadIdx.x & 31, G = p.H >> p.log2_pack;
  PaHead* head = reinterpret_cast<PaHead*>(p.ws);
  int longest = 0;
  if (p.B <= kPlanWarp) {
    PaReq q = {};
    int ok = lane < p.B ? pa_request(p, lane, q) : 0;
    if (__any_sync(0xffffffffu, ok < 0)) {  // (requests overlap only where an offset goes back)
      int all;
      if (q.q0 < pa_ends(q, ok, all) && ok > 0) {
        ok = -1;
        q = PaReq{};
      }
    }
    if (ok < 0 && blockIdx.x == 0) atomicOr(&head->err, SMLA_DEVERR_INDEX);
    PaTab v = {0, 0, 0};
    const int64_t tiles = pa_sum(p, q);
    if (ok > 0) {
      v.tiles = tiles * G;
      v.items = q.blocks * G;
      longest = pa_tiles(p, q, q.nq - 1);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    w.tab = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t a = __shfl_up_sync(0xffffffffu, w.tab.tiles, o);
      const int b = __shfl_up_sync(0xffffffffu, w.tab.items, o);
      if (lane >= o) {
        w.tab.tiles += a;
        w.tab.items += b;
      }
    }
    w.total.tiles = __shfl_sync(0xffffffffu, w.tab.tiles, 31);
    w.total.items = __shfl_sync(0xffffffffu, w.tab.items, 31);
    w.tab.tiles -= v.tiles;
    w.tab.items -= v.items;
  } else {
    w.total = pa_line(p, w, p.B);
    longest = __ldcg(&head->longest);
  }
  w.per = 0;
  w.cost = kPaItemCost;
  // Runs where the longest item is over a third of an SM's share (8191 tokens of 32 heads, 0.29 of it, take 2 % longer in
  // runs than off the counter; chunks of 2 x 1024 over 12k keys, 16 heads, 20 % longer off it than in runs).
  if (int64_t(longest) * 3 * gridDim.x <= w.total.tiles || w.total.items == 0) return;
  // an SM for every item, and none long enough to be cut: nothing to lay out
  if (w.total.items <= static_cast<int>(gridDim.x) && longest < 2 * kPaMinTiles) return;
  int64_t all = w.total.tiles + int64_t(w.total.items) * w.cost;
  if (all < int64_t(kPaMinTiles) * gridDim.x) {  // less than a run each: items count as one, so that every one gets an SM
    w.cost = kPaMinTiles;
    all = w.total.tiles + int64_t(w.total.items) * w.cost;
  }
  w.per = max(int64_t(kPaMinTiles), (all + gridDim.x - 1) / gridDim.x);
  w.cta = blockIdx.x;
  const int64_t x0 = w.cta * w.per, x1 = x0 + w.per;
  w.r = p.B;
  w.x = w.x_end = 0;
  w.end = 0;
  if (x0 >= all) return;
  w.from = pa_locate(p, w, x0, w.r, w.hg, w.block, w.x);
  if (w.from == kPaAll) {
    PaReq q;
    pa_request(p, w.r, q);
    pa_next(p, w, q);
  }
  w.x_end = all;
  if (x1 < all) {
    int r, hg, block;
    w.end = pa_locate(p, w, x1, r, hg, block, w.x_end);
  }
}

__device__ __forceinline__ void pa_fill(const PromptArgs& p, const PaReq& q, int hg, int block, PaItem& it) {
  it.q0 = q.q0;
  it.nq = q.nq;
  it.nk = q.nk;
  it.k0 = q.k0;
  it.prefix = q.prefix;
  it.tok0 = block * (kPaRows >> p.log2_pack);
  it.head0 = hg << p.log2_pack;
  it.kvh = it.head0 / (p.H / p.HK);
  it.pieces = 1;
  it.cta0 = it.piece = 0;
  it.last = 0;
}
// key tiles [from, to) of an item
__device__ __forceinline__ void pa_range(const PromptArgs& p, const PaReq& q, int from, int to, PaItem& it) {
  const int tt = kPaM >> p.log2_pack;  // tokens of a row tile
  const bool two = it.tok0 + tt < q.nq;
  const int n0 = pa_tiles(p, q, min(it.tok0 + tt, q.nq) - 1), n1 = two ? pa_tiles(p, q, min(it.tok0 + 2 * tt, q.nq) - 1) : 0;
  it.kt0 = from;
  it.n[0] = max(0, min(to, n0) - from);
  it.n[1] = max(0, min(to, n1) - from);
  // a lone row tile with several key tiles: both halves of the CTA work for it, on the even and on the odd ones
  it.paired = !two && n0 > 1;
  if (it.paired) {
    it.n[1] = it.n[0] / 2;
    it.n[0] -= it.n[1];
  }
}

// The next item of this CTA (by a whole warp); false when there are no more. idx: the item off the counter, without runs.
__device__ __forceinline__ bool pa_item(const PromptArgs& p, PaWalk& w, int idx, PaItem& it) {
  const int G = p.H >> p.log2_pack;
  PaReq q;
  if (w.per == 0) {
    if (idx >= w.total.items) return false;
    const int r = pa_find(p, w, 0, 1, idx);
    int i = idx - pa_line(p, w, r).items;
    pa_request(p, r, q);
    // heads at a time: their keys and values take up to 128 MB
    const int g = p.H / p.HK;
    const int kv_heads = max(1, min(p.HK, static_cast<int>((int64_t(128) << 20) / (int64_t(q.nk) * 512 + 1))));
    const int gc = kv_heads * (g >> p.log2_pack);
    const int64_t chunk_items = int64_t(gc) * q.blocks;
    const int chunk = static_cast<int>(i / chunk_items);
    i -= static_cast<int>(chunk * chunk_items);
    const int wide = min(gc, G - chunk * gc), block = q.blocks - 1 - i / wide;
    pa_fill(p, q, chunk * gc + i % wide, block, it);
    pa_range(p, q, 0, kPaAll, it);
    return true;
  }
  if (w.r >= p.B || w.x > w.x_end || (w.x == w.x_end && w.end == 0)) return false;
  pa_request(p, w.r, q);
  pa_fill(p, q, w.hg, w.block, it);
  const int n = pa_block_tiles(p, q, w.block);
  const int to = w.x == w.x_end ? min(w.end, n) : n;
  if (w.from > 0 || to < n) {  // the cuts of this item: runs' starts in it, in order
    const int64_t k0 = (w.x + w.per - 1) / w.per;
    int64_t lo = k0, hi = (w.x + n + w.cost - 1) / w.per;
    while (lo <= hi && pa_cut(n, w.cost, static_cast<int>(lo * w.per - w.x)) == 0) ++lo;
    while (hi >= lo && pa_cut(n, w.cost, static_cast<int>(hi * w.per - w.x)) == kPaAll) --hi;
    it.pieces = static_cast<int>(hi - lo + 2);
    it.cta0 = static_cast<int>(lo - 1);
    it.piece = w.cta - it.cta0;
  }
  pa_range(p, q, w.from, to, it);
  pa_next(p, w, q);
  return true;
}
// A part's place: a CTA leaves one of an item that it starts, and one of an item that another CTA started.
__device__ __forceinline__ int pa_slot(int cta0, int piece) { return 2 * (cta0 + piece) + (piece == 0); }

// ---------------------------------------------------------------- helpers

__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}
// One lane of a converged warp. The MMA warp runs as one and elects a lane for its instructions alone: a branch on the lane
// number around the whole loop made each MMA cost 80-200 clocks to issue (one 8191-token prompt: 837 us, 637 without it, then).
__device__ __forceinline__ bool pa_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 f2_parts(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {  // NaN if one of them is
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// 32 bytes to global memory: one whole sector
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// ---------------------------------------------------------------- the kernel

template <int ROPE, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const PromptArgs p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap v_map) {
  using Y = PaLay<ROPE>;
  constexpr int QU = Y::qk_units, R = Y::ring;
  extern __shared__ __align__(1024) uint8_t sm[];  // all of it: the swizzle atoms need its start
  const uint32_t sb = smem_u32(sm);
  auto bar = [&](int k) -> uint32_t { return sb + uint32_t(Y::bars) + 8u * k; };
  auto unit = [&](int u) -> uint32_t { return sb + uint32_t(Y::units) + uint32_t(u % R) * kPaUnit; };
  // the warp number comes from a shuffle, so that the compiler takes the warps' branches as uniform
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int32_t* err = reinterpret_cast<int32_t*>(p.ws);
  PaItem* items = reinterpret_cast<PaItem*>(sm + Y::item);
  int32_t* bad = reinterpret_cast<int32_t*>(sm + Y::bad);  // [item parity]: the first key whose values are not finite
  if (tid == 0) {
    for (int i = 0; i < R; ++i) mbar_init(bar(A_UFREE + i), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(A_QFULL + t), 1);
      mbar_init(bar(A_QFREE + t), 1);
      mbar_init(bar(A_S + t), 1);
      mbar_init(bar(A_P + 2 * t), 4);
      mbar_init(bar(A_P + 2 * t + 1), 4);
      mbar_init(bar(A_O + t), 1);
      mbar_init(bar(A_ITEM + t), 1);
      mbar_init(bar(A_TAKEN + t), 8 + 1 + kPaGuards);
      mbar_init(bar(A_HALF + t), 4);
    }
    for (int i = 0; i < kPaTiles; ++i) {
      mbar_init(bar(A_KFULL + i), 1);
      mbar_init(bar(A_VFULL + i), 1);
      mbar_init(bar(A_GFULL + i), 1);
      mbar_init(bar(A_READY + i), kPaGuards);
    }
    mbar_init(bar(A_PAIR), 8);
    mbar_init(bar(A_DRAIN), 1);
    tc::fence_mbarrier_init_cluster();
  }
  if (warp == kPaMmaWarp) tc::alloc(sb + uint32_t(Y::tmem), 512);
  if (tid == 32 * kPaLoadWarp) {
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
    if (ROPE) prefetch_tensormap(&rope_map);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait();  // the plan, where there is one, is complete, and with it what came before on the stream
  const uint32_t tm = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sm + Y::tmem), 0);
  bool ok = true;

  if (warp >= kPaMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------------------------------------------------------- items and loads
    if (warp == kPaLoadWarp) {
      int32_t* claim = &reinterpret_cast<PaHead*>(p.ws)->claim;
      int u = 0, nk = 0, nv = 0, ng = 0, nq[2] = {0, 0}, idx = blockIdx.x;  // a CTA's first item is its own
      PaWalk walk;
      pa_plan(p, walk);
      const bool counted = walk.per == 0 && walk.total.items > static_cast<int>(gridDim.x);
      auto room = [&](int at) { return at < R || mbar_wait(bar(A_UFREE + at % R), ((at / R) - 1) & 1); };
      for (int k = 0; ok; ++k) {
        PaItem it = {};
        const bool real = pa_item(p, walk, idx, it);
        it.last = !real;
        if (k >= 2 && !pa_wait(bar(A_TAKEN + (k & 1)), ((k >> 1) - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          items[k & 1] = it;
          bad[k & 1] = 0x7fffffff;
          mbar_arrive(bar(A_ITEM + (k & 1)));
        }
        __syncwarp();
        if (!real) break;
        int next = kPaAll;
        if (lane == 0) {
          if (counted) next = gridDim.x + atomicAdd(claim, 1);
          const int n = it.paired ? it.n[0] + it.n[1] : max(it.n[0], it.n[1]);
          const int seen = pa_lim(p.causal, it.nq, it.nk, it.prefix, it.tok0);
          // a key tile's units, and a value tile's, arrive at the barrier of their first one
          auto load_k = [&](int j) {
            const uint32_t full = bar(A_KFULL + nk % kPaTiles);
            ++nk;
            const int key = it.k0 + (it.kt0 + j) * kPaN;
            for (int c = 0; c < QU && ok; ++c, ++u) {
              if (!room(u)) { ok = false; break; }
              if (c == 0) mbar_arrive_expect_tx(full, QU * kPaUnit);
              if (c < 2) tma_load_3d(unit(u), &k_map, 64 * c, it.kvh, key, full);
              else tma_load_2d(unit(u), &rope_map, 0, key, full);
            }
          };
          auto load_v = [&](int j) {
            // values that not every row sees go to the guards, who pass them on
            const bool guarded = (it.kt0 + j + 1) * kPaN > seen;
            const uint32_t full = guarded ? bar(A_GFULL + ng % kPaTiles) : bar(A_VFULL + nv % kPaTiles);
            ++(guarded ? ng : nv);
            const int key = it.k0 + (it.kt0 + j) * kPaN;
            for (int c = 0; c < 2 && ok; ++c, ++u) {
              if (!room(u)) { ok = false; break; }
              if (c == 0) mbar_arrive_expect_tx(full, 2 * kPaUnit);
              tma_load_3d(unit(u), &v_map, 0, it.kvh, key + 64 * c, full);
              tma_load_3d(unit(u) + kPaUnit / 2, &v_map, 64, it.kvh, key + 64 * c, full);
            }
          };
          if (n > 0) load_k(0);
          for (int t = 0; t < 2 && ok; ++t) {
            if (it.n[t] == 0 || (t == 1 && it.paired)) continue;
            if (nq[t] > 0 && !mbar_wait(bar(A_QFREE + t), (nq[t] - 1) & 1)) { ok = false; break; }
            ++nq[t];
            mbar_arrive_expect_tx(bar(A_QFULL + t), QU * kPaUnit);
            for (int c = 0; c < QU; ++c)
              tma_load_3d(sb + uint32_t(Y::q) + (t * QU + c) * kPaUnit, &q_map, 64 * c, it.head0,
                          it.q0 + it.tok0 + t * (kPaM >> p.log2_pack), bar(A_QFULL + t));
          }
          const int ahead = it.paired ? 2 : 1;
          if (it.paired && ok && n > 1) load_k(1);
          for (int j = 0; j < n && ok; ++j) {
            load_v(j);
            if (j + ahead < n && ok) load_k(j + ahead);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        idx = __shfl_sync(0xffffffffu, next, 0);
      }
      if (lane == 0 && counted) {  // the last CTA to come here resets the counter for the next call: no other one takes items any more
        int32_t* done = &reinterpret_cast<PaHead*>(p.ws)->done;
        __threadfence();
        if (atomicAdd(done, 1) == static_cast<int>(gridDim.x) - 1) *claim = *done = 0;
      }
      if (lane == 0) {  // copies still in flight land before shared memory goes
        auto landed = [&](int first, int n) {
          for (int at = max(0, n - kPaTiles); at < n; ++at)
            if (!mbar_wait(bar(first + at % kPaTiles), (at / kPaTiles) & 1)) ok = false;
        };
        landed(A_KFULL, nk);
        landed(A_VFULL, nv);
        landed(A_GFULL, ng);
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0 && !mbar_wait(bar(A_QFULL + t), (nq[t] - 1) & 1)) ok = false;
      }
      __syncwarp();
    }
    // ---------------------------------------------------------------- MMA issue
    else if (warp == kPaMmaWarp) {
      constexpr uint32_t kIdQK = tc::idesc_bf16_f32(kPaM, kPaN, false, false), kIdPV = tc::idesc_bf16_f32(kPaM, 128, false, true);
      const uint64_t dq = tc::sdesc_sw128(sb + uint32_t(Y::q), 16, 1024), dk = tc::sdesc_sw128(sb + uint32_t(Y::units), 16, 1024),
                     dv = tc::sdesc_sw128(sb + uint32_t(Y::units), kPaUnit / 2, 1024);
      int base = 0, nk = 0, nv = 0, ng = 0, nq[2] = {0, 0}, ns[2] = {0, 0};
      for (int k = 0; ok; ++k) {
        if (!pa_wait(bar(A_ITEM + (k & 1)), (k >> 1) & 1)) { ok = false; break; }
        const PaItem& item = items[k & 1];
        auto uniform = [&](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        const int n0 = uniform(item.n[0]), n1 = uniform(item.n[1]), kt0 = uniform(item.kt0), last_item = uniform(item.last);
        const int seen = uniform(pa_lim(p.causal, item.nq, item.nk, item.prefix, item.tok0));  // keys that every row of the item sees
        const int paired = uniform(item.paired);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(A_TAKEN + (k & 1)));
        if (last_item) break;
        const int n = paired ? n0 + n1 : max(n0, n1), ahead = paired ? 2 : 1;
        // units of key tile j, and of its values
        auto uk = [&](int j) { return j < ahead ? base + j * QU : base + ahead * QU + (j - ahead) * (QU + 2) + 2; };
        auto uv = [&](int j) { return min(j + ahead, n) * QU + 2 * j + base; };
        auto qk = [&](int t, int j, bool last) -> bool {
          const bool first_use = paired || t == 0 || j >= n0, last_use = paired || t == 1 || j >= n1;
          const int tq = paired ? 0 : t;  // the row tile of q
          if (first_use) {
            if (!pa_wait(bar(A_KFULL + nk % kPaTiles), (nk / kPaTiles) & 1)) return false;
            ++nk;
          }
          tc::fence_after();
          const int u0 = uk(j);
          if (pa_elect()) {
#pragma unroll
            for (int c = 0; c < QU; ++c) {
              const uint64_t qa = dq + (tq * QU + c) * (kPaUnit >> 4), ka = dk + ((u0 + c) % R) * (kPaUnit >> 4);
#pragma unroll
              for (int s = 0; s < 4; ++s) tc::mma_ss(tm + 128 * t, qa + 2 * s, ka + 2 * s, kIdQK, c > 0 || s > 0);
              if (last_use) tc::commit(bar(A_UFREE + (u0 + c) % R));
            }
            tc::commit(bar(A_S + t));
            if (last) tc::commit(bar(A_QFREE + tq));
          }
          __syncwarp();
          return true;
        };
        auto pv = [&](int t, int j, bool first, bool last) -> bool {
          const bool first_use = paired || t == 0 || j >= n0, last_use = paired || t == 1 || j >= n1;
          if (first_use) {
            if ((kt0 + j + 1) * kPaN > seen) {
              if (!pa_wait(bar(A_READY + ng % kPaTiles), (ng / kPaTiles) & 1)) return false;
              ++ng;
            } else {
              if (!pa_wait(bar(A_VFULL + nv % kPaTiles), (nv / kPaTiles) & 1)) return false;
              ++nv;
            }
          }
          const int u0 = uv(j);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!pa_wait(bar(A_P + 2 * t + c), ns[t] & 1)) return false;
            tc::fence_after();
            if (pa_elect()) {
              const uint64_t va = dv + ((u0 + c) % R) * (kPaUnit >> 4);
#pragma unroll
              for (int s = 0; s < 4; ++s)
                tc::mma_ts(tm + 256 + 128 * t, tm + 128 * t + 32 * c + 8 * s, va + 128 * s, kIdPV, !first || c > 0 || s > 0);
              if (last_use) tc::commit(bar(A_UFREE + (u0 + c) % R));
              if (c == 1 && last) tc::commit(bar(A_O + t));
            }
            __syncwarp();
          }
          ++ns[t];
          return true;
        };
        if (paired) {
          if (n > 0) {
            ok = pa_wait(bar(A_QFULL), nq[0] & 1);
            ++nq[0];
            ok = ok && qk(0, 0, n == 1) && (n == 1 || qk(1, 1, n == 2));
          }
          for (int j = 0; j < n && ok; j += 2) {
            ok = pv(0, j, j == 0, j + 2 >= n);
            if (ok && j + 2 < n) ok = qk(0, j + 2, j + 3 == n);
            if (ok && j + 1 < n) ok = pv(1, j + 1, j == 0, j + 3 >= n);
            if (ok && j + 3 < n) ok = qk(1, j + 3, j + 4 == n);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : n0;
            if (!ok || nt == 0) continue;
            ok = pa_wait(bar(A_QFULL + t), nq[t] & 1);
            ++nq[t];
            if (ok) ok = qk(t, 0, nt == 1);
          }
          for (int j = 0; j < n && ok; ++j) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int nt = t ? n1 : n0;
              if (!ok || j >= nt) continue;
              ok = pv(t, j, j == 0, j + 1 == nt);
              if (ok && j + 1 < nt) ok = qk(t, j + 1, j + 2 == nt);
            }
          }
        }
        base += n * (QU + 2);
      }
      if (base > 0) {  // every MMA has completed before the tensor memory is released
        if (pa_elect()) tc::commit(bar(A_DRAIN));
        __syncwarp();
        if (!pa_wait(bar(A_DRAIN), 0)) ok = false;
      }
    }
    // ---------------------------------------------------------------- values that not every row sees
    else {
      const int g = warp - kPaGuardWarp;
      int base = 0, ready = 0;
      for (int k = 0; ok; ++k) {
        if (!pa_wait(bar(A_ITEM + (k & 1)), (k >> 1) & 1)) { ok = false; break; }
        const PaItem it = items[k & 1];
        if (it.last) break;
        const int n = it.paired ? it.n[0] + it.n[1] : max(it.n[0], it.n[1]), ahead = it.paired ? 2 : 1;
        const int seen = pa_lim(p.causal, it.nq, it.nk, it.prefix, it.tok0);
        for (int j = max(0, max(seen, 0) / kPaN - it.kt0); j < n && ok; ++j) {
          if (!pa_wait(bar(A_GFULL + ready % kPaTiles), (ready / kPaTiles) & 1)) { ok = false; break; }
          for (int c = 0; c < 2; ++c) {
            const int u = base + min(j + ahead, n) * QU + 2 * j + c;
            const int row = 32 * g + lane, key = (it.kt0 + j) * kPaN + 64 * c + row;
            const uint32_t at = unit(u) + uint32_t(row) * 128;
            bool zero = key >= it.nk;
            if (!zero && key >= seen) {
              uint32_t top = 0;  // the larger exponents of both halves of the words
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const uint4 y = lds128(at + (x >> 3) * (kPaUnit / 2) + (((x + lane) & 7) << 4));
                top = __vmaxu2(__vmaxu2(top, __vmaxu2(y.x & 0x7f807f80u, y.y & 0x7f807f80u)),
                               __vmaxu2(y.z & 0x7f807f80u, y.w & 0x7f807f80u));
              }
              zero = (top & 0xffffu) == 0x7f80u || (top >> 16) == 0x7f80u;
              if (zero) atomicMin(bad + (k & 1), key);
            }
            if (zero) {
              for (int x = 0; x < 16; ++x)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + (x >> 3) * (kPaUnit / 2) + (((x + lane) & 7) << 4)), "r"(0)
                             : "memory");
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(A_READY + ready % kPaTiles));
          ++ready;
        }
        base += n * (QU + 2);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(A_TAKEN + (k & 1)));
      }
    }
  }
  // ------------------------------------------------------------------ softmax and epilogue
  else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2, row = tid & 127;
    const uint32_t tl = tm + (uint32_t(32 * (warp & 3)) << 16), ts = tl + 128 * t, to = tl + 256 + 128 * t;
    int32_t* flag = reinterpret_cast<int32_t*>(sm + Y::flag) + t;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    int ns = 0, no = 0, nhalf = 0, npair = 0;
    auto meet = [&](int b, int& count) -> bool {  // the warps of a barrier, bounded as every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
      return pa_wait(bar(b), count++ & 1);
    };
    for (int k = 0; ok; ++k) {
      if (!pa_wait(bar(A_ITEM + (k & 1)), (k >> 1) & 1)) { ok = false; break; }
      const PaItem& it = items[k & 1];
      if (it.last) break;
      const bool paired = it.paired;
      const int first = it.tok0 + (paired ? 0 : t) * (kPaM >> p.log2_pack), token = first + (row >> p.log2_pack);
      const int hd = it.head0 + (row & ((1 << p.log2_pack) - 1));
      const bool mine = token < it.nq;
      const int lim = mine ? pa_lim(p.causal, it.nq, it.nk, it.prefix, token) : 0;
      const int all_see = pa_lim(p.causal, it.nq, it.nk, it.prefix, min(first, it.nq - 1));
      const int n = it.n[t], kt0 = it.kt0;
      float slope = 0.f;
      if (BIAS && mine) slope = __ldg(p.slopes + hd) * kLog2e;
      const int pos = it.nk - it.nq + token;
      // A lone row tile's m is the row's maximum itself: the largest weight is 1 then, which BF16 holds exactly, and a token whose
      // weight lies on few of many keys is as near as fp32 weights would make it (one over 50k keys: out is 0.0016 off 64 bits, 0.0035
      // with a stale m). Its rows are few, so that O is still rescaled rarely: no time lost. Rows that are no token's never move theirs
      // (-inf + inf is no number, which nothing exceeds).
      const float stale = !mine ? CUDART_INF_F : paired && !BIAS ? 0.f : kPaRescale;
      float m = -CUDART_INF_F, mu = 0.f;  // mu: m where it is finite
      uint64_t sum2 = 0;
      for (int j = 0; j < n; ++j, ++ns) {
        if (!pa_wait(bar(A_S + t), ns & 1)) { ok = false; break; }
        tc::fence_after();
        uint32_t raw[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, raw[c]);
        tc::wait_ld();
        float x[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = __uint_as_float(raw[i >> 5][i & 31]);
        const int key0 = (kt0 + (paired ? 2 * j + t : j)) * kPaN;
        const bool masked = key0 + kPaN > all_see;
        const int left = lim - key0;
        if constexpr (CAP) {
          if (masked) {  // four scores share a reciprocal: a hidden one that is not a number stays out of it
#pragma unroll
            for (int i = 0; i < 128; ++i) x[i] = i < left ? x[i] : 0.f;
          }
          float probe = 0.f;
#pragma unroll
          for (int i = 0; i < 128; i += 2) probe = max3_nan(probe, fabsf(x[i]), fabsf(x[i + 1]));
          // Each row goes by its own scores of this tile, so that no other row's change a bit of it; rows that are no token's go
          // along with the quick way. 2 x 1024 tokens over 12k keys, 16 heads, cap 30: 176 us where no score of a tile is large beside
          // the cap, 276 where every row has some, 303 where a warp has rows of both kinds and takes both ways (queries five
          // times as large; 274 with one way a warp, by vote).
          if (!mine || probe <= p.tanh_max) {
            // all |u| <= 0.625: cap tanh(u) as u times a polynomial in u^2 (least maximum error: 2^-25 of cap), without the
            // special functions that the weights need too
            uint64_t cf[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) cf[i] = f2(p.tanh_c[i], p.tanh_c[i]);
#pragma unroll
            for (int i = 0; i < 128; i += 2) {
              const uint64_t v = f2(x[i], x[i + 1]), t2 = f2_mul(v, v);
              uint64_t q = f2_fma(t2, cf[4], cf[3]);
#pragma unroll
              for (int c = 2; c >= 0; --c) q = f2_fma(t2, q, cf[c]);
              const float2 f = f2_parts(f2_mul(v, q));
              x[i] = f.x;
              x[i + 1] = f.y;
            }
          } else {
          if (probe != probe) sum2 = f2(CUDART_NAN_F, 0.f);
          // cap tanh(u) = cap - 2 cap / (1 + e^(2u)), within 2^-21 of cap; four quotients from one reciprocal of the
          // product (u is cut where tanh is 1 to 2^-29: the product stays finite)
          const float down = -2.f * p.cap2;
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            float e[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) e[c] = 1.f + ex2(fminf(x[i + c] * p.cap_in, 30.f));
            const float ab = e[0] * e[1], cd = e[2] * e[3], r = rcp(ab * cd) * down;
            const float rab = r * cd, rcd = r * ab;
            x[i] = fmaf(rab, e[1], p.cap2);
            x[i + 1] = fmaf(rab, e[0], p.cap2);
            x[i + 2] = fmaf(rcd, e[3], p.cap2);
            x[i + 3] = fmaf(rcd, e[2], p.cap2);
          }
          }
          __syncwarp();
        }
        if constexpr (BIAS) {
          const float d0 = float(pos - key0);  // the difference first: positions past 2^24 are not fp32 numbers
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = fmaf(-slope, fabsf(d0 - float(i)), CAP ? x[i] : x[i] * p.c2);
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = i < left ? x[i] : -CUDART_INF_F;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = x[c];
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], x[i + c], x[i + 4 + c]);
        float top = fmaxf(max3(mx[0], x[124], x[125]), max3(max3(mx[1], x[126], x[127]), mx[2], mx[3]));
        if (!CAP && !BIAS) top *= p.c2;
        const bool move = top > m + stale;
        if (__any_sync(0xffffffffu, move)) {
          const float to_m = BIAS ? top + kPaAhead : top;
          const float f = move ? ex2(m - to_m) : 1.f;  // 0 from -inf
          if (move) m = mu = to_m;
          const uint64_t ff = f2(f, f);
          sum2 = f2_fma(sum2, ff, 0);
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tc::ld16(to + 16 * c, o);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tc::st16(to + 16 * c, o);
            }
          }
        }
        const uint64_t cc = CAP || BIAS ? f2(1.f, 1.f) : f2(p.c2, p.c2), mm = f2(-mu, -mu);
        uint64_t part[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 d = f2_parts(f2_fma(f2(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]), cc, mm));
            const float a = ex2(d.x), b = ex2(d.y);
            part[i & 1] = f2_add(part[i & 1], f2(a, b));
            w[i] = pack_bf16x2(a, b);
          }
          tc::st16(ts + 16 * c, w);
          if (c & 1) {  // PV of the first half of the keys starts while the second half's weights are made
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(A_P + 2 * t + (c >> 1)));
          }
        }
        sum2 = f2_add(sum2, f2_add(part[0], part[1]));
      }
      if (!ok) break;
      if (n > 0) {
        if (!pa_wait(bar(A_O + t), no & 1)) { ok = false; break; }
        ++no;
        tc::fence_after();
      }
      const float2 s2 = f2_parts(sum2);
      float l = s2.x + s2.y;
      const int64_t at = int64_t(it.q0 + token) * p.H + hd;
      const float sink = p.sink && mine ? __ldg(p.sink + hd) * kLog2e : -CUDART_INF_F;
      auto finish = [&](float& m_, float& l_) -> float {  // with the sink: the factor of O
        const float mf = fmaxf(m_, sink), base = mf == -CUDART_INF_F ? 0.f : mf;
        const float f = m_ == -CUDART_INF_F ? 0.f : ex2(m_ - base);
        l_ = l_ * f + (sink == -CUDART_INF_F ? 0.f : ex2(sink - base));
        m_ = base;
        return l_ == 0.f ? 0.f : f / l_;
      };
      // chunks of 32 dims that this thread finishes: all four, or two of a paired item's row, out of both halves' sums
      const int c0 = paired ? 2 * t : 0, c1 = paired ? 2 * t + 2 : 4, n_other = it.n[1 - t];
      float fa = 1.f, fb = 0.f;
      if (paired) {
        float2* ml = reinterpret_cast<float2*>(sm + Y::ml);
        ml[t * kPaM + row] = make_float2(m, l);
        if (!meet(A_PAIR, npair)) { ok = false; break; }
        tc::fence_after();
        const float2 o = ml[(1 - t) * kPaM + row];
        const float both = fmaxf(m, o.x);
        fa = m == -CUDART_INF_F ? 0.f : ex2(m - both);
        fb = o.x == -CUDART_INF_F ? 0.f : ex2(o.x - both);
        l = l * fa + o.y * fb;
        m = both;
      }
      // A value this row sees is not finite. The guards have looked at the tiles of this half's own sums when those are there,
      // and at the other half's of a paired item once the halves have met.
      const bool spoilt = *reinterpret_cast<volatile int32_t*>(bad + (k & 1)) < lim;
      auto sums = [&](int c, float (&v)[32]) {
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
        if (n > 0) {
          tc::ld32(to + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * fa;
        }
        if (paired && n_other > 0) {
          tc::ld32(tl + 256 + 128 * (1 - t) + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), fb, v[i]);
        }
      };
      auto write = [&](int c, const float (&v)[32], float f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[16 * h + 2 * i] * f, v[16 * h + 2 * i + 1] * f);
          store32(static_cast<uint16_t*>(p.out) + at * 128 + 32 * c + 16 * h, w, wide);
        }
      };
      const bool writes_lse = mine && p.lse && (!paired || t == 0);
      if (it.pieces == 1) {
        float f = finish(m, l);
        if (spoilt) f = CUDART_NAN_F;
        if (writes_lse) p.lse[at] = (log2f(l) + m) * kLn2;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float v[32];
          sums(c, v);
          if (mine) write(c, v, f);
        }
        if (paired && !meet(A_PAIR, npair)) { ok = false; break; }  // both sums have been read
      } else {
        float* slot = p.parts + int64_t(pa_slot(it.cta0, it.piece)) * kPaSlotFloats;
        // a part's sums: [32 pieces of 4 dims][rows], so that a warp moves whole lines; a paired row's stand in the first row tile
        const int prow = (paired ? 0 : t * kPaM) + row;
        float4* po = reinterpret_cast<float4*>(slot) + prow;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float v[32];
          sums(c, v);
          if (mine) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              po[(8 * c + i) * kPaRows] = spoilt ? make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F)
                                                 : make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (mine) reinterpret_cast<float2*>(slot + kPaRows * 128)[t * kPaM + row] = make_float2(m, l);
        __threadfence();
        if (paired && !meet(A_PAIR, npair)) { ok = false; break; }
        if (!meet(A_HALF + t, nhalf)) { ok = false; break; }
        if (row == 0) {
          int32_t* count = p.counts + 2 * it.cta0 + t;
          const int old = atomicAdd(count, 1);
          if (old == it.pieces - 1) *count = 0;  // the last one: nobody else looks at it in this call
          *flag = old;
        }
        if (!meet(A_HALF + t, nhalf)) { ok = false; break; }
        if (*reinterpret_cast<volatile int32_t*>(flag) == it.pieces - 1 && mine) {
          __threadfence();
          auto part_of = [&](int q) { return p.parts + int64_t(pa_slot(it.cta0, q)) * kPaSlotFloats; };
          auto ml_of = [&](int q) {
            return __ldcg(reinterpret_cast<const float2*>(part_of(q) + kPaRows * 128) + t * kPaM + row);
          };
          float M = -CUDART_INF_F, Lsum = 0.f;
          for (int q = 0; q < it.pieces; ++q) M = fmaxf(M, ml_of(q).x);
          const float Mu = M == -CUDART_INF_F ? 0.f : M;
          for (int q = 0; q < it.pieces; ++q) {
            const float2 v = ml_of(q);
            Lsum += v.y * (v.x == -CUDART_INF_F ? 0.f : ex2(v.x - Mu));
          }
          const float f = finish(M, Lsum);
          // M may have moved to the sink's: the parts' factors are of Mu, f takes them there
          if (writes_lse) p.lse[at] = (log2f(Lsum) + M) * kLn2;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
            for (int q = 0; q < it.pieces; ++q) {
              const float mq = ml_of(q).x, fq = mq == -CUDART_INF_F ? 0.f : ex2(mq - Mu);
              const float4* pq = reinterpret_cast<const float4*>(part_of(q)) + prow;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v = __ldcg(pq + (8 * c + i) * kPaRows);
                acc[4 * i] = fmaf(v.x, fq, acc[4 * i]);
                acc[4 * i + 1] = fmaf(v.y, fq, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(v.z, fq, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(v.w, fq, acc[4 * i + 3]);
              }
            }
            write(c, acc, f);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(A_TAKEN + (k & 1)));
    }
  }
  if (!ok && lane == 0) atomicOr(err, SMLA_DEVERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kPaMmaWarp) tc::dealloc(tm, 512);
}

}  // namespace

// ---------------------------------------------------------------- host

PromptLayout prompt_layout(int64_t requests, int num_sms) {
  PromptLayout l;
  const size_t slots = 2 * size_t(num_sms);
  // What lasts from call to call, the head and the counters, comes first: where it is depends on the device alone, so that
  // calls of other descriptions on the same workspace find it as they left it and write nothing else there.
  l.counts = 256;
  size_t at = l.counts + slots * sizeof(int32_t);
  at = (at + 255) / 256 * 256;
  l.table = at;
  at += size_t(requests + 1) * sizeof(PaTab);
  at = (at + 255) / 256 * 256;
  l.parts = at;
  l.bytes = at + slots * kPaSlotFloats * sizeof(float);
  return l;
}

namespace {

cudaError_t map3(const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2, int b1, int b2, CUtensorMap* out) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (tensor_map_encoder(&encode) != cudaSuccess) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(d0), cuuint64_t(d1), cuuint64_t(d2)};
  const cuuint64_t strides[2] = {cuuint64_t(2 * s1), cuuint64_t(2 * s2)};
  const cuuint32_t box[3] = {64, cuuint32_t(b1), cuuint32_t(b2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int ROPE, bool CAP, bool BIAS>
cudaError_t launch_variant(const PromptArgs& a, cudaStream_t s) {
  CUtensorMap qm, km, rm, vm;
  const int pack = 1 << a.log2_pack;
  cudaError_t e = map3(a.q, 128 + ROPE, a.H, a.T, a.q_head, a.q_token, pack, kPaM / pack, &qm);
  if (e == cudaSuccess) e = map3(a.k, 128, a.HK, a.N, a.k_head, a.k_token, 1, kPaN, &km);
  if (e == cudaSuccess) e = map3(a.v, 128, a.HK, a.N, a.v_head, a.v_token, 1, kPaN / 2, &vm);
  if (e != cudaSuccess) return e;
  rm = km;
  if (ROPE) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {cuuint64_t(64), cuuint64_t(a.N)};
    const cuuint64_t strides[1] = {cuuint64_t(2 * a.rope_token)};
    const cuuint32_t box[2] = {64, kPaN}, estr[2] = {1, 1};
    if (encode(&rm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.rope), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // set on every device that a call runs on, once
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prompt_attention_kernel<ROPE, CAP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(PaLay<ROPE>::bytes));
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.B > kPlanWarp) {
    e = cudaLaunchKernelEx(&cfg, prompt_plan_kernel, a);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(a.sms));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = PaLay<ROPE>::bytes;
  return cudaLaunchKernelEx(&cfg, prompt_attention_kernel<ROPE, CAP, BIAS>, a, qm, km, rm, vm);
}

template <int ROPE>
cudaError_t launch_rope(const PromptArgs& a, cudaStream_t s) {
  if (a.slopes) return a.cap2 > 0.f ? launch_variant<ROPE, true, true>(a, s) : launch_variant<ROPE, false, true>(a, s);
  return a.cap2 > 0.f ? launch_variant<ROPE, true, false>(a, s) : launch_variant<ROPE, false, false>(a, s);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s) {
  return a.rope ? launch_rope<64>(a, s) : launch_rope<0>(a, s);
}

}  // namespace smla
