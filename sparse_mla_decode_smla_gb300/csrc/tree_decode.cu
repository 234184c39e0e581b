// Attention of drafted nodes over the paged latent cache, on the 5th-generation tensor cores:
// every node of a request attends the request's context and the nodes it sees (a bit mask, or
// the chain j <= i).
//
// out_h = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink_h}), s_j = sm_scale <q_h, k_j>, v_j = k_j[0:512],
// in one pass over the slots with a running maximum and sum.
//
// Work. The (node, head) rows of a request share its keys. 64 consecutive rows are a row tile, 64
// consecutive slots a key tile; a unit is one of each. The units of the batch, in the order (request,
// row tile, key tile), are cut into equal runs, one for each SM's CTA, from the lengths on the device: no
// launch depends on them, SMs are equally loaded however ragged the batch, and row tiles of a request
// run near one another, so that its keys are read from HBM once. A row tile that a run's end cuts leaves
// its part, normalised, with its log-sum-exp, in the workspace; a second kernel joins the parts in the
// order of the slots (equal results in every call). A CTA cuts at most two row tiles, so the workspace
// holds two parts an SM whatever the batch.
//
// A unit on one SM. The fp32 output of 64 rows x 512 dims takes half of the tensor memory when the
// halves of each row are stacked on its 128 lanes: lane l < 64 holds row l's dims [0, 256), lane 64 + l
// its dims [256, 512). q is stacked the same way.
//  * Scores: B stacks the 64 slots twice, their low dims over their high ones. Of the M128 N128 result,
//    lanes l < 64, columns 0-63 are the low partial scores, lanes 64 + l, columns 64-127 the high ones;
//    the four threads of a row exchange halves through shared memory and finish 16 slots each.
//  * Values: A = [P; 0] against the low dims and [0; P] against the high ones, into the same columns.
//  Half of every MMA is unused; in exchange nothing crosses between SMs and q stays in tensor memory.
//  Two SMs that share 128 rows, half of the dims each, fill their MMAs, but the exchange of partial scores and
//  of weights through distributed shared memory makes a tile's way too long for the three key buffers that fit:
//  5,613 us where this took 4,020 (16 requests x 64 nodes x 128 heads, contexts of 4k-16k, fp8_ds).
//
// Bound: no unit is full. The MMAs of a unit take 2,220 clocks (18 of N 128 at 66, 8 of N 256 at 128), and shared
// memory, at 128 bytes a clock, carries about 290 KB of it (2,270 clocks): keys in, operands, partial scores. It
// measures 3,990 clocks with fp8_ds (3,395 us for the batch above at 2,070 MHz: 702 TFLOP/s of useful work), 3,830 with
// per-tensor FP8 and 3,590 with BF16; 4 requests of 8k slots, whose runs are shorter, 4,185, 4,035 and 3,720. Two key
// buffers and one score buffer tie the tiles' ways (scores 1,250, read 800, softmax 2,000, values 1,050, the buffer's
// next keys about 1,000) together.
//
// Keys come by the loads of eight warps that know a tile's rows two tiles ahead, when they are prefetched into L2. FP8
// formats: into registers while PV still reads their place, then as f16 into the key tile (block scales applied,
// exact for powers of two). BF16: by asynchronous 16-byte copies into the key tile as PV frees it.
//
// What is hidden never counts: slots without a page or past the last node become zero rows with weight
// zero, and in tiles that hold nodes a row with a non-finite latent value is zeroed and marked, so that
// the scores of the nodes that see it become NaN and the others' sums never meet it.
//
// Per CTA (576 threads): warps 0-7 softmax and epilogue, 8-15 key tiles and q, 16 the tiles' rows, 17 MMA
// issue. Every wait is bounded in time; one that gives up sets SMLA_DEVERR_TIMEOUT.
#include <math_constants.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tree_decode.h"

namespace smla {
namespace {

constexpr int kTrN = 64;   // slots of a key tile
constexpr int kTrM = 64;   // rows of a row tile
constexpr int kTrSub = 16; // slots of a chunk: what PV frees at once
constexpr int kTrSoftWarps = 8, kTrFirstConv = kTrSoftWarps, kTrConvWarps = 8;
constexpr int kTrProducer = kTrFirstConv + kTrConvWarps, kTrMmaWarp = kTrProducer + 1;
constexpr int kTrThreads = 32 * (kTrMmaWarp + 1);
constexpr float kTrRescale = 8.f;  // the running maximum moves when it grows by more (log2 units)
// weights are 2^(s - m + 7): at most 2^15 between moves of the maximum, within f16, and exact to
// 2^-11 down to 2^-21 of the largest one
constexpr float kTrShift = 7.f;

constexpr int kTrPairBlk = 2 * kTrN * 128;  // 64 dims: [64 slots, low | the same slots, high]
constexpr int kTrKLat = 4 * kTrPairBlk;
constexpr int kTrPBlk = kTrM * kTrN * 2;
constexpr int kTrMeta = 8;  // key tiles between the rows' warp and the softmax at most: 6

// TMEM columns
constexpr uint32_t kTrTmO = 0, kTrTmQ = 256, kTrTmS = 384;

struct TreeRun {  // the units [u0, u1) of one CTA
  int64_t u0, u1, per;
  int64_t base0, base1;  // first units of the requests of unit u0 and of unit u1 - 1
  int r0, r1;            // those requests
};

template <int FMT>
struct Lay {
  static constexpr bool bf16 = FMT == SMLA_KV_BF16, tens = FMT == SMLA_KV_FP8_TENSOR;
  static constexpr int row = bf16 ? kBf16RowBytes : tens ? kFp8TensorRowBytes : kFp8RowBytes;
  static constexpr int rope_blk = 2 * kTrN * 64;
  static constexpr size_t K = 0;
  static constexpr size_t rope = K + 2 * size_t(kTrKLat);
  static constexpr size_t P = rope + 2 * size_t(rope_blk);  // [0 | P of even tiles | 0 | P of odd ones | 0]
  static constexpr size_t qr = P + 5 * size_t(kTrPBlk);
  static constexpr size_t xs = qr + 128 * 64;
  static constexpr size_t xm = xs + 256 * 64;   // xs: 16 partial scores a softmax thread
  static constexpr size_t qf = xm + 256 * 4;    // xm: a maximum a softmax thread
  static constexpr size_t rows = qf + 128 * 4;  // qf: factors of q; rows of the key tiles' slots, -1: none [buffer]
  static constexpr size_t meta = rows + 2 * kTrN * 4;
  static constexpr size_t bad = meta + kTrMeta * 8;
  static constexpr size_t keys = bad + kTrMeta * 8;
  static constexpr size_t run = keys + kTrMeta * 4;
  static constexpr size_t tmem = run + sizeof(TreeRun);
  static constexpr size_t bars = tmem + 16;
  static constexpr size_t bytes = bars + 32 * 8;
  static_assert(bytes <= 232448, "shared memory budget");
  static_assert(rope % 1024 == 0 && P % 1024 == 0 && qr % 1024 == 0 && bars % 8 == 0,
                "swizzle atoms and copies");
};
enum {
  R_ROWS = 0,               // [buffer]: the rows of its tile are known
  R_TAKEN = R_ROWS + 2,     // [buffer]: and have been taken
  R_K_FULL = R_TAKEN + 2,   // [buffer]
  R_K_FREE = R_K_FULL + 2,  // [buffer][16-slot chunk]
  R_S_FULL = R_K_FREE + 8,
  R_S_FREE,
  R_P_READY,                // [tile parity]
  R_Q = R_P_READY + 2, R_QRAW, R_QX, R_DRAIN, R_COUNT
};
static_assert(R_COUNT <= 32, "barriers");
// A tile's PV is done when its last chunk is free. (A barrier a tile parity: a wait that may be two tiles behind
// another tells their phases apart.)
__device__ __forceinline__ int pv_done(int t) { return R_K_FREE + 4 * (t & 1) + 3; }

// ---------------------------------------------------------------- the schedule

struct TreeReq {
  int ctx, n, cu0, kt;  // context, nodes, first row of q, key tiles
  int64_t units;        // row tiles x key tiles
};

// 1: a request with nodes, 0: without, -1: one that does not fit the description.
__device__ __forceinline__ int tree_request(const TreeArgs& p, int r, TreeReq& q) {
  const int a = *(p.cu + r), b = *(p.cu + r + 1), c = *(p.ctx + r);
  q.ctx = c;
  q.cu0 = a;
  q.n = 0;
  q.kt = 0;
  q.units = 0;
  if (a == b) return 0;
  const int64_t n = int64_t(b) - a;
  if (a < 0 || n < 0 || b > p.T || c < 0 || (p.W > 0 && n > 32 * int64_t(p.W)) ||
      c + n > (int64_t(p.stride) << p.log2_page))
    return -1;
  q.n = static_cast<int>(n);
  q.kt = static_cast<int>((c + n + kTrN - 1) / kTrN);
  q.units = (n * p.H + kTrM - 1) / kTrM * q.kt;
  return 1;
}

// The run of CTA g of G, for a whole CTA of NT threads, in two steps: each thread's requests (their loads
// pass behind what comes in between), then the run, which ends with a barrier.
template <int NT>
__device__ __forceinline__ int64_t tree_units(const TreeArgs& p, int32_t* err) {
  const int each = (p.B + NT - 1) / NT, ra = min(p.B, int(threadIdx.x) * each), rb = min(p.B, ra + each);
  TreeReq q;
  int64_t sum = 0;
  for (int r = ra; r < rb; ++r) {
    if (tree_request(p, r, q) < 0 && err) atomicOr(err, SMLA_DEVERR_INDEX);
    sum += q.units;
  }
  return sum;
}
template <int NT>
__device__ void tree_schedule(const TreeArgs& p, int64_t sum, int g, int G, TreeRun* run, int64_t* s_warp) {
  constexpr int kWarps = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.B + NT - 1) / NT;
  const int ra = min(p.B, tid * each), rb = min(p.B, ra + each);
  TreeReq q;
  int64_t v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int64_t all = lane < kWarps ? s_warp[lane] : 0;  // (a loop over the warps' sums takes 650 clocks more)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += x;
  }
  const int64_t total = __shfl_sync(0xffffffffu, all, 31), upto = __shfl_sync(0xffffffffu, all, warp ? warp - 1 : 0);
  const int64_t before = warp ? upto : 0;
  v += before - sum;  // units before this thread's requests
  const int64_t per = (total + G - 1) / G;
  const int64_t u0 = min(total, g * per), u1 = min(total, u0 + per);
  if (tid == 0) {
    run->u0 = u0;
    run->u1 = u1;
    run->per = per;
    run->r0 = run->r1 = p.B;
    run->base0 = run->base1 = total;
  }
  __syncthreads();
  if (u0 < u1 && v < u1 && u0 < v + sum) {
    for (int r = ra; r < rb; ++r) {
      tree_request(p, r, q);
      if (v <= u0 && u0 < v + q.units) { run->r0 = r; run->base0 = v; }
      if (v <= u1 - 1 && u1 - 1 < v + q.units) { run->r1 = r; run->base1 = v; }
      v += q.units;
    }
  }
  __syncthreads();
}

// What a run leaves for joining: the row tile it ends in, if later runs go on with it (a tile that several
// runs share is the last one of the first of them, so a run has one at most).
struct alignas(32) TreeJoin {
  int row0, rows;   // first row of out (token x H + head), rows of the tile; 0: nothing to join
  int parts, slot;  // runs that share it, from this one on; where this one's part is
  int head0, pad[3];  // head of the first row
};
__device__ __forceinline__ TreeJoin* tree_join_of(const TreeArgs& p, int g) {
  return reinterpret_cast<TreeJoin*>(p.ws + 256) + g;
}

// The same for up to 32 requests by one warp, a lane a request, without barriers: 0.4 us less on the way to the first copy
// than with the whole CTA (one request of 16 rows and 1000 slots: 15.9 us a call against 16.5).
__device__ void tree_schedule_warp(const TreeArgs& p, int g, int G, int32_t* err, TreeRun* out) {
  const int lane = threadIdx.x & 31;
  TreeReq q;
  q.units = 0;
  if (lane < p.B && tree_request(p, lane, q) < 0 && err) atomicOr(err, SMLA_DEVERR_INDEX);
  int64_t v = q.units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  const int64_t total = __shfl_sync(0xffffffffu, v, 31), before = v - q.units;
  TreeRun run;
  run.per = (total + G - 1) / G;
  run.u0 = min(total, g * run.per);
  run.u1 = min(total, run.u0 + run.per);
  const uint32_t m0 = __ballot_sync(0xffffffffu, before <= run.u0 && run.u0 < v);
  const uint32_t m1 = __ballot_sync(0xffffffffu, before < run.u1 && run.u1 <= v);
  run.r0 = m0 ? __ffs(m0) - 1 : p.B;
  run.r1 = m1 ? __ffs(m1) - 1 : p.B;
  run.base0 = __shfl_sync(0xffffffffu, before, run.r0 & 31);
  run.base1 = __shfl_sync(0xffffffffu, before, run.r1 & 31);
  if (lane == 0) *out = run;
}

struct TreeSeg {  // key tiles [k0, k1) of row tile m of a request
  int r, m, k0, k1;
  int from;  // the one that is worked on first; the others follow in a circle
  TreeReq q;
  bool whole, first;  // all of the row tile's key tiles; the run starts here
};

// Walks a run's segments; every thread of a warp calls it together.
struct TreeWalk {
  int64_t u, u0, u1, base;
  int r;
  TreeReq q;
  __device__ __forceinline__ TreeWalk(const TreeArgs& p, const TreeRun& run)
      : u(run.u0), u0(run.u0), u1(run.u1), base(run.base0), r(run.r0) {
    if (u < u1) tree_request(p, r, q);
  }
  __device__ __forceinline__ bool next(const TreeArgs& p, TreeSeg& s) {
    if (u >= u1) return false;
    if (u >= base + q.units) {  // the next request with nodes, 32 looked at together
      base += q.units;
      const int lane = threadIdx.x & 31;
      for (int x = r + 1; x < p.B; x += 32) {
        TreeReq c;
        const bool has = x + lane < p.B && tree_request(p, x + lane, c) == 1;
        const uint32_t b = __ballot_sync(0xffffffffu, has);
        if (b) {
          r = x + __ffs(b) - 1;
          break;
        }
      }
      tree_request(p, r, q);
    }
    const int64_t off = u - base;
    s.r = r;
    s.q = q;
    s.m = static_cast<int>(off / q.kt);
    s.k0 = static_cast<int>(off - int64_t(s.m) * q.kt);
    s.k1 = static_cast<int>(min(int64_t(q.kt), s.k0 + (u1 - u)));
    s.first = u == u0;
    s.whole = s.k0 == 0 && s.k1 == q.kt;
    // All of a row tile: its keys are taken from where the CTA would be, had it gone round the request's keys
    // since its start, as the other CTAs of this request do: they read the same keys at about the same time, and
    // batches whose keys are more than L2 holds meet them there (16 requests x 64 nodes x 128 heads, 16k contexts:
    // 4,865 us against 5,600 with BF16, 5,500 against 5,945 with fp8_ds).
    s.from = s.whole ? static_cast<int>(uint32_t(u - u0) % uint32_t(q.kt)) : s.k0;
    u += s.k1 - s.k0;
    return true;
  }
};

// Part `slot` (0: of the row tile a run starts in, 1: of the one it ends in) of CTA g: 64 rows of 512
// fp32 values, four dims of a row together, rows next to one another (a warp, a row a lane, stores 512
// consecutive bytes); then their log-sum-exps.
constexpr size_t kTrPart = size_t(kTrM) * (kLatent + 1) * 4;
__device__ __forceinline__ float* tree_part(const TreeArgs& p, int64_t g, int slot, int G) {
  return reinterpret_cast<float*>(p.ws + 256 + size_t(G) * sizeof(TreeJoin) + size_t(2 * g + slot) * kTrPart);
}

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 f2_split(uint64_t d) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
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

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Final factor of a row whose output is divided by its sum already, and its log-sum-exp, with the sink.
__device__ __forceinline__ void apply_sink(const float* sink, int h, float& lse, float& f) {
  if (!sink) return;
  const float sg = *(sink + h);
  if (sg == -CUDART_INF_F) return;
  const float both = fmaxf(lse, sg) + log1pf(expf(-fabsf(lse - sg)));
  f *= expf(lse - both);
  lse = both;
}

// The 64 visibility bits of key tile k for node i of a request: all context slots, and the nodes that
// its mask row shows.
__device__ __forceinline__ uint64_t tree_bits(const TreeArgs& p, const TreeReq& q, int i, int k) {
  const int64_t base = int64_t(k) * kTrN - q.ctx;  // node of the tile's first slot
  if (base + kTrN <= 0) return ~0ull;
  if (p.W == 0) {
    const int64_t last = i - base;  // the tile's last visible slot
    return last >= 63 ? ~0ull : last < 0 ? 0ull : (2ull << last) - 1;
  }
  const uint32_t* row = p.mask + int64_t(q.cu0 + i) * p.W;
  const int64_t from = base < 0 ? 0 : base;
  const int w = static_cast<int>(from >> 5), sh = static_cast<int>(from & 31);
  const uint64_t w0 = w < p.W ? *(row + w) : 0u, w1 = w + 1 < p.W ? *(row + w + 1) : 0u,
                 w2 = w + 2 < p.W ? *(row + w + 2) : 0u;
  uint64_t b = (w0 | (w1 << 32)) >> sh;
  if (sh) b |= w2 << (64 - sh);
  if (base < 0) b = (b << -base) | ((1ull << -base) - 1);  // -base in 1..63
  return b;
}

// ---------------------------------------------------------------- the kernel

// A pipeline wait of a whole warp: all lanes go on, or none does.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

template <int FMT>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_decode_kernel(const TreeArgs p, const __grid_constant__ CUtensorMap q_map) {
  using Y = Lay<FMT>;
  constexpr bool BF = Y::bf16, tens = Y::tens;
  extern __shared__ __align__(1024) uint8_t sm[];  // all of it: the swizzle atoms need its start
  const uint32_t sb = smem_u32(sm);
  auto bar = [&](int k) -> uint32_t { return sb + uint32_t(Y::bars) + 8u * k; };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* err = reinterpret_cast<int32_t*>(p.ws);
  volatile uint64_t* meta = reinterpret_cast<volatile uint64_t*>(sm + Y::meta);  // slots with a row, per tile
  uint32_t* bad = reinterpret_cast<uint32_t*>(sm + Y::bad);                     // non-finite rows, per tile
  volatile int32_t* keys = reinterpret_cast<volatile int32_t*>(sm + Y::keys);  // which key tile, per tile

  // ------------------------------------------------------------------ set-up
  if (tid == 32) prefetch_tensormap(&q_map);
  {
    uint4* zp = reinterpret_cast<uint4*>(sm + Y::P);  // the zero blocks beside P stay zero
    for (int k = tid; k < 5 * kTrPBlk / 16; k += kTrThreads) zp[k] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (tid == 0) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(R_ROWS + b), 1);
        mbar_init(bar(R_TAKEN + b), kTrConvWarps);
        mbar_init(bar(R_K_FULL + b), kTrConvWarps);
      }
      for (int c = 0; c < 8; ++c) mbar_init(bar(R_K_FREE + c), 1);
      mbar_init(bar(R_S_FULL), 1);
      mbar_init(bar(R_S_FREE), kTrSoftWarps);
      for (int x = 0; x < 2; ++x) mbar_init(bar(R_P_READY + x), kTrSoftWarps);
      mbar_init(bar(R_Q), kTrConvWarps);
      mbar_init(bar(R_QRAW), 1);
      mbar_init(bar(R_QX), kTrConvWarps);
      mbar_init(bar(R_DRAIN), 1);
      tc::fence_mbarrier_init_cluster();
    }
    if (warp == kTrMmaWarp) tc::alloc(sb + uint32_t(Y::tmem), 512);
    tc::fence_before();
    pdl_wait();  // what came before on the stream is complete; nothing of it is read before this line
    TreeRun* shared = reinterpret_cast<TreeRun*>(sm + Y::run);
    if (p.B <= 32) {
      if (warp == 0) tree_schedule_warp(p, blockIdx.x, gridDim.x, blockIdx.x == 0 ? err : nullptr, shared);
      __syncthreads();
    } else {
      const int64_t units = tree_units<kTrThreads>(p, blockIdx.x == 0 ? err : nullptr);
      tree_schedule<kTrThreads>(p, units, blockIdx.x, gridDim.x, shared, reinterpret_cast<int64_t*>(sm + Y::xs));
    }
    tc::fence_after();
  }
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + Y::tmem);
  const TreeRun run = *reinterpret_cast<const TreeRun*>(sm + Y::run);
  TreeWalk walk(p, run);
  if (tid == 32 * kTrMmaWarp) {  // the row tile this run ends in, for the joining kernel
    TreeJoin jn = {};
    if (run.u0 < run.u1) {
      TreeReq q;
      tree_request(p, run.r1, q);
      const int64_t m = (run.u1 - 1 - run.base1) / q.kt, ub = run.base1 + m * q.kt;
      if (ub >= run.u0 && ub + q.kt > run.u1) {
        jn.row0 = q.cu0 * p.H + static_cast<int>(m) * kTrM;
        jn.rows = static_cast<int>(min(int64_t(kTrM), int64_t(q.n) * p.H - m * kTrM));
        jn.parts = static_cast<int>((ub + q.kt - 1) / run.per - blockIdx.x + 1);
        jn.slot = ub > run.u0 ? 1 : 0;
        jn.head0 = static_cast<int>(m * kTrM % p.H);
      }
    }
    *tree_join_of(p, blockIdx.x) = jn;
  }
  TreeSeg seg;
  bool ok = true;
  int gi = 0;  // key tiles of this CTA so far: the barriers' phases follow it across segments

  // ------------------------------------------------------------------ rows of the key tiles
  if (warp == kTrProducer) {
    auto entries = [&](const TreeSeg& s, int k, int32_t& e0, int32_t& e1) {
      const int32_t* row = p.page_table + int64_t(s.r) * p.stride;
      const int64_t a = int64_t(k) * kTrN + lane, end = int64_t(s.q.ctx) + s.q.n;
      e0 = a < end ? *(row + (a >> p.log2_page)) : -2;  // -2: no such slot
      e1 = a + 32 < end ? *(row + ((a + 32) >> p.log2_page)) : -2;
    };
    const int P = 1 << p.log2_page;
    bool more = walk.next(p, seg);
    int k = seg.from;
    int32_t e0 = -2, e1 = -2;
    if (more) entries(seg, k, e0, e1);
    while (more && ok) {
      TreeSeg ns = seg;
      int nk = k + 1 == seg.k1 ? seg.k0 : k + 1;
      bool nm = true;
      if (nk == seg.from) {
        nm = walk.next(p, ns);
        nk = ns.from;
      }
      int32_t n0 = -2, n1 = -2;
      if (nm) entries(ns, nk, n0, n1);  // a tile ahead: their latency is hidden
      const bool ok0 = e0 >= 0 && e0 < p.num_pages, ok1 = e1 >= 0 && e1 < p.num_pages;
      if ((!ok0 && e0 != -2) || (!ok1 && e1 != -2)) atomicOr(err, SMLA_DEVERR_PAGE);
      const uint64_t v = uint64_t(__ballot_sync(0xffffffffu, ok0)) | uint64_t(__ballot_sync(0xffffffffu, ok1)) << 32;
      if (lane == 0) {
        meta[gi % kTrMeta] = v;
        keys[gi % kTrMeta] = k;
        bad[2 * (gi % kTrMeta)] = bad[2 * (gi % kTrMeta) + 1] = 0;
      }
      const int b = gi & 1;
      if (gi >= 2 && !warp_wait(bar(R_TAKEN + b), ((gi >> 1) - 1) & 1)) { ok = false; break; }
      int32_t* rows = reinterpret_cast<int32_t*>(sm + Y::rows) + kTrN * b;
      const int64_t s0 = int64_t(k) * kTrN + lane;
      rows[lane] = ok0 ? (e0 << p.log2_page) + static_cast<int32_t>(s0 & (P - 1)) : -1;
      rows[lane + 32] = ok1 ? (e1 << p.log2_page) + static_cast<int32_t>((s0 + 32) & (P - 1)) : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(R_ROWS + b));
      {  // the rows start on their way to L2: 118 -> 113 us for the 128k chain, 3,507 -> 3,463 for the trees above
        const int32_t ra = rows[lane], rb = rows[lane + 32];
#pragma unroll
        for (int o = 0; o < Y::row; o += 128) {
          if (ra >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.kv + int64_t(ra) * Y::row + o));
          if (rb >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.kv + int64_t(rb) * Y::row + o));
        }
      }
      seg = ns;
      k = nk;
      e0 = n0;
      e1 = n1;
      more = nm;
      ++gi;
    }
  }
  // ------------------------------------------------------------------ MMA issuer
  else if (warp == kTrMmaWarp) {
    constexpr uint32_t kIdQK = BF ? tc::idesc_bf16_f32(128, 128, false, false) : tc::idesc_f16_f32(128, 128, false, false);
    constexpr uint32_t kIdPV = BF ? tc::idesc_bf16_f32(128, 256, false, true) : tc::idesc_f16_f32(128, 256, false, true);
    const uint32_t qr = sb + uint32_t(Y::qr);
    const uint32_t d = tm + kTrTmS;
    int nseg = 0;
    while (ok && walk.next(p, seg)) {
      const int nt = seg.k1 - seg.k0;
      if (lane == 0) {
        auto qk_ready = [&](int g) {
          return mbar_test_wait(bar(R_K_FULL + (g & 1)), (g >> 1) & 1) && (g > gi || mbar_test_wait(bar(R_Q), nseg & 1)) &&
                 (g == 0 || mbar_test_wait(bar(R_S_FREE), (g - 1) & 1));
        };
        auto qk = [&](int g) {
          tc::fence_after();
          const uint32_t kt = sb + uint32_t(Y::K) + uint32_t((g & 1) * kTrKLat);
          const uint32_t rope = sb + uint32_t(Y::rope) + uint32_t((g & 1) * Y::rope_blk);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            tc::mma_ts(d, tm + kTrTmQ + 8 * j, tc::sdesc_sw128(kt + (j >> 2) * kTrPairBlk + (j & 3) * 32, 16, 1024), kIdQK, j > 0);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tc::mma_ss(d, tc::sdesc_sw64(qr + 32 * j, 16, 512),
                       tc::sdesc_sw64(rope + 32 * j, 16, 512), kIdQK, 1);
          tc::commit(bar(R_S_FULL));
        };
        auto pv = [&](int g) {
          tc::fence_after();
          const uint32_t kt = sb + uint32_t(Y::K) + uint32_t((g & 1) * kTrKLat);
          const uint32_t pa = sb + uint32_t(Y::P) + uint32_t((1 + 2 * (g & 1)) * kTrPBlk);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            tc::mma_ss(tm + kTrTmO, tc::sdesc_sw128(pa + 32 * s, 16, 1024), tc::sdesc_sw128(kt + 2048 * s, kTrPairBlk, 1024), kIdPV,
                       g > gi || s > 0);
            tc::mma_ss(tm + kTrTmO, tc::sdesc_sw128(pa - kTrPBlk + 32 * s, 16, 1024),
                       tc::sdesc_sw128(kt + kTrN * 128 + 2048 * s, kTrPairBlk, 1024), kIdPV, 1);
            tc::commit(bar(R_K_FREE + 4 * (g & 1) + s));
          }
        };
        int nqk = 0, npv = 0;
        uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 0; npv < nt && ok; ++it) {
          if (npv < nqk && mbar_test_wait(bar(R_P_READY + ((gi + npv) & 1)), ((gi + npv) >> 1) & 1)) {
            pv(gi + npv++);
          } else if (nqk < nt && nqk <= npv + 1 && qk_ready(gi + nqk)) {
            qk(gi + nqk++);
          } else {
            if ((it & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
              ok = false;
              break;
            }
            continue;
          }
          t0 = globaltimer_ns();
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      gi += nt;
      ++nseg;
    }
    if (lane == 0 && nseg > 0) {  // every MMA has completed before the tensor memory is released
      tc::commit(bar(R_DRAIN));
      if (!mbar_wait(bar(R_DRAIN), 0)) ok = false;
    }
    __syncwarp();
  }
  // ------------------------------------------------------------------ key tiles and q
  else if (warp >= kTrFirstConv) {
    const int dtid = tid - 32 * kTrFirstConv, dw = dtid >> 5;
    const int quarter = warp & 3, part = dw >> 2, half = quarter >> 1;
    const int hl = 32 * (quarter & 1) + lane, row = 32 * quarter + lane;
    const uint32_t lrow = tm + (uint32_t(32 * quarter) << 16);
    // FP8 formats: warp dw holds 256 dims (half dw >> 2) of the 16 slots of chunk dw & 3, and their share of the RoPE
    // dims, in registers from the moment it is done with the tile before. Four lanes take 64 consecutive bytes of a
    // row, a warp eight rows: the f16 stores, two 16-byte pieces a job, then spread over the 128-byte swizzle. (Bulk
    // copies into a ring in shared memory instead, read from there, put 84 KB a unit more on it: 3,507 us
    // where this takes 3,463, and 518 against 314 with pages of one slot.)
    const int q = dw & 3, hw = dw >> 2, total = static_cast<int>(run.u1 - run.u0);
    uint4 v[8], rv[2];
    float2 sc[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)};  // of slots lane / 4 and lane / 4 + 8
    uint32_t smax = 0, smin_p2 = ~0u, smin_other = ~0u;  // of the block scales seen: one of the four is this lane's to look at
    auto fetch = [&](int g) -> bool {
      const int fb = g & 1;
      if (!warp_wait(bar(R_ROWS + fb), (g >> 1) & 1)) return false;
      int32_t r[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        r[h] = static_cast<int32_t>(lds_u32(sb + uint32_t(Y::rows) + uint32_t(kTrN * fb + kTrSub * q + (lane >> 2) + 8 * h) * 4));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(R_TAKEN + fb));
      const uint8_t* src[2] = {p.kv + int64_t(max(r[0], 0)) * Y::row, p.kv + int64_t(max(r[1], 0)) * Y::row};
      const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = r[j & 1] >= 0 ? *reinterpret_cast<const uint4*>(src[j & 1] + 256 * hw + 64 * (j >> 1) + 16 * (lane & 3)) : none;
      if constexpr (tens) {
        rv[0] = r[hw] >= 0 ? *reinterpret_cast<const uint4*>(src[hw] + kLatent + 16 * (lane & 3)) : none;
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sc[h] = r[h] >= 0 ? *reinterpret_cast<const float2*>(src[h] + kScaleOff + 8 * hw) : make_float2(1.f, 1.f);
          rv[h] = r[h] >= 0 ? *reinterpret_cast<const uint4*>(src[h] + kRopeOffFp8 + 64 * hw + 16 * (lane & 3)) : none;
        }
      }
      return true;
    };
    int nseg = 0;
    while (ok && walk.next(p, seg)) {
      // q of this row tile, once the softmax has taken the last scores of the previous one (and with them
      // its factors of q): dims [256 half + 128 part, + 128) of
      // a row by this thread, and its 32 RoPE dims by part 1. FP8 formats: f16, scaled by a power of two
      // that brings the row's largest value into [1, 2); the factor goes back into the scores.
      // q arrives as nine boxes of 64 rows x 64 dims in the key-tile buffer that this warp group fills next. A lane
      // per row from global memory instead took 5-7 us.
      // PV of the tile that last used the buffer comes first; its wait also tells S_FREE's last phase from the
      // one before (a barrier's parity tells no more).
      const int qb = gi & 1;
      if (gi >= 2 && !warp_wait(bar(R_K_FREE + 4 * qb + 3), ((gi - 2) >> 1) & 1)) { ok = false; break; }
      if (gi > 0 && !warp_wait(bar(R_S_FREE), (gi - 1) & 1)) { ok = false; break; }
      const uint32_t qlat = sb + uint32_t(Y::K) + uint32_t(qb * kTrKLat);
      const uint32_t qrop = sb + uint32_t(Y::rope) + uint32_t(qb * Y::rope_blk);
      if (dw == 0) {
        if (lane == 0) mbar_arrive_expect_tx(bar(R_QRAW), 9u * kTrM * 128u);
        __syncwarp();
        if (lane < 9)
          tma_load_2d(lane < 8 ? qlat + lane * (kTrM * 128) : qrop, &q_map, 64 * lane, seg.q.cu0 * p.H + seg.m * kTrM, bar(R_QRAW));
      }
      if (!BF && gi == 0 && !fetch(0)) { ok = false; break; }
      {
        const bool have = int64_t(seg.m) * kTrM + hl < int64_t(seg.q.n) * p.H;
        if (!warp_wait(bar(R_QRAW), nseg & 1)) { ok = false; break; }
        tc::fence_after();
        // 16-byte piece c of this thread's 16 latent and 4 RoPE ones (FP8 formats: read twice, for the largest value and
        // for the conversion; held in registers, they spill: 1-2 % of every case)
        auto lat = [&](int c) {
          const uint32_t at = qlat + uint32_t(4 * half + 2 * part + (c >> 3)) * (kTrM * 128) + uint32_t(hl) * 128;
          return have ? lds128(at + (((c & 7) ^ (hl & 7)) << 4)) : make_uint4(0, 0, 0, 0);
        };
        auto rop = [&](int c) {
          return have ? lds128(qrop + uint32_t(hl) * 128 + (((4 * half + c) ^ (hl & 7)) << 4)) : make_uint4(0, 0, 0, 0);
        };
        float qdown = 1.f;
        int qe = 0;
        if constexpr (!BF) {
          uint32_t m4[4] = {0, 0, 0, 0};
          auto look = [&](const uint4 v) {
            m4[0] = bf16x2_max(m4[0], v.x & 0x7fff7fffu);
            m4[1] = bf16x2_max(m4[1], v.y & 0x7fff7fffu);
            m4[2] = bf16x2_max(m4[2], v.z & 0x7fff7fffu);
            m4[3] = bf16x2_max(m4[3], v.w & 0x7fff7fffu);
          };
#pragma unroll 4
          for (int c = 0; c < 16; ++c) look(lat(c));
          if (part == 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) look(rop(c));
          }
          const uint32_t mx = bf16x2_hmax_bits(bf16x2_max(bf16x2_max(m4[0], m4[1]), bf16x2_max(m4[2], m4[3])));
          // the two warps of a row meet in the halves of its factor's word
          const uint32_t at = sb + uint32_t(Y::qf) + uint32_t(row) * 4;
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2 * part), "h"(uint16_t(mx)) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(R_QX));
          if (!warp_wait(bar(R_QX), 0)) { ok = false; break; }
          const uint32_t both = lds_u32(at);
          qe = pow2_exponent_of_bf16(max(both & 0xffffu, both >> 16));
          qdown = exp2_int(-qe);
        }
        auto cvt = [&](uint32_t x) -> uint32_t { return BF ? x : pack_f16x2(bf16_lo(x) * qdown, bf16_hi(x) * qdown); };
        constexpr int kUnroll = BF ? 4 : 1;
#pragma unroll kUnroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t wv[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = lat(4 * ch + k);
            wv[4 * k] = cvt(v.x); wv[4 * k + 1] = cvt(v.y);
            wv[4 * k + 2] = cvt(v.z); wv[4 * k + 3] = cvt(v.w);
          }
          tc::st16(lrow + kTrTmQ + 64 * part + 16 * ch, wv);
        }
        tc::wait_st();
        if (part == 1) {
#pragma unroll kUnroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t dst = sb + uint32_t(Y::qr) + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
            const uint4 v = rop(c);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(cvt(v.x)), "r"(cvt(v.y)), "r"(cvt(v.z)),
                         "r"(cvt(v.w)) : "memory");
          }
          fence_proxy_async_smem();
        }
        // q (and the halves of the factors) has been read before it is written over
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R_QX));
        if (!warp_wait(bar(R_QX), BF ? nseg & 1 : 1)) { ok = false; break; }
        if constexpr (!BF) {
          if (part == 0)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + uint32_t(Y::qf) + uint32_t(row) * 4), "f"(exp2_int(qe)) : "memory");
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R_Q));
        ++nseg;
      }
      for (const int end = gi + seg.k1 - seg.k0; gi < end && ok; ++gi) {
        const int b = gi & 1;
        const uint32_t kt = sb + uint32_t(Y::K) + uint32_t(b * kTrKLat);
        // the tile holds drafted nodes (asked once its rows are known)
        auto has_nodes = [&] { return int64_t(keys[gi % kTrMeta] + 1) * kTrN > seg.q.ctx; };
        uint32_t* badw = bad + 2 * (gi % kTrMeta);
        if constexpr (BF) {
          // Warp dw loads slots [8 dw, 8 dw + 8), four of them (8 lanes of 16 bytes each) and 64 dims at a time, as soon
          // as PV has freed them; what has no row becomes zero. Copies by the threads keep pace whatever the page size,
          // where TMA boxes cost 65 clocks each, ten for every run of slots in one page: pages of 1, 8, 64 slots, 4
          // requests x 64 nodes x 128 heads, 4k contexts, 278 us each against 2,737, 475 and 302.
          if (!warp_wait(bar(R_ROWS + b), (gi >> 1) & 1)) { ok = false; break; }
          int32_t r[2];
#pragma unroll
          for (int g = 0; g < 2; ++g)
            r[g] = static_cast<int32_t>(lds_u32(sb + uint32_t(Y::rows) + uint32_t(kTrN * b + 8 * dw + 4 * g + (lane >> 3)) * 4));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(R_TAKEN + b));
          if (gi >= 2 && !warp_wait(bar(R_K_FREE + 4 * b + (dw >> 1)), ((gi >> 1) - 1) & 1)) { ok = false; break; }
          const uint32_t rp = sb + uint32_t(Y::rope) + uint32_t(b * Y::rope_blk), c = lane & 7;
          auto at = [&](int g, int bx) -> uint32_t {  // piece c of 64 dims of a slot
            const int sl = 8 * dw + 4 * g + (lane >> 3);
            return kt + (bx & 3) * kTrPairBlk + (bx >> 2) * (kTrN * 128) + sl * 128 + ((c ^ (sl & 7)) << 4);
          };
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint8_t* src = p.kv + int64_t(max(r[g], 0)) * kBf16RowBytes + 16 * c;
#pragma unroll
            for (int bx = 0; bx < 8; ++bx) cp_async16(at(g, bx), src + 128 * bx, r[g] >= 0 ? 16 : 0);
            const int rr = kTrN * (c >> 2) + 8 * dw + 4 * g + (lane >> 3);
            cp_async16(rp + rr * 64 + (((c & 3) ^ ((rr >> 1) & 3)) << 4), src + 1024, r[g] >= 0 ? 16 : 0);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          if (has_nodes()) {
#pragma unroll 1
            for (int x = 0; x < 16; ++x) {
              const uint4 y = lds128(at(x >> 3, x & 7));
              const uint32_t w4[4] = {y.x, y.y, y.z, y.w};
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) odd |= (w4[e] & 0x7f80u) == 0x7f80u || (w4[e] & 0x7f800000u) == 0x7f800000u;
              if (odd) {
                const int sl = 8 * dw + 4 * (x >> 3) + (lane >> 3);
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at(x >> 3, x & 7)), "r"(0) : "memory");
                atomicOr(badw + (sl >> 5), 1u << (sl & 31));
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(R_K_FULL + b));
        } else {
          const uint32_t vq = uint32_t(meta[gi % kTrMeta] >> (kTrSub * q)) & 0xffffu;
          const bool nodes = has_nodes();
          // 16 codes of job j -> f16; `whole`: every slot has a row and none is a node
          auto convert = [&](int j, uint32_t (&o)[8], bool whole) {
            const uint32_t wv[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            const __half2 s2 = __float2half2_rn(j < 4 ? sc[j & 1].x : sc[j & 1].y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              e4m3x4_to_f16x4(wv[e], o[2 * e], o[2 * e + 1]);  // exact
              if constexpr (!tens) {  // code * scale in f16
                __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&o[2 * e]), s2);
                __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&o[2 * e + 1]), s2);
                o[2 * e] = *reinterpret_cast<uint32_t*>(&x);
                o[2 * e + 1] = *reinterpret_cast<uint32_t*>(&y);
              }
            }
            if (whole) return;
            const int slot = (lane >> 2) + 8 * (j & 1);
            bool clear = !((vq >> slot) & 1);
            if (nodes) {
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) odd |= (o[e] & 0x7c00u) == 0x7c00u || (o[e] & 0x7c000000u) == 0x7c000000u;
              if (odd) atomicOr(badw + ((kTrSub * q + slot) >> 5), 1u << ((kTrSub * q + slot) & 31));
              clear |= odd;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = clear ? 0u : o[e];
          };
          // Job j's two 16-byte pieces c0, c0 + 1 (even c0) of row rr go to row rr's pieces c ^ (rr & 7): the
          // addresses of job 0 and a constant
          const int rr0 = kTrN * hw + kTrSub * q + (lane >> 2);
          const uint32_t at0 = kt + uint32_t(rr0) * 128 + (((2 * (lane & 3)) ^ (rr0 & 7)) << 4);
          auto put = [&](int j, const uint32_t (&o)[8]) {
            const uint32_t far = 1024u * (j & 1) + uint32_t(j >> 1) * kTrPairBlk;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at0 + far), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"((at0 ^ 16u) + far), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
          };
          if constexpr (!tens) {
            const float2 s2 = lane & 2 ? sc[1] : sc[0];
            const uint32_t a = __float_as_uint(lane & 1 ? s2.y : s2.x) & 0x7fffffffu;
            const bool p2 = (a & 0x7fffffu) == 0;
            smax = max(smax, a);
            smin_p2 = min(smin_p2, (p2 && a != 0) ? a : ~0u);
            smin_other = min(smin_other, p2 ? ~0u : a);
          }
          auto tile = [&](bool whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t o[8];
              convert(j, o, whole);
              put(j, o);
            }
          };
          // Rows [16q, 16q + 16) of the buffer are free once that chunk of PV, two tiles ago, is done. (Converting
          // some jobs before this wait is slower: none of 8 652 us, one 659, two 657, three 706; 4 requests x 64
          // nodes x 128 heads, 8k contexts, fp8_ds.)
          if (gi >= 2 && !warp_wait(bar(R_K_FREE + 4 * b + q), ((gi >> 1) - 1) & 1)) { ok = false; break; }
          // a tile without the checks of its slots takes 8 % less time than with them
          if (vq == 0xffffu && !nodes)
            tile(true);
          else
            tile(false);
          auto rope_put = [&](int rr, int c, uint4 x) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(sb + uint32_t(Y::rope) + uint32_t(b * Y::rope_blk) + rr * 64 +
                         ((c ^ ((rr >> 1) & 3)) << 4)), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
          };
          if constexpr (tens) {  // 16 RoPE dims of a slot
            uint4 x, y;
            e4m3x4_to_f16x4(rv[0].x, x.x, x.y);
            e4m3x4_to_f16x4(rv[0].y, x.z, x.w);
            e4m3x4_to_f16x4(rv[0].z, y.x, y.y);
            e4m3x4_to_f16x4(rv[0].w, y.z, y.w);
            const int rr = kTrN * ((lane >> 1) & 1) + kTrSub * q + 8 * hw + (lane >> 2), c = 2 * (lane & 1);
            rope_put(rr, c, x);
            rope_put(rr, c + 1, y);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              rope_put(kTrN * hw + kTrSub * q + (lane >> 2) + 8 * j, lane & 3,
                       make_uint4(bf16x2_to_f16x2(rv[j].x), bf16x2_to_f16x2(rv[j].y), bf16x2_to_f16x2(rv[j].z), bf16x2_to_f16x2(rv[j].w)));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(R_K_FULL + b));
          // the next tile's rows come while PV frees their place
          if (gi + 1 < total && !fetch(gi + 1)) { ok = false; break; }
        }
      }
    }
    if (FMT == SMLA_KV_FP8_DS) {  // the f16 window: largest scale, smallest power of two, smallest other one
      const bool out_of_window = smax > 0x43000000u || smin_p2 < 0x38000000u || smin_other < 0x38800000u;
      if (__any_sync(0xffffffffu, out_of_window) && lane == 0) atomicOr(err, SMLA_DEVERR_RANGE);
    }
    if (dtid == 0) pdl_trigger();  // the joining kernel may start launching
  }
  // ------------------------------------------------------------------ softmax + epilogue
  else {
    // Four threads hold a row: half (low or high partial scores) and sub (16 of 32 slots). Thread (half,
    // sub) finishes slots 32 half + 16 sub .. + 15: it takes the other half's partials of them from thread
    // (1 - half, sub) and gives it its own of that thread's slots. The four warps of a row group meet at
    // two named barriers a tile: partials written, maxima written.
    const int quarter = warp & 3, sub = warp >> 2, half = quarter >> 1, pr = quarter & 1;
    const int hl = 32 * pr + lane;
    const uint32_t lrow = tm + (uint32_t(32 * quarter) << 16);
    // 16 partials of (quarter, sub, lane): 16-byte piece k at k ^ ((lane >> 1) & 3), no bank conflicts
    const uint32_t xmine = sb + uint32_t(Y::xs) + uint32_t(32 * warp + lane) * 64;
    const uint32_t xpart = sb + uint32_t(Y::xs) + uint32_t(32 * (warp ^ 2) + lane) * 64;
    const uint32_t xsw = uint32_t((lane >> 1) & 3);
    // maxima of a row: [(half, sub)][row]
    const uint32_t mrow = sb + uint32_t(Y::xm) + uint32_t(hl) * 4;
    const uint32_t mmine = mrow + uint32_t(2 * half + sub) * 256;
    const int bar_x = 1 + pr, bar_m = 3 + pr;
    const float c2 = tens ? p.c2 * p.kv_scale : p.c2;
    int nseg = 0;
    while (ok && walk.next(p, seg)) {
      const int64_t R = int64_t(seg.m) * kTrM + hl;
      const bool real = R < int64_t(seg.q.n) * p.H;
      const int node = real ? static_cast<int>(R / p.H) : 0;
      const int h = real ? static_cast<int>(R - int64_t(node) * p.H) : 0;
      const int nt = seg.k1 - seg.k0;
      bool good = warp_wait(bar(R_Q), nseg & 1);
      float c2m = c2, c2p = c2;
      if constexpr (!BF) {
        c2m *= lds_f32(sb + uint32_t(Y::qf) + uint32_t(32 * quarter + lane) * 4);
        c2p *= lds_f32(sb + uint32_t(Y::qf) + uint32_t(32 * (quarter ^ 2) + lane) * 4);
      }
      float m = -CUDART_INF_F, l = 0.f;
      auto correct_o = [&](float a) {  // warp-wide: the whole warp calls it when any lane needs it
#pragma unroll 1
        for (int k = 8 * sub; k < 8 * sub + 8; k += 2) {
          uint32_t v0[16], v1[16];
          tc::ld16(lrow + kTrTmO + 16 * k, v0);
          tc::ld16(lrow + kTrTmO + 16 * k + 16, v1);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v0[e] = __float_as_uint(__uint_as_float(v0[e]) * a);
            v1[e] = __float_as_uint(__uint_as_float(v1[e]) * a);
          }
          tc::st16(lrow + kTrTmO + 16 * k, v0);
          tc::st16(lrow + kTrTmO + 16 * k + 16, v1);
        }
        tc::wait_st();
      };
      for (int i = 0; i < nt; ++i, ++gi) {
        uint32_t own[16], send[16];
        const bool got = good && warp_wait(bar(R_S_FULL), gi & 1);
        if (got) {
          tc::fence_after();
          tc::ld16(lrow + kTrTmS + 64 * half + 32 * (half ^ 1) + 16 * sub, send);
          tc::ld16(lrow + kTrTmS + 64 * half + 32 * half + 16 * sub, own);
          tc::wait_ld();
          tc::fence_before();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) own[e] = send[e] = 0u;
        }
        __syncwarp();
        if (lane == 0 && got) mbar_arrive(bar(R_S_FREE));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(xmine + ((k ^ xsw) << 4)), "r"(send[4 * k]),
                       "r"(send[4 * k + 1]), "r"(send[4 * k + 2]), "r"(send[4 * k + 3]) : "memory");
        if (!named_bar_and(bar_x, 128, got)) {
          ok = false;
          break;
        }
        float s[16];
        const uint64_t c2m2 = f2(c2m, c2m), c2p2 = f2(c2p, c2p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 xv = lds128(xpart + ((k ^ xsw) << 4));
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 r = f2_split(f2_fma(f2(__uint_as_float(own[4 * k + e]), __uint_as_float(own[4 * k + e + 1])), c2m2,
                                             f2_mul(f2(__uint_as_float(xw[e]), __uint_as_float(xw[e + 1])), c2p2)));
            s[4 * k + e] = r.x;
            s[4 * k + e + 1] = r.y;
          }
        }
        uint64_t vis = meta[gi % kTrMeta];
        uint32_t oddm = 0;
        const int key = keys[gi % kTrMeta];
        const bool nodes = int64_t(key + 1) * kTrN > seg.q.ctx;  // a tile with nodes
        if (nodes || vis != ~0ull) {
          if (nodes) {
            vis &= tree_bits(p, seg.q, node, key);
            oddm = reinterpret_cast<volatile uint32_t*>(bad)[2 * (gi % kTrMeta) + half] >> (16 * sub);
          }
          const uint32_t msk = uint32_t(vis >> (32 * half + 16 * sub)) & 0xffffu;
          oddm &= msk;
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = ((msk >> j) & 1u) ? s[j] : -CUDART_INF_F;
        }
        float mx = max3(s[0], s[1], s[2]), my = max3(s[3], s[4], s[5]);
#pragma unroll
        for (int j = 6; j < 14; j += 4) {
          mx = max3(mx, s[j], s[j + 1]);
          my = max3(my, s[j + 2], s[j + 3]);
        }
        mx = fmaxf(max3(mx, s[14], s[15]), my);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(mmine), "f"(mx) : "memory");
        if (oddm) {  // a visible row with a non-finite value: NaN
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((oddm >> j) & 1u) s[j] = CUDART_NAN_F;
        }
        named_bar(bar_m, 128);
        const float mn = fmaxf(fmaxf(fmaxf(lds_f32(mrow), lds_f32(mrow + 256)), fmaxf(lds_f32(mrow + 512), lds_f32(mrow + 768))), m);
        float a = 1.f;
        if (m == -CUDART_INF_F ? mn != -CUDART_INF_F : mn > m + kTrRescale) {
          a = exp2_fast(m - mn);  // 0 when m was -inf
          m = mn;
        }
        const float base = m == -CUDART_INF_F ? 0.f : m - kTrShift;
        const uint64_t nb2 = f2(-base, -base);
        uint64_t sum[2] = {0, 0};
        uint32_t pw2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 x = f2_split(f2_add(f2(s[2 * j], s[2 * j + 1]), nb2));
          const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
          // The weights enter PV in the keys' type, since an MMA takes both operands in one: bf16 with a BF16 cache
          // (each off by 2^-8 at most; results 0.0018-0.0021 off 64 bits where fp32 weights give 0.0017), else f16.
          sum[j & 1] = f2_add(sum[j & 1], f2(p0, p1));
          pw2[j] = BF ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
        }
        const float2 sums = f2_split(f2_add(sum[0], sum[1]));
        l = l * a + (sums.x + sums.y);
        // This P block is free: the scores that came are of keys that replaced those PV read two tiles ago. O is
        // free once PV of the previous tile is complete.
        if (good && i > 0 && __any_sync(0xffffffffu, a != 1.f)) {
          good = warp_wait(bar(pv_done(gi - 1)), ((gi - 1) >> 1) & 1);
          tc::fence_after();
          if (good) correct_o(a);
        }
        if (good) {
          const uint32_t prow = sb + uint32_t(Y::P) + uint32_t((1 + 2 * (gi & 1)) * kTrPBlk) + uint32_t(hl) * 128;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = 4 * half + 2 * sub + k;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(prow + ((c ^ (hl & 7)) << 4)), "r"(pw2[4 * k]),
                         "r"(pw2[4 * k + 1]), "r"(pw2[4 * k + 2]), "r"(pw2[4 * k + 3]) : "memory");
          }
          fence_proxy_async_smem();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0 && good) mbar_arrive(bar(R_P_READY + (gi & 1)));
      }
      if (!ok) break;
      // ---- epilogue: the four threads' sums of a row, then O lane -> output or part
      const bool fin = good && warp_wait(bar(pv_done(gi - 1)), ((gi - 1) >> 1) & 1);
      tc::fence_after();
      // the sums meet in the partials' places, which this group of four warps alone uses: those of the last
      // tile were read before its second barrier
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(xmine), "f"(l) : "memory");
      if (!named_bar_and(bar_x, 128, fin)) {
        ok = false;
        break;
      }
      const uint32_t lsum = sb + uint32_t(Y::xs) + uint32_t(32 * pr + lane) * 64;  // warps pr, pr + 2, pr + 4, pr + 6
      l = (lds_f32(lsum) + lds_f32(lsum + 64 * 64)) + (lds_f32(lsum + 128 * 64) + lds_f32(lsum + 192 * 64));
      named_bar(bar_m, 128);
      float lse = l == 0.f ? -CUDART_INF_F : (m - kTrShift + log2f(l)) * kLn2;
      float f = l == 0.f ? 0.f : (tens ? p.kv_scale : 1.f) / l;
      const int64_t orow = (int64_t(seg.q.cu0) + node) * p.H + h;
      float* part = nullptr;
      if (seg.whole) {
        apply_sink(p.sink, h, lse, f);
        if (p.lse && real && half == 0 && sub == 0) p.lse[orow] = lse;
      } else {
        part = tree_part(p, blockIdx.x, seg.first ? 0 : 1, gridDim.x);
        if (half == 0 && sub == 0) part[kTrM * kLatent + hl] = lse;
      }
#pragma unroll 1
      for (int k4 = 2 * sub; k4 < 2 * sub + 2; ++k4) {
        uint32_t v4[4][16];
#pragma unroll
        for (int j = 0; j < 4; ++j) tc::ld16(lrow + kTrTmO + 64 * k4 + 16 * j, v4[j]);
        tc::wait_ld();
        if (!real) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t* vv = v4[j];
          const int col = 256 * half + 64 * k4 + 16 * j;
          if (seg.whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kLatent + col);
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2(__uint_as_float(vv[2 * e]) * f, __uint_as_float(vv[2 * e + 1]) * f);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
          } else {
            float4* dst = reinterpret_cast<float4*>(part) + (col >> 2) * kTrM + hl;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e * kTrM] = make_float4(__uint_as_float(vv[4 * e]) * f, __uint_as_float(vv[4 * e + 1]) * f,
                                   __uint_as_float(vv[4 * e + 2]) * f, __uint_as_float(vv[4 * e + 3]) * f);
          }
        }
      }
      tc::fence_before();  // the next row tile's PV comes after this one's loads
      ++nseg;
    }
  }

  // ------------------------------------------------------------------ teardown
  if (!ok && lane == 0) atomicOr(err, SMLA_DEVERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  if (warp == kTrMmaWarp) {
    tc::fence_after();
    tc::dealloc(tm, 512);
  }
}

// ---------------------------------------------------------------- joining the parts

constexpr int kTrJoinThreads = 256, kTrJoinCtas = 4;  // CTAs an SM
constexpr int kTrMaxRuns = 512;

// The row tiles to join, 64 items each: four rows and 128 dims. out = sum_i w_i o_i / sum_i w_i with w_i =
// e^(lse_i - max) over a tile's parts i: the weights of the four rows go to shared memory, then a thread
// takes four dims of a row over the even or the odd parts, always in the same order. Bound by the latency of
// a few dependent loads: spread over the whole GPU it takes a few microseconds, where one CTA a run,
// two rows at a time, took 30-55 us.
__global__ void __launch_bounds__(kTrJoinThreads) tree_join_kernel(const TreeArgs p, int G) {
  __shared__ int s_list[kTrMaxRuns], s_found[kTrJoinThreads / 32];
  __shared__ float s_w[4][kTrMaxRuns], s_lse[4], s_f[4];
  __shared__ float4 s_acc[128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  // the runs that leave a row tile to join, in order; every thread looks at one (a warp at all of them took a
  // microsecond more)
  int count = 0;
  for (int x0 = 0; x0 < G; x0 += kTrJoinThreads) {
    const bool has = x0 + tid < G && tree_join_of(p, x0 + tid)->rows > 0;
    const uint32_t b = __ballot_sync(0xffffffffu, has);
    if (lane == 0) s_found[warp] = __popc(b);
    __syncthreads();
    for (int w = 0; w < kTrJoinThreads / 32; ++w) {
      if (w == warp && has) s_list[count + __popc(b & ((1u << lane) - 1))] = x0 + tid;
      count += s_found[w];
    }
    __syncthreads();
  }
  const int items = 64 * count;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int g = s_list[item >> 6];
    const TreeJoin jn = *tree_join_of(p, g);
    const int row0 = 4 * ((item >> 2) & 15);
    if (row0 >= jn.rows) continue;
    const int r = tid & 3, quad = 32 * (item & 3) + ((tid >> 2) & 31), odd = tid >> 7;
    auto piece = [&](int i) { return reinterpret_cast<const float4*>(tree_part(p, g + i, i ? 0 : jn.slot, G))[quad * kTrM + row0 + r]; };
    constexpr int kAhead = 4;  // loads that pass behind the weights
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (odd + 2 * k < jn.parts) ahead[k] = piece(odd + 2 * k);
    if (warp < 4) {  // the weights of row row0 + warp
      const int row = row0 + warp;
      float M = -CUDART_INF_F, W = 0.f;
      for (int i = lane; i < jn.parts; i += 32) {
        const float v = tree_part(p, g + i, i ? 0 : jn.slot, G)[kTrM * kLatent + row];
        s_w[warp][i] = v;
        M = fmaxf(M, v);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float ref = M == -CUDART_INF_F ? 0.f : M;
      for (int i = lane; i < jn.parts; i += 32) {
        const float w = expf(s_w[warp][i] - ref);
        s_w[warp][i] = w;
        W += w;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
      float lse = W == 0.f ? -CUDART_INF_F : ref + logf(W);
      float f = W == 0.f ? 0.f : 1.f / W;
      apply_sink(p.sink, (jn.head0 + row) % p.H, lse, f);
      if (lane == 0) {
        s_lse[warp] = lse;
        s_f[warp] = f;
      }
    }
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& o) {
      const float w = s_w[r][i];
      a.x = fmaf(w, o.x, a.x);
      a.y = fmaf(w, o.y, a.y);
      a.z = fmaf(w, o.z, a.z);
      a.w = fmaf(w, o.w, a.w);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (odd + 2 * k < jn.parts) add(odd + 2 * k, ahead[k]);
#pragma unroll 8
    for (int i = odd + 2 * kAhead; i < jn.parts; i += 2) add(i, piece(i));
    if (odd) s_acc[tid & 127] = a;
    __syncthreads();
    if (!odd && row0 + r < jn.rows) {
      const float4 o = s_acc[tid];
      const float f = s_f[r];
      const int64_t orow = int64_t(jn.row0) + row0 + r;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kLatent + 4 * quad) =
          make_uint2(pack_bf16x2((a.x + o.x) * f, (a.y + o.y) * f), pack_bf16x2((a.z + o.z) * f, (a.w + o.w) * f));
      if (p.lse && quad == 0) p.lse[orow] = s_lse[r];
    }
    __syncthreads();
  }
}

// q, [rows, 576] bf16, in boxes of a row tile x 64 dims, 128-byte swizzle.
cudaError_t tree_q_map(const void* base, int64_t rows, CUtensorMap* out) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (tensor_map_encoder(&encode) != cudaSuccess) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cuuint64_t(kDim), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(2 * kDim)};
  const cuuint32_t box[2] = {64, kTrM};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int FMT>
cudaError_t launch_fmt(const TreeArgs& a, int sms, const CUtensorMap& qmap, cudaStream_t s) {
  // devices (below 64) whose kernel attribute is set; concurrent first calls set it twice
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t(1) << dev) : 0;
  if (!(configured.load(std::memory_order_acquire) & bit) || !bit) {
    cudaError_t e = cudaFuncSetAttribute(tree_decode_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Lay<FMT>::bytes));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  // both kernels start up while what is before them on the stream ends, and wait for it themselves (pdl_wait)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(kTrThreads);
  cfg.dynamicSmemBytes = Lay<FMT>::bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_decode_kernel<FMT>, a, qmap);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(sms * kTrJoinCtas));
  cfg.blockDim = dim3(kTrJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel, a, sms);
}

}  // namespace

size_t tree_workspace_bytes(int num_sms) { return 256 + num_sms * (sizeof(TreeJoin) + 2 * kTrPart); }

cudaError_t launch_tree_decode(const TreeArgs& a, int num_sms, cudaStream_t s) {
  if (num_sms > kTrMaxRuns) return cudaErrorInvalidConfiguration;
  alignas(64) CUtensorMap qmap = {};
  const cudaError_t e = tree_q_map(a.q, int64_t(a.T) * a.H, &qmap);
  if (e != cudaSuccess) return e;
  if (a.kv_format == SMLA_KV_FP8_TENSOR) return launch_fmt<SMLA_KV_FP8_TENSOR>(a, num_sms, qmap, s);
  if (a.kv_format == SMLA_KV_FP8_DS) return launch_fmt<SMLA_KV_FP8_DS>(a, num_sms, qmap, s);
  return launch_fmt<SMLA_KV_BF16>(a, num_sms, qmap, s);
}

}  // namespace smla
