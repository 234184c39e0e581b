// Log probabilities of given tokens, the entropy and the most likely alternatives (smla_token_logprobs), from one
// pass over each row of logits.
//
// With z_i = scale x_i and m = max z:  S = sum e^{z_i - m},  W = sum e^{z_i - m} (z_i - m);
// log p_t = z_t - m - log S, entropy = log S - W / S. Every thread keeps its own m, S and W over the pieces it reads
// (powers of two of d = (x_i - m) log2(e) scale, the difference first: logits of the type's lowest value are as good a
// maximum as any other) and moves m when a piece exceeds it; they are joined in a fixed order at the end.
//
// Alternatives. Every thread keeps the largest value of each quarter of its pieces. The k-th largest of the threads' maxima
// bounds the k-th largest value of the CTA's part from below (k values are no less), and what reaches it is in the few
// quarters whose maximum does: those are read once more (a fiftieth of the row for k = 20), and the candidates found, 64-bit keys of
// value and index (larger value first, then lower index), are ranked by counting. More candidates than the buffer holds
// (rows of equal values) are found by a radix search over the part instead. Keys are distinct, so the order in which they
// came does not matter.
//
// 1024 rows of 129,280 bf16 logits take 55 us with 20 alternatives, 8 more than with none (265 MB: 39 us at the measured copy
// bandwidth). The reading and the ends of rows bound it, where a CTA's threads meet, all CTAs at nearly the same time: without
// the exponentials it takes as long, and so it does with twice as much on its way (by asynchronous copies to shared memory).
// Bounds raised on the way and candidates kept in the first reading: 82 us.
//
// Few rows are split over the CTAs of a cluster, which meet in the first CTA's shared memory.
#include <math_constants.h>

#include "common.cuh"
#include "prompt.h"
#include "tcgen05.cuh"

namespace smla {
namespace {

constexpr int kLpWide = 256, kLpNarrow = 64;  // threads of a CTA: for long rows, and for short ones
constexpr int kLpMaxCluster = 8;
constexpr int kLpUnroll = 4;      // 16-byte pieces a thread loads together
static_assert(kLpUnroll == 4, "pick");

struct LpSums {
  float m, s, w;  // the largest x, sum 2^d, sum 2^d d
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// values in an order that unsigned integers keep; -0 counts as +0
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_ordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) { return uint64_t(ordered(x)) << 32 | (0xffffffffu - i); }

__device__ __forceinline__ void join(LpSums& a, const LpSums& b, float c) {
  const float m = fmaxf(a.m, b.m);
  // an empty side (m = -inf, s = 0) adds nothing
  const float da = a.m == m ? 0.f : fmaxf((a.m - m) * c, -200.f), db = b.m == m ? 0.f : fmaxf((b.m - m) * c, -200.f);
  const float ea = ex2(da), eb = ex2(db);
  a.w = ea * fmaf(da, a.s, a.w) + eb * fmaf(db, b.s, b.w);
  a.s = ea * a.s + eb * b.s;
  a.m = m;
}

template <int TH>
struct __align__(16) LpShared {
  static constexpr int kCand = TH == kLpWide ? 1024 : 512;  // candidates a CTA keeps
  uint64_t cand[kCand];
  uint64_t best[(TH == kLpWide ? kLpMaxCluster : 1) * kLogprobMaxTop];  // the CTAs' first k, in the cluster's first CTA
  float maxima[TH];
  uint32_t hist[256];
  float quarter[4 * TH];  // the threads' maxima of each quarter of their pieces
  int32_t hot[4 * TH];    // the quarters whose maximum reaches the bound
  LpSums part[TH / 32];
  LpSums all[kLpMaxCluster];  // the CTAs' sums, in the first CTA
  LpSums total;
  uint32_t count, hot_count, pick, need;
  uint32_t bound;  // in the order of `ordered`
};

template <bool F32>
__device__ __forceinline__ float lp_load(const LogprobArgs& a, const void* row, int i) {
  if (F32) return static_cast<const float*>(row)[i];
  return __uint_as_float(uint32_t(static_cast<const uint16_t*>(row)[i]) << 16);
}

// A value that at least k of the threads' maxima reach -> sh.bound: the k-th largest one's upper 16 bits, found from the top
// by the first warp, eight maxima a lane (all of a BF16 value's bits; the few more that reach it in fp32 cost less than 16
// more steps).
template <int TH>
__device__ __forceinline__ void find_bound(LpShared<TH>& sh, float mine, int k) {
  sh.maxima[threadIdx.x] = mine;
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t key[TH / 32], found = 0;
#pragma unroll
    for (int i = 0; i < TH / 32; ++i) key[i] = ordered(sh.maxima[32 * i + threadIdx.x]);
    for (int b = 31; b >= 16; --b) {
      const uint32_t next = found | 1u << b;
      int n = 0;
#pragma unroll
      for (int i = 0; i < TH / 32; ++i) n += key[i] >= next ? 1 : 0;
      if (__reduce_add_sync(0xffffffffu, n) >= k) found = next;
    }
    if (threadIdx.x == 0) sh.bound = found;
  }
  __syncthreads();
}

// The k first keys of [v0, v1) by a radix search over the row: for parts with more candidates than the buffer holds.
// Eight bits of the 64-bit key a pass, from the top; then the keys from the k-th on are collected.
template <bool F32, int TH>
__device__ __noinline__ void radix_top(const LogprobArgs& a, const void* row, int v0, int v1, int k, LpShared<TH>& sh) {
  uint64_t prefix = 0;
  const int want = min(k, v1 - v0);
  if (threadIdx.x == 0) sh.need = want;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += TH) sh.hist[i] = 0;
    __syncthreads();
    for (int i = v0 + threadIdx.x; i < v1; i += TH) {
      const uint64_t key = key_of(lp_load<F32>(a, row, i), i);
      if (shift == 56 || (key >> (shift + 8)) == prefix) atomicAdd(&sh.hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t need = sh.need;
      int b = 255;
      while (b > 0 && sh.hist[b] < need) need -= sh.hist[b--];
      sh.need = need;
      sh.pick = b;
    }
    __syncthreads();
    prefix = prefix << 8 | sh.pick;
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  if (want > 0) {
    for (int i = v0 + threadIdx.x; i < v1; i += TH) {
      const uint64_t key = key_of(lp_load<F32>(a, row, i), i);
      if (key >= prefix) sh.cand[atomicAdd(&sh.count, 1u)] = key;  // exactly `want` keys: they are distinct
    }
  }
  __syncthreads();
}

// the k first of n distinct keys, in order, to dst (shared memory of this CTA or, by its cluster address, another's)
template <int TH>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, uint32_t dst) {
  for (int t = threadIdx.x; t < n; t += TH) {
    const uint64_t me = keys[t];
    int above = 0;
    for (int u = 0; u < n; ++u) above += keys[u] > me ? 1 : 0;
    if (above < k) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst + 8 * above), "l"(me) : "memory");
  }
}

template <bool F32, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) token_logprobs_kernel(const LogprobArgs a, int cluster) {
  extern __shared__ __align__(16) uint8_t lp_smem[];
  using Shared = LpShared<TH>;
  Shared& sh = *reinterpret_cast<Shared*>(lp_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? blockIdx.x % cluster : 0;
  constexpr int es = F32 ? 4 : 2, kPer = 16 / es;  // elements of a 16-byte piece
  const int k = a.top;
  const float c = a.scale * kLog2e;
  struct Part {  // of a row, in whole pieces; the first one also takes what stands before the first 16-byte border, the last one the end
    const uint8_t* row;
    int head, pieces, p0, p1;
  };
  auto part_of = [&](int64_t r) {
    Part q;
    q.row = static_cast<const uint8_t*>(a.x) + r * a.stride * es;
    q.head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(q.row) & 15)) & 15) / es));
    q.pieces = (a.V - q.head) / kPer;
    q.p0 = static_cast<int>(int64_t(q.pieces) * rank / cluster);
    q.p1 = static_cast<int>(int64_t(q.pieces) * (rank + 1) / cluster);
    return q;
  };
  constexpr int step = TH * kLpUnroll;
  uint4 next[kLpUnroll];
  auto load = [&](const uint4* from, int left) {  // left: pieces from there on; one past the end is nothing but lowest values
    if (left >= step) {
#pragma unroll
      for (int j = 0; j < kLpUnroll; ++j) next[j] = __ldg(from + j * TH);
    } else {
      const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
      for (int j = 0; j < kLpUnroll; ++j)
        next[j] = j * TH + tid < left ? __ldg(from + j * TH) : make_uint4(none, none, none, none);
    }
  };
  auto first_load = [&](const Part& q) { load(reinterpret_cast<const uint4*>(q.row + size_t(q.head) * es) + q.p0 + tid, q.p1 - q.p0); };
  const int64_t rows_apart = gridDim.x / cluster;
  int64_t r = blockIdx.x / cluster;
  pdl_wait();  // what came before on the stream is complete
  first_load(part_of(r));
  for (; r < a.n; r += rows_apart) {  // (one row where it is shared by a cluster)
  const Part part = part_of(r);
  const uint8_t* row = part.row;
  const int head = part.head, pieces = part.pieces, p0 = part.p0, p1 = part.p1;
  const int v0 = rank == 0 ? 0 : head + p0 * kPer, v1 = rank == cluster - 1 ? a.V : head + p1 * kPer;
  int given_id = -1;  // this thread's given token and its logit, on their way while the row is read
  float given_x = 0.f;
  if (rank == 0 && tid < a.given) {
    given_id = a.tokens[r * a.given + tid];
    if (given_id >= 0 && given_id < a.V) given_x = lp_load<F32>(a, row, given_id);
  }
  __syncthreads();  // the row before is done with shared memory
  if (tid == 0) sh.count = sh.hot_count = 0;
  if (k > 0)
    for (int i = tid; i < (cluster > 1 ? kLpMaxCluster * kLogprobMaxTop : k); i += TH) sh.best[i] = 0;
  __syncthreads();
  if (cluster > 1) tc::cluster_arrive();
  float m = -CUDART_INF_F, mu = 0.f, s = 0.f, w = 0.f, big = -CUDART_INF_F;  // mu: m where it is finite; big: the largest x of the pieces
  auto take = [&](float x) {
    const float d = max_nan((x - mu) * c, -200.f), e = ex2(d);
    s += e;
    w = fmaf(e, d, w);
  };
  auto lift = [&](float top) {  // the largest of the values to come
    if (top > m) {
      const float d = s > 0.f ? fmaxf((mu - top) * c, -200.f) : 0.f, e = ex2(d);
      w = e * fmaf(d, s, w);
      s *= e;
      m = mu = top;
    }
  };
  const uint4* body = reinterpret_cast<const uint4*>(row + size_t(head) * es);
  auto unpack = [&](const uint4& q, float* x) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (F32) {
        x[i] = __uint_as_float(u[i]);
      } else {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
      }
    }
  };
  auto pick = [](const uint4 (&q)[kLpUnroll], int j) {  // without a place in memory
    return j & 2 ? (j & 1 ? q[3] : q[2]) : (j & 1 ? q[1] : q[0]);
  };
  uint64_t s2 = 0, w2 = 0;  // the sums of the pieces, in pairs
  const uint4* at = body + p0 + tid;
  const int rounds = (p1 - p0 + step - 1) / step;
  int part_end = rounds >> 2, in_part = 0, round = 0;  // quarter i ends before round (i + 1) rounds / 4
  float here = -CUDART_INF_F;
  auto end_part = [&] {
    while (in_part < 4 && round == part_end) {
      sh.quarter[in_part * TH + tid] = here;
      here = -CUDART_INF_F;
      ++in_part;
      part_end = (in_part + 1) * rounds >> 2;
    }
  };
  if (k > 0) end_part();
  for (int p = p0; p < p1; p += step, at += step) {
    uint4 q[kLpUnroll];
#pragma unroll
    for (int j = 0; j < kLpUnroll; ++j) q[j] = next[j];
    if (p + step < p1) load(at + step, p1 - p - step);  // a round ahead
    float top, low;
    if (F32) {
      top = -CUDART_INF_F;
      low = CUDART_INF_F;
#pragma unroll
      for (int j = 0; j < kLpUnroll; ++j) {
        const float a = __uint_as_float(q[j].x), b = __uint_as_float(q[j].y), e = __uint_as_float(q[j].z), f = __uint_as_float(q[j].w);
        top = fmaxf(top, fmaxf(fmaxf(a, b), fmaxf(e, f)));
        low = fminf(low, fminf(fminf(a, b), fminf(e, f)));
      }
    } else {
      uint32_t hi = q[0].x, lo = q[0].x;
#pragma unroll
      for (int j = 0; j < kLpUnroll; ++j) {
        hi = bf16x2_max(hi, bf16x2_max(bf16x2_max(q[j].x, q[j].y), bf16x2_max(q[j].z, q[j].w)));
        lo = bf16x2_min(lo, bf16x2_min(bf16x2_min(q[j].x, q[j].y), bf16x2_min(q[j].z, q[j].w)));
      }
      top = fmaxf(bf16_lo(hi), bf16_hi(hi));
      low = fminf(bf16_lo(lo), bf16_hi(lo));
    }
    big = fmaxf(big, top);
    here = fmaxf(here, top);
    if (big > m) {
      const float d = s2 != 0 ? fmaxf((mu - big) * c, -200.f) : 0.f, e = ex2(d);
      const uint64_t ee = f2(e, e);
      w2 = f2_mul(f2_fma(f2(d, d), s2, w2), ee);
      s2 = f2_mul(s2, ee);
      m = mu = big;
    }
    const uint64_t cc = f2(c, c), mm = f2(-mu, -mu);
    // no value so low that its term vanishes (where the product with its exponent could be none): without a check each
    if (__all_sync(0xffffffffu, (low - mu) * c > -120.f)) {
#pragma unroll
      for (int j = 0; j < kLpUnroll; ++j) {
        float x[kPer];
        unpack(q[j], x);
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const uint64_t d = f2_mul(f2_add(f2(x[i], x[i + 1]), mm), cc);
          const float2 f = f2_parts(d);
          const uint64_t e = f2(ex2(f.x), ex2(f.y));
          s2 = f2_add(s2, e);
          w2 = f2_fma(e, d, w2);
        }
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < kLpUnroll; ++j) {
        float x[kPer];
        unpack(pick(q, j), x);
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const float a = max_nan((x[i] - mu) * c, -200.f), b = max_nan((x[i + 1] - mu) * c, -200.f);
          const uint64_t e = f2(ex2(a), ex2(b));
          s2 = f2_add(s2, e);
          w2 = f2_fma(e, f2(a, b), w2);
        }
      }
    }
    ++round;
    if (k > 0) end_part();
  }
  {
    const float2 a = f2_parts(s2), b = f2_parts(w2);
    s = a.x + a.y;
    w = b.x + b.y;
  }
  // the next row's first pieces, while this one's end is worked out
  const bool short_row = rounds <= 1;  // its pieces are all still in `next`
  if (!short_row && r + rows_apart < a.n) first_load(part_of(r + rows_apart));
  // (CTAs of the next kernel that come where some have two rows and some one take places unevenly: 1024 rows of 129,280 then take 59.7 us, 55 without)
  if (a.n <= rows_apart) pdl_trigger();
  float edge[2] = {-CUDART_INF_F, -CUDART_INF_F};  // a value before the first and one behind the last piece
  const int edge_at[2] = {rank == 0 && tid < head ? tid : -1,
                          rank == cluster - 1 && head + pieces * kPer + tid < a.V ? head + pieces * kPer + tid : -1};
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (edge_at[part] >= 0) {
      edge[part] = lp_load<F32>(a, row, edge_at[part]);
      lift(edge[part]);
      take(edge[part]);
    }
  }
  LpSums mine = {m, s, w};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LpSums other = {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o),
                    __shfl_xor_sync(0xffffffffu, mine.w, o)};
    if (lane & o) {  // the same order on both sides
      join(other, mine, c);
      mine = other;
    } else {
      join(mine, other, c);
    }
  }
  if (lane == 0) sh.part[warp] = mine;
  __syncthreads();
  if (k > 0) {
    find_bound(sh, fmaxf(big, fmaxf(edge[0], edge[1])), k);
    const uint32_t bound = sh.bound;
    auto keep = [&](float x, int i) {
      if (ordered(x) >= bound) {
        const uint32_t to = atomicAdd(&sh.count, 1u);
        if (to < Shared::kCand) sh.cand[to] = key_of(x, i);
      }
    };
#pragma unroll
    for (int part = 0; part < 2; ++part)
      if (edge_at[part] >= 0) keep(edge[part], edge_at[part]);
    auto look = [&](const uint4& v, int piece) {
      float x[kPer];
      unpack(v, x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < kPer; ++e) top = fmaxf(top, x[e]);
      if (ordered(top) >= bound) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) keep(x[e], head + piece * kPer + e);
      }
    };
    if (short_row) {
#pragma unroll 1
      for (int j = 0; j < kLpUnroll; ++j)
        if (p0 + j * TH + tid < p1) look(pick(next, j), p0 + j * TH + tid);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ordered(sh.quarter[i * TH + tid]) >= bound) sh.hot[atomicAdd(&sh.hot_count, 1u)] = i * TH + tid;
      __syncthreads();
      const int hot = sh.hot_count, each = ((rounds + 3) >> 2) * kLpUnroll;
      for (int i = tid; i < hot * each && sh.count <= Shared::kCand; i += TH) {
        const int q = sh.hot[i % hot], in = i / hot, first = (q / TH) * rounds >> 2, end = (q / TH + 1) * rounds >> 2;
        if (first + in / kLpUnroll >= end) continue;
        const int piece = p0 + (first * kLpUnroll + in) * TH + q % TH;
        if (piece < p1) look(__ldg(body + piece), piece);
      }
    }
    __syncthreads();
    if (sh.count > Shared::kCand) radix_top<F32, TH>(a, row, v0, v1, k, sh);
  }
  if (short_row && r + rows_apart < a.n) first_load(part_of(r + rows_apart));
  const uint32_t base = smem_u32(lp_smem);
  if (cluster > 1) tc::cluster_wait();  // the first CTA's shared memory has been set up before others write there
  const uint32_t first = cluster > 1 ? tc::mapa(base, 0) : base;
  if (warp == 0) {
    LpSums t = {-CUDART_INF_F, 0.f, 0.f};
    if (lane < (TH / 32)) t = sh.part[lane];
#pragma unroll
    for (int o = 1; o < (TH / 32); o *= 2) {  // lane 0: the warps' sums in order
      const LpSums other = {__shfl_down_sync(0xffffffffu, t.m, o), __shfl_down_sync(0xffffffffu, t.s, o), __shfl_down_sync(0xffffffffu, t.w, o)};
      join(t, other, c);
    }
    if (lane == 0) {
      const uint32_t to = first + uint32_t(offsetof(Shared, all)) + uint32_t(sizeof(LpSums)) * rank;
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(t.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(t.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(t.w) : "memory");
    }
  }
  if (k > 0) rank_keys<TH>(sh.cand, min(int(sh.count), Shared::kCand), k, first + uint32_t(offsetof(Shared, best)) + 8u * k * rank);
  if (cluster > 1) {
    tc::cluster_arrive();
    tc::cluster_wait();
    if (rank != 0) return;
  }
  __syncthreads();
  LpSums t = sh.all[0];
  for (int i = 1; i < cluster; ++i) join(t, sh.all[i], c);
  const float log2_s = log2f(t.s);
  auto logprob = [&](float x) { return fmaf(x - t.m, a.scale, -log2_s * kLn2); };
  if (tid == 0 && a.entropy) a.entropy[r] = (log2_s - t.w / t.s) * kLn2;
  for (int g = tid; g < a.given; g += TH) {
    const int id = g == tid ? given_id : a.tokens[r * a.given + g];
    float v = 0.f;
    if (id >= 0 && id < a.V) {
      v = logprob(g == tid ? given_x : lp_load<F32>(a, row, id));
    } else if (id != -1) {
      v = CUDART_NAN_F;
      if (a.err) atomicOr(a.err, SMLA_DEVERR_INDEX);
    }
    a.logprobs[r * a.given + g] = v;
  }
  if (k > 0) {
    const uint64_t* keys = sh.best;
    if (cluster > 1) {
      // zeros (a part with fewer than k values) rank last among themselves by place
      const int n = cluster * k;
      for (int i = tid; i < n; i += TH) {
        const uint64_t me = sh.best[i];
        int above = 0;
        for (int u = 0; u < n; ++u) above += sh.best[u] > me || (sh.best[u] == me && u < i) ? 1 : 0;
        if (above < k) sh.cand[above] = me;
      }
      __syncthreads();
      keys = sh.cand;
    }
    for (int i = tid; i < k; i += TH) {
      const uint64_t key = keys[i];
      const float x = of_ordered(uint32_t(key >> 32));
      a.top_ids[r * k + i] = key ? int32_t(0xffffffffu - uint32_t(key)) : -1;
      if (a.top_logprobs) a.top_logprobs[r * k + i] = key ? logprob(x) : -CUDART_INF_F;
    }
  }
  }
}

template <bool F32, int TH>
cudaError_t launch(const LogprobArgs& a, int cluster, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(TH);
  cfg.dynamicSmemBytes = sizeof(LpShared<TH>);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<F32, TH>, a, cluster);
}

template <bool F32>
cudaError_t launch_rows(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  // Four wide CTAs an SM go from row to row, or a row is split over up to eight of them while that leaves places without
  // work and every thread a piece or two. Many short rows take narrow CTAs, sixteen an SM: a row's fixed steps are most of its time
  // (2134 rows of 1862 fp32 logits, nothing in L2: 21 us, 31 with wide ones).
  const int64_t places = 4 * int64_t(num_sms);
  const int64_t bytes = int64_t(a.V) * (F32 ? 4 : 2);
  if (a.n > places && bytes <= kLpNarrow * 16 * 16) return launch<F32, kLpNarrow>(a, 1, static_cast<int>(a.n < 4 * places ? a.n : 4 * places), s);
  int cluster = 1;
  while (cluster < kLpMaxCluster && a.n * cluster * 2 <= places && bytes / (cluster * 2) >= kLpWide * 32) cluster *= 2;
  return launch<F32, kLpWide>(a, cluster, static_cast<int>(cluster > 1 ? a.n * cluster : a.n < places ? a.n : places), s);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch_rows<true>(a, num_sms, s) : launch_rows<false>(a, num_sms, s);
}

}  // namespace smla
