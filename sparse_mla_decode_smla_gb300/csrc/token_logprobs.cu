// Log probabilities of given tokens, the entropy and the most likely alternatives (smla_token_logprobs), from one
// pass over each row of logits.
//
// With z_i = scale x_i and m = max z:  S = sum e^{z_i - m},  W = sum e^{z_i - m} (z_i - m);
// log p_t = z_t - m - log S, entropy = log S - W / S. Every thread keeps its own m, S and W over the pieces it reads
// (powers of two of d = (x_i - m) log2(e) scale, the difference first: logits of the type's lowest value are as good a
// maximum as any other) and moves m when a piece exceeds it; they are joined in a fixed order at the end.
//
// Alternatives. After a CTA's first pieces, the k-th largest of its threads' maxima bounds the k-th largest
// value of its part from below (k values are no less): what reaches the bound is kept as a candidate, a 64-bit key of
// value and index (larger value first, then lower index). The bound is raised once more on the way. More candidates
// than the buffer holds (rows of equal or of ascending values) are found again by a radix search over the part instead. The
// k first of the candidates are ranked by counting; keys are distinct, so the order in which they came does not matter.
//
// Few rows are split over the CTAs of a cluster, which meet in the first CTA's shared memory.
#include <math_constants.h>

#include "common.cuh"
#include "prompt.h"
#include "tcgen05.cuh"

namespace smla {
namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpCand = 1024;     // candidates a CTA keeps
constexpr int kLpMaxCluster = 8;
constexpr int kLpUnroll = 4;      // 16-byte pieces a thread loads together

struct LpSums {
  float m, s, w;  // the largest x, sum 2^d, sum 2^d d
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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

struct __align__(16) LpShared {
  uint64_t cand[kLpCand];
  uint64_t best[kLpMaxCluster * kLogprobMaxTop];  // the CTAs' first k, in the cluster's first CTA
  float maxima[kLpThreads];
  uint32_t hist[256];
  LpSums part[kLpWarps];
  LpSums all[kLpMaxCluster];  // the CTAs' sums, in the first CTA
  LpSums total;
  uint32_t count, pick, need;
  float bound;
};

template <bool F32>
__device__ __forceinline__ float lp_load(const LogprobArgs& a, const void* row, int i) {
  if (F32) return static_cast<const float*>(row)[i];
  return __uint_as_float(uint32_t(static_cast<const uint16_t*>(row)[i]) << 16);
}

// the k-th largest of the threads' maxima -> sh.bound; -inf when there are fewer than k
__device__ __forceinline__ void raise_bound(LpShared& sh, float mine, int k) {
  sh.maxima[threadIdx.x] = mine;
  __syncthreads();
  const uint64_t me = key_of(mine, threadIdx.x);
  int above = 0;
#pragma unroll 8
  for (int t = 0; t < kLpThreads; ++t) above += key_of(sh.maxima[t], t) > me ? 1 : 0;
  if (above == k - 1) sh.bound = mine;
  __syncthreads();
}

// The k first keys of [v0, v1) by a radix search over the row: for parts with more candidates than the buffer holds.
// Eight bits of the 64-bit key a pass, from the top; then the keys from the k-th on are collected.
template <bool F32>
__device__ __noinline__ void radix_top(const LogprobArgs& a, const void* row, int v0, int v1, int k, LpShared& sh) {
  uint64_t prefix = 0;
  const int want = min(k, v1 - v0);
  if (threadIdx.x == 0) sh.need = want;
  for (int shift = 56; shift >= 0; shift -= 8) {
    sh.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = v0 + threadIdx.x; i < v1; i += kLpThreads) {
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
    for (int i = v0 + threadIdx.x; i < v1; i += kLpThreads) {
      const uint64_t key = key_of(lp_load<F32>(a, row, i), i);
      if (key >= prefix) sh.cand[atomicAdd(&sh.count, 1u)] = key;  // exactly `want` keys: they are distinct
    }
  }
  __syncthreads();
}

// the k first of n distinct keys, in order, to dst (shared memory of this CTA or, by its cluster address, another's)
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, uint32_t dst) {
  for (int t = threadIdx.x; t < n; t += kLpThreads) {
    const uint64_t me = keys[t];
    int above = 0;
    for (int u = 0; u < n; ++u) above += keys[u] > me ? 1 : 0;
    if (above < k) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst + 8 * above), "l"(me) : "memory");
  }
}

template <bool F32>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(const LogprobArgs a, int cluster) {
  extern __shared__ __align__(16) uint8_t lp_smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(lp_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? blockIdx.x % cluster : 0;
  const int64_t r = blockIdx.x / cluster;
  const int es = F32 ? 4 : 2, per = 16 / es;  // elements of a 16-byte piece
  const uint8_t* row = static_cast<const uint8_t*>(a.x) + r * a.stride * es;
  // this CTA's part: whole pieces; the first one also takes what stands before the first 16-byte border, the last one the end
  const int head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / es));
  const int pieces = (a.V - head) / per, p0 = static_cast<int>(int64_t(pieces) * rank / cluster),
            p1 = static_cast<int>(int64_t(pieces) * (rank + 1) / cluster);
  const int v0 = rank == 0 ? 0 : head + p0 * per, v1 = rank == cluster - 1 ? a.V : head + p1 * per;
  const int k = a.top;
  const float c = a.scale * kLog2e;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = -CUDART_INF_F;
  }
  if (k > 0)
    for (int i = tid; i < kLpMaxCluster * kLogprobMaxTop; i += kLpThreads) sh.best[i] = 0;
  __syncthreads();
  float m = -CUDART_INF_F, mu = 0.f, s = 0.f, w = 0.f, big = -CUDART_INF_F;  // mu: m where it is finite; big: the largest x
  float bound = CUDART_INF_F;  // nothing is kept before the first bound is known
  auto take = [&](const float* x, int n) {  // n values, the largest of which is known to be <= big
    for (int i = 0; i < n; ++i) {
      const float d = max_nan((x[i] - mu) * c, -200.f), e = ex2(d);
      s += e;
      w = fmaf(e, d, w);
    }
  };
  auto lift = [&](float top) {  // the largest of the values to come
    if (top > m) {
      const float d = s > 0.f ? fmaxf((mu - top) * c, -200.f) : 0.f, e = ex2(d);
      w = e * fmaf(d, s, w);
      s *= e;
      m = mu = top;
    }
  };
  auto keep = [&](float x, int i) {
    if (x >= bound) {
      const uint32_t at = atomicAdd(&sh.count, 1u);
      if (at < kLpCand) sh.cand[at] = key_of(x, i);
    }
  };
  const uint4* body = reinterpret_cast<const uint4*>(row + size_t(head) * es);
  constexpr int kPer = F32 ? 4 : 8;
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
  const int step = kLpThreads * kLpUnroll;
  int round = 0;
  for (int p = p0; p < p1; p += step, ++round) {
    uint4 q[kLpUnroll];
#pragma unroll
    for (int j = 0; j < kLpUnroll; ++j) {
      const int at = p + j * kLpThreads + tid;
      // a piece past the end is nothing but lowest values
      q[j] = at < p1 ? __ldg(body + at) : F32 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                                              : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    }
    float top[kLpUnroll];
#pragma unroll
    for (int j = 0; j < kLpUnroll; ++j) {
      float x[kPer];
      unpack(q[j], x);
      top[j] = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top[j] = fmaxf(top[j], x[i]);
      big = fmaxf(big, top[j]);
    }
    if (k > 0 && (round == 0 || round == 3)) {
      raise_bound(sh, big, k);
      bound = sh.bound;
    }
    lift(big);
#pragma unroll
    for (int j = 0; j < kLpUnroll; ++j) {
      const int at = p + j * kLpThreads + tid;
      if (at < p1) {
        float x[kPer];
        unpack(q[j], x);
        take(x, kPer);
        if (k > 0 && top[j] >= bound) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) keep(x[i], head + at * kPer + i);
        }
      }
    }
  }
  if (k > 0 && round == 0) {  // no whole piece: everything is kept
    bound = -CUDART_INF_F;
  }
  for (int part = 0; part < 2; ++part) {  // before the first and behind the last piece
    const int b0 = part ? (rank == cluster - 1 ? head + pieces * per : a.V) : rank == 0 ? 0 : a.V, b1 = part ? a.V : rank == 0 ? head : a.V;
    const int i = b0 + tid;
    if (i < b1) {
      const float x = lp_load<F32>(a, row, i);
      lift(x);
      take(&x, 1);
      if (k > 0) keep(x, i);
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
  if (k > 0 && sh.count > kLpCand) radix_top<F32>(a, row, v0, v1, k, sh);
  const uint32_t base = smem_u32(lp_smem);
  if (cluster > 1) {  // the first CTA's shared memory is set up before others write there
    tc::cluster_arrive();
    tc::cluster_wait();
  }
  const uint32_t first = cluster > 1 ? tc::mapa(base, 0) : base;
  if (tid == 0) {
    LpSums t = sh.part[0];
    for (int i = 1; i < kLpWarps; ++i) join(t, sh.part[i], c);
    const uint32_t at = first + uint32_t(offsetof(LpShared, all)) + uint32_t(sizeof(LpSums)) * rank;
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(t.m) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(t.s) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(t.w) : "memory");
  }
  if (k > 0) rank_keys(sh.cand, min(int(sh.count), kLpCand), k, first + uint32_t(offsetof(LpShared, best)) + 8u * k * rank);
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
  for (int g = tid; g < a.given; g += kLpThreads) {
    const int id = a.tokens[r * a.given + g];
    float v = 0.f;
    if (id >= 0 && id < a.V) {
      v = logprob(lp_load<F32>(a, row, id));
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
      for (int i = tid; i < n; i += kLpThreads) {
        const uint64_t me = sh.best[i];
        int above = 0;
        for (int u = 0; u < n; ++u) above += sh.best[u] > me || (sh.best[u] == me && u < i) ? 1 : 0;
        if (above < k) sh.cand[above] = me;
      }
      __syncthreads();
      keys = sh.cand;
    }
    for (int i = tid; i < k; i += kLpThreads) {
      const uint64_t key = keys[i];
      const float x = of_ordered(uint32_t(key >> 32));
      a.top_ids[r * k + i] = key ? int32_t(0xffffffffu - uint32_t(key)) : -1;
      if (a.top_logprobs) a.top_logprobs[r * k + i] = key ? logprob(x) : -CUDART_INF_F;
    }
  }
}

template <bool F32>
cudaError_t launch(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  // a row over one CTA, or over up to eight while that leaves SMs without work and every thread a piece or two
  int cluster = 1;
  while (cluster < kLpMaxCluster && a.n * cluster * 2 <= num_sms && a.V / (cluster * 2) >= kLpThreads * 8) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n * cluster));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = sizeof(LpShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<F32>, a, cluster);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}

}  // namespace smla
