// The row operators around a prompt: cache rows read back as bf16 (smla_cache_read), and the residual's
// addition with the RMS norm and its bf16 and E4M3 outputs (smla_add_rmsnorm). Both are bound by memory.
#include "common.cuh"
#include "kernels.h"
#include "prompt.h"
#include "quantise.cuh"

namespace smla {
namespace {

// ---------------------------------------------------------------- cache rows read back

constexpr int kRdRows = 64, kRdThreads = 256;  // rows and threads of a CTA: eight rows a warp

__device__ __forceinline__ uint4 bf16x8_of_e4m3(uint2 w, float scale) {
  uint32_t h[4], o[4];
  e4m3x4_to_f16x4(w.x, h[0], h[1]);
  e4m3x4_to_f16x4(w.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    o[i] = pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Bound by HBM: 24 contexts of 4k to 32k fp8_ds slots (796 MB in and out) take 120 us, 98 % of the measured copy bandwidth.
//
// Output row i belongs to the request r with cu[r] <= i < cu[r + 1] and receives its slot starts[r] + i - cu[r].
// A CTA finds the cache rows of its 64 output rows with one thread each (a binary search over cu, then the page
// table), so that the eight rows of a warp are loaded together: one memory round trip for all of them.
template <int FMT>
__global__ void __launch_bounds__(kRdThreads) cache_read_kernel(const ReadArgs a) {
  __shared__ int64_t slots[kRdRows];  // -1: zeros, -2: no request's row
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = int64_t(blockIdx.x) * kRdRows;
  if (tid < kRdRows) {
    const int64_t i = row0 + tid;
    int64_t slot = -2;
    if (i < a.N) {
      int lo = 0, hi = a.B;  // the last r with cu[r] <= i, if cu ascends
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= i) lo = mid; else hi = mid;
      }
      const int64_t c0 = __ldg(a.cu + lo), c1 = __ldg(a.cu + lo + 1);
      if (c0 >= 0 && c0 <= i && i < c1) {
        const int64_t at = int64_t(__ldg(a.starts + lo)) + i - c0, page_at = at >> a.log2_page;
        slot = -1;
        if (at < 0 || page_at >= a.stride) {
          if (a.err) atomicOr(a.err, SMLA_DEVERR_INDEX);
        } else {
          const int64_t page = __ldg(a.page_table + int64_t(lo) * a.stride + page_at);
          if (page < 0 || page >= a.num_pages) {
            if (a.err) atomicOr(a.err, SMLA_DEVERR_PAGE);
          } else {
            slot = (page << a.log2_page) + (at & ((int64_t(1) << a.log2_page) - 1));
          }
        }
      }
    }
    slots[tid] = slot;
  }
  __syncthreads();
  pdl_trigger();
  constexpr bool BF = FMT == SMLA_KV_BF16, tens = FMT == SMLA_KV_FP8_TENSOR;
  constexpr int R = BF ? kBf16RowBytes : tens ? kFp8TensorRowBytes : kFp8RowBytes;
  const uint4 none = make_uint4(0, 0, 0, 0);
  // RoPE parts: 8 lanes a row, four rows at a time
  uint4 rp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t s = slots[8 * warp + 4 * h + (lane >> 3)];
    const uint8_t* src = a.kv + s * R;
    rp[h] = none;
    if (s >= 0) {
      if constexpr (tens) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + kLatent + 8 * (lane & 7));
        rp[h].x = w.x;
        rp[h].y = w.y;
      } else {
        rp[h] = *reinterpret_cast<const uint4*>(src + (BF ? 2 * kLatent : kRopeOffFp8) + 16 * (lane & 7));
      }
    }
  }
#pragma unroll
  for (int g = 0; g < (BF ? 2 : 1); ++g) {
    constexpr int n = BF ? 4 : 8;  // rows at a time
    uint4 v[n][BF ? 2 : 1];
    float2 sc[n];
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int64_t s = slots[8 * warp + n * g + k];
      const uint8_t* src = a.kv + s * R;
      sc[k] = make_float2(a.kv_scale, a.kv_scale);
      v[k][0] = none;
      if constexpr (BF) v[k][1] = none;
      if (s >= 0) {
        if constexpr (BF) {
          v[k][0] = *reinterpret_cast<const uint4*>(src + 16 * lane);
          v[k][1] = *reinterpret_cast<const uint4*>(src + 512 + 16 * lane);
        } else {  // codes [8 lane, + 8) and [256 + 8 lane, + 8): both halves' outputs are stored by whole lines
          const uint2 w0 = *reinterpret_cast<const uint2*>(src + 8 * lane);
          const uint2 w1 = *reinterpret_cast<const uint2*>(src + 256 + 8 * lane);
          v[k][0] = make_uint4(w0.x, w0.y, w1.x, w1.y);
          if constexpr (!tens) {
            const float* f = reinterpret_cast<const float*>(src + kScaleOff);
            sc[k] = make_float2(f[lane >> 4], f[2 + (lane >> 4)]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int row = 8 * warp + n * g + k;
      if (slots[row] == -2) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.latent) + (row0 + row) * a.latent_stride);
      if constexpr (BF) {
        dst[lane] = v[k][0];
        dst[32 + lane] = v[k][1];
      } else {
        dst[lane] = bf16x8_of_e4m3(make_uint2(v[k][0].x, v[k][0].y), sc[k].x);
        dst[32 + lane] = bf16x8_of_e4m3(make_uint2(v[k][0].z, v[k][0].w), sc[k].y);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * warp + 4 * h + (lane >> 3);
    if (slots[row] == -2) continue;
    uint4 o = rp[h];
    if constexpr (tens) o = bf16x8_of_e4m3(make_uint2(o.x, o.y), a.kv_scale);
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.rope) + (row0 + row) * a.rope_stride)[lane & 7] = o;
  }
}

// ---------------------------------------------------------------- residual + RMS norm

// h = x + residual; y = h r w with r = 1 / sqrt(mean(h^2) + eps), in fp32 from the unrounded sum. A thread holds VPT pieces of
// eight consecutive dims of its row in registers: the row is read once. Sixteen lanes share a block of 128.
//
// A row's work on its VPT pieces, by LANES lanes of a warp (LANES <= 32), or by a CTA of T threads that meet in `part`
// (LANES = 0).
template <int LANES, int VPT>
struct NormRow {
  float h[VPT][8];

  // x and the residual -> h, its bf16 sum stored; the sum of squares
  __device__ __forceinline__ float add(const NormArgs& a, int64_t row, int t, int T, const uint4 (&xv)[VPT], const uint4 (&rv)[VPT]) {
    const int nv = a.dim >> 3;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t xw[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w}, rw[4] = {rv[k].x, rv[k].y, rv[k].z, rv[k].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[k][2 * i] = __fadd_rn(bf16_lo(xw[i]), bf16_lo(rw[i]));
        h[k][2 * i + 1] = __fadd_rn(bf16_hi(xw[i]), bf16_hi(rw[i]));
        o[i] = pack_bf16x2(h[k][2 * i], h[k][2 * i + 1]);
        ss = fmaf(h[k][2 * i + 1], h[k][2 * i + 1], fmaf(h[k][2 * i], h[k][2 * i], ss));
      }
      if (a.sum && k * T + t < nv)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.sum) + row * a.dim)[k * T + t] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return ss;
  }
  // the value that every lane of the row (part: of the CTA) gets
  template <typename F>
  __device__ __forceinline__ static float all(float v, int T, float* part, F f) {
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (LANES) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (T >> 5) ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
  // h -> y and its outputs
  __device__ __forceinline__ void finish(const NormArgs& a, int64_t row, int t, int T, float ss, const uint4 (&wv)[VPT], float* part) {
    const int nv = a.dim >> 3;
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, float(a.dim)), a.eps)));
    float amax[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t ww[4] = {wv[k].x, wv[k].y, wv[k].z, wv[k].w};
      uint32_t o[4];
      amax[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[k][2 * i] = __fmul_rn(__fmul_rn(h[k][2 * i], r), bf16_lo(ww[i]));
        h[k][2 * i + 1] = __fmul_rn(__fmul_rn(h[k][2 * i + 1], r), bf16_hi(ww[i]));
        o[i] = pack_bf16x2(h[k][2 * i], h[k][2 * i + 1]);
        amax[k] = fmaxf(amax[k], fmaxf(fabsf(h[k][2 * i]), fabsf(h[k][2 * i + 1])));
      }
      if (a.y && k * T + t < nv)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + row * a.dim)[k * T + t] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (!a.codes) return;
    if (a.group) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
    } else {
      float m = amax[0];
#pragma unroll
      for (int k = 1; k < VPT; ++k) m = fmaxf(m, amax[k]);
      m = all(m, T, part, [](float x, float y) { return fmaxf(x, y); });
#pragma unroll
      for (int k = 0; k < VPT; ++k) amax[k] = m;
    }
    const int groups = a.group ? (a.dim + 127) >> 7 : 1;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = k * T + t;
      if (v >= nv) continue;
      const float scale = block_scale(amax[k], a.scale_mode);
      uint16_t c[4];
      ScaleDiv(scale).codes_by_reciprocal<4>(h[k], c);
      reinterpret_cast<uint2*>(a.codes + row * a.dim)[v] = make_uint2(c[0] | (uint32_t(c[1]) << 16), c[2] | (uint32_t(c[3]) << 16));
      if (a.group ? (v & 15) == 0 : v == 0) a.scales[row * groups + (a.group ? v >> 4 : 0)] = scale;
    }
  }
};
__device__ __forceinline__ float norm_sum(float x, float y) { return x + y; }

__device__ __forceinline__ const uint4* norm_x(const NormArgs& a, int64_t row) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row * a.x_stride);
}
// Without a residual -0 is added, which leaves every x as it is, zeros of both signs among them.
__device__ __forceinline__ uint4 norm_no_res(const NormArgs& a) {
  const uint32_t z = a.residual ? 0u : 0x80008000u;
  return make_uint4(z, z, z, z);
}
__device__ __forceinline__ const uint4* norm_res(const NormArgs& a, int64_t row) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) + row * a.dim);
}

// Short rows, of up to 8 LANES VPT dims: LANES lanes of a warp a row.
constexpr int kNormSmallThreads = 256;
template <int LANES, int VPT>
__global__ void __launch_bounds__(kNormSmallThreads) add_rmsnorm_small_kernel(const NormArgs a) {
  const int t = threadIdx.x & (LANES - 1), nv = a.dim >> 3;
  const int64_t row = int64_t(blockIdx.x) * (kNormSmallThreads / LANES) + threadIdx.x / LANES;
  const bool real = row < a.n;  // (lanes of rows past the end go along: the warp shuffles together)
  pdl_wait();
  uint4 xv[VPT], rv[VPT], wv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * LANES + t;
    xv[k] = wv[k] = make_uint4(0, 0, 0, 0);
    rv[k] = norm_no_res(a);
    if (real && v < nv) {
      xv[k] = norm_x(a, row)[v];
      if (a.residual) rv[k] = norm_res(a, row)[v];
      wv[k] = __ldg(static_cast<const uint4*>(a.weight) + v);
    }
  }
  pdl_trigger();
  NormArgs b = a;
  if (!real) b.dim = 0;  // nothing of it is stored
  NormRow<LANES, VPT> r;
  const float ss = r.all(r.add(b, row, t, LANES, xv, rv), LANES, nullptr, norm_sum);
  r.finish(b, row, t, LANES, ss, wv, nullptr);
}

// Long rows: a CTA each, four or five an SM, whose loads, sums and stores overlap: 16384 x 7168 with the residual, y and a
// scale a row take 153 us, the measured copy bandwidth (6.9 TB/s). (A CTA that goes from row to row with the next ones on their
// way to shared memory holds fewer rows an SM and is slower: 206 us.)
constexpr int kNormVpt = 4;

template <int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 4 : 1) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  const int t = threadIdx.x, T = blockDim.x, nv = a.dim >> 3;
  const int64_t row = blockIdx.x;
  uint4 xv[kNormVpt], rv[kNormVpt], wv[kNormVpt];
  pdl_wait();
#pragma unroll
  for (int k = 0; k < kNormVpt; ++k) {
    const int v = k * T + t;
    xv[k] = make_uint4(0, 0, 0, 0);
    rv[k] = norm_no_res(a);
    if (v < nv) {
      xv[k] = norm_x(a, row)[v];
      if (a.residual) rv[k] = norm_res(a, row)[v];
    }
  }
  NormRow<0, kNormVpt> r;
  pdl_trigger();
  const float mine = r.add(a, row, t, T, xv, rv);
#pragma unroll
  for (int k = 0; k < kNormVpt; ++k)  // on their way while the threads meet (loaded with the row: 100 bytes of spills, 171 us)
    wv[k] = k * T + t < nv ? __ldg(static_cast<const uint4*>(a.weight) + k * T + t) : make_uint4(0, 0, 0, 0);
  const float ss = r.all(mine, T, part[0], norm_sum);
  r.finish(a, row, t, T, ss, wv, part[1]);
}

// A kernel that starts up while the one before it on the stream ends, and waits for it before it touches memory (pdl_wait).
template <typename A>
cudaError_t launch_early(void (*kernel)(A), int64_t ctas, int threads, const A& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  const int64_t ctas = (a.N + kRdRows - 1) / kRdRows;
  if (a.kv_format == SMLA_KV_BF16) return launch_early(cache_read_kernel<SMLA_KV_BF16>, ctas, kRdThreads, a, s);
  if (a.kv_format == SMLA_KV_FP8_DS) return launch_early(cache_read_kernel<SMLA_KV_FP8_DS>, ctas, kRdThreads, a, s);
  return launch_early(cache_read_kernel<SMLA_KV_FP8_TENSOR>, ctas, kRdThreads, a, s);
}

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  const int nv = a.dim >> 3;
  auto ctas = [&](int lanes) { return (a.n * lanes + kNormSmallThreads - 1) / kNormSmallThreads; };
  if (nv <= 32) return launch_early(add_rmsnorm_small_kernel<16, 2>, ctas(16), kNormSmallThreads, a, s);
  if (nv <= 128) return launch_early(add_rmsnorm_small_kernel<32, 4>, ctas(32), kNormSmallThreads, a, s);
  const int threads = ((nv + kNormVpt - 1) / kNormVpt + 31) & ~31;
  return threads <= 256 ? launch_early(add_rmsnorm_kernel<256>, a.n, threads, a, s)
                        : launch_early(add_rmsnorm_kernel<1024>, a.n, threads, a, s);
}

}  // namespace smla
