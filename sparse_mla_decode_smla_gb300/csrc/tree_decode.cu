// Attention of drafted nodes over the paged latent cache: every node of a request attends the
// request's context and the nodes it sees (a bit mask, or the chain j <= i).
//
// out_h = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink_h}), s_j = sm_scale <q_h, k_j>, v_j = k_j[0:512],
// in one pass over the slots with a running maximum and sum.
#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"
#include "tree_decode.h"

namespace smla {
namespace {

// One warp per (node, head). Lane l holds dims [16 l, 16 l + 16) of the latent and [2 l, 2 l + 2)
// of the RoPE part.
__global__ void __launch_bounds__(256) tree_simple_kernel(const TreeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (item >= int64_t(p.T) * p.H) return;
  const int t = static_cast<int>(item / p.H), h = static_cast<int>(item % p.H);
  int r = -1, cu0 = 0, n = 0;
  for (int i = 0; i < p.B; ++i) {
    const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
    if (t >= a && t < b) { r = i; cu0 = a; n = b - a; }
  }
  if (r < 0) return;
  int32_t* err = reinterpret_cast<int32_t*>(p.ws);
  const int ctx = __ldg(p.ctx + r), i = t - cu0;
  if (cu0 < 0 || cu0 + n > p.T || ctx < 0 || (p.mask && n > 32 * p.W) ||
      int64_t(ctx) + n > (int64_t(p.stride) << p.log2_page)) {
    if (lane == 0) atomicOr(err, SMLA_DEVERR_INDEX);
    return;
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + item * kDim;
  float ql[16], qr[2], o[16];
  for (int e = 0; e < 16; ++e) { ql[e] = __bfloat162float(q[16 * lane + e]); o[e] = 0.f; }
  for (int e = 0; e < 2; ++e) qr[e] = __bfloat162float(q[kLatent + 2 * lane + e]);
  float m = -CUDART_INF_F, l = 0.f;
  for (int s = 0; s < ctx + n; ++s) {
    if (s >= ctx) {
      const int j = s - ctx;
      const bool see = p.mask ? (p.mask[int64_t(t) * p.W + (j >> 5)] >> (j & 31)) & 1u : j <= i;
      if (!see) continue;
    }
    const int32_t page = __ldg(p.page_table + int64_t(r) * p.stride + (s >> p.log2_page));
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(err, SMLA_DEVERR_PAGE);
      continue;
    }
    const int64_t slot = (int64_t(page) << p.log2_page) + (s & ((1 << p.log2_page) - 1));
    float k[16], kr[2];
    if (p.kv_format == SMLA_KV_BF16) {
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(p.kv + slot * kBf16RowBytes);
      for (int e = 0; e < 16; ++e) k[e] = __bfloat162float(row[16 * lane + e]);
      for (int e = 0; e < 2; ++e) kr[e] = __bfloat162float(row[kLatent + 2 * lane + e]);
    } else {
      const bool ds = p.kv_format == SMLA_KV_FP8_DS;
      const uint8_t* row = p.kv + slot * (ds ? kFp8RowBytes : kFp8TensorRowBytes);
      const float sc = ds ? reinterpret_cast<const float*>(row + kScaleOff)[lane >> 3] : p.kv_scale;
      for (int e = 0; e < 16; e += 2) {
        const uint32_t x = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(row + 16 * lane + e));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
        k[e] = f.x * sc;
        k[e + 1] = f.y * sc;
      }
      if (ds) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(row + kRopeOffFp8)[lane];
        kr[0] = bf16_lo(w);
        kr[1] = bf16_hi(w);
      } else {
        const uint32_t x = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(row + kLatent + 2 * lane));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
        kr[0] = f.x * sc;
        kr[1] = f.y * sc;
      }
    }
    float d = qr[0] * kr[0] + qr[1] * kr[1];
    for (int e = 0; e < 16; ++e) d = fmaf(ql[e], k[e], d);
    for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    const float sc2 = d * p.c2;
    if (sc2 > m) {
      const float a = exp2f(m - sc2);
      l *= a;
      for (int e = 0; e < 16; ++e) o[e] *= a;
      m = sc2;
    }
    const float w = exp2f(sc2 - (m == -CUDART_INF_F ? 0.f : m));
    l += w;
    for (int e = 0; e < 16; ++e) o[e] = fmaf(w, k[e], o[e]);
  }
  float lse = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
  float f = l == 0.f ? 0.f : 1.f / l;
  if (p.sink) {
    const float sg = __ldg(p.sink + h);
    if (sg != -CUDART_INF_F) {
      const float both = fmaxf(lse, sg) + log1pf(expf(-fabsf(lse - sg)));
      f *= expf(lse - both);
      lse = both;
    }
  }
  if (p.lse && lane == 0) p.lse[item] = lse;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + item * kLatent + 16 * lane);
  uint32_t w[8];
  for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[2 * e] * f, o[2 * e + 1] * f);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace

size_t tree_workspace_bytes(int) { return 256; }

cudaError_t launch_tree_decode(const TreeArgs& a, int, cudaStream_t s) {
  const int64_t blocks = (int64_t(a.T) * a.H + 7) / 8;
  tree_simple_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace smla
