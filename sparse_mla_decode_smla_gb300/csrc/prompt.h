// Internal launchers of the operators around a prompt (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/smla.h"

namespace smla {

struct ReadArgs {
  const uint8_t* kv;
  const int32_t* page_table;
  const int32_t* starts;
  const int32_t* cu;
  void* latent;
  void* rope;
  int32_t* err;
  int32_t B, stride, log2_page, kv_format;
  int64_t num_pages, N, latent_stride, rope_stride;
  float kv_scale;
};
cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s);

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum;
  void* y;
  uint8_t* codes;
  float* scales;
  int64_t n, x_stride;
  int32_t dim, group, scale_mode;
  float eps;
};
constexpr int kNormMaxDim = 32768;
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);

struct LogprobArgs {
  const void* x;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* err;
  int64_t n, stride;
  int32_t V, given, top, f32;
  float scale;
};
constexpr int kLogprobMaxTop = 64, kLogprobMaxGiven = 1024, kLogprobMaxVocab = 1 << 24;
cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t s);

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* rope;         // NULL: none
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* prefix;    // NULL: none
  const float* slopes;      // NULL: none
  const float* sink;        // NULL: none
  void* out;
  float* lse;
  uint8_t* ws;              // error word and item counters
  int32_t* counts;          // [SM][row tile]: pieces that have ended, zero between calls
  uint8_t* table;           // a line a request
  float* parts;             // two an SM
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, rope_token;  // strides in elements
  int32_t T, N, H, HK, B, causal, log2_pack, sms;
  float c2;                 // sm_scale log2(e)
  float cap2, cap_in;       // cap log2(e) (0: no cap); 2 sm_scale log2(e) / cap
  float tanh_max;           // scores q.k up to this are capped by the polynomial
  float tanh_c[5];          // its coefficients, of odd powers of q.k
};
struct PromptLayout {
  size_t counts, table, parts, bytes;
};
PromptLayout prompt_layout(int64_t requests, int num_sms);
constexpr int kPromptMaxRequests = 1 << 16;
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s);

}  // namespace smla
