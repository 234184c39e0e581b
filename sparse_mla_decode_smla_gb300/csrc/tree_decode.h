// Internal launcher of the tree attention (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/smla.h"

namespace smla {

constexpr int kTreeMaxRequests = 1 << 16;

struct TreeArgs {
  const void* q;
  const uint8_t* kv;
  const int32_t* page_table;
  const int32_t* ctx;
  const int32_t* cu;
  const uint32_t* mask;
  const float* sink;
  void* out;
  float* lse;
  uint8_t* ws;  // error word at 0; from byte 256 on what each run leaves for joining, then the runs' parts
  int32_t T, H, B, W, stride, log2_page, kv_format;
  int64_t num_pages;
  float c2;        // sm_scale * log2(e)
  float kv_scale;  // per-tensor scale (1 for the other formats)
};

size_t tree_workspace_bytes(int num_sms);
cudaError_t launch_tree_decode(const TreeArgs& a, int num_sms, cudaStream_t s);

}  // namespace smla
