// Argument checks shared by the host sides of the model-side calls.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "attend/attend.cuh"

namespace bkv {
namespace host {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The checks of bkv_create's config, and what these kernels need of it.
inline bkv_status check(const bkv_config* c) {
  size_t bytes = 0;
  const bkv_status st = bkv_workspace_bytes(c, &bytes);
  if (st != BKV_OK) return st;
  if (c->heads / c->kv_heads > bkv::kMaxGroup) return BKV_ERR_UNSUPPORTED;
  return BKV_OK;
}

// A packed [tokens][heads][d] tensor whose tokens lie `stride` elements apart
// (no tokens: the pointer is not looked at).
inline bool strided_ok(const void* p, int64_t stride, int heads, int d, int tokens) {
  return (tokens == 0 || p) && aligned(p, 16) && stride >= (int64_t)heads * d && stride % 8 == 0 && stride < (1ll << 38);
}

inline bkv_status zero_status(uint32_t* status, cudaStream_t s) {
  if (status && cudaMemsetAsync(status, 0, sizeof(uint32_t), s) != cudaSuccess) return BKV_ERR_CUDA;
  return BKV_OK;
}

}  // namespace host
}  // namespace bkv
