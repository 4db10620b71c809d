// Moves an accepted path's rows to the end of the cache, in every layer:
//
//   K[len + i] = K_old[len + path[i]], V likewise, i < count
//
// One block per (layer, sequence, KV head) loads every row of the path into
// registers before it writes the first one, so a path may be in any order and
// name a node twice; units do not overlap. Rows that stay (path[i] = i) are
// neither read nor written. Bound: a block's chain of dependent loads (length, path,
// rows). A batch is some 20 rounds of five blocks per SM (40 layers, 48 sequences, 8 KV
// heads, 14.4 moved rows on average, 227 MB: 48 us, 4.7 TB/s; DRAM is 46 % busy), one
// sequence a single round (36 layers: 1.5 us a call in a captured graph).
#include "attend/attend.cuh"

namespace bkv {
namespace {

constexpr int kThreadsCommit = 256;
// 16 threads per row and tensor: 8 rows of K and of V per step
constexpr int kRowsPerStep = kThreadsCommit / 32;
constexpr int kSteps = kMaxNodes / kRowsPerStep;

__global__ void __launch_bounds__(kThreadsCommit) commit_kernel(const __grid_constant__ CommitParams P) {
  const int64_t u = blockIdx.x;
  const int h = (int)(u % P.kv_heads);
  const int b = (int)(u / P.kv_heads % P.batch);
  const int layer = (int)(u / ((int64_t)P.kv_heads * P.batch));
  const int tid = threadIdx.x;
  const int part = tid & 15, r = tid >> 5;
  uint4* base = ((tid & 16) ? P.V[layer] : P.K[layer]) + ((int64_t)b * P.kv_heads + h) * P.max_cache * 16 + part;
  depend_wait();
  depend_go();
  const int len = P.lens[b], given = P.count[b];
  const int count = min(max(given, 0), P.n);
  bool bad = count != given || len < 0 || len > P.max_cache;
  uint4 x[kSteps];
  bool move[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int i = k * kRowsPerStep + r;
    move[k] = false;
    if (i < count) {
      const int from = P.path[(int64_t)b * P.n + i];
      const bool ok = from >= 0 && from < P.n && len >= 0 && (int64_t)len + max(from, i) < P.max_cache;
      bad |= !ok;
      move[k] = ok && from != i;
      if (move[k]) x[k] = base[((int64_t)len + from) * 16];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    if (move[k]) base[((int64_t)len + k * kRowsPerStep + r) * 16] = x[k];
  if (bad) latch(P.status, BKV_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_commit(const CommitParams& p, cudaStream_t s) {
  const int64_t units = (int64_t)p.layers * p.batch * p.kv_heads;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(kThreadsCommit);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, commit_kernel, p);
}

}  // namespace bkv
