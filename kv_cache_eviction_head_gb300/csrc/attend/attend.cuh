// Declarations of the model-side calls over the caches: prompt and tree
// attention (k_attend.cu), key/value store (k_store.cu), path commit
// (k_commit.cu). Host checks and launches: attend_api.cu.
#pragma once

#include "bkv_internal.cuh"

namespace bkv {

constexpr int kMaxNodes = 64;    // one 64-bit ancestor mask per node
constexpr int kMaxGroup = 128;   // query heads per KV head: one token's rows fit a 128-row tile

// Programmatic dependent launch. These kernels are short and follow one another, so
// the next one's blocks may start (and set up barriers and TMEM) while the one
// before still runs: depend_wait() returns when everything before this kernel in
// its stream is complete and visible, and stands before every access to memory
// that other kernels may have written or still read; depend_go() lets the next
// kernel's blocks start once every block of this one has come so far. Between
// kernels that do not take part, launches are ordered as ever.
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void depend_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
inline cudaLaunchAttribute dependent_launch() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

struct AttendParams {
  CUtensorMap qmap;        // queries [tokens][heads][d], box (64, group, tpt)
  CUtensorMap omap;        // out, the same box
  CUtensorMap kmap, vmap;  // caches [batch * kv_heads][max_cache][d], box (64, 128, 1)
  const int32_t* cu;       // prompt: [batch + 1] token offsets; tree: null
  const int32_t* first;    // [batch] slots before the first token / node
  const int32_t* nodes;    // tree: optional [batch] nodes in use
  const int64_t* mask;     // tree: optional [batch][n] ancestor bits (null: a chain)
  __nv_bfloat16* out;      // [tokens][heads][d]
  float* lse;              // optional [tokens][heads]
  uint32_t* status;        // optional
  int batch, heads, kv_heads, group, max_cache;
  int total;               // packed tokens (tree: batch * n)
  int n;                   // tree: nodes per sequence
  int tpt;                 // tokens per 128-row tile
  int qblocks;             // tree: row blocks per (sequence, KV head)
  int stages;              // K/V ring stages
  float scale_log2;        // log2(e) / sqrt(d)
};
// nq: 128-row tiles per CTA (1 or 2); splits: CTAs per row block (1..16, a
// cluster), each taking a share of the keys; items: row blocks to launch.
cudaError_t launch_attend(const AttendParams& p, int nq, int splits, int64_t items, cudaStream_t s);
constexpr int kSms = 152;  // GB300
// CTAs that share an SM: with few rows a CTA waits for its keys most of the time,
// and two hide each other's latencies with three K/V stages each. More rows leave
// two CTAs only two stages; one CTA with six is faster (64 sequences of 80 rows over
// 1040 slots: 56.5 against 59.1 us).
constexpr int attend_ctas_per_sm(int nq, int rows) { return nq == 1 && rows <= 32 ? 2 : 1; }
// K/V ring stages that fit beside the rest of a CTA's shared memory.
int attend_stages(int nq, int group, int tpt);
// Fills p's tensor maps (host only). False on failure.
bool encode_attend_maps(AttendParams& p, const void* q, int64_t q_stride, const void* K, const void* V);

struct StoreParams {
  const uint4* q;          // token t, head h at q + t * q_stride + h * 16 (uint4 units); k, v likewise
  const uint4* k;
  const uint4* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu;       // [batch + 1]
  const int32_t* first;    // [batch] slot of a sequence's first token
  const int32_t* pos;      // [batch] its position
  const int32_t* depth;    // optional [total] offsets from pos (null: the place in the sequence)
  uint4* q_rot;            // [total][heads][d]
  uint4* K;                // [batch][kv_heads][max_cache][d]
  uint4* V;
  uint32_t* status;
  int batch, heads, kv_heads, max_cache, total;
  uint64_t turns[kRopePairs];  // theta^(-2i/d) / (2 pi) as a 64-bit fraction of a turn
};
cudaError_t launch_store(const StoreParams& p, cudaStream_t s);

struct CommitParams {
  uint4* K[kMaxLayers];
  uint4* V[kMaxLayers];
  const int32_t* lens;     // [batch]
  const int32_t* path;     // [batch][n]
  const int32_t* count;    // [batch]
  uint32_t* status;
  int batch, kv_heads, max_cache, n, layers;
};
cudaError_t launch_commit(const CommitParams& p, cudaStream_t s);

}  // namespace bkv
