// Declarations of the calls over paged caches: rotary store (k_store_paged.cu),
// attention of one new token (k_attend_paged.cu), prompt weights (k_weigh.cu),
// eviction by accumulated weight (k_evict_weight.cu). Host checks and launches:
// paged_api.cu.
#pragma once

#include <atomic>

#include "attend/attend.cuh"

namespace bkv {

// Slots of sequence b: slot j lies in page table[b][j / page_size] at place
// j % page_size; without a table the sequence's only page is page b. Page sizes
// under a table are multiples of 16, so 16 aligned slots lie in one page.
struct Pages {
  const int32_t* table;  // [batch][per_seq] or null
  int pages, page_size, per_seq;
  int cap;               // per_seq * page_size: slots a sequence may hold
  uint32_t mul, shift;   // j / page_size = (j * mul) >> shift, j < 2^31
};
// mul and shift for d in 1 .. 2^31 - 1 and j < 2^31: with L = ceil(log2 d) and
// mul = ceil(2^(31 + L) / d) the error j (mul d - 2^(31+L)) / (d 2^(31+L)) is below
// 2^31 / 2^(31+L) <= 1 / d, so the floor is that of j / d.
inline void set_division(Pages& p) {
  int l = 0;
  while ((1ull << l) < (unsigned long long)p.page_size) ++l;
  p.mul = (uint32_t)(((1ull << (31 + l)) + (unsigned)p.page_size - 1) / (unsigned)p.page_size);
  p.shift = 31 + l;
}
__device__ __forceinline__ int page_of(const Pages& p, int slot) {
  return (int)(((uint64_t)(uint32_t)slot * p.mul) >> p.shift);
}
// The pool's page for a sequence's page k, or -1 if the table names none.
__device__ __forceinline__ int pool_page(const Pages& p, int b, int k) {
  if (!p.table) return b;
  const int x = p.table[(int64_t)b * p.per_seq + k];
  return x >= 0 && x < p.pages ? x : -1;
}
// Row of a pool [pages][kv_heads][page_size] that holds slot `slot`, or -1.
__device__ __forceinline__ int64_t pool_row(const Pages& p, int kv_heads, int b, int h, int slot) {
  const int k = page_of(p, slot);
  const int page = pool_page(p, b, k);
  return page < 0 ? -1 : ((int64_t)page * kv_heads + h) * p.page_size + (slot - k * p.page_size);
}

// Allows a kernel its dynamic shared memory, once per device (a bit each; devices beyond
// the 64th every time).
template <typename Kernel>
cudaError_t allow_shared(Kernel fn, int bytes, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (configured.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured.fetch_or(bit);
  return e;
}

struct StorePagedParams {
  Pages pg;
  const uint4* q;          // token t, head h at q + t * q_stride + h * 16 (uint4 units); k, v likewise
  const uint4* k;
  const uint4* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu;       // [batch + 1]
  const int32_t* first;    // [batch] slot of a sequence's first token
  const int32_t* pos;      // [batch] its position
  const int32_t* depth;    // optional [total] offsets from pos (null: the place in the sequence)
  uint4* q_rot;            // [total][heads][d]
  uint4* K;
  uint4* V;
  uint32_t* status;
  int batch, heads, kv_heads, total;
  int rotary;              // rotated elements, a multiple of 16
  int interleaved;
  float scale;             // of cosines and sines
  uint64_t turns[kRopePairs];  // turns per position of every pair, as a 64-bit fraction
};
cudaError_t launch_store_paged(const StorePagedParams& p, cudaStream_t s);

// Attention of one token: the visible tiles of all (sequence, KV head, chunk of query
// heads) units stand in a row and are dealt out evenly to the warps of one launch.
constexpr int kAttendWarps = 5;                               // per CTA, at most
constexpr int kAttendCtas = 2 * kSms;                         // two per SM
constexpr int kAttendShares = kAttendCtas * kAttendWarps;     // warps of a launch, at most
constexpr int kTileSlots = 16;
struct AttendPagedParams {
  CUtensorMap kmap, vmap;  // pools [pages * kv_heads][page_size][d], box (64, 16, 1)
  Pages pg;
  const uint4* q;          // sequence b, head h at q + b * q_stride + h * 16 (uint4 units)
  int64_t q_stride;
  const uint4* K;
  const uint4* V;
  const int32_t* lens;     // [batch] visible slots
  uint4* out;              // [batch][heads][d]
  float* lse;              // optional [batch][heads]
  float* weights;          // optional [pages][kv_heads][page_size]
  uint32_t* status;
  float decay;
  float scale_log2;        // log2(e) / sqrt(d)
  int batch, heads, kv_heads, group;
  int chunk;               // query heads per unit: 8 or 16
  int chunks;              // units per KV head
  int shares;              // warps of the launch (set by the launch)
  int64_t tiles_cap;       // tiles the logits have room for
  // workspace
  float2* part_ml;         // [2 * shares][16] reference maximum (log2) and sum of a piece
  float4* part_o;          // [2 * shares][chunk][d / 4]
  float* lse2;             // [batch][heads] log2 of the sum, of units done by one warp
  int2* seq;               // [batch + 1] tiles in front of a sequence (all of them), its length
  float* logits;           // [tile][group][16], log2 units; with weights only
};
cudaError_t launch_attend_paged(const AttendPagedParams& p, cudaStream_t s);
// Fills p's tensor maps (host only). False on failure.
bool encode_attend_paged_maps(AttendPagedParams& p);

constexpr int kWeighRows = 96;  // query rows per tile: query heads per KV head, at most
struct WeighParams {
  CUtensorMap qmap;        // queries [tokens][heads][d], box (64, group, tpt)
  Pages pg;
  const uint4* K;
  const float* row_lse;    // [total][heads]
  const int32_t* cu;       // [batch + 1]
  const int32_t* first;    // [batch]
  float* weights;
  uint32_t* status;
  float decay;
  float scale_log2;
  int batch, heads, kv_heads, group, total;
  int tpt;                 // tokens per tile of query rows
  int splits;              // CTAs that share a tile of slots (set by the launch)
  int items;               // as given to the launch, fewer than 2^31 - 4096
};
// items: (sequence, KV head, tile of 128 slots) triples there can be
cudaError_t launch_weigh(const WeighParams& p, int64_t items, cudaStream_t s);
// Fills p's tensor map (host only). False on failure.
bool encode_weigh_map(WeighParams& p, const void* q, int64_t q_stride);

struct EvictWeightParams {
  Pages pg;
  uint4* K[kMaxLayers];
  uint4* V[kMaxLayers];
  float* W[kMaxLayers];
  const int32_t* lens;     // [batch]
  int32_t* kept;           // [layers][batch][kv_heads][budget]
  int32_t* new_lens;       // optional [batch]
  uint32_t* status;
  int layers, batch, kv_heads, budget, prefix, recent;
  int order_free;
  int cached;              // slots whose keys the selection keeps on chip (set by the launch)
};
cudaError_t launch_evict_weight(const EvictWeightParams& p, cudaStream_t s);

}  // namespace bkv
