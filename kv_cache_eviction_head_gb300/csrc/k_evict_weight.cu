// Eviction by accumulated attention weight, for every (layer, sequence, KV head):
//
//   keep = prefix + recent window + the slots with the largest weights, up to the budget
//   (equal weights: the lowest slots; NaN ranks below all numbers),
//   K[i] = K_old[kept[i]], V and weights likewise.
//
// Two launches. The first finds the keep set: a radix select over the weights' order-
// preserving bits (three passes of eleven bits, one histogram each: the first tells the
// exponents and two bits more apart, so that few threads meet in a bin) gives the smallest
// kept weight, a pass over the slots in order writes the kept list. The keys of the first
// 8192 slots stay in shared memory. The second launch moves the rows.
// In slot order kept[i] >= i ascends, so a block that walks up the list and loads a chunk
// of rows before it writes them never overwrites a row that is still to be read. Order-
// free, dropped slots below the budget take kept ones from behind it, which are disjoint.
//
// Bound: HBM; moved rows are read and written once, weights read once.
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;                                    // eleven bits of a key
constexpr int kMostCached = 8192;                              // slots whose keys stay in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;                                  // rows of K and of V per step
constexpr int kMoveLoads = kMoveRows * 32 / kMoveThreads;      // 16-byte pieces per thread and step
constexpr int kMoveWarps = kMoveThreads / 32;

struct Unit {
  int layer, b, h;
  int len;       // clamped
  bool bad;      // length out of range, or too short for an order-free eviction
  bool evicts;
};
__device__ __forceinline__ Unit unit_of(const EvictWeightParams& P) {
  Unit u;
  const int64_t i = blockIdx.x;
  u.h = (int)(i % P.kv_heads);
  u.b = (int)(i / P.kv_heads % P.batch);
  u.layer = (int)(i / ((int64_t)P.kv_heads * P.batch));
  const int given = P.lens[u.b];
  u.len = min(max(given, 0), P.pg.cap);
  u.bad = u.len != given;
  u.evicts = u.len > P.budget;
  if (u.evicts && P.order_free && u.len - P.budget < P.recent) {
    u.bad = true;
    u.evicts = false;
  }
  return u;
}

// Larger key: larger weight. -0 and 0 are equal, NaN is below everything.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t x = __float_as_uint(w + 0.f);
  return (x & 0x80000000u) ? ~x : x | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_weight_kernel(const __grid_constant__ EvictWeightParams P) {
  // the first P.cached slots' keys; order-free: kept slots below the budget as bits, and the
  // kept in front of every word
  extern __shared__ uint32_t dynamic[];
  __shared__ int hist[kBins];
  __shared__ int chosen, left;
  __shared__ int2 warp_sum[kSelectWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  depend_wait();
  depend_go();
  const Unit u = unit_of(P);
  int32_t* kept = P.kept + (int64_t)blockIdx.x * P.budget;
  if (tid == 0) {
    if (u.bad) latch(P.status, BKV_ERR_INVALID_ARG);
    if (P.new_lens && u.layer == 0 && u.h == 0) P.new_lens[u.b] = u.evicts ? P.budget : u.len;
  }
  if (!u.evicts) {
    // within the budget everything stays; a refused sequence has no keep set
    for (int i = tid; i < P.budget; i += kSelectThreads) kept[i] = i < u.len && u.len <= P.budget ? i : -1;
    return;
  }
  const float* W = P.W[u.layer];
  const int from = P.prefix, to = u.len - P.recent;  // candidates
  auto read_key = [&](int slot) {
    const int64_t row = pool_row(P.pg, P.kv_heads, u.b, u.h, slot);
    if (row < 0) {
      latch(P.status, BKV_ERR_INVALID_ARG);
      return 0u;
    }
    return BKV_IN_RANGE(row < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status) ? key_of(W[row]) : 0u;
  };
  uint32_t* cache = dynamic;
#pragma unroll 8
  for (int s = tid; s < min(to, P.cached); s += kSelectThreads) cache[s] = s >= from ? read_key(s) : 0u;
  // a thread only reads keys that it wrote itself
  auto key = [&](int slot) { return slot < P.cached ? cache[slot] : read_key(slot); };
  int need = P.budget - P.prefix - P.recent;  // of the candidates, fewer than there are
  uint32_t least = 0, known = 0;              // the smallest kept key, as far as its bits are known
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
#pragma unroll
      for (int i = 0; i < kBins / kSelectThreads; ++i) hist[i * kSelectThreads + tid] = 0;
      __syncthreads();
      for (int s = tid; s < to; s += kSelectThreads) {
        if (s < from) continue;
        const uint32_t k = key(s);
        if ((k & known) == least) atomicAdd(&hist[k >> shift & digit], 1);
      }
      __syncthreads();
      // the bin, from the top, in which the need-th largest lies: eight bins a thread
      int mine[kBins / kSelectThreads], sum = 0;
#pragma unroll
      for (int i = 0; i < kBins / kSelectThreads; ++i) {
        mine[i] = hist[kBins - 1 - (tid * (kBins / kSelectThreads) + i)];
        sum += mine[i];
      }
      int upto = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kAll, upto, off);
        if (lane >= off) upto += y;
      }
      if (lane == 31) warp_sum[warp].x = upto;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSelectWarps; ++k)
        if (k < warp) upto += warp_sum[k].x;
      if (upto - sum < need && upto >= need) {
        int above = upto - sum, i = 0;
        while (i < kBins / kSelectThreads - 1 && above + mine[i] < need) above += mine[i++];
        chosen = kBins - 1 - (tid * (kBins / kSelectThreads) + i);
        left = need - above;
      }
      __syncthreads();
      least |= (uint32_t)chosen << shift;
      known |= digit << shift;
      need = left;  // how many of those equal so far are kept
    }
  }
  const int ties = need;  // of the slots whose key is `least`, the lowest
  const bool any = P.budget - P.prefix - P.recent > 0;
  int above = 0, equal = 0;  // kept beyond the ties, and ties, in front of the slots looked at
  const int words = (P.budget + 31) / 32;
  uint32_t* bits = dynamic + P.cached;
  int* in_front = reinterpret_cast<int*>(bits + words);
  int below = 0;  // order-free: kept slots below the budget
  for (int s0 = 0; s0 < u.len; s0 += kSelectThreads) {
    const int s = s0 + tid;
    bool gt = false, eq = false;
    if (s < u.len) {
      if (s < from || s >= to) gt = true;
      else if (any) {
        const uint32_t k = key(s);
        gt = k > least;
        eq = k == least;
      }
    }
    const unsigned bg = __ballot_sync(kAll, gt), be = __ballot_sync(kAll, eq);
    if (lane == 0) warp_sum[warp] = make_int2(__popc(bg), __popc(be));
    __syncthreads();
    int g = above, e = equal;
#pragma unroll
    for (int k = 0; k < kSelectWarps; ++k) {
      const int2 x = warp_sum[k];
      if (k < warp) {
        g += x.x;
        e += x.y;
      }
      above += x.x;
      equal += x.y;
    }
    const unsigned lower = (1u << lane) - 1;
    g += __popc(bg & lower);
    e += __popc(be & lower);
    const bool keep = gt || (eq && e < ties);
    const int at = g + min(e, ties);  // kept slots in front of s
    if (!P.order_free) {
      if (keep && at < P.budget) kept[at] = s;
    } else {
      const unsigned bk = __ballot_sync(kAll, keep && s < P.budget);
      if (lane == 0 && s < P.budget) {
        bits[s >> 5] = bk;
        in_front[s >> 5] = at;
      }
      if (keep && s < P.budget) kept[s] = s;
    }
    __syncthreads();
    if (P.order_free && s0 + kSelectThreads >= P.budget && s0 < P.budget) {
      // the last word below the budget is written: kept slots below it
      below = in_front[words - 1] + __popc(bits[words - 1]);
    }
    if (P.order_free && keep && s >= P.budget) {
      // the (at - below)-th dropped slot below the budget takes this one
      const int t = at - below;
      int lo = 0, hi = words - 1;  // the last word with at most t dropped slots in front
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mid * 32 - in_front[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      uint32_t holes = ~bits[lo];
      for (int skip = t - (lo * 32 - in_front[lo]); skip > 0; --skip) holes &= holes - 1;
      const int hole = lo * 32 + __ffs(holes) - 1;
      if (holes != 0 && hole < P.budget) kept[hole] = s;
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_weight_kernel(const __grid_constant__ EvictWeightParams P) {
  __shared__ int64_t src[2 * kMoveThreads], dst[2 * kMoveThreads];  // rows that move
  __shared__ int moved_in[kMoveWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  depend_wait();
  depend_go();
  const Unit u = unit_of(P);
  if (!u.evicts) return;
  const int32_t* kept = P.kept + (int64_t)blockIdx.x * P.budget;
  uint4* pool = tid & 16 ? P.V[u.layer] : P.K[u.layer];
  float* W = P.W[u.layer];
  const int part = tid & 15;
  int count = 0;  // rows in the list
  for (int i0 = 0; i0 < P.budget; i0 += kMoveThreads) {
    const int i = i0 + tid;
    const int from = i < P.budget ? kept[i] : i;
    int64_t a = -1, b = -1;
    if (from != i && from >= 0 && from < u.len) {
      a = pool_row(P.pg, P.kv_heads, u.b, u.h, from);
      b = pool_row(P.pg, P.kv_heads, u.b, u.h, i);
      if (a < 0 || b < 0) latch(P.status, BKV_ERR_INVALID_ARG);
      if (b < 0 || !BKV_IN_RANGE(max(a, b) < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) a = -1;
    }
    const unsigned moving = __ballot_sync(kAll, a >= 0);
    if (lane == 0) moved_in[warp] = __popc(moving);
    __syncthreads();
    int at = count + __popc(moving & ((1u << lane) - 1));
#pragma unroll
    for (int k = 0; k < kMoveWarps; ++k) {
      const int n = moved_in[k];
      if (k < warp) at += n;
      count += n;
    }
    if (a >= 0) {
      src[at] = a;
      dst[at] = b;
    }
    __syncthreads();
    if (count <= kMoveThreads && i0 + kMoveThreads < P.budget) continue;
    // The next step's rows are loaded before this step's are written: their sources lie
    // behind all that this step writes.
    uint4 x[kMoveLoads], y[kMoveLoads];
    float wx = 0.f, wy = 0.f;
    auto load = [&](int c, uint4 (&v)[kMoveLoads], float& w) {
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kMoveWarps + warp;
        if (r < count) v[k] = pool[src[r] * 16 + part];
      }
      if (tid < kMoveRows && c + tid < count) w = W[src[c + tid]];
    };
    load(0, x, wx);
    for (int c = 0; c < count; c += kMoveRows) {
      load(c + kMoveRows, y, wy);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kMoveWarps + warp;
        if (r < count) pool[dst[r] * 16 + part] = x[k];
        x[k] = y[k];
      }
      if (tid < kMoveRows && c + tid < count) W[dst[c + tid]] = wx;
      wx = wy;
    }
    count = 0;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict_weight(const EvictWeightParams& given, cudaStream_t s) {
  EvictWeightParams p = given;
  p.cached = p.pg.cap < kMostCached ? p.pg.cap : kMostCached;
  const size_t mask = (size_t)p.cached * 4 + (p.order_free ? (size_t)((p.budget + 31) / 32) * 8 : 0);
  cudaError_t e = cudaFuncSetAttribute(select_weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p.layers * p.batch * p.kv_heads));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = mask;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select_weight_kernel, p);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, move_weight_kernel, p);
}

}  // namespace bkv
