// Eviction by accumulated attention weight, for every (layer, sequence, KV head):
//
//   keep = prefix + recent window + the slots with the largest weights, up to the budget
//   (equal weights: the lowest slots; NaN ranks below all numbers),
//   K[i] = K_old[kept[i]], V and weights likewise.
//
// Two launches. The first finds the keep set: a radix select over the weights' order-
// preserving bits (four passes of eight bits, one histogram each) gives the smallest kept
// weight, a pass over the slots in order writes the kept list. The second moves the rows.
// In slot order kept[i] >= i ascends, so a block that walks up the list and loads a chunk
// of rows before it writes them never overwrites a row that is still to be read. Order-
// free, dropped slots below the budget take kept ones from behind it, which are disjoint.
//
// Bound: HBM; moved rows are read and written once, weights read by each pass (from L2).
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;                                  // rows of K and of V per step
constexpr int kMoveLoads = kMoveRows * 32 / kMoveThreads;      // 16-byte pieces per thread and step

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
  extern __shared__ uint32_t mask_words[];  // order-free: kept slots below the budget as bits, then the kept in front of every word
  __shared__ int hist[256];
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
  auto key = [&](int slot) {
    const int64_t row = pool_row(P.pg, P.kv_heads, u.b, u.h, slot);
    if (row < 0) {
      latch(P.status, BKV_ERR_INVALID_ARG);
      return 0u;
    }
    return BKV_IN_RANGE(row < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status) ? key_of(W[row]) : 0u;
  };
  int need = P.budget - P.prefix - P.recent;  // of the candidates, fewer than there are
  uint32_t least = 0, known = 0;              // the smallest kept key, as far as its bits are known
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int s = from + tid; s < to; s += kSelectThreads) {
        const uint32_t k = key(s);
        if ((k & known) == least) atomicAdd(&hist[k >> shift & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // the bin, from the top, in which the need-th largest lies: eight bins a lane
        int mine[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mine[i] = hist[255 - (lane * 8 + i)];
          sum += mine[i];
        }
        int upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(kAll, upto, off);
          if (lane >= off) upto += y;
        }
        const unsigned hit = __ballot_sync(kAll, upto >= need);
        if (lane == __ffs(hit) - 1) {
          int above = upto - sum, i = 0;
          while (i < 7 && above + mine[i] < need) above += mine[i++];
          chosen = 255 - (lane * 8 + i);
          left = need - above;
        }
      }
      __syncthreads();
      least |= (uint32_t)chosen << shift;
      known |= 255u << shift;
      need = left;  // how many of those equal so far are kept
    }
  }
  const int ties = need;  // of the slots whose key is `least`, the lowest
  const bool any = P.budget - P.prefix - P.recent > 0;
  int above = 0, equal = 0;  // kept beyond the ties, and ties, in front of the slots looked at
  const int words = (P.budget + 31) / 32;
  uint32_t* bits = mask_words;
  int* in_front = reinterpret_cast<int*>(mask_words + words);
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
  __shared__ int64_t src[kMoveRows], dst[kMoveRows];
  const int tid = threadIdx.x;
  depend_wait();
  depend_go();
  const Unit u = unit_of(P);
  if (!u.evicts) return;
  const int32_t* kept = P.kept + (int64_t)blockIdx.x * P.budget;
  uint4* pool[2] = {P.K[u.layer], P.V[u.layer]};
  float* W = P.W[u.layer];
  const int part = tid & 15, kv = tid >> 4 & 1, r = tid >> 5;
  for (int i0 = 0; i0 < P.budget; i0 += kMoveRows) {
    float w = 0.f;
    bool moves = false;
    if (tid < kMoveRows) {
      const int i = i0 + tid;
      const int from = i < P.budget ? kept[i] : i;
      int64_t a = -1, b = -1;
      if (from != i && from >= 0 && from < u.len) {
        a = pool_row(P.pg, P.kv_heads, u.b, u.h, from);
        b = pool_row(P.pg, P.kv_heads, u.b, u.h, i);
        if (a < 0 || b < 0) {
          latch(P.status, BKV_ERR_INVALID_ARG);
        } else if (BKV_IN_RANGE(max(a, b) < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) {
          moves = true;
          w = W[a];
        }
      }
      src[tid] = moves ? a : -1;
      dst[tid] = b;
    }
    if (!__syncthreads_or(moves)) continue;
    uint4 x[kMoveLoads];
#pragma unroll
    for (int k = 0; k < kMoveLoads; ++k) {
      const int64_t a = src[k * (kMoveThreads / 32) + r];
      if (a >= 0) x[k] = pool[kv][a * 16 + part];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveLoads; ++k) {
      const int at = k * (kMoveThreads / 32) + r;
      if (src[at] >= 0) pool[kv][dst[at] * 16 + part] = x[k];
    }
    if (moves) W[dst[tid]] = w;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict_weight(const EvictWeightParams& p, cudaStream_t s) {
  const size_t mask = p.order_free ? (size_t)((p.budget + 31) / 32) * 8 : 0;
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
