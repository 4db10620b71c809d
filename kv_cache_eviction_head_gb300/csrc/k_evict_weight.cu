// Eviction by accumulated attention weight, for every (layer, sequence, KV head):
//
//   keep = prefix + recent window + the slots with the largest weights, up to the budget
//   (equal weights: the lowest slots; NaN ranks below all numbers),
//   K[i] = K_old[kept[i]], V and weights likewise.
//
// One block per unit. A radix select over the weights' order-preserving bits gives the
// smallest kept weight: a histogram of the top eleven bits (the exponents and two bits more,
// so that few threads meet in a bin) leaves one bin, whose keys are ranked against each
// other if they are few and told apart by their next bits otherwise. A pass over the slots
// writes the kept list. The keys of the first 8192 slots stay in shared memory. Then the
// rows move: in slot order kept[i] >= i ascends, so a block that walks up the list and loads
// rows before it writes in front of them never overwrites one that is still to be read.
// Order-free, dropped slots below the budget take kept ones from behind it, which are
// disjoint.
//
// Bound: HBM; moved rows are read and written once, weights read once. In one launch a
// block's selection, which is latency, lies under the copies of others.
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kEvictThreads = 256;
constexpr int kEvictCtas = 4;                               // per SM
constexpr int kWarps = kEvictThreads / 32;
constexpr int kBins = 2048;                                 // eleven bits of a key
constexpr int kPerThread = kBins / kEvictThreads;
constexpr int kMostCached = 8192;                           // slots whose keys stay in shared memory
constexpr int kFew = kEvictThreads;                         // keys of a bin that are ranked directly
constexpr int kMoveRows = 32;                               // rows of K and of V per step
constexpr int kMoveLoads = kMoveRows * 32 / kEvictThreads;  // 16-byte pieces per thread and step

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

struct Shared {
  union {
    int hist[kBins];         // in descending order of the digits
    uint32_t few[kFew];      // keys of the bin in question
    struct {
      int64_t src[kEvictThreads * 2], dst[kEvictThreads * 2];  // rows that move
    } list;
  };
  int chosen, left, found;
  int2 warp_sum[kWarps];
};

__global__ void __launch_bounds__(kEvictThreads, kEvictCtas) evict_weight_kernel(const __grid_constant__ EvictWeightParams P) {
  // the first P.cached slots' keys; order-free: kept slots below the budget as bits, and the
  // kept in front of every word
  extern __shared__ uint32_t dynamic[];
  __shared__ __align__(16) Shared S;
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
    for (int i = tid; i < P.budget; i += kEvictThreads) kept[i] = i < u.len && u.len <= P.budget ? i : -1;
    return;
  }
  float* W = P.W[u.layer];
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
  for (int s = tid; s < min(to, P.cached); s += kEvictThreads) cache[s] = s >= from ? read_key(s) : 0u;
  auto key = [&](int slot) { return slot < P.cached ? cache[slot] : read_key(slot); };

  // The smallest kept key, as far as its bits are known, and how many of those equal in these
  // bits are kept (the lowest slots): `need`.
  int need = P.budget - P.prefix - P.recent;  // of the candidates, fewer than there are
  const bool any = need > 0;
  uint32_t least = 0, known = 0;
  for (int shift = 21; any && shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
    const uint32_t digit = shift == 0 ? 1023u : 2047u;
    int4* clear = reinterpret_cast<int4*>(S.hist);
    clear[tid] = clear[tid + kEvictThreads] = make_int4(0, 0, 0, 0);
    if (tid == 0) S.found = 0;
    __syncthreads();
    for (int s = tid; s < to; s += kEvictThreads) {
      if (s < from) continue;
      const uint32_t k = key(s);
      if ((k & known) == least) atomicAdd(&S.hist[kBins - 1 - (k >> shift & digit)], 1);
    }
    __syncthreads();
    // the bin, from the top, in which the need-th largest lies: eight bins a thread
    int mine[kPerThread], sum = 0;
    *reinterpret_cast<int4*>(&mine[0]) = reinterpret_cast<const int4*>(S.hist)[2 * tid];
    *reinterpret_cast<int4*>(&mine[4]) = reinterpret_cast<const int4*>(S.hist)[2 * tid + 1];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) sum += mine[i];
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, off);
      if (lane >= off) upto += y;
    }
    if (lane == 31) S.warp_sum[warp].x = upto;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
      if (k < warp) upto += S.warp_sum[k].x;
    if (upto - sum < need && upto >= need) {
      int above = upto - sum, in = mine[0], bin = tid * kPerThread;
#pragma unroll
      for (int i = 1; i < kPerThread; ++i) {
        if (above + in >= need) break;
        above += in;
        in = mine[i];
        bin = tid * kPerThread + i;
      }
      S.chosen = kBins - 1 - bin;
      S.left = need - above;
      S.warp_sum[0].y = in;
    }
    __syncthreads();
    const int in_bin = S.warp_sum[0].y;
    least |= (uint32_t)S.chosen << shift;
    known |= digit << shift;
    need = S.left;
    if (in_bin == need || shift == 0) break;  // all of the bin are kept, or all equal
    if (in_bin <= kFew) {
      // few: each counts those above it
      __syncthreads();
      for (int s = tid; s < to; s += kEvictThreads) {
        if (s < from) continue;
        const uint32_t k = key(s);
        if ((k & known) == least) {
          const int at = atomicAdd(&S.found, 1);
          if (at < kFew) S.few[at] = k;
        }
      }
      __syncthreads();
      if (tid < in_bin) {
        const uint32_t k = S.few[tid];
        int above = 0, same = 0;
        for (int i = 0; i < in_bin; ++i) {
          const uint32_t y = S.few[i];
          above += y > k ? 1 : 0;
          same += y == k ? 1 : 0;
        }
        if (above < need && need <= above + same) {  // the key looked for: all that have it write the same
          S.chosen = (int)k;
          S.left = need - above;
        }
      }
      __syncthreads();
      least = (uint32_t)S.chosen;
      known = ~0u;
      need = S.left;
      break;
    }
    __syncthreads();
  }

  // The kept list. A warp takes neighbouring slots, counts what it keeps, and lists it behind
  // what the warps in front of it keep.
  const int ties = any ? need : 0;
  const int span = ((u.len + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int begin = min(warp * span, u.len), end = min(begin + span, u.len);
  auto look = [&](int s, bool& gt, bool& eq) {
    gt = eq = false;
    if (s >= end) return;
    if (s < from || s >= to) {
      gt = true;
    } else if (any) {
      const uint32_t k = key(s) & known;
      gt = k > least;
      eq = k == least;
    }
  };
  __syncthreads();  // the keys are all there; S.warp_sum is free
  {
    int g = 0, e = 0;
    for (int s0 = begin; s0 < end; s0 += 32) {
      bool gt, eq;
      look(s0 + lane, gt, eq);
      g += __popc(__ballot_sync(kAll, gt));
      e += __popc(__ballot_sync(kAll, eq));
    }
    if (lane == 0) S.warp_sum[warp] = make_int2(g, e);
  }
  __syncthreads();
  int g0 = 0, e0 = 0;  // in front of this warp's slots
  for (int k = 0; k < warp; ++k) {
    g0 += S.warp_sum[k].x;
    e0 += S.warp_sum[k].y;
  }
  const unsigned lower = (1u << lane) - 1;
  const int words = (P.budget + 31) / 32;
  uint32_t* bits = dynamic + P.cached;
  int* in_front = reinterpret_cast<int*>(bits + words);
  {
    int g = g0, e = e0;
    for (int s0 = begin; s0 < end; s0 += 32) {
      const int s = s0 + lane;
      bool gt, eq;
      look(s, gt, eq);
      const unsigned bg = __ballot_sync(kAll, gt), be = __ballot_sync(kAll, eq);
      const int rank = e + __popc(be & lower);
      const bool keep = gt || (eq && rank < ties);
      const int at = g + __popc(bg & lower) + min(rank, ties);  // kept slots in front of s
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
      g += __popc(bg);
      e += __popc(be);
    }
    if (P.order_free) {
      __syncthreads();
      // the t-th dropped slot below the budget takes the t-th kept one from there on
      const int below = in_front[words - 1] + __popc(bits[words - 1]);
      g = g0;
      e = e0;
      for (int s0 = begin; s0 < end; s0 += 32) {
        const int s = s0 + lane;
        bool gt, eq;
        look(s, gt, eq);
        const unsigned bg = __ballot_sync(kAll, gt), be = __ballot_sync(kAll, eq);
        const int rank = e + __popc(be & lower);
        const int t = g + __popc(bg & lower) + min(rank, ties) - below;
        if (s >= P.budget && (gt || (eq && rank < ties))) {
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
        g += __popc(bg);
        e += __popc(be);
      }
    }
  }
  __syncthreads();

  // The rows.
  uint4* pool = tid & 16 ? P.V[u.layer] : P.K[u.layer];
  const int part = tid & 15;
  int count = 0;  // rows in the list
  for (int i0 = 0; i0 < P.budget; i0 += kEvictThreads) {
    const int i = i0 + tid;
    const int source = i < P.budget ? kept[i] : i;
    int64_t a = -1, b = -1;
    if (source != i && source >= 0 && source < u.len) {
      a = pool_row(P.pg, P.kv_heads, u.b, u.h, source);
      b = pool_row(P.pg, P.kv_heads, u.b, u.h, i);
      if (a < 0 || b < 0) latch(P.status, BKV_ERR_INVALID_ARG);
      if (b < 0 || !BKV_IN_RANGE(max(a, b) < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) a = -1;
    }
    const unsigned moving = __ballot_sync(kAll, a >= 0);
    if (lane == 0) S.warp_sum[warp].x = __popc(moving);
    __syncthreads();
    int at = count + __popc(moving & lower);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const int n = S.warp_sum[k].x;
      if (k < warp) at += n;
      count += n;
    }
    if (a >= 0) {
      S.list.src[at] = a;
      S.list.dst[at] = b;
    }
    __syncthreads();
    if (count <= kEvictThreads && i0 + kEvictThreads < P.budget) continue;
    // The next step's rows are loaded before this step's are written: their sources lie
    // behind all that this step writes.
    uint4 x[kMoveLoads], y[kMoveLoads];
    float wx = 0.f, wy = 0.f;
    auto load = [&](int c, uint4 (&v)[kMoveLoads], float& w) {
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kWarps + warp;
        if (r < count) v[k] = pool[S.list.src[r] * 16 + part];
      }
      if (tid < kMoveRows && c + tid < count) w = W[S.list.src[c + tid]];
    };
    load(0, x, wx);
    for (int c = 0; c < count; c += kMoveRows) {
      load(c + kMoveRows, y, wy);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kWarps + warp;
        if (r < count) pool[S.list.dst[r] * 16 + part] = x[k];
        x[k] = y[k];
      }
      if (tid < kMoveRows && c + tid < count) W[S.list.dst[c + tid]] = wx;
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
  cudaError_t e = cudaFuncSetAttribute(evict_weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p.layers * p.batch * p.kv_heads));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = (size_t)p.cached * 4 + (p.order_free ? (size_t)((p.budget + 31) / 32) * 8 : 0);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_weight_kernel, p);
}

}  // namespace bkv
