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
// block's selection, which is latency, lies under the copies of others: 6,144 units of up to
// 2,048 slots cut to 1,792 take 1,679 us for 11.4 GB, a copy's rate (as two launches
// 1,640 + 164). Order-free, 16 rows of 4,096 units, 48 us: the selection's instructions (62 with
// a look-up of the row for every key, the first histogram in a pass of its own, and prefix and
// recent slots told by their numbers and not by their keys).
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kBins = 2048;                                 // eleven bits of a key
constexpr int kMostCached = 8192;                           // slots whose keys stay in shared memory
constexpr uint32_t kAlways = ~0u;                           // in place of a key: the slot is kept in any case. No weight
                                                            // has this key, nor one that shares its top eleven bits
constexpr int kMoveLoads = 4;                               // 16-byte pieces per thread and step

struct Unit {
  int layer, b, h;
  int len;       // clamped
  bool bad;      // length out of range, or too short for an order-free eviction
  bool evicts;
};
__device__ __forceinline__ Unit unit_of(const EvictWeightParams& P) {
  Unit u;
  const unsigned i = blockIdx.x / (unsigned)P.kv_heads;  // fewer than 2^31 units
  u.h = (int)(blockIdx.x - i * P.kv_heads);
  u.layer = (int)(i / (unsigned)P.batch);
  u.b = (int)(i - u.layer * P.batch);
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

template <int kThreads>
struct Shared {
  union {
    int hist[kBins];         // in descending order of the digits
    uint32_t few[kThreads];  // keys of a bin that are ranked directly
    struct {
      int64_t src[kThreads * 2], dst[kThreads * 2];  // rows that move
    } list;
  };
  int chosen, left, found;
  int2 warp_sum[kThreads / 32];
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) evict_weight_kernel(const __grid_constant__ EvictWeightParams P) {
  constexpr int kWarps = kThreads / 32, kPerThread = kBins / kThreads, kFew = kThreads;
  static_assert(kBins % (4 * kThreads) == 0, "a thread clears and reads its bins four at a time");
  constexpr int kMoveRows = kMoveLoads * kThreads / 32;  // rows of K and of V per step
  // the first P.cached slots' keys; order-free: kept slots below the budget as bits, and the
  // kept in front of every word
  extern __shared__ uint32_t dynamic[];
  __shared__ __align__(16) Shared<kThreads> S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < kPerThread / 4; ++i) reinterpret_cast<int4*>(S.hist)[tid + i * kThreads] = make_int4(0, 0, 0, 0);
  };
  clear();
  if (tid == 0) S.found = 0;
  __syncthreads();
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
    for (int i = tid; i < P.budget; i += kThreads) kept[i] = i < u.len && u.len <= P.budget ? i : -1;
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
  int need = P.budget - P.prefix - P.recent;  // of the candidates, fewer than there are
  const bool any = need > 0;

  // The keys of the first slots, four a thread (in one page), and the histogram of the first bits.
  uint32_t* cache = dynamic;
  const int cached = min(u.len, P.cached);
  const bool quads = P.pg.page_size % 4 == 0 && (reinterpret_cast<uintptr_t>(W) & 15) == 0;
  auto count_key = [&](uint32_t k, int shift, uint32_t digit) { atomicAdd(&S.hist[kBins - 1 - (k >> shift & digit)], 1); };
#pragma unroll 2
  for (int s = 4 * tid; s < cached; s += 4 * kThreads) {
    const int64_t row = pool_row(P.pg, P.kv_heads, u.b, u.h, s);
    float4 w = make_float4(__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""));
    if (row < 0) {
      latch(P.status, BKV_ERR_INVALID_ARG);
    } else if (BKV_IN_RANGE(row + min(3, u.len - 1 - s) < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) {
      if (quads) {
        w = *reinterpret_cast<const float4*>(W + row);
      } else {
        w.x = W[row];
        if (s + 1 < u.len) w.y = W[row + 1];
        if (s + 2 < u.len) w.z = W[row + 2];
        if (s + 3 < u.len) w.w = W[row + 3];
      }
    }
    uint32_t k[4] = {key_of(w.x), key_of(w.y), key_of(w.z), key_of(w.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (s + e < from || s + e >= to) k[e] = kAlways;
      else if (any) count_key(k[e], 21, 2047u);
    }
    *reinterpret_cast<uint4*>(cache + s) = make_uint4(k[0], k[1], k[2], k[3]);
  }
  auto key = [&](int slot) { return slot < cached ? cache[slot] : slot < from || slot >= to ? kAlways : read_key(slot); };
  const int behind = max(cached, from);  // candidates from here on have no key on chip
  if (any)
    for (int s = behind + tid; s < to; s += kThreads) count_key(read_key(s), 21, 2047u);

  // The smallest kept key, as far as its bits are known, and how many of those equal in these
  // bits are kept (the lowest slots): `need`. Without a candidate to keep, a key above all weights'.
  uint32_t least = any ? 0u : kAlways - 1, known = any ? 0u : ~0u;
  __syncthreads();
  for (int shift = 21; any && shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
    const uint32_t digit = shift == 0 ? 1023u : 2047u;
    if (shift < 21) {
      clear();
      __syncthreads();
      auto count = [&](uint32_t k) {
        if ((k & known) == least) count_key(k, shift, digit);
      };
      for (int s = tid; s < cached; s += kThreads) count(cache[s]);
      for (int s = behind + tid; s < to; s += kThreads) count(read_key(s));
      __syncthreads();
    }
    // the bin, from the top, in which the need-th largest lies: neighbouring bins a thread
    int mine[kPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread / 4; ++i)
      *reinterpret_cast<int4*>(&mine[4 * i]) = reinterpret_cast<const int4*>(S.hist)[tid * (kPerThread / 4) + i];
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
      auto list = [&](uint32_t k) {
        if ((k & known) == least) {
          const int at = atomicAdd(&S.found, 1);
          if (at < kFew) S.few[at] = k;
        }
      };
      for (int s = tid; s < cached; s += kThreads) list(cache[s]);
      for (int s = behind + tid; s < to; s += kThreads) list(read_key(s));
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

  // The kept list. A warp takes neighbouring slots: words of 32, as many as lanes at a time,
  // lane i keeping what is known of word i. It counts what it keeps, and lists it behind what
  // the warps in front of it keep.
  const int ties = any ? need : 0;
  const int span = ((u.len + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int begin = min(warp * span, u.len), end = min(begin + span, u.len);
  uint32_t greater = 0, equal = 0;  // word `lane` of the 32 looked at: slots kept in any case, slots equal to the least
  auto look = [&](int s0) {
    greater = equal = 0;
    const int n = min((end - s0 + 31) / 32, 32);
    auto word = [&](int i, uint32_t k) {
      const unsigned bg = __ballot_sync(kAll, (k & known) > least), be = __ballot_sync(kAll, (k & known) == least);
      if (lane == i) {
        greater = bg;
        equal = be;
      }
    };
    if (end <= cached) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) word(i, cache[s0 + i * 32 + lane]);
    } else {
      for (int i = 0; i < n; ++i) word(i, key(s0 + i * 32 + lane));
    }
    // slots behind the last one
    const int in = end - s0 - lane * 32;
    if (in < 32) {
      const uint32_t mask = in > 0 ? (1u << in) - 1 : 0u;
      greater &= mask;
      equal &= mask;
    }
  };
  __syncthreads();  // the keys are all there; S.warp_sum is free
  {
    int g = 0, e = 0;
    for (int s0 = begin; s0 < end; s0 += 1024) {
      look(s0);
      g += __popc(greater);
      e += __popc(equal);
    }
    g = __reduce_add_sync(kAll, g);
    e = __reduce_add_sync(kAll, e);
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
  uint32_t* bits = dynamic + (P.cached + 31) / 32 * 32;
  int* in_front = reinterpret_cast<int*>(bits + words);
  uint32_t keep = 0;  // of word `lane`: its kept slots, and those in front of it
  int at = 0;
  auto keep_words = [&](int s0) {
    if (span > 1024) look(s0);  // otherwise it was the only look
    int g = __popc(greater), e = __popc(equal);
    const int own_g = g, own_e = e;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(kAll, g, off), y = __shfl_up_sync(kAll, e, off);
      if (lane >= off) {
        g += x;
        e += y;
      }
    }
    const int g_all = __shfl_sync(kAll, g, 31), e_all = __shfl_sync(kAll, e, 31);
    g += g0 - own_g;
    e += e0 - own_e;
    at = g + min(e, ties);
    uint32_t low = equal;  // the lowest of the equal ones, up to `ties` in all
    for (int drop = own_e - max(ties - e, 0); drop > 0 && low; --drop) low &= ~(0x80000000u >> __clz(low));
    keep = greater | low;
    g0 += g_all;
    e0 += e_all;
  };
  const int g_begin = g0, e_begin = e0;
  for (int s0 = begin; s0 < end; s0 += 1024) {
    keep_words(s0);
    if (P.order_free) {
      const int w0 = s0 + lane * 32;
      if (w0 < min(end, P.budget)) {
        bits[w0 >> 5] = P.budget - w0 < 32 ? keep & ((1u << (P.budget - w0)) - 1) : keep;
        in_front[w0 >> 5] = at;
      }
    }
    for (int i = 0; i < 32 && s0 + i * 32 < end; ++i) {
      const uint32_t k = __shfl_sync(kAll, keep, i);
      const int to_slot = P.order_free ? s0 + i * 32 + lane : __shfl_sync(kAll, at, i) + __popc(k & lower);
      if ((k >> lane & 1) && (unsigned)to_slot < (unsigned)P.budget) kept[to_slot] = s0 + i * 32 + lane;
    }
  }
  __syncthreads();

  int count = 0;  // rows in the list
  auto rows_of = [&](int source, int i, int64_t& a, int64_t& b) {
    a = pool_row(P.pg, P.kv_heads, u.b, u.h, source);
    b = pool_row(P.pg, P.kv_heads, u.b, u.h, i);
    if (a < 0 || b < 0) latch(P.status, BKV_ERR_INVALID_ARG);
    if (b < 0 || !BKV_IN_RANGE(max(a, b) < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) a = -1;
  };
  bool listed = false;
  if (P.order_free) {
    // the t-th dropped slot below the budget takes the t-th kept one from there on
    const int below = in_front[words - 1] + __popc(bits[words - 1]);
    const int moved = P.budget - below;
    listed = moved <= 2 * kThreads;
    if (listed) {
      for (int t = tid; t < moved; t += kThreads) S.list.src[t] = -1;
      __syncthreads();
    }
    if (end > P.budget) {
      g0 = g_begin;
      e0 = e_begin;
      for (int s0 = begin; s0 < end; s0 += 1024) {
        keep_words(s0);
        for (int i = max(P.budget - s0, 0) / 32; i < 32 && s0 + i * 32 < end; ++i) {
          const uint32_t k = __shfl_sync(kAll, keep, i);
          const int t = __shfl_sync(kAll, at, i) + __popc(k & lower) - below, source = s0 + i * 32 + lane;
          if (source < P.budget || !(k >> lane & 1)) continue;
          int lo = 0, hi = words - 1;  // the last word with at most t dropped slots in front
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (mid * 32 - in_front[mid] <= t) lo = mid;
            else hi = mid - 1;
          }
          uint32_t holes = ~bits[lo];
          for (int skip = t - (lo * 32 - in_front[lo]); skip > 0 && holes; --skip) holes &= holes - 1;
          const int hole = lo * 32 + __ffs(holes) - 1;
          if (holes == 0 || hole >= P.budget) continue;
          kept[hole] = source;
          if (listed && t >= 0 && t < 2 * kThreads) {
            int64_t a, b;
            rows_of(source, hole, a, b);
            S.list.src[t] = a;
            S.list.dst[t] = b;
          }
        }
      }
    }
    if (listed) count = moved;
    __syncthreads();
  }

  // The rows.
  uint4* pool = tid & 16 ? P.V[u.layer] : P.K[u.layer];
  const int part = tid & 15;
  for (int i0 = listed ? P.budget - 1 : 0; i0 < P.budget; i0 += kThreads) {
    if (!listed) {
      const int i = i0 + tid;
      const int source = i < P.budget ? kept[i] : i;
      int64_t a = -1, b = -1;
      if (source != i && source >= 0 && source < u.len) rows_of(source, i, a, b);
      const unsigned moving = __ballot_sync(kAll, a >= 0);
      if (lane == 0) S.warp_sum[warp].x = __popc(moving);
      __syncthreads();
      int place = count + __popc(moving & lower);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const int n = S.warp_sum[k].x;
        if (k < warp) place += n;
        count += n;
      }
      if (a >= 0) {
        S.list.src[place] = a;
        S.list.dst[place] = b;
      }
      __syncthreads();
      if (count <= kThreads && i0 + kThreads < P.budget) continue;
    }
    // The next step's rows are loaded before this step's are written: their sources lie
    // behind all that this step writes.
    uint4 x[kMoveLoads], y[kMoveLoads];
    float wx = 0.f, wy = 0.f;
    auto load = [&](int c, uint4 (&v)[kMoveLoads], float& w) {
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kWarps + warp;
        if (r < count && S.list.src[r] >= 0) v[k] = pool[S.list.src[r] * 16 + part];
      }
      if (tid < kMoveRows && c + tid < count && S.list.src[c + tid] >= 0) w = W[S.list.src[c + tid]];
    };
    load(0, x, wx);
    for (int c = 0; c < count; c += kMoveRows) {
      load(c + kMoveRows, y, wy);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kMoveLoads; ++k) {
        const int r = c + k * kWarps + warp;
        if (r < count && S.list.src[r] >= 0) pool[S.list.dst[r] * 16 + part] = x[k];
        x[k] = y[k];
      }
      if (tid < kMoveRows && c + tid < count && S.list.src[c + tid] >= 0) W[S.list.dst[c + tid]] = wx;
      wx = wy;
    }
    count = 0;
    __syncthreads();
  }
}

template <int kThreads>
cudaError_t launch(const EvictWeightParams& p, cudaStream_t s) {
  const auto fn = evict_weight_kernel<kThreads>;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_shared(fn, 200 * 1024, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p.layers * p.batch * p.kv_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)((p.cached + 31) / 32 * 32) * 4 + (p.order_free ? (size_t)((p.budget + 31) / 32) * 8 : 0);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t launch_evict_weight(const EvictWeightParams& given, cudaStream_t s) {
  EvictWeightParams p = given;
  p.cached = p.pg.cap < kMostCached ? p.pg.cap : kMostCached;
  // Few units: 512 threads each (288 units of 2,064 slots: 27 us, with 256 threads 31, with 128
  // 44). Many: 256 (6,144 units of 2,048 slots: 1,680 us, with 512 1,673, with 128 1,719), or
  // order-free, where a unit is a chain of latencies and little else, 128 and so twice the
  // units at once (4,096 units of 1,040 slots: 48 us, with 256 70, with 512 109).
  const int64_t units = (int64_t)p.layers * p.batch * p.kv_heads;
  return units <= 2 * kSms ? launch<512>(p, s) : p.order_free ? launch<128>(p, s) : launch<256>(p, s);
}

}  // namespace bkv
