// Rotates packed queries and keys and writes keys and values to their cache
// slots.
//
//   (x_i, x_{i+64}) -> (x_i cos a - x_{i+64} sin a, x_{i+64} cos a + x_i sin a),
//   a = pos * theta^(-2i/d), i < 64 (rotate-half pairs)
//
// Angles of far positions: the frequency is held as a 64-bit fraction of a
// turn, so pos * frequency mod 2^64 is the angle's fraction of a turn with an
// error below pos * 2^-54 turns, in two integer multiplies and at no fp64 rate.
// Its top 32 bits go to sincospif as an fp32 in [-1, 1) (error 2^-25 turns).
// Rotations are fp32, rounded once to bf16.
//
// Bound: HBM. Every row is read and written once; a block's cosines and sines
// sit in shared memory, shared by all heads of a token. A thread's first loads
// start before its token's sequence is looked up (192 decode tokens: 6.2 -> 4.5 us
// on the device, 3.8 a call in a captured graph since calls start dependently).
#include "attend/attend.cuh"

namespace bkv {
namespace {

constexpr int kThreadsStore = 256;
constexpr int kRowThreads = 8;                           // threads per 256-byte row
constexpr int kRows = kThreadsStore / kRowThreads;       // rows per pass of a block

__device__ __forceinline__ void rotate8(const uint4& lo, const uint4& hi, const float2* cs, uint4& olo, uint4& ohi) {
  const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&lo);
  const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&hi);
  __nv_bfloat162* oa = reinterpret_cast<__nv_bfloat162*>(&olo);
  __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(&ohi);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = __bfloat1622float2(a2[e]), b = __bfloat1622float2(b2[e]);
    const float2 c0 = cs[2 * e], c1 = cs[2 * e + 1];
    oa[e] = __floats2bfloat162_rn(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y);
    ob[e] = __floats2bfloat162_rn(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y);
  }
}

// kTokens tokens per block, one warp each to find its sequence; a thread loads
// kAhead rows at a time.
template <int kTokens, int kAhead>
__global__ void __launch_bounds__(kThreadsStore, kTokens > 1 ? 8 : 1) store_kernel(const __grid_constant__ StoreParams P) {
  __shared__ __align__(16) float2 cs[kTokens][kRopePairs];
  __shared__ int64_t row_of[kTokens];  // cache row (sequence * kv_heads * max_cache + slot) or -1
  __shared__ int live[kTokens];        // the token belongs to a sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kTokens;
  const int rows = P.heads + 2 * P.kv_heads;
  const int part = tid % kRowThreads;  // elements [8 part, 8 part + 8) and their partners 64 on
  uint4 lo[kAhead], hi[kAhead];
  depend_wait();
  depend_go();
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kRows, k = r / rows, h = r - k * rows;
      const int t = t0 + k;
      if (r >= kTokens * rows || t >= P.total) continue;
      const uint4* src = h < P.heads               ? P.q + (int64_t)t * P.q_stride + h * 16
                         : h < P.heads + P.kv_heads ? P.k + (int64_t)t * P.k_stride + (h - P.heads) * 16
                                                    : P.v + (int64_t)t * P.v_stride + (h - P.heads - P.kv_heads) * 16;
      lo[i] = src[part];
      hi[i] = src[part + 8];
    }
  };
  load(tid / kRowThreads);  // the first rows need no answer from below
  if (blockIdx.x == 0 && warp == kThreadsStore / 32 - 1) {
    // offsets out of range or order, also those of sequences that no token leads to
    bool bad = false;
    for (int k = lane; k < P.batch; k += 32) bad |= P.cu[k] < 0 || P.cu[k + 1] < P.cu[k] || P.cu[k + 1] > P.total;
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) latch(P.status, BKV_ERR_INVALID_ARG);
  }
  if (warp < kTokens) {
    // a token's sequence: the number of sequences that end at or before it
    const int t = t0 + warp;
    int c = 0;
    for (int k = 1 + lane; k <= P.batch; k += 32) c += P.cu[k] <= t ? 1 : 0;
    const int b = min((int)__reduce_add_sync(0xFFFFFFFFu, c), P.batch);
    const int at = min(b, P.batch - 1);
    const int begin = P.cu[at], first = P.first[at], base = P.pos[at];
    const int i = t - begin;
    // in front of the first sequence or behind the last one: not a token of any
    const bool known = t < P.total && b < P.batch && begin >= 0 && i >= 0;
    const int64_t slot = (int64_t)first + i;
    const bool fits = slot >= 0 && slot < P.max_cache;
    const int64_t where = known ? (int64_t)base + (P.depth ? P.depth[t] : i) : 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t turn = (uint64_t)where * P.turns[lane + 32 * k];
      const float half = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // half turns, [-1, 1]
      float sn, co;
      sincospif(half, &sn, &co);
      cs[warp][lane + 32 * k] = make_float2(co, sn);
    }
    if (lane == 0) {
      row_of[warp] = known && fits ? (int64_t)b * P.kv_heads * P.max_cache + slot : -1;
      live[warp] = known;
      if (known && !fits) latch(P.status, BKV_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  for (int r0 = tid / kRowThreads; r0 < kTokens * rows; r0 += kAhead * kRows) {
    if (r0 >= kAhead * kRows) load(r0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kRows, k = r / rows, h = r - k * rows;
      if (r >= kTokens * rows || !live[k]) continue;
      uint4* dst;
      if (h < P.heads) {
        dst = P.q_rot + ((int64_t)(t0 + k) * P.heads + h) * 16;
      } else {
        const bool key = h < P.heads + P.kv_heads;
        const int64_t row = row_of[k] + (int64_t)(h - P.heads - (key ? 0 : P.kv_heads)) * P.max_cache;
        if (row_of[k] < 0 || !BKV_IN_RANGE(row < (int64_t)P.batch * P.kv_heads * P.max_cache, P.status)) continue;
        dst = (key ? P.K : P.V) + row * 16;
      }
      uint4 a = lo[i], b = hi[i];
      if (h < P.heads + P.kv_heads) rotate8(lo[i], hi[i], &cs[k][part * 8], a, b);
      dst[part] = a;
      dst[part + 8] = b;
    }
  }
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, cudaStream_t s) {
  // a decode step's tokens one to a block with both passes' loads under way at once;
  // long prompts two to a block, eight blocks to an SM (27,380 tokens of 48 rows:
  // 103 us, 6.5 TB/s; at 105.7 one pass ahead in four-token blocks took 107.8, two
  // passes 113)
  const int per_block = p.total <= 8 * kSms ? 1 : 2;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.total + per_block - 1) / per_block));
  cfg.blockDim = dim3(kThreadsStore);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return per_block == 1 ? cudaLaunchKernelEx(&cfg, store_kernel<1, 2>, p) : cudaLaunchKernelEx(&cfg, store_kernel<2, 1>, p);
}

}  // namespace bkv
