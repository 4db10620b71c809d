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
// sit in shared memory, shared by all heads of a token.
#include "attend/attend.cuh"

namespace bkv {
namespace {

constexpr int kThreadsStore = 256;
constexpr int kTokens = 4;  // tokens per block

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

__global__ void __launch_bounds__(kThreadsStore) store_kernel(const __grid_constant__ StoreParams P) {
  __shared__ __align__(16) float2 cs[kTokens][kRopePairs];
  __shared__ int64_t row_of[kTokens];  // cache row (sequence * kv_heads * max_cache + slot) or -1
  __shared__ int live[kTokens];        // the token belongs to a sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kTokens;
  if (warp < kTokens) {
    // one warp per token finds its sequence: the offsets at or below it
    const int t = t0 + warp;
    int b = -1, i = 0;
    int64_t row = -1;
    bool bad = false;
    if (t < P.total) {
      int c = 0;
      for (int k = 1 + lane; k <= P.batch; k += 32) c += P.cu[k] <= t ? 1 : 0;
      b = __reduce_add_sync(0xFFFFFFFFu, c);
      if (b < P.batch) {
        const int begin = P.cu[b];
        i = t - begin;
        if (i < 0) {
          bad = b > 0;  // before the first sequence: not a token of any
          b = -1;
        } else if (begin < 0) {
          bad = true;
          b = -1;
        } else {
          const int64_t slot = (int64_t)P.first[b] + i;
          if (slot >= 0 && slot < P.max_cache) row = (int64_t)b * P.kv_heads * P.max_cache + slot;
          else bad = true;
        }
      } else {
        b = -1;
      }
    }
    int64_t where = 0;
    if (b >= 0) where = (int64_t)P.pos[b] + (P.depth ? P.depth[t] : i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t turn = (uint64_t)where * P.turns[lane + 32 * k];
      const float half = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // half turns, [-1, 1]
      float sn, co;
      sincospif(half, &sn, &co);
      cs[warp][lane + 32 * k] = make_float2(co, sn);
    }
    if (lane == 0) {
      row_of[warp] = row;
      live[warp] = b >= 0;
      if (bad) latch(P.status, BKV_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  // 8 threads per row: thread `part` has elements [8 part, 8 part + 8) and their partners 64 on
  const int rows = P.heads + 2 * P.kv_heads;
  const int part = tid & 7;
  for (int r = tid >> 3; r < kTokens * rows; r += kThreadsStore / 8) {
    const int k = r / rows, h = r - k * rows;
    const int t = t0 + k;
    if (!live[k]) continue;
    const uint4* src;
    uint4* dst;
    bool turn = true;
    if (h < P.heads) {
      src = P.q + (int64_t)t * P.q_stride + h * 16;
      dst = P.q_rot + ((int64_t)t * P.heads + h) * 16;
    } else {
      if (row_of[k] < 0) continue;
      const bool key = h < P.heads + P.kv_heads;
      const int kh = h - P.heads - (key ? 0 : P.kv_heads);
      src = (key ? P.k + (int64_t)t * P.k_stride : P.v + (int64_t)t * P.v_stride) + kh * 16;
      dst = (key ? P.K : P.V) + (row_of[k] + (int64_t)kh * P.max_cache) * 16;
      turn = key;
      if (!BKV_IN_RANGE(row_of[k] + (int64_t)kh * P.max_cache < (int64_t)P.batch * P.kv_heads * P.max_cache, P.status))
        continue;
    }
    uint4 lo = src[part], hi = src[part + 8];
    if (turn) {
      uint4 a, b;
      rotate8(lo, hi, &cs[k][part * 8], a, b);
      lo = a;
      hi = b;
    }
    dst[part] = lo;
    dst[part + 8] = hi;
  }
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, cudaStream_t s) {
  store_kernel<<<(unsigned)((p.total + kTokens - 1) / kTokens), kThreadsStore, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace bkv
