// Rotates packed queries and keys, in any of the rotary layouts, and writes keys
// and values to their pages.
//
//   (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin) * scale, angle = pos * f_i,
//   (a, b) = (i, i + r/2) (half) or (2i, 2i + 1) (interleaved), i < r/2; elements from
//   r on stay.
//
// The angle is a 64-bit fraction of a turn, pos * f_i / (2 pi) mod 1 by one integer
// multiply: its error is below pos * 2^-54 turns at any position, and no fp64 unit is
// involved. Rotations are fp32, rounded once to bf16.
//
// A thread takes two 16-byte pieces of a row, the ones its eight pairs lie in: pieces
// p and p + r/16 of a half layout, 2p and 2p + 1 of an interleaved one; in both its
// pairs are 8p .. 8p + 7. Bound: HBM, every row read and written once (27,380 tokens of 56
// rows, interleaved, half of the head: 117 us, 6.7 TB/s, 0.99 of a copy; 192 decode tokens 6.7 us,
// the chain of offsets, slot, page and row).
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr int kThreadsStore = 256;
constexpr int kRowThreads = 8;                      // threads per 256-byte row
constexpr int kRows = kThreadsStore / kRowThreads;  // rows per pass of a block

__device__ __forceinline__ float2 turn(float2 x, float2 cs) {
  return make_float2(x.x * cs.x - x.y * cs.y, x.y * cs.x + x.x * cs.y);
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate_pieces(uint4& a, uint4& b, const float2* cs) {
  __nv_bfloat162* a2 = reinterpret_cast<__nv_bfloat162*>(&a);
  __nv_bfloat162* b2 = reinterpret_cast<__nv_bfloat162*>(&b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = __bfloat1622float2(a2[e]), y = __bfloat1622float2(b2[e]);
    if constexpr (kInterleaved) {
      const float2 u = turn(x, cs[e]), v = turn(y, cs[4 + e]);
      a2[e] = __floats2bfloat162_rn(u.x, u.y);
      b2[e] = __floats2bfloat162_rn(v.x, v.y);
    } else {
      const float2 u = turn(make_float2(x.x, y.x), cs[2 * e]), v = turn(make_float2(x.y, y.y), cs[2 * e + 1]);
      a2[e] = __floats2bfloat162_rn(u.x, v.x);
      b2[e] = __floats2bfloat162_rn(u.y, v.y);
    }
  }
}

// kTokens tokens per block, one warp each to find its sequence; a thread loads
// kAhead rows at a time.
template <bool kInterleaved, int kTokens, int kAhead>
__global__ void __launch_bounds__(kThreadsStore, kTokens > 1 ? 8 : 1)
    store_paged_kernel(const __grid_constant__ StorePagedParams P) {
  __shared__ __align__(16) float2 cs[kTokens][kRopePairs];
  __shared__ int64_t row_of[kTokens];  // pool row of KV head 0, or -1
  __shared__ int live[kTokens];        // the token belongs to a sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kTokens;
  const int rows = P.heads + 2 * P.kv_heads;
  const int part = tid % kRowThreads;
  // this thread's pieces of a row
  const int half = P.rotary / 16;  // threads that rotate
  const bool rotates = part < half;
  int pa = 2 * part, pb = 2 * part + 1;
  if (!kInterleaved && rotates) {
    pa = part;
    pb = part + half;
  }
  uint4 a[kAhead], b[kAhead];
  depend_wait();
  depend_go();
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kRows, k = r / rows, h = r - k * rows;
      const int t = t0 + k;
      if (r >= kTokens * rows || t >= P.total) continue;
      const uint4* src = h < P.heads                ? P.q + (int64_t)t * P.q_stride + h * 16
                         : h < P.heads + P.kv_heads ? P.k + (int64_t)t * P.k_stride + (h - P.heads) * 16
                                                    : P.v + (int64_t)t * P.v_stride + (h - P.heads - P.kv_heads) * 16;
      a[i] = src[pa];
      b[i] = src[pb];
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
    const int seq = min((int)__reduce_add_sync(0xFFFFFFFFu, c), P.batch);
    const int at = min(seq, P.batch - 1);
    const int begin = P.cu[at], first = P.first[at], base = P.pos[at];
    const int i = t - begin;
    // in front of the first sequence or behind the last one: not a token of any
    const bool known = t < P.total && seq < P.batch && begin >= 0 && i >= 0;
    const int64_t slot = (int64_t)first + i;
    const bool fits = slot >= 0 && slot < P.pg.cap;
    const int64_t where = known ? (int64_t)base + (P.depth ? P.depth[t] : i) : 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t turns = (uint64_t)where * P.turns[lane + 32 * k];
      const float halves = (float)(int32_t)(turns >> 32) * 0x1p-31f;  // half turns, [-1, 1]
      float sn, co;
      sincospif(halves, &sn, &co);
      cs[warp][lane + 32 * k] = make_float2(co * P.scale, sn * P.scale);
    }
    if (lane == 0) {
      const int64_t row = known && fits ? pool_row(P.pg, P.kv_heads, at, 0, (int)slot) : -1;
      row_of[warp] = row;
      live[warp] = known;
      if (known && row < 0) latch(P.status, BKV_ERR_INVALID_ARG);
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
        const int64_t row = row_of[k] + (int64_t)(h - P.heads - (key ? 0 : P.kv_heads)) * P.pg.page_size;
        if (row_of[k] < 0 || !BKV_IN_RANGE(row < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) continue;
        dst = (key ? P.K : P.V) + row * 16;
      }
      if (rotates && h < P.heads + P.kv_heads) rotate_pieces<kInterleaved>(a[i], b[i], &cs[k][part * 8]);
      dst[pa] = a[i];
      dst[pb] = b[i];
    }
  }
}

template <bool kInterleaved>
cudaError_t launch(const StorePagedParams& p, cudaStream_t s) {
  // a decode step's tokens one to a block with both passes' loads under way at once;
  // long prompts two to a block, eight blocks to an SM
  const int per_block = p.total <= 8 * kSms ? 1 : 2;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.total / per_block + (p.total % per_block ? 1 : 0)));
  cfg.blockDim = dim3(kThreadsStore);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return per_block == 1 ? cudaLaunchKernelEx(&cfg, store_paged_kernel<kInterleaved, 1, 2>, p)
                        : cudaLaunchKernelEx(&cfg, store_paged_kernel<kInterleaved, 2, 1>, p);
}

}  // namespace

cudaError_t launch_store_paged(const StorePagedParams& p, cudaStream_t s) {
  return p.interleaved ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace bkv
