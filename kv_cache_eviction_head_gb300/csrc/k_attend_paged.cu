// Attention of one new token per sequence over paged caches, and the weight every
// slot received from it.
//
//   o_h = sum_j p_hj V[j],  p_hj = exp(l_hj - lse_h),  l_hj = q_h . k_j / sqrt(d),
//   lse_h = ln sum_j exp(l_hj),  j < lens[b];  weights[j] = decay weights[j] + sum_h p_hj
//   over the query heads of slot j's KV head (the new token's own slot: sum_h p_hj).
//
// Bound: HBM, 512 bytes per visible slot and KV head for 4 d G operations. With at most
// 16 rows to multiply there is nothing for a 128-row tensor instruction to gain, and
// what counts is that every SM has loads under way all the time. So the work is cut to
// the warp: the visible tiles of 16 slots of all (sequence, KV head, chunk of query
// heads) units stand in a row, each warp of the launch takes an equal share of that row
// and runs on its own, without a barrier. A unit that lies in several shares leaves
// pieces (reference maximum, sum, unnormalised o) in the workspace, which a second
// launch joins in the order of the shares. The split goes by the lengths alone: the same
// call gives the same bits.
//
// A warp's ring of tiles is its own: one lane asks TMA for the four boxes of a tile
// (64 elements x 16 slots of K and of V, twice; SWIZZLE_128B, so that the fragments' loads
// meet no bank twice), the warp waits for their barrier. S = Q K^T (m16n8k16, rows: query
// heads, columns: slots); P as it leaves S is the B operand of O^T = V^T P^T (rows: d,
// columns: heads). Copied by the threads themselves (cp.async, 16 bytes each, in fragment
// order) the same tiles came at 4.7 TB/s whatever the number of warps and stages.
//
// Rounding: logits, maxima, sums, weights and O are fp32; P is rounded to bf16 for the
// product with bf16 V (at most 2^-8 relative per term, as the output), the sums and
// the weights take the unrounded values. The reference maximum moves only when a logit
// exceeds it by 8 in log2 (a factor of 256 in P, which costs no precision).
//
// Weights need the final sum: the first launch leaves its logits (fp32, 4 G bytes a
// slot) in the workspace, and the second turns them into probabilities.
//
// Measured on one GB300 (6.78 TB/s copy):
//   192 sequences of 1,857 - 2,063 slots, 32/8 heads, weights   260 us   6.0 TB/s  0.89 (227 + 22 us)
//   3 of 16,500 - 32,767 slots, 40/8 heads                       59 us   5.9 TB/s  0.87
//   64 of 0 - 4,112 slots, 28/4 heads, weights                   54 us   5.0 TB/s  0.73 (45 + 15)
//   one of 2,063 slots, 32/8 heads, weights                      12 us, the call on the host
// The first launch runs at the memory's rate; the second is a chain of look-ups (the
// sequences' places, pieces, old weights and logits) at a latency each.
#include "paged/device.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kBox = kTileSlots * 128;       // 16 slots x 64 elements
constexpr int kTileBox = 4 * kBox;           // K and V of a tile: 8 KB
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 3;                // per SM
constexpr int kAhead = 2;                   // heads whose logits are asked for ahead (ragged lengths: 53.6 us, with four 54.8)
constexpr int kJoinTiles = 16;              // tiles of a block's weights, at least
constexpr int kJoinHeads = 512;             // heads whose sums a block holds at a time
constexpr float kMinusInf = -__builtin_huge_valf();
constexpr float kLag = 8.f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four 8 x 8 tiles of 16-bit elements, plain or transposed; lane i gives the address of
// row i % 8 of tile i / 8.
__device__ __forceinline__ void load_tiles(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void load_tiles_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int len_of(const AttendPagedParams& P, int b) { return min(max(P.lens[b], 0), P.pg.cap); }
__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + kTileSlots - 1) / kTileSlots); }

// Tiles of the whole call per (KV head, chunk), fewer than 2^31 / units: one warp, all lanes
// get it. `bad`: a length was clamped.
__device__ __forceinline__ int all_tiles(const AttendPagedParams& P, int lane, bool& bad) {
  int n = 0;
  bad = false;
#pragma unroll 4
  for (int b = lane; b < P.batch; b += 32) {
    const int given = P.lens[b], len = min(max(given, 0), P.pg.cap);
    bad |= len != given;
    n += tiles_of(len);
  }
  bad = __any_sync(kAll, bad);
  return __reduce_add_sync(kAll, n);
}
// Tiles per share: four at least, or the pieces cost more to join than they save (30,000
// slots of one KV head: 17.1 us, with one 24.6, with six 17.4); more when there are not warps
// enough.
__device__ __forceinline__ int share_of(int tiles, int shares) { return max((tiles + shares - 1) / shares, 4); }
// The sequence that tile t (of `per` tiles for each of a sequence's own) lies in, and the
// sum of the tiles in front of it; b = batch behind the last. One warp.
__device__ __forceinline__ void find_sequence(const AttendPagedParams& P, int t, int per, int lane, int& b, int& before) {
  int base = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 32) {
    const int n = b0 + lane < P.batch ? tiles_of(len_of(P, b0 + lane)) : 0;
    int upto = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, off);
      if (lane >= off) upto += y;
    }
    const unsigned hit = __ballot_sync(kAll, t < (base + upto) * per);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      before = base + __shfl_sync(kAll, upto - n, src);
      return;
    }
    base += __shfl_sync(kAll, upto, 31);
  }
  b = P.batch;
  before = base;
}

// For the second launch: the tiles in front of every sequence and its length. One warp.
__device__ __forceinline__ void list_sequences(const AttendPagedParams& P, int lane) {
  int base = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 32) {
    const int len = b0 + lane < P.batch ? len_of(P, b0 + lane) : 0, n = tiles_of(len);
    int upto = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, off);
      if (lane >= off) upto += y;
    }
    if (b0 + lane < P.batch) P.seq[b0 + lane] = make_int2(base + upto - n, len);
    base += __shfl_sync(kAll, upto, 31);
  }
  if (lane == 0) P.seq[P.batch] = make_int2(base, 0);
}

// A place in the row of tiles.
struct Place {
  int b, u;        // sequence, unit within it (KV head * chunks + chunk)
  int i, n;        // tile of the unit, its tiles
  int len;
  int page;        // pool page of the tile, or -1
  int before;      // tiles (per unit) of the sequences in front
};
__device__ __forceinline__ void look_up(const AttendPagedParams& P, Place& p) {
  p.page = pool_page(P.pg, p.b, page_of(P.pg, p.i * kTileSlots));
}
// The next tile. Sequences without slots have none.
__device__ __forceinline__ void step(const AttendPagedParams& P, Place& p, int units) {
  if (++p.i < p.n) return;
  p.i = 0;
  if (++p.u < units) return;
  p.u = 0;
  p.before += p.n;
  do {
    if (++p.b >= P.batch) return;
    p.len = len_of(P, p.b);
    p.n = tiles_of(p.len);
  } while (p.n == 0);
}

template <int NT, int kAttendWarps, int kStages>
__global__ void __launch_bounds__(kAttendWarps * 32, 2) attend_paged_kernel(const __grid_constant__ AttendPagedParams P) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[kAttendWarps][kStages];
  __shared__ int rows_in[kAttendWarps][kStages];  // visible slots of a tile
  __shared__ Ctl ctl_of[kAttendWarps];            // a warp's waits end for itself alone
  constexpr int kChunk = 8 * NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane & 3, row = lane >> 2;
  const int w = blockIdx.x * kAttendWarps + warp;
  const int units = P.kv_heads * P.chunks;
  uint64_t* bar = full[warp];
  Ctl* ctl = &ctl_of[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bar[s], 1);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  depend_wait();
  depend_go();

  bool bad;
  const int total = all_tiles(P, lane, bad) * units;
  if (w == 0) {
    if (lane == 0 && bad) latch(P.status, BKV_ERR_INVALID_ARG);
    list_sequences(P, lane);
  }
  const int share = share_of(total, P.shares);
  const int64_t begin = (int64_t)w * share;
  if (begin >= total) return;
  const int t0 = (int)begin, count = min(share, total - t0);

  Place c;
  find_sequence(P, t0, units, lane, c.b, c.before);
  c.len = len_of(P, c.b);
  c.n = tiles_of(c.len);
  {
    const int in = t0 - c.before * units;
    c.u = in / c.n;
    c.i = in - c.u * c.n;
  }
  look_up(P, c);
  Place a = c;  // the next tile to copy; its page is looked up one tile ahead

  const uint32_t ring = ((smem_u32(raw) + 1023u) & ~1023u) + warp * kStages * kTileBox;
  const uint64_t policy = policy_evict_first();  // read once, unlike the workspace and the weights (ragged lengths: 67 -> 60 us)
  auto fetch = [&](int stage) {
    const int slot0 = a.i * kTileSlots;
    int rows = min(kTileSlots, a.len - slot0);
    const int z = a.page * P.kv_heads + a.u / P.chunks;
    if (a.page < 0) {
      rows = 0;
      if (lane == 0) latch(P.status, BKV_ERR_INVALID_ARG);
    } else if (!BKV_IN_RANGE(z < P.pg.pages * P.kv_heads, P.status)) {
      rows = 0;
    }
    if (lane == 0) {
      rows_in[warp][stage] = rows;
      if (rows > 0) {
        const int y = slot0 - page_of(P.pg, slot0) * P.pg.page_size;
        const uint32_t dst = ring + stage * kTileBox;
        mbar_expect_tx(&bar[stage], kTileBox);
        tma_rows(dst, &P.kmap, 0, y, z, &bar[stage], policy);
        tma_rows(dst + kBox, &P.kmap, 64, y, z, &bar[stage], policy);
        tma_rows(dst + 2 * kBox, &P.vmap, 0, y, z, &bar[stage], policy);
        tma_rows(dst + 3 * kBox, &P.vmap, 64, y, z, &bar[stage], policy);
      } else {
        mbar_arrive(&bar[stage]);
      }
    }
  };
  int ahead = 0;  // tiles copied or under way
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (ahead < count) {
      fetch(s);
      ++ahead;
      step(P, a, units);
      if (ahead < count) look_up(P, a);
    }
  }

  // a lane's row of the fragments' tiles: (slots 0-7, 16-byte pieces 0 and 1), (slots 8-15,
  // pieces 0 and 1)
  const int tile_row = lane & 7, piece0 = lane >> 3 & 1;
  const uint32_t slot_row = (uint32_t)((lane >> 4) * 8 + tile_row) * 128;

  uint32_t qlo[8][2], qhi[NT == 2 ? 8 : 1][2];
  float o[NT][8][4];
  float m[NT], l[NT];
  int first = 0;  // tile of the unit that this piece begins with
  bool fresh = true;
  int stage = 0;
  uint32_t phase = 0;
  int it = 0;
  for (; it < count; ++it) {
    const int h = c.u / P.chunks, head0 = (c.u - h * P.chunks) * kChunk;  // first query head of the chunk, in its group
    if (fresh) {
      fresh = false;
      first = c.i;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(P.q + (int64_t)c.b * P.q_stride + ((int64_t)h * P.group + head0) * 16) + quad;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        m[t] = kMinusInf;
        l[t] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
        const bool in = head0 + row + 8 * t < P.group;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = in ? q[(row + 8 * t) * 64 + k * 8 + e * 4] : 0u;
            if (t == 0) qlo[k][e] = x;
            else if constexpr (NT == 2) qhi[k][e] = x;
          }
      }
    }
    if (!__all_sync(kAll, mbar_wait(&bar[stage], phase, ctl, P.status))) break;
    const int rows = rows_in[warp][stage];
    const uint32_t at = ring + stage * kTileBox;
    // the stage that the tile before has left
    if (ahead < count) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      ++ahead;
      step(P, a, units);
      if (ahead < count) look_up(P, a);
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
    if (rows < kTileSlots) {  // what lies behind the last slot may be NaN: a weight of 0 does not undo it
      for (int i = lane; i < (kTileSlots - rows) * 16; i += 32)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + (2 + (i >> 3 & 1)) * kBox + (rows + (i >> 4)) * 128 + (i & 7) * 16), "r"(0) : "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
      __syncwarp();
    }

    float s[2][4], s1[2][4];  // two sums per eight slots halve the chain of products
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = s1[t][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t f[4];
      load_tiles(f, at + (k >> 2) * kBox + slot_row + (uint32_t)((((k & 3) * 2 + piece0) ^ tile_row) << 4));
      const uint32_t h0 = NT == 2 ? qhi[NT == 2 ? k : 0][0] : 0u, h1 = NT == 2 ? qhi[NT == 2 ? k : 0][1] : 0u;
      if (k & 1) {
        mma16816(s1[0], qlo[k][0], h0, qlo[k][1], h1, f[0], f[1]);
        mma16816(s1[1], qlo[k][0], h0, qlo[k][1], h1, f[2], f[3]);
      } else {
        mma16816(s[0], qlo[k][0], h0, qlo[k][1], h1, f[0], f[1]);
        mma16816(s[1], qlo[k][0], h0, qlo[k][1], h1, f[2], f[3]);
      }
    }
    // this thread's logits of head `row` (and row + 8): slots 2 quad, 2 quad + 1, and 8 on
    float x[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[t][e] = (s[e >> 1][2 * t + (e & 1)] + s1[e >> 1][2 * t + (e & 1)]) * P.scale_log2;
        if (rows < kTileSlots && 2 * quad + (e & 1) + 8 * (e >> 1) >= rows) x[t][e] = kMinusInf;
      }
    if (P.logits) {
      const int64_t tile = (int64_t)c.before * P.kv_heads + h * c.n + c.i;
      if (tile < P.tiles_cap) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (head0 + row + 8 * t < P.group) {
            float* to = P.logits + (tile * P.group + head0 + row + 8 * t) * kTileSlots + 2 * quad;
            *reinterpret_cast<float2*>(to) = make_float2(x[t][0], x[t][1]);
            *reinterpret_cast<float2*>(to + 8) = make_float2(x[t][2], x[t][3]);
          }
      }
    }
    // the reference maximum follows when a logit is far above it
    bool over = false;
    float top[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      top[t] = fmaxf(fmaxf(x[t][0], x[t][1]), fmaxf(x[t][2], x[t][3]));
      over |= top[t] > m[t] + kLag;
    }
    if (__any_sync(kAll, over)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        top[t] = fmaxf(top[t], __shfl_xor_sync(kAll, top[t], 1));
        top[t] = fmaxf(top[t], __shfl_xor_sync(kAll, top[t], 2));
        float f = 1.f;
        if (top[t] > m[t] + kLag) {
          f = exp2_approx(m[t] - top[t]);  // the first time: exp2(-inf) = 0
          m[t] = top[t];
          l[t] *= f;
        }
        const float f0 = __shfl_sync(kAll, f, 8 * quad), f1 = __shfl_sync(kAll, f, 8 * quad + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[t][k][0] *= f0;
          o[t][k][1] *= f1;
          o[t][k][2] *= f0;
          o[t][k][3] *= f1;
        }
      }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float ref = m[t] == kMinusInf ? 0.f : m[t];  // nothing visible so far: exp2(-inf) = 0
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = exp2_approx(x[t][e] - ref);
      l[t] += (p[0] + p[1]) + (p[2] + p[3]);
      pb[t][0] = pack2_bf16(p[0], p[1]);
      pb[t][1] = pack2_bf16(p[2], p[3]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t f[4];  // (d 0-7, slots 0-7), (d 8-15, slots 0-7), (d 0-7, slots 8-15), (d 8-15, slots 8-15)
      load_tiles_t(f, at + (2 + (k >> 2)) * kBox + slot_row + (uint32_t)((((k & 3) * 2 + piece0) ^ tile_row) << 4));
#pragma unroll
      for (int t = 0; t < NT; ++t) mma16816(o[t][k], f[0], f[1], f[2], f[3], pb[t][0], pb[t][1]);
    }

    if (c.i + 1 == c.n || it + 1 == count) {  // the unit ends here, or this share of it
      const bool whole = first == 0 && c.i + 1 == c.n;
      const int64_t piece = 2 * (int64_t)w + (first == 0 ? 1 : 0);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        l[t] += __shfl_xor_sync(kAll, l[t], 1);
        l[t] += __shfl_xor_sync(kAll, l[t], 2);
        const int g = head0 + row + 8 * t;
        const int64_t out_row = (int64_t)c.b * P.heads + h * P.group + head0 + 8 * t;
        if (quad == 0 && g < P.group) {
          if (whole) {
            const float lse2 = m[t] + log2f(l[t]);
            const float lse = lse2 * 0.6931471805599453f;
            if (P.lse) P.lse[out_row + row] = lse;
            P.lse2[out_row + row] = lse2;
            if (!(fabsf(lse) < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
          } else {
            P.part_ml[piece * 16 + row + 8 * t] = make_float2(m[t], l[t]);
          }
        }
        const float d0 = 1.f / __shfl_sync(kAll, l[t], 8 * quad), d1 = 1.f / __shfl_sync(kAll, l[t], 8 * quad + 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // head 2 quad + e of this eight: elements 16 k + row and 16 k + 8 + row
          if (head0 + 8 * t + 2 * quad + e >= P.group) continue;
          const float d = e ? d1 : d0;
          if (whole) {
            __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(P.out) + (out_row + 2 * quad + e) * kD + row;
            float check = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float y0 = o[t][k][e] * d, y1 = o[t][k][2 + e] * d;
              check += y0 * 0.f + y1 * 0.f;
              to[16 * k] = __float2bfloat16_rn(y0);
              to[16 * k + 8] = __float2bfloat16_rn(y1);
            }
            if (check != 0.f) latch(P.status, BKV_ERR_NONFINITE);
          } else {
            // a piece's elements in the order of the fragments
            float4* to = P.part_o + (piece * kChunk + 8 * t + 2 * quad + e) * 32 + row * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              to[k] = make_float4(o[t][2 * k][e], o[t][2 * k][2 + e], o[t][2 * k + 1][e], o[t][2 * k + 1][2 + e]);
          }
        }
      }
      fresh = true;
    }
    step(P, c, units);
  }
  // a wait ran out: copies under way land before the shared memory goes
  for (; it < ahead; ++it) {
    wait_done(&bar[stage], phase);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
}

// The pieces of unit u of a sequence: shares c0 .. c1, share c0's piece is its second.
struct Pieces {
  int c0, c1;
  __device__ __forceinline__ int at(int c) const { return 2 * c + (c == c0 ? 1 : 0); }
};
__device__ __forceinline__ Pieces pieces_of(int before, int u, int n, int units, int share) {
  const int from = before * units + u * n;
  return Pieces{from / share, (from + n - 1) / share};
}
// A head's largest reference over the unit's pieces and the sum relative to it. Eight lanes,
// all get it; the warp's four eights each have their own pieces (or none).
__device__ __forceinline__ float2 join_sum(const AttendPagedParams& P, const Pieces& pc, int in_chunk, int lane) {
  // four pieces a lane at once, more in rounds: a running maximum and sum
  float m = kMinusInf, l = 0.f;
  for (int c0 = pc.c0; c0 <= pc.c1; c0 += 32) {
    float2 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 8 + (lane & 7);
      x[k] = c <= pc.c1 ? P.part_ml[pc.at(c) * 16 + in_chunk] : make_float2(kMinusInf, 0.f);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, x[k].x);
    if (m != kMinusInf) l *= exp2_approx(m - top);
    // a piece without a finite logit has no part (its sum is 0, or NaN, which stays)
#pragma unroll
    for (int k = 0; k < 4; ++k) l += x[k].x == kMinusInf ? x[k].y : x[k].y * exp2_approx(x[k].x - top);
    m = top;
  }
  float top = m;
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
  if (m != kMinusInf) l *= exp2_approx(m - top);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) l += __shfl_xor_sync(kAll, l, off);
  return make_float2(top, l);
}

// A row's running state over some of its pieces: reference, sum, and this lane's four elements.
struct Joined {
  float m, l;
  float4 y;
};
__device__ __forceinline__ void join_in(Joined& j, float m, float l, const float4& y) {
  const float top = fmaxf(j.m, m);
  const float f = j.m == kMinusInf ? 1.f : exp2_approx(j.m - top);  // without a finite logit so far: 0, or NaN, as it is
  const float g = m == kMinusInf ? 1.f : exp2_approx(m - top);
  j.m = top;
  j.l = j.l * f + l * g;
  j.y.x = j.y.x * f + y.x * g;
  j.y.y = j.y.y * f + y.y * g;
  j.y.z = j.y.z * f + y.z * g;
  j.y.w = j.y.w * f + y.w * g;
}
__device__ __forceinline__ Joined join_pieces(const AttendPagedParams& P, const Pieces& pc, int in_chunk, int from, int by, int lane) {
  Joined j{kMinusInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int c0 = from; c0 <= pc.c1; c0 += 4 * by) {
    float2 ml[4];
    float4 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * by;
      ml[k] = make_float2(kMinusInf, 0.f);
      y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c <= pc.c1) {
        ml[k] = P.part_ml[pc.at(c) * 16 + in_chunk];
        y[k] = P.part_o[(int64_t)(pc.at(c) * P.chunk + in_chunk) * 32 + lane];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) join_in(j, ml[k].x, ml[k].y, y[k]);
  }
  return j;
}

// Outputs of units that lie in several shares, and weights.
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) join_paged_kernel(const __grid_constant__ AttendPagedParams P) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float4 sums[kWarps][32];
  __shared__ float2 sums_ml[kWarps];
  __shared__ float lse2[kJoinHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = P.kv_heads * P.chunks;
  depend_wait();
  depend_go();
  const int x0 = tid < P.batch ? P.seq[tid].x : 0;
  const int tiles = P.seq[P.batch].x;
  const int share = share_of(tiles * units, P.shares);

  // Outputs, also those of sequences without a slot. Few rows: a block each (the last blocks,
  // the first have weights to do), its warps take the pieces in turn; many: a warp each.
  const int rows = P.batch * P.heads;
  const bool wide = rows <= (int)gridDim.x;
  const int block = gridDim.x - 1 - blockIdx.x;
  for (int r = wide ? block : block * kWarps + warp; r < rows; r += gridDim.x * (wide ? 1 : kWarps)) {
    const int b = r / P.heads, head = r - b * P.heads;
    const int2 q = P.seq[b];
    if (q.y == 0) {
      if (wide && warp != 0) continue;
      reinterpret_cast<uint2*>(P.out)[(int64_t)r * 32 + lane] = make_uint2(0, 0);
      if (lane == 0 && P.lse) P.lse[r] = kMinusInf;
      continue;
    }
    const int h = head / P.group, g = head - h * P.group, u = h * P.chunks + g / P.chunk, in = g % P.chunk;
    const Pieces pc = pieces_of(q.x, u, tiles_of(q.y), units, share);
    if (pc.c0 == pc.c1) continue;  // one answer for the whole block where it shares a row
    Joined j = join_pieces(P, pc, in, pc.c0 + (wide ? warp : 0), wide ? kWarps : 1, lane);
    if (wide) {
      sums[warp][lane] = j.y;
      if (lane == 0) sums_ml[warp] = make_float2(j.m, j.l);
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k) join_in(j, sums_ml[k].x, sums_ml[k].y, sums[k][lane]);
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const float inv = 1.f / j.l;
    float4 y = make_float4(j.y.x * inv, j.y.y * inv, j.y.z * inv, j.y.w * inv);
    if (j.l == 0.f) y.x = y.y = y.z = y.w = __builtin_nanf("");  // every logit is -inf
    // elements (lane / 4) + 8 i, i = 4 (lane % 4) .. + 3: the order of the fragments
    __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(P.out) + (int64_t)r * kD + (lane >> 2) + (lane & 3) * 32;
    to[0] = __float2bfloat16_rn(y.x);
    to[8] = __float2bfloat16_rn(y.y);
    to[16] = __float2bfloat16_rn(y.z);
    to[24] = __float2bfloat16_rn(y.w);
    const float check = (y.x * 0.f + y.y * 0.f) + (y.z * 0.f + y.w * 0.f);
    if (check != 0.f) latch(P.status, BKV_ERR_NONFINITE);
    if (lane == 0) {
      const float lse = (j.m + log2f(j.l)) * 0.6931471805599453f;
      if (P.lse) P.lse[r] = lse;
      if (!(fabsf(lse) < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
    }
  }

  if (!P.weights) return;
  // Weights: a block takes an equal share of the (sequence, KV head, tile) row, sequence by
  // sequence: its warps find the heads' sums, then a thread takes four slots of a tile.
  const int64_t all = (int64_t)tiles * P.kv_heads;
  if (all > P.tiles_cap) {  // a page in two tables: more tiles than the pool has slots for
    if (blockIdx.x == 0 && tid == 0) latch(P.status, BKV_ERR_INVALID_ARG);
    return;
  }
  const int each = max((int)((all + gridDim.x - 1) / gridDim.x), kJoinTiles);
  const int64_t begin = (int64_t)blockIdx.x * each;
  if (begin >= all) return;
  int t = (int)begin;
  const int end = (int)min(begin + each, all);
  // the sequence of tile t: the last with at most t tiles in front of it that has any itself
  int b = -1;
  for (int b0 = 0; b0 < P.batch; b0 += kJoinThreads) {
    const int n = __syncthreads_count(b0 + tid < P.batch && (b0 == 0 ? x0 : P.seq[b0 + tid].x) * P.kv_heads <= t);
    b += n;
    if (n < kJoinThreads) break;
  }
  const int most_heads = kJoinHeads / P.group;  // KV heads whose sums fit
  while (true) {
    const int2 seq = P.seq[b];
    const int len = seq.y, n = tiles_of(len), before = seq.x;
    if (len == 0) {  // none of its own; there are tiles left, so a later sequence has them
      if (++b >= P.batch) return;
      continue;
    }
    const int i0 = t - before * P.kv_heads, h0 = i0 / n;  // place in the sequence's tiles
    const int cnt = min(min(n * P.kv_heads, n * (h0 + most_heads)) - i0, end - t);
    const int heads = ((i0 + cnt - 1) / n - h0 + 1) * P.group;
    // four slots of a tile: their pool row, old weights and the first heads' logits, asked for
    // before the sums are looked for
    struct Slots {
      int64_t row;
      int in, h;
      float old[4];
      float4 x[kAhead];
    };
    auto fetch = [&](int q, Slots& v) {
      v.row = -1;
      if (q >= cnt * 4) return;
      const int i = i0 + q / 4;
      v.h = i / n;
      const int slot = (i - v.h * n) * kTileSlots + q % 4 * 4;
      v.in = min(4, len - slot);
      if (v.in <= 0) return;
      v.row = pool_row(P.pg, P.kv_heads, b, v.h, slot);
      if (!BKV_IN_RANGE(v.row + v.in <= (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) v.row = -1;
      if (v.row < 0) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) v.old[e] = e < v.in && P.decay != 0.f && slot + e != len - 1 ? P.weights[v.row + e] : 0.f;
      const float4* x = reinterpret_cast<const float4*>(P.logits + (int64_t)(t + q / 4) * P.group * kTileSlots) + q % 4;
#pragma unroll
      for (int g = 0; g < kAhead; ++g)
        if (g < P.group) v.x[g] = x[g * 4];
    };
    Slots now, next;
    fetch(tid, now);
    for (int k0 = warp * 4; k0 < heads; k0 += kWarps * 4) {
      const int k = min(k0 + (lane >> 3), heads - 1);
      const int h = h0 + k / P.group, g = k % P.group;
      Pieces pc = pieces_of(before, h * P.chunks + g / P.chunk, n, units, share);
      const bool whole = pc.c0 == pc.c1;
      if (whole) --pc.c1;  // no pieces
      float x = whole ? P.lse2[(int64_t)b * P.heads + h0 * P.group + k] : 0.f;
      const float2 ml = join_sum(P, pc, g % P.chunk, lane);
      if (!whole) x = ml.x + log2f(ml.y);
      if ((lane & 7) == 0) lse2[k] = x;  // lanes behind the last head write that one's again
    }
    __syncthreads();
    for (int q = tid; q < cnt * 4; q += kJoinThreads) {
      fetch(q + kJoinThreads, next);
      if (now.row >= 0) {
        const float* z = lse2 + (now.h - h0) * P.group;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](const float4& v, float l) {
          sum[0] += exp2_approx(v.x - l);
          sum[1] += exp2_approx(v.y - l);
          sum[2] += exp2_approx(v.z - l);
          sum[3] += exp2_approx(v.w - l);
        };
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
          if (g < P.group) add(now.x[g], z[g]);
        const float4* x = reinterpret_cast<const float4*>(P.logits + (int64_t)(t + q / 4) * P.group * kTileSlots) + q % 4;
#pragma unroll 4
        for (int g = kAhead; g < P.group; ++g) add(x[g * 4], z[g]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < now.in) P.weights[now.row + e] = fmaf(P.decay, now.old[e], sum[e]);
      }
      now = next;
    }
    t += cnt;
    if (t >= end) return;
    if (i0 + cnt == n * P.kv_heads && ++b >= P.batch) return;
    __syncthreads();
  }
}

template <int NT, int kWarps, int kStages>
cudaError_t launch(const AttendPagedParams& given, cudaStream_t s) {
  constexpr int kSmem = kWarps * kStages * kTileBox + 1024;
  static_assert(kWarps <= kAttendWarps, "the workspace holds the pieces of kAttendWarps warps per CTA");
  AttendPagedParams p = given;
  p.shares = kAttendCtas * kWarps;
  const auto fn = attend_paged_kernel<NT, kWarps, kStages>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = allow_shared(fn, kSmem, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kAttendCtas);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(kJoinCtas * kSms);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_paged_kernel, p);
}

}  // namespace

bool encode_attend_paged_maps(AttendPagedParams& p) {
  const cuuint64_t row = (cuuint64_t)kD * 2, plane = (cuuint64_t)p.pg.page_size * row;
  const cuuint64_t planes = (cuuint64_t)p.pg.pages * p.kv_heads;
  return encode_rows(&p.kmap, p.K, (cuuint64_t)p.pg.page_size, row, planes, plane, kTileSlots, 1) &&
         encode_rows(&p.vmap, p.V, (cuuint64_t)p.pg.page_size, row, planes, plane, kTileSlots, 1);
}

cudaError_t launch_attend_paged(const AttendPagedParams& p, cudaStream_t s) {
  // five warps with two tiles under way each: 192 sequences 269 us; four with three 280, three
  // with four 280, two with six 341. Sixteen rows leave registers for four.
  return p.chunk == 8 ? launch<1, 5, 2>(p, s) : launch<2, 4, 3>(p, s);
}

}  // namespace bkv
