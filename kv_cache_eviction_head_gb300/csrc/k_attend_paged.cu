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
// A warp's ring of tiles is private down to the thread: every thread copies (cp.async)
// the 16-byte pieces that its own matrix fragments are made of and reads back only
// those, so the ring needs no barrier and its shared-memory accesses no swizzle. This
// works since the fragments' inner dimensions may be permuted freely: S = Q K^T
// (m16n8k16, rows: query heads, columns: slots) takes as its k-steps the four 16-byte
// pieces q + 4j of a key row that thread q of a quad holds, on both sides alike;
// O^T = V^T P^T (rows: d, columns: heads) takes two neighbouring slots' pieces, whose
// elements are paired by byte permutes; and P as it leaves S is that product's B operand.
//
// Rounding: logits, maxima, sums, weights and O are fp32; P is rounded to bf16 for the
// product with bf16 V (at most 2^-8 relative per term, as the output), the sums and
// the weights take the unrounded values. The reference maximum moves only when a logit
// exceeds it by 8 in log2 (a factor of 256 in P, which costs no precision).
//
// Weights need the final sum: the first launch leaves its logits (fp32, 4 G bytes a
// slot) in the workspace, and the second turns them into probabilities.
#include "paged/paged.cuh"

namespace bkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kStages = 3;                  // tiles under way per warp
constexpr int kTileBytes16 = 2 * kTileSlots * kD * 2;  // K and V of a tile: 8 KB
constexpr int kAttendSmem = kAttendWarps * kStages * kTileBytes16;
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 5;                // per SM
constexpr int kJoinTiles = 16;              // tiles of a block's weights, at least
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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Copies 16 bytes, or writes 16 zero bytes.
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
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
// Tiles per share. One tile per warp at least; more when there are not warps enough.
__device__ __forceinline__ int share_of(int tiles) { return max((tiles + kAttendShares - 1) / kAttendShares, 1); }
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

template <int NT>
__global__ void __launch_bounds__(kAttendWarps * 32, 2) attend_paged_kernel(const __grid_constant__ AttendPagedParams P) {
  extern __shared__ __align__(128) unsigned char ring_bytes[];
  __shared__ int rows_in[kAttendWarps][kStages];  // visible slots of a tile
  constexpr int kChunk = 8 * NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane & 3, row = lane >> 2;
  const int w = blockIdx.x * kAttendWarps + warp;
  const int units = P.kv_heads * P.chunks;
  depend_wait();
  depend_go();

  bool bad;
  const int total = all_tiles(P, lane, bad) * units;
  if (w == 0 && lane == 0 && bad) latch(P.status, BKV_ERR_INVALID_ARG);
  const int share = share_of(total);
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

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_bytes) + warp * kStages * kTileBytes16 + lane * 16;
  auto fetch = [&](int stage) {
    const int slot0 = a.i * kTileSlots;
    const int h = a.u / P.chunks;
    int rows = min(kTileSlots, a.len - slot0);
    int64_t base = 0;
    if (a.page >= 0) {
      base = ((int64_t)a.page * P.kv_heads + h) * P.pg.page_size + (slot0 - page_of(P.pg, slot0) * P.pg.page_size);
    } else {
      rows = 0;
      if (lane == 0) latch(P.status, BKV_ERR_INVALID_ARG);
    }
    if (!BKV_IN_RANGE(base >= 0 && base + rows <= (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) rows = 0, base = 0;
    if (lane == 0) rows_in[warp][stage] = rows;
    const uint32_t dst = ring + stage * kTileBytes16;
    const uint4* k = P.K + base * 16 + (row * 16 + quad);
    const uint4* v = P.V + base * 16 + (quad * 32 + row);
    if (rows == kTileSlots) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) copy16(dst + (t * 4 + j) * 512, k + t * 128 + 4 * j);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) copy16(dst + (8 + s * 2 + j) * 512, v + (s & 1) * 16 + (s >> 1) * 128 + 8 * j);
    } else {  // zeros for the slots behind the last: what lies there may be NaN
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bool in = row + 8 * t < rows;
#pragma unroll
        for (int j = 0; j < 4; ++j) copy16_if(dst + (t * 4 + j) * 512, in ? k + t * 128 + 4 * j : P.K, in);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool in = 2 * quad + (s & 1) + 8 * (s >> 1) < rows;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          copy16_if(dst + (8 + s * 2 + j) * 512, in ? v + (s & 1) * 16 + (s >> 1) * 128 + 8 * j : P.V, in);
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
    copies_commit();
  }

  uint32_t qlo[8][2], qhi[NT == 2 ? 8 : 1][2];
  float o[NT][8][4];
  float m[NT], l[NT];
  int first = 0;  // tile of the unit that this piece begins with
  bool fresh = true;
  int stage = 0;
  for (int it = 0; it < count; ++it) {
    const int h = c.u / P.chunks, head0 = (c.u - h * P.chunks) * kChunk;  // first query head of the chunk, in its group
    if (fresh) {
      fresh = false;
      first = c.i;
      const uint4* q = P.q + (int64_t)c.b * P.q_stride + ((int64_t)h * P.group + head0) * 16 + quad;
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
        for (int j = 0; j < 4; ++j) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (in) x = q[(row + 8 * t) * 16 + 4 * j];
          if (t == 0) {
            qlo[2 * j][0] = x.x;
            qlo[2 * j][1] = x.y;
            qlo[2 * j + 1][0] = x.z;
            qlo[2 * j + 1][1] = x.w;
          } else if constexpr (NT == 2) {
            qhi[2 * j][0] = x.x;
            qhi[2 * j][1] = x.y;
            qhi[2 * j + 1][0] = x.z;
            qhi[2 * j + 1][1] = x.w;
          }
        }
      }
    }
    copies_wait<kStages - 2>();
    __syncwarp();
    const int rows = rows_in[warp][stage];
    const uint32_t at = ring + stage * kTileBytes16;
    // the stage that the tile before has left
    if (ahead < count) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      ++ahead;
      step(P, a, units);
      if (ahead < count) look_up(P, a);
    }
    copies_commit();
    stage = stage == kStages - 1 ? 0 : stage + 1;

    // all of the tile's pieces are asked for at once; two sums per eight slots halve the
    // chain of products
    uint4 kf[8], vf[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) kf[i] = lds16(at + i * 512);
#pragma unroll
    for (int i = 0; i < 8; ++i) vf[i] = lds16(at + (8 + i) * 512);
    float s[2][4], s1[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = s1[t][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4 k = kf[t * 4 + j];
        mma16816(s[t], qlo[2 * j][0], NT == 2 ? qhi[NT == 2 ? 2 * j : 0][0] : 0u, qlo[2 * j][1],
                 NT == 2 ? qhi[NT == 2 ? 2 * j : 0][1] : 0u, k.x, k.y);
        mma16816(s1[t], qlo[2 * j + 1][0], NT == 2 ? qhi[NT == 2 ? 2 * j + 1 : 0][0] : 0u, qlo[2 * j + 1][1],
                 NT == 2 ? qhi[NT == 2 ? 2 * j + 1 : 0][1] : 0u, k.z, k.w);
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
    for (int j = 0; j < 2; ++j) {
      const uint4 v0 = vf[j], v1 = vf[2 + j], v2 = vf[4 + j], v3 = vf[6 + j];
      const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
      const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a0 = __byte_perm(w0[e], w1[e], 0x5410), a1 = __byte_perm(w0[e], w1[e], 0x7632);
        const uint32_t a2 = __byte_perm(w2[e], w3[e], 0x5410), a3 = __byte_perm(w2[e], w3[e], 0x7632);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[t][j * 4 + e], a0, a1, a2, a3, pb[t][0], pb[t][1]);
      }
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
        for (int e = 0; e < 2; ++e) {  // head 2 quad + e of this eight
          if (head0 + 8 * t + 2 * quad + e >= P.group) continue;
          const float d = e ? d1 : d0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[2 * k] = o[t][j * 4 + k][e];
              y[2 * k + 1] = o[t][j * 4 + k][2 + e];
            }
            if (whole) {
              float check = 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                y[k] *= d;
                check += y[k] * 0.f;
              }
              if (check != 0.f) latch(P.status, BKV_ERR_NONFINITE);
              P.out[(out_row + 2 * quad + e) * 16 + row + 8 * j] =
                  make_uint4(pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3]), pack2_bf16(y[4], y[5]), pack2_bf16(y[6], y[7]));
            } else {
              float4* to = P.part_o + (piece * kChunk + 8 * t + 2 * quad + e) * 32 + (row + 8 * j) * 2;
              to[0] = make_float4(y[0], y[1], y[2], y[3]);
              to[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
      }
      fresh = true;
    }
    step(P, c, units);
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
// A head's largest reference over the unit's pieces and the sum relative to it. One warp,
// all lanes get it.
__device__ __forceinline__ float2 join_sum(const AttendPagedParams& P, const Pieces& pc, int in_chunk, int lane) {
  // eight pieces a lane at once, more in rounds: a running maximum and sum
  float m = kMinusInf, l = 0.f;
  for (int c0 = pc.c0; c0 <= pc.c1; c0 += 256) {
    float2 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = c0 + k * 32 + lane;
      x[k] = c <= pc.c1 ? P.part_ml[pc.at(c) * 16 + in_chunk] : make_float2(kMinusInf, 0.f);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, x[k].x);
    if (m != kMinusInf) l *= exp2_approx(m - top);
    // a piece without a finite logit has no part (its sum is 0, or NaN, which stays)
#pragma unroll
    for (int k = 0; k < 8; ++k) l += x[k].x == kMinusInf ? x[k].y : x[k].y * exp2_approx(x[k].x - top);
    m = top;
  }
  float top = m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
  if (m != kMinusInf) l *= exp2_approx(m - top);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(kAll, l, off);
  return make_float2(top, l);
}

// Outputs of units that lie in several shares, and weights.
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) join_paged_kernel(const __grid_constant__ AttendPagedParams P) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float4 sums[kWarps][32];
  __shared__ float lse2[kMaxGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = P.kv_heads * P.chunks;
  depend_wait();
  depend_go();
  bool bad;
  const int tiles = all_tiles(P, lane, bad);
  const int share = share_of(tiles * units);

  // Outputs, also those of sequences without a slot. Few rows: a block each (the last blocks,
  // the first have weights to do), its warps take the pieces in turn; many: a warp each.
  const int rows = P.batch * P.heads;
  const bool wide = rows <= (int)gridDim.x;
  const int block = gridDim.x - 1 - blockIdx.x;
  for (int r = wide ? block : block * kWarps + warp; r < rows; r += gridDim.x * (wide ? 1 : kWarps)) {
    const int b = r / P.heads, head = r - b * P.heads;
    const int len = len_of(P, b);
    if (len == 0) {
      if (wide && warp != 0) continue;
      reinterpret_cast<uint2*>(P.out)[(int64_t)r * 32 + lane] = make_uint2(0, 0);
      if (lane == 0 && P.lse) P.lse[r] = kMinusInf;
      continue;
    }
    const int h = head / P.group, g = head - h * P.group, u = h * P.chunks + g / P.chunk, in = g % P.chunk;
    int before = 0;
    for (int x = lane; x < b; x += 32) before += tiles_of(len_of(P, x));
    before = __reduce_add_sync(kAll, before);
    const Pieces pc = pieces_of(before, u, tiles_of(len), units, share);
    if (pc.c0 == pc.c1) continue;  // one answer for the whole block where it shares a row
    const float2 ml = join_sum(P, pc, in, lane);
    const float inv = 1.f / ml.y;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const int by = wide ? kWarps : 1;
#pragma unroll 8
    for (int c = pc.c0 + (wide ? warp : 0); c <= pc.c1; c += by) {
      const float m = P.part_ml[pc.at(c) * 16 + in].x;
      const float4 x = P.part_o[(int64_t)(pc.at(c) * P.chunk + in) * 32 + lane];
      const float f = m == kMinusInf ? 1.f : exp2_approx(m - ml.x) * inv;  // without a finite logit: o is 0, or NaN
      y.x = fmaf(f, x.x, y.x);
      y.y = fmaf(f, x.y, y.y);
      y.z = fmaf(f, x.z, y.z);
      y.w = fmaf(f, x.w, y.w);
    }
    if (wide) {
      sums[warp][lane] = y;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
          const float4 x = sums[k][lane];
          y.x += x.x;
          y.y += x.y;
          y.z += x.z;
          y.w += x.w;
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    if (ml.y == 0.f) y.x = y.y = y.z = y.w = __builtin_nanf("");  // every logit is -inf
    reinterpret_cast<uint2*>(P.out)[(int64_t)r * 32 + lane] = make_uint2(pack2_bf16(y.x, y.y), pack2_bf16(y.z, y.w));
    const float check = (y.x * 0.f + y.y * 0.f) + (y.z * 0.f + y.w * 0.f);
    if (check != 0.f) latch(P.status, BKV_ERR_NONFINITE);
    if (lane == 0) {
      const float lse = (ml.x + log2f(ml.y)) * 0.6931471805599453f;
      if (P.lse) P.lse[r] = lse;
      if (!(fabsf(lse) < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
    }
  }

  if (!P.weights) return;
  // Weights: a block takes an equal share of the (sequence, KV head, tile) row, unit by unit:
  // its warps find the heads' sums, then a thread takes four slots of a tile.
  const int64_t room = P.tiles_cap;
  const int64_t all = (int64_t)tiles * P.kv_heads;
  if (all > room) {  // a page in two tables: more tiles than the pool has slots for
    if (blockIdx.x == 0 && tid == 0) latch(P.status, BKV_ERR_INVALID_ARG);
    return;
  }
  const int each = max((int)((all + gridDim.x - 1) / gridDim.x), kJoinTiles);
  const int64_t begin = (int64_t)blockIdx.x * each;
  if (begin >= all) return;
  int t = (int)begin;
  const int end = (int)min(begin + each, all);
  int b, before;
  find_sequence(P, t, P.kv_heads, lane, b, before);
  int len = len_of(P, b), n = tiles_of(len), h = (t - before * P.kv_heads) / n, i0 = t - before * P.kv_heads - h * n;
  while (true) {
    const int cnt = min(n - i0, end - t);
    for (int g = warp; g < P.group; g += kWarps) {
      const Pieces pc = pieces_of(before, h * P.chunks + g / P.chunk, n, units, share);
      float x;
      if (pc.c0 == pc.c1) {
        x = P.lse2[(int64_t)b * P.heads + h * P.group + g];
      } else {
        const float2 ml = join_sum(P, pc, g % P.chunk, lane);
        x = ml.x + log2f(ml.y);
      }
      if (lane == 0) lse2[g] = x;
    }
    __syncthreads();
    for (int q = tid; q < cnt * 4; q += kJoinThreads) {
      const int slot = (i0 + q / 4) * kTileSlots + q % 4 * 4, in = min(4, len - slot);
      if (in <= 0) continue;
      const int64_t row = pool_row(P.pg, P.kv_heads, b, h, slot);
      if (row < 0 || !BKV_IN_RANGE(row + in <= (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status)) continue;
      float* w = P.weights + row;
      float old[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) old[e] = e < in && P.decay != 0.f && slot + e != len - 1 ? w[e] : 0.f;
      const float4* x = reinterpret_cast<const float4*>(P.logits + (int64_t)(t + q / 4) * P.group * kTileSlots) + q % 4;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int g = 0; g < P.group; ++g) {
        const float4 v = x[g * 4];
        const float z = lse2[g];
        sum[0] += exp2_approx(v.x - z);
        sum[1] += exp2_approx(v.y - z);
        sum[2] += exp2_approx(v.z - z);
        sum[3] += exp2_approx(v.w - z);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < in) w[e] = fmaf(P.decay, old[e], sum[e]);
    }
    t += cnt;
    if (t >= end) return;
    __syncthreads();
    i0 = 0;
    if (++h == P.kv_heads) {
      h = 0;
      before += n;
      do {  // there are tiles left, so a sequence has them
        if (++b >= P.batch) return;
        len = len_of(P, b);
      } while (len == 0);
      n = tiles_of(len);
    }
  }
}

template <int NT>
cudaError_t launch(const AttendPagedParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attend_paged_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttendSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = dependent_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kAttendCtas);
  cfg.blockDim = dim3(kAttendWarps * 32);
  cfg.dynamicSmemBytes = kAttendSmem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attend_paged_kernel<NT>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(kJoinCtas * kSms);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_paged_kernel, p);
}

}  // namespace

cudaError_t launch_attend_paged(const AttendPagedParams& p, cudaStream_t s) {
  return p.chunk == 8 ? launch<1>(p, s) : launch<2>(p, s);
}

}  // namespace bkv
