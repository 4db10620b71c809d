// The attention weight that packed prompt queries give to every slot, summed over the
// queries and the query heads of a KV head, on the fifth-generation tensor cores.
//
//   S_j = sum_{i, g: first + i >= j} exp(q_ig . k_j / sqrt(d) - lse_ig)
//   weights[j] = decay weights[j] + S_j (j < first), S_j (j >= first)
//
// The product is taken transposed: the 128 slots of a tile are the rows (TMEM lanes) and
// the queries the columns, so a thread owns a slot and adds up its row in registers;
// no reduction over lanes, no atomics, the same bits every time. The tile's keys stay in
// TMEM as operand A for all queries (every thread loads its own slot's 256 bytes, whatever
// page they are in), so a product reads only the queries from shared memory: 64 bytes
// per clock and SM, with as much again from TMA writing the next ones.
//
// A tile of columns is tpt = 96 / G tokens with the G query heads of the KV head. Two
// buffers of 96 columns and the keys' 64 take 256 columns of TMEM, so that two CTAs
// share an SM and one's set-up, ends and hand-overs lie under the other's products.
// CTA: 8 warps that exponentiate and add, four for each buffer (so for every other tile), a
// TMA producer that also looks up the columns' log-sum-exps, an MMA issuer. Blocks of the
// grid take the slots' tiles in order, those that most queries see first. Where there are
// few such tiles, the CTAs of a cluster share one's queries and join their sums, in rank
// order, through distributed shared memory.
//
// Rounding: products and sums are fp32, nothing is rounded to fewer bits.
//
// Measured on one GB300 (1,924 TFLOP/s cuBLAS bf16): 2 prompts of 8,190 tokens, 28/4 heads, 362 us,
// 0.68; 8 of 1,359 - 2,064 tokens, 32/8 heads, 99 us, 0.52. A tile's product and its
// exponentials take 384 clocks of their units each; a CTA's tile takes 1,000 - 1,100, four of
// ten waiting for a buffer's way to the issuer and back (550 clocks beside the products in
// front of it), and an item 10,000 for its set-up, first logits and end. Not kept (against
// 366 and 102): three buffers of 64 columns 462 and 124, four CTAs of one such buffer 495 and
// 144, look-ups of the columns six tiles ahead 392 and 107. One adding warp for each 32 slots took 588 and 146.
#include <cstddef>

#include "paged/device.cuh"

namespace bkv {
namespace {

constexpr int kCols = kWeighRows, kHalf = kCols / 2;
constexpr int kQSlab = kCols * 128;              // 96 rows x 64 bf16
constexpr int kQTile = 2 * kQSlab;               // 24 KB
constexpr int kQStages = 4;
constexpr int kAdders = 8;                       // warps 0 - 7: warp w adds up every other tile (w / 4) for slots 32 (w % 4) ..
constexpr int kMostSplits = 8;
constexpr int kProducer = kAdders, kIssuer = kAdders + 1;
constexpr int kWeighThreads = 32 * (kAdders + 2);
constexpr int kColStages = 4;
constexpr uint32_t kTmemCols = 256, kTmemKeys = 192;  // two buffers of 96 columns, the keys behind them
constexpr int kWeighSmem = kQStages * kQTile + 1024;

struct WeighControl {
  uint64_t full[kQStages], empty[kQStages];
  uint64_t keys, keys_free;       // the keys are in TMEM; its products are done
  uint64_t sfull[2], sempty[2];   // a tile's logits are in TMEM and its columns written; the logits have been read
  uint64_t others[2];             // the odd tiles are added up; items in turn
  Ctl ctl;
  // -lse log2(e) of a tile's columns. Tile i's place is written when buffer i % 2 is free for
  // it, so after tile i - 2 has been read, and by the same warps tile i - 4 added up
  alignas(16) float col[kColStages][kCols];
  // per item (in turn): the odd tiles' sums. A group without a tile of an item is done with it
  // before the other group may have read those of the item in front, but no earlier than that
  // one's keys are all there, and so those of the item before it read
  float other[2][128];
  // per item (in turn) and warp: a key holds an infinity or NaN, which would make NaN of the
  // products with rows that no token fills
  int odd[2][kAdders];
  uint64_t ranks;                 // rank 0: the other ranks' sums are here
  float rank_sum[kMostSplits - 1][128];
};
static_assert(offsetof(WeighControl, col) % 16 == 0 && (kCols * sizeof(float)) % 16 == 0, "read as float4");

__device__ __forceinline__ uint32_t lane_elected() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e;
}
// A bounded wait, with one answer for the warp.
__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, Ctl* ctl, uint32_t* status) {
  return __all_sync(kFull, mbar_wait(b, parity, ctl, status));
}
// A (128 slots x 16 bf16) from TMEM, B (96 query rows) from shared memory.
template <uint32_t kAStep, uint32_t kBStep>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // SBO, version, SWIZZLE_128B
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 b;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %8, 0;\n add.u32 x, %1, %5;\n add.u32 y, %2, %6;\n"
      " mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kAStep), "n"(kBStep), "n"(kHi), "r"(elected));
}
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 TMEM lanes x 48 consecutive columns.
__device__ __forceinline__ void load_half(uint32_t taddr, float (&v)[kHalf]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int i = 0; i < kHalf; i += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]),
          "=r"(r[i + 7]), "=r"(r[i + 8]), "=r"(r[i + 9]), "=r"(r[i + 10]), "=r"(r[i + 11]), "=r"(r[i + 12]),
          "=r"(r[i + 13]), "=r"(r[i + 14]), "=r"(r[i + 15])
        : "r"(taddr + i));
}
// A value that tcgen05.ld delivers is there only after the wait: ties the registers to it.
__device__ __forceinline__ void tie(float (&v)[kHalf]) {
#pragma unroll
  for (int i = 0; i < kHalf; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7]));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Adds up the exponentials of half a tile's columns.
__device__ __forceinline__ void add_half(const float (&v)[kHalf], const float* col, uint64_t scale, uint64_t (&part)[2]) {
  const float4* cols = reinterpret_cast<const float4*>(col);
#pragma unroll
  for (int q = 0; q < kHalf / 4; ++q) {
    const float4 c = cols[q];
    float a0, a1, a2, a3;
    unpair(fma_pair(pair(v[4 * q], v[4 * q + 1]), scale, pair(c.x, c.y)), a0, a1);
    unpair(fma_pair(pair(v[4 * q + 2], v[4 * q + 3]), scale, pair(c.z, c.w)), a2, a3);
    part[0] = add_pair(part[0], pair(fast_exp2(a0), fast_exp2(a1)));
    part[1] = add_pair(part[1], pair(fast_exp2(a2), fast_exp2(a3)));
  }
}
// The same of columns from .. to - 1 only.
__device__ __forceinline__ void add_half_of(const float (&v)[kHalf], const float* col, int from, int to, uint64_t scale,
                                            uint64_t (&part)[2]) {
  const float4* cols = reinterpret_cast<const float4*>(col);
#pragma unroll
  for (int q = 0; q < kHalf / 4; ++q) {
    const float4 c = cols[q];
    float a[4];
    unpair(fma_pair(pair(v[4 * q], v[4 * q + 1]), scale, pair(c.x, c.y)), a[0], a[1]);
    unpair(fma_pair(pair(v[4 * q + 2], v[4 * q + 3]), scale, pair(c.z, c.w)), a[2], a[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = 4 * q + e >= from && 4 * q + e < to ? fast_exp2(a[e]) : 0.f;
    part[0] = add_pair(part[0], pair(a[0], a[1]));
    part[1] = add_pair(part[1], pair(a[2], a[3]));
  }
}

// Clusters: the CTAs of one share an item's tiles of columns.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_rank0(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void store_cluster(uint32_t a, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A bounded wait for what other CTAs of the cluster have written.
__device__ __forceinline__ bool wait_cluster(uint64_t* b, uint32_t parity, Ctl* ctl, uint32_t* status) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    if (__all_sync(kFull, ok)) return true;
    if (__any_sync(kFull, ctl->abort || clock64() - t0 > kWaitCycles)) {
      latch(status, BKV_ERR_TIMEOUT);
      ctl->abort = 1;
      return false;
    }
  }
}

// What a CTA works on: one tile of slots of one (sequence, KV head).
struct WeighItem {
  int b, h;
  int j0;         // first slot
  int i0, n;      // first token that sees a slot of the tile, tokens of the sequence
  int begin;      // packed index of the sequence's first token
  int first;      // slots before the first token
  int slots;      // slots of the sequence: first + n, at most what its table holds
  int tiles;      // tiles of query rows; 0: nothing to do
  int own;        // those of this CTA: rank, rank + splits, ...
};
// A sequence as the call may read it; `bad`: something had to be clamped.
__device__ __forceinline__ void read_sequence(const WeighParams& P, int b, int& begin, int& n, int& first, int& slots, bool& bad) {
  const int x = P.cu[b], y = P.cu[b + 1], f = P.first[b];
  begin = min(max(x, 0), P.total);
  const int end = min(max(y, begin), P.total);
  n = end - begin;
  first = min(max(f, 0), P.pg.cap);
  const int64_t most = (int64_t)first + n;
  slots = n == 0 ? 0 : (int)min(most, (int64_t)P.pg.cap);
  bad = begin != x || end != y || (n > 0 && (first != f || most > P.pg.cap));
}
__device__ __forceinline__ WeighItem item_of(const WeighParams& P, int item, int rank) {
  WeighItem w;
  const unsigned v = (unsigned)item / (unsigned)P.kv_heads, tile = v / (unsigned)P.batch;
  w.h = item - (int)v * P.kv_heads;
  w.b = (int)(v - tile * P.batch);
  bool bad;
  read_sequence(P, w.b, w.begin, w.n, w.first, w.slots, bad);
  w.j0 = (int)(tile * 128);  // a table holds fewer than 2^31 - 4096 slots, and the items come from it
  w.tiles = 0;
  w.i0 = 0;
  if (w.j0 < w.slots) {
    w.i0 = max(0, w.j0 - w.first);
    w.tiles = (w.n - w.i0 + P.tpt - 1) / P.tpt;
  }
  w.own = (w.tiles - rank + P.splits - 1) / P.splits;
  return w;
}

__global__ void __launch_bounds__(kWeighThreads, 2) weigh_kernel(const __grid_constant__ WeighParams P) {
  extern __shared__ unsigned char raw[];
  __shared__ WeighControl C;
  __shared__ int items;
  unsigned char* qring = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Ctl* ctl = &C.ctl;
  const int rank = P.splits > 1 ? (int)cluster_rank() : 0;
  const int item0 = blockIdx.x / P.splits, item_step = gridDim.x / P.splits;
  if (tid == 0) {
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&C.full[i], 1);
      mbar_init(&C.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&C.sfull[i], 2);
      mbar_init(&C.sempty[i], kAdders / 2);
    }
    mbar_init(&C.keys, kAdders);
    mbar_init(&C.keys_free, 1);
    mbar_init(&C.ranks, max((P.splits - 1) * kAdders / 2, 1));
    for (int i = 0; i < 2; ++i) mbar_init(&C.others[i], kAdders / 2);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tmem_alloc(&ctl->tmem_base, kTmemCols);
  // rows that no token fills are zero in every stage: their logits are finite
  const int filled = P.tpt * P.group;
  for (int i = tid; i < kQStages * 2 * (kCols - filled) * 8; i += kWeighThreads) {
    const int slab = i / ((kCols - filled) * 8), in = i - slab * (kCols - filled) * 8;
    *reinterpret_cast<uint4*>(qring + slab * kQSlab + filled * 128 + in * 16) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  depend_wait();
  // tiles of slots of the longest sequence: the order of items is tile by tile. A block or
  // cluster that has one item only needs no answer but that its item is there.
  const bool one = item_step >= P.items;
  if (warp == 0 && (!one || blockIdx.x == 0)) {
    int most = 0;
    bool bad = false;
    for (int b = lane; b < P.batch; b += 32) {
      int begin, n, first, slots;
      bool clamped;
      read_sequence(P, b, begin, n, first, slots, clamped);
      bad |= clamped;
      most = max(most, slots);
    }
    most = __reduce_max_sync(kFull, most);
    if (__any_sync(kFull, bad) && lane == 0 && blockIdx.x == 0) latch(P.status, BKV_ERR_INVALID_ARG);
    if (lane == 0) items = (int)(((unsigned)most + 127) / 128) * P.batch * P.kv_heads;
  }
  tc_fence_before();
  __syncthreads();
  depend_go();  // with the TMEM allocated: a later kernel's block on this SM must not get there first
  if (P.splits > 1) cluster_sync();  // the ranks' barriers are there
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = one ? P.items : items;

  if (warp == kProducer) {
    // Copies run two tiles ahead of the columns, which need a free buffer of logits.
    const uint64_t keep = policy_evict_last();  // queries are read once per tile of slots
    int ct[3], at[3];  // this lane's columns of a tile: token (none: never in the sequence), place in the log-sum-exps
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const int c = lane + 32 * p, t = c / P.group;
      ct[p] = c < filled ? t : 0x7FFFFFFF;
      at[p] = c < filled ? t * P.heads + c - t * P.group : 0;
    }
    uint32_t it = 0, ci = 0;  // tiles copied, columns written
    bool go = true;
    for (int item = item0; go && item < total; item += item_step) {
      const WeighItem w = item_of(P, item, rank);
      if (w.own <= 0) continue;
      const float* lse = P.row_lse + ((int64_t)w.begin + w.i0 + (int64_t)rank * P.tpt) * P.heads + w.h * P.group;
      int left = w.n - w.i0 - rank * P.tpt;  // tokens from the first of the tile on
      float next[3];
      auto columns = [&] {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          next[p] = -__builtin_huge_valf();
          if (ct[p] < left) next[p] = lse[at[p]];
        }
        lse += (int64_t)P.splits * P.tpt * P.heads;
        left -= P.splits * P.tpt;
      };
      columns();
      for (int k = 0; go && k < w.own + 2; ++k) {
        if (k < w.own) {
          const int s = it % kQStages;
          go = wait(&C.empty[s], (it / kQStages & 1) ^ 1, ctl, P.status);
          if (!go) break;
          if (lane == 0) {
            mbar_expect_tx(&C.full[s], (uint32_t)(2 * filled * 128));
            const int t = w.begin + w.i0 + (k * P.splits + rank) * P.tpt;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              tma_rows(smem_u32(qring + s * kQTile + x * kQSlab), &P.qmap, x * 64, w.h * P.group, t, &C.full[s], keep);
          }
          __syncwarp();
          ++it;
        }
        if (k >= 2) {
          go = wait(&C.sempty[ci & 1], (ci / 2 & 1) ^ 1, ctl, P.status);
          if (!go) break;
          float* col = C.col[ci % kColStages];
          // a row that sees nothing gives nothing
#pragma unroll
          for (int p = 0; p < 3; ++p) col[lane + 32 * p] = next[p] == -__builtin_huge_valf() ? next[p] : -next[p] * kLog2e;
          __syncwarp();
          if (lane == 0) mbar_arrive(&C.sfull[ci & 1]);
          ++ci;
          columns();
        }
      }
    }
    // copies under way land before the CTA's shared memory goes
    for (uint32_t k = it > kQStages ? it - kQStages : 0; k < it; ++k)
      wait_done(&C.full[k % kQStages], k / kQStages & 1);
  } else if (warp == kIssuer) {
    const uint32_t e = lane_elected();
    const uint32_t idesc = idesc_bf16(128, kCols);
    uint32_t it = 0, nth = 0;
    bool go = true;
    for (int item = item0; go && item < total; item += item_step) {
      const WeighItem w = item_of(P, item, rank);
      if (w.own <= 0) continue;
      go = wait(&C.keys, nth & 1, ctl, P.status);
      tc_fence_after();
      for (int k = 0; go && k < w.own; ++k, ++it) {
        const int s = it % kQStages, x = it & 1;
        go = wait(&C.full[s], it / kQStages & 1, ctl, P.status) && wait(&C.sempty[x], (it / 2 & 1) ^ 1, ctl, P.status);
        if (!go) break;
        tc_fence_after();
        const uint32_t q = smem_u32(qring + s * kQTile);
        const uint32_t b0 = ((q & 0x3FFFFu) >> 4) | (1u << 16), b1 = (((q + kQSlab) & 0x3FFFFu) >> 4) | (1u << 16);
        const uint32_t d = tmem + x * kCols, a = tmem + kTmemKeys;
        mma_ts<0, 0>(d, a, b0, idesc, 0, e);
        mma_ts<8, 2>(d, a, b0, idesc, 1, e);
        mma_ts<16, 4>(d, a, b0, idesc, 1, e);
        mma_ts<24, 6>(d, a, b0, idesc, 1, e);
        mma_ts<32, 0>(d, a, b1, idesc, 1, e);
        mma_ts<40, 2>(d, a, b1, idesc, 1, e);
        mma_ts<48, 4>(d, a, b1, idesc, 1, e);
        mma_ts<56, 6>(d, a, b1, idesc, 1, e);
        commit_if(&C.empty[s], e);
        commit_if(&C.sfull[x], e);
      }
      commit_if(&C.keys_free, e);
      ++nth;
    }
    // products under way are done before TMEM goes
    if (nth > 0) wait_done(&C.keys_free, (nth - 1) & 1);
  } else {
    uint32_t nth = 0, done = 0, phase = 0;  // items and tiles so far, parity of this group's buffer
    bool go = true;
    const int group = warp >> 2, mine = tid & 127;  // buffer, slot of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_mine = tmem + lanes + group * kCols;
    for (int item = item0; go && item < total; item += item_step) {
      const WeighItem w = item_of(P, item, rank);
      if (w.tiles == 0) continue;
      // this thread's key, one half of it, into its lane of TMEM
      const int slot = w.j0 + mine;
      const int64_t row = slot < w.slots ? pool_row(P.pg, P.kv_heads, w.b, w.h, slot) : -1;
      if (slot < w.slots && row < 0) latch(P.status, BKV_ERR_INVALID_ARG);
      const bool in = row >= 0 && BKV_IN_RANGE(row < (int64_t)P.pg.pages * P.kv_heads * P.pg.page_size, P.status);
      float s = 0.f;
      if (w.own > 0) {
        if (nth > 0) go = wait(&C.keys_free, (nth - 1) & 1, ctl, P.status);
        if (!go) break;
        tc_fence_after();
        uint32_t odd = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t r[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = in ? P.K[row * 16 + group * 8 + x * 4 + k] : make_uint4(0, 0, 0, 0);
            r[4 * k] = v.x;
            r[4 * k + 1] = v.y;
            r[4 * k + 2] = v.z;
            r[4 * k + 3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) odd |= ((r[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
          tmem_store16(tmem + lanes + kTmemKeys + group * 32 + x * 16, r);
        }
        odd = __any_sync(kFull, odd != 0);
        if (lane == 0) C.odd[nth & 1][warp] = (int)odd;  // the other group's warp reads it after a product with these keys
        tmem_stored();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.keys);
        ++nth;

        const uint64_t scale = pair(P.scale_log2, P.scale_log2);
        uint64_t sum[2] = {0ull, 0ull};  // of whole tiles of columns: tens of thousands of terms, so a tile's are added up first
        // this group's tiles of the item: every other one of the CTA's
        const int begin = ((done & 1) ^ group) * P.splits + rank, by = 2 * P.splits;
        uint32_t tile = done + ((done & 1) ^ group);  // counted over the CTA's items
        done += w.own;
        // tiles of columns in front of `seen` hold rows that do not see all slots, those from `full`
        // on rows of other sequences
        const int full = (w.n - w.i0) / P.tpt;
        int seen = (int)min(max((int64_t)w.j0 + 127 - w.first - w.i0 + P.tpt - 1, (int64_t)0) / P.tpt, (int64_t)full);
#pragma unroll 1
        for (int k = begin; k < w.tiles; k += by) {
          go = wait(&C.sfull[group], phase, ctl, P.status);
          if (!go) break;
          phase ^= 1;
          tc_fence_after();
          // the other group's keys have been looked at: a product with them is done
          if (k == begin && (odd | C.odd[(nth - 1) & 1][warp ^ 4])) seen = full;
          const bool whole = k >= seen && k < full;
          // this thread sees the columns from G * (slot - first - token of the tile's first row) on
          int from = 0, to = 0;
          if (!whole) {
            const int i = w.i0 + k * P.tpt;
            from = (int)min(max((int64_t)P.group * ((int64_t)slot - w.first - i), (int64_t)0), (int64_t)kCols);
            to = (int)min((int64_t)filled, (int64_t)(w.n - i) * P.group);
          }
          const float* col = C.col[tile % kColStages];
          tile += 2;
          uint64_t part[2] = {0ull, 0ull};
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += kHalf) {
            float v[kHalf];
            load_half(t_mine + c0, v);
            tmem_wait_ld();
            tie(v);
            if (c0 > 0) {  // read: the buffer may be filled again
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&C.sempty[group]);
            }
            if (whole) add_half(v, col + c0, scale, part);
            else add_half_of(v, col + c0, from - c0, to - c0, scale, part);
          }
          sum[0] = add_pair(sum[0], part[0]);
          sum[1] = add_pair(sum[1], part[1]);
        }
        if (!go) break;
        float a0, a1, a2, a3;
        unpair(sum[0], a0, a1);
        unpair(sum[1], a2, a3);
        s = (a0 + a1) + (a2 + a3);
        if (group == 1) {
          C.other[(nth - 1) & 1][mine] = s;
          __syncwarp();
          if (lane == 0) mbar_arrive(&C.others[(nth - 1) & 1]);
        } else {
          go = wait(&C.others[(nth - 1) & 1], (nth - 1) / 2 & 1, ctl, P.status);
          if (!go) break;
          s += C.other[(nth - 1) & 1][mine];
        }
      }
      if (group == 1) continue;
      if (rank > 0) {
        store_cluster(in_rank0(&C.rank_sum[rank - 1][mine]), s);
        __syncwarp();
        if (lane == 0) arrive_cluster(in_rank0(&C.ranks));
        continue;
      }
      if (P.splits > 1) {  // in the order of the ranks; such a cluster has one item
        go = wait_cluster(&C.ranks, 0, ctl, P.status);
        if (!go) break;
        for (int r = 1; r < P.splits; ++r) s += C.rank_sum[r - 1][mine];
      }
      if (in) {
        float old = 0.f;
        if (slot < w.first && P.decay != 0.f) old = P.decay * P.weights[row];
        P.weights[row] = old + s;
        if (!(fabsf(old + s) < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, kTmemCols);
  if (P.splits > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

}  // namespace

bool encode_weigh_map(WeighParams& p, const void* q, int64_t q_stride) {
  return encode_rows(&p.qmap, q, (cuuint64_t)p.heads, (cuuint64_t)kD * 2, (cuuint64_t)p.total, (cuuint64_t)q_stride * 2,
                     (cuuint32_t)p.group, (cuuint32_t)p.tpt);
}

cudaError_t launch_weigh(const WeighParams& p, int64_t items, cudaStream_t s) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_shared(weigh_kernel, kWeighSmem, configured);
  if (e != cudaSuccess) return e;
  WeighParams q = p;
  q.items = (int)items;
  // Shares are halved while that keeps all CTAs in three or so rounds of 2 x 152 and leaves
  // eight tiles of queries to each, for prompts of the average length
  const int64_t tiles = p.total / p.batch / p.tpt;
  q.splits = 1;
  while (q.splits < kMostSplits && items * q.splits < 4 * kSms && 16 * q.splits <= tiles) q.splits *= 2;
  cudaLaunchAttribute at[2];
  at[0] = dependent_launch();
  cudaLaunchConfig_t cfg{};
  // blocks walk on from there; a cluster has one item
  cfg.gridDim = dim3((unsigned)(items * q.splits < 8 * 2 * kSms || q.splits > 1 ? items * q.splits : 8 * 2 * kSms));
  cfg.blockDim = dim3(kWeighThreads);
  cfg.dynamicSmemBytes = kWeighSmem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (q.splits > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)q.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, weigh_kernel, q);
}

}  // namespace bkv
