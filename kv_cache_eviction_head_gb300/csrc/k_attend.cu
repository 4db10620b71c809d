// Softmax attention of packed prompt tokens, or of a tree of drafted tokens,
// over the caches, on the fifth-generation tensor cores.
//
//   o[r] = sum_j p_rj V[j],  p_rj = exp(l_rj - lse_r),  l_rj = q_r . k_j / sqrt(d),
//   lse_r = ln sum_j exp(l_rj), over the slots j that row r sees.
//
// A row is (token, query head of the group); a tile is the 128 rows of
// tpt = 128 / G consecutive tokens, so that the G query heads that share a KV
// head read its keys once. One pass over the keys with a running maximum and
// sum: per 128-key tile S = Q K^T goes to TMEM, one thread per row reads its
// 128 logits, subtracts its reference maximum, exponentiates and writes P back
// over S as bf16, and O += P V accumulates in TMEM with P as the TMEM operand.
//
// Rounding: l, the maximum, the sum and O are fp32; P is rounded to bf16 for
// the product with bf16 V (at most 2^-8 relative per term, like the output's own
// rounding); the sum adds the unrounded values.
//
// The reference maximum only moves when a tile's maximum exceeds it by more
// than 8 (a factor 256 in P, which costs bf16 and fp32 no precision); O and
// the sum are rescaled then. The QK^T of a tile is issued after the PV of the
// tile before (one thread's MMAs run in the order of issue), so a row that has
// its logits may rescale O without further synchronisation.
//
// Instances by prompts or trees, persistent CTAs or a cluster per row block (an
// instance each keeps the others' code out of the instruction caches), and one or two
// row tiles; prompts of two tiles are many row blocks, so they have no cluster form.
// NQ = 2: two tiles per CTA share every K and V tile (64 KB per 8.4 MMAC, 32 bytes
// per clock and SM), their MMAs alternate, and 512 TMEM columns hold both S and both O. NQ = 1: one tile, 256 columns, for few rows;
// up to 32 rows two CTAs share an SM. Warps: 4 per tile for softmax, 4 for the
// output (NQ = 2; with one tile the softmax warps write it), one TMA producer,
// one MMA issuer, one scheduler. K and V tiles alternate in one ring of 32 KB
// stages.
//
// Few row blocks: the keys of a block are split over the CTAs of a cluster;
// each keeps its own maximum, sum and O, and the partial results are joined
// through distributed shared memory, in rank order, so results do not vary.
//
// Slots behind a sequence's last one may hold anything: their logits are replaced,
// not added to, and their V rows are zeroed in shared memory. Slots that only later
// rows of the call see keep their V, with P = 0.
//
// Measured on one GB300 (6.78 TB/s copy, 1,933 TFLOP/s cuBLAS bf16, 1,721 sustained):
//   two prompts of 8,190 tokens, 28/4 heads       595 us   1.60 PFLOP/s, 0.83 (0.93 of sustained)
//   8 prompts of 1,359 - 2,064 tokens, 32/8       157 us   1.26 PFLOP/s, 0.65 (0.73)
//   64 trees of 64 nodes over 4,112 slots, 28/4   190 us   1.14 PFLOP/s, 0.59 (0.66)
//   192 sequences decoding over 2,063 slots       229 us   6.75 TB/s,    1.00
// Decoding a batch is bound by HBM. Prompts and large trees lose 6 - 9 % to the board's
// power limit (first 200 calls against steady: prompts of 2,000 tokens 144 and 154 us,
// trees 170 and 186, the long prompts 551 and 592); the rest lies in the kernel and the
// launch. Between two key tiles a row tile's products take 2 x 512 clocks; its softmax
// 1,000 - 1,200 (in isolation 910: 430 of exponentials, 160 maximum, 170 TMEM, 95
// sums), the hand-overs 300. The two tiles alternate, so a pair of key tiles takes
// 2,340 - 2,400 clocks instead of the products' 2,048, and a row block 4,000 more
// (first logits, ragged last tile, both tiles' softmax at once); row blocks are handed
// out whole, so the last round of them leaves SMs idle (trees: 27 us on average).
// The last tile's products end with its last visible quarter: 160 -> 157 us for the
// prompts of 2,000, trees 191 -> 187. The next block's first product between the last
// ones of this block cut 1,850 clocks per block and, at the power limit, no time.
// Before: without the uniform issuer (below) the long prompts took 764 us, with one
// thread computing descriptors in a branch 882, with the whole row unpacked 995.
// Measured and not kept (the long prompts, against 625 us then): half a row per
// thread, 691; three hand-overs per tile, 669; two issuers, 832; logits read twice
// from TMEM in rolled loops, 653.
#include <atomic>

#include "attend/attend.cuh"
#include "score_common.cuh"

namespace bkv {
namespace {

// A wait of this kernel: bounded like mbar_wait, in a third of its instructions
// (there are forty of them; with the others and all kinds of call in one kernel it was
// 118 KB of code, 47 - 65 KB an instance now: long prompts 625 -> 600 us). A wait
// that runs out raises the abort flag; the status is latched once, at the end. In the
// bounds-checked build a test can lower the bound (bkv_checked_wait_cycles) and see
// waits run out at any point of a call; its waits do not suspend the thread, which
// could outlast a short bound.
#ifdef BKV_CHECKED
__device__ uint32_t wait_cycles = (uint32_t)kWaitCycles;
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
#else
constexpr uint32_t wait_cycles = (uint32_t)kWaitCycles;
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) { return mbar_test(b, parity); }
#endif
__device__ __forceinline__ uint32_t clock32() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, Ctl* ctl) {
  if (bar_test(b, parity)) return true;
  const uint32_t t0 = clock32();
  do {
    if (bar_test(b, parity)) return true;
  } while (!ctl->abort && clock32() - t0 < wait_cycles);
  ctl->abort = 1;
  return false;
}
// Waits for work already handed to the hardware (a copy, an MMA), whatever has become
// of the call: shared memory and TMEM must not change hands before it is done.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity, Ctl* ctl) {
  const uint32_t t0 = clock32();
  while (!mbar_test(b, parity)) {
    if (clock32() - t0 >= (uint32_t)kWaitCycles) {
      ctl->abort = 1;
      return;
    }
  }
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kNaN = __builtin_nanf("");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // log2 units by which the reference maximum may lag

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// One lane of the warp, the same one every time (elect.sync).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e;
}
// One MMA of 16 along K, issued by the lane with `elected` set. The whole warp
// runs these, with warp-uniform operands: under a branch on the lane the
// operands take vector registers and a detour to the uniform ones, and the
// issuer falls behind the tensor core whenever the softmax warps are busy.
// Shared-memory descriptors travel as their low words plus a constant step.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // SBO, version, SWIZZLE_128B
template <uint32_t kAStep, uint32_t kBStep>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate,
                                        uint32_t elected) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %8, 0;\n add.u32 x, %1, %5;\n add.u32 y, %2, %6;\n"
      " mov.b64 a, {x, %7};\n mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kAStep), "n"(kBStep), "r"(kDescHi), "r"(elected));
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
// A (the 128 x 16 bf16 probabilities) from TMEM, two elements per 32-bit column.
template <uint32_t kAStep, uint32_t kBStep>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                        uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 b;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %8, 0;\n add.u32 x, %1, %5;\n add.u32 y, %2, %6;\n"
      " mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kAStep), "n"(kBStep), "r"(kDescHi), "r"(elected));
}
__device__ __forceinline__ void umma_commit_if(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A value that tcgen05.ld delivers is there only after the wait: this ties the
// registers to what precedes it, so that no use moves in front of the wait.
__device__ __forceinline__ void pin(float (&v)[32]) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                    "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                    "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                    "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

// Low words. Q and K [row][d], d contiguous: K-major SWIZZLE_128B (sw128_desc).
// V [keys][d] as B operand: MN-major SWIZZLE_128B; one atom is 64 d x 8 keys (8
// rows of 128 bytes), the next 8 keys follow 1024 bytes on (SBO), the next 64 d
// one slab on (LBO).
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(kSlabBytes >> 4) << 16);
}
constexpr uint32_t kIdescBMn = 1u << 16;  // instruction descriptor: B is MN-major

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Takes a block of this grid that has not started (its work is then this CTA's):
// 16 bytes that say which arrive in shared memory.
__device__ __forceinline__ void take_block(void* result, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(result)),
               "r"(smem_u32(bar))
               : "memory");
}
// The block taken, or -1: none is left.
__device__ __forceinline__ int taken_block(const void* result) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b32 y, z, w;\n .reg .b64 lo, hi;\n"
      " ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 r, {lo, hi};\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.b32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(result))
      : "memory");
  return got ? (int)x : -1;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// What one row block works on.
struct Block {
  int b, h;      // sequence, KV head
  int64_t row0;  // packed index of its first token
  int cnt;       // its tokens
  int past;      // slots before its first token (causal: token i sees past + i + 1 slots)
  int L;         // tree: committed slots (every node sees them)
  int nodes;     // tree: nodes visible in the cache
  int kv_len;    // slots that some row may see
  int v_len;     // slots that some row of the call may see
  int i0;        // its first token's place in the sequence
  bool bad;      // a length had to be clamped
};

// Where a search for a prompt's row block may begin: `before` blocks lie in the
// sequences before b0.
struct Cursor {
  int b0 = 0, before = 0;
};

// Prompt: row blocks sequence by sequence, the last (longest) first. One warp, 128
// sequences a step. Items behind the last block return cnt = 0.
__device__ __forceinline__ Block find_prompt_block(const AttendParams& P, int item, int tpi, Cursor& cur) {
  const int lane = threadIdx.x & 31;
  Block k;
  k.h = item % P.kv_heads;
  const int at = item / P.kv_heads;
  k.b = 0;
  k.row0 = 0;
  k.cnt = k.past = k.L = k.nodes = k.kv_len = k.v_len = k.i0 = 0;
  k.bad = false;
  if (at < cur.before) cur = Cursor{};
  for (; cur.b0 < P.batch; cur.b0 += 128) {
    const int b = cur.b0 + 4 * lane;  // this lane's four sequences
    int edge[5], nb[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) edge[i] = P.cu[min(b + i, P.batch)];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int begin = min(max(edge[i], 0), P.total), end = min(max(edge[i + 1], begin), P.total);
      if (b + i < P.batch) k.bad |= begin != edge[i] || end != edge[i + 1];
      nb[i] = b + i < P.batch ? (end - begin + tpi - 1) / tpi : 0;
      sum += nb[i];
    }
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, upto, off);
      if (lane >= off) upto += y;
    }
    k.bad = __any_sync(kFull, k.bad);
    const unsigned hit = __ballot_sync(kFull, at - cur.before < upto);
    if (!hit) {
      cur.before += __shfl_sync(kFull, upto, 31);
      continue;
    }
    // the lane that has the block, then which of its four sequences
    const int src = __ffs(hit) - 1;
    int left = at - cur.before - (upto - sum), which = 0, blocks = nb[0], beg = edge[0], end = edge[1];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (which == i - 1 && left >= nb[i - 1]) {
        left -= nb[i - 1];
        which = i;
        blocks = nb[i];
        beg = edge[i];
        end = edge[i + 1];
      }
    k.b = __shfl_sync(kFull, b + which, src);
    beg = min(max(__shfl_sync(kFull, beg, src), 0), P.total);
    end = min(max(__shfl_sync(kFull, end, src), beg), P.total);
    k.i0 = (__shfl_sync(kFull, blocks, src) - 1 - __shfl_sync(kFull, left, src)) * tpi;
    k.row0 = (int64_t)beg + k.i0;
    k.cnt = min(tpi, end - beg - k.i0);
    const int f = P.first[k.b];
    const int fc = min(max(f, 0), P.max_cache);
    k.past = fc + k.i0;
    k.kv_len = (int)min((int64_t)k.past + k.cnt, (int64_t)P.max_cache);
    k.v_len = (int)min((int64_t)fc + (end - beg), (int64_t)P.max_cache);
    k.bad |= fc != f || (int64_t)k.past + k.cnt > P.max_cache;
    return k;
  }
  return k;
}

__device__ __forceinline__ Block find_tree_block(const AttendParams& P, int item, int tpi) {
  Block k;
  const int qb = item % P.qblocks, u = item / P.qblocks;
  k.h = u % P.kv_heads;
  k.b = u / P.kv_heads;
  const int len = P.first[k.b];
  const int nn = P.nodes ? P.nodes[k.b] : P.n;
  const int used = min(max(nn, 0), P.n);
  k.L = min(max(len, 0), P.max_cache);
  k.nodes = min(used, P.max_cache - k.L);
  k.kv_len = k.v_len = k.L + k.nodes;
  k.bad = k.L != len || used != nn || k.nodes != used;
  k.i0 = qb * tpi;
  k.row0 = (int64_t)k.b * P.n + k.i0;
  k.cnt = min(tpi, used - k.i0);
  k.past = k.L + k.i0;
  return k;
}

constexpr int kMaxStages = 6;
constexpr int kWarpOut = 32 * 128;       // staging of a warp's output rows, one 64-column half at a time
constexpr int kTileOut = 2 * kSlabBytes;  // output warps: both halves of a tile

// What a row block needs in shared memory, handed from the scheduler to the other warps.
struct Work {
  Block blk;      // blk.cnt = 0: no more work
  int t_lo, nt;   // this CTA's key tiles
};

// Quarters (32 keys) of the last tile `tile` that row tile q sees some of, at least one.
// Products stop there: the rows after a block's first ones end inside a tile, and at the
// board's power limit every MMA left out counts.
template <bool kTree>
__device__ __forceinline__ int last_quarters(const Block& k, int q, int tpt, int tile) {
  const int end = kTree ? k.kv_len : min(k.past + (q + 1) * tpt, k.kv_len);
  return min(max((end - tile * kTileKeys + 31) >> 5, 1), 4);
}

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];  // K/V ring
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];      // a tile's logits are in TMEM (and its PV before is done)
  uint64_t pfull[2][2];   // half of its probabilities are
  uint64_t ofull[2], ofree[2];  // O is complete; O (and the row statistics) have been read
  uint64_t rfull[2];            // a tile's row statistics are in shared memory
  uint64_t staged[2], unstaged[2];  // output warps: a half tile is in its buffer; the buffer may be filled
  uint64_t wfull[2], wempty[2];  // work slots
  uint64_t want, taken;   // the producer runs out of work; a block has been taken
  uint64_t done;          // every MMA of the CTA is done
  uint4 block;            // its name
  Work work[2];
  Ctl ctl;
};

// With two tiles per CTA four more warps write the output, so that the softmax
// warps go on with the next row block at once. With one tile two CTAs share the SM
// (and its registers), and one's output overlaps the other's work anyway.
__host__ __device__ constexpr bool output_warps(int nq) { return nq == 2; }

struct Smem {
  uint32_t slab_q, q, ring, out, stats, control, total;
};
// The ring starts behind the rows in use; an MMA reads 128 rows of Q whatever
// their number, the rest of them from the ring: rows nobody looks at.
__host__ __device__ inline Smem attend_smem(int nq, int group, int tpt, int stages) {
  Smem s;
  const int rows = group * tpt;
  s.slab_q = (uint32_t)((rows + 7) / 8) * 1024;
  s.q = 0;
  s.ring = s.q + (uint32_t)nq * 2 * s.slab_q;
  s.out = s.ring + (uint32_t)stages * kTileBytes;
  s.stats = s.out + (output_warps(nq) ? kTileOut : (uint32_t)((rows + 31) / 32) * kWarpOut);
  s.control = s.stats + (output_warps(nq) ? (uint32_t)nq * 128 * 8 : 0);
  s.total = s.control + (uint32_t)((sizeof(Control) + 15) / 16 * 16);
  return s;
}

__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f ? (m + fast_log2(l)) * kLn2 : (l == 0.f ? kNegInf : l);  // no visible slot: -inf; NaN stays
}
__device__ __forceinline__ float row_scale(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }

// Whether a token or node of a block sees any slot. One that does and still has a sum of
// zero has logits of -inf alone: its softmax is not a number.
__device__ __forceinline__ bool sees_any(const AttendParams& P, const Block& k, int tok) {
  if (!P.mask || k.L > 0) return true;
  return ((uint64_t)P.mask[k.row0 + tok] << (64 - k.nodes)) != 0;  // nodes: 1 .. 64
}

// 64 columns of one warp's 32 rows of O, out of TMEM: normalised, rounded and put
// into a SWIZZLE_128B slab (row r of the warp at slab + r * 128 bytes). `check`
// stays finite unless some value is not. `free_bar`, if any, gets the warp's
// arrival once the columns have been read.
__device__ __forceinline__ void stage_half(uint32_t t_o, uint4* slab, uint64_t inv2, uint64_t (&check)[2], uint64_t* free_bar) {
  const int lane = threadIdx.x & 31;
  const uint64_t tiny2 = pack2(0x1p-10f, 0x1p-10f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float o[32];
    tmem_ld32(t_o + (uint32_t)c * 32, o);
    tmem_wait_ld();
    pin(o);
    if (c == 1 && free_bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(free_bar);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t x = mul2(pack2(o[i * 8 + 2 * e], o[i * 8 + 2 * e + 1]), inv2);
        check[e & 1] = fma2(x, tiny2, check[e & 1]);
        float a, b;
        unpack2(x, a, b);
        y[e] = pack_bf16(a, b);
      }
      slab[lane * 8 + ((c * 4 + i) ^ (lane & 7))] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}
// The warp's rows of a staged half to memory, 8 lanes per row. `mine`: where this
// lane's row goes, in rows from orow0, or -1.
__device__ __forceinline__ void write_half(const AttendParams& P, const uint4* slab, int64_t orow0, int mine, int half) {
  const int lane = threadIdx.x & 31;
  uint4* dst = reinterpret_cast<uint4*>(P.out) + orow0 * 16 + half * 8 + (lane & 7);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    uint4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (k + i) + (lane >> 3);
      y[i] = slab[r * 8 + ((lane & 7) ^ (r & 7))];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = __shfl_sync(kFull, mine, 4 * (k + i) + (lane >> 3));
      if (at >= 0 && BKV_IN_RANGE(orow0 + at >= 0 && orow0 + at < (int64_t)P.total * P.heads, P.status))
        dst[(int64_t)at * 16] = y[i];
    }
  }
}
// This lane's log-sum-exp, and the verdict on its row.
__device__ __forceinline__ void write_lse(const AttendParams& P, int64_t orow, float m, float l, const uint64_t (&check)[2]) {
  if (!BKV_IN_RANGE(orow >= 0 && orow < (int64_t)P.total * P.heads, P.status)) return;
  const float lse = row_lse(m, l);
  if (P.lse) P.lse[orow] = lse;
  float a, b;
  unpack2(add2(check[0], check[1]), a, b);
  if (!(fabsf(a + b) < __builtin_huge_valf()) || !(lse < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
}

// kTree: node masks and one length per sequence; else packed prompts. kCluster:
// one row block per cluster of `splits` CTAs; else persistent CTAs, splits = 1. An
// instance for each keeps the others' code out of the instruction caches.
template <int NQ, bool kTree, bool kCluster>
__global__ void __launch_bounds__(NQ * 128 + (output_warps(NQ) ? 256 : 128), NQ == 1 ? 2 : 1)
attend_kernel(const __grid_constant__ AttendParams P, const int splits_given) {
  extern __shared__ __align__(1024) unsigned char smem[];  // swizzled tiles: 1 KB aligned
  if (smem_u32(smem) & 1023u) {
    depend_wait();
    latch(P.status, BKV_ERR_INTERNAL);
    return;
  }
  const int splits = kCluster ? splits_given : 1;
  constexpr int kSoftmaxWarps = NQ * 4;
  constexpr bool kOut = output_warps(NQ);
  constexpr int kControl = kSoftmaxWarps + (kOut ? 4 : 0);  // first warp of the control warpgroup
  constexpr int kProducer = kControl, kIssuer = kControl + 1, kScheduler = kControl + 2;
  constexpr uint32_t kCols = NQ * 256;  // per tile: 128 columns of S (and P), 128 of O
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int tpi = NQ * P.tpt;

  const Smem lay = attend_smem(NQ, P.group, P.tpt, P.stages);
  unsigned char* q_s = smem + lay.q;
  unsigned char* ring = smem + lay.ring;
  float2* ml = reinterpret_cast<float2*>(q_s);  // [NQ * 128] partial maximum and sum, once Q is done with
  float2* stats_s = reinterpret_cast<float2*>(smem + lay.stats);  // [2][128] a finished tile's maximum and sum per row
  Control& C = *reinterpret_cast<Control*>(smem + lay.control);
  Ctl* ctl = &C.ctl;
  const int S = P.stages;
  const int wpt = (P.group * P.tpt + 31) / 32;  // softmax warps with rows in a full tile

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      mbar_init(&C.full[i], 1);
      mbar_init(&C.empty[i], 1);
    }
#pragma unroll 1
    for (int q = 0; q < NQ; ++q) {
      mbar_init(&C.qfull[q], 1);
      mbar_init(&C.qempty[q], 1);
      mbar_init(&C.sfull[q], 1);
      mbar_init(&C.pfull[q][0], (uint32_t)wpt);
      mbar_init(&C.pfull[q][1], (uint32_t)wpt);
      mbar_init(&C.ofull[q], 1);
      mbar_init(&C.ofree[q], (uint32_t)wpt);
      mbar_init(&C.rfull[q], (uint32_t)wpt);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&C.wfull[i], 1);
      mbar_init(&C.staged[i], (uint32_t)wpt);
      mbar_init(&C.unstaged[i], 1);
      mbar_init(&C.wempty[i], (uint32_t)((NQ + (kOut ? 1 : 0)) * wpt + 2));
    }
    mbar_init(&C.want, 1);
    mbar_init(&C.taken, 1);
    mbar_init(&C.done, 1);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tmem_alloc(&ctl->tmem_base, kCols);
  if (warp == kProducer && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &P.qmap : lane == 1 ? &P.kmap : &P.vmap) : "memory");
  depend_wait();
  const int first_item = (int)(blockIdx.x / (unsigned)splits);
  // Every warp's start: barriers and TMEM are there. The scheduler comes to it with
  // the first block found.
  auto start = [&]() {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    depend_go();  // with the TMEM allocated: a later kernel's block on this SM must not get there first
    return __shfl_sync(kFull, ctl->tmem_base, 0);
  };

  // The next piece of work; false: none is left, or a wait ran out. Every lane of
  // a warp gets it; one arrival per warp frees the slot.
  int works = 0;
  auto next_work = [&](Work& w) {
    const int slot = works & 1;
    if (!__all_sync(kFull, bar_wait(&C.wfull[slot], (uint32_t)((works >> 1) & 1), ctl))) return false;
    w = C.work[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&C.wempty[slot]);
    ++works;
    return w.blk.cnt > 0;
  };

  // One warp's part of a cluster's partial results: O as it is, 16-byte chunk c of a
  // row at c ^ (row & 31) against bank conflicts, and the row's maximum and sum.
  auto write_partial = [&](uint32_t t_o, int q, int row, float m, float l, bool any) {
    ml[q * 128 + row] = make_float2(m, l);
    if (!any) return;
    float4* part = reinterpret_cast<float4*>(ring) + (size_t)(q * 128 + row) * 32;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[32];
      tmem_ld32(t_o + (uint32_t)c * 32, o);
      tmem_wait_ld();
      pin(o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[(c * 8 + i) ^ lane] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  };

  // The softmax warps hold a row's 128 logits; the control warpgroup (producer,
  // issuer, scheduler, one idle warp) and the output warps give them registers:
  // 48 + 208 = 2 * 128 a thread for one tile, 56 + 104 + 2 * 176 = 4 * 128 for two.
  if (warp >= kControl) {
    regs_dec<NQ == 1 ? 48 : 56>();
    if (warp == kScheduler) {
      // ---------------------------------------------------------- scheduler
      // The grid has one CTA per row block, the longest first; a CTA that runs out
      // of work takes a block that has not started (the hardware hands them out),
      // so the setup and the pipeline's ends are paid once per SM and the order of
      // the grid still balances the load. A cluster works on its one block.
      int item = first_item;
      int n = 0, tries = 0;
      bool started = false;
      Cursor cursor;
      bool ok = true;
      auto publish = [&](const Work& w) {
        const int slot = n & 1;
        if (n >= 2) ok = __all_sync(kFull, bar_wait(&C.wempty[slot], (uint32_t)(((n >> 1) - 1) & 1), ctl));
        if (ok && lane == 0) {
          C.work[slot] = w;
          mbar_arrive(&C.wfull[slot]);
        }
        ++n;
      };
      while (ok) {
        Work w;
        if constexpr (kTree) w.blk = find_tree_block(P, item, tpi);
        else w.blk = find_prompt_block(P, item, tpi, cursor);
        if (!started) start();
        started = true;
        if (w.blk.bad && lane == 0) latch(P.status, BKV_ERR_INVALID_ARG);
        if (w.blk.cnt > 0) {
          const int T = (w.blk.kv_len + kTileKeys - 1) / kTileKeys;
          // splits <= 16 and T < 2^24: no overflow
          w.t_lo = T * rank / splits;
          w.nt = T * (rank + 1) / splits - w.t_lo;
          publish(w);
          if (ok && !kCluster) ok = __all_sync(kFull, bar_wait(&C.want, (uint32_t)((n - 1) & 1), ctl));
        }
        if (!ok || kCluster) break;
        if (lane == 0) {
          mbar_expect_tx(&C.taken, 16);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last name has been read
          take_block(&C.block, &C.taken);
        }
        ok = __all_sync(kFull, bar_wait(&C.taken, (uint32_t)(tries & 1), ctl));
        if (!ok) {  // the name must land before the CTA exits
          drain(&C.taken, (uint32_t)(tries & 1), ctl);
          break;
        }
        ++tries;
        item = taken_block(&C.block);
        __syncwarp();
        if (item < 0) break;
      }
      if (ok) {
        Work w;
        w.blk.cnt = 0;
        publish(w);
      }
    } else if (warp == kProducer) {
      // ---------------------------------------------------------- TMA producer
      start();
      const uint64_t pol = policy_evict_normal();
      const uint32_t qbytes = (uint32_t)(P.group * P.tpt) * 128;
      int st = 0;
      uint32_t loads0 = 0, loads1 = 0;  // of each row tile's queries
      long long g = 0;
      uint32_t ph = 0;
      bool ok = true;
      Work w;
      while (ok && next_work(w)) {
        if (lane == 0 && w.nt > 0) {
          const Block& blk = w.blk;
          const int nq = NQ == 1 || blk.cnt <= P.tpt ? 1 : 2;
          const int z = blk.b * P.kv_heads + blk.h;
          const int call = 2 * w.nt > 8 ? 2 * w.nt - 8 : 0;  // four tiles before the end
#pragma unroll 1
          for (int i = 0; i < 2 * w.nt && ok; ++i) {
            if (i == call) mbar_arrive(&C.want);
            if (g >= S) ok = bar_wait(&C.empty[st], ph ^ 1u, ctl);
            if (!ok) break;
            mbar_expect_tx(&C.full[st], kTileBytes);
            const uint32_t dst = smem_u32(ring) + (uint32_t)st * kTileBytes;
            const CUtensorMap* map = (i & 1) ? &P.vmap : &P.kmap;
            const int y = (w.t_lo + (i >> 1)) * kTileKeys;
            tma_load_3d(dst, map, 0, y, z, &C.full[st], pol);
            tma_load_3d(dst + kSlabBytes, map, 64, y, z, &C.full[st], pol);
            ++g;
            if (++st == S) {
              st = 0;
              ph ^= 1u;
            }
            // Queries behind the first keys, which need not wait for the last block's
            // products; a tile's own as soon as its last logits are there.
            if (i == 0) {
#pragma unroll 1
              for (int q = 0; q < nq && ok; ++q) {
                const uint32_t n = q ? loads1 : loads0;
                if (n > 0) ok = bar_wait(&C.qempty[q], (n - 1) & 1u, ctl);
                if (!ok) break;
                if (q) ++loads1;
                else ++loads0;
                mbar_expect_tx(&C.qfull[q], 2 * qbytes);
#pragma unroll 1
                for (int s = 0; s < 2; ++s)
                  tma_load_3d(smem_u32(q_s) + (uint32_t)(2 * q + s) * lay.slab_q, &P.qmap, 64 * s, blk.h * P.group,
                              (int)(blk.row0 + q * P.tpt), &C.qfull[q], pol);
              }
            }
          }
        }
        ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
      }
      // The loads land before the CTA exits, also if another warp gives up after this
      // point. st and ph are the next load's, so the last load of a stage in front of st
      // was ph's, of one at or behind it the round's before.
      if (lane == 0) {
        if (loads0 > 0) drain(&C.qfull[0], (loads0 - 1) & 1u, ctl);
        if (loads1 > 0) drain(&C.qfull[1], (loads1 - 1) & 1u, ctl);
#pragma unroll 1
        for (int s = 0; s < S && s < g; ++s) drain(&C.full[s], s < st ? ph : ph ^ 1u, ctl);
      }
      __syncwarp();
    } else if (warp == kIssuer) {
      // ---------------------------------------------------------- MMA issuer
      // The tensor core takes few MMAs ahead, so whatever lies between two of them
      // shows up as idle time: the waits on K and V stages sit in the middle of a
      // product whose MMAs are queued, and only the waits for probabilities stand
      // between two products.
      const uint32_t tmem = start();
      constexpr uint32_t id_pv = idesc_bf16(128, 128) | kIdescBMn;
      const uint32_t qd = desc_k(smem_u32(q_s)), kd = desc_k(smem_u32(ring)), vd = desc_mn(smem_u32(ring));
      const uint32_t slab_step = lay.slab_q >> 4;  // descriptors count 16 bytes
      const uint32_t el = elect_one();
      // the two 64-column halves of a logit product
      auto issue_qk = [&](int q, int st, int half, uint32_t id_qk) {
        const uint32_t d = tmem + (uint32_t)q * 256;
        const uint32_t a = qd + (uint32_t)(2 * q + half) * slab_step;
        const uint32_t b = kd + (uint32_t)st * (kTileBytes >> 4) + (uint32_t)half * (kSlabBytes >> 4);
        umma_ss<0, 0>(d, a, b, id_qk, (uint32_t)half, el);
        umma_ss<2, 2>(d, a, b, id_qk, 1u, el);
        umma_ss<4, 4>(d, a, b, id_qk, 1u, el);
        umma_ss<6, 6>(d, a, b, id_qk, 1u, el);
      };
      // 32 keys of a PV product
      auto issue_pv = [&](int q, int st, int quarter, uint32_t acc) {
        const uint32_t s = tmem + (uint32_t)q * 256, p = s + (uint32_t)quarter * 16;
        const uint32_t b = vd + (uint32_t)st * (kTileBytes >> 4) + (uint32_t)quarter * 256;
        umma_ts<0, 0>(s + 128, p, b, id_pv, acc, el);
        umma_ts<8, 128>(s + 128, p, b, id_pv, 1u, el);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kFull, bar_wait(bar, parity, ctl));
      };
      auto step = [&](int& st, uint32_t& ph) {
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
      };
      // per row tile, one bit each: parity of the queries' loads, of the key tiles and of
      // the row blocks done, and whether there was one
      uint32_t loads = 0, tiles = 0, outs = 0, any = 0;
      int st = 0;  // next stage of the ring
      uint32_t ph = 0;
      bool ok = true, issued = false;
      int nt = 0, nq = 0, sv = 0;  // the present block; stage of V_j, which K_{j+1} follows
      int last0 = 4, last1 = 4;    // quarters of its last tile
      auto quarters = [&](int q) { return q ? last1 : last0; };
      Work w;
      // A turn: the last products of one block and the first of the next, row tile by row
      // tile, so that one tile's softmax has its logits while the other's is still at work.
      for (;;) {
        const bool more = next_work(w) && w.nt > 0;
        const int nq1 = !more ? 0 : NQ == 1 || w.blk.cnt <= P.tpt ? 1 : 2;
#pragma unroll 1
        for (int q = 0; q < NQ && ok; ++q) {
          if (q < nq) {
            const uint32_t par = ((tiles >> q) ^ (uint32_t)(nt - 1)) & 1u;
            ok = wait(&C.pfull[q][0], par);
            if (!ok) break;
            tc_fence_after();
            issue_pv(q, sv, 0, nt > 1 ? 1u : 0u);
            if (quarters(q) > 1) issue_pv(q, sv, 1, 1u);
            ok = wait(&C.pfull[q][1], par);
            if (!ok) break;
            tc_fence_after();
            if (quarters(q) > 2) issue_pv(q, sv, 2, 1u);
            if (quarters(q) > 3) issue_pv(q, sv, 3, 1u);
            umma_commit_if(&C.ofull[q], el);
          }
          if (q < nq1) {
            ok = (q > 0 || wait(&C.full[st], ph)) && wait(&C.qfull[q], (loads >> q) & 1u);
            if (!ok) break;
            tc_fence_after();
            issued = true;
            const uint32_t id = idesc_bf16(128, w.nt == 1 ? 32 * last_quarters<kTree>(w.blk, q, P.tpt, w.t_lo) : 128);
            issue_qk(q, st, 0, id);
            issue_qk(q, st, 1, id);
            umma_commit_if(&C.sfull[q], el);
            if (w.nt == 1) umma_commit_if(&C.qempty[q], el);
          }
        }
        if (!ok) break;
        if (nq > 0) umma_commit_if(&C.empty[sv], el);
        if (nt & 1) tiles ^= nq == 2 ? 3u : 1u;
        if (!more) break;
        umma_commit_if(&C.empty[st], el);
        nt = w.nt;
        nq = nq1;
        last0 = last_quarters<kTree>(w.blk, 0, P.tpt, w.t_lo + nt - 1);
        last1 = last_quarters<kTree>(w.blk, 1, P.tpt, w.t_lo + nt - 1);
        loads ^= nq == 2 ? 3u : 1u;
        step(st, ph);
        sv = st;
        ok = wait(&C.full[sv], ph);
#pragma unroll 1
        for (int q = 0; q < nq; ++q)  // the last block's O has been read
          if ((any >> q) & 1u) ok = ok && wait(&C.ofree[q], ((outs >> q) & 1u) ^ 1u);
        any |= nq == 2 ? 3u : 1u;
        outs ^= nq == 2 ? 3u : 1u;
#pragma unroll 1
        for (int j = 0; j + 1 < nt && ok; ++j) {
          step(st, ph);
          const int sk = st;  // stages of K_{j+1} and V_{j+1}
          const uint32_t pk = ph;
          step(st, ph);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (q >= nq || !ok) break;
            const uint32_t par = ((tiles >> q) ^ (uint32_t)j) & 1u;
            ok = wait(&C.pfull[q][0], par);
            if (!ok) break;
            tc_fence_after();
            issue_pv(q, sv, 0, j > 0 ? 1u : 0u);
            issue_pv(q, sv, 1, 1u);
            ok = wait(&C.pfull[q][1], par);
            if (!ok) break;
            tc_fence_after();
            issue_pv(q, sv, 2, 1u);
            if (q == 0) ok = wait(&C.full[sk], pk);
            issue_pv(q, sv, 3, 1u);
            if (q == nq - 1) umma_commit_if(&C.empty[sv], el);
            if (!ok) break;
            const uint32_t id = idesc_bf16(128, j + 2 == nt ? 32 * quarters(q) : 128);
            issue_qk(q, sk, 0, id);
            if (q == nq - 1) ok = wait(&C.full[st], ph);
            issue_qk(q, sk, 1, id);
            umma_commit_if(&C.sfull[q], el);
            if (j + 2 == nt) umma_commit_if(&C.qempty[q], el);
          }
          // Only a stage whose products are issued is given back: without its K the loop
          // above has left before them, and a second copy would join the one under way.
          if (!ok) break;
          umma_commit_if(&C.empty[sk], el);
          sv = st;
        }
        if (!ok) break;
        step(st, ph);
        // the last tile: V rows behind the sequence may hold NaN, and 0 * NaN is NaN
        const int live = w.blk.v_len - (w.t_lo + nt - 1) * kTileKeys;
        if (live < kTileKeys) {
          uint4* rows = reinterpret_cast<uint4*>(ring + (size_t)sv * kTileBytes);
#pragma unroll 1
          for (int i = live * 8 + lane; i < quarters(nq - 1) * 256; i += 32) {
            rows[i] = make_uint4(0, 0, 0, 0);
            rows[kSlabBytes / 16 + i] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
      if (issued) {
        // the MMAs, and the arrivals of the commits before this one, before the TMEM is
        // freed and the CTA exits: after an abort nobody has waited for them
        umma_commit_if(&C.done, el);
        drain(&C.done, 0u, ctl);
      }
      __syncwarp();
    } else {
      start();
    }
    if constexpr (kCluster) {  // the join's two barriers, see below
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else if (kOut && warp >= kSoftmaxWarps) {
    // ------------------------------------------------------------ output
    regs_dec<104>();
    const uint32_t tmem = start();
    const int wq = warp & 3, row = wq * 32 + lane;
    const int tok_q = row / P.group, g_q = row - tok_q * P.group;  // token in its tile, query head in its group
    uint32_t outs = 0, stats = 0;  // parities, one bit per tile
    int uses = 0;
    bool ok = true;
    Work w;
    while (wq < wpt && ok && next_work(w)) {
      const Block& blk = w.blk;
      const int64_t orow0 = blk.row0 * P.heads + (int64_t)blk.h * P.group;
      const int nq = blk.cnt <= P.tpt ? 1 : 2;
#pragma unroll 1
      for (int q = 0; q < nq; ++q) {
        const int rows = min(blk.cnt - q * P.tpt, P.tpt) * P.group;
        const uint32_t t_o = tmem + ((uint32_t)wq << 21) + (uint32_t)q * 256 + 128;
        ok = __all_sync(kFull, bar_wait(&C.rfull[q], (stats >> q) & 1u, ctl));
        stats ^= 1u << q;
        if (ok && w.nt > 0) {
          ok = __all_sync(kFull, bar_wait(&C.ofull[q], (outs >> q) & 1u, ctl));
          // a cluster's partial results go where the other tile's V may still be read
          if (kCluster && ok && nq == 2)
            ok = __all_sync(kFull, bar_wait(&C.ofull[q ^ 1], (outs >> q) & 1u, ctl));
          outs ^= 1u << q;
          tc_fence_after();
        }
        if (!ok) break;
        const float2 x = stats_s[q * 128 + row];
        const int tok = q * P.tpt + tok_q;
        if constexpr (kCluster) {
          write_partial(t_o, q, row, x.x, x.y, w.nt > 0 && wq * 32 < rows);
          continue;
        }
        // A full tile leaves as two tensor stores: written by the warps themselves, its
        // 32 KB hold up the softmax warps' exponentials in the same queue. A ragged one
        // may not write behind its last token.
        const bool whole = rows == P.group * P.tpt;
        const float inv = row_scale(x.y);
        const int mine = row < rows ? tok * P.heads + g_q : -1;
        uint64_t check[2] = {0ull, 0ull};
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (uses > 0) {
            if (wq == 0 && lane == 0) {
              bulk_wait_read<1>();  // the store before the last one is done reading this buffer
              mbar_arrive(&C.unstaged[half]);
            }
            ok = __all_sync(kFull, bar_wait(&C.unstaged[half], (uint32_t)((uses - 1) & 1), ctl));
            if (!ok) break;
          }
          uint4* slab = reinterpret_cast<uint4*>(smem + lay.out + (uint32_t)half * kSlabBytes) + wq * (kWarpOut / 16);
          stage_half(t_o + (uint32_t)half * 64, slab, pack2(inv, inv), check, half ? &C.ofree[q] : nullptr);
          if (whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (!whole && wq * 32 < rows) write_half(P, slab, orow0, mine, half);
          if (lane == 0) mbar_arrive(&C.staged[half]);
          if (wq == 0) {
            ok = __all_sync(kFull, bar_wait(&C.staged[half], (uint32_t)(uses & 1), ctl));
            if (!ok) break;
            if (lane == 0) {
              if (whole)
                tma_store_3d(&P.omap, smem_u32(smem + lay.out) + (uint32_t)half * kSlabBytes, 64 * half,
                             blk.h * P.group, (int)(blk.row0 + q * P.tpt));
              bulk_commit();
            }
          }
        }
        if (!ok) break;
        ++uses;
        if (mine >= 0) write_lse(P, orow0 + mine, x.x, x.y, check);
      }
    }
    if (wq == 0 && lane == 0) bulk_wait_all();
    __syncwarp();
    if constexpr (kCluster) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<NQ == 1 ? 208 : 176>();
    const uint32_t tmem = start();
    const int q = NQ == 1 ? 0 : warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 TMEM lanes
    const uint32_t t_s = tl + (uint32_t)q * 256, t_o = t_s + 128;
    const int tok_q = row / P.group, g_q = row - tok_q * P.group;  // token in its tile, query head in its group
    const uint64_t scale2 = pack2(P.scale_log2, P.scale_log2);
    int tiles = 0, outs = 0;
    bool ok = true;
    Work w;
    w.blk.cnt = 0;
    w.nt = 0;
    int rows = 0;  // of this row tile in the present block
    // warps that never have a row take no part
    while ((warp & 3) < wpt && ok && next_work(w)) {
      const Block& blk = w.blk;
      const int nt = w.nt;
      rows = min(blk.cnt - q * P.tpt, P.tpt) * P.group;
      if (rows <= 0) continue;
      const bool active = (warp & 3) * 32 < rows;
      const bool valid = row < rows;
      const int tok = q * P.tpt + (valid ? tok_q : 0);
      // slots [0, lim) are visible, and the tree's slots L + i whose bit is set
      int lim = min(blk.past + tok + 1, blk.kv_len);
      // tiles that end at or below every row's bound need no mask
      int lim_min = min(blk.past + q * P.tpt + 1, blk.kv_len);
      uint64_t bits = 0;
      if constexpr (kTree) {
        if (P.mask) {
          lim = lim_min = blk.L;
          if (valid) bits = (uint64_t)P.mask[blk.row0 + tok];
          if (blk.nodes < 64) bits &= (1ull << blk.nodes) - 1ull;
        }
      }
      const int last = last_quarters<kTree>(blk, q, P.tpt, w.t_lo + nt - 1);
      float m = kNegInf, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        ok = __all_sync(kFull, bar_wait(&C.sfull[q], (uint32_t)(tiles & 1), ctl));
        ++tiles;
        if (!ok) break;
        if (!active) {
          if (lane == 0) {
            mbar_arrive(&C.pfull[q][0]);
            mbar_arrive(&C.pfull[q][1]);
          }
          continue;
        }
        tc_fence_after();
        float v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + (uint32_t)c * 32, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) pin(v[c]);
        const int base = (w.t_lo + j) * kTileKeys;
        if (base + kTileKeys > lim_min) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int lo = base + 32 * c;
            const int n = min(max(lim - lo, 0), 32);
            uint32_t see = n >= 32 ? ~0u : (1u << n) - 1u;
            if constexpr (kTree) {
              const int sh = lo - blk.L;
              if (sh >= 0) see |= sh < 64 ? (uint32_t)(bits >> sh) : 0u;
              else if (sh > -32) see |= (uint32_t)(bits << -sh);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c][i] = (see >> i) & 1u ? v[c][i] : kNegInf;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = v[c][0];
#pragma unroll
          for (int i = 1; i < 31; i += 2) mx[c] = fmaxf(fmaxf(mx[c], v[c][i]), v[c][i + 1]);
          mx[c] = fmaxf(mx[c], v[c][31]);
        }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.scale_log2;
        // Each row by its own logits alone, or its last bits would vary with its
        // neighbours', and with what lies in the rows behind the last one.
        const bool raise = valid && (mt > m + kRescale || (m == kNegInf && mt > kNegInf));
        if (j == 0) {
          m = mt;
        } else if (__any_sync(kFull, raise)) {
          const float m_new = raise ? mt : m;
          const float f = !raise ? 1.f : m == kNegInf ? 0.f : fast_exp2(m - m_new);
          l *= f;
          m = m_new;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[16];
            tmem_ld16(t_o + (uint32_t)c * 16, o);
            tmem_wait_ld();
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              asm volatile("" : "+f"(o[i]));  // as pin()
              r[i] = __float_as_uint(o[i] * f);
            }
            tmem_st16(t_o + (uint32_t)c * 16, r);
          }
        }
        const float off = m == kNegInf ? 0.f : -m;
        const uint64_t off2 = pack2(off, off);
        uint64_t sum[2] = {0ull, 0ull};
        auto exps = [&](int c, uint32_t* p) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            unpack2(fma2(pack2(v[c][2 * i], v[c][2 * i + 1]), scale2, off2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[i & 1] = add2(sum[i & 1], pack2(a, b));
            p[i] = pack_bf16(a, b);
          }
        };
        auto hand_over = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&C.pfull[q][half]);
        };
        uint32_t p[4][16];
        exps(0, p[0]);
        tmem_st16(t_s, p[0]);
        exps(1, p[1]);
        tmem_st16(t_s + 16, p[1]);
        if (j + 1 < nt || last > 2) {
          exps(2, p[2]);
          hand_over(0);
          tmem_st16(t_s + 32, p[2]);
          exps(3, p[3]);
          tmem_st16(t_s + 48, p[3]);
        } else {
          hand_over(0);
        }
        hand_over(1);
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      if (!kCluster && l == 0.f && (lim > 0 || bits != 0)) l = kNaN;  // only logits of -inf
      if (kOut) {
        // the output warps have read the last block's statistics
        if (outs > 0) ok = __all_sync(kFull, bar_wait(&C.ofree[q], (uint32_t)((outs - 1) & 1), ctl));
        ++outs;
        if (!ok) break;
        stats_s[q * 128 + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.rfull[q]);
        continue;
      }
      if (nt > 0) {
        ok = __all_sync(kFull, bar_wait(&C.ofull[q], (uint32_t)(outs & 1), ctl));
        ++outs;
        if (!ok) break;
        tc_fence_after();
      }
      if constexpr (kCluster) {
        write_partial(t_o, q, row, m, l, nt > 0 && active);
      } else if (active) {
        // rows go out through shared memory: 8 lanes write 128 bytes of a row at a time
        // instead of every lane 16 bytes of its own row
        uint4* slab = reinterpret_cast<uint4*>(smem + lay.out) + (warp & 3) * (kWarpOut / 16);
        const int64_t orow0 = blk.row0 * P.heads + (int64_t)blk.h * P.group;
        const int mine = valid ? tok * P.heads + g_q : -1;
        const float inv = row_scale(l);
        uint64_t check[2] = {0ull, 0ull};
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          stage_half(t_o + (uint32_t)half * 64, slab, pack2(inv, inv), check, half ? &C.ofree[q] : nullptr);
          __syncwarp();
          write_half(P, slab, orow0, mine, half);
          __syncwarp();
        }
        if (valid) write_lse(P, orow0 + mine, m, l, check);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.ofree[q]);
      }
    }
    if constexpr (kCluster) {
      // ---------------------------------------------------------- join
      // Rank r joins rows r, r + splits, ...; a warp takes 32 / splits of them at a time,
      // so that all their statistics come in one load per lane (lane = row, share). The
      // loops over rows stay loops: in a short call, code is as far away as data.
      __syncwarp();
      cluster_sync();
      const Block blk = C.work[0].blk;  // every CTA of the cluster had the same block
      if (!ctl->abort && blk.cnt > 0) {
        const int nq = NQ == 1 || blk.cnt <= P.tpt ? 1 : 2;
        const uint32_t part = smem_u32(ring), mls = smem_u32(ml);
        const int64_t orow0 = blk.row0 * P.heads + (int64_t)blk.h * P.group;
        const int sh = 31 - __clz(splits), share = lane & (splits - 1);  // splits: a power of two
#pragma unroll 1
        for (int t = 0; t < nq; ++t) {
          const int n = min(blk.cnt - t * P.tpt, P.tpt) * P.group;
#pragma unroll 1
          for (int k = warp; rank + k * splits < n; k += kSoftmaxWarps << (5 - sh)) {
            auto row_at = [&](int i) { return rank + (k + i * kSoftmaxWarps) * splits; };  // i-th of the warp's rows
            auto out_row = [&](int r) { return orow0 + (int64_t)(t * P.tpt + r / P.group) * P.heads + r % P.group; };
            const int r = row_at(lane >> sh);
            float2 x = make_float2(kNegInf, 0.f);
            if (r < n) x = ld_cluster2(map_rank(mls + (uint32_t)(t * 128 + r) * 8, (uint32_t)share));
            float M = x.x;
#pragma unroll 1
            for (int off = splits >> 1; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
            // a share without a visible key has no part in the sums (its sum is 0, or NaN)
            float wt = x.x == kNegInf ? x.y : fast_exp2(x.x - M);
            float l = wt * x.y;
#pragma unroll 1
            for (int off = splits >> 1; off > 0; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
            wt = wt == 0.f ? 0.f : wt * row_scale(l);
            if (r < n && l == 0.f && sees_any(P, blk, t * P.tpt + r / P.group)) wt = l = kNaN;  // only logits of -inf
            if (r < n && share == 0) {
              const float lse = row_lse(M, l);
              const int64_t orow = out_row(r);
              if (P.lse && BKV_IN_RANGE(orow >= 0 && orow < (int64_t)P.total * P.heads, P.status)) P.lse[orow] = lse;
              if (!(lse < __builtin_huge_valf())) latch(P.status, BKV_ERR_NONFINITE);
            }
#pragma unroll 1
            for (int i = 0; i < 32 >> sh && row_at(i) < n; ++i) {
              const int rr = row_at(i);
              const uint32_t at = part + ((uint32_t)(t * 128 + rr) * 32 + (uint32_t)(lane ^ (rr & 31))) * 16;
              float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
              for (int c0 = 0; c0 < splits; c0 += 8) {
                float4 y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  if (c0 + c < splits) y[c] = ld_cluster4(map_rank(at, (uint32_t)(c0 + c)));
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float wc = __shfl_sync(kFull, wt, (i << sh) + ((c0 + c) & (splits - 1)));
                  if (c0 + c < splits && wc != 0.f) {  // a share without weight may not have written its O
                    o.x = fmaf(wc, y[c].x, o.x);
                    o.y = fmaf(wc, y[c].y, o.y);
                    o.z = fmaf(wc, y[c].z, o.z);
                    o.w = fmaf(wc, y[c].w, o.w);
                  }
                }
              }
              const int64_t orow = out_row(rr);
              if (!BKV_IN_RANGE(orow >= 0 && orow < (int64_t)P.total * P.heads, P.status)) continue;
              reinterpret_cast<uint2*>(P.out)[orow * 32 + lane] = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
              const float check = (o.x * 0.f + o.y * 0.f) + (o.z * 0.f + o.w * 0.f);
              if (check != 0.f) latch(P.status, BKV_ERR_NONFINITE);
            }
          }
        }
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while another still reads its partial results
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(ctl->tmem_base, kCols);
  if (tid == 0 && ctl->abort) latch(P.status, BKV_ERR_TIMEOUT);
}

}  // namespace

// K/V stages that fit. Two CTAs share an SM's 228 KB; fewer stages than the most
// would fit three there, and three ask for more TMEM columns (256 each) than it has.
int attend_stages(int nq, int group, int tpt) {
  const uint32_t room = attend_ctas_per_sm(nq, group * tpt) == 2 ? 228 * 1024 / 2 - 1024 : 227 * 1024;
  int n = kMaxStages;
  while (n > 0 && attend_smem(nq, group, tpt, n).total > room) --n;
  return n;
}

bool encode_attend_maps(AttendParams& p, const void* q, int64_t q_stride, const void* K, const void* V) {
  // the driver's encoder, looked up once per process (thread-safe static initialisation)
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult qres;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qres) !=
            cudaSuccess ||
        qres != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  auto one = [&](CUtensorMap* map, const void* base, cuuint64_t d1, cuuint64_t s1, cuuint64_t d2, cuuint64_t s2,
                 cuuint32_t b1, cuuint32_t b2) {
    const cuuint64_t dims[3] = {(cuuint64_t)kD, d1, d2};
    const cuuint64_t strides[2] = {s1, s2};
    const cuuint32_t box[3] = {64, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t row = (cuuint64_t)kD * 2;
  const cuuint64_t heads = (cuuint64_t)p.batch * p.kv_heads, plane = (cuuint64_t)p.max_cache * row;
  return one(&p.qmap, q, (cuuint64_t)p.heads, row, (cuuint64_t)p.total, (cuuint64_t)q_stride * 2,
             (cuuint32_t)p.group, (cuuint32_t)p.tpt) &&
         one(&p.omap, p.out, (cuuint64_t)p.heads, row, (cuuint64_t)p.total, (cuuint64_t)p.heads * row,
             (cuuint32_t)p.group, (cuuint32_t)p.tpt) &&
         one(&p.kmap, K, (cuuint64_t)p.max_cache, row, heads, plane, (cuuint32_t)kTileKeys, 1) &&
         one(&p.vmap, V, (cuuint64_t)p.max_cache, row, heads, plane, (cuuint32_t)kTileKeys, 1);
}

namespace {

template <int NQ, bool kTree, bool kCluster>
cudaError_t launch_instance(const AttendParams& p, int splits, int64_t items, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const auto fn = attend_kernel<NQ, kTree, kCluster>;
  static std::atomic<unsigned long long> configured{0};  // once per device (one bit each)
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess && kCluster) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  if (p.stages < 2) return cudaErrorInvalidConfiguration;  // V_j and K_{j+1}
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * splits));
  cfg.blockDim = dim3((unsigned)(NQ * 128 + (output_warps(NQ) ? 256 : 128)));
  cfg.dynamicSmemBytes = attend_smem(NQ, p.group, p.tpt, p.stages).total;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  if (kCluster) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = (unsigned)splits;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  // one sequence decoding 12.3 -> 9.6 us, 64 trees of 16 nodes 56.5 -> 54.1, prompt
  // chunks of 500 tokens 74.2 -> 72.6; long calls as without it
  at[cfg.numAttrs++] = dependent_launch();
  return cudaLaunchKernelEx(&cfg, fn, p, splits);
}

template <int NQ, bool kTree>
cudaError_t launch_tiles(const AttendParams& p, int splits, int64_t items, cudaStream_t s) {
  return splits > 1 ? launch_instance<NQ, kTree, true>(p, splits, items, s)
                    : launch_instance<NQ, kTree, false>(p, 1, items, s);
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, int nq, int splits, int64_t items, cudaStream_t s) {
  // prompts take two tiles for many row blocks only, whose keys are never split
  if (p.cu) return nq == 1 ? launch_tiles<1, false>(p, splits, items, s) : launch_instance<2, false, false>(p, 1, items, s);
  return nq == 1 ? launch_tiles<1, true>(p, splits, items, s) : launch_tiles<2, true>(p, splits, items, s);
}

}  // namespace bkv

#ifdef BKV_CHECKED
// Tests only: the bound of the attention kernels' waits on the current device, in clocks.
extern "C" bkv_status bkv_checked_wait_cycles(uint32_t cycles) {
  return cudaMemcpyToSymbol(bkv::wait_cycles, &cycles, sizeof(cycles)) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}
#endif
