// Host side of the model-side calls over the caches (bkv_store_kv,
// bkv_attend_prompt, bkv_attend_tree, bkv_commit_tree): argument checks and
// launches. No handle, no workspace, no device allocation.
#include <cmath>

#include "attend/attend.cuh"
#include "attend/host.cuh"

namespace {

using namespace bkv::host;

// CTAs per row block: the keys are split over a cluster while all clusters run at
// once. GB300's GPCs hold 7 clusters of 16, 15 of 8, 36 of 4 and 76 of 2 at one CTA
// per SM, twice that at two; one cluster too many waits for a whole other one (one
// node of 16 KV heads over 2063 slots: 14.9 us in clusters of 16, 10.0 in clusters of
// 8). Two CTAs per SM take 32 clusters of 8 well (11.5 us, 12.2 in clusters of 4).
int splits_for(int64_t items, int ctas_per_sm, int max_cache) {
  const int tiles = (max_cache + 127) / 128;
  const int64_t most[4] = {7 * ctas_per_sm, ctas_per_sm == 2 ? 32 : 15, 36 * ctas_per_sm, 76 * ctas_per_sm};
  for (int i = 0; i < 4; ++i)
    if (items <= most[i] && (16 >> i) <= tiles) return 16 >> i;
  return 1;
}

}  // namespace

extern "C" {

bkv_status bkv_store_kv(const bkv_config* cfg, const void* q_pre, int64_t q_stride, const void* k_pre,
                        int64_t k_stride, const void* v, int64_t v_stride, int32_t total, const int32_t* cu_seqlens,
                        const int32_t* first_slot, const int32_t* first_pos, const int32_t* depth, void* q_rot,
                        void* K, void* V, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_store_kv");
  const bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  if (total < 0 || !cu_seqlens || !first_slot || !first_pos || (total > 0 && !q_rot) || !K || !V || !aligned(cu_seqlens, 4) ||
      !aligned(first_slot, 4) || !aligned(first_pos, 4) || !aligned(depth, 4) || !aligned(q_rot, 16) ||
      !aligned(K, 16) || !aligned(V, 16) || !aligned(status, 4))
    return BKV_ERR_INVALID_ARG;
  if (!strided_ok(q_pre, q_stride, c.heads, c.d, total) || !strided_ok(k_pre, k_stride, c.kv_heads, c.d, total) ||
      !strided_ok(v, v_stride, c.kv_heads, c.d, total))
    return BKV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  if (total == 0) return BKV_OK;
  bkv::StoreParams p{};
  p.q = static_cast<const uint4*>(q_pre);
  p.k = static_cast<const uint4*>(k_pre);
  p.v = static_cast<const uint4*>(v);
  p.q_stride = q_stride / 8;
  p.k_stride = k_stride / 8;
  p.v_stride = v_stride / 8;
  p.cu = cu_seqlens;
  p.first = first_slot;
  p.pos = first_pos;
  p.depth = depth;
  p.q_rot = static_cast<uint4*>(q_rot);
  p.K = static_cast<uint4*>(K);
  p.V = static_cast<uint4*>(V);
  p.status = status;
  p.batch = c.batch;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.max_cache = c.max_cache;
  p.total = total;
  // theta^(-2i/d) as theta^(-16a/d) theta^(-2b/d), i = 8a + b: 16 powers, one more rounding
  double coarse[8], fine[8];
  for (int i = 0; i < 8; ++i) {
    coarse[i] = std::pow(c.rope_theta, -16.0 * i / (double)c.d) * 0.15915494309189535;  // 1 / (2 pi)
    fine[i] = std::pow(c.rope_theta, -2.0 * i / (double)c.d);
  }
  for (int i = 0; i < bkv::kRopePairs; ++i) {
    double turns = coarse[i / 8] * fine[i % 8];
    turns -= std::floor(turns);
    p.turns[i] = turns < 1.0 ? (uint64_t)std::ldexp(turns, 64) : 0ull;
  }
  return bkv::launch_store(p, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_attend_prompt(const bkv_config* cfg, const void* q, int64_t q_stride, const void* K, const void* V,
                             const int32_t* cu_seqlens, const int32_t* first_slot, int32_t total, void* out,
                             float* lse, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_attend_prompt");
  const bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  if (total < 0 || !K || !V || !cu_seqlens || !first_slot || (total > 0 && !out) || !aligned(K, 16) || !aligned(V, 16) ||
      !aligned(cu_seqlens, 4) || !aligned(first_slot, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(status, 4) || !strided_ok(q, q_stride, c.heads, c.d, total))
    return BKV_ERR_INVALID_ARG;
  bkv::AttendParams p{};
  p.cu = cu_seqlens;
  p.first = first_slot;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = status;
  p.batch = c.batch;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = c.heads / c.kv_heads;
  p.max_cache = c.max_cache;
  p.total = total;
  p.tpt = 128 / p.group < total ? 128 / p.group : (total > 0 ? total : 1);
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.d));
  // row blocks of nq tiles: at most total / (nq tpt) full ones and one ragged one per sequence
  auto items_of = [&](int nq) { return ((int64_t)total / (nq * p.tpt) + c.batch) * c.kv_heads; };
  const int nq = items_of(2) > bkv::kSms / 2 && p.tpt < total ? 2 : 1;
  const int64_t items = items_of(nq);
  if (items > 0x7FFFFFFF / 16) return BKV_ERR_UNSUPPORTED;
  p.stages = bkv::attend_stages(nq, p.group, p.tpt);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (total > 0 && !bkv::encode_attend_maps(p, q, q_stride, K, V)) return BKV_ERR_CUDA;
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  if (total == 0) return BKV_OK;
  // a few tokens behind a long context leave most of the GPU idle unless their keys are
  // split; two tiles per CTA are only taken by row blocks enough for every SM
  const int splits = nq == 2 ? 1 : splits_for(items, bkv::attend_ctas_per_sm(nq, p.group * p.tpt), c.max_cache);
  return bkv::launch_attend(p, nq, splits, items, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_attend_tree(const bkv_config* cfg, const void* q, int64_t q_stride, const void* K, const void* V,
                           const int32_t* cache_lens, int32_t n, const int64_t* mask, const int32_t* nodes, void* out,
                           float* lse, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_attend_tree");
  const bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  if (n < 1 || !K || !V || !cache_lens || !out || !aligned(K, 16) || !aligned(V, 16) || !aligned(cache_lens, 4) ||
      !aligned(mask, 8) || !aligned(nodes, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(status, 4) ||
      !strided_ok(q, q_stride, c.heads, c.d, 1))
    return BKV_ERR_INVALID_ARG;
  if (n > bkv::kMaxNodes || (int64_t)c.batch * n > 0x7FFFFFFF) return BKV_ERR_UNSUPPORTED;
  bkv::AttendParams p{};
  p.first = cache_lens;
  p.nodes = nodes;
  p.mask = mask;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = status;
  p.batch = c.batch;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = c.heads / c.kv_heads;
  p.max_cache = c.max_cache;
  p.total = c.batch * n;
  p.n = n;
  p.tpt = 128 / p.group < n ? 128 / p.group : n;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.d));
  const int nq = p.tpt < n ? 2 : 1;
  p.qblocks = (n + nq * p.tpt - 1) / (nq * p.tpt);
  const int64_t items = (int64_t)c.batch * c.kv_heads * p.qblocks;
  if (items > 0x7FFFFFFF / 16) return BKV_ERR_UNSUPPORTED;
  const int splits = splits_for(items, bkv::attend_ctas_per_sm(nq, p.group * p.tpt), c.max_cache);
  p.stages = bkv::attend_stages(nq, p.group, p.tpt);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (!bkv::encode_attend_maps(p, q, q_stride, K, V)) return BKV_ERR_CUDA;
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  return bkv::launch_attend(p, nq, splits, items, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_commit_tree(const bkv_config* cfg, void* const* K, void* const* V, const int32_t* cache_lens,
                           const int32_t* path, const int32_t* count, int32_t n, uint32_t* status,
                           void* cuda_stream) {
  NvtxRange nvtx("bkv_commit_tree");
  const bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  if (n < 1 || !K || !V || !cache_lens || !path || !count || !aligned(cache_lens, 4) || !aligned(path, 4) ||
      !aligned(count, 4) || !aligned(status, 4))
    return BKV_ERR_INVALID_ARG;
  for (int l = 0; l < c.layers; ++l)
    if (!K[l] || !V[l] || !aligned(K[l], 16) || !aligned(V[l], 16)) return BKV_ERR_INVALID_ARG;
  if (n > bkv::kMaxNodes) return BKV_ERR_UNSUPPORTED;
  bkv::CommitParams p{};
  for (int l = 0; l < c.layers; ++l) {
    p.K[l] = static_cast<uint4*>(K[l]);
    p.V[l] = static_cast<uint4*>(V[l]);
  }
  p.lens = cache_lens;
  p.path = path;
  p.count = count;
  p.status = status;
  p.batch = c.batch;
  p.kv_heads = c.kv_heads;
  p.max_cache = c.max_cache;
  p.n = n;
  p.layers = c.layers;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  return bkv::launch_commit(p, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

}  // extern "C"
