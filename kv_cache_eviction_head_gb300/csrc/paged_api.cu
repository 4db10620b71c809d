// Host side of the calls over paged caches (bkv_store_paged, bkv_attend_paged,
// bkv_weigh_prompt, bkv_evict_weight): argument checks and launches. No handle, no
// device allocation.
#include <algorithm>
#include <cmath>

#include "attend/host.cuh"
#include "paged/paged.cuh"

namespace {

using namespace bkv::host;

constexpr double kPi = 3.14159265358979323846;

// The caller's pages (NULL: the dense caches of the config) as the kernels take them.
bkv_status take_pages(const bkv_config& c, const bkv_pages* pages, bkv::Pages& out) {
  if (!pages) {
    out.table = nullptr;
    out.pages = c.batch;
    out.page_size = c.max_cache;
    out.per_seq = 1;
  } else {
    if (pages->pages < 1 || pages->page_size < 1 || pages->per_seq < 1 || !pages->table || !aligned(pages->table, 4))
      return BKV_ERR_INVALID_ARG;
    if (pages->page_size % bkv::kTileSlots) return BKV_ERR_UNSUPPORTED;
    out.table = pages->table;
    out.pages = pages->pages;
    out.page_size = pages->page_size;
    out.per_seq = pages->per_seq;
  }
  const int64_t cap = (int64_t)out.page_size * out.per_seq;
  if (cap > 0x7FFFFFFF - 4096) return BKV_ERR_UNSUPPORTED;
  out.cap = (int)cap;
  bkv::set_division(out);
  return BKV_OK;
}

// Tiles of 16 slots that the sequences' slots can take, for each KV head, when no page
// is in two tables: every sequence may end inside a tile.
int64_t most_tiles(const bkv_config& c, const bkv::Pages& p) {
  const int64_t by_table = (int64_t)c.batch * ((p.cap + bkv::kTileSlots - 1) / bkv::kTileSlots);
  const int64_t by_pool = (int64_t)p.pages * ((p.page_size + bkv::kTileSlots - 1) / bkv::kTileSlots);
  return std::min(by_table, by_pool);
}

struct Workspace {
  size_t part_ml, part_o, lse2, seq, logits, bytes;
};
Workspace lay_out(const bkv_config& c, const bkv::Pages& p, bool weighed) {
  const size_t g = (size_t)(c.heads / c.kv_heads), pieces = 2 * (size_t)bkv::kAttendShares;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w{};
  w.part_ml = 0;
  w.part_o = up(pieces * 16 * sizeof(float2));
  w.lse2 = w.part_o + up(pieces * (g > 8 ? 16 : 8) * bkv::kD * sizeof(float));
  w.seq = w.lse2 + up((size_t)c.batch * c.heads * sizeof(float));
  w.logits = w.seq + up(((size_t)c.batch + 1) * sizeof(int2));
  w.bytes = w.logits + (weighed ? up((size_t)most_tiles(c, p) * c.heads * bkv::kTileSlots * sizeof(float)) : 0);
  return w;
}

bool decay_ok(float d) { return d >= 0.f && d <= 1.f; }

}  // namespace

extern "C" {

bkv_status bkv_make_rope(bkv_rope* out, double theta, int32_t rotary_dim, int32_t interleaved, int32_t scaling,
                         double factor, double original_len) {
  if (!out || !(theta > 0.0) || !std::isfinite(theta) || rotary_dim < 0 || (interleaved != 0 && interleaved != 1) ||
      scaling < BKV_ROPE_NONE || scaling > BKV_ROPE_YARN)
    return BKV_ERR_INVALID_ARG;
  if (scaling != BKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return BKV_ERR_INVALID_ARG;
  if (scaling == BKV_ROPE_YARN && (!(original_len > 0.0) || !std::isfinite(original_len))) return BKV_ERR_INVALID_ARG;
  if (rotary_dim > bkv::kD || rotary_dim % 16) return BKV_ERR_UNSUPPORTED;
  out->rotary_dim = rotary_dim;
  out->interleaved = interleaved;
  out->scale = scaling == BKV_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  const double r = rotary_dim;
  if (scaling == BKV_ROPE_NTK && rotary_dim > 0) theta *= std::pow(factor, r / (r - 2.0));
  for (int i = 0; i < bkv::kRopePairs; ++i) {
    double f = 0.0;
    if (i < rotary_dim / 2) {
      f = std::pow(theta, -2.0 * i / r);
      if (scaling == BKV_ROPE_LINEAR) f /= factor;
      if (scaling == BKV_ROPE_YARN) {
        const double turns = original_len * f / (2.0 * kPi);
        const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
        f *= keep + (1.0 - keep) / factor;
      }
    }
    out->inv_freq[i] = f;
  }
  return BKV_OK;
}

bkv_status bkv_store_paged(const bkv_config* cfg, const bkv_pages* pages, const bkv_rope* rope, const void* q_pre,
                           int64_t q_stride, const void* k_pre, int64_t k_stride, const void* v, int64_t v_stride,
                           int32_t total, const int32_t* cu_seqlens, const int32_t* first_slot, const int32_t* first_pos,
                           const int32_t* depth, void* q_rot, void* K, void* V, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_store_paged");
  bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  bkv::StorePagedParams p{};
  st = take_pages(c, pages, p.pg);
  if (st != BKV_OK) return st;
  if (!rope || total < 0 || !cu_seqlens || !first_slot || !first_pos || (total > 0 && !q_rot) || !K || !V || !aligned(cu_seqlens, 4) ||
      !aligned(first_slot, 4) || !aligned(first_pos, 4) || !aligned(depth, 4) || !aligned(q_rot, 16) || !aligned(K, 16) ||
      !aligned(V, 16) || !aligned(status, 4))
    return BKV_ERR_INVALID_ARG;
  if (!strided_ok(q_pre, q_stride, c.heads, c.d, total) || !strided_ok(k_pre, k_stride, c.kv_heads, c.d, total) ||
      !strided_ok(v, v_stride, c.kv_heads, c.d, total))
    return BKV_ERR_INVALID_ARG;
  if (rope->rotary_dim < 0 || (rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->scale)) return BKV_ERR_INVALID_ARG;
  if (rope->rotary_dim > bkv::kD || rope->rotary_dim % 16) return BKV_ERR_UNSUPPORTED;
  for (int i = 0; i < rope->rotary_dim / 2; ++i) {
    if (!std::isfinite(rope->inv_freq[i])) return BKV_ERR_INVALID_ARG;
    double turns = rope->inv_freq[i] / (2.0 * kPi);
    turns -= std::floor(turns);
    p.turns[i] = turns < 1.0 ? (uint64_t)std::ldexp(turns, 64) : 0ull;
  }
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  if (total == 0) return BKV_OK;
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
  p.total = total;
  p.rotary = rope->rotary_dim;
  p.interleaved = rope->interleaved;
  p.scale = (float)rope->scale;
  return bkv::launch_store_paged(p, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_attend_paged_bytes(const bkv_config* cfg, const bkv_pages* pages, int32_t weighed, size_t* bytes) {
  bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  if (!bytes) return BKV_ERR_INVALID_ARG;
  bkv::Pages p{};
  st = take_pages(*cfg, pages, p);
  if (st != BKV_OK) return st;
  *bytes = lay_out(*cfg, p, weighed != 0).bytes;
  return BKV_OK;
}

bkv_status bkv_attend_paged(const bkv_config* cfg, const bkv_pages* pages, const void* q, int64_t q_stride, const void* K,
                            const void* V, const int32_t* lens, void* out, float* lse, float* weights, float decay,
                            void* workspace, size_t workspace_bytes, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_attend_paged");
  bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  bkv::AttendPagedParams p{};
  st = take_pages(c, pages, p.pg);
  if (st != BKV_OK) return st;
  if (!K || !V || !lens || !out || !aligned(K, 16) || !aligned(V, 16) || !aligned(lens, 4) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(weights, 4) || !aligned(status, 4) || !strided_ok(q, q_stride, c.heads, c.d, 1) ||
      (weights && !decay_ok(decay)))
    return BKV_ERR_INVALID_ARG;
  const Workspace w = lay_out(c, p.pg, weights != nullptr);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.bytes) return BKV_ERR_WORKSPACE;
  p.q = static_cast<const uint4*>(q);
  p.q_stride = q_stride / 8;
  p.K = static_cast<const uint4*>(K);
  p.V = static_cast<const uint4*>(V);
  p.lens = lens;
  p.out = static_cast<uint4*>(out);
  p.lse = lse;
  p.weights = weights;
  p.status = status;
  p.decay = decay;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.d));
  p.batch = c.batch;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = c.heads / c.kv_heads;
  p.chunk = p.group > 8 ? 16 : 8;
  p.chunks = (p.group + p.chunk - 1) / p.chunk;
  // the kernels count tiles of 16 slots, output rows and (page, KV head) planes in 32 bits
  if ((int64_t)p.pg.pages * c.kv_heads > 0x7FFFFFFF ||
      (int64_t)c.batch * ((p.pg.cap + bkv::kTileSlots - 1) / bkv::kTileSlots) * c.kv_heads * p.chunks > 0x7FFF0000 ||
      (int64_t)c.batch * c.heads > 0x7FFFFFFF / 32)
    return BKV_ERR_UNSUPPORTED;
  p.tiles_cap = weights ? most_tiles(c, p.pg) * c.kv_heads : 0;
  char* base = static_cast<char*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(base + w.part_ml);
  p.part_o = reinterpret_cast<float4*>(base + w.part_o);
  p.lse2 = reinterpret_cast<float*>(base + w.lse2);
  p.seq = reinterpret_cast<int2*>(base + w.seq);
  p.logits = weights ? reinterpret_cast<float*>(base + w.logits) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (!bkv::encode_attend_paged_maps(p)) return BKV_ERR_CUDA;
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  return bkv::launch_attend_paged(p, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_weigh_prompt(const bkv_config* cfg, const bkv_pages* pages, const void* q, int64_t q_stride, const float* lse,
                            const void* K, const int32_t* cu_seqlens, const int32_t* first_slot, int32_t total,
                            float* weights, float decay, uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_weigh_prompt");
  bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  bkv::WeighParams p{};
  st = take_pages(c, pages, p.pg);
  if (st != BKV_OK) return st;
  if (total < 0 || !K || !weights || !cu_seqlens || !first_slot || (total > 0 && !lse) || !aligned(K, 16) || !aligned(weights, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(first_slot, 4) || !aligned(lse, 4) || !aligned(status, 4) ||
      !strided_ok(q, q_stride, c.heads, c.d, total) || !decay_ok(decay))
    return BKV_ERR_INVALID_ARG;
  p.group = c.heads / c.kv_heads;
  if (p.group > bkv::kWeighRows) return BKV_ERR_UNSUPPORTED;
  p.K = static_cast<const uint4*>(K);
  p.row_lse = lse;
  p.cu = cu_seqlens;
  p.first = first_slot;
  p.weights = weights;
  p.status = status;
  p.decay = decay;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.d));
  p.batch = c.batch;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.total = total;
  p.tpt = bkv::kWeighRows / p.group;
  // tiles of 128 slots there can be; the kernel counts them in 32 bits
  const int64_t items = (int64_t)c.batch * c.kv_heads * ((p.pg.cap + 127) / 128);
  if (items > 0x7FFFFFFF - 4096) return BKV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (total > 0 && !bkv::encode_weigh_map(p, q, q_stride)) return BKV_ERR_CUDA;
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  if (total == 0) return BKV_OK;
  return bkv::launch_weigh(p, items, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

bkv_status bkv_evict_weight(const bkv_config* cfg, const bkv_pages* pages, void* const* K, void* const* V,
                            float* const* weights, const int32_t* cache_lens, int32_t* kept, int32_t* new_lens,
                            uint32_t* status, void* cuda_stream) {
  NvtxRange nvtx("bkv_evict_weight");
  bkv_status st = check(cfg);
  if (st != BKV_OK) return st;
  const bkv_config& c = *cfg;
  bkv::EvictWeightParams p{};
  st = take_pages(c, pages, p.pg);
  if (st != BKV_OK) return st;
  if (!K || !V || !weights || !cache_lens || !kept || new_lens == cache_lens || !aligned(cache_lens, 4) || !aligned(kept, 4) ||
      !aligned(new_lens, 4) || !aligned(status, 4))
    return BKV_ERR_INVALID_ARG;
  for (int l = 0; l < c.layers; ++l)
    if (!K[l] || !V[l] || !weights[l] || !aligned(K[l], 16) || !aligned(V[l], 16) || !aligned(weights[l], 4))
      return BKV_ERR_INVALID_ARG;
  p.order_free = (c.flags & BKV_FLAG_ORDER_FREE) != 0;
  const int64_t units = (int64_t)c.layers * c.batch * c.kv_heads;
  // the kernel counts slots of the keep set in 32 bits, a block's width at a time
  if (units > 0x7FFFFFFF || c.budget > 0x7FFFFFFF - 4096 || (p.order_free && c.budget > (1 << 19))) return BKV_ERR_UNSUPPORTED;
  for (int l = 0; l < c.layers; ++l) {
    p.K[l] = static_cast<uint4*>(K[l]);
    p.V[l] = static_cast<uint4*>(V[l]);
    p.W[l] = weights[l];
  }
  p.lens = cache_lens;
  p.kept = kept;
  p.new_lens = new_lens;
  p.status = status;
  p.layers = c.layers;
  p.batch = c.batch;
  p.kv_heads = c.kv_heads;
  p.budget = c.budget;
  p.prefix = c.prefix;
  p.recent = c.recent;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (zero_status(status, s) != BKV_OK) return BKV_ERR_CUDA;
  return bkv::launch_evict_weight(p, s) == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

}  // extern "C"
