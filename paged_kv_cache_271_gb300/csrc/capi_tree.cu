// C ABI of the speculative-decoding operators: argument checks and dispatch of the fused norm +
// rotation + append, the tree attention and the path commit.
#include <algorithm>
#include <cmath>

#include <cuda.h>

#include "capi_util.h"
#include "pkv.h"
#include "pkv_internal.h"

using namespace pkv;

namespace {

// Query rows of a unit, tokens of a tile, least tiles of a CTA, cost of a pass in tiles, the weights
// of narrow and wide passes (tree_plan.cuh) and the CTAs of one wave of the kernel that a call uses.
struct TreeSplit {
  int rows, tokens, min_tiles, pass_cost, narrow_rows, wide_tile, wave;
  bool tc;
};

// bf16 queries run on the tensor cores, fp32 queries (whose weights keep 24 bits) on CUDA cores.
// Measured on the tensor cores, 8-bit caches: a pass costs as much as about 12 narrow tiles (128
// requests of 128 .. 8192 tokens, 192 rows a head: 409 us with 4, 376 with 8, 366 with 12, 382 with
// 24); bf16: 8 (64 requests, 64 rows: 122 us with 4, 118 with 8, 128 with 24). A wide tile costs as
// much as one and a half narrow ones (the 192-row batch: 446 us when counted as one, 376 as one and
// a half, 382 as two; bf16, ragged drafts of up to 256 rows: 163, 141, 138).
TreeSplit tree_split(int dtype_q, int kv, int head_dim) {
  if (dtype_q == PKV_BF16)
    return TreeSplit{kTreeTcRows,     kTreeTcTokens, 2, is_coded(kv) ? 12 : 8,
                     kTreeTcRows / 2, 3,             kTreeTcWave, true};
  return TreeSplit{kTreeSimtRows, kTreeSimtTokens, 1, 1,
                   kTreeSimtRows, 2,               tree_simt_wave(head_dim), false};
}

size_t tree_acc_bytes(const TreeSplit& t, int ctas, int head_dim) {
  return align256((size_t)ctas * 2 * t.rows * head_dim * sizeof(float));
}
size_t tree_ml_bytes(const TreeSplit& t, int ctas) {
  return align256((size_t)ctas * 2 * t.rows * 2 * sizeof(float));
}

int check_tree_types(const char* who, int dtype_q, int kv) {
  if (dtype_q != PKV_F32 && dtype_q != PKV_BF16)
    return set_error(PKV_EDTYPE, "%s: q dtype must be F32 or BF16", who);
  if (!is_coded(kv) && kv != dtype_q)
    return set_error(PKV_EDTYPE, "%s: q dtype must match an F32/BF16 cache", who);
  return PKV_OK;
}

// a b, or 2^60 where that is less (a, b in [0, 2^62]).
long long capped_product(long long a, long long b) {
  constexpr long long most = 1ll << 60;
  return b != 0 && a > most / b ? most : a * b;
}

// Half tiles of work (tree_plan.cuh) that the call's table could hold at most (up to 2^60).
long long tree_most_work(const TreeSplit& t, int batch, int nodes, int h_q, int h_kv,
                         int max_pages) {
  const long long units = ((long long)nodes * (h_q / h_kv) + t.rows - 1) / t.rows;
  const long long tiles = ((long long)max_pages * 16 + t.tokens - 1) / t.tokens;
  const long long passes = capped_product((long long)batch * h_kv, units);
  return capped_product(passes, tiles * t.wide_tile + 2 * t.pass_cost);
}

// CTAs of a call: one wave, or fewer when the table cannot hold that many shares.
int tree_ctas(const TreeSplit& t, int batch, int nodes, int h_q, int h_kv, int max_pages) {
  const long long work = tree_most_work(t, batch, nodes, h_q, h_kv, max_pages);
  return (int)std::max(1ll, std::min<long long>(t.wave, work / (2 * t.min_tiles) + 1));
}

int check_tree_sizes(const char* who, int batch, int nodes, int h_q, int h_kv, int max_pages) {
  if (batch < 0 || nodes < 0 || h_q <= 0 || h_kv <= 0 || max_pages <= 0)
    return set_error(PKV_EINVAL, "%s: bad batch, tree width, head count or table width", who);
  if (h_q % h_kv != 0)
    return set_error(PKV_ESHAPE, "%s: num_q_heads %% num_kv_heads != 0", who);
  if (nodes > PKV_MAX_TREE_NODES || h_q / h_kv > PKV_MAX_TREE_GROUP)
    return set_error(PKV_ESHAPE, "%s: at most %d nodes and %d query heads per KV head", who,
                     PKV_MAX_TREE_NODES, PKV_MAX_TREE_GROUP);
  if (h_kv > 65535 || batch > 65535)
    return set_error(PKV_ESHAPE, "%s: batch and kv heads must be <= 65535", who);
  if (max_pages > (1 << 27) - 16)  // (positions and tile ends stay below 2^31)
    return set_error(PKV_ESHAPE, "%s: a table row holds 2^31 positions or more", who);
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, int32_t dtype, int32_t num_tokens,
                            int32_t num_q_heads, const void* q_weight, const void* k_weight,
                            float eps, const float* cos_sin, int32_t max_positions,
                            int32_t rot_dim, int32_t interleaved, const int32_t* positions,
                            const int64_t* slot_mapping, void* q_out, int64_t q_out_stride,
                            void* k_cache, void* v_cache, const pkv_cache_desc* desc,
                            const float* k_scales, const float* v_scales, void* stream) {
  const char* who = "pkv_qk_norm_rope_append";
  int st = check_desc(desc, who);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_q_heads <= 0)
    return set_error(PKV_EINVAL, "%s: bad token or head count", who);
  if (num_tokens == 0) return PKV_OK;
  const int D = desc->head_dim, h_kv = desc->num_kv_heads, kv = desc->cache_dtype;
  if (!q || !k || !v || !q_out || !k_cache || !v_cache || !slot_mapping)
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (dtype != PKV_F32 && dtype != PKV_BF16)
    return set_error(PKV_EDTYPE, "%s: q, k and v must be F32 or BF16", who);
  if (!is_coded(kv) && kv != dtype)
    return set_error(PKV_EDTYPE, "%s: input dtype must equal an F32/BF16 cache's", who);
  if (is_coded(kv) && (!k_scales || !v_scales))
    return set_error(PKV_EINVAL, "%s: FP8/INT8 cache needs scales", who);
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
    return set_error(PKV_ESHAPE, "%s: rot_dim %d is not a multiple of 16 in [0, head_dim]", who,
                     rot_dim);
  if (rot_dim > 0 && (!cos_sin || !positions || max_positions <= 0))
    return set_error(PKV_EINVAL, "%s: a rotation needs cos_sin, positions and max_positions", who);
  if (interleaved != 0 && interleaved != 1)
    return set_error(PKV_EINVAL, "%s: interleaved must be 0 or 1", who);
  if (!(eps >= 0.f) || std::isinf(eps))
    return set_error(PKV_EINVAL, "%s: eps must be finite and >= 0", who);
  const int eb = dtype_bytes(dtype);
  const int64_t need_q = (int64_t)num_q_heads * D, need_kv = (int64_t)h_kv * D;
  if (need_q >= (1ll << 31) || need_kv * desc->page_size >= (1ll << 31))
    return set_error(PKV_ESHAPE, "%s: a token's queries or a page hold 2^31 elements or more", who);
  if (num_tokens > 1 && (q_stride < need_q || k_stride < need_kv || v_stride < need_kv ||
                         q_out_stride < need_q))
    return set_error(PKV_ESHAPE, "%s: a token stride is smaller than the token's row", who);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(cos_sin) || !aligned16(q_weight) ||
      !aligned16(k_weight) ||
      (num_tokens > 1 && (q_stride * eb % 16 || k_stride * eb % 16 || v_stride * eb % 16 ||
                          q_out_stride * eb % 16)))
    return set_error(PKV_EALIGN, "%s: pointers and token strides must be 16-byte aligned", who);
  NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.max_positions = max_positions;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.slots = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = is_coded(kv) ? k_scales : nullptr;
  a.v_scales = is_coded(kv) ? v_scales : nullptr;
  a.num_tokens = num_tokens;
  a.h_q = num_q_heads;
  a.h_kv = h_kv;
  a.head_dim = D;
  a.num_slots = (int64_t)desc->num_pages * desc->page_size;
  st = error_word(&a.err);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = traced("qk_norm_rope_append", s,
                         [&] { return launch_qk_norm_rope_append(a, dtype, kv, s); });
  return cuda_status(e, "qk_norm_rope_append launch");
}

size_t pkv_tree_decode_workspace_size(int32_t dtype_q, int32_t cache_dtype, int32_t batch,
                                      int32_t tree_width, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t head_dim,
                                      int32_t max_pages_per_seq) {
  if (batch <= 0 || tree_width <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_pages_per_seq <= 0)
    return 0;
  const TreeSplit t = tree_split(dtype_q, cache_dtype, head_dim);
  const int ctas = tree_ctas(t, batch, tree_width, num_q_heads, num_kv_heads, max_pages_per_seq);
  return tree_acc_bytes(t, ctas, head_dim) + tree_ml_bytes(t, ctas);
}

int pkv_tree_decode_attention(const void* q, int32_t dtype_q, int32_t batch, int32_t tree_width,
                              int32_t num_q_heads, const void* k_cache, const void* v_cache,
                              const pkv_cache_desc* desc, const int32_t* block_tables,
                              int32_t max_pages_per_seq, const int32_t* context_lens,
                              const int32_t* tree_lens, const uint64_t* tree_mask,
                              int64_t mask_batch_stride, float scale, const float* k_scales,
                              const float* v_scales, void* out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const char* who = "pkv_tree_decode_attention";
  int st = check_desc(desc, who);
  if (st != PKV_OK) return st;
  const int h_kv = desc->num_kv_heads, D = desc->head_dim, kv = desc->cache_dtype;
  st = check_tree_sizes(who, batch, tree_width, num_q_heads, h_kv, max_pages_per_seq);
  if (st != PKV_OK) return st;
  st = check_tree_types(who, dtype_q, kv);
  if (st != PKV_OK) return st;
  if (batch == 0 || tree_width == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (is_coded(kv) && (!k_scales || !v_scales))
    return set_error(PKV_EINVAL, "%s: FP8/INT8 cache needs k_scales and v_scales", who);
  if (!(scale > 0.f) || std::isinf(scale))
    return set_error(PKV_EINVAL, "%s: scale must be positive and finite", who);
  const int words = (tree_width + 63) / 64;
  if (tree_mask && mask_batch_stride != 0 &&
      mask_batch_stride < (int64_t)tree_width * words)
    return set_error(PKV_ESHAPE, "%s: mask_batch_stride must be 0 or at least tree_width * "
                     "ceil(tree_width / 64)", who);
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return set_error(PKV_EALIGN, "%s: q, out and pools must be 16-byte, the mask 8-byte aligned",
                     who);
  if (dtype_q == PKV_BF16 && kv == PKV_BF16 &&
      (long long)desc->num_pages * h_kv * desc->page_size >= (1ll << 31))
    return set_error(PKV_ESHAPE, "%s: a bf16 pool must have fewer than 2^31 rows", who);
  const TreeSplit t = tree_split(dtype_q, kv, D);
  if (tree_most_work(t, batch, tree_width, num_q_heads, h_kv, max_pages_per_seq) >= (1ll << 30))
    return set_error(PKV_ESHAPE, "%s: the table can hold 2^30 half tiles of work or more", who);
  TreeArgs a{};
  a.ctas = tree_ctas(t, batch, tree_width, num_q_heads, h_kv, max_pages_per_seq);
  const size_t acc = tree_acc_bytes(t, a.ctas, D), need = acc + tree_ml_bytes(t, a.ctas);
  if (!workspace || workspace_bytes < need)
    return set_error(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", who, need,
                     workspace ? workspace_bytes : 0);
  if (!aligned16(workspace)) return set_error(PKV_EALIGN, "%s: workspace alignment", who);
  a.q = q;
  a.out = out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.tree_lens = tree_lens;
  a.mask = tree_mask;
  a.mask_stride = mask_batch_stride;
  a.mask_words = words;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + acc);
  a.batch = batch;
  a.nodes = tree_width;
  a.h_q = num_q_heads;
  a.h_kv = h_kv;
  a.group = num_q_heads / h_kv;
  a.num_pages = desc->num_pages;
  a.max_pages = max_pages_per_seq;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.unit_rows = t.rows;
  a.tile_tokens = t.tokens;
  a.min_tiles = t.min_tiles;
  a.pass_cost = t.pass_cost;
  a.narrow_rows = t.narrow_rows;
  a.wide_tile = t.wide_tile;
  st = error_word(&a.err);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap tk{}, tv{};
  if (t.tc && kv == PKV_BF16) {
    int rank = 2;
    st = pool_tensor_map(k_cache, desc, &tk, &rank, true);
    if (st == PKV_OK) st = pool_tensor_map(v_cache, desc, &tv, &a.tma_rank);
    if (st != PKV_OK) return st;
  }
  cudaError_t e = traced("tree_attention", s, [&] {
    return t.tc ? launch_tree_tc(a, kv, D, &tk, &tv, s) : launch_tree_simt(a, kv, D, s);
  });
  st = cuda_status(e, "tree_attention launch");
  if (st != PKV_OK || a.ctas == 1) return st;  // (one CTA finishes every pass)
  e = traced("tree_combine", s, [&] { return launch_tree_combine(a, dtype_q, D, s); });
  return cuda_status(e, "tree_combine launch");
}

int pkv_tree_commit(void* k_cache, void* v_cache, const pkv_cache_desc* desc,
                    const int32_t* block_tables, int32_t max_pages_per_seq,
                    const int32_t* context_lens, const int32_t* tree_lens, const int32_t* path,
                    const int32_t* path_lens, int32_t batch, int32_t max_path, int32_t* new_lens,
                    void* stream) {
  const char* who = "pkv_tree_commit";
  int st = check_desc(desc, who);
  if (st != PKV_OK) return st;
  if (batch < 0 || max_path < 0 || max_pages_per_seq <= 0)
    return set_error(PKV_EINVAL, "%s: bad batch, path or table width", who);
  if (batch == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !tree_lens || !path_lens ||
      (max_path > 0 && !path))
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (new_lens == context_lens || new_lens == tree_lens || new_lens == path_lens ||
      (new_lens && new_lens == path))
    return set_error(PKV_EINVAL, "%s: new_lens must not be one of the inputs", who);
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return set_error(PKV_EALIGN, "%s: pools must be 16-byte aligned", who);
  CommitArgs a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.tree_lens = tree_lens;
  a.path = path;
  a.path_lens = path_lens;
  a.new_lens = new_lens;
  a.batch = batch;
  a.max_path = max_path;
  a.max_pages = max_pages_per_seq;
  a.num_pages = desc->num_pages;
  a.h_kv = desc->num_kv_heads;
  a.row_bytes = desc->head_dim * dtype_bytes(desc->cache_dtype);
  if ((long long)a.h_kv * (a.row_bytes / 16) > 65535ll * 128)
    return set_error(PKV_ESHAPE, "%s: too many KV heads", who);
  st = error_word(&a.err);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = traced("tree_commit", s, [&] { return launch_tree_commit(a, s); });
  return cuda_status(e, "tree_commit launch");
}

int pkv_tree_masks(const int32_t* parents, int64_t n_trees, int32_t tree_width,
                   uint64_t* masks_out, int32_t* depths_out) {
  const char* who = "pkv_tree_masks";
  if (n_trees < 0 || tree_width < 0 || tree_width > PKV_MAX_TREE_NODES)
    return set_error(PKV_EINVAL, "%s: bad tree count or width", who);
  if (n_trees == 0 || tree_width == 0) return PKV_OK;
  if (!parents || !masks_out) return set_error(PKV_EINVAL, "%s: null pointer", who);
  const int words = (tree_width + 63) / 64;
  for (int64_t i = 0; i < n_trees * tree_width; ++i) {
    const int32_t node = (int32_t)(i % tree_width), p = parents[i];
    if (p < -1 || p >= node)
      return set_error(PKV_EINVAL, "%s: node %d of tree %lld has parent %d (-1 or an earlier "
                       "node)", who, node, (long long)(i / tree_width), p);
  }
  for (int64_t t = 0; t < n_trees; ++t) {
    const int32_t* par = parents + t * tree_width;
    uint64_t* m = masks_out + t * tree_width * words;
    for (int32_t i = 0; i < tree_width; ++i) {
      const int32_t p = par[i];
      for (int w = 0; w < words; ++w)
        m[(int64_t)i * words + w] = p < 0 ? 0 : m[(int64_t)p * words + w];
      m[(int64_t)i * words + i / 64] |= 1ull << (i % 64);
      if (depths_out)
        depths_out[t * tree_width + i] = p < 0 ? 0 : depths_out[t * tree_width + p] + 1;
    }
  }
  return PKV_OK;
}

}  // extern "C"
