// C ABI of the operators on chunks of new tokens and of the eviction: argument checks and dispatch.
#include <algorithm>
#include <cmath>

#include <cuda.h>

#include "capi_util.h"
#include "chunk_plan.cuh"
#include "pkv.h"
#include "pkv_internal.h"
#include "weigh_plan.cuh"

using namespace pkv;

namespace {

// Rows of a unit, tokens of a tile, least tiles of a CTA, cost of a unit in tiles, the weights of narrow
// and wide tiles (chunk_plan.cuh) and the CTAs of one wave of the kernel that a call uses.
struct ChunkSplit {
  int rows, tokens, min_tiles, pass_cost, narrow_rows, wide_tile, wave;
  bool tc;
};

// The tensor cores' constants were measured in graphs (64 biased decode steps; an 8191-token prompt; a
// window): 132, 431 and 244 us; with a unit's cost of 1 tile 134, 472, 254, of 6 138, 439, 245; with wide
// tiles (more than 128 rows) of weight 2 against a narrow one's 2 132, 435, 246, of 4 132, 440, 251; least
// tiles of 1 or 4 make no difference there.
// bf16 queries run on the tensor cores, fp32 queries (whose weights keep 24 bits) on CUDA cores.
ChunkSplit chunk_split(int dtype_q, int kv, int head_dim) {
  if (dtype_q == PKV_BF16)
    return ChunkSplit{kChunkTcRows, kChunkTcTokens, 2, 3, kChunkTcRows / 2, 3, kChunkTcWave, true};
  return ChunkSplit{kChunkSimtRows, kChunkSimtTokens, 1, 1, kChunkSimtRows, 2,
                    chunk_simt_wave(head_dim), false};
}

// a b, or 2^60 where that is less (a, b in [0, 2^62]).
long long capped_product(long long a, long long b) {
  constexpr long long most = 1ll << 60;
  return b != 0 && a > most / b ? most : a * b;
}

// Units of one KV head that num_rows tokens of `batch` requests can have at most.
long long chunk_most_units(int rows, int num_rows, int batch, int group) {
  const long long tokens = std::max(1, rows / group), subs = (group + rows - 1) / rows;
  const long long used = std::min(batch, num_rows);  // (requests with rows)
  return ((num_rows - used) / tokens + used) * subs;
}

// Half tiles of work that the call's rows and table could hold at most (up to 2^60).
long long chunk_most_work(const ChunkSplit& t, int num_rows, int batch, int h_q, int h_kv,
                          int max_pages) {
  const long long units =
      capped_product(chunk_most_units(t.rows, num_rows, batch, h_q / h_kv), h_kv);
  const long long tiles = ((long long)max_pages * kPageSize + t.tokens - 1) / t.tokens;
  return capped_product(units, tiles * t.wide_tile + 2 * t.pass_cost);
}

// CTAs of a call: one wave, or fewer when rows and table cannot hold that many shares.
int chunk_ctas(const ChunkSplit& t, int num_rows, int batch, int h_q, int h_kv, int max_pages) {
  const long long work = chunk_most_work(t, num_rows, batch, h_q, h_kv, max_pages);
  return (int)std::max(1ll, std::min<long long>(t.wave, work / (2 * t.min_tiles) + 1));
}

struct ChunkSpace {
  size_t acc, ml, all;  // offsets of the partials' (max, sum) and the records, bytes in all
};

ChunkSpace chunk_space(const ChunkSplit& t, int ctas, int head_dim) {
  ChunkSpace s;
  s.acc = align256((size_t)ctas * 2 * t.rows * head_dim * sizeof(float));
  s.ml = s.acc + align256((size_t)ctas * 2 * t.rows * 2 * sizeof(float));
  s.all = s.ml + align256((size_t)ctas * sizeof(ChunkRecord));
  return s;
}

// What the attention and the weights check alike; fills in what both kernels read.
int check_chunk(const char* who, const void* q, int dtype_q, int num_rows, int batch, int h_q,
                const void* k_cache, const pkv_cache_desc* desc, const int32_t* block_tables,
                int max_pages, const int32_t* context_lens, const int32_t* query_starts,
                const pkv_score_form* form, const float* k_scales, ChunkArgs& a) {
  int st = check_desc(desc, who);
  if (st != PKV_OK) return st;
  const int h_kv = desc->num_kv_heads, kv = desc->cache_dtype;
  if (num_rows < 0 || batch < 0 || h_q <= 0 || h_kv <= 0 || max_pages <= 0)
    return set_error(PKV_EINVAL, "%s: bad row count, batch, head count or table width", who);
  if (h_q % h_kv != 0) return set_error(PKV_ESHAPE, "%s: num_q_heads %% num_kv_heads != 0", who);
  if (h_q / h_kv > PKV_MAX_CHUNK_GROUP)
    return set_error(PKV_ESHAPE, "%s: at most %d query heads per KV head", who,
                     PKV_MAX_CHUNK_GROUP);
  if (h_kv > 65535 || batch > 65535)
    return set_error(PKV_ESHAPE, "%s: batch and kv heads must be <= 65535", who);
  if (max_pages > (1 << 27) - 16)  // (positions and tile ends stay below 2^31)
    return set_error(PKV_ESHAPE, "%s: a table row holds 2^31 positions or more", who);
  if ((long long)num_rows * h_q >= (1ll << 31))
    return set_error(PKV_ESHAPE, "%s: 2^31 query heads of rows or more", who);
  if (dtype_q != PKV_F32 && dtype_q != PKV_BF16)
    return set_error(PKV_EDTYPE, "%s: q dtype must be F32 or BF16", who);
  if (!is_coded(kv) && kv != dtype_q)
    return set_error(PKV_EDTYPE, "%s: q dtype must match an F32/BF16 cache", who);
  if (!form) return set_error(PKV_EINVAL, "%s: null score form", who);
  if (!(form->scale > 0.f) || std::isinf(form->scale))
    return set_error(PKV_EINVAL, "%s: scale must be positive and finite", who);
  if (!(form->softcap >= 0.f) || std::isinf(form->softcap))
    return set_error(PKV_EINVAL, "%s: softcap must be finite and >= 0", who);
  // The kernels take scale log2(e), 1 / softcap and scale / softcap as fp32, beyond which 0 times infinity
  // would be a score. Caps are moved to where they are in range: below 2^-100 all of them leave weights that
  // are equal, above 2^100 the scores (up to 2^88) as they are, to the last bit.
  const float cap = form->softcap > 0.f ? std::min(std::max(form->softcap, 0x1p-100f), 0x1p100f) : 0.f;
  if (!(form->scale <= 0x1p126f) || (cap > 0.f && !(form->scale / cap <= 0x1p120f)))
    return set_error(PKV_EINVAL, "%s: scale beyond 2^126, or 2^120 times softcap", who);
  if (form->window < 0 || form->sink_tokens < 0 || (form->window == 0 && form->sink_tokens != 0))
    return set_error(PKV_EINVAL, "%s: window and sink_tokens must be >= 0; sinks need a window",
                     who);
  if (dtype_q == PKV_BF16 && kv == PKV_BF16 &&
      (long long)desc->num_pages * h_kv * desc->page_size >= (1ll << 31))
    return set_error(PKV_ESHAPE, "%s: a bf16 pool must have fewer than 2^31 rows", who);
  if (batch == 0) return PKV_OK;
  if (num_rows > 0 && (!q || !k_cache || !block_tables))
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (!context_lens || !query_starts) return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (num_rows > 0 && is_coded(kv) && !k_scales)
    return set_error(PKV_EINVAL, "%s: FP8/INT8 cache needs scales", who);
  if (!aligned16(q) || !aligned16(k_cache))
    return set_error(PKV_EALIGN, "%s: q and pools must be 16-byte aligned", who);
  a.q = q;
  a.k_cache = k_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_starts = query_starts;
  a.slopes = form->alibi_slopes;
  a.k_scales = k_scales;
  a.num_rows = num_rows;
  a.batch = batch;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.group = h_q / h_kv;
  a.num_pages = desc->num_pages;
  a.max_pages = max_pages;
  a.scale = form->scale;
  a.softcap = cap;
  a.window = form->window;
  a.sink = form->sink_tokens;
  return PKV_OK;
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

void set_tile(ChunkArgs& a, int rows, int tokens) {
  a.unit_rows = rows;
  a.rows_shift = log2_of(rows);
  a.tile_tokens = tokens;
  a.tile_shift = log2_of(tokens);
}

void set_split(ChunkArgs& a, const ChunkSplit& t) {
  set_tile(a, t.rows, t.tokens);
  a.unit_tokens = std::max(1, t.rows / a.group);
  a.subs = (a.group + t.rows - 1) / t.rows;
  a.min_tiles = t.min_tiles;
  a.pass_cost = t.pass_cost;
  a.narrow_rows = t.narrow_rows;
  a.wide_tile = t.wide_tile;
}

// The same for the weights' sums (weigh_plan.cuh): rows of a step, positions of an item, CTAs.
struct WeighSplit {
  int rows, tokens, wave;
  bool tc;
};

WeighSplit weigh_split(int dtype_q, int head_dim) {
  if (dtype_q == PKV_BF16) return WeighSplit{kWeighTcRows, kWeighTcTokens, kWeighTcWave, true};
  return WeighSplit{kChunkSimtRows, kChunkSimtTokens, weigh_simt_wave(head_dim), false};
}

// Steps that the call's rows and sums could take at most (up to 2^60).
long long weigh_most_work(const WeighSplit& t, int num_rows, int batch, int h_q, int h_kv,
                          int64_t width) {
  const long long items = capped_product((width + t.tokens - 1) / t.tokens, h_kv);
  // (every request's items: two each, besides a step for every t.rows rows and a broken one)
  const long long steps = (long long)num_rows * (h_q / h_kv) / t.rows + 3ll * batch;
  return capped_product(items, steps);
}

int weigh_ctas(const WeighSplit& t, int num_rows, int batch, int h_q, int h_kv, int64_t width) {
  const long long work = weigh_most_work(t, num_rows, batch, h_q, h_kv, width);
  return (int)std::max(1ll, std::min<long long>(t.wave, work / 2 + 1));
}

ChunkSpace weigh_space(const WeighSplit& t, int ctas) {
  ChunkSpace s;
  s.acc = s.ml = align256((size_t)ctas * 2 * t.tokens * sizeof(float));
  s.all = s.ml + align256((size_t)ctas * sizeof(WeighRecord));
  return s;
}

}  // namespace

extern "C" {

size_t pkv_chunk_workspace_size(int32_t dtype_q, int32_t cache_dtype, int32_t num_rows,
                                int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t max_pages_per_seq) {
  if (num_rows <= 0 || batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_pages_per_seq <= 0 || num_q_heads < num_kv_heads)
    return 0;
  const ChunkSplit t = chunk_split(dtype_q, cache_dtype, head_dim);
  return chunk_space(
             t, chunk_ctas(t, num_rows, batch, num_q_heads, num_kv_heads, max_pages_per_seq),
             head_dim)
      .all;
}

int pkv_chunk_attention(const void* q, int32_t dtype_q, int32_t num_rows, int32_t batch,
                        int32_t num_q_heads, const void* k_cache, const void* v_cache,
                        const pkv_cache_desc* desc, const int32_t* block_tables,
                        int32_t max_pages_per_seq, const int32_t* context_lens,
                        const int32_t* query_starts, const pkv_score_form* form,
                        const float* k_scales, const float* v_scales, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "pkv_chunk_attention";
  ChunkArgs a{};
  int st = check_chunk(who, q, dtype_q, num_rows, batch, num_q_heads, k_cache, desc, block_tables,
                       max_pages_per_seq, context_lens, query_starts, form, k_scales, a);
  if (st != PKV_OK || batch == 0 || num_rows == 0) return st;
  const int kv = desc->cache_dtype, D = desc->head_dim;
  if (!v_cache || !out) return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (is_coded(kv) && !v_scales)
    return set_error(PKV_EINVAL, "%s: FP8/INT8 cache needs k_scales and v_scales", who);
  if (!aligned16(out) || !aligned16(v_cache))
    return set_error(PKV_EALIGN, "%s: out and pools must be 16-byte aligned", who);
  const ChunkSplit t = chunk_split(dtype_q, kv, D);
  if (chunk_most_work(t, num_rows, batch, a.h_q, a.h_kv, a.max_pages) >= (1ll << 30))
    return set_error(PKV_ESHAPE, "%s: rows and table can hold 2^30 half tiles of work or more", who);
  a.ctas = chunk_ctas(t, num_rows, batch, a.h_q, a.h_kv, a.max_pages);
  set_split(a, t);
  const ChunkSpace space = chunk_space(t, a.ctas, D);
  if (!workspace || workspace_bytes < space.all)
    return set_error(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", who, space.all,
                     workspace ? workspace_bytes : 0);
  if (!aligned16(workspace)) return set_error(PKV_EALIGN, "%s: workspace alignment", who);
  a.out = out;
  a.lse = lse;
  a.v_cache = v_cache;
  a.v_scales = v_scales;
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + space.acc);
  a.ws_rec = static_cast<char*>(workspace) + space.ml;
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
  cudaError_t e = traced("chunk_attention", s, [&] {
    return t.tc ? launch_chunk_tc(a, kv, D, &tk, &tv, s) : launch_chunk_simt(a, kv, D, s);
  });
  st = cuda_status(e, "chunk_attention launch");
  if (st != PKV_OK || a.ctas == 1) return st;  // (one CTA finishes every unit)
  e = traced("chunk_combine", s, [&] { return launch_chunk_combine(a, dtype_q, D, s); });
  return cuda_status(e, "chunk_combine launch");
}

size_t pkv_chunk_weights_workspace_size(int32_t dtype_q, int32_t num_rows, int32_t batch,
                                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int64_t width) {
  if (num_rows < 0 || batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      width <= 0 || num_q_heads < num_kv_heads)
    return 0;
  const WeighSplit t = weigh_split(dtype_q, head_dim);
  return weigh_space(t, weigh_ctas(t, num_rows, batch, num_q_heads, num_kv_heads, width)).all;
}

int pkv_chunk_weights(const void* q, int32_t dtype_q, int32_t num_rows, int32_t batch,
                      int32_t num_q_heads, const void* k_cache, const pkv_cache_desc* desc,
                      const int32_t* block_tables, int32_t max_pages_per_seq,
                      const int32_t* context_lens, const int32_t* query_starts,
                      const pkv_score_form* form, const float* k_scales, const float* lse,
                      int32_t last_rows, const float* add_to, float* weights_out, int64_t width,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "pkv_chunk_weights";
  ChunkArgs a{};
  int st = check_chunk(who, q, dtype_q, num_rows, batch, num_q_heads, k_cache, desc, block_tables,
                       max_pages_per_seq, context_lens, query_starts, form, k_scales, a);
  if (st != PKV_OK) return st;
  if (width < 0 || last_rows < 0)
    return set_error(PKV_EINVAL, "%s: bad width or last_rows", who);
  if (batch == 0 || width == 0) return PKV_OK;
  const int kv = desc->cache_dtype, D = desc->head_dim;
  if (!weights_out || (num_rows > 0 && !lse)) return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (width >= (1ll << 31) - 256)
    return set_error(PKV_ESHAPE, "%s: a row of sums holds 2^31 positions or more", who);
  // Few rows a request on the mean: K is read once, straight into registers (the choice is made on what
  // the host knows; both kernels take any rows), by passes of 8 rows or 32. Measured, us, 64 requests of
  // 512 .. 4096 tokens, 8 KV heads, at 4 / 8 / 16 / 32 / 64 rows of each:
  //   FP8,  passes of 8: 37 / 37 / 67 / 128 / 247, of 32: 91 / 92 / 92 / 95 / 191, tcgen05: 135 (64: 139)
  //   bf16, passes of 8: 52 / 53 / 97 / 183 / 357, of 32: 103 / 104 / 105 / 107 / 209, tcgen05: 72
  // and for 8 requests at 16 / 32 rows: FP8 15 / 24, 24 / 25, 22 / 22; bf16 15 / 26, 24 / 26, 16 / 15.
  // What the host does not know is how uneven the rows are. One prompt beside 255 decode steps (4 heads to a
  // KV head, 512 .. 4096 tokens each), FP8, this rule / tcgen05: 300 tokens of it 543 / 651 us, 1500 of it
  // 2963 / 774 (a pass of 32 rows reads the prompt's K again, where a step there is 128 rows); bf16, whose
  // mean is beyond the rule there, 296 and 350. The sums are as good either way.
  const long long counted = last_rows > 0 ? std::min<long long>((long long)last_rows * batch, num_rows)
                                          : num_rows;
  const long long mean = (counted * a.group + batch - 1) / batch;
  const bool codes = kv == PKV_FP8_E4M3 || kv == PKV_INT8;
  const int blocks = mean <= 16 ? 1 : 4;
  const WeighSplit few{8 * blocks, kPageSize, weigh_few_wave(blocks), false};
  const long long work = weigh_most_work(few, num_rows, batch, a.h_q, a.h_kv, width);
  if (dtype_q == PKV_BF16 && mean <= (codes ? kWeighFewRowsCodes : kWeighFewRows) &&
      work < (1ll << 30)) {
    set_tile(a, few.rows, few.tokens);
    a.ctas = (int)std::max(1ll, std::min<long long>(few.wave, work / 4 + 1));
    a.lse = const_cast<float*>(lse);
    a.add_to = add_to;
    a.weights_out = weights_out;
    a.width = width;
    a.last_rows = last_rows;
    st = error_word(&a.err);
    if (st != PKV_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = traced("chunk_weights", s,
                           [&] { return launch_chunk_weights_few(a, kv, D, blocks, s); });
    return cuda_status(e, "chunk_weights launch");
  }
  const WeighSplit t = weigh_split(dtype_q, D);
  if (weigh_most_work(t, num_rows, batch, a.h_q, a.h_kv, width) >= (1ll << 30))
    return set_error(PKV_ESHAPE, "%s: rows and width can hold 2^30 steps of work or more", who);
  set_tile(a, t.rows, t.tokens);
  a.ctas = weigh_ctas(t, num_rows, batch, a.h_q, a.h_kv, width);
  const ChunkSpace space = weigh_space(t, a.ctas);
  if (!workspace || workspace_bytes < space.all)
    return set_error(PKV_EINVAL, "%s: workspace of %zu bytes needed, %zu given", who, space.all,
                     workspace ? workspace_bytes : 0);
  if (!aligned16(workspace)) return set_error(PKV_EALIGN, "%s: workspace alignment", who);
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_rec = static_cast<char*>(workspace) + space.ml;
  st = error_word(&a.err);
  if (st != PKV_OK) return st;
  a.lse = const_cast<float*>(lse);
  a.add_to = add_to;
  a.weights_out = weights_out;
  a.width = width;
  a.last_rows = last_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap tk{}, tq{};
  if (t.tc && kv == PKV_BF16 && num_rows > 0) {
    int rank = 2;
    st = pool_tensor_map(k_cache, desc, &tk, &rank, true);
    // a step's rows are whole tokens where the heads divide them: a box
    if (st == PKV_OK && kWeighTcRows % a.group == 0) {
      a.step_tokens = kWeighTcRows / a.group;
      st = query_tensor_map(q, num_rows, a.h_q, D, a.group, a.step_tokens, &tq);
    }
    if (st != PKV_OK) return st;
  }
  cudaError_t e = traced("chunk_weights", s, [&] {
    return t.tc ? launch_chunk_weights_tc(a, kv, D, &tk, &tq, s) : launch_chunk_weights_simt(a, kv, D, s);
  });
  st = cuda_status(e, "chunk_weights launch");
  if (st != PKV_OK || a.ctas == 1) return st;  // (one CTA finishes every item)
  e = traced("chunk_weights_combine", s, [&] { return launch_chunk_weights_combine(a, s); });
  return cuda_status(e, "chunk_weights_combine launch");
}

int pkv_evict_select(const float* weights, int64_t width, const int32_t* context_lens, int32_t batch,
                     int32_t num_kv_heads, int32_t budget, int32_t recent, int32_t sink_tokens,
                     int32_t* kept, int32_t* kept_lens, void* stream) {
  const char* who = "pkv_evict_select";
  if (batch < 0 || num_kv_heads <= 0 || width < 0)
    return set_error(PKV_EINVAL, "%s: bad batch, head count or width", who);
  if (budget <= 0 || recent < 0 || sink_tokens < 0 || (long long)recent + sink_tokens > budget)
    return set_error(PKV_EINVAL, "%s: budget must be positive and hold recent and sink_tokens", who);
  if (num_kv_heads > 65535 || batch > 65535)
    return set_error(PKV_ESHAPE, "%s: batch and kv heads must be <= 65535", who);
  if (width >= (1ll << 31) - 65536 || budget >= (1ll << 31) - 65536)
    return set_error(PKV_ESHAPE, "%s: a row holds 2^31 positions or more", who);
  if (batch == 0) return PKV_OK;
  if ((!weights && width > 0) || !context_lens || !kept || !kept_lens)
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (kept_lens == context_lens)
    return set_error(PKV_EINVAL, "%s: kept_lens must not be context_lens", who);
  EvictSelectArgs a{};
  a.weights = weights;
  a.width = width;
  a.context_lens = context_lens;
  a.kept = kept;
  a.kept_lens = kept_lens;
  a.batch = batch;
  a.h_kv = num_kv_heads;
  a.budget = budget;
  a.recent = recent;
  a.sink = sink_tokens;
  int st = error_word(&a.err);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = traced("evict_select", s, [&] { return launch_evict_select(a, s); });
  return cuda_status(e, "evict_select launch");
}

int pkv_evict_move(void* k_cache, void* v_cache, const pkv_cache_desc* desc,
                   const int32_t* block_tables, int32_t max_pages_per_seq, const int32_t* kept,
                   const int32_t* kept_lens, int32_t batch, int32_t budget,
                   const int32_t* new_tables, int32_t new_pages_per_seq, const float* weights,
                   int64_t width, float* new_weights, int64_t new_width, void* stream) {
  const char* who = "pkv_evict_move";
  int st = check_desc(desc, who);
  if (st != PKV_OK) return st;
  if (batch < 0 || budget <= 0 || max_pages_per_seq <= 0 || new_pages_per_seq <= 0 || width < 0 ||
      new_width < 0)
    return set_error(PKV_EINVAL, "%s: bad batch, budget, table width or row of sums", who);
  if (desc->num_kv_heads > 65535 || batch > 65535)
    return set_error(PKV_ESHAPE, "%s: batch and kv heads must be <= 65535", who);
  if (budget >= (1ll << 31) - 65536)
    return set_error(PKV_ESHAPE, "%s: a row holds 2^31 positions or more", who);
  if (batch == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !kept || !kept_lens || !new_tables)
    return set_error(PKV_EINVAL, "%s: null pointer", who);
  if (weights && !new_weights)
    return set_error(PKV_EINVAL, "%s: sums need new_weights", who);
  if (weights && weights == new_weights)
    return set_error(PKV_EINVAL, "%s: new_weights must not be weights", who);
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return set_error(PKV_EALIGN, "%s: pools must be 16-byte aligned", who);
  EvictMoveArgs a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.new_tables = new_tables;
  a.kept = kept;
  a.kept_lens = kept_lens;
  a.weights = weights;
  a.new_weights = new_weights;
  a.width = width;
  a.new_width = new_width;
  a.batch = batch;
  a.h_kv = desc->num_kv_heads;
  a.budget = budget;
  a.max_pages = max_pages_per_seq;
  a.new_pages = new_pages_per_seq;
  a.num_pages = desc->num_pages;
  a.row_bytes = desc->head_dim * dtype_bytes(desc->cache_dtype);
  st = error_word(&a.err);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = traced("evict_move", s, [&] { return launch_evict_move(a, s); });
  return cuda_status(e, "evict_move launch");
}

}  // extern "C"
