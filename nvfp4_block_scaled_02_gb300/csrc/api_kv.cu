// api_kv.cu -- the C ABI of the operators around the NVFP4 KV cache: argument
// validation (all synchronous, before anything is enqueued) and dispatch.
#include <cmath>
#include <cstdint>

#include "kv.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool dim_ok(int d) { return d == 64 || d == 128; }
nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }
constexpr int64_t kMaxI32 = INT32_MAX;
constexpr int32_t kMaxHeads = 65536;

// Bytes of a tensor of heads, pages and tokens must stay inside int64 (8 bytes
// per element at most).
bool fits(int64_t a, int64_t b, int64_t c) {
  int64_t n = 0;
  return a >= 0 && b >= 0 && c >= 0 && !__builtin_mul_overflow(a, b, &n) &&
         !__builtin_mul_overflow(n, c, &n) && n <= (INT64_MAX >> 3);
}

nvfp4_status check_rows(const nvfp4_rows& r, int64_t tokens, int64_t heads, int32_t dim) {
  if (heads == 0) return NVFP4_OK;
  if (!r.ptr) return NVFP4_ERR_NULL;
  if (r.stride < heads * dim || r.stride % 8 != 0 || !fits(tokens, r.stride, 1))
    return NVFP4_ERR_SHAPE;
  return aligned(r.ptr, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_cache(const nvfp4_kv_cache* c) {
  if (!c) return NVFP4_ERR_NULL;
  if (!dim_ok(c->head_dim) || c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->page_size < 16 ||
      c->page_size % 16 != 0 || c->pages < 0 ||
      !fits(c->pages, (int64_t)c->page_size * c->kv_heads, c->head_dim) ||
      // rows (a token of a head) are counted in 32 bits: 309 GB of cache at head_dim 64
      c->pages * c->page_size * c->kv_heads > UINT32_MAX)
    return NVFP4_ERR_SHAPE;
  if (c->four_over_six != 0 && c->four_over_six != 1) return NVFP4_ERR_ENUM;
  return NVFP4_OK;
}
nvfp4_status check_cache_ptrs(const nvfp4_kv_cache* c) {
  if (!c->k_amax || !c->v_amax || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
    return NVFP4_ERR_NULL;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16) || !aligned(c->k_amax, 4) || !aligned(c->v_amax, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}
float outer_max(const nvfp4_kv_cache* c) { return c->four_over_six ? 256.0f : 448.0f; }

nvfp4_status check_qk(const nvfp4_qk_config* c) {
  if (!c) return NVFP4_ERR_NULL;
  if (c->tokens < 0 || c->tokens > kMaxI32 || c->q_heads < 0 || c->kv_heads < 0 ||
      c->q_heads > kMaxHeads || c->kv_heads > kMaxHeads || !dim_ok(c->head_dim) ||
      c->rotary_dim < 16 || c->rotary_dim % 16 != 0 || c->rotary_dim > c->head_dim ||
      c->max_pos < 1 || !fits(c->max_pos, c->rotary_dim, 1))
    return NVFP4_ERR_SHAPE;
  if ((c->interleaved != 0 && c->interleaved != 1) || !(c->eps >= 0.0f) || !std::isfinite(c->eps))
    return NVFP4_ERR_ENUM;
  return NVFP4_OK;
}
nvfp4_status check_qk_ptrs(const nvfp4_qk_config* c, int32_t* status) {
  if (!c->positions || !c->cos_sin) return NVFP4_ERR_NULL;
  if (!aligned(c->positions, 4) || !aligned(c->cos_sin, 16) || !aligned(c->q_weight, 16) ||
      !aligned(c->k_weight, 16) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}
void fill_qk(nvfp4::QkRopeParams& p, const nvfp4_qk_config* c, const nvfp4_rows& q,
             const nvfp4_rows& k, const nvfp4_rows& qo, const nvfp4_rows& ko, int32_t* status) {
  p.T = c->tokens;
  p.hq = c->q_heads;
  p.hk = c->kv_heads;
  p.R = c->rotary_dim;
  p.eps = c->eps;
  p.qw = static_cast<const uint4*>(c->q_weight);
  p.kw = static_cast<const uint4*>(c->k_weight);
  p.pos = c->positions;
  p.cs = c->cos_sin;
  p.max_pos = c->max_pos;
  p.q = static_cast<const uint16_t*>(q.ptr);
  p.q_st = q.stride;
  p.k = static_cast<const uint16_t*>(k.ptr);
  p.k_st = k.stride;
  p.qo = static_cast<uint16_t*>(qo.ptr);
  p.qo_st = qo.stride;
  p.ko = static_cast<uint16_t*>(ko.ptr);
  p.ko_st = ko.stride;
  p.status = status;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_plan(const int32_t* cached_len, const int32_t* new_len, int64_t requests,
                           int32_t* block_table, int64_t table_cols, int32_t page_size,
                           const int32_t* free_pages, int64_t free_count, int64_t tokens,
                           int32_t* seq_len, int32_t* q_start, int64_t* slots, int32_t* positions,
                           int32_t* pages_used, int32_t* status, void* stream) {
  if (requests < 0 || requests > kMaxI32 || table_cols < 0 || table_cols > kMaxI32 ||
      page_size < 1 || free_count < 0 || free_count > kMaxI32 || tokens < 0 || tokens > kMaxI32)
    return NVFP4_ERR_SHAPE;
  if (!q_start || !pages_used || (requests > 0 && (!cached_len || !new_len || !seq_len)) ||
      (requests > 0 && table_cols > 0 && !block_table) || (free_count > 0 && !free_pages) ||
      (tokens > 0 && (!slots || !positions)))
    return NVFP4_ERR_NULL;
  if (!aligned(cached_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(seq_len, 4) || !aligned(q_start, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(pages_used, 4) ||
      !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::KvPlanParams p{};
  p.cached = cached_len;
  p.fresh = new_len;
  p.B = (int32_t)requests;
  p.table = block_table;
  p.cols = (int32_t)table_cols;
  p.by_page = nvfp4::make_fastdiv((uint32_t)page_size);
  p.P = page_size;
  p.free_pages = free_pages;
  p.n_free = (int32_t)free_count;
  p.T = (int32_t)tokens;
  p.seq_len = seq_len;
  p.q_start = q_start;
  p.slots = slots;
  p.positions = positions;
  p.used = pages_used;
  p.status = status;
  return cuda_status(nvfp4::launch_kv_plan(p, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_qk_norm_rope(const nvfp4_qk_config* cfg, nvfp4_rows q, nvfp4_rows k,
                                nvfp4_rows q_out, nvfp4_rows k_out, int32_t* status,
                                void* stream) {
  nvfp4_status e = check_qk(cfg);
  if (e != NVFP4_OK) return e;
  if (cfg->tokens == 0 || cfg->q_heads + cfg->kv_heads == 0) return NVFP4_OK;
  if ((e = check_qk_ptrs(cfg, status)) != NVFP4_OK) return e;
  for (const nvfp4_rows* r : {&q, &q_out})
    if ((e = check_rows(*r, cfg->tokens, cfg->q_heads, cfg->head_dim)) != NVFP4_OK) return e;
  for (const nvfp4_rows* r : {&k, &k_out})
    if ((e = check_rows(*r, cfg->tokens, cfg->kv_heads, cfg->head_dim)) != NVFP4_OK) return e;
  nvfp4::QkRopeParams p{};
  fill_qk(p, cfg, q, k, q_out, k_out, status);
  return cuda_status(nvfp4::launch_qk_rope(p, cfg->head_dim, cfg->interleaved != 0,
                                           static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_qk_norm_rope_ws_bytes(void) { return nvfp4::kQkWsBytes; }

nvfp4_status nvfp4_qk_norm_rope_bwd(const nvfp4_qk_config* cfg, nvfp4_rows gq_out,
                                    nvfp4_rows gk_out, nvfp4_rows q, nvfp4_rows k, nvfp4_rows gq,
                                    nvfp4_rows gk, float* gq_weight, float* gk_weight,
                                    void* workspace, size_t ws_bytes, int32_t* status,
                                    void* stream) {
  nvfp4_status e = check_qk(cfg);
  if (e != NVFP4_OK) return e;
  if ((cfg->q_weight == nullptr) != (gq_weight == nullptr) ||
      (cfg->k_weight == nullptr) != (gk_weight == nullptr))
    return NVFP4_ERR_NULL;
  if (!aligned(gq_weight, 4) || !aligned(gk_weight, 4)) return NVFP4_ERR_ALIGN;
  const bool weights = gq_weight || gk_weight;
  if (weights) {
    if (!workspace) return NVFP4_ERR_NULL;
    if (ws_bytes < nvfp4::kQkWsBytes) return NVFP4_ERR_SHAPE;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cfg->tokens == 0 || cfg->q_heads + cfg->kv_heads == 0) {  // sums over nothing
    cudaError_t z = cudaSuccess;
    for (float* w : {gq_weight, gk_weight})
      if (w && z == cudaSuccess)
        z = nvfp4::launch_zero_words(reinterpret_cast<uint32_t*>(w), cfg->head_dim, st);
    return cuda_status(z);
  }
  if ((e = check_qk_ptrs(cfg, status)) != NVFP4_OK) return e;
  for (const nvfp4_rows* r : {&gq_out, &q, &gq})
    if ((e = check_rows(*r, cfg->tokens, cfg->q_heads, cfg->head_dim)) != NVFP4_OK) return e;
  for (const nvfp4_rows* r : {&gk_out, &k, &gk})
    if ((e = check_rows(*r, cfg->tokens, cfg->kv_heads, cfg->head_dim)) != NVFP4_OK) return e;
  nvfp4::QkRopeParams p{};
  fill_qk(p, cfg, q, k, gq, gk, status);
  p.gq = static_cast<const uint16_t*>(gq_out.ptr);
  p.gq_st = gq_out.stride;
  p.gk = static_cast<const uint16_t*>(gk_out.ptr);
  p.gk_st = gk_out.stride;
  p.gqw = gq_weight;
  p.gkw = gk_weight;
  p.ws = static_cast<float*>(workspace);
  return cuda_status(nvfp4::launch_qk_rope_bwd(p, cfg->head_dim, cfg->interleaved != 0, st));
}

nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, nvfp4_rows k, nvfp4_rows v,
                             const int64_t* slots, int64_t tokens, void* k_dq, void* v_dq,
                             int32_t* status, void* stream) {
  nvfp4_status e = check_cache(cache);
  if (e != NVFP4_OK) return e;
  if (tokens < 0 || tokens > kMaxI32) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if ((e = check_cache_ptrs(cache)) != NVFP4_OK) return e;
  if (!slots) return NVFP4_ERR_NULL;
  if (!aligned(slots, 8) || !aligned(k_dq, 16) || !aligned(v_dq, 16) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  for (const nvfp4_rows* r : {&k, &v})
    if ((e = check_rows(*r, tokens, cache->kv_heads, cache->head_dim)) != NVFP4_OK) return e;
  nvfp4::KvAppendParams p{};
  p.x[0] = static_cast<const uint16_t*>(k.ptr);
  p.x[1] = static_cast<const uint16_t*>(v.ptr);
  p.st[0] = k.stride;
  p.st[1] = v.stride;
  p.codes[0] = cache->k_codes;
  p.codes[1] = cache->v_codes;
  p.scales[0] = cache->k_scales;
  p.scales[1] = cache->v_scales;
  p.amax[0] = cache->k_amax;
  p.amax[1] = cache->v_amax;
  p.dq[0] = static_cast<uint4*>(k_dq);
  p.dq[1] = static_cast<uint4*>(v_dq);
  p.slots = slots;
  p.T = tokens;
  p.n_slots = cache->pages * cache->page_size;
  p.H = cache->kv_heads;
  p.P = cache->page_size;
  p.M = outer_max(cache);
  p.status = status;
  return cuda_status(nvfp4::launch_kv_append(p, cache->head_dim, cache->four_over_six != 0,
                                             static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_kv_attention_ws_bytes(void) { return nvfp4::kAttnWsBytes; }

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_cache* cache, const nvfp4_attention_config* cfg,
                                nvfp4_rows q, void* out, float* lse, void* workspace,
                                size_t ws_bytes, int32_t* status, void* stream) {
  nvfp4_status e = check_cache(cache);
  if (e != NVFP4_OK) return e;
  if (!cfg) return NVFP4_ERR_NULL;
  const int64_t group = cfg->q_heads / std::max(cache->kv_heads, 1);
  if (cfg->requests < 0 || cfg->requests > (1 << 30) || cfg->table_cols < 0 ||
      cfg->table_cols > kMaxI32 || cfg->tokens < 0 || cfg->tokens > kMaxI32 || cfg->max_q < 0 ||
      cfg->window < 0 || cfg->q_heads < 1 || cfg->q_heads > kMaxHeads ||
      cfg->q_heads % cache->kv_heads != 0 || cfg->max_q * group > kMaxI32 - 1024 ||
      !fits(cfg->tokens, cfg->q_heads, cache->head_dim) || ws_bytes < nvfp4::kAttnWsBytes)
    return NVFP4_ERR_SHAPE;
  if (!std::isfinite(cfg->scale)) return NVFP4_ERR_ENUM;
  if (cfg->tokens == 0 || cfg->requests == 0) return NVFP4_OK;
  if ((cache->pages > 0 && (e = check_cache_ptrs(cache)) != NVFP4_OK)) return e;
  if (!cache->k_amax || !cache->v_amax || !cfg->seq_len || !cfg->q_start ||
      (cfg->table_cols > 0 && !cfg->block_table) || !out || !workspace)
    return NVFP4_ERR_NULL;
  if (!aligned(cfg->block_table, 4) || !aligned(cfg->seq_len, 4) || !aligned(cfg->q_start, 4) ||
      !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  if ((e = check_rows(q, cfg->tokens, cfg->q_heads, cache->head_dim)) != NVFP4_OK) return e;
  nvfp4::KvAttnParams p{};
  p.kc = cache->k_codes;
  p.ks = cache->k_scales;
  p.vc = cache->v_codes;
  p.vs = cache->v_scales;
  p.k_amax = cache->k_amax;
  p.v_amax = cache->v_amax;
  p.M = outer_max(cache);
  p.pages = cache->pages;
  p.hk = cache->kv_heads;
  p.P = cache->page_size;
  p.page_shift = (p.P & (p.P - 1)) == 0 ? __builtin_ctz((unsigned)p.P) : -1;
  p.by_page = nvfp4::make_fastdiv((uint32_t)p.P);
  p.table = cfg->block_table;
  p.seq_len = cfg->seq_len;
  p.q_start = cfg->q_start;
  p.B = (int32_t)cfg->requests;
  // a cache without pages holds no token: every length but 0 is past its table
  p.cols = cache->pages > 0 ? (int32_t)cfg->table_cols : 0;
  p.T = (int32_t)cfg->tokens;
  p.hq = cfg->q_heads;
  p.G = (int32_t)group;
  p.by_group = nvfp4::make_fastdiv((uint32_t)group);
  p.max_q = cfg->max_q;
  p.window = cfg->window;
  p.scale = cfg->scale;
  p.q = static_cast<const uint16_t*>(q.ptr);
  p.q_st = q.stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.tickets = static_cast<uint32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                    (size_t)nvfp4::kAttnTickets * 4);
  p.status = status;
  // The requests share the call, their row counts are on the device: each kernel
  // takes the requests that are its own, and the one for many rows is launched
  // only if max_q allows such a request.
  p.few_rows = nvfp4::kAttnRows;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t ce = nvfp4::launch_kv_few(p, cache->head_dim, st);
  if (ce == cudaSuccess && cfg->max_q * group > p.few_rows)
    ce = nvfp4::launch_kv_prefill(p, cache->head_dim, st);
  return cuda_status(ce);
}

}  // extern "C"
