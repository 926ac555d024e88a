// C ABI of the paged 8-bit cache (include/rtp.h): argument validation and
// dispatch.  No allocation, no synchronisation.
#include <cstdint>
#include <string>

#include "q8.h"

namespace rtp {
namespace {

int fail(int code, const std::string& msg) {
  set_error(msg);
  return code;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int log2_block(int block_size, int* log_bs) {
  for (int l = 4; l <= 7; ++l)
    if (block_size == 1 << l) {
      *log_bs = l;
      return RTP_OK;
    }
  return fail(RTP_ERR_SHAPE, "block_size must be 16, 32, 64 or 128");
}

// The layer's shape, and what a paged cache asks of the configuration.
int q8_shape(const rtp_layer_cfg* cfg, int block_size, Shape* sh, int* log_bs) {
  int rc = make_shape(cfg, sh);
  if (rc != RTP_OK) return rc;
  if (cfg->top_p != 1.0f || cfg->top_k != 0 || cfg->local_cap != 0)
    return fail(RTP_ERR_SHAPE, "the paged cache takes no selection and no ring: top_p must be 1, top_k and local_cap 0");
  return log2_block(block_size, log_bs);
}

int q8_pool(const Shape& sh, const rtp_q8_cache* c, int log_bs, Q8Pool* pool) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->status)
    return fail(RTP_ERR_INVALID, "cache k/v/k_scale/v_scale/status is NULL");
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return fail(RTP_ERR_INVALID, "cache buffers must be 16-byte aligned");
  if (c->n_blocks < 1 || (((long long)c->n_blocks * sh.Hkv) << log_bs) > INT32_MAX)
    return fail(RTP_ERR_SHAPE, "n_blocks must be >= 1 and n_blocks * n_kv_heads * block_size below 2^31");
  pool->k = c->k;
  pool->v = c->v;
  pool->k_scale = c->k_scale;
  pool->v_scale = c->v_scale;
  pool->status = c->status;
  pool->n_blocks = c->n_blocks;
  pool->log_bs = log_bs;
  pool->table_cols = (sh.Lmax + c->block_size - 1) >> log_bs;
  return RTP_OK;
}

int rope_axes(const Shape& sh, const rtp_rope_axes* r, RopeAxes* out) {
  for (int k = 0; k < 64; ++k) out->axis[k] = 0;
  out->n_axes = 1;
  if (!r) return RTP_OK;
  if (r->n_axes < 1 || r->n_axes > 4) return fail(RTP_ERR_SHAPE, "n_axes must be in [1, 4]");
  out->n_axes = r->n_axes;
  for (int k = 0; k < sh.D / 2; ++k) {
    if (r->axis[k] >= r->n_axes) return fail(RTP_ERR_SHAPE, "a rotary pair's axis must be below n_axes");
    out->axis[k] = r->axis[k];
  }
  return RTP_OK;
}

// Elements between tokens' rows: 0 means dense.
int row_stride(const Shape& sh, int64_t given, int heads, const char* name, int64_t* out) {
  const int64_t dense = (int64_t)heads * sh.D;
  *out = given == 0 ? dense : given;
  if (*out < dense || *out * sh.esize % 16 != 0 || *out > (1ll << 40))
    return fail(RTP_ERR_SHAPE, std::string(name) + " must be 0, or at least heads * head_dim and a multiple of 16 bytes");
  return RTP_OK;
}

int attn_bounds(const Shape& sh, int n_tokens, int max_q, int* max_seq_len) {
  if (n_tokens < 0) return fail(RTP_ERR_SHAPE, "n_tokens must be >= 0");
  if (max_q < 1 || max_q > sh.Lmax) return fail(RTP_ERR_SHAPE, "max_q must be in [1, max_ctx]");
  if (*max_seq_len < 0 || *max_seq_len > sh.Lmax) return fail(RTP_ERR_SHAPE, "max_seq_len must be in [0, max_ctx]");
  if (*max_seq_len == 0) *max_seq_len = sh.Lmax;
  if (!attn_q8_fits(sh, max_q, *max_seq_len))
    return fail(RTP_ERR_SHAPE, "batch * n_kv_heads * query row chunks * (ceil(max_seq_len / 32) + 16) must stay below 2^31");
  return RTP_OK;
}

}  // namespace
}  // namespace rtp

using namespace rtp;

extern "C" {

int rtp_q8_cache_bytes(const rtp_layer_cfg* cfg, int n_blocks, int block_size, size_t* kv_bytes, size_t* scale_bytes) {
  Shape sh;
  int log_bs, rc = q8_shape(cfg, block_size, &sh, &log_bs);
  if (rc != RTP_OK) return rc;
  if (n_blocks < 1 || (((long long)n_blocks * sh.Hkv) << log_bs) > INT32_MAX)
    return fail(RTP_ERR_SHAPE, "n_blocks must be >= 1 and n_blocks * n_kv_heads * block_size below 2^31");
  if (kv_bytes) *kv_bytes = (((size_t)n_blocks * sh.Hkv) << log_bs) * sh.D;
  if (scale_bytes) *scale_bytes = (size_t)n_blocks * sh.Hkv * sizeof(float);
  return RTP_OK;
}

int rtp_page_plan(const rtp_layer_cfg* cfg, int block_size, const int* ctx_len, const int* new_len,
                  int* block_table, int* free_list, int free_cap, const int* n_free, int* seq_len,
                  int* cu_new, int64_t* slot_map, int* positions, int max_tokens, int* n_free_out,
                  int* status, void* stream) {
  Shape sh;
  int log_bs, rc = q8_shape(cfg, block_size, &sh, &log_bs);
  if (rc != RTP_OK) return rc;
  if (sh.B > kMaxPlanBatch) return fail(RTP_ERR_SHAPE, "a page plan takes at most 4096 requests");
  if (max_tokens < 0 || max_tokens > (1 << 30)) return fail(RTP_ERR_SHAPE, "max_tokens must be in [0, 2^30]");
  if (free_cap < 0 || free_cap > (1 << 30)) return fail(RTP_ERR_SHAPE, "free_cap must be in [0, 2^30]");
  if (!ctx_len || !new_len || !block_table || !n_free || !seq_len || !cu_new || !n_free_out || !status ||
      (free_cap > 0 && !free_list) || (max_tokens > 0 && (!slot_map || !positions)))
    return fail(RTP_ERR_INVALID, "a page plan buffer is NULL");
  if ((max_tokens > 0 && (!aligned16(slot_map) || !aligned16(positions))))
    return fail(RTP_ERR_INVALID, "slot_map and positions must be 16-byte aligned");
  const int cols = (sh.Lmax + block_size - 1) >> log_bs;
  return launch_page_plan(sh, log_bs, cols, ctx_len, new_len, block_table, free_list, free_cap, n_free, seq_len,
                          cu_new, slot_map, positions, max_tokens, n_free_out, status, (cudaStream_t)stream);
}

int rtp_append_q8(const rtp_layer_cfg* cfg, const rtp_q8_cache* cache, const void* k_pre, int64_t k_stride,
                  const void* v_in, int64_t v_stride, const int64_t* slot_map, const int* pos,
                  const rtp_rope_axes* rope, int n_tokens, void* stream) {
  if (!cache) return fail(RTP_ERR_INVALID, "cache is NULL");
  Shape sh;
  int log_bs, rc = q8_shape(cfg, cache->block_size, &sh, &log_bs);
  if (rc != RTP_OK) return rc;
  Q8Pool pool;
  if ((rc = q8_pool(sh, cache, log_bs, &pool)) != RTP_OK) return rc;
  RopeAxes axes;
  if ((rc = rope_axes(sh, rope, &axes)) != RTP_OK) return rc;
  if (n_tokens < 0) return fail(RTP_ERR_SHAPE, "n_tokens must be >= 0");
  if ((rc = row_stride(sh, k_stride, sh.Hkv, "k_stride", &k_stride)) != RTP_OK) return rc;
  if ((rc = row_stride(sh, v_stride, sh.Hkv, "v_stride", &v_stride)) != RTP_OK) return rc;
  if (n_tokens == 0) return RTP_OK;
  if (!k_pre || !v_in || !slot_map || !pos) return fail(RTP_ERR_INVALID, "k_pre/v_in/slot_map/pos is NULL");
  if (!aligned16(k_pre) || !aligned16(v_in)) return fail(RTP_ERR_INVALID, "k_pre and v_in must be 16-byte aligned");
  return launch_append_q8(sh, pool, k_pre, k_stride, v_in, v_stride, slot_map, pos, axes, n_tokens,
                          (cudaStream_t)stream);
}

int rtp_attn_q8_workspace_bytes(const rtp_layer_cfg* cfg, int block_size, int n_tokens, int max_q, int max_seq_len,
                                size_t* bytes) {
  Shape sh;
  int log_bs, rc = q8_shape(cfg, block_size, &sh, &log_bs);
  if (rc != RTP_OK) return rc;
  if (!bytes) return fail(RTP_ERR_INVALID, "bytes is NULL");
  if ((rc = attn_bounds(sh, n_tokens, max_q, &max_seq_len)) != RTP_OK) return rc;
  *bytes = attn_q8_workspace_bytes(sh, n_tokens, max_q);
  return RTP_OK;
}

int rtp_attn_q8(const rtp_layer_cfg* cfg, const rtp_q8_cache* cache, const void* q_pre, int64_t q_stride,
                const int* cu_q, const int* seq_len, const int* block_table, const int* pos,
                const rtp_rope_axes* rope, int n_tokens, int max_q, int max_seq_len, void* out,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache) return fail(RTP_ERR_INVALID, "cache is NULL");
  Shape sh;
  int log_bs, rc = q8_shape(cfg, cache->block_size, &sh, &log_bs);
  if (rc != RTP_OK) return rc;
  Q8Pool pool;
  if ((rc = q8_pool(sh, cache, log_bs, &pool)) != RTP_OK) return rc;
  RopeAxes axes;
  if ((rc = rope_axes(sh, rope, &axes)) != RTP_OK) return rc;
  if ((rc = attn_bounds(sh, n_tokens, max_q, &max_seq_len)) != RTP_OK) return rc;
  if ((rc = row_stride(sh, q_stride, sh.Hq, "q_stride", &q_stride)) != RTP_OK) return rc;
  if (n_tokens == 0) return RTP_OK;
  if (!q_pre || !cu_q || !seq_len || !block_table || !pos || !out)
    return fail(RTP_ERR_INVALID, "q_pre/cu_q/seq_len/block_table/pos/out is NULL");
  if (!aligned16(q_pre) || !aligned16(out)) return fail(RTP_ERR_INVALID, "q_pre and out must be 16-byte aligned");
  if (!workspace) return fail(RTP_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(RTP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (workspace_bytes < attn_q8_workspace_bytes(sh, n_tokens, max_q))
    return fail(RTP_ERR_WORKSPACE, "workspace smaller than rtp_attn_q8_workspace_bytes");
  AttnQ8Call c;
  c.q_pre = q_pre; c.q_stride = q_stride; c.cu_q = cu_q; c.seq_len = seq_len; c.block_table = block_table;
  c.pos = pos; c.n_tokens = n_tokens; c.max_q = max_q; c.max_seq_len = max_seq_len; c.out = out;
  return launch_attn_q8(sh, pool, axes, c, workspace, (cudaStream_t)stream);
}

}  // extern "C"
