// Host-side declarations of the paged 8-bit cache (rtp_page_plan,
// rtp_append_q8, rtp_attn_q8).
#pragma once

#include "internal.h"

namespace rtp {

constexpr int kMaxPlanBatch = 4096;  // requests a page plan takes (its scan sits in shared memory)

// Geometry of a pool and its block tables.
struct Q8Pool {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int* status;
  int n_blocks;
  int log_bs;      // log2(block_size)
  int table_cols;  // entries of a block-table row: ceil(max_ctx / block_size)
};

// Rotary axes as the kernels take them.
struct RopeAxes {
  int n_axes;
  unsigned char axis[64];
};

int launch_page_plan(const Shape& sh, int log_bs, int table_cols, const int* ctx_len, const int* new_len,
                     int* block_table, int* free_list, int free_cap, const int* n_free, int* seq_len,
                     int* cu_new, int64_t* slot_map, int* positions, int max_tokens, int* n_free_out,
                     int* status, cudaStream_t st);

int launch_append_q8(const Shape& sh, const Q8Pool& pool, const void* k_pre, int64_t k_stride, const void* v_in,
                     int64_t v_stride, const int64_t* slot_map, const int* pos, const RopeAxes& rope,
                     int n_tokens, cudaStream_t st);

struct AttnQ8Call {
  const void* q_pre;
  int64_t q_stride;
  const int* cu_q;
  const int* seq_len;
  const int* block_table;
  const int* pos;
  int n_tokens, max_q, max_seq_len;
  void* out;
};
size_t attn_q8_workspace_bytes(const Shape& sh, int n_tokens, int max_q);
bool attn_q8_fits(const Shape& sh, int max_q, int max_seq_len);
int launch_attn_q8(const Shape& sh, const Q8Pool& pool, const RopeAxes& rope, const AttnQ8Call& c, void* ws,
                   cudaStream_t st);

}  // namespace rtp
