// What the two attention kernels of the paged 8-bit cache share: the streaming
// kernel (attn_q8.cu) and the chunk kernel (attn_q8_tc.cu).
#pragma once

#include <cuda.h>  // CUtensorMap

#include "q8.cuh"

namespace rtp {

constexpr float kAqRescale = 8.f;  // the running maximum moves when a tile exceeds it by 2^8
constexpr float kAqLift = 6.f;     // weights are held 2^6 up (at most 2^14 in fp16), away from fp16's small end
// Value scales lie up to 2^185 apart.  A weight that vanishes beside another's scale,
// 2^(x - M) = 0, may still have its share of l, w / vs: where a tile's scales lie more
// than 2^64 below the largest that M may hold, the tile adds to l from the logits
// without the scales.  (Nearer ones lose less than 2^-44 of l: M is at most the largest
// logit plus log2 of that scale, so a weight that vanishes is below 2^-67 of the largest.)
// l is held 2^24 up besides, which keeps its ends, 2^-115 for the largest scale and
// 2^101 for 2^23 positions of the least, away from fp32's.
constexpr float kAqFar = 64.f;
constexpr float kAqSumLift = 24.f;
constexpr float kAqSumUnit = 16777216.f;  // 2^24

// 256 query rows of one (request, KV head): row r is token (row0 + r) / G of
// the request, at position i0 + that, and query head (row0 + r) % G of the
// group.  Its tiles of 128 positions are [0, ns) and from w0 on.
struct __align__(16) ChunkItem {
  int b, h, row0, n_rows;
  int q0, i0, i_hi, tiles;  // first packed row, its position; position of the item's last row
  int ns, w0, ret, pad;
};

// An item that the cut behind a CTA's share goes through first: its partials
// lie in slots [slot0, slot0 + np); np = 0: there is none.
struct __align__(16) JoinJob {
  int np, n_rows;
  uint32_t slot0;
  int h, row0, q0, pad0, pad1;
};

struct __align__(64) AttnQ8Args {
  // first what every CTA reads at once (each line of the parameters misses at a kernel's start)
  AttnQ8Call c;
  Q8Pool pool;
  int B, Hq, Hkv, G, S, W, rows;
  int log_g;          // G is a power of two
  int small_rows;     // requests of more query rows (n G) a KV head go to the chunk kernel
  uint32_t n_slots;   // partials that the workspace holds
  uint64_t ret_mask;
  float* part;        // [n_slots][rows][D] O, and (M, l)
  float* part_ml;
  JoinJob* jobs;  // [CTAs] what each cut of the line leaves to join
  unsigned long long wait_ns;
  // the chunk kernel's share of the workspace
  ChunkItem* items;
  long long* prefix;  // units of the line ahead of each item, then their number; [max_chunk_items + 1]: a CTA's share of them
  int* req_items;     // [B + 1] items ahead of each request
  float* cpart;       // partials of cut items: [2 CTAs][D / 4][256][4], and (M, l)
  float* cpart_ml;
  int max_chunk_items;
  __half* cq;         // rotated queries, [n_tokens][Hq][D], each row by its power-of-two scale
  float* cq_unit;     // [n_tokens][Hq]: from their products to base-2 logits
  uint64_t turns[64]; // rotary frequencies
  RopeAxes rope;
  CUtensorMap tm_k, tm_v;    // the pool as [n_blocks Hkv block_size][D] bytes, boxes of min(32, block_size) rows
  CUtensorMap tm_q;          // cq, boxes of 64 dims x G heads x 128 / G tokens
  CUtensorMap tm_ck, tm_cv;  // the pool as rows of D bytes, boxes of min(128, block_size) rows
};

// First packed row, number of queries and cached positions of request b;
// n = 0 where it has nothing to do or is refused (`flags`).
struct ReqRows {
  int q0, n, L;
};

__device__ __forceinline__ ReqRows load_rows(const AttnQ8Args& a, int b, int& flags) {
  const int q0 = a.c.cu_q[b], q1 = a.c.cu_q[b + 1], L = a.c.seq_len[b];
  const long long n = (long long)q1 - q0;
  if (n < 0 || n > a.c.max_q || q0 < 0 || q1 > a.c.n_tokens) {
    flags |= RTP_DEV_POSITION;
    return ReqRows{0, 0, 0};
  }
  if (n == 0) return ReqRows{0, 0, 0};
  if (L < n || L > a.c.max_seq_len) {
    flags |= RTP_DEV_SEQ_LEN;
    return ReqRows{0, 0, 0};
  }
  return ReqRows{q0, (int)n, L};
}

// Factor 2^e that brings a query row's largest magnitude m into [2^8, 2^9), so
// that neither fp16's largest value nor its smallest step is in the way; not below
// 2^least, which rows of m < 2^(least + 8) are left under.  At -118 the factor's
// reciprocal is still a normal number.
template <int least>
__device__ __forceinline__ float query_scale(float m) {
  int e = (int)(__float_as_uint(m) >> 23) - 127 - 8;
  e = m == 0.f ? 0 : min(max(e, least), 119);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// l 2^d, d <= 0, in two steps: 2^d alone may vanish where the product does not.
__device__ __forceinline__ float lower(float l, float d) {
  const float e = fmaxf(d, -120.f);
  return l * ex2f(e) * ex2f(d - e);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// out = O / l of one row element (l held 2^24 up).
template <typename T>
__device__ __forceinline__ T finish(float o, float l) {
  return from_f32<T>(l == 0.f ? 0.f : o * kAqSumUnit / l);  // l = 0: no position of the row is there
}

// The chunk kernel (bf16 layers): workspace, and its launches for the requests
// of more than a.small_rows query rows a KV head.
size_t chunk_workspace_bytes(const Shape& sh, int n_tokens, int max_q, int small_rows);
bool chunk_carve(const Shape& sh, int n_tokens, int max_q, int small_rows, void* ws, AttnQ8Args* a);
cudaError_t launch_attn_q8_chunks(const Shape& sh, const AttnQ8Args& a, cudaStream_t st);

}  // namespace rtp
