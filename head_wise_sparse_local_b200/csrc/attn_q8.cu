// rtp_attn_q8 for few queries a request (decode, drafts to verify): one stream
// over the paged 8-bit cache.
//
// Mathematics.  A query row (token t, query head g of a KV head's group) at
// position i attends to the positions its head sees; with the stored e4m3
// values k', v' and their block's scales ks, vs
//   x_j = q.k'_j ks / sqrt(D) log2(e) + log2(vs),   w_j = 2^(x_j - M),
//   O = sum_j w_j v'_j,   l = sum_j w_j / vs_j,   out = O / l.
// Taking vs into the exponent keeps the value blocks' scales out of the
// products; M is the running maximum of x, moved only when a tile exceeds it by
// 2^8, so weights are at most 2^8 whatever the scales are, and 2^14 as held in
// fp16 (2^6 up), whose largest is 2^16 less 32.  l is another matter: see kAqFar.
//
// Work.  A tile is 32 positions of one (request, KV head, row chunk) item.  All
// tiles of all items, and some units an item for its start and end, form one
// line that is cut into equal shares, one for each CTA (two an SM), so ragged
// batches and the short local heads load the SMs evenly; an item that a cut goes through leaves one partial (O, M, l) a
// CTA, and a second kernel joins them in order, from a note that the item's
// first CTA leaves it (finding the items anew cost it 4 us at 128K; a join by
// the CTA that arrives last, counted by compare-and-swap so that the workspace
// needs no clearing, 30 us for 70 CTAs an item).  Inside a CTA each of 4 warps
// takes every fourth tile and keeps its own softmax state and accumulators;
// they meet once an item.
//
// A warp stages its own tiles (K and V, 2 x 32 x D bytes) three deep by TMA,
// which also swizzles the rows for conflict-free reads; there is no barrier
// between warps in the loop.  Products are mma.sync m16n8k16 in fp16: e4m3
// values convert to fp16 exactly, one instruction for two.  S = Q K^T takes Q
// as the 16-row operand: 8 rows as a high and a low fp16 part (22 bits), or 16
// rows in one part where there are more.  Its accumulator layout is the layout
// the second product wants the weights in, O^T = V^T W^T with V^T read
// transposed by byte-wise ldmatrix.
//
// Bound: memory.  128 positions of K and V are 32 KB; at 6.5 TB/s an SM gets
// 23 B a clock, so 1400 clocks; the products are 192 mma.sync of 2 clocks each and 512
// conversions of about 1 clock.  (tcgen05 would spend as long: its 128-row operand would be
// 8 or 16 rows full.)
//
// Measured, 32 query / 8 KV heads, D = 128, bf16, both kernels of a call in a
// replayed graph (a call from a host program that makes one after another takes 1
// to 3 us more): one request at 1M positions 92.5 us (543 MB, 5.9 TB/s, 90% of a
// copy's rate), at 128K 20.7 us (70 MB); 8 requests of 8K to 32K positions 24.8 us
// (95 MB), as drafts 39.2 us (16 rows a chunk, so their tiles are read twice).
// Value scales of any size cost 0.2 of the 24.8 and 0.6 of the 39.2.
#include "attn_q8.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace rtp {
namespace {

constexpr int kAqWarps = 4;
constexpr int kAqThreads = kAqWarps * 32;
constexpr int kAqTile = 32;   // positions a tile
constexpr int kAqStages = 3;  // tiles in flight a warp
// Units of the line after an item's tiles: its start and end cost about as much as so many
// tiles (none: 27.2 us for 8 requests of 8K to 32K, 43.1 for drafts there; 8: 25.1 and 40.8;
// 16: 24.2 and 38.6; 28: 25.4 and 39.6).
constexpr int kAqItemCost = 16;
constexpr int kAqCtasPerSm = 2;
constexpr int kAqMaxCtas = 148 * kAqCtasPerSm;  // every SM of a B200

// A request's queries and tiles.
struct ReqQ8 {
  int q0, n, L;   // first packed row, queries, cached positions
  int rc;         // row chunks
  int tr, tl;     // tiles of a retrieval and of a local KV head
  int ns, w0;     // a local head's tiles: [0, ns) and [w0, tr)
  __device__ __forceinline__ uint32_t units(int R, int Hkv) const {  // of the line
    return (uint32_t)rc * (uint32_t)(R * tr + (Hkv - R) * tl + Hkv * kAqItemCost);
  }
};

__device__ __forceinline__ ReqQ8 load_req(const AttnQ8Args& a, int b, int& flags) {
  ReqQ8 r = {};
  const ReqRows x = load_rows(a, b, flags);
  if (x.n == 0 || (long long)x.n * a.G > a.small_rows) return r;
  const int L = x.L;
  r.q0 = x.q0;
  r.n = x.n;
  r.L = L;
  r.rc = (x.n * a.G + a.rows - 1) / a.rows;
  r.tr = (L - 1) / kAqTile + 1;
  r.ns = min((a.S + kAqTile - 1) / kAqTile, r.tr);
  r.w0 = max(0, L - r.n - a.W + 1) / kAqTile;
  if (r.w0 <= r.ns) {
    r.ns = r.w0 = 0;
    r.tl = r.tr;
  } else {
    r.tl = r.ns + r.tr - r.w0;
  }
  return r;
}

// Units a CTA takes: an equal share of the line, at least one a warp, or the
// items' mean where that is less (short contexts: four one-tile items after one
// another took 16 us where a CTA each takes 7).
__device__ __forceinline__ uint32_t share_of(uint32_t total, uint32_t items) {
  return max((total + kAqMaxCtas - 1) / kAqMaxCtas, min((uint32_t)kAqWarps, total / max(items, 1u) - kAqItemCost));
}

// Where position `part` * share of the line lies (every warp for itself): its
// request, and the units and items ahead of that.  b < 0: past the end.
struct LineAt {
  int b;
  uint32_t at, share, total, units, items;
};

__device__ __forceinline__ LineAt locate(const AttnQ8Args& a, uint32_t part, int& flags) {
  const int lane = threadIdx.x & 31, R = __popcll(a.ret_mask);
  LineAt p = {-1, 0u, 0u, 0u, 0u, 0u};
  auto sums = [&](int b0, uint32_t& t, uint32_t& it, uint32_t& ts, uint32_t& is) {
    ReqQ8 r = {};
    if (b0 + lane < a.B) r = load_req(a, b0 + lane, flags);
    t = r.units(R, a.Hkv);
    it = (uint32_t)(r.rc * a.Hkv);
    ts = warp_incl_scan_u32(t);
    is = warp_incl_scan_u32(it);
  };
  uint32_t t, it, ts, is;
  sums(0, t, it, ts, is);
  p.total = __shfl_sync(0xffffffffu, ts, 31);
  uint32_t all_items = __shfl_sync(0xffffffffu, is, 31);
  for (int b0 = 32; b0 < a.B; b0 += 32) {
    uint32_t t2, it2, ts2, is2;
    sums(b0, t2, it2, ts2, is2);
    p.total += __shfl_sync(0xffffffffu, ts2, 31);
    all_items += __shfl_sync(0xffffffffu, is2, 31);
  }
  p.share = share_of(p.total, all_items);
  p.at = part * p.share;
  if (p.at >= p.total) return p;
  for (int b0 = 0;;) {
    const unsigned m = __ballot_sync(0xffffffffu, p.units + ts > p.at);
    if (m) {
      const int l = __ffs(m) - 1;
      p.b = b0 + l;
      p.units += __shfl_sync(0xffffffffu, ts - t, l);
      p.items += __shfl_sync(0xffffffffu, is - it, l);
      return p;
    }
    p.units += __shfl_sync(0xffffffffu, ts, 31);
    p.items += __shfl_sync(0xffffffffu, is, 31);
    b0 += 32;
    sums(b0, t, it, ts, is);
  }
}

// The item at `rel` units into a request: its KV head and row chunk; `rel`
// becomes the tile's number in it (not below nt in the units after its tiles).
struct ItemAt {
  int h, rch, nt;  // nt: its tiles
};
__device__ __forceinline__ ItemAt item_at(const AttnQ8Args& a, const ReqQ8& r, uint32_t& rel) {
  ItemAt x = {0, 0, 0};
  for (;; ++x.h) {
    x.nt = (a.ret_mask >> x.h) & 1ull ? r.tr : r.tl;
    const uint32_t all = (uint32_t)((x.nt + kAqItemCost) * r.rc);
    if (rel < all) break;
    rel -= all;
  }
  if (r.rc > 1) {
    const uint32_t each = (uint32_t)(x.nt + kAqItemCost);
    x.rch = (int)(rel / each);
    rel -= (uint32_t)x.rch * each;
  }
  return x;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two 16 x 16 byte matrices, transposed: rows at the 32 lanes' addresses (16
// bytes each, lanes 0-15 the first matrix).  Lane l gets of each matrix the
// bytes of rows 4 (l % 4) .. + 3 in columns l / 4 and l / 4 + 8.
__device__ __forceinline__ void ldsm_b8_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// What a tile's consumers need beside its rows; the scales arrive by cp.async.
struct __align__(16) TileMeta {
  float ks[2], vs[2];  // scales of its first and second 16 positions
  int there;           // bit q: those 16 positions' block is in the pool
};

template <int D, int ROWS>
struct AqSmem {
  static constexpr int kStage = 2 * kAqTile * D;                       // K, then V
  static constexpr int kRing = kAqWarps * kAqStages * kStage;
  static constexpr int kQPitch = D + 4;
  static constexpr int kOffQ = kRing;                                  // rotated queries, fp32
  static constexpr int kOffMeta = kOffQ + ROWS * kQPitch * 4;
  static constexpr int kBytes = kOffMeta + kAqWarps * kAqStages * (int)sizeof(TileMeta) + 1024;
  static constexpr int kMPitch = D + 4;                                // joining the warps: O rows, M, l (over the ring)
  static_assert(kAqWarps * ROWS * kMPitch * 4 <= kRing, "the warps' partials fit in the ring");
};

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kAqThreads, kAqCtasPerSm) attn_q8_kernel(const __grid_constant__ AttnQ8Args a) {
  using SM = AqSmem<D, ROWS>;
  constexpr bool kTwoParts = ROWS == 8;          // queries as high + low fp16 parts
  constexpr bool kWLow = sizeof(T) == 4;         // weights as well (fp32 layers)
  constexpr int NR = ROWS / 8;                   // rows a lane quad holds scores of; column groups of O^T
  constexpr int KS = D / 16;
  static_assert(!kWLow || kTwoParts, "fp32 layers run 8 rows");
  extern __shared__ __align__(1024) unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t s_bar[kAqWarps][kAqStages];
  __shared__ float s_qs[ROWS];  // per row: factor from products to base-2 logits
  __shared__ int s_abort;
  __shared__ uint64_t s_turns[D / 2];  // (lanes that index the parameters apart are served one by one)
  __shared__ int s_axis[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  unsigned char* dsm = dsm_raw + ((1024u - (smem_u32(dsm_raw) & 1023u)) & 1023u);
  unsigned char* ring = dsm + warp * kAqStages * SM::kStage;
  float* s_q = reinterpret_cast<float*>(dsm + SM::kOffQ);
  TileMeta* meta = reinterpret_cast<TileMeta*>(dsm + SM::kOffMeta) + warp * kAqStages;
  uint64_t* bar = s_bar[warp];
  if (tid == 0) {
    // two arrivals a phase: the copies' expect_tx and the scales' cp.async
    for (int w = 0; w < kAqWarps; ++w)
      for (int s = 0; s < kAqStages; ++s) mbar_init(&s_bar[w][s], 2);
    s_abort = 0;
  }
  if (tid < D / 2) {
    s_turns[tid] = a.turns[tid];
    s_axis[tid] = a.rope.n_axes > 1 ? a.rope.axis[tid] : 0;
  }
  __syncthreads();
  griddep_wait();
  griddep_launch();

  const int R = __popcll(a.ret_mask);
  int flags = 0;
  LineAt line = locate(a, blockIdx.x, flags);
  if (blockIdx.x == 0 && warp == 0 && flags) atomicOr(a.pool.status, flags);
  flags = 0;
  JoinJob job = {};
  if (line.b < 0) {  // uniform
    if (tid == 0) a.jobs[blockIdx.x] = job;
    return;
  }
  uint32_t at = line.at;
  const uint32_t end = min(line.total, at + line.share);
  int b = line.b;

  const uint64_t pol = l2_evict_first();
  const int bs1 = (1 << a.pool.log_bs) - 1;
  const bool split = a.pool.log_bs == 4;  // a tile is two blocks
  int st = 0;        // ring position of the next tile to consume,
  uint32_t ph = 0u;  // and its phase
  ReqQ8 rq = load_req(a, b, flags);

  while (at < end) {
    // ---- the segment: tiles [u0, u1) of item (b, h, rch) ----
    uint32_t rel = at - line.units;
    while (rel >= rq.units(R, a.Hkv)) {  // on to the next request that has tiles
      line.units += rq.units(R, a.Hkv);
      line.items += (uint32_t)(rq.rc * a.Hkv);
      rel = at - line.units;
      rq = load_req(a, ++b, flags);
    }
    const ItemAt x = item_at(a, rq, rel);
    const int h = x.h, rch = x.rch, nt = x.nt;
    const uint32_t next = at + (uint32_t)(nt + kAqItemCost) - rel;  // the next item
    if (rel >= (uint32_t)nt) {
      at = next;
      continue;
    }
    const bool ret = (a.ret_mask >> h) & 1ull;
    const int u0 = (int)rel;
    const int u1 = (int)min((uint32_t)nt, rel + (end - at));
    const uint32_t item = line.items + (uint32_t)(h * rq.rc + rch);
    const int row0 = rch * ROWS, n_rows = min(ROWS, rq.n * a.G - row0);
    const int i0 = rq.L - rq.n;                            // position of the request's first query
    const int i_lo = i0 + (row0 >> a.log_g), i_hi = i0 + ((row0 + n_rows - 1) >> a.log_g);  // of this chunk's rows
    const int* tab = a.c.block_table + (size_t)b * a.pool.table_cols;
    const int mine = u0 + warp < u1 && !s_abort ? (u1 - u0 - warp + kAqWarps - 1) / kAqWarps : 0;  // this warp's tiles

    auto tile_key = [&](int n) {  // first position of the warp's n-th tile
      const int u = u0 + warp + n * kAqWarps;
      return (ret || u < rq.ns ? u : rq.w0 + u - rq.ns) * kAqTile;
    };
    // ids of the blocks of a tile's two halves (lane 0)
    auto block_ids = [&](int n, int (&id)[2]) {
      const int j0 = tile_key(n);
      const int c0 = j0 >> a.pool.log_bs;
      id[0] = tab[c0];
      id[1] = split ? (j0 + 16 < rq.L ? tab[c0 + 1] : -1) : id[0];
    };
    auto issue = [&](int n, int s, const int (&id)[2]) {  // one lane: tile n into ring stage s
      const int j0 = tile_key(n);
      int there = 0, y[2], blk[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = (unsigned)id[q] < (unsigned)a.pool.n_blocks;
        if (!in && j0 + 16 * q < rq.L) flags |= RTP_DEV_BLOCKS;
        there |= (in ? 1 : 0) << q;
        blk[q] = in ? id[q] : 0;
        y[q] = ((blk[q] * a.Hkv + h) << a.pool.log_bs) + (split ? 0 : j0 & bs1);
      }
      TileMeta* m = meta + s;
      m->there = there;
      unsigned char* dst = ring + s * SM::kStage;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const size_t bh = (size_t)blk[q] * a.Hkv + h;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(&m->ks[q])), "l"(a.pool.k_scale + bh) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(&m->vs[q])), "l"(a.pool.v_scale + bh) : "memory");
      }
      cp_async_arrive_noinc(&bar[s]);
      mbar_expect_tx(&bar[s], (uint32_t)SM::kStage);
      tma_load_2d(dst, &a.tm_k, 0, y[0], &bar[s], pol);
      if (split) tma_load_2d(dst + 16 * D, &a.tm_k, 0, y[1], &bar[s], pol);
      tma_load_2d(dst + kAqTile * D, &a.tm_v, 0, y[0], &bar[s], pol);
      if (split) tma_load_2d(dst + kAqTile * D + 16 * D, &a.tm_v, 0, y[1], &bar[s], pol);
    };
    // ---- queries: asked for before the stream's copies, which fill the memory system for
    // microseconds; a thread turns a rotary pair of all the chunk's rows of one token ----
    const int tok0 = row0 >> a.log_g, n_tok = ((row0 + n_rows - 1) >> a.log_g) - tok0 + 1;
    struct Pair {
      uint64_t turns;
      int pos, ra, rb;     // rows [ra, rb) of the chunk
      float x1[8], x2[8];  // a token has at most 8 rows
    };
    auto load_pair = [&](int task, Pair& y) {
      const int tl = task / (D / 2), k = task % (D / 2), tok = rq.q0 + tok0 + tl;
      y.turns = s_turns[k];
      y.pos = a.c.pos[(size_t)s_axis[k] * a.c.n_tokens + tok];
      y.ra = max(((tok0 + tl) << a.log_g) - row0, 0);
      y.rb = min(((tok0 + tl + 1) << a.log_g) - row0, n_rows);
      const T* q = static_cast<const T*>(a.c.q_pre) + (size_t)tok * a.c.q_stride +
                   (size_t)(h * a.G + ((row0 + y.ra) & (a.G - 1))) * D + k;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (y.ra + r < y.rb) {
          y.x1[r] = to_f32(q[(size_t)r * D]);
          y.x2[r] = to_f32(q[(size_t)r * D + D / 2]);
        }
    };
    Pair pair;
    if (tid < n_tok * (D / 2)) load_pair(tid, pair);

    // the first tiles, a lane each, so that their block numbers are read at once
    if (lane < kAqStages && lane < mine) {
      int id[2], s = st + lane;
      block_ids(lane, id);
      issue(lane, s >= kAqStages ? s - kAqStages : s, id);
    }
    int next_id[2] = {0, 0};  // blocks of the next tile to issue
    if (lane == 0 && mine > kAqStages) block_ids(kAqStages, next_id);

    // ---- rotated in fp32, then fp16 operands of a power-of-two scale a row ----
    for (int task = tid; task < n_tok * (D / 2); task += kAqThreads) {
      if (task != tid) load_pair(task, pair);
      const int k = task % (D / 2);
      float c, s;
      rope_turns(pair.pos, pair.turns, c, s);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (pair.ra + r < pair.rb) {
          s_q[(pair.ra + r) * SM::kQPitch + k] = pair.x1[r] * c - pair.x2[r] * s;
          s_q[(pair.ra + r) * SM::kQPitch + k + D / 2] = pair.x2[r] * c + pair.x1[r] * s;
        }
    }
    for (int i = n_rows * D + tid; i < ROWS * D; i += kAqThreads) s_q[(i / D) * SM::kQPitch + i % D] = 0.f;
    __syncthreads();
    for (int r = warp; r < ROWS; r += kAqWarps) {
      float m = 0.f;
      for (int k = lane; k < D; k += 32) m = fmaxf(m, fabsf(s_q[r * SM::kQPitch + k]));
      m = warp_max(m);
      if (lane == 0) s_qs[r] = query_scale<-118>(m);
    }
    __syncthreads();
    uint32_t qa[KS][4];
    float sc[NR];
    {
      const float inv0 = 1.f / s_qs[g];
      const float inv1 = kTwoParts ? inv0 : 1.f / s_qs[(g + 8) % ROWS];
      const float unit = 1.4426950408889634f * rsqrtf((float)D);
      sc[0] = s_qs[g] * unit;
      if constexpr (NR == 2) sc[1] = s_qs[g + 8] * unit;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(s_q + g * SM::kQPitch + t4 * (D / 4) + 4 * j);
        const float v[4] = {x.x * inv0, x.y * inv0, x.z * inv0, x.w * inv0};
        qa[j][0] = pack_f16(v[0], v[1]);
        qa[j][2] = pack_f16(v[2], v[3]);
        if constexpr (kTwoParts) {
          float lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) lo[e] = v[e] - __half2float(__float2half_rn(v[e]));
          qa[j][1] = pack_f16(lo[0], lo[1]);
          qa[j][3] = pack_f16(lo[2], lo[3]);
        } else {
          const float4 y = *reinterpret_cast<const float4*>(s_q + (g + 8) * SM::kQPitch + t4 * (D / 4) + 4 * j);
          qa[j][1] = pack_f16(y.x * inv1, y.y * inv1);
          qa[j][3] = pack_f16(y.z * inv1, y.w * inv1);
        }
      }
    }
    int pi[NR];  // position of the lane's score rows (-1: no such row)
#pragma unroll
    for (int r = 0; r < NR; ++r) pi[r] = g + 8 * r < n_rows ? i0 + ((row0 + g + 8 * r) >> a.log_g) : -1;

    // ---- the stream ----
    float o[KS][NR][4];
    float M[NR], l[NR], lv_low = -CUDART_INF_F;  // lv_low: kAqFar below log2 of the largest value scale that M may hold
#pragma unroll
    for (int m = 0; m < KS; ++m)
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][r][e] = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      M[r] = -CUDART_INF_F;
      l[r] = 0.f;
    }
    int n = 0;
    for (; n < mine; ++n) {
      const bool ok = mbar_wait_bounded(&bar[st], ph, a.wait_ns, a.pool.status);
      if (!__all_sync(0xffffffffu, ok)) {
        s_abort = 1;
        break;
      }
      const unsigned char* kt = ring + st * SM::kStage;
      const uint32_t vt = smem_u32(kt + kAqTile * D);
      const TileMeta m = meta[st];
      const int j0 = tile_key(n);
      // S = Q K^T: column c of product u is position 16 (u/2) + 4 (c/2) + 2 (u%2) + c%2
      float s[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
        const int kr = 16 * (u >> 1) + 4 * (g >> 1) + 2 * (u & 1) + (g & 1);
        uint32_t w[D / 16];
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(kt + kr * 128 + (((2 * t4) ^ (kr & 7)) << 4));
          const uint4 y = *reinterpret_cast<const uint4*>(kt + kr * 128 + (((2 * t4 + 1) ^ (kr & 7)) << 4));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(kt + kr * 64 + ((t4 ^ ((kr >> 1) & 3)) << 4));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          uint32_t b0, b1;
          e4m3x4_to_f16x4(w[j], b0, b1);
          mma_f16(s[u], qa[j][0], qa[j][1], qa[j][2], qa[j][3], b0, b1);
        }
      }
      // base-2 logits with the value scale's exponent
      const float lv[2] = {__log2f(fmaxf(m.vs[0], kQ8ScaleMin)), __log2f(fmaxf(m.vs[1], kQ8ScaleMin))};
      float x[NR][8];  // [2 u + e]
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float f = sc[r] * fmaxf(m.ks[u >> 1], kQ8ScaleMin);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x[r][2 * u + e] = fmaf(kTwoParts ? s[u][e] + s[u][2 + e] : s[u][2 * r + e], f, lv[u >> 1]);
        }
      // every position there and seen by every row?
      const bool all_there = m.there == 3 && j0 + kAqTile - 1 <= i_hi;
      const bool whole =
          all_there && j0 + kAqTile - 1 <= i_lo && (ret || j0 + kAqTile - 1 < a.S || j0 > i_hi - a.W);
      if (!whole) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = j0 + 16 * (u >> 1) + 4 * t4 + 2 * (u & 1) + e;
              const bool see = j <= pi[r] && (m.there >> (u >> 1) & 1) && (ret || j < a.S || j > pi[r] - a.W);
              x[r][2 * u + e] = see ? x[r][2 * u + e] : -CUDART_INF_F;
            }
      }
      float mx[NR];
      bool move = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        mx[r] = x[r][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx[r] = fmaxf(mx[r], x[r][e]);
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        move = move || mx[r] > M[r] + kAqRescale || (M[r] == -CUDART_INF_F && mx[r] > M[r]);
      }
      if (__any_sync(0xffffffffu, move)) {
        lv_low = fmaxf(lv_low, fmaxf(lv[0], lv[1]) - kAqFar);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float mn = fmaxf(M[r], mx[r]);
          const float f = M[r] == -CUDART_INF_F ? 0.f : ex2f(M[r] - mn);
          l[r] = M[r] == -CUDART_INF_F ? 0.f : lower(l[r], M[r] - mn);
          M[r] = mn;
          // O^T's columns are rows 2 t4 and 2 t4 + 1 of the row group
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * t4), f1 = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[k][r][0] *= f0;
            o[k][r][1] *= f1;
            o[k][r][2] *= f0;
            o[k][r][3] *= f1;
          }
        }
      }
      float rv[2] = {ex2f(kAqSumLift - lv[0]), ex2f(kAqSumLift - lv[1])};
      if (fminf(lv[0], lv[1]) < lv_low) {  // (the warp agrees) the tile's share of l from the logits without the scales
        rv[0] = rv[1] = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            l[r] += ex2f(x[r][e] - lv[e >> 2] + (kAqLift + kAqSumLift - (M[r] == -CUDART_INF_F ? 0.f : M[r])));
      }
      uint32_t wh[2][NR][2], wl[2][NR][2];  // [16 positions][row group][b0, b1]
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float sub = kAqLift - (M[r] == -CUDART_INF_F ? 0.f : M[r]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2f(x[r][4 * q + e] + sub);
          l[r] = fmaf((w[0] + w[1]) + (w[2] + w[3]), rv[q], l[r]);
          wh[q][r][0] = pack_f16(w[0], w[1]);
          wh[q][r][1] = pack_f16(w[2], w[3]);
          if constexpr (kWLow) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] -= __half2float(__float2half_rn(w[e]));
            wl[q][r][0] = pack_f16(w[0], w[1]);
            wl[q][r][1] = pack_f16(w[2], w[3]);
          }
        }
      }
      // O^T += V^T W^T; rows of V that are not there may hold anything: zero (0 x NaN is not 0)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t keep = 0xffffffffu;
        if (!all_there) {
          keep = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((m.there >> q & 1) && j0 + 16 * q + 4 * t4 + e <= i_hi) keep |= 0xffu << (8 * e);
        }
        const int vr = 16 * q + (lane & 15);
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          const int c = k + (lane >> 4);
          uint32_t v[4];
          ldsm_b8_t(v, D == 128 ? vt + vr * 128 + ((c ^ (vr & 7)) << 4) : vt + vr * 64 + ((c ^ ((vr >> 1) & 3)) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] &= keep;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(v[2 * p], a0, a2);
            e4m3x4_to_f16x4(v[2 * p + 1], a1, a3);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              mma_f16(o[k + p][r], a0, a1, a2, a3, wh[q][r][0], wh[q][r][1]);
              if constexpr (kWLow) mma_f16(o[k + p][r], a0, a1, a2, a3, wl[q][r][0], wl[q][r][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0 && n + kAqStages < mine) {
        const int id[2] = {next_id[0], next_id[1]};
        if (n + kAqStages + 1 < mine) block_ids(n + kAqStages + 1, next_id);
        issue(n + kAqStages, st, id);
      }
      if (++st == kAqStages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (n < mine) {  // gave up: let the copies in flight land before anything else
      for (int k = n; k < min(mine, n + kAqStages); ++k) {
        mbar_wait_bounded(&bar[st], ph, a.wait_ns, a.pool.status);
        if (++st == kAqStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // ---- join the warps (their partials over the ring, once every warp is done with it) ----
    __syncthreads();
    float* mg = reinterpret_cast<float*>(dsm);
    {
      float* mw = mg + warp * ROWS * SM::kMPitch;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t4 == 0) {
          mw[(g + 8 * r) * SM::kMPitch + D] = M[r];
          mw[(g + 8 * r) * SM::kMPitch + D + 1] = l[r];
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mw[(8 * r + 2 * t4 + (e & 1)) * SM::kMPitch + k * 16 + g + 8 * (e >> 1)] = o[k][r][e];
      }
    }
    __syncthreads();
    const bool alone = u0 == 0 && u1 == nt;  // the whole item is here
    const uint32_t slot = blockIdx.x + item;
    auto write_out = [&](int r, int d, const float4& o, float l) {
      const int tok = rq.q0 + ((row0 + r) >> a.log_g), hq = h * a.G + ((row0 + r) & (a.G - 1));
      T* p = static_cast<T*>(a.c.out) + ((size_t)tok * a.Hq + hq) * D + d;
      const T y[4] = {finish<T>(o.x, l), finish<T>(o.y, l), finish<T>(o.z, l), finish<T>(o.w, l)};
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(y);
      else *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(y);
    };
    for (int i = tid; i < n_rows * (D / 4); i += kAqThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      const float* p = mg + r * SM::kMPitch;
      constexpr int kW = ROWS * SM::kMPitch;  // between warps
      float m = p[D];
#pragma unroll
      for (int w = 1; w < kAqWarps; ++w) m = fmaxf(m, p[w * kW + D]);
      const float ms = m == -CUDART_INF_F ? 0.f : m;
      float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
#pragma unroll
      for (int w = 0; w < kAqWarps; ++w) {
        const float f = ex2f(p[w * kW + D] - ms);
        const float4 v = *reinterpret_cast<const float4*>(p + w * kW + d);
        os.x = fmaf(v.x, f, os.x);
        os.y = fmaf(v.y, f, os.y);
        os.z = fmaf(v.z, f, os.z);
        os.w = fmaf(v.w, f, os.w);
        ls += lower(p[w * kW + D + 1], p[w * kW + D] - ms);
      }
      if (alone) {
        write_out(r, d, os, ls);
      } else if (slot < a.n_slots) {  // always, unless cu_q goes back and forth
        *reinterpret_cast<float4*>(a.part + ((size_t)slot * ROWS + r) * D + d) = os;
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + ((size_t)slot * ROWS + r) * 2) = make_float2(m, ls);
      }
    }
    if (u0 == 0 && u1 < nt) {  // the cut behind this CTA is the item's first
      job.np = (int)((at + (uint32_t)nt - 1) / line.share - blockIdx.x) + 1;
      job.n_rows = slot + (uint32_t)job.np <= a.n_slots ? n_rows : 0;
      job.slot0 = slot;
      job.h = h;
      job.row0 = row0;
      job.q0 = rq.q0;
    }
    fence_async_smem();  // the ring held ordinary stores; the next segment's copies overwrite them
    __syncthreads();
    at = next;
  }
  if (tid == 0) a.jobs[blockIdx.x] = job;
  if (flags) atomicOr(a.pool.status, flags);
}

// Joins the partials of an item (x: the CTA whose note it is) for one row (y):
// a lane a partial for the weights, then the warps the partials in turn.
constexpr int kAqJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kAqJoinWarps * 32) attn_q8_join_kernel(const __grid_constant__ AttnQ8Args a) {
  constexpr int E = D / 32;  // dims a lane
  __shared__ float s_o[kAqJoinWarps][D], s_f[kAqMaxCtas], s_l[kAqJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.y;
  griddep_wait();
  const JoinJob job = a.jobs[blockIdx.x];
  if (job.np == 0 || r >= job.n_rows) return;
  const float* ml = a.part_ml + ((size_t)job.slot0 * a.rows + r) * 2;
  const float* po = a.part + ((size_t)job.slot0 * a.rows + r) * D + lane * E;
  // the first partials of each warp are on their way before their weights are known
  constexpr int kFirst = 8;
  float2 v[kFirst][E / 2];
#pragma unroll
  for (int k = 0; k < kFirst; ++k)
    if (warp + k * kAqJoinWarps < job.np) {
#pragma unroll
      for (int e = 0; e < E / 2; ++e)
        v[k][e] = reinterpret_cast<const float2*>(po + (size_t)(warp + k * kAqJoinWarps) * a.rows * D)[e];
    }
  float m = -CUDART_INF_F;
  for (int p = lane; p < job.np; p += 32) m = fmaxf(m, ml[(size_t)p * a.rows * 2]);
  m = warp_max(m);
  const float ms = m == -CUDART_INF_F ? 0.f : m;
  float l = 0.f;
  for (int p = tid; p < job.np; p += kAqJoinWarps * 32) {
    const float2 y = *reinterpret_cast<const float2*>(ml + (size_t)p * a.rows * 2);
    s_f[p] = ex2f(y.x - ms);
    l += lower(y.y, y.x - ms);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kFirst; ++k)
    if (warp + k * kAqJoinWarps < job.np) {
      const float f = s_f[warp + k * kAqJoinWarps];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        o[2 * e] = fmaf(v[k][e].x, f, o[2 * e]);
        o[2 * e + 1] = fmaf(v[k][e].y, f, o[2 * e + 1]);
      }
    }
#pragma unroll 4
  for (int p = warp + kFirst * kAqJoinWarps; p < job.np; p += kAqJoinWarps) {
    const float f = s_f[p];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 y = *reinterpret_cast<const float2*>(po + (size_t)p * a.rows * D + e);
      o[e] = fmaf(y.x, f, o[e]);
      o[e + 1] = fmaf(y.y, f, o[e + 1]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (tid >= D) return;
  float os = 0.f, ls = 0.f;
#pragma unroll
  for (int w = 0; w < kAqJoinWarps; ++w) {
    os += s_o[w][tid];
    ls += s_l[w];
  }
  const int row = job.row0 + r;
  const int tok = job.q0 + (row >> a.log_g), hq = job.h * a.G + (row & (a.G - 1));
  static_cast<T*>(a.c.out)[((size_t)tok * a.Hq + hq) * D + tid] = finish<T>(os, ls);
}

// Requests of up to this many query rows a KV head (n G) are streamed, larger
// ones of bf16 layers are chunks.  Streaming reads the cache once for each 16
// rows; a chunk's 128-row products cost the same for any number up to 128.
constexpr int kAqSmallRows = 32;

// All requests streamed, all chunks, or (by their rows, on the device) some of each.
int small_rows(const Shape& sh, int max_q) {
  if (sh.dtype == RTP_FP32 || (long long)max_q * sh.G <= kAqSmallRows) return INT32_MAX;
  return sh.B == 1 ? 0 : kAqSmallRows;
}

// Queries that a streamed request can have.
int small_q(const Shape& sh, int max_q) {
  const int s = small_rows(sh, max_q);
  return s == INT32_MAX ? max_q : s / sh.G;
}

// Query rows of a streamed item: 8 (queries in two fp16 parts) for fp32 layers
// and where a KV head's rows fit in 8, else 16.
int item_rows(const Shape& sh, int max_q) {
  return sh.dtype == RTP_FP32 || (long long)small_q(sh, max_q) * sh.G <= 8 ? 8 : 16;
}

long long max_items(const Shape& sh, int n_tokens, int max_q) {
  // sum over requests of ceil(n G / rows)
  const int rows = item_rows(sh, max_q), q = small_q(sh, max_q);
  const long long reqs = sh.B < n_tokens ? sh.B : n_tokens;
  const long long by_tokens = (long long)n_tokens * sh.G / rows + reqs;
  const long long by_max = reqs * (((long long)q * sh.G + rows - 1) / rows);
  return sh.Hkv * (by_tokens < by_max ? by_tokens : by_max);
}

template <typename T, int D, int ROWS>
cudaError_t launch(const AttnQ8Args& a, int most_rows, cudaStream_t st) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int smem = AqSmem<D, ROWS>::kBytes;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(attn_q8_kernel<T, D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  e = launch_pdl(attn_q8_kernel<T, D, ROWS>, dim3(kAqMaxCtas), dim3(kAqThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q8_join_kernel<T, D>, dim3(kAqMaxCtas - 1, ROWS < most_rows ? ROWS : most_rows),
                    dim3(kAqJoinWarps * 32), 0, st, a);
}

}  // namespace

namespace {
size_t stream_workspace_bytes(const Shape& sh, int n_tokens, int max_q) {
  if (small_rows(sh, max_q) == 0) return 0;
  const size_t slots = (size_t)kAqMaxCtas + (size_t)max_items(sh, n_tokens, max_q);
  const size_t bytes = slots * item_rows(sh, max_q) * (sh.D + 2) * sizeof(float) + kAqMaxCtas * sizeof(JoinJob);
  return (bytes + 255) / 256 * 256;
}
}  // namespace

size_t attn_q8_workspace_bytes(const Shape& sh, int n_tokens, int max_q) {
  size_t bytes = stream_workspace_bytes(sh, n_tokens, max_q);
  const int small = small_rows(sh, max_q);
  if (small != INT32_MAX) bytes += chunk_workspace_bytes(sh, n_tokens, max_q, small);
  return bytes < 256 ? 256 : bytes;
}

// The line's positions are 32-bit numbers.
bool attn_q8_fits(const Shape& sh, int max_q, int max_seq_len) {
  const int q = small_q(sh, max_q);
  const long long chunks = ((long long)q * sh.G + item_rows(sh, max_q) - 1) / item_rows(sh, max_q);
  return (double)sh.B * sh.Hkv * (double)chunks * ((max_seq_len - 1) / kAqTile + 1 + kAqItemCost) < 2147483648.0;
}

int launch_attn_q8(const Shape& sh, const Q8Pool& pool, const RopeAxes& rope, const AttnQ8Call& c, void* ws,
                   cudaStream_t st) {
  AttnQ8Args a;
  const unsigned long long pool_rows = ((unsigned long long)pool.n_blocks * sh.Hkv) << pool.log_bs;
  const unsigned box = pool.log_bs == 4 ? 16 : kAqTile;
  const CUtensorMapSwizzle sw = sh.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_tensor_map(&a.tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, pool.k, sh.D, pool_rows, sh.D, box, sw,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !make_tensor_map(&a.tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, pool.v, sh.D, pool_rows, sh.D, box, sw,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B)) {
    set_error("attn q8: could not encode the K/V tensor maps (cuTensorMapEncodeTiled)");
    return RTP_ERR_CUDA;
  }
  a.pool = pool;
  a.rope = rope;
  a.B = sh.B; a.Hq = sh.Hq; a.Hkv = sh.Hkv; a.G = sh.G; a.S = sh.S; a.W = sh.W;
  a.log_g = sh.G == 1 ? 0 : sh.G == 2 ? 1 : sh.G == 4 ? 2 : 3;
  a.ret_mask = 0;
  for (int h = 0; h < sh.Hkv; ++h)
    if (sh.ret_rank[h] >= 0) a.ret_mask |= 1ull << h;
  a.c = c;
  a.rows = item_rows(sh, c.max_q);
  a.wait_ns = 400ull * 1000 * 1000;
  for (int i = 0; i < 64; ++i) a.turns[i] = sh.turns[i];
  a.small_rows = small_rows(sh, c.max_q);
  const long long items = max_items(sh, c.n_tokens, c.max_q);
  a.jobs = static_cast<JoinJob*>(ws);
  a.part = reinterpret_cast<float*>(a.jobs + kAqMaxCtas);
  a.n_slots = (uint32_t)(kAqMaxCtas + items);
  a.part_ml = a.part + (size_t)a.n_slots * a.rows * sh.D;
  const bool chunks = a.small_rows != INT32_MAX;
  if (chunks && !chunk_carve(sh, c.n_tokens, c.max_q, a.small_rows,
                             static_cast<unsigned char*>(ws) + stream_workspace_bytes(sh, c.n_tokens, c.max_q), &a)) {
    set_error("attn q8: could not encode the queries' tensor map (cuTensorMapEncodeTiled)");
    return RTP_ERR_CUDA;
  }
  cudaError_t e = cudaSuccess;
  trace_begin(RTP_STAGE_ATTN_Q8, st);
  if (a.small_rows > 0) {
    const long long rows = (long long)small_q(sh, c.max_q) * sh.G;  // that a request can have
    const int most = rows < 16 ? (int)rows : 16;
    if (sh.dtype == RTP_BF16) {
      if (a.rows == 8) e = sh.D == 128 ? launch<__nv_bfloat16, 128, 8>(a, most, st) : launch<__nv_bfloat16, 64, 8>(a, most, st);
      else e = sh.D == 128 ? launch<__nv_bfloat16, 128, 16>(a, most, st) : launch<__nv_bfloat16, 64, 16>(a, most, st);
    } else {
      e = sh.D == 128 ? launch<float, 128, 8>(a, most, st) : launch<float, 64, 8>(a, most, st);
    }
  }
  if (chunks && e == cudaSuccess) e = launch_attn_q8_chunks(sh, a, st);
  trace_end(RTP_STAGE_ATTN_Q8, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error(std::string("attn q8 launch: ") + cudaGetErrorString(e));
    return RTP_ERR_CUDA;
  }
  return RTP_OK;
}

}  // namespace rtp
