// rtp_attn_q8 for chunks: attention of many queries a request over the paged
// 8-bit cache, on the fifth-generation tensor cores (tcgen05 + TMEM).
//
// Mathematics as in attn_q8.cu (weights 2^(x - M) with the value blocks' scales
// in the exponent).  e4m3 values are exact in fp16, so the operands are fp16:
// K and V as stored, without their scales; Q scaled by a power of two a row;
// the weights.  The block scales enter as one multiplier and one addend of the
// base-2 logits, which the softmax's fused multiply-add takes for nothing.
//
// Work.  An item is 256 query rows of one (request, KV head): row r is token
// r / G, query head r % G of the group, so the G heads share every tile of K
// and V and a chunk of 64 G-head tokens fills the tensor cores' rows.  A tile
// is 128 positions.  The tiles of all items, and three more units an item for its
// start and end (without them the CTAs with many short window items finished a
// tenth late: 418 us for 384), form one line that is cut into equal shares, one
// a CTA (one an SM): causal triangles, windows and ragged batches load the SMs
// evenly.  A cut item leaves partials that a last kernel joins.
//
// Roles (16 warps):
//   warps 0-3, 4-7   the softmax of slot 0 and slot 1 (128 rows each), one
//                    thread a row: 64 columns of S at a time are read from TMEM
//                    and their fp16 weights against the running maximum written
//                    over columns already read; where they exceed the maximum by
//                    2^9, it moves, up to a whole number, and O and the tile's weights
//                    so far are rescaled by the exact power of two.  One rolled loop: the same in straight-line code
//                    for 4 x 32 columns took 475 us for the 418 (the instruction
//                    cache could not feed it), a rolled loop over 32 columns 409
//                    for 384, whole rows in registers and S read twice more still;
//   warps 8-11       convert a tile's e4m3 rows to fp16 in the operands' swizzled layout;
//   warp 12          issues the products in the order S0(i), PV1(i-1), S1(i),
//                    PV0(i): each slot's softmax runs beside the other's products;
//   warp 13          loads by TMA: Q of the next item, K and V rows of the next
//                    tile from their blocks, and reads the blocks' scales.
// The roles run on from item to item on their own; nothing synchronises the CTA
// between its first and its last tile.
//
// The first kernel lays the line out and rotates the queries: fp16 rows and
// their scales, once a token, not once a CTA in a prologue that stalls its
// products (33000 clocks an item, measured).
//
// Every wait is bounded: on expiry the CTA sets RTP_DEV_TIMEOUT, stops issuing,
// waits (bounded) for what it issued and frees its TMEM.
//
// Bound: the tensor cores.  A tile of 256 x 128 pairs at D = 128 is 16.8 MFLOP,
// 2048 clocks at the dense fp16 rate; its weights are 32768 exponentials, 2048
// clocks of the MUFU pipe, of which a quarter go to the FMA pipe (none: 399 us
// for 384; an eighth 393; a half 421).
//
// Measured, 2K queries of 32 heads at 32K positions, D = 128: 359 us for the
// three kernels in a replayed graph (319 GFLOP, 890 TFLOP/s, 54% of a large matrix
// product's rate).
// A tile takes 4950 clocks: a slot's softmax 2700 of them, then its own two
// products and the turn of the other slot's (1700), 250 from one to the next;
// an item's end and start about as long as three tiles.
// Halves of a tile with their own products, so that a slot's softmax need not
// wait for them, made the products' issue the bound instead (64-column products
// are 48 clocks for half the work of 64.5): 411 us.
#include <mutex>

#include "attn_q8.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace rtp {
namespace {

constexpr int kCRows = 128;               // query rows a slot = TMEM lanes
constexpr int kCGroup = 256;              // query rows an item
constexpr int kCKeys = 128;               // positions a tile
constexpr int kCThreads = 16 * 32;
constexpr int kCRegion = 128 * 128;       // bytes of 128 rows x 64 fp16 dims
constexpr int kCCtas = 148;               // one an SM of a B200
constexpr int kCItemCost = 3;             // units of the line after an item's tiles: its start and end cost about as much
constexpr int kCMinShare = 4;             // units a CTA takes at least
constexpr int kCTmemCols = 512;
// The running maximum moves past 2^9: weights reach 2^15, and 2^15.5 where M is rounded by a half
// (from 2^24, scores of 2^23), below fp16's largest.
constexpr float kCRescale = 9.f;

template <int D>
struct CSmem {
  static constexpr int kOp = (D / 64) * kCRegion;  // one operand tile: Q of a slot, K or V of a stage
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kOp;
  static constexpr int kOffV = kOffK + 2 * kOp;
  static constexpr int kRaw = kCKeys * D;          // e4m3 rows of a tile
  static constexpr int kOffRaw = kOffV + 2 * kOp;  // K, then V
  static constexpr int kBytes = kOffRaw + 2 * kRaw + 1024;  // + alignment slack
};

// Scales of 16 positions of a tile, and which 32-position words are there.
struct __align__(16) CMeta {
  // k scale, log2(v scale), 2^24 / v scale (0 where `far`, and for blocks that are not there); g[0].w: 1 where all are there and not `far`
  float4 g[8];
  uint32_t there[4];
  int far;  // the value scales so far, of the item's tiles in this CTA, lie more than kAqFar apart
};

// First position of an item's u-th tile.
__device__ __forceinline__ int tile_pos(const ChunkItem& c, int u) { return (u < c.ns ? u : c.w0 + u - c.ns) * kCKeys; }

__device__ __forceinline__ ChunkItem chunk_item(const AttnQ8Args& a, const ReqRows& r, int b, int h, int grp) {
  ChunkItem c;
  c.b = b;
  c.h = h;
  c.row0 = grp * kCGroup;
  c.n_rows = min(kCGroup, r.n * a.G - c.row0);
  c.q0 = r.q0;
  c.i0 = r.L - r.n;
  c.i_hi = c.i0 + ((c.row0 + c.n_rows - 1) >> a.log_g);
  c.ret = (int)((a.ret_mask >> h) & 1ull);
  c.pad = 0;
  const int nt = c.i_hi / kCKeys + 1;
  c.ns = min((a.S + kCKeys - 1) / kCKeys, nt);
  c.w0 = max(0, c.i0 + (c.row0 >> a.log_g) - a.W + 1) / kCKeys;
  if (c.ret || c.w0 <= c.ns) c.ns = c.w0 = 0;
  c.tiles = c.ns + nt - c.w0;
  return c;
}

constexpr int kCPrep = 256;  // threads of the first kernel

// Exclusive scan over the block and its total.
__device__ __forceinline__ long long block_scan(long long v, long long& total, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kCPrep / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  return x - v + before;
}

// Block 0 lays out the line: items in the order (request, KV head, group), and
// the units ahead of each.  The others rotate queries: a warp a token and 8
// heads; every row becomes fp16 of its power-of-two scale, and its factor from
// products to base-2 logits.
template <int D>
__global__ void __launch_bounds__(kCPrep) chunk_prep_kernel(const __grid_constant__ AttnQ8Args a) {
  if (blockIdx.x > 0) {
    constexpr int PP = D / 64, H = D / 2;
    struct __align__(2 * PP) Pairs { __nv_bfloat16 x[PP]; };  // a lane's dims, below H or from H on
    struct __align__(2 * PP) Halves { __half x[PP]; };
    const int lane = threadIdx.x & 31;
    const int hb = (a.Hq + 7) / 8;
    const long long task = (long long)(blockIdx.x - 1) * (kCPrep / 32) + (threadIdx.x >> 5);
    // lanes that index the parameters apart are served one by one: once a CTA, not once a warp
    __shared__ uint64_t s_turns[H];
    __shared__ int s_axis[H];
    if (threadIdx.x < H) {
      s_turns[threadIdx.x] = a.turns[threadIdx.x];
      s_axis[threadIdx.x] = a.rope.axis[threadIdx.x];
    }
    __syncthreads();
    griddep_wait();
    griddep_launch();
    if (task >= (long long)a.c.n_tokens * hb) return;
    const int t = (int)(task / hb), h0 = (int)(task % hb) * 8;
    const float unit = 1.4426950408889634f * rsqrtf((float)D);
    float c[PP], s[PP];
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int k = lane * PP + i;
      rope_turns(a.c.pos[(size_t)s_axis[k] * a.c.n_tokens + t], s_turns[k], c[i], s[i]);
    }
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.c.q_pre) + (size_t)t * a.c.q_stride + (size_t)h0 * D + lane * PP;
    const int nh = min(a.Hq - h0, 8);
    float x1[8][PP], x2[8][PP];
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < nh) {
        const Pairs u = *reinterpret_cast<const Pairs*>(q + h * D), v = *reinterpret_cast<const Pairs*>(q + h * D + H);
#pragma unroll
        for (int i = 0; i < PP; ++i) {
          x1[h][i] = to_f32(u.x[i]);
          x2[h][i] = to_f32(v.x[i]);
        }
      }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      if (h >= nh) break;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        const float y1 = x1[h][i] * c[i] - x2[h][i] * s[i];
        x2[h][i] = x2[h][i] * c[i] + x1[h][i] * s[i];
        x1[h][i] = y1;
        m = fmaxf(m, fmaxf(fabsf(y1), fabsf(x2[h][i])));
      }
      // (times the least key scale, 2^-64, and log2(e) / sqrt(D) the factor stays above 0: it multiplies the -inf of masked positions)
      const float sc = query_scale<-59>(warp_max(m)), inv = 1.f / sc;
      const size_t row = (size_t)t * a.Hq + h0 + h;
      __half* o = a.cq + row * D + lane * PP;
      Halves y1, y2;
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        y1.x[i] = __float2half_rn(x1[h][i] * inv);
        y2.x[i] = __float2half_rn(x2[h][i] * inv);
      }
      *reinterpret_cast<Halves*>(o) = y1;
      *reinterpret_cast<Halves*>(o + H) = y2;
      if (lane == 0) a.cq_unit[row] = sc * unit;
    }
    return;
  }
  __shared__ long long s_warp[kCPrep / 32];
  __shared__ int s_req[kCPrep];  // req_items, where they fit
  griddep_wait();
  griddep_launch();
  int flags = 0;
  long long n_items = 0;
  for (int b0 = 0; b0 < a.B; b0 += kCPrep) {
    const int b = b0 + threadIdx.x;
    long long v = 0;
    if (b < a.B) {
      const ReqRows r = load_rows(a, b, flags);
      const long long rows = (long long)r.n * a.G;
      if (rows > a.small_rows) v = a.Hkv * ((rows + kCGroup - 1) / kCGroup);
    }
    long long total;
    const long long x = n_items + block_scan(v, total, s_warp);
    if (b < a.B) s_req[threadIdx.x] = a.req_items[b] = (int)min(x, (long long)a.max_chunk_items);
    n_items += total;
  }
  n_items = min(n_items, (long long)a.max_chunk_items);  // more only if cu_q goes back and forth
  if (threadIdx.x == 0) a.req_items[a.B] = (int)n_items;
  __syncthreads();
  const int* req = a.B <= kCPrep ? s_req : a.req_items;
  long long tiles = 0;
  for (int i0 = 0; i0 < n_items; i0 += kCPrep) {
    const int i = i0 + threadIdx.x;
    long long v = 0;
    ChunkItem it = {};
    if (i < n_items) {
      int b = 0, hi = a.B;  // the last request with req_items <= i
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (req[mid] <= i) b = mid;
        else hi = mid;
      }
      const ReqRows r = load_rows(a, b, flags);
      const int ng = (r.n * a.G + kCGroup - 1) / kCGroup, rel = i - req[b];
      it = chunk_item(a, r, b, rel / ng, rel % ng);
      v = it.tiles + kCItemCost;
    }
    long long total;
    const long long x = tiles + block_scan(v, total, s_warp);
    if (i < n_items) {
      a.items[i] = it;
      a.prefix[i] = x;
    }
    tiles += total;
  }
  if (threadIdx.x == 0) {
    a.prefix[n_items] = tiles;
    a.prefix[a.max_chunk_items + 1] = max((tiles + kCCtas - 1) / kCCtas, (long long)kCMinShare);
  }
  if (flags) atomicOr(a.pool.status, flags);
}

// The item whose units hold line position `at` (one warp; prefix[n] > at).
__device__ __forceinline__ int find_item(const long long* prefix, int n, long long at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + min(lane * step, len - 1);
    const unsigned m = __ballot_sync(0xffffffffu, prefix[i] <= at && lane * step < len);  // lane 0's holds
    const int k = 31 - __clz(m);
    const int nlo = lo + k * step;
    len = min(step, lo + len - nlo);
    lo = nlo;
  }
  return lo;
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b) {  // (x, y) = (x, y) a + b
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}

// (x, y) = (2^x, 2^y) on the FMA pipe, the cubic of ex2_poly on a pair.  Below -125, masked
// positions among them, 2^-125: 0 in fp16, and in l 2^(24 - 125) / vs, in all under 2^-44 of it
// beside scales up to 2^64 larger; where they lie farther apart l is not formed from these.
__device__ __forceinline__ void ex2_poly2(float& x, float& y) {
  const float a = fmaxf(x, -125.f), b = fmaxf(y, -125.f);
  asm("{\n\t.reg .b64 v, t, f, p, c;\n\t.reg .b32 t0, t1, p0, p1;\n\t"
      "mov.b64 v, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\tadd.rn.f32x2 t, v, c;\n\t"    // round(x) in t's low bits
      "mov.b64 c, {%5, %5};\n\tadd.rn.f32x2 f, t, c;\n\t"
      "mov.b64 c, {%6, %6};\n\tfma.rn.f32x2 f, f, c, v;\n\t"                          // x - round(x)
      "mov.b64 c, {%7, %7};\n\tmov.b64 p, {%8, %8};\n\tfma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 c, {%9, %9};\n\tfma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 c, {%10, %10};\n\tfma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 {t0, t1}, t;\n\tmov.b64 {p0, p1}, p;\n\t"
      "shl.b32 t0, t0, 23;\n\tshl.b32 t1, t1, 23;\n\tadd.s32 p0, p0, t0;\n\tadd.s32 p1, p1, t1;\n\t"
      "mov.b32 %0, p0;\n\tmov.b32 %1, p1;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(12582912.f), "f"(-12582912.f), "f"(-1.f), "f"(0.24261111f), "f"(0.05517161f),
        "f"(0.69326097f), "f"(0.99992806f));
}

__device__ __noinline__ bool c_wait_long(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, int* status,
                                         volatile int* s_abort) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_sleep(bar, parity, kWaitHintNs)) {
    if (*s_abort) return false;
    if (global_ns() - t0 > limit_ns) {
      *s_abort = 1;
      atomicOr(status, RTP_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
// Bounded wait that also gives up once another role has; the warp agrees on the outcome.
__device__ __forceinline__ bool c_wait(uint64_t* bar, uint32_t parity, const AttnQ8Args& a, volatile int* s_abort) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = c_wait_long(bar, parity, a.wait_ns, a.pool.status, s_abort);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* tm, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
               :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(0), "r"(y)
               : "memory");
}

// The CTA's share of the line, walked item by item (each role for itself).
struct CWalk {
  int item;
  long long at, end;
  // the current segment: tiles [u0, u0 + nt) of item c
  ChunkItem c;
  int u0, nt;
  bool two;  // it has rows for the second slot
  __device__ __forceinline__ bool start(const AttnQ8Args& a) {
    const int n_items = a.req_items[a.B];
    const long long total = a.prefix[n_items], share = a.prefix[a.max_chunk_items + 1];
    at = (long long)blockIdx.x * share;
    end = min(total, at + share);
    if (at >= end) return false;
    item = find_item(a.prefix, n_items, at);
    load(a);
    return nt > 0 || next(a);
  }
  __device__ __forceinline__ void load(const AttnQ8Args& a) {
    c = a.items[item];
    u0 = (int)(at - a.prefix[item]);
    nt = (int)min((long long)c.tiles - u0, end - at);  // none or fewer if the share starts in the units after the item's tiles
    two = c.n_rows > kCRows;
  }
  __device__ __forceinline__ bool next(const AttnQ8Args& a) {
    at = a.prefix[++item];
    if (at >= end) return false;
    load(a);
    return true;
  }
};

// A row's maximum and l after a tile whose value scales lie far below the largest: its share of l
// comes from the logits without the scales, against the tile's own maximum, to which O and l are
// brought first.  Seldom called, so it is kept out of the softmax's loop.
template <int D>
__device__ __forceinline__ float2 far_tile(const CMeta& m, uint32_t tSs, uint32_t tOs, bool has_o, float rs, float M, float l) {
  float mx = M;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint32_t s[16];
    tmem_ld16(tSs + 16 * q, s);
    tmem_wait_ld();
    const float4 g = m.g[q];
    float t = -CUDART_INF_F;
#pragma unroll
    for (int e = 0; e < 16; ++e) t = fmaxf(t, __uint_as_float(s[e]));
    mx = fmaxf(mx, fmaf(t, rs * g.x, g.y));
  }
  mx = ceilf(mx);
  const float f = M == -CUDART_INF_F ? 0.f : ex2f(M - mx);
  l = M == -CUDART_INF_F ? 0.f : lower(l, M - mx);
  if (has_o) {
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
      uint32_t o[16];
      tmem_ld16(tOs + k * 16, o);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st16(tOs + k * 16, o);
    }
    tmem_wait_st();
  }
  const float sub = kAqLift + kAqSumLift - (mx == -CUDART_INF_F ? 0.f : mx);
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint32_t s[16];
    tmem_ld16(tSs + 16 * q, s);
    tmem_wait_ld();
    const float fq = rs * m.g[q].x;
#pragma unroll
    for (int e = 0; e < 16; ++e) l += ex2f(fmaf(__uint_as_float(s[e]), fq, sub));
  }
  return make_float2(mx, l);
}

struct CBars {
  uint64_t raw_full[2], raw_empty[2];                       // K's rows as stored, and V's
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];    // by stage
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2];  // by slot
  uint64_t fin;
};

// Asks for the rows of the CTA's tile T, whose blocks the lanes hold in `id`, and writes its scales.
// `span`: log2 of the least and the largest value scale so far of the item's tiles in this CTA.
template <int D>
__device__ __forceinline__ bool load_rows_of_tile(const AttnQ8Args& a, const CWalk& w, int T, int id, CBars& bars,
                                                  unsigned char* raw, CMeta* meta, volatile int* s_abort, uint32_t (&asked)[2],
                                                  float2& span) {
  const int lane = threadIdx.x & 31;
  const int per = kCKeys >> a.pool.log_bs, box = 1 << a.pool.log_bs;  // copies a tile, of so many rows
  float ks = 0.f, vs = 0.f;
  if (id >= 0) {
    ks = a.pool.k_scale[(size_t)id * a.Hkv + w.c.h];
    vs = a.pool.v_scale[(size_t)id * a.Hkv + w.c.h];
  }
  // copy p < per covers the blocks of lanes p * 8 / per ..; a block that is not there: any rows, they become zeros
  const int mine = __shfl_sync(0xffffffffu, id, (lane & 7) * (8 / per) & 7);
  const int y = (((mine < 0 ? 0 : mine) * a.Hkv + w.c.h) << a.pool.log_bs);  // (a tile starts on a block)
  const unsigned there = __ballot_sync(0xffffffffu, lane < 8 && id >= 0);
  vs = fmaxf(vs, kQ8ScaleMin);
  const float lv = __log2f(vs);
  if (id >= 0) {
    span.x = fminf(span.x, lv);
    span.y = fmaxf(span.y, lv);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {  // (lanes 8 and up repeat the first ones)
    span.x = fminf(span.x, __shfl_xor_sync(0xffffffffu, span.x, o));
    span.y = fmaxf(span.y, __shfl_xor_sync(0xffffffffu, span.y, o));
  }
  const bool far = span.x < span.y - kAqFar;
  const float4 g = make_float4(fmaxf(ks, kQ8ScaleMin), lv, id < 0 || far ? 0.f : kAqSumUnit / vs, there == 0xffu && !far ? 1.f : 0.f);
  if (!c_wait(&bars.raw_empty[0], ((uint32_t)T & 1u) ^ 1u, a, s_abort)) return false;
  CMeta& m = meta[T & 7];
  if (lane < 8) m.g[lane] = g;
  if (lane == 0) m.far = far;
  if (lane < 4)
    m.there[lane] = ((there >> (2 * lane) & 1u) ? 0xffffu : 0u) | ((there >> (2 * lane + 1) & 1u) ? 0xffff0000u : 0u);
  __syncwarp();
  if (lane == 0) mbar_expect_tx(&bars.raw_full[0], (uint32_t)(kCKeys * D));
  __syncwarp();
  if (lane < per) tma_rows(raw + lane * box * D, &a.tm_ck, y, &bars.raw_full[0]);
  ++asked[0];
  if (!c_wait(&bars.raw_empty[1], ((uint32_t)T & 1u) ^ 1u, a, s_abort)) return false;
  if (lane == 0) mbar_expect_tx(&bars.raw_full[1], (uint32_t)(kCKeys * D));
  __syncwarp();
  if (lane < per) tma_rows(raw + kCKeys * D + lane * box * D, &a.tm_cv, y, &bars.raw_full[1]);
  ++asked[1];
  return true;
}

template <int D>
__global__ void __launch_bounds__(kCThreads, 1) attn_q8_chunk_kernel(const __grid_constant__ AttnQ8Args a) {
  using SM = CSmem<D>;
  extern __shared__ __align__(1024) unsigned char dsm_raw[];
  __shared__ __align__(8) CBars bars;
  // tile i's scales, read by the softmax after S(i); rewritten for tile i + 8, whose rows are
  // asked for once tile i + 7 is converted, S of tile i + 5 complete and the weights of tile i + 4 formed
  __shared__ CMeta s_meta[8];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* dsm = dsm_raw + ((1024u - (smem_u32(dsm_raw) & 1023u)) & 1023u);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.raw_full[s], 1);
      mbar_init(&bars.raw_empty[s], 128);
      mbar_init(&bars.k_full[s], 128);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.v_full[s], 128);
      mbar_init(&bars.v_empty[s], 1);
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 1);
      mbar_init(&bars.s_full[s], 2);  // the products' commit, and the issuer (who has seen the scales)
      mbar_init(&bars.p_full[s], kCRows);
      mbar_init(&bars.o_full[s], 1);
      mbar_init(&bars.o_empty[s], kCRows);
    }
    mbar_init(&bars.fin, 1);
    s_abort = 0;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&s_tmem)), "r"(kCTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  griddep_launch();

  if (warp < 8) {
    // ---- softmax: one thread a row ----
    const int slot = warp >> 2, quad = warp & 3, r = tid;  // row of the item
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tSs = tmem + slot * kCKeys + lane_off, tOs = tmem + (2 + slot) * kCKeys + lane_off;
    uint32_t ph = 0u, seg = 0u;  // tiles and items of this slot so far
    int gt = 0;                  // tiles of the CTA
    CWalk w;
    bool ok = true;
    for (bool more = w.start(a); more && ok; gt += w.nt, more = w.next(a)) {
      if (slot == 1 && !w.two) continue;
      const ChunkItem& c = w.c;
      const bool rv = r < c.n_rows;
      const int pi = c.i0 + ((c.row0 + r) >> a.log_g);                // the row's position
      const int s_lo = c.i0 + ((c.row0 + slot * kCRows) >> a.log_g);  // the slot's first, and its last row's
      const int s_hi = min(c.i_hi, c.i0 + ((c.row0 + slot * kCRows + kCRows - 1) >> a.log_g));
      const int tok = c.q0 + ((c.row0 + r) >> a.log_g), hq = w.c.h * a.G + ((c.row0 + r) & (a.G - 1));
      const float rs = rv ? a.cq_unit[(size_t)tok * a.Hq + hq] : 1.f;
      float M = -CUDART_INF_F, l = 0.f;
      bool poison = false;
      for (int i = 0; i < w.nt; ++i, ph ^= 1u) {
        const int kt = tile_pos(c, w.u0 + i);
        if (!c_wait(&bars.s_full[slot], ph, a, &s_abort)) { ok = false; break; }
        tc_fence_after();
        const CMeta& m = s_meta[(gt + i) & 7];
        const bool whole = kt + kCKeys - 1 <= s_lo && (c.ret || kt + kCKeys - 1 < a.S || kt > s_hi - a.W) &&
                           m.g[0].w != 0.f;
        if (!whole) {  // (the slot agrees) S of the positions that the row does not see becomes -inf
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            const int base = kt + 32 * x;
            const int nc = pi - base + 1;
            const uint32_t causal = !rv || nc <= 0 ? 0u : nc >= 32 ? 0xffffffffu : (1u << nc) - 1u;
            uint32_t near = 0xffffffffu;
            if (!c.ret) {
              const int nsk = a.S - base, nw = pi - a.W + 1 - base;
              near = (nsk <= 0 ? 0u : nsk >= 32 ? 0xffffffffu : (1u << nsk) - 1u) |
                     (nw <= 0 ? 0xffffffffu : nw >= 32 ? 0u : ~((1u << nw) - 1u));
            }
            const uint32_t bits = causal & near & m.there[x];
            if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
            float v[32];
            tmem_ld32(tSs + x * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (bits >> e) & 1u ? v[e] : -CUDART_INF_F;
            tmem_st32(tSs + x * 32, v);
          }
          tmem_wait_st();
          if (m.far) {  // (the slot agrees)
            const float2 y = far_tile<D>(m, tSs, tOs, i > 0, rs, M, l);
            M = y.x;
            l = y.y;
          }
        }
        // ---- the weights against the running maximum, 64 columns at a time (one rolled loop:
        // the instruction cache feeds it), their fp16 over columns already read ----
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          float v[64];
          tmem_ld64(tSs + 64 * x, v);
          float4 g[4];  // of 16 columns each
#pragma unroll
          for (int q = 0; q < 4; ++q) g[q] = m.g[4 * x + q];
          tmem_wait_ld();
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* y = v + 16 * q;
            float t0 = max3_nan(y[0], y[1], y[2]), t1 = max3_nan(y[3], y[4], y[5]);
            t0 = max3_nan(t0, y[6], y[7]);
            t1 = max3_nan(t1, y[8], y[9]);
            t0 = max3_nan(t0, y[10], y[11]);
            t1 = max3_nan(t1, y[12], y[13]);
            t0 = max3_nan(t0, y[14], y[15]);
            mx = max_nan(mx, fmaf(max_nan(t0, t1), rs * g[q].x, g[q].y));
          }
          poison = poison || mx != mx;  // a stored NaN that the row sees
          const bool need = mx > M + kCRescale || (M == -CUDART_INF_F && mx > M);
          if (__any_sync(0xffffffffu, need)) {
            // rare after an item's first columns: the maximum moves, and with it O, l and the
            // tile's weights so far (by whole powers of two: in fp16 too the factor is exact)
            mx = ceilf(mx);
            const float f = need ? (M == -CUDART_INF_F ? 0.f : ex2f(M - mx)) : 1.f;
            M = need ? mx : M;
            l *= f;
            // PV of the slot's previous tile has completed (S(i) was issued after it)
            if (i > 0) {
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k) {
                uint32_t o[16];
                tmem_ld16(tOs + k * 16, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(tOs + k * 16, o);
              }
            }
            tmem_wait_st();
            const __half2 f2 = __float2half2_rn(f);
#pragma unroll 1
            for (int y = 0; y < 2 * x; ++y) {
              uint32_t o[16];
              tmem_ld16(tSs + y * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __half2 t = __hmul2(*reinterpret_cast<__half2*>(&o[e]), f2);
                o[e] = *reinterpret_cast<const uint32_t*>(&t);
              }
              tmem_st16(tSs + y * 16, o);
            }
          }
          const float base = kAqLift - (M == -CUDART_INF_F ? 0.f : M);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float fq = rs * g[2 * w + q].x, add = g[2 * w + q].y + base;
              float s0 = 0.f, s1 = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float x0 = v[32 * w + 16 * q + 2 * e], x1 = v[32 * w + 16 * q + 2 * e + 1];
                fma2(x0, x1, fq, add);
                if ((e & 3) == 3) {  // one weight in four on the FMA pipe
                  ex2_poly2(x0, x1);
                } else {
                  x0 = ex2f(x0);
                  x1 = ex2f(x1);
                }
                add2(s0, s1, x0, x1);
                pk[8 * q + e] = pack_f16(x0, x1);
              }
              l = fmaf(s0 + s1, g[2 * w + q].z, l);
            }
            tmem_st16(tSs + 32 * x + 16 * w, pk);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_full[slot]);
      }
      if (!ok || !c_wait(&bars.o_full[slot], seg & 1u, a, &s_abort)) { ok = false; break; }
      tc_fence_after();
      if (poison) l = CUDART_NAN_F;
      else if (M == -CUDART_INF_F) l = 0.f;  // the row sees nothing (ex2_poly2 gives masked positions 2^-125, not 0)
      const bool alone = w.u0 == 0 && w.nt == c.tiles;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.c.out) + ((size_t)tok * a.Hq + hq) * D;
      const size_t pn = (size_t)(2 * blockIdx.x + (w.u0 > 0 ? 0 : 1));  // the partial: four dims of all rows lie together
      const float inv = l == 0.f ? 0.f : kAqSumUnit / l;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        float o[32];
        tmem_ld32(tOs + k * 32, o);
        tmem_wait_ld();
        if (!rv) continue;
        if (alone) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 u;
            u.x = pack_bf16(o[e] * inv, o[e + 1] * inv);
            u.y = pack_bf16(o[e + 2] * inv, o[e + 3] * inv);
            u.z = pack_bf16(o[e + 4] * inv, o[e + 5] * inv);
            u.w = pack_bf16(o[e + 6] * inv, o[e + 7] * inv);
            *reinterpret_cast<uint4*>(orow + k * 32 + e) = u;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(a.cpart + ((pn * (D / 4) + k * 8 + e / 4) * kCGroup + r) * 4) =
                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (rv && !alone) *reinterpret_cast<float2*>(a.cpart_ml + (pn * kCGroup + r) * 2) = make_float2(M, l);
      tc_fence_before();
      mbar_arrive(&bars.o_empty[slot]);
      ++seg;
    }
  } else if (warp < 12) {
    // ---- K and V rows to fp16, swizzled ----
    constexpr int LPR = D / 16;          // lanes a row (16 bytes each)
    constexpr int RPI = 4 * (32 / LPR);  // rows the four warps take at once
    const int r_lane = (warp - 8) * (32 / LPR) + lane / LPR, cl = lane % LPR;
    // 16 dims are two 16-byte chunks of a 64-dim region; lanes of the two
    // regions take them in opposite order, so eight lanes hit eight chunks
    const int reg = cl >> 2, ch = (2 * cl) & 7, odd = reg & 1;
    const int off0 = reg * kCRegion + r_lane * 128 + (((ch + odd) ^ (r_lane & 7)) << 4);
    const int off1 = reg * kCRegion + r_lane * 128 + (((ch + 1 - odd) ^ (r_lane & 7)) << 4);
    static_assert(RPI % 8 == 0, "a lane's rows share their swizzle");
    auto convert = [&](const unsigned char* raw, unsigned char* dst, const CMeta& m, int n_valid, bool all) {
#pragma unroll 4
      for (int r = 0; r < kCKeys; r += RPI) {
        uint4 x = *reinterpret_cast<const uint4*>(raw + (r + r_lane) * D + cl * 16);
        // rows past the item's last position, or whose block is not there, hold anything: zeros
        if (!all && (r + r_lane >= n_valid || !(m.there[(r + r_lane) >> 5] >> ((r + r_lane) & 31) & 1u)))
          x = make_uint4(0u, 0u, 0u, 0u);
        uint4 lo, hi;
        e4m3x4_to_f16x4(x.x, lo.x, lo.y);
        e4m3x4_to_f16x4(x.y, lo.z, lo.w);
        e4m3x4_to_f16x4(x.z, hi.x, hi.y);
        e4m3x4_to_f16x4(x.w, hi.z, hi.w);
        *reinterpret_cast<uint4*>(dst + r * 128 + off0) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(dst + r * 128 + off1) = odd ? lo : hi;
      }
    };
    CWalk w;
    int T = 0;
    bool ok = true;
    for (bool more = w.start(a); more && ok; more = w.next(a)) {
      for (int i = 0; i < w.nt; ++i, ++T) {
        const int st = T & 1;
        const uint32_t par = ((uint32_t)(T >> 1) & 1u) ^ 1u;
        const CMeta& m = s_meta[T & 7];
        const int n_valid = w.c.i_hi - tile_pos(w.c, w.u0 + i) + 1;
        if (!(ok = c_wait(&bars.raw_full[0], (uint32_t)T & 1u, a, &s_abort))) break;
        const bool all = n_valid >= kCKeys && m.g[0].w != 0.f;
        if (!(ok = c_wait(&bars.k_empty[st], par, a, &s_abort))) break;
        convert(dsm + SM::kOffRaw, dsm + SM::kOffK + st * SM::kOp, m, n_valid, all);
        fence_async_smem();
        mbar_arrive(&bars.raw_empty[0]);
        mbar_arrive(&bars.k_full[st]);
        if (!(ok = c_wait(&bars.raw_full[1], (uint32_t)T & 1u, a, &s_abort))) break;
        if (!(ok = c_wait(&bars.v_empty[st], par, a, &s_abort))) break;
        convert(dsm + SM::kOffRaw + SM::kRaw, dsm + SM::kOffV + st * SM::kOp, m, n_valid, all);
        fence_async_smem();
        mbar_arrive(&bars.raw_empty[1]);
        mbar_arrive(&bars.v_full[st]);
      }
    }
  } else {
    if (warp == 12) {
      // ---- the products ----
      constexpr uint32_t idS = umma_idesc(kCRows, kCKeys, false, true);
      constexpr uint32_t idO = umma_idesc(kCRows, D, true, true);
      const uint64_t dq0 = umma_desc(smem_u32(dsm + SM::kOffQ), 16, 1024), dk0 = umma_desc(smem_u32(dsm + SM::kOffK), 16, 1024);
      const uint64_t dv0 = umma_desc(smem_u32(dsm + SM::kOffV), kCRegion, 1024);
      const uint32_t lead = elect_lane();
      auto uni = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };  // a value that the warp agrees on
      const uint32_t tm = uni(tmem);
      auto issue_s = [&](int slot, int stage) {
        const uint64_t dq = dq0 + (uint64_t)((slot * SM::kOp) >> 4), dk = dk0 + (uint64_t)uni((stage * SM::kOp) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (uint32_t)(((kk / 4) * kCRegion + (kk % 4) * 32) >> 4);
          umma_f16_by(lead, tm + slot * kCKeys, dq + off, dk + off, idS, kk > 0 ? 1u : 0u);
        }
        mbar_arrive_by(lead, &bars.s_full[slot]);
        umma_commit_by(lead, &bars.s_full[slot]);
      };
      auto issue_pv = [&](int slot, int stage, bool acc) {
        const uint64_t dv = dv0 + (uint64_t)uni((stage * SM::kOp) >> 4);
        const uint32_t ac = uni(acc ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < kCKeys / 16; ++kk)
          umma_f16_ts_by(lead, tm + (2 + slot) * kCKeys, tm + slot * kCKeys + kk * 8, dv + (uint64_t)((kk * 2048) >> 4),
                         idO, kk > 0 ? 1u : ac);
      };
      auto commit = [&](uint64_t* bar) { umma_commit_by(lead, bar); };
      auto wait = [&](uint64_t* bar, uint32_t par) { return c_wait(bar, par, a, &s_abort); };
      auto wait_tmem = [&](uint64_t* bar, uint32_t par) {  // for what other warps did to TMEM
        const bool ok = c_wait(bar, par, a, &s_abort);
        tc_fence_after();
        return ok;
      };
      int T = 0;
      uint32_t seg0 = 0u, seg1 = 0u, ph1 = 0u;  // items of each slot; phase of slot 1's weights
      bool owed = false, owed_first = false, owed_last = false;  // PV1 of the tile before is still to issue
      auto pay = [&]() {  // PV1 of tile T - 1
        if (!wait_tmem(&bars.p_full[1], ph1)) return false;
        if (owed_first && !wait_tmem(&bars.o_empty[1], (seg1 & 1u) ^ 1u)) return false;  // the last item's O has been read
        ph1 ^= 1u;
        issue_pv(1, (T - 1) & 1, !owed_first);
        commit(&bars.v_empty[(T - 1) & 1]);
        if (owed_last) {
          commit(&bars.o_full[1]);
          ++seg1;
        }
        owed = false;
        return true;
      };
      CWalk w;
      bool ok = true;
      for (bool more = w.start(a); more && ok; more = w.next(a)) {
        uint32_t q1 = 0u;
        for (int i = 0; i < w.nt; ++i, ++T) {
          const int st = T & 1;
          const uint32_t par = (uint32_t)(T >> 1) & 1u;
          const bool first = i == 0, last = i + 1 == w.nt;
          if (first && !(ok = wait(&bars.q_full[0], seg0 & 1u))) break;
          if (!(ok = wait(&bars.k_full[st], par))) break;
          issue_s(0, st);
          if (last) commit(&bars.q_empty[0]);
          if (owed && !(ok = pay())) break;
          if (w.two) {
            if (first) {
              q1 = seg1 & 1u;
              if (!(ok = wait(&bars.q_full[1], q1))) break;
            }
            issue_s(1, st);
            if (last) commit(&bars.q_empty[1]);
          }
          commit(&bars.k_empty[st]);
          if (!(ok = wait(&bars.v_full[st], par))) break;
          if (!(ok = wait_tmem(&bars.p_full[0], (uint32_t)T & 1u))) break;
          if (first && !(ok = wait_tmem(&bars.o_empty[0], (seg0 & 1u) ^ 1u))) break;
          issue_pv(0, st, !first);
          if (last) {
            commit(&bars.o_full[0]);
            ++seg0;
          }
          if (w.two) {
            owed = true;
            owed_first = first;
            owed_last = last;
          } else {
            commit(&bars.v_empty[st]);
          }
        }
      }
      if (ok && owed) pay();
      // every product issued has completed before TMEM is freed
      commit(&bars.fin);
      mbar_wait_bounded(&bars.fin, 0u, a.wait_ns, a.pool.status);
    } else if (warp == 13) {
      // ---- loads: Q (128 rows of a slot are 128 / G tokens of the group's G
      // heads), then the tiles' rows from their blocks ----
      CWalk w;
      uint32_t nq[2] = {0u, 0u}, nr[2] = {0u, 0u};  // loads so far: each slot's Q; K rows and V rows
      int T = 0, flags = 0;
      bool ok = true;
      for (bool more = w.start(a); more && ok; more = w.next(a)) {
        float2 span = make_float2(CUDART_INF_F, -CUDART_INF_F);
        for (int i = 0; i < w.nt && ok; ++i, ++T) {
          // lane g < 8: the block of positions [16 g, 16 g + 16) of the tile; -1: there is none
          int id = -1;
          const int j = tile_pos(w.c, w.u0 + i) + 16 * (lane & 7);
          if (j <= w.c.i_hi) {
            id = a.c.block_table[(size_t)w.c.b * a.pool.table_cols + (j >> a.pool.log_bs)];
            if ((unsigned)id >= (unsigned)a.pool.n_blocks) {
              flags |= RTP_DEV_BLOCKS;
              id = -1;
            }
          }
          ok = load_rows_of_tile<D>(a, w, T, id, bars, dsm + SM::kOffRaw, s_meta, &s_abort, nr, span);
          if (i > 0) continue;
          for (int slot = 0; slot < (w.two ? 2 : 1) && ok; ++slot) {
            if (!(ok = c_wait(&bars.q_empty[slot], (nq[slot] & 1u) ^ 1u, a, &s_abort))) break;
            if (lane == 0) {
              mbar_expect_tx(&bars.q_full[slot], (uint32_t)SM::kOp);
#pragma unroll
              for (int x = 0; x < D / 64; ++x)
                tma_load_3d(dsm + SM::kOffQ + slot * SM::kOp + x * kCRegion, &a.tm_q, x * 64, w.c.h * a.G,
                            w.c.q0 + ((w.c.row0 + slot * kCRows) >> a.log_g), &bars.q_full[slot]);
            }
            __syncwarp();
            ++nq[slot];
          }
        }
      }
      if (flags) atomicOr(a.pool.status, flags);
      // where the CTA gave up, its copies land before it leaves
      for (int x = 0; x < 2; ++x) {
        if (nq[x] > 0) mbar_wait_bounded(&bars.q_full[x], (nq[x] - 1u) & 1u, a.wait_ns, a.pool.status);
        if (nr[x] > 0) mbar_wait_bounded(&bars.raw_full[x], (nr[x] - 1u) & 1u, a.wait_ns, a.pool.status);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kCTmemCols) : "memory");
  }
}

// Joins the partials of the items that cuts of the line go through: CTA column x
// is the cut ahead of share x + 1, and works if it is its item's first.
template <int D>
__global__ void __launch_bounds__(256) attn_q8_chunk_join_kernel(const __grid_constant__ AttnQ8Args a) {
  // a CTA takes 64 rows and half the dims, a thread J times four of them: the chain of loads
  // that finds the item and its weights is walked once
  constexpr int kRows = 64, J = D / 32;
  griddep_wait();
  const int n_items = a.req_items[a.B];
  const long long total = a.prefix[n_items], share = a.prefix[a.max_chunk_items + 1];
  const int cut = blockIdx.x + 1;
  const long long at = cut * share;
  if (at >= total) return;
  const int item = find_item(a.prefix, n_items, at);
  const long long first = a.prefix[item];
  if (first == at || at - share > first) return;  // between two items, or not the item's first cut
  const ChunkItem c = a.items[item];
  if (at - first >= c.tiles) return;
  const int c1 = (int)((first + c.tiles - 1) / share);
  const int r = (blockIdx.y & 3) * kRows + (threadIdx.x & 63), d4 = (blockIdx.y >> 2) * (D / 8) + (threadIdx.x >> 6) * J;
  if (r >= c.n_rows) return;
  // the share that starts the item keeps its partial second, the later ones first
  auto part = [&](int k) { return (size_t)(k == cut - 1 ? 2 * k + 1 : 2 * k); };
  float m = -CUDART_INF_F;
  for (int k = cut - 1; k <= c1; ++k) m = fmaxf(m, a.cpart_ml[(part(k) * kCGroup + r) * 2]);
  const float ms = m == -CUDART_INF_F ? 0.f : m;
  float4 o[J];
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 2
  for (int k = cut - 1; k <= c1; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(a.cpart_ml + (part(k) * kCGroup + r) * 2);
    float4 p[J];
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = *reinterpret_cast<const float4*>(a.cpart + ((part(k) * (D / 4) + d4 + j) * kCGroup + r) * 4);
    const float f = ex2f(ml.x - ms);
    l += lower(ml.y, ml.x - ms);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      o[j].x = fmaf(p[j].x, f, o[j].x);
      o[j].y = fmaf(p[j].y, f, o[j].y);
      o[j].z = fmaf(p[j].z, f, o[j].z);
      o[j].w = fmaf(p[j].w, f, o[j].w);
    }
  }
  const int tok = c.q0 + ((c.row0 + r) >> a.log_g), hq = c.h * a.G + ((c.row0 + r) & (a.G - 1));
  const float inv = l == 0.f ? 0.f : kAqSumUnit / l;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.c.out) + ((size_t)tok * a.Hq + hq) * D + d4 * 4;
#pragma unroll
  for (int j = 0; j < J; j += 2) {
    uint4 v;
    v.x = pack_bf16(o[j].x * inv, o[j].y * inv);
    v.y = pack_bf16(o[j].z * inv, o[j].w * inv);
    v.z = pack_bf16(o[j + 1].x * inv, o[j + 1].y * inv);
    v.w = pack_bf16(o[j + 1].z * inv, o[j + 1].w * inv);
    *reinterpret_cast<uint4*>(out + j * 4) = v;
  }
}

long long max_chunk_items(const Shape& sh, int n_tokens, int max_q, int small) {
  // sum over requests of ceil(n G / 256), each of more than `small` rows
  const long long rows = (long long)n_tokens * sh.G;
  long long reqs = rows / (small + 1);
  if (reqs > sh.B) reqs = sh.B;
  const long long by_rows = rows / kCGroup + reqs;
  const long long by_max = reqs * (((long long)max_q * sh.G + kCGroup - 1) / kCGroup);
  return sh.Hkv * (by_rows < by_max ? by_rows : by_max);
}

struct ChunkLayout {
  size_t prefix, items, reqs, part, ml, q, unit, total;
};
ChunkLayout chunk_layout(const Shape& sh, int n_tokens, long long items) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  ChunkLayout l;
  l.prefix = 0;
  l.items = up((size_t)(items + 2) * sizeof(long long));
  l.reqs = l.items + up((size_t)items * sizeof(ChunkItem));
  l.part = l.reqs + up((size_t)(sh.B + 1) * sizeof(int));
  l.ml = l.part + (size_t)2 * kCCtas * kCGroup * sh.D * sizeof(float);
  l.q = l.ml + up((size_t)2 * kCCtas * kCGroup * 2 * sizeof(float));
  l.unit = l.q + up((size_t)n_tokens * sh.Hq * sh.D * sizeof(__half));
  l.total = l.unit + up((size_t)n_tokens * sh.Hq * sizeof(float));
  return l;
}

template <int D>
cudaError_t launch_chunks(const AttnQ8Args& a, cudaStream_t st) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(attn_q8_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CSmem<D>::kBytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  const long long tasks = (long long)a.c.n_tokens * ((a.Hq + 7) / 8);
  e = launch_pdl(chunk_prep_kernel<D>, dim3((unsigned)(1 + (tasks + kCPrep / 32 - 1) / (kCPrep / 32))), dim3(kCPrep), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(attn_q8_chunk_kernel<D>, dim3(kCCtas), dim3(kCThreads), CSmem<D>::kBytes, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(attn_q8_chunk_join_kernel<D>, dim3(kCCtas - 1, 2 * kCGroup / 64), dim3(256), 0, st, a);
  return e;
}

}  // namespace

size_t chunk_workspace_bytes(const Shape& sh, int n_tokens, int max_q, int small_rows) {
  return chunk_layout(sh, n_tokens, max_chunk_items(sh, n_tokens, max_q, small_rows)).total;
}

bool chunk_carve(const Shape& sh, int n_tokens, int max_q, int small_rows, void* ws, AttnQ8Args* a) {
  const unsigned long long rows = ((unsigned long long)a->pool.n_blocks * sh.Hkv) << a->pool.log_bs;
  const unsigned box_rows = 1u << a->pool.log_bs;
  if (!make_tensor_map(&a->tm_ck, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a->pool.k, sh.D, rows, sh.D, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !make_tensor_map(&a->tm_cv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a->pool.v, sh.D, rows, sh.D, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return false;
  const long long items = max_chunk_items(sh, n_tokens, max_q, small_rows);
  const ChunkLayout l = chunk_layout(sh, n_tokens, items);
  unsigned char* p = static_cast<unsigned char*>(ws);
  a->prefix = reinterpret_cast<long long*>(p + l.prefix);
  a->items = reinterpret_cast<ChunkItem*>(p + l.items);
  a->req_items = reinterpret_cast<int*>(p + l.reqs);
  a->cpart = reinterpret_cast<float*>(p + l.part);
  a->cpart_ml = reinterpret_cast<float*>(p + l.ml);
  a->max_chunk_items = (int)items;
  a->cq = reinterpret_cast<__half*>(p + l.q);
  a->cq_unit = reinterpret_cast<float*>(p + l.unit);
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)sh.D, (cuuint64_t)sh.Hq, (cuuint64_t)n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)sh.D * 2, (cuuint64_t)sh.Hq * sh.D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)sh.G, (cuuint32_t)(kCRows / sh.G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(&a->tm_q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, a->cq, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attn_q8_chunks(const Shape& sh, const AttnQ8Args& a, cudaStream_t st) {
  return sh.D == 128 ? launch_chunks<128>(a, st) : launch_chunks<64>(a, st);
}

}  // namespace rtp
