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
// is 128 positions.  The tiles of all items form one line that is cut into equal
// shares, one a CTA (one an SM): causal triangles, windows and ragged batches
// load the SMs evenly.  A cut item leaves partials that a second kernel joins.  A first,
// one-CTA kernel lays the line out.
//
// Roles (13 warps):
//   warps 0-3, 4-7   the softmax of slot 0 and slot 1 (128 rows each), one
//                    thread a row: its weights against the running maximum as
//                    S is read from TMEM once, kept packed in registers until
//                    the tile's maximum is known not to exceed it by 2^8 (else
//                    O is rescaled and the weights formed again), then written
//                    over S in TMEM;
//   warps 8-11       fetch K and V from their blocks into registers one tile
//                    ahead, convert e4m3 to fp16 and store the operands' swizzled layout
//                    (fetching through registers and not by TMA saves a pass
//                    through shared memory, whose bandwidth the products need);
//   warp 12          issues the products in the order S0(i), PV1(i-1), S1(i),
//                    PV0(i): each slot's softmax runs beside the other's products.
//
// Every wait is bounded: on expiry the CTA sets RTP_DEV_TIMEOUT, stops issuing,
// waits (bounded) for what it issued and frees its TMEM.
//
// Bound: the tensor cores.  A tile of 256 x 128 pairs at D = 128 is 16.8 MFLOP,
// 2048 clocks at the dense fp16 rate; its weights are 32768 exponentials, 2048
// clocks of the MUFU pipe, of which a quarter go to the FMA pipe.
#include <mutex>

#include "attn_q8.cuh"
#include "tc.cuh"

namespace rtp {
namespace {

constexpr int kCRows = 128;               // query rows a slot = TMEM lanes
constexpr int kCGroup = 256;              // query rows an item
constexpr int kCKeys = 128;               // positions a tile
constexpr int kCThreads = 13 * 32;
constexpr int kCRegion = 128 * 128;       // bytes of 128 rows x 64 fp16 dims
constexpr int kCCtas = 148;               // one an SM of a B200
constexpr int kCMinShare = 4;             // tiles a CTA takes at least: a segment's start and end cost about as much
constexpr int kCTmemCols = 512;

template <int D>
struct CSmem {
  static constexpr int kOp = (D / 64) * kCRegion;  // one operand tile: Q of a slot, K or V of a stage
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kOp;
  static constexpr int kOffV = kOffK + 2 * kOp;
  static constexpr int kBytes = kOffV + 2 * kOp + 1024;  // + alignment slack
};

// Scales of 16 positions of a tile, and which 32-position words are there.
struct __align__(16) CMeta {
  float4 g[8];  // k scale, log2(v scale), 1 / v scale
  uint32_t there[4];
};

// An item's geometry.
struct CItem {
  int q0, n, i0, n_rows, row0, i_lo, i_hi, ns, w0, tiles;
  bool ret;
  __device__ __forceinline__ int key(int u) const { return (ret || u < ns ? u : w0 + u - ns) * kCKeys; }
};

__device__ __forceinline__ CItem chunk_item(const AttnQ8Args& a, const ReqRows& r, int h, int grp) {
  CItem c;
  c.q0 = r.q0;
  c.n = r.n;
  c.i0 = r.L - r.n;
  c.row0 = grp * kCGroup;
  c.n_rows = min(kCGroup, r.n * a.G - c.row0);
  c.i_lo = c.i0 + c.row0 / a.G;
  c.i_hi = c.i0 + (c.row0 + c.n_rows - 1) / a.G;
  c.ret = (a.ret_mask >> h) & 1ull;
  const int nt = c.i_hi / kCKeys + 1;
  c.ns = min((a.S + kCKeys - 1) / kCKeys, nt);
  c.w0 = max(0, c.i_lo - a.W + 1) / kCKeys;
  if (c.ret || c.w0 <= c.ns) {
    c.ns = c.w0 = 0;
    c.tiles = nt;
  } else {
    c.tiles = c.ns + nt - c.w0;
  }
  return c;
}

__device__ __forceinline__ long long chunk_share(long long total) {
  return max((total + kCCtas - 1) / kCCtas, (long long)kCMinShare);
}

// Exclusive scan over the block (1024 threads) and its total.
__device__ __forceinline__ long long block_scan_1024(long long v, long long& total, long long* s_warp) {
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
  long long w = s_warp[lane], ws = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += y;
  }
  total = __shfl_sync(0xffffffffu, ws, 31);
  return x - v + __shfl_sync(0xffffffffu, ws - w, warp);
}

// The line: items in the order (request, KV head, group), and the tiles ahead of each.
__global__ void __launch_bounds__(1024) chunk_line_kernel(const __grid_constant__ AttnQ8Args a) {
  __shared__ long long s_warp[32];
  griddep_wait();
  int flags = 0;
  long long n_items = 0;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    long long v = 0;
    if (b < a.B) {
      const ReqRows r = load_rows(a, b, flags);
      const long long rows = (long long)r.n * a.G;
      if (rows > a.small_rows) v = a.Hkv * ((rows + kCGroup - 1) / kCGroup);
    }
    long long total;
    const long long x = n_items + block_scan_1024(v, total, s_warp);
    if (b < a.B) a.req_items[b] = (int)min(x, (long long)a.max_chunk_items);
    n_items += total;
  }
  n_items = min(n_items, (long long)a.max_chunk_items);  // more only if cu_q goes back and forth
  if (threadIdx.x == 0) a.req_items[a.B] = (int)n_items;
  __syncthreads();
  long long tiles = 0;
  for (int i0 = 0; i0 < n_items; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    long long v = 0;
    ChunkItem it = {0, 0, 0, 0};
    if (i < n_items) {
      int b = 0, hi = a.B;  // the last request with req_items <= i
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (a.req_items[mid] <= i) b = mid;
        else hi = mid;
      }
      const ReqRows r = load_rows(a, b, flags);
      const int ng = (r.n * a.G + kCGroup - 1) / kCGroup, rel = i - a.req_items[b];
      it.b = b;
      it.h = rel / ng;
      it.grp = rel % ng;
      it.tiles = chunk_item(a, r, it.h, it.grp).tiles;
      v = it.tiles;
    }
    long long total;
    const long long x = tiles + block_scan_1024(v, total, s_warp);
    if (i < n_items) {
      a.items[i] = it;
      a.prefix[i] = x;
    }
    tiles += total;
  }
  if (threadIdx.x == 0) a.prefix[n_items] = tiles;
  if (flags) atomicOr(a.pool.status, flags);
}

// The item whose tiles hold line position `at` (one warp; prefix[n] > at).
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

__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
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

__device__ __forceinline__ bool c_wait(uint64_t* bar, uint32_t parity, const AttnQ8Args& a, volatile int* s_abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_sleep(bar, parity, kWaitHintNs)) {
    if (*s_abort) return false;
    if (global_ns() - t0 > a.wait_ns) {
      *s_abort = 1;
      atomicOr(a.pool.status, RTP_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kCThreads, 1) attn_q8_chunk_kernel(const __grid_constant__ AttnQ8Args a) {
  using SM = CSmem<D>;
  constexpr int H = D / 2;
  extern __shared__ __align__(1024) unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t bar_k_full[2], bar_k_empty[2], bar_v_full[2], bar_v_empty[2];
  __shared__ __align__(8) uint64_t bar_s_full[2], bar_p_full[2], bar_o_done, bar_fin;
  // tile i's scales, read by the softmax after S(i); rewritten for tile i + 4, after S1(i + 2)
  // has completed, which follows both slots' weights of tile i + 1
  __shared__ CMeta s_meta[4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_item;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* dsm = dsm_raw + ((1024u - (smem_u32(dsm_raw) & 1023u)) & 1023u);
  const uint32_t sQ = smem_u32(dsm + SM::kOffQ), sK = smem_u32(dsm + SM::kOffK), sV = smem_u32(dsm + SM::kOffV);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar_k_full[s], 128);
      mbar_init(&bar_k_empty[s], 1);
      mbar_init(&bar_v_full[s], 128);
      mbar_init(&bar_v_empty[s], 1);
      mbar_init(&bar_s_full[s], 2);  // the products' commit, and the issuer (who has seen the scales)
      mbar_init(&bar_p_full[s], kCRows);
    }
    mbar_init(&bar_o_done, 1);
    mbar_init(&bar_fin, 1);
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

  const int n_items = a.req_items[a.B];
  const long long total = a.prefix[n_items], share = chunk_share(total);
  long long at = (long long)blockIdx.x * share;
  const long long end = min(total, at + share);
  int flags = 0;
  // tiles so far: phases of the K and V stages, and of each slot's barriers (slot 1 idles where an item has no row for it)
  int gt = 0, gs1 = 0;
  uint32_t seg_par = 0u;
  if (at < end && warp == 0) {
    const int it = find_item(a.prefix, n_items, at);
    if (lane == 0) s_item = it;
  }
  __syncthreads();
  int item = s_item;

  while (at < end) {
    const ChunkItem ci = a.items[item];
    int dummy = 0;
    const ReqRows rr = load_rows(a, ci.b, dummy);
    const CItem c = chunk_item(a, rr, ci.h, ci.grp);
    const int h = ci.h;
    const int u0 = (int)(at - a.prefix[item]);
    const int nt = (int)min((long long)c.tiles - u0, end - at);  // tiles [u0, u0 + nt) of the item
    const bool two = c.n_rows > kCRows;
    // ---- Q: cos and sin of the item's tokens (over the K stages), then each
    // row rotated, scaled by its power of two and stored as fp16, swizzled ----
    float2* s_cs = reinterpret_cast<float2*>(dsm + SM::kOffK);
    const int tok0 = c.row0 / a.G, n_tok = (c.row0 + c.n_rows - 1) / a.G - tok0 + 1;
    float rs = 1.f;  // the thread's row: factor from products to base-2 logits
    static_assert(4 * SM::kOp >= kCGroup * H * (int)sizeof(float2), "the table fits over the K and V stages");
    for (int i = tid; i < n_tok * H; i += kCThreads) {
      const int t = c.q0 + tok0 + i / H, k = i % H;
      float2 cs;
      rope_cos_sin(a.c.pos[(size_t)a.rope.axis[k] * a.c.n_tokens + t], a.inv_freq[k], cs.x, cs.y);
      s_cs[i] = cs;
    }
    __syncthreads();
    if (warp < 8) {
      const int r = tid;  // row of the item
      unsigned char* qs = dsm + SM::kOffQ + (r / kCRows) * SM::kOp + (r % kCRows) * 128;
      if (r < c.n_rows) {
        const int tl = (c.row0 + r) / a.G - tok0;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.c.q_pre) +
                                 (size_t)(c.q0 + tok0 + tl) * a.c.q_stride + (size_t)(h * a.G + (c.row0 + r) % a.G) * D;
        const float2* cs = s_cs + tl * H;
        float m = 0.f;
#pragma unroll 2
        for (int k8 = 0; k8 < H; k8 += 8) {
          float x1[8], x2[8];
          load_row<__nv_bfloat16, 8>(q + k8, x1);
          load_row<__nv_bfloat16, 8>(q + H + k8, x2);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = cs[k8 + e];
            m = fmaxf(m, fmaxf(fabsf(x1[e] * f.x - x2[e] * f.y), fabsf(x2[e] * f.x + x1[e] * f.y)));
          }
        }
        const float s = query_scale(m), inv = 1.f / s;
        rs = s * (1.4426950408889634f * rsqrtf((float)D));
#pragma unroll 2
        for (int k8 = 0; k8 < H; k8 += 8) {
          float x1[8], x2[8];
          load_row<__nv_bfloat16, 8>(q + k8, x1);
          load_row<__nv_bfloat16, 8>(q + H + k8, x2);
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 f = cs[k8 + e], g = cs[k8 + e + 1];
            lo[e / 2] = pack_f16((x1[e] * f.x - x2[e] * f.y) * inv, (x1[e + 1] * g.x - x2[e + 1] * g.y) * inv);
            hi[e / 2] = pack_f16((x2[e] * f.x + x1[e] * f.y) * inv, (x2[e + 1] * g.x + x1[e + 1] * g.y) * inv);
          }
          const int d1 = k8, d2 = H + k8;
          *reinterpret_cast<uint4*>(qs + (d1 / 64) * kCRegion + ((((d1 % 64) / 8) ^ (r & 7)) * 16)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          *reinterpret_cast<uint4*>(qs + (d2 / 64) * kCRegion + ((((d2 % 64) / 8) ^ (r & 7)) * 16)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
      } else if (r < kCRows || two) {  // rows that the item does not have
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          *reinterpret_cast<uint4*>(qs + (k / 8) * kCRegion + (k % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    fence_async_smem();
    __syncthreads();

    if (warp >= 8 && warp < 12) {
      // ---- K and V: fetched a tile ahead, converted, stored ----
      constexpr int LPR = D / 16;          // lanes a row (16 bytes each)
      constexpr int RPI = 4 * (32 / LPR);  // rows the four warps fetch at once
      constexpr int IT = kCKeys / RPI;
      const int cw = warp - 8;
      const int r_lane = cw * (32 / LPR) + lane / LPR, cl = lane % LPR;
      const int bs1 = (1 << a.pool.log_bs) - 1;
      const int* tab = a.c.block_table + (size_t)ci.b * a.pool.table_cols;
      // lane g < 8: the block of positions [16 g, 16 g + 16) of tile u, -1 if it has none
      auto block_id = [&](int u) {
        const int j = c.key(u) + 16 * (lane & 7);
        if (j > c.i_hi) return -1;
        const int id = tab[j >> a.pool.log_bs];
        if ((unsigned)id < (unsigned)a.pool.n_blocks) return id;
        flags |= RTP_DEV_BLOCKS;
        return -1;
      };
      auto fetch = [&](const void* pool, int u, int id, uint4 (&x)[IT]) {
        const int j0 = c.key(u);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int r = i * RPI + r_lane, j = j0 + r;
          const int blk = __shfl_sync(0xffffffffu, id, r >> 4);
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (blk >= 0 && j <= c.i_hi)
            x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(pool) +
                         (((((size_t)blk * a.Hkv + h) << a.pool.log_bs) + (j & bs1)) * D + cl * 16)));
        }
      };
      auto store = [&](unsigned char* dst, const uint4 (&x)[IT]) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int r = i * RPI + r_lane;
          const uint4 lo = make_uint4(e4m3x2_to_f16x2(x[i].x), e4m3x2_to_f16x2(x[i].x >> 16),
                                      e4m3x2_to_f16x2(x[i].y), e4m3x2_to_f16x2(x[i].y >> 16));
          const uint4 hi = make_uint4(e4m3x2_to_f16x2(x[i].z), e4m3x2_to_f16x2(x[i].z >> 16),
                                      e4m3x2_to_f16x2(x[i].w), e4m3x2_to_f16x2(x[i].w >> 16));
          // 16 dims are two 16-byte chunks of a 64-dim region; lanes of the two
          // regions take them in opposite order, so eight lanes hit eight chunks
          const int reg = cl >> 2, ch = (2 * cl) & 7, odd = reg & 1;
          unsigned char* p = dst + reg * kCRegion + r * 128;
          *reinterpret_cast<uint4*>(p + (((ch + odd) ^ (r & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(p + (((ch + 1 - odd) ^ (r & 7)) << 4)) = odd ? lo : hi;
        }
      };
      uint4 xk[IT], xv[IT];
      int id = block_id(u0);
      fetch(a.pool.k, u0, id, xk);
      fetch(a.pool.v, u0, id, xv);
      float ks = 0.f, vs = 0.f;
      if (cw == 0 && id >= 0) {
        ks = a.pool.k_scale[(size_t)id * a.Hkv + h];
        vs = a.pool.v_scale[(size_t)id * a.Hkv + h];
      }
      for (int i = 0; i < nt; ++i) {
        const int T = gt + i, st = T & 1;
        const uint32_t par = ((uint32_t)(T >> 1) & 1u) ^ 1u;
        const int id_next = i + 1 < nt ? block_id(u0 + i + 1) : -1;
        if (!__all_sync(0xffffffffu, c_wait(&bar_k_empty[st], par, a, &s_abort))) break;
        store(dsm + SM::kOffK + st * SM::kOp, xk);
        if (cw == 0) {
          CMeta& m = s_meta[T & 3];
          const unsigned there = __ballot_sync(0xffffffffu, lane < 8 && id >= 0);
          vs = fmaxf(vs, kQ8ScaleMin);
          if (lane < 8) m.g[lane] = make_float4(fmaxf(ks, kQ8ScaleMin), __log2f(vs), 1.f / vs, 0.f);
          if (lane < 4) m.there[lane] = ((there >> (2 * lane) & 1u) ? 0xffffu : 0u) | ((there >> (2 * lane + 1) & 1u) ? 0xffff0000u : 0u);
          ks = vs = 0.f;
          if (id_next >= 0) {
            ks = a.pool.k_scale[(size_t)id_next * a.Hkv + h];
            vs = a.pool.v_scale[(size_t)id_next * a.Hkv + h];
          }
        }
        if (i + 1 < nt) fetch(a.pool.k, u0 + i + 1, id_next, xk);
        fence_async_smem();
        mbar_arrive(&bar_k_full[st]);
        if (!__all_sync(0xffffffffu, c_wait(&bar_v_empty[st], par, a, &s_abort))) break;
        store(dsm + SM::kOffV + st * SM::kOp, xv);
        if (i + 1 < nt) fetch(a.pool.v, u0 + i + 1, id_next, xv);
        fence_async_smem();
        mbar_arrive(&bar_v_full[st]);
        id = id_next;
      }
    } else if (warp == 12) {
      // ---- the products ----
      constexpr uint32_t idS = umma_idesc(kCRows, kCKeys, false, true);
      constexpr uint32_t idO = umma_idesc(kCRows, D, true, true);
      const uint32_t tS[2] = {tmem, tmem + kCKeys};
      const uint32_t tO[2] = {tmem + 2 * kCKeys, tmem + 3 * kCKeys};
      const uint64_t dq0 = umma_desc(sQ, 16, 1024), dk0 = umma_desc(sK, 16, 1024), dv0 = umma_desc(sV, kCRegion, 1024);
      auto issue_s = [&](int slot, int st) {
        if (lane == 0) {
          const uint64_t dq = dq0 + (uint64_t)((slot * SM::kOp) >> 4), dk = dk0 + (uint64_t)((st * SM::kOp) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (uint32_t)(((kk / 4) * kCRegion + (kk % 4) * 32) >> 4);
            umma_f16(tS[slot], dq + off, dk + off, idS, kk > 0 ? 1u : 0u);
          }
          mbar_arrive(&bar_s_full[slot]);
          umma_commit(&bar_s_full[slot]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int slot, int st, bool acc) {
        if (lane == 0) {
          const uint64_t dv = dv0 + (uint64_t)((st * SM::kOp) >> 4);
#pragma unroll
          for (int kk = 0; kk < kCKeys / 16; ++kk)
            umma_f16_ts(tO[slot], tS[slot] + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), idO, (acc || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t par) {
        const bool ok = __all_sync(0xffffffffu, c_wait(bar, par, a, &s_abort));
        tc_fence_after();
        return ok;
      };
      bool ok = true;
      for (int i = 0; i < nt && ok; ++i) {
        const int T = gt + i, st = T & 1;
        const uint32_t par = (uint32_t)(T >> 1) & 1u;
        ok = wait(&bar_k_full[st], par);
        if (!ok) break;
        issue_s(0, st);
        if (two) {
          if (i > 0) {
            ok = wait(&bar_p_full[1], (uint32_t)(gs1 + i - 1) & 1u);
            if (!ok) break;
            issue_pv(1, st ^ 1, i > 1);
            if (lane == 0) umma_commit(&bar_v_empty[st ^ 1]);
          }
          issue_s(1, st);
        }
        if (lane == 0) umma_commit(&bar_k_empty[st]);
        ok = wait(&bar_v_full[st], par);
        if (!ok) break;
        ok = wait(&bar_p_full[0], (uint32_t)T & 1u);
        if (!ok) break;
        issue_pv(0, st, i > 0);
        if (!two && lane == 0) umma_commit(&bar_v_empty[st]);
      }
      if (ok && two) {
        ok = wait(&bar_p_full[1], (uint32_t)(gs1 + nt - 1) & 1u);
        if (ok) {
          issue_pv(1, (gt + nt - 1) & 1, nt > 1);
          if (lane == 0) umma_commit(&bar_v_empty[(gt + nt - 1) & 1]);
        }
      }
      if (lane == 0) umma_commit(&bar_o_done);
      __syncwarp();
    } else if (warp < 8) {
      // ---- softmax: one thread a row ----
      const int slot = warp >> 2, quad = warp & 3;
      if (slot == 0 || two) {
        const int r = tid;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tSs = tmem + slot * kCKeys + lane_off, tOs = tmem + (2 + slot) * kCKeys + lane_off;
        const bool rv = r < c.n_rows;
        const int pi = c.i0 + (c.row0 + r) / a.G;          // the row's position
        const int s_lo = c.i0 + (c.row0 + slot * kCRows) / a.G;  // the slot's first, and its last row's
        const int s_hi = min(c.i_hi, c.i0 + (c.row0 + slot * kCRows + kCRows - 1) / a.G);
        const int g0 = slot == 0 ? gt : gs1;
        float M = -CUDART_INF_F, l = 0.f;
        bool ok = true, poison = false;
        for (int i = 0; i < nt; ++i) {
          const int kt = c.key(u0 + i);
          if (!__all_sync(0xffffffffu, c_wait(&bar_s_full[slot], (uint32_t)(g0 + i) & 1u, a, &s_abort))) { ok = false; break; }
          tc_fence_after();
          const CMeta& m = s_meta[(gt + i) & 3];
          const bool whole = kt + kCKeys - 1 <= s_lo && (c.ret || kt + kCKeys - 1 < a.S || kt > s_hi - a.W) &&
                             (m.there[0] & m.there[1] & m.there[2] & m.there[3]) == 0xffffffffu;
          auto keep_word = [&](int w) {  // of positions [kt + 32 w, + 32), those that the row sees
            const int base = kt + 32 * w;
            const int nc = pi - base + 1;
            const uint32_t causal = !rv || nc <= 0 ? 0u : nc >= 32 ? 0xffffffffu : (1u << nc) - 1u;
            uint32_t near = 0xffffffffu;
            if (!c.ret) {
              const int nsk = a.S - base, nw = pi - a.W + 1 - base;
              near = (nsk <= 0 ? 0u : nsk >= 32 ? 0xffffffffu : (1u << nsk) - 1u) |
                     (nw <= 0 ? 0xffffffffu : nw >= 32 ? 0u : ~((1u << nw) - 1u));
            }
            return causal & near & m.there[w];
          };
          // weights of 32 positions against `mm`, their packed fp16, the row's sum, and the largest logit
          auto chunk = [&](int w, float mm, uint32_t (&pk)[16], float& ls, float& mx) {
            float v[32];
            tmem_ld32(tSs + w * 32, v);
            tmem_wait_ld();
            if (!whole) {
              const uint32_t bits = keep_word(w);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = (bits >> e) & 1u ? v[e] : -CUDART_INF_F;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 g = m.g[2 * w + q];
              const float f = rs * g.x;
              float t = v[16 * q];
#pragma unroll
              for (int e = 1; e < 15; e += 2) t = max3_nan(t, v[16 * q + e], v[16 * q + e + 1]);
              t = max_nan(t, v[16 * q + 15]);
              mx = max_nan(mx, fmaf(t, f, g.y));
              const float add = g.y + kAqLift - mm;
              float s0 = 0.f, s1 = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float x0 = v[16 * q + 2 * e], x1 = v[16 * q + 2 * e + 1];
                fma2(x0, x1, f, add);
                const float p0 = ex2f(x0), p1 = (e & 1) ? ex2_poly(x1) : ex2f(x1);
                add2(s0, s1, p0, p1);
                pk[8 * q + e] = pack_f16(p0, p1);
              }
              ls = fmaf(s0 + s1, g.z, ls);
            }
          };
          const float mspec = M == -CUDART_INF_F ? 0.f : M;
          uint32_t pk[4][16];
          float ls = 0.f, mx = -CUDART_INF_F;
#pragma unroll
          for (int w = 0; w < 4; ++w) chunk(w, mspec, pk[w], ls, mx);
          if (mx != mx) {  // a stored NaN that the row sees
            poison = true;
            mx = -CUDART_INF_F;
          }
          float mn = M, f = 1.f;
          if (mx > M + kAqRescale || (M == -CUDART_INF_F && mx > M)) {
            mn = mx;
            f = M == -CUDART_INF_F ? 0.f : ex2f(M - mn);
          }
          if (__any_sync(0xffffffffu, mn != M)) {
            // PV of the slot's previous tile has completed (S(i) was issued after it)
            if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                float o[32];
                tmem_ld32(tOs + k * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) mul2(o[e], o[e + 1], f);
                tmem_st32(tOs + k * 32, o);
              }
            }
            ls = 0.f;
            float again = 0.f;
            const float ms = mn == -CUDART_INF_F ? 0.f : mn;
#pragma unroll
            for (int w = 0; w < 4; ++w) chunk(w, ms, pk[w], ls, again);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) tmem_st16(tSs + 16 * w, pk[w]);
          M = mn;
          l = fmaf(l, f, ls);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bar_p_full[slot]);
        }
        if (ok && __all_sync(0xffffffffu, c_wait(&bar_o_done, seg_par, a, &s_abort))) {
          tc_fence_after();
          if (poison) l = CUDART_NAN_F;
          const bool alone = u0 == 0 && nt == c.tiles;
          const int tok = c.q0 + (c.row0 + r) / a.G, hq = h * a.G + (c.row0 + r) % a.G;
          __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.c.out) + ((size_t)tok * a.Hq + hq) * D;
          const size_t prow = (size_t)(2 * blockIdx.x + (u0 > 0 ? 0 : 1)) * kCGroup + r;
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            float o[32];
            tmem_ld32(tOs + k * 32, o);
            tmem_wait_ld();
            if (!rv) continue;
            if (alone) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 v;
                v.x = pack_bf16(o[e] * inv, o[e + 1] * inv);
                v.y = pack_bf16(o[e + 2] * inv, o[e + 3] * inv);
                v.z = pack_bf16(o[e + 4] * inv, o[e + 5] * inv);
                v.w = pack_bf16(o[e + 6] * inv, o[e + 7] * inv);
                *reinterpret_cast<uint4*>(orow + k * 32 + e) = v;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(a.cpart + prow * D + k * 32 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (rv && !alone) *reinterpret_cast<float2*>(a.cpart_ml + prow * 2) = make_float2(M, l);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s_abort) break;  // uniform
    gt += nt;
    if (two) gs1 += nt;
    seg_par ^= 1u;
    at += nt;
    ++item;
  }
  if (flags) atomicOr(a.pool.status, flags);
  // every product issued has completed before TMEM is freed
  if (warp == 12) {
    if (lane == 0) {
      umma_commit(&bar_fin);
      mbar_wait_bounded(&bar_fin, 0u, a.wait_ns, a.pool.status);
    }
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kCTmemCols) : "memory");
  }
}

// Joins the partials of the items that cuts of the line go through: CTA column x
// is the cut ahead of share x + 1, and works if it is its item's first.
template <int D>
__global__ void __launch_bounds__(256) attn_q8_chunk_join_kernel(const __grid_constant__ AttnQ8Args a) {
  constexpr int LPR = D / 4;  // threads a row
  griddep_wait();
  const int n_items = a.req_items[a.B];
  const long long total = a.prefix[n_items], share = chunk_share(total);
  const int cut = blockIdx.x + 1;
  const long long at = cut * share;
  if (at >= total) return;
  const int item = find_item(a.prefix, n_items, at);
  const long long first = a.prefix[item];
  if (first == at || at - share > first) return;  // between two items, or not the item's first cut
  const int c1 = (int)((a.prefix[item + 1] - 1) / share);
  const ChunkItem ci = a.items[item];
  int dummy = 0;
  const CItem c = chunk_item(a, load_rows(a, ci.b, dummy), ci.h, ci.grp);
  const int r = blockIdx.y * (256 / LPR) + threadIdx.x / LPR, d = (threadIdx.x % LPR) * 4;
  if (r >= c.n_rows) return;
  // the share that starts the item keeps its partial second, the later ones first
  auto row = [&](int k) { return (size_t)(k == cut - 1 ? 2 * k + 1 : 2 * k) * kCGroup + r; };
  float m = -CUDART_INF_F;
  for (int k = cut - 1; k <= c1; ++k) m = fmaxf(m, a.cpart_ml[row(k) * 2]);
  const float ms = m == -CUDART_INF_F ? 0.f : m;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 2
  for (int k = cut - 1; k <= c1; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(a.cpart_ml + row(k) * 2);
    const float4 p = *reinterpret_cast<const float4*>(a.cpart + row(k) * D + d);
    const float f = ex2(ml.x - ms);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(p.x, f, o.x);
    o.y = fmaf(p.y, f, o.y);
    o.z = fmaf(p.z, f, o.z);
    o.w = fmaf(p.w, f, o.w);
  }
  const int tok = c.q0 + (c.row0 + r) / a.G, hq = ci.h * a.G + (c.row0 + r) % a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 v;
  v.x = pack_bf16(o.x * inv, o.y * inv);
  v.y = pack_bf16(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.c.out) + ((size_t)tok * a.Hq + hq) * D + d) = v;
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
  size_t prefix, items, reqs, part, ml, total;
};
ChunkLayout chunk_layout(const Shape& sh, long long items) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  ChunkLayout l;
  l.prefix = 0;
  l.items = up((size_t)(items + 1) * sizeof(long long));
  l.reqs = l.items + up((size_t)items * sizeof(ChunkItem));
  l.part = l.reqs + up((size_t)(sh.B + 1) * sizeof(int));
  l.ml = l.part + (size_t)2 * kCCtas * kCGroup * sh.D * sizeof(float);
  l.total = l.ml + up((size_t)2 * kCCtas * kCGroup * 2 * sizeof(float));
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
  e = launch_pdl(chunk_line_kernel, dim3(1), dim3(1024), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(attn_q8_chunk_kernel<D>, dim3(kCCtas), dim3(kCThreads), CSmem<D>::kBytes, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(attn_q8_chunk_join_kernel<D>, dim3(kCCtas - 1, kCGroup * (D / 4) / 256), dim3(256), 0, st, a);
  return e;
}

}  // namespace

size_t chunk_workspace_bytes(const Shape& sh, int n_tokens, int max_q, int small_rows) {
  return chunk_layout(sh, max_chunk_items(sh, n_tokens, max_q, small_rows)).total;
}

void chunk_carve(const Shape& sh, int n_tokens, int max_q, int small_rows, void* ws, AttnQ8Args* a) {
  const long long items = max_chunk_items(sh, n_tokens, max_q, small_rows);
  const ChunkLayout l = chunk_layout(sh, items);
  unsigned char* p = static_cast<unsigned char*>(ws);
  a->prefix = reinterpret_cast<long long*>(p + l.prefix);
  a->items = reinterpret_cast<ChunkItem*>(p + l.items);
  a->req_items = reinterpret_cast<int*>(p + l.reqs);
  a->cpart = reinterpret_cast<float*>(p + l.part);
  a->cpart_ml = reinterpret_cast<float*>(p + l.ml);
  a->max_chunk_items = (int)items;
}

cudaError_t launch_attn_q8_chunks(const Shape& sh, const AttnQ8Args& a, cudaStream_t st) {
  return sh.D == 128 ? launch_chunks<128>(a, st) : launch_chunks<64>(a, st);
}

}  // namespace rtp
