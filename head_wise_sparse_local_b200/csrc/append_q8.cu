// rtp_append_q8: rotary positions (one or several axes), then keys and values
// as e4m3 into their blocks, with a power-of-two scale for each (block, head).
//
// A run is a maximal stretch of packed tokens that go to consecutive slots of
// one block; its first token leads.  The scale needs the run's largest
// magnitude, so a group of warps holds a whole run of one head in registers (8
// rows a warp), reduces the maximum, and stores: every input is read once.
// Where a block already held rows and its scale grows, the group also rounds
// those rows again.
//
// The rotation is done in 64 bits and reaches the e4m3 rounding through a
// 32-bit value rounded to odd (truncated, the lowest bit set if anything was
// cut off): scaling it by a power of two is exact, and rounding it to nearest
// gives what rounding the 64-bit value would, so a stored value is off by one
// rounding and by nothing else.
//
// Bound: memory, the inputs read once and half (bf16) of their bytes written.
#include <cfloat>

#include "q8.cuh"

namespace rtp {
namespace {

constexpr int kAppWarps = 8;
constexpr int kAppRows = 8;  // rows a warp holds

struct AppQ8Args {
  Q8Pool pool;
  RopeAxes rope;
  int Hkv, n_tokens, tile, wpr, heads;  // wpr: warps a run; heads: KV heads a CTA goes through
  const void* k_pre;
  const void* v_in;
  long long k_stride, v_stride;
  const int64_t* slot;
  const int* pos;
  double inv_freq[64];
};

__device__ __forceinline__ float round_to_odd(double y) {
  float f = __double2float_rz(y);
  if ((double)f != y) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// One row of a head, as the lane holds it: the rotary pairs (k, k + D/2) for
// k = lane * PP + i, rotated, and the value dims of the same numbers.
template <int PP>
struct AppRow {
  float k1[PP], k2[PP], v1[PP], v2[PP];
};

template <typename T, int D>
__global__ void __launch_bounds__(kAppWarps * 32) append_q8_kernel(const __grid_constant__ AppQ8Args a) {
  constexpr int PP = D / 64, H = D / 2;
  extern __shared__ double2 s_cs[];  // [8 wpr rows][H] cos, sin
  __shared__ float s_max[kAppWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wpr = a.wpr, hpc = kAppWarps / wpr, sub = warp % wpr, grp = warp / wpr;
  const int bs = 1 << a.pool.log_bs;
  const long long n_slots = (long long)a.pool.n_blocks << a.pool.log_bs;
  const int rows_per = wpr * kAppRows;  // rows of a run a pass holds
  griddep_wait();
  griddep_launch();
  const int t0 = blockIdx.x * a.tile;
  // ---- this tile's leaders (every warp finds the same) ----
  unsigned leaders;
  {
    bool lead = false;
    const int t = t0 + lane;
    if (lane < a.tile && t < a.n_tokens) {
      const long long s = a.slot[t];
      if (s >= n_slots) atomicOr(a.pool.status, RTP_DEV_BLOCKS);
      else if (s >= 0) lead = t == 0 || (s & (bs - 1)) == 0 || a.slot[t - 1] != s - 1;
    }
    leaders = __ballot_sync(0xffffffffu, lead);
  }
  for (; leaders; leaders &= leaders - 1) {
    const int tl = t0 + __ffs(leaders) - 1;
    const long long s0 = a.slot[tl];
    const int off = (int)(s0 & (bs - 1));
    const size_t blk = (size_t)(s0 >> a.pool.log_bs);
    const int most = min(bs - off, a.n_tokens - tl);
    int n = 0;  // the run's tokens
    for (;;) {
      const bool in = n + lane < most && a.slot[tl + n + lane] == s0 + n + lane;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      if (m != 0xffffffffu) break;
    }
    const int passes = (n + rows_per - 1) / rows_per;
    auto fill_angles = [&](int base) {  // cos and sin of rows [base, base + rows_per) of the run
      for (int i = tid; i < min(rows_per, n - base) * H; i += kAppWarps * 32) {
        const int r = i / H, k = i % H;
        const int p = a.pos[(size_t)a.rope.axis[k] * a.n_tokens + tl + base + r];
        double sn, c;
        sincos((double)p * a.inv_freq[k], &sn, &c);
        s_cs[i] = make_double2(c, sn);
      }
    };
    __syncthreads();
    if (passes == 1) fill_angles(0);
    __syncthreads();
    for (int h0 = blockIdx.y * a.heads; h0 < min(a.Hkv, (int)(blockIdx.y + 1) * a.heads); h0 += hpc) {
      const int h = h0 + grp;
      const bool on = h < a.Hkv && h < (int)(blockIdx.y + 1) * a.heads;
      AppRow<PP> row[kAppRows];
      unsigned bad = 0;  // rows of this warp that hold a value that is not finite
      // rows [base + 8 sub, + 8) of the run into registers
      auto load = [&](int base) {
        bad = 0;
#pragma unroll
        for (int r = 0; r < kAppRows; ++r) {
          const int rr = sub * kAppRows + r;
          if (!on || base + rr >= n) continue;
          const size_t t = (size_t)(tl + base + rr);
          const T* kp = static_cast<const T*>(a.k_pre) + t * a.k_stride + (size_t)h * D;
          const T* vp = static_cast<const T*>(a.v_in) + t * a.v_stride + (size_t)h * D;
          bool fin = true;
#pragma unroll
          for (int i = 0; i < PP; ++i) {
            const int k = lane * PP + i;
            const double x1 = to_f32(kp[k]), x2 = to_f32(kp[k + H]);
            const double2 cs = s_cs[rr * H + k];
            const double y1 = x1 * cs.x - x2 * cs.y, y2 = x2 * cs.x + x1 * cs.y;
            fin = fin && fabs(y1) <= (double)FLT_MAX && fabs(y2) <= (double)FLT_MAX;
            row[r].k1[i] = round_to_odd(y1);
            row[r].k2[i] = round_to_odd(y2);
            row[r].v1[i] = to_f32(vp[k]);
            row[r].v2[i] = to_f32(vp[k + H]);
            fin = fin && fabsf(row[r].v1[i]) <= FLT_MAX && fabsf(row[r].v2[i]) <= FLT_MAX;
          }
          if (__any_sync(0xffffffffu, !fin)) bad |= 1u << r;
        }
      };
      auto grow = [&](int base, float& mk, float& mv) {
#pragma unroll
        for (int r = 0; r < kAppRows; ++r) {
          if (!on || base + sub * kAppRows + r >= n || (bad >> r & 1u)) continue;
#pragma unroll
          for (int i = 0; i < PP; ++i) {
            mk = fmaxf(mk, fmaxf(fabsf(row[r].k1[i]), fabsf(row[r].k2[i])));
            mv = fmaxf(mv, fmaxf(fabsf(row[r].v1[i]), fabsf(row[r].v2[i])));
          }
        }
      };
      float mk = 0.f, mv = 0.f;
      for (int p = 0; p < passes; ++p) {
        if (passes > 1) {
          __syncthreads();
          fill_angles(p * rows_per);
          __syncthreads();
        }
        load(p * rows_per);
        grow(p * rows_per, mk, mv);
      }
      mk = warp_max(mk);
      mv = warp_max(mv);
      if (wpr > 1) {
        __syncthreads();
        if (lane == 0) {
          s_max[warp][0] = mk;
          s_max[warp][1] = mv;
        }
        __syncthreads();
        for (int w = 0; w < wpr; ++w) {
          mk = fmaxf(mk, s_max[grp * wpr + w][0]);
          mv = fmaxf(mv, s_max[grp * wpr + w][1]);
        }
      }
      // ---- scales; where one grows, the rows that the block held are rounded again ----
      const size_t bh = blk * a.Hkv + (on ? h : 0);
      unsigned char* kb = static_cast<unsigned char*>(a.pool.k) + ((bh << a.pool.log_bs)) * D;
      unsigned char* vb = static_cast<unsigned char*>(a.pool.v) + ((bh << a.pool.log_bs)) * D;
      float ks = q8_scale(mk), vs = q8_scale(mv);
      const float ks_old = on && off > 0 ? fmaxf(a.pool.k_scale[bh], kQ8ScaleMin) : 0.f;
      const float vs_old = on && off > 0 ? fmaxf(a.pool.v_scale[bh], kQ8ScaleMin) : 0.f;
      ks = fmaxf(ks, ks_old);
      vs = fmaxf(vs, vs_old);
      auto again = [&](unsigned char* base, float f) {  // rows [0, off), shared out among the run's warps
        uint32_t* w = reinterpret_cast<uint32_t*>(base);
        for (int i = sub * 32 + lane; i < off * (D / 4); i += wpr * 32) {
          const uint32_t u = w[i];
          uint32_t x, y;
          e4m3x4_to_f16x4(u, x, y);
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&y));
          w[i] = f32x2_to_e4m3x2(lo.x * f, lo.y * f) | (f32x2_to_e4m3x2(hi.x * f, hi.y * f) << 16);
        }
      };
      if (on && off > 0 && ks > ks_old) again(kb, ks_old * q8_inverse(ks));
      if (on && off > 0 && vs > vs_old) again(vb, vs_old * q8_inverse(vs));
      // every lane and warp of the run has read the old scales
      if (wpr > 1) __syncthreads();
      else __syncwarp();
      if (on && sub == 0 && lane == 0) {
        a.pool.k_scale[bh] = ks;
        a.pool.v_scale[bh] = vs;
      }
      const float ki = q8_inverse(ks), vi = q8_inverse(vs);
      for (int p = 0; p < passes; ++p) {
        if (passes > 1) {
          __syncthreads();
          fill_angles(p * rows_per);
          __syncthreads();
          load(p * rows_per);
        }
#pragma unroll
        for (int r = 0; r < kAppRows; ++r) {
          const int rr = p * rows_per + sub * kAppRows + r;
          if (!on || rr >= n) continue;
          unsigned char* kd = kb + (size_t)(off + rr) * D + lane * PP;
          unsigned char* vd = vb + (size_t)(off + rr) * D + lane * PP;
          if (bad >> r & 1u) {
#pragma unroll
            for (int i = 0; i < PP; ++i) {
              kd[i] = kd[H + i] = 0x7f;
              vd[i] = vd[H + i] = 0;
            }
            continue;
          }
          if constexpr (PP == 2) {
            *reinterpret_cast<uint16_t*>(kd) = (uint16_t)f32x2_to_e4m3x2(row[r].k1[0] * ki, row[r].k1[1] * ki);
            *reinterpret_cast<uint16_t*>(kd + H) = (uint16_t)f32x2_to_e4m3x2(row[r].k2[0] * ki, row[r].k2[1] * ki);
            *reinterpret_cast<uint16_t*>(vd) = (uint16_t)f32x2_to_e4m3x2(row[r].v1[0] * vi, row[r].v1[1] * vi);
            *reinterpret_cast<uint16_t*>(vd + H) = (uint16_t)f32x2_to_e4m3x2(row[r].v2[0] * vi, row[r].v2[1] * vi);
          } else {
            const uint32_t kk = f32x2_to_e4m3x2(row[r].k1[0] * ki, row[r].k2[0] * ki);
            const uint32_t vv = f32x2_to_e4m3x2(row[r].v1[0] * vi, row[r].v2[0] * vi);
            kd[0] = (unsigned char)kk;
            kd[H] = (unsigned char)(kk >> 8);
            vd[0] = (unsigned char)vv;
            vd[H] = (unsigned char)(vv >> 8);
          }
        }
      }
    }
  }
}

}  // namespace

int launch_append_q8(const Shape& sh, const Q8Pool& pool, const void* k_pre, int64_t k_stride, const void* v_in,
                     int64_t v_stride, const int64_t* slot_map, const int* pos, const RopeAxes& rope,
                     int n_tokens, cudaStream_t st) {
  AppQ8Args a;
  a.pool = pool;
  a.rope = rope;
  a.Hkv = sh.Hkv;
  a.n_tokens = n_tokens;
  a.k_pre = k_pre; a.v_in = v_in; a.k_stride = k_stride; a.v_stride = v_stride;
  a.slot = slot_map; a.pos = pos;
  for (int i = 0; i < 64; ++i) a.inv_freq[i] = sh.inv_freq[i];
  // Steps of a few tokens a request: a warp a run and a CTA for each possible
  // leader.  Chunks: the warps that hold a whole block, and a CTA for each 16
  // tokens (no block is shorter).
  const bool step = (long long)n_tokens <= 8ll * sh.B;
  a.tile = step ? 1 : 16;
  a.wpr = step ? 1 : (1 << pool.log_bs) / kAppRows > kAppWarps ? kAppWarps : (1 << pool.log_bs) / kAppRows;
  const int hpc = kAppWarps / a.wpr;
  a.heads = hpc > 4 ? hpc : 4;
  const dim3 grid((n_tokens + a.tile - 1) / a.tile, (sh.Hkv + a.heads - 1) / a.heads);
  const size_t smem = (size_t)a.wpr * kAppRows * (sh.D / 2) * sizeof(double2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kAppWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*k)(AppQ8Args) = sh.dtype == RTP_BF16
                             ? (sh.D == 128 ? append_q8_kernel<__nv_bfloat16, 128> : append_q8_kernel<__nv_bfloat16, 64>)
                             : (sh.D == 128 ? append_q8_kernel<float, 128> : append_q8_kernel<float, 64>);
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
  trace_begin(RTP_STAGE_APPEND_Q8, st);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k, a);
  trace_end(RTP_STAGE_APPEND_Q8, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error(std::string("append q8 launch: ") + cudaGetErrorString(e));
    return RTP_ERR_CUDA;
  }
  return RTP_OK;
}

}  // namespace rtp
