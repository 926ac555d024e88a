// rtp_append_q8: rotary positions (one or several axes), then keys and values
// as e4m3 into their blocks, with a power-of-two scale for each (block, head).
//
// A run is a maximal stretch of packed tokens that go to consecutive slots of
// one block; its first token leads.  The scale needs the run's largest
// magnitude, so a group of warps holds a whole run of one head in registers, as
// loaded (8 rows a warp), rotates it once for the maximum and once more to store:
// every input is read once.  Where a block already held rows and its scale grows,
// the group also rounds those rows again.
//
// The stored value is the exact rotation rounded once.  The rotation is formed
// in fp32, off by at most e = 1.125 2^-22 (|x1| + |x2|) (cos and sin by 2^-23,
// the products and their sum by 2^-24 each; the eighth is for forming y - e and
// y + e); where those two round to the same e4m3 value, that is the answer, and
// where they do not (one value in 10^4) the pair is formed again in 64 bits.
// The same holds for the scale: the maximum less and plus the largest e nearly
// always name one power of two.
//
// Measured in a replayed graph, 8K tokens of 8 heads, D = 128, bf16, three axes: 26 us
// (50 MB, 1.9 TB/s); 64 bits throughout, with a table of cosines in shared memory, took 36;
// the fp32 way with the cosines of a run shared through shared memory 29 to 40;
// without any cosines, 19 to 21: what is left is the chain slots, rows, maximum,
// store of each CTA with 16 warps an SM.
// Bound: memory, the inputs read once and half (bf16) of their bytes written.
#include <cfloat>
#include <type_traits>

#include "q8.cuh"

namespace rtp {
namespace {

constexpr int kAppMaxWarps = 16;
constexpr int kAppRows = 8;  // rows a warp of a chunk holds

struct AppQ8Args {
  Q8Pool pool;
  int Hkv, n_tokens, tile, wpr;  // tile: tokens whose leaders a CTA serves; wpr: warps a run
  const void* k_pre;
  const void* v_in;
  long long k_stride, v_stride;
  const int64_t* slot;
  const int* pos;
  uint64_t turns[64];
  RopeAxes rope;
};

// The rotation of one pair in 64 bits, each result rounded to odd (truncated,
// the lowest bit set if anything was cut off): scaling it by a power of two is
// exact, and rounding it to nearest gives what rounding the 64-bit value would.
// The angle is split as in rope_turns; Taylor sums to r^17 and r^16.
__device__ __noinline__ float2 exact_pair(float x1, float x2, int pos, uint64_t turns) {
  const uint64_t f = (uint64_t)(long long)pos * turns;
  const uint32_t q = (uint32_t)((f + (1ull << 61)) >> 62);                              // quarter turns
  const double r = (double)(long long)(f - ((uint64_t)q << 62)) * 3.4061215800307446e-19;  // the rest, 2 pi / 2^64
  const double x = r * r;
  double s = fma(x, 2.8114572543455206e-15, -7.6471637318198164e-13);
  s = fma(s, x, 1.6059043836821613e-10);
  s = fma(s, x, -2.5052108385441720e-08);
  s = fma(s, x, 2.7557319223985893e-06);
  s = fma(s, x, -1.9841269841269841e-04);
  s = fma(s, x, 8.3333333333333332e-03);
  s = fma(s, x, -1.6666666666666666e-01);
  s = fma(s * x, r, r);
  double c = fma(x, 4.7794773323873853e-14, -1.1470745597729725e-11);
  c = fma(c, x, 2.0876756987868100e-09);
  c = fma(c, x, -2.7557319223985888e-07);
  c = fma(c, x, 2.4801587301587302e-05);
  c = fma(c, x, -1.3888888888888889e-03);
  c = fma(c, x, 4.1666666666666664e-02);
  c = fma(c, x, -0.5);
  c = fma(c, x, 1.0);
  double u = q & 1u ? s : c, v = q & 1u ? c : s;
  if ((q + 1u) & 2u) u = -u;
  if (q & 2u) v = -v;
  const double y[2] = {(double)x1 * u - (double)x2 * v, (double)x2 * u + (double)x1 * v};
  float z[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    z[i] = __double2float_rz(y[i]);
    if ((double)z[i] != y[i]) z[i] = __uint_as_float(__float_as_uint(z[i]) | 1u);
  }
  return make_float2(z[0], z[1]);
}

// Four elements as they lie in memory.
template <typename T>
struct Four {
  typename std::conditional<sizeof(T) == 2, uint2, uint4>::type u;
  __device__ __forceinline__ void load(const T* p) { u = __ldg(reinterpret_cast<const decltype(u)*>(p)); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    if constexpr (sizeof(T) == 2) {
      const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
      const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    } else {
      x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
  }
};

// e4m3 of four values times f.
__device__ __forceinline__ uint32_t quant4(const float (&y)[4], float f) {
  return f32x2_to_e4m3x2(y[0] * f, y[1] * f) | (f32x2_to_e4m3x2(y[2] * f, y[3] * f) << 16);
}
__device__ __forceinline__ uint32_t quant4_off(const float (&y)[4], float f, float off) {
  return f32x2_to_e4m3x2(fmaf(y[0], f, off), fmaf(y[1], f, off)) | (f32x2_to_e4m3x2(fmaf(y[2], f, off), fmaf(y[3], f, off)) << 16);
}

// A lane's part of a row as loaded: 4 rotary pairs (k, k + D/2) of the key, and
// the value dims of the same numbers.
template <typename T>
struct AppPart {
  Four<T> k1, k2, v1, v2;
};

// The largest number >= 0 of the warp.
__device__ __forceinline__ float warp_max_positive(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// A warp holds ST steps of RPS rows: kAppRows for chunks; one step where a
// request brings a few tokens, since steps without rows are worked on all the
// same (a decode step of 8 requests: 3.1 us for 5.0).
constexpr int rows_a_step(int D) { return 32 / (D / 8); }

template <typename T, int D, int ST>
__global__ void __launch_bounds__(kAppMaxWarps * 32) append_q8_kernel(const __grid_constant__ AppQ8Args a) {
  constexpr int H = D / 2;
  constexpr int LPR = D / 8;            // lanes a row
  constexpr int RPS = rows_a_step(D);
  constexpr int kRows = ST * RPS;
  __shared__ float s_max[2][kAppMaxWarps][3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int wpr = a.wpr, hpc = nw / wpr, sub = warp % wpr, grp = warp / wpr;
  const int bs = 1 << a.pool.log_bs;
  const long long n_slots = (long long)a.pool.n_blocks << a.pool.log_bs;
  const int rows_per = wpr * kRows;  // rows of a run that a pass holds
  const int rl = lane / LPR, k0 = (lane % LPR) * 4;  // the lane's row of a step and its first pair
  const int h = blockIdx.y * hpc + grp;
  const bool on = h < a.Hkv;
  const bool axes = a.rope.n_axes > 1;
  // lanes that index the parameters apart are served one by one: once a CTA
  __shared__ uint64_t s_turns[H];
  __shared__ int s_axis[H];
  for (int k = tid; k < H; k += blockDim.x) {
    s_turns[k] = a.turns[k];
    s_axis[k] = axes ? a.rope.axis[k] : 0;
  }
  __syncthreads();
  uint64_t turns[4];  // of the lane's pairs
  int axis[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    turns[e] = s_turns[k0 + e];
    axis[e] = s_axis[k0 + e];
  }
  griddep_wait();
  griddep_launch();
  int turn = 0;  // which half of s_max
  const int t_end = min((int)(blockIdx.x + 1) * a.tile, a.n_tokens);
  for (int t0 = blockIdx.x * a.tile; t0 < t_end; t0 += 32) {
    // ---- the leaders among 32 tokens (every warp finds the same) ----
    bool lead = false;
    {
      const int t = t0 + lane;
      if (t < t_end) {
        const long long s = a.slot[t], before = t > 0 ? a.slot[t - 1] : -1;
        if (s >= n_slots) atomicOr(a.pool.status, RTP_DEV_BLOCKS);
        else if (s >= 0) lead = t == 0 || (s & (bs - 1)) == 0 || before != s - 1;
      }
    }
    for (unsigned leaders = __ballot_sync(0xffffffffu, lead); leaders; leaders &= leaders - 1) {
      const int tl = t0 + __ffs(leaders) - 1;
      const long long s0 = a.slot[tl];
      const int off = (int)(s0 & (bs - 1));
      const size_t blk = (size_t)(s0 >> a.pool.log_bs);
      const int most = min(bs - off, a.n_tokens - tl);
      int n = 0;  // the run's tokens: at most 128, looked at together
      {
        unsigned in[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = 32 * q + lane;
          in[q] = i < most && a.slot[tl + i] == s0 + i ? 1u : 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const unsigned m = __ballot_sync(0xffffffffu, in[q] != 0u);
          if (n == 32 * q) n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        }
      }
      const int passes = (n + rows_per - 1) / rows_per;
      AppPart<T> part[ST] = {};
      float cs[ST][4], sn[ST][4];
      auto row_of = [&](int p, int st) { return p * rows_per + sub * kRows + st * RPS + rl; };
      auto key_at = [&](int r) {
        return static_cast<const T*>(a.k_pre) + (size_t)(tl + r) * a.k_stride + (size_t)h * D + k0;
      };
      auto pos_at = [&](int r, int k) {
        return a.pos[(size_t)(tl + r) + (size_t)s_axis[k] * a.n_tokens];
      };
      auto load = [&](int p) {  // a pass's rows, and the cosines of their positions
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          const int r = row_of(p, st);
          if (!on || r >= n) continue;
          const T* kp = key_at(r);
          const T* vp = static_cast<const T*>(a.v_in) + (size_t)(tl + r) * a.v_stride + (size_t)h * D + k0;
          part[st].k1.load(kp);
          part[st].k2.load(kp + H);
          part[st].v1.load(vp);
          part[st].v2.load(vp + H);
        }
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          const int r = min(row_of(p, st), n - 1);
          int pos[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pos[e] = e > 0 && !axes ? pos[0] : a.pos[(size_t)axis[e] * a.n_tokens + (tl + r)];
#pragma unroll
          for (int e = 0; e < 4; ++e) rope_turns(pos[e], turns[e], cs[st][e], sn[st][e]);
        }
      };
      // the lane's pairs of a row, rotated
      auto rotate = [&](int st, float (&y1)[4], float (&y2)[4], float (&x1)[4], float (&x2)[4]) {
        part[st].k1.get(x1);
        part[st].k2.get(x2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y1[e] = x1[e] * cs[st][e] - x2[e] * sn[st][e];
          y2[e] = x2[e] * cs[st][e] + x1[e] * sn[st][e];
        }
      };
      float off_e[ST];  // of each step: the bound on the rotation's error
      float mk = 0.f, mv = 0.f, me = 0.f;
      unsigned bad = 0;  // steps whose row, here, holds a value that is not finite (of the last pass loaded)
      auto scan = [&](int p) {
        bad = 0;
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          // (rows that are not there are worked on all the same, without a branch, and left out below)
          const bool lv = on && row_of(p, st) < n;
          float xk = 0.f, xv = 0.f, xe = 0.f, y1[4], y2[4], x1[4], x2[4], v1[4], v2[4];
          rotate(st, y1, y2, x1, x2);
          part[st].v1.get(v1);
          part[st].v2.get(v2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xk = max3_nan(xk, fabsf(y1[e]), fabsf(y2[e]));
            xv = max3_nan(xv, fabsf(v1[e]), fabsf(v2[e]));
            xe = fmaxf(xe, fabsf(x1[e]) + fabsf(x2[e]));
          }
          xe *= 2.682209e-07f;  // 1.125 2^-22
          off_e[st] = xe;
          const unsigned m = __ballot_sync(0xffffffffu, lv && !(xk <= FLT_MAX && xv <= FLT_MAX));  // an infinity or a NaN
          const bool bd = (m >> (rl * LPR) & (LPR == 16 ? 0xffffu : 0xffu)) != 0u;
          bad |= bd ? 1u << st : 0u;
          mk = lv && !bd ? fmaxf(mk, xk) : mk;
          mv = lv && !bd ? fmaxf(mv, xv) : mv;
          me = lv && !bd ? fmaxf(me, xe) : me;
        }
      };
      for (int p = 0; p < passes; ++p) {
        load(p);
        scan(p);
      }
      // ---- the run's maxima; lane w of every warp works out those of warp w's run ----
      mk = warp_max_positive(mk);
      mv = warp_max_positive(mv);
      me = warp_max_positive(me);
      if (lane == 0) {
        s_max[turn][warp][0] = mk;
        s_max[turn][warp][1] = mv;
        s_max[turn][warp][2] = me;
      }
      __syncthreads();
      mk = mv = me = 0.f;
      if (lane < nw) {
        mk = s_max[turn][lane][0];
        mv = s_max[turn][lane][1];
        me = s_max[turn][lane][2];
      }
      turn ^= 1;
      for (int o = 1; o < wpr; o <<= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        me = fmaxf(me, __shfl_xor_sync(0xffffffffu, me, o));
      }
      float ks = q8_scale(fminf(mk + me, FLT_MAX));
      const bool close = q8_scale(fmaxf(mk - me, 0.f)) != ks;
      // some head's maximum lies next to 448 times a power of two (the CTA agrees): those in 64 bits
      if (__any_sync(0xffffffffu, close)) {
        const bool mine = __shfl_sync(0xffffffffu, close, grp * wpr);
        float m = 0.f;
        for (int p = 0; p < passes; ++p) {
          if (passes > 1) {
            load(p);
            float k_ = mk, v_ = mv, e_ = me;
            scan(p);
            mk = k_; mv = v_; me = e_;
          }
#pragma unroll 1
          for (int st = 0; st < ST; ++st) {
            const int r = row_of(p, st);
            if (!mine || !on || r >= n || (bad >> st & 1u)) continue;
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              const float2 y = exact_pair(to_f32(key_at(r)[e]), to_f32(key_at(r)[e + H]), pos_at(r, k0 + e), s_turns[k0 + e]);
              m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
          }
        }
        __syncwarp();
        m = warp_max_positive(m);
        if (lane == 0) s_max[turn][warp][0] = m;
        __syncthreads();
        m = lane < nw ? s_max[turn][lane][0] : 0.f;
        turn ^= 1;
        for (int o = 1; o < wpr; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (close) ks = q8_scale(m);
      }
      ks = __shfl_sync(0xffffffffu, ks, grp * wpr);
      float vs = __shfl_sync(0xffffffffu, q8_scale(mv), grp * wpr);
      // ---- scales; where one grows, the rows that the block held are rounded again ----
      const size_t bh = blk * a.Hkv + (on ? h : 0);
      unsigned char* kb = static_cast<unsigned char*>(a.pool.k) + (bh << a.pool.log_bs) * D;
      unsigned char* vb = static_cast<unsigned char*>(a.pool.v) + (bh << a.pool.log_bs) * D;
      if (off > 0) {  // (the CTA agrees)
        const float ks_old = on ? fmaxf(a.pool.k_scale[bh], kQ8ScaleMin) : 0.f;
        const float vs_old = on ? fmaxf(a.pool.v_scale[bh], kQ8ScaleMin) : 0.f;
        ks = fmaxf(ks, ks_old);
        vs = fmaxf(vs, vs_old);
        auto again = [&](unsigned char* base, float f) {  // rows [0, off), shared out among the run's warps
          uint32_t* w = reinterpret_cast<uint32_t*>(base);
          for (int i = sub * 32 + lane; i < off * (D / 4); i += wpr * 32) {
            uint32_t x, y;
            e4m3x4_to_f16x4(w[i], x, y);
            const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&x));
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&y));
            const float v[4] = {lo.x, lo.y, hi.x, hi.y};
            w[i] = quant4(v, f);
          }
        };
        if (on && ks > ks_old) again(kb, ks_old * q8_inverse(ks));
        if (on && vs > vs_old) again(vb, vs_old * q8_inverse(vs));
        __syncthreads();  // every lane and warp of the run has read the old scales
      }
      if (on && sub == 0 && lane == 0) {
        a.pool.k_scale[bh] = ks;
        a.pool.v_scale[bh] = vs;
      }
      const float ki = q8_inverse(ks), vi = q8_inverse(vs);
      for (int p = 0; p < passes; ++p) {
        if (passes > 1) {
          load(p);
          scan(p);  // (for the rows that are bad)
        }
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          const int r = row_of(p, st);
          const bool lv = on && r < n, bd = bad >> st & 1u;
          float y1[4], y2[4], x1[4], x2[4], v[4];
          rotate(st, y1, y2, x1, x2);
          const float e = off_e[st] * ki;
          uint32_t q1 = quant4_off(y1, ki, e), q2 = quant4_off(y2, ki, e);
          uint32_t off_by = (q1 ^ quant4_off(y1, ki, -e)) | (q2 ^ quant4_off(y2, ki, -e));
          part[st].v1.get(v);
          uint32_t w1 = quant4(v, vi);
          part[st].v2.get(v);
          uint32_t w2 = quant4(v, vi);
          off_by = lv && !bd ? off_by : 0u;
          while (off_by) {  // pair i lies too near a border
            const int i = (__ffs(off_by) - 1) >> 3;
            const float2 x = exact_pair(to_f32(key_at(r)[i]), to_f32(key_at(r)[i + H]), pos_at(r, k0 + i), s_turns[k0 + i]);
            const uint32_t z = f32x2_to_e4m3x2(x.x * ki, x.y * ki);
            q1 = (q1 & ~(0xffu << (8 * i))) | (z & 0xffu) << (8 * i);
            q2 = (q2 & ~(0xffu << (8 * i))) | (z >> 8) << (8 * i);
            off_by &= ~(0xffu << (8 * i));
          }
          if (bd) {
            q1 = q2 = 0x7f7f7f7fu;
            w1 = w2 = 0u;
          }
          if (lv) {
            uint32_t* kd = reinterpret_cast<uint32_t*>(kb + (size_t)(off + r) * D + k0);
            uint32_t* vd = reinterpret_cast<uint32_t*>(vb + (size_t)(off + r) * D + k0);
            kd[0] = q1;
            kd[H / 4] = q2;
            vd[0] = w1;
            vd[H / 4] = w2;
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
  for (int i = 0; i < 64; ++i) a.turns[i] = sh.turns[i];
  // Steps of a few tokens a request: the warps that hold its tokens, and a CTA
  // for each possible leader.  Chunks: the warps that hold a whole block, and a
  // CTA for each block's worth of tokens.
  const bool step = (long long)n_tokens <= 8ll * sh.B;
  const int bs = 1 << pool.log_bs;
  a.tile = step ? 1 : bs;
  a.wpr = bs / kAppRows;
  if (step && n_tokens == sh.B) {
    a.wpr = 1;  // a token each
  } else if (step) {
    // any one request may bring a whole block: two warps a run at least, more while the CTAs are few
    // (200 tokens of one of 256 requests: 31 us with 8 rows a warp, 39 with one warp of 2, 20 with two;
    // 256 requests of a token each 4.2 with one warp, 6.8 with two, 12.5 with four)
    for (a.wpr = 2; a.wpr < 8 && ((long long)a.wpr * rows_a_step(sh.D) * sh.B < n_tokens ||
                                  2ll * a.wpr * n_tokens * sh.Hkv <= 8 * 512);)
      a.wpr *= 2;
  }
  // eight warps at least, but none for heads that the layer has not got (they
  // do the work all the same: 10.1 for 9.3 us on a 2-head layer)
  const int hpc = a.wpr >= 8 ? 1 : 8 / a.wpr < sh.Hkv ? 8 / a.wpr : sh.Hkv, warps = hpc * a.wpr;
  const dim3 grid((n_tokens + a.tile - 1) / a.tile, (sh.Hkv + hpc - 1) / hpc);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(warps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*k)(AppQ8Args);
  auto pick = [&](auto few, auto many) { k = step ? few : many; };
  if (sh.dtype == RTP_BF16) {
    if (sh.D == 128) pick(append_q8_kernel<__nv_bfloat16, 128, 1>, append_q8_kernel<__nv_bfloat16, 128, kAppRows / rows_a_step(128)>);
    else pick(append_q8_kernel<__nv_bfloat16, 64, 1>, append_q8_kernel<__nv_bfloat16, 64, kAppRows / rows_a_step(64)>);
  } else {
    if (sh.D == 128) pick(append_q8_kernel<float, 128, 1>, append_q8_kernel<float, 128, kAppRows / rows_a_step(128)>);
    else pick(append_q8_kernel<float, 64, 1>, append_q8_kernel<float, 64, kAppRows / rows_a_step(64)>);
  }
  trace_begin(RTP_STAGE_APPEND_Q8, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, a);
  trace_end(RTP_STAGE_APPEND_Q8, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error(std::string("append q8 launch: ") + cudaGetErrorString(e));
    return RTP_ERR_CUDA;
  }
  return RTP_OK;
}

}  // namespace rtp
