// rtp_page_plan: block tables, slot map and positions of one serving step, from
// the requests' lengths and a stack of free blocks.
//
// Everything follows from three prefix sums over the requests (blocks that
// ended requests give back, blocks that the others need, tokens that they
// bring), so one launch does it all: a cluster of 1 to 16 CTAs, each of which
// forms the sums for itself (B lengths, a few KB from L2) and then writes its
// share of the tables and of the token arrays.  The one cluster barrier stands
// between "every CTA has read the lengths and the stack's height, and the
// returned blocks are on the stack" and "blocks are taken and results
// written"; it is what lets seq_len be ctx_len and n_free_out be n_free.
//
// Bound: latency for a decode step (B = 8: one CTA, a chain of two dependent
// loads, the sums and a store); for large chunks the 12 bytes per token that
// are written.
//
// Measured in a replayed graph: 8 decoding requests 4.5 us; 256 requests that decode, end and bring
// chunks 11 us (26 before a warp formed its sums by itself and a block was looked
// up once for four tokens).
#include "common.cuh"
#include "q8.h"

namespace rtp {
namespace {

constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanMaxCluster = 16;  // the largest cluster (more than 8 have to be asked for)

struct PlanArgs {
  int B, log_bs, cols, free_cap, max_tokens, max_ctx;
  const int* ctx_len;
  const int* new_len;
  int* table;
  int* free_list;
  const int* n_free;
  int* seq_len;
  int* cu_new;
  int64_t* slot_map;
  int* positions;
  int* n_free_out;
  int* status;
};

// What a CTA keeps of each request.
struct PlanReq {
  int ctx;   // cached positions
  int base;  // stack index: of the first block given back, or `before` (turned into the index of the first block taken)
  int add;   // new tokens; -1: ended
  int cu;    // first packed row (min(., max_tokens))
};

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// to[i] = from[dir i] for i = first, first + step, .. below n, eight loads on their way at once.
__device__ __forceinline__ void copy_ids(int* to, const int* from, int dir, int first, int n, int step) {
  for (int i0 = first; i0 < n; i0 += 8 * step) {
    int v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * step < n) v[k] = from[dir * (i0 + k * step)];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * step < n) to[i0 + k * step] = v[k];
  }
}

__global__ void __launch_bounds__(kPlanMaxThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ PlanReq s_req[];  // [B] and one past the end (cu only)
  __shared__ long long s_warp[3][32];
  __shared__ int s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
  const int rank = blockIdx.x, n_cta = gridDim.x;  // the grid is one cluster
  const int bs1 = (1 << a.log_bs) - 1;
  griddep_wait();
  int flags = 0;
  int height = *(volatile const int*)a.n_free;
  if (height < 0 || height > a.free_cap) {
    height = min(max(height, 0), a.free_cap);
    flags |= RTP_DEV_BLOCKS;
  }
  if (tid == 0) s_taken = 0;
  // ---- the sums: blocks given back, blocks needed, tokens brought ----
  long long run[3] = {0, 0, 0};
  for (int b0 = 0; b0 < a.B; b0 += nthr) {
    const int b = b0 + tid;
    int ctx = 0, add = 0;
    long long v[3] = {0, 0, 0};
    if (b < a.B) {
      ctx = a.ctx_len[b];
      add = a.new_len[b];
      if (ctx < 0 || ctx > a.max_ctx) {
        flags |= RTP_DEV_SEQ_LEN;
        ctx = 0;
        add = min(add, 0);
      }
      const long long have = (ctx + bs1) >> a.log_bs;
      if (add < 0) {
        add = -1;
        v[0] = have;
      } else {
        v[2] = add;
        if ((long long)ctx + add <= a.max_ctx) v[1] = ((ctx + add + bs1) >> a.log_bs) - have;
      }
    }
    long long x[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long y = __shfl_up_sync(0xffffffffu, x[k], o);
        if (lane >= o) x[k] += y;
      }
    }
    if (lane == 31)
      for (int k = 0; k < 3; ++k) s_warp[k][warp] = x[k];
    __syncthreads();
    long long tot[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {  // the warps' sums, a lane each
      long long y = lane < nwarp ? s_warp[k][lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      tot[k] = __shfl_sync(0xffffffffu, y, 31);
      const long long before = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
      x[k] += run[k] + (warp > 0 ? before : 0) - v[k];  // exclusive
    }
    if (b < a.B) {
      // sums past the stack or the token arrays only have to stay past them
      const long long base = add < 0 ? height + x[0] : x[1];
      s_req[b] = PlanReq{ctx, (int)min(base, (long long)INT32_MAX), add, (int)min(x[2], (long long)a.max_tokens)};
    }
    for (int k = 0; k < 3; ++k) run[k] += tot[k];
    __syncthreads();
  }
  const int n_tok = (int)min(run[2], (long long)a.max_tokens);
  if (run[2] > a.max_tokens) flags |= RTP_DEV_POSITION;
  if (height + run[0] > a.free_cap) flags |= RTP_DEV_BLOCKS;
  const int top = (int)min(height + run[0], (long long)a.free_cap);
  if (tid == 0) s_req[a.B].cu = n_tok;
  __syncthreads();
  // ---- ended requests' blocks onto the stack (`per` warps a request) ----
  const int all_warps = n_cta * nwarp, per = max(1, all_warps / a.B);
  const int my_req = (rank * nwarp + warp) / per, my_first = (rank * nwarp + warp) % per * 32 + lane;
  if (run[0] > 0 && my_req * per + per <= all_warps) {
    for (int b = my_req; b < a.B; b += all_warps / per) {
      const PlanReq r = s_req[b];
      if (r.add >= 0) continue;
      const int have = (int)min((long long)((r.ctx + bs1) >> a.log_bs), (long long)a.free_cap - r.base);
      const int* from = a.table + (size_t)b * a.cols;
      int* to = a.free_list + r.base;
      copy_ids(to, from, 1, my_first, have, per * 32);
    }
  }
  cluster_arrive_wait();
  // ---- who is served; `base` becomes the stack index of the first block taken ----
  for (int b = tid; b < a.B; b += nthr) {
    PlanReq r = s_req[b];
    int seq = 0;
    if (r.add >= 0) {
      const int have = (r.ctx + bs1) >> a.log_bs;
      bool ok = (long long)r.ctx + r.add <= a.max_ctx;
      if (!ok) flags |= RTP_DEV_POSITION;
      if (ok && r.add > 0 && (long long)r.cu + r.add > a.max_tokens) ok = false;  // flagged above
      const int need = ok ? ((r.ctx + r.add + bs1) >> a.log_bs) - have : 0;
      if (ok && need > 0 && (long long)r.base + need > top) {
        flags |= RTP_DEV_BLOCKS;
        ok = false;
      }
      if (ok && need > 0) atomicAdd(&s_taken, need);
      seq = ok ? r.ctx + r.add : r.ctx;
      s_req[b].base = ok ? top - 1 - r.base : -1;
      s_req[b].add = ok ? r.add : -2;  // -2: refused
    }
    if (rank == 0) {
      a.seq_len[b] = seq;
      a.cu_new[b] = r.cu;
    }
  }
  __syncthreads();
  if (rank == 0 && tid == 0) {
    a.cu_new[a.B] = n_tok;
    *a.n_free_out = top - s_taken;
  }
  // ---- table entries of the blocks taken ----
  if (my_req * per + per <= all_warps) {
    for (int b = my_req; b < a.B; b += all_warps / per) {
      const PlanReq r = s_req[b];
      if (r.add <= 0) continue;
      const int have = (r.ctx + bs1) >> a.log_bs;
      const int need = ((r.ctx + r.add + bs1) >> a.log_bs) - have;
      const int* from = a.free_list + r.base;
      int* to = a.table + (size_t)b * a.cols + have;
      copy_ids(to, from, -1, my_first, need, per * 32);
    }
  }
  // ---- slots and positions, four consecutive tokens a thread ----
  for (int t0 = (rank * nthr + tid) * 4; t0 < a.max_tokens; t0 += n_cta * nthr * 4) {
    int64_t slot[4];
    int pos[4];
    int b = 0, next = 0;
    if (t0 < n_tok) {  // the request whose rows hold t0: the last one with cu <= t0
      int hi = a.B;
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (s_req[mid].cu <= t0) b = mid;
        else hi = mid;
      }
      next = s_req[b + 1].cu;
    }
    PlanReq r = s_req[b];
    int have = (r.ctx + bs1) >> a.log_bs;
    int col = -1, blk = -1;  // the block of the last token looked up (four tokens are seldom in more than one)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + e;
      slot[e] = -1;
      pos[e] = 0;
      if (t >= n_tok) continue;
      if (t >= next) {
        while (t >= next) next = s_req[++b + 1].cu;  // t < n_tok = cu of the end
        r = s_req[b];
        have = (r.ctx + bs1) >> a.log_bs;
        col = -1;
      }
      const int p = r.ctx + t - r.cu;
      pos[e] = p;
      if (r.add < 0) continue;
      const int c = p >> a.log_bs;
      if (c != col) {
        col = c;
        blk = c < have ? a.table[(size_t)b * a.cols + c] : a.free_list[r.base - (c - have)];
        if (blk < 0) flags |= RTP_DEV_BLOCKS;
      }
      if (blk >= 0) slot[e] = ((int64_t)blk << a.log_bs) + (p & bs1);
    }
    if (t0 + 4 <= a.max_tokens) {
      reinterpret_cast<longlong2*>(a.slot_map + t0)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2*>(a.slot_map + t0)[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int e = 0; e < 4; ++e)
        if (t0 + e < a.max_tokens) {
          a.slot_map[t0 + e] = slot[e];
          a.positions[t0 + e] = pos[e];
        }
    }
  }
  if (flags) atomicOr(a.status, flags);
}

}  // namespace

int launch_page_plan(const Shape& sh, int log_bs, int table_cols, const int* ctx_len, const int* new_len,
                     int* block_table, int* free_list, int free_cap, const int* n_free, int* seq_len,
                     int* cu_new, int64_t* slot_map, int* positions, int max_tokens, int* n_free_out,
                     int* status, cudaStream_t st) {
  PlanArgs a;
  a.B = sh.B; a.log_bs = log_bs; a.cols = table_cols; a.free_cap = free_cap; a.max_tokens = max_tokens;
  a.max_ctx = sh.Lmax;
  a.ctx_len = ctx_len; a.new_len = new_len; a.table = block_table; a.free_list = free_list; a.n_free = n_free;
  a.seq_len = seq_len; a.cu_new = cu_new; a.slot_map = slot_map; a.positions = positions;
  a.n_free_out = n_free_out; a.status = status;
  // one CTA for a decode step; more once there are tokens for them to write
  const int threads = sh.B <= 256 && max_tokens <= 1024 ? 256 : kPlanMaxThreads;
  int n_cta = 1;
  while (n_cta < kPlanMaxCluster && (long long)n_cta * threads * 4 < max_tokens) n_cta *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_cta);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)(sh.B + 1) * sizeof(PlanReq);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_cta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaSuccess;
  if (n_cta > 8) e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && cfg.dynamicSmemBytes > 40 * 1024)  // past what a kernel may take unasked
    e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((kMaxPlanBatch + 1) * sizeof(PlanReq)));
  trace_begin(RTP_STAGE_PAGE_PLAN, st);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, page_plan_kernel, a);
  trace_end(RTP_STAGE_PAGE_PLAN, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error(std::string("page plan launch: ") + cudaGetErrorString(e));
    return RTP_ERR_CUDA;
  }
  return RTP_OK;
}

}  // namespace rtp
