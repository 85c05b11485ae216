// Packed sequences of different lengths: prefill forward and backward over S sequences laid end to end
// (attn_fwd_varlen, attn_bwd_varlen).
//
// The lengths are in device memory, so the host can size the launch only by bounds. A plan kernel of one
// block checks the offsets and lists the blocks of work of every sequence, heaviest first (a counting sort by
// the number of tiles a block walks), with where each block lies; the prefill kernel's CTAs claim blocks of
// that list. Launched programmatically, the main kernel sets up while the plan runs.
#include <cuda_bf16.h>
#include <math.h>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn {

// ---- plan ------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;      // of the counting sort
constexpr int kPlanOwnBlocks = 8;    // blocks of a sequence that one thread lists by itself
constexpr int kFwdBlockRows = 256;   // query rows of a forward block (two tiles of 128, in one CTA or a pair)
constexpr int kTileRows = 128;

struct PlanSeq {
  int q0, nq, k0, nkv;
};

// Forward: blocks of query rows, and the tiles of 128 keys that block `blk` walks (0: none of its rows sees a key).
struct PlanFwd {
  static __device__ __forceinline__ int blocks(const PlanSeq& s) { return (s.nq + kFwdBlockRows - 1) / kFwdBlockRows; }
  static __device__ __forceinline__ int longest(const PlanSeq& s) { return (s.nkv + kTileRows - 1) / kTileRows; }
  static __device__ __forceinline__ int tiles(const PlanSeq& s, int blk, int causal) {
    const int left = s.nq - blk * kFwdBlockRows;
    const int end = causal ? min(s.nkv, min(kFwdBlockRows, left) + s.nkv - left) : s.nkv;
    return end > 0 ? (end + kTileRows - 1) / kTileRows : 0;
  }
  static __device__ __forceinline__ VarUnit unit(const PlanSeq& s, int seq, int blk) {
    return VarUnit{s.q0 + blk * kFwdBlockRows, s.nq - blk * kFwdBlockRows, s.k0, s.nkv, seq, {0, 0, 0}};
  }
};
// Backward: blocks of 128 keys, and the tiles of 128 query rows that block `blk` walks.
struct PlanBwd {
  static __device__ __forceinline__ int blocks(const PlanSeq& s) { return (s.nkv + kTileRows - 1) / kTileRows; }
  static __device__ __forceinline__ int longest(const PlanSeq& s) { return (s.nq + kTileRows - 1) / kTileRows; }
  static __device__ __forceinline__ int tiles(const PlanSeq& s, int blk, int causal) {
    return max(0, longest(s) - first_q_tile(causal, s.nq, s.nkv - blk * kTileRows));
  }
  static __device__ __forceinline__ VarUnit unit(const PlanSeq& s, int seq, int blk) {
    return VarUnit{s.q0, s.nq, s.k0 + blk * kTileRows, s.nkv - blk * kTileRows, seq, {0, 0, 0}};
  }
};

// The plan, by one block of kPlanThreads threads. Returns the tiles of all blocks (to thread 0) and the most that
// one block walks at most.
struct PlanSum {
  unsigned long long tiles;
  int longest;
};
template <class P>
__device__ __forceinline__ PlanSum make_plan(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int S,
                                             int Tq, int Tk, int causal, const VarPlan& plan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ---- check the offsets, and the largest number of tiles
  __shared__ int bins[kPlanBins], warp_sum[kPlanThreads / 32], most;
  __shared__ unsigned long long sum;
  if (threadIdx.x == 0) {
    most = 0;
    sum = 0;
  }
  bins[threadIdx.x] = 0;
  bool bad = false;
  int mx = 0;
  for (int s = threadIdx.x; s < S; s += kPlanThreads) {
    const int a = cu_q[s], b = cu_q[s + 1], c = cu_k[s], e = cu_k[s + 1];
    bad |= a < 0 || b < a || b > Tq || c < 0 || e < c || e > Tk;
    mx = max(mx, P::longest(PlanSeq{a, b - a, c, e - c}));
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) {
      *plan.count = -1;
      *plan.claim = 0;
      atomicOr(&g_error_word, kErrBadLengthBit);
    }
    return PlanSum{0, 0};
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) atomicMax(&most, mx);
  __syncthreads();
  const int max_tiles = most;
  auto bin_of = [&](int tiles) -> int {  // 0: heaviest
    return max_tiles < kPlanBins ? max_tiles - tiles : int((long long)(max_tiles - tiles) * (kPlanBins - 1) / max_tiles);
  };
  // f(number of the sequence, sequence, block) for every block: a thread takes a sequence, a warp one with many blocks
  auto each_block = [&](auto f) {
    for (int s0 = warp * 32; s0 < S; s0 += kPlanThreads) {
      const int s = s0 + lane;
      PlanSeq q = {0, 0, 0, 0};
      if (s < S) {
        q.q0 = cu_q[s];
        q.nq = cu_q[s + 1] - q.q0;
        q.k0 = cu_k[s];
        q.nkv = cu_k[s + 1] - q.k0;
      }
      const int nb = P::blocks(q);
      if (nb <= kPlanOwnBlocks)
        for (int i = 0; i < nb; ++i) f(s, q, i);
      for (unsigned many = __ballot_sync(0xffffffffu, nb > kPlanOwnBlocks); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const PlanSeq w = {__shfl_sync(0xffffffffu, q.q0, src), __shfl_sync(0xffffffffu, q.nq, src),
                           __shfl_sync(0xffffffffu, q.k0, src), __shfl_sync(0xffffffffu, q.nkv, src)};
        const int wnb = __shfl_sync(0xffffffffu, nb, src);
        for (int i = lane; i < wnb; i += 32) f(s0 + src, w, i);
      }
    }
  };
  unsigned long long tiles = 0;
  each_block([&](int, const PlanSeq& q, int i) {
    const int t = P::tiles(q, i, causal);
    tiles += t;
    atomicAdd(&bins[bin_of(t)], 1);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  if (lane == 0 && tiles) atomicAdd(&sum, tiles);
  __syncthreads();
  // exclusive scan of the bins
  const int mine = bins[threadIdx.x];
  int scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int before = scan - mine;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  bins[threadIdx.x] = before;
  if (threadIdx.x == kPlanThreads - 1) {
    *plan.count = int(min((long long)(before + mine), plan.max_blocks));
    *plan.claim = 0;
  }
  __syncthreads();
  each_block([&](int seq, const PlanSeq& q, int i) {
    const int at = atomicAdd(&bins[bin_of(P::tiles(q, i, causal))], 1);
    if (at < plan.max_blocks) plan.units[at] = P::unit(q, seq, i);
  });
  return PlanSum{sum, max_tiles};
}
static_assert(kPlanBins == kPlanThreads, "one bin per thread");

__global__ void __launch_bounds__(kPlanThreads)
    varlen_plan_kernel(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int S, int Tq, int Tk,
                       int causal, int Hq, int Hkv, int groups, int ctas, VarPlan plan) {
  pdl_launch();
  const PlanSum sum = make_plan<PlanFwd>(cu_q, cu_k, S, Tq, Tk, causal, plan);
  // `groups` groups of heads, one after the other, would keep each group's K/V in L2; but every group ends with its
  // own longest blocks still running, so no more of them than leave each CTA half as much again as the longest
  // block in every group. Measured: sixteen causal sequences of 4096 with 16 heads 1000 us in 6 groups, 1140 us in
  // one; 8192 + 5003 + 3001 (this rule: one group) 376 us, 395 us in 4.
  if (threadIdx.x == 0) {
    const unsigned long long room = 2 * sum.tiles * Hq / (3ull * ctas * max(1, sum.longest));
    const int n = max(1, int(min((unsigned long long)min(groups, Hkv), room)));
    plan.count[1] = Hq / Hkv * ((Hkv + n - 1) / n);
  }
}

// Workspace of a plan: count and claim counter, blocks.
long long fwd_max_blocks(int S, int Tq) { return (long long)Tq / kFwdBlockRows + S; }
long long bwd_max_blocks(int S, int Tk) { return (long long)Tk / kTileRows + S; }
size_t plan_bytes(long long max_blocks) { return 256 + (size_t(max_blocks) * sizeof(VarUnit) + 255) / 256 * 256; }

VarPlan plan_at(void* workspace, long long max_blocks) {
  char* w = static_cast<char*>(workspace);
  VarPlan p;
  p.count = reinterpret_cast<int*>(w);
  p.claim = reinterpret_cast<unsigned int*>(w + 128);
  p.units = reinterpret_cast<VarUnit*>(w + 256);
  p.max_blocks = max_blocks;
  return p;
}

// The sequence that owns packed row t (-1: none): the last s with cu[s] <= t, if t < cu[s + 1].
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int S, int t) {
  if (t < cu[0] || t >= cu[S]) return -1;
  int lo = 0, hi = S;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ---- backward: pre- and post-pass ------------------------------------------------------------------------
// The workspace after the plan: the fp32 dQ accumulator [acc_rows, Hq, 128] and per head the LSE' and D rows
// [Hq, lse_rows], in which every sequence starts at a box or tile of its own (padded_row), and the accumulator
// row of each packed row (-1: of no sequence).
struct BwdSpace {
  float* acc;
  float* lse2;
  float* dd;
  int32_t* row_of;
  long long acc_rows, lse_rows;
};

// Block 0 makes the plan. The others take a packed query row per warp, 16 lanes per head: D = sum_e dO_e O_e and
// LSE' = LSE log2 e (+inf for a row without keys, so that its P is 0), and the row of the accumulator zeroed, with
// the padding rows of its last box after a sequence's last row. Every place a row of a sequence writes to lies
// inside the arrays whatever the other offsets are; offsets out of order leave results unused (the plan says so).
__global__ void __launch_bounds__(kPlanThreads)
    varlen_bwd_pre_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
                          const float* __restrict__ lse, const int32_t* __restrict__ cu_q,
                          const int32_t* __restrict__ cu_k, int S, int Tq, int Tk, int Hq, int causal, VarPlan plan,
                          BwdSpace w) {
  pdl_launch();
  if (blockIdx.x == 0) {
    make_plan<PlanBwd>(cu_q, cu_k, S, Tq, Tk, causal, plan);
    return;
  }
  const int lane = threadIdx.x & 31, seg = lane & 15;
  const int n_warps = int(gridDim.x - 1) * (kPlanThreads / 32);
  for (long long t = (blockIdx.x - 1ll) * (kPlanThreads / 32) + (threadIdx.x >> 5); t < Tq; t += n_warps) {
    int s = seq_of_row(cu_q, S, int(t));
    const int first = s < 0 ? -1 : cu_q[s];
    if (first < 0) s = -1;
    const int i = int(t) - first;
    const size_t acc_row = s < 0 ? 0 : padded_row(first, s, kAccRows) + i;
    if (lane == 0) w.row_of[t] = s < 0 ? -1 : int(acc_row);
    if (s < 0) continue;
    const size_t lse_row = padded_row(first, s, kTileRows) + i;
    const int zero_rows = i + 1 == cu_q[s + 1] - first ? (i / kAccRows + 1) * kAccRows - i : 1;
    for (int h0 = 0; h0 < Hq; h0 += 2) {
      const int h = h0 + (lane >> 4);
      const bool real = h < Hq;
      float dsum = 0.f;
      if (real) {
        const size_t row = (size_t(t) * Hq + h) * bwd::D;
        const uint4 a = reinterpret_cast<const uint4*>(o + row)[seg];
        const uint4 c = reinterpret_cast<const uint4*>(dout + row)[seg];
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dsum = fmaf(__uint_as_float(wa[k] << 16), __uint_as_float(wc[k] << 16), dsum);
          dsum = fmaf(__uint_as_float(wa[k] & 0xFFFF0000u), __uint_as_float(wc[k] & 0xFFFF0000u), dsum);
        }
        for (int r = 0; r < zero_rows; ++r) {
          float4* z = reinterpret_cast<float4*>(w.acc + ((acc_row + r) * Hq + h) * bwd::D) + 2 * seg;
          z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
          z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, off);
      if (real && seg == 0) {
        const float L = lse[size_t(h) * Tq + t];
        w.lse2[h * w.lse_rows + lse_row] = (L == -INFINITY) ? INFINITY : L * 1.4426950408889634f;
        w.dd[h * w.lse_rows + lse_row] = dsum;
      }
    }
  }
}

// dQ = scale * accumulator, bf16, for the rows that a sequence owns: a warp per packed row, all heads.
constexpr int kPostThreads = 256;
__global__ void __launch_bounds__(kPostThreads)
    varlen_bwd_post_kernel(const int* count, const float* acc, const int32_t* row_of, __nv_bfloat16* __restrict__ dq,
                           int Tq, int Hq, float scale) {
  pdl_wait();
  if (*count < 0) return;
  const int per_row = Hq * (bwd::D / 4), lane = threadIdx.x & 31;
  const int n_warps = int(gridDim.x) * (kPostThreads / 32);
  for (long long t = blockIdx.x * (kPostThreads / 32) + (threadIdx.x >> 5); t < Tq; t += n_warps) {
    const int r = row_of[t];
    if (r < 0) continue;
    const float4* src = reinterpret_cast<const float4*>(acc) + size_t(r) * per_row;
    uint2* dst = reinterpret_cast<uint2*>(dq) + size_t(t) * per_row;
#pragma unroll 4
    for (int e = lane; e < per_row; e += 32) {
      const float4 v = src[e];
      dst[e] = make_uint2(pack_bf16x2(v.x * scale, v.y * scale), pack_bf16x2(v.z * scale, v.w * scale));
    }
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The backward workspace: its size (workspace null), or where its parts are.
size_t bwd_space(void* workspace, int S, int Tq, int Tk, int Hq, VarPlan* plan, BwdSpace* w) {
  const long long max_blocks = bwd_max_blocks(S, Tk);
  w->acc_rows = ((long long)Tq / kAccRows + S) * kAccRows;
  w->lse_rows = ((long long)Tq / kTileRows + S) * kTileRows;
  const size_t acc = up256(plan_bytes(max_blocks)), lse2 = acc + up256(size_t(w->acc_rows) * Hq * bwd::D * sizeof(float)),
               dd = lse2 + up256(size_t(w->lse_rows) * Hq * sizeof(float)),
               row_of = dd + up256(size_t(w->lse_rows) * Hq * sizeof(float));
  if (workspace != nullptr) {
    char* b = static_cast<char*>(workspace);
    *plan = plan_at(workspace, max_blocks);
    w->acc = reinterpret_cast<float*>(b + acc);
    w->lse2 = reinterpret_cast<float*>(b + lse2);
    w->dd = reinterpret_cast<float*>(b + dd);
    w->row_of = reinterpret_cast<int32_t*>(b + row_of);
  }
  return row_of + up256(size_t(Tq) * sizeof(int32_t));
}

// Rows `stride` elements apart that hold heads * d dense elements: 16-byte aligned rows, and byte offsets
// that the tensor maps take.
bool token_stride_ok(long long stride, int heads, int d) {
  return stride >= (long long)heads * d && stride % 8 == 0 && stride < (1ll << 31);
}

namespace {
attn_status_t varlen_args_status(const void* const* ptrs16, int n, const float* lse, const int32_t* cu_q,
                                 const int32_t* cu_k, int S, int Tq, int Tk, int Hq, int Hkv, int d, long long qs,
                                 long long ks, long long vs, float scale, int causal) {
  for (int i = 0; i < n; ++i)
    if (!ptrs16[i] || !is_aligned16(ptrs16[i])) return ATTN_ERR_INVALID_ARG;
  if (!lse || !cu_q || !cu_k) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3u)
    return ATTN_ERR_INVALID_ARG;
  if (S < 1 || Tq < 1 || Tk < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (d != 32 && d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (!token_stride_ok(qs, Hq, d) || !token_stride_ok(ks, Hkv, d) || !token_stride_ok(vs, Hkv, d))
    return ATTN_ERR_INVALID_ARG;
  if (S > kVarMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}
}  // namespace

}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_fwd_varlen_workspace_bytes(int S, int Tq) {
  if (S < 1 || Tq < 1 || S > kVarMaxSeqs) return 0;
  return plan_bytes(fwd_max_blocks(S, Tq));
}

attn_status_t attn_fwd_varlen(const void* q, const void* k, const void* v, const int32_t* cu_q, const int32_t* cu_k,
                              void* o, float* lse, int S, int Tq, int Tk, int Hq, int Hkv, int d, long long q_stride,
                              long long k_stride, long long v_stride, float scale, int causal, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  const void* ptrs[] = {q, k, v, o};
  attn_status_t st =
      varlen_args_status(ptrs, 4, lse, cu_q, cu_k, S, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, causal);
  if (st != ATTN_OK) return st;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < attn_fwd_varlen_workspace_bytes(S, Tq))
    return ATTN_ERR_WORKSPACE;
  const long long max_blocks = fwd_max_blocks(S, Tq);
  if (max_blocks * Hq > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;  // units are counted in 32 bits
  const int ctas = fwd_varlen_ctas(d);
  if (ctas <= 0) return ATTN_ERR_CUDA;
  const VarPlan plan = plan_at(workspace, max_blocks);
  varlen_plan_kernel<<<1, kPlanThreads, 0, stream>>>(cu_q, cu_k, S, Tq, Tk, causal, Hq, Hkv,
                                                     fwd_varlen_groups(Tk, Hkv, d, causal), ctas, plan);
  if (cudaPeekAtLastError() != cudaSuccess) return cudaGetLastError(), ATTN_ERR_CUDA;
  return fwd_varlen_dispatch(plan, q, k, v, o, lse, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, causal,
                             stream);
}

size_t attn_bwd_varlen_workspace_bytes(int S, int Tq, int Tk, int Hq, int d) {
  if (S < 1 || Tq < 1 || Tk < 1 || Hq < 1 || d < 1 || S > kVarMaxSeqs) return 0;
  VarPlan plan;
  BwdSpace w;
  return bwd_space(nullptr, S, Tq, Tk, Hq, &plan, &w);
}

attn_status_t attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse,
                              const void* dout, const int32_t* cu_q, const int32_t* cu_k, void* dq, void* dk, void* dv,
                              int S, int Tq, int Tk, int Hq, int Hkv, int d, long long q_stride, long long k_stride,
                              long long v_stride, float scale, int causal, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  const void* ptrs[] = {q, k, v, o, dout, dq, dk, dv};
  attn_status_t st =
      varlen_args_status(ptrs, 8, lse, cu_q, cu_k, S, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, causal);
  if (st != ATTN_OK) return st;
  if (d != 128) return ATTN_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < attn_bwd_varlen_workspace_bytes(S, Tq, Tk, Hq, d))
    return ATTN_ERR_WORKSPACE;
  VarPlan plan;
  BwdSpace w;
  bwd_space(workspace, S, Tq, Tk, Hq, &plan, &w);
  // tile coordinates, and the grid, are 32-bit
  if (plan.max_blocks * Hkv > 0x7FFFFFFFll || w.acc_rows > 0x7FFFFFFFll || w.lse_rows > 0x7FFFFFFFll)
    return ATTN_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // a warp per row, at most two blocks of them per SM
  const long long want = ((long long)Tq + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
  const unsigned rows_grid = unsigned(want < 2ll * sms ? want : 2ll * sms);
  varlen_bwd_pre_kernel<<<1 + rows_grid, kPlanThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, cu_q, cu_k, S, Tq, Tk, Hq,
      causal, plan, w);
  if (cudaPeekAtLastError() != cudaSuccess) return cudaGetLastError(), ATTN_ERR_CUDA;
  st = bwd_varlen_launch(plan, q, k, v, dout, dk, dv, w.acc, w.acc_rows, w.lse2, w.dd, w.lse_rows, Tq, Tk, Hq, Hkv,
                         q_stride, k_stride, v_stride, scale, causal, stream);
  if (st != ATTN_OK) return st;
  const long long post = ((long long)Tq + kPostThreads / 32 - 1) / (kPostThreads / 32);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(unsigned(post < 16ll * sms ? post : 16ll * sms));
  lc.blockDim = dim3(kPostThreads);
  lc.stream = stream;
  lc.attrs = at;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, varlen_bwd_post_kernel, static_cast<const int*>(plan.count),
                         static_cast<const float*>(w.acc), static_cast<const int32_t*>(w.row_of),
                         static_cast<__nv_bfloat16*>(dq), Tq, Hq, scale) != cudaSuccess)
    return cudaGetLastError(), ATTN_ERR_CUDA;
  return ATTN_OK;
}

}  // extern "C"
