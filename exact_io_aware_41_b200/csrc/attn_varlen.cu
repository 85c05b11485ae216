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

// Tiles of 128 keys that forward block `blk` of a sequence walks (0: none of its rows sees a key).
__device__ __forceinline__ int fwd_block_tiles(const PlanSeq& s, int blk, int causal) {
  const int left = s.nq - blk * kFwdBlockRows;
  const int end = causal ? min(s.nkv, min(kFwdBlockRows, left) + s.nkv - left) : s.nkv;
  return end > 0 ? (end + kTileRows - 1) / kTileRows : 0;
}

__global__ void __launch_bounds__(kPlanThreads)
    varlen_plan_kernel(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int S, int Tq, int Tk,
                       int causal, VarPlan plan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  // ---- check the offsets, and the largest number of tiles
  __shared__ int bins[kPlanBins], warp_sum[kPlanThreads / 32], most;
  if (threadIdx.x == 0) most = 0;
  bins[threadIdx.x] = 0;
  bool bad = false;
  int mx = 0;
  for (int s = threadIdx.x; s < S; s += kPlanThreads) {
    const int a = cu_q[s], b = cu_q[s + 1], c = cu_k[s], e = cu_k[s + 1];
    bad |= a < 0 || b < a || b > Tq || c < 0 || e < c || e > Tk;
    mx = max(mx, e - c);
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) {
      *plan.count = 0;
      *plan.claim = 0;
      atomicOr(&g_error_word, kErrBadLengthBit);
    }
    return;
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) atomicMax(&most, mx);
  __syncthreads();
  const int max_tiles = (most + kTileRows - 1) / kTileRows;
  auto bin_of = [&](int tiles) -> int {  // 0: heaviest
    return max_tiles < kPlanBins ? max_tiles - tiles : int((long long)(max_tiles - tiles) * (kPlanBins - 1) / max_tiles);
  };
  // f(sequence, block) for every block: a thread takes a sequence, a warp one with many blocks
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
      const int nb = (q.nq + kFwdBlockRows - 1) / kFwdBlockRows;
      if (nb <= kPlanOwnBlocks)
        for (int i = 0; i < nb; ++i) f(q, i);
      for (unsigned many = __ballot_sync(0xffffffffu, nb > kPlanOwnBlocks); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const PlanSeq w = {__shfl_sync(0xffffffffu, q.q0, src), __shfl_sync(0xffffffffu, q.nq, src),
                           __shfl_sync(0xffffffffu, q.k0, src), __shfl_sync(0xffffffffu, q.nkv, src)};
        const int wnb = __shfl_sync(0xffffffffu, nb, src);
        for (int i = lane; i < wnb; i += 32) f(w, i);
      }
    }
  };
  each_block([&](const PlanSeq& q, int i) { atomicAdd(&bins[bin_of(fwd_block_tiles(q, i, causal))], 1); });
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
  each_block([&](const PlanSeq& q, int i) {
    const int at = atomicAdd(&bins[bin_of(fwd_block_tiles(q, i, causal))], 1);
    if (at >= plan.max_blocks) return;
    VarUnit u;
    u.q_row = q.q0 + i * kFwdBlockRows;
    u.nq = q.nq - i * kFwdBlockRows;
    u.k_row = q.k0;
    u.nkv = q.nkv;
    plan.units[at] = u;
  });
}
static_assert(kPlanBins == kPlanThreads, "one bin per thread");

// Workspace of a plan: count and claim counter, blocks.
long long fwd_max_blocks(int S, int Tq) { return (long long)Tq / kFwdBlockRows + S; }
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

// 1 in ok[0] if both offset arrays are in order, else 0 and the error bit.
__global__ void __launch_bounds__(1024) varlen_check_kernel(const int32_t* __restrict__ cu_q,
                                                            const int32_t* __restrict__ cu_k, int S, int Tq, int Tk,
                                                            int* ok) {
  bool bad = false;
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const int a = cu_q[s], b = cu_q[s + 1], c = cu_k[s], e = cu_k[s + 1];
    bad |= a < 0 || b < a || b > Tq || c < 0 || e < c || e > Tk;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    *ok = bad ? 0 : 1;
    if (bad) atomicOr(&g_error_word, kErrBadLengthBit);
  }
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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct VarArgs {
  const __nv_bfloat16 *q, *k, *v, *o, *dout;
  const int32_t *cu_q, *cu_k;
  __nv_bfloat16 *out, *dq, *dk, *dv;
  float* lse;
  const int* ok;
  int S, Tq, Tk, Hq, Hkv;
  long long qs, ks, vs;
  float scale;
  int causal;
};

template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int lane, float* x) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = __bfloat162float(p[lane + 32 * i]);
}

__global__ void __launch_bounds__(256) varlen_dq_simple_kernel(const VarArgs a) {
  constexpr int D = 128;
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5;
  if (*a.ok == 0 || w >= (long long)a.Tq * a.Hq) return;
  const int t = int(w / a.Hq), h = int(w % a.Hq), g = h / (a.Hq / a.Hkv);
  const int s = seq_of_row(a.cu_q, a.S, t);
  if (s < 0) return;
  const int i = t - a.cu_q[s], nq = a.cu_q[s + 1] - a.cu_q[s], k0 = a.cu_k[s], nk = a.cu_k[s + 1] - k0;
  const int end = a.causal ? min(nk, i + nk - nq + 1) : nk;
  const size_t row = (size_t(t) * a.Hq + h) * D;
  float q[4], o[4], g_o[4], k[4], v[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  load_row<D>(a.q + t * a.qs + h * D, lane, q);
  load_row<D>(a.o + row, lane, o);
  load_row<D>(a.dout + row, lane, g_o);
  const float dd = warp_sum(o[0] * g_o[0] + o[1] * g_o[1] + o[2] * g_o[2] + o[3] * g_o[3]);
  const float L = a.lse[size_t(h) * a.Tq + t];
  for (int j = 0; j < end; ++j) {
    load_row<D>(a.k + (k0 + j) * a.ks + g * D, lane, k);
    load_row<D>(a.v + (k0 + j) * a.vs + g * D, lane, v);
    const float x = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * a.scale;
    const float dp = warp_sum(g_o[0] * v[0] + g_o[1] * v[1] + g_o[2] * v[2] + g_o[3] * v[3]);
    const float ds = expf(x - L) * (dp - dd);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) a.dq[row + lane + 32 * e] = __float2bfloat16_rn(acc[e] * a.scale);
}

__global__ void __launch_bounds__(256) varlen_dkv_simple_kernel(const VarArgs a) {
  constexpr int D = 128;
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5;
  if (*a.ok == 0 || w >= (long long)a.Tk * a.Hkv) return;
  const int t = int(w / a.Hkv), g = int(w % a.Hkv), G = a.Hq / a.Hkv;
  const int s = seq_of_row(a.cu_k, a.S, t);
  if (s < 0) return;
  const int j = t - a.cu_k[s], nk = a.cu_k[s + 1] - a.cu_k[s], q0 = a.cu_q[s], nq = a.cu_q[s + 1] - q0;
  float k[4], v[4], q[4], o[4], g_o[4], dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
  load_row<D>(a.k + t * a.ks + g * D, lane, k);
  load_row<D>(a.v + t * a.vs + g * D, lane, v);
  for (int i = a.causal ? max(0, j - (nk - nq)) : 0; i < nq; ++i)
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const size_t row = (size_t(q0 + i) * a.Hq + h) * D;
      load_row<D>(a.q + (q0 + i) * a.qs + h * D, lane, q);
      load_row<D>(a.o + row, lane, o);
      load_row<D>(a.dout + row, lane, g_o);
      const float x = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * a.scale;
      const float dd = warp_sum(o[0] * g_o[0] + o[1] * g_o[1] + o[2] * g_o[2] + o[3] * g_o[3]);
      const float dp = warp_sum(g_o[0] * v[0] + g_o[1] * v[1] + g_o[2] * v[2] + g_o[3] * v[3]);
      const float p = expf(x - a.lse[size_t(h) * a.Tq + q0 + i]), ds = p * (dp - dd);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dv[e] = fmaf(p, g_o[e], dv[e]);
        dk[e] = fmaf(ds, q[e], dk[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a.dk[(size_t(t) * a.Hkv + g) * D + lane + 32 * e] = __float2bfloat16_rn(dk[e] * a.scale);
    a.dv[(size_t(t) * a.Hkv + g) * D + lane + 32 * e] = __float2bfloat16_rn(dv[e]);
  }
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

unsigned warps_grid(long long warps) { return unsigned((warps + 7) / 8); }
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
  const VarPlan plan = plan_at(workspace, max_blocks);
  varlen_plan_kernel<<<1, kPlanThreads, 0, stream>>>(cu_q, cu_k, S, Tq, Tk, causal, plan);
  if (cudaPeekAtLastError() != cudaSuccess) return cudaGetLastError(), ATTN_ERR_CUDA;
  return fwd_varlen_dispatch(plan, q, k, v, o, lse, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, causal,
                             stream);
}

size_t attn_bwd_varlen_workspace_bytes(int S, int Tq, int Tk, int Hq, int d) {
  if (S < 1 || Tq < 1 || Tk < 1 || Hq < 1 || d < 1 || S > kVarMaxSeqs) return 0;
  return 256;
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
  VarArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.o = static_cast<const __nv_bfloat16*>(o);
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.lse = const_cast<float*>(lse);
  a.ok = static_cast<int*>(workspace);
  a.S = S;
  a.Tq = Tq;
  a.Tk = Tk;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.scale = scale;
  a.causal = causal;
  varlen_check_kernel<<<1, 1024, 0, stream>>>(cu_q, cu_k, S, Tq, Tk, static_cast<int*>(workspace));
  varlen_dq_simple_kernel<<<warps_grid((long long)Tq * Hq), 256, 0, stream>>>(a);
  varlen_dkv_simple_kernel<<<warps_grid((long long)Tk * Hkv), 256, 0, stream>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : (cudaGetLastError(), ATTN_ERR_CUDA);
}

}  // extern "C"
