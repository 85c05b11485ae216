// Packed sequences of different lengths: prefill forward and backward over S sequences laid end to end
// (attn_fwd_varlen, attn_bwd_varlen). Plain kernels: one warp per output row, keys (or queries) one after
// the other.
#include <cuda_bf16.h>
#include <math.h>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn {

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

template <int D>
__global__ void __launch_bounds__(256) varlen_fwd_simple_kernel(const VarArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5;
  if (*a.ok == 0 || w >= (long long)a.Tq * a.Hq) return;
  const int t = int(w / a.Hq), h = int(w % a.Hq), g = h / (a.Hq / a.Hkv);
  const int s = seq_of_row(a.cu_q, a.S, t);
  if (s < 0) return;
  const int i = t - a.cu_q[s], nq = a.cu_q[s + 1] - a.cu_q[s], k0 = a.cu_k[s], nk = a.cu_k[s + 1] - k0;
  const int end = a.causal ? min(nk, i + nk - nq + 1) : nk;
  float q[D / 32], k[D / 32], acc[D / 32];
  load_row<D>(a.q + t * a.qs + h * D, lane, q);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    load_row<D>(a.k + (k0 + j) * a.ks + g * D, lane, k);
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x = fmaf(q[e], k[e], x);
    x = warp_sum(x) * a.scale;
    const float mn = fmaxf(m, x), f = expf(m - mn), p = expf(x - mn);
    m = mn;
    l = l * f + p;
    load_row<D>(a.v + (k0 + j) * a.vs + g * D, lane, k);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(p, k[e], acc[e] * f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) a.out[(size_t(t) * a.Hq + h) * D + lane + 32 * e] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0) a.lse[size_t(h) * a.Tq + t] = l > 0.f ? m + logf(l) : -INFINITY;
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
  return 256;
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
  VarArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
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
  const unsigned grid = warps_grid((long long)Tq * Hq);
  switch (d) {
    case 32: varlen_fwd_simple_kernel<32><<<grid, 256, 0, stream>>>(a); break;
    case 64: varlen_fwd_simple_kernel<64><<<grid, 256, 0, stream>>>(a); break;
    case 128: varlen_fwd_simple_kernel<128><<<grid, 256, 0, stream>>>(a); break;
    default: varlen_fwd_simple_kernel<256><<<grid, 256, 0, stream>>>(a); break;
  }
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : (cudaGetLastError(), ATTN_ERR_CUDA);
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
