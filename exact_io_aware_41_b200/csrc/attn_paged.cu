// Paged KV cache: single-token attention over it (attn_decode_paged) and the writes into it
// (attn_cache_append). Plain decode kernel: one warp per query head row, tokens one after the other.
#include <cuda_bf16.h>
#include <math.h>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn {

// Length of a sequence within the pages its table row can name; flags others.
__device__ __forceinline__ int paged_len(const int32_t* kv_lens, int b, long long cap) {
  const int L = kv_lens[b];
  if (L < 0 || L > cap) {
    atomicOr(&g_error_word, kErrBadLengthBit);
    return L < 0 ? 0 : int(cap);
  }
  return L;
}

// Page number within the pool; flags others.
__device__ __forceinline__ int page_in_pool(int p, int n_pages) {
  if (unsigned(p) >= unsigned(n_pages)) {
    atomicOr(&g_error_word, kErrBadPageBit);
    return p < 0 ? 0 : n_pages - 1;
  }
  return p;
}

template <int D>
__global__ void __launch_bounds__(128)
    decode_paged_simple_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kp,
                               const __nv_bfloat16* __restrict__ vp, const int32_t* __restrict__ table,
                               const int32_t* __restrict__ kv_lens, int n_pages, int page_size, int max_pages,
                               __nv_bfloat16* __restrict__ o, float* __restrict__ lse, int B, int Hq, int Hkv,
                               long long q_stride, float scale) {
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5;
  if (w >= (long long)B * Hq) return;
  const int b = int(w / Hq), h = int(w % Hq), g = h / (Hq / Hkv);
  const int L = paged_len(kv_lens, b, (long long)max_pages * page_size);
  float qf[D / 32], x[D / 32], acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    qf[i] = __bfloat162float(q[b * q_stride + h * D + lane + 32 * i]);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < L; ++t) {
    const int p = page_in_pool(table[size_t(b) * max_pages + t / page_size], n_pages);
    const size_t row = ((size_t(p) * page_size + t % page_size) * Hkv + g) * D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(qf[i], __bfloat162float(kp[row + lane + 32 * i]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= scale;
    const float mn = fmaxf(m, s), f = expf(m - mn), pr = expf(s - mn);
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = __bfloat162float(vp[row + lane + 32 * i]);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(pr, x[i], acc[i] * f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[(size_t(b) * Hq + h) * D + lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
  if (lane == 0) lse[size_t(b) * Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

// New rows into the pages of their sequences: pure copies. A block takes `rows` consecutive packed rows:
// its first threads look up where each of them goes (the sequence by bisection of the offsets, the page
// from the table; -1 for a row that is not written), then all threads copy 16-byte units of K and V.
// Bound by memory: every row is read and written once (2 * 2 * Hkv * d bytes per token).
constexpr int kAppendRows = 8;   // most rows of one block
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads)
    cache_append_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                        const int32_t* __restrict__ cu, const int32_t* __restrict__ table,
                        const int32_t* __restrict__ kv_lens, uint4* __restrict__ k_pages, uint4* __restrict__ v_pages,
                        int B, int T, int n_pages, int page_size, int max_pages, int units, long long ks_units,
                        long long vs_units, int rows) {
  __shared__ long long dst[kAppendRows];  // 16-byte unit of the row's place in the pools, or -1
  const int t0 = blockIdx.x * rows;
  if (threadIdx.x < rows) {
    const int t = t0 + threadIdx.x;
    long long at = -1;
    if (t < T) {
      int b = t, i = 0, n = 1;
      bool owned = true;
      if (cu != nullptr) {
        owned = t >= cu[0] && t < cu[B];
        if (owned) {
          int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t)
              lo = mid;
            else
              hi = mid;
          }
          b = lo;
          i = t - cu[b];
          n = cu[b + 1] - cu[b];
        }
      }
      if (owned) {
        const long long pos = (long long)kv_lens[b] - n + i;
        if (pos < 0 || pos >= (long long)max_pages * page_size) {
          atomicOr(&g_error_word, kErrBadLengthBit);
        } else {
          const int p = table[size_t(b) * max_pages + int(pos / page_size)];
          if (unsigned(p) >= unsigned(n_pages))
            atomicOr(&g_error_word, kErrBadPageBit);
          else
            at = ((long long)p * page_size + pos % page_size) * units;
        }
      }
    }
    dst[threadIdx.x] = at;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < rows * units; u += kAppendThreads) {
    const int r = u / units, c = u - r * units;
    const long long at = dst[r];
    if (at < 0) continue;
    const uint4 a = k_new[(t0 + r) * ks_units + c], b = v_new[(t0 + r) * vs_units + c];
    k_pages[at + c] = a;
    v_pages[at + c] = b;
  }
}

}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1) return 0;
  return 16;
}

attn_status_t attn_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                                const int32_t* kv_lens, int n_pages, int page_size, int max_pages, void* o, float* lse,
                                int B, int Hq, int Hkv, int d, long long q_stride, float scale, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned16(q) || !is_aligned16(k_pages) || !is_aligned16(v_pages) || !is_aligned16(o) ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(page_table) |
        reinterpret_cast<uintptr_t>(kv_lens)) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || n_pages < 1 || page_size < 1 || max_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if ((d != 32 && d != 64 && d != 128 && d != 256) || Hq / Hkv > 16) return ATTN_ERR_UNSUPPORTED;
  if (!token_stride_ok(q_stride, Hq, d)) return ATTN_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || page_size > 65536) return ATTN_ERR_UNSUPPORTED;
  if (workspace == nullptr || !is_aligned16(workspace) ||
      workspace_bytes < attn_decode_paged_workspace_bytes(B, Hq, Hkv, d))
    return ATTN_ERR_WORKSPACE;
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* kb = static_cast<const __nv_bfloat16*>(k_pages);
  const auto* vb = static_cast<const __nv_bfloat16*>(v_pages);
  auto* ob = static_cast<__nv_bfloat16*>(o);
  const unsigned grid = unsigned(((long long)B * Hq + 3) / 4);
  switch (d) {
    case 32:
      decode_paged_simple_kernel<32><<<grid, 128, 0, stream>>>(qb, kb, vb, page_table, kv_lens, n_pages, page_size,
                                                               max_pages, ob, lse, B, Hq, Hkv, q_stride, scale);
      break;
    case 64:
      decode_paged_simple_kernel<64><<<grid, 128, 0, stream>>>(qb, kb, vb, page_table, kv_lens, n_pages, page_size,
                                                               max_pages, ob, lse, B, Hq, Hkv, q_stride, scale);
      break;
    case 128:
      decode_paged_simple_kernel<128><<<grid, 128, 0, stream>>>(qb, kb, vb, page_table, kv_lens, n_pages, page_size,
                                                                max_pages, ob, lse, B, Hq, Hkv, q_stride, scale);
      break;
    default:
      decode_paged_simple_kernel<256><<<grid, 128, 0, stream>>>(qb, kb, vb, page_table, kv_lens, n_pages, page_size,
                                                                max_pages, ob, lse, B, Hq, Hkv, q_stride, scale);
  }
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : (cudaGetLastError(), ATTN_ERR_CUDA);
}

attn_status_t attn_cache_append(const void* k_new, const void* v_new, const int32_t* cu, const int32_t* page_table,
                                const int32_t* kv_lens, void* k_pages, void* v_pages, int B, int T, int n_pages,
                                int page_size, int max_pages, int Hkv, int d, long long k_stride, long long v_stride,
                                cudaStream_t stream) {
  if (!k_new || !v_new || !page_table || !kv_lens || !k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
  if (!is_aligned16(k_new) || !is_aligned16(v_new) || !is_aligned16(k_pages) || !is_aligned16(v_pages) ||
      ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(page_table) |
        reinterpret_cast<uintptr_t>(kv_lens)) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || n_pages < 1 || page_size < 1 || max_pages < 1 || Hkv < 1 || d < 1) return ATTN_ERR_INVALID_ARG;
  if ((long long)Hkv * d % 8 != 0 || (long long)Hkv * d > (1 << 24)) return ATTN_ERR_INVALID_ARG;
  if (!token_stride_ok(k_stride, Hkv, d) || !token_stride_ok(v_stride, Hkv, d)) return ATTN_ERR_INVALID_ARG;
  if (cu == nullptr && T != B) return ATTN_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // one row per block while that leaves SMs idle (latency), up to kAppendRows where there are many
  const long long per = T / (8ll * sms);
  const int rows = per < 1 ? 1 : per > kAppendRows ? kAppendRows : int(per);
  cache_append_kernel<<<unsigned((T + (long long)rows - 1) / rows), kAppendThreads, 0, stream>>>(
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), cu, page_table, kv_lens,
      static_cast<uint4*>(k_pages), static_cast<uint4*>(v_pages), B, T, n_pages, page_size, max_pages, Hkv * d / 8,
      k_stride / 8, v_stride / 8, rows);
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : (cudaGetLastError(), ATTN_ERR_CUDA);
}

}  // extern "C"
