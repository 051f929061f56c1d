// Many adapters on one base: the tokens grouped by adapter, the adapters' term of
// the forward pass and its gradients (see qlora_adapters_fwd in qlora_nf4.h).
#pragma once

#include <cuda_bf16.h>

#include "nf4_device.cuh"
#include "sm100_ptx.cuh"

namespace qlora {

// ---------------------------------------------------------------------------
// Tokens grouped by adapter: a stable counting sort in one CTA.  Warp w owns the
// w-th contiguous piece of the tokens and counts its keys in its own row of
// shared counters; a running sum over (key, warp) turns the counts into first
// places; each warp then walks its piece again, 32 tokens at a time, and places
// them with the rank among equal keys that match gives.  Key n: no adapter.
// ---------------------------------------------------------------------------
constexpr int kGroupThreads = 1024;

__device__ __forceinline__ int group_key(const int32_t *idx, int64_t t, int n, uint32_t *status) {
  const int a = idx[t];
  if (a >= 0 && a < n) return a;
  if (a != -1) raise_status(status, QLORA_ERR_INVALID_ARGUMENT);
  return n;
}

__global__ void __launch_bounds__(kGroupThreads) adapter_groups_kernel(const int32_t *__restrict__ idx, int64_t M, int n,
                                                                       int32_t *__restrict__ order,
                                                                       int32_t *__restrict__ offsets, uint32_t *status) {
  extern __shared__ int32_t group_counts[];  // [warps][n + 1]
  __shared__ int32_t scan[kGroupThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, keys = n + 1;
  int32_t *mine = group_counts + warp * keys;
  for (int i = threadIdx.x; i < warps * keys; i += blockDim.x) group_counts[i] = 0;
  __syncthreads();
  const int64_t per = ((M + warps - 1) / warps + 31) / 32 * 32;
  const int64_t t0 = warp * per, t1 = min(M, t0 + per);
  for (int64_t t = t0 + lane; t < t1; t += 32) atomicAdd(&mine[group_key(idx, t, n, status)], 1);
  __syncthreads();
  // first place of each key, then of each (key, warp)
  const int per_thread = (keys + blockDim.x - 1) / blockDim.x, k0 = threadIdx.x * per_thread;
  int32_t sum = 0;
  for (int k = k0; k < min(keys, k0 + per_thread); ++k)
    for (int w = 0; w < warps; ++w) sum += group_counts[w * keys + k];
  scan[threadIdx.x] = sum;
  __syncthreads();
  for (int o = 1; o < static_cast<int>(blockDim.x); o <<= 1) {
    const int32_t x = threadIdx.x >= o ? scan[threadIdx.x - o] : 0;
    __syncthreads();
    scan[threadIdx.x] += x;
    __syncthreads();
  }
  int32_t at = scan[threadIdx.x] - sum;
  for (int k = k0; k < min(keys, k0 + per_thread); ++k) {
    offsets[k] = at;  // key n: the number of tokens with an adapter
    for (int w = 0; w < warps; ++w) {
      const int32_t c = group_counts[w * keys + k];
      group_counts[w * keys + k] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t b = t0; b < t1; b += 32) {
    const int64_t t = b + lane;
    const bool in = t < t1;
    const int key = in ? group_key(idx, t, n, nullptr) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (in) order[mine[key] + before] = static_cast<int32_t>(t);
    __syncwarp();
    if (in && before == 0) mine[key] += __popc(same);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// The plain kernels: every output element from its formula, in float32.
// ---------------------------------------------------------------------------
struct PoolArgs {
  const __nv_bfloat16 *A, *B;  // [n, r, K], [n, N, r]
  const int32_t *ranks;        // nullable
  const float *scales;
  int n, r;
  int64_t M, N, K;
  const int32_t *order, *offsets;
  uint32_t *status;
};

// Rank of adapter a: a multiple of 8 in [0, r].
__device__ __forceinline__ int pool_rank(const PoolArgs &p, int a) {
  if (!p.ranks) return p.r;
  const int k = p.ranks[a], c = min(max(k, 0), p.r) & ~7;
  if (c != k) raise_status(p.status, QLORA_ERR_INVALID_ARGUMENT);
  return c;
}

// Adapter of place i of order; -1 past the last group.
__device__ __forceinline__ int pool_adapter(const PoolArgs &p, int64_t i) {
  if (i >= p.offsets[p.n]) return -1;
  int lo = 0, hi = p.n - 1;  // the last adapter whose group begins at or before i
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.offsets[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int64_t pool_token(const PoolArgs &p, int64_t i) {
  const int64_t t = p.order[i];
  if (t >= 0 && t < p.M) return t;
  raise_status(p.status, QLORA_ERR_INVALID_ARGUMENT);
  return -1;
}

// The intermediates T = X A^T and U = dY B are [M, r] in float32 and kept as three bf16 planes [3, M, r], each the rounding
// of what the ones before leave: 24 bits together, in the type the tensor cores take beside bf16 operands.
constexpr int kPoolPlanes = 3;

__device__ __forceinline__ float pool_value(const __nv_bfloat16 *P, int64_t plane, int64_t i) {
  return __bfloat162float(P[i]) + (__bfloat162float(P[plane + i]) + __bfloat162float(P[2 * plane + i]));
}

// P = V W_a: a warp per (place, rank).  T: V = X, W = A^T; U: V = dY, W = B.
__global__ void pool_down_kernel(const PoolArgs p, const __nv_bfloat16 *__restrict__ V, int64_t ldv, int64_t len,
                                 bool transposed, __nv_bfloat16 *__restrict__ P) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + (threadIdx.x >> 5); w < p.M * p.r; w += warps) {
    const int64_t i = w / p.r;
    const int j = static_cast<int>(w - i * p.r);
    const int a = pool_adapter(p, i);
    if (a < 0) return;
    const int64_t t = pool_token(p, i);
    if (t < 0) continue;
    float s = 0.0f;
    if (j < pool_rank(p, a))
      for (int64_t k = lane; k < len; k += 32) {
        const __nv_bfloat16 wv = transposed ? p.B[(a * p.N + k) * p.r + j] : p.A[(static_cast<int64_t>(a) * p.r + j) * p.K + k];
        s = fmaf(__bfloat162float(V[t * ldv + k]), __bfloat162float(wv), s);
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      for (int q = 0; q < kPoolPlanes; ++q) {
        const __nv_bfloat16 h = __float2bfloat16_rn(s);
        P[q * p.M * p.r + t * p.r + j] = h;
        s -= __bfloat162float(h);
      }
    }
  }
}

// Out[t] += s_a P[t] W_a: a thread per (place, column).  Y: W = B^T; dX: W = A.
template <typename O>
__global__ void pool_up_kernel(const PoolArgs p, const __nv_bfloat16 *__restrict__ P,
                               bool transposed, int64_t cols, O *__restrict__ Out, int64_t ldo) {
  const int64_t total = p.M * cols;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; w < total;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t i = w / cols, c = w - i * cols;
    const int a = pool_adapter(p, i);
    if (a < 0) return;
    const int64_t t = pool_token(p, i);
    if (t < 0) continue;
    const int rank = pool_rank(p, a);
    float s = 0.0f;
    for (int j = 0; j < rank; ++j) {
      const __nv_bfloat16 wv = transposed ? p.B[(a * p.N + c) * p.r + j] : p.A[(static_cast<int64_t>(a) * p.r + j) * p.K + c];
      s = fmaf(pool_value(P, p.M * p.r, t * p.r + j), __bfloat162float(wv), s);
    }
    if (rank) Out[t * ldo + c] = static_cast<O>(static_cast<float>(Out[t * ldo + c]) + p.scales[a] * s);
  }
}

// Grad_a = s_a sum_t P[t]^T V[t]: a thread per (adapter, rank, column).  dA [n, r, cols]: P = U, V = X;
// dB [n, cols, r] (by_column): P = T, V = dY.
template <typename O>
__global__ void pool_grad_kernel(const PoolArgs p, const __nv_bfloat16 *__restrict__ P,
                                 const __nv_bfloat16 *__restrict__ V, int64_t ldv, int64_t cols, bool by_column,
                                 O *__restrict__ Grad) {
  const int64_t total = static_cast<int64_t>(p.n) * p.r * cols;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; w < total;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t aj = w / cols, c = w - aj * cols;
    const int a = static_cast<int>(aj / p.r), j = static_cast<int>(aj - static_cast<int64_t>(a) * p.r);
    float s = 0.0f;
    if (j < pool_rank(p, a))
      for (int64_t i = max(p.offsets[a], 0); i < min(static_cast<int64_t>(p.offsets[a + 1]), p.M); ++i) {
        const int64_t t = pool_token(p, i);
        if (t < 0) continue;
        s = fmaf(pool_value(P, p.M * p.r, t * p.r + j), __bfloat162float(V[t * ldv + c]), s);
      }
    Grad[by_column ? (a * cols + c) * p.r + j : w] = static_cast<O>(p.scales[a] * s);
  }
}

}  // namespace qlora
