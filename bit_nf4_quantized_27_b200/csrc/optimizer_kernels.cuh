// One optimiser step over a list of tensors: the norm of all gradients with the
// factor that clips it, and AdamW with states in 32 bits or in 8.
//
// A list is a device table: the qlora_tensor structs, then one (tensor, chunk)
// pair for each chunk of 2048 elements, so that a CTA finds its work with two
// loads whatever the tensors' sizes.
#pragma once

#include <cuda_bf16.h>

#include "nf4_device.cuh"
#include "sm100_ptx.cuh"

namespace qlora {

constexpr int kOptThreads = 256;
constexpr int kOptChunk = 2048;  // elements: eight warps x one block of 256
static_assert(kOptChunk == (kOptThreads / 32) * QLORA_STATE_BLOCK, "one state block per warp and chunk");

struct TensorTable {
  const qlora_tensor *tensors;
  const int2 *chunks;  // (tensor, chunk of it)
  int64_t n_chunks;
};

// Table entries travel as kernel arguments: no host memory outlives the call.
constexpr int kTablePerLaunch = 48;
struct TableWrite {
  qlora_tensor t[kTablePerLaunch];
  int64_t first_chunk[kTablePerLaunch + 1];
  qlora_tensor *tensors;
  int2 *chunks;
  int base;  // list place of t[0]
};
static_assert(sizeof(TableWrite) <= 4096, "kernel arguments");

// Block x writes entry x and its chunk pairs.
__global__ void tensor_table_kernel(const __grid_constant__ TableWrite w) {
  const int i = blockIdx.x;
  if (threadIdx.x == 0) w.tensors[w.base + i] = w.t[i];
  const int64_t c0 = w.first_chunk[i], n = w.first_chunk[i + 1] - c0;
  for (int64_t c = threadIdx.x; c < n; c += blockDim.x) w.chunks[c0 + c] = make_int2(w.base + i, static_cast<int>(c));
}

// ---------------------------------------------------------------------------
// Norm of all gradients.  Each thread sums the squares of its elements in
// float64 (a float32 square overflows above 1.8e19, and its sums lose what a
// long list of small tensors needs); CTA sums go to ws in CTA order and the CTA that
// finishes last adds them in that order, so the result does not depend on the
// schedule.
// ---------------------------------------------------------------------------
constexpr int kNormMaxCtas = 1184;

__device__ __forceinline__ double block_sum(double x, double *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_down_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kOptThreads / 32; ++i) s += red[i];
  return s;  // thread 0
}

template <typename G>
__global__ void __launch_bounds__(kOptThreads) grad_norm_kernel(const TensorTable tab, float max_norm,
                                                                float *__restrict__ out, uint32_t *counter,
                                                                double *partial) {
  __shared__ double red[kOptThreads / 32];
  __shared__ bool last;
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < tab.n_chunks; c += gridDim.x) {
    const int2 tc = tab.chunks[c];
    const G *g = static_cast<const G *>(tab.tensors[tc.x].grad);
    const int64_t n = tab.tensors[tc.x].n, e0 = static_cast<int64_t>(tc.y) * kOptChunk;
    for (int64_t e = e0 + threadIdx.x; e < n && e < e0 + kOptChunk; e += kOptThreads) {
      const double x = static_cast<double>(static_cast<float>(g[e]));
      s += x * x;
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) {
    partial[blockIdx.x] = s;
    __threadfence();
    last = atomicAdd(counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kOptThreads) t += __ldcg(partial + i);
  t = block_sum(t, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(t);
    const bool ok = isfinite(static_cast<float>(norm));
    out[0] = static_cast<float>(norm);
    out[1] = ok ? static_cast<float>(fmin(1.0, static_cast<double>(max_norm) / (norm + 1e-6))) : __int_as_float(0x7fc00000);
    *counter = 0;
  }
}

// ---------------------------------------------------------------------------
// AdamW.  The arithmetic is adamw_one's, float32 operation by operation.  8-bit
// states: a warp holds one block of 256 elements, eight consecutive ones per
// lane; the block's new maxima come from warp shuffles, the codes from adding
// random bits below the last mantissa bit kept and cutting them off.  The result is
// unbiased, which round-to-nearest is not where it matters: a step changes the
// variance by 1 - beta2 of itself, far less than half an E5M2 step, and a rounded
// variance would never move.
// ---------------------------------------------------------------------------
struct AdamWMulti {
  float beta1, beta2, eps, sqrt_bc2;
  double lr, weight_decay, step_size;  // step_size = lr / bc1
  const float *clip;                   // nullable [2]
  uint32_t seed;
};

// 32 bits for an element: multiplications by the first fraction bits of the golden
// ratio and of the square roots of 2 and 3, with the high half folded down between them.
__device__ __forceinline__ uint32_t state_hash(uint32_t element, uint32_t stream) {
  uint32_t x = (element + stream) * 0x9E3779B9u;
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// x >= 0 to a float8 value (as float32) at or next to it, up with the probability
// of rnd's kDrop bits.  Below the format's least normal value kLeast the step is
// that of the first binade: adding kLeast puts x there.
template <int kDrop>
__device__ __forceinline__ float round_float8(float x, uint32_t rnd, float least, float most) {
  const bool small = x < least;
  const float z = small ? __fadd_rn(x, least) : x;
  const float y = __uint_as_float((__float_as_uint(z) + rnd) & ~((1u << kDrop) - 1u));
  return fminf(small ? __fsub_rn(y, least) : y, most);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = (y > x || y != y) ? y : x;  // a NaN stays
  }
  return x;
}

template <typename G, bool EIGHT>
__global__ void __launch_bounds__(kOptThreads) adamw_multi_kernel(const TensorTable tab, const AdamWMulti a) {
  const float clip = a.clip ? a.clip[1] : 1.0f;
  if (clip != clip) return;  // the norm was not finite: the step changes nothing
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float omb1 = 1.0f - a.beta1, omb2 = 1.0f - a.beta2;
  for (int64_t c = blockIdx.x; c < tab.n_chunks; c += gridDim.x) {
    const int2 tc = tab.chunks[c];
    const qlora_tensor t = tab.tensors[tc.x];
    const double lr_scale = static_cast<double>(t.lr_scale);
    const float decay = static_cast<float>(1.0 - a.lr * lr_scale * a.weight_decay);
    const float step_size = static_cast<float>(a.step_size * lr_scale);
    const int64_t blk = static_cast<int64_t>(tc.y) * (kOptThreads / 32) + warp;
    const int64_t e0 = blk * QLORA_STATE_BLOCK;
    if (e0 >= t.n) continue;
    float m[8], v[8];
    float sm = 0.0f, sv = 0.0f;
    if (EIGHT) { sm = t.exp_avg_scale[blk]; sv = t.exp_avg_sq_scale[blk]; }
    float mm = 0.0f, vm = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t e = e0 + 8 * lane + i;
      m[i] = v[i] = 0.0f;
      if (e >= t.n) continue;
      float p = t.param[e];
      const float g = __fmul_rn(static_cast<float>(static_cast<const G *>(t.grad)[e]), clip);
      if (EIGHT) {
        m[i] = __fmul_rn(scale_code_value(static_cast<const uint8_t *>(t.exp_avg)[e], QLORA_SCALE_E4M3), sm);
        v[i] = __fmul_rn(scale_code_value(static_cast<const uint8_t *>(t.exp_avg_sq)[e], QLORA_SCALE_E5M2), sv);
      } else {
        m[i] = static_cast<const float *>(t.exp_avg)[e];
        v[i] = static_cast<const float *>(t.exp_avg_sq)[e];
      }
      m[i] = __fadd_rn(__fmul_rn(a.beta1, m[i]), __fmul_rn(omb1, g));
      v[i] = __fadd_rn(__fmul_rn(a.beta2, v[i]), __fmul_rn(omb2, __fmul_rn(g, g)));
      const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(v[i]), a.sqrt_bc2), a.eps);
      p = __fsub_rn(__fmul_rn(p, decay), __fdiv_rn(__fmul_rn(step_size, m[i]), denom));
      t.param[e] = p;
      if (t.param_bf16) static_cast<__nv_bfloat16 *>(t.param_bf16)[e] = __float2bfloat16_rn(p);
      if (!EIGHT) {
        static_cast<float *>(t.exp_avg)[e] = m[i];
        static_cast<float *>(t.exp_avg_sq)[e] = v[i];
      }
      const float am = fabsf(m[i]);
      mm = (am > mm || am != am) ? am : mm;
      vm = (v[i] > vm || v[i] != v[i]) ? v[i] : vm;
    }
    if (EIGHT) {
      mm = warp_max(mm);
      vm = warp_max(vm);
      // a maximum below 2^-100 is a block of zeros: its reciprocal would overflow
      const float im = mm < 0x1p-100f ? 0.0f : __fdiv_rn(448.0f, mm), iv = vm < 0x1p-100f ? 0.0f : __fdiv_rn(57344.0f, vm);
      if (lane == 0) {
        t.exp_avg_scale[blk] = mm < 0x1p-100f ? 0.0f : __fdiv_rn(mm, 448.0f);
        t.exp_avg_sq_scale[blk] = vm < 0x1p-100f ? 0.0f : __fdiv_rn(vm, 57344.0f);
      }
      const uint32_t stream = a.seed * 0xB7E15163u + static_cast<uint32_t>(tc.x) * 0x3504F333u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t e = e0 + 8 * lane + i;
        if (e >= t.n) continue;
        const uint32_t h = state_hash(static_cast<uint32_t>(e), stream);
        const float qm = round_float8<20>(__fmul_rn(fabsf(m[i]), im), h & 0xFFFFFu, 0x1p-6f, 448.0f);
        float qv = round_float8<21>(__fmul_rn(v[i], iv), h >> 11, 0x1p-14f, 57344.0f);
        if (v[i] > 0.0f && iv > 0.0f) qv = fmaxf(qv, 0x1p-16f);
        static_cast<uint8_t *>(t.exp_avg)[e] = f32_to_e4m3(copysignf(qm, m[i]));
        static_cast<uint8_t *>(t.exp_avg_sq)[e] = scale_code_encode(qv, QLORA_SCALE_E5M2);
      }
    }
  }
}

}  // namespace qlora
