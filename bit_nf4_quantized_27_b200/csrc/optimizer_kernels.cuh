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

// Eight consecutive gradients as float32: wide loads where the address allows them.
__device__ __forceinline__ void load_grads8(const float *g, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(g)), b = __ldcs(reinterpret_cast<const float4 *>(g) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load_grads8(const __nv_bfloat16 *g, float (&x)[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(g));
  x[0] = bf16lo_to_f32(a.x); x[1] = bf16hi_to_f32(a.x); x[2] = bf16lo_to_f32(a.y); x[3] = bf16hi_to_f32(a.y);
  x[4] = bf16lo_to_f32(a.z); x[5] = bf16hi_to_f32(a.z); x[6] = bf16lo_to_f32(a.w); x[7] = bf16hi_to_f32(a.w);
}

template <typename G>
__global__ void __launch_bounds__(kOptThreads) grad_norm_kernel(const TensorTable tab, float max_norm,
                                                                float *__restrict__ out, uint32_t *counter,
                                                                double *partial) {
  __shared__ double red[kOptThreads / 32];
  __shared__ bool last;
  double s = 0.0;
  // A CTA's chunks are neighbours, mostly of one tensor: its entry stays in L1.  Eight CTAs an SM keep the loads going (two or
  // four chunks ahead in fewer CTAs were slower: 16.7 and 24.9 against 15.8 us for 27M bf16 gradients).
  const int64_t per = (tab.n_chunks + gridDim.x - 1) / gridDim.x, c0 = blockIdx.x * per, c1 = min(tab.n_chunks, c0 + per);
  for (int64_t c = c0; c < c1; ++c) {
    const int2 tc = tab.chunks[c];
    const G *g = static_cast<const G *>(tab.tensors[tc.x].grad);
    const int64_t n = tab.tensors[tc.x].n, e = static_cast<int64_t>(tc.y) * kOptChunk + threadIdx.x * 8;
    if ((reinterpret_cast<uintptr_t>(g) & 15) == 0 && e + 8 <= n) {
      float x[8];
      load_grads8(g + e, x);
      double t = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), t);
      s += t;
    } else {
      for (int i = 0; i < 8; ++i)
        if (e + i < n) {
          const double x = static_cast<double>(static_cast<float>(g[e + i]));
          s = fma(x, x, s);
        }
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
  __syncthreads();  // red is read by thread 0 until here
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
// AdamW.  The arithmetic is adamw_one's, float32 operation by operation (with 8-bit
// states but for the update's root and quotient).  8-bit states: a warp holds one
// block of 256 elements, eight consecutive ones per lane; the block's new maxima come from warp shuffles, the codes from adding
// random bits below the last mantissa bit kept and cutting them off.  The result is
// unbiased, which round-to-nearest is not where it matters: a step changes the
// variance by 1 - beta2 of itself, far less than half an E5M2 step, and a rounded
// variance would never move.
// ---------------------------------------------------------------------------
struct AdamWMulti {
  float beta1, beta2, eps, sqrt_bc2, inv_sqrt_bc2;
  double lr, weight_decay, step_size;  // step_size = lr / bc1
  const float *clip;                   // nullable [2]
  uint32_t seed;
  int per;  // chunks a CTA
};

// 32 bits for an element: multiplications by the first fraction bits of the golden
// ratio and of the square roots of 2 and 3, with the high half folded down between them.
__device__ __forceinline__ uint32_t state_hash(uint32_t element, uint32_t stream) {
  uint32_t x = (element + stream) * 0x9E3779B9u;
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// x >= 0 to the code of a float8 value at or next to it, up with the probability of rnd's kDrop bits: added below the last
// mantissa bit kept, they carry into it, and the shift cuts the rest off.  Below the format's least normal value kLeast
// the step is that of the first binade: adding kLeast puts x there, kBinade codes up.  kBias: the float32 code of the
// format's exponent 0, shifted alike.
template <int kDrop>
__device__ __forceinline__ uint32_t round_float8(float x, uint32_t rnd, float least, uint32_t bias, uint32_t binade, uint32_t most) {
  const bool small = x < least;
  const float z = __fadd_rn(x, small ? least : 0.0f);
  return min((__float_as_uint(z) + rnd - (bias << kDrop) - (small ? binade << kDrop : 0u)) >> kDrop, most);
}
__device__ __forceinline__ uint32_t round_e4m3(float x, uint32_t rnd) { return round_float8<20>(x, rnd, 0x1p-6f, 120u << 3, 8u, 126u); }
__device__ __forceinline__ uint32_t round_e5m2(float x, uint32_t rnd) { return round_float8<21>(x, rnd, 0x1p-14f, 112u << 2, 4u, 123u); }

// The larger one; a NaN stays.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// The warp's largest magnitude; a NaN stays.
__device__ __forceinline__ float warp_max_abs(float x) {
  float r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight elements of one lane.  WIDE: whole and at addresses for wide accesses; else element by element, those below n.
template <bool WIDE>
__device__ __forceinline__ void load_f32x8(const float *p, int valid, float (&x)[8]) {
  if (WIDE) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < valid ? p[i] : 0.0f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_f32x8(float *p, int valid, const float (&x)[8]) {
  if (WIDE) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = x[i];
  }
}
template <bool WIDE>
__device__ __forceinline__ uint2 load_codes8(const uint8_t *p, int valid) {
  if (WIDE) return __ldcs(reinterpret_cast<const uint2 *>(p));
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
template <bool WIDE>
__device__ __forceinline__ void store_codes8(uint8_t *p, int valid, const uint32_t (&w)[2]) {
  if (WIDE) {
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

template <typename G, bool EIGHT, bool WIDE>
__device__ __forceinline__ void adamw_block(const qlora_tensor &t, const AdamWMulti &a, int place, int64_t blk, int lane, float clip,
                                            float decay, float step_size) {
  const int64_t e0 = blk * QLORA_STATE_BLOCK + 8 * lane;
  const int valid = WIDE ? 8 : static_cast<int>(max(int64_t(0), min(int64_t(8), t.n - e0)));
  float p[8], g[8], m[8], v[8];
  load_f32x8<WIDE>(t.param + e0, valid, p);
  const G *grad = static_cast<const G *>(t.grad) + e0;
  if (WIDE) {
    load_grads8(grad, g);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = i < valid ? static_cast<float>(grad[i]) : 0.0f;
  }
  uint2 cm, cv;
  float sm = 0.0f, sv = 0.0f;
  if (EIGHT) {
    cm = load_codes8<WIDE>(static_cast<const uint8_t *>(t.exp_avg) + e0, valid);
    cv = load_codes8<WIDE>(static_cast<const uint8_t *>(t.exp_avg_sq) + e0, valid);
    sm = t.exp_avg_scale[blk];
    sv = t.exp_avg_sq_scale[blk];
  } else {
    load_f32x8<WIDE>(static_cast<const float *>(t.exp_avg) + e0, valid, m);
    load_f32x8<WIDE>(static_cast<const float *>(t.exp_avg_sq) + e0, valid, v);
  }
  const float omb1 = 1.0f - a.beta1, omb2 = 1.0f - a.beta2;
  float mm = 0.0f, vm = 0.0f;
  if (EIGHT) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 x = scale_code_value2((i < 4 ? cm.x : cm.y) >> (8 * (i & 2)), QLORA_SCALE_E4M3);
      const float2 y = scale_code_value2((i < 4 ? cv.x : cv.y) >> (8 * (i & 2)), QLORA_SCALE_E5M2);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float gi = __fmul_rn(g[i + k], clip);
        m[i + k] = __fadd_rn(__fmul_rn(a.beta1, __fmul_rn(k ? x.y : x.x, sm)), __fmul_rn(omb1, gi));
        v[i + k] = __fadd_rn(__fmul_rn(a.beta2, __fmul_rn(k ? y.y : y.x, sv)), __fmul_rn(omb2, __fmul_rn(gi, gi)));
      }
      // The states were read to 2^-4 and 2^-3, so the update needs no last bit: approximate root and reciprocal (a few
      // 2^-23 of the update) in place of IEEE ones, which made this path issue-bound (112
      // instructions a parameter, 243 us for 54M).  The states' own chain stays in single roundings.
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float denom = fmaf(sqrt_approx(v[i + k]), a.inv_sqrt_bc2, a.eps);
        p[i + k] = fmaf(p[i + k], decay, -__fmul_rn(__fmul_rn(step_size, m[i + k]), rcp_approx(denom)));
      }
      mm = max_nan(mm, max_nan(fabsf(m[i]), fabsf(m[i + 1])));
      vm = max_nan(vm, max_nan(v[i], v[i + 1]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gi = __fmul_rn(g[i], clip);
      m[i] = __fadd_rn(__fmul_rn(a.beta1, m[i]), __fmul_rn(omb1, gi));
      v[i] = __fadd_rn(__fmul_rn(a.beta2, v[i]), __fmul_rn(omb2, __fmul_rn(gi, gi)));
      const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(v[i]), a.sqrt_bc2), a.eps);
      p[i] = __fsub_rn(__fmul_rn(p[i], decay), __fdiv_rn(__fmul_rn(step_size, m[i]), denom));
    }
  }
  store_f32x8<WIDE>(t.param + e0, valid, p);
  if (t.param_bf16) {
    __nv_bfloat16 *p16 = static_cast<__nv_bfloat16 *>(t.param_bf16) + e0;
    if (WIDE) {
      __stcs(reinterpret_cast<uint4 *>(p16), make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                                                        pack_bf16x2(p[6], p[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) p16[i] = __float2bfloat16_rn(p[i]);
    }
  }
  if (!EIGHT) {
    store_f32x8<WIDE>(static_cast<float *>(t.exp_avg) + e0, valid, m);
    store_f32x8<WIDE>(static_cast<float *>(t.exp_avg_sq) + e0, valid, v);
    return;
  }
  mm = warp_max_abs(mm);
  vm = warp_max_abs(vm);
  // Factors for the codes (lanes 0 and 1), the largest code times the maximum's reciprocal, and scales (lanes 2 and 3) in
  // one division.  A maximum below 2^-100 is a block of zeros: its reciprocal would overflow.
  const bool of_v = lane & 1, scale = lane & 2;
  const float top = of_v ? vm : mm, most = of_v ? 57344.0f : 448.0f;
  float quot = top < 0x1p-100f ? 0.0f : __fdiv_rn(scale ? top : 1.0f, scale ? most : top);
  if (!scale) quot = __fmul_rn(most, quot);
  if (lane == 2) t.exp_avg_scale[blk] = quot;
  if (lane == 3) t.exp_avg_sq_scale[blk] = quot;
  const float im = __shfl_sync(0xffffffffu, quot, 0), iv = __shfl_sync(0xffffffffu, quot, 1);
  const uint32_t stream = a.seed * 0xB7E15163u + static_cast<uint32_t>(place) * 0x3504F333u;
  uint32_t wm[2] = {0u, 0u}, wv[2] = {0u, 0u};
  const uint32_t least_v = iv > 0.0f ? 1u : 0u;  // a variance that is not zero keeps a code above zero
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t h = state_hash(static_cast<uint32_t>(e0) + i + k, stream);
      const uint32_t qm = round_e4m3(__fmul_rn(fabsf(m[i + k]), im), h & 0xFFFFFu);
      const uint32_t qv = round_e5m2(__fmul_rn(v[i + k], iv), h >> 11);
      wm[i >> 2] |= (qm | (__float_as_uint(m[i + k]) >> 24 & 0x80u)) << (8 * ((i + k) & 3));
      wv[i >> 2] |= (v[i + k] > 0.0f ? max(qv, least_v) : qv) << (8 * ((i + k) & 3));
    }
  }
  store_codes8<WIDE>(static_cast<uint8_t *>(t.exp_avg) + e0, valid, wm);
  store_codes8<WIDE>(static_cast<uint8_t *>(t.exp_avg_sq) + e0, valid, wv);
}

template <typename G, bool EIGHT>
__global__ void __launch_bounds__(kOptThreads, EIGHT ? 4 : 3) adamw_multi_kernel(const TensorTable tab, const AdamWMulti a) {
  const float clip = a.clip ? a.clip[1] : 1.0f;
  if (clip != clip) return;  // the norm was not finite: the step changes nothing
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a CTA's chunks are neighbours, mostly of one tensor, whose entry is read once; the next chunk's place is read ahead
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.per, c1 = min(tab.n_chunks, c0 + a.per);
  int2 next = tab.chunks[c0];
  int at = -1;
  __shared__ qlora_tensor t;  // not in registers: they are what bounds the warps on an SM
  float decay = 0.0f, step_size = 0.0f;
  bool wide = false;
  for (int64_t c = c0; c < c1; ++c) {
    const int2 tc = next;
    if (c + 1 < c1) next = tab.chunks[c + 1];
    if (tc.x != at) {
      at = tc.x;
      __syncthreads();  // the last entry is done with
      if (threadIdx.x == 0) t = tab.tensors[at];
      __syncthreads();
      const double lr_scale = static_cast<double>(t.lr_scale);
      decay = static_cast<float>(1.0 - a.lr * lr_scale * a.weight_decay);
      step_size = static_cast<float>(a.step_size * lr_scale);
      // wide accesses where all addresses allow them (16 bytes; codes 8), and the block is whole
      const uintptr_t any = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.param_bf16) |
                            reinterpret_cast<uintptr_t>(t.grad) |
                            (reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq)) * (EIGHT ? 2 : 1);
      wide = (any & 15) == 0;
    }
    const int64_t blk = static_cast<int64_t>(tc.y) * (kOptThreads / 32) + warp, e0 = blk * QLORA_STATE_BLOCK;
    if (e0 >= t.n) continue;
    if (wide && e0 + QLORA_STATE_BLOCK <= t.n)
      adamw_block<G, EIGHT, true>(t, a, at, blk, lane, clip, decay, step_size);
    else
      adamw_block<G, EIGHT, false>(t, a, at, blk, lane, clip, decay, step_size);
  }
}

}  // namespace qlora
