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
// The products.  Two kernels, on the tensor cores (tcgen05, accumulators in TMEM) with
// ranks, or features, in the 128 rows of the accumulator and tokens, or ranks, in its
// columns:
//
//   term  P = V W1_a over the long dimension, then Out += s_a P W2_a: T and Y in the
//         forward, U and dX in the backward
//   grad  s_a P^T V over the tokens of an adapter: dA, dB
//
// A tile holds tokens of one adapter, wherever their rows lie: runs of 32 rows come
// with one tiled load, others four rows to a gather, and a short tile loads only the
// rows it has.  Columns of the accumulator are independent, so a short tile's unused
// columns need no zeros, and neither do rows past an adapter's rank.  How the tiles
// fall follows from offsets, which only the device knows: each CTA adds up the
// adapters' tile counts first and walks the tiles from there.
//
// Both are bound by HBM at ranks up to about 128 (r flops a byte of X, dY, Y or dX).
// ---------------------------------------------------------------------------
// The intermediates T = X A^T and U = dY B are [M, r] in float32 and kept as three bf16 planes [3, M, r], each the rounding
// of what the ones before leave: 24 bits together, in the type the tensor cores take beside bf16 operands.  A bf16 result
// is computed from the first two (16 bits), a float32 one from all.
constexpr int kPoolPlanes = 3;

struct PoolArgs {
  const int32_t *ranks;  // nullable
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

// Places [lo, hi) of adapter a's tokens in order.
__device__ __forceinline__ int2 pool_group(const PoolArgs &p, int a) {
  const int m = static_cast<int>(p.M);
  const int lo = min(max(p.offsets[a], 0), m);
  return make_int2(lo, min(max(p.offsets[a + 1], lo), m));
}

// Token at place i (below M); -1 if it is out of range.
__device__ __forceinline__ int pool_token(const PoolArgs &p, int i) {
  const int t = __ldg(p.order + i);
  if (t >= 0 && t < p.M) return t;
  raise_status(p.status, QLORA_ERR_INVALID_ARGUMENT);
  return -1;
}

// The same for a load of four rows, which needs some row in range: row 0 then, whose result is not written.
__device__ __forceinline__ int4 pool_rows(const PoolArgs &p, int i, int last) {
  int4 y;
  y.x = max(pool_token(p, min(i, last)), 0);
  y.y = max(pool_token(p, min(i + 1, last)), 0);
  y.z = max(pool_token(p, min(i + 2, last)), 0);
  y.w = max(pool_token(p, min(i + 3, last)), 0);
  return y;
}

// Loads of token rows into a stage: 32 consecutive rows of memory come with one tiled load (box 64 x 32), other rows
// four to a gather.  A gather costs the loading thread as much as a tiled load eight times its size (reading 67 MB by
// gathers alone took 46 us), and requests of a packed batch are runs of rows.
//
// Whether the eight lanes from lane & ~7, with four rows each, hold 32 consecutive rows.  valid: rows of the tile; those
// past it may be any rows where `loose` (at least half of the 32 must be wanted).
__device__ __forceinline__ bool pool_run32(const int4 &y, int lane, int first, int valid, bool loose) {
  const int base = __shfl_sync(0xffffffffu, y.x, lane & ~7) + 4 * (lane & 7), left = valid - first;
  const bool seq = (y.x == base || left < 1) && (y.y == base + 1 || left < 2) && (y.z == base + 2 || left < 3) &&
                   (y.w == base + 3 || left < 4);
  const uint32_t all = __ballot_sync(0xffffffffu, seq);
  const int wanted = valid - (first - 4 * (lane & 7));
  return ((all >> (lane & ~7)) & 0xffu) == 0xffu && wanted >= (loose ? 16 : 32);
}

// Position in a ring of stages, with the phase of its barriers.
struct RingPos {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++s == stages) { s = 0; ph ^= 1; }
  }
};

// The last (up to) `stages` stages filled have landed: nothing may be in flight when the CTA's memory goes.
__device__ __forceinline__ void ring_drain(uint64_t *full, RingPos pos, uint32_t stages, uint32_t issued) {
  for (uint32_t i = 0; i < stages && i < issued; ++i) {
    if (pos.s == 0) { pos.s = stages - 1; pos.ph ^= 1; } else { --pos.s; }
    ptx::mbar_wait(&full[pos.s], pos.ph, nullptr);
  }
}

// Barriers and flags of a CTA, behind its buffers.
constexpr uint32_t kPoolMostStages = 12, kPoolBars = 2 * kPoolMostStages + 9, kPoolTailBytes = 512;
struct PoolSmem {
  uint8_t *buf;   // 1024-byte aligned, `bytes` of it
  uint64_t *bars;
  uint32_t *tmem_slot;
  volatile int *abort_flag;
};
__device__ __forceinline__ PoolSmem pool_smem(uint8_t *raw, uint32_t bytes) {
  PoolSmem s;
  s.buf = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.bars = reinterpret_cast<uint64_t *>(s.buf + bytes);
  s.tmem_slot = reinterpret_cast<uint32_t *>(s.bars + kPoolBars);
  s.abort_flag = reinterpret_cast<volatile int *>(s.tmem_slot + 1);
  return s;
}
__host__ __device__ constexpr uint32_t pool_smem_bytes(uint32_t bytes) { return 1024 + bytes + kPoolTailBytes; }

// Set-up of both kernels: barriers (one arrival each; four, one of each warp of a set, from place `four` on), TMEM, then
// the wait for the kernel ahead.  The next kernel may start only after that wait: one that reads early, or that waits for
// this kernel alone, then finds everything before this kernel complete too.
__device__ __forceinline__ uint32_t pool_setup(const PoolSmem &s, uint32_t tmem_cols, uint32_t four) {
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kPoolBars; ++i) ptx::mbar_init(&s.bars[i], i < four ? 1 : 4);
    *s.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x >> 5 == 1) {
    ptx::tmem_alloc(s.tmem_slot, tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::griddep_wait();
  ptx::griddep_launch();
  return *s.tmem_slot;
}

__device__ __forceinline__ void pool_teardown(uint32_t tmem, uint32_t tmem_cols) {
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x >> 5 == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, tmem_cols);
  }
}

// All threads of the cluster; a warp may have split before it.
__device__ __forceinline__ void pool_cluster_sync() {
  __syncwarp();
  ptx::cluster_sync();
}

__device__ __forceinline__ void pool_fail(const PoolSmem &s, uint32_t *status) {
  raise_status(status, QLORA_ERR_TIMEOUT);
  *s.abort_flag = 1;
}

// ---------------------------------------------------------------------------
// term: g CTAs of a cluster take a tile of 64 tokens (32 above rank 128); g, at most the cluster, follows on the device from
// the number of tiles.
//
// 1. Its CTAs each sum a part of the long dimension, with the accumulator's rows as ranks and its columns as
//    tokens; the steps of 64 go round four accumulators, which keeps each one's chain of float32 additions
//    short (the tensor cores' additions cut off: one chain over 1400 elements was 3e-6 off, all to one side).
// 2. Each CTA leaves its float32 partial sums in shared memory; each then adds up a share of the tokens over
//    the g CTAs, in CTA order, splits the sums into planes, and writes them into the shared memory of
//    every CTA of the tile (and to HBM, where the backward needs them).  No partial planes in HBM, no
//    second launch, and the same bits every time.
// 3. Each CTA takes every g-th block of 128 features: W2's block by TMA, rows of the accumulator as
//    features, then Out += s accumulator.  Two sets of four epilogue warps take turns, each with two of four
//    accumulators: while one is stored, the next is multiplied.
//    The lanes hold features; where Out's rows are 16-byte aligned, 16 tokens at a time pass through
//    shared memory, so that four lanes (bf16; eight for float32) then share a token's 32 features in
//    16-byte pieces, loaded before the accumulator is waited for (element by element the epilogue took 47
//    instructions an element and warp, and bound the kernel on issue).  Other outputs, odd strides or
//    columns of a wider tensor, go element by element.
//
//   warp 0  loads; warp 1  products; warps 2..9  accumulators -> shared memory, epilogue; all  the sums
// W_MN false (forward): W1 = A [n][r][len], W2 = B [n][cols][r], both K-major; true (backward): W1 = B
// [n][len][r], W2 = A [n][r][cols], both MN-major.
// ---------------------------------------------------------------------------
constexpr int kPoolTermThreads = 320;
constexpr uint32_t kPoolTermTmem = 256;
constexpr uint32_t kPoolTermMostBytes = 218 * 1024;
// Shared memory of a warp's 16 tokens x 32 features: a pitch of 36 floats keeps 16-byte pieces aligned and both
// directions without bank conflicts.
constexpr int kPoolPitch = 36, kPoolWarpBuf = 16 * kPoolPitch;

// Sizes that follow from the rank and the planes.  Two CTAs share an SM up to rank 64, unless the call is `roomy`: too
// small to give every SM one, so that a deeper ring is worth more. 
struct PoolTermLayout {
  int tn;               // tokens a tile
  int rpad;             // floats a token of the partial sums
  uint32_t stage;       // bytes
  uint32_t stages;
  uint32_t plane;       // bytes of one 64-rank chunk of one plane
  uint32_t planes_at, exch_at, bytes;
};
__host__ __device__ constexpr PoolTermLayout pool_term_layout(int r, int planes, bool roomy) {
  PoolTermLayout l{};
  l.tn = r <= 128 ? 64 : 32;
  l.rpad = r <= 64 ? 64 : r <= 128 ? 128 : 256;
  l.stage = l.tn * 128u + l.rpad * 128u;  // token rows and W1's
  if (l.stage < 16384u) l.stage = 16384u;  // a block of W2
  l.plane = l.tn * 128u;
  const uint32_t budget = r <= 64 && !roomy ? 107u * 1024u : kPoolTermMostBytes, p_bytes = (r + 63) / 64 * planes * l.plane;
  const uint32_t exch = l.tn * l.rpad * 4u > 8 * kPoolWarpBuf * 4u ? l.tn * l.rpad * 4u : 8 * kPoolWarpBuf * 4u;
  const uint32_t fit = (budget - p_bytes - exch) / l.stage;
  l.stages = fit < kPoolMostStages ? fit : kPoolMostStages;
  l.planes_at = l.stages * l.stage;
  l.exch_at = l.planes_at + p_bytes;
  l.bytes = l.exch_at + exch;
  return l;
}
static_assert(pool_term_layout(64, 3, false).stages >= 3 && pool_term_layout(128, 3, false).stages >= 3 &&
                  pool_term_layout(256, 3, false).stages >= 3,
              "a ring of three stages at least");
static_assert(pool_smem_bytes(pool_term_layout(64, 3, false).bytes) + 2048 <= 114 * 1024 &&
                  pool_smem_bytes(pool_term_layout(256, 3, false).bytes) <= 225 * 1024,
              "shared memory");

struct PoolTermArgs {
  PoolArgs p;
  int64_t len;         // columns of V
  int64_t cols, ldo;   // of Out
  void *out;           // nullable: P alone
  __nv_bfloat16 *P;    // nullable [3, M, r]
  int planes;          // used for Out
  PoolTermLayout l;
};

__device__ __forceinline__ float pool_load(const float *p) { return __ldcg(p); }
__device__ __forceinline__ float pool_load(const __nv_bfloat16 *p) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(p))) << 16);
}
__device__ __forceinline__ void pool_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void pool_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes of Out: y + s v, rounded once.  kElems elements; a row's 32 features take 32 / kElems lanes, so that each
// instruction covers whole sectors.  kTokens: one item of a warp, 2 KB; two are in flight.
template <typename O>
struct PoolPiece;
template <>
struct PoolPiece<float> {
  static constexpr int kElems = 4, kTokens = 16;
  float4 y;
  __device__ __forceinline__ void load(const float *p) { y = __ldcg(reinterpret_cast<const float4 *>(p)); }
  __device__ __forceinline__ void add(float s, const float *v) {
    const float4 u = *reinterpret_cast<const float4 *>(v);
    y = make_float4(fmaf(s, u.x, y.x), fmaf(s, u.y, y.y), fmaf(s, u.z, y.z), fmaf(s, u.w, y.w));
  }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = y; }
};
template <>
struct PoolPiece<__nv_bfloat16> {
  static constexpr int kElems = 8, kTokens = 32;
  uint4 y;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { y = __ldcg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void add(float s, const float *v) {
    const float4 u = reinterpret_cast<const float4 *>(v)[0], w = reinterpret_cast<const float4 *>(v)[1];
    y.x = pack_bf16x2(fmaf(s, u.x, bf16lo_to_f32(y.x)), fmaf(s, u.y, bf16hi_to_f32(y.x)));
    y.y = pack_bf16x2(fmaf(s, u.z, bf16lo_to_f32(y.y)), fmaf(s, u.w, bf16hi_to_f32(y.y)));
    y.z = pack_bf16x2(fmaf(s, w.x, bf16lo_to_f32(y.z)), fmaf(s, w.y, bf16hi_to_f32(y.z)));
    y.w = pack_bf16x2(fmaf(s, w.z, bf16lo_to_f32(y.w)), fmaf(s, w.w, bf16hi_to_f32(y.w)));
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = y; }
};

// The tile at hand.
struct PoolTile {
  int ad, lo, cnt, rank;
  float scale;
};

template <bool W_MN, typename O, bool VEC>
__global__ void __launch_bounds__(kPoolTermThreads, 2)
    pool_term_kernel(const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmW2,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmVt, const PoolTermArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int64_t row_at[64];  // of the tile's tokens in Out, in elements; -1: not a token
  __shared__ int4 row4[16];
  __shared__ int warp_sum[kPoolTermThreads / 32];
  __shared__ PoolTile tile_s;
  // descriptor words (128-byte swizzle, groups of eight rows 1024 bytes apart): the high one is the same for all operands,
  // the low one is the address and the distance of 64-element blocks, which MN-major operands use (8192 bytes); 16
  // elements on, a K-major operand is 32 bytes away and an MN-major one 2048
  constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
  constexpr uint32_t kWLbo = W_MN ? ((8192u >> 4) - (16u >> 4)) << 16 : 0u, kW16 = W_MN ? 128u : 2u;
  const PoolArgs &p = a.p;
  const PoolTermLayout &l = a.l;
  const PoolSmem sm = pool_smem(pool_raw, l.bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tn = l.tn;
  const uint32_t stages = l.stages, v_bytes = tn * 128u;
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *sum_full = sm.bars + 2 * kPoolMostStages;
  uint64_t *acc_full = sum_full + 1, *acc_empty = acc_full + 4;
  float *exch = reinterpret_cast<float *>(sm.buf + l.exch_at);
  uint8_t *planes = sm.buf + l.planes_at;
  if (tid < 4) ptx::prefetch_tmap(tid == 0 ? &tmW1 : tid == 1 ? &tmW2 : tid == 2 ? &tmV : &tmVt);
  const uint32_t tmem = pool_setup(sm, kPoolTermTmem, 2 * kPoolMostStages + 5);

  // this thread's adapters, ad0 .. ad0 + per: what is known of the first stays in registers
  const int per = (p.n + kPoolTermThreads - 1) / kPoolTermThreads, ad0 = tid * per;
  int2 group0 = make_int2(0, 0);
  int sum = 0, rank0 = 0;
  float scale0 = 0.0f;
  if (ad0 < p.n) {
    group0 = pool_group(p, ad0);
    rank0 = pool_rank(p, ad0);
    scale0 = p.scales[ad0];
    sum = (group0.y - group0.x + tn - 1) / tn;
    for (int i = 1; i < per && ad0 + i < p.n; ++i) {
      const int2 grp = pool_group(p, ad0 + i);
      sum += (grp.y - grp.x + tn - 1) / tn;
    }
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int before = inc - sum, tiles = 0;
#pragma unroll
  for (int w = 0; w < kPoolTermThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    tiles += warp_sum[w];
  }

  // a tile is shared by g CTAs of the cluster: the largest divisor with which all tiles are at work at once
  const int cluster = static_cast<int>(ptx::cluster_nctarank()), crank = static_cast<int>(ptx::cluster_ctarank());
  int g = cluster;
  while (g > 1 && (static_cast<int64_t>(tiles) * g > gridDim.x || cluster % g)) --g;
  const int q = crank % g, peers = crank - q;  // the g CTAs from rank `peers` of the cluster
  const int k_steps = static_cast<int>((a.len + 63) / 64), k_per = (k_steps + g - 1) / g;
  const int nblk = a.out ? static_cast<int>((a.cols + 127) / 128) : 0;
  const int nrb = (p.r + 127) / 128, acc_cols = tn * nrb;  // one of the four accumulators of the sums
  RingPos pos;
  uint32_t sum_phase = 0, issued = 0, blocks = 0;  // blocks: accumulators of features used so far
  bool ok = true;
  // all CTAs of a cluster walk as long as the first of its tiles exists
  for (int lead = (blockIdx.x - crank) / g; lead < tiles; lead += gridDim.x / g) {
    const int tile = lead + crank / g;
    if (tile >= tiles && tid == 0) {
      tile_s.ad = tile_s.lo = tile_s.cnt = tile_s.rank = 0;
      tile_s.scale = 0.0f;
    }
    if (tile >= before && tile < before + sum) {  // among this thread's
      int2 grp = group0;
      int ad = ad0, t = tile - before, nt;
      while (t >= (nt = (grp.y - grp.x + tn - 1) / tn)) {
        t -= nt;
        grp = pool_group(p, ++ad);
      }
      tile_s.ad = ad;
      tile_s.lo = grp.x + t * tn;
      tile_s.cnt = min(tn, grp.y - tile_s.lo);
      tile_s.rank = ad > ad0 ? pool_rank(p, ad) : rank0;
      tile_s.scale = ad > ad0 ? p.scales[ad] : scale0;
    }
    __syncthreads();
    const int ad = tile_s.ad, lo = tile_s.lo, cnt = tile_s.cnt, rank = tile_s.rank;
    const int kb = rank > 0 ? min(q * k_per, k_steps) : 0, ke = rank > 0 ? min(k_steps, kb + k_per) : 0;
    const int nch = rank > 0 ? (rank + 63) / 64 : 0;
    const int mine = rank > 0 && nblk > q ? (nblk - q + g - 1) / g : 0;  // blocks q, q + g, ...
    const uint32_t idesc = ptx::idesc_bf16(128, (cnt + 15) / 16 * 16, W_MN ? 1 : 0, 0);
    const int quad = warp & 3, set = (warp - 2) >> 2;

    // epilogue: a warp's items are (block, group of tokens), the blocks being those whose accumulator is its set's
    constexpr int kGroup = PoolPiece<O>::kTokens, kElems = PoolPiece<O>::kElems, kLanes = 32 / kElems, kRows = 32 / kLanes;
    constexpr int kPieces = kGroup / kRows;
    const int tr = lane / kLanes, part = lane % kLanes;
    const int b_first = (set ^ blocks) & 1;
    const bool few = cnt <= 4;  // a column of the accumulator is then a token's feature of each lane, straight to Out
    const bool pieces = VEC && !few && warp >= 2;
    PoolPiece<O> y0[kPieces], y1[kPieces];
    // an item's loads: rows that are not tokens, and columns past the last, load something that is and are not stored
    auto load_y = [&](PoolPiece<O>(&y)[kPieces], int b, int g0) {
      const int64_t f = static_cast<int64_t>(q + b * g) * 128 + quad * 32 + part * kElems;
      const O *out = static_cast<const O *>(a.out) + (f < a.cols ? f : 0);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int64_t at = row_at[min(g0 + kRows * i + tr, cnt - 1)];
        y[i].load(out + (at < 0 ? 0 : at));
      }
    };

    // the lines of this warp's features in a whole block, towards L2: a block ahead of the loads (16 KB an item's warp)
    auto prefetch_block = [&](int b) {
      const int64_t f = static_cast<int64_t>(q + b * g) * 128 + quad * 32;
      if (f >= a.cols || (sizeof(O) == 2 && (quad & 1))) return;  // two warps' bf16 features share a line
      for (int c = lane; c < cnt; c += 32) {
        const int64_t at = row_at[c];
        if (at >= 0) ptx::prefetch_line_l2(static_cast<const O *>(a.out) + f + at);
      }
    };

    // warp 0's thread: stages [i0, i1) of W2's blocks, 64 ranks of a block each
    auto load_w2 = [&](int i0, int i1) {
      int b = i0 / max(nch, 1), ch = i0 - b * nch;
      for (int i = i0; i < i1; ++i) {
        if (!ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag)) { ok = false; break; }
        const int f = (q + b * g) * 128, x = ch * 64;
        uint8_t *st = sm.buf + pos.s * l.stage;
        ptx::mbar_arrive_expect_tx(&full[pos.s], 16384u);
        if (W_MN) {
          ptx::tma_load_3d(st, &tmW2, &full[pos.s], f, x, ad);
          ptx::tma_load_3d(st + 8192, &tmW2, &full[pos.s], f + 64, x, ad);
        } else {
          ptx::tma_load_3d(st, &tmW2, &full[pos.s], x, f, ad);
        }
        if (++ch == nch) { ch = 0; ++b; }
        ++issued;
        pos.next(stages);
      }
    };

    // ------------------------------------------------------------ 1. the sums over the long dimension
    if (warp == 0) {
      const int4 rows = cnt > 0 ? pool_rows(p, lo + 4 * min(lane, tn / 4 - 1), lo + cnt - 1) : make_int4(0, 0, 0, 0);
      const bool mine4 = 4 * lane < cnt;
      const bool run = pool_run32(rows, lane, 4 * lane, cnt, true);
      const uint32_t tile_loads = __ballot_sync(0xffffffffu, run && (lane & 7) == 0 && mine4);
      const uint32_t gathers = __ballot_sync(0xffffffffu, !run && mine4);
      if (lane < 16) row4[lane] = rows;
      __syncwarp();
      if (ok && ptx::elect_one()) {
        // W1's ranks [0, min(r, 256)): K-major in boxes of up to 128 rows, MN-major in boxes of 64 ranks
        const int w_loads = W_MN ? (p.r + 63) / 64 : nrb;
        const uint32_t w_box = W_MN ? 8192u : static_cast<uint32_t>(min(p.r, 128)) * 128u;
        const uint32_t bytes = w_loads * w_box + __popc(tile_loads) * 4096u + __popc(gathers) * 512u;
        for (int ks = kb; ks < ke; ++ks) {
          if (!ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag)) { ok = false; break; }
          uint8_t *st = sm.buf + pos.s * l.stage;
          uint64_t *bar = &full[pos.s];
          ptx::mbar_arrive_expect_tx(bar, bytes);
          for (int i = 0; i < w_loads; ++i)
            ptx::tma_load_3d(st + v_bytes + i * (W_MN ? 8192 : 16384), &tmW1, bar, W_MN ? i * 64 : ks * 64, W_MN ? ks * 64 : i * 128,
                             ad);
          for (uint32_t m = tile_loads; m; m &= m - 1) {
            const int i = __ffs(m) - 1;
            ptx::tma_load_2d(st + i * 512, &tmVt, bar, ks * 64, row4[i].x);
          }
          for (uint32_t m = gathers; m; m &= m - 1) {
            const int i = __ffs(m) - 1;
            ptx::tma_gather4(st + i * 512, &tmV, bar, ks * 64, row4[i]);
          }
          ++issued;
          pos.next(stages);
        }
        // the first of W2's blocks follow through the ring while the sums are joined
        if (ok) load_w2(0, min(mine * nch, static_cast<int>(stages)));
        if (!ok) pool_fail(sm, p.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      if (ok && ptx::elect_one()) {
        const uint32_t v_lo = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024));
        for (int ks = kb; ks < ke; ++ks) {
          if (!ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t v = v_lo + pos.s * (l.stage >> 4), w = v + (v_bytes >> 4) + kWLbo, d = tmem + ((ks - kb) & 3) * acc_cols;
          const uint32_t more = ks - kb >= 4 ? 1u : 0u;
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            ptx::mma_bf16_lohi(d, w + k16 * kW16, kDescHi, v + k16 * 2, kDescHi, idesc, k16 ? 1u : more);
          if (nrb > 1) {  // ranks 128 and up
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16)
              ptx::mma_bf16_lohi(d + tn, w + 1024 + k16 * kW16, kDescHi, v + k16 * 2, kDescHi, idesc, k16 ? 1u : more);
          }
          ptx::mma_commit(&empty[pos.s]);
          pos.next(stages);
        }
        if (ok && ke > kb) ptx::mma_commit(sum_full);
        if (!ok) pool_fail(sm, p.status);
      }
      __syncwarp();
    } else {
      if (tid - 64 < tn) {
        const int t = tid - 64 < cnt ? pool_token(p, lo + tid - 64) : -1;
        row_at[tid - 64] = t < 0 ? -1 : t * a.ldo;
      }
      ptx::named_bar_sync(1, kPoolTermThreads - 64);
      if (pieces && b_first < mine) {  // the first ones', while the sums are formed
        load_y(y0, b_first, 0);
        prefetch_block(b_first);
      }
      if (ke > kb && ok) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(sum_full, sum_phase, sm.abort_flag));
        sum_phase ^= 1;
        if (!ok && lane == 0) pool_fail(sm, p.status);
      }
      ptx::tc_fence_after();
      const int nacc = ok ? min(4, ke - kb) : 0, c_end = min(cnt, (set + 1) * (tn / 2));
      for (int rb = 0; rb < nrb; ++rb) {
        if (rb * 128 + quad * 32 >= p.r) break;
        for (int c0 = set * (tn / 2); c0 < c_end; c0 += 16) {
          const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + rb * tn + c0;
          float x[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            if (i >= nacc) break;
            uint32_t v[16], w[16];
            ptx::tmem_ld16(from + i * acc_cols, v);
            if (i + 1 < nacc) ptx::tmem_ld16(from + (i + 1) * acc_cols, w);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] += __uint_as_float(v[j]) + (i + 1 < nacc ? __uint_as_float(w[j]) : 0.0f);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c0 + j < c_end) exch[(c0 + j) * l.rpad + rb * 128 + quad * 32 + lane] = x[j];
        }
      }
      ptx::tc_fence_before();
    }

    // ------------------------------------------------------------ 2. the sums over the cluster
    pool_cluster_sync();
    {
      const int pt = (cnt + g - 1) / g, c_lo = min(cnt, q * pt), c_hi = min(cnt, c_lo + pt);
      const int n4 = (p.r + 15) / 16 * 4;  // groups of 4 ranks; products take 16 at a time
      const uint32_t exch_addr = ptx::smem_addr(exch), planes_addr = ptx::smem_addr(planes);
      for (int e = tid; e < (c_hi - c_lo) * n4; e += kPoolTermThreads) {
        const int c = c_lo + e / n4, j = e % n4 * 4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < rank) {
          const uint32_t src = exch_addr + (c * l.rpad + j) * 4;
#pragma unroll
          for (int r0 = 0; r0 < 8; r0 += 4) {
            if (r0 >= g) break;
            float4 u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (r0 + r < g) u[r] = ptx::ld_cluster_f32x4(ptx::mapa_shared(src, peers + r0 + r));
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (r0 + r < g) { x.x += u[r].x; x.y += u[r].y; x.z += u[r].z; x.w += u[r].w; }
          }
        }
        const int t = a.P ? pool_token(p, lo + c) : -1;
        const uint32_t dst = planes_addr + (j >> 6) * a.planes * l.plane + c * 128 + ((((j >> 3) & 7) ^ (c & 7)) << 4) + (j & 4) * 2;
#pragma unroll
        for (int pl = 0; pl < kPoolPlanes; ++pl) {
          const uint2 h = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
          x.x -= bf16lo_to_f32(h.x);
          x.y -= bf16hi_to_f32(h.x);
          x.z -= bf16lo_to_f32(h.y);
          x.w -= bf16hi_to_f32(h.y);
          if (t >= 0 && j < p.r) *reinterpret_cast<uint2 *>(a.P + (static_cast<int64_t>(pl) * p.M + t) * p.r + j) = h;
          if (a.out && pl < a.planes) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (r < g) ptx::st_cluster_u32x2(ptx::mapa_shared(dst + pl * l.plane, peers + r), h);
          }
        }
      }
    }
    ptx::fence_proxy_async_cluster();  // the planes are read by the tensor cores
    pool_cluster_sync();

    // ------------------------------------------------------------ 3. the features
    if (warp == 0) {
      if (ok && ptx::elect_one()) {
        load_w2(min(mine * nch, static_cast<int>(stages)), mine * nch);
        if (!ok) pool_fail(sm, p.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      ptx::fence_proxy_async_cluster();
      const uint32_t p_lo = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024));
      // one thread issues a chunk of a block's products
      auto issue = [&](uint32_t acc, int ch) {
        ptx::tc_fence_after();
        const int left = min(64, rank - ch * 64);  // a multiple of 8; products go 16 ranks at a time
        const uint32_t w = p_lo + pos.s * (l.stage >> 4) + kWLbo, pc = p_lo + ((l.planes_at + ch * a.planes * l.plane) >> 4);
#pragma unroll
        for (int k16 = 0; k16 < 4; ++k16) {
          if (k16 * 16 >= left) break;
#pragma unroll
          for (int pl = 0; pl < kPoolPlanes; ++pl)
            if (pl < a.planes)
              ptx::mma_bf16_lohi(tmem + acc * 64, w + k16 * kW16, kDescHi, pc + pl * (l.plane >> 4) + k16 * 2, kDescHi, idesc,
                                 (ch || k16 || pl) ? 1u : 0u);
        }
        ptx::mma_commit(&empty[pos.s]);
        if (ch == nch - 1) ptx::mma_commit(&acc_full[acc]);
      };
      const bool one = ptx::elect_one();
      if (!(rank & 8) || rank == p.r) {
        if (ok && one) {
          for (int b = 0; b < mine && ok; ++b) {
            const uint32_t n = blocks + b, acc = n & 3;
            ok = ptx::mbar_wait(&acc_empty[acc], ((n >> 2) & 1) ^ 1, sm.abort_flag);
            for (int ch = 0; ch < nch && ok; ++ch) {
              if (!(ok = ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag))) break;
              issue(acc, ch);
              pos.next(stages);
            }
          }
          if (!ok) pool_fail(sm, p.status);
        }
      } else {
        // The 8 ranks past the adapter's meet zeros in P and have to be finite: the warp clears them in each last chunk.
        const int leader = __ffs(__ballot_sync(0xffffffffu, one)) - 1;
        pos.s = __shfl_sync(0xffffffffu, pos.s, leader);
        pos.ph = __shfl_sync(0xffffffffu, pos.ph, leader);
        ok = __all_sync(0xffffffffu, ok);
        for (int b = 0; b < mine && ok; ++b) {
          const uint32_t n = blocks + b, acc = n & 3;
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_empty[acc], ((n >> 2) & 1) ^ 1, sm.abort_flag));
          for (int ch = 0; ch < nch && ok; ++ch) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
            if (!ok) break;
            if (ch == nch - 1) {
              uint8_t *st = sm.buf + pos.s * l.stage;
              const int at_rank = rank & 63;
#pragma unroll
              for (int i = lane; i < 128; i += 32) {
                const int at = W_MN ? (i >> 6) * 8192 + (at_rank + ((i >> 3) & 7)) * 128 + (i & 7) * 16
                                    : i * 128 + (((at_rank >> 3) ^ (i & 7)) << 4);
                *reinterpret_cast<uint4 *>(st + at) = make_uint4(0u, 0u, 0u, 0u);
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
            }
            if (one) issue(acc, ch);
            __syncwarp();
            pos.next(stages);
          }
        }
        if (!ok && lane == 0) pool_fail(sm, p.status);
      }
      __syncwarp();
    } else {
      const float s = tile_s.scale;
      uint32_t acc = 0, d = 0;
      auto wait = [&](int b) {
        const uint32_t n = blocks + b;
        acc = n & 3;
        d = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 64;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], (n >> 2) & 1, sm.abort_flag));
        ptx::tc_fence_after();
        return ok;
      };
      auto done = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&acc_empty[acc]);
      };
      if (few) {
        const int64_t f0 = static_cast<int64_t>(q) * 128 + quad * 32 + lane;
        float y[4], next[4];
        auto load_few = [&](float(&z)[4], int b) {
          const int64_t f = f0 + static_cast<int64_t>(b) * g * 128;
          const O *out = static_cast<const O *>(a.out) + (f < a.cols ? f : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t at = row_at[min(j, cnt - 1)];
            z[j] = pool_load(out + (at < 0 ? 0 : at));
          }
        };
        if (b_first < mine) load_few(y, b_first);
        for (int b = b_first; b < mine && ok; b += 2) {
          if (b + 2 < mine) load_few(next, b + 2);
          if (!wait(b)) break;
          uint32_t v[4];
          ptx::tmem_ld4(d, v);
          ptx::tmem_ld_wait();
          done();
          const int64_t f = f0 + static_cast<int64_t>(b) * g * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t at = j < cnt && f < a.cols ? row_at[j] : -1;
            if (at >= 0) pool_store(static_cast<O *>(a.out) + f + at, fmaf(s, __uint_as_float(v[j]), y[j]));
            y[j] = next[j];
          }
        }
      } else if (VEC) {
        float *buf = exch + (warp - 2) * kPoolWarpBuf;
        auto add_store = [&](PoolPiece<O>(&y)[kPieces], int b, int g0) {
          if (g0 == 0 && !wait(b)) return;
          const int64_t f = static_cast<int64_t>(q + b * g) * 128 + quad * 32 + part * kElems;
          O *out = static_cast<O *>(a.out) + f;
#pragma unroll
          for (int k = 0; k < kGroup / 16; ++k) {
            if (g0 + 16 * k >= cnt) break;
            uint32_t v[16];
            ptx::tmem_ld16(d + g0 + 16 * k, v);
            ptx::tmem_ld_wait();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) buf[j * kPoolPitch + lane] = __uint_as_float(v[j]);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 16 / kRows; ++h) {
              const int i = 16 / kRows * k + h, c = g0 + kRows * i + tr;
              y[i].add(s, buf + (kRows * h + tr) * kPoolPitch + part * kElems);
              const int64_t at = c < cnt && f < a.cols ? row_at[c] : -1;
              if (at >= 0) y[i].store(out + at);
            }
          }
          if (g0 + kGroup >= cnt) done();
        };
        // (block, group of tokens) after (block, group of tokens), the next one's loads ahead
        int b = b_first, g0 = 0;
        auto step = [&](PoolPiece<O>(&y)[kPieces], PoolPiece<O>(&next)[kPieces]) {
          int nb = b, ng = g0 + kGroup;
          if (ng >= cnt) { ng = 0; nb += 2; }
          if (nb < mine) load_y(next, nb, ng);
          if (g0 == 0 && b + 2 < mine) prefetch_block(b + 2);
          add_store(y, b, g0);
          b = nb;
          g0 = ng;
          return ok && b < mine;
        };
        if (b < mine && ok)
          while (step(y0, y1) && step(y1, y0)) {
          }
      } else {
        for (int b = b_first; b < mine && ok; b += 2) {
          const int64_t f0 = static_cast<int64_t>(q + b * g) * 128 + quad * 32;
          bool ready = false;
          const bool in = f0 + lane < a.cols;
          O *out = static_cast<O *>(a.out) + f0 + lane;
          for (int c0 = 0; c0 < cnt; c0 += 16) {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t at = c0 + j < cnt ? row_at[c0 + j] : -1;
              y[j] = at >= 0 && in ? pool_load(out + at) : 0.0f;
            }
            if (!ready && !wait(b)) break;
            ready = true;
            uint32_t v[16];
            ptx::tmem_ld16(d + c0, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t at = c0 + j < cnt ? row_at[c0 + j] : -1;
              if (at >= 0 && in) pool_store(out + at, fmaf(s, __uint_as_float(v[j]), y[j]));
            }
          }
          done();
        }
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    }
    blocks += mine;
    __syncthreads();  // the tile's tokens, planes and buffers are done with
  }
  if (issued && *sm.abort_flag) ring_drain(full, pos, stages, issued);  // the thread that loads
  pool_teardown(tmem, kPoolTermTmem);
}

// ---------------------------------------------------------------------------
// grad: one unit is 128 features x 64 ranks of one adapter's dA or dB, summed over its tokens;
// the CTAs of a cluster each take a part of the tokens and add up as in down.  Both
// operands come as token rows (MN-major).  An adapter without tokens gets zeros.
//   warp 0  loads; warp 1  products; warps 2..5  accumulator -> shared memory; all  the sum
// ---------------------------------------------------------------------------
constexpr int kPoolGradThreads = 192;
constexpr uint32_t kPoolGradTmem = 64;
constexpr uint32_t kPoolGradBytes = 98 * 1024;  // two CTAs share an SM

struct PoolGradArgs {
  PoolArgs p;
  void *dA, *dB;  // [n, r, K], [n, N, r]
  int planes;
};

template <typename O>
__global__ void __launch_bounds__(kPoolGradThreads) pool_grad_kernel(const __grid_constant__ CUtensorMap tmX,
                                                                     const __grid_constant__ CUtensorMap tmU,
                                                                     const __grid_constant__ CUtensorMap tmDY,
                                                                     const __grid_constant__ CUtensorMap tmT,
                                                                     const __grid_constant__ CUtensorMap tmXt,
                                                                     const __grid_constant__ CUtensorMap tmUt,
                                                                     const __grid_constant__ CUtensorMap tmDYt,
                                                                     const __grid_constant__ CUtensorMap tmTt,
                                                                     const PoolGradArgs a) {
  extern __shared__ uint8_t pool_raw[];
  const PoolSmem sm = pool_smem(pool_raw, kPoolGradBytes);
  const PoolArgs &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = 16384u + a.planes * 8192u, stages = min(kPoolGradBytes / stage_bytes, kPoolMostStages);
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *acc_full = sm.bars + 2 * kPoolMostStages;
  const uint32_t tmem = pool_setup(sm, kPoolGradTmem, kPoolBars);
  const int nrb = (p.r + 63) / 64;
  const int in_a = static_cast<int>((p.K + 127) / 128) * nrb, per_adapter = in_a + static_cast<int>((p.N + 127) / 128) * nrb;
  const int64_t units = static_cast<int64_t>(p.n) * per_adapter;
  const int cs = static_cast<int>(ptx::cluster_nctarank()), q = static_cast<int>(ptx::cluster_ctarank());
  float *exch = reinterpret_cast<float *>(sm.buf);
  RingPos pos;
  uint32_t acc_phase = 0, issued = 0;
  bool ok = true;
  for (int64_t u = blockIdx.x / cs; u < units; u += gridDim.x / cs) {
    const int ad = static_cast<int>(u / per_adapter);
    int w = static_cast<int>(u - static_cast<int64_t>(ad) * per_adapter);
    const bool is_a = w < in_a;
    if (!is_a) w -= in_a;
    const int fb = w / nrb, rb = w - fb * nrb;
    const int64_t cols = is_a ? p.K : p.N;
    const int2 grp = pool_group(p, ad);
    const int cnt = grp.y - grp.x, live = pool_rank(p, ad) - rb * 64;
    const int steps = live > 0 ? (cnt + 63) / 64 : 0;
    const int s_per = (steps + cs - 1) / cs, sb = min(q * s_per, steps), se = min(steps, sb + s_per);
    if (warp == 0) {
      const CUtensorMap *tmV = is_a ? &tmX : &tmDY, *tmP = is_a ? &tmU : &tmT;
      const CUtensorMap *tmVt = is_a ? &tmXt : &tmDYt, *tmPt = is_a ? &tmUt : &tmTt;
      const int g = lane & 15;
      int4 rows = make_int4(0, 0, 0, 0);
      if (sb < se) rows = pool_rows(p, grp.x + sb * 64 + 4 * g, grp.y - 1);
      for (int st = sb; st < se && ok; ++st) {
        const int groups = (min(64, cnt - st * 64) + 15) / 16 * 4;  // whole steps of 16 tokens
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag));
        if (!ok) break;
        uint8_t *d = sm.buf + pos.s * stage_bytes;
        // a group of 32 that is not whole is gathered: rows of other adapters' tokens must not meet the padding
        const bool run = pool_run32(rows, lane, 4 * g, cnt - st * 64, false), tile_load = run && (lane & 7) == 0;
        const bool gather = !run && g < groups;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[pos.s], groups * 512u * (2 + a.planes));
        __syncwarp();
        uint8_t *dv = d + (lane >> 4) * 8192 + g * 512;
        const int xv = fb * 128 + (lane >> 4) * 64;
        if (tile_load) ptx::tma_load_2d(dv, tmVt, &full[pos.s], xv, rows.x);
        if (gather) ptx::tma_gather4(dv, tmV, &full[pos.s], xv, rows);
        for (int pl = lane >> 4; pl < a.planes; pl += 2) {
          const int o = pl * static_cast<int>(p.M);
          uint8_t *dp = d + 16384 + pl * 8192 + g * 512;
          if (tile_load) ptx::tma_load_2d(dp, tmPt, &full[pos.s], rb * 64, rows.x + o);
          if (gather) ptx::tma_gather4(dp, tmP, &full[pos.s], rb * 64, make_int4(rows.x + o, rows.y + o, rows.z + o, rows.w + o));
        }
        if (st + 1 < se) rows = pool_rows(p, grp.x + (st + 1) * 64 + 4 * g, grp.y - 1);
        __syncwarp();
        ++issued;
        pos.next(stages);
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    } else if (warp == 1) {
      const uint32_t idesc = ptx::idesc_bf16(128, 64, 1, 1);
      for (int st = sb; st < se && ok; ++st) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
        if (!ok) break;
        uint8_t *d = sm.buf + pos.s * stage_bytes;
        const int valid = min(64, cnt - st * 64);
        if (valid & 15) {
          // the last 16 tokens are not all there: zero rows of P meet repeated rows of V
          const int pad = 16 - (valid & 15);
          for (int i = lane; i < pad * 8 * a.planes; i += 32) {
            const int pl = i / (pad * 8), e = i - pl * pad * 8;
            *reinterpret_cast<uint4 *>(d + 16384 + pl * 8192 + (valid + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        ptx::tc_fence_after();
        if (lane == 0) {
          const uint32_t v = ptx::smem_addr(d), b = v + 16384;
          for (int k16 = 0; k16 * 16 < valid; ++k16)
            for (int pl = 0; pl < a.planes; ++pl)
              ptx::mma_bf16(tmem, ptx::smem_desc_sw128(v + k16 * 2048, 8192, 1024),
                            ptx::smem_desc_sw128(b + pl * 8192 + k16 * 2048, 8192, 1024), idesc, (st != sb || k16 || pl) ? 1u : 0u);
          ptx::mma_commit(&empty[pos.s]);
        }
        __syncwarp();
        pos.next(stages);
      }
      if (ok && se > sb && lane == 0) ptx::mma_commit(acc_full);
      if (!ok && lane == 0) pool_fail(sm, p.status);
      __syncwarp();
    } else if (steps > 0) {
      const int quad = warp & 3, f = quad * 32 + lane;
      if (se > sb && ok) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_full, acc_phase, sm.abort_flag));
        acc_phase ^= 1;
        if (!ok && lane == 0) pool_fail(sm, p.status);
      }
      ptx::tc_fence_after();
      // dA: [rank][feature], dB: [feature][rank] with a pitch that keeps pairs aligned and lanes on 16 banks
      const int pitch = is_a ? 128 : 1, lane_pitch = is_a ? 1 : 66;
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t v[32];
        if (se > sb && ok) {
          ptx::tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0, v);
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) exch[(c0 + j) * pitch + f * lane_pitch] = __uint_as_float(v[j]);
      }
      ptx::tc_fence_before();
    }
    if (steps > 0) pool_cluster_sync();
    // this CTA's share, in pairs of consecutive elements of the output
    const float s = p.scales[ad];
    const uint32_t exch_addr = ptx::smem_addr(exch);
    const int rows = is_a ? 64 : 128, width = is_a ? 64 : 32, pitch = is_a ? 128 : 66;  // pairs a row
    const int per = (rows + cs - 1) / cs, r_lo = min(rows, q * per), r_hi = min(rows, r_lo + per);
    for (int e = threadIdx.x; e < (r_hi - r_lo) * width; e += kPoolGradThreads) {
      const int row = r_lo + e / width, x = 2 * (e % width);
      const int j = rb * 64 + (is_a ? row : x);
      const int64_t f = static_cast<int64_t>(fb) * 128 + (is_a ? x : row);
      if (j >= p.r || f >= cols) continue;  // r and cols are even, and so is x
      float2 v = make_float2(0.0f, 0.0f);
      if (steps > 0 && j - rb * 64 < live) {
        for (int r = 0; r < cs; ++r) {
          const float2 o = ptx::ld_cluster_f32x2(ptx::mapa_shared(exch_addr + (row * pitch + x) * 4, r));
          v.x += o.x;
          v.y += o.y;
        }
        v.x *= s;
        v.y *= s;
      }
      const int64_t at = is_a ? (static_cast<int64_t>(ad) * p.r + j) * p.K + f : (static_cast<int64_t>(ad) * p.N + f) * p.r + j;
      O *out = static_cast<O *>(is_a ? a.dA : a.dB) + at;
      if (sizeof(O) == 4)
        *reinterpret_cast<float2 *>(out) = v;
      else
        *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(v.x, v.y);
    }
    if (steps > 0) {
      ptx::fence_proxy_async_smem();  // the next unit's loads overwrite what was read and written here
      pool_cluster_sync();
    }
  }
  if (warp == 0 && lane == 0 && *sm.abort_flag) ring_drain(full, pos, stages, issued);
  pool_teardown(tmem, kPoolGradTmem);
}

}  // namespace qlora
