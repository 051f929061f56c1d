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
// The products.  Three kernels, all on the tensor cores (tcgen05, accumulators in
// TMEM) with the adapters' matrices, or features, in the 128 rows of the
// accumulator and tokens, or ranks, in its columns:
//
//   down  P = V W_a over the long dimension: T = X A^T, U = dY B     [rank x token]
//   up    Out += s_a P W_a over the rank: Y with B^T, dX with A      [feature x token]
//   grad  s_a P^T V over the tokens of an adapter: dA, dB            [feature x rank]
//
// A tile holds tokens of one adapter, wherever their rows lie: one warp gathers them,
// four rows to an instruction (TMA gather, 128-byte swizzle), and a short tile loads
// only the rows it has.  Columns of the accumulator are independent, so a short
// tile's unused columns need no zeros, and neither do rows past an adapter's rank.
// How the tiles fall follows from offsets, which only the device knows: each CTA sums
// the adapters' tile counts into shared memory first, and walks tiles from there.
//
// All three are bound by HBM at ranks up to about 128 (r flops a byte of X, dY, Y or
// dX), so the loads run ahead in a ring of 64-column stages and two CTAs share an SM.
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

// The same for a gather, which needs some row in range: row 0 then, whose result is not written.
__device__ __forceinline__ int4 pool_rows(const PoolArgs &p, int i, int last) {
  int4 y;
  y.x = max(pool_token(p, min(i, last)), 0);
  y.y = max(pool_token(p, min(i + 1, last)), 0);
  y.z = max(pool_token(p, min(i + 2, last)), 0);
  y.w = max(pool_token(p, min(i + 3, last)), 0);
  return y;
}

// Loads of token rows into a stage: 32 consecutive rows of memory come with one tiled load (box 64 x 32), other rows
// four to a gather.  A gather costs the loading thread as much as a tiled load eight times its size (the down kernel
// took 46 us to read 67 MB by gathers alone), and requests of a packed batch are runs of rows.
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

// pre[a] = tiles of tn tokens of the adapters before a, a = 0 .. n; returns pre[n].  The whole block.
__device__ __forceinline__ int pool_scan(const PoolArgs &p, int tn, int *pre) {
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n + blockDim.x - 1) / blockDim.x, a0 = tid * per, a1 = min(p.n, a0 + per);
  int sum = 0;
  for (int a = a0; a < a1; ++a) {
    const int2 g = pool_group(p, a);
    sum += (g.y - g.x + tn - 1) / tn;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int a = a0; a < a1; ++a) {
    pre[a] = at;
    const int2 g = pool_group(p, a);
    at += (g.y - g.x + tn - 1) / tn;
  }
  if (tid == static_cast<int>(blockDim.x) - 1) pre[p.n] = at;
  __syncthreads();
  return pre[p.n];
}

// The adapter of a tile: the last one with pre[a] <= tile.
__device__ __forceinline__ int pool_find(const int *pre, int n, int tile) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
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

// Shared memory of one CTA: two share an SM's 227 KB, whatever the rank.
constexpr uint32_t kPoolRingBytes = 98 * 1024;
__host__ __device__ constexpr uint32_t pool_smem_bytes(int n) {
  return 1024 + kPoolRingBytes + 512 + (static_cast<uint32_t>(n) + 1) * 4;
}
struct PoolSmem {
  uint8_t *ring;      // 1024-byte aligned
  uint64_t *bars;     // 24
  uint32_t *tmem_slot;
  volatile int *abort_flag;
  int *pre;           // [n + 1]
};
__device__ __forceinline__ PoolSmem pool_smem(uint8_t *raw) {
  PoolSmem s;
  s.ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.bars = reinterpret_cast<uint64_t *>(s.ring + kPoolRingBytes);
  s.tmem_slot = reinterpret_cast<uint32_t *>(s.bars + 24);
  s.abort_flag = reinterpret_cast<volatile int *>(s.tmem_slot + 1);
  s.pre = reinterpret_cast<int *>(s.ring + kPoolRingBytes + 512);
  return s;
}

// Set-up that all three share: barriers (one arrival each, but `acc_empty`), TMEM, then the wait for the kernel ahead.  The
// next kernel may start only after that wait: one that reads early, or that waits for this kernel alone, then finds
// everything before this kernel complete too.
__device__ __forceinline__ uint32_t pool_setup(const PoolSmem &s, uint32_t tmem_cols, int acc_empty0, int acc_empty_count) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 24; ++i)
      ptx::mbar_init(&s.bars[i], acc_empty0 >= 0 && (i == acc_empty0 || i == acc_empty0 + 1) ? acc_empty_count : 1);
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
// down: one unit is 128 tokens x 128 ranks; the CTAs of a cluster each sum a part of
// the long dimension, leave their float32 partial accumulators in shared memory, and
// each then adds a share of the tokens over all of them, in CTA order, through
// distributed shared memory: no partial planes in HBM, no second launch, and the same
// bits every time.
//   warp 0  loads; warp 1  products; warps 2..5  accumulator -> shared memory; all  the sum
// W_MN false: W is [n][r][len] (K-major); true: [n][len][r] (MN-major).
// ---------------------------------------------------------------------------
constexpr int kPoolDownThreads = 192;
constexpr int kPoolDownTile = 128;
constexpr uint32_t kPoolDownTmem = 128;

struct PoolDownArgs {
  PoolArgs p;
  int k_steps;  // of 64
  __nv_bfloat16 *P;
};

template <bool W_MN>
__global__ void __launch_bounds__(kPoolDownThreads) pool_down_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                     const __grid_constant__ CUtensorMap tmV,
                                                                     const __grid_constant__ CUtensorMap tmVt,
                                                                     const PoolDownArgs a) {
  extern __shared__ uint8_t pool_raw[];
  const PoolSmem sm = pool_smem(pool_raw);
  const PoolArgs &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a stage: W's rows (64 of them when r <= 64; the accumulator's upper rows then multiply what follows in
  // memory and are not read), then 128 token rows
  const uint32_t w_bytes = p.r <= 64 ? 8192u : 16384u, stage_bytes = w_bytes + 16384u, stages = kPoolRingBytes / stage_bytes;
  uint64_t *full = sm.bars, *empty = sm.bars + 4, *acc_full = sm.bars + 8;
  const uint32_t tmem = pool_setup(sm, kPoolDownTmem, -1, 1);
  const int tiles = pool_scan(p, kPoolDownTile, sm.pre);
  const int nrb = (p.r + 127) / 128;
  const int64_t units = static_cast<int64_t>(tiles) * nrb;
  const int cs = static_cast<int>(ptx::cluster_nctarank()), q = static_cast<int>(ptx::cluster_ctarank());
  const int k_per = (a.k_steps + cs - 1) / cs;
  float *exch = reinterpret_cast<float *>(sm.ring);
  RingPos pos;
  uint32_t acc_phase = 0, issued = 0;
  bool ok = true;
  for (int64_t u = blockIdx.x / cs; u < units; u += gridDim.x / cs) {
    const int tile = static_cast<int>(u / nrb), rb = static_cast<int>(u - static_cast<int64_t>(tile) * nrb);
    const int ad = pool_find(sm.pre, p.n, tile);
    const int2 grp = pool_group(p, ad);
    const int lo = grp.x + (tile - sm.pre[ad]) * kPoolDownTile, cnt = min(kPoolDownTile, grp.y - lo);
    const int live = pool_rank(p, ad) - rb * 128;  // ranks of this block that exist
    const int rw = min(128, p.r - rb * 128);
    const int kb = live > 0 ? min(q * k_per, a.k_steps) : 0, ke = live > 0 ? min(a.k_steps, kb + k_per) : 0;
    if (warp == 0) {
      const int4 rows = pool_rows(p, lo + 4 * lane, lo + cnt - 1);
      const bool run = pool_run32(rows, lane, 4 * lane, cnt, true), tile_load = run && (lane & 7) == 0;
      const bool gather = !run && 4 * lane < cnt;
      const int w_loads = W_MN ? (rw + 63) / 64 : 1;
      const uint32_t bytes = (W_MN ? w_loads * 8192u : static_cast<uint32_t>(min(p.r, 128)) * 128u) +
                             __popc(__ballot_sync(0xffffffffu, tile_load)) * 4096u +
                             __popc(__ballot_sync(0xffffffffu, gather)) * 512u;
      for (int ks = kb; ks < ke && ok; ++ks) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag));
        if (!ok) break;
        uint8_t *st = sm.ring + pos.s * stage_bytes;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&full[pos.s], bytes);
          if (W_MN)
            for (int i = 0; i < w_loads; ++i) ptx::tma_load_3d(st + i * 8192, &tmW, &full[pos.s], rb * 128 + i * 64, ks * 64, ad);
          else
            ptx::tma_load_3d(st, &tmW, &full[pos.s], ks * 64, rb * 128, ad);
        }
        __syncwarp();
        if (tile_load) ptx::tma_load_2d(st + w_bytes + lane * 512, &tmVt, &full[pos.s], ks * 64, rows.x);
        if (gather) ptx::tma_gather4(st + w_bytes + lane * 512, &tmV, &full[pos.s], ks * 64, rows);
        ++issued;
        pos.next(stages);
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    } else if (warp == 1) {
      const uint32_t idesc = ptx::idesc_bf16(128, (cnt + 15) / 16 * 16, W_MN ? 1 : 0, 0);
      for (int ks = kb; ks < ke && ok; ++ks) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        if (lane == 0) {
          const uint32_t w = ptx::smem_addr(sm.ring + pos.s * stage_bytes), v = w + w_bytes;
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            ptx::mma_bf16(tmem, W_MN ? ptx::smem_desc_sw128(w + k16 * 2048, 8192, 1024) : ptx::smem_desc_sw128(w + k16 * 32, 16, 1024),
                          ptx::smem_desc_sw128(v + k16 * 32, 16, 1024), idesc, (ks != kb || k16) ? 1u : 0u);
          ptx::mma_commit(&empty[pos.s]);
        }
        __syncwarp();
        pos.next(stages);
      }
      if (ok && ke > kb && lane == 0) ptx::mma_commit(acc_full);
      if (!ok && lane == 0) pool_fail(sm, p.status);
      __syncwarp();
    } else {
      const int quad = warp & 3;
      if (ke > kb && ok) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_full, acc_phase, sm.abort_flag));
        acc_phase ^= 1;
        if (!ok && lane == 0) pool_fail(sm, p.status);
      }
      ptx::tc_fence_after();
      if (quad * 32 < rw)
        for (int c0 = 0; c0 < cnt; c0 += 32) {
          uint32_t v[32];
          if (ke > kb && ok) {
            ptx::tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0, v);
            ptx::tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j < cnt) exch[(c0 + j) * 128 + quad * 32 + lane] = __uint_as_float(v[j]);
        }
      ptx::tc_fence_before();
    }
    pool_cluster_sync();
    // this CTA's share of the tokens
    const int per = (cnt + cs - 1) / cs, c_lo = min(cnt, q * per), c_hi = min(cnt, c_lo + per), half = rw / 2;
    const uint32_t exch_addr = ptx::smem_addr(exch);
    for (int e = threadIdx.x; e < (c_hi - c_lo) * half; e += kPoolDownThreads) {
      const int c = c_lo + e / half, j = 2 * (e % half);
      float2 s = make_float2(0.0f, 0.0f);
      for (int r = 0; r < cs; ++r) {
        const float2 v = ptx::ld_cluster_f32x2(ptx::mapa_shared(exch_addr + (c * 128 + j) * 4, r));
        s.x += v.x;
        s.y += v.y;
      }
      if (j >= live) s = make_float2(0.0f, 0.0f);  // a multiple of 8, so both
      const int t = pool_token(p, lo + c);
      if (t < 0) continue;
      __nv_bfloat16 *out = a.P + static_cast<int64_t>(t) * p.r + rb * 128 + j;
#pragma unroll
      for (int pl = 0; pl < kPoolPlanes; ++pl) {
        const uint32_t h = pack_bf16x2(s.x, s.y);
        *reinterpret_cast<uint32_t *>(out + pl * p.M * p.r) = h;
        s.x -= bf16lo_to_f32(h);
        s.y -= bf16hi_to_f32(h);
      }
    }
    ptx::fence_proxy_async_smem();  // the next unit's loads overwrite what was read and written here
    pool_cluster_sync();
  }
  if (warp == 0 && lane == 0 && *sm.abort_flag) ring_drain(full, pos, stages, issued);
  pool_teardown(tmem, kPoolDownTmem);
}

// ---------------------------------------------------------------------------
// up: one unit is a tile of tokens and a run of 128-feature blocks.  P's rows of the tile
// are loaded once, the blocks of W stream through the ring, and the accumulator of one
// block is computed while the one before is added to Out.  A warp of the epilogue takes 32
// features x half of the tile's tokens.  Its lanes hold features; where Out's rows are
// 16-byte aligned, 16 tokens at a time pass through shared memory, so that four lanes (bf16;
// eight for float32) then share a token's 32 features in 16-byte pieces, all loaded before the accumulator is waited
// for (64 KB in flight on an SM; element by element the epilogue took 47 instructions an
// element and warp and bound the kernel on issue).  Other outputs, odd strides or columns of a
// wider tensor, go element by element.
//   warp 0  loads; warp 1  products; warps 2..9  Out += s_a accumulator
// W_MN false: W is [n][cols][r] (Y: B); true: [n][r][cols] (dX: A).
// ---------------------------------------------------------------------------
constexpr int kPoolUpThreads = 320;
constexpr uint32_t kPoolUpTmem = 256;  // two accumulators of up to 128 tokens

struct PoolUpArgs {
  PoolArgs p;
  int64_t cols, ldo;
  void *out;
  int planes;
  int tn;  // tokens a tile: 128, 64 or 32
};

// Tokens of an up tile: as many as keep P's planes within 48 KB, which leaves the ring two stages or more.
constexpr uint32_t kPoolUpPlaneBytes = 48 * 1024, kPoolUpRingBytes = 80 * 1024;
__host__ __device__ constexpr int pool_up_tile(int r, int planes) {
  const uint32_t row = (r + 63) / 64 * planes * 128u;
  return row * 128 <= kPoolUpPlaneBytes ? 128 : row * 64 <= kPoolUpPlaneBytes ? 64 : 32;
}
static_assert(pool_up_tile(256, 3) == 32 && 4 * 3 * 32 * 128 <= kPoolUpPlaneBytes, "the largest rank fits");
// Shared memory of a warp's 16 tokens x 32 features: a pitch of 36 floats keeps 16-byte pieces aligned and both
// directions without bank conflicts.
constexpr int kPoolUpPitch = 36, kPoolUpBuf = 16 * kPoolUpPitch;
static_assert(kPoolUpRingBytes + 8 * kPoolUpBuf * 4 <= kPoolRingBytes, "shared memory");

__device__ __forceinline__ float pool_load(const float *p) { return __ldcg(p); }
__device__ __forceinline__ float pool_load(const __nv_bfloat16 *p) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(p))) << 16);
}
__device__ __forceinline__ void pool_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void pool_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes of Out: y + s v, rounded once.  kElems elements; a row's 32 features take 32 / kElems lanes, so that each
// instruction covers whole sectors.  kTokens: loaded ahead by a warp, 4 KB.
template <typename O>
struct PoolPiece;
template <>
struct PoolPiece<float> {
  static constexpr int kElems = 4, kTokens = 32;
  float4 y;
  __device__ __forceinline__ void zero() { y = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const float *p) { y = __ldcg(reinterpret_cast<const float4 *>(p)); }
  __device__ __forceinline__ void add_store(float *p, float s, const float *v) const {
    const float4 u = *reinterpret_cast<const float4 *>(v);
    *reinterpret_cast<float4 *>(p) = make_float4(fmaf(s, u.x, y.x), fmaf(s, u.y, y.y), fmaf(s, u.z, y.z), fmaf(s, u.w, y.w));
  }
};
template <>
struct PoolPiece<__nv_bfloat16> {
  static constexpr int kElems = 8, kTokens = 64;
  uint4 y;
  __device__ __forceinline__ void zero() { y = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { y = __ldcg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void add_store(__nv_bfloat16 *p, float s, const float *v) const {
    const float4 u = reinterpret_cast<const float4 *>(v)[0], w = reinterpret_cast<const float4 *>(v)[1];
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(fmaf(s, u.x, bf16lo_to_f32(y.x)), fmaf(s, u.y, bf16hi_to_f32(y.x))),
                                               pack_bf16x2(fmaf(s, u.z, bf16lo_to_f32(y.y)), fmaf(s, u.w, bf16hi_to_f32(y.y))),
                                               pack_bf16x2(fmaf(s, w.x, bf16lo_to_f32(y.z)), fmaf(s, w.y, bf16hi_to_f32(y.z))),
                                               pack_bf16x2(fmaf(s, w.z, bf16lo_to_f32(y.w)), fmaf(s, w.w, bf16hi_to_f32(y.w))));
  }
};

template <bool W_MN, typename O, bool VEC>
__global__ void __launch_bounds__(kPoolUpThreads, 2) pool_up_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                    const __grid_constant__ CUtensorMap tmP,
                                                                    const __grid_constant__ CUtensorMap tmPt,
                                                                    const PoolUpArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int token[128];
  const PoolSmem sm = pool_smem(pool_raw);
  const PoolArgs &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tn = a.tn;
  const uint32_t plane_bytes = tn * 128u, p_bytes = (p.r + 63) / 64 * a.planes * plane_bytes;
  const uint32_t stages = min((kPoolUpRingBytes - p_bytes) / 16384u, 4u);
  uint8_t *ring = sm.ring + p_bytes;
  uint64_t *full = sm.bars, *empty = sm.bars + 4, *acc_full = sm.bars + 8, *acc_empty = sm.bars + 10, *p_full = sm.bars + 12;
  const uint32_t tmem = pool_setup(sm, kPoolUpTmem, 10, 8);
  const int tiles = pool_scan(p, tn, sm.pre);
  const int nblk = static_cast<int>((a.cols + 127) / 128);
  // runs of blocks: as many as give every CTA a unit
  int runs = min(max(static_cast<int>(gridDim.x) / max(tiles, 1), 1), nblk);
  const int run = (nblk + runs - 1) / runs;
  runs = (nblk + run - 1) / run;
  const int64_t units = static_cast<int64_t>(tiles) * runs;
  RingPos pos;
  uint32_t p_phase = 0, issued = 0, blocks = 0;  // blocks: accumulators used so far
  bool ok = true;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = static_cast<int>(u / runs), b0 = static_cast<int>(u - static_cast<int64_t>(tile) * runs) * run;
    const int b1 = min(nblk, b0 + run);
    const int ad = pool_find(sm.pre, p.n, tile);
    const int2 grp = pool_group(p, ad);
    const int lo = grp.x + (tile - sm.pre[ad]) * tn, cnt = min(tn, grp.y - lo);
    const int rank = pool_rank(p, ad), nch = (rank + 63) / 64;
    if (rank == 0) continue;
    if (warp >= 2) {
      const int i = threadIdx.x - 64;
      if (i < 128) token[i] = i < cnt ? pool_token(p, lo + i) : -1;
    }
    __syncthreads();
    if (warp == 0) {
      const int4 rows = pool_rows(p, lo + 4 * lane, lo + cnt - 1);
      const bool run_32 = pool_run32(rows, lane, 4 * lane, cnt, true), tile_load = run_32 && (lane & 7) == 0;
      const bool gather = !run_32 && 4 * lane < cnt;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, tile_load)) * 4096u + __popc(__ballot_sync(0xffffffffu, gather)) * 512u;
      if (ok) {
        if (lane == 0) ptx::mbar_arrive_expect_tx(p_full, nch * a.planes * bytes);
        __syncwarp();
        for (int i = 0; i < nch * a.planes; ++i) {
          const int o = i % a.planes * static_cast<int>(p.M), x = i / a.planes * 64;
          uint8_t *d = sm.ring + i * plane_bytes + lane * 512;
          if (tile_load) ptx::tma_load_2d(d, &tmPt, p_full, x, rows.x + o);
          if (gather) ptx::tma_gather4(d, &tmP, p_full, x, make_int4(rows.x + o, rows.y + o, rows.z + o, rows.w + o));
        }
        __syncwarp();
      }
      for (int b = b0; b < b1 && ok; ++b)
        for (int ch = 0; ch < nch && ok; ++ch) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag));
          if (!ok) break;
          if (lane == 0) {
            uint8_t *st = ring + pos.s * 16384u;
            ptx::mbar_arrive_expect_tx(&full[pos.s], 16384u);
            if (W_MN) {
              ptx::tma_load_3d(st, &tmW, &full[pos.s], b * 128, ch * 64, ad);
              ptx::tma_load_3d(st + 8192, &tmW, &full[pos.s], b * 128 + 64, ch * 64, ad);
            } else {
              ptx::tma_load_3d(st, &tmW, &full[pos.s], ch * 64, b * 128, ad);
            }
          }
          __syncwarp();
          ++issued;
          pos.next(stages);
        }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    } else if (warp == 1) {
      const uint32_t idesc = ptx::idesc_bf16(128, (cnt + 15) / 16 * 16, W_MN ? 1 : 0, 0);
      const uint32_t p_addr = ptx::smem_addr(sm.ring);
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(p_full, p_phase, sm.abort_flag));
      uint32_t n = blocks;
      for (int b = b0; b < b1 && ok; ++b, ++n) {
        const uint32_t acc = n & 1;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_empty[acc], ((n >> 1) & 1) ^ 1, sm.abort_flag));
        for (int ch = 0; ch < nch && ok; ++ch) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
          if (!ok) break;
          uint8_t *st = ring + pos.s * 16384u;
          const int left = min(64, rank - ch * 64);  // a multiple of 8
          if ((left & 8) && rank < p.r) {
            // products go 16 ranks at a time: the 8 past the adapter's rank meet zeros in P and have to be finite
            if (W_MN) {
              for (int i = lane; i < 128; i += 32)
                *reinterpret_cast<uint4 *>(st + (i >> 6) * 8192 + (left + ((i >> 3) & 7)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            } else {
              for (int i = lane; i < 128; i += 32)
                *reinterpret_cast<uint4 *>(st + i * 128 + (((left >> 3) ^ (i & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          ptx::tc_fence_after();
          if (lane == 0) {
            const uint32_t w = ptx::smem_addr(st);
            for (int k16 = 0; k16 * 16 < left; ++k16)
              for (int pl = 0; pl < a.planes; ++pl)
                ptx::mma_bf16(tmem + acc * 128,
                              W_MN ? ptx::smem_desc_sw128(w + k16 * 2048, 8192, 1024) : ptx::smem_desc_sw128(w + k16 * 32, 16, 1024),
                              ptx::smem_desc_sw128(p_addr + (ch * a.planes + pl) * plane_bytes + k16 * 32, 16, 1024), idesc,
                              (ch || k16 || pl) ? 1u : 0u);
            ptx::mma_commit(&empty[pos.s]);
          }
          __syncwarp();
          pos.next(stages);
        }
        if (ok && lane == 0) ptx::mma_commit(&acc_full[acc]);
        __syncwarp();
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    } else {
      const int quad = warp & 3, half = (warp - 2) >> 2;
      const int c_lo = half * (tn / 2), c_hi = min(cnt, c_lo + tn / 2);
      const float s = p.scales[ad];
      uint32_t n = blocks;
      for (int b = b0; b < b1 && ok; ++b, ++n) {
        const uint32_t acc = n & 1;
        const int64_t f = static_cast<int64_t>(b) * 128 + quad * 32 + lane;
        O *out = static_cast<O *>(a.out) + f;
        bool ready = false;
        if (VEC) {
          float *buf = reinterpret_cast<float *>(sm.ring + kPoolUpRingBytes) + (warp - 2) * kPoolUpBuf;
          constexpr int kGroup = PoolPiece<O>::kTokens, kElems = PoolPiece<O>::kElems, kLanes = 32 / kElems, kRows = 32 / kLanes;
          const int tr = lane / kLanes, part = lane % kLanes;
          const int64_t f8 = static_cast<int64_t>(b) * 128 + quad * 32 + part * kElems;
          O *out8 = static_cast<O *>(a.out) + f8;
          for (int g0 = c_lo; g0 < c_hi; g0 += kGroup) {
            PoolPiece<O> y[kGroup / kRows];
#pragma unroll
            for (int i = 0; i < kGroup / kRows; ++i) {
              const int c = g0 + kRows * i + tr, t = c < c_hi ? token[c] : -1;
              if (t >= 0 && f8 < a.cols) y[i].load(out8 + t * a.ldo);
              else y[i].zero();
            }
            if (!ready) {
              ready = true;
              ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], (n >> 1) & 1, sm.abort_flag));
              if (!ok) break;
              ptx::tc_fence_after();
            }
#pragma unroll
            for (int k = 0; k < kGroup / 16; ++k) {
              if (g0 + 16 * k >= c_hi) break;
              uint32_t v[16];
              ptx::tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 128 + g0 + 16 * k, v);
              ptx::tmem_ld_wait();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 16; ++j) buf[j * kPoolUpPitch + lane] = __uint_as_float(v[j]);
              __syncwarp();
#pragma unroll
              for (int h = 0; h < 16 / kRows; ++h) {
                const int c = g0 + 16 * k + kRows * h + tr, t = c < c_hi ? token[c] : -1;
                if (t >= 0 && f8 < a.cols)
                  y[16 / kRows * k + h].add_store(out8 + t * a.ldo, s, buf + (kRows * h + tr) * kPoolUpPitch + part * kElems);
              }
            }
          }
        } else {
          for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int t = c0 + j < c_hi ? token[c0 + j] : -1;
              y[j] = t >= 0 && f < a.cols ? pool_load(out + t * a.ldo) : 0.0f;
            }
            if (!ready) {
              ready = true;
              ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], (n >> 1) & 1, sm.abort_flag));
              if (!ok) break;
              ptx::tc_fence_after();
            }
            uint32_t v[32];
            ptx::tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 128 + c0, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int t = c0 + j < c_hi ? token[c0 + j] : -1;
              if (t >= 0 && f < a.cols) pool_store(out + t * a.ldo, fmaf(s, __uint_as_float(v[j]), y[j]));
            }
          }
        }
        if (!ready && ok)  // no tokens in this half
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], (n >> 1) & 1, sm.abort_flag));
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&acc_empty[acc]);
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    }
    p_phase ^= 1;
    blocks += b1 - b0;
    __syncthreads();  // the tile's rows of P and its tokens are done with
  }
  if (warp == 0 && lane == 0 && *sm.abort_flag) {
    ring_drain(full, pos, stages, issued);
    ptx::mbar_wait(p_full, p_phase ^ 1, nullptr);
  }
  pool_teardown(tmem, kPoolUpTmem);
}

// ---------------------------------------------------------------------------
// grad: one unit is 128 features x 64 ranks of one adapter's dA or dB, summed over its tokens;
// the CTAs of a cluster each take a part of the tokens and add up as in down.  Both
// operands come as token rows (MN-major).  An adapter without tokens gets zeros.
//   warp 0  loads; warp 1  products; warps 2..5  accumulator -> shared memory; all  the sum
// ---------------------------------------------------------------------------
constexpr int kPoolGradThreads = 192;
constexpr uint32_t kPoolGradTmem = 64;

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
  const PoolSmem sm = pool_smem(pool_raw);
  const PoolArgs &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = 16384u + a.planes * 8192u, stages = min(kPoolRingBytes / stage_bytes, 4u);
  uint64_t *full = sm.bars, *empty = sm.bars + 4, *acc_full = sm.bars + 8;
  const uint32_t tmem = pool_setup(sm, kPoolGradTmem, -1, 1);
  const int nrb = (p.r + 63) / 64;
  const int in_a = static_cast<int>((p.K + 127) / 128) * nrb, per_adapter = in_a + static_cast<int>((p.N + 127) / 128) * nrb;
  const int64_t units = static_cast<int64_t>(p.n) * per_adapter;
  const int cs = static_cast<int>(ptx::cluster_nctarank()), q = static_cast<int>(ptx::cluster_ctarank());
  float *exch = reinterpret_cast<float *>(sm.ring);
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
        uint8_t *d = sm.ring + pos.s * stage_bytes;
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
        uint8_t *d = sm.ring + pos.s * stage_bytes;
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
