// Many adapters on one base: the tokens grouped by adapter, the adapters' term of
// the forward pass and its gradients (see qlora_adapters_fwd in qlora_nf4.h).
#pragma once

#include <cuda_bf16.h>

#include "nf4_device.cuh"
#include "sm100_ptx.cuh"

namespace qlora {

// ---------------------------------------------------------------------------
// Tokens grouped by adapter: a stable counting sort by the CTAs of one cluster (one CTA for
// few tokens).  Warp w of CTA b owns the (b, w)-th contiguous piece of the tokens and counts
// its keys in its own row of shared counters, 32 tokens at a time: match gives the lanes of
// equal keys, and their first adds for all (runs of one request would serialise atomics).  Each
// CTA then needs, of each key, the counts of the CTAs before it and of all, read
// through distributed shared memory, and a running sum over the keys; that turns the counters
// into first places, and a second walk places the tokens with the rank among equal keys.
// Key n: no adapter.  Latency bound: 22 us with one CTA for 65536 tokens of 512 adapters.
// ---------------------------------------------------------------------------
constexpr int kGroupThreads = 1024, kGroupWarps = kGroupThreads / 32;
constexpr int kGroupCluster = 8;
// Tokens up to which one CTA is faster (64 adapters: 1024 tokens 5.3 us against 6.4 with the cluster, 2048 7.3 against 6.6).
constexpr int64_t kGroupOneCta = 1536;

__device__ __forceinline__ int group_key(const int32_t *idx, int64_t t, int n, uint32_t *status) {
  const int a = idx[t];
  if (a >= 0 && a < n) return a;
  if (a != -1) raise_status(status, QLORA_ERR_INVALID_ARGUMENT);
  return n;
}

__global__ void __launch_bounds__(kGroupThreads) adapter_groups_kernel(const int32_t *__restrict__ idx, int64_t M, int n,
                                                                       int32_t *__restrict__ order,
                                                                       int32_t *__restrict__ offsets, uint32_t *status) {
  extern __shared__ int32_t group_counts[];  // [warps][n + 1], then [n + 1] of the CTA
  __shared__ int32_t warp_sum[kGroupWarps];
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, keys = n + 1;
  const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
  int32_t *mine = group_counts + warp * keys, *cta = group_counts + kGroupWarps * keys;
  for (int i = tid; i < kGroupWarps * keys; i += kGroupThreads) group_counts[i] = 0;
  __syncthreads();
  const int64_t pieces = static_cast<int64_t>(ctas) * kGroupWarps;
  const int64_t per = ((M + pieces - 1) / pieces + 31) / 32 * 32;
  const int64_t t0 = (static_cast<int64_t>(rank) * kGroupWarps + warp) * per, t1 = min(M, t0 + per);
  for (int64_t b = t0; b < t1; b += 32) {
    const int64_t t = b + lane;
    const int key = t < t1 ? group_key(idx, t, n, status) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && (same & ((1u << lane) - 1u)) == 0) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // a thread's key (at most one key more than threads: QLORA_MAX_ADAPTERS + 1, so the last thread may have two)
  for (int k = tid; k < keys; k += kGroupThreads) {
    int32_t s = 0;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) s += group_counts[w * keys + k];
    cta[k] = s;
  }
  if (ctas > 1) ptx::cluster_sync(); else __syncthreads();
  // of key k: the count of all CTAs, and of those before this one
  auto totals = [&](int k, int32_t &before) {
    int32_t all = 0;
    before = 0;
    const uint32_t at = ptx::smem_addr(cta + k);
    for (int c = 0; c < ctas; ++c) {
      const int32_t x = ctas > 1 ? static_cast<int32_t>(ptx::ld_cluster_u32(ptx::mapa_shared(at, c))) : cta[k];
      all += x;
      if (c < rank) before += x;
    }
    return all;
  };
  int32_t before = 0, extra_before = 0;
  const int32_t all = tid < keys ? totals(tid, before) : 0;
  const bool two = tid == kGroupThreads - 1 && keys > kGroupThreads;  // the last key
  if (two) totals(kGroupThreads, extra_before);
  int32_t inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int32_t first = inc - all;
  for (int w = 0; w < warp; ++w) first += warp_sum[w];
  auto place = [&](int k, int32_t at, int32_t ahead) {
    if (rank == 0) offsets[k] = at;  // key n: the number of tokens with an adapter
    at += ahead;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) {
      const int32_t c = group_counts[w * keys + k];
      group_counts[w * keys + k] = at;
      at += c;
    }
  };
  if (tid < keys) place(tid, first, before);
  if (two) place(kGroupThreads, first + all, extra_before);
  __syncthreads();
  for (int64_t b = t0; b < t1; b += 32) {
    const int64_t t = b + lane;
    const int key = t < t1 ? group_key(idx, t, n, nullptr) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, key);
    const int ahead = __popc(same & ((1u << lane) - 1u));
    if (key >= 0) order[mine[key] + ahead] = static_cast<int32_t>(t);
    __syncwarp();
    if (key >= 0 && ahead == 0) mine[key] += __popc(same);
    __syncwarp();
  }
  if (ctas > 1) ptx::cluster_sync();  // the counts are read by the others
}

// ---------------------------------------------------------------------------
// The products.  Three kernels, on the tensor cores (tcgen05, accumulators in TMEM) with
// ranks, or features, in the 128 rows of the accumulator and tokens, or ranks, in its
// columns:
//
//   down  P = V W_a over the long dimension: T = X A^T, U = dY B
//   up    Out += s_a P W_a over the rank: Y with B^T, dX with A
//   grad  s_a P^T V over the tokens of an adapter: dA, dB
//
// A tile holds tokens of one adapter, wherever their rows lie: runs of 16, 32 or 64 rows come
// with one tiled load, others four rows to a gather, and a short tile loads only the
// rows it has.  Columns of the accumulator are independent, so a short tile's unused
// columns need no zeros, and neither do rows past an adapter's rank.  How the tiles
// fall follows from offsets, which only the device knows: each CTA adds up the
// adapters' tile counts first and walks the tiles from there.
//
// By their work all are bound by HBM at ranks up to about 128 (r flops a byte of X, dY, Y or dX); up over long outputs
// comes near it (0.72 of the copy rate for 4096 tokens on 22016 float32 columns), smaller calls are latency.
// ---------------------------------------------------------------------------
// The intermediates T = X A^T and U = dY B are [M, r] in float32 and kept as three bf16 planes [3, M, r], each the rounding
// of what the ones before leave: 24 bits together, in the type the tensor cores take beside bf16 operands.  A bf16 result
// is computed from the first two (16 bits), a float32 one from all.  With all three a bf16 result is as far from 64 bits,
// 1.7e-3 of it by its own rounding, differs from float32 products' in fewer places (1e-5 of the result against 1e-4), and
// takes longer (48 decode tokens 34.1 us against 30.0, 2039 packed 29.4 against 28.5, 1003 backward 23.1 against 21.8).
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
  const int k = __ldcg(p.ranks + a), c = min(max(k, 0), p.r) & ~7;
  if (c != k) raise_status(p.status, QLORA_ERR_INVALID_ARGUMENT);
  return c;
}

// Places [lo, hi) of adapter a's tokens in order.
__device__ __forceinline__ int2 pool_group(const PoolArgs &p, int a) {
  const int m = static_cast<int>(p.M);
  const int lo = min(max(__ldcg(p.offsets + a), 0), m);
  return make_int2(lo, min(max(__ldcg(p.offsets + a + 1), lo), m));
}

// An entry of the order; -1 if it is out of range.
__device__ __forceinline__ int pool_checked(const PoolArgs &p, int t) {
  if (t >= 0 && t < p.M) return t;
  raise_status(p.status, QLORA_ERR_INVALID_ARGUMENT);
  return -1;
}
// Token at place i (below M).
__device__ __forceinline__ int pool_token(const PoolArgs &p, int i) { return pool_checked(p, __ldcg(p.order + i)); }

// Four entries for a load of rows, as they are, and checked: the load needs some row in range, row 0 then, whose result is
// not written.  Apart, so that a step's entries can be on their way during the step before.
__device__ __forceinline__ int4 pool_entries(const PoolArgs &p, int i, int last) {
  return make_int4(__ldcg(p.order + min(i, last)), __ldcg(p.order + min(i + 1, last)), __ldcg(p.order + min(i + 2, last)),
                   __ldcg(p.order + min(i + 3, last)));
}
__device__ __forceinline__ int4 pool_rows(const PoolArgs &p, const int4 &e) {
  return make_int4(max(pool_checked(p, e.x), 0), max(pool_checked(p, e.y), 0), max(pool_checked(p, e.z), 0),
                   max(pool_checked(p, e.w), 0));
}

// Loads of token rows into a stage: 64, 32 or 16 consecutive rows of memory come with one tiled load, other rows four to a
// gather, and 64 rows of all planes that are used come with one load too.  Requests of a packed batch are runs of rows, and
// a load costs the loading thread 100 to 160 cycles, whatever its rows: gathers alone bound a step of 64 tokens at many
// times its time (reading 67 MB by them took 46 us), and with runs of 32 and planes one by one the backward over 2048
// tokens took 87 us, with these 78.
struct PoolMaps {
  CUtensorMap row, row16, row32, row64;
};

// Whether the kRows / 4 lanes that share this one's run hold kRows consecutive rows, four a lane.  first: of this lane's
// rows in the tile; valid: rows of the tile; those past it may be any rows where `loose` (half of the run must be
// wanted).
template <int kRows>
__device__ __forceinline__ bool pool_run(const int4 &y, int lane, int first, int valid, bool loose) {
  constexpr int kLanes = kRows / 4;
  const int lead = lane & ~(kLanes - 1), base = __shfl_sync(0xffffffffu, y.x, lead) + 4 * (lane - lead), left = valid - first;
  const bool seq = (y.x == base || left < 1) && (y.y == base + 1 || left < 2) && (y.z == base + 2 || left < 3) &&
                   (y.w == base + 3 || left < 4);
  const uint32_t all = __ballot_sync(0xffffffffu, seq);
  const int wanted = valid - (first - 4 * (lane - lead));
  return ((all >> lead) & ((1u << kLanes) - 1u)) == (1u << kLanes) - 1u && wanted >= (loose ? kRows / 2 : kRows);
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
  // an offset, not a rounded pointer: the compiler has to see that this is shared memory (through generic addresses
  // 2039 packed tokens took 32.6 us instead of 30.0)
  s.buf = raw + ((1024u - (ptx::smem_addr(raw) & 1023u)) & 1023u);
  s.bars = reinterpret_cast<uint64_t *>(s.buf + bytes);
  s.tmem_slot = reinterpret_cast<uint32_t *>(s.bars + kPoolBars);
  s.abort_flag = reinterpret_cast<volatile int *>(s.tmem_slot + 1);
  return s;
}
__host__ __device__ constexpr uint32_t pool_smem_bytes(uint32_t bytes) { return 1024 + bytes + kPoolTailBytes; }

// Set-up of the kernels: barriers (one arrival each; two, of two loading warps, below place `two`; four, one of each warp
// of a set, from place `four` on) and TMEM.
__device__ __forceinline__ uint32_t pool_setup(const PoolSmem &s, uint32_t tmem_cols, uint32_t four, uint32_t two = 0) {
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kPoolBars; ++i) ptx::mbar_init(&s.bars[i], i < two ? 2 : i < four ? 1 : 4);
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
  return *s.tmem_slot;
}

// The wait for the kernel ahead.  The next kernel may start only after it: one that reads early, or that waits for this
// kernel alone, then finds everything before this kernel complete too.  So up and grad, which follow a kernel with this
// order in the same call, may read before their wait, through L2, all that the kernel ahead does not write (the groups,
// the pool, Y, X and dY), which hides their start behind that kernel's end; what it writes (the planes), and writes of
// their own, come after.  Where grad is ahead of up, which share nothing but what both read, up does not wait for it
// at all and fills the SMs as grad's CTAs end.  Each CTA waits before it ends, whatever it had to do.
__device__ __forceinline__ void pool_wait_ahead() {
  ptx::griddep_wait();
  ptx::griddep_launch();
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
// How both kernels below find their tiles: every thread holds some of the adapters (in order) and the number of
// tiles before them; the thread whose adapters a tile is among publishes it.
// ---------------------------------------------------------------------------
constexpr int kPoolThreads = 320;

struct PoolTile {
  int ad, lo, cnt, rank;
  float scale;
};
struct PoolWalk {
  int per, ad0;      // this thread's adapters: ad0 .. ad0 + per
  int before, sum;   // tiles before them, and theirs
  int tiles;         // of all
  int2 group0;       // what is known of ad0
  int rank0;
  float scale0;
};

__device__ __forceinline__ PoolWalk pool_walk(const PoolArgs &p, int tn, int *warp_sum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  PoolWalk w;
  w.per = (p.n + kPoolThreads - 1) / kPoolThreads;
  w.ad0 = tid * w.per;
  w.group0 = make_int2(0, 0);
  w.sum = w.rank0 = 0;
  w.scale0 = 0.0f;
  if (w.ad0 < p.n) {
    w.group0 = pool_group(p, w.ad0);
    w.rank0 = pool_rank(p, w.ad0);
    w.scale0 = __ldcg(p.scales + w.ad0);
    w.sum = (w.group0.y - w.group0.x + tn - 1) / tn;
    for (int i = 1; i < w.per && w.ad0 + i < p.n; ++i) {
      const int2 g = pool_group(p, w.ad0 + i);
      w.sum += (g.y - g.x + tn - 1) / tn;
    }
  }
  int inc = w.sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  w.before = inc - w.sum;
  w.tiles = 0;
#pragma unroll
  for (int i = 0; i < kPoolThreads / 32; ++i) {
    if (i < warp) w.before += warp_sum[i];
    w.tiles += warp_sum[i];
  }
  return w;
}

// *out = the tile (an empty one past the last); the caller synchronises.
__device__ __forceinline__ void pool_find(const PoolArgs &p, const PoolWalk &w, int tn, int tile, PoolTile *out) {
  if (tile >= w.tiles && threadIdx.x == 0) {
    out->ad = out->lo = out->cnt = out->rank = 0;
    out->scale = 0.0f;
  }
  if (tile >= w.before && tile < w.before + w.sum) {
    int2 g = w.group0;
    int ad = w.ad0, t = tile - w.before, nt;
    while (t >= (nt = (g.y - g.x + tn - 1) / tn)) {
      t -= nt;
      g = pool_group(p, ++ad);
    }
    out->ad = ad;
    out->lo = g.x + t * tn;
    out->cnt = min(tn, g.y - out->lo);
    out->rank = ad > w.ad0 ? pool_rank(p, ad) : w.rank0;
    out->scale = ad > w.ad0 ? __ldcg(p.scales + ad) : w.scale0;
  }
}

// How up to 64 token rows, four a lane of the first 16 (the others the same again), are loaded: as 64 rows from row64, or
// (row64 < 0) by masks over lanes.
struct PoolRowLoads {
  int row64;
  uint32_t runs32, runs16, gathers;
  __device__ __forceinline__ uint32_t bytes() const {  // of 64 columns
    return row64 >= 0 ? 8192u : __popc(runs32) * 4096u + __popc(runs16) * 2048u + __popc(gathers) * 512u;
  }
};
// valid: rows that exist; wanted: lanes with rows to load; loose: as pool_run.  The whole warp; writes row4.
__device__ __forceinline__ PoolRowLoads pool_row_loads(const int4 &rows, int lane, int valid, int wanted, bool loose, int4 *row4) {
  const int i = lane & 15;
  PoolRowLoads l = {-1, 0u, 0u, 0u};
  const int first = __shfl_sync(0xffffffffu, rows.x, 0);
  if (valid >= (loose ? 33 : 64)) {  // the same for the whole warp, as are the ballots' results
    const int base = first + 4 * i, left = valid - 4 * i;
    if (__all_sync(0xffffffffu, (rows.x == base || left < 1) && (rows.y == base + 1 || left < 2) &&
                                    (rows.z == base + 2 || left < 3) && (rows.w == base + 3 || left < 4))) {
      l.row64 = first;
      return l;
    }
  }
  const bool run32 = pool_run<32>(rows, lane, 4 * i, valid, loose);
  bool run16 = pool_run<16>(rows, lane, 4 * i, valid, loose);  // outside any condition: the whole warp takes part
  run16 = run16 && !run32;
  l.runs32 = __ballot_sync(0xffffffffu, run32 && (i & 7) == 0 && i < wanted) & 0xffffu;
  l.runs16 = __ballot_sync(0xffffffffu, run16 && (i & 3) == 0 && i < wanted) & 0xffffu;
  l.gathers = __ballot_sync(0xffffffffu, !run32 && !run16 && i < wanted) & 0xffffu;
  if (lane < 16) row4[lane] = rows;
  __syncwarp();
  return l;
}
// One thread: columns [x, x + 64) of the rows, moved down by `down` rows, to dst.
__device__ __forceinline__ void pool_load_parts(const PoolRowLoads &l, const int4 *row4, uint8_t *dst, const PoolMaps *maps,
                                                uint64_t *bar, int x, int down) {
  for (uint32_t m = l.runs32; m; m &= m - 1) {
    const int i = __ffs(m) - 1;
    ptx::tma_load_2d(dst + i * 512, &maps->row32, bar, x, row4[i].x + down);
  }
  for (uint32_t m = l.runs16; m; m &= m - 1) {
    const int i = __ffs(m) - 1;
    ptx::tma_load_2d(dst + i * 512, &maps->row16, bar, x, row4[i].x + down);
  }
  for (uint32_t m = l.gathers; m; m &= m - 1) {
    const int i = __ffs(m) - 1;
    const int4 y = row4[i];
    ptx::tma_gather4(dst + i * 512, &maps->row, bar, x, make_int4(y.x + down, y.y + down, y.z + down, y.w + down));
  }
}
__device__ __forceinline__ void pool_load_rows(const PoolRowLoads &l, const int4 *row4, uint8_t *dst, const PoolMaps *maps,
                                               uint64_t *bar, int x) {
  if (l.row64 >= 0)
    ptx::tma_load_2d(dst, &maps->row64, bar, x, l.row64);
  else
    pool_load_parts(l, row4, dst, maps, bar, x, 0);
}
// The same of the planes [3, M, r], `pitch` bytes from one to the next.
__device__ __forceinline__ void pool_load_planes(const PoolRowLoads &l, const int4 *row4, uint8_t *dst, const PoolMaps *maps,
                                                 uint64_t *bar, int x, int planes, int M, uint32_t pitch) {
  if (l.row64 >= 0)
    ptx::tma_load_3d(dst, &maps->row64, bar, x, l.row64, 0);  // pitch: 8192
  else
    for (int pl = 0; pl < planes; ++pl) pool_load_parts(l, row4, dst + pl * pitch, maps, bar, x, pl * M);
}
// The same of a tile of up to 64 tokens.
__device__ __forceinline__ PoolRowLoads pool_tile_loads(const PoolArgs &p, const PoolTile &t, int lane, int4 *row4) {
  const int4 rows = t.cnt > 0 ? pool_rows(p, pool_entries(p, t.lo + 4 * (lane & 15), t.lo + t.cnt - 1)) : make_int4(0, 0, 0, 0);
  return pool_row_loads(rows, lane, t.cnt, (t.cnt + 3) / 4, true, row4);
}

// Descriptor words (128-byte swizzle, groups of eight rows 1024 bytes apart): the high one is the same for all operands,
// the low one is the address and the distance of 64-element blocks, which MN-major operands use (8192 bytes); 16
// elements on, a K-major operand is 32 bytes away and an MN-major one 2048.
constexpr uint32_t kPoolDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__host__ __device__ constexpr uint32_t pool_desc_lbo(bool mn) { return mn ? ((8192u >> 4) - (16u >> 4)) << 16 : 0u; }
__host__ __device__ constexpr uint32_t pool_desc_16(bool mn) { return mn ? 128u : 2u; }

// ---------------------------------------------------------------------------
// down: g CTAs of a cluster take a tile of 64 tokens (32 above rank 128) and sum a part of the long dimension each,
// with the accumulator's rows as ranks and its columns as tokens.  The steps of 64 go round four accumulators, which
// keeps each one's chain of float32 additions short (the tensor cores' additions cut off: one chain over 1400 elements
// was 3e-6 off, all to one side); after kPoolDownFold steps they are added to the partial sums and start anew.  Each CTA
// leaves its float32 partial sums in shared memory; each then adds up a share of the tokens over the g CTAs, in CTA
// order, through distributed shared memory, and writes the planes: no partial planes in HBM, no further launch, and the
// same bits every time.  g, a divisor of the cluster, follows on the device from the number of tiles.
//   warp 0  loads V; warp 2 W (one thread that loaded both bounded the kernel: 480 cycles a step); warp 1  products;
//   warps 2..9  accumulators -> shared memory; all  the sums
// A launch has one or two sums to do (a backward whose T was not kept does U and T, which saves a launch that would wait
// for the other's last tiles); each has clusters of its own.
// mn false: W is [n][r][len], K-major (T: A); true: [n][len][r], MN-major (U: B).
// ---------------------------------------------------------------------------
constexpr uint32_t kPoolDownTmem = 256;
// Steps of 64 until the accumulators start anew: chains of 64 additions.  U summed by one CTA over 11008 elements put dA
// 1.7e-6 further off before, and T over 20008 was 5.4e-6 off; such calls take as long as before within 1% (8192 tokens of
// 11008 x 4096, one adapter, backward 216 us, forward of 22016 -> 8192 186).
constexpr int kPoolDownFold = 64;
// Shared memory: two CTAs an SM, or all of it for one.
constexpr uint32_t kPoolHalfBytes = 107 * 1024, kPoolFullBytes = 218 * 1024;

struct PoolDownLayout {
  int tn;        // tokens a tile
  int rpad;      // floats a token of the partial sums
  uint32_t stage, stages, exch_at, bytes;
};
// Two CTAs an SM up to rank 128; above it a stage is 36 KB and needs all of the shared memory.  (A ring twice as deep in
// calls too small for two CTAs an SM was no faster: 8 tokens 13.0 against 13.1 us, 16 tokens 16.3 against 15.1.)
__host__ __device__ constexpr PoolDownLayout pool_down_layout(int r) {
  PoolDownLayout l{};
  l.tn = r <= 128 ? 64 : 32;
  l.rpad = r <= 64 ? 64 : r <= 128 ? 128 : 256;
  l.stage = l.tn * 128u + l.rpad * 128u;  // token rows, then W's
  const uint32_t exch = l.tn * l.rpad * 4u;
  const uint32_t fit = ((r <= 128 ? kPoolHalfBytes : kPoolFullBytes) - exch) / l.stage;
  l.stages = fit < kPoolMostStages ? fit : kPoolMostStages;
  l.exch_at = l.stages * l.stage;
  l.bytes = l.exch_at + exch;
  return l;
}
static_assert(pool_down_layout(64).stages >= 3 && pool_down_layout(128).stages >= 3 && pool_down_layout(256).stages >= 3,
              "a ring of three stages at least");

struct PoolDownJob {
  CUtensorMap W;
  PoolMaps V;
  int64_t len;       // columns of V
  __nv_bfloat16 *P;  // [3, M, r]
  int first, clusters;  // its clusters
  bool mn;
};
struct PoolDownArgs {
  PoolDownJob job[2];
  PoolArgs p;
  PoolDownLayout l;
};

// What plane h leaves of x.  An infinity is all in the first plane: inf - inf would make the others, and so every result, NaN.
__device__ __forceinline__ float pool_rest(float x, float h, bool first) {
  return first && fabsf(h) == __int_as_float(0x7f800000) ? 0.0f : x - h;
}

// kSums: T, U, or both (found at run time, they cost a call with one token 0.9 us of 12.8).
enum PoolSums { kPoolT, kPoolU, kPoolBoth };
// kFold: a CTA may have more than kPoolDownFold steps.
template <PoolSums kSums, bool kFold>
__global__ void __launch_bounds__(kPoolThreads, 2) pool_down_kernel(const __grid_constant__ PoolDownArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int4 row4[16];
  __shared__ int warp_sum[kPoolThreads / 32];
  __shared__ PoolTile tile_s;
  const int cluster = static_cast<int>(ptx::cluster_nctarank()), crank = static_cast<int>(ptx::cluster_ctarank());
  const PoolDownJob &job = a.job[kSums == kPoolBoth && blockIdx.x / cluster >= a.job[0].clusters];
  const int grid = kSums == kPoolBoth ? job.clusters * cluster : gridDim.x;
  const int bid = kSums == kPoolBoth ? blockIdx.x - job.first * cluster : blockIdx.x;
  const bool mn = kSums == kPoolBoth ? job.mn : kSums == kPoolU;
  const PoolArgs &p = a.p;
  const PoolDownLayout &l = a.l;
  const PoolSmem sm = pool_smem(pool_raw, l.bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tn = l.tn;
  const uint32_t stages = l.stages, v_bytes = tn * 128u;
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *sum_full = sm.bars + 2 * kPoolMostStages;
  float *exch = reinterpret_cast<float *>(sm.buf + l.exch_at);
  if (tid < 5) ptx::prefetch_tmap(tid == 0 ? &job.W : tid == 1 ? &job.V.row : tid == 2 ? &job.V.row16 : tid == 3 ? &job.V.row32 : &job.V.row64);
  uint64_t *sum_empty0 = sum_full + 1, *sum_empty1 = sum_full + 2;  // from the two sets of four warps
  const uint32_t tmem = pool_setup(sm, kPoolDownTmem, 2 * kPoolMostStages + 1, kPoolMostStages);
  pool_wait_ahead();
  const PoolWalk walk = pool_walk(p, tn, warp_sum);
  // a tile is shared by g CTAs of the cluster: the largest divisor with which all tiles are at work at once
  int g = cluster;
  while (g > 1 && (static_cast<int64_t>(walk.tiles) * g > grid || cluster % g)) --g;
  const int q = crank % g, peers = crank - q;  // the g CTAs from rank `peers` of the cluster
  const int k_steps = static_cast<int>((job.len + 63) / 64), k_per = (k_steps + g - 1) / g;
  const int nrb = (p.r + 127) / 128, acc_cols = tn * nrb;  // one of the four accumulators
  RingPos pos;
  uint32_t sum_phase = 0, issued = 0;
  bool ok = true;
  // all CTAs of a cluster walk as long as the first of its tiles exists
  for (int lead = (bid - crank) / g; lead < walk.tiles; lead += grid / g) {
    pool_find(p, walk, tn, lead + crank / g, &tile_s);
    __syncthreads();
    const int ad = tile_s.ad, lo = tile_s.lo, cnt = tile_s.cnt, rank = tile_s.rank;
    const int kb = rank > 0 ? min(q * k_per, k_steps) : 0, ke = rank > 0 ? min(k_steps, kb + k_per) : 0;
    const uint32_t idesc = ptx::idesc_bf16(128, (cnt + 15) / 16 * 16, mn ? 1 : 0, 0);
    if (warp == 0) {
      const PoolRowLoads rows = pool_tile_loads(p, tile_s, lane, row4);
      const bool one = ptx::elect_one();  // the whole warp, whatever a lane's own `ok`
      if (ok && one) {
        const uint32_t bytes = rows.bytes();
        for (int ks = kb; ks < ke; ++ks) {
          // (a wait takes 140 cycles even where it is over: none for the first filling of the ring)
          if (issued >= stages && !ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(&full[pos.s], bytes);
          pool_load_rows(rows, row4, sm.buf + pos.s * l.stage, &job.V, &full[pos.s], ks * 64);
          ++issued;
          pos.next(stages);
        }
        if (!ok) pool_fail(sm, p.status);
      }
      ok = __all_sync(0xffffffffu, ok);  // for all lanes, so that the warp stays together
    } else if (warp == 1) {
      const bool one = ptx::elect_one();
      if (ok && one) {
        const uint32_t w_lbo = pool_desc_lbo(mn), w_16 = pool_desc_16(mn);
        const uint32_t v_lo = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024));
        for (int ks = kb; ks < ke; ++ks) {
          const int in_part = kFold ? (ks - kb) % kPoolDownFold : ks - kb;
          if (kFold && in_part == 0 && ks > kb) {
            ptx::mma_commit(sum_full);
            if (!ptx::mbar_wait(sum_empty0, sum_phase, sm.abort_flag) || !ptx::mbar_wait(sum_empty1, sum_phase, sm.abort_flag)) {
              ok = false;
              break;
            }
            sum_phase ^= 1;
          }
          if (!ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t v = v_lo + pos.s * (l.stage >> 4), w = v + (v_bytes >> 4) + w_lbo, d = tmem + (in_part & 3) * acc_cols;
          const uint32_t more = in_part >= 4 ? 1u : 0u;
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            ptx::mma_bf16_lohi(d, w + k16 * w_16, kPoolDescHi, v + k16 * 2, kPoolDescHi, idesc, k16 ? 1u : more);
          if (nrb > 1) {  // ranks 128 and up
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16)
              ptx::mma_bf16_lohi(d + tn, w + 1024 + k16 * w_16, kPoolDescHi, v + k16 * 2, kPoolDescHi, idesc, k16 ? 1u : more);
          }
          ptx::mma_commit(&empty[pos.s]);
          pos.next(stages);
        }
        if (ok && ke > kb) ptx::mma_commit(sum_full);
        if (!ok) pool_fail(sm, p.status);
      }
      ok = __all_sync(0xffffffffu, ok);
    } else {
      const int quad = warp & 3, set = (warp - 2) >> 2;
      // a part at a time: W's loads for it, then its accumulators
      for (int part = kb;; part += kPoolDownFold) {
        const int end = kFold ? min(ke, part + kPoolDownFold) : ke;
        if (warp == 2) {
          const bool one = ptx::elect_one();
          if (ok && one) {
            // W's ranks [0, min(r, 256)): K-major in boxes of up to 128 rows, MN-major in boxes of 64 ranks
            const int w_loads = mn ? (p.r + 63) / 64 : nrb;
            const uint32_t bytes = w_loads * (mn ? 8192u : static_cast<uint32_t>(min(p.r, 128)) * 128u);
            for (int ks = kFold ? part : kb; ks < end; ++ks) {
              if (issued >= stages && !ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag)) { ok = false; break; }
              uint8_t *st = sm.buf + pos.s * l.stage + v_bytes;
              uint64_t *bar = &full[pos.s];
              ptx::mbar_arrive_expect_tx(bar, bytes);
              for (int i = 0; i < w_loads; ++i)
                ptx::tma_load_3d(st + i * (mn ? 8192 : 16384), &job.W, bar, mn ? i * 64 : ks * 64, mn ? ks * 64 : i * 128, ad);
              ++issued;
              pos.next(stages);
            }
            if (!ok) pool_fail(sm, p.status);
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        if (ke > kb && ok) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(sum_full, sum_phase, sm.abort_flag));
          sum_phase ^= 1;
          if (!ok && lane == 0) pool_fail(sm, p.status);
        }
        ptx::tc_fence_after();
        int rpad = l.rpad;
        asm volatile("" : "+r"(rpad));  // in a register: read again as a parameter, each store took 60 ns
        const int nacc = ok ? min(4, end - (kFold ? part : kb)) : 0, c_end = min(cnt, (set + 1) * (tn / 2));
        for (int rb = 0; rb < nrb; ++rb) {
          if (rb * 128 + quad * 32 >= p.r) break;
          for (int c0 = set * (tn / 2); c0 < c_end; c0 += 16) {
            const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + rb * tn + c0;
            float *to = exch + c0 * rpad + rb * 128 + quad * 32 + lane;
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
            if (kFold && part > kb) {
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] += to[j * rpad];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) to[j * rpad] = x[j];  // up to 15 that are not tokens: not read
          }
        }
        ptx::tc_fence_before();
        if (!kFold || end >= ke || !ok) break;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(set ? sum_empty1 : sum_empty0);
      }
    }

    pool_cluster_sync();
    // this CTA's share of the tokens, four ranks a thread
    {
      const int pt = (cnt + g - 1) / g, c_lo = min(cnt, q * pt), c_hi = min(cnt, c_lo + pt), n4 = p.r / 4;
      const uint32_t exch_addr = ptx::smem_addr(exch);
      for (int e = tid; e < (c_hi - c_lo) * n4; e += kPoolThreads) {
        const int c = c_lo + e / n4, j = e % n4 * 4;
        const int t = pool_token(p, lo + c);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < rank) {
          const uint32_t src = exch_addr + (c * l.rpad + j) * 4;
          float4 u[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < g) u[r] = ptx::ld_cluster_f32x4(ptx::mapa_shared(src, peers + r));
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < g) { x.x += u[r].x; x.y += u[r].y; x.z += u[r].z; x.w += u[r].w; }
        }
        if (t < 0) continue;
        __nv_bfloat16 *out = job.P + static_cast<int64_t>(t) * p.r + j;
#pragma unroll
        for (int pl = 0; pl < kPoolPlanes; ++pl) {
          const uint2 h = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
          x.x = pool_rest(x.x, bf16lo_to_f32(h.x), pl == 0);
          x.y = pool_rest(x.y, bf16hi_to_f32(h.x), pl == 0);
          x.z = pool_rest(x.z, bf16lo_to_f32(h.y), pl == 0);
          x.w = pool_rest(x.w, bf16hi_to_f32(h.y), pl == 0);
          *reinterpret_cast<uint2 *>(out + pl * p.M * p.r) = h;
        }
      }
    }
    pool_cluster_sync();  // the partial sums, and the tile, are done with
  }
  if (issued && *sm.abort_flag) ring_drain(full, pos, stages, issued);  // the threads that load
  pool_teardown(tmem, kPoolDownTmem);
}

// ---------------------------------------------------------------------------
// up: one unit is a tile of 64 tokens (32 where the planes are many) and every runs-th block of 128 features.  P's rows
// come once, W's blocks stream through the ring, rows of the accumulator are features.  Two sets of four epilogue warps
// take turns with the blocks, each with two of four accumulators: while one is added to Out, the next is multiplied.
// The lanes hold features; where Out's rows are 16-byte aligned, 16 tokens at a time pass through shared memory, so that
// four lanes (bf16; eight for float32) then share a token's 32 features in 16-byte pieces (element by element the
// epilogue took 47 instructions an element and warp, and bound the kernel on issue).  The pieces are loaded an item
// ahead, and the lines of the next block are prefetched to L2 (203 -> 172 us for 4096 tokens on 22016 float32 columns).
// Tiles of up to four tokens go straight from the accumulator to Out (32 decode tokens 16.8 -> 16.3 us), and other outputs,
// odd strides or columns of a wider tensor, element by element.
//   warp 0  loads; warp 1  products; warps 2..9  Out += s accumulator
// W_MN false: W is [n][cols][r], K-major (Y: B); true: [n][r][cols], MN-major (dX: A).
// ---------------------------------------------------------------------------
constexpr uint32_t kPoolUpTmem = 256;
// Shared memory of a warp's 16 tokens x 32 features: a pitch of 36 floats keeps 16-byte pieces aligned and both
// directions without bank conflicts.
constexpr int kPoolPitch = 36, kPoolWarpBuf = 16 * kPoolPitch;
constexpr uint32_t kPoolUpStage = 16384;  // 128 features x 64 ranks

struct PoolUpLayout {
  int tn;          // tokens a tile
  uint32_t plane;  // bytes of one 64-rank chunk of one plane
  uint32_t stages, planes_at, buf_at, bytes;
};
__host__ __device__ constexpr PoolUpLayout pool_up_layout(int r, int planes) {
  PoolUpLayout l{};
  const int chunks = (r + 63) / 64 * planes;
  l.tn = chunks <= 6 ? 64 : 32;
  l.plane = l.tn * 128u;
  const uint32_t rest = chunks * l.plane + 8 * kPoolWarpBuf * 4u;
  l.stages = (kPoolHalfBytes - rest) / kPoolUpStage;
  l.planes_at = l.stages * kPoolUpStage;
  l.buf_at = l.planes_at + chunks * l.plane;
  l.bytes = l.planes_at + rest;
  return l;
}
static_assert(pool_up_layout(64, 3).stages >= 3 && pool_up_layout(128, 3).stages >= 2 && pool_up_layout(256, 3).stages >= 2 &&
                  pool_up_layout(64, 2).stages <= kPoolMostStages,
              "a ring of two stages at least");
static_assert(pool_smem_bytes(kPoolHalfBytes) + 2048 <= 114 * 1024 && pool_smem_bytes(kPoolFullBytes) <= 225 * 1024, "shared memory");

struct PoolUpArgs {
  PoolArgs p;
  int64_t cols, ldo;  // of Out
  void *out;
  int planes;
  bool after_down;  // the kernel ahead writes P; else it is grad, which has waited for the one that did
  PoolUpLayout l;
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

template <bool W_MN, typename O, bool VEC>
__global__ void __launch_bounds__(kPoolThreads, 2) pool_up_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                  const __grid_constant__ PoolMaps tmP, const PoolUpArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int64_t row_at[64];  // of the tile's tokens in Out, in elements; -1: not a token
  __shared__ int4 row4[16];
  __shared__ int warp_sum[kPoolThreads / 32];
  __shared__ PoolTile tile_s;
  constexpr uint32_t kWLbo = pool_desc_lbo(W_MN), kW16 = pool_desc_16(W_MN);
  const PoolArgs &p = a.p;
  const PoolUpLayout &l = a.l;
  const PoolSmem sm = pool_smem(pool_raw, l.bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tn = l.tn;
  const uint32_t stages = l.stages;
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *p_full = sm.bars + 2 * kPoolMostStages;
  uint64_t *acc_full = p_full + 1, *acc_empty = acc_full + 4;
  if (tid < 5) ptx::prefetch_tmap(tid == 0 ? &tmW : tid == 1 ? &tmP.row : tid == 2 ? &tmP.row16 : tid == 3 ? &tmP.row32 : &tmP.row64);
  const uint32_t tmem = pool_setup(sm, kPoolUpTmem, 2 * kPoolMostStages + 5);
  const PoolWalk walk = pool_walk(p, tn, warp_sum);
  // runs of blocks a tile: as many as give every CTA a unit
  const int nblk = static_cast<int>((a.cols + 127) / 128);
  const int g = min(max(static_cast<int>(gridDim.x) / max(walk.tiles, 1), 1), nblk);
  const int64_t units = static_cast<int64_t>(walk.tiles) * g;
  RingPos pos;
  uint32_t p_phase = 0, issued = 0, blocks = 0;  // blocks: accumulators used so far
  bool ok = true;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = static_cast<int>(u / g), q = static_cast<int>(u - static_cast<int64_t>(tile) * g);
    pool_find(p, walk, tn, tile, &tile_s);
    __syncthreads();
    const int ad = tile_s.ad, lo = tile_s.lo, cnt = tile_s.cnt, rank = tile_s.rank;
    const int nch = (rank + 63) / 64;
    const int mine = rank > 0 ? (nblk - q + g - 1) / g : 0;  // blocks q, q + g, ...
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

    if (warp == 0) {
      const PoolRowLoads rows = pool_tile_loads(p, tile_s, lane, row4);
      const bool one = ptx::elect_one();
      if (ok && mine > 0 && one) {
        // the first blocks of W, then P's rows, then the other blocks
        int b = 0, ch = 0;
        for (int i = 0; i < mine * nch; ++i) {
          if (i == min(static_cast<int>(stages), mine * nch) - 1) {
            if (a.after_down && issued < stages) pool_wait_ahead();  // the first unit's
            ptx::mbar_arrive_expect_tx(p_full, nch * a.planes * rows.bytes());
            for (int c = 0; c < nch; ++c)
              pool_load_planes(rows, row4, sm.buf + l.planes_at + c * a.planes * l.plane, &tmP, p_full, c * 64, a.planes,
                               static_cast<int>(p.M), l.plane);
          }
          if (issued >= stages && !ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag)) { ok = false; break; }
          const int f = (q + b * g) * 128, x = ch * 64;
          uint8_t *st = sm.buf + pos.s * kPoolUpStage;
          ptx::mbar_arrive_expect_tx(&full[pos.s], kPoolUpStage);
          if (W_MN) {
            ptx::tma_load_3d(st, &tmW, &full[pos.s], f, x, ad);
            ptx::tma_load_3d(st + 8192, &tmW, &full[pos.s], f + 64, x, ad);
          } else {
            ptx::tma_load_3d(st, &tmW, &full[pos.s], x, f, ad);
          }
          if (++ch == nch) { ch = 0; ++b; }
          ++issued;
          pos.next(stages);
        }
        if (!ok) pool_fail(sm, p.status);
      }
      ok = __all_sync(0xffffffffu, ok);
    } else if (warp == 1) {
      if (mine > 0 && ok) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(p_full, p_phase, sm.abort_flag));
        if (!ok && lane == 0) pool_fail(sm, p.status);
      }
      const uint32_t p_lo = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024));
      // one thread issues a chunk of a block's products
      auto issue = [&](uint32_t acc, int ch) {
        ptx::tc_fence_after();
        const int left = min(64, rank - ch * 64);  // a multiple of 8; products go 16 ranks at a time
        const uint32_t w = p_lo + pos.s * (kPoolUpStage >> 4) + kWLbo, pc = p_lo + ((l.planes_at + ch * a.planes * l.plane) >> 4);
#pragma unroll
        for (int k16 = 0; k16 < 4; ++k16) {
          if (k16 * 16 >= left) break;
#pragma unroll
          for (int pl = 0; pl < kPoolPlanes; ++pl)
            if (pl < a.planes)
              ptx::mma_bf16_lohi(tmem + acc * 64, w + k16 * kW16, kPoolDescHi, pc + pl * (l.plane >> 4) + k16 * 2, kPoolDescHi, idesc,
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
        ok = __all_sync(0xffffffffu, ok);
      } else {
        // The 8 ranks past the adapter's meet zeros in P and have to be finite: the warp clears them in each last chunk.
        const int leader = __ffs(__ballot_sync(0xffffffffu, one)) - 1;
        pos.s = __shfl_sync(0xffffffffu, pos.s, leader);
        pos.ph = __shfl_sync(0xffffffffu, pos.ph, leader);
        for (int b = 0; b < mine && ok; ++b) {
          const uint32_t n = blocks + b, acc = n & 3;
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_empty[acc], ((n >> 2) & 1) ^ 1, sm.abort_flag));
          for (int ch = 0; ch < nch && ok; ++ch) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
            if (!ok) break;
            if (ch == nch - 1) {
              uint8_t *st = sm.buf + pos.s * kPoolUpStage;
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
      if (tid - 64 < tn) {
        const int t = tid - 64 < cnt ? pool_token(p, lo + tid - 64) : -1;
        row_at[tid - 64] = t < 0 ? -1 : t * a.ldo;
      }
      ptx::named_bar_sync(1, kPoolThreads - 64);
      if (pieces && b_first < mine) {  // the first ones', while the products are formed
        load_y(y0, b_first, 0);
        prefetch_block(b_first);
      }
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
        float *buf = reinterpret_cast<float *>(sm.buf + l.buf_at) + (warp - 2) * kPoolWarpBuf;
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
            __syncwarp();
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
    if (mine > 0) p_phase ^= 1;
    blocks += mine;
    __syncthreads();  // the tile's tokens and planes are done with
  }
  if (issued && *sm.abort_flag) {  // the thread that loads
    ring_drain(full, pos, stages, issued);
    ptx::mbar_wait(p_full, p_phase ^ 1, nullptr);
  }
  pool_wait_ahead();
  pool_teardown(tmem, kPoolUpTmem);
}

// ---------------------------------------------------------------------------
// grad: one unit is 128 features x 64 ranks of one adapter's dA or dB, summed over its tokens.  Both operands come as
// token rows (MN-major), 64 tokens a step.  The first plane's products go round three accumulators and the other
// planes' into a fourth; after kPoolGradFold steps the epilogue adds them to float32 sums in its registers and they start
// anew.  Both keep an accumulator's chain of additions short: the tensor cores cut off where a float32 addition rounds,
// which put a sum off by 2e-8 of itself for each addition in a chain.  While one unit is stored the next one's tokens are
// loaded.  Units are taken longest adapter first, back and forth over the CTAs, so that long and short ones
// meet: a CTA has one or two, and their lengths differ.  An adapter without tokens gets zeros.
//   warp 0  loads; warp 1  products; warps 2..9  accumulators -> dA or dB
// ---------------------------------------------------------------------------
constexpr uint32_t kPoolGradTmem = 256;
// Steps of 64 tokens until the accumulators start anew: chains of 60 additions.  One adapter, float32, error of dB: 8192
// tokens 3.7e-6 -> 1.8e-6, 65536 2.6e-5 -> 1.8e-6; 16384 tokens of 11008 x 4096 take 420 us instead of 414.
constexpr int kPoolGradFold = 45;

struct PoolGradArgs {
  PoolArgs p;
  void *dA, *dB;  // [n, r, K], [n, N, r]
  int planes;
  uint32_t stages, bytes;
};
// Shared memory: the ring, then of each adapter the places of its tokens and the adapters by length.
__host__ __device__ constexpr uint32_t pool_grad_stage(int planes) { return 16384u + planes * 8192u; }
__host__ __device__ constexpr uint32_t pool_grad_lists(int n) { return (static_cast<uint32_t>(n) * 12u + 15u) & ~15u; }
__host__ __device__ constexpr uint32_t pool_grad_stages(int planes, int n) {
  return (kPoolHalfBytes - pool_grad_lists(n)) / pool_grad_stage(planes);
}
__host__ __device__ constexpr uint32_t pool_grad_bytes(int planes, int n) {
  return pool_grad_stages(planes, n) * pool_grad_stage(planes) + pool_grad_lists(n);  // barriers follow: 16-byte aligned
}
static_assert(pool_grad_bytes(3, 1) % 16 == 0 && pool_grad_bytes(2, 7) % 16 == 0, "the barriers' alignment");
static_assert(pool_grad_stages(3, QLORA_MAX_ADAPTERS) >= 2 && pool_grad_stages(2, 1) <= kPoolMostStages, "a ring of two stages at least");

struct PoolGradUnit {
  int ad, lo, cnt, live, fb, rb;
  bool is_a;
};

// sum += 16 columns of the accumulators of `steps` steps (those that took part): three at 0, 64 and 128 with the first
// plane's products, and the other planes' at 192.
__device__ __forceinline__ void pool_add_accumulators(uint32_t from, int steps, float *sum) {
  uint32_t v[16], w[16];
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (steps > 1) {
    ptx::tmem_ld16(from + 64, v);
    if (steps > 2) ptx::tmem_ld16(from + 128, w);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]) + (steps > 2 ? __uint_as_float(w[i]) : 0.0f);
  }
  ptx::tmem_ld16(from, v);
  ptx::tmem_ld16(from + 192, w);
  ptx::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] += (__uint_as_float(v[i]) + x[i]) + __uint_as_float(w[i]);
}

// kFold: a unit may have more than kPoolGradFold steps.
template <typename O, bool kFold>
__global__ void __launch_bounds__(kPoolThreads, 2)
    pool_grad_kernel(const __grid_constant__ PoolMaps tmX, const __grid_constant__ PoolMaps tmU,
                     const __grid_constant__ PoolMaps tmDY, const __grid_constant__ PoolMaps tmT, const PoolGradArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int4 row4[16];
  const PoolSmem sm = pool_smem(pool_raw, a.bytes);
  const PoolArgs &p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage_bytes = pool_grad_stage(a.planes), stages = a.stages;
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *acc_full = sm.bars + 2 * kPoolMostStages;
  uint64_t *acc_empty0 = acc_full + 1, *acc_empty1 = acc_full + 2;  // from the two sets of four warps
  int2 *group = reinterpret_cast<int2 *>(sm.buf + stages * stage_bytes);
  int *by_length = reinterpret_cast<int *>(group + p.n);
  const uint32_t tmem = pool_setup(sm, kPoolGradTmem, 2 * kPoolMostStages + 1);
  for (int i = tid; i < p.n; i += kPoolThreads) group[i] = pool_group(p, i);
  __syncthreads();
  for (int i = tid; i < p.n; i += kPoolThreads) {
    // its place among the adapters, the longest first (more of them than threads: in their own order)
    int place = i;
    if (p.n <= kPoolThreads) {
      const int mine = group[i].y - group[i].x;
      place = 0;
      for (int k = 0; k < p.n; ++k) {
        const int len = group[k].y - group[k].x;
        place += len > mine || (len == mine && k < i);
      }
    }
    by_length[place] = i;
  }
  __syncthreads();
  const int nrb = (p.r + 63) / 64;
  const int in_a = static_cast<int>((p.K + 127) / 128) * nrb, per_adapter = in_a + static_cast<int>((p.N + 127) / 128) * nrb;
  const int64_t units = static_cast<int64_t>(p.n) * per_adapter;
  const int G = gridDim.x;
  // the unit of this CTA in a round; false if the round has none for it
  auto unit_of = [&](int64_t round, PoolGradUnit &u) {
    const int64_t i = round * G + (round & 1 ? G - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
    if (i >= units) return false;
    const int at = static_cast<int>(i / per_adapter);
    int w = static_cast<int>(i - static_cast<int64_t>(at) * per_adapter);
    u.ad = by_length[at];
    u.is_a = w < in_a;
    if (!u.is_a) w -= in_a;
    u.fb = w / nrb;
    u.rb = w - u.fb * nrb;
    u.lo = group[u.ad].x;
    u.cnt = group[u.ad].y - u.lo;
    u.live = pool_rank(p, u.ad) - u.rb * 64;
    return true;
  };
  RingPos pos;
  uint32_t issued = 0, acc_phase = 0;
  bool ok = true;
  const int64_t rounds = (units + G - 1) / G;
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    // in registers: read again as parameters at each use, they took part of this thread's time, which bounds a step
    int planes = a.planes, m = static_cast<int>(p.M);
    uint32_t sbytes = stage_bytes, nst = stages;
    asm volatile("" : "+r"(planes), "+r"(m), "+r"(sbytes), "+r"(nst));
    for (int64_t round = 0; round < rounds && ok; ++round) {
      PoolGradUnit u;
      if (!unit_of(round, u) || u.live <= 0 || u.cnt == 0) continue;
      const PoolMaps *tmV = u.is_a ? &tmX : &tmDY, *tmP = u.is_a ? &tmU : &tmT;
      const int g = lane & 15, last = u.lo + u.cnt - 1;
      int4 entries = pool_entries(p, u.lo + 4 * g, last);
      for (int t0 = 0; t0 < u.cnt && ok; t0 += 64) {
        const int left = u.cnt - t0, groups = (min(64, left) + 15) / 16 * 4;  // whole steps of 16 tokens
        // a run that is not whole is gathered: rows of other adapters' tokens must not meet the padding
        const PoolRowLoads loads = pool_row_loads(pool_rows(p, entries), lane, left, groups, false, row4);
        if (t0 + 64 < u.cnt) entries = pool_entries(p, u.lo + t0 + 64 + 4 * g, last);
        __syncwarp();
        if (ptx::elect_one()) {
          ok = ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag);
          if (ok) {
            uint8_t *d = sm.buf + pos.s * sbytes;
            ptx::mbar_arrive_expect_tx(&full[pos.s], loads.bytes() * (2 + planes));
            pool_load_rows(loads, row4, d, tmV, &full[pos.s], u.fb * 128);
            pool_load_rows(loads, row4, d + 8192, tmV, &full[pos.s], u.fb * 128 + 64);
            if (issued == 0) pool_wait_ahead();
            pool_load_planes(loads, row4, d + 16384, tmP, &full[pos.s], u.rb * 64, planes, m, 8192);
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        pos.next(nst);
      }
    }
    if (!ok && lane == 0) pool_fail(sm, p.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    const uint32_t idesc = ptx::idesc_bf16(128, 64, 1, 1);
    constexpr uint32_t kLbo = pool_desc_lbo(true), k16s = pool_desc_16(true);
    const uint32_t base = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024)) + kLbo;
    const bool one = ptx::elect_one();
    for (int64_t round = 0; round < rounds && ok; ++round) {
      PoolGradUnit u;
      if (!unit_of(round, u) || u.live <= 0 || u.cnt == 0) continue;
      for (int part = 0; part < u.cnt && ok; part += kPoolGradFold * 64) {
        const int end = kFold ? min(u.cnt, part + kPoolGradFold * 64) : u.cnt;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_empty0, acc_phase ^ 1, sm.abort_flag) &&
                                         ptx::mbar_wait(acc_empty1, acc_phase ^ 1, sm.abort_flag));
        acc_phase ^= 1;
        uint32_t turn = 0, used = 0;
        for (int t0 = kFold ? part : 0; t0 < end && ok; t0 += 64) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[pos.s], pos.ph, sm.abort_flag));
          if (!ok) break;
          const int valid = min(64, u.cnt - t0);
          if (valid & 15) {
            // the last 16 tokens are not all there: zero rows of P meet repeated rows of V
            uint8_t *d = sm.buf + pos.s * stage_bytes + 16384;
            const int pad = 16 - (valid & 15);
            for (int i = lane; i < pad * 8 * a.planes; i += 32) {
              const int pl = i / (pad * 8), e = i - pl * pad * 8;
              *reinterpret_cast<uint4 *>(d + pl * 8192 + (valid + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          ptx::tc_fence_after();
          if (one) {
            const uint32_t v = base + pos.s * (stage_bytes >> 4), b = v + (16384 >> 4), d = tmem + turn * 64;
            const uint32_t more = used & (1u << turn) ? 1u : 0u, rest = used ? 1u : 0u;
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16) {
              if (k16 * 16 >= valid) break;
              ptx::mma_bf16_lohi(d, v + k16 * k16s, kPoolDescHi, b + k16 * k16s, kPoolDescHi, idesc, k16 ? 1u : more);
#pragma unroll
              for (int pl = 1; pl < kPoolPlanes; ++pl)
                if (pl < a.planes)
                  ptx::mma_bf16_lohi(tmem + 192, v + k16 * k16s, kPoolDescHi, b + pl * (8192 >> 4) + k16 * k16s, kPoolDescHi, idesc,
                                     (k16 || pl > 1) ? 1u : rest);
            }
            ptx::mma_commit(&empty[pos.s]);
            if (t0 + 64 >= end) ptx::mma_commit(acc_full);
          }
          __syncwarp();
          used |= 1u << turn;
          turn = turn == 2 ? 0 : turn + 1;
          pos.next(stages);
        }
        if (!kFold) break;
      }
    }
    if (!ok && lane == 0) pool_fail(sm, p.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ the gradients
    const int quad = warp & 3, half = (warp - 2) >> 2;
    pool_wait_ahead();  // zeros are written without a load
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 32;
    for (int64_t round = 0; round < rounds && ok; ++round) {
      PoolGradUnit u;
      if (!unit_of(round, u)) continue;
      const bool sums = u.live > 0 && u.cnt > 0;
      const int steps = (u.cnt + 63) / 64, j0 = u.rb * 64 + half * 32;  // ranks j0 .. j0 + 32
      const float s = p.scales[u.ad];
      const int64_t cols = u.is_a ? p.K : p.N, f = static_cast<int64_t>(u.fb) * 128 + quad * 32 + lane;
      auto wait = [&]() {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_full, acc_phase, sm.abort_flag));
        acc_phase ^= 1;
        if (ok) ptx::tc_fence_after();
        return ok;
      };
      auto done = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(half ? acc_empty1 : acc_empty0);
      };
      float sum[kFold ? 32 : 16];  // with one part, half of the ranks at a time, the first stored while the others are read
      if (kFold) {
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i % (kFold ? 32 : 16)] = 0.0f;
        for (int at = 0; sums && at < steps && wait(); at += kPoolGradFold) {
#pragma unroll
          for (int c = 0; c < 32; c += 16) pool_add_accumulators(from + c, steps - at, sum + (kFold ? c : 0));
          done();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i % (kFold ? 32 : 16)] = sums && half * 32 + i < u.live ? s * sum[i % (kFold ? 32 : 16)] : 0.0f;
      } else if (sums) {
        wait();
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        float *x = sum + (kFold ? c : 0);
        if (!kFold) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = 0.0f;
          if (sums) {
            pool_add_accumulators(from + c, steps, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = half * 32 + c + i < u.live ? s * x[i] : 0.0f;
          }
        }
        if (f >= cols) {
        } else if (u.is_a) {
          O *out = static_cast<O *>(a.dA) + (static_cast<int64_t>(u.ad) * p.r + j0 + c) * p.K + f;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j0 + c + i < p.r) pool_store(out + i * p.K, x[i]);
        } else {
          O *out = static_cast<O *>(a.dB) + (static_cast<int64_t>(u.ad) * p.N + f) * p.r + j0 + c;
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            if (j0 + c + i >= p.r) break;  // r is a multiple of 8
            if (sizeof(O) == 4) {
              reinterpret_cast<float4 *>(out + i)[0] = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
              reinterpret_cast<float4 *>(out + i)[1] = make_float4(x[i + 4], x[i + 5], x[i + 6], x[i + 7]);
            } else {
              *reinterpret_cast<uint4 *>(out + i) = make_uint4(pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3]),
                                                               pack_bf16x2(x[i + 4], x[i + 5]), pack_bf16x2(x[i + 6], x[i + 7]));
            }
          }
        }
        __syncwarp();
      }
      if (!kFold && sums) done();
    }
    if (!ok && lane == 0) pool_fail(sm, p.status);
  }
  if (issued && *sm.abort_flag) ring_drain(full, pos, stages, issued);  // the thread that loads
  pool_wait_ahead();
  pool_teardown(tmem, kPoolGradTmem);
}

// ---------------------------------------------------------------------------
// grad, split: the same for calls with so few units that CTAs would be idle.  The CTAs of a cluster each take a part of
// a unit's tokens, sum it in the four accumulators as grad does (in one, 131072 tokens were 5e-5 off; now 1.1e-6), and add
// up as in down.
//   warp 0  loads; warp 1  products; warps 2..5  accumulators -> shared memory; all  the sum
// ---------------------------------------------------------------------------
constexpr int kPoolGradSplitThreads = 192;
// Units of 128 features x 64 ranks of all adapters' dA and dB.
__host__ __device__ constexpr int64_t pool_grad_units(int n, int r, int64_t K, int64_t N) {
  return static_cast<int64_t>(n) * ((r + 63) / 64) * ((K + 127) / 128 + (N + 127) / 128);
}
// An adapter's tokens are split over CTAs where units are few, so that CTAs are idle, and tokens many (gradients, 16 units:
// 8192 tokens 32.2 us against 89.1 by pool_grad_kernel, 2048 19.9 against 30.1, 1024 16.8 against 20.4, but 512 15.4 against
// 15.4 and 256 14.6 against 13.1; 64 units of 512 tokens 24.9 against 17.1, of 1024 27.6 against 26.9).
__host__ __device__ constexpr bool pool_grad_splits(int64_t units, int64_t M, int n, int sms) {
  return 2 * units < sms && M >= 1024 * static_cast<int64_t>(n);
}
constexpr uint32_t kPoolGradSplitBytes = 98 * 1024;  // two CTAs share an SM

template <typename O>
__global__ void __launch_bounds__(kPoolGradSplitThreads, 2)
    pool_grad_split_kernel(const __grid_constant__ PoolMaps tmX, const __grid_constant__ PoolMaps tmU,
                           const __grid_constant__ PoolMaps tmDY, const __grid_constant__ PoolMaps tmT, const PoolGradArgs a) {
  extern __shared__ uint8_t pool_raw[];
  __shared__ int4 row4[16];
  const PoolSmem sm = pool_smem(pool_raw, kPoolGradSplitBytes);
  const PoolArgs &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = 16384u + a.planes * 8192u, stages = min(kPoolGradSplitBytes / stage_bytes, kPoolMostStages);
  uint64_t *full = sm.bars, *empty = sm.bars + kPoolMostStages, *acc_full = sm.bars + 2 * kPoolMostStages;
  uint64_t *acc_empty = acc_full + 1;  // from the four warps
  const uint32_t tmem = pool_setup(sm, kPoolGradTmem, 2 * kPoolMostStages + 1);
  pool_wait_ahead();
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
      const PoolMaps *tmV = is_a ? &tmX : &tmDY, *tmP = is_a ? &tmU : &tmT;
      const int g = lane & 15;
      int4 entries = make_int4(0, 0, 0, 0);
      if (sb < se) entries = pool_entries(p, grp.x + sb * 64 + 4 * g, grp.y - 1);
      for (int st = sb; st < se && ok; ++st) {
        const int left = cnt - st * 64, groups = (min(64, left) + 15) / 16 * 4;  // whole steps of 16 tokens
        // a run that is not whole is gathered: rows of other adapters' tokens must not meet the padding
        const PoolRowLoads loads = pool_row_loads(pool_rows(p, entries), lane, left, groups, false, row4);
        if (st + 1 < se) entries = pool_entries(p, grp.x + (st + 1) * 64 + 4 * g, grp.y - 1);
        if (ptx::elect_one()) {
          ok = ptx::mbar_wait(&empty[pos.s], pos.ph ^ 1, sm.abort_flag);
          if (ok) {
            uint8_t *d = sm.buf + pos.s * stage_bytes;
            ptx::mbar_arrive_expect_tx(&full[pos.s], loads.bytes() * (2 + a.planes));
            pool_load_rows(loads, row4, d, tmV, &full[pos.s], fb * 128);
            pool_load_rows(loads, row4, d + 8192, tmV, &full[pos.s], fb * 128 + 64);
            pool_load_planes(loads, row4, d + 16384, tmP, &full[pos.s], rb * 64, a.planes, static_cast<int>(p.M), 8192);
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        pos.next(stages);
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
    } else if (warp == 1) {
      const uint32_t idesc = ptx::idesc_bf16(128, 64, 1, 1);
      constexpr uint32_t kLbo = pool_desc_lbo(true), k16s = pool_desc_16(true);
      const uint32_t base = static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(sm.buf), 16, 1024)) + kLbo;
      uint32_t turn = 0, used = 0;
      for (int st = sb; st < se && ok; ++st) {
        const int in_part = (st - sb) % kPoolGradFold;
        if (in_part == 0) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_empty, acc_phase ^ 1, sm.abort_flag));
          if (!ok) break;
          acc_phase ^= 1;
          turn = used = 0;
        }
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
          const uint32_t v = base + pos.s * (stage_bytes >> 4), b = v + (16384 >> 4), acc = tmem + turn * 64;
          const uint32_t more = used & (1u << turn) ? 1u : 0u, rest = used ? 1u : 0u;
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16) {
            if (k16 * 16 >= valid) break;
            ptx::mma_bf16_lohi(acc, v + k16 * k16s, kPoolDescHi, b + k16 * k16s, kPoolDescHi, idesc, k16 ? 1u : more);
#pragma unroll
            for (int pl = 1; pl < kPoolPlanes; ++pl)
              if (pl < a.planes)
                ptx::mma_bf16_lohi(tmem + 192, v + k16 * k16s, kPoolDescHi, b + pl * (8192 >> 4) + k16 * k16s, kPoolDescHi, idesc,
                                   (k16 || pl > 1) ? 1u : rest);
          }
          ptx::mma_commit(&empty[pos.s]);
          if (in_part == kPoolGradFold - 1 || st + 1 == se) ptx::mma_commit(acc_full);
        }
        __syncwarp();
        used |= 1u << turn;
        turn = turn == 2 ? 0 : turn + 1;
        pos.next(stages);
      }
      if (!ok && lane == 0) pool_fail(sm, p.status);
      __syncwarp();
    } else if (steps > 0) {
      const int quad = warp & 3, f = quad * 32 + lane;
      float sum[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = 0.0f;
      for (int done = sb; done < se && ok; done += kPoolGradFold) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_full, acc_phase, sm.abort_flag));
        acc_phase ^= 1;
        if (!ok) {
          if (lane == 0) pool_fail(sm, p.status);
          break;
        }
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 16)
          pool_add_accumulators(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, se - done, sum + c);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(acc_empty);
      }
      // dA: [rank][feature], dB: [feature][rank] with a pitch that keeps pairs aligned and lanes on 16 banks
      const int pitch = is_a ? 128 : 1, lane_pitch = is_a ? 1 : 66;
#pragma unroll
      for (int j = 0; j < 64; ++j) exch[j * pitch + f * lane_pitch] = sum[j];
    }
    if (steps > 0) pool_cluster_sync();
    // this CTA's share, in pairs of consecutive elements of the output
    const float s = p.scales[ad];
    const uint32_t exch_addr = ptx::smem_addr(exch);
    const int rows = is_a ? 64 : 128, width = is_a ? 64 : 32, pitch = is_a ? 128 : 66;  // pairs a row
    const int per = (rows + cs - 1) / cs, r_lo = min(rows, q * per), r_hi = min(rows, r_lo + per);
    for (int e = threadIdx.x; e < (r_hi - r_lo) * width; e += kPoolGradSplitThreads) {
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
  if (issued && *sm.abort_flag) ring_drain(full, pos, stages, issued);  // the thread that loads
  pool_teardown(tmem, kPoolGradTmem);
}

}  // namespace qlora
