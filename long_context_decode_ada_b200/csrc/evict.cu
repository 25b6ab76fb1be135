// evict.cu -- eviction by accumulated attention weight: per (sequence, kv
// head) the sink, the recent window, the protected tokens and the highest
// scores stay resident, in their tier and with their bytes; the others are
// dropped and the kept rows packed into new tier-homogeneous pages.
//
// Three kernels.  Select: a cluster of up to 16 blocks per unit finds the cut
// by a radix select (three digits of 11, 11 and 10 bits, most significant
// first, the blocks' histograms summed over distributed shared memory), then
// ranks the kept tokens per tier in position order: tiers, row map and, per new
// row, its old row.  Up to 131072 positions a thread keeps its 8 or 16
// positions in registers from load to store; longer sequences go through
// shared memory (the 128K context to half: 107 us against 50).  Plan: one
// block turns the units' counts into the page table's offsets.  Move: the
// pages' ids and headers, and every new row's bytes from its old page.
//
// What bounds it: the move, by DRAM traffic and its latency.  The pages keep
// two rows' values in every 16 bytes, so that a kept row brings its
// neighbours' bytes along: 518 MB read and 232 MB written on the ragged batch
// (175 us, 4.3 TB/s) for some 255 MB of kept rows; at 6.5 TB/s those bytes would
// take 118 us.  The rest of its 224 us is the select, with DRAM idle (on the 128K
// context some 50 of 128).  The register selects spill 60 (8 positions a thread)
// and 128 bytes (16).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace skv {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr uint32_t kGone = 3;      // state: not resident
constexpr uint32_t kHeld = 4;      // state bit: stays whatever its score
constexpr uint32_t kStay = 8;      // state bit: stays

// Scores as unsigned integers of the same order (-0 equals +0, NaN lowest).
__device__ __forceinline__ uint32_t score_key(float x) {
  x += 0.0f;
  const uint32_t b = __float_as_uint(x);
  if (x != x) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct SelShared {
  __align__(16) uint32_t hist[3][kBins];
  uint32_t scan[kSelWarps];
  uint32_t part[4];             // this block's totals, read by the cluster
  uint32_t part2[4];
  uint32_t warp[3][kSelWarps];
  uint32_t bin, above;
  int live;                     // candidates of the unit
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t x) {
  return __reduce_add_sync(0xFFFFFFFFu, x);
}

// Sum over the cluster of word `k` of part / part2, and the sum before this block.
template <class Cluster>
__device__ __forceinline__ void cluster_sum(Cluster& cl, uint32_t* word, uint32_t& before,
                                            uint32_t& total) {
  before = total = 0;
  const unsigned me = cl.block_rank(), n = cl.num_blocks();
  for (unsigned r = 0; r < n; ++r) {
    const uint32_t x = *cl.map_shared_rank(word, r);
    if (r < me) before += x;
    total += x;
  }
}

// The bin of digit d (summed over the cluster's blocks) that holds the left-th
// highest key, and the keys above it: sm.bin, sm.above.  (Block-wide, between
// barriers.)
template <class Cluster>
__device__ __forceinline__ void find_bin(Cluster& cl, SelShared& sm, int d, uint32_t left) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // bins from the highest: thread t holds bins 4 t' .. 4 t' + 3, t' from the top
  uint32_t c[4] = {0, 0, 0, 0};
  const int b0 = kBins - 4 - 4 * tid;
  const unsigned me = cl.block_rank(), blocks = cl.num_blocks();
#pragma unroll 4
  for (unsigned k = 0; k < blocks; ++k) {
    // every block starts at another one's histogram: no block serves all at once
    const unsigned r = me + k < blocks ? me + k : me + k - blocks;
    const uint4 x = *reinterpret_cast<const uint4*>(cl.map_shared_rank(&sm.hist[d][b0], r));
    c[3] += x.x;
    c[2] += x.y;
    c[1] += x.z;
    c[0] += x.w;
  }
  const uint32_t tot = c[0] + c[1] + c[2] + c[3];
  uint32_t inc = tot;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sm.scan[w] = inc;
  __syncthreads();
  // the totals of the warps before this one
  uint32_t ex = lane < w ? sm.scan[lane & (kSelWarps - 1)] : 0u;
  ex = warp_sum(ex) + inc - tot;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (ex < left && left <= ex + c[e]) {
      sm.bin = (uint32_t)(b0 + 3 - e);
      sm.above = ex;
    }
    ex += c[e];
  }
  __syncthreads();
}

// Select for sequences of up to 16 blocks of 512 PT positions: a thread holds
// PT consecutive positions in registers from its loads to its stores.
constexpr int kSelBlocks = 16;   // of a cluster (above 8 by opt-in)

template <int PT, class T>
__device__ __forceinline__ void load_run(T (&x)[PT], const T* from, int n) {
  constexpr int kVec = 16 / sizeof(T);
  if (n >= PT && (reinterpret_cast<uintptr_t>(from) & 15) == 0 && PT % kVec == 0) {
#pragma unroll
    for (int i = 0; i < PT; i += kVec) *reinterpret_cast<uint4*>(&x[i]) = *reinterpret_cast<const uint4*>(from + i);
  } else {
#pragma unroll
    for (int i = 0; i < PT; ++i) x[i] = i < n ? from[i] : T(0);
  }
}
template <int PT, class T>
__device__ __forceinline__ void store_run(const T (&x)[PT], T* to, int n) {
  constexpr int kVec = 16 / sizeof(T);
  if (n >= PT && (reinterpret_cast<uintptr_t>(to) & 15) == 0 && PT % kVec == 0) {
#pragma unroll
    for (int i = 0; i < PT; i += kVec) *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(&x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PT; ++i)
      if (i < n) to[i] = x[i];
  }
}

template <int PT>
__global__ void __launch_bounds__(kSelThreads, 2)
    evict_select_regs_kernel(const __grid_constant__ EvictParams p) {
  __shared__ __align__(16) SelShared sm;
  __shared__ unsigned long long warp64[kSelWarps], part64;
  cg::cluster_group cl = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const unsigned me = cl.block_rank(), blocks = cl.num_blocks();
  const long long u = blockIdx.x / blocks;
  const int b = (int)(u / p.Hkv);
  const long long T = min(max((long long)p.seq_lens[b], 0ll), p.Tmax);
  const long long keep = p.keep[b];
  const long long lo = ((long long)me * kSelThreads + tid) * PT;   // the thread's positions
  const int len = (int)min((long long)PT, max(0ll, p.Tmax - lo));
  const long long base = u * p.Tmax + lo;

  __align__(16) float sc[PT];
  __align__(16) int32_t old[PT];
  __align__(16) uint8_t ti[PT];
  load_run<PT>(ti, p.tier + base, len);
  load_run<PT>(sc, p.score + base, len);
  load_run<PT>(old, p.row_of + base, len);
  for (int i = tid; i < 3 * kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4*>(&sm.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  uint32_t cand = 0, held = 0, key[PT];
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const long long t = lo + i;
    key[i] = score_key(sc[i]);
    if (i >= len || t >= T || ti[i] >= kGone) continue;
    if (t < p.sink || t >= T - p.recent || (p.protect && p.protect[base + i]))
      held |= 1u << i;
    else
      cand |= 1u << i;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PT; ++i)
    if ((cand >> i) & 1) atomicAdd(&sm.hist[0][key[i] >> 21], 1u);
  const uint32_t n_cand = warp_sum(__popc(cand)), n_held = warp_sum(__popc(held));
  if (lane == 0) {
    sm.warp[0][w] = n_cand;
    sm.warp[1][w] = n_held;
  }
  __syncthreads();
  if (w == 0) {
    const uint32_t a = warp_sum(lane < kSelWarps ? sm.warp[0][lane] : 0u);
    const uint32_t c = warp_sum(lane < kSelWarps ? sm.warp[1][lane] : 0u);
    if (lane == 0) {
      sm.part[0] = a;
      sm.part[1] = c;
    }
  }
  cl.sync();
  uint32_t before, cands, helds;
  cluster_sum(cl, &sm.part[0], before, cands);
  cluster_sum(cl, &sm.part[1], before, helds);
  const long long want = keep - helds;
  // all candidates stay, none does, or the `need` highest
  const uint32_t need = want <= 0 ? 0u : (uint32_t)min(want, (long long)cands);
  uint32_t stay = held | (need > 0 ? cand : 0u);
  if (need > 0 && need < cands) {
    uint32_t left = need, prefix = 0;
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
      const int up = d == 1 ? 21 : 10;   // bits of the prefix from here
      if (d > 0) {
#pragma unroll
        for (int i = 0; i < PT; ++i)
          if (((cand >> i) & 1) && (key[i] >> up) == (prefix >> up))
            atomicAdd(&sm.hist[d][(key[i] >> shift) & (d == 2 ? 1023u : 2047u)], 1u);
        cl.sync();
      }
      find_bin(cl, sm, d, left);
      prefix |= sm.bin << shift;
      left -= sm.above;
      __syncthreads();
    }
    // keys above the cut stay, and the first `left` equal to it
    uint32_t above = 0, tie = 0;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      if (key[i] > prefix) above |= 1u << i;
      if (key[i] == prefix) tie |= 1u << i;
    }
    above &= cand;
    tie &= cand;
    const uint32_t n = __popc(tie);
    uint32_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sm.warp[0][w] = inc;
    __syncthreads();
    const uint32_t x = lane < kSelWarps ? sm.warp[0][lane] : 0u;
    uint32_t at = warp_sum(lane < w ? x : 0u) + inc - n;
    const uint32_t all = warp_sum(x);
    if (tid == 0) sm.part2[3] = all;
    cl.sync();
    uint32_t total;
    cluster_sum(cl, &sm.part2[3], before, total);
    at += before;
    const uint32_t room = left > at ? left - at : 0u;
    while ((uint32_t)__popc(tie) > room) tie ^= 0x80000000u >> __clz(tie);  // the last ones go
    stay = held | above | tie;
  }

  // ranks of the kept tokens by tier (three counts of 21 bits)
  unsigned long long n3 = 0;
#pragma unroll
  for (int i = 0; i < PT; ++i)
    if ((stay >> i) & 1) n3 += 1ull << (21 * ti[i]);
  unsigned long long inc3 = n3;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, inc3, o);
    if (lane >= o) inc3 += y;
  }
  if (lane == 31) warp64[w] = inc3;
  __syncthreads();
  unsigned long long at3 = inc3 - n3, all3 = 0;
#pragma unroll
  for (int k = 0; k < kSelWarps; ++k) {
    if (k < w) at3 += warp64[k];
    all3 += warp64[k];
  }
  if (tid == 0) part64 = all3;
  cl.sync();
  unsigned long long total3 = 0;
  for (unsigned r = 0; r < blocks; ++r) {
    const unsigned long long x = *cl.map_shared_rank(&part64, r);
    if (r < me) at3 += x;
    total3 += x;
  }
  const uint32_t P = (uint32_t)p.P;
  uint32_t at[3], total[3];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    at[t] = (uint32_t)(at3 >> (21 * t)) & 0x1FFFFFu;
    total[t] = (uint32_t)(total3 >> (21 * t)) & 0x1FFFFFu;
  }
  // the tiers' first rows in the unit's page list
  at[1] += (total[0] + P - 1) / P * P;
  at[2] += (total[0] + P - 1) / P * P + (total[1] + P - 1) / P * P;
  if (tid == 0 && me == 0)
    for (int t = 0; t < 3; ++t) p.counts[3 * u + t] = (int32_t)total[t];
  int32_t* const src = p.src + u * p.src_stride;
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    int row = -1;
    const int t = ti[i];
    ti[i] = (uint8_t)SKV_TIER_DROP;
    if ((stay >> i) & 1) {
      row = (int)(t == 0 ? at[0] : (t == 1 ? at[1] : at[2]));
      at[0] += t == 0;
      at[1] += t == 1;
      at[2] += t == 2;
      src[row] = old[i];
      ti[i] = (uint8_t)t;
    }
    old[i] = row;
  }
  store_run<PT>(old, p.row_of_out + base, len);
  store_run<PT>(ti, p.tier_out + base, len);
  cl.sync();  // no block leaves while another reads its shared memory
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ SelShared sm;
  cg::cluster_group cl = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const long long u = blockIdx.x / p.clusters;
  const int b = (int)(u / p.Hkv);
  const long long T = min(max((long long)p.seq_lens[b], 0ll), p.Tmax);
  const long long lo = (long long)cl.block_rank() * p.chunk;
  const int len = (int)max(0ll, min((long long)p.chunk, p.Tmax - lo));
  uint32_t* const keys = reinterpret_cast<uint32_t*>(raw);
  uint8_t* const smst = raw + (p.cached ? 4 * (size_t)p.chunk : 0);
  const long long base = u * p.Tmax + lo;

  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
  __syncthreads();

  // states (one byte a position) and keys; the first digit's histogram
  uint32_t n_cand = 0, n_held = 0;
  for (int i = tid; i < len; i += kSelThreads) {
    const long long t = lo + i;
    uint32_t st = t < T ? p.tier[base + i] : kGone;
    if (st >= kGone) st = kGone;
    if (st != kGone && (t < p.sink || t >= T - p.recent || (p.protect && p.protect[base + i])))
      st |= kHeld;
    smst[i] = (uint8_t)st;
    if (st < kGone) {
      const uint32_t k = score_key(p.score[base + i]);
      if (p.cached) keys[i] = k;
      atomicAdd(&sm.hist[0][k >> 21], 1u);
      ++n_cand;
    } else if (st & kHeld) {
      ++n_held;
    }
  }
  n_cand = warp_sum(n_cand);
  n_held = warp_sum(n_held);
  if (lane == 0) {
    sm.warp[0][w] = n_cand;
    sm.warp[1][w] = n_held;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, c = 0;
    for (int k = 0; k < kSelWarps; ++k) {
      a += sm.warp[0][k];
      c += sm.warp[1][k];
    }
    sm.part[0] = a;
    sm.part[1] = c;
  }
  cl.sync();
  uint32_t before, cand, held;
  cluster_sum(cl, &sm.part[0], before, cand);
  cluster_sum(cl, &sm.part[1], before, held);
  const long long want = (long long)p.keep[b] - held;
  // all candidates stay, none does, or the `need` highest
  const uint32_t need = want <= 0 ? 0u : (uint32_t)min(want, (long long)cand);
  uint32_t cut = 0, ties = 0;  // keys above `cut` stay, and the first `ties` equal to it
  const bool some = need > 0 && need < cand;
  if (some) {
    uint32_t left = need, prefix = 0;
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
      const int up = d == 1 ? 21 : 10;   // bits of the prefix from here
      if (d > 0) {
        for (int i = tid; i < len; i += kSelThreads) {
          if (smst[i] >= kGone) continue;
          const uint32_t k = p.cached ? keys[i] : score_key(p.score[base + i]);
          if ((k >> up) == (prefix >> up))
            atomicAdd(&sm.hist[d][(k >> shift) & (d == 2 ? 1023u : 2047u)], 1u);
        }
        cl.sync();
      }
      find_bin(cl, sm, d, left);
      prefix |= sm.bin << shift;
      left -= sm.above;
      __syncthreads();
    }
    cut = prefix;
    ties = left;
  }

  // ties in position order: warp w takes the w-th part of the block's span
  const int span = (((len + kSelWarps - 1) / kSelWarps) + 31) / 32 * 32;
  const int i0 = min(len, w * span), i1 = min(len, i0 + span);
  uint32_t tie_at = 0;
  if (some) {
    uint32_t cnt = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
      if (smst[i] >= kGone) continue;
      cnt += (p.cached ? keys[i] : score_key(p.score[base + i])) == cut;
    }
    cnt = warp_sum(cnt);
    if (lane == 0) sm.warp[0][w] = cnt;
    __syncthreads();
    if (tid == 0) {
      uint32_t a = 0;
      for (int k = 0; k < kSelWarps; ++k) a += sm.warp[0][k];
      sm.part2[3] = a;
    }
    cl.sync();
    uint32_t total;
    cluster_sum(cl, &sm.part2[3], tie_at, total);
    for (int k = 0; k < w; ++k) tie_at += sm.warp[0][k];
  }

  // who stays, and how many of each tier
  uint32_t n[3] = {0, 0, 0};
  const uint32_t lt = (1u << lane) - 1;
  for (int i = i0; i < i1; i += 32) {
    const int k = i + lane;
    uint32_t st = k < i1 ? smst[k] : kGone;
    bool stay = (st & kHeld) != 0;
    if (some) {
      const uint32_t key = st < kGone ? (p.cached ? keys[k] : score_key(p.score[base + k])) : 0u;
      const bool tie = st < kGone && key == cut;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, tie);
      if (st < kGone) stay = key > cut || (tie && tie_at + __popc(m & lt) < ties);
      tie_at += __popc(m);
    } else if (st < kGone) {
      stay = need > 0;
    }
    if (k < i1 && stay) smst[k] = (uint8_t)(st | kStay);
#pragma unroll
    for (int t = 0; t < 3; ++t)
      n[t] += __popc(__ballot_sync(0xFFFFFFFFu, stay && (st & 3u) == (uint32_t)t));
  }
  __syncthreads();  // the tie counts of sm.warp are read above
  if (lane == 0)
    for (int t = 0; t < 3; ++t) sm.warp[t][w] = n[t];
  __syncthreads();
  if (tid < 3) {
    uint32_t a = 0;
    for (int k = 0; k < kSelWarps; ++k) a += sm.warp[tid][k];
    sm.part2[tid] = a;
  }
  cl.sync();
  uint32_t at[3], total[3];
#pragma unroll
  for (int t = 0; t < 3; ++t) cluster_sum(cl, &sm.part2[t], at[t], total[t]);
  const uint32_t P = (uint32_t)p.P;
  uint32_t first[3];  // the tier's first row in the unit's page list
  first[0] = 0;
  first[1] = (total[0] + P - 1) / P * P;
  first[2] = first[1] + (total[1] + P - 1) / P * P;
  if (tid == 0 && cl.block_rank() == 0)
    for (int t = 0; t < 3; ++t) p.counts[3 * u + t] = (int32_t)total[t];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    for (int k = 0; k < w; ++k) at[t] += sm.warp[t][k];
    at[t] += first[t];
  }
  int32_t* const src = p.src + u * p.src_stride;
  for (int i = i0; i < i1; i += 32) {
    const int k = i + lane;
    const uint32_t st = k < i1 ? smst[k] : 0u;
    const bool stay = (st & kStay) != 0;
    int row = -1;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      const bool mine = stay && (st & 3u) == (uint32_t)t;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) row = (int)(at[t] + __popc(m & lt));
      at[t] += __popc(m);
    }
    if (k < i1) {
      p.tier_out[base + k] = (uint8_t)(stay ? st & 3u : (uint32_t)SKV_TIER_DROP);
      p.row_of_out[base + k] = row;
      if (stay) src[row] = p.row_of[base + k];
    }
  }
  cl.sync();  // no block leaves while another reads its shared memory
}

// One block: the page offsets of every (unit, tier) and its first free-list
// entry, by a scan of the units' page counts.
__global__ void __launch_bounds__(1024) evict_plan_kernel(const __grid_constant__ EvictParams p) {
  __shared__ long long sc[32][4];
  asm volatile("griddepcontrol.launch_dependents;");
  const int U = p.B * p.Hkv, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (U + 1023) / 1024, lgP = __ffs(p.P) - 1;
  const int a = min(U, tid * per), z = min(U, a + per);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  long long n[4] = {0, 0, 0, 0};
  for (int u = a; u < z; ++u)
#pragma unroll
    for (int t = 0; t < 3; ++t) n[t] += (p.counts[3 * u + t] + p.P - 1) >> lgP;
  n[3] = n[0] + n[1] + n[2];
  long long ex[4], tot[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    long long x = n[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sc[w][k] = x;
    ex[k] = x - n[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // the totals of the warps, summed up to this one
    long long x = sc[lane][k];
    tot[k] = x;
    if (lane >= w) x = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      tot[k] += __shfl_xor_sync(0xFFFFFFFFu, tot[k], o);
    }
    ex[k] += x;
  }
  for (int u = a; u < z; ++u) {
    p.indptr_out[u] = (int32_t)ex[3];
    for (int t = 0; t < 3; ++t) {
      const long long c = (p.counts[3 * u + t] + p.P - 1) >> lgP;
      if (p.tier_indptr_out) p.tier_indptr_out[3 * u + t] = (int32_t)ex[3];
      p.tbase[3 * u + t] = (int32_t)ex[t];
      ex[3] += c;
      ex[t] += c;
    }
  }
  if (tid == 0) {
    p.indptr_out[U] = (int32_t)tot[3];
    if (p.tier_indptr_out) p.tier_indptr_out[3 * U] = (int32_t)tot[3];
    if (tot[3] > p.out_cap) report(p.err, SKV_ERR_POOL);
    for (int t = 0; t < 3; ++t) {
      const int c = p.cursor[t];
      if (c < 0 || c + tot[t] > p.free_len[t]) report(p.err, SKV_ERR_POOL);
      if (p.cursor_out) p.cursor_out[t] = (int32_t)min(c + tot[t], 0x7FFFFFFFll);
    }
  }
}

__device__ __forceinline__ uint4 load4(const uint8_t* at) {
  return at ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
}

// 16 rows of a new page.
struct Job {
  int u, t, rows;     // unit, tier, rows in use from row0 on (16 at most)
  int row0;           // of the page
  int local;          // first row within the unit's pages
  int place;          // page of its tier within the unit
  long long g;        // page of the list (below 0: no job)
};

// Job `task` (page task >> lg); u: a unit at or before its own.
__device__ __forceinline__ Job locate(const EvictParams& p, long long task, long long end, int lg,
                                      int& u) {
  Job j;
  j.g = -1;
  j.u = u;
  j.t = j.rows = j.row0 = j.local = j.place = 0;
  if (task >= end) return j;
  const int P = p.P, lgP = __ffs(P) - 1;
  j.g = task >> lg;
  while (j.g >= p.indptr_out[u + 1]) ++u;
  j.u = u;
  int pg = (int)(j.g - p.indptr_out[u]);
  j.row0 = 16 * (int)(task & ((1 << lg) - 1));
  j.local = pg * P + j.row0;
  const int n0 = p.counts[3 * u], n1 = p.counts[3 * u + 1], n2 = p.counts[3 * u + 2];
  const int p0 = (n0 + P - 1) >> lgP, p1 = (n1 + P - 1) >> lgP;
  int n = n0;
  if (pg >= p0 + p1) {
    j.t = 2;
    n = n2;
    pg -= p0 + p1;
  } else if (pg >= p0) {
    j.t = 1;
    n = n1;
    pg -= p0;
  }
  j.place = pg;
  j.rows = min(min(P, n - pg * P) - j.row0, 16);
  return j;
}

// A warp per 16 rows of a new page.  A row's values lie in 16-byte chunks
// shared with its pair row (the matrix-fragment order): a new chunk is the
// byte (T1 / T2) or half-word (T0) interleave of two old ones.  A job needs
// three loads one after the other (its rows' old places, their pages' ids,
// the bytes): the first two run two jobs and one job ahead.
constexpr int kMoveBlocks = 2;   // resident blocks of an SM
__global__ void __launch_bounds__(256, kMoveBlocks) evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int U = p.B * p.Hkv, P = p.P, lane = threadIdx.x & 31, lgP = __ffs(P) - 1;
  const int lg = lgP - 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long total = min((long long)p.indptr_out[U], p.out_cap) << lg;
  const long long nw = ((long long)gridDim.x * blockDim.x) >> 5;
  const long long me = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long per = (total + nw - 1) / nw;
  long long task = me * per;
  const long long end = min(total, task + per);
  if (task >= end) return;
  int u = 0, hi = U;
  while (hi - u > 1) {  // the unit of the first page
    const int mid = (u + hi) >> 1;
    if (p.indptr_out[mid] <= (task >> lg)) u = mid; else hi = mid;
  }
  const int row = lane & 15;
  // raw loads, checked when they are used
  const auto load_src = [&](const Job& j) {
    return j.g >= 0 && row < j.rows ? p.src[(long long)j.u * p.src_stride + j.local + row] : -1;
  };
  const auto load_id = [&](const Job& j, int loc) {
    if (loc < 0) return 0xFFFFFFFFu;
    const long long g = (long long)p.indptr[j.u] + (loc >> lgP);
    return g >= 0 && g < p.indptr[j.u + 1] && g < p.page_cap ? p.ids[g] : 0xFFFFFFFFu;
  };
  const auto load_slot = [&](const Job& j) {
    if (j.g < 0) return 0xFFFFFFFFu;
    const long long fi = (long long)p.cursor[j.t] + p.tbase[3 * j.u + j.t] + j.place;
    return fi >= 0 && fi < p.free_len[j.t] ? p.free_ids[j.t][fi] : 0xFFFFFFFFu;
  };
  Job a = locate(p, task, end, lg, u);
  int loc_a = load_src(a);
  uint32_t id_a = load_id(a, loc_a), slot_a = load_slot(a);
  Job b = locate(p, task + 1, end, lg, u);
  int loc_b = load_src(b);
  for (; task < end; ++task) {
    const uint32_t id_b = load_id(b, loc_b), slot_b = load_slot(b);
    const Job c = locate(p, task + 2, end, lg, u);
    const int loc_c = load_src(c);
    const int t = a.t;
    if (slot_a > 0x3FFFFFFFu || (long long)slot_a >= p.slots[t]) {
      if (lane == 0) report(p.err, SKV_ERR_POOL);
    } else {
      uint8_t* const page = p.pool[t] + (long long)slot_a * p.stride[t];
      if (a.row0 == 0 && lane == 0) {
        p.ids_out[a.g] = ((uint32_t)t << 30) | slot_a;
        const int all = min(P, p.counts[3 * a.u + t] - a.place * P);
        *reinterpret_cast<uint4*>(page) =
            make_uint4((uint32_t)all | ((uint32_t)t << 16) | ((uint32_t)kPageMagic << 24),
                       (uint32_t)(a.u / p.Hkv), (uint32_t)(a.u % p.Hkv), (uint32_t)a.place);
      }
      // lane: the old page and row of new row row0 + (lane & 15)
      const uint8_t* op = nullptr;
      if (row < a.rows) {
        const uint32_t old = id_a & 0x3FFFFFFFu;
        if ((int)(id_a >> 30) == t && (long long)old < p.slots[t])
          op = p.pool[t] + (long long)old * p.stride[t];
        else if (lane < 16)
          report(p.err, SKV_ERR_CORRUPT);
      }
      const int ro = loc_a & (P - 1);
      const auto page_of = [&](int r) {
        return reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(op), r));
      };
      const auto row_of = [&](int r) { return __shfl_sync(0xFFFFFFFFu, ro, r); };
      const int t4 = lane & 3;  // values: lane (g, t4) holds rows 2 t4, 2 t4 + 1 of each 8
      const uint8_t *pa[2], *pb[2];
      int ra[2], rb[2], la[2], lb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pa[h] = page_of(8 * h + 2 * t4);
        pb[h] = page_of(8 * h + 2 * t4 + 1);
        ra[h] = row_of(8 * h + 2 * t4);
        rb[h] = row_of(8 * h + 2 * t4 + 1);
        la[h] = 16 * ((lane & ~3) + ((ra[h] & 7) >> 1));
        lb[h] = 16 * ((lane & ~3) + ((rb[h] & 7) >> 1));
      }
      if (t == SKV_TIER_T0) {
        const int vs = kHdrBytes + 256 * P;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // keys: 16 chunks a row, two rows at a time
          uint4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 8 * h + 2 * k + (lane >> 4), ch = lane & 15;
            const uint8_t* o = page_of(r);
            const int q = row_of(r);
            x[k] = load4(o ? o + kHdrBytes + q * 256 + (ch ^ (4 * (q & 1))) * 16 : nullptr);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = a.row0 + 8 * h + 2 * k + (lane >> 4), ch = lane & 15;
            *reinterpret_cast<uint4*>(page + kHdrBytes + r * 256 + (ch ^ (4 * (r & 1))) * 16) = x[k];
          }
          const uint32_t sel = (ra[h] & 1 ? 0x32u : 0x10u) | (rb[h] & 1 ? 0x7600u : 0x5400u);
          const uint8_t* const fa = pa[h] ? pa[h] + vs + (ra[h] >> 3) * 2048 + la[h] : nullptr;
          const uint8_t* const fb = pb[h] ? pb[h] + vs + (rb[h] >> 3) * 2048 + lb[h] : nullptr;
          uint4 y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] = load4(fa ? fa + 512 * k : nullptr);
            y[k] = load4(fb ? fb + 512 * k : nullptr);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(page + vs + (a.row0 / 8 + h) * 2048 + 512 * k + 16 * lane) =
                make_uint4(__byte_perm(x[k].x, y[k].x, sel), __byte_perm(x[k].y, y[k].y, sel),
                           __byte_perm(x[k].z, y[k].z, sel), __byte_perm(x[k].w, y[k].w, sel));
        }
      } else {
        const int cb = t == SKV_TIER_T1 ? 64 : 48, ch = cb / 16;
        // radius (lanes 0-15) and scale (lanes 16-31)
        const int sec = kHdrBytes + (lane >= 16 ? (2 + cb) * P : 0);
        const uint16_t rs = op ? *reinterpret_cast<const uint16_t*>(op + sec + 2 * ro) : (uint16_t)0;
        // codes: cb / 16 chunks a row; the first 32 / (cb / 16) rows, then the rest
        const int cr = t == SKV_TIER_T1 ? lane >> 2 : lane / 3, cc = lane - cr * ch;
        const int step = t == SKV_TIER_T1 ? 8 : 10;   // (T2: rows 0-9, then 10-15)
        uint4 code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = cr + step * h;
          const uint8_t* o = page_of(r & 15);
          const int q = row_of(r & 15);
          const bool mine = r < 16 && cr < step;
          code[h] = load4(o && mine ? o + kHdrBytes + 2 * P + cb * q + 16 * cc : nullptr);
        }
        const int vs = kHdrBytes + (4 + cb) * P;
        uint4 x[4], y[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* const fa = pa[h] ? pa[h] + vs + (ra[h] >> 3) * 1024 + la[h] : nullptr;
          const uint8_t* const fb = pb[h] ? pb[h] + vs + (rb[h] >> 3) * 1024 + lb[h] : nullptr;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            x[2 * h + k] = load4(fa ? fa + 512 * k : nullptr);
            y[2 * h + k] = load4(fb ? fb + 512 * k : nullptr);
          }
        }
        *reinterpret_cast<uint16_t*>(page + sec + 2 * (a.row0 + row)) = rs;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = cr + step * h;
          if (r < 16 && cr < step)
            *reinterpret_cast<uint4*>(page + kHdrBytes + 2 * P + cb * (a.row0 + r) + 16 * cc) = code[h];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // bytes (row 2 t4, row 2 t4 + 1) x (dims d, d + 8) of each word
          const uint32_t sel = ra[h] & 1 ? (rb[h] & 1 ? 0x7351u : 0x6341u) : (rb[h] & 1 ? 0x7250u : 0x6240u);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 z = x[2 * h + k], v = y[2 * h + k];
            *reinterpret_cast<uint4*>(page + vs + (a.row0 / 8 + h) * 1024 + 512 * k + 16 * lane) =
                make_uint4(__byte_perm(z.x, v.x, sel), __byte_perm(z.y, v.y, sel),
                           __byte_perm(z.z, v.z, sel), __byte_perm(z.w, v.w, sel));
          }
        }
      }
    }
    a = b;
    loc_a = loc_b;
    id_a = id_b;
    slot_a = slot_b;
    b = c;
    loc_b = loc_c;
  }
}

// Blocks per unit: chunks of about 16384 positions, at most 8 (the portable
// cluster size).  The keys stay in shared memory while they fit.
int evict_clusters(long long Tmax) {
  int c = 1;
  while (c < 8 && Tmax > 16384ll * c) c *= 2;
  return c;
}

}  // namespace

size_t evict_workspace_bytes(int B, int Hkv, long long Tmax, int P) {
  const size_t U = (size_t)B * Hkv;
  return 4 * (6 * U + U * (size_t)(Tmax + 3 * P));
}

void evict_carve(EvictParams& p, void* ws) {
  const size_t U = (size_t)p.B * p.Hkv;
  int32_t* w = static_cast<int32_t*>(ws);
  p.counts = w;
  p.tbase = w + 3 * U;
  p.src = w + 6 * U;
  p.src_stride = p.Tmax + 3 * p.P;
}

cudaError_t launch_evict(EvictParams& p, cudaStream_t stream) {
  const long long U = (long long)p.B * p.Hkv;
  if (U == 0) return cudaSuccess;
  cudaError_t e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto blocks_of = [&](int span) {
    int c = 1;
    while (c < kSelBlocks && p.Tmax > (long long)span * c) c *= 2;
    return c;
  };
  constexpr int kWide = kSelThreads * 16, kNarrow = kSelThreads * 8;
  if (p.Tmax <= (long long)kWide * kSelBlocks) {
    // 8 positions a thread where that still leaves every block its own SM
    // (half the latency of a block's phases), else 16
    const bool narrow = p.Tmax <= (long long)kNarrow * kSelBlocks && U * blocks_of(kNarrow) <= 148;
    p.clusters = blocks_of(narrow ? kNarrow : kWide);
    const auto kernel = narrow ? evict_select_regs_kernel<8> : evict_select_regs_kernel<16>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(U * p.clusters));
    attr[0].val.clusterDim.x = (unsigned)p.clusters;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
  } else {
    p.clusters = evict_clusters(p.Tmax);
    p.chunk = (int)((p.Tmax + p.clusters - 1) / p.clusters + 15) / 16 * 16;
    constexpr int kMaxSmem = 160 * 1024;
    p.cached = 5ll * p.chunk <= kMaxSmem;
    const long long smem = (p.cached ? 5ll : 1ll) * p.chunk;
    if (smem > 200 * 1024) return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             200 * 1024);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(U * p.clusters));
    cfg.dynamicSmemBytes = (size_t)smem;
    attr[0].val.clusterDim.x = (unsigned)p.clusters;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  }
  if (e != cudaSuccess) return e;
  // plan and move: their launches overlap the grid before them, their work
  // waits for it
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  e = cudaLaunchKernelEx(&cfg, evict_plan_kernel, p);
  if (e != cudaSuccess) return e;
  // several short blocks for each place: tiers cost differently, and blocks
  // that end early make room (ragged batch: 240 us with one block a place,
  // 235 with four, 227 with eight, 229 with sixteen)
  cfg.gridDim = dim3(148 * kMoveBlocks * 8);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace skv
