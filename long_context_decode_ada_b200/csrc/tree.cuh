// tree.cuh -- what the two kernels of the tree attention share: conversions,
// the split of the page list into runs, and the writing of a finished row.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace skv {
namespace tree {

constexpr float kRaise = 8.0f;       // log2 units a score may pass the running maximum

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ldg128(const uint8_t* a) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a));
  return v;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 h =
      __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of fp32: a * b + c, a + b, each rounded once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
// floor(a / b) for a < 2^52, 0 < b < 2^52 (2^20 units of 2^25 pages in 2^16 runs
// stay below): one double division, off by at most one, corrected with exact
// products
__device__ __forceinline__ unsigned long long divide(unsigned long long a, unsigned long long b) {
  unsigned long long q = (unsigned long long)((double)a / (double)b);
  if (q * b > a)
    --q;
  else if ((q + 1) * b <= a)
    ++q;
  return q;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float from16(uint16_t x, int bf16) {
  return bf16 ? __bfloat162float(__ushort_as_bfloat16(x)) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ float2 from16x2(uint32_t x, int bf16) {
  return make_float2(from16((uint16_t)x, bf16), from16((uint16_t)(x >> 16), bf16));
}
// |x| of both halves as one comparable word: the larger bit pattern
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t x) {
  return max(m, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
}
// the same over bf16 halves that fp16's range holds (up to 65280)
__device__ __forceinline__ uint32_t held_bits(uint32_t m, uint32_t x) {
  const uint32_t a = x & 0x7FFFu, b = (x >> 16) & 0x7FFFu;
  return max(m, max(a <= 0x477Fu ? a : 0u, b <= 0x477Fu ? b : 0u));
}
// e with 2^e |x| in [2^14, 2^15) for the largest |x| (bit pattern m)
__device__ __forceinline__ int scale_exp(uint32_t m, int bf16) {
  if (m == 0) return 0;
  const uint32_t b = __float_as_uint(from16((uint16_t)m, bf16));
  const int e = 141 - (int)(b >> 23);
  return b >= 0x7F800000u ? 0 : min(100, e);
}

// The key pairs of the codes at radius 1 (share times cosine and sine) in
// fp16: T1 entry e (the code byte) at tbl1 + step e, T2 entry e (angle |
// share << 4) at tbl2 + step e, each in 32 copies of 4 bytes (copy L is read by
// lane L).
__device__ __forceinline__ void key_tables(const TreeParams& p, uint32_t tbl1, int step,
                                           uint32_t tbl2, int tid, int threads) {
  for (int i = tid; i < 8 * (256 + 64); i += threads) {
    const int e = i >> 3;
    float cs, sn, w;
    if (e < 256 && p.t1_scheme) {
      cs = p.cos5[e >> 3];
      sn = p.sin5[e >> 3];
      w = (float)((e & 7) + 1) / 32.0f;
    } else if (e < 256) {
      cs = p.cos6[e >> 2];
      sn = p.sin6[e >> 2];
      w = p.rho[e & 3];
    } else {
      cs = p.cos4[(e - 256) & 15];
      sn = p.sin4[(e - 256) & 15];
      w = p.rho[(e - 256) >> 4];
    }
    const uint32_t h = pack_f16x2(w * cs, w * sn);
    sts128((e < 256 ? tbl1 + step * e : tbl2 + step * (e - 256)) + 16 * (i & 7), make_uint4(h, h, h, h));
  }
}

// Asks for a page's bytes in L2.
__device__ __forceinline__ void prefetch_page(const uint8_t* a, int P, int tier) {
  const uint32_t bytes = (uint32_t)(kHdrBytes + P * tier_row_bytes(tier));
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(bytes) : "memory");
}

// cap tanh(z) for |z| at most 1/2: the Taylor series up to z^13, whose rest is
// below 5e-8.  (1 - 2 / (1 + e^(2 z)) is off by some 3e-7 whatever z: with a cap
// far above the scores, by more than the scores.)
__device__ __forceinline__ float cap_series(float z, float cap) {
  const float u = z * z, az = cap * z;
  float y = fmaf(21844.0f / 6081075.0f, u, -1382.0f / 155925.0f);
  y = fmaf(y, u, 62.0f / 2835.0f);
  y = fmaf(y, u, -17.0f / 315.0f);
  y = fmaf(y, u, 2.0f / 15.0f);
  y = fmaf(y, u, -1.0f / 3.0f);
  return fmaf(y * u, az, az);
}
// Caps up to which 1 - 2 / (1 + e^(2 z)) serves for every z: it is then off by at
// most 6e-5 of a weight (an fp16 result's rounding is 5e-4).
constexpr float kLowCap = 128.0f;
__device__ __forceinline__ float cap_any(float z, float cap) {
  const float x = fmaf(-2.0f * cap, rcpf(1.0f + ex2f(z * (2.0f * 1.4426950408889634f))), cap);
  return fabsf(z) <= 0.5f ? cap_series(z, cap) : x;
}

// ------------------------------------------------------------------ the split
// Pages of a unit by tier and their costs.  A dense page's bytes take 2.6
// times a coded one's, but its conversion less: it counts twice.  A unit's
// rows count by the kernel's own measure (rows_cost, with the tokens of its
// tiles, kTile; taking up a unit counts as kBegin coded tokens of few rows).
struct Unit {
  long long first;     // index of the first page
  int np, n;           // pages, drafted tokens
  int nt[3];
  int w[3];
  int begin;           // cost of taking the unit up, before its first tile
  unsigned long long last, cost;  // start of the last item, all
};

template <class Cost>
__device__ __forceinline__ Unit unit_of(const TreeParams& p, int u, Cost rows_cost) {
  Unit x;
  const long long a = max(0, p.indptr[u]), z = min((long long)p.indptr[u + 1], p.page_cap);
  const int b = u / p.Hkv;
  // (hidden from the compiler, which would make a loop for every combination)
  const int32_t *count = p.count, *tier_indptr = p.tier_indptr;
  const void* K = p.K;
  asm volatile("" : "+l"(count), "+l"(tier_indptr), "+l"(K));
  x.n = count ? min(max(count[b], 0), p.N) : p.N;
  x.first = a;
  x.np = (int)max(0ll, z - a);
  int n0 = 0, n1 = x.np;
  if (tier_indptr) {
    const int t0 = tier_indptr[3 * u], t1 = tier_indptr[3 * u + 1], t2 = tier_indptr[3 * u + 2];
    n0 = min(max(t1 - t0, 0), x.np);
    n1 = min(max(t2 - t1, 0), x.np - n0);
  }
  x.nt[0] = n0;
  x.nt[1] = n1;
  x.nt[2] = x.np - n0 - n1;
  const int f = rows_cost(x.n * (p.Hq / p.Hkv));
  x.w[0] = 2 * f;
  x.w[1] = x.w[2] = f;
  const unsigned long long pages =
      (unsigned long long)x.w[0] * x.nt[0] + (unsigned long long)f * (x.nt[1] + x.nt[2]);
  const int ipp = Cost::kTile / p.P;
  x.begin = 2 * Cost::kBegin / p.P;
  if (x.n == 0) {
    x.last = x.cost = 0;
  } else if (K || x.np == 0) {
    x.last = x.begin + pages;
    x.cost = x.last + (unsigned long long)(f * ipp);
  } else {
    const int k = (x.np - 1) & ~(ipp - 1);  // the last tile's first page
    const int a0 = min(k, n0);
    x.last = x.begin + (unsigned long long)x.w[0] * a0 + (unsigned long long)f * (k - a0);
    x.cost = x.begin + pages;
  }
  return x;
}

// The first tile of the unit that starts at cost y or above (T1 and T2 pages
// cost the same).
__device__ __forceinline__ int tile_at(const Unit& x, long long y, int ipp) {
  y -= x.begin;
  if (y <= 0) return 0;
  const long long dense = (long long)x.nt[0] * x.w[0];
  const bool first = y <= dense;
  const uint32_t w = first ? x.w[0] : x.w[1];
  const uint32_t z = (uint32_t)min(first ? y : y - dense, 0x7FFFFFF0ll);
  const int g = min((first ? 0 : x.nt[0]) + (int)((z + w - 1) / w), x.np);
  return (g + ipp - 1) >> (__ffs(ipp) - 1);
}

// The split as one run sees it.
struct Run {
  unsigned long long tot, from, to;   // total cost, the run's part of it
  unsigned long long before;          // cost before the unit that holds `from`
  int S;                              // runs with a part
  int unit;                           // that unit (U: none)
};

// scan: a word a warp, out: filled by the thread that finds the unit.
// (Block-wide, with barriers.)
template <int THREADS, class Cost>
__device__ __forceinline__ void find_run(const TreeParams& p, int c, unsigned long long* scan,
                                         Run* out, Cost rows_cost) {
  const int U = p.B * p.Hkv, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (U + THREADS - 1) / THREADS;
  const int u0 = min(U, tid * per), u1 = min(U, u0 + per);
  unsigned long long mine = 0;
#pragma unroll 1
  for (int u = u0; u < u1; ++u) mine += unit_of(p, u, rows_cost).cost;
  unsigned long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[w] = x;
  __syncthreads();
  unsigned long long before = x - mine, tot = 0;
#pragma unroll 1
  for (int k = 0; k < THREADS / 32; ++k) {
    if (k < w) before += scan[k];
    tot += scan[k];
  }
  // a run has a tile of the least cost at least
  const unsigned long long tiles =
      divide(tot, (unsigned long long)(rows_cost(1) * (Cost::kTile / p.P)));
  const int S = (int)min((unsigned long long)p.S, max(1ull, tiles));
  const bool live = c < S && tot > 0;
  unsigned long long from = 0, to = 0;
  if (live) {
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      from = to;
      to = divide((unsigned long long)(c + k) * tot + S - 1, S);
    }
  }
  if (tid == 0) {
    out->tot = tot;
    out->from = from;
    out->to = to;
    out->S = S;
    if (!live) out->unit = U;
  }
  if (live) {
    unsigned long long cc = before;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      const unsigned long long k = per == 1 ? mine : unit_of(p, u, rows_cost).cost;
      if (cc <= from && from < cc + k) {
        out->unit = u;
        out->before = cc;
      }
      cc += k;
    }
  }
  __syncthreads();
}

// The part of unit u (cost cc before it) in run c: false when it has none.
struct Share {
  int k, kend;     // its tiles of pages
  bool draft;      // and the drafted tokens
  int slot;        // where its sums go, -1: the unit lies in this run
  int last;        // the last run of the unit
  bool starts;     // the run is the unit's first of several
};
__device__ __forceinline__ bool share_of(const TreeParams& p, const Unit& x, const Run& r, int c,
                                         unsigned long long cc, int ipp, Share& o) {
  if (x.cost == 0 || cc + x.last < r.from) return false;
  o.k = tile_at(x, (long long)(r.from - cc), ipp);
  o.kend = tile_at(x, (long long)(r.to - cc), ipp);
  o.draft = p.K != nullptr && cc + x.last < r.to;
  const bool begins = cc >= r.from, ends = cc + x.last < r.to;
  o.slot = begins ? (ends ? -1 : 2 * c + 1) : 2 * c;
  o.starts = begins && !ends;
  o.last = o.starts ? (int)divide((cc + x.last) * r.S, r.tot) : c;
  return true;
}

// Four dims (d0 ..) of one row of the result, by one of LANES lanes that
// share the row: v is O relative to M, L the row's sum.  Drafted values
// outside fp16's range are added here.
template <bool CAP, bool BIAS, int LANES>
__device__ __forceinline__ void write_row(const TreeParams& p, int unit, int n, int slot, bool bad,
                                          int r, float M, float L, float (&v)[4], int d0, int lane) {
  const int G = p.Hq / p.Hkv, i = r >> (__ffs(G) - 1), g = r & (G - 1);
  const int b = unit / p.Hkv, h = unit - b * p.Hkv, hq = h * G + g;
  const long long tok = (long long)b * p.N + i;
  if (bad) {
    const uint32_t group = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1) << (lane & ~(LANES - 1) & 31);
    const int l = lane & (LANES - 1);
    constexpr int kEach = kHeadDim / LANES;
    unsigned long long bits = p.mask ? p.mask[tok] : (i == 63 ? ~0ull : (2ull << i) - 1);
    if (n < 64) bits &= (1ull << n) - 1;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + tok * p.q_stride + (long long)hq * kHeadDim;
#pragma unroll 1
    while (bits) {
      const int j = __ffsll((long long)bits) - 1;
      bits &= bits - 1;
      const long long at = ((long long)b * p.N + j) * p.kv_stride + (long long)h * kHeadDim;
      float y[4], s = 0.0f;
      bool out = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = from16(static_cast<const uint16_t*>(p.V)[at + d0 + e], p.kv_bf16);
        if (fabsf(y[e]) <= 65504.0f)
          y[e] = 0.0f;
        else
          out = true;
      }
      if (!__any_sync(group, out)) continue;
#pragma unroll 1
      for (int e = kEach * l; e < kEach * (l + 1); ++e)
        s += from16(q[e], p.q_bf16) * from16(static_cast<const uint16_t*>(p.K)[at + e], p.kv_bf16);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o);
      s *= p.qk_scale;
      if (CAP) s = p.softcap * tanhf(s / p.softcap);
      if (BIAS)
        s -= p.slopes[hq] * (float)(p.q_pos[tok] - p.q_pos[(long long)b * p.N + j]);
      const float w = exp2f(s * 1.4426950408889634f - M);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (y[e] != 0.0f) v[e] += w * y[e];
    }
  }
  if (slot >= 0) {
    const long long at = (long long)slot * (p.N * G) + r;
    *reinterpret_cast<float4*>(p.part + at * kHeadDim + d0) = make_float4(v[0], v[1], v[2], v[3]);
    if (d0 == 0) p.part_ml[at] = make_float2(M, L);
    return;
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint2 w;
  if (p.q_bf16)
    w = make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
  else
    w = make_uint2(pack_f16x2(v[0] * inv, v[1] * inv), pack_f16x2(v[2] * inv, v[3] * inv));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (tok * p.Hq + hq) * kHeadDim + d0) = w;
  if (d0 == 0 && p.lse)
    p.lse[tok * p.Hq + hq] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace tree
}  // namespace skv
