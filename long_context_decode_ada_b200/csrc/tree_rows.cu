// tree_rows.cu -- the tree attention for few rows: at most 32 (drafted
// tokens times query heads) a kv head, single tokens among them.
//
// Every warp takes 16 tokens at a time and keeps everything in registers: the
// keys are rebuilt from their codes by gathers from a replicated table and
// enter mma.sync (m16n8k16, A = 16 keys, B = 8 rows of Q) as they come, the
// weights are transposed between the products by movmatrix, and the values
// (A = V^T, in the pages' fragment order) go from global memory through the
// int8 -> fp16 conversion (exact) straight into the second product; their
// scales go with the weights, which enter as two fp16 parts.  No barrier lies
// between a warp's loads and its sums; the warps' sums meet once per segment
// in shared memory.  Up to 8 rows a warp has one column block, up to 16 two;
// with 17 to 32 rows two warps share the tokens, 16 rows each (the second
// gather costs less than the products).
//
// The loads of a warp's next 16 tokens are issued as soon as the registers
// of the present ones are free.  Shared memory stays at 128 KB: loads in
// flight pass through the L1, and with 28 KB of it (shared memory full) the
// ragged batch of 64 with 8 tokens took 487 us against 415.
//
// What bounds it: latency.  Instruction issue is 39 to 42% busy with three warps
// a scheduler (registers allow no more), HBM gives 2.9 TB/s on single tokens
// over the 128K store (74 us), tensor cores are 23% busy on the ragged batch
// (309 us, of which 3.6 segments a block cost some 10 us each to take up and to
// put down behind block-wide barriers; 364 us in the tensor-memory form, which
// wins from 33 rows on: its conversion costs the same for 1 row as for 64).
// 12 warps: 16 with 128 registers each spill (biased single tokens 260 us
// against 214), 8 hide less.  L2 prefetches ahead of the loads cost more than they
// hide (333 against 316 us).  Two column blocks spill 48 bytes a thread (136 with
// a bias), one up to 24.
#include <algorithm>

#include "tree.cuh"

namespace skv {

namespace {

using namespace tree;

constexpr int kWindow = 512;                   // page ids held at once
constexpr int kRunTile = 64;                   // tokens a run is cut by
constexpr int kObufRow = kHeadDim + 4;         // floats
constexpr uint32_t kRowsTbl = 65536;
// Shared memory ends behind the tables (128 KB): what is left of the SM's
// 256 KB is the L1 that the loads in flight pass through.
constexpr uint32_t kRowsSmem = 131072;

template <int NT>
struct Shape {
  static constexpr int kWarps = 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT;         // rows of a warp
  static constexpr int kHalf = kWarps / 2;     // warps whose sums meet in shared memory
  // cost of a tile by the rows: one or two warps take its tokens.  A unit
  // taken up costs about 1024 tokens (64 ragged sequences x 4 tokens: 349 us
  // at 256 tokens, 328 at 512, 310 at 1024, 318 at 1536, 323 at 2048)
  struct Cost {
    static constexpr int kTile = kRunTile, kBegin = 1024;
    __device__ __forceinline__ int operator()(int rows) const {
      return NT == 1 || rows <= kRows ? 2 : 4;
    }
  };
};

struct __align__(16) Segment {   // a unit, or the part of it that lies in the run
  long long first;                // page of the list
  int pages, dparts;              // pages, 16-row parts of drafted tokens
  int u, n, slot;                 // unit, drafted tokens, partial slot (-1: all here)
};

template <int NT>
struct __align__(16) RowsFixed {
  uint32_t ids[2][kWindow];       // page ids of this segment and the next, in turn
  unsigned long long scan[Shape<NT>::kWarps];
  Run run;
  Segment seg[32];                // the next segments
  int nseg;                       // of them
  int unit;                       // the first unit not looked at, and the cost before it
  unsigned long long before;
  int bad[2];                     // a drafted value lies outside fp16 (segments in turn)
  float m[Shape<NT>::kHalf][Shape<NT>::kRows], l[Shape<NT>::kHalf][Shape<NT>::kRows];
  __align__(16) float o[Shape<NT>::kHalf][Shape<NT>::kRows][kObufRow];
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Lane 4 g + t: rows g, g + 8 of the 16 tokens for keys and scales; rows 2 t,
// 2 t + 1 of both halves for values.
struct Raw {
  uint4 k[2], v[4];
  uint32_t r[2], s[2];
  uint32_t hd;           // the page's header word
  int pos[2];
};

__device__ __forceinline__ void raw_keys(const uint8_t* page, uint32_t tier, int at, int P, int g,
                                         int t, Raw& o) {
  if (tier < 3) o.hd = *reinterpret_cast<const uint32_t*>(page);
  const uint8_t* a = page + kHdrBytes;
  if (tier == SKV_TIER_T1 || tier == SKV_TIER_T2) {
    o.r[0] = *reinterpret_cast<const uint16_t*>(a + 2 * (at + g));
    o.r[1] = *reinterpret_cast<const uint16_t*>(a + 2 * (at + g) + 16);
    a += 2 * P;
    if (tier == SKV_TIER_T1) {
      a += 64 * (at + g) + 16 * t;
      o.k[0] = ldg128(a);
      o.k[1] = ldg128(a + 512);
    } else {
      a += 48 * (at + g);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 n = *reinterpret_cast<const uint2*>(a + 384 * h + 8 * t);
        o.k[h].x = n.x;
        o.k[h].y = n.y;
        o.k[h].z = *reinterpret_cast<const uint32_t*>(a + 384 * h + 32 + 4 * t);
      }
    }
  }
}
__device__ __forceinline__ void raw_values(const uint8_t* page, uint32_t tier, int at, int P,
                                           int g, int lane, Raw& o) {
  if (tier == SKV_TIER_T1 || tier == SKV_TIER_T2) {
    const uint8_t* a = page + kHdrBytes + (tier == SKV_TIER_T1 ? 66 : 50) * P;
    o.s[0] = *reinterpret_cast<const uint16_t*>(a + 2 * (at + g));
    o.s[1] = *reinterpret_cast<const uint16_t*>(a + 2 * (at + g) + 16);
    a += 2 * P + 128 * at + 16 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = ldg128(a + 512 * i);
  }
}

// Asks for 16 dense rows' keys or values (4 KB, a line a lane) in L2: dense rows
// are loaded when they are used.
__device__ __forceinline__ void prefetch_rows(const uint8_t* a, int lane) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a + 128 * lane));
}

template <int NT>
struct Frag {
  uint32_t q[16];         // B fragments of the rows (one column block; two: from qs)
  uint32_t qs;            // the same in shared memory
  float acc[NT][8][4];    // O^T times gain: dims 16 mt + g (+ 8), rows 2 t, 2 t + 1
  float m[NT][2], l[NT][2];
  float gain;             // of the weights, a power of two
};

// S^T += keys (A: two registers a row) x rows for k-step s
template <int NT>
__device__ __forceinline__ void qk(float (&c)[NT][4], const Frag<NT>& f, int s, uint32_t a0,
                                   uint32_t a1, uint32_t a2, uint32_t a3) {
  if constexpr (NT == 1) {
    mma_16816k16_f16(c[0], a0, a1, a2, a3, f.q[2 * s], f.q[2 * s + 1]);
  } else {
    const uint4 q = lds128(f.qs + 1024 * s);
    mma_16816k16_f16(c[0], a0, a1, a2, a3, q.x, q.y);
    mma_16816k16_f16(c[NT - 1], a0, a1, a2, a3, q.z, q.w);
  }
}

__device__ __forceinline__ uint32_t tbl1(uint32_t w, int k, uint32_t tb) {
  return lds32(__byte_perm(w, tb, 0x7604u | (uint32_t)(k << 4)));
}
__device__ __forceinline__ uint32_t tbl2(const uint4& w, int j, uint32_t tb) {
  const int sn = 4 * (j & 7) - 8, sc = 2 * j - 12;
  const uint32_t nw = j < 8 ? w.x : w.y;
  const uint32_t xn = sn >= 0 ? (nw >> sn) : (nw << -sn);
  const uint32_t xc = sc >= 0 ? (w.z >> sc) : (w.z << -sc);
  return lds32((xn & 0xF00u) | (xc & 0x3000u) | tb);
}

// CAP: 0 none, 1 up to kLowCap, 2 above it by cap_any (one capped token over the
// 128K context: 87 us with it, 81 without).

// What a warp knows of its rows' scores (columns 2 t, 2 t + 1 of block n).
template <int NT>
struct Score {
  float c[NT][2];         // what a product is scaled by: to the log2 domain, or to parts of the cap
  float cap;
  float slope[NT][2], rel[NT][2];
};

// Weights (2^4 at most above 1, see kRise) times a value scale times the warp's
// gain stay within fp16: scale times gain is at most kTop.  The gain starts high
// and is lowered (with the sums: powers of two, exact) when a value scale
// asks for it, so that small weights of small values stay normal numbers: with a
// gain of 4 for all, weights of 2^-12 were lost where values are below 0.01.
constexpr float kRise = 4.0f, kTop = 4094.0f, kFirstGain = 0x1p100f;

// Weights as B fragments: each is the sum of two fp16 numbers, so that nothing
// of a weight above some 2^-36 is lost to their rounding (the products for it
// cost less than scaling the values, which would round them: one fp16 store
// 0.0002 off, as its output's rounding alone, against 0.00034).  bf16 results
// would not show it: they take the same path, 17 us of the ragged batch's 309,
// rather than instances of their own.
template <int NT>
struct Weights {
  uint32_t hi[NT][2], lo[NT][2];
};

__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = transposed(*reinterpret_cast<const uint32_t*>(&h));
  lo = transposed(pack_f16x2(x - f.x, y - f.y));
}

// Scores to weights: c holds the products of tokens g, g + 8, rA / rB what
// the keys are scaled by, vA / vB what the values are; bit 4 n + e of `see`:
// the score counts.
template <int NT, int CAP, bool BIAS>
__device__ __forceinline__ void weights(Frag<NT>& f, const Score<NT>& sc, float (&c)[NT][4],
                                        float rA, float rB, float vA, float vB, float posA,
                                        float posB, uint32_t see, Weights<NT>& b) {
  constexpr uint32_t kAll = (1u << (4 * NT)) - 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = e & 1;
      float x = c[n][e] * (e < 2 ? rA : rB);
      if (CAP || BIAS) x *= sc.c[n][j];
      if (CAP == 1) x = fmaf(-2.0f * sc.cap, rcpf(1.0f + ex2f(x)), sc.cap);
      if (CAP == 2) x = cap_any(x, sc.cap);
      if (BIAS) x = fmaf(sc.slope[n][j], (e < 2 ? posA : posB) - sc.rel[n][j], x);
      c[n][e] = x;
    }
  }
  if (see != kAll) {
#pragma unroll
    for (int k = 0; k < 4 * NT; ++k)
      if (!((see >> k) & 1)) c[k >> 2][k & 3] = -INFINITY;
  }
  // z = score - maximum; above kRise (or without a maximum: not a number or
  // infinite) the maximum rises first.  Value scales above kTop lower the gain
  float z[NT][4], top = -INFINITY;
  const auto less = [&](int n, int e, float m) {
    return CAP || BIAS ? c[n][e] - m : fmaf(c[n][e], sc.c[n][e & 1], -m);
  };
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[n][e] = less(n, e, f.m[n][e & 1]);
      top = fmaxf(top, z[n][e]);
    }
  const float big = fmaxf(fabsf(vA), fabsf(vB));
  if (__any_sync(0xFFFFFFFFu, top > kRise || big > kTop)) {
    float v = big;
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
    // (v d in [2^11, 2^12))
    const float d = v > kTop ? __uint_as_float((265u - (__float_as_uint(v) >> 23)) << 23) : 1.0f;
    f.gain *= d;
    vA *= d;
    vB *= d;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float a[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = fmaxf(less(n, j, 0.0f), less(n, j + 2, 0.0f));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
        x = x > f.m[n][j] + kRise ? x : f.m[n][j];
        a[j] = x == f.m[n][j] ? 1.0f : ex2f(f.m[n][j] - x);
        f.m[n][j] = x;
        f.l[n][j] *= a[j];
        a[j] *= d;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        f.acc[n][mt][0] *= a[0];
        f.acc[n][mt][1] *= a[1];
        f.acc[n][mt][2] *= a[0];
        f.acc[n][mt][3] *= a[1];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        z[n][e] = less(n, e, f.m[n][e & 1] == -INFINITY ? 0.0f : f.m[n][e & 1]);
  } else if (see != kAll) {
    // a row that has seen nothing so far
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c[n][e] == -INFINITY) z[n][e] = -INFINITY;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float w0 = ex2f(z[n][0]), w1 = ex2f(z[n][1]), w2 = ex2f(z[n][2]), w3 = ex2f(z[n][3]);
    f.l[n][0] += w0 + w2;
    f.l[n][1] += w1 + w3;
    split(w0 * vA, w1 * vA, b.hi[n][0], b.lo[n][0]);
    split(w2 * vB, w3 * vB, b.hi[n][1], b.lo[n][1]);
  }
}

template <int NT>
__device__ __forceinline__ void pv(Frag<NT>& f, int mt, uint32_t a0, uint32_t a1, uint32_t a2,
                                   uint32_t a3, const Weights<NT>& b) {
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_16816k16_f16(f.acc[n][mt], a0, a1, a2, a3, b.lo[n][0], b.lo[n][1]);
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_16816k16_f16(f.acc[n][mt], a0, a1, a2, a3, b.hi[n][0], b.hi[n][1]);
}

// both halves of a mask of rows 2 t, 2 t + 1 that lie below `rows`
__device__ __forceinline__ uint32_t pair_mask(int row, int rows) {
  return (row < rows ? 0xFFFFu : 0u) | (row + 1 < rows ? 0xFFFF0000u : 0u);
}

// int8 values to fp16: v + 128 as the low byte of 1024 + x, less 1152 (exact)
__device__ __forceinline__ uint32_t whole(uint32_t u, uint32_t sel) {
  const uint32_t x = __byte_perm(u, 0x64646464u, sel);
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 drafted tokens from j0 on (scratch: 2 KB of shared memory of the warp).
// Rolled loops: a unit's drafted tokens are few, their code should be too.
template <int NT, int CAP, bool BIAS>
__device__ __forceinline__ void draft_tokens(const TreeParams& p, Frag<NT>& f, const Score<NT>& sc,
                                             const Segment& sg, int j0, int row0, int G, int lane,
                                             uint32_t scratch, int* bad) {
  const int g = lane >> 2, t = lane & 3, n = sg.n, R = n * G;
  const int b = sg.u / p.Hkv, h = sg.u - b * p.Hkv;
  const long long tok0 = (long long)b * p.N, off = (long long)h * kHeadDim;
  const uint16_t* K = static_cast<const uint16_t*>(p.K) + off + 8 * t;
  float c[NT][4] = {}, up[2], down[2], pos[2] = {0.0f, 0.0f};
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int j = j0 + g + 8 * y;
    uint32_t mx = 0;
    if (j < n) {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(K + (tok0 + j) * p.kv_stride + 32 * i);
        mx = max_bits(max_bits(max_bits(max_bits(mx, x.x), x.y), x.z), x.w);
      }
      if (BIAS) pos[y] = (float)(p.q_pos[tok0 + j] - p.q_pos[tok0]);
    }
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    const int e = scale_exp(mx, p.kv_bf16);
    up[y] = pow2i(e);
    down[y] = pow2i(-e);
  }
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    uint32_t a[2][4];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int j = j0 + g + 8 * y;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (j < n) x = *reinterpret_cast<const uint4*>(K + (tok0 + j) * p.kv_stride + 32 * i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 z = from16x2(w[k], p.kv_bf16);
        a[y][k] = pack_f16x2(z.x * up[y], z.y * up[y]);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 q = lds128(f.qs + 1024 * (2 * i + k));
      mma_16816k16_f16(c[0], a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1], q.x, q.y);
      if (NT == 2)
        mma_16816k16_f16(c[NT - 1], a[0][2 * k], a[1][2 * k], a[0][2 * k + 1], a[1][2 * k + 1], q.z, q.w);
    }
  }
  // small bf16 values enter times a power of two, their largest between 1 and 2,
  // the weights back (further up the weights would lose what the values gain)
  const int tok = lane >> 1;
  const uint16_t* V = static_cast<const uint16_t*>(p.V) + (tok0 + j0 + tok) * p.kv_stride + off;
  float vup = 1.0f, vdown = f.gain;
  if (p.kv_bf16) {
    uint32_t mx = 0;
    if (j0 + tok < n) {
#pragma unroll 4
      for (int k = lane & 1; k < 16; k += 2) {
        const uint4 x = *reinterpret_cast<const uint4*>(V + 8 * k);
        mx = held_bits(held_bits(held_bits(held_bits(mx, x.x), x.y), x.z), x.w);
      }
    }
    const int e = max(0, scale_exp(__reduce_max_sync(0xFFFFFFFFu, mx), 1) - 14);
    vup = pow2i(e);
    vdown *= pow2i(-e);
  }
  uint32_t see = 0;
  Weights<NT> w;
#pragma unroll 1
  for (int e = 0; e < 4 * NT; ++e) {
    const int r = row0 + 8 * (e >> 2) + 2 * t + (e & 1), j = j0 + g + 8 * ((e >> 1) & 1);
    if (r < R && j < n) {
      const int i = r >> (__ffs(G) - 1);
      if (p.mask ? (p.mask[tok0 + i] >> j) & 1 : j <= i) see |= 1u << e;
    }
  }
  weights<NT, CAP, BIAS>(f, sc, c, down[0], down[1], vdown, vdown, pos[0], pos[1], see, w);
  // values: 64 dims at a time as fp16 rows of 128 bytes (16-byte chunks permuted
  // by the token's low bits), read back transposed.  A value that fp16 does
  // not hold enters as 0 and is added by write_row.
  bool out = false;
  const int m = lane >> 3, from = (lane & 7) + 8 * (m >> 1);
#pragma unroll
  for (int hv = 0; hv < 2; ++hv) {
    __syncwarp();
#pragma unroll 1
    for (int k = 4 * (lane & 1); k < 4 * (lane & 1) + 4; ++k) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (j0 + tok < n) x = *reinterpret_cast<const uint4*>(V + 64 * hv + 8 * k);
      uint32_t z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 y = from16x2(z[e], p.kv_bf16);
        if (!(fabsf(y.x) <= 65504.0f)) {
          y.x = 0.0f;
          out = true;
        }
        if (!(fabsf(y.y) <= 65504.0f)) {
          y.y = 0.0f;
          out = true;
        }
        z[e] = pack_f16x2(y.x * vup, y.y * vup);
      }
      sts128(scratch + 128 * tok + ((k ^ (tok & 7)) << 4), make_uint4(z[0], z[1], z[2], z[3]));
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                   : "r"(scratch + 128 * from + (((2 * k + (m & 1)) ^ (from & 7)) << 4))
                   : "memory");
      pv<NT>(f, 4 * hv + k, a[0], a[1], a[2], a[3], w);
    }
  }
  if (out) *(volatile int*)bad = 1;
}

template <int NT, int CAP, bool BIAS, bool DRAFT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
    tree_rows_kernel(const __grid_constant__ TreeParams p) {
  using S = Shape<NT>;
  using Fixed = RowsFixed<NT>;
  static_assert(sizeof(Fixed) + 1024 <= kRowsTbl, "the tables start at 64 KB");
  constexpr uint32_t kScratch = sizeof(Fixed::o) / S::kWarps / 16 * 16;   // a warp's, for drafted values
  static_assert(kScratch >= 2048, "16 tokens, 64 dims");
  extern __shared__ __align__(128) uint8_t raw[];
  Fixed& f = *reinterpret_cast<Fixed*>(raw);
  const uint32_t base = smem_u32(raw);
  const uint32_t tbl = (base + (uint32_t)sizeof(Fixed) + kRowsTbl - 1) & ~(kRowsTbl - 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (tbl + kRowsTbl > base + kRowsSmem) {
    // (the window starts at 1 KB: it fits)
    if (tid == 0) report(p.err, SKV_ERR_CUDA);
    return;
  }
  // (entry e of T1's table at 256 e, T2's in the other halves)
  key_tables(p, tbl, 256, tbl + 128, tid, S::kThreads);
  const int c = blockIdx.x, G = p.Hq / p.Hkv, lgG = __ffs(G) - 1, P = p.P, ipp = kRunTile / P;
  const int lgp = __ffs(P) - 5, ppp = 1 << lgp;   // 16-row parts of a page
  const uint32_t tb = tbl + 4 * lane;
  find_run<S::kThreads>(p, c, f.scan, &f.run, typename S::Cost());
  // the next segments, by one warp: a lane per unit
  const auto look_ahead = [&]() {
    const int U = p.B * p.Hkv, u = f.unit + lane;
    Unit x = {};
    if (u < U) x = unit_of(p, u, typename S::Cost());
    unsigned long long cc = x.cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, cc, o);
      if (lane >= o) cc += y;
    }
    cc += f.before;                      // behind the unit
    const Run run = f.run;
    Share y;
    const bool mine = u < U && cc - x.cost < run.to && share_of(p, x, run, c, cc - x.cost, ipp, y);
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine);
    if (mine) {
      Segment g;
      g.first = x.first + (long long)y.k * ipp;
      g.pages = max(0, min(y.kend * ipp, x.np) - y.k * ipp);
      g.dparts = y.draft ? (x.n + 15) >> 4 : 0;
      g.u = u;
      g.n = x.n;
      g.slot = y.slot;
      f.seg[__popc(all & ((1u << lane) - 1))] = g;
      if (y.starts) p.join[c] = make_int2(u, y.last);
    }
    __syncwarp();
    if (lane == 31) {
      f.nseg = __popc(all);
      f.before = cc;
      f.unit = cc < run.to ? u + 1 : U;
    }
    __syncwarp();
  };
  // the next segments, while there are units: the count in f.nseg (block-wide
  // between barriers; whole batches of units may lie outside the run)
  const auto refill = [&]() {
    if (warp == 0) {
      do {
        look_ahead();
      } while (f.nseg == 0 && f.unit < p.B * p.Hkv);
    }
  };
  constexpr int kEach = (kWindow + S::kThreads - 1) / S::kThreads;
  const auto load_ids = [&](const Segment& g, int w0, uint32_t (&id)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int k = tid + e * S::kThreads;
      id[e] = k < min(kWindow, g.pages - w0) ? p.ids[g.first + w0 + k] : 0xFFFFFFFFu;
    }
  };
  const auto keep_ids = [&](int buf, const uint32_t (&id)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (tid + e * S::kThreads < kWindow) f.ids[buf][tid + e * S::kThreads] = id[e];
  };
  uint32_t id[kEach];
  if (tid == 0) {
    p.join[c] = make_int2(-1, 0);
    f.bad[0] = f.bad[1] = 0;
    f.unit = f.run.unit;
    f.before = f.run.before;
    f.nseg = 0;
  }
  __syncthreads();
  int at_seg = 0, nseg = 0;
#pragma unroll 1
  for (int seg = 0;; seg ^= 1) {
    if (at_seg == nseg) {
      refill();
      __syncthreads();
      at_seg = 0;
      nseg = f.nseg;
      if (nseg == 0) break;
      load_ids(f.seg[0], 0, id);
      keep_ids(seg, id);
      __syncthreads();
    }
    // (read again where it is used: registers are short)
    const Segment& sg = f.seg[at_seg];
    const int b = sg.u / p.Hkv, h = sg.u - b * p.Hkv, R = sg.n * G;
    const int blocks = R > S::kRows ? 2 : 1;      // (at most 2 S::kRows rows)
    const int streams = blocks == 2 ? S::kHalf : S::kWarps;
    const int stream = blocks == 2 ? warp >> 1 : warp;
    const int row0 = blocks == 2 ? S::kRows * (warp & 1) : 0;
    const long long tok0 = (long long)b * p.N;
    const int q0 = BIAS ? p.q_pos[tok0] : 0;

    const bool more = at_seg + 1 < nseg;
    if (more) load_ids(f.seg[at_seg + 1], 0, id);
    // the rows as B fragments: fp16 scaled by a power of two a row
    Frag<NT> fr;
    Score<NT> sc;
    sc.cap = p.softcap * 1.4426950408889634f;
    // (also in shared memory: k-step s of a row block at 1 KB steps, in the halves
    // that the tables leave free; a warp's fragments serve all streams)
    fr.qs = tbl + 256 * (64 + 32 * (row0 != 0) + (lane >> 3)) + 128 + 16 * (lane & 7);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int r = row0 + 8 * k + g, i = r >> lgG;
      uint4 x[4];
      uint32_t mx = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x[y] = make_uint4(0, 0, 0, 0);
        if (r < R)
          x[y] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                 (tok0 + i) * p.q_stride +
                                                 (long long)(h * G + r - i * G) * kHeadDim +
                                                 32 * y + 8 * t);
        mx = max_bits(max_bits(max_bits(max_bits(mx, x[y].x), x[y].y), x[y].z), x[y].w);
      }
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const int e = scale_exp(mx, p.q_bf16);
      const float up = pow2i(e);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t w[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float2 a = from16x2(w[v], p.q_bf16);
          const uint32_t q = pack_f16x2(a.x * up, a.y * up);
          if (NT == 1) fr.q[4 * y + v] = q;
          if (stream == 0) sts32(fr.qs + 1024 * (2 * y + (v >> 1)) + 8 * k + 4 * (v & 1), q);
        }
      }
      // of the lane's two score columns
      float scale = p.qk_scale * pow2i(-e);
      if (CAP)   // (0 times it stays 0)
        scale = fminf(scale * (CAP == 1 ? 2.0f * 1.4426950408889634f : 1.0f) / p.softcap, 3.0e38f);
      else
        scale *= 1.4426950408889634f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc.c[k][j] = __shfl_sync(0xFFFFFFFFu, scale, 8 * t + 4 * j);
        fr.m[k][j] = -INFINITY;
        fr.l[k][j] = 0.0f;
        sc.slope[k][j] = sc.rel[k][j] = 0.0f;
        const int rr = row0 + 8 * k + 2 * t + j;
        if (BIAS && rr < R) {
          const int ii = rr >> lgG;
          sc.slope[k][j] = p.slopes[h * G + rr - ii * G] * 1.4426950408889634f;
          sc.rel[k][j] = (float)(p.q_pos[tok0 + ii] - q0);
        }
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        fr.acc[k][mt][0] = fr.acc[k][mt][1] = fr.acc[k][mt][2] = fr.acc[k][mt][3] = 0.0f;
    }
    fr.gain = kFirstGain;

    if (more) keep_ids(seg ^ 1, id);
    // the rows' fragments in shared memory are there (one column block: only the
    // drafted tokens read them)
    if (NT == 2 || (DRAFT && sg.dparts > 0)) __syncthreads();
    for (int w0 = 0; w0 < sg.pages || w0 == 0; w0 += kWindow) {
      const int held = min(kWindow, sg.pages - w0);
      if (w0 > 0) {
        load_ids(sg, w0, id);
        __syncthreads();
        keep_ids(seg, id);
        __syncthreads();
      }
      const int store = held << lgp;
      const int total = store + (w0 + kWindow >= sg.pages ? sg.dparts : 0);
      Raw o;
      o.r[0] = o.r[1] = o.s[0] = o.s[1] = o.hd = 0;
      o.pos[0] = o.pos[1] = q0;
      const uint8_t* page = nullptr;
      uint32_t tier = 3;
      int at = 0;
      // the pages' headers come with their rows: a pass over the headers
      // alone would wait for a translation per page
      const auto look = [&](int q) {
        tier = 3;
        if (q < store) {
          const uint32_t x = f.ids[seg][q >> lgp], sl = x & 0x3FFFFFFFu;
          at = 16 * (q & (ppp - 1));
          tier = x >> 30;
          if (tier > 2 || (long long)sl >= p.slots[tier]) {
            if (lane == 0) report(p.err, SKV_ERR_CORRUPT);
            tier = 3;
            return;
          }
          page = p.pool[tier] + (long long)sl * p.stride[tier];
          if (tier == SKV_TIER_T0) {
            if (blocks == 1 || row0 == 0) prefetch_rows(page + kHdrBytes + 256 * at, lane);
            if (blocks == 1 || row0 > 0) prefetch_rows(page + kHdrBytes + 256 * (P + at), lane);
          }
        }
      };
      const auto raw_pos = [&](int q) {
        if (BIAS && q < store) {
          const int32_t* a = p.row_pos + ((sg.first + w0 + (q >> lgp)) * P + at + g);
          o.pos[0] = a[0];   // (below 0: no position names the row)
          o.pos[1] = a[8];
        }
      };
      // (the first turn only loads)
#pragma unroll 1
      for (int q = stream - streams; q < total; q += streams) {
        if (DRAFT && q >= store) {
          draft_tokens<NT, CAP, BIAS>(p, fr, sc, sg, 16 * (q - store), row0, G, lane,
                                      smem_u32(&f.o[0][0][0]) + warp * kScratch,
                                      &f.bad[seg]);
          continue;
        }
        const uint8_t* const pg = page;
        const uint32_t ti = tier;
        const int a0 = at;
        int nr = 0;
        if (ti < 3) {
          if ((o.hd >> 16) != (ti | ((uint32_t)kPageMagic << 8)) || (o.hd & 0xFFFFu) > (uint32_t)P) {
            if (lane == 0) report(p.err, SKV_ERR_CORRUPT);
          } else {
            nr = min((int)(o.hd & 0xFFFFu) - a0, 16);
          }
        }
        // (one column block: two chains of products, which halves their latency)
        float cc[NT][4] = {}, cd[NT == 1 ? 1 : NT][4] = {};
        float(&co)[NT][4] = NT == 1 ? cd : cc;
        float rA = 1.0f, rB = 1.0f, vA = fr.gain, vB = fr.gain, posA = 0.0f, posB = 0.0f;
        uint32_t placed = ~0u;
        if (BIAS) {
          posA = (float)(o.pos[0] - q0);
          posB = (float)(o.pos[1] - q0);
          if (o.pos[0] < 0) placed &= 0xCCCCCCCCu;
          if (o.pos[1] < 0) placed &= 0x33333333u;
        }
        if (nr <= 0) {
          // nothing there
        } else if (ti == SKV_TIER_T1) {
          const uint32_t wa[4] = {o.k[0].x, o.k[0].y, o.k[0].z, o.k[0].w};
          const uint32_t wb[4] = {o.k[1].x, o.k[1].y, o.k[1].z, o.k[1].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qk<NT>(cc, fr, 2 * i, tbl1(wa[i], 0, tb), tbl1(wb[i], 0, tb), tbl1(wa[i], 1, tb),
                   tbl1(wb[i], 1, tb));
            qk<NT>(co, fr, 2 * i + 1, tbl1(wa[i], 2, tb), tbl1(wb[i], 2, tb), tbl1(wa[i], 3, tb),
                   tbl1(wb[i], 3, tb));
          }
        } else if (ti == SKV_TIER_T2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qk<NT>(cc, fr, 2 * i, tbl2(o.k[0], 4 * i, tb + 128), tbl2(o.k[1], 4 * i, tb + 128),
                   tbl2(o.k[0], 4 * i + 1, tb + 128), tbl2(o.k[1], 4 * i + 1, tb + 128));
            qk<NT>(co, fr, 2 * i + 1, tbl2(o.k[0], 4 * i + 2, tb + 128),
                   tbl2(o.k[1], 4 * i + 2, tb + 128), tbl2(o.k[0], 4 * i + 3, tb + 128),
                   tbl2(o.k[1], 4 * i + 3, tb + 128));
          }
        } else {
          const uint8_t* a = pg + kHdrBytes + 256 * (a0 + g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ch = 16 * ((4 * i + t) ^ (4 * (g & 1)));
            const uint4 x = ldg128(a + ch), y = ldg128(a + 2048 + ch);
            qk<NT>(cc, fr, 2 * i, x.x, y.x, x.y, y.y);
            qk<NT>(co, fr, 2 * i + 1, x.z, y.z, x.w, y.w);
          }
        }
        if (ti != SKV_TIER_T0) {
          rA = __half2float(__ushort_as_half((uint16_t)o.r[0]));
          rB = __half2float(__ushort_as_half((uint16_t)o.r[1]));
          // (rows that are not there may hold anything)
          vA = g < nr ? fr.gain * __half2float(__ushort_as_half((uint16_t)o.s[0])) : 0.0f;
          vB = g + 8 < nr ? fr.gain * __half2float(__ushort_as_half((uint16_t)o.s[1])) : 0.0f;
        }
        look(q + streams);
        raw_pos(q + streams);
        raw_keys(page, tier, at, P, g, t, o);
        if (nr > 0) {
          uint32_t see = ~0u;
          Weights<NT> w;
          if (nr < 16) see = (g < nr ? 0x33333333u : 0u) | (g + 8 < nr ? 0xCCCCCCCCu : 0u);
          if (BIAS && (see & ~placed)) {
            report(p.err, SKV_ERR_CORRUPT);
            see &= placed;
          }
          see &= (1u << (4 * NT)) - 1;
          if (NT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) cc[0][e] += cd[0][e];
          }
          weights<NT, CAP, BIAS>(fr, sc, cc, rA, rB, vA, vB, posA, posB, see, w);
          if (ti != SKV_TIER_T0) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t va[4] = {o.v[y].x, o.v[y].y, o.v[y].z, o.v[y].w};
              const uint32_t vb[4] = {o.v[y + 2].x, o.v[y + 2].y, o.v[y + 2].z, o.v[y + 2].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t ua = va[k] ^ 0x80808080u, ub = vb[k] ^ 0x80808080u;
                pv<NT>(fr, 4 * y + k, whole(ua, 0x4140), whole(ua, 0x4342), whole(ub, 0x4140),
                       whole(ub, 0x4342), w);
              }
            }
          } else {
            const uint32_t m0 = pair_mask(2 * t, nr), m1 = pair_mask(2 * t + 8, nr);
            const uint8_t* a = pg + kHdrBytes + 256 * (P + a0) + 16 * lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 x = ldg128(a + 512 * k), y = ldg128(a + 2048 + 512 * k);
              pv<NT>(fr, 2 * k, x.x & m0, x.y & m0, y.x & m1, y.y & m1, w);
              pv<NT>(fr, 2 * k + 1, x.z & m0, x.w & m0, y.z & m1, y.w & m1, w);
            }
          }
        }
        raw_values(page, tier, at, P, g, lane, o);
      }
    }

    if (DRAFT && sg.dparts > 0) __syncthreads();  // (the drafted values' scratch lies where the sums go)
    // the warps' sums meet: the second half's in the first half's registers,
    // those in shared memory (a warp and the one kHalf behind it have the
    // same rows)
#pragma unroll
    for (int k = 0; k < NT; ++k) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fr.l[k][j] += __shfl_xor_sync(0xFFFFFFFFu, fr.l[k][j], 4);
        fr.l[k][j] += __shfl_xor_sync(0xFFFFFFFFu, fr.l[k][j], 8);
        fr.l[k][j] += __shfl_xor_sync(0xFFFFFFFFu, fr.l[k][j], 16);
      }
    }
    const int slot0 = warp < S::kHalf ? warp : warp - S::kHalf;
    const float off = 1.0f / fr.gain;   // (exact)
    for (int half = 1; half >= 0; --half) {
      if (warp / S::kHalf == half) {
#pragma unroll
        for (int k = 0; k < NT; ++k) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = 8 * k + 2 * t + j;
            float* const to = &f.o[slot0][r][g];
            if (half == 0) {
              const float m1 = f.m[slot0][r], l1 = f.l[slot0][r], m0 = fr.m[k][j];
              const float m = fmaxf(m0, m1);
              const float a0 = m0 == m ? 1.0f : ex2f(m0 - m), a1 = m1 == m ? 1.0f : ex2f(m1 - m);
              fr.m[k][j] = m;
              fr.l[k][j] = fr.l[k][j] * a0 + l1 * a1;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                fr.acc[k][mt][j] = fr.acc[k][mt][j] * (a0 * off) + to[16 * mt] * a1;
                fr.acc[k][mt][j + 2] = fr.acc[k][mt][j + 2] * (a0 * off) + to[16 * mt + 8] * a1;
              }
              __syncwarp();   // (every lane has read the row's m and l)
            }
            if (g == 0) {
              f.m[slot0][r] = fr.m[k][j];
              f.l[slot0][r] = fr.l[k][j];
            }
            const float o = half == 0 ? 1.0f : off;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              to[16 * mt] = fr.acc[k][mt][j] * o;
              to[16 * mt + 8] = fr.acc[k][mt][j + 2] * o;
            }
          }
        }
      }
      __syncthreads();
    }
    if (tid == 0) f.bad[seg ^ 1] = 0;
    const bool bad = DRAFT && *(volatile int*)&f.bad[seg] != 0;
    for (int r = warp; r < sg.n * G; r += S::kWarps) {
      const int blk = r >= S::kRows ? 1 : 0, lr = r - S::kRows * blk;
      float m = -INFINITY, l = 0.0f;
      if (lane < S::kHalf / blocks) {
        const int w = blocks * lane + blk;
        m = f.m[w][lr];
        l = f.l[w][lr];
      }
      float M = m;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, k));
      const float a = m == -INFINITY ? 0.0f : ex2f(m - M);
      // (a sum without a maximum: 0, or NaN where every score is NaN)
      float L = m == -INFINITY ? l : l * a;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, k);
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int k = 0; k < S::kHalf / blocks; ++k) {
        const float ak = __shfl_sync(0xFFFFFFFFu, a, k);
        const float4 x = *reinterpret_cast<const float4*>(&f.o[blocks * k + blk][lr][4 * lane]);
        v[0] += ak * x.x;
        v[1] += ak * x.y;
        v[2] += ak * x.z;
        v[3] += ak * x.w;
      }
      write_row<CAP != 0, BIAS, 32>(p, sg.u, sg.n, sg.slot, bad, r, M, L, v, 4 * lane, lane);
    }
    __syncthreads();
    ++at_seg;
  }
}

template <int NT, int CAP, bool BIAS>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
  // few rows over the store alone: the drafted tokens' code in the loop costs them
  // registers (one capped token over the 128K context: 76 us with it, 73 without,
  // 64 sequences with one biased token 238 and 221)
  const auto kernel = NT == 1 && !p.K ? tree_rows_kernel<NT, CAP, BIAS, NT != 1>
                                      : tree_rows_kernel<NT, CAP, BIAS, true>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kRowsSmem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)p.S, Shape<NT>::kThreads, kRowsSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int NT>
cudaError_t launch_score(const TreeParams& p, cudaStream_t stream) {
  if (p.softcap > kLowCap)
    return p.slopes ? launch<NT, 2, true>(p, stream) : launch<NT, 2, false>(p, stream);
  if (p.softcap > 0.0f)
    return p.slopes ? launch<NT, 1, true>(p, stream) : launch<NT, 1, false>(p, stream);
  return p.slopes ? launch<NT, 0, true>(p, stream) : launch<NT, 0, false>(p, stream);
}

}  // namespace

cudaError_t launch_tree_rows(const TreeParams& p, cudaStream_t stream) {
  return p.N * (p.Hq / p.Hkv) <= 8 ? launch_score<1>(p, stream) : launch_score<2>(p, stream);
}

}  // namespace skv
