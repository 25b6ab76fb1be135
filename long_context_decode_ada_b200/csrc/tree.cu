// tree.cu -- attention of the drafted tokens of a tree over the paged store:
// every row (drafted token i, query head) sees the store's resident tokens
// and the drafted tokens its mask names, with scores optionally capped by a
// tanh or biased by distance (the same keys and values as the decode: logits
// from the radius and angle codes, int8 or fp16 values).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace skv {

namespace {

constexpr int kTreeThreads = 128;
constexpr int kTreeWarps = kTreeThreads / 32;

// Positions of the store's rows: row_pos[page * P + row] = t, by the row map.
__global__ void __launch_bounds__(256) tree_positions_kernel(const __grid_constant__ TreeParams p) {
  const long long u = blockIdx.y;
  const long long T = min((long long)p.seq_lens[u / p.Hkv], p.Tmax);
  const long long a = p.indptr[u], rows = ((long long)p.indptr[u + 1] - a) * p.P;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < T;
       t += (long long)gridDim.x * blockDim.x) {
    const long long r = p.row_of[u * p.Tmax + t];
    if (r < 0) continue;
    if (a < 0 || r >= rows || a * p.P + r >= p.page_cap * p.P)
      report(p.err, SKV_ERR_CORRUPT);
    else
      p.row_pos[a * p.P + r] = (int32_t)t;
  }
}

__device__ __forceinline__ float load16(const void* base, long long i, int bf16) {
  const uint16_t x = static_cast<const uint16_t*>(base)[i];
  return bf16 ? __bfloat162float(__ushort_as_bfloat16(x)) : __half2float(__ushort_as_half(x));
}

// The four key components 4 lane .. 4 lane + 3 of row `row` of a page.
__device__ __forceinline__ void key4(const TreeParams& p, const uint8_t* page, int tier, int row,
                                     int lane, float (&k)[4]) {
  if (tier == SKV_TIER_T0) {
    const uint2 w = *reinterpret_cast<const uint2*>(
        page + kHdrBytes + row * 256 + (((lane >> 1) ^ (4 * (row & 1))) * 16) + (lane & 1) * 8);
    const __half2 a = *reinterpret_cast<const __half2*>(&w.x);
    const __half2 b = *reinterpret_cast<const __half2*>(&w.y);
    k[0] = __low2float(a);
    k[1] = __high2float(a);
    k[2] = __low2float(b);
    k[3] = __high2float(b);
    return;
  }
  const uint8_t* rs = page + kHdrBytes;
  const float r = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(rs + 2 * row)));
  const int cb = tier == SKV_TIER_T1 ? 64 : 48;
  const uint8_t* c = rs + 2 * p.P + cb * row;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int pr = 2 * lane + e;
    const int g = (pr & 15) >> 2, j = 4 * (pr >> 4) + (pr & 3);
    float cs, sn, w;
    if (tier == SKV_TIER_T1) {
      const uint32_t x = c[16 * g + j];
      if (p.t1_scheme) {
        cs = p.cos5[x >> 3];
        sn = p.sin5[x >> 3];
        w = (float)((x & 7) + 1) / 32.0f;
      } else {
        cs = p.cos6[x >> 2];
        sn = p.sin6[x >> 2];
        w = p.rho[x & 3];
      }
    } else {
      const uint32_t a = (c[8 * g + (j >> 1)] >> (4 * (j & 1))) & 15u;
      const uint32_t s = (c[32 + 4 * g + (j >> 2)] >> (2 * (j & 3))) & 3u;
      cs = p.cos4[a];
      sn = p.sin4[a];
      w = p.rho[s];
    }
    k[2 * e] = r * w * cs;
    k[2 * e + 1] = r * w * sn;
  }
}

__device__ __forceinline__ void value4(const TreeParams& p, const uint8_t* page, int tier, int row,
                                       int lane, float (&v)[4]) {
  if (tier == SKV_TIER_T0) {
    const uint8_t* vs = page + kHdrBytes + 256 * p.P;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = __half2float(__ushort_as_half(
          *reinterpret_cast<const uint16_t*>(vs + v_frag_offset(row, 4 * lane + e, 2))));
    return;
  }
  const int cb = tier == SKV_TIER_T1 ? 64 : 48;
  const uint8_t* ss = page + kHdrBytes + (2 + cb) * p.P;
  const float s = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(ss + 2 * row)));
  const int8_t* vs = reinterpret_cast<const int8_t*>(ss + 2 * p.P);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = s * (float)vs[v_frag_offset(row, 4 * lane + e, 1)];
}

template <int G>
struct TreeState {
  float m[G], l[G], o[G][4];
};

// One key / value into the running softmax of the G heads (log2 domain).
template <int G>
__device__ __forceinline__ void tree_step(const TreeParams& p, TreeState<G>& st,
                                          const float (&q)[G][4], const float (&slope)[G],
                                          const float (&k)[4], const float (&v)[4], float dist) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float s = q[g][0] * k[0] + q[g][1] * k[1] + q[g][2] * k[2] + q[g][3] * k[3];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= p.qk_scale;
    if (p.softcap > 0.0f) s = p.softcap * tanhf(s / p.softcap);
    s = (s - slope[g] * dist) * 1.4426950408889634f;
    const float mn = fmaxf(st.m[g], s);
    const float a = st.m[g] == mn ? 1.0f : exp2f(st.m[g] - mn);
    const float w = mn == -INFINITY ? 0.0f : exp2f(s - mn);
    st.l[g] = st.l[g] * a + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) st.o[g][e] = st.o[g][e] * a + w * v[e];
    st.m[g] = mn;
  }
}

// A block per (unit, drafted token): its warps share the rows of each page,
// warp 0 takes the drafted tokens, and the four states meet at the end.
template <int G>
__global__ void __launch_bounds__(kTreeThreads)
    tree_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float sm[kTreeWarps][G][2];
  __shared__ float so[kTreeWarps][G][kHeadDim];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long u = blockIdx.x / p.N;
  const int i = (int)(blockIdx.x - u * p.N);
  const int b = (int)(u / p.Hkv), h = (int)(u - (long long)b * p.Hkv);
  const int n = p.count ? min(max(p.count[b], 0), p.N) : p.N;
  if (i >= n) return;
  const long long tok = (long long)b * p.N + i;
  float q[G][4], slope[G];
  TreeState<G> st;
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[g][e] = load16(p.q, tok * p.q_stride + (long long)(h * G + g) * kHeadDim + 4 * lane + e,
                       p.q_bf16);
      st.o[g][e] = 0.0f;
    }
    slope[g] = p.slopes ? p.slopes[h * G + g] : 0.0f;
    st.m[g] = -INFINITY;
    st.l[g] = 0.0f;
  }
  const int qpos = p.slopes ? p.q_pos[tok] : 0;
  const long long g0 = max(0, p.indptr[u]), g1 = min((long long)p.indptr[u + 1], p.page_cap);
  for (long long pg = g0; pg < g1; ++pg) {
    const uint32_t id = p.ids[pg];
    const int tier = (int)(id >> 30);
    const long long slot = id & 0x3FFFFFFFu;
    if (tier > 2 || slot >= p.slots[tier]) {
      if (threadIdx.x == 0) report(p.err, SKV_ERR_CORRUPT);
      continue;
    }
    const uint8_t* page = p.pool[tier] + slot * p.stride[tier];
    const uint32_t hdr = *reinterpret_cast<const uint32_t*>(page);
    const int rows = (int)(hdr & 0xFFFFu);
    if ((hdr >> 16) != ((uint32_t)tier | ((uint32_t)kPageMagic << 8)) || rows > p.P) {
      if (threadIdx.x == 0) report(p.err, SKV_ERR_CORRUPT);
      continue;
    }
    for (int r = w; r < rows; r += kTreeWarps) {
      float k[4], v[4];
      key4(p, page, tier, r, lane, k);
      value4(p, page, tier, r, lane, v);
      const float dist = p.slopes ? (float)(qpos - p.row_pos[pg * p.P + r]) : 0.0f;
      tree_step<G>(p, st, q, slope, k, v, dist);
    }
  }
  if (p.K && w == 0) {
    unsigned long long bits = p.mask ? p.mask[tok] : (i == 63 ? ~0ull : (2ull << i) - 1);
    if (n < 64) bits &= (1ull << n) - 1;
    while (bits) {
      const int j = __ffsll((long long)bits) - 1;
      bits &= bits - 1;
      const long long at = ((long long)b * p.N + j) * p.kv_stride + (long long)h * kHeadDim;
      float k[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[e] = load16(p.K, at + 4 * lane + e, p.kv_bf16);
        v[e] = load16(p.V, at + 4 * lane + e, p.kv_bf16);
      }
      const float dist = p.slopes ? (float)(qpos - p.q_pos[(long long)b * p.N + j]) : 0.0f;
      tree_step<G>(p, st, q, slope, k, v, dist);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (lane == 0) {
      sm[w][g][0] = st.m[g];
      sm[w][g][1] = st.l[g];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) so[w][g][4 * lane + e] = st.o[g][e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < G * kHeadDim; x += kTreeThreads) {
    const int g = x / kHeadDim, d = x % kHeadDim;
    float M = -INFINITY, L = 0.0f, o = 0.0f;
    for (int k = 0; k < kTreeWarps; ++k) M = fmaxf(M, sm[k][g][0]);
    for (int k = 0; k < kTreeWarps; ++k) {
      const float a = sm[k][g][0] == M ? 1.0f : exp2f(sm[k][g][0] - M);
      L += a * sm[k][g][1];
      o += a * so[k][g][d];
    }
    o = L > 0.0f ? o / L : (L == 0.0f ? 0.0f : o);
    const long long at = (tok * p.Hq + h * G + g) * kHeadDim + d;
    if (p.q_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(o);
    if (d == 0 && p.lse)
      p.lse[tok * p.Hq + h * G + g] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  const long long U = (long long)p.B * p.Hkv;
  if (U == 0) return cudaSuccess;
  if (U * p.N > 0x7FFFFFFFLL || U > 65535) return cudaErrorInvalidValue;
  if (p.slopes && p.Tmax > 0) {
    const long long bx = std::min<long long>((p.Tmax + 255) / 256, std::max<long long>(1, 1184 / U));
    tree_positions_kernel<<<dim3((unsigned)bx, (unsigned)U), 256, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)(U * p.N);
  switch (p.Hq / p.Hkv) {
    case 1: tree_kernel<1><<<grid, kTreeThreads, 0, stream>>>(p); break;
    case 2: tree_kernel<2><<<grid, kTreeThreads, 0, stream>>>(p); break;
    default: tree_kernel<4><<<grid, kTreeThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace skv
