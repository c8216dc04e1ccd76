// norm_rotate.cuh — per-head RMS norm of queries and keys with the rotation by position in the same
// pass, and its backward pass.
//
//   n = x * r * g,  r = 1 / sqrt(mean over the head's columns of x^2 + eps)
//   a pair (u, v) of n's leading `rot` columns becomes (u cos a - v sin a, u sin a + v cos a), a = p * base^(-2 i / rot)
// backward, with dn = the pairs of dy turned by -a:
//   dg = sum over rows and heads of dn * x * r
//   dx = r * (dn * g) - x * r^3 * mean(dn * g * x)
//
// Work split. A head is LPH = d_head / V lanes of V = 16 bytes of columns each, and those LPH lanes take
// one row and walk its heads: the angles of a row are the same for every head, so each pair's sine and
// cosine is formed once per row (V / 2 pairs a lane, handed round by shuffles in the halves layout)
// and the gains stay in registers. A warp's lanes cover 32 / LPH rows; a head's columns are one 64- or
// 128-byte segment, so loads and stores are whole sectors. Everything is held in fp32 and rounded once, at
// the store. Angles are reduced in fp64, in turns: p times base^(-2i/rot) / 2 pi keeps 2^-53 of the
// product where fp32 would lose the angle of a far position.
#pragma once

#include "ptx.cuh"

namespace whale {

constexpr int kNrThreads = 256;
constexpr int kNrMaxPairs = 64;  // d_head <= 128

struct NrPart {
  const void* x;
  void* y;           // forward: output; backward: dx
  const void* dy;    // backward only
  const float* gain;  // [d_head]
  const int* pos;     // [rows]
  long long rows, ldx, ldy, lddy;
  int heads;
};

struct NrArgs {
  NrPart part[2];
  int blocks0;       // blocks [0, blocks0) take part 0, the rest part 1
  int rot;           // leading columns of a head that turn
  float eps;
  float* partial;    // backward: [gridDim.x, d_head] column sums of dg
  double turns[kNrMaxPairs];  // base^(-2 i / rot) / (2 pi)
};

// 16 bytes of columns as fp32.
template <typename T>
struct NrVec;
template <>
struct NrVec<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct NrVec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

template <int LPH>
__device__ __forceinline__ float nr_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sines and cosines that this lane's V columns need, as full-length factors: with w the other column of
// the pair, the rotated column is c * own + s * w. Columns that do not turn get (1, 0).
//  halves:   column e < rot/2 pairs with e + rot/2, held by the lane `hop` lanes on (or back)
//  adjacent: columns 2 i and 2 i + 1 pair, both in this lane; c and s are per pair there
template <int V, int LPH, bool ADJ>
__device__ __forceinline__ void nr_angles(const NrArgs& a, int p, int li, float (&c)[ADJ ? V / 2 : V],
                                          float (&s)[ADJ ? V / 2 : V], int hop) {
  float mc[V / 2], ms[V / 2];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const int i = li * (V / 2) + k;
    mc[k] = 1.f;
    ms[k] = 0.f;
    if (i < a.rot / 2) {
      const double t = (double)p * a.turns[i];
      sincospif((float)(2.0 * (t - rint(t))), &ms[k], &mc[k]);
    }
  }
  if constexpr (ADJ) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      c[k] = mc[k];
      s[k] = ms[k];
    }
  } else {
    // columns e0 .. e0 + V - 1 of pairs (e mod rot/2): formed by lanes 2 l' and 2 l' + 1 of the head
    const int l2 = li < hop ? li : li - hop;  // lane of the pair's first column
    const bool turns = li < 2 * hop;
    const int base = (threadIdx.x & 31 & ~(LPH - 1)) + ((2 * l2) & (LPH - 1));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int src = base + (k >= V / 2 ? 1 : 0);
      const float cc = __shfl_sync(0xffffffffu, mc[k % (V / 2)], src);
      const float ss = __shfl_sync(0xffffffffu, ms[k % (V / 2)], src);
      c[k] = turns ? cc : 1.f;
      s[k] = turns ? (li < hop ? -ss : ss) : 0.f;
    }
  }
}

// y = rotation of n by the factors of nr_angles, `w` = the partner lane's columns (halves layout only)
template <int V, bool ADJ, bool BACK>
__device__ __forceinline__ void nr_turn(const float (&n)[V], const float (&w)[V], const float (&c)[ADJ ? V / 2 : V],
                                        const float (&s)[ADJ ? V / 2 : V], float (&y)[V]) {
  if constexpr (ADJ) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const float sn = BACK ? -s[k] : s[k];
      y[2 * k] = n[2 * k] * c[k] - n[2 * k + 1] * sn;
      y[2 * k + 1] = n[2 * k] * sn + n[2 * k + 1] * c[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] = n[k] * c[k] + w[k] * (BACK ? -s[k] : s[k]);
  }
}

template <typename T, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrThreads) norm_rotate_kernel(const __grid_constant__ NrArgs a) {
  constexpr int V = NrVec<T>::V, LPH = DH / V, RPW = 32 / LPH, HU = 4;
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPH;
  const int hop = a.rot / 2 / V;
  const long long row = ((long long)block * (kNrThreads / 32) + warp) * RPW + lane / LPH;
  const bool live = row < p.rows;  // every lane keeps step: the shuffles need the whole warp
  const long long r0 = live ? row : 0;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + r0 * p.ldx) + li;
  uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(p.y) + r0 * p.ldy) + li;
  if (row - lane / LPH >= p.rows) return;  // a whole warp past the end
  uint4 w[HU];
#pragma unroll
  for (int u = 0; u < HU; ++u)
    if (live && u < p.heads) w[u] = x[u * LPH];
  float g[V], gw[V];  // gains of this lane's columns and of their partners
  const bool turns = !ADJ && li < 2 * hop;
  const int partner = turns ? (li < hop ? lane + hop : lane - hop) : lane;
  const int le = turns ? (li < hop ? li + hop : li - hop) : li;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    g[k] = p.gain[li * V + k];
    gw[k] = p.gain[le * V + k];
  }
  float c[ADJ ? V / 2 : V], s[ADJ ? V / 2 : V];
  nr_angles<V, LPH, ADJ>(a, live ? p.pos[row] : 0, li, c, s, hop);
  for (int h0 = 0; h0 < p.heads; h0 += HU) {
    uint4 nx[HU];
#pragma unroll
    for (int u = 0; u < HU; ++u)
      if (live && h0 + HU + u < p.heads) nx[u] = x[(h0 + HU + u) * LPH];
#pragma unroll
    for (int u = 0; u < HU; ++u) {
      if (h0 + u >= p.heads) break;
      float f[V], v[V], out[V];
      NrVec<T>::unpack(w[u], f);
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) q = fmaf(f[k], f[k], q);
      const float r = rsqrtf(nr_sum<LPH>(q) * (1.0f / DH) + a.eps);
      if constexpr (!ADJ) {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, w[u].x, partner);
        o.y = __shfl_sync(0xffffffffu, w[u].y, partner);
        o.z = __shfl_sync(0xffffffffu, w[u].z, partner);
        o.w = __shfl_sync(0xffffffffu, w[u].w, partner);
        NrVec<T>::unpack(o, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] *= r * gw[k];
      }
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] *= r * g[k];
      nr_turn<V, ADJ, false>(f, v, c, s, out);
      if (live) y[(h0 + u) * LPH] = NrVec<T>::pack(out);
    }
#pragma unroll
    for (int u = 0; u < HU; ++u) w[u] = nx[u];
  }
}

// Gradient rows as fp32, V columns of a lane.
template <typename GT, int V>
__device__ __forceinline__ void nr_load_grad(const GT* row, int col, float (&f)[V]) {
  if constexpr (sizeof(GT) == 4) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float4 t = *reinterpret_cast<const float4*>(row + col + 4 * k);
      f[4 * k] = t.x;
      f[4 * k + 1] = t.y;
      f[4 * k + 2] = t.z;
      f[4 * k + 3] = t.w;
    }
  } else {
    static_assert(sizeof(GT) == 4 || V == 8, "bf16 gradients come with bf16 rows");
    NrVec<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(row + col), f);
  }
}
template <typename GT, int V>
__device__ __forceinline__ void nr_store_grad(GT* row, int col, const float (&f)[V]) {
  if constexpr (sizeof(GT) == 4) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k)
      *reinterpret_cast<float4*>(row + col + 4 * k) = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
  } else {
    *reinterpret_cast<uint4*>(row + col) = NrVec<__nv_bfloat16>::pack(f);
  }
}

// dx, and each block's column sums of dg (a lane keeps its columns over every row and head it takes, so dg
// needs no atomics: the warps' sums meet in shared memory, the blocks' in norm_rotate_gain_kernel, each in a
// fixed order).
template <typename T, typename GT, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrThreads) norm_rotate_backward_kernel(const __grid_constant__ NrArgs a) {
  constexpr int V = NrVec<T>::V, LPH = DH / V, RPW = 32 / LPH, WARPS = kNrThreads / 32;
  __shared__ float sums[WARPS][DH];
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int blocks = second ? gridDim.x - a.blocks0 : a.blocks0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPH;
  const int hop = a.rot / 2 / V;
  const bool turns = !ADJ && li < 2 * hop;
  const int partner = turns ? (li < hop ? lane + hop : lane - hop) : lane;
  float g[V], dg[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    g[k] = p.gain[li * V + k];
    dg[k] = 0.f;
  }
  for (long long base = ((long long)block * WARPS + warp) * RPW; base < p.rows; base += (long long)blocks * WARPS * RPW) {
    const long long row = base + lane / LPH;
    const bool live = row < p.rows;
    const long long r0 = live ? row : 0;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + r0 * p.ldx) + li;
    const GT* dy = static_cast<const GT*>(p.dy) + r0 * p.lddy;
    GT* dx = static_cast<GT*>(p.y) + r0 * p.ldy;
    float c[ADJ ? V / 2 : V], s[ADJ ? V / 2 : V];
    nr_angles<V, LPH, ADJ>(a, live ? p.pos[row] : 0, li, c, s, hop);
#pragma unroll 2
    for (int h = 0; h < p.heads; ++h) {
      float f[V], d[V], e[V], dn[V];
      const uint4 w = live ? x[h * LPH] : make_uint4(0u, 0u, 0u, 0u);
      if (live) nr_load_grad<GT, V>(dy, h * DH + li * V, d);
      else {
#pragma unroll
        for (int k = 0; k < V; ++k) d[k] = 0.f;
      }
      NrVec<T>::unpack(w, f);
      if constexpr (!ADJ) {
#pragma unroll
        for (int k = 0; k < V; ++k) e[k] = __shfl_sync(0xffffffffu, d[k], partner);
      }
      nr_turn<V, ADJ, true>(d, e, c, s, dn);
      float q = 0.f, t = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        q = fmaf(f[k], f[k], q);
        t = fmaf(dn[k] * g[k], f[k], t);
      }
      const float r = rsqrtf(nr_sum<LPH>(q) * (1.0f / DH) + a.eps);
      const float m = nr_sum<LPH>(t) * (1.0f / DH) * r * r * r;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (live) dg[k] = fmaf(dn[k], f[k] * r, dg[k]);  // a dead lane's r is 1 / sqrt(eps): infinite at eps 0
        e[k] = r * dn[k] * g[k] - f[k] * m;
      }
      if (live) nr_store_grad<GT, V>(dx, h * DH + li * V, e);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) dg[k] += __shfl_xor_sync(0xffffffffu, dg[k], o);
    if (lane < LPH) sums[warp][li * V + k] = dg[k];
  }
  __syncthreads();
  for (int col = threadIdx.x; col < DH; col += kNrThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) t += sums[w][col];
    a.partial[(size_t)blockIdx.x * DH + col] = t;
  }
}

// d_gain[part] = the sum of its blocks' partials; one block per part, DH columns x (1024 / DH) strides.
__global__ void __launch_bounds__(1024)
    norm_rotate_gain_kernel(const float* __restrict__ partial, int blocks0, int blocks, int dh, float* g0, float* g1) {
  __shared__ float sums[1024];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.x ? g1 : g0;
  const int lo = blockIdx.x ? blocks0 : 0, hi = blockIdx.x ? blocks : blocks0;
  const int col = threadIdx.x % dh, k0 = threadIdx.x / dh, ks = 1024 / dh;
  float t = 0.f;
  for (int b = lo + k0; b < hi; b += ks) t += partial[(size_t)b * dh + col];
  sums[threadIdx.x] = t;
  __syncthreads();
  if (k0 == 0 && out) {
    for (int k = 1; k < ks; ++k) t += sums[k * dh + col];
    out[col] = t;
  }
}

}  // namespace whale
