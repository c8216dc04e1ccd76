// norm_rotate.cuh — per-head RMS norm of queries and keys with the rotation by position in the same
// pass, and its backward pass.
//
//   n = x * r * g,  r = 1 / sqrt(mean over the head's columns of x^2 + eps)
//   a pair (u, v) of n's leading `rot` columns becomes (u cos a - v sin a, u sin a + v cos a), a = p * base^(-2 i / rot)
// backward, with dn = the pairs of dy turned by -a:
//   dg = sum over rows and heads of dn * x * r
//   dx = r * (dn * g) - x * r^3 * mean(dn * g * x)
//
// Work split. A head is LPH = d_head / V lanes of V columns (16 bytes) each, and those LPH lanes take one row
// and walk its heads: the angles of a row are the same for every head, so each sine and cosine is formed once per
// row, by the lane that uses it, and multiplied into the gains. A lane holds both columns of its V / 2 pairs
// (halves layout: two 8-byte pieces rot / 2 apart), so nothing passes between lanes but the sum of squares. A
// warp's lanes cover 32 / LPH rows; a head's columns are one segment of 32 bytes or more, so loads and stores are whole
// sectors. The next kNrHeads heads (the next row's first ones at a row's end) are loaded before the
// present ones are used. Everything is held in fp32 and rounded once, at the store. Angles are reduced
// in fp64, in turns: p times base^(-2i/rot) / 2 pi keeps 2^-53 of the product where fp32 would lose the angle of a
// far position.
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

// V columns of a lane as fp32, read and written as two pieces of C = V / 2 columns.
template <typename T, int V>
struct NrRaw {
  uint32_t w[V * sizeof(T) / 4];
};
template <typename T, int V>
__device__ __forceinline__ NrRaw<T, V> nr_load(const T* row, int o1, int o2, bool whole) {
  NrRaw<T, V> r;
  constexpr int N = V * sizeof(T) / 4;  // words: 4, or 8 (fp32 gradients of bf16 rows)
  if constexpr (N == 4) {
    if (whole) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + o1);
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(row + o1), b = *reinterpret_cast<const uint2*>(row + o2);
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
    }
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(row + o1), b = *reinterpret_cast<const uint4*>(row + o2);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void nr_unpack(const NrRaw<T, V>& r, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(r.w[i]);
    else f[i] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
  }
}
template <typename T, int V>
__device__ __forceinline__ void nr_store(T* row, int o1, int o2, bool whole, const float (&f)[V]) {
  uint32_t w[V * sizeof(T) / 4];
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(f[i]);
      w[i + 1] = __float_as_uint(f[i + 1]);
    } else {
      w[i / 2] = pack_bf16x2(f[i], f[i + 1]);
    }
  }
  if constexpr (V * sizeof(T) == 16) {
    if (whole) {
      *reinterpret_cast<uint4*>(row + o1) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + o1) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + o2) = make_uint2(w[2], w[3]);
    }
  } else {
    *reinterpret_cast<uint4*>(row + o1) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + o2) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int LPH>
__device__ __forceinline__ float nr_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane's columns are: pieces [o1, o1 + V/2) and [o2, o2 + V/2) of the head. Pair k of the lane is
// (f[k], f[V/2 + k]) in the halves layout, (f[2k], f[2k+1]) in the adjacent one; it is pair first + k of the head, and turns if
// that is below rot / 2. Columns past rot come in the same form and do not turn.
struct NrLane {
  int o1, o2, first;
};
template <int V, bool ADJ>
__device__ __forceinline__ NrLane nr_lane(int rot, int li) {
  constexpr int C = V / 2;
  NrLane l;
  l.first = li * C;
  const bool turns = !ADJ && l.first < rot / 2;
  l.o1 = turns ? l.first : (ADJ ? li * V : rot + (l.first - rot / 2) * 2);
  l.o2 = turns ? rot / 2 + l.first : l.o1 + C;
  return l;
}
template <bool ADJ, int V>
__device__ __forceinline__ constexpr int nr_a(int k) { return ADJ ? 2 * k : k; }
template <bool ADJ, int V>
__device__ __forceinline__ constexpr int nr_b(int k) { return ADJ ? 2 * k + 1 : V / 2 + k; }

template <int C>
__device__ __forceinline__ void nr_angles(const NrArgs& a, int p, int first, float (&c)[C], float (&s)[C]) {
#pragma unroll
  for (int k = 0; k < C; ++k) {
    c[k] = 1.f;
    s[k] = 0.f;
    if (first + k < a.rot / 2) {
      const double t = (double)p * a.turns[first + k];
      sincospif((float)(2.0 * (t - rint(t))), &s[k], &c[k]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void nr_gains(const float* gain, const NrLane& l, float (&g)[V]) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    g[k] = gain[l.o1 + k];
    g[V / 2 + k] = gain[l.o2 + k];
  }
}

constexpr int kNrHeads = 4;

template <typename T, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrThreads) norm_rotate_kernel(const __grid_constant__ NrArgs a) {
  constexpr int V = 16 / sizeof(T), C = V / 2, LPH = DH / V, RPW = 32 / LPH, HU = kNrHeads, WARPS = kNrThreads / 32;
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int blocks = second ? gridDim.x - a.blocks0 : a.blocks0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const NrLane l = nr_lane<V, ADJ>(a.rot, lane % LPH);
  const bool whole = l.o2 == l.o1 + C;
  const long long step = (long long)blocks * WARPS * RPW;
  long long base = ((long long)block * WARPS + warp) * RPW;
  if (base >= p.rows) return;
  long long row = base + lane / LPH;  // past the end: the last row, not stored (the shuffles need the whole warp)
  auto src_of = [&](long long r) { return static_cast<const T*>(p.x) + (r < p.rows ? r : p.rows - 1) * p.ldx; };
  const T* x = src_of(row);
  NrRaw<T, V> w[HU], nx[HU];
#pragma unroll
  for (int u = 0; u < HU; ++u)
    if (u < p.heads) w[u] = nr_load<T, V>(x + u * DH, l.o1, l.o2, whole);
  int pos = p.pos[row < p.rows ? row : p.rows - 1];
  float g[V];
  nr_gains<T, V>(p.gain, l, g);
  for (; base < p.rows; base += step) {
    row = base + lane / LPH;
    const bool live = row < p.rows, more = base + step < p.rows;
    T* y = static_cast<T*>(p.y) + (live ? row : 0) * p.ldy;
    const T* next = src_of(row + step);
    const int next_pos = more ? p.pos[row + step < p.rows ? row + step : p.rows - 1] : 0;
    // turn and gain in one: y_a = r (a ca - b sb), y_b = r (a sa + b cb)
    float ca[C], sa[C], cb[C], sb[C];
    {
      float c[C], s[C];
      nr_angles<C>(a, pos, l.first, c, s);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float ga = g[nr_a<ADJ, V>(k)], gb = g[nr_b<ADJ, V>(k)];
        ca[k] = c[k] * ga;
        sa[k] = s[k] * ga;
        cb[k] = c[k] * gb;
        sb[k] = s[k] * gb;
      }
    }
    for (int h0 = 0; h0 < p.heads; h0 += HU) {
      const bool last = h0 + HU >= p.heads;
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        if (!last) {
          if (h0 + HU + u < p.heads) nx[u] = nr_load<T, V>(x + (h0 + HU + u) * DH, l.o1, l.o2, whole);
        } else if (more && u < p.heads) {
          nx[u] = nr_load<T, V>(next + u * DH, l.o1, l.o2, whole);
        }
      }
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        if (h0 + u < p.heads) {
          float f[V], out[V];
          nr_unpack<T, V>(w[u], f);
          float q0 = 0.f, q1 = 0.f;
#pragma unroll
          for (int k = 0; k < V; k += 2) {
            q0 = fmaf(f[k], f[k], q0);
            q1 = fmaf(f[k + 1], f[k + 1], q1);
          }
          const float r = rsqrtf(nr_sum<LPH>(q0 + q1) * (1.0f / DH) + a.eps);
#pragma unroll
          for (int k = 0; k < C; ++k) {
            const float xa = f[nr_a<ADJ, V>(k)], xb = f[nr_b<ADJ, V>(k)];
            out[nr_a<ADJ, V>(k)] = (xa * ca[k] - xb * sb[k]) * r;
            out[nr_b<ADJ, V>(k)] = (xa * sa[k] + xb * cb[k]) * r;
          }
          if (live) nr_store<T, V>(y + (h0 + u) * DH, l.o1, l.o2, whole, out);
        }
      }
#pragma unroll
      for (int u = 0; u < HU; ++u) w[u] = nx[u];
    }
    x = next;
    pos = next_pos;
  }
}

// dx, and each block's column sums of dg (a lane keeps its columns over every row and head it takes, so dg
// needs no atomics: the warps' sums meet in shared memory, the blocks' in norm_rotate_gain_kernel, each in a
// fixed order).
template <typename T, typename GT, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrThreads) norm_rotate_backward_kernel(const __grid_constant__ NrArgs a) {
  constexpr int V = 16 / sizeof(T), C = V / 2, LPH = DH / V, RPW = 32 / LPH, WARPS = kNrThreads / 32, HU = 2;
  __shared__ float sums[WARPS][DH];
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int blocks = second ? gridDim.x - a.blocks0 : a.blocks0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const NrLane l = nr_lane<V, ADJ>(a.rot, lane % LPH);
  const bool whole = l.o2 == l.o1 + C;
  float g[V], dg[V];
  nr_gains<T, V>(p.gain, l, g);
#pragma unroll
  for (int k = 0; k < V; ++k) dg[k] = 0.f;
  const long long step = (long long)blocks * WARPS * RPW;
  for (long long base = ((long long)block * WARPS + warp) * RPW; base < p.rows; base += step) {
    const long long row = base + lane / LPH;
    const bool live = row < p.rows;
    const long long r0 = live ? row : p.rows - 1;
    const T* x = static_cast<const T*>(p.x) + r0 * p.ldx;
    const GT* dy = static_cast<const GT*>(p.dy) + r0 * p.lddy;
    GT* dx = static_cast<GT*>(p.y) + r0 * p.ldy;
    NrRaw<T, V> wx[HU], nx[HU];
    NrRaw<GT, V> wd[HU], nd[HU];
#pragma unroll
    for (int u = 0; u < HU; ++u)
      if (u < p.heads) {
        wx[u] = nr_load<T, V>(x + u * DH, l.o1, l.o2, whole);
        wd[u] = nr_load<GT, V>(dy + u * DH, l.o1, l.o2, whole);
      }
    float c[C], s[C];
    nr_angles<C>(a, p.pos[r0], l.first, c, s);
    for (int h0 = 0; h0 < p.heads; h0 += HU) {
#pragma unroll
      for (int u = 0; u < HU; ++u)
        if (h0 + HU + u < p.heads) {
          nx[u] = nr_load<T, V>(x + (h0 + HU + u) * DH, l.o1, l.o2, whole);
          nd[u] = nr_load<GT, V>(dy + (h0 + HU + u) * DH, l.o1, l.o2, whole);
        }
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        if (h0 + u < p.heads) {
          float f[V], d[V], dn[V], e[V];
          nr_unpack<T, V>(wx[u], f);
          nr_unpack<GT, V>(wd[u], d);
          float q = 0.f, t = 0.f;
#pragma unroll
          for (int k = 0; k < C; ++k) {
            constexpr auto A = nr_a<ADJ, V>;
            constexpr auto B = nr_b<ADJ, V>;
            dn[A(k)] = d[A(k)] * c[k] + d[B(k)] * s[k];
            dn[B(k)] = d[B(k)] * c[k] - d[A(k)] * s[k];
          }
#pragma unroll
          for (int k = 0; k < V; ++k) {
            q = fmaf(f[k], f[k], q);
            e[k] = dn[k] * g[k];
            t = fmaf(e[k], f[k], t);
          }
          const float r = rsqrtf(nr_sum<LPH>(q) * (1.0f / DH) + a.eps);
          const float m = nr_sum<LPH>(t) * (1.0f / DH) * r * r * r;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if (live) dg[k] = fmaf(dn[k], f[k] * r, dg[k]);  // a row past the end counts once
            e[k] = r * e[k] - f[k] * m;
          }
          if (live) nr_store<GT, V>(dx + (h0 + u) * DH, l.o1, l.o2, whole, e);
        }
      }
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        wx[u] = nx[u];
        wd[u] = nd[u];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) dg[k] += __shfl_xor_sync(0xffffffffu, dg[k], o);
    if (lane < LPH) sums[warp][k < C ? l.o1 + k : l.o2 + k - C] = dg[k];
  }
  __syncthreads();
  for (int col = threadIdx.x; col < DH; col += kNrThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) t += sums[w][col];
    a.partial[(size_t)blockIdx.x * DH + col] = t;
  }
}

// d_gain[part] = the sum of its blocks' partials, in fp64 (the partials are large beside what a rounding of
// theirs may lose); one block per part, DH columns x (1024 / DH) strides.
__global__ void __launch_bounds__(1024)
    norm_rotate_gain_kernel(const float* __restrict__ partial, int blocks0, int blocks, int dh, float* g0, float* g1) {
  __shared__ double sums[1024];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.x ? g1 : g0;
  const int lo = blockIdx.x ? blocks0 : 0, hi = blockIdx.x ? blocks : blocks0;
  const int col = threadIdx.x % dh, k0 = threadIdx.x / dh, ks = 1024 / dh;
  double t = 0.0;
  for (int b = lo + k0; b < hi; b += ks) t += (double)partial[(size_t)b * dh + col];
  sums[threadIdx.x] = t;
  __syncthreads();
  if (k0 == 0 && out) {
    for (int k = 1; k < ks; ++k) t += sums[k * dh + col];
    out[col] = (float)t;
  }
}

}  // namespace whale
