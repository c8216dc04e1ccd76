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
// in 64-bit fixed point: a position times the fraction of a turn that one position turns, modulo 1, keeps 2^-31 of
// a turn at any position, where fp32 would lose the angle of a far one.
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
  unsigned long long turns[kNrMaxPairs];  // fraction of base^(-2 i / rot) / (2 pi), times 2^64
};

// V columns of a lane as fp32, read and written as two pieces of C = V / 2 columns (one piece of V in the adjacent layout).
template <typename T, int V>
struct NrRaw {
  uint32_t w[V * sizeof(T) / 4];
};
template <typename T, int V, bool ADJ>
__device__ __forceinline__ NrRaw<T, V> nr_load(const T* p1, const T* p2) {
  NrRaw<T, V> r;
  if constexpr (V * sizeof(T) == 32) {  // fp32 gradients of bf16 rows
    const uint4 a = *reinterpret_cast<const uint4*>(p1), b = *reinterpret_cast<const uint4*>(p2);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  } else if constexpr (ADJ) {
    const uint4 a = *reinterpret_cast<const uint4*>(p1);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p1), b = *reinterpret_cast<const uint2*>(p2);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
  }
  return r;
}
// First columns of the lane's pairs in f[0 .. C), second ones in f[C .. V): column i of the two pieces is
// f[nr_slot(i)].
template <int V, bool ADJ>
__host__ __device__ constexpr int nr_slot(int i) {
  return ADJ ? i / 2 + (i & 1) * (V / 2) : i;
}
template <typename T, int V, bool ADJ>
__device__ __forceinline__ void nr_unpack(const NrRaw<T, V>& r, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 4) f[nr_slot<V, ADJ>(i)] = __uint_as_float(r.w[i]);
    else f[nr_slot<V, ADJ>(i)] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
  }
}
template <typename T, int V, bool ADJ>
__device__ __forceinline__ void nr_store(T* p1, T* p2, const float (&f)[V]) {
  uint32_t w[V * sizeof(T) / 4];
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float x0 = f[nr_slot<V, ADJ>(i)], x1 = f[nr_slot<V, ADJ>(i + 1)];
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(x0);
      w[i + 1] = __float_as_uint(x1);
    } else {
      w[i / 2] = pack_bf16x2(x0, x1);
    }
  }
  if constexpr (V * sizeof(T) == 32) {
    *reinterpret_cast<uint4*>(p1) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p2) = make_uint4(w[4], w[5], w[6], w[7]);
  } else if constexpr (ADJ) {
    *reinterpret_cast<uint4*>(p1) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(p1) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p2) = make_uint2(w[2], w[3]);
  }
}

// The angles' table in shared memory: lanes read different entries, which the parameter bank would serve one by one.
__device__ __forceinline__ void nr_table(const NrArgs& a, unsigned long long (&turns)[kNrMaxPairs]) {
  if (threadIdx.x < kNrMaxPairs) turns[threadIdx.x] = a.turns[threadIdx.x];
  __syncthreads();
}

template <int LPH>
__device__ __forceinline__ float nr_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane's columns are: pieces [o1, o1 + V/2) and [o2, o2 + V/2) of the head. Its pairs are the head's pairs
// first, first + 1, ..; they turn below rot / 2. Columns past rot come in the same form and do not turn.
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
// FAST (bf16 rows): sines and cosines off by up to 2^-20, far below a rounding of the result.
template <int C, bool FAST>
__device__ __forceinline__ void nr_angles(const unsigned long long* turns, int rot, int p, int first, float (&c)[C],
                                          float (&s)[C]) {
#pragma unroll
  for (int k = 0; k < C; ++k) {
    c[k] = 1.f;
    s[k] = 0.f;
    if (first + k < rot / 2) {
      const unsigned long long t = (unsigned long long)(long long)p * turns[first + k];
      const float half_turns = (float)(int)(t >> 32) * 0x1p-31f;  // in [-1, 1]
      if constexpr (FAST) __sincosf(half_turns * 3.14159265358979f, &s[k], &c[k]);
      else sincospif(half_turns, &s[k], &c[k]);
    }
  }
}

// Column of the head that f[j] holds.
template <int V, bool ADJ>
__device__ __forceinline__ int nr_col(const NrLane& l, int j) {
  constexpr int C = V / 2;
  if constexpr (ADJ) return l.o1 + 2 * (j % C) + j / C;
  else return j < C ? l.o1 + j : l.o2 + j - C;
}
template <int V, bool ADJ>
__device__ __forceinline__ void nr_gains(const float* gain, const NrLane& l, float (&g)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) g[j] = gain[nr_col<V, ADJ>(l, j)];
}

// Sum of the V products, two at a time.
template <int V>
__device__ __forceinline__ float nr_dot(const float (&x)[V], const float (&y)[V]) {
  uint64_t q = fmul2(f2pack(x[0], x[1]), f2pack(y[0], y[1]));
#pragma unroll
  for (int k = 2; k < V; k += 2) q = ffma2(f2pack(x[k], x[k + 1]), f2pack(y[k], y[k + 1]), q);
  float q0, q1;
  f2unpack(q, q0, q1);
  return q0 + q1;
}

constexpr int kNrHeads = 4;
constexpr int kNrFwdBlocksPerSM = 3;  // resident at once

// A warp's rows, one block of which is resident from start to end. FULL: the heads are a multiple of kNrHeads.
template <typename T, int DH, bool ADJ, bool FULL>
__device__ __forceinline__ void norm_rotate_rows(const NrArgs& a, const NrPart& p, const unsigned long long* turns,
                                                 long long base, long long step) {
  constexpr int V = 16 / sizeof(T), C = V / 2, LPH = DH / V, HU = kNrHeads;
  const int lane = threadIdx.x & 31;
  const NrLane l = nr_lane<V, ADJ>(a.rot, lane % LPH);
  const int heads = p.heads, gap = l.o2 - l.o1;
  // past the end: the last row, not stored (the shuffles need the whole warp)
  long long row = base + lane / LPH;
  auto src_of = [&](long long r) { return static_cast<const T*>(p.x) + (r < p.rows ? r : p.rows - 1) * p.ldx + l.o1; };
  const T* x = src_of(row);
  NrRaw<T, V> w[HU], nx[HU];
#pragma unroll
  for (int u = 0; u < HU; ++u)
    if (FULL || u < heads) w[u] = nr_load<T, V, ADJ>(x + u * DH, x + u * DH + gap);
  int pos = p.pos[row < p.rows ? row : p.rows - 1];
  float g[V];
  nr_gains<V, ADJ>(p.gain, l, g);
  for (; base < p.rows; base += step) {
    row = base + lane / LPH;
    const bool live = row < p.rows, more = base + step < p.rows;
    T* y = static_cast<T*>(p.y) + (live ? row : 0) * p.ldy + l.o1;
    const T* next = src_of(row + step);
    const int next_pos = p.pos[row + step < p.rows ? row + step : p.rows - 1];
    // turn and gain in one: y_a = r (a ca - b sb), y_b = r (a sa + b cb)
    float ca[C], sa[C], cb[C], sb[C];
    {
      float c[C], s[C];
      nr_angles<C, sizeof(T) == 2>(turns, a.rot, pos, l.first, c, s);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        ca[k] = c[k] * g[k];
        sa[k] = s[k] * g[k];
        cb[k] = c[k] * g[C + k];
        sb[k] = -s[k] * g[C + k];
      }
    }
#pragma unroll 1
    for (int h0 = 0; h0 < heads; h0 += HU) {
      x = h0 + HU < heads ? x + HU * DH : next;
      if (h0 + HU < heads || more) {
#pragma unroll
        for (int u = 0; u < HU; ++u)
          if (FULL || (h0 + HU < heads ? h0 + HU + u : u) < heads) nx[u] = nr_load<T, V, ADJ>(x + u * DH, x + u * DH + gap);
      }
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        if (FULL || h0 + u < heads) {
          float f[V], out[V];
          nr_unpack<T, V, ADJ>(w[u], f);
          const float r = rsqrtf(nr_sum<LPH>(nr_dot<V>(f, f)) * (1.0f / DH) + a.eps);
#pragma unroll
          for (int k = 0; k < C; k += 2) {
            const uint64_t xa = f2pack(f[k], f[k + 1]), xb = f2pack(f[C + k], f[C + k + 1]), rr = f2pack(r, r);
            const uint64_t ya = fmul2(ffma2(xa, f2pack(ca[k], ca[k + 1]), fmul2(xb, f2pack(sb[k], sb[k + 1]))), rr);
            const uint64_t yb = fmul2(ffma2(xb, f2pack(cb[k], cb[k + 1]), fmul2(xa, f2pack(sa[k], sa[k + 1]))), rr);
            f2unpack(ya, out[k], out[k + 1]);
            f2unpack(yb, out[C + k], out[C + k + 1]);
          }
          if (live) nr_store<T, V, ADJ>(y + u * DH, y + u * DH + gap, out);
        }
      }
      y += HU * DH;
#pragma unroll
      for (int u = 0; u < HU; ++u) w[u] = nx[u];
    }
    pos = next_pos;
  }
}

template <typename T, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrThreads, kNrFwdBlocksPerSM) norm_rotate_kernel(const __grid_constant__ NrArgs a) {
  constexpr int RPW = 32 / (DH * (int)sizeof(T) / 16), WARPS = kNrThreads / 32;
  __shared__ __align__(16) unsigned long long turns[kNrMaxPairs];
  nr_table(a, turns);
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int blocks = second ? gridDim.x - a.blocks0 : a.blocks0;
  const long long base = ((long long)block * WARPS + (threadIdx.x >> 5)) * RPW, step = (long long)blocks * WARPS * RPW;
  if (base >= p.rows) return;
  if (p.heads % kNrHeads == 0) norm_rotate_rows<T, DH, ADJ, true>(a, p, turns, base, step);
  else norm_rotate_rows<T, DH, ADJ, false>(a, p, turns, base, step);
}

// The backward's ring: a thread brings its own pieces of kNrStages - 1 steps ahead into its own slots of shared memory by
// cp.async (no other thread reads them, so no barrier either). Small blocks, so that the registers hold 20 warps an SM
// and not 16. 512 + 109605 rows, d 512, bf16: 61 us, 5.6 TB/s; with blocks of 256 threads 68 us; with one step
// ahead in registers instead of the ring 78 us.
constexpr int kNrBwdThreads = 128, kNrStages = 3, kNrStepHeads = 2;
template <typename T, typename GT>
struct NrRing {
  static constexpr int V = 16 / sizeof(T);
  static constexpr int ITEMS = kNrStepHeads * (1 + V * (int)sizeof(GT) / 16);  // 16-byte slots of a step
  static constexpr int SMEM = kNrStages * ITEMS * kNrBwdThreads * 16;
  static constexpr int BLOCKS = sizeof(T) == 4 ? 7 : (sizeof(GT) == 4 ? 4 : 5);  // resident at once: what registers and ring allow
};
inline int nr_backward_blocks_per_sm(bool bf16_rows, bool bf16_grads) {
  return !bf16_rows ? NrRing<float, float>::BLOCKS
                    : (bf16_grads ? NrRing<__nv_bfloat16, __nv_bfloat16>::BLOCKS : NrRing<__nv_bfloat16, float>::BLOCKS);
}
template <int BYTES>
__device__ __forceinline__ void nr_copy(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// A lane's pieces into its slots (slot stride: the block's threads), and back.
template <typename T, int V, bool ADJ>
__device__ __forceinline__ void nr_fetch(uint32_t slot, const T* p1, const T* p2) {
  if constexpr (V * sizeof(T) == 32) {
    nr_copy<16>(slot, p1);
    nr_copy<16>(slot + 16 * kNrBwdThreads, p2);
  } else if constexpr (ADJ) {
    nr_copy<16>(slot, p1);
  } else {
    nr_copy<8>(slot, p1);
    nr_copy<8>(slot + 8, p2);
  }
}
template <typename T, int V>
__device__ __forceinline__ NrRaw<T, V> nr_take(uint32_t slot) {
  NrRaw<T, V> r;
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 16; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[4 * i]), "=r"(r.w[4 * i + 1]), "=r"(r.w[4 * i + 2]), "=r"(r.w[4 * i + 3])
                 : "r"(slot + 16 * kNrBwdThreads * i));
  return r;
}

// dx, and each block's column sums of dg (a lane keeps its columns over every row and head it takes, so dg
// needs no atomics: the warps' sums meet in shared memory, the blocks' in norm_rotate_gain_kernel, each in a
// fixed order).
template <typename T, typename GT, int DH, bool ADJ>
__global__ void __launch_bounds__(kNrBwdThreads, NrRing<T, GT>::BLOCKS)
    norm_rotate_backward_kernel(const __grid_constant__ NrArgs a) {
  using R = NrRing<T, GT>;
  constexpr int V = R::V, C = V / 2, LPH = DH / V, RPW = 32 / LPH, WARPS = kNrBwdThreads / 32, HU = kNrStepHeads;
  constexpr int GI = V * (int)sizeof(GT) / 16;  // slots of a head's gradient piece
  extern __shared__ __align__(16) uint8_t nr_ring[];
  __shared__ float sums[WARPS][DH];
  __shared__ __align__(16) unsigned long long turns[kNrMaxPairs];
  nr_table(a, turns);
  pdl_wait();
  pdl_trigger();
  const int second = blockIdx.x >= (unsigned)a.blocks0;
  const NrPart& p = a.part[second];
  const int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int blocks = second ? gridDim.x - a.blocks0 : a.blocks0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = p.heads;
  const NrLane l = nr_lane<V, ADJ>(a.rot, lane % LPH);
  const int gap = l.o2 - l.o1;
  const uint32_t ring = smem_u32(nr_ring) + threadIdx.x * 16;
  float g[V], dg[V];
  nr_gains<V, ADJ>(p.gain, l, g);
#pragma unroll
  for (int k = 0; k < V; ++k) dg[k] = 0.f;
  const long long step = (long long)blocks * WARPS * RPW;
  long long base = ((long long)block * WARPS + warp) * RPW;
  // past the end: the last row, which counts nowhere (the shuffles need the whole warp)
  auto row_of = [&](long long b) {
    const long long r = b + lane / LPH;
    return r < p.rows ? r : p.rows - 1;
  };
  long long f_base = base;  // the step to fetch next: rows at f_base, heads from f_h
  int f_h = 0;
  const T* fx = static_cast<const T*>(p.x) + l.o1;
  const GT* fdy = static_cast<const GT*>(p.dy) + l.o1;
  if (base < p.rows) {
    fx += row_of(base) * p.ldx;
    fdy += row_of(base) * p.lddy;
  }
  auto fetch = [&](uint32_t st) {
    if (f_base < p.rows) {
#pragma unroll
      for (int u = 0; u < HU; ++u)
        if (f_h + u < heads) {
          const uint32_t slot = st + u * (1 + GI) * 16 * kNrBwdThreads;
          nr_fetch<T, V, ADJ>(slot, fx + u * DH, fx + u * DH + gap);
          nr_fetch<GT, V, ADJ>(slot + 16 * kNrBwdThreads, fdy + u * DH, fdy + u * DH + gap);
        }
      f_h += HU;
      fx += HU * DH;
      fdy += HU * DH;
      if (f_h >= heads) {
        f_h = 0;
        f_base += step;
        if (f_base < p.rows) {
          fx = static_cast<const T*>(p.x) + row_of(f_base) * p.ldx + l.o1;
          fdy = static_cast<const GT*>(p.dy) + row_of(f_base) * p.lddy + l.o1;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  constexpr uint32_t STAGE = R::ITEMS * 16 * kNrBwdThreads;
#pragma unroll
  for (int i = 0; i < kNrStages - 1; ++i) fetch(ring + i * STAGE);
  int stage = 0;
  int pos = base < p.rows ? p.pos[row_of(base)] : 0;
  for (; base < p.rows; base += step) {
    const bool live = base + lane / LPH < p.rows;
    GT* dx = static_cast<GT*>(p.y) + row_of(base) * p.ldy + l.o1;
    float c[C], s[C];
    nr_angles<C, sizeof(T) == 2>(turns, a.rot, pos, l.first, c, s);
    pos = base + step < p.rows ? p.pos[row_of(base + step)] : 0;
#pragma unroll 1
    for (int h0 = 0; h0 < heads; h0 += HU) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kNrStages - 2) : "memory");
      const uint32_t st = ring + stage * STAGE;
      fetch(ring + (stage == 0 ? kNrStages - 1 : stage - 1) * STAGE);
      stage = stage == kNrStages - 1 ? 0 : stage + 1;
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        if (h0 + u < heads) {
          const uint32_t slot = st + u * (1 + GI) * 16 * kNrBwdThreads;
          float f[V], d[V], dn[V], e[V];
          nr_unpack<T, V, ADJ>(nr_take<T, V>(slot), f);
          nr_unpack<GT, V, ADJ>(nr_take<GT, V>(slot + 16 * kNrBwdThreads), d);
#pragma unroll
          for (int k = 0; k < C; k += 2) {
            const uint64_t da = f2pack(d[k], d[k + 1]), db = f2pack(d[C + k], d[C + k + 1]);
            const uint64_t cc = f2pack(c[k], c[k + 1]), ss = f2pack(s[k], s[k + 1]), ns = f2pack(-s[k], -s[k + 1]);
            f2unpack(ffma2(da, cc, fmul2(db, ss)), dn[k], dn[k + 1]);
            f2unpack(ffma2(db, cc, fmul2(da, ns)), dn[C + k], dn[C + k + 1]);
          }
#pragma unroll
          for (int k = 0; k < V; k += 2)
            f2unpack(fmul2(f2pack(dn[k], dn[k + 1]), f2pack(g[k], g[k + 1])), e[k], e[k + 1]);
          const float r = rsqrtf(nr_sum<LPH>(nr_dot<V>(f, f)) * (1.0f / DH) + a.eps);
          const float m = nr_sum<LPH>(nr_dot<V>(e, f)) * (1.0f / DH) * r * r * r;
          if (live) {
            const uint64_t rr = f2pack(r, r), nm = f2pack(-m, -m);
#pragma unroll
            for (int k = 0; k < V; k += 2) {
              const uint64_t ff = f2pack(f[k], f[k + 1]);
              f2unpack(ffma2(f2pack(dn[k], dn[k + 1]), fmul2(ff, rr), f2pack(dg[k], dg[k + 1])), dg[k], dg[k + 1]);
              f2unpack(ffma2(f2pack(e[k], e[k + 1]), rr, fmul2(ff, nm)), e[k], e[k + 1]);
            }
            nr_store<GT, V, ADJ>(dx + u * DH, dx + u * DH + gap, e);
          }
        }
      }
      dx += HU * DH;
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) dg[k] += __shfl_xor_sync(0xffffffffu, dg[k], o);
    if (lane < LPH) sums[warp][nr_col<V, ADJ>(l, k)] = dg[k];
  }
  __syncthreads();
  for (int col = threadIdx.x; col < DH; col += kNrBwdThreads) {
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
