// history_cache.cuh — projected K|V rows of growing histories in a paged cache: writing rows (as bf16, or
// quantised to e4m3 with one power-of-two scale per row and head) and reading them back.
//
// Layout. pages [n_pages][planes][kv_heads][page_size][d_head], planes = K, V (K alone with shared K = V);
// scales [n_pages][planes][kv_heads][page_size], one byte e + 127. Head-major inside a page: the rows
// that one head's attention streams are contiguous (page_size * d_head numbers, their scales beside one
// another), so a tile is one copy and an e4m3 row of 32 bytes costs no half-used sectors.
//
// Quantisation of a row x (one head's K or V): e = the least integer with max|x| <= 448 * 2^e, kept in
// [-100, 119] (119: 448 * 2^119 is finite; -100: 2^-109, the least e4m3 number times 2^-100, is a bf16 number),
// 0 for a row of zeros; stored = e4m3(x * 2^-e), round to nearest even. The scaling is exact, so the
// stored number has one rounding, does not depend on how the division is done, and number * 2^e is
// exact in bf16. A NaN stays a NaN (and does not count for e); an infinity becomes +-448 * 2^119.
#pragma once

#include <cuda_fp8.h>

#include "chunk_index.h"
#include "ptx.cuh"

namespace whale {

constexpr unsigned kErrPages = 4u;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 numbers as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

struct RowsArgs {
  ChunkView c;
  const __nv_bfloat16* src;  // append: kv [total, ld]
  __nv_bfloat16* dst;        // read: kv [total, ld]
  long long ld;
  uint8_t* pages;
  uint8_t* scales;
};

constexpr int kRowsThreads = 256;
// Rows of a block: one pass of its threads, 16 bytes of a head each (two passes of the read took 65 us where one takes 61:
// 48 histories, d 256, e4m3).
constexpr int rows_per_block(int dh) { return kRowsThreads / (dh / 8); }
// Heads whose 16 bytes a lane has in flight at once (append: and as many more while it uses those).
constexpr int kAppendHeads = 4, kReadHeads = 8;

// Append: a row's d_head / 8 lanes take its heads one after another, 16 bytes a lane, the first kAppendHeads loaded
// before the row's place in the cache is looked up; the amax of a head is log2(lanes) shuffles. HBM-bound: each
// number is read once and written once. 24 histories (152k rows, d 512) as e4m3: 72 us, 6.2 TB/s; with 8 heads in flight
// and 3 blocks an SM, 75 us.
template <int DH, bool FP8>
__global__ void __launch_bounds__(kRowsThreads, 5) cache_append_kernel(const RowsArgs a) {
  constexpr int LPH = DH / 8, RPW = 32 / LPH, HU = kAppendHeads;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, li = lane % LPH;
  const long long row = ((long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5)) * RPW + lane / LPH;
  const int heads = a.c.planes * a.c.kv_heads;
  const bool mine = row < a.c.total && row < a.c.offsets[a.c.B];
  const uint4* src = reinterpret_cast<const uint4*>(a.src + (mine ? row : 0) * a.ld) + li;
  uint4 w[HU];
#pragma unroll
  for (int u = 0; u < HU; ++u) w[u] = mine && u < heads ? src[u * LPH] : make_uint4(0u, 0u, 0u, 0u);
  long long at = -1;
  if (mine) {
    const int b = chunk_seq(a.c, row);
    at = cache_row(a.c, b, (long long)a.c.lengths[b] - (a.c.offsets[b + 1] - row));
    if (at < 0) atomicOr(&g_device_error, kErrPages);
  }
  const bool live = at >= 0;
  if (!__any_sync(0xffffffffu, live)) return;
  for (int h0 = 0; h0 < heads; h0 += HU) {
    uint4 nx[HU];
#pragma unroll
    for (int u = 0; u < HU; ++u)
      nx[u] = live && h0 + HU + u < heads ? src[(h0 + HU + u) * LPH] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < HU; ++k) {
      if (h0 + k >= heads) break;
      const long long out = at + ((long long)(h0 + k) << a.c.page_shift);
      if constexpr (!FP8) {
        if (live) *reinterpret_cast<uint4*>(a.pages + (out * DH + li * 8) * 2) = w[k];
      } else {
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
        float f[8], m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(u[i] << 16);
          f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
          m = fmaxf(m, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
        }
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = scale_exponent(m);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          q[i] = (uint32_t)e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
                 ((uint32_t)e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16);
        if (live) {
          *reinterpret_cast<uint2*>(a.pages + out * DH + li * 8) = make_uint2(q[0], q[1]);
          if (li == 0) a.scales[out] = (uint8_t)(e + 127);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < HU; ++u) w[u] = nx[u];
  }
}

// Read: the same lanes the other way; rows in no page come back as zeros. Each row's place is looked up by one
// thread of the block (every load waits for it: 60 us where every lane looking up its own row took 69 us, 48
// histories of 3000 to 6000 rows, d 256, e4m3). bf16 rows take 101.2 us with registers
// for 4 blocks an SM, 102.3 for 5 (24 histories, d 512); e4m3 rows need fewer and have 5.
template <int DH, bool FP8>
__global__ void __launch_bounds__(kRowsThreads, FP8 ? 5 : 4) cache_read_kernel(const RowsArgs a) {
  constexpr int LPH = DH / 8, HU = kReadHeads, ROWS = rows_per_block(DH);
  __shared__ long long places[ROWS];
  pdl_wait();
  pdl_trigger();
  const int li = threadIdx.x % LPH;
  const long long first = (long long)blockIdx.x * ROWS;
  const int heads = a.c.planes * a.c.kv_heads;
  if (threadIdx.x < ROWS) {
    const long long row = first + threadIdx.x;
    long long at = -2;  // behind the last sequence; -1: in no page
    if (row < a.c.total && row < a.c.offsets[a.c.B]) {
      const int b = chunk_seq(a.c, row);
      at = cache_row(a.c, b, (long long)a.c.lengths[b] - (a.c.offsets[b + 1] - row));
      if (at < 0) atomicOr(&g_device_error, kErrPages);
    }
    places[threadIdx.x] = at;
  }
  __syncthreads();
  const int r = threadIdx.x / LPH;
  const long long at = places[r];
  if (at == -2) return;
  uint4* dst = reinterpret_cast<uint4*>(a.dst + (first + r) * a.ld) + li;
  for (int h0 = 0; h0 < heads; h0 += HU) {
    uint4 w[HU];
    uint32_t sc[HU];
#pragma unroll
    for (int k = 0; k < HU; ++k) {
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      sc[k] = 0u;
      if (at >= 0 && h0 + k < heads) {
        const long long in = at + ((long long)(h0 + k) << a.c.page_shift);
        if constexpr (!FP8) {
          w[k] = *reinterpret_cast<const uint4*>(a.pages + (in * DH + li * 8) * 2);
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(a.pages + in * DH + li * 8);
          w[k].x = q.x;
          w[k].y = q.y;
        }
      }
    }
    if constexpr (FP8) {  // behind all numbers: 61 us; each scale beside its head's numbers 69 us (the same histories)
#pragma unroll
      for (int k = 0; k < HU; ++k)
        if (at >= 0 && h0 + k < heads) sc[k] = a.scales[at + ((long long)(h0 + k) << a.c.page_shift)];
    }
#pragma unroll
    for (int k = 0; k < HU; ++k) {
      if (h0 + k >= heads) break;
      if constexpr (FP8) {
        const float f = __uint_as_float(sc[k] << 23);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = e4m3x2_f16x2((uint16_t)((i < 2 ? w[k].x : w[k].y) >> (16 * (i & 1))));
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v));
          o[i] = pack_bf16x2(x.x * f, x.y * f);
        }
        w[k] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      dst[(h0 + k) * LPH] = w[k];
    }
  }
}

}  // namespace whale
