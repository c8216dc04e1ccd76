// cache_attention.cuh — attention of a chunk of rows over the paged cache, few rows per sequence (a new event,
// a request's tokens):
//   a_i = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j / sqrt(d_head)) over the sequence's cached positions j
//   (causal: j <= position of row i; a row that sees nothing gives 0).
// Query head h reads K|V head h * kv_heads / n_heads, so the n_b * group rows (token, head of the group) of one
// sequence and K|V head share every cached row: row r is token r / group, head kvh * group + r % group.
//
// Bound: HBM (each cached row is read once; 2 * n_b * group operations per byte of bf16).
// 64 users, d 512, histories of up to 15000 rows: one row 138 to 144 us (bf16, 6.0 to 6.2 TB/s) and 100 us (e4m3), 32 rows 159 and 171 us.
//
// Split. Units of kCaTile positions of one (sequence, K|V head, block of BM rows) are laid end to end, and warp w of
// W takes the contiguous slice [w T / W, (w + 1) T / W): every warp streams the same number of bytes whatever the
// lengths. A warp works alone (its own ring of shared memory, no block barrier after the prologue), keeps (m, l, o)
// of its BM rows in registers, and leaves a partial in the workspace where its slice cuts an item: at most two a
// warp. cache_attend_merge_kernel joins them in the order of the warps, so results do not depend on timing.
//
// The stream: cp.async, STAGES - 1 tiles ahead; the lanes look up the page of one position each, a tile earlier still.
// Rows past the end and rows in no page are zero-filled, so what unwritten rows hold is never used.
//
// Products: warp-level m16n8k16 with fp32 sums. bf16 cache: K and V by ldmatrix; weights are rounded to bf16, V's
// type, which both operands of a product have (one event's relative error is then 0.0023 where the rounding of the result
// alone leaves 0.0016; the packed path rounds its weights the same way). e4m3 cache: the fragments are converted from the
// bytes in registers, to f16 (every e4m3 number is an f16 number); a lane's bytes of a K row are contiguous (the order of
// d_head inside a product is free as long as q has the same), and the positions of a tile are numbered so that a lane's
// scores are 8 neighbouring ones, whose scales it reads as one word. K's scale multiplies the score, V's the weight.
// Queries are brought into f16's range by a power of two of each row (all bits down to 2^-28 of the row's largest, to
// 2^-39 of it below).
// f16 weights have 11 significant bits, where bf16 ones have 8, but 2^-24 is their least step, so V's scales must not
// push them there: a unit's positions are taken in passes, each with those whose scale is within 2^kCaWindow of the
// largest one left, E (one pass where the scales are alike, as a history's are; each further one costs as much again). A
// weight is 2^(s - m - 8 + 15 + e - E), off by at most 2^-24 of the largest weight where it is less than 2^-13 of it. A
// pass's sums are fp32 of their own, times 2^(E - 15) added to the row's: what a row does not see, and rows of zeros
// (whose e is 0), can shift nothing out of it. Sums of a unit's own cost 3 % at 32 rows (171 us where one running E
// took 167) and 1 % at one.
#pragma once

#include <cuda_fp16.h>

#include "attention_bwd.cuh"
#include "history_cache.cuh"

namespace whale {

struct CacheAttnArgs {
  ChunkView c;
  const __nv_bfloat16* q;  // [total, ldq]
  __nv_bfloat16* a;        // [total, lda]
  long long ldq, lda;
  const uint8_t* pages;
  const uint8_t* scales;
  int group, causal;       // query heads of a K|V head
  int max_new;             // rows of a sequence, at most
  int rows_lo, rows_hi;    // this kernel's sequences: more than rows_lo rows x group, at most rows_hi
  float scale_log2;        // log2(e) / sqrt(d_head)
  float* part_o;           // [2 W, BM, DH]
  float* part_ml;          // [2 W, BM, 2]
  struct CaCut* cuts;      // [W] the item that each slice leaves to the next ones
};

// An item that begins in a slice and does not end there: its rows, and the partials that make it up.
struct CaCut {
  int first_row, row0, n_rows, head0;  // packed row of the sequence, first row of the block, rows, first query head
  int parts, slot;                     // slices (0: nothing to join), the first one's slot; the next ones' are 2 w
  int pad[2];
};
__device__ __forceinline__ void ca_write_cut(CaCut* c, int first_row, int row0, int n_rows, int head0, int parts, int slot) {
  reinterpret_cast<int4*>(c)[0] = make_int4(first_row, row0, n_rows, head0);
  reinterpret_cast<int4*>(c)[1] = make_int4(parts, slot, 0, 0);
}
// Slice of W that holds unit u of T.
__device__ __forceinline__ long long ca_slice_of(long long u, long long W, long long T) { return ((u + 1) * W - 1) / T; }

constexpr int kCaTile = 32;     // positions of a unit
// Warps of a CTA (one CTA per SM) for blocks of 16 mt rows. What is in flight is the same; the conversions of e4m3 fragments
// leave gaps that more warps fill: 64 users, one row, d 512, histories of up to 15000 rows 121 us with 8 warps, 103 with
// 12, 102 with 16. With 32 rows 12 warps have too few registers, and pairs of warps that share the tiles and
// convert them twice take 178 us with 16 warps where 8 warps of 32 rows took 165 (both before the passes by scale).
constexpr int ca_warps(bool fp8, int mt) { return fp8 && mt == 1 ? 12 : 8; }
constexpr int kCaMinUnits = 2;  // a warp's least share where there is little work: 12.1 us for one row of 8 heads over
                                // 5000 positions; with 4 the units take longer, with 1 the join does (12.9, 13.3 us)
constexpr float kCaLazy = 8.0f; // log2 headroom before the reference is raised; weights are 2^(s - reference - 8), at most
                                // 1, so that one times the largest V is finite
constexpr int kCaWindow = 8;    // log2 of the range of V's scales that one pass takes (e4m3)

template <int DH, bool FP8, int MT>
struct CaTile {
  static constexpr int ROW = FP8 ? DH : 2 * DH;           // bytes of a row
  static constexpr int PLANE = kCaTile * ROW;
  static constexpr int SCALES = FP8 ? 2 * kCaTile : 0;    // K's, V's
  static constexpr int BYTES = 2 * PLANE + SCALES;
  static constexpr int SHARE = 196608 / ca_warps(FP8, MT);
  static constexpr int STAGES = SHARE / BYTES < 8 ? SHARE / BYTES : 8;
  static constexpr int SMEM = ca_warps(FP8, MT) * STAGES * BYTES;
  static_assert(STAGES >= 3 && BYTES % 16 == 0 && SMEM <= 220 * 1024, "ring");
  // byte offset of 16-byte chunk `ch` of row r: conflict-free for the fragment reads below
  static __device__ __forceinline__ int at(int r, int ch) {
    if constexpr (!FP8) return r * ROW + ((ch ^ (DH == 64 ? r & 7 : (r >> 1) & 3)) << 4);
    // one line of 128 bytes holds the rows that lanes t = 0..3 read together (8 positions apart): give each its quarter
    else if constexpr (DH == 64) return (r ^ ((r >> 4) & 1)) * ROW + ((ch ^ ((r >> 2) & 2)) << 4);
    else return (r ^ (((r >> 2) & 2) | ((r >> 4) & 1))) * ROW + (ch << 4);
  }
};

// Units of sequence b per (K|V head, row block), its rows and positions.
struct CaSeq {
  int first_row, rows, take; // rows of the packed tensor; of them within max_new
  int len;                  // positions, within the cache's bounds
  int units, blocks;        // tiles (1 for an empty history: its rows are written as zeros), row blocks
};
__device__ __forceinline__ CaSeq ca_seq(const CacheAttnArgs& p, int b, int bm) {
  CaSeq s;
  s.first_row = chunk_off(p.c, b);
  s.rows = chunk_off(p.c, b + 1) - s.first_row;
  s.take = min(s.rows, p.max_new);
  const long long n = p.c.lengths[b];
  s.len = (int)(n < 0 ? 0 : (n > p.c.capacity ? p.c.capacity : n));
  s.units = s.len <= kCaTile ? 1 : (s.len + kCaTile - 1) / kCaTile;
  const int rows = max(s.take, 0) * p.group;
  s.blocks = rows > p.rows_lo && rows <= p.rows_hi ? (rows + bm - 1) / bm : 0;
  return s;
}
// Rows beyond the host's bound of them, and positions beyond the cache's: by one block, whether or not the sequence has work.
__device__ __forceinline__ void ca_report(const CacheAttnArgs& p, int b, const CaSeq& s) {
  if (s.rows > s.take) atomicOr(&g_device_error, kErrOffsets);
  if (s.rows > 0 && p.c.lengths[b] > s.len) atomicOr(&g_device_error, kErrPages);
}
__device__ __forceinline__ long long ca_units(const CacheAttnArgs& p, int b, int bm) {
  const CaSeq s = ca_seq(p, b, bm);
  return (long long)s.units * s.blocks * p.c.kv_heads;
}
__device__ __forceinline__ long long ca_workers(long long T, long long W) {
  const long long w = (T + kCaMinUnits - 1) / kCaMinUnits;
  return w < W ? w : W;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with zeros for the sums so far.
__device__ __forceinline__ void mma_f16_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

template <int DH, bool FP8, int MT>
__global__ void __launch_bounds__(32 * ca_warps(FP8, MT), 1) cache_attend_kernel(const CacheAttnArgs p) {
  using L = CaTile<DH, FP8, MT>;
  constexpr int kCaWarps = ca_warps(FP8, MT), kCaThreads = 32 * kCaWarps;
  constexpr int BM = 16 * MT, NT = kCaTile / 8, KS = DH / 16, ND = DH / 8, STAGES = L::STAGES;
  extern __shared__ __align__(128) uint8_t ring_all[];
  __shared__ long long sums[kCaThreads + 1];
  __shared__ __align__(16) float factors[kCaWarps][2 * kCaTile];  // e4m3: K's and V's factor of each position of a unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();

  // units before each thread's run of sequences
  const int run = (p.c.B + kCaThreads - 1) / kCaThreads;
  const int b_lo = min(p.c.B, tid * run), b_hi = min(p.c.B, b_lo + run);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const CaSeq s = ca_seq(p, b, BM);
    mine += (long long)s.units * s.blocks * p.c.kv_heads;
    if (blockIdx.x == 0) ca_report(p, b, s);
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  long long base = 0;
  for (int w = 0; w < warp; ++w) base += sums[w];
  __syncthreads();
  sums[tid + 1] = base + scan;
  if (tid == 0) sums[0] = 0;
  __syncthreads();
  const long long T = sums[kCaThreads];
  const long long W = ca_workers(T, (long long)gridDim.x * kCaWarps);
  const long long gw = (long long)warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
  const long long u_lo = gw < W ? gw * T / W : T, u_hi = gw < W ? (gw + 1) * T / W : T;
  if (u_lo >= u_hi) {
    if (lane == 0) ca_write_cut(p.cuts + gw, 0, 0, 0, 0, 0, 0);
    return;
  }

  // the sequence of the first unit
  int b, lo = 0, hi = kCaThreads - 1;
  while (lo < hi) {  // largest run that starts at or before u_lo and is not empty behind it
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= u_lo) lo = mid;
    else hi = mid - 1;
  }
  b = min(p.c.B, lo * run);
  long long at = sums[lo];
  for (;;) {
    const long long n = ca_units(p, b, BM);
    if (at + n > u_lo || b + 1 >= p.c.B) break;
    at += n;
    ++b;
  }

  const uint32_t ring = smem_u32(ring_all) + warp * (STAGES * L::BYTES);
  const uint8_t* const pages = p.pages;
  long long u = u_lo;
  while (u < u_hi) {
    const CaSeq s = ca_seq(p, b, BM);
    const long long n_b = (long long)s.units * s.blocks * p.c.kv_heads;
    if (u >= at + n_b) {
      if (b + 1 >= p.c.B) {  // cannot be: the units are the sequences'
        if (lane == 0) ca_write_cut(p.cuts + gw, 0, 0, 0, 0, 0, 0);
        return;
      }
      at += n_b;
      ++b;
      continue;
    }
    const int item = (int)((u - at) / s.units), t_lo = (int)((u - at) - (long long)item * s.units);
    const int t_hi = (int)min((long long)s.units, t_lo + (u_hi - u));
    const int kvh = item / s.blocks, r0 = (item - kvh * s.blocks) * BM;
    const int n_rows = min(BM, s.take * p.group - r0);
    const long long pos0 = (long long)p.c.lengths[b] - s.rows;  // position of the sequence's first row

    // queries as A fragments, ends of the rows
    uint32_t qf[MT][KS][4];
    int end[MT][2];
    float fac[MT][2];  // log2(e) / sqrt(d_head), and for e4m3 the power of two taken out of the row
    int end_min = s.len;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = 16 * m + 8 * hh + g;
        const bool live = r < n_rows;
        const int tok = live ? (r0 + r) / p.group : 0;
        const int head = kvh * p.group + (live ? (r0 + r) % p.group : 0);
        const __nv_bfloat16* src = p.q + (long long)(s.first_row + tok) * p.ldq + head * DH;
        fac[m][hh] = p.scale_log2;
        const long long e = p.causal ? min((long long)s.len, pos0 + tok + 1) : (long long)s.len;
        end[m][hh] = live ? (int)max(e, 0ll) : 0;
        if (live) end_min = min(end_min, end[m][hh]);
        if constexpr (!FP8) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[m][k][hh] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t) : 0u;
            qf[m][k][2 + hh] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t + 8) : 0u;
          }
        } else {
          uint32_t w[2 * KS];
          float f[4 * KS], mx = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint2 v = live ? *reinterpret_cast<const uint2*>(src + t * (DH / 4) + 4 * k) : make_uint2(0u, 0u);
            w[2 * k] = v.x;
            w[2 * k + 1] = v.y;
          }
#pragma unroll
          for (int k = 0; k < 2 * KS; ++k) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            mx = fmaxf(mx, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int ex = (int)(__float_as_uint(mx) >> 23) - 127;  // mx in [2^ex, 2^(ex+1))
          ex = mx == 0.f ? 14 : max(-100, min(ex, 127));
          const float down = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
          fac[m][hh] = p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[m][k][hh] = pack_f16x2(f[4 * k] * down, f[4 * k + 1] * down);
            qf[m][k][2 + hh] = pack_f16x2(f[4 * k + 2] * down, f[4 * k + 3] * down);
          }
        }
      }
    end_min = __reduce_min_sync(0xffffffffu, end_min);

    float o[MT][ND][4], mr[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[m][d][k] = 0.f;
      mr[m][0] = mr[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }

    const long long kv_off = (long long)kvh << p.c.page_shift;
    const uint32_t vpl = p.c.planes == 2 ? L::PLANE : 0;  // V's plane of a stage (K's with shared K = V)
    const long long v_off = p.c.planes == 2 ? (long long)p.c.kv_heads << p.c.page_shift : 0;
    const long long v_bytes = v_off * L::ROW;
    // the page of this lane's position of tile i: only loaded here, and looked at a tile later
    const int* const table = p.c.table + (long long)b * p.c.table_stride;
    auto look = [&](int i) -> int {
      const int pos = i * kCaTile + lane;
      return i < t_hi && pos < s.len ? table[pos >> p.c.page_shift] : 0;
    };
    auto fetch = [&](int i, int page) {
      if (i >= t_hi) return;
      int row = -1;  // in the pool (this head's K plane), whose rows are numbered in 31 bits; -1: none
      if (i * kCaTile + lane < s.len) {
        row = (int)page_row(p.c, page, i * kCaTile + lane);
        if (row < 0) atomicOr(&g_device_error, kErrPages);
        else row += (int)kv_off;
      }
      const uint32_t st = ring + (uint32_t)((i - t_lo) % STAGES) * L::BYTES;
      constexpr int CH = L::ROW / 16, RPI = 32 / CH;  // 16-byte chunks of a row, rows of one instruction
#pragma unroll
      for (int k = 0; k < kCaTile / RPI; ++k) {
        const int r = k * RPI + lane / CH, ch = lane % CH;
        const int src = __shfl_sync(0xffffffffu, row, r);
        const uint32_t n = src < 0 ? 0u : 16u;
        const uint8_t* a = pages + (long long)max(src, 0) * L::ROW + ch * 16;
        cp_async16(st + L::at(r, ch), a, n);
        if (vpl) cp_async16(st + L::PLANE + L::at(r, ch), src < 0 ? a : a + v_bytes, n);
      }
      if constexpr (FP8) {
        const int src = __shfl_sync(0xffffffffu, row, 4 * (lane & 7));
        if (lane < 16 && src < 0)  // rows in no page are zeros: any scale will do, but not a stale one
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + 2 * L::PLANE + (lane >> 3) * kCaTile + 4 * (lane & 7)), "r"(0u)
                       : "memory");
        else if (lane < 16)
          cp_async4(st + 2 * L::PLANE + (lane >> 3) * kCaTile + 4 * (lane & 7), p.scales + src + (lane >> 3) * v_off);
      }
    };

    __syncwarp();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      fetch(t_lo + i, look(t_lo + i));
      cp_async_commit();
    }
    int ahead = look(t_lo + STAGES - 1);

    bool more = false;  // e4m3: the unit has positions for another pass, those with V's code
    int below = 256;    // below this
    for (int i = t_lo; i < t_hi; i += !more) {
      if (!more) {
        cp_async_wait<STAGES - 2>();
        __syncwarp();
        fetch(i + STAGES - 1, ahead);
        cp_async_commit();
        ahead = look(i + STAGES);
        below = 256;
      }
      const bool first = !more;
      const uint32_t st = ring + (uint32_t)((i - t_lo) % STAGES) * L::BYTES;
      const int pos = i * kCaTile;

      // scores
      float sc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[m][j][k] = 0.f;
      if constexpr (!FP8) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t b0, b1, b2, b3;  // positions 8 j .., d_head 16 k .. 16 k + 31
            ldsm_x4(st + L::at(8 * j + (lane & 7), 2 * k + (lane >> 3)), b0, b1, b2, b3);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_bf16_16816(sc[m][j], qf[m][k][0], qf[m][k][1], qf[m][k][2], qf[m][k][3], b0, b1);
              mma_bf16_16816(sc[m][j], qf[m][k + 1][0], qf[m][k + 1][1], qf[m][k + 1][2], qf[m][k + 1][3], b2, b3);
            }
          }
      } else {
        // column c of n-tile j is position 8 (c / 2) + 2 j + c % 2
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = 8 * (g >> 1) + 2 * j + (g & 1);
          uint32_t w[KS];
          if constexpr (DH == 64) {
            const uint4 v = lds128(st + L::at(r, t));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else {
            const uint2 v = lds64(st + L::at(r, t >> 1) + 8 * (t & 1));
            w[0] = v.x, w[1] = v.y;
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t b0 = e4m3x2_f16x2((uint16_t)w[k]), b1 = e4m3x2_f16x2((uint16_t)(w[k] >> 16));
#pragma unroll
            for (int m = 0; m < MT; ++m)
              mma_f16_16816(sc[m][j], qf[m][k][0], qf[m][k][1], qf[m][k][2], qf[m][k][3], b0, b1);
          }
        }
      }

      // scales: K's into the scores, V's as factors of the weights (8 neighbouring positions a lane)
      uint64_t vf[NT];  // pairs
      float o_unit = 0.f;  // e4m3: what 1 in the pass's sums is in o
      if constexpr (FP8) {
        const bool ok = pos + lane < s.len;  // rows past the end hold any code
        uint32_t ck, cv;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(ck) : "r"(st + 2 * L::PLANE + lane));
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(cv) : "r"(st + 2 * L::PLANE + kCaTile + lane));
        cv = ok && (int)cv < below ? cv : 0u;
        const int e_max = (int)__reduce_max_sync(0xffffffffu, cv);  // E + 127
        const bool in = (int)cv + kCaWindow >= e_max;
        more = __any_sync(0xffffffffu, cv != 0u && !in);
        below = e_max - kCaWindow;
        o_unit = __uint_as_float((uint32_t)max(e_max - 15, 0) << 23);
        // each lane makes its position's two factors, 2^e and 2^(e - E + 15); then a lane takes those of its 8 positions
        const uint32_t fs = smem_u32(factors[warp]);
        __syncwarp();
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(fs + 4 * lane), "r"(ck << 23) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(fs + 128 + 4 * lane), "r"(in ? (cv - e_max + 142) << 23 : 0u)
                     : "memory");
        __syncwarp();
        uint64_t kf[NT];
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          const uint4 a = lds128(fs + 32 * t + 8 * j), b = lds128(fs + 128 + 32 * t + 8 * j);
          kf[j] = f2pack(__uint_as_float(a.x), __uint_as_float(a.y));
          kf[j + 1] = f2pack(__uint_as_float(a.z), __uint_as_float(a.w));
          vf[j] = f2pack(__uint_as_float(b.x), __uint_as_float(b.y));
          vf[j + 1] = f2pack(__uint_as_float(b.z), __uint_as_float(b.w));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              f2unpack(fmul2(f2pack(sc[m][j][2 * hh], sc[m][j][2 * hh + 1]), fmul2(kf[j], f2pack(fac[m][hh], fac[m][hh]))),
                       sc[m][j][2 * hh], sc[m][j][2 * hh + 1]);
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[m][j][k] *= p.scale_log2;
      }
      if (pos + kCaTile > end_min) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int x = pos + (FP8 ? 8 * t + 2 * j + (k & 1) : 8 * j + 2 * t + (k & 1));
              if (x >= end[m][k >> 1]) sc[m][j][k] = -INFINITY;
            }
      }

      // running maximum, raised when the tile's exceeds it by kCaLazy; weights as A fragments
      uint32_t pf[MT][NT][2];
      bool raise = false;
      float mn[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x = fmaxf(sc[m][0][2 * hh], sc[m][0][2 * hh + 1]);
#pragma unroll
          for (int j = 1; j < NT; ++j) x = fmax3(x, sc[m][j][2 * hh], sc[m][j][2 * hh + 1]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const bool up = x > mr[m][hh] + kCaLazy;
          mn[m][hh] = up ? x : mr[m][hh];
          raise |= up;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float f = mn[m][hh] == mr[m][hh] ? 1.f : fast_exp2(mr[m][hh] - mn[m][hh]);
            mr[m][hh] = mn[m][hh];
            l[m][hh] *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              o[m][d][2 * hh] *= f;
              o[m][d][2 * hh + 1] *= f;
            }
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float ref = (mr[m][hh] == -INFINITY ? 0.f : mr[m][hh]) + kCaLazy;
          const uint64_t nr = f2pack(-ref, -ref);
          uint64_t sum2 = f2pack(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float w0, w1;
            f2unpack(fadd2(f2pack(sc[m][j][2 * hh], sc[m][j][2 * hh + 1]), nr), w0, w1);
            w0 = fast_exp2(w0);
            w1 = fast_exp2(w1);
            const uint64_t w = f2pack(w0, w1);
            sum2 = fadd2(sum2, w);
            if constexpr (FP8) {
              f2unpack(fmul2(w, vf[j]), w0, w1);
              pf[m][j][hh] = pack_f16x2(w0, w1);
            } else {
              pf[m][j][hh] = pack_bf16x2(w0, w1);
            }
          }
          float sum, sum1;
          f2unpack(sum2, sum, sum1);
          sum += sum1;
          l[m][hh] += first ? sum : 0.f;
        }

      // o += weights x V
      if constexpr (!FP8) {
#pragma unroll
        for (int k = 0; k < NT / 2; ++k)  // 16 positions a step: n-tiles 2 k and 2 k + 1 of the scores
#pragma unroll
          for (int d = 0; d < ND; d += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(st + vpl + L::at(16 * k + (lane & 15), d + (lane >> 4)), b0, b1, b2, b3);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_bf16_16816(o[m][d], pf[m][2 * k][0], pf[m][2 * k][1], pf[m][2 * k + 1][0], pf[m][2 * k + 1][1], b0, b1);
              mma_bf16_16816(o[m][d + 1], pf[m][2 * k][0], pf[m][2 * k][1], pf[m][2 * k + 1][0], pf[m][2 * k + 1][1], b2, b3);
            }
          }
      } else {
        // column n of n-tile d is column n * ND + d of V: a lane's bytes are contiguous
        uint32_t v[NT / 2][4][ND / 4];
#pragma unroll
        for (int k = 0; k < NT / 2; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = 8 * t + 4 * k + x;
            if constexpr (DH == 64) {
              const uint2 w = lds64(st + vpl + L::at(r, g >> 1) + 8 * (g & 1));
              v[k][x][0] = w.x;
              v[k][x][1] = w.y;
            } else {
              v[k][x][0] = lds32(st + vpl + L::at(r, g >> 2) + 4 * (g & 3));
            }
          }
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
          float c[MT][2][4];
#pragma unroll
          for (int k = 0; k < NT / 2; ++k) {
            const uint32_t sel = (d & 2) ? 0x7362u : 0x5140u;  // bytes d, d + 1 of the two rows, interleaved
            const uint32_t lo2 = __byte_perm(v[k][0][d / 4], v[k][1][d / 4], sel);
            const uint32_t hi2 = __byte_perm(v[k][2][d / 4], v[k][3][d / 4], sel);
            const uint32_t b0 = e4m3x2_f16x2((uint16_t)lo2), b1 = e4m3x2_f16x2((uint16_t)hi2);
            const uint32_t b2 = e4m3x2_f16x2((uint16_t)(lo2 >> 16)), b3 = e4m3x2_f16x2((uint16_t)(hi2 >> 16));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t a0 = pf[m][2 * k][0], a1 = pf[m][2 * k][1], a2 = pf[m][2 * k + 1][0], a3 = pf[m][2 * k + 1][1];
              if (k == 0) {
                mma_f16_16816_first(c[m][0], a0, a1, a2, a3, b0, b1);
                mma_f16_16816_first(c[m][1], a0, a1, a2, a3, b2, b3);
              } else {
                mma_f16_16816(c[m][0], a0, a1, a2, a3, b0, b1);
                mma_f16_16816(c[m][1], a0, a1, a2, a3, b2, b3);
              }
            }
          }
          const uint64_t unit = f2pack(o_unit, o_unit);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 4; k += 2)
                f2unpack(ffma2(f2pack(c[m][e][k], c[m][e][k + 1]), unit, f2pack(o[m][d + e][k], o[m][d + e][k + 1])),
                         o[m][d + e][k], o[m][d + e][k + 1]);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // the item's output where the slice holds all of it, else a partial
    const bool whole = t_lo == 0 && t_hi == s.units;
    const long long slot = 2 * gw + (u != u_lo);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float sum = l[m][hh];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = 16 * m + 8 * hh + g;
        if (r >= n_rows) continue;
        const float f = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        float* po = p.part_o + (slot * BM + r) * DH;
        const int tok = (r0 + r) / p.group, head = kvh * p.group + (r0 + r) % p.group;
        __nv_bfloat16* dst = p.a + (long long)(s.first_row + tok) * p.lda + head * DH;
        // this lane's columns: 8 d + 2 t, + 1 (bf16), or 2 ND t + d, 2 ND t + ND + d (e4m3)
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const float x0 = o[m][d][2 * hh] * f, x1 = o[m][d][2 * hh + 1] * f;
          if constexpr (!FP8) {
            if (whole) *reinterpret_cast<uint32_t*>(dst + 8 * d + 2 * t) = pack_bf16x2(x0, x1);
            else *reinterpret_cast<float2*>(po + 8 * d + 2 * t) = make_float2(x0, x1);
          } else {
            o[m][d][2 * hh] = x0;
            o[m][d][2 * hh + 1] = x1;
          }
        }
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 0; d < ND; d += 4) {
              const int col = (2 * t + e) * ND + d;
              const float x[4] = {o[m][d][2 * hh + e], o[m][d + 1][2 * hh + e], o[m][d + 2][2 * hh + e], o[m][d + 3][2 * hh + e]};
              if (whole) *reinterpret_cast<uint2*>(dst + col) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
              else *reinterpret_cast<float4*>(po + col) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        if (!whole && t == 0)
          *reinterpret_cast<float2*>(p.part_ml + (slot * BM + r) * 2) = make_float2(mr[m][hh], sum);
      }
    u += t_hi - t_lo;
    if (u >= u_hi && lane == 0) {
      const bool starts = !whole && t_lo == 0;
      ca_write_cut(p.cuts + gw, s.first_row, r0, n_rows, kvh * p.group,
                   starts ? (int)(ca_slice_of(u - t_hi + s.units - 1, W, T) - gw) + 1 : 0, (int)slot);
    }
  }
}

}  // namespace whale
