// cache_attention_e4m3.cuh — attention of up to 32 rows (tokens x heads of a group) per sequence and K|V head over
// the e4m3 cache, with positions where the other kernels have rows: S^T = K Q^T (128 positions x 32 rows) and
// O^T += V^T P^T on tcgen05. The formula, the row order and the masks are those of cache_attention.cuh.
//
// Why transposed: 32 rows would leave three quarters of a 128-row tile empty, its softmax warps with it; 128 positions
// fill it. A softmax thread then has one position, whose scales are one factor each: K's of its 32 scores, V's of its 32
// weights. And every byte of the cache is converted once, by the producers, to f16 (exact), where warp-level
// products convert in each warp's registers: 83 us where that kernel takes 166 (64 users, 32 tokens, 8 heads, d 512,
// histories of up to 15000 rows).
//
// Bound: HBM, then the conversions (16 numbers: one shared load, 8 converts, 2 shared stores).
//
// Two CTAs per SM, each with a slice of the units as in cache_attention_tc.cuh:
//   warps 0-1  raw bytes by cp.async two units ahead; converted to f16 tiles, K's once S^T has read the last one,
//              V's (two buffers) once O^T has; the queries, brought into f16's range by a power of two per row
//   warp 2     the products. V^T's rows are repeated to make 128 (the shapes with 64 take as long)
//   warps 4-7  one position per thread. The row's maximum lies across threads, so the reference is one that some earlier
//              unit needed: a thread that finds a weight above 2^8 of it, or a scale above the largest so far, calls for a
//              new one, all warps agree on that by a barrier's vote, and O^T, in tensor memory, and the sums follow.
//              Weights go to shared memory as f16, 2^(s - m + 7 + e - E): see cache_attention.cuh.
#pragma once

#include "cache_attention_tc.cuh"

namespace whale {

constexpr int kCeRows = 32;      // rows of an item
constexpr int kCeThreads = 256;
constexpr int kCeBlocksPerSM = 2;

template <int DH>
struct CeSmem {
  static constexpr int ROW = 2 * DH;                       // bytes of a converted row
  static constexpr uint32_t TILE = kCpUnit * ROW;
  static constexpr uint32_t RAW = kCpUnit * DH;            // raw bytes of a plane
  static constexpr uint32_t RAW_STAGE = 2 * RAW + 2 * kCpUnit;  // K, V, K's scales, V's
  static constexpr int RST = 3;
  // from the start of the block's shared memory
  static constexpr int OFF_RAW = 0;
  static constexpr int OFF_CODE = OFF_RAW + RST * (int)RAW_STAGE;  // [2] units: K's and V's scales
  static constexpr int OFF_FAC = OFF_CODE + 2 * 2 * kCpUnit;       // [2] segments: factor of each row
  static constexpr int OFF_REF = OFF_FAC + 2 * kCeRows * 4;        // reference and last position + 1 of each row; sums
  static constexpr int OFF_BAR = OFF_REF + (2 + 5 + 4) * kCeRows * 4;
  static constexpr int LOW = OFF_BAR + 6 * 8 + 16;
  // from the next 1024-byte boundary
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + (int)TILE;          // [2]
  static constexpr int OFF_P = OFF_V + 2 * (int)TILE;      // 128 positions x 32 rows, 64 bytes each
  static constexpr int OFF_Q = OFF_P + kCpUnit * 64;       // 32 rows
  static constexpr size_t BYTES = LOW + 1024 + OFF_Q + kCeRows * ROW;
  static_assert(2 * (BYTES + 1024 + 1024) <= 233472, "two CTAs on an SM, with their walks and what the system takes");
  static __device__ __forceinline__ uint32_t at(int r, int ch) { return CpSmem<DH>::at(r, ch); }
  static __device__ __forceinline__ uint64_t desc(uint32_t a) { return CpSmem<DH>::desc(a); }
  // V as the transposed A operand: every group of 64 (32) columns of M is the tile itself
  static __device__ __forceinline__ uint64_t desc_vt(uint32_t a) { return CpSmem<DH>::desc(a) & ~((uint64_t)0x3FFFu << 16); }
  // P: rows of 64 bytes, the 64-byte swizzle
  static __device__ __forceinline__ uint64_t desc_p(uint32_t a) { return CpSmem<32>::desc(a); }
};

constexpr uint32_t ce_idesc(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// OR of a predicate over the 128 softmax threads (a barrier).
__device__ __forceinline__ bool ce_vote(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// v[q] summed (or its maximum taken) over the warp's lanes, for lane q: 31 exchanges for 32 values.
template <bool MAX>
__device__ __forceinline__ float ce_across(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 16; n > 0; n >>= 1)
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const bool up = lane & n;
      const float mine = up ? v[j + n] : v[j], other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + n], n);
      v[j] = MAX ? fmaxf(mine, other) : mine + other;
    }
  return v[0];
}

template <int DH>
__global__ void __launch_bounds__(kCeThreads, kCeBlocksPerSM)
    cache_attend_e4m3_kernel(const __grid_constant__ CacheAttnArgs p) {
  using L = CeSmem<DH>;
  using Walk = CpWalk<kCeRows>;
  extern __shared__ __align__(16) uint8_t ce_low[];
  uint8_t* const low = ce_low;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(low) + L::LOW + 1023) & ~uintptr_t(1023));
  // [2]: by the unit's number, where the one that waits may be a unit behind
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(low + L::OFF_BAR);
  uint64_t* pfull = kvfull + 1;   // P in shared memory, S^T read
  uint64_t* sfull = pfull + 1;    // [2] S^T in tensor memory; K's tile and the queries read
  uint64_t* pvdone = sfull + 2;   // [2] O^T updated; V's tile and P read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pvdone + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ CpSlice<kCeThreads> slice;
  __shared__ Walk walks[8], ahead[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(kvfull, 2);
    mbar_init(pfull, 4);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pvdone[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 128);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  cp_slice<kCeRows, kCeThreads>(p, slice);
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;  // S^T: columns 0 and 32, O^T: 64
  const long long T = slice.T, W = slice.W, u_lo = slice.u_lo, u_hi = slice.u_hi;
  Walk& walk = walks[warp];
  if (lane == 0 && u_lo < u_hi) {
    walk.begin(p, slice.b, slice.at, u_lo, u_hi - u_lo);
    if (warp < 2) ahead[warp] = walk;
  }
  __syncwarp();
  const uint32_t k_tile = smem_u32(smem + L::OFF_K), v_tile = smem_u32(smem + L::OFF_V), q_tile = smem_u32(smem + L::OFF_Q);
  const uint32_t p_tile = smem_u32(smem + L::OFF_P);

  if (u_lo >= u_hi) {  // no units: nothing but the common end
    if (tid == 0) ca_write_cut(p.cuts + blockIdx.x, 0, 0, 0, 0, 0, 0);
  } else if (warp < 2) {
    // ---------------- producers: 64 of a unit's 128 positions each ----------------
    constexpr int CH = DH / 16, RPI = 32 / CH;  // 16-byte chunks of a raw row, rows of a warp's instruction
    const long long v_off = p.c.planes == 2 ? (long long)p.c.kv_heads << p.c.page_shift : 0;
    const uint32_t raw0 = smem_u32(low + L::OFF_RAW);
    Walk& far = ahead[warp];
    int f_t = far.t_lo, f_n = 0;  // the unit to fetch next, and how many were
    bool f_more = true;
    long long at[2];
    auto look = [&]() {  // the cache's rows (K plane) of this lane's two positions of the unit to fetch
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        at[k] = -1;
        const int pos = f_t * kCpUnit + warp * 64 + k * 32 + lane;
        if (f_more && pos < far.s.len) {
          const long long r = cache_row(p.c, far.b, pos);
          if (r < 0) atomicOr(&g_device_error, kErrPages);
          else at[k] = r + ((long long)far.kvh << p.c.page_shift);
        }
      }
    };
    auto fetch = [&]() {
      if (f_more) {
        const uint32_t st = raw0 + (f_n % L::RST) * L::RAW_STAGE;
#pragma unroll
        for (int k = 0; k < 64 / RPI; ++k) {
          const int r = k * RPI + lane / CH, ch = lane % CH;
          const long long src = __shfl_sync(0xffffffffu, k * RPI < 32 ? at[0] : at[1], r & 31);
          const uint8_t* a = p.pages + (src < 0 ? 0 : src) * DH + ch * 16;
          const uint32_t dst = st + (warp * 64 + r) * DH + ch * 16, bytes = src < 0 ? 0u : 16u;
          cp_async16(dst, a, bytes);
          cp_async16(dst + L::RAW, a + (src < 0 ? 0 : v_off * DH), bytes);
        }
        // four scales a lane (positions 4 i ..: one page): lanes 0-15 K's, 16-31 V's
        const int i = lane & 15;
        const long long s0 = __shfl_sync(0xffffffffu, at[0], 4 * (i & 7)), s1 = __shfl_sync(0xffffffffu, at[1], 4 * (i & 7));
        const long long src = i < 8 ? s0 : s1;
        const uint32_t dst = st + 2 * L::RAW + (lane >> 4) * kCpUnit + warp * 64 + 4 * i;
        if (src >= 0) cp_async4(dst, p.scales + src + (lane >> 4) * v_off);
        else asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(0u) : "memory");
        ++f_n;
        if (++f_t >= far.t_hi) {
          f_more = far.next(p);
          f_t = far.t_lo;
        }
        look();
      }
      cp_async_commit();
    };
    look();
    fetch();
    fetch();
    int n = 0, seg = 0;
    bool ok = true;
    do {
      const int blocks = walk.t_hi - walk.t_lo;
      if (tid == 0 && p.c.lengths[walk.b] > walk.s.len) atomicOr(&g_device_error, kErrPages);
      if (tid == 0 && walk.s.rows > walk.s.take) atomicOr(&g_device_error, kErrOffsets);
      for (int i = 0; i < blocks; ++i, ++n) {
        fetch();
        cp_async_wait<2>();
        __syncwarp();
        if ((n >= 1 && !warp_wait(&sfull[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag)) ||
            (n >= 2 && !warp_wait(&pvdone[n & 1], ((n - 2) >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (i == 0) {  // the segment's queries, 16 rows a warp
          constexpr int QL = DH / 8, QR = 32 / QL;  // lanes of a row, rows at a time
          float* fac = reinterpret_cast<float*>(low + L::OFF_FAC) + (seg & 1) * kCeRows;
#pragma unroll
          for (int k = 0; k < 16 / QR; ++k) {
            const int r = warp * 16 + k * QR + lane / QL, ch = lane % QL;
            const bool live = r < walk.n_rows;
            const int row = walk.qb * kCeRows + (live ? r : 0), tok = row / p.group, head = walk.kvh * p.group + row % p.group;
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (live) w = *reinterpret_cast<const uint4*>(p.q + (long long)(walk.s.first_row + tok) * p.ldq + head * DH + ch * 8);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float f[8], mx = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] = __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
              mx = fmaxf(mx, fabsf(f[j]));
            }
#pragma unroll
            for (int d = QL / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            int ex = (int)(__float_as_uint(mx) >> 23) - 127;
            ex = mx == 0.f ? 14 : max(-100, min(ex, 120));
            const float down = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            sts128(q_tile + L::at(r, ch), make_uint4(pack_f16x2(f[0] * down, f[1] * down), pack_f16x2(f[2] * down, f[3] * down),
                                                     pack_f16x2(f[4] * down, f[5] * down), pack_f16x2(f[6] * down, f[7] * down)));
            if (ch == 0) fac[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
          }
        }
        const uint32_t st = raw0 + (n % L::RST) * L::RAW_STAGE;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
          const uint32_t dst = pl ? v_tile + (n & 1) * L::TILE : k_tile;
#pragma unroll 4
          for (int k = 0; k < 64 / RPI; ++k) {
            const int r = warp * 64 + k * RPI + lane / CH, ch = lane % CH;
            const uint4 w = lds128(st + pl * L::RAW + r * DH + ch * 16);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              h[2 * j] = e4m3x2_f16x2((uint16_t)u[j]);
              h[2 * j + 1] = e4m3x2_f16x2((uint16_t)(u[j] >> 16));
            }
            sts128(dst + L::at(r, 2 * ch), make_uint4(h[0], h[1], h[2], h[3]));
            sts128(dst + L::at(r, 2 * ch + 1), make_uint4(h[4], h[5], h[6], h[7]));
          }
        }
        {  // 64 scales of each plane: lanes 0-15 K's, 16-31 V's
          const uint32_t off = (lane >> 4) * kCpUnit + warp * 64 + 4 * (lane & 15);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(smem_u32(low + L::OFF_CODE) + (n & 1) * 2 * kCpUnit + off),
                       "r"(lds32(st + 2 * L::RAW + off))
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kvfull);
      }
      ++seg;
    } while (ok && walk.next(p));
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 2) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc_s = ce_idesc(128, kCeRows);
    constexpr uint32_t idesc_o = ce_idesc(128, kCeRows) | kIdescAMnMajor | kIdescBMnMajor;
    int n = 0;
    bool late = false, late_first = false, ok = true;
    auto flush = [&]() {  // O^T of unit n - 1
      if (!late) return;
      late = false;
      if (!warp_wait(pfull, (n - 1) & 1, abort_flag)) {
        ok = false;
        return;
      }
      tc_fence_after();
      const uint32_t v_base = v_tile + ((n - 1) & 1) * L::TILE;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16_elect(tmem_base + 64, L::desc_vt(v_base + k * 16 * L::ROW), L::desc_p(p_tile + k * 16 * 64), idesc_o,
                       !late_first || k > 0 ? 1u : 0u);
      umma_commit_elect(&pvdone[(n - 1) & 1]);
    };
    do {
      const int blocks = walk.t_hi - walk.t_lo;
      for (int i = 0; i < blocks && ok; ++i) {
        if (!warp_wait(kvfull, n & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < DH / 16; ++k)
          umma_f16_elect(tmem_base + (n & 1) * 32, L::desc(k_tile + k * 32), L::desc(q_tile + k * 32), idesc_s, k > 0 ? 1u : 0u);
        umma_commit_elect(&sfull[n & 1]);
        flush();
        late = true;
        late_first = i == 0;
        ++n;
      }
    } while (ok && walk.next(p));
    if (ok) flush();
  } else if (warp >= 4) {
    // ---------------- softmax and output: one thread per position ----------------
    const int q4 = warp & 3, th = q4 * 32 + lane;  // position in the unit
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16, o_tm = tmem_base + 64 + lane_off;
    float* const ref_s = reinterpret_cast<float*>(low + L::OFF_REF);      // [32]
    int* const end_s = reinterpret_cast<int*>(ref_s + kCeRows);            // [32]
    float* const part_s = ref_s + 2 * kCeRows;                             // [4][32] of one kind, [32] factors
    float* const sum_s = part_s + 5 * kCeRows;                             // [4][32]
    const uint8_t* const codes = low + L::OFF_CODE;
    int n = 0, seg = 0;
    bool ok = true;
    do {
      const int blocks = walk.t_hi - walk.t_lo, len = walk.s.len;
      float l[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) l[q] = 0.f;
      int e_ref = 0;
      if (th < kCeRows) {
        const bool live = th < walk.n_rows;
        long long e = len;
        if (p.causal) e = max(0ll, min(e, walk.pos0 + (walk.qb * kCeRows + (live ? th : 0)) / p.group + 1));
        ref_s[th] = -INFINITY;
        end_s[th] = live ? (int)e : 0;
      }
      int end_min = len;
      if (p.causal) end_min = (int)max(0ll, min((long long)len, walk.pos0 + (walk.qb * kCeRows) / p.group + 1));
      ce_vote(false);  // the rows' table is set
      const float* const fac = reinterpret_cast<const float*>(low + L::OFF_FAC) + (seg & 1) * kCeRows;
      for (int i = 0; i < blocks; ++i, ++n) {
        if (ok && !warp_wait(&sfull[n & 1], (n >> 1) & 1, abort_flag)) ok = false;
        tc_fence_after();
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem_base + (n & 1) * 32 + lane_off, v);
        const int pos = (walk.t_lo + i) * kCpUnit + th;
        const bool in = pos < len;
        const uint32_t ck = codes[(n & 1) * 2 * kCpUnit + th];
        const int cv = in ? codes[(n & 1) * 2 * kCpUnit + kCpUnit + th] : 0;
        const float kf = __uint_as_float(ck << 23);
        tmem_ld_wait();
        float x[32], top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(fac + q);
          x[q] = __uint_as_float(v[q]) * (f4.x * kf);
          x[q + 1] = __uint_as_float(v[q + 1]) * (f4.y * kf);
          x[q + 2] = __uint_as_float(v[q + 2]) * (f4.z * kf);
          x[q + 3] = __uint_as_float(v[q + 3]) * (f4.w * kf);
        }
        if ((walk.t_lo + i + 1) * kCpUnit > end_min) {
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (pos >= end_s[q]) x[q] = -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(ref_s + q);
          top = fmax3(top, x[q] > m4.x + kCaLazy ? 1.f : 0.f, x[q + 1] > m4.y + kCaLazy ? 1.f : 0.f);
          top = fmax3(top, x[q + 2] > m4.z + kCaLazy ? 1.f : 0.f, x[q + 3] > m4.w + kCaLazy ? 1.f : 0.f);
        }
        if (ce_vote(top > 0.f || cv > e_ref || !ok)) {
          // new references: the unit's maximum where it is larger by 2^8, its largest scale
          float mx[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) mx[q] = x[q];
          part_s[q4 * kCeRows + lane] = ce_across<true>(mx);
          if (lane == 0) sum_s[q4] = 0.f;
          const int ce = __reduce_max_sync(0xffffffffu, cv);
          if (lane == 0) sum_s[q4] = (float)ce;
          const bool bad = ce_vote(!ok);
          float f = 1.f;
          if (th < kCeRows) {
            const float old = ref_s[th];
            const float t = fmaxf(fmaxf(part_s[th], part_s[32 + th]), fmaxf(part_s[64 + th], part_s[96 + th]));
            const float now = t > old + kCaLazy ? t : old;
            f = now == old ? 1.f : fast_exp2(old - now);
            ref_s[th] = now;
            part_s[4 * kCeRows + th] = f;
          }
          const int e_new = max(e_ref, (int)fmaxf(fmaxf(sum_s[0], sum_s[1]), fmaxf(sum_s[2], sum_s[3])));
          const float fe = e_ref == 0 ? 0.f : fast_exp2((float)(e_ref - e_new));
          e_ref = e_new;
          if (bad) ok = false;
          // O^T up to the unit before is complete
          if (ok && i > 0 && !warp_wait(&pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag)) ok = false;
          ce_vote(false);  // the factors are set
          if (i > 0) {
            tc_fence_after();
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_tm, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float g = part_s[4 * kCeRows + q];
              l[q] *= g;
              o[q] = __float_as_uint(__uint_as_float(o[q]) * (g * fe));
            }
            tmem_st_32x32b_x32(o_tm, o);
            tmem_st_wait();
          }
        }
        // weights; P of the unit before has been read
        const int d = cv - e_ref + 127 + 7;
        const float vf = __uint_as_float((uint32_t)(in ? max(0, min(d, 134)) : 0) << 23);
        uint32_t pk[16];
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(ref_s + q);
          const float w0 = fast_exp2(x[q] - (m4.x == -INFINITY ? 0.f : m4.x)), w1 = fast_exp2(x[q + 1] - (m4.y == -INFINITY ? 0.f : m4.y));
          const float w2 = fast_exp2(x[q + 2] - (m4.z == -INFINITY ? 0.f : m4.z)), w3 = fast_exp2(x[q + 3] - (m4.w == -INFINITY ? 0.f : m4.w));
          l[q] += w0;
          l[q + 1] += w1;
          l[q + 2] += w2;
          l[q + 3] += w3;
          pk[q / 2] = pack_f16x2(w0 * vf, w1 * vf);
          pk[q / 2 + 1] = pack_f16x2(w2 * vf, w3 * vf);
        }
        if (ok && n > 0 && !warp_wait(&pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag)) ok = false;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts128(p_tile + CpSmem<32>::at(th, c), make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]));
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }
      // sums over the positions, output
      sum_s[q4 * kCeRows + lane] = ce_across<false>(l);
      if (ok && !warp_wait(&pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag)) ok = false;
      if (ce_vote(!ok)) ok = false;
      const bool whole = walk.t_lo == 0 && walk.t_hi == walk.units;
      const long long slot = 2 * (long long)blockIdx.x + !walk.first;
      if (ok) {
        tc_fence_after();
        uint32_t o[32];
        if (32 * q4 < DH) {  // this warp's lanes are columns of the head
          tmem_ld_32x32b_x32(o_tm, o);
          tmem_ld_wait();
          const float unscale = __uint_as_float((uint32_t)max(e_ref - 7, 0) << 23);
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            if (q < walk.n_rows) {
              const float sum = (sum_s[q] + sum_s[32 + q]) + (sum_s[64 + q] + sum_s[96 + q]);
              const float y = __uint_as_float(o[q]) * unscale;
              if (whole) {
                const int row = walk.qb * kCeRows + q, tok = row / p.group, head = walk.kvh * p.group + row % p.group;
                p.a[(long long)(walk.s.first_row + tok) * p.lda + head * DH + th] = __float2bfloat16_rn(sum == 0.f ? 0.f : y / sum);
              } else {
                p.part_o[(slot * kCeRows + q) * DH + th] = y;
              }
            }
          }
        }
        if (!whole && th < walk.n_rows)
          *reinterpret_cast<float2*>(p.part_ml + (slot * kCeRows + th) * 2) =
              make_float2(ref_s[th], (sum_s[th] + sum_s[32 + th]) + (sum_s[64 + th] + sum_s[96 + th]));
        tc_fence_before();
      }
      if (th == 0 && walk.left <= 0) {  // the slice's last segment
        const long long u0 = u_hi - walk.t_hi;
        ca_write_cut(p.cuts + blockIdx.x, walk.s.first_row, walk.qb * kCeRows, walk.n_rows, walk.kvh * p.group,
                     !whole && walk.t_lo == 0 ? (int)(ca_slice_of(u0 + walk.units - 1, W, T) - blockIdx.x) + 1 : 0, (int)slot);
      }
      ce_vote(false);  // the tables are read
      ++seg;
    } while (ok && walk.next(p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 128);
  }
}

}  // namespace whale
