// cache_attention_tc.cuh — attention of a chunk over the paged cache, many rows per sequence (chunks of new events,
// candidates' tokens): the products on tcgen05, the softmax between them in registers. The formula, the row order
// and the masks are those of cache_attention.cuh.
//
// Bound: the exponentials. A tile of 128 rows x 128 positions takes 16384 of them, 1024 cycles of the SM's
// special-function units (16 a cycle), beside 2 * 128 * 128 * d_head multiply-adds in 128 (d_head 32) or 256 cycles
// each. (A share of them on the FMA pipe gained nothing: a softmax warp is as busy with the rest of a score.)
// Four users' chunks of 1000 rows against histories of up to 15000 (8 heads, d 512): 117 us, 520 TFLOP/s; on e4m3 130 us.
//
// One CTA per SM takes a contiguous slice of the units (128 positions of one item = (sequence, K|V head, block of 256
// rows)), all items' units laid end to end; causal items end at their last row's position. Partials where a slice cuts an
// item, joined by cache_attend_merge_kernel in the order of the slices. Inside a CTA, for two tiles of 128 rows:
//   warps 0-1   bf16: queries, and K and V of a unit, into stages by cp.async. e4m3: raw bytes by bulk copies, up to three
//               units ahead, from which warps 12-15 make the bf16 number that number * 2^e is. Rows in no page or
//               past the end are zeros.
//   warps 2-3   a tile each: S = Q K^T (128 x 128, K = d_head) and O += P V (128 x d_head, K = 128)
//   warps 4-11  one thread per row: scores out of tensor memory, running maximum (the reference is raised when the
//               tile's maximum exceeds it by 2^8, with the rescale of O in tensor memory then), weights as bf16 back
//               to tensor memory, where P V reads them, sums in fp32; at an item's end O / l, or the partial.
#pragma once

#include "cache_attention.cuh"

namespace whale {

constexpr int kCpRows = 256;     // rows of an item: two tiles
constexpr int kCpUnit = 128;     // positions of a unit
// Three warpgroups for bf16 pages: loads and products, and two of softmax; a fourth that converts for e4m3 ones.
constexpr int cp_threads(bool fp8) { return fp8 ? 512 : 384; }
constexpr int cp_producers(bool fp8) { return fp8 ? 4 : 2; }  // warps that write the tiles
// Registers after the start: a row's 128 scores stay in a softmax thread's. With what the block was launched with
// (65536 / threads, a multiple of 8) they must add up, or the last one would wait for ever. The compiler allots the launch's
// 168 (128) to all of them and spills 40 (24) bytes of a thread.
constexpr int kCpRegsLoad = 88, kCpRegsSoftmax = 208;                               // bf16: 3 x 168
constexpr int kCpRegsLoadE4m3 = 64, kCpRegsConvert = 96, kCpRegsSoftmaxE4m3 = 176;  // e4m3: 4 x 128
static_assert(kCpRegsLoad + 2 * kCpRegsSoftmax <= 3 * 168 && kCpRegsLoadE4m3 + kCpRegsConvert + 2 * kCpRegsSoftmaxE4m3 <= 4 * 128,
              "the warpgroups share what the block was launched with");
constexpr int kCpMinUnits = 2;

template <int DH, bool FP8>
struct CpSmem {
  static constexpr int ROW = 2 * DH;                         // bytes of a row of Q, K, V
  static constexpr uint32_t TILE = 128 * ROW;                // 128 rows
  static constexpr int ST = FP8 ? 3 : 4;
  static constexpr uint32_t RAW = FP8 ? 128 * DH : 0;         // raw e4m3 bytes of a plane
  static constexpr uint32_t RAW_STAGE = FP8 ? 2 * RAW + 256 : 0;  // K, V, K's scales, V's
  static constexpr int RST = 3;
  static constexpr int OFF_Q = 0;                            // [2 buffers][2 tiles]
  static constexpr int OFF_KV = OFF_Q + 4 * (int)TILE;       // [ST][K, V]
  static constexpr int OFF_RAW = OFF_KV + ST * 2 * (int)TILE;  // [RST]
  static constexpr int OFF_BAR = OFF_RAW + RST * (int)RAW_STAGE;
  // kvfull[ST], kvempty[ST], qfree[2], sfull[2], sfree[2], pfull[2], pfree[2], rawfull[RST], rawfree[RST], tmem slot,
  // abort flags[2], which 16 rows of a raw stage are there [RST]
  static constexpr size_t BYTES = 1024 + OFF_BAR + (2 * ST + 10 + 2 * RST) * 8 + 12 + 4 * RST;
  static_assert(BYTES <= 232448 - 1024, "shared memory of one CTA");
  // byte offset of 16-byte chunk ch of row r: the 128-byte (d_head 64) or 64-byte swizzle
  static __device__ __forceinline__ uint32_t at(int r, int ch) {
    return (uint32_t)r * ROW + (uint32_t)((ch ^ (DH == 64 ? r & 7 : (r >> 1) & 3)) << 4);
  }
  // matrix descriptors of rows of ROW bytes: K-major (Q, K), MN-major (V)
  static __device__ __forceinline__ uint64_t desc(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)1u << 46;
    d |= (uint64_t)((8 * ROW) >> 4) << 32;                   // 8-row groups
    d |= (uint64_t)(DH == 64 ? 2u : 4u) << 61;
    return d;
  }
};

// Units of one (K|V head, row block) of a sequence, and of all its row blocks.
__device__ __forceinline__ int cp_units(const CacheAttnArgs& p, const CaSeq& s, long long pos0, int qb) {
  long long e = s.len;
  if (p.causal) {
    const int last = (min(s.take * p.group, (qb + 1) * kCpRows) - 1) / p.group;
    e = min(e, pos0 + last + 1);
  }
  return e <= kCpUnit ? 1 : (int)((e + kCpUnit - 1) / kCpUnit);
}
__device__ __forceinline__ long long cp_head_units(const CacheAttnArgs& p, const CaSeq& s, int b, int blocks) {
  if (!p.causal) return blocks ? (long long)blocks * cp_units(p, s, 0, 0) : 0;
  const long long pos0 = (long long)p.c.lengths[b] - s.rows;
  long long n = 0;
  for (int qb = 0; qb < blocks; ++qb) n += cp_units(p, s, pos0, qb);
  return n;
}
__device__ __forceinline__ long long cp_workers(long long T, long long W) {
  const long long w = (T + kCpMinUnits - 1) / kCpMinUnits;
  return w < W ? w : W;
}

// A CTA's slice, segment by segment; every warp walks it for itself (in shared memory: the softmax warps have no
// registers to spare). Only the first segment is searched for: the next one begins the next item.
struct CpWalk {
  long long left;          // units after the present segment
  int b, kvh, qb;
  int t_lo, t_hi, units;   // the segment's units, and the item's
  int n_rows, first;       // rows of the item; the slice's first segment
  long long pos0;
  CaSeq s;

  __device__ __forceinline__ void sequence(const CacheAttnArgs& p, int b_) {
    b = b_;
    s = ca_seq(p, b, kCpRows);
    pos0 = (long long)p.c.lengths[b] - s.rows;
  }
  __device__ __forceinline__ void item(const CacheAttnArgs& p, int from) {
    units = cp_units(p, s, pos0, qb);
    n_rows = min(kCpRows, s.take * p.group - qb * kCpRows);
    t_lo = from;
    t_hi = (int)min((long long)units, t_lo + left);
    left -= t_hi - t_lo;
  }
  // Unit u of the slice's sequence b_, whose units begin at `at`; n units to take.
  __device__ __forceinline__ void begin(const CacheAttnArgs& p, int b_, long long at, long long u, long long n) {
    sequence(p, b_);
    const long long head = cp_head_units(p, s, b, s.blocks);
    kvh = (int)((u - at) / head);
    long long rem = u - at - kvh * head;
    if (!p.causal) {
      const int per = cp_units(p, s, pos0, 0);
      qb = (int)(rem / per);
      rem -= (long long)qb * per;
    } else {
      int per;
      for (qb = 0; rem >= (per = cp_units(p, s, pos0, qb)); ++qb) rem -= per;
    }
    left = n;
    first = 1;
    item(p, (int)rem);
  }
  // One lane: to the next segment, if there is one.
  __device__ __forceinline__ bool step(const CacheAttnArgs& p) {
    if (left <= 0) return false;
    first = 0;
    if (++qb >= s.blocks) {
      qb = 0;
      if (++kvh >= p.c.kv_heads) {
        kvh = 0;
        do {
          if (b + 1 >= p.c.B) return false;
          sequence(p, b + 1);
        } while (s.blocks == 0);
      }
    }
    item(p, 0);
    return true;
  }
  // The whole warp. Begin with the present segment: do { .. } while (next(p)).
  __device__ __forceinline__ bool next(const CacheAttnArgs& p) {
    __syncwarp();
    int more = 0;
    if ((threadIdx.x & 31) == 0) more = step(p);
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0);
  }
};

// Eight e4m3 numbers times 2^e as bf16 (exact).
__device__ __forceinline__ uint4 cp_bf16x8(uint2 q, float f) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = e4m3x2_f16x2((uint16_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1))));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v));
    o[i] = pack_bf16x2(x.x * f, x.y * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Bulk copy of `bytes` (a multiple of 16, as both addresses are) to shared memory, counted on `bar`.
__device__ __forceinline__ void cp_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The MMAs of a whole warp, issued by one elected lane. _ts: A (M = 128 rows, 16 bf16 columns as 8 words a row)
// in tensor memory.
__device__ __forceinline__ void umma_f16_elect(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar))
      : "memory");
}

// The whole warp's wait: one answer, so that a wait that ran out ends every lane's work at the same place.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(cp_threads(FP8), 1) cache_attend_tc_kernel(const __grid_constant__ CacheAttnArgs p) {
  using L = CpSmem<DH, FP8>;
  constexpr int kCpThreads = cp_threads(FP8);
  constexpr int ST = L::ST;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long sums[kCpThreads / 32 + 1];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* kvempty = kvfull + ST;
  uint64_t* qfree = kvempty + ST;  // [2] queries of a segment read by its last S
  uint64_t* sfull = qfree + 2;     // [2] per tile, as in attention_qtile.cuh
  uint64_t* sfree = sfull + 2;
  uint64_t* pfull = sfree + 2;
  uint64_t* pfree = pfull + 2;
  uint64_t* rawfull = pfree + 2;   // [RST] e4m3: raw bytes of a unit there, and read by both producers
  uint64_t* rawfree = rawfull + L::RST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rawfree + L::RST);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* pieces_of = reinterpret_cast<volatile uint32_t*>(tmem_slot + 3);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kvfull[s], cp_producers(FP8));
      mbar_init(&kvempty[s], 2);  // both tiles
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&qfree[h], 2);
      mbar_init(&sfull[h], 1);
      mbar_init(&sfree[h], 4);
      mbar_init(&pfull[h], 4);
      mbar_init(&pfree[h], 1);
    }
    for (int s = 0; s < L::RST; ++s) {
      mbar_init(&rawfull[s], 1);
      mbar_init(&rawfree[s], cp_producers(FP8));
    }
    abort_flag[0] = abort_flag[1] = 0;  // [1]: of the wait for copies in flight at the end
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();

  // units before each thread's run of sequences; the slice; its first sequence
  __shared__ int start_b;
  __shared__ long long start_at;
  const int run = (p.c.B + kCpThreads - 1) / kCpThreads;
  const int b_lo = min(p.c.B, tid * run), b_hi = min(p.c.B, b_lo + run);
  auto seq_units = [&](int b) {
    const CaSeq s = ca_seq(p, b, kCpRows);
    return cp_head_units(p, s, b, s.blocks) * p.c.kv_heads;
  };
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += seq_units(b);
    if (blockIdx.x == 0) ca_report(p, b, ca_seq(p, b, kCpRows));
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  long long base = 0, T = 0;
  for (int w = 0; w < kCpThreads / 32; ++w) {
    base += w < warp ? sums[w] : 0;
    T += sums[w];
  }
  const long long W = cp_workers(T, gridDim.x);
  __shared__ CpWalk walks[kCpThreads / 32];
  const long long u_lo = W > (long long)blockIdx.x ? (long long)blockIdx.x * T / W : T;
  const long long u_hi = W > (long long)blockIdx.x ? ((long long)blockIdx.x + 1) * T / W : T;
  {
    long long at = base + scan - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = seq_units(b);
      if (at <= u_lo && u_lo < at + n) {
        start_b = b;
        start_at = at;
      }
      at += n;
    }
  }
  // nothing to join, until the slice's last segment says otherwise: a wait that runs out ends the slice before that
  if (tid == 0) ca_write_cut(p.cuts + blockIdx.x, 0, 0, 0, 0, 0, 0);
  __syncthreads();
  CpWalk& walk = walks[warp];
  if (lane == 0 && u_lo < u_hi) walk.begin(p, start_b, start_at, u_lo, u_hi - u_lo);
  __syncwarp();

  // A segment's queries into its buffer, the producers' warps each a part of the rows, by cp.async.
  auto queries = [&](int seg, int part) -> bool {
    constexpr int CH = L::ROW / 16, RPI = 32 / CH, PARTS = cp_producers(FP8);
    if (seg >= 2 && !warp_wait(&qfree[seg & 1], ((seg >> 1) - 1) & 1, abort_flag)) return false;
    const uint32_t q_base = smem_u32(smem + L::OFF_Q) + (seg & 1) * 2 * L::TILE;
#pragma unroll 4
    for (int k = 0; k < kCpRows / PARTS / RPI; ++k) {
      const int r = part * (kCpRows / PARTS) + k * RPI + lane / CH, ch = lane % CH;
      const bool live = r < walk.n_rows;
      const int row = walk.qb * kCpRows + (live ? r : 0), tok = row / p.group, head = walk.kvh * p.group + row % p.group;
      cp_async16(q_base + (r >> 7) * L::TILE + L::at(r & 127, ch),
                 p.q + (long long)(walk.s.first_row + tok) * p.ldq + head * DH + ch * 8, live ? 16u : 0u);
    }
    return true;
  };

  if (u_lo >= u_hi) {  // no units: nothing but the common end
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FP8 ? kCpRegsLoadE4m3 : kCpRegsLoad));
    if (warp < 2) {
      if constexpr (!FP8) {
        // ---------------- bf16: queries and tiles, 64 of a unit's positions a warp ----------------
        constexpr int CH = L::ROW / 16, RPI = 32 / CH;  // 16-byte chunks of a row, rows of a warp's instruction
        int n = 0, seg = 0;                             // tiles and segments so far
        bool ok = true;
        const long long v_off = p.c.planes == 2 ? (long long)p.c.kv_heads << p.c.page_shift : 0;
        do {
          const long long kv_off = (long long)walk.kvh << p.c.page_shift;
          const int t_lo = walk.t_lo, t_hi = walk.t_hi, len = walk.s.len, seq = walk.b;
          // rows (of each plane's first head) of this lane's two positions of unit i: the warp has 64 of the 128
          long long at[2];
          auto look = [&](int i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int pos = i * kCpUnit + warp * 64 + k * 32 + lane;
              at[k] = -1;
              if (i < t_hi && pos < len) {
                const long long r = cache_row(p.c, seq, pos);
                if (r < 0) atomicOr(&g_device_error, kErrPages);
                else at[k] = r + kv_off;
              }
            }
          };
          look(t_lo);
          if (!queries(seg, warp)) break;
          for (int i = t_lo; i < t_hi; ++i, ++n) {
            if (n >= ST && !warp_wait(&kvempty[n % ST], (n / ST - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t st = smem_u32(smem + L::OFF_KV) + (n % ST) * 2 * L::TILE;
            const long long a0 = at[0], a1 = at[1];
            look(i + 1);
#pragma unroll
            for (int k = 0; k < 64 / RPI; ++k) {
              const int r = k * RPI + lane / CH, ch = lane % CH;
              const long long src = __shfl_sync(0xffffffffu, k * RPI < 32 ? a0 : a1, r & 31);
              const uint8_t* a = p.pages + (src < 0 ? 0 : src) * L::ROW + ch * 16;
              const uint32_t dst = st + L::at(warp * 64 + r, ch), bytes = src < 0 ? 0u : 16u;
              cp_async16(dst, a, bytes);
              cp_async16(dst + L::TILE, a + (src < 0 ? 0 : v_off * L::ROW), bytes);
            }
            cp_async_commit();
            // handed on at once: waiting to fill the next stage first would tie this tile to the P V two tiles back
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kvfull[n % ST]);
          }
          ++seg;
        } while (ok && walk.next(p));
        asm volatile("cp.async.wait_all;" ::: "memory");
      } else if (warp == 0) {
        // ---------------- e4m3: raw bytes by bulk copies, a lane per piece of a page's rows ----------------
        const int rows = min(1 << p.c.page_shift, kCpUnit), pieces = kCpUnit / rows;  // 16 to 128 rows, 8 to 1 pieces
        const long long v_off = p.c.planes == 2 ? (long long)p.c.kv_heads << p.c.page_shift : 0;
        int n = 0;
        bool ok = true;
        do {
          const long long kv_off = (long long)walk.kvh << p.c.page_shift;
          auto look = [&](int t) -> long long {  // the cache's row where this lane's piece of unit t begins
            const int pos = t * kCpUnit + lane * rows;
            if (lane >= pieces || t >= walk.t_hi || pos >= walk.s.len) return -1;
            const long long r = cache_row(p.c, walk.b, pos);
            if (r < 0) atomicOr(&g_device_error, kErrPages);
            return r;
          };
          long long at = look(walk.t_lo);
          for (int t = walk.t_lo; t < walk.t_hi; ++t, ++n) {
            const int s = n % L::RST;
            if (n >= L::RST && !warp_wait(&rawfree[s], (n / L::RST - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t have = __ballot_sync(0xffffffffu, at >= 0);
            if (lane == 0) {
              uint32_t bits = 0;  // of 16 rows each
              for (int k = 0; k < pieces; ++k)
                if (have >> k & 1) bits |= ((1u << (rows >> 4)) - 1) << (k * (rows >> 4));
              pieces_of[s] = bits;
              mbar_arrive_expect_tx(&rawfull[s], __popc(have) * rows * 2 * (DH + 1));
            }
            __syncwarp();
            if (at >= 0) {
              const uint32_t st = smem_u32(smem + L::OFF_RAW) + s * L::RAW_STAGE, r = lane * rows;
              const long long k_row = at + kv_off, v_row = k_row + v_off;
              cp_bulk(st + r * DH, p.pages + k_row * DH, rows * DH, &rawfull[s]);
              cp_bulk(st + L::RAW + r * DH, p.pages + v_row * DH, rows * DH, &rawfull[s]);
              cp_bulk(st + 2 * L::RAW + r, p.scales + k_row, rows, &rawfull[s]);
              cp_bulk(st + 2 * L::RAW + 128 + r, p.scales + v_row, rows, &rawfull[s]);
            }
            at = look(t + 1);
          }
        } while (ok && walk.next(p));
        // nothing may be in flight when the block ends, also where a wait ran out
        for (int k = max(0, n - L::RST); k < n; ++k)
          mbar_wait(&rawfull[k % L::RST], (k / L::RST) & 1, abort_flag + 1, 100000000ull);
      }
    } else {
      // ---------------- MMA issuers: warp 2 + h for tile h ----------------
      // A unit's S as soon as the softmax warps have read the S before it, across segments too, then the P V of the
      // unit before. The whole warp runs this with one lane elected per instruction, so that descriptors are uniform.
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DH) | kIdescBMnMajor;
      const int h = warp - 2;
      const uint32_t kv0 = smem_u32(smem + L::OFF_KV), q0 = smem_u32(smem + L::OFF_Q);
      const uint32_t s_tm = tmem_base + h * 128, o_tm = tmem_base + 256 + h * 64, p_tm = tmem_base + 384 + h * 64;
      int n = 0, seg = 0, c = 0;       // units, segments, and units that have this tile, so far
      int late = -1;                   // unit whose P V is to come
      bool late_first = false, ok = true;
      auto flush = [&]() {
        if (late < 0) return;
        if (!warp_wait(&pfull[h], (c - 1) & 1, abort_flag)) {
          ok = false;
          return;
        }
        tc_fence_after();
        const uint32_t v_base = kv0 + ((late % ST) * 2 + 1) * L::TILE;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_ts(o_tm, p_tm + k * 8, L::desc(v_base + k * 16 * L::ROW), idesc_pv, !late_first || k > 0 ? 1u : 0u);
        umma_commit_elect(&pfree[h]);
        umma_commit_elect(&kvempty[late % ST]);
        late = -1;
      };
      do {
        const int blocks = walk.t_hi - walk.t_lo;
        const bool active = walk.n_rows > 128 * h;
        const uint32_t q_base = q0 + ((seg & 1) * 2 + h) * L::TILE;
        for (int i = 0; i < blocks && ok; ++i, ++n) {
          ok = warp_wait(&kvfull[n % ST], (n / ST) & 1, abort_flag);
          if (!ok) break;
          if (!active) {
            flush();
            if (lane == 0) {
              mbar_arrive(&kvempty[n % ST]);
              if (i == blocks - 1) mbar_arrive(&qfree[seg & 1]);
            }
            continue;
          }
          if (c > 0 && !warp_wait(&sfree[h], (c - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t k_base = kv0 + (n % ST) * 2 * L::TILE;
#pragma unroll
          for (int k = 0; k < DH / 16; ++k)
            umma_f16_elect(s_tm, L::desc(q_base + k * 32), L::desc(k_base + k * 32), idesc_s, k > 0 ? 1u : 0u);
          umma_commit_elect(&sfull[h]);
          if (i == blocks - 1) umma_commit_elect(&qfree[seg & 1]);
          flush();
          late = n;
          late_first = i == 0;
          ++c;
        }
        ++seg;
      } while (ok && walk.next(p));
      if (ok) flush();
    }
  } else if (FP8 && warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCpRegsConvert));
    // ---------------- e4m3: queries, and raw bytes to tiles, 32 of a unit's positions a warp ----------------
    const int cw = warp - 12;
    int n = 0, seg = 0;
    bool ok = true;
    do {
      const int t_lo = walk.t_lo, t_hi = walk.t_hi, len = walk.s.len;
      if (!queries(seg, cw)) break;
      constexpr int RCH = DH / 16, RRPI = 32 / RCH, PASS = 32 / RRPI;  // raw rows are DH bytes
      for (int i = t_lo; i < t_hi; ++i, ++n) {
        if (!warp_wait(&rawfull[n % L::RST], (n / L::RST) & 1, abort_flag) ||
            (n >= ST && !warp_wait(&kvempty[n % ST], (n / ST - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        // rows past the end, and rows in no page, are zeros, whatever their raw bytes are
        const uint32_t there = pieces_of[n % L::RST];
        const int left = len - i * kCpUnit;
        const uint8_t* const raw = smem + L::OFF_RAW + (n % L::RST) * L::RAW_STAGE;
        const uint32_t st = smem_u32(smem + L::OFF_KV) + (n % ST) * 2 * L::TILE;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
          uint4 w[PASS];
          float f[PASS];
#pragma unroll
          for (int k = 0; k < PASS; ++k) {
            const int r = cw * 32 + k * RRPI + lane / RCH;
            w[k] = *reinterpret_cast<const uint4*>(raw + pl * L::RAW + (cw * 32 + k * RRPI) * DH + lane * 16);
            const uint32_t code = raw[2 * L::RAW + pl * 128 + r];
            if (r >= left || !(there >> (r >> 4) & 1)) {
              w[k] = make_uint4(0u, 0u, 0u, 0u);
              f[k] = 0.f;
            } else {
              f[k] = __uint_as_float(code << 23);
            }
          }
#pragma unroll
          for (int k = 0; k < PASS; ++k) {
            const int r = cw * 32 + k * RRPI + lane / RCH, ch = lane % RCH;
            sts128(st + pl * L::TILE + L::at(r, 2 * ch), cp_bf16x8(make_uint2(w[k].x, w[k].y), f[k]));
            sts128(st + pl * L::TILE + L::at(r, 2 * ch + 1), cp_bf16x8(make_uint2(w[k].z, w[k].w), f[k]));
          }
        }
        if (i == t_lo) {  // the queries too
          cp_async_commit();
          cp_async_wait<0>();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&kvfull[n % ST]);
          mbar_arrive(&rawfree[n % L::RST]);
        }
      }
      ++seg;
    } while (ok && walk.next(p));
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FP8 ? kCpRegsSoftmaxE4m3 : kCpRegsSoftmax));
    // ---------------- softmax and output: one thread per row ----------------
    const int q4 = warp & 3, h = (warp - 4) >> 2, row = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_tm = tmem_base + h * 128 + lane_off, o_tm = tmem_base + 256 + h * 64 + lane_off;
    const uint32_t p_tm = tmem_base + 384 + h * 64 + lane_off;  // weights, two a word
    int c = 0;  // blocks of this tile so far
    bool ok = true;
    do {
      const int blocks = walk.t_hi - walk.t_lo;
      if (walk.n_rows <= 128 * h) continue;
      const int r = 128 * h + row;
      const bool live = r < walk.n_rows;
      int end = walk.s.len;  // of the positions from the segment's first on
      if (p.causal) end = (int)max(0ll, min((long long)end, walk.pos0 + (walk.qb * kCpRows + (live ? r : 0)) / p.group + 1));
      end -= walk.t_lo * kCpUnit;
      float m_run = -INFINITY, l = 0.f;
      for (int i = 0; i < blocks && ok; ++i, ++c) {
        if (!warp_wait(&sfull[h], c & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[128];
        tmem_ld_32x32b_x32(s_tm + 0, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
        tmem_ld_32x32b_x32(s_tm + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
        tmem_ld_32x32b_x32(s_tm + 64, *reinterpret_cast<uint32_t(*)[32]>(&v[64]));
        tmem_ld_32x32b_x32(s_tm + 96, *reinterpret_cast<uint32_t(*)[32]>(&v[96]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[h]);
        const int nv = end - i * kCpUnit;  // positions of the block that this row sees
        const bool full = __all_sync(0xffffffffu, nv >= kCpUnit);
        if (!full) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= nv) v[j] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 128; j += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmax3(mx[k], __uint_as_float(v[j + 2 * k]), __uint_as_float(v[j + 2 * k + 1]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        const float m_new = mt > m_run + kCaLazy ? mt : m_run;
        bool may_write = i == 0;  // P of the block before has been read and O updated
        if (i > 0 && __any_sync(0xffffffffu, m_new != m_run)) {
          if (!warp_wait(&pfree[h], (c - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          may_write = true;
          tc_fence_after();
          const float f = m_new == m_run ? 1.f : fast_exp2(m_run - m_new);
#pragma unroll 1
          for (int k = 0; k < DH / 32; ++k) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_tm + k * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st_32x32b_x32(o_tm + k * 32, o);
          }
          tmem_st_wait();
          tc_fence_before();
          l *= f;
        }
        m_run = m_new;
        const float ref = (m_run == -INFINITY ? 0.f : m_run) + kCaLazy;
        const uint64_t sc2 = f2pack(p.scale_log2, p.scale_log2), nr2 = f2pack(-ref, -ref);
        {
          uint64_t ls[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // 64 positions each
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int j = 64 * half + 2 * k;
              const uint64_t x = ffma2(f2pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sc2, nr2);
              float w0, w1;
              f2unpack(x, w0, w1);
              w0 = fast_exp2(w0);
              w1 = fast_exp2(w1);
              ls[k & 1] = fadd2(ls[k & 1], f2pack(w0, w1));
              pk[k] = pack_bf16x2(w0, w1);
            }
            if (half == 0 && !may_write) {
              if (!warp_wait(&pfree[h], (c - 1) & 1, abort_flag)) ok = false;
              tc_fence_after();
            }
            tmem_st_32x32b_x32(p_tm + 32 * half, pk);
          }
          float a0, a1;
          f2unpack(fadd2(ls[0], ls[1]), a0, a1);
          l += a0 + a1;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[h]);
      }
      if (!ok || !warp_wait(&pfree[h], (c - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = walk.t_lo == 0 && walk.t_hi == walk.units;
      const long long slot = 2 * (long long)blockIdx.x + !walk.first;
      const float f = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.f;
      const int srow = walk.qb * kCpRows + (live ? r : 0), tok = srow / p.group, head = walk.kvh * p.group + srow % p.group;
      __nv_bfloat16* dst = p.a + (long long)(walk.s.first_row + tok) * p.lda + head * DH;
      float* po = p.part_o + (slot * kCpRows + r) * DH;
#pragma unroll 1
      for (int k = 0; k < DH / 32; ++k) {  // collective: every lane loads, live rows are stored
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_tm + k * 32, o);
        tmem_ld_wait();
        if (!live) continue;
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(dst + k * 32 + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(po + k * 32 + 4 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      if (live && !whole) *reinterpret_cast<float2*>(p.part_ml + (slot * kCpRows + r) * 2) = make_float2(m_run, l);
      if (r == 0 && walk.left <= 0) {  // the slice's last segment
        const long long u0 = u_hi - walk.t_hi;  // the item's first unit
        ca_write_cut(p.cuts + blockIdx.x, walk.s.first_row, walk.qb * kCpRows, walk.n_rows, walk.kvh * p.group,
                     !whole && walk.t_lo == 0 ? (int)(ca_slice_of(u0 + walk.units - 1, W, T) - blockIdx.x) + 1 : 0, (int)slot);
      }
      tc_fence_before();
    } while (ok && walk.next(p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// One CTA per slice and kCaMergeRows rows: joins the partials of the item that begins in the slice and does not end
// there, in the order of the slices.
constexpr int kCaMergeThreads = 256, kCaMergeRows = 32;
template <int DH, int BM>
__global__ void __launch_bounds__(kCaMergeThreads) cache_attend_merge_kernel(const CacheAttnArgs p) {
  __shared__ float4 so[kCaMergeThreads];
  __shared__ float2 sml[kCaMergeThreads];
  pdl_wait();
  pdl_trigger();
  const int4* const cut = reinterpret_cast<const int4*>(p.cuts + blockIdx.x);
  const int4 c0 = cut[0], c1 = cut[1];
  const int first_row = c0.x, head0 = c0.w, n = c1.x, slot0 = c1.y;
  const int row0 = blockIdx.y * kCaMergeRows, n_rows = min(kCaMergeRows, c0.z - row0);  // of the block
  if (n_rows <= 0 || !cut_valid(p.c, p.group, BM, gridDim.x, blockIdx.x, first_row, c0.y, c0.z, head0, n, slot0)) return;
  const int vecs = n_rows * (DH / 4);
  // `groups` threads take every groups-th partial of one vector of 4 columns
  int groups = 1;
  while (groups * 2 * vecs <= kCaMergeThreads && groups < n) groups *= 2;
  const int per = kCaMergeThreads / groups, grp = threadIdx.x / per;
  auto join = [](float& m, float& l, float4& o, const float2& ml, const float4& x) {
    const float mn = fmaxf(m, ml.x);
    const float fo = m == mn ? 1.f : fast_exp2(m - mn), fx = ml.x == mn ? 1.f : fast_exp2(ml.x - mn);
    m = mn;
    l = l * fo + ml.y * fx;
    o.x = o.x * fo + x.x * fx;
    o.y = o.y * fo + x.y * fx;
    o.z = o.z * fo + x.z * fx;
    o.w = o.w * fo + x.w * fx;
  };
  for (int v0 = 0; v0 < vecs; v0 += per) {
    const int v = v0 + threadIdx.x % per, r = v / (DH / 4), c4 = v % (DH / 4);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (v < vecs) {
#pragma unroll 8
      for (int k = grp; k < n; k += groups) {
        const long long slot = (long long)(k == 0 ? slot0 : 2 * ((int)blockIdx.x + k)) * BM + row0 + r;
        join(m, l, o, *reinterpret_cast<const float2*>(p.part_ml + slot * 2),
             *reinterpret_cast<const float4*>(p.part_o + slot * DH + 4 * c4));
      }
    }
    if (groups > 1) {  // one round: vecs <= per
      so[threadIdx.x] = o;
      sml[threadIdx.x] = make_float2(m, l);
      __syncthreads();
      if (grp == 0 && v < vecs)
        for (int k = 1; k < groups; ++k) join(m, l, o, sml[k * per + v], so[k * per + v]);
    }
    if (grp == 0 && v < vecs) {
      const float f = l == 0.f ? 0.f : 1.f / l;
      const int row = c0.y + row0 + r, tok = row / p.group, head = head0 + row % p.group;
      *reinterpret_cast<uint2*>(p.a + (long long)(first_row + tok) * p.lda + head * DH + 4 * c4) =
          make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    }
  }
}

}  // namespace whale
