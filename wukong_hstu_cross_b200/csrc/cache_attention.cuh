// cache_attention.cuh — attention of a chunk of rows over the paged cache:
//   a_i = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j / sqrt(d_head)) over the sequence's cached positions j
//   (causal: j <= position of row i; a row that sees nothing gives 0).
// Query head h reads K|V head h * kv_heads / n_heads.
#pragma once

#include "history_cache.cuh"

namespace whale {

struct CacheAttnArgs {
  ChunkView c;
  const __nv_bfloat16* q;  // [total, ldq]
  __nv_bfloat16* a;        // [total, lda]
  long long ldq, lda;
  const uint8_t* pages;
  const uint8_t* scales;
  int heads, group, causal;
  float scale_log2;  // log2(e) / sqrt(d_head)
};

// One warp per (row, head): a lane takes every 32nd position with a running maximum, sum and output of its
// own (fp32); the lanes meet by shuffles at the end.
template <int DH, bool FP8>
__global__ void __launch_bounds__(128) cache_attend_simple_kernel(const CacheAttnArgs p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long row = item / p.heads;
  const int h = (int)(item % p.heads), kvh = h / p.group;
  if (row >= p.c.total || row >= p.c.offsets[p.c.B]) return;
  const int b = chunk_seq(p.c, row);
  const long long len = min((long long)p.c.lengths[b], p.c.capacity);
  const long long pos = p.c.lengths[b] - (p.c.offsets[b + 1] - row);
  if (p.c.lengths[b] > len && lane == 0) atomicOr(&g_device_error, kErrPages);
  const long long end = p.causal ? min(len, pos + 1) : len;
  float q[DH], o[DH], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < DH; ++k) {
    q[k] = __bfloat162float(p.q[row * p.ldq + h * DH + k]) * p.scale_log2;
    o[k] = 0.f;
  }
  for (long long j = lane; j < end; j += 32) {
    const long long at = cache_row(p.c, b, j);
    if (at < 0) atomicOr(&g_device_error, kErrPages);
    float kv[2][DH];
#pragma unroll
    for (int pl = 0; pl < 2; ++pl) {
      const long long r = at + ((long long)((p.c.planes == 2 ? pl : 0) * p.c.kv_heads + kvh) << p.c.page_shift);
      const float sc = FP8 && at >= 0 ? __uint_as_float((uint32_t)p.scales[r] << 23) : 1.f;
#pragma unroll
      for (int k = 0; k < DH; ++k) {
        if (at < 0) kv[pl][k] = 0.f;
        else if constexpr (FP8) {
          __half_raw hr = __nv_cvt_fp8_to_halfraw(p.pages[r * DH + k], __NV_E4M3);
          kv[pl][k] = __half2float(*reinterpret_cast<__half*>(&hr)) * sc;
        } else kv[pl][k] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.pages)[r * DH + k]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < DH; ++k) s = fmaf(q[k], kv[0][k], s);
    const float mn = fmaxf(m, s), f = fast_exp2(m - mn), w = fast_exp2(s - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int k = 0; k < DH; ++k) o[k] = fmaf(o[k], f, w * kv[1][k]);
  }
  float mx = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const float f = m == -INFINITY ? 0.f : fast_exp2(m - mx);
  l *= f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
  for (int k = 0; k < DH; ++k) {
    float t = o[k] * f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    if (lane == k % 32) p.a[row * p.lda + h * DH + k] = __float2bfloat16_rn(l > 0.f ? t / l : 0.f);
  }
}

}  // namespace whale
