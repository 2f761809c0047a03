// Attention over the paged grouped-head cache, one block per (query, head):
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  s_j = scale q . k_j
// Every warp walks its own keys with a running maximum, sum and accumulator
// (fp32); the four are joined at the end.
#pragma once

#include "paged_common.cuh"

namespace mla {

namespace pg {

constexpr int kRowThreads = 128;

template <typename T, int kD>
__global__ void __launch_bounds__(kRowThreads) attend_row_kernel(GqaParams p) {
  constexpr int E = kD / 32;
  __shared__ int32_t cu_shared[kCuShared + 1];
  __shared__ float sm[4], sl[4], so[4][kD];
  CuSearch cs{};
  if (p.cu) {
    cs = stage_cu(p.cu, p.B, cu_shared);
    __syncthreads();
  }
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, hk = h / p.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t b;
  int64_t n, i;
  if (p.cu) {
    b = sequence_of(cs, cu_shared, (int32_t)t);
    if (b < 0) return;
    const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
    if (t >= c1) return;
    n = c1 - c0;
    i = t - c0;
    if (c0 < 0 || c1 > p.T || n > p.max_new) {
      if (threadIdx.x == 0) record_error(p.status, MLA_ERR_BOUNDS);
      return;
    }
  } else {
    b = (int32_t)(t / p.Lq);
    n = p.Lq;
    i = t % p.Lq;
  }
  int64_t L = p.seq_lens[b];
  if (L < 0 || L > (int64_t)p.bt_stride * kPage) {
    if (threadIdx.x == 0) record_error(p.status, MLA_ERR_BOUNDS);
    L = 0;
  }
  const int64_t keys = L - n + i + 1;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const T* qp = static_cast<const T*>(p.q) + (t * p.Hq + h) * kD;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = (float)qp[lane + 32 * e] * p.scale_log2;
    o[e] = 0.f;
  }
  for (int64_t j = warp; j < keys; j += 4) {
    const int64_t block = p.block_table[(int64_t)b * p.bt_stride + j / kPage];
    if (block < 0 || block >= p.num_blocks) {
      if (lane == 0) record_error(p.status, MLA_ERR_BOUNDS);
      continue;
    }
    const int64_t at = ((block * p.Hk + hk) * kPage + j % kPage) * kD + lane;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * (float)static_cast<const T*>(p.k_pool)[at + 32 * e];
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s), a = exp2f(m - mn), x = exp2f(s - mn);
    m = mn;
    l = l * a + x;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + x * (float)static_cast<const T*>(p.v_pool)[at + 32 * e];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  if (threadIdx.x < kD) {
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float total = 0.f, x = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float a = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - top);
      total += sl[w] * a;
      x += so[w][threadIdx.x] * a;
    }
    static_cast<T*>(p.out)[(t * p.Hq + h) * kD + threadIdx.x] = (T)(total > 0.f ? x / total : 0.f);
  }
}

}  // namespace pg
}  // namespace mla
