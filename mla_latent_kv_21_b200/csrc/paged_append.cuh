// Appending to the paged caches, with the position rotation on the way.
//
//   x'[a] = x[a] cos - x[b] sin,  x'[b] = x[b] cos + x[a] sin   per pair (a, b)
//
// in fp32, rounded once. A thread owns a unit of two 16-byte vectors that hold
// whole pairs: vectors u and u + D/2 of the half style, vectors 2u and 2u + 1
// of the interleaved style, and (either style) two neighbouring vectors of the
// part that is not rotated. Both styles need the same slice of the rotation
// table for a unit, so a thread loads its cos and sin once and walks heads.
#pragma once

#include "paged_common.cuh"

namespace mla {

struct AppendParams {
  // sources (element strides)
  const void* k; int64_t k_ts, k_hs;
  const void* v; int64_t v_ts, v_hs;
  const void* q; int64_t q_ts, q_hs;
  void* q_out;
  void* k_pool;            // grouped heads; latent: the pool or the codes
  void* v_pool;            // grouped heads; FP8 latent: the RoPE keys
  float* kv_scale;         // FP8 latent
  void* kv_rows;           // latent
  int32_t* status;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu;
  const float* table;
  int64_t table_rows, num_blocks, T;
  int32_t bt_stride, B, Lq;
  int32_t Hq, Hk, d;       // latent: Hq query heads, d unused
  int32_t D, r;            // rotated elements; latent rank
  int32_t heads_per_cta;
};

namespace pg {

// Where token t goes: its position and its row slot in the cache (block * 64 +
// slot), or pos = -1 if it has no place (not a token of a sequence, or an
// error, which is recorded by the calling thread if `tell`). The lengths are the
// decode's: without prefix sums those below Lq are none.
struct Place {
  int64_t pos;
  int64_t block;
  int32_t slot;
};
__device__ __forceinline__ Place place_of(const AppendParams& p, const CuSearch& cs, const int32_t* cu_shared,
                                          int64_t t, bool tell) {
  Place r{-1, 0, 0};
  int32_t b;
  int64_t n, i;
  if (p.cu) {
    b = sequence_of(cs, cu_shared, (int32_t)t);
    if (b < 0) return r;
    const int64_t c0 = cs.step == 1 ? cu_shared[b] : p.cu[b], c1 = cs.step == 1 ? cu_shared[b + 1] : p.cu[b + 1];
    if (t >= c1) return r;          // prefix sums that do not rise own no such token
    n = c1 - c0;
    i = t - c0;
    if (c0 < 0 || c1 > p.T) {
      if (tell) record_error(p.status, MLA_ERR_BOUNDS);
      return r;
    }
  } else {
    b = (int32_t)(t / p.Lq);
    n = p.Lq;
    i = t - (int64_t)b * p.Lq;
  }
  const int64_t L = p.seq_lens[b], pos = L - n + i;
  // without prefix sums a slot of L < Lq tokens (0: idle) has only its last L rows
  if (!p.cu && L >= 0 && pos < 0) return r;
  bool ok = L >= (p.cu ? n : 0) && L <= kMaxLen && L <= (int64_t)p.bt_stride * kPage && (p.D == 0 || pos < p.table_rows);
  if (ok) {
    r.block = p.block_table[(int64_t)b * p.bt_stride + pos / kPage];
    r.slot = (int32_t)(pos % kPage);
    ok = r.block >= 0 && r.block < p.num_blocks;
  }
  if (!ok) {
    if (tell) record_error(p.status, MLA_ERR_BOUNDS);
    return r;
  }
  r.pos = pos;
  return r;
}

// ------------------------------------------------------ 16-byte vectors ------
template <typename T> struct Vec {                 // 8 values of a 16-bit type
  static constexpr int n = 8;
  static __device__ __forceinline__ void to(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Pack<T>::to(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 of(const float (&x)[8]) {
    return make_uint4(Pack<T>::of(x[0], x[1]), Pack<T>::of(x[2], x[3]), Pack<T>::of(x[4], x[5]),
                      Pack<T>::of(x[6], x[7]));
  }
};
template <> struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void to(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 of(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// A unit's place in a head of which D elements rotate, and its angles.
template <typename T> struct Unit {
  static constexpr int V = Vec<T>::n;
  int u, at0, at1;         // its number; element offsets of its two vectors
  bool turn, half;
  float c[V], s[V];

  __device__ __forceinline__ Unit(int u_, int D, bool half_style) : u(u_), half(half_style) {
    turn = u < D / (2 * V);
    at0 = turn && half ? u * V : 2 * u * V;
    at1 = at0 + (turn && half ? D / 2 : V);
  }
  __device__ __forceinline__ void angles(const float* row, int D) {
    if (!turn) return;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(row + u * V + i);
      const float4 b = *reinterpret_cast<const float4*>(row + D / 2 + u * V + i);
      c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
      s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
    }
  }
  // x0, x1: the values of the two vectors
  __device__ __forceinline__ void rotate(float (&x0)[V], float (&x1)[V]) const {
    if (!turn) return;
    if (half) {
#pragma unroll
      for (int i = 0; i < V; ++i) pair(x0[i], x1[i], c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        pair(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
        pair(x1[2 * i], x1[2 * i + 1], c[V / 2 + i], s[V / 2 + i]);
      }
    }
  }
  static __device__ __forceinline__ void pair(float& a, float& b, float c, float s) {
    const float ra = a * c - b * s, rb = b * c + a * s;
    a = ra;
    b = rb;
  }
};

// One thread's unit of every step-th head from h0 to h1 - 1 of one token, four
// heads' loads at a time and the next four under way while a batch is turned and
// stored.
// place(): where the token goes and its angles, false if it goes nowhere; it is
// called with the first loads in flight, since its chain of dependent reads
// (prefix sums, length, block, table row) is as long as theirs.
template <typename T, typename Src, typename Place, typename Dst>
__device__ __forceinline__ void walk_heads(Unit<T>& unit, int h0, int h1, int step, int turned, Src src, Place place, Dst dst) {
  uint4 a[4], b[4];
  auto load = [&](int hb) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (hb + j * step < h1) {
        const T* x = src(hb + j * step);
        a[j] = *reinterpret_cast<const uint4*>(x + unit.at0);
        b[j] = *reinterpret_cast<const uint4*>(x + unit.at1);
      }
  };
  load(h0);
  if (!place()) return;
  for (int hb = h0; hb < h1; hb += 4 * step) {
    uint4 x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      y[j] = b[j];
    }
    if (hb + 4 * step < h1) load(hb + 4 * step);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int h = hb + j * step;
      if (h < h1) {
        if (unit.turn && h < turned) {
          float x0[Unit<T>::V], x1[Unit<T>::V];
          Vec<T>::to(x[j], x0);
          Vec<T>::to(y[j], x1);
          unit.rotate(x0, x1);
          x[j] = Vec<T>::of(x0);
          y[j] = Vec<T>::of(x1);
        }
        T* z = dst(h);
        *reinterpret_cast<uint4*>(z + unit.at0) = x[j];
        *reinterpret_cast<uint4*>(z + unit.at1) = y[j];
      }
    }
  }
}

// The threads of a block: units x `lanes` heads x tokens. Measured with 1 / 2 / 4 /
// 8 lanes (heads of a token read by neighbouring threads): latent append of 16K
// tokens with 128 query heads 115 / 112 / 111 / 107 us (its queries are pieces of
// 128 bytes), grouped-head append of 14K tokens 51.6 / 52.2 / 53.6 / 63 us (pieces of
// 256 bytes, and each block has fewer tokens for its one look at the prefix sums).
constexpr int kAppendThreads = 128;
constexpr int kGqaLanes = 1, kLatentLanes = 8;

// ----------------------------------------------------- grouped-head cache ----
// Block (x, y): tokens, and heads [y * heads_per_cta, ..) of the list q heads, k
// heads, v heads.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) gqa_append_kernel(AppendParams p, int half_style) {
  __shared__ int32_t cu_shared[kCuShared + 1];
  // Every access waits for the grid before this one; only then may the next
  // grid's blocks be placed, so that what they read ahead of their own wait
  // (weights) is past whatever wrote it.
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  CuSearch cs{};
  if (p.cu) {
    cs = stage_cu(p.cu, p.B, cu_shared);
    __syncthreads();
  }
  const int units = p.d / 16;
  const int64_t t = (int64_t)blockIdx.x * (kAppendThreads / (units * kGqaLanes)) + threadIdx.x / (units * kGqaLanes);
  if (t >= p.T) return;
  Unit<T> unit(threadIdx.x % units, p.D, half_style != 0);
  const int nq = p.q ? p.Hq : 0, H = nq + 2 * p.Hk;
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(H, h0 + p.heads_per_cta), lane = threadIdx.x / units % kGqaLanes;
  Place at;
  walk_heads<T>(
      unit, h0 + lane, h1, kGqaLanes, nq + p.Hk,
      [&](int h) {
        return h < nq ? static_cast<const T*>(p.q) + t * p.q_ts + h * p.q_hs
             : h < nq + p.Hk ? static_cast<const T*>(p.k) + t * p.k_ts + (h - nq) * p.k_hs
                             : static_cast<const T*>(p.v) + t * p.v_ts + (h - nq - p.Hk) * p.v_hs;
      },
      [&]() {
        at = place_of(p, cs, cu_shared, t, unit.u == 0 && lane == 0 && blockIdx.y == 0);
        if (at.pos >= 0) unit.angles(p.table + at.pos * p.D, p.D);
        return at.pos >= 0;
      },
      [&](int h) {
        if (h < nq) return static_cast<T*>(p.q_out) + (t * p.Hq + h) * p.d;
        const bool is_k = h < nq + p.Hk;
        const int hk = h - nq - (is_k ? 0 : p.Hk);
        return static_cast<T*>(is_k ? p.k_pool : p.v_pool) + ((at.block * p.Hk + hk) * kPage + at.slot) * p.d;
      });
}

// ----------------------------------------------------------- latent cache ----
constexpr int kNarrowThreads = 256;

// One pair of the rotated part, element by element (any D, any alignment).
template <typename T>
__device__ __forceinline__ void turn_pair(const T* src, int i, int D, bool half, const float* row, float& xa, float& xb,
                                          int& ia, int& ib) {
  ia = half ? i : 2 * i;
  ib = half ? i + D / 2 : 2 * i + 1;
  const float a = to_float(src[ia]), b = to_float(src[ib]), c = row[i], s = row[D / 2 + i];
  xa = a * c - b * s;
  xb = b * c + a * s;
}

// Narrow path (bf16 and fp32 caches): one block per token, element by element.
template <typename T>
__global__ void __launch_bounds__(kNarrowThreads) latent_append_narrow_kernel(AppendParams p, int half_style) {
  __shared__ int32_t cu_shared[kCuShared + 1];
  // Every access waits for the grid before this one; only then may the next
  // grid's blocks be placed, so that what they read ahead of their own wait
  // (weights) is past whatever wrote it.
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  CuSearch cs{};
  if (p.cu) {
    cs = stage_cu(p.cu, p.B, cu_shared);
    __syncthreads();
  }
  const int64_t t = blockIdx.x;
  const Place at = place_of(p, cs, cu_shared, t, threadIdx.x == 0);
  if (at.pos < 0) return;
  const float* row = p.table + at.pos * p.D;
  const int width = p.r + p.D;
  const T* c = static_cast<const T*>(p.k) + t * p.k_ts;
  const T* kr = static_cast<const T*>(p.v) + t * p.v_ts;
  T* dst = static_cast<T*>(p.k_pool) + (at.block * kPage + at.slot) * (int64_t)width;
  T* rows = p.kv_rows ? static_cast<T*>(p.kv_rows) + t * width : nullptr;
  for (int i = threadIdx.x; i < p.r; i += kNarrowThreads) {
    dst[i] = c[i];
    if (rows) rows[i] = c[i];
  }
  float xa, xb;
  int ia, ib;
  for (int i = threadIdx.x; i < p.D / 2; i += kNarrowThreads) {
    turn_pair(kr, i, p.D, half_style != 0, row, xa, xb, ia, ib);
    dst[p.r + ia] = from_float<T>(xa);
    dst[p.r + ib] = from_float<T>(xb);
    if (rows) {
      rows[p.r + ia] = from_float<T>(xa);
      rows[p.r + ib] = from_float<T>(xb);
    }
  }
  if (!p.q) return;
  for (int e = threadIdx.x; e < p.Hq * (p.D / 2); e += kNarrowThreads) {
    const int h = e / (p.D / 2), i = e % (p.D / 2);
    turn_pair(static_cast<const T*>(p.q) + t * p.q_ts + h * p.q_hs, i, p.D, half_style != 0, row, xa, xb, ia, ib);
    T* qo = static_cast<T*>(p.q_out) + (t * p.Hq + h) * (int64_t)p.D;
    qo[ia] = from_float<T>(xa);
    qo[ib] = from_float<T>(xb);
  }
}

// Wide path. The first blocks write the latent rows, a warp per token; the
// others turn the query heads as the grouped-head append does.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(AppendParams p, int half_style) {
  using VT = Vec<T>;
  constexpr int V = VT::n;
  __shared__ int32_t cu_shared[kCuShared + 1];
  // Every access waits for the grid before this one; only then may the next
  // grid's blocks be placed, so that what they read ahead of their own wait
  // (weights) is past whatever wrote it.
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  CuSearch cs{};
  if (p.cu) {
    cs = stage_cu(p.cu, p.B, cu_shared);
    __syncthreads();
  }
  const int64_t row_blocks = (p.T + 3) / 4;
  if (blockIdx.x >= row_blocks) {
    const int units = p.D / (2 * V), tokens = kAppendThreads / (units * kLatentLanes);
    const int64_t token_blocks = (p.T + tokens - 1) / tokens, i = blockIdx.x - row_blocks;
    const int64_t t = i % token_blocks * tokens + threadIdx.x / (units * kLatentLanes);
    if (t >= p.T || (int)threadIdx.x >= tokens * units * kLatentLanes) return;
    Unit<T> unit(threadIdx.x % units, p.D, half_style != 0);
    const int h0 = (int)(i / token_blocks) * p.heads_per_cta, h1 = min(p.Hq, h0 + p.heads_per_cta);
    walk_heads<T>(
        unit, h0 + (int)threadIdx.x / units % kLatentLanes, h1, kLatentLanes, h1, [&](int h) { return static_cast<const T*>(p.q) + t * p.q_ts + h * p.q_hs; },
        [&]() {
          const Place at = place_of(p, cs, cu_shared, t, false);   // told by the latent row's warp
          if (at.pos >= 0) unit.angles(p.table + at.pos * p.D, p.D);
          return at.pos >= 0;
        },
        [&](int h) { return static_cast<T*>(p.q_out) + (t * p.Hq + h) * (int64_t)p.D; });
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int width = p.r + p.D, lane = threadIdx.x & 31;
  const T* c = static_cast<const T*>(p.k) + t * p.k_ts;
  const T* kr = static_cast<const T*>(p.v) + t * p.v_ts;
  // the latent: up to 512 elements, 16 per lane (FP8: 16 neighbours; else every 32nd vector)
  constexpr int N = 16 / V;
  uint4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = kFp8 ? 16 * lane + V * i : V * (lane + 32 * i);
    v[i] = e < p.r ? *reinterpret_cast<const uint4*>(c + e) : make_uint4(0, 0, 0, 0);
  }
  const Place at = place_of(p, cs, cu_shared, t, lane == 0);
  if (at.pos < 0) return;
  const float* row = p.table + at.pos * p.D;
  const int64_t cell = at.block * kPage + at.slot;
  T* rows = p.kv_rows ? static_cast<T*>(p.kv_rows) + t * width : nullptr;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = kFp8 ? 16 * lane + V * i : V * (lane + 32 * i);
    if (e >= p.r) continue;
    if (rows) *reinterpret_cast<uint4*>(rows + e) = v[i];
    if constexpr (!kFp8) *reinterpret_cast<uint4*>(static_cast<T*>(p.k_pool) + cell * width + e) = v[i];
  }
  float scale = 1.f;
  if constexpr (kFp8) {
    float x[16], top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) VT::to(v[i], *reinterpret_cast<float(*)[V]>(x + V * i));
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // correctly rounded divisions: the scale and the codes are those of the
    // definition, bit for bit. The floor keeps s a normal number and
    // k_rope / s inside bf16's range for a latent row of zeros.
    scale = fmaxf(__fdiv_rn(top, 448.f), 5.421010862427522e-20f);   // 2^-64
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = ptx::cvt_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
             ptx::cvt_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16;
    if (16 * lane < p.r)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_pool) + cell * p.r + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane == 0) p.kv_scale[cell] = scale;
  }
  for (int u = lane; u < p.D / (2 * V); u += 32) {
    Unit<T> unit(u, p.D, half_style != 0);
    unit.angles(row, p.D);
    float x0[V], x1[V];
    VT::to(*reinterpret_cast<const uint4*>(kr + unit.at0), x0);
    VT::to(*reinterpret_cast<const uint4*>(kr + unit.at1), x1);
    unit.rotate(x0, x1);
    if (rows) {
      *reinterpret_cast<uint4*>(rows + p.r + unit.at0) = VT::of(x0);
      *reinterpret_cast<uint4*>(rows + p.r + unit.at1) = VT::of(x1);
    }
    T* dst;
    if constexpr (kFp8) {
      dst = static_cast<T*>(p.v_pool) + cell * p.D;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x0[i] = __fdiv_rn(x0[i], scale);
        x1[i] = __fdiv_rn(x1[i], scale);
      }
    } else {
      dst = static_cast<T*>(p.k_pool) + cell * width + p.r;
    }
    *reinterpret_cast<uint4*>(dst + unit.at0) = VT::of(x0);
    *reinterpret_cast<uint4*>(dst + unit.at1) = VT::of(x1);
  }
}

}  // namespace pg
}  // namespace mla
