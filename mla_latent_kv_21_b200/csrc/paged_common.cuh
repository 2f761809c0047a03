// Shared definitions of the paged-cache operators (include/mla_paged.h): types
// and conversions, the lookup of a packed token's sequence, tensor maps.
#pragma once

#include "../../include/mla_paged.h"
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace pg {

constexpr int kPage = 64;   // tokens per cache block

template <typename T> struct Pack;   // two values of a 16-bit type in 32 bits
template <> struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t of(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 to(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <> struct Pack<__half> {
  static __device__ __forceinline__ uint32_t of(float lo, float hi) { return ptx::cvt_f16x2(lo, hi); }
  static __device__ __forceinline__ float2 to(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
};

// ------------------------------------------------------------ parameters -----
}  // namespace pg

struct GqaParams {
  const void* q;           // [T, Hq, d]
  const void* k_pool;      // [num_blocks, Hk, 64, d]
  const void* v_pool;
  void* out;               // [T, Hq, d]
  int32_t* status;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu;       // prefill
  float* o_part;           // decode workspace: partial sums of split items
  float2* ml_part;         // their running maxima and sums
  int2* tails;             // per worker, the item it began and did not finish
  int64_t num_blocks, T;
  int32_t bt_stride, B, Lq, Hq, Hk, G, W;
  int32_t key_parts;       // decode, up to 16 rows: four key parts, no column halves
  int32_t max_new;         // prefill: largest count of the plan
  int2* order;             // prefill workspace: (sequence, pair of tiles), longest first; NULL: one item per block
  int32_t* order_state;    // workspace header: {items drawn, items}
  int32_t order_room;
  float scale_log2;
  uint64_t wait_limit_ns;
  int32_t withhold;        // self-test of the timeout path only: barriers that one arrival too few completes
};

namespace pg {

// The sequence b with cu[b] <= t < cu[b + 1] of a packed token t, or -1 for a
// row that belongs to none. The prefix sums (or every `step`-th of them, where
// there are more than kCuShared) are in shared memory: a search over global
// memory would cost a dependent L2 round trip per halving.
constexpr int kCuShared = 1024;
struct CuSearch {
  const int32_t* cu;       // global, [B + 1]
  int32_t B, step, n;      // n samples cu[0], cu[step], ..
};
__device__ __forceinline__ CuSearch stage_cu(const int32_t* cu, int32_t B, int32_t* shared) {
  CuSearch s{cu, B, B / kCuShared + 1, 0};
  s.n = B / s.step + 1;
  for (int i = threadIdx.x; i < s.n; i += blockDim.x) shared[i] = cu[i * s.step];
  return s;   // the caller synchronises the block
}
__device__ __forceinline__ int32_t sequence_of(const CuSearch& s, const int32_t* shared, int32_t t) {
  int lo = 0, hi = s.n - 1;   // the last sample <= t
  if (shared[0] > t) return -1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (shared[mid] <= t) lo = mid; else hi = mid - 1;
  }
  if (s.step == 1) return lo < s.B ? lo : -1;
  int a = lo * s.step, e = min(a + s.step - 1, s.B);
  while (a < e) {
    const int mid = (a + e + 1) >> 1;
    if (s.cu[mid] <= t) a = mid; else e = mid - 1;
  }
  return a < s.B ? a : -1;
}

// Softmax weights are rounded once, to the 16-bit type: the tensor core takes both
// operands of the second product in it, and a second term for the residual would
// double that product. Their sum is of the unrounded weights, in fp32, so an output
// is off by at most half a step times sum_j p_j |v_j| from that (with random keys
// 2.2e-3 of the output's norm in bf16 and 2.5e-4 in fp16, where rounding the output
// alone gives 1.7e-3 and 2.1e-4). ex2.approx adds 2^-22.
// fp16 softmax weights: 2^-14 is the smallest normal value, so the weights of the
// largest score are 2^8 instead of 1 and the maximum moves after 2^6; weights
// then stay below 2^14 and are normal numbers down to 2^-22 of the largest.
// bf16 has fp32's range: the maximum moves after 2^8.
template <typename T> struct WeightScale { static constexpr float bias = 0.f, lazy = 8.f; };
template <> struct WeightScale<__half> { static constexpr float bias = 8.f, lazy = 6.f; };

// The tokens of sequence b; a length out of range counts as 0 (`tell`: record
// it). Lengths stay so far below 2^31 that a step past them is still an int32.
constexpr int32_t kMaxLen = 0x7ffff000;
__device__ __forceinline__ int32_t checked_len(const GqaParams& p, int32_t b, bool tell) {
  const int32_t L = p.seq_lens[b];
  if (L >= 0 && L <= kMaxLen && (int64_t)L <= (int64_t)p.bt_stride * kPage) return L;
  if (tell) record_error(p.status, MLA_ERR_BOUNDS);
  return 0;
}
__device__ __forceinline__ int32_t pages_of(int32_t L) { return (L + kPage - 1) / kPage; }

// ------------------------------------------------------------ tensor maps ----
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A pool [num_blocks * Hk, 64, d] of a 16-bit type as (d, 64, pages): boxes of
// 64 columns of one page, rows of 128 bytes in the 128-byte swizzle.
inline bool pool_map(CUtensorMap* m, const void* pool, int64_t pages, int d, bool bf16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, kPage, (cuuint64_t)pages};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * kPage};
  const cuuint32_t box[3] = {64, kPage, 1}, es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(pool),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pg
}  // namespace mla
