// Decode attention over the paged grouped-head cache, split over the cache's
// length and joined.
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . k_j
//
// An item is a (sequence, key head): its G Lq query rows read every key and
// value of the item once, 2 L d values for 4 G Lq L d operations, so the kernel
// is bound by the cache's bytes up to the 64 rows it takes. The pages of all
// items lie on one line (sequence by sequence, head by head), each item behind
// kItemCost empty places that stand for what a segment costs beside its pages.
// The line is cut into W equal ranges, one per worker (a block; two share an
// SM). A range is walked page by page with one pass of a running maximum and
// sum. An item that lies inside one range is finished there; of the others each
// range writes its part's maximum, sum and accumulator in fp32, and a second
// kernel joins the parts of an item in page order.
//
// A worker is a producer warp, which copies pages by TMA into a ring of key and
// value slots, and four consumer warps on mma.sync (m16n8k16): with at most 64
// rows of a page the product is far below what a tcgen05 tile (128 rows) would
// hold, and the fragments stay in registers from the scores to the weighted
// sum. MT = 1, 2 or 4 tiles of 16 rows. With 2 tiles two warps share a tile and
// take half the keys of each page, with their own running maximum and sum, joined
// when the segment ends. With 1 tile there are two layouts (key_parts): four such
// warps, or two pairs, each with half of the output columns (both compute the same
// scores, 16 more products a page, and the join moves a quarter of what four key
// parts would).
//
// Measured on one B200 (graph replay): 16 x 8192 tokens, 32 heads of their own,
// 2147.7 MB in 328 to 331 us (6.5 TB/s; the copy rate is 6.55); 1 x 131071 tokens,
// 64 / 4 heads, 53 to 55 us (4.9 to 5.1 TB/s); 64 x 500, 32 / 8 heads, 30 us (4.4 TB/s);
// one page 3.9 us. A segment's fixed part (queries, joining the warps, storing, the
// latency of one page) is thousands of cycles. At 256 x 64 tokens a warp that does
// not issue waits for loads (2.3 warps per issued instruction) or for fixed
// latencies (2.1), less for shared memory (0.7), barriers (0.6) and instructions
// (0.4); loading the next segment's queries early changed no case by more than 2%.
#pragma once

#include "paged_common.cuh"

namespace mla {
namespace pg {

constexpr int kDecodeThreads = 160;
// Loading an item's queries, joining the warps and storing takes a worker about
// as long as this many pages. Measured (graph replay, two runs of each in turn, with
// column halves where there are up to 16 rows) at 64
// sequences of 1 to 16384 tokens, 8 key heads (many items of one page): 90.5 us with
// 0, 56.7 with 2, 56.6 with 3, 56.1 with 4, 56.8 with 6; at 128 x 200 tokens 31.5, 30.6,
// 30.9, 31.1 and 31.3, at 32 x 4000 with 32 rows a key head 97.9, 97.2, 96.8, 97.4 and
// 98.3: from 2 to 4 it hardly matters. Only one short item is better off with 0 (1 x
// 500: 6.9 instead of 7.6).
constexpr int kItemCost = 4;

template <int kD> struct DecodeSmem {
  static constexpr uint32_t slot_bytes = kPage * kD * 2;           // one page's keys or values
  static constexpr int slots = kD == 128 ? 6 : 12;                 // keys and values alternate
  static constexpr uint32_t ring = 0;
  static constexpr uint32_t join = slots * slot_bytes;             // 16 rows x d of fp32
  static constexpr uint32_t ml = join + 16 * kD * 4;               // [4 warps][16 rows] maxima, then sums
  static constexpr uint32_t count = ml + 2 * 64 * 4;               // keys in each slot's page
  static constexpr uint32_t bars = count + 64;
  static constexpr uint32_t scan = bars + 16 * slots;              // int64 [5 + 3]
  static constexpr uint32_t alloc = scan + 64 + 1024;              // the ring starts on 1 KB
  static_assert(2 * (alloc + 1024) <= 228 * 1024, "two workers share an SM");
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// An item's places on the line.
__device__ __forceinline__ int64_t line_of(int32_t pages) { return pages ? pages + kItemCost : 0; }

// Walks a worker's range of the page line, segment by segment.
struct Segments {
  int64_t at, end;         // line positions: the next segment's start, the range's end
  int64_t item0;           // line position of the current item's first page (its empty places are before it)
  int32_t b, h, L, pages;  // the current item
  int32_t p0, p1;          // the segment's pages

  // b0, pos0: a sequence with pages and its first line position, at or before the range's start
  __device__ __forceinline__ bool init(const GqaParams& p, int64_t begin, int64_t end_, int32_t b0, int64_t pos0) {
    at = begin;
    end = end_;
    if (at >= end) return false;
    b = b0;
    for (;;) {
      L = checked_len(p, b, false);
      pages = pages_of(L);
      const int64_t line = line_of(pages) * p.Hk;
      if (at < pos0 + line) break;
      pos0 += line;
      if (++b >= p.B) return false;   // only where lengths change under the kernel
    }
    h = (int32_t)((at - pos0) / line_of(pages));
    item0 = pos0 + h * line_of(pages) + kItemCost;
    return cut();
  }
  __device__ __forceinline__ bool next(const GqaParams& p) {
    at = item0 + p1;
    if (at >= end) return false;
    item0 += line_of(pages);
    if (++h == p.Hk) {
      h = 0;
      do {
        if (++b >= p.B) return false;
        L = checked_len(p, b, false);
        pages = pages_of(L);
      } while (pages == 0);
    }
    // the empty places have the next item's width whatever its pages are
    return cut();
  }
  // a range that ends in an item's empty places has none of its pages
  __device__ __forceinline__ bool cut() {
    p0 = at > item0 ? (int32_t)(at - item0) : 0;
    const int64_t left = end - item0;
    if (left <= p0) return false;
    p1 = left < pages ? (int32_t)left : pages;
    return true;
  }
};

// kHalves: warps with the same rows and keys, each with its output columns
template <typename T, int kD, int MT, int kHalves>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, GqaParams p) {
  using namespace ptx;
  using S = DecodeSmem<kD>;
  using WS = WeightScale<T>;
  constexpr int kParts = 4 / (MT * kHalves);       // warps with the same rows and columns, each with its keys
  constexpr int kKeys = kPage / kParts;            // keys of a page per warp
  constexpr int NT = kKeys / 8;
  constexpr int kDW = kD / kHalves;                // output columns of a warp
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto full = [&](int s) -> uint32_t { return base + S::bars + 16u * s; };
  auto empty = [&](int s) -> uint32_t { return base + S::bars + 16u * s + 8u; };
  int32_t* count = reinterpret_cast<int32_t*>(gbase + S::count);
  int64_t* scan = reinterpret_cast<int64_t*>(gbase + S::scan);
  const int w = blockIdx.x, rows = p.G * p.Lq;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::slots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4 + p.withhold);
    }
    fence_mbarrier_init_cluster();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // Every access waits for the grid before this one; only then may the next
  // grid's blocks be placed, so that what they read ahead of their own wait
  // (weights) is past whatever wrote it.
  grid_dependency_wait();
  grid_launch_dependents();
  // ---- the page line: every thread sums the pages of a run of sequences, a scan gives the runs' places
  const int per = (p.B + kDecodeThreads - 1) / kDecodeThreads;
  const int b_lo = min(p.B, (int)threadIdx.x * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += line_of(pages_of(checked_len(p, b, w == 0))) * p.Hk;
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
  }
  // no more ranges than places on the line: none is empty
  const int64_t W = min((int64_t)p.W, total);
  const int64_t begin = w < W ? w * total / W : 0, end = w < W ? (w + 1) * total / W : 0;
  const int64_t run0 = before + upto - mine;
  if (begin < end && run0 <= begin && begin < run0 + mine) {   // one thread: the run that holds the range's start
    scan[5] = b_lo;
    scan[6] = run0;
  }
  __syncthreads();
  Segments seg;
  bool have = seg.init(p, begin, end, (int32_t)scan[5], scan[6]);
  bool ok = true;

  if (warp == 4) {
    // ------------------------------------------------------------ producer --
    uint32_t it = 0;
    for (; have && ok; have = seg.next(p)) {
      const int32_t* table = p.block_table + (int64_t)seg.b * p.bt_stride;
      int32_t ids = 0;
      for (int pg = seg.p0; pg < seg.p1 && ok; ++pg) {
        const int o = (pg - seg.p0) & 31;
        if (o == 0 && pg + lane < seg.p1) ids = table[pg + lane];
        const int32_t id = __shfl_sync(0xffffffffu, ids, o);
        const bool good = id >= 0 && (int64_t)id < p.num_blocks;
        if (lane == 0) {
          const int keys = good ? min(kPage, seg.L - pg * kPage) : 0;
          if (!good) record_error(p.status, MLA_ERR_BOUNDS);
          const int32_t z = good ? id * p.Hk + seg.h : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int s = it % S::slots;
            if (ok && it >= (uint32_t)S::slots) ok = mbar_wait(empty(s), ((it / S::slots) - 1) & 1, p.wait_limit_ns);
            if (!ok) break;
            count[s] = keys;
            if (!good) {
              mbar_arrive_local(full(s));
              continue;
            }
            const uint32_t dst = base + S::ring + s * S::slot_bytes;
            mbar_arrive_expect_tx_local(full(s), S::slot_bytes);
#pragma unroll
            for (int c = 0; c < kD; c += 64) tma_load_3d(dst + c * 128, kv ? &tm_v : &tm_k, c, 0, z, full(s));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    }
    if (!ok && lane == 0) {
      record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
      // copies still in flight land before the block ends
      for (uint32_t i = it > (uint32_t)S::slots ? it - S::slots : 0; i < it; ++i)
        (void)mbar_wait(full(i % S::slots), (i / S::slots) & 1, p.wait_limit_ns);
    }
  } else {
    // ----------------------------------------------------------- consumers --
    // idle slots: sequences without a token give zeros
    for (int b = w; b < p.B; b += p.W)
      if (checked_len(p, b, false) == 0) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (int64_t)b * p.Lq * p.Hq * kD);
        for (int i = threadIdx.x; i < p.Lq * p.Hq * (kD / 8); i += 128) o[i] = make_uint4(0, 0, 0, 0);
      }
    const int tile = warp % MT, part = warp / MT % kParts, half = warp / (MT * kParts);
    const int g = lane >> 2, t4 = lane & 3;
    const int row0 = 16 * tile + g, row1 = row0 + 8;
    const int key0 = part * kKeys;           // this warp's first key of a page
    // per row, from an item's first query: its elements' offset, and how many keys
    // less than the item's length its token sees (a row past `rows` stands for the
    // last token: finite, never stored)
    const bool real0 = row0 < rows, real1 = row1 < rows;
    const int last0 = real0 ? row0 : rows - 1, last1 = real1 ? row1 : rows - 1;
    const int off0 = (last0 / p.G * p.Hq + last0 % p.G) * kD + 2 * t4, off1 = (last1 / p.G * p.Hq + last1 % p.G) * kD + 2 * t4;
    const int less0 = p.Lq - 1 - last0 / p.G, less1 = p.Lq - 1 - last1 / p.G;
    float* sm = reinterpret_cast<float*>(gbase + S::ml);
    float* sl = sm + 64;
    float* join = reinterpret_cast<float*>(gbase + S::join);
    // shared-memory offsets of this lane's ldmatrix rows
    const uint32_t k_row = key0 + (lane & 7), k_chunk = lane >> 3;
    const uint32_t v_row = key0 + ((lane >> 3) & 1) * 8 + (lane & 7), v_chunk = half * (kDW / 8) + (lane >> 4);
    uint32_t it = 0;
    int2 tail = make_int2(-1, 0);
    for (; have; have = seg.next(p)) {
      uint32_t q[kD / 16][4];
      const int64_t item = ((int64_t)seg.b * p.Lq * p.Hq + seg.h * p.G) * kD;   // its first query's elements
      {
        const T* a = static_cast<const T*>(p.q) + item + off0;
        const T* c = static_cast<const T*>(p.q) + item + off1;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          q[k][0] = *reinterpret_cast<const uint32_t*>(a + 16 * k);
          q[k][1] = *reinterpret_cast<const uint32_t*>(c + 16 * k);
          q[k][2] = *reinterpret_cast<const uint32_t*>(a + 16 * k + 8);
          q[k][3] = *reinterpret_cast<const uint32_t*>(c + 16 * k + 8);
        }
      }
      const int lim0 = seg.L - less0, lim1 = seg.L - less1;     // keys that the rows see
      float o[kDW / 8][4];
#pragma unroll
      for (int n = 0; n < kDW / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

      for (int pg = seg.p0; pg < seg.p1; ++pg, it += 2) {
        const int ks = it % S::slots, vs = (it + 1) % S::slots;
        const uint32_t par_k = (it / S::slots) & 1, par_v = ((it + 1) / S::slots) & 1;
        if (ok) ok = mbar_wait(full(ks), par_k, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int keys = count[ks];
        const uint32_t kb = base + S::ring + ks * S::slot_bytes;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) {
          const uint32_t chunk = 4 * k + k_chunk;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t r = k_row + 8 * n;
            uint32_t f[4];
            ldsm4(f, kb + (chunk >> 3) * 8192 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
            mma16816<T>(s[n], q[2 * k], f[0], f[1]);
            mma16816<T>(s[n], q[2 * k + 1], f[2], f[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_local(empty(ks));
        const int j0 = pg * kPage + key0 + 2 * t4;
        if (keys < kPage || pg * kPage + kPage > seg.L - p.Lq + 1) {
          const int past = pg * kPage + keys;   // slots past the page's tokens hold anything
          const int e0 = min(lim0, past), e1 = min(lim1, past);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int j = j0 + 8 * n;
            if (j >= e0) s[n][0] = -INFINITY;
            if (j + 1 >= e0) s[n][1] = -INFINITY;
            if (j >= e1) s[n][2] = -INFINITY;
            if (j + 1 >= e1) s[n][3] = -INFINITY;
          }
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          t0 = fmaxf(t0, fmaxf(s[n][0], s[n][1]));
          t1 = fmaxf(t1, fmaxf(s[n][2], s[n][3]));
        }
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2)) * p.scale_log2;
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2)) * p.scale_log2;
        // the maximum moves when it has to by more than `lazy` (and at a row's first visible key)
        if (__any_sync(0xffffffffu, t0 > m0 + WS::lazy || t1 > m1 + WS::lazy)) {
          const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
          const float a0 = n0 == m0 ? 1.f : ex2_approx(m0 - n0), a1 = n1 == m1 ? 1.f : ex2_approx(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int n = 0; n < kDW / 8; ++n) {
            o[n][0] *= a0;
            o[n][1] *= a0;
            o[n][2] *= a1;
            o[n][3] *= a1;
          }
        }
        const float d0 = m0 == -INFINITY ? 0.f : WS::bias - m0, d1 = m1 == -INFINITY ? 0.f : WS::bias - m1;
        uint32_t a[NT / 2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float x0 = ex2_approx(fmaf(s[n][0], p.scale_log2, d0)), x1 = ex2_approx(fmaf(s[n][1], p.scale_log2, d0));
          const float y0 = ex2_approx(fmaf(s[n][2], p.scale_log2, d1)), y1 = ex2_approx(fmaf(s[n][3], p.scale_log2, d1));
          l0 += x0 + x1;
          l1 += y0 + y1;
          a[n >> 1][2 * (n & 1)] = Pack<T>::of(x0, x1);
          a[n >> 1][2 * (n & 1) + 1] = Pack<T>::of(y0, y1);
        }
        ok = mbar_wait(full(vs), par_v, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t vb = base + S::ring + vs * S::slot_bytes;
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
          const uint32_t r = v_row + 16 * k;
          // values of slots past the page's tokens: their weight is 0, but 0 times NaN is not
          const int k0 = key0 + 16 * k + 2 * t4;
          uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
          if (keys < kPage) {
            z0 = (k0 < keys ? 0x0000ffffu : 0u) | (k0 + 1 < keys ? 0xffff0000u : 0u);
            z1 = (k0 + 8 < keys ? 0x0000ffffu : 0u) | (k0 + 9 < keys ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int n = 0; n < kDW / 16; ++n) {
            const uint32_t chunk = 2 * n + v_chunk;
            uint32_t f[4];
            ldsm4_t(f, vb + (chunk >> 3) * 8192 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
            mma16816<T>(o[2 * n], a[k], f[0] & z0, f[1] & z1);
            mma16816<T>(o[2 * n + 1], a[k], f[2] & z0, f[3] & z1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_local(empty(vs));
      }

      // ---- the segment's end: sums over the row's lanes, then over the warps of a tile
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if constexpr (kParts > 1) {
        if (t4 == 0) {
          sm[16 * warp + g] = m0;
          sm[16 * warp + g + 8] = m1;
          sl[16 * warp + g] = l0;
          sl[16 * warp + g + 8] = l1;
        }
        named_barrier(1, 128);
        float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          n0 = fmaxf(n0, sm[16 * ((half * kParts + i) * MT + tile) + g]);
          n1 = fmaxf(n1, sm[16 * ((half * kParts + i) * MT + tile) + g + 8]);
        }
        const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0), a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
        l0 = l1 = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int x = 16 * ((half * kParts + i) * MT + tile) + g;
          if (sm[x] != -INFINITY) l0 += sl[x] * ex2_approx(sm[x] - n0);
          if (sm[x + 8] != -INFINITY) l1 += sl[x + 8] * ex2_approx(sm[x + 8] - n1);
        }
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int n = 0; n < kDW / 8; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
        // part i hands its accumulators to part 0 through 16 x d floats, MT
        // tiles with d / MT columns at a time
#pragma unroll
        for (int c = 0; c < MT; ++c) {
#pragma unroll
          for (int i = 1; i < kParts; ++i) {
            named_barrier(1, 128);
            float* buf = join + (half * MT + tile) * (16 * kDW / MT) + lane * 4;
            if (part == i) {
#pragma unroll
              for (int n = 0; n < kDW / 8 / MT; ++n)
                *reinterpret_cast<float4*>(buf + 128 * n) = make_float4(o[c * (kDW / 8 / MT) + n][0], o[c * (kDW / 8 / MT) + n][1],
                                                                        o[c * (kDW / 8 / MT) + n][2], o[c * (kDW / 8 / MT) + n][3]);
            }
            named_barrier(1, 128);
            if (part == 0) {
#pragma unroll
              for (int n = 0; n < kDW / 8 / MT; ++n) {
                const float4 x = *reinterpret_cast<const float4*>(buf + 128 * n);
                float(&y)[4] = o[c * (kDW / 8 / MT) + n];
                y[0] += x.x;
                y[1] += x.y;
                y[2] += x.z;
                y[3] += x.w;
              }
            }
          }
        }
      }
      // an item's first segment that does not finish it: the worker's last; any
      // other part of a split item: the worker's first
      const bool first = seg.p0 == 0, whole = first && seg.p1 == seg.pages;
      if (part == 0) {
        if (whole) {
          const float i0 = l0 > 0.f ? 1.f / l0 : 0.f, i1 = l1 > 0.f ? 1.f / l1 : 0.f;
          T* d0 = static_cast<T*>(p.out) + item + off0 + half * kDW;
          T* d1 = static_cast<T*>(p.out) + item + off1 + half * kDW;
#pragma unroll
          for (int n = 0; n < kDW / 8; ++n) {
            if (real0) *reinterpret_cast<uint32_t*>(d0 + 8 * n) = Pack<T>::of(o[n][0] * i0, o[n][1] * i0);
            if (real1) *reinterpret_cast<uint32_t*>(d1 + 8 * n) = Pack<T>::of(o[n][2] * i1, o[n][3] * i1);
          }
        } else {
          const int64_t slot = (2 * (int64_t)w + (first ? 1 : 0)) * rows;
          if (real0) {
            float* d = p.o_part + (slot + row0) * kD + half * kDW + 2 * t4;
#pragma unroll
            for (int n = 0; n < kDW / 8; ++n) *reinterpret_cast<float2*>(d + 8 * n) = make_float2(o[n][0], o[n][1]);
            if (t4 == 0 && half == 0) p.ml_part[slot + row0] = make_float2(m0, l0);
          }
          if (real1) {
            float* d = p.o_part + (slot + row1) * kD + half * kDW + 2 * t4;
#pragma unroll
            for (int n = 0; n < kDW / 8; ++n) *reinterpret_cast<float2*>(d + 8 * n) = make_float2(o[n][2], o[n][3]);
            if (t4 == 0 && half == 0) p.ml_part[slot + row1] = make_float2(m1, l1);
          }
        }
      }
      // the item this worker begins and others finish, and the last of them: the
      // last worker whose range starts before the item's end
      if (first && !whole) tail = make_int2(seg.b * p.Hk + seg.h, (int)(((seg.item0 + seg.pages) * W - 1) / total));
      if constexpr (kParts > 1) named_barrier(1, 128);   // the join's buffers are free again
    }
    if (threadIdx.x == 0) p.tails[w] = tail;
    if (!ok && lane == 0) record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
  }
}

// Adds one part of an item (its maximum, sum and accumulator) to another.
template <int E>
__device__ __forceinline__ void add_part(float& m, float& l, float (&o)[E], float m1, float l1, const float (&x)[E]) {
  if (m1 == -INFINITY) return;
  const float n = fmaxf(m, m1), a = m == -INFINITY ? 0.f : exp2f(m - n), c = exp2f(m1 - n);
  m = n;
  l = l * a + l1 * c;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = o[e] * a + x[e] * c;
}

// Joins the parts of the items that workers left unfinished. Block (x, y): the
// items that workers x `group` to (x + 1) `group` - 1 began, rows y `per` to
// (y + 1) `per` - 1, 8 / per warps to a row.
constexpr int kJoinThreads = 256;

template <typename T, int kD, int kAhead>
__global__ void __launch_bounds__(kJoinThreads) gqa_join_kernel(GqaParams p, int group, int per) {
  constexpr int E = kD / 32;                 // kAhead: parts whose loads are in flight
  __shared__ float so[8][kD];
  __shared__ float sm[8], sl[8];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.G * p.Lq, share = 8 / per;
  const int row = blockIdx.y * per + warp / share, first = warp % share;
  const int w_end = min(p.W - 1, (int)(blockIdx.x + 1) * group);
  for (int w0 = blockIdx.x * group; w0 < w_end; w0 += 32) {
    // What the workers left lies in the workspace: where two calls share one by
    // mistake it may be another call's, and none is followed out of this call's
    // items and workers. (Warps that then see different items leave at different
    // times; a barrier waits for those that are left.)
    int2 mine = w0 + lane < w_end ? p.tails[w0 + lane] : make_int2(-1, 0);
    if (mine.x >= p.B * p.Hk || mine.y >= p.W) {
      record_error(p.status, MLA_ERR_BOUNDS);
      mine.x = -1;
    }
    uint32_t open = __ballot_sync(0xffffffffu, mine.x >= 0);
    for (; open; open &= open - 1) {          // the same for every warp
      const int i0 = __ffs(open) - 1, w = w0 + i0;
      const int item = __shfl_sync(0xffffffffu, mine.x, i0), parts = __shfl_sync(0xffffffffu, mine.y, i0) - w + 1;
      float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
      if (row < rows) {
        auto slot = [&](int i) { return (2 * (int64_t)(w + i) + (i == 0 ? 1 : 0)) * rows + row; };
        for (int i1 = first; i1 < parts; i1 += kAhead * share) {
          float2 ml[kAhead];
          float x[kAhead][E];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int i = i1 + u * share;
            ml[u] = i < parts ? p.ml_part[slot(i)] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) x[u][e] = i < parts ? p.o_part[slot(i) * kD + lane + 32 * e] : 0.f;
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) add_part(m, l, o, ml[u].x, ml[u].y, x[u]);
        }
      }
      if (share > 1) {
        __syncthreads();                      // the last item's sums have been read
        if (lane == 0) {
          sm[warp] = m;
          sl[warp] = l;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
        __syncthreads();
        if (first == 0)
          for (int i = warp + 1; i < warp + share; ++i) {
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = so[i][lane + 32 * e];
            add_part(m, l, o, sm[i], sl[i], x);
          }
      }
      if (row < rows && first == 0) {
        const int b = item / p.Hk, h = item % p.Hk;
        T* d = static_cast<T*>(p.out) + (((int64_t)b * p.Lq + row / p.G) * p.Hq + h * p.G + row % p.G) * kD + lane;
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) d[32 * e] = (T)(o[e] * inv);
      }
    }
  }
}

// ------------------------------------------------------------------ host ---
template <typename T, int kD, int MT, int kHalves>
cudaError_t launch_decode_tiles(const GqaParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
  using S = DecodeSmem<kD>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(gqa_decode_kernel<T, kD, MT, kHalves>), (int)S::alloc);
  if (e != cudaSuccess) return e;
  return launch_dependent(gqa_decode_kernel<T, kD, MT, kHalves>, dim3(p.W), dim3(kDecodeThreads), S::alloc, stream, tm_k, tm_v, p);
}

template <typename T, int kD>
cudaError_t launch_decode(const GqaParams& p, int64_t items, cudaStream_t stream) {
  CUtensorMap tm_k, tm_v;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  if (!pool_map(&tm_k, p.k_pool, p.num_blocks * p.Hk, kD, bf16) || !pool_map(&tm_v, p.v_pool, p.num_blocks * p.Hk, kD, bf16))
    return cudaErrorInvalidValue;
  const int rows = p.G * p.Lq;
  cudaError_t e = rows > 32   ? launch_decode_tiles<T, kD, 4, 1>(p, tm_k, tm_v, stream)
                : rows > 16   ? launch_decode_tiles<T, kD, 2, 1>(p, tm_k, tm_v, stream)
                : p.key_parts ? launch_decode_tiles<T, kD, 1, 1>(p, tm_k, tm_v, stream)
                              : launch_decode_tiles<T, kD, 1, 2>(p, tm_k, tm_v, stream);
  if (e != cudaSuccess || p.W == 1) return e;
  // Where workers outnumber items, about every W / items-th begins one, of about
  // as many parts. A block looks through that many workers; a row has one, four or
  // eight warps, and a warp as many loads in flight as it has parts, up to 8.
  // Measured at 22 shapes with 1, 2, 4 and 8 warps to a row and 4 or 8 loads; the
  // borders' sides, us: 5 parts (8 x 2000, 8 key heads, 32 rows) one warp with 4 / 8
  // loads 23.0 / 21.6, four warps 24.8 / 29.3; 8 parts (1 x 500, 8 key heads) one warp
  // 7.6 / 7.3, four 7.6 / 7.8; 10 parts (4 x 8000, 8 key heads) one warp 30.1 / 29.8, four
  // 29.5 / 29.2, with 32 rows 34.8 / 33.4 and 32.5 / 34.7; 25 parts (3 x 9000, 4 key heads, 16
  // rows) four 19.3 / 18.0, eight 18.3 / 17.9; 37 parts (8 x 4000, one key head, 32 rows)
  // four 14.5 / 13.5, eight 13.1 / 12.4; 100 parts (1 x 20000, one key head) four 14.3 / 14.1,
  // eight 12.6 / 12.3. (From 70 parts on, blocks that look through a quarter of the
  // workers would gain up to 8%: 1 x 100000, one key head, 25.4 / 23.3.) Joining in the
  // decode kernel, by the worker that comes last, was slower: 9.3 us against 8.3 at
  // 1 x 500, 35 against 30 at 64 x 500 (with the first form of this kernel).
  const int group = (int)std::max<int64_t>(1, p.W / items), parts = (int)ceil_div64(p.W, items);
  const int per = parts <= 8 ? 8 : parts <= 32 ? 2 : 1;
  const dim3 grid((unsigned)((p.W - 1 + group - 1) / group), (unsigned)((rows + per - 1) / per));
  return parts * per <= 4 * 8 ? launch_dependent(gqa_join_kernel<T, kD, 4>, grid, dim3(kJoinThreads), 0, stream, p, group, per)
                              : launch_dependent(gqa_join_kernel<T, kD, 8>, grid, dim3(kJoinThreads), 0, stream, p, group, per);
}

}  // namespace pg
}  // namespace mla
