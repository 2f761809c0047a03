// Causal attention of packed prompts over the paged grouped-head cache on
// tcgen05 tensor cores.
//
//   out[t,h] = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q[t,h] . k_j,  j <= pos(t)
//
// The G query heads of a key head read the same keys, so a tile of 128 rows is
// 128 / G tokens x G heads (row = token G + head, as a TMA box of the packed
// queries lays it down; the rows left over where G does not divide 128 are
// zero). A block takes two such tiles of one sequence and key head and streams
// the keys and values of 128 tokens (two pages) at a time: each byte that
// reaches shared memory serves 256 rows. Per tile and step,
//   S = Q K^T   (M 128, N 128, K d)   into the tile's 128 columns of tensor memory,
//   P           (16-bit pairs)        over the first half of those columns,
//   O += P V    (M 128, N d, K 128, A from tensor memory).
// Warps: 0 producer, 1 MMA issuer, 4-7 and 8-11 the softmax of tile 0 and 1 (a
// row per thread, running maximum and sum in fp32). The two tiles alternate:
// while one tile's weights are computed, the tensor core works for the other.
// The MMAs of a tile run in the order S(0), O(0), S(1), O(1), ..; one thread
// issues them, so S(j + 1) may overwrite the P(j) that O(j) has read, and a
// full S(j + 1) means that O(j) is complete.
#pragma once

#include "paged_common.cuh"

namespace mla {
namespace pg {

constexpr int kPrefillThreads = 384;
constexpr int kTile = 128;               // rows of a tile, keys of a step
constexpr int kEarlyKeys = 64;           // keys whose weights are handed over early

template <int kD> struct PrefillSmem {
  static constexpr uint32_t tile_bytes = kTile * kD * 2;         // a query tile; a step's keys or values
  static constexpr int slots = kD == 128 ? 5 : 8;                // keys and values alternate
  static constexpr uint32_t q = 0;
  static constexpr uint32_t ring = 2 * tile_bytes;
  static constexpr uint32_t bars = ring + slots * tile_bytes;
  static constexpr uint32_t misc = bars + 256;
  static constexpr uint32_t alloc = misc + 64 + 1024;            // the tiles start on 1 KB
  static_assert(alloc <= 227 * 1024, "shared memory of one block");
};

// kind::f16 with fp32 accumulation for either 16-bit type (bf16 = 1, f16 = 0 in
// both operand formats).
template <typename T> constexpr uint32_t idesc16(int M, int N, int a_mn, int b_mn) {
  const uint32_t d = ptx::idesc_bf16_f32(M, N, a_mn, b_mn);
  return std::is_same<T, __half>::value ? d & ~((1u << 7) | (1u << 10)) : d;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A from tensor memory: two 16-bit values per column, B by descriptor.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Two fp32 lanes per instruction, each rounded as the scalar one.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max_three(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <typename T, int kD>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, GqaParams p, int32_t steps) {
  using namespace ptx;
  using S = PrefillSmem<kD>;
  using WS = WeightScale<T>;
  constexpr int kSlots = S::slots;
  extern __shared__ uint8_t smem_raw[];
  // ---- this block's tokens: the last ones of every sequence first (they see most keys)
  const int bh = blockIdx.x % (p.B * p.Hk), b = bh / p.Hk, hk = bh % p.Hk;
  const int32_t pair = steps - 1 - (int32_t)(blockIdx.x / (p.B * p.Hk));
  const int tokens = kTile / p.G;                                   // of one tile
  // the next grid's blocks may be placed once all of this one's are; each waits
  // for the grid before it ahead of its first access
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t c0 = p.cu[b], c1 = p.cu[b + 1], n = c1 - c0;
  const int64_t t0 = (int64_t)pair * 2 * tokens;                    // first token of the block, in its sequence
  if (c0 < 0 || n < 0 || c1 > p.T || n > p.max_new) {
    if (threadIdx.x == 0 && pair == 0) record_error(p.status, MLA_ERR_BOUNDS);
    return;
  }
  if (t0 >= n) return;
  const int32_t L = checked_len(p, b, threadIdx.x == 0);
  // tile i sees the keys up to its last token's position: nk[i] steps
  const int64_t ahead = (int64_t)L - n;                             // position of token t: ahead + t
  const bool two_tiles = t0 + tokens < n;
  auto steps_of = [&](int i) {
    const int64_t last = ahead + min(t0 + (int64_t)(i + 1) * tokens, n) - 1;
    return last < 0 ? 0 : (int)(last / kTile) + 1;
  };
  const int nk0 = steps_of(0), nk1 = two_tiles ? steps_of(1) : 0, nk = max(nk0, nk1);
  const int pages = min(pages_of(L), 2 * nk);
  const int32_t* table = p.block_table + (int64_t)b * p.bt_stride;

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto full = [&](int s) -> uint32_t { return base + S::bars + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return base + S::bars + 8u * (kSlots + s); };
  auto q_full = [&](int i) -> uint32_t { return base + S::bars + 8u * (2 * kSlots + i); };
  auto s_full = [&](int i) -> uint32_t { return base + S::bars + 8u * (2 * kSlots + 2 + i); };
  auto p_full = [&](int i) -> uint32_t { return base + S::bars + 8u * (2 * kSlots + 4 + i); };
  auto o_full = [&](int i) -> uint32_t { return base + S::bars + 8u * (2 * kSlots + 6 + i); };
  auto p_part = [&](int i) -> uint32_t { return base + S::bars + 8u * (2 * kSlots + 8 + i); };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(gbase + S::misc);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * kSlots; ++s) mbar_init(full(s), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_part(i), 4);    // the four softmax warps of the tile
      mbar_init(p_full(i), 4);
      mbar_init(o_full(i), 1);
    }
    fence_mbarrier_init_cluster();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc<1>(base + S::misc, 512);
    tmem_relinquish<1>();
  }
  // rows of the query tiles that no token fills
  const int used = tokens * p.G;
  for (int i = threadIdx.x; i < 2 * (kTile - used) * (kD / 8); i += kPrefillThreads) {
    const int r = i / (kD / 8), c = i % (kD / 8), tile = r / (kTile - used), row = used + r % (kTile - used);
    *reinterpret_cast<uint4*>(gbase + S::q + tile * S::tile_bytes + (c >> 3) * (kTile * 128) + row * 128 + (c & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  // pages whose block is out of range: their keys are not seen
  bool bad = false;
  for (int i = threadIdx.x; i < pages; i += kPrefillThreads) {
    const int32_t id = table[i];
    bad |= id < 0 || (int64_t)id >= p.num_blocks;
  }
  tc_fence_before();
  const bool any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tbase = *tslot;
  constexpr uint32_t kTmemO = 256;       // S (and P) of tile i: columns [128 i, +128); O: [256 + d i, +d)
  bool ok = true;
  // 384 x 168 registers at launch: 128 x 72 + 256 x 216

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    const int32_t q0 = (int32_t)(c0 + t0);
    if (lane == 0 && nk > 0) {
      for (int i = 0; i < (two_tiles ? 2 : 1); ++i) {
        mbar_arrive_expect_tx_local(q_full(i), (uint32_t)used * kD * 2);
        for (int c = 0; c < kD / 64; ++c)
          tma_load_3d(base + S::q + i * S::tile_bytes + c * (kTile * 128), &tm_q, 64 * c, hk * p.G, q0 + i * tokens, q_full(i));
      }
    }
    const int32_t nowhere = (int32_t)(p.num_blocks * p.Hk);   // past the pool: the copy fills zeros
    int32_t ids = 0;
    uint32_t it = 0;
    for (int j = 0; j < nk && ok; ++j) {
      if ((j & 15) == 0) {
        const int x = 2 * j + lane;
        const int32_t id = x < pages ? table[x] : -1;
        ids = id >= 0 && (int64_t)id < p.num_blocks ? id * p.Hk + hk : nowhere;
        if (any_bad && x < pages && ids == nowhere) record_error(p.status, MLA_ERR_BOUNDS);
      }
      const int32_t z0 = __shfl_sync(0xffffffffu, ids, (2 * j) & 31), z1 = __shfl_sync(0xffffffffu, ids, (2 * j + 1) & 31);
      if (lane == 0) {
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int s = it % kSlots;
          if (it >= (uint32_t)kSlots) ok = mbar_wait(empty(s), ((it / kSlots) - 1) & 1, p.wait_limit_ns);
          if (!ok) break;
          const uint32_t dst = base + S::ring + s * S::tile_bytes;
          const CUtensorMap* m = kv ? &tm_v : &tm_k;
          mbar_arrive_expect_tx_local(full(s), S::tile_bytes);
          for (int c = 0; c < kD / 64; ++c) {
            tma_load_3d(dst + c * (kTile * 128), m, 64 * c, 0, z0, full(s));
            tma_load_3d(dst + c * (kTile * 128) + 8192, m, 64 * c, 0, z1, full(s));
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (!ok && lane == 0) {
      record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
      // copies still in flight land before the block ends
      for (uint32_t i = it > (uint32_t)kSlots ? it - kSlots : 0; i < it; ++i)
        (void)mbar_wait(full(i % kSlots), (i / kSlots) & 1, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer --
    // The warp stays converged and one elected lane issues: descriptors and
    // addresses are then uniform, and an MMA costs a few issue slots. (Issued
    // by lane 0 of a diverged warp, the 32 MMAs of a step took 4270 cycles.)
    if (nk > 0) {
      constexpr uint32_t idesc_s = idesc16<T>(128, 128, 0, 0), idesc_o = idesc16<T>(128, kD, 0, 1);
      const bool leader = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      };
      auto scores = [&](int i, int s) {
        if (!ok || !leader) return;
        const uint64_t a = smem_desc_sw128(base + S::q + i * S::tile_bytes, 16, 1024);
        const uint64_t k = smem_desc_sw128(base + S::ring + s * S::tile_bytes, 16, 1024);
#pragma unroll
        for (int x = 0; x < kD / 16; ++x) {
          const uint64_t off = (uint64_t)((x / 4) * ((kTile * 128) >> 4) + 2 * (x % 4));
          mma_f16<1>(tbase + 128 * i, a + off, k + off, idesc_s, x ? 1u : 0u);
        }
        tc_commit<1>(s_full(i));
      };
      auto values = [&](int i, int s, bool more, auto x0, auto x1) {
        if (!ok || !leader) return;
        const uint64_t v = smem_desc_sw128(base + S::ring + s * S::tile_bytes, kTile * 128, 1024);
#pragma unroll
        for (int x = x0; x < x1; ++x)
          mma_ts(tbase + kTmemO + kD * i, tbase + 128 * i + 8 * x, v + (uint64_t)(128 * x), idesc_o, more || x ? 1u : 0u);
      };
      auto done = [&](uint32_t bar) {
        if (ok && leader) tc_commit<1>(bar);
      };
      constexpr std::integral_constant<int, 0> k0{};
      constexpr std::integral_constant<int, kEarlyKeys / 16> kEarly{};
      constexpr std::integral_constant<int, kTile / 16> kAll{};
      uint32_t it = 0;                   // the next ring item
      auto arrived = [&]() {
        wait(full(it % kSlots), (it / kSlots) & 1);
        return (int)(it++ % kSlots);
      };
      const int s = arrived();
      // a tile that sees no key is waited for too: its copy lands before the block ends
      wait(q_full(0), 0);
      if (nk0 > 0) scores(0, s);
      if (two_tiles) wait(q_full(1), 0);
      if (nk1 > 0) scores(1, s);
      done(empty(s));
      for (int j = 0; j < nk && ok; ++j) {
        const int vs = arrived();
        int ks = 0;
        if (j < nk0) {
          wait(p_part(0), j & 1);
          values(0, vs, j > 0, k0, kEarly);
          wait(p_full(0), j & 1);
          values(0, vs, j > 0, kEarly, kAll);
          if (j + 1 == nk0) done(o_full(0));
        }
        if (j + 1 < nk) {
          ks = arrived();
          if (j + 1 < nk0) scores(0, ks);
        }
        if (j < nk1) {
          wait(p_part(1), j & 1);
          values(1, vs, j > 0, k0, kEarly);
          wait(p_full(1), j & 1);
          values(1, vs, j > 0, kEarly, kAll);
          if (j + 1 == nk1) done(o_full(1));
        }
        done(empty(vs));
        if (j + 1 < nk) {
          if (j + 1 < nk1) scores(1, ks);
          done(empty(ks));
        }
      }
      if (!ok && lane == 0) record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------------- softmax --
    const int tile = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const int64_t t = t0 + (int64_t)tile * tokens + row / p.G;      // this row's token, in its sequence
    const bool real = row < used && t < n;
    // keys that the row sees; a row without a query is computed and not stored
    const int64_t sees = real ? max((int64_t)0, ahead + t + 1) : (int64_t)1 << 40;
    const int steps_here = tile ? nk1 : nk0;
    const uint32_t s_cols = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * tile;
    const uint32_t o_cols = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kTmemO + kD * tile;
    float m = -INFINITY, l = 0.f;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = mbar_wait(bar, parity, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
    };
    for (int j = 0; j < steps_here; ++j) {
      wait(s_full(tile), j & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t r[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32(s_cols + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
      tmem_wait_ld();
      const int64_t left = sees - (int64_t)j * kTile;
      if (left < kTile) {
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c >= (int)left) r[c] = 0xff800000u;
      }
      if (any_bad) {
        for (int half = 0; half < 2; ++half) {
          const int x = 2 * j + half;
          const int32_t id = x < pages ? table[x] : 0;
          if (id < 0 || (int64_t)id >= p.num_blocks) {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (c / kPage == half) r[c] = 0xff800000u;
          }
        }
      }
      float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kTile; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = max_three(x[e], __uint_as_float(r[c + 2 * e]), __uint_as_float(r[c + 2 * e + 1]));
      const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
      const bool move = top > m + WS::lazy;      // also a row's first visible key (m = -inf)
      const float mn = move ? top : m;
      if (__any_sync(0xffffffffu, move && l > 0.f)) {
        // the products up to step j - 1 are complete (S(j) is), and no other is under way
        const float a = m == mn ? 1.f : ex2_approx(m - mn);
        l *= a;
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_cols + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st32(o_cols + c, o);
        }
      }
      m = mn;
      if ((j + 1) * kTile > L && (tile == 0 || j >= nk0)) {
        // the cache's last step: values of slots without a token may hold
        // anything, and 0 times NaN is not 0. The first tile to use them
        // clears them before its weights are handed over.
        const int s = (2 * j + 1) % kSlots;
        wait(full(s), ((2 * j + 1) / kSlots) & 1);
        if (ok)
          for (int i = row; i < ((j + 1) * kTile - L) * (kD / 8); i += 128) {
            const int x = kTile - 1 - i / (kD / 8), c = i % (kD / 8);
            *reinterpret_cast<uint4*>(gbase + S::ring + s * S::tile_bytes + (c >> 3) * (kTile * 128) + x * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async_smem();
      }
      const float shift = m == -INFINITY ? 0.f : WS::bias - m;
      const uint64_t sc = two(p.scale_log2, p.scale_log2), sh = two(shift, shift);
      uint64_t sum0 = two(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float2 a = apart(fma_two(two(__uint_as_float(r[c + e]), __uint_as_float(r[c + e + 1])), sc, sh));
          const float2 d = apart(fma_two(two(__uint_as_float(r[c + e + 2]), __uint_as_float(r[c + e + 3])), sc, sh));
          const float y0 = ex2_approx(a.x), y1 = ex2_approx(a.y), y2 = ex2_approx(d.x), y3 = ex2_approx(d.y);
          sum0 = add_two(sum0, two(y0, y1));
          sum1 = add_two(sum1, two(y2, y3));
          w[e / 2] = Pack<T>::of(y0, y1);
          w[e / 2 + 1] = Pack<T>::of(y2, y3);
        }
        tmem_st16(s_cols + c / 2, w);   // over scores that are in registers
        if (c + 32 == kEarlyKeys) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_local(p_part(tile));
        }
      }
      const float2 u0 = apart(sum0), u1 = apart(sum1);
      l += (u0.x + u0.y) + (u1.x + u1.y);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_local(p_full(tile));
    }
    // ---- O / l
    if (steps_here > 0) wait(o_full(tile), 0);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      T* out = static_cast<T*>(p.out) + ((c0 + t) * p.Hq + hk * p.G + row % p.G) * (int64_t)kD;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (steps_here > 0) {
          tmem_ld32(o_cols + c, o);
          tmem_wait_ld();
        }
        if (!real) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = l > 0.f ? Pack<T>::of(__uint_as_float(o[e + 2 * x]) * inv, __uint_as_float(o[e + 2 * x + 1]) * inv) : 0u;
          *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (!ok && lane == 0) record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<1>(tbase, 512);
}

// ------------------------------------------------------------------ host ---
// The packed queries [T, Hq, d] as (d, Hq, T): boxes of 64 columns x G heads x
// the tokens of a tile.
inline bool query_map(CUtensorMap* m, const void* q, int64_t T, int Hq, int G, int d, bool bf16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)Hq * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTile / G)}, es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of one launch: a pair of tiles of every sequence's longest possible count, per key head.
inline int64_t prefill_steps(int32_t max_new, int G) { return (max_new + 2 * (kTile / G) - 1) / (2 * (kTile / G)); }

template <typename T, int kD>
cudaError_t launch_prefill(const GqaParams& p, cudaStream_t stream) {
  using S = PrefillSmem<kD>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  CUtensorMap tm_q, tm_k, tm_v;
  if (!query_map(&tm_q, p.q, p.T, p.Hq, p.G, kD, bf16) ||
      !pool_map(&tm_k, p.k_pool, p.num_blocks * p.Hk, kD, bf16) || !pool_map(&tm_v, p.v_pool, p.num_blocks * p.Hk, kD, bf16))
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(gqa_prefill_kernel<T, kD>), (int)S::alloc);
  if (e != cudaSuccess) return e;
  const int64_t steps = prefill_steps(p.max_new, p.G);
  return launch_dependent(gqa_prefill_kernel<T, kD>, dim3((unsigned)(steps * p.B * p.Hk)), dim3(kPrefillThreads), S::alloc,
                          stream, tm_q, tm_k, tm_v, p, (int32_t)steps);
}

}  // namespace pg
}  // namespace mla
