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
// Warps: 0 producer, 1 MMA issuer, 2 scheduler, 4-7 and 8-11 the softmax of tile
// 0 and 1 (a row per thread, running maximum and sum in fp32). The two tiles
// alternate: while one tile's weights are computed, the tensor core works for
// the other. The MMAs of a tile run in the order S(0), O(0), S(1), O(1), ..; one
// thread issues them, so S(j + 1) may overwrite the P(j) that O(j) has read, and
// a full S(j + 1) means that O(j) is complete.
//
// Blocks stay: one per SM works through items (a pair of tiles), each drawn from
// a list that a first small kernel sorts by the number of steps, longest first.
// The next item's queries, keys and first scores come while the last one is
// divided and stored. (With a block per item, about 10 us of set-up and drain
// each: 64 us instead of 51 at eight prompts of 63 to 1331 tokens, 480 instead of
// 427 at 8K tokens and 32 heads. Items drawn without the sort, last pairs of
// every sequence first: 140 us instead of 116 at five chunks over 3 to 5.3K cached
// tokens, 51.8 instead of 50.5 at the eight prompts.)
//
// What bounds it: a step of two tiles takes 3190 cycles (both head sizes). The
// chain of one tile is scores in tensor memory -> registers 70, maximum 370,
// weights 1450 (1024 of special-function unit, shared with the other tile's
// warps), P V and Q K^T 1180; the tensor core is busy for 2048 of the cycles at
// d = 128. At 8K tokens that is 437 us while the clock stays at 1965 MHz (1260
// TFLOP/s); in a loop the power cap lowers it and it takes 480 to 525 us. Tried and
// no faster: the maximum found beside the first weights, with those made again
// where it moves (3370 cycles); for d = 64, weights in columns of their own, so
// that S(j + 1) is computed during the softmax of step j (3700 cycles: the two
// tiles fall into step and share the special-function unit; 3320 when started half
// a step apart); a quarter or half of the exponentials by a polynomial, and bf16
// rounding by integer instructions, alone and together (up to 10% slower at
// d = 128, within the power cap's noise at d = 64). The products themselves run at
// the tensor core's rate when issued back to back (64 cycles per 128 x 128 x 16
// from either operand form), also beside tensor-memory loads and exponentials.
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
  static constexpr uint32_t work = bars + 320;
  static constexpr uint32_t misc = work + 128;
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

// An item: 2 (128 / G) tokens of one sequence and one key head.
struct Item {
  int64_t c0;              // the sequence's first packed row
  int64_t n, t0, ahead;    // its new tokens; the item's first; position of token t: ahead + t
  int32_t L, b, hk;        // b < 0: no more items
  int32_t nk0, nk1;        // steps of the two tiles (0: none, or no key is seen)
  int32_t two_tiles, pages, any_bad;

  __device__ __forceinline__ int nk() const { return max(nk0, nk1); }
};

// The new tokens of sequence b as they are, or -1 where the prefix sums are not
// those of the packed rows or exceed the plan (told by `tell`).
__device__ __forceinline__ int64_t new_tokens(const GqaParams& p, int32_t b, bool tell) {
  const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
  if (c0 >= 0 && c0 <= c1 && c1 <= p.T && c1 - c0 <= p.max_new) return c1 - c0;
  if (tell) record_error(p.status, MLA_ERR_BOUNDS);
  return -1;
}

// Steps of 128 keys that the tokens up to t (not included) of a sequence see.
__device__ __forceinline__ int32_t steps_to(int64_t ahead, int64_t t) {
  const int64_t last = ahead + t - 1;
  return last < 0 ? 0 : (int32_t)(last / kTile) + 1;
}

// Sorts the items of a call by their steps, longest first (a counting sort; the
// order among equals is not fixed and moves no result): p.order[i] = (sequence,
// pair of tiles), p.order_state = {items drawn, items}.
constexpr int kOrderThreads = 1024;      // and buckets: items of 1023 steps or more share one
__global__ void __launch_bounds__(kOrderThreads) gqa_prefill_order_kernel(GqaParams p) {
  __shared__ int32_t bucket[kOrderThreads];
  __shared__ int32_t warp_sum[32];
  bucket[threadIdx.x] = 0;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = 2 * (kTile / p.G);
  auto walk = [&](bool tell, auto put) {
    for (int b = warp; b < p.B; b += 32) {
      const int64_t n = new_tokens(p, b, tell && lane == 0);
      const int64_t ahead = checked_len(p, b, false) - n;
      for (int64_t i = lane; i * tokens < n; i += 32) {
        const int32_t nk = steps_to(ahead, min(n, (i + 1) * tokens));
        put(kOrderThreads - 1 - min(nk, kOrderThreads - 1), b, (int32_t)i);   // long ones first
      }
    }
  };
  walk(true, [&](int k, int, int) { atomicAdd(bucket + k, 1); });
  __syncthreads();
  // exclusive prefix sums over the buckets
  const int32_t mine = bucket[threadIdx.x];
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int32_t sums = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += x;
  }
  const int32_t before = warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0, total = __shfl_sync(0xffffffffu, sums, 31);
  bucket[threadIdx.x] = before + upto - mine;
  __syncthreads();
  walk(false, [&](int k, int b, int i) {
    const int32_t at = atomicAdd(bucket + k, 1);
    if (at < p.order_room) p.order[at] = make_int2(b, i);
    else record_error(p.status, MLA_ERR_BOUNDS);   // prefix sums that overlap
  });
  if (threadIdx.x == 0) {
    p.order_state[0] = 0;
    p.order_state[1] = min(total, p.order_room);
  }
}

template <typename T, int kD>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, GqaParams p) {
  using namespace ptx;
  using S = PrefillSmem<kD>;
  using WS = WeightScale<T>;
  constexpr int kSlots = S::slots;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return base + S::bars + 8u * i; };
  auto full = [&](int s) -> uint32_t { return bar(s); };                     // ring items
  auto empty = [&](int s) -> uint32_t { return bar(kSlots + s); };
  auto q_full = [&](int i) -> uint32_t { return bar(2 * kSlots + i); };      // per tile
  auto q_empty = [&](int i) -> uint32_t { return bar(2 * kSlots + 2 + i); };
  auto s_full = [&](int i) -> uint32_t { return bar(2 * kSlots + 4 + i); };
  auto p_part = [&](int i) -> uint32_t { return bar(2 * kSlots + 6 + i); };
  auto p_full = [&](int i) -> uint32_t { return bar(2 * kSlots + 8 + i); };
  auto o_full = [&](int i) -> uint32_t { return bar(2 * kSlots + 10 + i); };
  auto o_empty = [&](int i) -> uint32_t { return bar(2 * kSlots + 12 + i); };
  const uint32_t w_full = bar(2 * kSlots + 14), w_empty = bar(2 * kSlots + 15);   // the work item
  const uint32_t drained = bar(2 * kSlots + 16);                                  // after a timeout
  Item* work = reinterpret_cast<Item*>(gbase + S::work);
  static_assert(sizeof(Item) <= 128 && 8 * (2 * kSlots + 17) <= 320, "shared memory layout");
  uint32_t* tslot = reinterpret_cast<uint32_t*>(gbase + S::misc);
  const int tokens = kTile / p.G, used = tokens * p.G;              // of one tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kSlots + 17; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < 2; ++i) {        // the four softmax warps of the tile
      mbar_init(p_part(i), 4);
      mbar_init(p_full(i), 4 + p.withhold);
      mbar_init(o_empty(i), 4);
    }
    mbar_init(w_empty, 10);              // producer, MMA issuer, softmax warps
    fence_mbarrier_init_cluster();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc<1>(base + S::misc, 512);
    tmem_relinquish<1>();
  }
  // rows of the query tiles that no token fills; no copy writes them
  for (int i = threadIdx.x; i < 2 * (kTile - used) * (kD / 8); i += kPrefillThreads) {
    const int r = i / (kD / 8), c = i % (kD / 8), tile = r / (kTile - used), row = used + r % (kTile - used);
    *reinterpret_cast<uint4*>(gbase + S::q + tile * S::tile_bytes + (c >> 3) * (kTile * 128) + row * 128 + (c & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  constexpr uint32_t kTmemO = 256;       // S (and P) of tile i: columns [128 i, +128); O: [256 + d i, +d)
  bool ok = true;
  // Every access waits for the grid before this one; only then may the next
  // grid's blocks be placed, so that what they read ahead of their own wait
  // (weights) is past whatever wrote it.
  grid_dependency_wait();
  grid_launch_dependents();

  // Every role walks the same items in the same order. Barriers are used in
  // phases that each role counts for itself: `items` so far, ring copies, and per
  // tile the items and steps in which it took part.
  uint32_t items = 0;
  // the next item, by converged warps; the place for the one after it is free
  // when every role has copied this one (the producer says so later, once its
  // copies are issued, so that a block does not draw far ahead)
  auto draw = [&](Item& x, bool free_now) {
    if (ok) ok = mbar_wait(w_full, items & 1, p.wait_limit_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    x = *work;
    ++items;
    __syncwarp();
    if (free_now && lane == 0) mbar_arrive_local(w_empty);
    return x.b >= 0;
  };

  if (warp < 4) {
    // 384 x 168 registers at launch: 128 x 72 + 256 x 216
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 2) {
      // ---------------------------------------------------------- scheduler --
      Item x{};
      uint32_t ticket = blockIdx.x;
      for (bool more = true; more && ok; ++items) {
        // One lane reads and the warp agrees on what it read. The list lies in the
        // workspace: where two calls share one by mistake its entries may be another
        // call's, and none is followed out of this call's sequences.
        int32_t b = -1, pair = 0, c0 = 0, n = 0, L = 0;
        if (lane == 0) {
          const uint32_t place = ticket / (uint32_t)p.Hk;
          if (p.order) {
            const int32_t count = min(p.order_state[1], p.order_room);
            const int2 at = p.order[min(place, (uint32_t)p.order_room - 1)];   // read beside the count
            if (count > 0 && place < (uint32_t)count) {
              b = at.x;
              pair = at.y;
              if (b < 0 || b >= p.B || pair < 0) b = -2;
            }
          } else if (items == 0) {       // one item per block
            b = (int32_t)(place % (uint32_t)p.B);
            pair = (int32_t)(place / (uint32_t)p.B);
          }
          if (b >= 0) {
            c0 = p.cu[b];
            L = checked_len(p, b, false);
            n = (int32_t)new_tokens(p, b, !p.order && pair == 0);
            if ((int64_t)pair * 2 * tokens >= n) b = p.order ? -2 : -1;
            else if (L == 0) (void)checked_len(p, b, true);
          }
          if (b == -2) record_error(p.status, MLA_ERR_BOUNDS);
        }
        x.b = __shfl_sync(0xffffffffu, b, 0);
        more = x.b >= 0;
        if (more) {
          x.hk = (int32_t)(ticket % (uint32_t)p.Hk);
          x.t0 = (int64_t)__shfl_sync(0xffffffffu, pair, 0) * 2 * tokens;
          x.c0 = __shfl_sync(0xffffffffu, c0, 0);
          x.n = __shfl_sync(0xffffffffu, n, 0);
          x.L = __shfl_sync(0xffffffffu, L, 0);
          x.ahead = x.L - x.n;
          x.two_tiles = x.t0 + tokens < x.n;
          x.nk0 = steps_to(x.ahead, min(x.t0 + tokens, x.n));
          x.nk1 = x.two_tiles ? steps_to(x.ahead, min(x.t0 + 2 * tokens, x.n)) : 0;
          x.pages = min(pages_of(x.L), 2 * x.nk());
          // pages whose block is out of range: their keys are not seen
          bool bad = false;
          for (int i = lane; i < x.pages; i += 32) {
            const int32_t id = p.block_table[(int64_t)x.b * p.bt_stride + i];
            bad |= id < 0 || (int64_t)id >= p.num_blocks;
          }
          x.any_bad = __any_sync(0xffffffffu, bad);
          if (x.any_bad && lane == 0) record_error(p.status, MLA_ERR_BOUNDS);
        }
        // the last item has been read by every role, and its copies are issued
        if (items > 0) ok = mbar_wait(w_empty, (items - 1) & 1, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          *work = x;
          mbar_arrive_local(w_full);
          if (more && p.order) ticket = gridDim.x + (uint32_t)atomicAdd(p.order_state, 1);
        }
        ticket = __shfl_sync(0xffffffffu, ticket, 0);
      }
      if (!ok && lane == 0) record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
    } else if (warp == 0) {
      // ----------------------------------------------------------- producer --
      const int32_t nowhere = (int32_t)(p.num_blocks * p.Hk);   // past the pool: the copy fills zeros
      uint32_t it = 0, q_uses[2] = {0, 0};
      Item x;
      while (draw(x, false)) {
        const int32_t* table = p.block_table + (int64_t)x.b * p.bt_stride;
        const int nk = x.nk();
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if ((i ? x.nk1 : x.nk0) == 0 || !ok) continue;
            if (q_uses[i] > 0) ok = mbar_wait(q_empty(i), (q_uses[i] - 1) & 1, p.wait_limit_ns);
            if (!ok) continue;
            ++q_uses[i];
            mbar_arrive_expect_tx_local(q_full(i), (uint32_t)used * kD * 2);
            for (int c = 0; c < kD / 64; ++c)
              tma_load_3d(base + S::q + i * S::tile_bytes + c * (kTile * 128), &tm_q, 64 * c, x.hk * p.G,
                          (int32_t)(x.c0 + x.t0) + i * tokens, q_full(i));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        int32_t ids = 0;
        for (int j = 0; j < nk && ok; ++j) {
          if ((j & 15) == 0) {
            const int pg = 2 * j + lane;
            const int32_t id = pg < x.pages ? table[pg] : -1;
            ids = id >= 0 && (int64_t)id < p.num_blocks ? id * p.Hk + x.hk : nowhere;
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
        if (!ok) break;
        if (lane == 0) mbar_arrive_local(w_empty);
      }
      if (!ok && lane == 0) {
        record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
        // copies still in flight land before the block ends
        for (int i = 0; i < 2; ++i)
          if (q_uses[i] > 0) (void)mbar_wait(q_full(i), (q_uses[i] - 1) & 1, p.wait_limit_ns);
        for (uint32_t i = it > (uint32_t)kSlots ? it - kSlots : 0; i < it; ++i)
          (void)mbar_wait(full(i % kSlots), (i / kSlots) & 1, p.wait_limit_ns);
      }
    } else if (warp == 1) {
      // --------------------------------------------------------- MMA issuer --
      // The warp stays converged and one elected lane issues: descriptors and
      // addresses are then uniform, and an MMA costs a few issue slots. (Issued
      // by lane 0 of a diverged warp, the 32 MMAs of a step took 4270 cycles; a
      // step took 3350 with this change, and takes 3190 now.)
      constexpr uint32_t idesc_s = idesc16<T>(128, 128, 0, 0), idesc_o = idesc16<T>(128, kD, 0, 1);
      constexpr std::integral_constant<int, 0> k0{};
      constexpr std::integral_constant<int, kEarlyKeys / 16> kEarly{};
      constexpr std::integral_constant<int, kTile / 16> kAll{};
      const bool leader = elect_one();
      auto wait = [&](uint32_t b, uint32_t parity) {
        ok = ok && mbar_wait(b, parity, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      };
      auto done = [&](uint32_t b) {
        if (ok && leader) tc_commit<1>(b);
      };
      auto scores = [&](int i, int s) {
        if (!ok || !leader) return;
        const uint64_t a = smem_desc_sw128(base + S::q + i * S::tile_bytes, 16, 1024);
        const uint64_t k = smem_desc_sw128(base + S::ring + s * S::tile_bytes, 16, 1024);
#pragma unroll
        for (int y = 0; y < kD / 16; ++y) {
          const uint64_t off = (uint64_t)((y / 4) * ((kTile * 128) >> 4) + 2 * (y % 4));
          mma_f16<1>(tbase + 128 * i, a + off, k + off, idesc_s, y ? 1u : 0u);
        }
        tc_commit<1>(s_full(i));
      };
      auto values = [&](int i, int s, bool more, auto from, auto to) {
        if (!ok || !leader) return;
        const uint64_t v = smem_desc_sw128(base + S::ring + s * S::tile_bytes, kTile * 128, 1024);
#pragma unroll
        for (int y = from; y < to; ++y)
          mma_ts(tbase + kTmemO + kD * i, tbase + 128 * i + 8 * y, v + (uint64_t)(128 * y), idesc_o, more || y ? 1u : 0u);
      };
      uint32_t it = 0, uses[2] = {0, 0}, steps[2] = {0, 0};
      auto arrived = [&]() {             // the next ring item's slot
        wait(full(it % kSlots), (it / kSlots) & 1);
        return (int)(it++ % kSlots);
      };
      Item x;
      while (draw(x, true)) {
        const int nk = x.nk();
        if (nk == 0) continue;
        const int ks0 = arrived();
        // the first scores of a tile; its query slot is free again after its last
        auto begin = [&](int i, int n) {
          if (n == 0) return;
          wait(q_full(i), uses[i]++ & 1);
          scores(i, ks0);
          if (n == 1) done(q_empty(i));
        };
        begin(0, x.nk0);
        begin(1, x.nk1);
        done(empty(ks0));
        // O = P V of step j; the last item's O has been read before the first
        auto step = [&](int i, int n, int j, int vs) {
          if (j >= n) return;
          if (j == 0 && uses[i] > 1) wait(o_empty(i), (uses[i] - 2) & 1);
          wait(p_part(i), steps[i] & 1);
          values(i, vs, j > 0, k0, kEarly);
          wait(p_full(i), steps[i]++ & 1);
          values(i, vs, j > 0, kEarly, kAll);
          if (j + 1 == n) done(o_full(i));
        };
        auto next_scores = [&](int i, int n, int j, int ks) {
          if (j + 1 >= n) return;
          scores(i, ks);
          if (j + 2 == n) done(q_empty(i));
        };
        for (int j = 0; j < nk && ok; ++j) {
          const int vs = arrived();
          int ks = 0;
          step(0, x.nk0, j, vs);
          if (j + 1 < nk) {
            ks = arrived();
            next_scores(0, x.nk0, j, ks);
          }
          step(1, x.nk1, j, vs);
          done(empty(vs));
          if (j + 1 < nk) {
            next_scores(1, x.nk1, j, ks);
            done(empty(ks));
          }
        }
        if (!ok) break;
      }
      // the last commit has arrived before the block ends
      if (it > 0) wait(empty((it - 1) % kSlots), ((it - 1) / kSlots) & 1);
      if (!ok) {
        if (lane == 0) record_error(p.status, MLA_ERR_DEVICE_TIMEOUT);
        // products that were issued are complete before their operands and
        // accumulators are given back
        if (leader) tc_commit<1>(drained);
        __syncwarp();
        (void)mbar_wait(drained, 0, p.wait_limit_ns);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------------- softmax --
    const int tile = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t s_cols = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * tile;
    const uint32_t o_cols = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kTmemO + kD * tile;
    uint32_t it0 = 0, uses = 0, steps = 0;
    auto wait = [&](uint32_t b, uint32_t parity) {
      if (ok) ok = mbar_wait(b, parity, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
    };
    const int row_token = tile * tokens + row / p.G;
    for (;;) {
      int32_t sees, nk, L, clear_from;   // clear_from: the step from which on this tile clears the cache's last values
      int32_t it_next;
      const int32_t* table = nullptr;    // of a sequence with pages that are out of range
      int32_t pages = 0;
      T* out = nullptr;                  // this row's, if it is one of the item's
      {
        Item x;
        if (!draw(x, true)) break;
        // keys that the row sees; a row without a query is computed and not stored
        const int64_t t = x.t0 + row_token;                           // this row's token, in its sequence
        const bool real = row < used && t < x.n;
        sees = real ? (int32_t)max((int64_t)0, x.ahead + t + 1) : 0x7fffffff;
        if (real) out = static_cast<T*>(p.out) + ((x.c0 + t) * p.Hq + x.hk * p.G + row % p.G) * (int64_t)kD;
        nk = tile ? x.nk1 : x.nk0;
        L = x.L;
        clear_from = tile ? x.nk0 : 0;
        it_next = it0 + 2 * x.nk();
        if (x.any_bad) {
          table = p.block_table + (int64_t)x.b * p.bt_stride;
          pages = x.pages;
        }
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nk; ++j) {
        wait(s_full(tile), steps++ & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(s_cols + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
        tmem_wait_ld();
        const int32_t left = sees - j * kTile;
        if (left < kTile) {
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c >= left) r[c] = 0xff800000u;
        }
        if (table) {
          for (int half = 0; half < 2; ++half) {
            const int pg = 2 * j + half;
            const int32_t id = pg < pages ? table[pg] : 0;
            if (id < 0 || (int64_t)id >= p.num_blocks) {
#pragma unroll
              for (int c = 0; c < kTile; ++c)
                if (c / kPage == half) r[c] = 0xff800000u;
            }
          }
        }
        float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kTile; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = max_three(y[e], __uint_as_float(r[c + 2 * e]), __uint_as_float(r[c + 2 * e + 1]));
        const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * p.scale_log2;
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
        if (L - j * kTile < kTile && j >= clear_from) {
          // the cache's last step: values of slots without a token may hold
          // anything, and 0 times NaN is not 0. The first tile to use them
          // clears them before its weights are handed over.
          const uint32_t it = it0 + 2 * j + 1;
          wait(full(it % kSlots), (it / kSlots) & 1);
          if (ok)
            for (int i = row; i < (kTile - (L - j * kTile)) * (kD / 8); i += 128) {
              const int z = kTile - 1 - i / (kD / 8), c = i % (kD / 8);
              *reinterpret_cast<uint4*>(gbase + S::ring + it % kSlots * S::tile_bytes + (c >> 3) * (kTile * 128) + z * 128 +
                                        (c & 7) * 16) = make_uint4(0, 0, 0, 0);
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
      it0 = it_next;
      // ---- O / l, read before the next item's first product may overwrite it
      if (nk > 0) wait(o_full(tile), uses++ & 1);
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (nk > 0) {
          tmem_ld32(o_cols + c, o);
          tmem_wait_ld();
        }
        if (!out) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = l > 0.f ? Pack<T>::of(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv) : 0u;
          *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (nk > 0 && lane == 0) mbar_arrive_local(o_empty(tile));
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

// Pairs of tiles of the longest count that a plan allows.
inline int64_t prefill_pairs(int32_t max_new, int G) { return (max_new + 2 * (kTile / G) - 1) / (2 * (kTile / G)); }

// Items whose order a workspace has room for: pairs of tiles of any prefix sums over T rows.
inline int64_t prefill_order_room(int64_t T, int32_t B, int G) { return T / (2 * (kTile / G)) + B; }

template <typename T, int kD>
cudaError_t launch_prefill(GqaParams p, int32_t sms, cudaStream_t stream) {
  using S = PrefillSmem<kD>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  CUtensorMap tm_q, tm_k, tm_v;
  if (!query_map(&tm_q, p.q, p.T, p.Hq, p.G, kD, bf16) ||
      !pool_map(&tm_k, p.k_pool, p.num_blocks * p.Hk, kD, bf16) || !pool_map(&tm_v, p.v_pool, p.num_blocks * p.Hk, kD, bf16))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(gqa_prefill_kernel<T, kD>), (int)S::alloc);
  if (e != cudaSuccess) return e;
  // as many items as blocks fit at once: each takes its own, no order is needed
  int64_t blocks = prefill_pairs(p.max_new, p.G) * p.B * p.Hk;
  if (blocks <= sms) {
    p.order = nullptr;
  } else {
    blocks = std::min<int64_t>(sms, (int64_t)p.order_room * p.Hk);
    e = launch_dependent(gqa_prefill_order_kernel, dim3(1), dim3(kOrderThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(gqa_prefill_kernel<T, kD>, dim3((unsigned)blocks), dim3(kPrefillThreads), S::alloc, stream, tm_q, tm_k,
                          tm_v, p);
}

}  // namespace pg
}  // namespace mla
