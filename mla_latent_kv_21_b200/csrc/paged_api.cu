// Host side of the paged-cache operators (include/mla_paged.h): checks of the
// arguments, plans, launches.
#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "paged_append.cuh"
#include "paged_decode.cuh"
#include "paged_prefill.cuh"

using namespace mla;

struct mla_gqa_decode_plan {
  mla_gqa_dims_t dims;
  int32_t B, W, key_parts;
  size_t o_off, ml_off, tails_off, total;
};

struct mla_gqa_prefill_plan {
  mla_gqa_dims_t dims;
  int32_t B, max_new, order_room;
  int64_t T;
  size_t total;
};

namespace {

constexpr size_t kHeaderBytes = 1024;

mla_status_t check_dims(const mla_gqa_dims_t& d) {
  if (d.num_q_heads < 1 || d.num_kv_heads < 1 || d.num_q_heads % d.num_kv_heads != 0 || d.head_dim < 1 ||
      d.q_len < 1 || d.rope_dim < 0 || d.rope_dim > d.head_dim || !std::isfinite(d.softmax_scale) ||
      d.softmax_scale <= 0.f || (d.rope_style != MLA_ROPE_HALF && d.rope_style != MLA_ROPE_INTERLEAVED))
    return MLA_ERR_INVALID_ARG;
  if (d.dtype != MLA_BF16 && d.dtype != MLA_FP16)
    return d.dtype == MLA_FP32 || d.dtype == MLA_FP8_CACHE ? MLA_ERR_UNSUPPORTED : MLA_ERR_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128) || d.page_size != 64 || d.rope_dim % 16 != 0 || d.num_q_heads > 4096)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool multiple(int64_t a, int64_t b, int64_t n) { return a % n == 0 && b % n == 0; }

bool sm_count(int32_t* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    return true;
  (void)cudaGetLastError();
  return false;
}

// A failed launch leaves no error behind for a later call to find.
mla_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  (void)cudaGetLastError();
  return MLA_ERR_CUDA;
}

// Heads of a block of an append whose threads stand for `lanes` heads: 16 per
// thread where that still fills the machine (its angles are then loaded once for
// them; 1184 blocks are 8 to each of a B200's 148 SMs), else 4 (one batch of loads). Measured with 4 / 8 / 16 / 32: grouped-head
// append of 14K tokens 60.2 / 55.0 / 51.8 / 50.2 us; with 8 / 16 in the latent
// append of 16K tokens 118 / 107 us.
int heads_per_block(int64_t token_blocks, int H, int lanes) {
  return lanes * (token_blocks * ((H + 16 * lanes - 1) / (16 * lanes)) >= 1184 ? 16 : 4);
}

// How the four warps of a decode worker share a page where up to 16 rows read it:
// four key parts, or two key parts times two halves of the output columns. The
// halves compute the scores twice and join a quarter as much when a segment ends.
// At d = 128 they suit short segments; at d = 64 very short and long ones, for a
// reason that is not established. By the mean pages of a segment (a sequence's share of one worker); four key parts
// against halves, graph replay, medians of seven runs in turn, us:
//   d = 128: 0.9 pages (256 x 64, 8 heads) 29.0 / 24.5, 3.1 (128 x 200) 33.0 / 31.2, 5 (64 x
//     500) 30.3 / 29.9, 12 (1 x 60000, 4 heads) 31.4 / 31.1, 15 (32 x 2000) 51.0 / 51.0,
//     20 (16 x 2048, 32 heads) 90.6 / 91.1, 27 (1 x 131071, 4 heads) 53.3 / 53.3,
//     30 (16 x 3000) 128.1 / 128.9, 41 (16 x 4096) 170.7 / 173.3, 81 (16 x 8192) 328.8 / 332.8
//   d = 64: 0.9 pages 21.8 / 19.7, 1.7 (1 x 4000) 9.7 / 9.6, 3.1 23.1 / 23.4, 10 (16 x 1000, 32
//     heads) 29.6 / 30.8, 12 22.2 / 22.7, 15 30.1 / 30.4, 22 (32 x 3000) 40.0 / 39.8, 30 71.0 / 67.5,
//     41 92.9 / 90.4, 81 176.7 / 168.0
bool four_key_parts(int d, int64_t pages, int64_t segments) {
  return d == 128 ? pages >= 16 * segments : pages >= 3 * segments && pages < 20 * segments;
}

// Rows of the cache and of the batch: tensor-map and grid coordinates are 32-bit.
bool fits32(int64_t rows) { return rows < (int64_t(1) << 31); }
bool fits32(int64_t blocks, int32_t heads) { return fits32(blocks) && fits32(blocks * heads); }

// The waits of one run: the normal limit, or a self-test of the timeout path
// (short limit, barriers that expect one arrival more than they get).
struct Waits {
  uint64_t limit_ns = ptx::kWaitLimitNs;
  int32_t withhold = 0;
};

bool selftest_limit(uint64_t ns) { return ns >= 1000 && ns <= ptx::kWaitLimitNs; }

mla_status_t decode_run(mla_gqa_decode_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                        int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                        const int32_t* seq_lens_dev, void* out, void* workspace, size_t workspace_bytes, void* stream_,
                        Waits waits) {
  if (!plan || !q || !k_pool || !v_pool || !block_table || !seq_lens_dev || !out || !workspace || num_blocks < 1 ||
      block_table_stride < 1 || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const mla_gqa_dims_t& d = plan->dims;
  if (!fits32(num_blocks, d.num_kv_heads)) return MLA_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  GqaParams p{};
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.out = out;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.block_table = block_table;
  p.seq_lens = seq_lens_dev;
  p.o_part = reinterpret_cast<float*>(ws + plan->o_off);
  p.ml_part = reinterpret_cast<float2*>(ws + plan->ml_off);
  p.tails = reinterpret_cast<int2*>(ws + plan->tails_off);
  p.wait_limit_ns = waits.limit_ns;
  p.withhold = waits.withhold;
  p.num_blocks = num_blocks;
  p.bt_stride = block_table_stride;
  p.B = plan->B;
  p.Lq = d.q_len;
  p.T = (int64_t)plan->B * d.q_len;
  p.Hq = d.num_q_heads;
  p.Hk = d.num_kv_heads;
  p.G = p.Hq / p.Hk;
  p.W = plan->W;
  p.key_parts = plan->key_parts;
  p.scale_log2 = d.softmax_scale * 1.4426950408889634f;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int64_t items = (int64_t)p.B * p.Hk;
  const bool bf = d.dtype == MLA_BF16;
  const cudaError_t e = bf && d.head_dim == 128 ? pg::launch_decode<__nv_bfloat16, 128>(p, items, stream)
                      : bf                      ? pg::launch_decode<__nv_bfloat16, 64>(p, items, stream)
                      : d.head_dim == 128       ? pg::launch_decode<__half, 128>(p, items, stream)
                                                : pg::launch_decode<__half, 64>(p, items, stream);
  return launched(e);
}

mla_status_t prefill_run(mla_gqa_prefill_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                         int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                         const int32_t* cu_seqlens_dev, const int32_t* seq_lens_dev, void* out, void* workspace,
                         size_t workspace_bytes, void* stream_, Waits waits) {
  if (!plan || !workspace || num_blocks < 1 || block_table_stride < 1) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (plan->T == 0) return MLA_OK;
  if (!q || !k_pool || !v_pool || !block_table || !cu_seqlens_dev || !seq_lens_dev || !out || !aligned16(q) ||
      !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return MLA_ERR_INVALID_ARG;
  const mla_gqa_dims_t& d = plan->dims;
  if (!fits32(num_blocks, d.num_kv_heads)) return MLA_ERR_UNSUPPORTED;
  GqaParams p{};
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.out = out;
  p.status = static_cast<int32_t*>(workspace);
  p.block_table = block_table;
  p.seq_lens = seq_lens_dev;
  p.cu = cu_seqlens_dev;
  p.num_blocks = num_blocks;
  p.bt_stride = block_table_stride;
  p.B = plan->B;
  p.T = plan->T;
  p.Hq = d.num_q_heads;
  p.Hk = d.num_kv_heads;
  p.G = p.Hq / p.Hk;
  p.max_new = plan->max_new;
  p.order_state = static_cast<int32_t*>(workspace) + 4;
  p.order = reinterpret_cast<int2*>(static_cast<char*>(workspace) + kHeaderBytes);
  p.order_room = plan->order_room;
  int32_t sms = 0;
  if (!sm_count(&sms)) return MLA_ERR_NO_DEVICE;
  p.scale_log2 = d.softmax_scale * 1.4426950408889634f;
  p.wait_limit_ns = waits.limit_ns;
  p.withhold = waits.withhold;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const bool bf = d.dtype == MLA_BF16;
  const cudaError_t e = bf && d.head_dim == 128 ? pg::launch_prefill<__nv_bfloat16, 128>(p, sms, stream)
                      : bf                      ? pg::launch_prefill<__nv_bfloat16, 64>(p, sms, stream)
                      : d.head_dim == 128       ? pg::launch_prefill<__half, 128>(p, sms, stream)
                                                : pg::launch_prefill<__half, 64>(p, sms, stream);
  return launched(e);
}

}  // namespace

extern "C" {

mla_status_t mla_gqa_append(const mla_gqa_dims_t* dims, const mla_gqa_append_args_t* args, void* workspace,
                            size_t workspace_bytes, void* stream_) {
  if (!dims || !args || !workspace) return MLA_ERR_INVALID_ARG;
  const mla_gqa_dims_t& d = *dims;
  const mla_gqa_append_args_t& a = *args;
  const mla_status_t st = check_dims(d);
  if (st != MLA_OK) return st;
  if (workspace_bytes < kHeaderBytes) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (a.batch < 1 || a.num_tokens < 0 || a.num_blocks < 1 || a.block_table_stride < 1 || a.rope_positions < 0)
    return MLA_ERR_INVALID_ARG;
  if (!a.cu_seqlens && a.num_tokens != (int64_t)a.batch * d.q_len) return MLA_ERR_INVALID_ARG;
  if (a.num_tokens == 0) return MLA_OK;
  if (!a.k || !a.v || !a.k_pool || !a.v_pool || !a.block_table || !a.seq_lens || (a.q && !a.q_out) ||
      (d.rope_dim > 0 && !a.rope_table))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.q) || !aligned16(a.q_out) || !aligned16(a.k_pool) ||
      !aligned16(a.v_pool) || !aligned16(a.rope_table) || !multiple(a.k_token_stride, a.k_head_stride, 8) ||
      !multiple(a.v_token_stride, a.v_head_stride, 8) || (a.q && !multiple(a.q_token_stride, a.q_head_stride, 8)))
    return MLA_ERR_INVALID_ARG;
  if (!fits32(a.num_tokens) || !fits32(a.num_blocks, d.num_kv_heads)) return MLA_ERR_UNSUPPORTED;
  AppendParams p{};
  p.k = a.k; p.k_ts = a.k_token_stride; p.k_hs = a.k_head_stride;
  p.v = a.v; p.v_ts = a.v_token_stride; p.v_hs = a.v_head_stride;
  p.q = a.q; p.q_ts = a.q_token_stride; p.q_hs = a.q_head_stride;
  p.q_out = a.q_out;
  p.k_pool = a.k_pool;
  p.v_pool = a.v_pool;
  p.status = static_cast<int32_t*>(workspace);
  p.block_table = a.block_table;
  p.bt_stride = a.block_table_stride;
  p.seq_lens = a.seq_lens;
  p.cu = a.cu_seqlens;
  p.table = a.rope_table;
  p.table_rows = a.rope_positions;
  p.num_blocks = a.num_blocks;
  p.T = a.num_tokens;
  p.B = a.batch;
  p.Lq = d.q_len;
  p.Hq = d.num_q_heads;
  p.Hk = d.num_kv_heads;
  p.d = d.head_dim;
  p.D = d.rope_dim;
  const int H = (a.q ? p.Hq : 0) + 2 * p.Hk, tokens = pg::kAppendThreads / (p.d / 16 * pg::kGqaLanes);
  const int64_t gx = (p.T + tokens - 1) / tokens;
  p.heads_per_cta = heads_per_block(gx, H, pg::kGqaLanes);
  const dim3 grid((unsigned)gx, (unsigned)((H + p.heads_per_cta - 1) / p.heads_per_cta));
  const int half = d.rope_style == MLA_ROPE_HALF;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const dim3 block(pg::kAppendThreads);
  return launched(d.dtype == MLA_BF16 ? launch_dependent(pg::gqa_append_kernel<__nv_bfloat16>, grid, block, 0, stream, p, half)
                                      : launch_dependent(pg::gqa_append_kernel<__half>, grid, block, 0, stream, p, half));
}

mla_status_t mla_latent_append(const mla_dims_t* dims, int32_t rope_style, const mla_latent_append_args_t* args,
                               void* workspace, size_t workspace_bytes, void* stream_) {
  if (!dims || !args || !workspace) return MLA_ERR_INVALID_ARG;
  const mla_dims_t& d = *dims;
  const mla_latent_append_args_t& a = *args;
  if (d.num_heads < 1 || d.latent_rank < 1 || d.rope_dim < 0 || d.q_len < 1 ||
      (rope_style != MLA_ROPE_HALF && rope_style != MLA_ROPE_INTERLEAVED))
    return MLA_ERR_INVALID_ARG;
  if (d.dtype != MLA_BF16 && d.dtype != MLA_FP32 && d.dtype != MLA_FP8_CACHE) return MLA_ERR_INVALID_ARG;
  const bool fp8 = d.dtype == MLA_FP8_CACHE;
  if (d.page_size != 64 || d.rope_dim % 2 != 0 || d.latent_rank > 512 || d.latent_rank + d.rope_dim > 576 ||
      d.num_heads > 4096 || (fp8 && (d.latent_rank % 16 != 0 || d.rope_dim % 16 != 0 || d.rope_dim > 256)))
    return MLA_ERR_UNSUPPORTED;
  if (workspace_bytes < kHeaderBytes) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (a.batch < 1 || a.num_tokens < 0 || a.num_blocks < 1 || a.block_table_stride < 1 || a.rope_positions < 0)
    return MLA_ERR_INVALID_ARG;
  if (!a.cu_seqlens && a.num_tokens != (int64_t)a.batch * d.q_len) return MLA_ERR_INVALID_ARG;
  if (a.num_tokens == 0) return MLA_OK;
  const bool rot = d.rope_dim > 0;
  if (!a.ckv || !a.kv_pool || !a.block_table || !a.seq_lens || (rot && (!a.k_rope || !a.rope_table)) ||
      (a.q_rope && (!rot || !a.q_rope_out)) || (fp8 && ((rot && !a.kv_rope) || !a.kv_scale)))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(a.rope_table)) return MLA_ERR_INVALID_ARG;
  const int V = d.dtype == MLA_FP32 ? 4 : 8;
  const bool wide = aligned16(a.ckv) && aligned16(a.k_rope) && aligned16(a.q_rope) && aligned16(a.q_rope_out) &&
                    aligned16(a.kv_pool) && aligned16(a.kv_rope) && aligned16(a.kv_rows) && d.latent_rank % V == 0 &&
                    d.rope_dim % (2 * V) == 0 && d.rope_dim / (2 * V) * pg::kLatentLanes <= pg::kAppendThreads && a.ckv_token_stride % V == 0 &&
                    (!rot || a.k_rope_token_stride % V == 0) &&
                    (!a.q_rope || multiple(a.q_rope_token_stride, a.q_rope_head_stride, V));
  if (fp8 && !wide) return MLA_ERR_INVALID_ARG;
  if (!fits32(a.num_tokens) || !fits32(a.num_blocks)) return MLA_ERR_UNSUPPORTED;
  AppendParams p{};
  p.k = a.ckv; p.k_ts = a.ckv_token_stride;
  p.v = a.k_rope; p.v_ts = a.k_rope_token_stride;
  p.q = a.q_rope; p.q_ts = a.q_rope_token_stride; p.q_hs = a.q_rope_head_stride;
  p.q_out = a.q_rope_out;
  p.k_pool = a.kv_pool;
  p.v_pool = a.kv_rope;
  p.kv_scale = a.kv_scale;
  p.kv_rows = a.kv_rows;
  p.status = static_cast<int32_t*>(workspace);
  p.block_table = a.block_table;
  p.bt_stride = a.block_table_stride;
  p.seq_lens = a.seq_lens;
  p.cu = a.cu_seqlens;
  p.table = a.rope_table;
  p.table_rows = a.rope_positions;
  p.num_blocks = a.num_blocks;
  p.T = a.num_tokens;
  p.B = a.batch;
  p.Lq = d.q_len;
  p.Hq = d.num_heads;
  p.D = d.rope_dim;
  p.r = d.latent_rank;
  const int half = rope_style == MLA_ROPE_HALF;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (wide) {
    int64_t blocks = (p.T + 3) / 4;
    if (a.q_rope) {
      const int tokens = pg::kAppendThreads / (p.D / (2 * V) * pg::kLatentLanes);
      const int64_t gx = (p.T + tokens - 1) / tokens;
      p.heads_per_cta = heads_per_block(gx, p.Hq, pg::kLatentLanes);
      blocks += gx * ((p.Hq + p.heads_per_cta - 1) / p.heads_per_cta);
    }
    if (!fits32(blocks)) return MLA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks), block(pg::kAppendThreads);
    return launched(fp8      ? launch_dependent(pg::latent_append_kernel<__nv_bfloat16, true>, grid, block, 0, stream, p, half)
                    : V == 8 ? launch_dependent(pg::latent_append_kernel<__nv_bfloat16, false>, grid, block, 0, stream, p, half)
                             : launch_dependent(pg::latent_append_kernel<float, false>, grid, block, 0, stream, p, half));
  }
  const dim3 grid((unsigned)p.T), block(pg::kNarrowThreads);
  return launched(V == 8 ? launch_dependent(pg::latent_append_narrow_kernel<__nv_bfloat16>, grid, block, 0, stream, p, half)
                         : launch_dependent(pg::latent_append_narrow_kernel<float>, grid, block, 0, stream, p, half));
}

mla_status_t mla_gqa_decode_plan(const mla_gqa_dims_t* dims, int32_t batch, const int32_t* seq_lens_host,
                                 const mla_plan_options_t* opts, mla_gqa_decode_plan_t* plan_out,
                                 size_t* workspace_bytes) {
  if (!dims || !seq_lens_host || !plan_out || batch < 1) return MLA_ERR_INVALID_ARG;
  *plan_out = nullptr;
  const mla_status_t st = check_dims(*dims);
  if (st != MLA_OK) return st;
  const mla_gqa_dims_t& d = *dims;
  const int G = d.num_q_heads / d.num_kv_heads;
  if ((int64_t)G * d.q_len > 64 || !fits32((int64_t)batch * d.q_len * d.num_q_heads)) return MLA_ERR_UNSUPPORTED;
  mla_plan_options_t o{};
  if (opts) o = *opts;
  int32_t sms = o.num_sms;
  if (sms < 0 || o.num_workers < 0 || o.kernel != MLA_KERNEL_AUTO) return MLA_ERR_INVALID_ARG;
  if (sms == 0 && !sm_count(&sms)) return MLA_ERR_NO_DEVICE;
  int64_t pages = 0, items = 0;
  for (int b = 0; b < batch; ++b) {
    if (seq_lens_host[b] < 0) return MLA_ERR_INVALID_ARG;
    pages += ceil_div64(seq_lens_host[b], pg::kPage) * d.num_kv_heads;
    items += seq_lens_host[b] > 0 ? d.num_kv_heads : 0;
  }
  // Two workers per SM, down to one page each; only an item cut into more than
  // about 100 parts of a few pages costs more to join than it gains. Measured
  // with one key head, 20000 tokens (313 pages) and 8 / 16 / 64 rows: 296 workers
  // 17.3 / 17.4 / 21.3 us, 104 workers 11.6 / 11.7 / 18.0, 52 workers 12.5 / 12.6
  // / 21.6; with 8 key heads, 500 tokens: 64 workers 7.4, 32 7.8, 16 9.7.
  const int64_t most = o.num_workers > 0 ? o.num_workers : std::min<int64_t>(2 * sms, std::max(100 * items, pages / 4));
  struct mla_gqa_decode_plan* p = new (std::nothrow) struct mla_gqa_decode_plan();
  if (!p) return MLA_ERR_INVALID_ARG;
  p->dims = d;
  p->B = batch;
  p->W = (int32_t)std::max<int64_t>(1, std::min<int64_t>({most, pages, 4096}));
  p->key_parts = four_key_parts(d.head_dim, pages, p->W + items);
  const size_t rows = (size_t)2 * p->W * G * d.q_len;
  p->o_off = kHeaderBytes;
  p->ml_off = align_up(p->o_off + rows * d.head_dim * sizeof(float), 1024);
  p->tails_off = align_up(p->ml_off + rows * sizeof(float2), 1024);
  p->total = align_up(p->tails_off + p->W * sizeof(int2), 1024);
  *plan_out = p;
  if (workspace_bytes) *workspace_bytes = p->total;
  return MLA_OK;
}

mla_status_t mla_gqa_decode_run(mla_gqa_decode_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                                int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                                const int32_t* seq_lens_dev, void* out, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return decode_run(plan, q, k_pool, v_pool, num_blocks, block_table, block_table_stride, seq_lens_dev, out, workspace,
                    workspace_bytes, stream, Waits{});
}

mla_status_t mla_gqa_decode_selftest_timeout(mla_gqa_decode_plan_t plan, const void* q, const void* k_pool,
                                             const void* v_pool, int64_t num_blocks, const int32_t* block_table,
                                             int32_t block_table_stride, const int32_t* seq_lens_dev, void* out,
                                             void* workspace, size_t workspace_bytes, uint64_t wait_limit_ns,
                                             void* stream) {
  if (!selftest_limit(wait_limit_ns)) return MLA_ERR_INVALID_ARG;
  return decode_run(plan, q, k_pool, v_pool, num_blocks, block_table, block_table_stride, seq_lens_dev, out, workspace,
                    workspace_bytes, stream, Waits{wait_limit_ns, 1});
}

void mla_gqa_decode_plan_destroy(mla_gqa_decode_plan_t plan) { delete plan; }

mla_status_t mla_gqa_prefill_plan(const mla_gqa_dims_t* dims, int32_t batch, const int32_t* new_tokens_host,
                                  mla_gqa_prefill_plan_t* plan_out, size_t* workspace_bytes) {
  if (!dims || !new_tokens_host || !plan_out || batch < 1) return MLA_ERR_INVALID_ARG;
  *plan_out = nullptr;
  const mla_status_t st = check_dims(*dims);
  if (st != MLA_OK) return st;
  const mla_gqa_dims_t& d = *dims;
  int64_t T = 0;
  int32_t most = 0;
  for (int b = 0; b < batch; ++b) {
    if (new_tokens_host[b] < 0) return MLA_ERR_INVALID_ARG;
    T += new_tokens_host[b];
    most = std::max(most, new_tokens_host[b]);
  }
  const int G = d.num_q_heads / d.num_kv_heads;
  if (G > 128 || !fits32(T + 2 * pg::kTile) || !fits32(pg::prefill_order_room(T, batch, G) * d.num_kv_heads))
    return MLA_ERR_UNSUPPORTED;
  struct mla_gqa_prefill_plan* p = new (std::nothrow) struct mla_gqa_prefill_plan();
  if (!p) return MLA_ERR_INVALID_ARG;
  p->dims = d;
  p->B = batch;
  p->T = T;
  p->max_new = most;
  p->order_room = (int32_t)pg::prefill_order_room(T, batch, G);
  p->total = align_up(kHeaderBytes + p->order_room * sizeof(int2), 1024);
  *plan_out = p;
  if (workspace_bytes) *workspace_bytes = p->total;
  return MLA_OK;
}

mla_status_t mla_gqa_prefill_run(mla_gqa_prefill_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                                 int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                                 const int32_t* cu_seqlens_dev, const int32_t* seq_lens_dev, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return prefill_run(plan, q, k_pool, v_pool, num_blocks, block_table, block_table_stride, cu_seqlens_dev, seq_lens_dev,
                     out, workspace, workspace_bytes, stream, Waits{});
}

mla_status_t mla_gqa_prefill_selftest_timeout(mla_gqa_prefill_plan_t plan, const void* q, const void* k_pool,
                                              const void* v_pool, int64_t num_blocks, const int32_t* block_table,
                                              int32_t block_table_stride, const int32_t* cu_seqlens_dev,
                                              const int32_t* seq_lens_dev, void* out, void* workspace,
                                              size_t workspace_bytes, uint64_t wait_limit_ns, void* stream) {
  if (!selftest_limit(wait_limit_ns)) return MLA_ERR_INVALID_ARG;
  return prefill_run(plan, q, k_pool, v_pool, num_blocks, block_table, block_table_stride, cu_seqlens_dev, seq_lens_dev,
                     out, workspace, workspace_bytes, stream, Waits{wait_limit_ns, 1});
}

void mla_gqa_prefill_plan_destroy(mla_gqa_prefill_plan_t plan) { delete plan; }

}  // extern "C"
