"""Torch-tensor wrappers of the paged-cache operators (include/mla_paged.h):
the cache writers, and attention over the grouped-head cache. Marshalling and
argument checks only; every computation runs inside libmla_decode.so.

Every run() works on its tensors' device, on `stream` or that device's current
stream, without synchronising; errors found on the device are read with
read_status(). An object's workspace serves one call in flight: use one object
per stream (or per captured graph) that may overlap with another.
"""

from __future__ import annotations

import contextlib
from typing import Optional, Sequence

from . import _lib as L

_DTYPES = {"bf16": L.MLA_BF16, "fp16": L.MLA_FP16, "fp32": L.MLA_FP32, "fp8": L.MLA_FP8_CACHE}
_STYLES = {"half": L.MLA_ROPE_HALF, "interleaved": L.MLA_ROPE_INTERLEAVED}


def gqa_dims_for(q_heads: int, kv_heads: int, head_dim: int, softmax_scale: float, dtype: str = "bf16",
                 q_len: int = 1, rope_dim: int = 0, rope_style: str = "half", page_size: int = 64) -> L.mla_gqa_dims_t:
    return L.mla_gqa_dims_t(q_heads, kv_heads, head_dim, q_len, page_size, rope_dim, _STYLES[rope_style],
                            _DTYPES[dtype], float(softmax_scale))


def rope_table(positions: int, rope_dim: int, base: float = 10000.0, device="cuda"):
    """The rotation table [positions, rope_dim] of the angles p * base^(-2i / rope_dim): cos in the first half of
    the columns, sin in the second; computed in 64 bits, stored as float32. Other frequencies or scalings: build the
    same layout from their angles."""
    import torch
    inv = float(base) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / max(rope_dim, 1))
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().to(device)


class _Bound:
    """A workspace, its status word and the checks that the classes share."""

    workspace = None
    workspace_bytes = 1024

    def allocate_workspace(self, device, stream: Optional[int] = None):
        """Allocates and clears the workspace on `stream` (default: the device's current stream)."""
        import torch
        device = torch.device(device)
        with torch.cuda.device(device):
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device="cuda")
            if stream is None:
                stream = torch.cuda.current_stream().cuda_stream
            L.mla_workspace_init(self.workspace.data_ptr(), self.workspace_bytes, stream)
        return self

    def read_status(self, stream: Optional[int] = None) -> int:
        """The first error the device recorded since the last call (an mla_status_t), cleared; synchronises."""
        import torch
        with torch.cuda.device(self.workspace.device):
            if stream is None:
                stream = torch.cuda.current_stream().cuda_stream
            return L.mla_decode_read_status(self.workspace.data_ptr(), stream)

    def _enter(self, t, stream):
        """(context that makes t's device current, stream handle), with the workspace in place."""
        import torch
        dev = t.device
        if self.workspace is None:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("allocate_workspace() before capturing: memory allocated under a capture belongs "
                                   "to the graph")
            self.allocate_workspace(dev)
            if stream is not None:  # the allocation and its clearing are ordered on the current stream
                torch.cuda.ExternalStream(stream, device=dev).wait_stream(torch.cuda.current_stream(dev))
        elif self.workspace.device != dev:
            raise ValueError(f"the workspace is on {self.workspace.device}, the tensors on {dev}")
        if stream is None:
            stream = torch.cuda.current_stream(dev).cuda_stream
        here = contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
        return here, stream


def _say(name, t, dtype, shape):
    want = tuple("*" if e is None else e for e in shape)
    return ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, needed: {dtype} {want}")


def _shape(name, t, dtype, shape):
    """dtype and shape of one argument (None: any extent). The C ABI sees bare pointers, so a mismatch is caught here."""
    got = t.shape
    if t.dtype != dtype or len(got) != len(shape):
        raise _say(name, t, dtype, shape)
    for e, n in zip(shape, got):
        if e is not None and e != n:
            raise _say(name, t, dtype, shape)


def _placed(dev, sources, dense) -> None:
    """sources: views whose last dimension is contiguous; dense: contiguous tensors; all on one device."""
    for name, t in dense:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
    for name, t in sources:
        if not t.is_cuda or (t.numel() and t.stride(-1) != 1):
            raise ValueError(f"{name} must be a CUDA tensor with a contiguous last dimension")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")


def _act(code):
    import torch
    return {L.MLA_FP32: torch.float32, L.MLA_FP16: torch.float16}.get(code, torch.bfloat16)


class GqaAppend(_Bound):
    """Appends keys and values to the paged grouped-head cache and rotates keys and queries on the way
    (mla_gqa_append)."""

    def __init__(self, dims: L.mla_gqa_dims_t):
        self.dims = dims
        self._dtype = _act(dims.dtype)

    def run(self, k, v, k_pool, v_pool, block_table, seq_lens, rope_table=None, q=None, q_out=None, cu_seqlens=None,
            stream: Optional[int] = None) -> None:
        """k, v [T, Hk, d] and q [T, Hq, d]: the new tokens before rotation (views whose last dimension is contiguous);
        k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; seq_lens int32 [B] with the new tokens counted;
        rope_table float32 [positions, rope_dim]; q_out [T, Hq, d], the rotated queries; cu_seqlens int32 [B + 1], or
        None: dims.q_len new tokens for every sequence."""
        import torch
        d, act, i32 = self.dims, self._dtype, torch.int32
        T, Hq, Hk, hd = k.shape[0], d.num_q_heads, d.num_kv_heads, d.head_dim
        B = seq_lens.shape[0]
        _shape("k", k, act, (T, Hk, hd))
        _shape("v", v, act, (T, Hk, hd))
        _shape("k_pool", k_pool, act, (None, Hk, d.page_size, hd))
        _shape("v_pool", v_pool, act, k_pool.shape)
        _shape("block_table", block_table, i32, (B, None))
        _shape("seq_lens", seq_lens, i32, (B,))
        sources = [("k", k), ("v", v)]
        dense = [("k_pool", k_pool), ("v_pool", v_pool), ("block_table", block_table), ("seq_lens", seq_lens)]
        if not d.rope_dim:
            rope_table = None
        elif rope_table is None:
            raise ValueError("rope_table is needed: the dims rotate")
        else:
            _shape("rope_table", rope_table, torch.float32, (None, d.rope_dim))
            dense.append(("rope_table", rope_table))
        if cu_seqlens is not None:
            _shape("cu_seqlens", cu_seqlens, i32, (B + 1,))
            dense.append(("cu_seqlens", cu_seqlens))
        elif T != B * d.q_len:
            raise ValueError(f"k: {T} tokens, needed without cu_seqlens: {B} x {d.q_len}")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        if q is not None:
            _shape("q", q, act, (T, Hq, hd))
            _shape("q_out", q_out, act, (T, Hq, hd))
            sources.append(("q", q))
            dense.append(("q_out", q_out))
        _placed(k.device, sources, dense)
        args = L.mla_gqa_append_args_t(
            k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
            *((None, 0, 0, None) if q is None else (q.data_ptr(), q.stride(0), q.stride(1), q_out.data_ptr())),
            k_pool.data_ptr(), v_pool.data_ptr(), k_pool.shape[0], block_table.data_ptr(), block_table.shape[1], B,
            seq_lens.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), T,
            None if rope_table is None else rope_table.data_ptr(), 0 if rope_table is None else rope_table.shape[0])
        here, stream = self._enter(k, stream)
        with here:
            L.mla_gqa_append(d, args, self.workspace.data_ptr(), self.workspace_bytes, stream)


class LatentAppend(_Bound):
    """Appends latent rows to the cache of a DecodePlan with the same dims (bf16, fp32 or FP8) and rotates the RoPE
    key and the queries' RoPE parts on the way (mla_latent_append)."""

    def __init__(self, dims: L.mla_dims_t, rope_style: str = "half"):
        self.dims = dims
        self.style = _STYLES[rope_style]
        self._dtype = _act(dims.dtype)

    def run(self, ckv, k_rope, kv_pool, block_table, seq_lens, rope_table, q_rope=None, q_rope_out=None, kv_rows=None,
            cu_seqlens=None, stream: Optional[int] = None) -> None:
        """ckv [T, r], k_rope [T, D] and q_rope [T, H, D]: the new tokens before rotation (views whose last dimension
        is contiguous); kv_pool [num_blocks, 64, r + D]; block_table int32 [B, *]; seq_lens int32 [B] with the new
        tokens counted; rope_table float32 [positions, D]; q_rope_out [T, H, D]; kv_rows [T, r + D]: also the packed
        rows that PrefillPlan.run reads; cu_seqlens int32 [B + 1], or None: dims.q_len new tokens per sequence."""
        d = self.dims
        if d.dtype == L.MLA_FP8_CACHE:
            raise ValueError("dims of the FP8 cache append with run_fp8")
        _shape("kv_pool", kv_pool, self._dtype, (None, d.page_size, d.latent_rank + d.rope_dim))
        self._run(ckv, k_rope, (("kv_pool", kv_pool),), block_table, seq_lens, rope_table, q_rope, q_rope_out, kv_rows,
                  cu_seqlens, stream)

    def run_fp8(self, ckv, k_rope, kv_codes, kv_rope, kv_scale, block_table, seq_lens, rope_table, q_rope=None,
                q_rope_out=None, kv_rows=None, cu_seqlens=None, stream: Optional[int] = None) -> None:
        """As run, into the three tensors of an FP8 latent cache (kv_codes uint8, kv_rope bfloat16, kv_scale float32:
        the layout of DecodePlan.run_fp8)."""
        import torch
        d = self.dims
        if d.dtype != L.MLA_FP8_CACHE:
            raise ValueError("run_fp8 needs dims made with dtype 'fp8'")
        _shape("kv_codes", kv_codes, torch.uint8, (None, d.page_size, d.latent_rank))
        nb = kv_codes.shape[0]
        _shape("kv_rope", kv_rope, torch.bfloat16, (nb, d.page_size, d.rope_dim))
        _shape("kv_scale", kv_scale, torch.float32, (nb, d.page_size))
        self._run(ckv, k_rope, (("kv_codes", kv_codes), ("kv_rope", kv_rope), ("kv_scale", kv_scale)), block_table,
                  seq_lens, rope_table, q_rope, q_rope_out, kv_rows, cu_seqlens, stream)

    def _run(self, ckv, k_rope, pools, block_table, seq_lens, rope_table, q_rope, q_rope_out, kv_rows, cu_seqlens,
             stream):
        import torch
        d, act, i32 = self.dims, self._dtype, torch.int32
        T, H, r, D = ckv.shape[0], d.num_heads, d.latent_rank, d.rope_dim
        B = seq_lens.shape[0]
        _shape("ckv", ckv, act, (T, r))
        _shape("block_table", block_table, i32, (B, None))
        _shape("seq_lens", seq_lens, i32, (B,))
        sources = [("ckv", ckv)]
        dense = [*pools, ("block_table", block_table), ("seq_lens", seq_lens)]
        if D:
            if k_rope is None or rope_table is None:
                raise ValueError("k_rope and rope_table are needed: the dims rotate")
            _shape("k_rope", k_rope, act, (T, D))
            _shape("rope_table", rope_table, torch.float32, (None, D))
            sources.append(("k_rope", k_rope))
            dense.append(("rope_table", rope_table))
        else:
            k_rope = rope_table = None
        if (q_rope is None) != (q_rope_out is None):
            raise ValueError("q_rope and q_rope_out come together")
        if q_rope is not None:
            _shape("q_rope", q_rope, act, (T, H, D))
            _shape("q_rope_out", q_rope_out, act, (T, H, D))
            sources.append(("q_rope", q_rope))
            dense.append(("q_rope_out", q_rope_out))
        if kv_rows is not None:
            _shape("kv_rows", kv_rows, act, (T, r + D))
            dense.append(("kv_rows", kv_rows))
        if cu_seqlens is not None:
            _shape("cu_seqlens", cu_seqlens, i32, (B + 1,))
            dense.append(("cu_seqlens", cu_seqlens))
        elif T != B * d.q_len:
            raise ValueError(f"ckv: {T} tokens, needed without cu_seqlens: {B} x {d.q_len}")
        _placed(ckv.device, sources, dense)
        pool, rope, scale = [t for _, t in pools] + [None] * (3 - len(pools))
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        args = L.mla_latent_append_args_t(
            ckv.data_ptr(), ckv.stride(0), at(k_rope), 0 if k_rope is None else k_rope.stride(0),
            *((None, 0, 0, None) if q_rope is None else (q_rope.data_ptr(), q_rope.stride(0), q_rope.stride(1),
                                                         q_rope_out.data_ptr())),
            pool.data_ptr(), at(rope), at(scale), at(kv_rows), pool.shape[0], block_table.data_ptr(),
            block_table.shape[1], B, seq_lens.data_ptr(), at(cu_seqlens), T, at(rope_table),
            0 if rope_table is None else rope_table.shape[0])
        here, stream = self._enter(ckv, stream)
        with here:
            L.mla_latent_append(d, self.style, args, self.workspace.data_ptr(), self.workspace_bytes, stream)


class _GqaPlan(_Bound):
    """Owns one plan handle of an attention over the grouped-head cache."""

    handle = None
    _destroy = None

    def _attend(self, q, out, k_pool, v_pool, shape, more):
        import torch
        d, act = self.dims, self._dtype
        _shape("q", q, act, shape)
        _shape("out", out, act, shape)
        _shape("k_pool", k_pool, act, (None, d.num_kv_heads, d.page_size, d.head_dim))
        _shape("v_pool", v_pool, act, k_pool.shape)
        for name, t, extent in more:
            _shape(name, t, torch.int32, extent)
        _placed(q.device, (), (("q", q), ("out", out), ("k_pool", k_pool), ("v_pool", v_pool),
                               *[(name, t) for name, t, _ in more]))

    def close(self) -> None:
        if self.handle:
            type(self)._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GqaDecodePlan(_GqaPlan):
    """Attention of every sequence's newest dims.q_len tokens over the paged grouped-head cache (mla_gqa_decode_run).
    seq_lens_host gives the lengths to balance for; a run's own lengths may differ."""

    _destroy = staticmethod(L.mla_gqa_decode_plan_destroy)

    def __init__(self, dims: L.mla_gqa_dims_t, seq_lens_host: Sequence[int], num_sms: int = 0, num_workers: int = 0):
        self.dims = dims
        self.batch = len(seq_lens_host)
        self._dtype = _act(dims.dtype)
        self.handle, self.workspace_bytes = L.mla_gqa_decode_plan(dims, list(seq_lens_host), num_sms, num_workers)

    def run(self, q, k_pool, v_pool, block_table, seq_lens, out, stream: Optional[int] = None) -> None:
        """q, out [B, Lq, Hq, d]; k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; seq_lens int32 [B],
        the Lq queries' tokens counted: contiguous CUDA tensors."""
        d, B = self.dims, self.batch
        self._attend(q, out, k_pool, v_pool, (B, d.q_len, d.num_q_heads, d.head_dim),
                     (("block_table", block_table, (B, None)), ("seq_lens", seq_lens, (B,))))
        here, stream = self._enter(q, stream)
        with here:
            L.mla_gqa_decode_run(self.handle, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), k_pool.shape[0],
                                 block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), out.data_ptr(),
                                 self.workspace.data_ptr(), self.workspace_bytes, stream)


class GqaPrefillPlan(_GqaPlan):
    """Causal attention of packed prompts over the paged grouped-head cache, which holds their keys and values already
    (mla_gqa_prefill_run)."""

    _destroy = staticmethod(L.mla_gqa_prefill_plan_destroy)

    def __init__(self, dims: L.mla_gqa_dims_t, new_tokens_host: Sequence[int]):
        self.dims = dims
        self.new_tokens = [int(x) for x in new_tokens_host]
        self.tokens = sum(self.new_tokens)
        self._dtype = _act(dims.dtype)
        self.handle, self.workspace_bytes = L.mla_gqa_prefill_plan(dims, self.new_tokens)

    def run(self, q, k_pool, v_pool, block_table, cu_seqlens, seq_lens, out, stream: Optional[int] = None) -> None:
        """q, out [T, Hq, d] packed; k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; cu_seqlens int32
        [B + 1], the prefix sums of the new tokens; seq_lens int32 [B], all tokens: contiguous CUDA tensors."""
        d, B = self.dims, len(self.new_tokens)
        self._attend(q, out, k_pool, v_pool, (self.tokens, d.num_q_heads, d.head_dim),
                     (("block_table", block_table, (B, None)), ("cu_seqlens", cu_seqlens, (B + 1,)),
                      ("seq_lens", seq_lens, (B,))))
        here, stream = self._enter(q, stream)
        with here:
            L.mla_gqa_prefill_run(self.handle, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), k_pool.shape[0],
                                  block_table.data_ptr(), block_table.shape[1], cu_seqlens.data_ptr(),
                                  seq_lens.data_ptr(), out.data_ptr(), self.workspace.data_ptr(), self.workspace_bytes,
                                  stream)
