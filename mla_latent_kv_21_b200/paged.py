"""Torch-tensor wrappers of the paged-cache operators (include/mla_paged.h):
the cache writers, and attention over the grouped-head cache. Marshalling and
argument checks only; every computation runs inside libmla_decode.so.

Every run() works on its tensors' device, on `stream` or that device's current
stream, without synchronising; errors found on the device are read with
read_status(). An object's workspace serves one call in flight: use one object
per stream (or per captured graph) that may overlap with another. An object may
be dropped while its call runs, but not while a graph that captured one lives.
"""

from __future__ import annotations

from typing import Optional, Sequence

from . import _lib as L
from ._workspace import Workspace

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


class _Bound(Workspace):
    """A workspace and the launch that the classes share."""

    def _launch(self, dev: int, stream, call, *args) -> None:
        """call(*args, workspace, workspace bytes, stream) with device `dev` current."""
        import torch
        stream = self._stream(dev, stream)
        if dev == torch.cuda.current_device():
            call(*args, self._at[1], self.workspace_bytes, stream)
        else:
            with torch.cuda.device(dev):
                call(*args, self._at[1], self.workspace_bytes, stream)


def _check(dev: int, sources, dense) -> None:
    """(name, tensor, dtype, shape) of every argument: `dense` contiguous, `sources` views whose last dimension is; all
    on device `dev`. The C ABI sees bare pointers, so a mismatch is caught here."""
    ok = dev >= 0
    for _, t, dtype, shape in dense:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            ok = False
    for _, t, dtype, shape in sources:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or (t.stride()[-1] != 1 and t.numel()):
            ok = False
    if ok:
        return
    for name, t, dtype, shape in (*sources, *dense):
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, needed: {dtype} {tuple(shape)}")
    for name, t, _, _ in dense:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    for name, t, _, _ in sources:
        if not t.is_cuda or t.stride(-1) != 1:
            raise ValueError(f"{name} must be a CUDA tensor with a contiguous last dimension")
    names = ", ".join(f"{name} on {t.device}" for name, t, _, _ in (*sources, *dense))
    raise ValueError(f"the tensors are not on one device: {names}")


def _act(code):
    import torch
    return {L.MLA_FP32: torch.float32, L.MLA_FP16: torch.float16}.get(code, torch.bfloat16)


class GqaAppend(_Bound):
    """Appends keys and values to the paged grouped-head cache and rotates keys and queries on the way
    (mla_gqa_append)."""

    def __init__(self, dims: L.mla_gqa_dims_t):
        self.dims = dims
        self._dtype = _act(dims.dtype)
        self._sizes = dims.num_q_heads, dims.num_kv_heads, dims.head_dim, dims.rope_dim, dims.page_size

    def run(self, k, v, k_pool, v_pool, block_table, seq_lens, rope_table=None, q=None, q_out=None, cu_seqlens=None,
            stream: Optional[int] = None) -> None:
        """k, v [T, Hk, d] and q [T, Hq, d]: the new tokens before rotation (views whose last dimension is contiguous);
        k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; seq_lens int32 [B] with the new tokens counted;
        rope_table float32 [positions, rope_dim]; q_out [T, Hq, d], the rotated queries; cu_seqlens int32 [B + 1], or
        None: dims.q_len new tokens for every sequence (where the cache holds fewer, 0 in an idle slot, its last ones)."""
        import torch
        d, act, i32 = self.dims, self._dtype, torch.int32
        Hq, Hk, hd, D, P = self._sizes
        T, B, pool = k.shape[0], seq_lens.shape[0], (k_pool.shape[0], Hk, P, hd)
        width = block_table.shape[-1]
        sources = [("k", k, act, (T, Hk, hd)), ("v", v, act, (T, Hk, hd))]
        dense = [("k_pool", k_pool, act, pool), ("v_pool", v_pool, act, pool), ("block_table", block_table, i32, (B, width)),
                 ("seq_lens", seq_lens, i32, (B,))]
        q_args, cu, table, positions = (None, 0, 0, None), None, None, 0
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        if D and rope_table is None:
            raise ValueError("rope_table is needed: the dims rotate")
        if D:
            positions = rope_table.shape[0]
            dense.append(("rope_table", rope_table, torch.float32, (positions, D)))
            table = rope_table.data_ptr()
        if cu_seqlens is not None:
            dense.append(("cu_seqlens", cu_seqlens, i32, (B + 1,)))
            cu = cu_seqlens.data_ptr()
        if q is not None:
            sources.append(("q", q, act, (T, Hq, hd)))
            dense.append(("q_out", q_out, act, (T, Hq, hd)))
        dev = k.get_device()
        if cu is None and T != B * d.q_len:
            raise ValueError(f"k: {T} tokens, needed without cu_seqlens: {B} x {d.q_len}")
        _check(dev, sources, dense)
        if q is not None:
            q_args = (q.data_ptr(), *q.stride()[:2], q_out.data_ptr())
        args = L.mla_gqa_append_args_t(k.data_ptr(), *k.stride()[:2], v.data_ptr(), *v.stride()[:2], *q_args,
                                       k_pool.data_ptr(), v_pool.data_ptr(), pool[0], block_table.data_ptr(), width, B,
                                       seq_lens.data_ptr(), cu, T, table, positions)
        self._launch(dev, stream, L.mla_gqa_append, d, args)


class LatentAppend(_Bound):
    """Appends latent rows to the cache of a DecodePlan with the same dims (bf16, fp32 or FP8) and rotates the RoPE
    key and the queries' RoPE parts on the way (mla_latent_append). Clear a fresh pool once: the latent decode needs
    the unused slots of a page finite."""

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
        pools = [("kv_pool", kv_pool, self._dtype, (kv_pool.shape[0], d.page_size, d.latent_rank + d.rope_dim))]
        self._run(ckv, k_rope, pools, block_table, seq_lens, rope_table, q_rope, q_rope_out, kv_rows, cu_seqlens, stream)

    def run_fp8(self, ckv, k_rope, kv_codes, kv_rope, kv_scale, block_table, seq_lens, rope_table, q_rope=None,
                q_rope_out=None, kv_rows=None, cu_seqlens=None, stream: Optional[int] = None) -> None:
        """As run, into the three tensors of an FP8 latent cache (kv_codes uint8, kv_rope bfloat16, kv_scale float32:
        the layout of DecodePlan.run_fp8)."""
        import torch
        d = self.dims
        if d.dtype != L.MLA_FP8_CACHE:
            raise ValueError("run_fp8 needs dims made with dtype 'fp8'")
        nb, P = kv_codes.shape[0], d.page_size
        pools = [("kv_codes", kv_codes, torch.uint8, (nb, P, d.latent_rank)),
                 ("kv_rope", kv_rope, torch.bfloat16, (nb, P, d.rope_dim)), ("kv_scale", kv_scale, torch.float32, (nb, P))]
        self._run(ckv, k_rope, pools, block_table, seq_lens, rope_table, q_rope, q_rope_out, kv_rows, cu_seqlens, stream)

    def _run(self, ckv, k_rope, pools, block_table, seq_lens, rope_table, q_rope, q_rope_out, kv_rows, cu_seqlens,
             stream):
        import torch
        d, act, i32 = self.dims, self._dtype, torch.int32
        H, r, D = d.num_heads, d.latent_rank, d.rope_dim
        T, B, width = ckv.shape[0], seq_lens.shape[0], block_table.shape[-1]
        sources = [("ckv", ckv, act, (T, r))]
        dense = [*pools, ("block_table", block_table, i32, (B, width)), ("seq_lens", seq_lens, i32, (B,))]
        if (q_rope is None) != (q_rope_out is None):
            raise ValueError("q_rope and q_rope_out come together")
        if D and (k_rope is None or rope_table is None):
            raise ValueError("k_rope and rope_table are needed: the dims rotate")
        if D:
            sources.append(("k_rope", k_rope, act, (T, D)))
            dense.append(("rope_table", rope_table, torch.float32, (rope_table.shape[0], D)))
        if q_rope is not None:
            sources.append(("q_rope", q_rope, act, (T, H, D)))
            dense.append(("q_rope_out", q_rope_out, act, (T, H, D)))
        if kv_rows is not None:
            dense.append(("kv_rows", kv_rows, act, (T, r + D)))
        if cu_seqlens is not None:
            dense.append(("cu_seqlens", cu_seqlens, i32, (B + 1,)))
        if cu_seqlens is None and T != B * d.q_len:
            raise ValueError(f"ckv: {T} tokens, needed without cu_seqlens: {B} x {d.q_len}")
        dev = ckv.get_device()
        _check(dev, sources, dense)
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        key = (k_rope.data_ptr(), k_rope.stride(0)) if D else (None, 0)
        q_args = (None, 0, 0, None) if q_rope is None else (q_rope.data_ptr(), *q_rope.stride()[:2], q_rope_out.data_ptr())
        out = [t.data_ptr() for _, t, _, _ in pools] + [None] * (3 - len(pools))
        table = (rope_table.data_ptr(), rope_table.shape[0]) if D else (None, 0)
        args = L.mla_latent_append_args_t(ckv.data_ptr(), ckv.stride(0), *key, *q_args, *out, at(kv_rows),
                                          pools[0][3][0], block_table.data_ptr(), width, B,
                                          seq_lens.data_ptr(), at(cu_seqlens), T, *table)
        self._launch(dev, stream, L.mla_latent_append, d, self.style, args)


class _GqaPlan(_Bound):
    """Owns one plan handle of an attention over the grouped-head cache."""

    handle = None
    _destroy = None

    def _attend(self, run, stream, q, out, k_pool, v_pool, block_table, *lengths):
        """The checks and the call; lengths: (name, tensor, dtype, shape) in the call's order."""
        import torch
        act = self._dtype
        blocks, width = k_pool.shape[0], block_table.shape[-1]
        pool = (blocks, *self._page)
        dev = q.get_device()
        _check(dev, (), (("q", q, act, self._rows), ("out", out, act, self._rows), ("k_pool", k_pool, act, pool),
                         ("v_pool", v_pool, act, pool), ("block_table", block_table, torch.int32, (self.batch, width)),
                         *lengths))
        self._launch(dev, stream, run, self.handle, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), blocks,
                     block_table.data_ptr(), width, *[x[1].data_ptr() for x in lengths], out.data_ptr())

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
        self._rows = self.batch, dims.q_len, dims.num_q_heads, dims.head_dim
        self._page = dims.num_kv_heads, dims.page_size, dims.head_dim
        self.handle, self.workspace_bytes = L.mla_gqa_decode_plan(dims, list(seq_lens_host), num_sms, num_workers)

    def run(self, q, k_pool, v_pool, block_table, seq_lens, out, stream: Optional[int] = None) -> None:
        """q, out [B, Lq, Hq, d]; k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; seq_lens int32 [B],
        the Lq queries' tokens counted: contiguous CUDA tensors."""
        import torch
        self._attend(L.mla_gqa_decode_run, stream, q, out, k_pool, v_pool, block_table,
                     ("seq_lens", seq_lens, torch.int32, (self.batch,)))


class GqaPrefillPlan(_GqaPlan):
    """Causal attention of packed prompts over the paged grouped-head cache, which holds their keys and values already
    (mla_gqa_prefill_run)."""

    _destroy = staticmethod(L.mla_gqa_prefill_plan_destroy)

    def __init__(self, dims: L.mla_gqa_dims_t, new_tokens_host: Sequence[int]):
        self.dims = dims
        self.new_tokens = [int(x) for x in new_tokens_host]
        self.batch, self.tokens = len(self.new_tokens), sum(self.new_tokens)
        self._dtype = _act(dims.dtype)
        self._rows = self.tokens, dims.num_q_heads, dims.head_dim
        self._page = dims.num_kv_heads, dims.page_size, dims.head_dim
        self.handle, self.workspace_bytes = L.mla_gqa_prefill_plan(dims, self.new_tokens)

    def run(self, q, k_pool, v_pool, block_table, cu_seqlens, seq_lens, out, stream: Optional[int] = None) -> None:
        """q, out [T, Hq, d] packed; k_pool, v_pool [num_blocks, Hk, 64, d]; block_table int32 [B, *]; cu_seqlens int32
        [B + 1], the prefix sums of the new tokens; seq_lens int32 [B], all tokens: contiguous CUDA tensors."""
        import torch
        self._attend(L.mla_gqa_prefill_run, stream, q, out, k_pool, v_pool, block_table,
                     ("cu_seqlens", cu_seqlens, torch.int32, (self.batch + 1,)), ("seq_lens", seq_lens, torch.int32, (self.batch,)))
