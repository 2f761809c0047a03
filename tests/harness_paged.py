"""Shared helpers of the paged-cache operators' tests: caches in random page
order with poisoned unused slots, and comparisons with bounds from the rounding
steps.

Attention (u: half a step of the type, eps / 2). The kernels round each weight
p_j once (relative u), which moves an output by at most u sum_j p_j |v_j|, and
the output once (u |ref|). A score is a sum of d products in fp32, each addition
off by at most a step 2^-23 of the running sum (truncating accumulation
included), so its absolute error is at most d 2^-23 S, S = the largest
scale sum |q k| of the row, and twice that is the relative error of a
normalised weight; the exponential and the fp32 sums of up to 2^20 terms in
blocks add less than 2^-18. fp16 weights below the normal range have an
absolute step 2^-24 relative to a largest weight of 1 (half of it is the
error): n 2^-25 sum |v| / L is bounded with max|v|.

Rotation: two products and a sum in fp32, 3 roundings of 2^-24 of the products'
size, then one rounding to the type.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import gqa_oracle

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def generator(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


def block_tables(lens, gen, spare=3, width=None):
    """(int32 [B, width] with -1 for unused entries, number of blocks): pages in random order, `spare` blocks unused."""
    need = [-(-n // PAGE) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).tolist()
    width = max(1, max(need)) if width is None else width
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    return table, total


def paged_kv(lens, heads, d, dtype, gen, table, blocks, fill=float("nan")):
    """(k_pool, v_pool, per-sequence (k, v) [L, heads, d]); slots without a token hold `fill`."""
    kp = torch.full((blocks, heads, PAGE, d), fill, dtype=dtype)
    vp = torch.full((blocks, heads, PAGE, d), fill, dtype=dtype)
    seqs = []
    for b, n in enumerate(lens):
        k = torch.randn((n, heads, d), generator=gen).to(dtype)
        v = torch.randn((n, heads, d), generator=gen).to(dtype)
        for j in range(0, n, PAGE):
            e = min(n, j + PAGE)
            kp[table[b, j // PAGE], :, :e - j] = k[j:e].transpose(0, 1)
            vp[table[b, j // PAGE], :, :e - j] = v[j:e].transpose(0, 1)
        seqs.append((k, v))
    return kp, vp, seqs


def f64(t) -> np.ndarray:
    return t.double().cpu().numpy()


def check_attention(got, q, k, v, scale, dtype, what=""):
    """got, q [n, Hq, d], k, v [L, Hk, d] of one sequence."""
    ref, mean, size = gqa_oracle.attend(f64(q), f64(k), f64(v), scale)
    got = f64(got)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    u, d = half_step(dtype), q.shape[-1]
    rel = (u + 2.0 * (d * 2.0 ** -23 * size + 2.0 ** -18))[..., None]
    bound = u * np.abs(ref) + rel * mean
    if dtype == torch.float16:
        bound = bound + k.shape[0] * 2.0 ** -25 * (np.abs(f64(v)).max() if v.numel() else 0.0) + 2.0 ** -25
    off = np.abs(got - ref)
    assert (off <= bound + 1e-30).all(), (
        f"{what}: max |got - ref| {off.max():.3e}, worst ratio to its bound {(off / (bound + 1e-30)).max():.3f}")


def check_rotated(got, x, table, positions, style, dtype, what=""):
    ref, size = gqa_oracle.rotate(f64(x), f64(table), np.asarray(positions), style)
    off = np.abs(f64(got) - ref)
    bound = half_step(dtype) * np.abs(ref) + 3 * 2.0 ** -24 * size * (1 + half_step(dtype))
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25   # subnormal results
    assert (off <= bound).all(), f"{what}: worst ratio to its bound {(off / np.maximum(bound, 1e-300)).max():.3f}"


def same_bits(a, b) -> bool:
    view = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))
