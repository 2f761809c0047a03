"""Latent decode steps directly behind kernels that let them be placed early.

A decode step is three programmatic launches. The combine waits for no grid: it
reads the absorb kernel's prefix sums, length flag and cleared segment counts,
and must not start before they are this step's. Here a long kernel of few blocks
(a short chunk attended over a long grouped-head cache) or the cache's writer
runs ahead on the same stream, with no other launch and no synchronisation in
between, first over a fresh workspace and then with other lengths and inputs;
16 heads and few pages leave most SMs free, so that nothing but the waits keeps
the kernels in order. Every element against the oracle.
"""

import numpy as np
import pytest
import torch

import mla_latent_kv_21_b200 as M
from mla_workloads import WORKLOADS, generate
from oracle import fp8_cache, mla_oracle

from harness import assert_close, dims_of, oracle_out, to_device
from harness_paged import f64

pytestmark = pytest.mark.gpu

WL = {"bf16": WORKLOADS["deepseek_v3"].with_(heads=16), "fp8": WORKLOADS["deepseek_v3_fp8"].with_(heads=16)}
STEPS = [[70, 130, 5], [300, 64, 129], [1, 700, 33]]


class LongChunk:
    """16 new tokens over a long cache: 8 items, one block each, a few hundred steps of keys."""

    def __init__(self, device, cached=40000):
        dims = M.gqa_dims_for(8, 8, 128, 128 ** -0.5, "bf16")
        gen = torch.Generator(device=device).manual_seed(3)
        self.q = torch.randn((16, 8, 128), device=device, generator=gen).to(torch.bfloat16)
        self.pools = [torch.randn((32, 8, 64, 128), device=device, generator=gen).to(torch.bfloat16) for _ in range(2)]
        self.bt = (torch.arange(-(-cached // 64), device=device, dtype=torch.int32) % 32)[None].contiguous()
        self.cu = torch.tensor([0, 16], dtype=torch.int32, device=device)
        self.sl = torch.tensor([cached], dtype=torch.int32, device=device)
        self.out = torch.empty_like(self.q)
        self.plan = M.GqaPrefillPlan(dims, [16]).allocate_workspace(device)

    def run(self):
        self.plan.run(self.q, *self.pools, self.bt, self.cu, self.sl, self.out)


def _pools(dev, dtype):
    return [dev[n] for n in (("kv_codes", "kv_rope", "kv_scale") if dtype == "fp8" else ("kv_pool",))]


def _decode(plan, dev, dtype, out, q_rope=None):
    q_rope = dev["q_rope"] if q_rope is None else q_rope
    run = plan.run_fp8 if dtype == "fp8" else plan.run
    run(dev["q_nope"], q_rope, *_pools(dev, dtype), dev["block_table"], dev["seq_lens"], dev["w_uk"], dev["w_uv"], out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("ahead", ["chunk", "step"])
def test_decode_behind_a_long_kernel_or_another_step(cuda_device, dtype, ahead):
    wl = WL[dtype]
    plan = M.DecodePlan(dims_of(wl), [300] * 3)
    chunk = LongChunk(cuda_device)
    inputs = [generate(wl.with_(seed=40 + i), seq_lens=lens) for i, lens in enumerate(STEPS)]
    devs = [to_device(x, cuda_device) for x in inputs]
    outs = [torch.full((3, 1, 16, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device) for _ in STEPS]
    plan.allocate_workspace(cuda_device)
    torch.cuda.synchronize(cuda_device)
    if ahead == "step":
        chunk.run()
    for dev, out in zip(devs, outs):
        if ahead == "chunk":
            chunk.run()
        _decode(plan, dev, dtype, out)
    torch.cuda.synchronize(cuda_device)
    assert plan.read_status() == 0 and chunk.plan.read_status() == 0
    for i, (x, out) in enumerate(zip(inputs, outs)):
        assert_close(f64(out), oracle_out(wl, x), dtype, f"step {i} behind a {ahead}")
    plan.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_decode_behind_the_cache_writer(cuda_device, dtype):
    """Each step appends a token to every sequence and decodes, directly behind each other."""
    wl = WL[dtype]
    dims, lens = dims_of(wl), [70, 127, 5]
    inputs = generate(wl, seq_lens=[n + 8 for n in lens])
    dev = to_device(inputs, cuda_device)
    for pool in _pools(dev, dtype):
        pool.zero_()
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    append = M.LatentAppend(dims, rope_style="interleaved").allocate_workspace(cuda_device)
    plan = M.DecodePlan(dims, lens).allocate_workspace(cuda_device)
    rope = M.rope_table(256, 64, device=cuda_device)
    put = append.run_fp8 if dtype == "fp8" else append.run
    # the cached tokens, as packed prompts
    T = sum(lens)
    kv = torch.randn((T, 576), device=cuda_device, generator=gen).to(torch.bfloat16)
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device=cuda_device)
    sl = [torch.tensor([n + i for n in lens], dtype=torch.int32, device=cuda_device) for i in range(4)]
    steps = []
    for i in range(1, 4):
        steps.append(dict(kv=torch.randn((3, 576), device=cuda_device, generator=gen).to(torch.bfloat16), sl=sl[i],
                          q=torch.randn((3, 16, 64), device=cuda_device, generator=gen).to(torch.bfloat16),
                          q_out=torch.full((3, 16, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device),
                          out=torch.full((3, 1, 16, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)))
    chunk = LongChunk(cuda_device)
    torch.cuda.synchronize(cuda_device)
    chunk.run()
    put(kv[:, :512], kv[:, 512:], *_pools(dev, dtype), dev["block_table"], sl[0], rope, cu_seqlens=cu)
    for s in steps:
        put(s["kv"][:, :512], s["kv"][:, 512:], *_pools(dev, dtype), dev["block_table"], s["sl"], rope, q_rope=s["q"],
            q_rope_out=s["q_out"])
        _decode(plan, dict(dev, seq_lens=s["sl"]), dtype, s["out"], s["q_out"][:, None])
    torch.cuda.synchronize(cuda_device)
    assert plan.read_status() == 0 and append.read_status() == 0
    table = inputs["block_table"]
    for i, s in enumerate(steps):
        ckv, kr = {}, {}
        for b, L in enumerate(s["sl"].tolist()):
            pages = table[b, :-(-L // 64)].long()
            cut = [p.cpu()[pages].flatten(0, 1)[:L] for p in _pools(dev, dtype)]
            if dtype == "fp8":
                ckv[b], kr[b] = fp8_cache.logical_cache_fp8(cut[0].numpy(), f64(cut[1]), f64(cut[2]))
            else:
                ckv[b], kr[b] = f64(cut[0][:, :512]), f64(cut[0][:, 512:])
        ref = mla_oracle.mla_decode(f64(inputs["q_nope"]), f64(s["q_out"][:, None]), ckv, kr, f64(inputs["w_uk"]),
                                    f64(inputs["w_uv"]), wl.softmax_scale)
        assert_close(f64(s["out"]), ref, dtype, f"appended step {i}")
    plan.close()
