"""The paged-cache operators as a server runs them: prompts appended and
attended in chunks, then decode steps; and the latent caches written by the
append and read by the MLA prefill and decode."""

import numpy as np
import pytest
import torch

import mla_latent_kv_21_b200 as M
from mla_workloads import WORKLOADS
from oracle import fp8_cache, gqa_oracle, mla_oracle

from harness import assert_close, assert_close_prefill
from harness_paged import block_tables, check_attention, f64, generator

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,Hq,Hk,d", [("bf16", 32, 8, 128), ("fp16", 14, 2, 128), ("bf16", 4, 4, 64)])
def test_gqa_serving(cuda_device, dtype, Hq, Hk, d):
    """Two chunks of every prompt, then three decode steps of one token and one of two, all on one stream without a
    synchronisation in between; every attention against the oracle on the cache's own (rounded) keys."""
    act = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    gen = generator(21)
    B, chunks, steps = 4, [[100, 1, 64, 30], [29, 130, 0, 200]], [1, 1, 2, 1]
    total = [sum(c[b] for c in chunks) + sum(steps) for b in range(B)]
    table, blocks = block_tables(total, gen)
    bt = table.to(cuda_device)
    kp = torch.full((blocks, Hk, 64, d), float("nan"), dtype=act, device=cuda_device)
    vp = kp.clone()
    rope = M.rope_table(max(total), d, device=cuda_device)
    dims = {n: M.gqa_dims_for(Hq, Hk, d, d ** -0.5, dtype, q_len=n, rope_dim=d) for n in (1, 2)}
    append = {n: M.GqaAppend(dims[n]).allocate_workspace(cuda_device) for n in (1, 2)}
    decode = {n: M.GqaDecodePlan(dims[n], total).allocate_workspace(cuda_device) for n in (1, 2)}
    lens, done = [0] * B, []
    for counts, decoding in [(c, False) for c in chunks] + [([n] * B, True) for n in steps]:
        lens = [x + n for x, n in zip(lens, counts)]
        T, n = sum(counts), counts[0]
        qkv = torch.randn((T, Hq + 2 * Hk, d), generator=gen).to(act).to(cuda_device)
        sl = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
        cu = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device=cuda_device)
        q, out = torch.empty((T, Hq, d), dtype=act, device=cuda_device), torch.empty((T, Hq, d), dtype=act, device=cuda_device)
        op = append[n if decoding else 1]
        op.run(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], kp, vp, bt, sl, rope, q=qkv[:, :Hq], q_out=q,
               cu_seqlens=None if decoding else cu)
        if decoding:
            decode[n].run(q.view(B, n, Hq, d), kp, vp, bt, sl, out.view(B, n, Hq, d))
        else:
            plan = M.GqaPrefillPlan(dims[1], counts)
            plan.run(q, kp, vp, bt, cu, sl, out)
        done.append((counts, list(lens), q, out))
    torch.cuda.synchronize(cuda_device)
    assert all(x.read_status() == 0 for x in (*append.values(), *decode.values()))
    for counts, lens, q, out in done:
        at = 0
        for b, (n, L) in enumerate(zip(counts, lens)):
            pages = table[b, :-(-L // 64)].long()
            k, v = (p.cpu()[pages].transpose(1, 2).reshape(-1, Hk, d)[:L] for p in (kp, vp))
            check_attention(out[at:at + n], q[at:at + n], k, v, d ** -0.5, act, f"sequence {b} at {L}")
            at += n


@pytest.mark.parametrize("n", [1, 2])
def test_gqa_steps_with_idle_slots(cuda_device, n):
    """A served batch of fixed slots: some idle, one shorter than the step, filled and emptied between steps; append and
    decode take the same lengths, without an error, and a query without a key gives zeros."""
    Hq, Hk, d, B = 16, 4, 128, 6
    gen = generator(25)
    table, blocks = block_tables([200] * B, gen)
    bt = table.to(cuda_device)
    kp, vp = (torch.randn((blocks, Hk, 64, d), generator=gen).to(torch.bfloat16).to(cuda_device) for _ in range(2))
    rope = M.rope_table(200, d, device=cuda_device)
    dims = M.gqa_dims_for(Hq, Hk, d, d ** -0.5, "bf16", q_len=n, rope_dim=d)
    append = M.GqaAppend(dims).allocate_workspace(cuda_device)
    decode = M.GqaDecodePlan(dims, [100] * B).allocate_workspace(cuda_device)
    done = []
    for lens in ([0, 1, 130, 0, 64, 65], [n, 0, 130 + n, 0, 0, 65 + n], [0] * B):
        qkv = torch.randn((B * n, Hq + 2 * Hk, d), generator=gen).to(torch.bfloat16).to(cuda_device)
        sl = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
        q = torch.full((B * n, Hq, d), float("nan"), dtype=torch.bfloat16, device=cuda_device)
        out = q.clone()
        append.run(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], kp, vp, bt, sl, rope, q=qkv[:, :Hq], q_out=q)
        decode.run(q.view(B, n, Hq, d), kp, vp, bt, sl, out.view(B, n, Hq, d))
        done.append((lens, q, out.view(B, n, Hq, d), kp.clone(), vp.clone()))
    assert append.read_status() == 0 and decode.read_status() == 0
    for lens, q, out, k_now, v_now in done:
        for b, L in enumerate(lens):
            seen = min(n, L)       # the queries with a key
            assert (out[b, :n - seen] == 0).all() and torch.isnan(q.view(B, n, Hq, d)[b, :n - seen]).all()
            if seen:
                pages = table[b, :-(-L // 64)].long()
                k, v = (p.cpu()[pages].transpose(1, 2).reshape(-1, Hk, d)[:L] for p in (k_now, v_now))
                check_attention(out[b, n - seen:], q.view(B, n, Hq, d)[b, n - seen:], k, v, d ** -0.5, torch.bfloat16,
                                f"slot {b} of {lens}")


def _latent_inputs(T, H, gen, device):
    kv = torch.randn((T, 576), generator=gen).to(torch.bfloat16).to(device)
    q = torch.randn((T, H, 192), generator=gen).to(torch.bfloat16).to(device)
    return kv, q


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_latent_prompts_and_decode(cuda_device, dtype):
    """Prompts appended (with the packed rows) and attended by the MLA prefill, then a decode step appended and decoded."""
    wl = WORKLOADS["deepseek_v3"].with_(heads=16)
    gen = generator(22)
    prompts, H = [70, 128, 5], 16
    lens = [n + 1 for n in prompts]
    table, blocks = block_tables(lens, gen, spare=0)
    bt = table.to(cuda_device)
    rope = M.rope_table(200, 64, device=cuda_device)
    w_uk = (torch.randn((H, 128, 512), generator=gen) * 512 ** -0.5).to(torch.bfloat16).to(cuda_device)
    w_uv = (torch.randn((H, 512, 128), generator=gen) * 512 ** -0.5).to(torch.bfloat16).to(cuda_device)
    dims = M.dims_for(H, 512, 64, 128, 128, 1, wl.softmax_scale, dtype)
    append = M.LatentAppend(dims, rope_style="interleaved").allocate_workspace(cuda_device)
    # slots of a partial page that no token fills have to be finite for the latent decode
    if dtype == "fp8":
        pools = (torch.zeros((blocks, 64, 512), dtype=torch.uint8, device=cuda_device),
                 torch.zeros((blocks, 64, 64), dtype=torch.bfloat16, device=cuda_device),
                 torch.zeros((blocks, 64), device=cuda_device))
        put = append.run_fp8
    else:
        pools = (torch.zeros((blocks, 64, 576), dtype=torch.bfloat16, device=cuda_device),)
        put = append.run
    T = sum(prompts)
    kv, q = _latent_inputs(T, H, gen, cuda_device)
    cu = torch.tensor([0] + np.cumsum(prompts).tolist(), dtype=torch.int32, device=cuda_device)
    rows = torch.empty((T, 576), dtype=torch.bfloat16, device=cuda_device)
    q_rope = torch.empty((T, H, 64), dtype=torch.bfloat16, device=cuda_device)
    sl = torch.tensor(prompts, dtype=torch.int32, device=cuda_device)
    put(kv[:, :512], kv[:, 512:], *pools, bt, sl, rope, q_rope=q[:, :, 128:], q_rope_out=q_rope, kv_rows=rows, cu_seqlens=cu)
    q_nope = q[:, :, :128].contiguous()
    out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=cuda_device)
    bf = M.dims_for(H, 512, 64, 128, 128, 1, wl.softmax_scale, "bf16")
    prefill = M.PrefillPlan(bf, prompts).allocate_workspace(cuda_device)
    prefill.run(q_nope, q_rope, rows, cu, w_uk, w_uv, out)
    # the rows hold the latent as it is and the rotated RoPE key
    pos = np.concatenate([np.arange(n) for n in prompts])
    ref_key, size = gqa_oracle.rotate(f64(kv[:, None, 512:]), f64(rope), pos, "interleaved")
    assert torch.equal(rows[:, :512], kv[:, :512])
    assert (np.abs(f64(rows[:, None, 512:]) - ref_key) <= 2.0 ** -8 * np.abs(ref_key) + 2.0 ** -22 * size).all()
    pairs = [(t, h) for t in (0, 69, 70, 150, 197, 198, 202) for h in range(H)]
    ref, mean = mla_oracle.mla_prefill(f64(q_nope), f64(q_rope), f64(rows), cu.tolist(), f64(w_uk), f64(w_uv),
                                       wl.softmax_scale, pairs, abs_weighted=True)
    got = np.stack([f64(out[t, h]) for t, h in pairs])
    assert_close_prefill(got, ref, mean, "prefill of appended prompts")
    # one decode step
    kv1, q1 = _latent_inputs(3, H, gen, cuda_device)
    sl1 = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    q1_rope = torch.empty((3, H, 64), dtype=torch.bfloat16, device=cuda_device)
    put(kv1[:, :512], kv1[:, 512:], *pools, bt, sl1, rope, q_rope=q1[:, :, 128:], q_rope_out=q1_rope)
    assert append.read_status() == 0
    plan = M.DecodePlan(dims, lens).allocate_workspace(cuda_device)
    out1 = torch.empty((3, 1, H, 128), dtype=torch.bfloat16, device=cuda_device)
    args = (q1[:, None, :, :128].contiguous(), q1_rope[:, None], *pools, bt, sl1, w_uk, w_uv, out1)
    (plan.run_fp8 if dtype == "fp8" else plan.run)(*args)
    torch.cuda.synchronize(cuda_device)
    assert plan.read_status() == 0
    ckv, kr = {}, {}
    for b, L in enumerate(lens):
        pages = table[b, :-(-L // 64)].long()
        cut = [p.cpu()[pages].flatten(0, 1)[:L] for p in pools]
        if dtype == "fp8":
            ckv[b], kr[b] = fp8_cache.logical_cache_fp8(cut[0].numpy(), f64(cut[1]), f64(cut[2]))
        else:
            ckv[b], kr[b] = f64(cut[0][:, :512]), f64(cut[0][:, 512:])
    ref1 = mla_oracle.mla_decode(f64(args[0]), f64(args[1]), ckv, kr, f64(w_uk), f64(w_uv), wl.softmax_scale)
    assert_close(f64(out1), ref1, dtype, f"decode over the appended {dtype} cache")
