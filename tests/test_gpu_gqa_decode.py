"""Decode attention over the paged grouped-head cache against the 64-bit oracle,
every element, with bounds from the rounding steps (harness_paged). Unused slots
and the slots behind a sequence's end hold NaN."""

import pytest
import torch

import mla_latent_kv_21_b200 as M

from harness_paged import TYPES, block_tables, check_attention, generator, paged_kv

pytestmark = pytest.mark.gpu


def _inputs(lens, Hk, G, d, Lq, dtype, seed, device, fill=float("nan"), q_std=1.0, width=None):
    gen = generator(seed)
    table, blocks = block_tables(lens, gen, width=width)
    kp, vp, seqs = paged_kv(lens, Hk, d, dtype, gen, table, blocks, fill)
    q = (torch.randn((len(lens), Lq, Hk * G, d), generator=gen) * q_std).to(dtype)
    dev = dict(q=q.to(device), kp=kp.to(device), vp=vp.to(device), bt=table.to(device),
               sl=torch.tensor(lens, dtype=torch.int32, device=device))
    return dev, q, seqs


def _run(plan, dev, out, stream=None):
    plan.run(dev["q"], dev["kp"], dev["vp"], dev["bt"], dev["sl"], out, stream=stream)


def _dims(Hk, G, d, Lq, dtype):
    return M.gqa_dims_for(Hk * G, Hk, d, d ** -0.5, dtype, q_len=Lq)


def _check(out, q, seqs, d, dtype, what):
    for b, (k, v) in enumerate(seqs):
        check_attention(out[b], q[b], k, v, d ** -0.5, TYPES[dtype], f"{what}, sequence {b}")


RAGGED = [1, 63, 64, 65, 0, 127, 128, 129, 700, 1000, 5, 0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk,G,Lq", [(2, 4, 1), (1, 1, 1), (3, 1, 2), (1, 7, 1), (2, 8, 2), (1, 16, 1), (1, 5, 4),
                                     (2, 12, 3), (1, 64, 1), (2, 8, 8)])
def test_ragged_batches(cuda_device, dtype, d, Hk, G, Lq):
    dev, q, seqs = _inputs(RAGGED, Hk, G, d, Lq, TYPES[dtype], Hk * 100 + G, cuda_device)
    for workers in (0, 1, 5):
        plan = M.GqaDecodePlan(_dims(Hk, G, d, Lq, dtype), RAGGED, num_workers=workers).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        _check(out, q, seqs, d, dtype, f"{workers} workers")
        plan.close()


@pytest.mark.parametrize("lens", [[1], [64], [200], [5000], [0, 0, 9000], [300] * 70, [1] * 300])
def test_splits(cuda_device, lens):
    """One short or long sequence, many equal ones: the split over the length from none to many parts."""
    dev, q, seqs = _inputs(lens, 2, 4, 128, 1, torch.bfloat16, len(lens), cuda_device)
    for workers in (0, 3, 97):
        plan = M.GqaDecodePlan(_dims(2, 4, 128, 1, "bf16"), lens, num_workers=workers).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        again = torch.full_like(out, float("nan"))
        _run(plan, dev, again)
        assert plan.read_status() == 0 and torch.equal(out, again)
        _check(out, q, seqs, 128, "bf16", f"{workers} workers")
        plan.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_std", [0.0, 30.0])
def test_flat_and_peaked_scores(cuda_device, dtype, q_std):
    """Equal weights, and scores hundreds apart (one key takes all the weight, the running maximum moves far)."""
    lens = [1000, 77, 4000]
    dev, q, seqs = _inputs(lens, 2, 4, 128, 2, TYPES[dtype], 5, cuda_device, q_std=q_std)
    plan = M.GqaDecodePlan(_dims(2, 4, 128, 2, dtype), lens, num_workers=7).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    assert plan.read_status() == 0
    _check(out, q, seqs, 128, dtype, "scores")


def test_growing_scores(cuda_device):
    """Keys whose scores rise with the position, so that the running maximum moves in every tile."""
    lens, d = [1500], 128
    dev, q, seqs = _inputs(lens, 1, 4, d, 1, torch.bfloat16, 6, cuda_device)
    k, v = seqs[0]
    u = torch.ones(d)
    k += (torch.arange(1500)[:, None, None] * 0.02 * u).to(k.dtype)
    q[:] = u.to(q.dtype)
    dev["q"].copy_(q)
    for j in range(0, 1500, 64):
        e = min(1500, j + 64)
        dev["kp"][dev["bt"][0, j // 64], :, :e - j] = k[j:e].transpose(0, 1).to(cuda_device)
    plan = M.GqaDecodePlan(_dims(1, 4, d, 1, "bf16"), lens, num_workers=2).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    _check(out, q, seqs, d, "bf16", "growing")


def test_plan_lengths_affect_balance_only(cuda_device):
    lens = [500, 0, 1200, 64]
    dev, q, seqs = _inputs(lens, 2, 2, 128, 1, torch.bfloat16, 8, cuda_device, width=40)
    for planned in ([1, 1, 1, 1], [2000, 2000, 2000, 2000], [0, 0, 0, 0]):
        plan = M.GqaDecodePlan(_dims(2, 2, 128, 1, "bf16"), planned).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        _check(out, q, seqs, 128, "bf16", f"planned {planned}")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("Hk,G,Lq", [(2, 4, 1), (1, 16, 1), (2, 5, 3)])
def test_both_layouts_of_the_warps(cuda_device, dtype, d, Hk, G, Lq):
    """Plans for short, medium and long segments choose how the warps share a page; each with the same ragged lengths."""
    lens = [1, 63, 64, 65, 0, 700, 2000, 5]
    dev, q, seqs = _inputs(lens, Hk, G, d, Lq, TYPES[dtype], 17, cuda_device)
    for planned, workers in ((64, 0), (64 * 8, 1), (64 * 10, 3), (64 * 200, 5), (64 * 200, 300)):
        plan = M.GqaDecodePlan(_dims(Hk, G, d, Lq, dtype), [planned] * len(lens), num_workers=workers)
        plan.allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        _check(out, q, seqs, d, dtype, f"planned {planned}, {workers} workers")
        plan.close()


def test_many_sequences(cuda_device):
    """More sequences than a worker has threads, many of them idle."""
    lens = [(b * 37) % 150 if b % 3 else 0 for b in range(2500)]
    dev, q, seqs = _inputs(lens, 1, 2, 64, 1, torch.float16, 18, cuda_device)
    for workers in (0, 2):
        plan = M.GqaDecodePlan(_dims(1, 2, 64, 1, "fp16"), lens, num_workers=workers).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        host = out.cpu()
        for b, (k, v) in enumerate(seqs):
            check_attention(host[b], q[b], k, v, 64 ** -0.5, torch.float16, f"{workers} workers, sequence {b}")
        plan.close()


@pytest.mark.parametrize("Hk,G,Lq", [(1, 4, 1), (2, 16, 2)])
def test_as_many_workers_as_pages(cuda_device, Hk, G, Lq):
    """An item of many parts: the join looks through more workers than a warp has lanes."""
    lens = [40000, 100]
    dev, q, seqs = _inputs(lens, Hk, G, 128, Lq, torch.bfloat16, 19, cuda_device)
    for workers in (4096, 500, 70):
        plan = M.GqaDecodePlan(_dims(Hk, G, 128, Lq, "bf16"), lens, num_workers=workers).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        _check(out, q, seqs, 128, "bf16", f"{workers} workers")
        plan.close()


def test_bad_lengths_and_blocks_are_recorded(cuda_device):
    """A length past the table or below zero counts as 0; a page whose block is out of range is not seen; the other
    sequences are right."""
    lens = [100, 200, 300]
    dev, q, seqs = _inputs(lens, 2, 4, 128, 1, torch.bfloat16, 9, cuda_device)
    plan = M.GqaDecodePlan(_dims(2, 4, 128, 1, "bf16"), lens).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    for bad in (-1, 64 * dev["bt"].shape[1] + 1, 2 ** 31 - 1):
        dev["sl"][1] = bad
        _run(plan, dev, out)
        assert plan.read_status() == M.MLA_ERR_BOUNDS
        assert plan.read_status() == 0
        assert (out[1] == 0).all()
        for b in (0, 2):
            check_attention(out[b], q[b], *seqs[b], 128 ** -0.5, torch.bfloat16, f"sequence {b}")
    dev["sl"][1] = 200
    for bad in (-1, dev["kp"].shape[0], 2 ** 31 - 1):
        keep = dev["bt"][2, 1].clone()
        dev["bt"][2, 1] = bad
        _run(plan, dev, out)
        assert plan.read_status() == M.MLA_ERR_BOUNDS
        dev["bt"][2, 1] = keep
        for b in (0, 1):
            check_attention(out[b], q[b], *seqs[b], 128 ** -0.5, torch.bfloat16, f"sequence {b}")
        k, v = seqs[2]
        seen = torch.tensor([j for j in range(300) if j // 64 != 1])
        check_attention(out[2], q[2], k[seen], v[seen], 128 ** -0.5, torch.bfloat16, "the pages that remain")
    dev["bt"][2, :] = -1
    _run(plan, dev, out)
    assert plan.read_status() == M.MLA_ERR_BOUNDS and (out[2] == 0).all()


def test_offsets_past_32_bits(cuda_device):
    """Pages whose element offsets lie past 2^31 (and byte offsets past 2^32)."""
    lens, Hk, d = [150, 64], 8, 128
    blocks = 2 ** 31 // (Hk * 64 * d) + 40
    dev, q, seqs = _inputs(lens, Hk, 2, d, 1, torch.bfloat16, 10, cuda_device)
    big = torch.empty((2, blocks, Hk, 64, d), dtype=torch.bfloat16, device=cuda_device)
    small = dev["kp"].shape[0]
    big[0, -small:], big[1, -small:] = dev["kp"], dev["vp"]
    table = torch.where(dev["bt"] >= 0, dev["bt"] + (blocks - small), -1).to(torch.int32)
    plan = M.GqaDecodePlan(_dims(Hk, 2, d, 1, "bf16"), lens).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    plan.run(dev["q"], big[0], big[1], table, dev["sl"], out)
    assert plan.read_status() == 0
    _check(out, q, seqs, d, "bf16", "far pages")


def test_streams_graphs_and_two_plans(cuda_device):
    """A captured step replayed with other lengths and queries in the same buffers; two plans on two streams at once."""
    lens = [700, 65, 300, 0, 2048]
    dev, q, seqs = _inputs(lens, 2, 4, 128, 1, torch.bfloat16, 11, cuda_device)
    dims = _dims(2, 4, 128, 1, "bf16")
    plan = M.GqaDecodePlan(dims, lens).allocate_workspace(cuda_device)
    other = M.GqaDecodePlan(dims, lens, num_workers=9).allocate_workspace(cuda_device)
    out, out2 = torch.zeros_like(dev["q"]), torch.zeros_like(dev["q"])
    side = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize(cuda_device)
    for _ in range(20):
        _run(plan, dev, out)
        _run(other, dev, out2, stream=side.cuda_stream)
    torch.cuda.synchronize(cuda_device)
    _check(out, q, seqs, 128, "bf16", "current stream")
    _check(out2, q, seqs, 128, "bf16", "other stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(plan, dev, out)
    for seed in (12, 13):
        new, q, seqs = _inputs([x for x in (64, 700, 0, 30, 1999)] if seed == 13 else lens, 2, 4, 128, 1, torch.bfloat16, seed,
                               cuda_device, width=dev["bt"].shape[1])
        n = min(new["kp"].shape[0], dev["kp"].shape[0])
        assert n == new["kp"].shape[0]
        dev["kp"][:n], dev["vp"][:n] = new["kp"], new["vp"]
        for name in ("q", "bt", "sl"):
            dev[name].copy_(new[name])
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize(cuda_device)
        assert plan.read_status() == 0
        _check(out, q, seqs, 128, "bf16", "replay")
    del g


def test_first_run_inside_a_capture_is_refused_without_a_workspace(cuda_device):
    lens = [10]
    dev, _, _ = _inputs(lens, 1, 1, 64, 1, torch.bfloat16, 14, cuda_device)
    plan = M.GqaDecodePlan(_dims(1, 1, 64, 1, "bf16"), lens)
    out = torch.zeros_like(dev["q"])
    x = torch.zeros(4, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x += 1
        with pytest.raises(RuntimeError, match="allocate_workspace"):
            _run(plan, dev, out)
    del g
    _run(plan, dev, out)      # outside of a capture it is allocated on the way
    assert plan.read_status() == 0


def test_sequences_that_share_pages(cuda_device):
    """Two sequences with the same prefix pages, and the same sequence twice."""
    lens = [300, 200, 300]
    dev, q, seqs = _inputs(lens, 2, 4, 128, 1, torch.bfloat16, 15, cuda_device)
    dev["bt"][1, :2] = dev["bt"][0, :2]
    dev["bt"][2] = dev["bt"][0]
    k, v = (torch.cat([a[:128], b[128:]]) for a, b in zip(seqs[0], seqs[1]))
    plan = M.GqaDecodePlan(_dims(2, 4, 128, 1, "bf16"), lens).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    assert plan.read_status() == 0
    _check(out, q, [seqs[0], (k, v), seqs[0]], 128, "bf16", "shared pages")


def test_binding_refuses_mixed_devices_and_strided_tensors(cuda_device):
    lens = [300, 200]
    dev, _, _ = _inputs(lens, 2, 4, 128, 1, torch.bfloat16, 16, cuda_device)
    plan = M.GqaDecodePlan(_dims(2, 4, 128, 1, "bf16"), lens)
    assert plan.read_status() == 0
    out = torch.zeros_like(dev["q"])
    for name in ("q", "kp", "vp", "bt", "sl"):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            _run(plan, dict(dev, **{name: dev[name].cpu()}), out)
        wide = torch.stack([dev[name], dev[name]], dim=-1)[..., 0]
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            _run(plan, dict(dev, **{name: wide}), out)
    with pytest.raises(ValueError, match="out must be a contiguous CUDA tensor"):
        _run(plan, dev, out.cpu())
    assert plan.workspace is None and (out == 0).all()
    plan.close()
    with pytest.raises(M.MlaError):      # a closed plan
        _run(plan, dev, out)
