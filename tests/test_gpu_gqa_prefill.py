"""Causal attention of packed prompts over the paged grouped-head cache against
the 64-bit oracle, every element, with bounds from the rounding steps
(harness_paged). Unused slots and the slots behind a sequence's end hold NaN."""

import pytest
import torch

import mla_latent_kv_21_b200 as M

from harness_paged import TYPES, block_tables, check_attention, generator, paged_kv

pytestmark = pytest.mark.gpu


def _inputs(new, lens, Hk, G, d, dtype, seed, device, extra_rows=0, q_std=1.0):
    gen = generator(seed)
    table, blocks = block_tables(lens, gen)
    kp, vp, seqs = paged_kv(lens, Hk, d, dtype, gen, table, blocks)
    T = sum(new) + extra_rows
    q = (torch.randn((T, Hk * G, d), generator=gen) * q_std).to(dtype)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    dev = dict(q=q.to(device), kp=kp.to(device), vp=vp.to(device), bt=table.to(device),
               cu=torch.tensor(cu, dtype=torch.int32, device=device), sl=torch.tensor(lens, dtype=torch.int32, device=device))
    return dev, q, cu, seqs


def _run(plan, dev, out, stream=None):
    plan.run(dev["q"], dev["kp"], dev["vp"], dev["bt"], dev["cu"], dev["sl"], out, stream=stream)


def _dims(Hk, G, d, dtype):
    return M.gqa_dims_for(Hk * G, Hk, d, d ** -0.5, dtype)


def _check(out, q, cu, seqs, d, dtype, what):
    for b, (k, v) in enumerate(seqs):
        rows = slice(cu[b], cu[b + 1])
        check_attention(out[rows], q[rows], k, v, d ** -0.5, TYPES[dtype], f"{what}, sequence {b}")


# (new tokens, all tokens) of each sequence
WHOLE = [(1, 1), (64, 64), (0, 0), (63, 63), (129, 129), (300, 300), (2, 2), (65, 65)]
CHUNKS = [(1, 200), (64, 128), (0, 70), (37, 100), (130, 513), (5, 5), (128, 129), (3, 900)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk,G", [(2, 1), (1, 2), (1, 3), (2, 4), (1, 5), (1, 7), (2, 8), (1, 16), (1, 48), (1, 128)])
def test_prompts_and_chunks(cuda_device, dtype, d, Hk, G):
    for counts in (WHOLE, CHUNKS):
        new, lens = [c[0] for c in counts], [c[1] for c in counts]
        dev, q, cu, seqs = _inputs(new, lens, Hk, G, d, TYPES[dtype], Hk * 10 + G, cuda_device)
        plan = M.GqaPrefillPlan(_dims(Hk, G, d, dtype), new).allocate_workspace(cuda_device)
        out = torch.full_like(dev["q"], float("nan"))
        _run(plan, dev, out)
        assert plan.read_status() == 0
        _check(out, q, cu, seqs, d, dtype, "prompts")
        plan.close()


@pytest.mark.parametrize("new,lens", [([1], [1]), ([256], [256]), ([257], [257]), ([1000], [1000]), ([1500], [2100]),
                                      ([1], [3000])])
@pytest.mark.parametrize("Hk,G,d", [(1, 1, 128), (2, 4, 128), (1, 3, 64)])
def test_single_prompts(cuda_device, new, lens, Hk, G, d):
    dev, q, cu, seqs = _inputs(new, lens, Hk, G, d, torch.bfloat16, new[0], cuda_device)
    plan = M.GqaPrefillPlan(_dims(Hk, G, d, "bf16"), new).allocate_workspace(cuda_device)
    out, again = torch.full_like(dev["q"], float("nan")), torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    _run(plan, dev, again)
    assert plan.read_status() == 0 and torch.equal(out, again)
    _check(out, q, cu, seqs, d, "bf16", "prompt")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_std", [0.0, 30.0])
def test_flat_and_peaked_scores(cuda_device, dtype, q_std):
    new, lens = [400, 33], [700, 33]
    dev, q, cu, seqs = _inputs(new, lens, 2, 2, 128, TYPES[dtype], 3, cuda_device, q_std=q_std)
    plan = M.GqaPrefillPlan(_dims(2, 2, 128, dtype), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    assert plan.read_status() == 0
    _check(out, q, cu, seqs, 128, dtype, "scores")


def test_queries_that_see_no_key_and_more_new_tokens_than_cached(cuda_device):
    """L_b < n_b: the first n_b - L_b queries see nothing and give zeros."""
    new, lens = [10, 200, 70], [4, 0, 66]
    dev, q, cu, seqs = _inputs(new, lens, 2, 4, 128, torch.bfloat16, 4, cuda_device)
    plan = M.GqaPrefillPlan(_dims(2, 4, 128, "bf16"), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    assert plan.read_status() == 0
    assert (out[:6] == 0).all() and (out[10:210] == 0).all()
    _check(out, q, cu, seqs, 128, "bf16", "short caches")


def test_rows_behind_the_last_sequence_stay(cuda_device):
    """A plan and buffers of 300 rows; the call's sequences own 250 of them."""
    new, lens = [100, 0, 150], [100, 7, 180]
    dev, q, cu, seqs = _inputs(new, lens, 2, 4, 128, torch.bfloat16, 5, cuda_device, extra_rows=50)
    plan = M.GqaPrefillPlan(_dims(2, 4, 128, "bf16"), [100, 50, 150]).allocate_workspace(cuda_device)
    dev["q"][250:] = float("nan")
    out = torch.full_like(dev["q"], 7.0)
    _run(plan, dev, out)
    assert plan.read_status() == 0
    assert (out[250:] == 7.0).all()
    _check(out, q, cu, seqs, 128, "bf16", "padded batch")


def test_bad_metadata_is_recorded(cuda_device):
    new, lens = [100, 90, 80], [100, 150, 80]
    dev, q, cu, seqs = _inputs(new, lens, 2, 4, 128, torch.bfloat16, 6, cuda_device)
    plan = M.GqaPrefillPlan(_dims(2, 4, 128, "bf16"), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], 7.0)

    def others(bad):
        for b in range(3):
            if b != bad:
                rows = slice(cu[b], cu[b + 1])
                check_attention(out[rows], q[rows], *seqs[b], 128 ** -0.5, torch.bfloat16, f"sequence {b}")

    for bad in (-5, 64 * dev["bt"].shape[1] + 1):
        dev["sl"][1] = bad
        out.fill_(7.0)
        _run(plan, dev, out)
        assert plan.read_status() == M.MLA_ERR_BOUNDS
        assert (out[100:190] == 0).all()
        others(1)
    dev["sl"][1] = 150
    dev["bt"][1, 1] = dev["kp"].shape[0]
    _run(plan, dev, out)
    assert plan.read_status() == M.MLA_ERR_BOUNDS
    others(1)
    k, v = seqs[1]     # without the keys 64 to 127, the last query sees the rest
    seen = torch.tensor([j for j in range(150) if j // 64 != 1])
    check_attention(out[189:190], q[189:190], k[seen], v[seen], 128 ** -0.5, torch.bfloat16, "the pages that remain")
    dev["bt"][1, 1] = 0
    # prefix sums past the packed rows, or a count above the plan's largest: those rows are left alone
    dev["cu"][3] = 400
    out.fill_(7.0)
    _run(plan, dev, out)
    assert plan.read_status() == M.MLA_ERR_BOUNDS and (out[190:] == 7.0).all()
    check_attention(out[:100], q[:100], *seqs[0], 128 ** -0.5, torch.bfloat16, "first")


# More items than the device has blocks: every block draws several from the sorted list.
MANY = [(700, 900), (1, 1), (0, 30), (1300, 1300), (64, 500), (333, 333), (1, 2000), (900, 901), (0, 0), (65, 64), (1100, 1500),
        (20, 0)]


@pytest.mark.parametrize("dtype,Hk,G,d", [("bf16", 4, 4, 128), ("fp16", 8, 7, 64), ("bf16", 8, 1, 128), ("fp16", 2, 40, 128),
                                          ("bf16", 1, 128, 64)])
def test_many_items(cuda_device, dtype, Hk, G, d):
    new, lens = [c[0] for c in MANY], [c[1] for c in MANY]
    dev, q, cu, seqs = _inputs(new, lens, Hk, G, d, TYPES[dtype], 31, cuda_device, extra_rows=9)
    counts = list(new)
    counts[2] = 9    # rows that the call's prefix sums leave over
    plan = M.GqaPrefillPlan(_dims(Hk, G, d, dtype), counts).allocate_workspace(cuda_device)
    out, again = torch.full_like(dev["q"], 7.0), torch.full_like(dev["q"], 7.0)
    _run(plan, dev, out)
    _run(plan, dev, again)
    assert plan.read_status() == 0 and torch.equal(out, again)
    assert (out[-9:] == 7.0).all()
    _check(out, q, cu, seqs, d, dtype, "many items")


def test_many_items_with_bad_metadata(cuda_device):
    new, lens = [1000, 1200, 900, 800], [1000, 1300, 900, 2000]
    dev, q, cu, seqs = _inputs(new, lens, 4, 4, 128, torch.bfloat16, 32, cuda_device)
    plan = M.GqaPrefillPlan(_dims(4, 4, 128, "bf16"), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], 7.0)

    def check(bad):
        assert plan.read_status() == M.MLA_ERR_BOUNDS and plan.read_status() == 0
        for b in range(4):
            if b not in bad:
                rows = slice(cu[b], cu[b + 1])
                check_attention(out[rows], q[rows], *seqs[b], 128 ** -0.5, torch.bfloat16, f"sequence {b}")

    dev["sl"][1] = -1
    _run(plan, dev, out)
    check([1])
    assert (out[1000:2200] == 0).all()
    dev["sl"][1] = 1300
    keep = dev["bt"].clone()
    dev["bt"][3, 5], dev["bt"][3, 6] = -1, dev["kp"].shape[0]
    _run(plan, dev, out)
    check([3])
    k, v = seqs[3]
    seen = torch.tensor([j for j in range(2000) if j // 64 not in (5, 6)])
    check_attention(out[-50:], q[-50:], k[seen], v[seen], 128 ** -0.5, torch.bfloat16, "the pages that remain")
    dev["bt"].copy_(keep)
    out.fill_(7.0)
    dev["cu"][2] = 2300     # 1300 and 800 new tokens: the first is above the plan's largest count
    _run(plan, dev, out)
    check([1, 2])
    assert (out[1000:2300] == 7.0).all()
    out.fill_(7.0)
    dev["cu"].copy_(torch.tensor([0, 1000, 0, 1000, 1800], dtype=torch.int32))   # sums that fall
    _run(plan, dev, out)
    assert plan.read_status() == M.MLA_ERR_BOUNDS


def test_many_sequences(cuda_device):
    """700 short prompts, some empty."""
    new = [(b * 5) % 9 for b in range(700)]
    lens = [n + (b * 3) % 70 for b, n in enumerate(new)]
    dev, q, cu, seqs = _inputs(new, lens, 2, 4, 64, torch.float16, 33, cuda_device)
    plan = M.GqaPrefillPlan(_dims(2, 4, 64, "fp16"), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    _run(plan, dev, out)
    assert plan.read_status() == 0
    _check(out, q, cu, seqs, 64, "fp16", "many sequences")


def test_offsets_past_32_bits(cuda_device):
    new, lens, Hk, d = [150, 64], [150, 100], 8, 128
    blocks = 2 ** 31 // (Hk * 64 * d) + 40
    dev, q, cu, seqs = _inputs(new, lens, Hk, 2, d, torch.bfloat16, 10, cuda_device)
    big = torch.empty((2, blocks, Hk, 64, d), dtype=torch.bfloat16, device=cuda_device)
    small = dev["kp"].shape[0]
    big[0, -small:], big[1, -small:] = dev["kp"], dev["vp"]
    table = torch.where(dev["bt"] >= 0, dev["bt"] + (blocks - small), -1).to(torch.int32)
    plan = M.GqaPrefillPlan(_dims(Hk, 2, d, "bf16"), new).allocate_workspace(cuda_device)
    out = torch.full_like(dev["q"], float("nan"))
    plan.run(dev["q"], big[0], big[1], table, dev["cu"], dev["sl"], out)
    assert plan.read_status() == 0
    _check(out, q, cu, seqs, d, "bf16", "far pages")


@pytest.mark.parametrize("new,lens,Hk", [([300, 20], [300, 500], 2), ([900, 1, 1400, 260], [900, 700, 1500, 260], 8)])
def test_capture_replay_and_another_stream(cuda_device, new, lens, Hk):
    """One item per block, and items drawn from the sorted list; the replays have other counts and lengths."""
    dev, q, cu, seqs = _inputs(new, lens, Hk, 4, 128, torch.bfloat16, 11, cuda_device)
    plan = M.GqaPrefillPlan(_dims(Hk, 4, 128, "bf16"), new).allocate_workspace(cuda_device)
    other = M.GqaPrefillPlan(_dims(Hk, 4, 128, "bf16"), new).allocate_workspace(cuda_device)
    out, out2 = torch.full_like(dev["q"], float("nan")), torch.full_like(dev["q"], float("nan"))
    side = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize(cuda_device)
    for _ in range(5):   # two calls in flight at once
        _run(plan, dev, out, stream=side.cuda_stream)
        _run(other, dev, out2)
    torch.cuda.synchronize(cuda_device)
    _check(out, q, cu, seqs, 128, "bf16", "side stream")
    assert torch.equal(out, out2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(plan, dev, out)
    for seed in (12, 13):
        counts = list(new) if seed == 12 else [new[0] - 7, *new[1:-1], new[-1] + 3 if len(new) > 2 else new[-1]]
        fresh, q, cu, seqs = _inputs(counts, lens, Hk, 4, 128, torch.bfloat16, seed, cuda_device, extra_rows=sum(new) - sum(counts))
        for name in dev:
            dev[name].copy_(fresh[name])
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize(cuda_device)
        assert plan.read_status() == 0
        _check(out, q, cu, seqs, 128, "bf16", "replay")
    del g
