"""The cache writers: what is stored, where, what stays untouched, and what is
refused on the device. Rotated values against the 64-bit oracle with the bound
of the rounding steps; copied values, FP8 codes and scales bit for bit."""

import numpy as np
import pytest
import torch

import mla_latent_kv_21_b200 as M
from oracle import fp8_cache

from harness_paged import TYPES, block_tables, check_rotated, f64, generator, half_step, same_bits

pytestmark = pytest.mark.gpu

COUNTS = [(3, 3), (1, 64), (0, 5), (1, 65), (70, 200), (64, 64), (0, 0), (2, 129)]   # (new, all) tokens


def _positions(counts):
    return [p for n, L in counts for p in range(L - n, L)]


def _cells(counts, table):
    return [(int(table[b, p // 64]), p % 64) for b, (n, L) in enumerate(counts) for p in range(L - n, L)]


def _poison(shape, dtype, device):
    return torch.full(shape, float("nan"), dtype=dtype, device=device)


def _others_untouched(pool, before, cells, dim_heads):
    """Every slot that is not in `cells` holds its old bits."""
    mask = torch.ones(pool.shape[0], 64, dtype=torch.bool)
    for blk, slot in cells:
        mask[blk, slot] = False
    a, b = pool.cpu(), before.cpu()
    if dim_heads:
        a, b = a.transpose(1, 2), b.transpose(1, 2)
    assert same_bits(a[mask], b[mask])


class Gqa:
    """One call's tensors; q, k and v are views of one projection."""

    def __init__(self, counts, Hq, Hk, d, D, dtype, device, seed=1, extra_rows=0, positions=256, style="half", packed=True):
        gen = generator(seed)
        self.counts, self.dtype, self.style = counts, TYPES[dtype], style
        T = sum(n for n, _ in counts) + extra_rows
        self.table, blocks = block_tables([L for _, L in counts], gen)
        qkv = torch.randn((T, Hq + 2 * Hk, d), generator=gen).to(self.dtype).to(device)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        self.kp = _poison((blocks, Hk, 64, d), self.dtype, device)
        self.vp = torch.randn((blocks, Hk, 64, d), generator=gen).to(self.dtype).to(device)
        self.before = (self.kp.clone(), self.vp.clone())
        self.bt = self.table.to(device)
        self.sl = torch.tensor([L for _, L in counts], dtype=torch.int32, device=device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in counts])]), dtype=torch.int32, device=device)
        self.rope = M.rope_table(positions, D, device=device) if D else None
        self.q_out = torch.full((T, Hq, d), 9.0, dtype=self.dtype, device=device)
        n = max(1, counts[0][0])
        self.op = M.GqaAppend(M.gqa_dims_for(Hq, Hk, d, 1.0, dtype, q_len=n, rope_dim=D, rope_style=style))
        self.op.allocate_workspace(device)
        self.packed = packed

    def run(self, **kw):
        a = dict(k=self.k, v=self.v, k_pool=self.kp, v_pool=self.vp, block_table=self.bt, seq_lens=self.sl,
                 rope_table=self.rope, q=self.q, q_out=self.q_out, cu_seqlens=self.cu if self.packed else None)
        a.update(kw)
        self.op.run(**a)

    def check(self, rows=None, counts=None):
        counts = counts or self.counts
        pos, cells = _positions(counts), _cells(counts, self.table)
        rows = list(range(len(pos))) if rows is None else rows
        kp, vp = self.kp.cpu(), self.vp.cpu()
        blk, slot = [c[0] for c in cells], [c[1] for c in cells]
        assert same_bits(vp[blk, :, slot], self.v[rows].cpu())
        table = self.rope if self.rope is not None else torch.zeros((1, 0))
        at = pos if self.rope is not None else [0] * len(pos)
        check_rotated(kp[blk, :, slot], self.k[rows], table, at, self.style, self.dtype, "keys")
        check_rotated(self.q_out[rows], self.q[rows], table, at, self.style, self.dtype, "queries")
        _others_untouched(self.kp, self.before[0], cells, True)
        _others_untouched(self.vp, self.before[1], cells, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hk,d,D", [(8, 2, 128, 128), (3, 3, 64, 64), (7, 1, 128, 64), (4, 4, 64, 32), (2, 1, 128, 16),
                                       (5, 1, 128, 0)])
def test_gqa_packed(cuda_device, dtype, style, Hq, Hk, d, D):
    c = Gqa(COUNTS, Hq, Hk, d, D, dtype, cuda_device, style=style)
    c.run()
    assert c.op.read_status() == 0
    c.check()
    bits = c.kp.clone(), c.vp.clone(), c.q_out.clone()
    c.run()      # writing the same tokens again changes nothing
    assert all(same_bits(a, b) for a, b in zip(bits, (c.kp, c.vp, c.q_out)))


@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("B", [1, 7, 40])
def test_gqa_step(cuda_device, n, B):
    counts = [(n, n + (b * 37) % 190) for b in range(B)]
    c = Gqa(counts, 32, 8, 128, 128, "bf16", cuda_device, packed=False)
    c.run()
    assert c.op.read_status() == 0
    c.check()


def test_gqa_without_queries_and_in_place(cuda_device):
    c = Gqa(COUNTS, 4, 2, 128, 128, "bf16", cuda_device)
    c.run(q=None, q_out=None)
    assert (c.q_out == 9.0).all()
    q = c.q.contiguous()
    c.run(q=q, q_out=q)
    c.q_out = q
    assert c.op.read_status() == 0
    c.check()


def test_gqa_large_prompts_take_long_head_lists(cuda_device):
    """Enough tokens that a thread walks 16 heads; an odd number of heads."""
    counts = [(9000, 9000), (12001, 12500)]
    c = Gqa(counts, 15, 3, 128, 128, "bf16", cuda_device, positions=12500)
    c.run()
    assert c.op.read_status() == 0
    c.check()


def test_many_sequences(cuda_device):
    """More sequences than the prefix sums that a block keeps: the search has two levels."""
    counts = [((b * 7) % 4, 4 + b % 120) for b in range(2500)]
    c = Gqa(counts, 2, 1, 64, 64, "bf16", cuda_device)
    c.run()
    assert c.op.read_status() == 0
    c.check()


def test_rows_behind_the_last_sequence_stay(cuda_device):
    c = Gqa(COUNTS, 4, 2, 128, 128, "bf16", cuda_device, extra_rows=5)
    c.run()
    assert c.op.read_status() == 0
    assert (c.q_out[-5:] == 9.0).all()
    c.check()


@pytest.mark.parametrize("what", ["short", "long", "block", "far block", "table", "negative"])
def test_bad_metadata_is_recorded_and_skipped(cuda_device, what):
    counts = [(3, 3), (4, 130), (2, 50)]
    c = Gqa(counts, 4, 2, 128, 128, "bf16", cuda_device, positions=100 if what == "table" else 256)
    if what in ("short", "long", "negative"):
        c.sl[1] = {"short": 3, "long": 64 * c.bt.shape[1] + 1, "negative": -7}[what]
    elif what != "table":
        c.bt[1, 2] = -1 if what == "block" else c.kp.shape[0]
        c.bt[1, 1] = c.bt[1, 2]
    c.run()
    assert c.op.read_status() == M.MLA_ERR_BOUNDS
    assert c.op.read_status() == 0
    assert (c.q_out[3:7] == 9.0).all()
    table = c.table.clone()
    c.table = torch.stack([table[0], table[2]])
    c.check(rows=[0, 1, 2, 7, 8], counts=[counts[0], counts[2]])


def test_prefix_sums_past_the_rows(cuda_device):
    counts = [(3, 3), (4, 130)]
    c = Gqa(counts, 4, 2, 128, 128, "bf16", cuda_device)
    c.cu[2] = 20
    c.run()
    assert c.op.read_status() == M.MLA_ERR_BOUNDS
    c.check(rows=[0, 1, 2], counts=counts[:1])


def test_gqa_no_tokens(cuda_device):
    c = Gqa([(0, 4), (0, 0)], 4, 2, 128, 128, "bf16", cuda_device)
    c.run()
    assert c.op.read_status() == 0
    assert same_bits(c.kp, c.before[0])


def test_gqa_offsets_past_32_bits(cuda_device):
    Hk, d = 8, 128
    blocks = 2 ** 31 // (Hk * 64 * d) + 30
    c = Gqa([(5, 70), (1, 1)], 8, Hk, d, d, "bf16", cuda_device)
    small = c.kp.shape[0]
    big = torch.empty((2, blocks, Hk, 64, d), dtype=torch.bfloat16, device=cuda_device)
    big[0, -small:], big[1, -small:] = c.kp, c.vp
    bt = torch.where(c.bt >= 0, c.bt + (blocks - small), -1).to(torch.int32)
    c.run(k_pool=big[0], v_pool=big[1], block_table=bt)
    assert c.op.read_status() == 0
    c.kp, c.vp = big[0, -small:], big[1, -small:]
    c.check()


def test_gqa_graph_and_stream(cuda_device):
    c = Gqa([(1, 10 + 20 * b) for b in range(9)], 8, 2, 128, 128, "bf16", cuda_device, packed=False)
    side = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize(cuda_device)
    c.run(stream=side.cuda_stream)
    torch.cuda.synchronize(cuda_device)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    # the captured step with other lengths: each sequence one token further
    for name, pool in zip(("kp", "vp"), c.before):
        getattr(c, name).copy_(pool)
    c.counts = [(1, L + 1) for _, L in c.counts]
    c.sl += 1
    g.replay()
    torch.cuda.synchronize(cuda_device)
    assert c.op.read_status() == 0
    c.check()
    del g


IDLE = [70, 0, 1, 2, 64, 0, 200, 3]   # with Lq new tokens each: idle slots, and caches shorter than Lq


def _kept(n):
    """(rows with a place, (new, all) tokens as they are appended) of a step of n tokens over IDLE."""
    rows = [b * n + i for b, L in enumerate(IDLE) for i in range(n) if i >= n - L]
    return rows, [(min(n, L), L) for L in IDLE]


@pytest.mark.parametrize("n", [1, 3])
def test_gqa_step_with_idle_and_short_slots(cuda_device, n):
    """The lengths that the decode takes: a slot without a token is no error, one with L < Lq takes its last L tokens."""
    c = Gqa([(n, L) for L in IDLE], 8, 2, 128, 128, "bf16", cuda_device, packed=False)
    c.run()
    assert c.op.read_status() == 0
    rows, counts = _kept(n)
    c.check(rows=rows, counts=counts)
    others = [t for t in range(n * len(IDLE)) if t not in rows]
    assert (c.q_out[others] == 9.0).all()
    c.sl[1] = -1        # a negative length is one
    c.run()
    assert c.op.read_status() == M.MLA_ERR_BOUNDS


# ---------------------------------------------------------------- latent cache --
class Latent:
    def __init__(self, counts, H, r, D, dtype, device, seed=2, style="half", packed=True, rows=True, shift=0, positions=256,
                 std=1.0):
        gen = generator(seed)
        self.counts, self.style, self.fp8 = counts, style, dtype == "fp8"
        self.act = torch.bfloat16 if self.fp8 else TYPES[dtype]
        T = sum(n for n, _ in counts)
        self.table, blocks = block_tables([L for _, L in counts], gen)
        # the latent and the key's rotary part are views of one projection; `shift` moves them off 16-byte addresses
        kv = (torch.randn((T, r + D + shift), generator=gen) * std).to(self.act).to(device)
        q = torch.randn((T, H, 32 + D + shift), generator=gen).to(self.act).to(device)
        self.ckv, self.kr, self.q = kv[:, shift:shift + r], kv[:, shift + r:], q[:, :, 32 + shift:]
        if self.fp8:
            self.codes = torch.randint(0, 100, (blocks, 64, r), dtype=torch.uint8, generator=gen).to(device)
            self.kvr = _poison((blocks, 64, D), self.act, device)
            self.scale = _poison((blocks, 64), torch.float32, device)
            self.pools = (self.codes, self.kvr, self.scale)
        else:
            self.pools = (_poison((blocks, 64, r + D), self.act, device),)
        self.before = [p.clone() for p in self.pools]
        self.bt = self.table.to(device)
        self.sl = torch.tensor([L for _, L in counts], dtype=torch.int32, device=device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in counts])]), dtype=torch.int32, device=device)
        self.rope = M.rope_table(positions, D, device=device) if D else None
        self.q_out = torch.full((T, H, D), 9.0, dtype=self.act, device=device)
        self.rows = torch.full((T, r + D), 9.0, dtype=self.act, device=device) if rows else None
        self.r, self.D = r, D
        dims = M.dims_for(H, r, D, 128, 128, max(1, counts[0][0]), 0.1, dtype)
        self.op = M.LatentAppend(dims, rope_style=style).allocate_workspace(device)
        self.packed = packed

    def run(self, **kw):
        a = dict(q_rope=self.q if self.D else None, q_rope_out=self.q_out if self.D else None, kv_rows=self.rows,
                 cu_seqlens=self.cu if self.packed else None)
        a.update(kw)
        f = self.op.run_fp8 if self.fp8 else self.op.run
        f(self.ckv, self.kr if self.D else None, *self.pools, self.bt, self.sl, self.rope, **a)

    def check(self, rows=None, counts=None):
        counts = counts or self.counts
        pos, cells = _positions(counts), _cells(counts, self.table)
        rows = list(range(len(pos))) if rows is None else rows
        blk, slot = [c[0] for c in cells], [c[1] for c in cells]
        ckv, kr = self.ckv[rows].cpu(), self.kr[rows].cpu()[:, None]
        table = self.rope if self.D else torch.zeros((1, 0))
        at = pos if self.D else [0] * len(pos)
        if self.fp8:
            c = ckv.float().numpy()
            scale = np.maximum(np.abs(c).max(axis=1) / np.float32(448.0), np.float32(2.0 ** -64)).astype(np.float32)
            want = torch.from_numpy(c / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(self.codes.cpu()[blk, slot], want)
            assert same_bits(self.scale.cpu()[blk, slot], torch.from_numpy(scale))
            got = f64(self.kvr.cpu()[blk, slot])[:, None] * scale.astype(np.float64)[:, None, None]
            from oracle import gqa_oracle
            ref, size = gqa_oracle.rotate(f64(kr), f64(table), np.asarray(at), self.style)
            # rotation in fp32 (3 roundings), a division (1), one rounding to bf16
            bound = 2.0 ** -8 * np.abs(ref) + 4 * 2.0 ** -24 * 1.01 * size
            assert (np.abs(got - ref) <= bound).all()
        else:
            pool = self.pools[0].cpu()[blk, slot]
            assert same_bits(pool[:, :self.r], ckv)
            if self.D:
                check_rotated(pool[:, None, self.r:], kr, table, at, self.style, self.act, "RoPE key")
        if self.rows is not None:
            assert same_bits(self.rows[rows][:, :self.r].cpu(), ckv)
            if self.D:
                check_rotated(self.rows[rows][:, None, self.r:], kr, table, at, self.style, self.act, "rows")
        if self.D:
            check_rotated(self.q_out[rows], self.q[rows], table, at, self.style, self.act, "queries")
        for p, b in zip(self.pools, self.before):
            _others_untouched(p, b, cells, False)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,H,r,D", [("bf16", 128, 512, 64), ("bf16", 16, 256, 64), ("fp32", 8, 64, 16), ("fp32", 4, 512, 64),
                                         ("fp8", 128, 512, 64), ("fp8", 5, 512, 64), ("fp8", 8, 256, 64), ("fp8", 3, 16, 16), ("bf16", 3, 64, 512), ("fp32", 2, 64, 256), ("bf16", 2, 320, 256), ("fp8", 2, 320, 256), ("fp8", 2, 464, 0), ("bf16", 3, 50, 6), ("fp32", 3, 37, 2),
                                         ("bf16", 4, 512, 0), ("fp32", 2, 72, 24)])
def test_latent_packed(cuda_device, style, dtype, H, r, D):
    c = Latent(COUNTS, H, r, D, dtype, cuda_device, style=style)
    c.run()
    assert c.op.read_status() == 0
    c.check()
    c = Latent(COUNTS, H, r, D, dtype, cuda_device, style=style, rows=False, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_latent_unaligned_views(cuda_device, dtype):
    c = Latent(COUNTS, 16, 512, 64, dtype, cuda_device, shift=1)
    assert c.ckv.data_ptr() % 16 != 0
    c.run()
    assert c.op.read_status() == 0
    c.check()


def test_fp8_refuses_unaligned_views(cuda_device):
    c = Latent(COUNTS, 16, 512, 64, "fp8", cuda_device, shift=1)
    with pytest.raises(M.MlaError) as e:
        c.run()
    assert e.value.status == M.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("B,n", [(1, 1), (64, 1), (9, 3)])
def test_latent_step(cuda_device, dtype, B, n):
    c = Latent([(n, n + (b * 41) % 180) for b in range(B)], 16, 512, 64, dtype, cuda_device, packed=False, rows=False)
    c.run()
    assert c.op.read_status() == 0
    c.check()


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("dtype,r,D", [("bf16", 512, 64), ("fp32", 512, 64), ("fp8", 512, 64), ("bf16", 50, 6)])
def test_latent_step_with_idle_and_short_slots(cuda_device, dtype, r, D, n):
    c = Latent([(n, L) for L in IDLE], 16, r, D, dtype, cuda_device, packed=False)
    c.run()
    assert c.op.read_status() == 0
    rows, counts = _kept(n)
    c.check(rows=rows, counts=counts)
    others = [t for t in range(n * len(IDLE)) if t not in rows]
    assert (c.q_out[others] == 9.0).all() and (c.rows[others] == 9.0).all()


@pytest.mark.parametrize("std", [1e-30, 1e-3, 1e4])
def test_fp8_scales_of_any_size(cuda_device, std):
    """Latents whose largest value is far below, near and above one; rows of zeros take the smallest scale."""
    c = Latent(COUNTS, 2, 512, 64, "fp8", cuda_device, std=std)
    c.ckv[5] = 0.0
    c.ckv[7, 1:] = 0.0
    c.kr.copy_(torch.randn(c.kr.shape, generator=generator(4)).to(torch.bfloat16))
    c.run()
    assert c.op.read_status() == 0
    c.check()
    assert torch.isfinite(c.kvr[c.bt[4, 2].item()][2:8].float()).all()   # its tokens 130 to 135


def test_fp8_cache_reads_back(cuda_device):
    """The codes, decoded by the oracle from the format's bit fields, give the latent within e4m3's step."""
    c = Latent(COUNTS, 2, 512, 64, "fp8", cuda_device)
    c.run()
    cells = _cells(c.counts, c.table)
    blk, slot = [x[0] for x in cells], [x[1] for x in cells]
    scale = c.scale.cpu()[blk, slot]
    ckv, _ = fp8_cache.logical_cache_fp8(c.codes.cpu()[blk, slot].numpy(), f64(c.kvr.cpu()[blk, slot]), f64(scale))
    x = f64(c.ckv)
    # half a step: 2^-4 of a normal code, 2^-10 (times the scale) of a subnormal one; the division adds 2^-24
    bound = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * f64(scale)[:, None]) * (1 + 2.0 ** -20)
    assert (np.abs(ckv - x) <= bound).all()


def test_latent_bad_metadata(cuda_device):
    counts = [(3, 3), (4, 130), (2, 50)]
    for dtype in ("bf16", "fp32", "fp8"):
        c = Latent(counts, 4, 512, 64, dtype, cuda_device)
        c.sl[1] = 2
        c.run()
        assert c.op.read_status() == M.MLA_ERR_BOUNDS
        assert (c.q_out[3:7] == 9.0).all() and (c.rows[3:7] == 9.0).all()
        table = c.table
        c.table = torch.stack([table[0], table[2]])
        c.check(rows=[0, 1, 2, 7, 8], counts=[counts[0], counts[2]])


def test_latent_graph_and_stream(cuda_device):
    c = Latent([(1, 10 + 20 * b) for b in range(9)], 8, 512, 64, "fp8", cuda_device, packed=False)
    side = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize(cuda_device)
    c.run(stream=side.cuda_stream)
    torch.cuda.synchronize(cuda_device)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for pool, old in zip(c.pools, c.before):
        pool.copy_(old)
    c.counts = [(1, L + 1) for _, L in c.counts]
    c.sl += 1
    g.replay()
    torch.cuda.synchronize(cuda_device)
    assert c.op.read_status() == 0
    c.check()
    del g
