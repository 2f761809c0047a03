"""Workspaces and streams: a plan dropped while its call runs on another stream
keeps its memory until the call is done; a stream that uses a workspace waits
until it is cleared; nothing is allocated for a stream under capture."""

import pytest
import torch

import mla_latent_kv_21_b200 as M
from mla_latent_kv_21_b200 import _lib as L

from mla_workloads import WORKLOADS, generate

from harness import assert_close, dims_of, oracle_out, to_device
from harness_paged import block_tables, check_attention, f64, generator, paged_kv

pytestmark = pytest.mark.gpu

LENS, HK, G, D = [700, 64, 0, 2100], 2, 4, 128


class Case:
    """Decode (one query per sequence) and prefill (20 new tokens per sequence) over one cache."""

    def __init__(self, device, seed=1):
        gen = generator(seed)
        table, blocks = block_tables(LENS, gen)
        kp, vp, self.seqs = paged_kv(LENS, HK, D, torch.bfloat16, gen, table, blocks)
        self.kp, self.vp, self.bt = kp.to(device), vp.to(device), table.to(device)
        self.sl = torch.tensor(LENS, dtype=torch.int32, device=device)
        self.dims = M.gqa_dims_for(HK * G, HK, D, D ** -0.5, "bf16")
        self.q = torch.randn((4, 1, HK * G, D), generator=gen).to(torch.bfloat16).to(device)
        self.new = [20, 20, 0, 20]
        self.cu = torch.tensor([0, 20, 40, 40, 60], dtype=torch.int32, device=device)
        self.qp = torch.randn((60, HK * G, D), generator=gen).to(torch.bfloat16).to(device)

    def make(self, what):
        return M.GqaDecodePlan(self.dims, LENS) if what == "decode" else M.GqaPrefillPlan(self.dims, self.new)

    def run(self, plan, what, stream=None):
        q = self.q if what == "decode" else self.qp
        out = torch.full_like(q, float("nan"))
        torch.cuda.synchronize()
        self.launch(plan, what, out, stream)
        return out

    def launch(self, plan, what, out, stream=None):
        if what == "decode":
            plan.run(self.q, self.kp, self.vp, self.bt, self.sl, out, stream=stream)
        else:
            plan.run(self.qp, self.kp, self.vp, self.bt, self.cu, self.sl, out, stream=stream)

    def check(self, out, what):
        for b, (k, v) in enumerate(self.seqs):
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            q, o = (self.q[b], out[b]) if what == "decode" else (self.qp[rows], out[rows])
            check_attention(o, q, k, v, D ** -0.5, torch.bfloat16, f"{what}, sequence {b}")


def _keep_busy(stream, device):
    """Products of a few tenths of a second on `stream`, with tensors that stay alive."""
    with torch.cuda.stream(stream):
        a = torch.randn((8192, 8192), device=device, dtype=torch.bfloat16)
        b = torch.empty_like(a)
        for _ in range(500):
            torch.matmul(a, a, out=b)
    return a, b


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_a_plan_dropped_while_its_call_waits_on_another_stream(cuda_device, what):
    c = Case(cuda_device)
    side = torch.cuda.Stream(cuda_device)
    c.run(c.make(what), what)         # loads the kernels, which may synchronise
    _keep_busy(side, cuda_device)
    out = torch.full_like(c.q if what == "decode" else c.qp, float("nan"))
    torch.cuda.synchronize()
    busy = _keep_busy(side, cuda_device)
    plan = c.make(what)
    c.launch(plan, what, out, side.cuda_stream)
    size, at = plan.workspace_bytes, plan.workspace.data_ptr()
    del plan                          # no cycle holds it: its memory goes back at once
    assert not side.query()           # the call has not run yet
    others = [torch.full((size,), 0x5b, dtype=torch.uint8, device=cuda_device) for _ in range(4)]
    ranges = [(t.data_ptr(), t.data_ptr() + size) for t in others]
    torch.cuda.synchronize()
    assert all(at + size <= lo or hi <= at for lo, hi in ranges)
    c.check(out, what)
    del busy


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_a_stream_waits_until_the_workspace_is_cleared(cuda_device, what):
    """Allocated on the busy current stream, first used on another one; and allocated for another stream directly."""
    c = Case(cuda_device)
    side, third = torch.cuda.Stream(cuda_device), torch.cuda.Stream(cuda_device)
    c.run(c.make(what), what)         # loads the kernels, which may synchronise
    _keep_busy(torch.cuda.current_stream(), cuda_device)
    for direct in (False, True):
        plan = c.make(what)
        outs = [torch.full_like(c.q if what == "decode" else c.qp, float("nan")) for _ in range(2)]
        torch.cuda.synchronize()
        busy = _keep_busy(torch.cuda.current_stream(), cuda_device)
        if direct:
            plan.allocate_workspace(cuda_device, stream=side.cuda_stream)
        else:
            plan.allocate_workspace(cuda_device)
        c.launch(plan, what, outs[0], side.cuda_stream)
        assert not side.query()       # it waits for the current stream's products
        side.synchronize()
        c.launch(plan, what, outs[1], third.cuda_stream)
        torch.cuda.synchronize()
        assert plan.read_status() == 0
        for out in outs:
            c.check(out, what)
        del busy


def test_the_default_stream_by_its_handle(cuda_device):
    """Handle 0 while another stream is current."""
    c = Case(cuda_device)
    plan = c.make("decode")
    side = torch.cuda.Stream(cuda_device)
    with torch.cuda.stream(side):
        out = c.run(plan, "decode", stream=0)
        assert torch.cuda.default_stream(cuda_device).cuda_stream in plan._streams
        torch.cuda.synchronize()
    assert plan.read_status(0) == 0
    c.check(out, "decode")


def test_a_first_run_on_a_capturing_stream_is_refused(cuda_device):
    """`stream` captures, the current stream does not."""
    c = Case(cuda_device)
    side = torch.cuda.Stream(cuda_device)
    x = torch.zeros(4, device=cuda_device)
    plan, ready = c.make("decode"), c.make("decode").allocate_workspace(cuda_device)
    out = torch.full_like(c.q, float("nan"))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        x += 1
        with torch.cuda.stream(torch.cuda.default_stream(cuda_device)):
            with pytest.raises(RuntimeError, match="allocate_workspace"):
                c.launch(plan, "decode", out, side.cuda_stream)
            with pytest.raises(RuntimeError, match="before capturing"):
                plan.allocate_workspace(cuda_device, stream=side.cuda_stream)
        c.launch(ready, "decode", out, side.cuda_stream)
    assert plan.workspace is None
    g.replay()
    torch.cuda.synchronize()
    assert ready.read_status() == 0 and (x == 1).all()
    c.check(out, "decode")
    out.fill_(float("nan"))
    c.launch(ready, "decode", out, side.cuda_stream)      # eager after the capture, on the stream that captured
    torch.cuda.synchronize()
    c.check(out, "decode")
    del g


def test_a_workspace_on_another_device_is_refused(cuda_device):
    c = Case(cuda_device)
    plan = c.make("decode").allocate_workspace(cuda_device)
    plan._at = 1, plan._at[1]
    with pytest.raises(ValueError, match="the workspace is on device 1"):
        c.run(plan, "decode")


def test_a_status_is_read_and_cleared_in_the_streams_order(cuda_device):
    """On a stream of its own, while the default stream is busy: the clearing waits for neither, and an error that the
    next call records is not cleared with the last one's."""
    c = Case(cuda_device)
    side = torch.cuda.Stream(cuda_device)
    plan = c.make("decode").allocate_workspace(cuda_device)
    out = c.run(plan, "decode", stream=side.cuda_stream)
    bad = c.sl.clone()
    bad[1] = -1
    torch.cuda.synchronize()
    default = torch.cuda.default_stream(cuda_device)
    busy = _keep_busy(default, cuda_device)
    good, c.sl = c.sl, bad
    for _ in range(3):
        c.launch(plan, "decode", out, side.cuda_stream)
        assert plan.read_status(side.cuda_stream) == M.MLA_ERR_BOUNDS
    assert not default.query()
    torch.cuda.synchronize()
    assert plan.read_status(side.cuda_stream) == 0
    c.sl = good
    del busy


def _batch(lens, new, Hk, d, device, seed):
    """Tensors of a decode (new None) or a prefill call and a function that launches it with a workspace."""
    gen = torch.Generator(device=device).manual_seed(seed)
    table, blocks = block_tables(lens, generator(seed))
    kp, vp = (torch.randn((blocks, Hk, 64, d), device=device, generator=gen).to(torch.bfloat16) for _ in range(2))
    bt, sl = table.to(device), torch.tensor(lens, dtype=torch.int32, device=device)
    dims = M.gqa_dims_for(4 * Hk, Hk, d, d ** -0.5, "bf16")
    if new is None:
        plan, size = L.mla_gqa_decode_plan(dims, lens)
        q = torch.randn((len(lens), 1, 4 * Hk, d), device=device, generator=gen).to(torch.bfloat16)
    else:
        plan, size = L.mla_gqa_prefill_plan(dims, new)
        q = torch.randn((sum(new), 4 * Hk, d), device=device, generator=gen).to(torch.bfloat16)
        cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=device)

    def launch(out, workspace, stream):
        if new is None:
            L.mla_gqa_decode_run(plan, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), blocks, bt.data_ptr(), bt.shape[1],
                                 sl.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.numel(), stream)
        else:
            L.mla_gqa_prefill_run(plan, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), blocks, bt.data_ptr(), bt.shape[1],
                                  cu.data_ptr(), sl.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                  stream)
    return size, torch.zeros_like(q), launch


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_a_workspace_that_two_calls_share_by_mistake(cuda_device, what):
    """Against the rule, two calls in flight use one workspace: their results are not defined, but nothing outside of
    the calls' own tensors is touched, both end, and the next calls in order are right."""
    if what == "decode":
        calls = [_batch([1 + 37 * b % 900 for b in range(300)], None, 2, 128, cuda_device, 1),
                 _batch([0, 40000], None, 1, 128, cuda_device, 2)]
    else:
        calls = [_batch([70] * 500, [1 + b % 7 for b in range(500)], 2, 64, cuda_device, 3),
                 _batch([1500, 900, 2000], [1300, 900, 700], 8, 128, cuda_device, 4)]
    workspace = torch.zeros(max(c[0] for c in calls), dtype=torch.uint8, device=cuda_device)
    streams = [torch.cuda.Stream(cuda_device) for _ in calls]
    current = torch.cuda.current_stream(cuda_device).cuda_stream
    want = []
    for _, out, launch in calls:
        launch(out, workspace, current)
        torch.cuda.synchronize()
        want.append(out.clone())
    assert L.mla_decode_read_status(workspace.data_ptr(), current) == 0
    for _ in range(30):
        for (_, out, launch), stream in zip(calls, streams):
            launch(out, workspace, stream.cuda_stream)
    torch.cuda.synchronize()
    assert L.mla_decode_read_status(workspace.data_ptr(), current) in (0, M.MLA_ERR_BOUNDS)
    for (_, out, launch), ref in zip(calls, want):
        out.fill_(float("nan"))
        launch(out, workspace, current)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert L.mla_decode_read_status(workspace.data_ptr(), current) == 0


# ------------------------------------------------------------- the latent plans --
class Latent:
    """A latent decode step (bf16 or FP8 cache), or the MLA-form prefill of three prompts."""

    def __init__(self, what, device):
        self.what, lens = what, [70, 300, 5]
        self.wl = WORKLOADS["deepseek_v3_fp8" if what == "fp8" else "deepseek_v3"].with_(heads=16)
        self.inputs = generate(self.wl, seq_lens=lens)
        self.dev = to_device(self.inputs, device)
        self.lens = lens
        if what == "prefill":
            gen = torch.Generator(device=device).manual_seed(8)
            T = sum(lens)
            self.x = [torch.randn(shape, device=device, generator=gen).to(torch.bfloat16)
                      for shape in ((T, 16, 128), (T, 16, 64), (T, 576))]
            self.x.append(torch.tensor([0, 70, 370, 375], dtype=torch.int32, device=device))
        self.shape = (sum(lens), 16, 128) if what == "prefill" else (3, 1, 16, 128)
        self.device = device
        # loads the kernels, which may synchronise
        self.want = self.empty()
        self.launch(self.make(), self.want)
        torch.cuda.synchronize()
        if what != "prefill":
            assert_close(f64(self.want), oracle_out(self.wl, self.inputs), self.wl.dtype, what)

    def empty(self):
        return torch.full(self.shape, float("nan"), dtype=torch.bfloat16, device=self.device)

    def make(self):
        return (M.PrefillPlan if self.what == "prefill" else M.DecodePlan)(dims_of(self.wl), self.lens)

    def launch(self, plan, out, stream=None):
        d = self.dev
        if self.what == "prefill":
            plan.run(*self.x, d["w_uk"], d["w_uv"], out, stream=stream)
        elif self.what == "fp8":
            plan.run_fp8(d["q_nope"], d["q_rope"], d["kv_codes"], d["kv_rope"], d["kv_scale"], d["block_table"],
                         d["seq_lens"], d["w_uk"], d["w_uv"], out, stream=stream)
        else:
            plan.run(d["q_nope"], d["q_rope"], d["kv_pool"], d["block_table"], d["seq_lens"], d["w_uk"], d["w_uv"], out,
                     stream=stream)


@pytest.mark.parametrize("what", ["bf16", "fp8", "prefill"])
def test_latent_plans_on_other_streams(cuda_device, what):
    """Dropped while the call waits; first used on a stream before the busy one has cleared the workspace."""
    c = Latent(what, cuda_device)
    side = torch.cuda.Stream(cuda_device)
    _keep_busy(side, cuda_device)
    out = c.empty()
    torch.cuda.synchronize()
    busy = _keep_busy(side, cuda_device)
    plan = c.make()
    c.launch(plan, out, side.cuda_stream)
    size, at = plan.workspace_bytes, plan.workspace.data_ptr()
    del plan
    assert not side.query()
    others = [torch.full((size,), 0x5b, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    ranges = [(t.data_ptr(), t.data_ptr() + size) for t in others]
    torch.cuda.synchronize()
    assert all(at + size <= lo or hi <= at for lo, hi in ranges)
    assert torch.equal(out, c.want)
    del busy, others
    out = c.empty()
    plan = c.make()
    torch.cuda.synchronize()
    busy = _keep_busy(torch.cuda.current_stream(), cuda_device)
    plan.allocate_workspace(cuda_device)
    c.launch(plan, out, side.cuda_stream)
    assert not side.query()
    torch.cuda.synchronize()
    assert plan.read_status() == 0 and torch.equal(out, c.want)
    del busy


@pytest.mark.parametrize("what", ["bf16", "prefill"])
def test_latent_plans_may_run_first_under_a_capture(cuda_device, what):
    """Their workspace is then the graph's memory, as it always was."""
    c = Latent(what, cuda_device)
    plan, out = c.make(), c.empty()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.launch(plan, out)
    g.replay()
    torch.cuda.synchronize()
    assert plan.read_status() == 0 and torch.equal(out, c.want)
    del g
