"""The bounded-wait error path of the grouped-head attention kernels, driven on
the GPU: a self-test run has barriers that expect one arrival more than they get
and a wait limit of a millisecond, so that every role gives up, waits for its own
copies and products, gives its tensor memory back and leaves. The call must
return quickly, report the timeout once, and leave the plan, the workspace and
the context usable: the next normal run is right, every element."""

import time

import pytest
import torch

import mla_latent_kv_21_b200 as M
from mla_latent_kv_21_b200 import _lib as L

from harness_paged import TYPES, block_tables, check_attention, generator, paged_kv

pytestmark = pytest.mark.gpu


def _timed(call, device):
    torch.cuda.synchronize(device)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize(device)
    return time.perf_counter() - t0


def _pool_args(kp, vp, bt):
    return kp.data_ptr(), vp.data_ptr(), kp.shape[0], bt.data_ptr(), bt.shape[1]


@pytest.mark.parametrize("dtype,Hk,G,Lq,d,workers", [("bf16", 2, 4, 1, 128, 1), ("bf16", 2, 4, 1, 128, 5),
                                                     ("fp16", 1, 8, 3, 64, 2), ("bf16", 1, 16, 4, 128, 3)])
def test_decode(cuda_device, dtype, Hk, G, Lq, d, workers):
    lens = [2048, 700, 0, 65]
    gen = generator(51)
    table, blocks = block_tables(lens, gen)
    kp, vp, seqs = paged_kv(lens, Hk, d, TYPES[dtype], gen, table, blocks)
    q = torch.randn((len(lens), Lq, Hk * G, d), generator=gen).to(TYPES[dtype])
    kp, vp, bt, qd = kp.to(cuda_device), vp.to(cuda_device), table.to(cuda_device), q.to(cuda_device)
    sl = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    plan = M.GqaDecodePlan(M.gqa_dims_for(Hk * G, Hk, d, d ** -0.5, dtype, q_len=Lq), lens, num_workers=workers)
    plan.allocate_workspace(cuda_device)
    out = torch.zeros_like(qd)
    stream = torch.cuda.current_stream(cuda_device).cuda_stream
    plan.run(qd, kp, vp, bt, sl, out)        # the kernels are loaded
    for _ in range(2):
        took = _timed(lambda: L.mla_gqa_decode_selftest_timeout(
            plan.handle, qd.data_ptr(), *_pool_args(kp, vp, bt), sl.data_ptr(), out.data_ptr(),
            plan.workspace.data_ptr(), plan.workspace_bytes, 1_000_000, stream), cuda_device)
        assert plan.read_status() == M.MLA_ERR_DEVICE_TIMEOUT
        assert plan.read_status() == 0
        assert took < 1.0, took              # a few waits of 1 ms, far below the normal 2 s
        out.fill_(float("nan"))
        plan.run(qd, kp, vp, bt, sl, out)
        assert plan.read_status() == 0
        for b, (k, v) in enumerate(seqs):
            check_attention(out[b], q[b], k, v, d ** -0.5, TYPES[dtype], f"after the timeout, sequence {b}")


@pytest.mark.parametrize("dtype,Hk,G,d", [("bf16", 2, 4, 128), ("fp16", 2, 2, 64)])
@pytest.mark.parametrize("new", [[300, 1, 64], [900, 0, 2000, 1500, 700, 1100, 800]])
def test_prefill(cuda_device, dtype, Hk, G, d, new):
    """One item per block, and items drawn from the sorted list."""
    Hk = Hk * 4 if len(new) > 3 else Hk
    lens = [n + 70 * b for b, n in enumerate(new)]
    gen = generator(52)
    table, blocks = block_tables(lens, gen)
    kp, vp, seqs = paged_kv(lens, Hk, d, TYPES[dtype], gen, table, blocks)
    q = torch.randn((sum(new), Hk * G, d), generator=gen).to(TYPES[dtype])
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    kp, vp, bt, qd = kp.to(cuda_device), vp.to(cuda_device), table.to(cuda_device), q.to(cuda_device)
    sl = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    cud = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    plan = M.GqaPrefillPlan(M.gqa_dims_for(Hk * G, Hk, d, d ** -0.5, dtype), new).allocate_workspace(cuda_device)
    out = torch.zeros_like(qd)
    stream = torch.cuda.current_stream(cuda_device).cuda_stream
    plan.run(qd, kp, vp, bt, cud, sl, out)   # the kernels are loaded
    for _ in range(2):
        took = _timed(lambda: L.mla_gqa_prefill_selftest_timeout(
            plan.handle, qd.data_ptr(), *_pool_args(kp, vp, bt), cud.data_ptr(), sl.data_ptr(), out.data_ptr(),
            plan.workspace.data_ptr(), plan.workspace_bytes, 1_000_000, stream), cuda_device)
        assert plan.read_status() == M.MLA_ERR_DEVICE_TIMEOUT
        assert plan.read_status() == 0
        assert took < 1.0, took
        out.fill_(float("nan"))
        plan.run(qd, kp, vp, bt, cud, sl, out)
        assert plan.read_status() == 0
        picked = range(len(new)) if len(new) == 3 else (0, 3)
        for b in picked:
            rows = slice(cu[b], cu[b + 1])
            check_attention(out[rows], q[rows], *seqs[b], d ** -0.5, TYPES[dtype], f"after the timeout, sequence {b}")
