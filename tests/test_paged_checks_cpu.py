"""Refusals of the paged-cache operators that need no GPU: plans and dims in the
C ABI, null and misaligned pointers, and the Python binding's dtype, shape and
device checks, which name the argument."""

import ctypes

import pytest
import torch

import mla_latent_kv_21_b200 as M
from mla_latent_kv_21_b200 import _lib as L


def _dims(**kw):
    a = dict(q_heads=8, kv_heads=2, head_dim=128, softmax_scale=0.1, dtype="bf16", q_len=1, rope_dim=128)
    a.update(kw)
    return M.gqa_dims_for(**a)


BAD_DIMS = [
    (dict(q_heads=0), L.MLA_ERR_INVALID_ARG), (dict(kv_heads=3), L.MLA_ERR_INVALID_ARG),
    (dict(softmax_scale=float("inf")), L.MLA_ERR_INVALID_ARG), (dict(softmax_scale=0.0), L.MLA_ERR_INVALID_ARG),
    (dict(q_len=0), L.MLA_ERR_INVALID_ARG), (dict(rope_dim=144), L.MLA_ERR_INVALID_ARG),
    (dict(rope_dim=24), L.MLA_ERR_UNSUPPORTED), (dict(head_dim=96, rope_dim=0), L.MLA_ERR_UNSUPPORTED),
    (dict(page_size=32), L.MLA_ERR_UNSUPPORTED), (dict(dtype="fp32"), L.MLA_ERR_UNSUPPORTED),
    (dict(dtype="fp8"), L.MLA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_bad_dims(kw, status):
    d = _dims(**kw)
    for call in (lambda: M.GqaDecodePlan(d, [10], num_sms=148), lambda: M.GqaPrefillPlan(d, [10]),
                 lambda: L.mla_gqa_append(d, L.mla_gqa_append_args_t(), 1 << 20, 1024)):
        with pytest.raises(M.MlaError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("q_heads,kv_heads,q_len,ok", [(64, 1, 1, True), (65, 1, 1, False), (32, 8, 16, True), (32, 8, 17, False)])
def test_decode_rows(q_heads, kv_heads, q_len, ok):
    d = _dims(q_heads=q_heads, kv_heads=kv_heads, q_len=q_len)
    if ok:
        M.GqaDecodePlan(d, [10, 0], num_sms=148).close()
    else:
        with pytest.raises(M.MlaError) as e:
            M.GqaDecodePlan(d, [10, 0], num_sms=148)
        assert e.value.status == L.MLA_ERR_UNSUPPORTED


def test_plan_lengths():
    for make in (lambda x: M.GqaDecodePlan(_dims(), x, num_sms=148), lambda x: M.GqaPrefillPlan(_dims(), x)):
        for bad in ([], [5, -1]):
            with pytest.raises(M.MlaError) as e:
                make(bad)
            assert e.value.status == L.MLA_ERR_INVALID_ARG
        make([0]).close()
    with pytest.raises(M.MlaError) as e:
        M.GqaPrefillPlan(_dims(q_heads=129, kv_heads=1), [1])
    assert e.value.status == L.MLA_ERR_UNSUPPORTED


def test_workspace_holds_two_partials_per_worker():
    for lens, workers, G, n in (([1000] * 50, 0, 4, 1), ([10], 0, 4, 2), ([100000], 17, 16, 4)):
        plan = M.GqaDecodePlan(_dims(q_heads=2 * G, kv_heads=2, q_len=n), lens, num_sms=148, num_workers=workers)
        W = min(workers or 296, 2 * sum(-(-x // 64) for x in lens))
        assert plan.workspace_bytes >= 1024 + 2 * W * G * n * (128 + 2) * 4
        plan.close()


def test_null_and_misaligned_pointers():
    """Fake addresses: every check comes before any use."""
    fake = 1 << 20
    plan, ws = L.mla_gqa_decode_plan(_dims(), [100], num_sms=148)
    good = dict(plan=plan, q=fake, k_pool=fake, v_pool=fake, num_blocks=4, block_table=fake, block_table_stride=2,
                seq_lens_dev=fake, out=fake, workspace=fake, workspace_bytes=ws)
    for name, bad, status in [("q", 0, 1), ("q", fake + 8, 1), ("k_pool", fake + 2, 1), ("v_pool", 0, 1), ("out", fake + 4, 1),
                              ("block_table", 0, 1), ("seq_lens_dev", 0, 1), ("workspace", 0, 1), ("num_blocks", 0, 1),
                              ("block_table_stride", 0, 1), ("workspace_bytes", ws - 1, 3), ("num_blocks", 2 ** 31, 2)]:
        with pytest.raises(M.MlaError) as e:
            L.mla_gqa_decode_run(**dict(good, **{name: bad}))
        assert e.value.status == status, (name, bad)
    L.mla_gqa_decode_plan_destroy(plan)
    plan, ws = L.mla_gqa_prefill_plan(_dims(), [100])
    good = dict(plan=plan, q=fake, k_pool=fake, v_pool=fake, num_blocks=4, block_table=fake, block_table_stride=2,
                cu_seqlens_dev=fake, seq_lens_dev=fake, out=fake, workspace=fake, workspace_bytes=ws)
    for name, bad, status in [("q", fake + 8, 1), ("k_pool", 0, 1), ("cu_seqlens_dev", 0, 1), ("out", 0, 1),
                              ("workspace_bytes", ws - 1, 3), ("num_blocks", 2 ** 31, 2)]:
        with pytest.raises(M.MlaError) as e:
            L.mla_gqa_prefill_run(**dict(good, **{name: bad}))
        assert e.value.status == status, (name, bad)
    L.mla_gqa_prefill_plan_destroy(plan)


def test_block_counts_whose_product_overflows():
    """num_blocks times the key heads past 64 bits is too many, not few."""
    fake = 1 << 20
    plan, ws = L.mla_gqa_decode_plan(_dims(), [100], num_sms=148)
    plan2, ws2 = L.mla_gqa_prefill_plan(_dims(), [100])
    for blocks in (2 ** 62, 2 ** 63 - 1):
        for call in (lambda: L.mla_gqa_decode_run(plan, fake, fake, fake, blocks, fake, 2, fake, fake, fake, ws),
                     lambda: L.mla_gqa_prefill_run(plan2, fake, fake, fake, blocks, fake, 2, fake, fake, fake, fake, ws2),
                     lambda: L.mla_gqa_append(_dims(), _gqa_args(num_blocks=blocks), fake, 1024)):
            with pytest.raises(M.MlaError) as e:
                call()
            assert e.value.status == L.MLA_ERR_UNSUPPORTED
    L.mla_gqa_decode_plan_destroy(plan)
    L.mla_gqa_prefill_plan_destroy(plan2)


def test_timeout_selftest_limits():
    """[1 us, 2 s], checked before any device work."""
    fake = 1 << 20
    plan, ws = L.mla_gqa_decode_plan(_dims(), [100], num_sms=148)
    plan2, ws2 = L.mla_gqa_prefill_plan(_dims(), [100])
    for limit in (0, 999, 2_000_000_001):
        with pytest.raises(M.MlaError) as e:
            L.mla_gqa_decode_selftest_timeout(plan, fake, fake, fake, 4, fake, 2, fake, fake, fake, ws, limit)
        assert e.value.status == L.MLA_ERR_INVALID_ARG
        with pytest.raises(M.MlaError) as e:
            L.mla_gqa_prefill_selftest_timeout(plan2, fake, fake, fake, 4, fake, 2, fake, fake, fake, fake, ws2, limit)
        assert e.value.status == L.MLA_ERR_INVALID_ARG
    with pytest.raises(M.MlaError) as e:
        L.mla_gqa_decode_selftest_timeout(plan, fake, fake, fake, 4, fake, 2, fake, fake, fake, ws - 1, 1_000_000)
    assert e.value.status == L.MLA_ERR_WORKSPACE_TOO_SMALL
    L.mla_gqa_decode_plan_destroy(plan)
    L.mla_gqa_prefill_plan_destroy(plan2)


def _gqa_args(**kw):
    f = 1 << 20
    a = dict(k=f, k_token_stride=256, k_head_stride=128, v=f, v_token_stride=256, v_head_stride=128, q=f, q_token_stride=1024,
             q_head_stride=128, q_out=f, k_pool=f, v_pool=f, num_blocks=4, block_table=f, block_table_stride=2, batch=3,
             seq_lens=f, cu_seqlens=f, num_tokens=5, rope_table=f, rope_positions=10)
    a.update(kw)
    return L.mla_gqa_append_args_t(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=(1 << 20) + 8), 1), (dict(k_token_stride=12), 1), (dict(q_head_stride=4), 1),
    (dict(q_out=None), 1), (dict(k_pool=None), 1), (dict(rope_table=None), 1), (dict(rope_table=(1 << 20) + 4), 1),
    (dict(batch=0), 1), (dict(num_tokens=-1), 1), (dict(cu_seqlens=None), 1), (dict(block_table_stride=0), 1),
    (dict(num_blocks=2 ** 31), 2), (dict(num_tokens=2 ** 31), 2),
])
def test_gqa_append_arguments(kw, status):
    with pytest.raises(M.MlaError) as e:
        L.mla_gqa_append(_dims(), _gqa_args(**kw), 1 << 20, 1024)
    assert e.value.status == status
    with pytest.raises(M.MlaError) as e:
        L.mla_gqa_append(_dims(), _gqa_args(), 1 << 20, 1023)
    assert e.value.status == L.MLA_ERR_WORKSPACE_TOO_SMALL


def test_nothing_to_append_is_no_launch():
    L.mla_gqa_append(_dims(), _gqa_args(num_tokens=0, k=None, v=None), 1 << 20, 1024)


@pytest.mark.parametrize("dims,kw,status", [
    (dict(), dict(ckv=None), 1), (dict(), dict(k_rope=None), 1), (dict(), dict(q_rope_out=None), 1), (dict(), dict(rope_table=None), 1),
    (dict(), dict(kv_pool=None), 1), (dict(dtype="fp8"), dict(kv_scale=None), 1), (dict(dtype="fp8"), dict(ckv=(1 << 20) + 2), 1),
    (dict(dtype="fp8", latent_rank=250), dict(), 2), (dict(dtype="fp8", rope_dim=24), dict(), 2),
    (dict(dtype="fp8", latent_rank=256, rope_dim=272), dict(), 2), (dict(rope_dim=63), dict(), 2), (dict(latent_rank=520), dict(), 2),
    (dict(page_size=16), dict(), 2), (dict(heads=0), dict(), 1), (dict(), dict(cu_seqlens=None), 1), (dict(), dict(num_blocks=0), 1),
])
def test_latent_append_arguments(dims, kw, status):
    f = 1 << 20
    d = dict(heads=4, latent_rank=512, rope_dim=64, nope_dim=128, v_dim=128, q_len=1, softmax_scale=0.1, dtype="bf16")
    d.update(dims)
    a = dict(ckv=f, ckv_token_stride=576, k_rope=f, k_rope_token_stride=576, q_rope=f, q_rope_token_stride=256,
             q_rope_head_stride=64, q_rope_out=f, kv_pool=f, kv_rope=f, kv_scale=f, kv_rows=None, num_blocks=4, block_table=f,
             block_table_stride=2, batch=3, seq_lens=f, cu_seqlens=f, num_tokens=5, rope_table=f, rope_positions=10)
    a.update(kw)
    with pytest.raises(M.MlaError) as e:
        L.mla_latent_append(M.dims_for(**d), 0, L.mla_latent_append_args_t(**a), f, 1024)
    assert e.value.status == status


def test_fp16_is_not_a_type_of_the_latent_operators():
    d = M.dims_for(4, 512, 64, 128, 128, 1, 0.1, "bf16")
    d.dtype = L.MLA_FP16
    with pytest.raises(M.MlaError):
        L.mla_decode_plan(d, [10], 148)
    with pytest.raises(M.MlaError) as e:
        L.mla_latent_append(d, 0, L.mla_latent_append_args_t(), 1 << 20, 1024)
    assert e.value.status == L.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------ the binding's checks --
def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


GQA_APPEND = dict(k=_z(5, 2, 128), v=_z(5, 2, 128), k_pool=_z(4, 2, 64, 128), v_pool=_z(4, 2, 64, 128), block_table=_i(3, 2),
                  seq_lens=_i(3), rope_table=_z(9, 128, dtype=torch.float32), q=_z(5, 8, 128), q_out=_z(5, 8, 128), cu_seqlens=_i(4))
DECODE = dict(q=_z(3, 1, 8, 128), k_pool=_z(4, 2, 64, 128), v_pool=_z(4, 2, 64, 128), block_table=_i(3, 2), seq_lens=_i(3),
              out=_z(3, 1, 8, 128))
PREFILL = dict(q=_z(6, 8, 128), k_pool=_z(4, 2, 64, 128), v_pool=_z(4, 2, 64, 128), block_table=_i(3, 2), cu_seqlens=_i(4),
               seq_lens=_i(3), out=_z(6, 8, 128))
LATENT = dict(ckv=_z(5, 512), k_rope=_z(5, 64), kv_pool=_z(4, 64, 576), block_table=_i(3, 2), seq_lens=_i(3),
              rope_table=_z(9, 64, dtype=torch.float32), q_rope=_z(5, 4, 64), q_rope_out=_z(5, 4, 64), kv_rows=_z(5, 576),
              cu_seqlens=_i(4))


def _latent():
    return M.LatentAppend(M.dims_for(4, 512, 64, 128, 128, 1, 0.1, "bf16"))


CALLS = {"append": (lambda: M.GqaAppend(_dims()), GQA_APPEND), "latent": (_latent, LATENT),
         "decode": (lambda: M.GqaDecodePlan(_dims(), [1, 2, 3], num_sms=148), DECODE),
         "prefill": (lambda: M.GqaPrefillPlan(_dims(), [1, 2, 3]), PREFILL)}


@pytest.mark.parametrize("which", sorted(CALLS))
def test_every_argument_is_checked(which):
    """CPU tensors of the right shape stop at the device check; a wrong type or shape names its argument."""
    make, good = CALLS[which]
    with pytest.raises(ValueError, match="CUDA tensor"):
        make().run(**good)
    for name, t in good.items():
        wrong = t.double() if t.is_floating_point() else t.long()
        with pytest.raises(ValueError, match=f"^{name}"):
            make().run(**dict(good, **{name: wrong}))
        with pytest.raises(ValueError, match="needed"):
            make().run(**dict(good, **{name: t[..., None]}))
        if name not in ("block_table", "k_pool"):   # any width; the first pool sets the number of blocks
            with pytest.raises(ValueError):
                make().run(**dict(good, **{name: t[..., :-1].contiguous()}))


def test_missing_and_mixed_arguments():
    with pytest.raises(ValueError, match="together"):
        M.GqaAppend(_dims()).run(**dict(GQA_APPEND, q_out=None))
    with pytest.raises(ValueError, match="rope_table is needed"):
        M.GqaAppend(_dims()).run(**dict(GQA_APPEND, rope_table=None))
    with pytest.raises(ValueError, match="without cu_seqlens"):
        M.GqaAppend(_dims()).run(**dict(GQA_APPEND, cu_seqlens=None))
    with pytest.raises(ValueError, match="without cu_seqlens"):
        _latent().run(**dict(LATENT, cu_seqlens=None))
    with pytest.raises(ValueError, match="run_fp8"):
        M.LatentAppend(M.dims_for(4, 512, 64, 128, 128, 1, 0.1, "fp8")).run(**LATENT)
    with pytest.raises(ValueError, match="dtype 'fp8'"):
        _latent().run_fp8(*([None] * 8))
    with pytest.raises(KeyError):
        M.gqa_dims_for(8, 2, 128, 0.1, rope_style="other")


def test_struct_layouts_match_the_header():
    """Sizes of the argument structs as the C compiler lays them out (LP64: every member naturally aligned)."""
    assert ctypes.sizeof(L.mla_gqa_dims_t) == 36
    assert ctypes.sizeof(L.mla_gqa_append_args_t) == 8 * 14 + 8 + 8 * 5
    assert ctypes.sizeof(L.mla_latent_append_args_t) == 8 * 14 + 8 + 8 * 5


def test_rope_table():
    t = M.rope_table(300, 64, device="cpu")
    assert t.shape == (300, 64) and t.dtype == torch.float32 and (t[0, :32] == 1).all() and (t[0, 32:] == 0).all()
    a = 299 * 10000.0 ** (-10 / 64)
    assert abs(float(t[299, 5]) - torch.cos(torch.tensor(a, dtype=torch.float64)).item()) < 1e-7
