"""The serving operators around a paged cache, as a user's program calls them, with
their plain forms: appending keys and values to the grouped-head cache and latent
rows to the MLA caches (bf16 and FP8) with the position rotation on the way,
attention of the newest tokens over the paged grouped-head cache, and causal
attention of packed prompts over the same cache.

Where `own` is false, `run` computes an operator with elementary torch operations in
32 bits; where it is true, it calls the library. Both write into the same buffers.
"""

import math
import random

import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.bfloat16}
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -64   # smallest token scale of the FP8 cache


# ------------------------------------------------------------------- cases ----
def listed():
    return [
        # One decode step of a small batch: the new token's keys and values go into the cache and its query is rotated.
        dict(name="gqa_append step 4", op="gqa_append", dtype="bf16", q_heads=32, kv_heads=8, head_dim=128, rope_dim=128,
             style="half", batch=4, new=1, len_lo=40, len_hi=700, pick=1),
        # Ragged prompts written behind earlier chunks, rotation of half the head in the interleaved order.
        dict(name="gqa_append prompts 16K", op="gqa_append", dtype="fp16", q_heads=32, kv_heads=4, head_dim=128, rope_dim=64,
             style="interleaved", batch=12, new=0, len_lo=200, len_hi=4000, pick=2),
        # One decode step over the FP8 latent cache: 64 sequences, 128 query heads.
        dict(name="latent_append fp8 step 64", op="latent_append", dtype="fp8", heads=128, rank=512, rope_dim=64,
             style="interleaved", batch=64, new=1, len_lo=60, len_hi=900, rows=False, pick=3),
        # Two long prompts into the bf16 latent cache, with the packed rows that the prefill attends over.
        dict(name="latent_append bf16 prompts", op="latent_append", dtype="bf16", heads=128, rank=512, rope_dim=64,
             style="half", batch=2, new=0, len_lo=8192, len_hi=8192, rows=True, pick=4),
        # A single user's decode step on a short context: latency counts.
        dict(name="gqa_decode 1 x 500", op="gqa_decode", dtype="bf16", q_heads=32, kv_heads=8, head_dim=128, q_len=1,
             batch=1, len_lo=500, len_hi=500, idle=False, pick=5),
        # The multi-head original of the 16 x 8K decode workload: 32 heads with a key and a value each.
        dict(name="gqa_decode 16 x 8K mha", op="gqa_decode", dtype="bf16", q_heads=32, kv_heads=32, head_dim=128, q_len=1,
             batch=16, len_lo=8192, len_hi=8192, idle=False, pick=6),
        # A served batch of mixed lengths with two query tokens per sequence and idle slots.
        dict(name="gqa_decode 64 ragged mtp", op="gqa_decode", dtype="fp16", q_heads=64, kv_heads=8, head_dim=128, q_len=2,
             batch=64, len_lo=1, len_hi=16384, idle=True, pick=7),
        # One very long context: the split over the cache's length carries it.
        dict(name="gqa_decode 1 x 128K", op="gqa_decode", dtype="bf16", q_heads=64, kv_heads=4, head_dim=128, q_len=1,
             batch=1, len_lo=131071, len_hi=131071, idle=False, pick=8),
        # A chat prompt of a few words.
        dict(name="gqa_prefill 1 x 37", op="gqa_prefill", dtype="bf16", q_heads=32, kv_heads=8, head_dim=128, batch=1,
             new_lo=37, new_hi=37, prefix_hi=0, pick=9),
        # A packed batch of prompts of different lengths, seven query heads to a key head.
        dict(name="gqa_prefill 8 ragged", op="gqa_prefill", dtype="fp16", q_heads=28, kv_heads=4, head_dim=128, batch=8,
             new_lo=30, new_hi=2999, prefix_hi=0, pick=10),
        # The long prompt.
        dict(name="gqa_prefill 1 x 8K", op="gqa_prefill", dtype="bf16", q_heads=32, kv_heads=8, head_dim=128, batch=1,
             new_lo=8192, new_hi=8192, prefix_hi=0, pick=11),
        # Chunks of prompts whose earlier chunks are in the cache, small heads.
        dict(name="gqa_prefill chunks d64", op="gqa_prefill", dtype="bf16", q_heads=16, kv_heads=16, head_dim=64, batch=5,
             new_lo=400, new_hi=1100, prefix_hi=5000, pick=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gqa_append", "latent_append", "gqa_decode", "gqa_decode", "gqa_prefill", "gqa_prefill"])
    pick = rng.randrange(1 << 30)
    if op == "latent_append":
        return dict(op=op, dtype=rng.choice(["bf16", "fp8", "fp32"]), heads=rng.choice([8, 16, 32, 64, 128]),
                    rank=rng.choice([256, 512]), rope_dim=64, style=rng.choice(["half", "interleaved"]),
                    batch=_log_int(rng, 1, 64), new=rng.choice([0, 1, 1, 2]), len_lo=_log_int(rng, 2, 200), len_hi=_log_int(rng, 200, 500),
                    rows=rng.random() < 0.5, pick=pick)
    kv_heads = rng.choice([1, 2, 4, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * kv_heads <= 64])
    head = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), q_heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=rng.choice([64, 128, 128]), pick=pick)
    if op == "gqa_append":
        return dict(head, rope_dim=rng.choice([head["head_dim"], head["head_dim"] // 2, 32]), style=rng.choice(["half", "interleaved"]),
                    batch=_log_int(rng, 1, 64), new=rng.choice([0, 1, 1, 3]), len_lo=_log_int(rng, 3, 100), len_hi=_log_int(rng, 100, 500))
    if op == "gqa_decode":
        q_len = rng.choice([1, 1, 2, 3, 4])
        q_len = min(q_len, 64 // group)
        batch = _log_int(rng, 1, 128)
        most = max(2, min(60000, 4_000_000 // (batch * kv_heads)))   # at most 4 M key rows of 128 (2 GB with the values)
        hi = _log_int(rng, 2, most)
        return dict(head, q_len=q_len, batch=batch, len_lo=_log_int(rng, 1, hi), len_hi=hi, idle=rng.random() < 0.3)
    batch = _log_int(rng, 1, 16)
    most = int(math.sqrt(1.0e9 / (batch * head["q_heads"])))         # the scores of a pass: at most 1e9
    hi = _log_int(rng, 1, most)
    prefix = rng.choice([0, 0, _log_int(rng, 1, 2000)])
    prefix = min(prefix, most * most // hi - hi)
    return dict(head, batch=batch, new_lo=_log_int(rng, 1, hi), new_hi=hi, prefix_hi=max(0, prefix))


def _between(rng, lo, hi):
    return lo if lo == hi else _log_int(rng, lo, hi)


def _counts(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    rng = random.Random(case["pick"])
    B = case["batch"]
    if case["op"] == "gqa_prefill":
        new = [_between(rng, case["new_lo"], case["new_hi"]) for _ in range(B)]
        return new, [n + rng.randint(0, case["prefix_hi"]) for n in new]
    lens = [_between(rng, case["len_lo"], case["len_hi"]) for _ in range(B)]
    if case["op"] == "gqa_decode":
        if case["idle"]:
            lens = [0 if b % 5 == 4 else n for b, n in enumerate(lens)]
        return [case["q_len"]] * B, lens
    if case["new"]:
        return [case["new"]] * B, [max(n, case["new"]) for n in lens]
    # prompts: the last two thirds or more of what the cache then holds
    return [n - rng.randint(0, n // 3) if case["len_lo"] != case["len_hi"] else n for n in lens], lens


# ------------------------------------------------------------------ inputs ----
def _normal(shape, dtype, gen, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _pages(lens, gen):
    """A block table in random page order (-1 where a sequence has no page), and the number of pages."""
    need = [-(-n // PAGE) for n in lens]
    total, width = max(1, sum(need)), max(1, max(need))
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    row = torch.arange(width, device="cuda")
    need_t = torch.tensor(need, device="cuda")
    start = torch.cumsum(need_t, 0) - need_t
    at = (start[:, None] + row[None, :]).clamp(max=total - 1)
    return torch.where(row[None, :] < need_t[:, None], order[at], -1).to(torch.int32).contiguous(), total


def _table(positions, rope_dim, base=10000.0):
    """cos in the first half of the columns, sin in the second."""
    inv = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device="cuda") / rope_dim)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1_000_003 + case["pick"] % 999_983)
    new, lens = _counts(case)
    T, op, dt = sum(new), case["op"], TYPES[case["dtype"]]
    s = dict(case=case, new=new, lens=lens, T=T, seq_lens=_int32(lens))
    s["block_table"], blocks = _pages(lens, gen)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = _int32(cu)
    if op == "latent_append":
        r, dr, H = case["rank"], case["rope_dim"], case["heads"]
        # one projection gives the latent and the key's rotary part, another the queries of all heads
        kv = _normal((T, r + dr), dt, gen)
        q = _normal((T, H, 128 + dr), dt, gen)
        s.update(ckv=kv[:, :r], k_rope=kv[:, r:], q_rope=q[:, :, 128:], q_rope_out=torch.zeros((T, H, dr), dtype=dt, device="cuda"),
                 table=_table(max(lens) + 1, dr), kv_rows=torch.zeros((T, r + dr), dtype=dt, device="cuda") if case["rows"] else None)
        if case["dtype"] == "fp8":
            s.update(codes=torch.randint(0, 120, (blocks, PAGE, r), dtype=torch.uint8, device="cuda", generator=gen),
                     rope=_normal((blocks, PAGE, dr), dt, gen, 30.0), scale=torch.rand((blocks, PAGE), device="cuda", generator=gen) + 0.01)
        else:
            s["pool"] = _normal((blocks, PAGE, r + dr), dt, gen)
    else:
        Hq, Hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        s["k_pool"] = _normal((blocks, Hk, PAGE, d), dt, gen)
        s["v_pool"] = _normal((blocks, Hk, PAGE, d), dt, gen)
        if op == "gqa_append":
            qkv = _normal((T, Hq + 2 * Hk, d), dt, gen)
            s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], q_out=torch.zeros((T, Hq, d), dtype=dt, device="cuda"),
                     table=_table(max(lens) + 1, case["rope_dim"]))
        elif op == "gqa_decode":
            # queries of twice the unit size: scores spread like those of trained heads
            s["q"] = _normal((case["batch"], case["q_len"], Hq, d), dt, gen, 2.0)
        else:
            s["q"] = _normal((T, Hq, d), dt, gen, 2.0)
        s["out"] = torch.zeros_like(s["q"]) if op != "gqa_append" else None
        s["softmax_scale"] = d ** -0.5
    if own:
        s["call"] = _own_call(case, s)
    return s


# ---------------------------------------------------------- the library's calls ----
def _own_call(case, s):
    """The plan or handle that a program keeps for these inputs."""
    import mla_latent_kv_21_b200 as M
    op = case["op"]
    if op == "latent_append":
        dims = M.dims_for(case["heads"], case["rank"], case["rope_dim"], 128, 128, max(1, case["new"]),
                          (128 + case["rope_dim"]) ** -0.5, case["dtype"])
        return M.LatentAppend(dims, rope_style=case["style"]).allocate_workspace("cuda")
    if op == "gqa_append":
        return M.GqaAppend(M.gqa_dims_for(case["q_heads"], case["kv_heads"], case["head_dim"], s["softmax_scale"], case["dtype"],
                                          q_len=max(1, case["new"]), rope_dim=case["rope_dim"],
                                          rope_style=case["style"])).allocate_workspace("cuda")
    dims = M.gqa_dims_for(case["q_heads"], case["kv_heads"], case["head_dim"], s["softmax_scale"], case["dtype"],
                          q_len=case.get("q_len", 1))
    if op == "gqa_decode":
        return M.GqaDecodePlan(dims, s["lens"]).allocate_workspace("cuda")
    return M.GqaPrefillPlan(dims, s["new"]).allocate_workspace("cuda")


def _run_own(s):
    case, call = s["case"], s["call"]
    op = case["op"]
    if op == "latent_append":
        more = dict(q_rope=s["q_rope"], q_rope_out=s["q_rope_out"], kv_rows=s["kv_rows"], cu_seqlens=None if case["new"] else s["cu"])
        if case["dtype"] == "fp8":
            call.run_fp8(s["ckv"], s["k_rope"], s["codes"], s["rope"], s["scale"], s["block_table"], s["seq_lens"], s["table"], **more)
        else:
            call.run(s["ckv"], s["k_rope"], s["pool"], s["block_table"], s["seq_lens"], s["table"], **more)
    elif op == "gqa_append":
        call.run(s["k"], s["v"], s["k_pool"], s["v_pool"], s["block_table"], s["seq_lens"], s["table"], q=s["q"], q_out=s["q_out"],
                 cu_seqlens=None if case["new"] else s["cu"])
    elif op == "gqa_decode":
        call.run(s["q"], s["k_pool"], s["v_pool"], s["block_table"], s["seq_lens"], s["out"])
    else:
        call.run(s["q"], s["k_pool"], s["v_pool"], s["block_table"], s["cu"], s["seq_lens"], s["out"])
    return _outputs(s)


def _outputs(s):
    op = s["case"]["op"]
    if op == "latent_append":
        got = [s["codes"].view(torch.float8_e4m3fn), s["rope"], s["scale"]] if s["case"]["dtype"] == "fp8" else [s["pool"]]
        return got + [s["q_rope_out"]] + ([s["kv_rows"]] if s["kv_rows"] is not None else [])
    return [s["k_pool"], s["v_pool"], s["q_out"]] if op == "gqa_append" else s["out"]


# -------------------------------------------------------------- plain forms ----
def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "latent_append":
        return _plain_latent_append(s)
    if op == "gqa_append":
        return _plain_gqa_append(s)
    return _plain_decode(s) if op == "gqa_decode" else _plain_prefill(s)


def _places(s):
    """(position, block, slot) of every new token."""
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - (cu[b + 1] - t)
    return pos, s["block_table"][b, pos // PAGE].long(), pos % PAGE


def _rotated(x, table, pos, style):
    """x [T, heads, d] in 32 bits with its first columns rotated by the positions' angles."""
    dr = table.shape[1]
    cos, sin = table[pos, None, :dr // 2], table[pos, None, dr // 2:]
    x = x.float()
    if style == "half":
        a, b, rest = x[..., :dr // 2], x[..., dr // 2:dr], x[..., dr:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)
    a, b, rest = x[..., 0:dr:2], x[..., 1:dr:2], x[..., dr:]
    pair = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([pair, rest], dim=-1)


def _plain_gqa_append(s):
    pos, block, slot = _places(s)
    style = s["case"]["style"]
    s["k_pool"][block, :, slot] = _rotated(s["k"], s["table"], pos, style).to(s["k_pool"].dtype)
    s["v_pool"][block, :, slot] = s["v"]
    s["q_out"].copy_(_rotated(s["q"], s["table"], pos, style))
    return _outputs(s)


def _plain_latent_append(s):
    pos, block, slot = _places(s)
    case = s["case"]
    key = _rotated(s["k_rope"][:, None, :], s["table"], pos, case["style"])[:, 0]
    if case["dtype"] == "fp8":
        c = s["ckv"].float()
        scale = (c.abs().amax(dim=1) / E4M3_MAX).clamp(min=MIN_SCALE)
        s["codes"][block, slot] = (c / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["rope"][block, slot] = (key / scale[:, None]).to(torch.bfloat16)
        s["scale"][block, slot] = scale
    else:
        s["pool"][block, slot] = torch.cat([s["ckv"], key.to(s["pool"].dtype)], dim=1)
    if s["kv_rows"] is not None:
        s["kv_rows"].copy_(torch.cat([s["ckv"].float(), key], dim=1))
    s["q_rope_out"].copy_(_rotated(s["q_rope"], s["table"], pos, case["style"]))
    return _outputs(s)


def _cache(pool, table):
    """[B, heads, tokens, d] in 32 bits: every sequence's pages side by side."""
    x = pool[table.clamp(min=0).long()]
    B, P, H, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * PAGE, d).float()


def _attend(q, k, v, visible, scale):
    """q [B, Hk, rows, d], k and v [B, Hk, tokens, d], visible [B, 1, rows, tokens]; a row that sees nothing is zero."""
    s = torch.matmul(q, k.transpose(2, 3)).mul_(scale)
    s = s.masked_fill_(~visible, -math.inf)
    top = s.amax(dim=3, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=3, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_decode(s):
    case = s["case"]
    B, n, Hq, d = s["q"].shape
    Hk = case["kv_heads"]
    G = Hq // Hk
    k, v = _cache(s["k_pool"], s["block_table"]), _cache(s["v_pool"], s["block_table"])
    # beyond a sequence's end the values are other sequences' or old ones
    inside = torch.arange(v.shape[2], device=v.device)[None, :] < s["seq_lens"][:, None]
    v = v.mul_(inside[:, None, :, None])
    q = s["q"].float().view(B, n, Hk, G, d).transpose(1, 2).reshape(B, Hk, n * G, d)
    row = torch.arange(n * G, device=q.device) // G
    last = s["seq_lens"][:, None] - n + row[None, :]
    visible = torch.arange(k.shape[2], device=q.device)[None, None, :] <= last[:, :, None]
    o = _attend(q, k, v, visible[:, None], s["softmax_scale"])
    s["out"].copy_(o.view(B, Hk, n, G, d).transpose(1, 2).reshape(B, n, Hq, d))
    return s["out"]


def _plain_prefill(s):
    case = s["case"]
    T, Hq, d = s["q"].shape
    Hk = case["kv_heads"]
    G, B, most = Hq // Hk, case["batch"], max(s["new"])
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    k, v = _cache(s["k_pool"], s["block_table"]), _cache(s["v_pool"], s["block_table"])
    inside = torch.arange(v.shape[2], device=v.device)[None, :] < lens[:, None]
    v = v.mul_(inside[:, None, :, None])
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device=k.device)
    real = i[None, :] < count[:, None]
    at = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    q = s["q"][at].float().view(B, most, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * most, d)
    last = torch.where(real, lens[:, None] - count[:, None] + i[None, :], -1)
    visible = torch.arange(k.shape[2], device=k.device)[None, None, :] <= last[:, :, None]
    o = _attend(q, k, v, visible.repeat(1, G, 1)[:, None], s["softmax_scale"])
    o = o.view(B, Hk, G, most, d).permute(0, 3, 1, 2, 4).reshape(B, most, Hq, d)
    s["out"].copy_(o[real])
    return s["out"]


# --------------------------------------------------------------------- work ----
def work(case):
    new, lens = _counts(case)
    T, e = sum(new), 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "latent_append":
        r, dr, H = case["rank"], case["rope_dim"], case["heads"]
        token = (r + dr) * e + 2 * H * dr * e + dr * 4            # latent and key in, queries in and out, table row
        token += r + 2 * dr + 4 if case["dtype"] == "fp8" else (r + dr) * e
        token += (r + dr) * e if case["rows"] else 0
        return {"bytes": T * token, "flops": T * (3 * dr * (H + 1) + (2 * r if case["dtype"] == "fp8" else 0))}
    Hq, Hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "gqa_append":
        return {"bytes": T * ((2 * Hq + 4 * Hk) * d * e + case["rope_dim"] * 4), "flops": T * 3 * case["rope_dim"] * (Hq + Hk)}
    seen = sum(max(0, L - n + i + 1) for n, L in zip(new, lens) for i in range(n))
    return {"bytes": 2 * T * Hq * d * e + 2 * sum(lens) * Hk * d * e, "flops": 4 * d * Hq * seen}


# ------------------------------------------------- the definitions in 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gqa_decode", "gqa_prefill"):
        return _exact_attention(s)
    turn = _exact_turn(s)
    table, PG = s["block_table"].tolist(), PAGE
    where = []
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        where += [(table[b][p // PG], p % PG) for p in range(L - n, L)]
    blk = torch.tensor([w[0] for w in where], device="cuda")
    slot = torch.tensor([w[1] for w in where], device="cuda")
    if op == "gqa_append":
        k, v = s["k_pool"].double(), s["v_pool"].double()
        k[blk, :, slot] = turn(s["k"].double())
        v[blk, :, slot] = s["v"].double()
        return [k, v, turn(s["q"].double())]
    c, key = s["ckv"].double(), turn(s["k_rope"].double().unsqueeze(1)).squeeze(1)
    if case["dtype"] == "fp8":
        size = torch.linalg.vector_norm(c, ord=math.inf, dim=1).div(E4M3_MAX).clamp(min=MIN_SCALE)
        codes = s["codes"].view(torch.float8_e4m3fn).double()
        codes[blk, slot] = (c / size.unsqueeze(1)).float().to(torch.float8_e4m3fn).double()
        rope, scale = s["rope"].double(), s["scale"].double()
        rope[blk, slot] = key / size.unsqueeze(1)
        scale[blk, slot] = size
        got = [codes, rope, scale]
    else:
        pool = s["pool"].double()
        pool[blk, slot] = torch.hstack([c, key])
        got = [pool]
    return got + [turn(s["q_rope"].double())] + ([torch.hstack([c, key])] if s["kv_rows"] is not None else [])


def _exact_turn(s):
    """The rotation as a product with a complex number per pair."""
    where = torch.tensor([p for n, L in zip(s["new"], s["lens"]) for p in range(L - n, L)], device="cuda")
    t = s["table"].double()[where]
    half = t.shape[1] // 2
    unit = torch.complex(t[:, :half], t[:, half:]).unsqueeze(1)

    def turn(x):
        y = x.clone()
        even, odd = (slice(0, half), slice(half, 2 * half)) if s["case"]["style"] == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        z = torch.complex(x[..., even], x[..., odd]) * unit
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    return turn


def _exact_attention(s):
    """One sequence and one key head at a time, softmax over the keys that a query sees."""
    case = s["case"]
    if work(case)["flops"] > 3e12:
        return None
    Hq, Hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    G, q = Hq // Hk, s["q"].reshape(-1, Hq, d)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        rows = slice(start, start + n)
        start += n
        if L == 0:
            continue
        ids = s["block_table"][b, :-(-L // PAGE)].long()
        # a query at position p sees the keys 0 to p; one before the cache's first key sees none
        first = max(0, n - L)
        unseen = torch.ones(n - first, L, device="cuda", dtype=torch.bool).triu(L - (n - first) + 1)
        for h in range(Hk):
            k = s["k_pool"][ids, h].reshape(-1, d)[:L].double()
            v = s["v_pool"][ids, h].reshape(-1, d)[:L].double()
            for g in range(h * G, (h + 1) * G):
                e = q[rows, g].double()[first:] @ k.T * s["softmax_scale"]
                out[rows, g][first:] = e.masked_fill(unseen, -math.inf).softmax(dim=1) @ v
    return out.reshape(s["q"].shape)
