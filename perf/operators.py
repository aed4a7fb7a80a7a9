"""Measured cases of the packed-prompt and attention-cache operators.

Four operators of one serving step of a hybrid model whose requests have different lengths:

  tables   request lengths -> block table, slot map, positions, packed offsets (whole numbers)
  append   a step's keys and values into the paged 4-bit cache, and back as the values it holds
  attend   causal grouped-query attention over that cache: one token per request, drafts, prompt chunks
  gdn      the gated delta rule over packed prompts: every token's output and the state after each prompt

``run`` computes them in plain torch where ``own`` is false and through the library where it is true.
``exact`` is the definition in 64 bits.  Lengths follow from a case's own ``lens_seed``, values from the
seed given to ``prepare``.

The cache is uint8 [pages][kv heads][page_size * 9/8 * head_dim]; the bytes of one page and head are the K
codes [page_size][head_dim / 2] (element 2i in the low half of byte i), the K block scales
[page_size][head_dim / 16], then V's codes and scales.  A code is e2m1, a block scale e4m3 over 16 elements,
and a value is code * block scale * tensor scale, the tensor scale a power of two.
"""
import math
import random

import torch

own = False

HEADS_GDN = 32   # heads of the Gated DeltaNet workload (d_k = d_v = 128)
Q_HEADS, KV_HEADS, HEAD_DIM = 32, 2, 128  # attention layer of the hybrid step
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's bookkeeping: one token for each of 256 requests, ragged contexts
        dict(name="tables_decode_b256", op="tables", batch=256, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8192,
             page=64, pad=0, lens_seed=1),
        # a packed prefill step: prompts of 0 to 4096 tokens, some continuing, padded to a fixed capacity
        dict(name="tables_prefill_b96", op="tables", batch=96, new_lo=0, new_hi=4096, ctx_lo=0, ctx_hi=2048,
             page=16, pad=1000, lens_seed=2),
        # the write of a decode step (256 tokens, 2 key/value heads)
        dict(name="append_decode_t256", op="append", tokens=256, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64,
             k_exp=0, v_exp=-2, lens_seed=3),
        # the write of a packed prefill step, an odd number of tokens, 8 heads of 64
        dict(name="append_prefill_t65521", op="append", tokens=65521, kv_heads=8, dim=64, page=16, k_exp=1,
             v_exp=-3, lens_seed=4),
        # one request decoding alone over a long context: latency
        dict(name="attend_b1_c4096", op="attend", batch=1, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=4096,
             q_heads=Q_HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, k_exp=0, v_exp=-2, lens_seed=5),
        # the hybrid step's attention layer at its own batch and context
        dict(name="attend_b256_c4096", op="attend", batch=256, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=4096,
             q_heads=Q_HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=64, k_exp=0, v_exp=-2, lens_seed=6),
        # speculative verify: 4 drafts per request, ragged contexts, small pages, 4 query heads per kv head
        dict(name="attend_verify_b128_k4", op="attend", batch=128, new_lo=4, new_hi=4, ctx_lo=1, ctx_hi=8192,
             q_heads=32, kv_heads=8, dim=64, page=16, k_exp=1, v_exp=0, lens_seed=7),
        # a chunk of each prompt attending to the chunks before it
        dict(name="attend_chunk_b8", op="attend", batch=8, new_lo=100, new_hi=512, ctx_lo=0, ctx_hi=4096,
             q_heads=Q_HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=32, k_exp=0, v_exp=0, lens_seed=8),
        # a handful of short prompts, an empty one among them possible: latency
        dict(name="gdn_short_b8", op="gdn", batch=8, len_lo=0, len_hi=64, heads=HEADS_GDN, dk=128, dv=128,
             type="bf16", state=True, lens_seed=9),
        # a packed batch of ragged prompts at the Gated DeltaNet workload's shape
        dict(name="gdn_ragged_b64", op="gdn", batch=64, len_lo=1, len_hi=1024, heads=HEADS_GDN, dk=128, dv=128,
             type="bf16", state=True, lens_seed=10),
        # one long prompt alone
        dict(name="gdn_long_b1", op="gdn", batch=1, len_lo=8191, len_hi=8191, heads=HEADS_GDN, dk=128, dv=128,
             type="bf16", state=False, lens_seed=11),
        # fp32 inputs and a smaller state (the library's other input type)
        dict(name="gdn_f32_b16", op="gdn", batch=16, len_lo=1, len_hi=200, heads=16, dk=64, dv=64, type="f32",
             state=True, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "gdn", "gdn"])
    seed = rng.randrange(1 << 20)
    if op == "tables":
        b = _log(rng, 1, 256)
        new_hi = rng.choice([1, 4, _log(rng, 1, max(1, min(4096, 196608 // b)))])
        return dict(op=op, batch=b, new_lo=rng.choice([0, min(1, new_hi)]), new_hi=new_hi, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 8192), page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 1, 333]),
                    lens_seed=seed)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), k_exp=rng.randint(-3, 3), v_exp=rng.randint(-3, 3),
                    lens_seed=seed)
    if op == "attend":
        kv, group, dim = rng.choice([1, 2, 8]), rng.choice([1, 4, 7, 16]), rng.choice([64, 128])
        kind = rng.choice(["decode", "verify", "chunk"])
        if kind == "chunk":
            b, new = _log(rng, 1, 4), _log(rng, 9, 256)
            kv = min(kv, 2)
        else:
            b, new = _log(rng, 1, 128), 1 if kind == "decode" else rng.randint(2, 8)
        ctx = _log(rng, 1, max(1, min(2048 if kind == "chunk" else 8192, 524288 // (b * kv))))
        return dict(op=op, batch=b, new_lo=1 if kind == "chunk" else new, new_hi=new, ctx_lo=ctx // 3, ctx_hi=ctx,
                    q_heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    k_exp=rng.randint(-2, 2), v_exp=rng.randint(-2, 2), lens_seed=seed)
    typ = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 128]) if typ == "f32" else 128
    dv = dim if typ == "f32" else rng.choice([64, 128])
    heads = rng.choice([4, 16, 32]) if typ == "bf16" else rng.choice([4, 16])
    b = _log(rng, 1, 48)
    hi = _log(rng, 1, max(1, min(4096 if typ == "bf16" else 200, 24576 // b)))
    return dict(op=op, batch=b, len_lo=min(1, hi // 2), len_hi=hi, heads=heads, dk=dim, dv=dv, type=typ,
                state=rng.random() < 0.5, lens_seed=seed)


def _lens(case):
    """The lengths of a case's requests, from the case alone."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "gdn":
        lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
        return [max(1, lens[0])] + lens[1:]  # at least one token in all
    return ([r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])],
            [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])])


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend,
            "gdn": _prepare_gdn}[case["op"]](case, g) | {"case": dict(case)}


def _prepare_tables(case, g):
    ctx, new = _lens(case)
    ps = case["page"]
    held = [_ceil(c, ps) for c in ctx]
    width = max(1, max(_ceil(c + n, ps) for c, n in zip(ctx, new)))
    need = sum(_ceil(c + n, ps) - h for c, n, h in zip(ctx, new, held))
    pages = torch.randperm(sum(held) + need + 7, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")
    mine = at < torch.tensor(held, device="cuda")[:, None]
    table[mine] = pages[:sum(held)]
    return dict(cached_len=_i32(ctx), new_len=_i32(new), free_pages=pages[sum(held):].clone(), free_head=_i32([3]),
                block_table=table, page_size=ps, max_tokens=max(1, sum(new) + case["pad"]))


def _kv(case, g, tokens):
    """Keys with a few strong channels and values, both bf16, as projections give them."""
    sh = (tokens, case["kv_heads"], case["dim"])
    chan = torch.exp(0.7 * torch.randn((1,) + sh[1:], generator=g, device="cuda"))
    k = torch.randn(sh, generator=g, device="cuda") * chan * 2.0 ** case["k_exp"]
    v = torch.randn(sh, generator=g, device="cuda") * 2.0 ** case["v_exp"]
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _prepare_append(case, g):
    n, ps = case["tokens"], case["page"]
    k, v = _kv(case, g, n)
    pages = _ceil(n, ps) + 3
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    slots = order[(t // ps).long()] * ps + t % ps
    cache = torch.zeros((pages, case["kv_heads"], ps * case["dim"] * 9 // 8), dtype=torch.uint8, device="cuda")
    return dict(k=k, v=v, slot_map=slots, cache=cache, k_scale=2.0 ** (case["k_exp"] - 4), v_scale=2.0 ** (case["v_exp"] - 4))


def _prepare_attend(case, g):
    ctx, new = _lens(case)
    ps, D, Hk = case["page"], case["dim"], case["kv_heads"]
    total = [c + n for c, n in zip(ctx, new)]
    held = [_ceil(t, ps) for t in total]
    pages, width = sum(held) + 1, max(held)
    k_scale, v_scale = 2.0 ** (case["k_exp"] - 4), 2.0 ** (case["v_exp"] - 4)
    cache = torch.empty((pages, Hk, ps * D * 9 // 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (Hk * ps * D))
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        k, v = _kv(case, g, n * ps)
        cache[p0:p0 + n] = _pack(_quantise(k.float(), k_scale), _quantise(v.float(), v_scale), n, ps)
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    mine = torch.arange(width, device="cuda") < torch.tensor(held, device="cuda")[:, None]
    table[mine] = order[:sum(held)]
    q = torch.randn((sum(new), case["q_heads"], D), generator=g, device="cuda") * 2.0 ** -case["k_exp"]
    return dict(q=q.to(torch.bfloat16), cache=cache, block_table=table, seq_len=_i32(total), cu_q=_i32(_cu(new)),
                max_q=max(new), max_seq=max(total), k_scale=k_scale, v_scale=v_scale)


def _prepare_gdn(case, g):
    lens = _lens(case)
    T, H, N, P = sum(lens), case["heads"], case["dk"], case["dv"]
    t = torch.bfloat16 if case["type"] == "bf16" else torch.float32
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = unit(rnd(T, H, N)).to(t), unit(rnd(T, H, N)).to(t)
    v = rnd(T, H, P).to(t)
    beta = torch.sigmoid(rnd(T, H))
    alpha = torch.exp(-torch.log1p(torch.exp(rnd(T, H) - 3.0)))  # a state that lasts for tens of tokens
    S0 = 0.1 * rnd(case["batch"], H, P, N) if case["state"] else None
    return dict(q=q, k=k, v=v, alpha=alpha, beta=beta, cu_seqlens=_i32(_cu(lens)), S0=S0, longest=max(lens))


# ---------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        from checkpoint_input_replay_rssm_b200 import rssm

        if op == "tables":
            return (s["block_table"],) + tuple(rssm.build_tables(
                s["cached_len"], s["new_len"], s["free_pages"], s["free_head"], s["block_table"], s["page_size"],
                s["max_tokens"]))
        if op == "append":
            rssm.kv4_append(s["k"], s["v"], s["slot_map"], s["cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return rssm.kv4_export(s["slot_map"], s["cache"], s["case"]["dim"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        if op == "attend":
            return rssm.kv4_attend(s["q"], s["cache"], s["block_table"], s["seq_len"], s["cu_q"], s["max_q"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], max_seq=s["max_seq"])
        return rssm.gdn_prefill(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["cu_seqlens"], S0=s["S0"])
    return {"tables": _tables, "append": _append, "attend": _attend, "gdn": _gdn}[op](s)


def _tables(s):
    """New pages go to the requests in order, from the free list at its head; a token's slot is
    page * page_size + offset; rows behind the last token hold -1."""
    ps, table, n = s["page_size"], s["block_table"], s["max_tokens"]
    cached, new = s["cached_len"].long(), s["new_len"].long()
    B, width = table.shape
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    seq = cached + new
    cu = torch.cat([zero, new.cumsum(0)])
    held, want = (cached + ps - 1) // ps, (seq + ps - 1) // ps
    first = torch.cat([zero, (want - held).cumsum(0)])
    at = torch.arange(width, device=table.device)
    fresh = (at >= held[:, None]) & (at < want[:, None])
    src = s["free_head"].long() + first[:-1, None] + at - held[:, None]
    src = torch.where(fresh, src, 0)
    table = torch.where(fresh, s["free_pages"][src], table)
    marks = torch.zeros(n + 1, dtype=torch.int64, device=table.device).index_add_(
        0, cu[1:], torch.ones(B, dtype=torch.int64, device=table.device))
    of = marks.cumsum(0)[:n].clamp(max=B - 1)
    t = torch.arange(n, device=table.device)
    pos = cached[of] + t - cu[of]
    live = t < cu[-1]
    pos = torch.where(live, pos, 0)
    slot = torch.where(live, table[of, pos // ps].long() * ps + pos % ps, -1)
    pos = torch.where(live, pos, -1)
    i32 = torch.int32
    return (table, cu.to(i32), seq.to(i32), slot.to(i32), pos.to(i32), (s["free_head"] + first[-1]).to(i32))


def _quantise(x, scale):
    """x fp32 [..., D] -> (signed code index 0..15 [..., D], block scales e4m3 [..., D / 16])."""
    y = x * (1.0 / scale)
    blocks = y.reshape(*y.shape[:-1], -1, 16)
    sc = (blocks.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sc.float()[..., None]
    r = (blocks / torch.where(f > 0, f, 1.0)) * (f > 0)
    a = r.abs()
    # round to nearest, a tie to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (r < 0).to(torch.uint8)
    return code.reshape(y.shape).to(torch.uint8), sc


def _dequantise(code, sc, scale):
    """(codes 0..15, block scales) -> fp32 values."""
    table = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=code.device)
    v = table[code.int()].reshape(*code.shape[:-1], -1, 16) * sc.float()[..., None]
    return v.reshape(code.shape) * scale


def _pack(kq, vq, pages, ps):
    """Codes and scales of [pages * ps, heads, D] -> the bytes of those pages."""
    parts = []
    for code, sc in (kq, vq):
        b = code[..., 0::2] | (code[..., 1::2] << 4)
        for x in (b, sc.view(torch.uint8)):
            x = x.reshape(pages, ps, x.shape[1], x.shape[2]).transpose(1, 2)
            parts.append(x.reshape(pages, x.shape[1], -1))
    return torch.cat(parts, -1)


def _append(s):
    k, v = s["k"].float(), s["v"].float()
    out = []
    for x, scale in ((k, s["k_scale"]), (v, s["v_scale"])):
        out.append(_dequantise(*_quantise(x, scale), scale).to(torch.bfloat16))
    return tuple(out)


def _unpack(pages, ps, D):
    """Bytes [..., heads, page bytes] -> K codes, K scales, V codes, V scales, each [..., heads, ps, :]."""
    c, e = ps * D // 2, ps * D // 16
    out = []
    for at in (0, c + e):
        b = pages[..., at:at + c].reshape(*pages.shape[:-1], ps, D // 2)
        out.append(torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], D))
        out.append(pages[..., at + c:at + c + e].contiguous().view(torch.float8_e4m3fn)
                   .reshape(*pages.shape[:-1], ps, D // 16))
    return out


def _attend(s):
    """softmax(q K^T / sqrt(D)) V over each request's cached tokens, query i of n seeing the first
    seq_len - n + i + 1 of them; requests padded to the longest."""
    case, q, table = s["case"], s["q"].float(), s["block_table"]
    D, ps, Hk = case["dim"], case["page"], case["kv_heads"]
    B, width, M = table.shape[0], table.shape[1], s["max_q"]
    group = case["q_heads"] // Hk
    kc, ks, vc, vs = _unpack(s["cache"][table.clamp(min=0).long()], ps, D)
    K = _dequantise(kc, ks, s["k_scale"]).transpose(1, 2).reshape(B, Hk, width * ps, D)
    V = _dequantise(vc, vs, s["v_scale"]).transpose(1, 2).reshape(B, Hk, width * ps, D)
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(M, device=q.device)
    real = i < n[:, None]
    rows = torch.where(real, cu[:-1, None] + i, 0)
    Q = q[rows].reshape(B, M, Hk, group, D).transpose(1, 2).reshape(B, Hk, M * group, D)
    S = (Q @ K.transpose(-1, -2)) * D ** -0.5
    seen = s["seq_len"].long()[:, None] - n[:, None] + i + 1
    ok = torch.arange(width * ps, device=q.device) < seen[..., None]
    ok = ok[:, None, :, None].expand(B, Hk, M, group, width * ps).reshape(S.shape)
    S = torch.where(ok, S, -math.inf)
    top = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    O = (p @ V) / torch.where(total > 0, total, 1.0)
    O = O.reshape(B, Hk, M, group, D).transpose(1, 2).reshape(B, M, Hk * group, D)
    return O[real].to(torch.bfloat16)


def _gdn(s):
    """Chunks of 64 tokens: the pseudo-values u of a chunk solve a unit lower-triangular system, whose
    inverse is the product of I + (-A)^(2^i); the state moves by one decay and a rank-64 update."""
    C, lens = 64, s["cu_seqlens"][1:].long() - s["cu_seqlens"][:-1].long()
    B, (_, H, N), P = lens.shape[0], s["q"].shape, s["v"].shape[2]
    nc = max(1, _ceil(s["longest"], C))
    t = torch.arange(nc * C, device="cuda")
    real = t < lens[:, None]
    at = torch.where(real, s["cu_seqlens"][:-1, None].long() + t, 0)

    def chunks(x):  # [T, H, ...] -> [B, nc, H, C, ...], zero behind each prompt
        x = x.float()[at] * real.reshape(real.shape + (1,) * (x.dim() - 1))
        return x.reshape(B, nc, C, *x.shape[2:]).transpose(2, 3)

    q, k, v, beta = (chunks(s[n]) for n in ("q", "k", "v", "beta"))
    la = torch.where(real[..., None], s["alpha"].double().log()[at], 0.0)
    lam = la.reshape(B, nc, C, H).transpose(2, 3).cumsum(-1)
    low = torch.ones(C, C, device="cuda").tril()
    decay = torch.exp((lam[..., :, None] - lam[..., None, :]).where(low > 0, -math.inf)).float()
    A = (k @ k.transpose(-1, -2)) * decay * beta[..., None] * low.tril(-1)
    inv, power = torch.eye(C, device="cuda") - A, A
    for _ in range(5):
        power = power @ power
        inv = inv + inv @ power
    M = (q @ k.transpose(-1, -2)) * decay
    into, left = lam.exp().float()[..., None], (lam[..., -1:] - lam).exp().float()[..., None]
    S = torch.zeros(B, H, P, N, device="cuda") if s["S0"] is None else s["S0"]
    o = torch.empty(B, nc, H, C, P, device="cuda")
    for c in range(nc):
        St = S.transpose(-1, -2)
        u = inv[:, c] @ (beta[:, c, ..., None] * (v[:, c] - into[:, c] * (k[:, c] @ St)))
        o[:, c] = into[:, c] * (q[:, c] @ St) + M[:, c] @ u
        S = S * into[:, c, :, -1:] + (u * left[:, c]).transpose(-1, -2) @ k[:, c]
    return o.transpose(2, 3).reshape(B, nc * C, H, P)[real], S


# ---------------------------------------------------------------- the least work
def work(case):
    op = case["op"]
    if op == "tables":
        ctx, new = _lens(case)
        fresh = sum(_ceil(c + n, case["page"]) - _ceil(c, case["page"]) for c, n in zip(ctx, new))
        # lengths in; packed offsets and totals out; new pages in and into the table; slot and position a token
        return dict(bytes=16 * case["batch"] + 8 * fresh + 8 * max(1, sum(new) + case["pad"]), flops=0)
    if op == "append":
        e = case["tokens"] * case["kv_heads"] * case["dim"] * 2  # keys and values
        return dict(bytes=e * (2 + 2 * 9 / 16 + 2) + 8 * case["tokens"], flops=4 * e)
    if op == "attend":
        ctx, new = _lens(case)
        D = case["dim"]
        kv = sum(c + n for c, n in zip(ctx, new)) * case["kv_heads"] * 2 * D * 9 / 16
        seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        return dict(bytes=kv + 4 * sum(new) * case["q_heads"] * D + 4 * sum(_ceil(c + n, case["page"]) for c, n in zip(ctx, new)),
                    flops=4 * D * case["q_heads"] * seen)
    n, H, N, P = sum(_lens(case)), case["heads"], case["dk"], case["dv"]
    e = 2 if case["type"] == "bf16" else 4
    state = 4 * case["batch"] * H * P * N
    return dict(bytes=n * H * (e * (2 * N + P) + 8 + 4 * P) + state * (2 if case["state"] else 1), flops=7 * n * H * P * N)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": lambda s: None, "append": _append64, "attend": _attend64, "gdn": _gdn64}[case["op"]](s)


def _grid(x, step_of):
    """x >= 0 in 64 bits to the nearest multiple of step_of(x), a tie to the even multiple."""
    step = step_of(x)
    return torch.round(x / step) * step


def _held64(x, scale):
    """The value that the cache holds for each element, from the definition."""
    y = x.double() / scale
    b = y.unflatten(-1, (-1, 16))
    power = lambda z, least: torch.exp2(torch.floor(torch.log2(z.clamp(min=1e-300))).clamp(min=least))  # noqa: E731
    sc = _grid(b.abs().amax(-1, keepdim=True) / 6, lambda z: power(z, -6) / 8).clamp(max=448)
    r = torch.where(sc > 0, b.abs() / sc.clamp(min=2.0 ** -9), 0.0)
    m = _grid(r, lambda z: power(z, 0) / 2).clamp(max=6)
    return (torch.sign(b) * m * sc).flatten(-2) * scale


def _append64(s):
    return _held64(s["k"], s["k_scale"]), _held64(s["v"], s["v_scale"])


def _attend64(s):
    case, q, out = s["case"], s["q"].double(), []
    D, ps, Hk, g = case["dim"], case["page"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    value = torch.tensor([(-1) ** (c >> 3) * E2M1[c & 7] for c in range(16)], dtype=torch.float64, device="cuda")
    cu, total, table = s["cu_q"].tolist(), s["seq_len"].tolist(), s["block_table"]
    for b, n in enumerate(total):
        page = s["cache"][table[b, :_ceil(n, ps)].long()]
        kv = []
        for at, scale in ((0, s["k_scale"]), (ps * D * 9 // 16, s["v_scale"])):
            byte = page[:, :, at:at + ps * D // 2].reshape(-1, Hk, ps, D // 2)
            e = page[:, :, at + ps * D // 2:at + ps * D * 9 // 16].contiguous().view(torch.float8_e4m3fn).double()
            x = torch.stack((value[(byte % 16).long()], value[(byte // 16).long()]), -1).reshape(-1, Hk, ps, D // 16, 16)
            x = x * e.reshape(-1, Hk, ps, D // 16, 1) * scale
            kv.append(x.reshape(-1, Hk, ps, D).transpose(0, 1).reshape(Hk, -1, D)[:, :n])
        m = cu[b + 1] - cu[b]
        qb = q[cu[b]:cu[b + 1]].reshape(m, Hk, g, D).permute(1, 2, 0, 3)  # [Hk, g, m, D]
        w = torch.einsum("hgmd,hnd->hgmn", qb, kv[0]) / math.sqrt(D)
        hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(m, device="cuda")[:, None] + (n - m)
        w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
        out.append(torch.einsum("hgmn,hnd->mhgd", w, kv[1]).reshape(m, Hk * g, D))
    return torch.cat(out)


def _gdn64(s):
    """The recurrence, token by token, all requests side by side."""
    lens = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    B, (T, H, N), P = lens.shape[0], s["q"].shape, s["v"].shape[2]
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    o = torch.zeros(T, H, P, dtype=torch.float64, device="cuda")
    q, k, v, a, b = (s[n].double() for n in ("q", "k", "v", "alpha", "beta"))
    start = s["cu_seqlens"][:-1].long()
    order = torch.argsort(lens, descending=True)
    S, start, sorted_lens = S[order].contiguous(), start[order], lens[order].tolist()
    alive = B
    for t in range(s["longest"]):
        while sorted_lens[alive - 1] <= t:
            alive -= 1
        at, X = start[:alive] + t, S[:alive]
        X *= a[at][..., None, None]
        err = v[at] - torch.einsum("bhpn,bhn->bhp", X, k[at])
        X += (b[at][..., None] * err)[..., None] * k[at][..., None, :]
        o[at] = torch.einsum("bhpn,bhn->bhp", X, q[at])
    back = torch.empty_like(S)
    back[order] = S
    return o, back
