"""Operators on packed requests (block tables, the 4-bit key/value cache and its attention, the gated
delta rule over packed prompts) against the fp64 / whole-number oracle, on the GPU.

Tolerances.
 * Tables and held cache values are exact.
 * Attention: its output is bf16 (half a step is 2^-8 of the value); the probabilities enter the second
   product as fp16 (2^-11 each, against sum_j p_j |v_j|); a score is an fp32 sum of D products, so it
   errs by at most (D + 4) 2^-24 of the sum of its terms' sizes and moves every probability and their
   sum by that much; exp2 and the sums over tokens add less than 2^-14 of sum_j p_j |v_j|.  Below
   2^-14 an fp16 number is a multiple of 2^-24, so a probability (relative to the largest, which is 1, so
   that their sum is at least 1) errs by up to 2^-25 however small it is: 2^-25 sum_j |v_j| in all.
 * The gated delta rule: an fp32 operand enters the tensor cores as two bf16 parts.  The first leaves up
   to 2^-9 of the value, the second 2^-9 of that: 2^-18.  On the way to one element of the state are R,
   T, the dropped product of their second parts and w U, 4 * 2^-18 = 1.5e-5 of the sum of its terms' sizes
   per chunk if every rounding were the worst one.  In the 2-norm they are not, and 1e-5 is asked for.
   One element may be 1e-4 off, the tolerance of the library's fp32 read path, of the RMS or, where the
   element is larger, of the element: a state of few tokens is a sum of few terms, whose size is the
   element's and not the RMS (one token's: the outer product of v and k, which has elements of 20 RMS,
   so that 1.5e-5 of them is 3e-4 RMS).
"""
import numpy as np
import pytest

from checkpoint_input_replay_rssm_b200 import rssm
from oracle import packed

pytestmark = pytest.mark.gpu


def _t(x, dtype="float32"):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to(getattr(torch, dtype)).cuda()


def _i(x):
    return _t(np.asarray(x, np.int32), "int32")


def _np(t):
    return t.double().cpu().numpy()


def _err():
    return _i([0, 0, 0, 0])


def _cu(lens, first=0):
    return [first] + [first + int(c) for c in np.cumsum(lens)]


# ---------------------------------------------------------------- gated delta rule
def _gdn_inputs(lens, H, N, P, dtype, seed, first=0, pad=0, keep=3.0, state=True):
    r = np.random.default_rng(seed)
    cu = _cu(lens, first)
    T = cu[-1] + pad
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    d = dict(q=_t(unit(r.normal(size=(T, H, N))), dtype), k=_t(unit(r.normal(size=(T, H, N))), dtype),
             v=_t(r.normal(size=(T, H, P)), dtype), alpha=_t(np.exp(-np.logaddexp(0, r.normal(size=(T, H)) - keep))),
             beta=_t(1 / (1 + np.exp(-r.normal(size=(T, H))))))
    S0 = _t(0.1 * r.normal(size=(len(lens), H, P, N))) if state else None
    return d, cu, S0


def _gdn_run(d, cu, S0, **kw):
    err = _err()
    y, S = rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], _i(cu), S0, err=err, **kw)
    assert err.tolist() == [0, 0, 0, 0]
    return _np(y), _np(S)


def _gdn_ref(d, cu, S0):
    return packed.gdn(*(_np(d[n]) for n in ("q", "k", "v", "alpha", "beta")), cu, None if S0 is None else _np(S0))


def _close(got, want, what):
    live = ~np.isnan(want)
    g, w = got[live], want[live]
    rms = np.sqrt(np.mean(w * w)) if w.size else 0.0
    assert np.isfinite(g).all(), what
    assert np.sqrt(np.mean((g - w) ** 2)) <= 1e-5 * rms if w.size else True, what
    assert np.max(np.abs(g - w) / np.maximum(rms, np.abs(w)), initial=0.0) <= 1e-4, what


SHAPES = [(128, 128, "bfloat16"), (128, 64, "bfloat16"), (128, 256, "bfloat16"), (128, 72, "bfloat16"),
          (64, 64, "bfloat16"), (32, 40, "bfloat16"), (16, 8, "float32"), (64, 64, "float32"), (128, 128, "float32")]


@pytest.mark.parametrize("N,P,dtype", SHAPES)
def test_gdn_ragged_prompts(N, P, dtype):
    """Lengths around the chunk and staging borders, empty prompts, rows before and behind."""
    lens = [1, 0, 63, 64, 65, 130, 0, 16, 17, 2]
    d, cu, S0 = _gdn_inputs(lens, 3, N, P, dtype, 7, first=5, pad=9)
    import torch

    y = torch.full((d["q"].shape[0], 3, P), 7.25, device="cuda")
    got, S = _gdn_run(d, cu, S0, y=y)
    want, Sw = _gdn_ref(d, cu, S0)
    _close(got, want, "y")
    _close(S, Sw, "state")
    assert (got[:5] == 7.25).all() and (got[cu[-1]:] == 7.25).all(), "rows of no request were written"
    assert np.array_equal(S[1], _np(S0)[1]) and np.array_equal(S[6], _np(S0)[6])


@pytest.mark.parametrize("lens", [[1], [5], [1] * 9, [700], [0, 0, 1], [64 * 5]])
def test_gdn_from_a_zero_state(lens):
    d, cu, _ = _gdn_inputs(lens, 2, 128, 128, "bfloat16", 11, state=False)
    got, S = _gdn_run(d, cu, None)
    want, Sw = _gdn_ref(d, cu, None)
    _close(got, want, "y")
    _close(S, Sw, "state")


@pytest.mark.parametrize("keep", [-4.0, 0.0, 8.0])
def test_gdn_gates_from_quick_to_almost_none(keep):
    """keep -4: a state of a token or less, whose decay over a chunk underflows; 8: hardly any decay."""
    d, cu, S0 = _gdn_inputs([400, 129], 2, 128, 128, "bfloat16", 13, keep=keep)
    got, S = _gdn_run(d, cu, S0)
    want, Sw = _gdn_ref(d, cu, S0)
    _close(got, want, "y")
    _close(S, Sw, "state")


def test_gdn_gates_of_exactly_zero_and_one_and_writes_of_strength_zero_and_one():
    d, cu, S0 = _gdn_inputs([200, 70], 2, 128, 64, "bfloat16", 17)
    r = np.random.default_rng(18)
    a, b = _np(d["alpha"]), _np(d["beta"])
    a[r.random(a.shape) < 0.1] = 0.0
    a[r.random(a.shape) < 0.1] = 1.0
    a[90:97, 0] = 0.0
    b[r.random(b.shape) < 0.1] = 0.0
    b[r.random(b.shape) < 0.1] = 1.0
    d["alpha"], d["beta"] = _t(a), _t(b)
    got, S = _gdn_run(d, cu, S0)
    want, Sw = _gdn_ref(d, cu, S0)
    _close(got, want, "y")
    _close(S, Sw, "state")


def test_gdn_repeated_keys_keep_the_system_solvable():
    """One key throughout, full strength, no decay: the chunk's triangular system is all ones below the
    diagonal, whose powers grow; every token overwrites the value of the one before.  The state is then the
    telescoping sum of the writes u_t = v_t - v_{t-1}, so that its error is not in proportion to itself:
    R_t leaves 2^-18 |v_t| and comes into u_t and u_{t+1}, u_t leaves 2^-18 (|v_t| + |v_{t-1}|), together
    at most 4 * 2^-18 sum_t |v_t| (T is +-1, exact)."""
    d, cu, S0 = _gdn_inputs([150], 1, 128, 64, "bfloat16", 19)
    import torch

    k = torch.zeros_like(d["k"])
    k[:, :, 3] = 1.0
    d["k"], d["beta"], d["alpha"] = k, torch.ones_like(d["beta"]), torch.ones_like(d["alpha"])
    got, S = _gdn_run(d, cu, S0)
    want, Sw = _gdn_ref(d, cu, S0)
    tol = 4 * 2.0 ** -18 * np.abs(_np(d["v"])).sum(0)[0] + 1e-6  # [P]
    assert (np.abs(S - Sw)[0, 0] <= tol[:, None]).all() and (np.abs(got - want)[:, 0] <= tol).all()
    assert (np.abs(S[0, 0, :, 3] - _np(d["v"])[-1, 0]) <= tol).all()


def test_gdn_state_of_a_prompt_in_two_parts_is_that_of_the_whole():
    d, cu, S0 = _gdn_inputs([333], 2, 128, 128, "bfloat16", 23)
    y, S = _gdn_run(d, cu, S0)
    part = lambda a, b: {n: t[a:b].contiguous() for n, t in d.items()}  # noqa: E731
    y1, S1 = _gdn_run(part(0, 100), [0, 100], S0)
    y2, S2 = _gdn_run(part(100, 333), [0, 233], _t(S1))
    _close(np.concatenate([y1, y2]), y, "y")
    _close(S2, S, "state")


def test_gdn_bad_offsets_are_reported_and_skipped():
    import torch

    d, _, S0 = _gdn_inputs([20, 20, 20], 2, 128, 64, "bfloat16", 29)
    good, _, _ = _gdn_inputs([20, 20, 20], 2, 128, 64, "bfloat16", 29)
    for cu, bad in (([0, 20, 10, 60], [1]), ([0, 20, 40, 61], [2]), ([-1, 20, 40, 60], [0]),
                    ([0, 20, 2 ** 31 - 1, 60], [1, 2])):
        err = _err()
        y = torch.full((60, 2, 64), 7.25, device="cuda")
        So = torch.full_like(S0, 7.25)
        rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], _i(cu), S0, y=y, S_out=So, err=err)
        assert err[0].item() == rssm.RSSM_DEV_BAD_LENGTHS and err[1].item() in bad
        for b in range(3):
            if b in bad:
                assert (So[b] == 7.25).all()
            else:
                w = packed.gdn(*(_np(good[n]) for n in ("q", "k", "v", "alpha", "beta")), [cu[b], cu[b + 1]],
                               _np(S0)[b:b + 1])[1]
                _close(_np(So)[b:b + 1], w, b)


# ---------------------------------------------------------------- block tables
def _tables_case(seed, B, ps, ctx_hi, new_hi, pad=0, spare=2):
    r = np.random.default_rng(seed)
    cached, new = r.integers(0, ctx_hi + 1, B).tolist(), r.integers(0, new_hi + 1, B).tolist()
    held = [-(-c // ps) for c in cached]
    need = sum(-(-(c + n) // ps) - h for c, n, h in zip(cached, new, held))
    width = max(1, max(-(-(c + n) // ps) for c, n in zip(cached, new)))
    pages = r.permutation(sum(held) + need + spare).tolist()
    table, at = [], 0
    for h in held:
        table.append(pages[at:at + h] + [-1] * (width - h))
        at += h
    return cached, new, [10 ** 6, 10 ** 6] + pages[at:], 2, table, ps, max(1, sum(new) + pad)


def _tables_run(case):
    cached, new, free, head, table, ps, mt = case
    tab, err = _i(table), _err()
    out = rssm.build_tables(_i(cached), _i(new), _i(free), _i([head]), tab, ps, mt, err=err)
    return tab.tolist(), [o.tolist() for o in out], err.tolist()


@pytest.mark.parametrize("B,ps,ctx,new,pad", [(1, 16, 0, 1, 0), (1, 16, 0, 0, 3), (3, 16, 40, 40, 5), (256, 64, 500, 1, 0),
                                              (511, 1, 9, 3, 1), (513, 7, 60, 9, 0), (1500, 32, 300, 20, 77),
                                              (16384, 16, 40, 2, 0), (5, 65536, 100, 100, 0), (40, 16, 5000, 3000, 11)])
def test_tables_equal_the_oracle(B, ps, ctx, new, pad):
    case = _tables_case(B + ps, B, ps, ctx, new, pad)
    tab, out, err = _tables_run(case)
    want = packed.tables(*case)
    assert err == [0, 0, 0, 0]
    assert tab == want[0]
    for got, w in zip(out, want[1:5]):
        assert got == w
    assert out[4] == [want[5]]


@pytest.mark.parametrize("what", ["negative cached", "negative new", "row too short", "sum past 2^31", "map too short",
                                  "no pages", "head past the list", "head below it"])
def test_tables_refuse_a_step_that_does_not_fit(what):
    cached, new, free, head, table, ps, mt = _tables_case(5, 70, 16, 100, 50)
    code, who = rssm.RSSM_DEV_BAD_LENGTHS, -1
    if what == "negative cached":
        cached[33], who = -1, 33
    elif what == "negative new":
        new[69], who = -5, 69
    elif what == "row too short":
        new[7], who = len(table[0]) * 16 - cached[7] + 1, 7
    elif what == "sum past 2^31":
        new[0] = new[1] = 2 ** 31 - 1
        who = 0
    elif what == "map too short":
        mt = sum(new) - 1
    else:
        code = rssm.RSSM_DEV_NO_PAGES
        if what == "no pages":
            need = packed.tables(cached, new, free, head, table, ps, mt)[5]
            free = free[:need - 1]
        else:
            head = len(free) + 1 if what == "head past the list" else -1
    assert packed.tables(cached, new, free, head, table, ps, mt) is None
    tab, out, err = _tables_run((cached, new, free, head, table, ps, mt))
    assert err[:2] == [code, who]
    assert tab == table and out[0] == [0] * 71 and out[1] == cached and out[4] == [head]
    assert out[2] == [-1] * mt and out[3] == [-1] * mt


# ---------------------------------------------------------------- the 4-bit cache
def _kv(r, T, Hk, D, spread=0.7):
    x = r.normal(size=(T, Hk, D)) * np.exp(spread * r.normal(size=(1, Hk, D)))
    return _t(x, "bfloat16")


@pytest.mark.parametrize("T,Hk,D,ps,ke,ve", [(1, 1, 64, 16, 0, 0), (37, 2, 128, 16, -4, -6), (300, 3, 64, 48, 5, -60),
                                             (129, 8, 128, 256, -3, 60)])
def test_cache_holds_the_nearest_values(T, Hk, D, ps, ke, ve):
    import torch

    r = np.random.default_rng(T)
    k, v = _kv(r, T, Hk, D), (_kv(r, T, Hk, D).float() * 2.0 ** ve).to(torch.bfloat16)
    k[0, 0, :16] = 0.0             # a block of zeros
    k[0, 0, 16:32] *= 2.0 ** -30   # a block below the smallest scale
    k[0, -1, 32:48] = 1e30         # saturates
    pages = -(-T // ps) + 2
    cache = rssm.kv4_cache(pages, Hk, ps, D)
    guard = cache.clone()
    slots = r.permutation(pages * ps)[:T]
    err = _err()
    kw = dict(k_scale=2.0 ** ke, v_scale=2.0 ** ve, err=err)
    rssm.kv4_append(k, v, _i(slots), cache, **kw)
    gk, gv = rssm.kv4_export(_i(slots), cache, D, **kw)
    assert err.tolist() == [0, 0, 0, 0]
    assert np.array_equal(_np(gk), packed.hold(_np(k), 2.0 ** ke))
    assert np.array_equal(_np(gv), packed.hold(_np(v), 2.0 ** ve))
    free = np.setdiff1d(np.arange(pages * ps), slots)
    gk, gv = rssm.kv4_export(_i(free), cache, D, **kw)
    assert not gk.any() and not gv.any(), "a slot that was not named was written"
    # a second write of some slots, others left alone
    rssm.kv4_append(v, k, _i(np.where(np.arange(T) % 2, slots, -1)), cache, **kw)
    gk2, _ = rssm.kv4_export(_i(slots), cache, D, **kw)
    want = np.where((np.arange(T) % 2)[:, None, None], packed.hold(_np(v), 2.0 ** ke), packed.hold(_np(k), 2.0 ** ke))
    assert np.array_equal(_np(gk2), want)
    assert guard.shape == cache.shape


@pytest.mark.parametrize("e", [0, -7, 60])
def test_cache_codes_of_every_quotient(e):
    """Every 8-bit value as a block's largest, so that every scale occurs, and every 8-bit value of
    ten binades below it, so that every code and every border between two is met, exactly."""
    import torch

    m = np.arange(128, 256)
    rest = np.concatenate([m * 2.0 ** -j for j in range(10)])
    rest = np.concatenate([rest, -rest, np.zeros(-2 * len(rest) % 15)]).reshape(-1, 15)
    top = np.repeat(m * 1.0, len(rest))[:, None]
    x = np.concatenate([top, np.minimum(np.tile(rest, (128, 1)), top)], 1).reshape(-1, 2, 64) * 2.0 ** (e - 4)
    k = _t(x, "bfloat16")
    assert np.array_equal(_np(k), x)
    cache = rssm.kv4_cache(-(-len(x) // 32), 2, 32, 64)
    slots = _i(range(len(x)))
    kw = dict(k_scale=2.0 ** e, v_scale=2.0 ** (e - 2))
    rssm.kv4_append(k, k, slots, cache, **kw)
    gk, gv = (_np(t) for t in rssm.kv4_export(slots, cache, 64, **kw))
    assert np.array_equal(gk, packed.hold(x, 2.0 ** e)) and np.array_equal(gv, packed.hold(x, 2.0 ** (e - 2)))


def test_cache_keeps_infinities_finite_and_nan_as_nan():
    import torch

    k = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 3], k[0, 0, 4], k[0, 0, 20], k[1, 0, 0] = float("inf"), -float("inf"), float("nan"), 1.0
    cache = rssm.kv4_cache(1, 1, 16, 64)
    rssm.kv4_append(k, k, _i([4, 9]), cache, k_scale=2.0, v_scale=1.0)
    gk, gv = (_np(t) for t in rssm.kv4_export(_i([4, 9]), cache, 64, k_scale=2.0, v_scale=1.0))
    assert gk[0, 0, 3] == 448 * 6 * 2 and gk[0, 0, 4] == -448 * 6 * 2 and gv[0, 0, 3] == 448 * 6
    assert np.isnan(gk[0, 0, 16:32]).all() and not np.isnan(gk[0, 0, 32:]).any() and not np.isnan(gk[0, 0, :16]).any()


def test_cache_slots_outside_it_are_reported_and_not_touched():
    import torch

    r = np.random.default_rng(3)
    k = _kv(r, 4, 2, 64)
    cache = rssm.kv4_cache(2, 2, 16, 64)
    err = _err()
    rssm.kv4_append(k, k, _i([-1, -2 ** 31, -7, -1]), cache, err=err)
    assert err.tolist() == [0, 0, 0, 0] and not cache.any()
    rssm.kv4_append(k, k, _i([32, 2 ** 31 - 1, 31, -1]), cache, err=err)
    assert err[0].item() == rssm.RSSM_DEV_BAD_PAGE
    gk, _ = rssm.kv4_export(_i([31, 32, 0]), cache, 64, err=_err())
    assert np.array_equal(_np(gk)[0], packed.hold(_np(k), 1.0)[2]) and not gk[1:].any()
    assert torch.count_nonzero(cache[0]).item() == 0


# ---------------------------------------------------------------- attention over it
def _attend_case(seed, lens, news, Hq, Hk, D, ps, ke=0, ve=0, pad=0, first=0, spare=1, fill=0xFF):
    """Random pages; every byte that no request's token owns holds `fill` (0xFF: NaN scales)."""
    import torch

    r = np.random.default_rng(seed)
    held = [-(-n // ps) for n in lens]
    width = max(1, max(held)) + spare
    pages = sum(held) + 2
    order, at = r.permutation(pages), 0
    cache = torch.full((pages, Hk, ps * D * 9 // 8), fill, dtype=torch.uint8, device="cuda")
    table = np.full((len(lens), width), -1)
    slots = []
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
        slots += [table[b, t // ps] * ps + t % ps for t in range(lens[b])]
    kw = dict(k_scale=2.0 ** ke, v_scale=2.0 ** ve)
    K, V = [np.zeros((0, Hk, D))] * len(lens), [np.zeros((0, Hk, D))] * len(lens)
    if slots:
        k, v = _kv(r, len(slots), Hk, D), _kv(r, len(slots), Hk, D, 0.1)
        rssm.kv4_append(k, v, _i(slots), cache, **kw)
        hk, hv = (_np(t) for t in rssm.kv4_export(_i(slots), cache, D, **kw))
        ends = np.cumsum([0] + list(lens))
        K, V = ([x[a:b] for a, b in zip(ends, ends[1:])] for x in (hk, hv))
    cu = _cu(news, first)
    q = _t(r.normal(size=(max(1, cu[-1] + pad), Hq, D)), "bfloat16")
    return dict(q=q, cache=cache, table=_i(table), lens=_i(lens), cu=cu, K=K, V=V, kw=kw, max_q=max(1, max(news)))


def _attend_check(c, got, scale=None):
    D = c["q"].shape[2]
    want, mean, big, flat = packed.attend(_np(c["q"]), c["K"], c["V"], c["cu"], D ** -0.5 if scale is None else scale)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14 + 2 * (D + 4) * 2.0 ** -24 * big[..., None]) * mean
    tol += 2.0 ** -25 * flat
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all()
    bad = np.abs(got - want)[live] > tol[live]
    assert not bad.any(), (bad.sum(), np.max(np.abs(got - want)[live]))


def _attend_run(c, **kw):
    import torch

    err = _err()
    out = torch.full_like(c["q"], 7.25)
    rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], _i(c["cu"]), c["max_q"], out=out, err=err, **c["kw"], **kw)
    assert err.tolist() == [0, 0, 0, 0]
    got = _np(out)
    assert (got[:c["cu"][0]] == 7.25).all() and (got[c["cu"][-1]:] == 7.25).all(), "rows of no request were written"
    return got


HEADS = [(1, 1, 64), (4, 4, 128), (8, 2, 64), (16, 1, 128), (7, 1, 128), (40, 2, 64), (34, 2, 128)]


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
def test_attend_one_token(Hq, Hk, D):
    lens = [1, 2, 15, 16, 17, 100, 33, 257]
    c = _attend_case(Hq + D, lens, [1] * 8, Hq, Hk, D, 16, ke=1, ve=-2)
    _attend_check(c, _attend_run(c))


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("ps", [16, 48, 256])
def test_attend_ragged_rows(Hq, Hk, D, ps):
    """Drafts and prompt chunks, requests without rows, rows before and behind, pages that end inside a tile."""
    news = [4, 0, 1, 9, 33, 70, 8]
    lens = [4, 20, 131, 64, 33, 200, 9]
    c = _attend_case(Hq + D + ps, lens, news, Hq, Hk, D, ps, first=3, pad=5)
    _attend_check(c, _attend_run(c))


def test_attend_rows_that_see_nothing_are_zero():
    """More rows than cached tokens (the first ones see none), and nothing cached at all."""
    c = _attend_case(3, [3, 0, 1], [7, 2, 1], 8, 2, 128, 16)
    got = _attend_run(c)
    _attend_check(c, got)
    assert not got[:4].any() and not got[7:9].any() and got[9].any()


@pytest.mark.parametrize("L", [1000, 4097, 20000])
def test_attend_long_context_alone(L):
    """One request over a long context: the tokens are split over the machine and joined."""
    c = _attend_case(L, [L], [2], 8, 2, 128, 64)
    _attend_check(c, _attend_run(c))


def test_attend_long_and_short_together_and_bounds_beyond_them():
    c = _attend_case(9, [5000, 1, 0, 77, 2049], [1, 1, 1, 3, 2], 8, 2, 64, 32, spare=500)
    _attend_check(c, _attend_run(c))
    a = _attend_run(c, max_seq=5000)
    _attend_check(c, a)


def test_attend_large_scores_and_a_scale_of_its_own():
    """Scores far apart (one token takes all the weight) and a zero scale (all tokens alike)."""
    c = _attend_case(21, [300, 40], [2, 1], 8, 2, 128, 16)
    c["q"] = (c["q"].float() * 100).to(c["q"].dtype)
    _attend_check(c, _attend_run(c))
    c["q"] = (c["q"].float() * 2.0 ** 60).to(c["q"].dtype)
    _attend_check(c, _attend_run(c, sm_scale=2.0 ** -62), 2.0 ** -62)
    _attend_check(c, _attend_run(c, sm_scale=0.0), 0.0)


def test_attend_rows_of_zeros_and_of_tiny_numbers():
    c = _attend_case(22, [50, 60], [3, 2], 4, 2, 64, 16)
    c["q"][0] = 0
    c["q"][1] = (c["q"][1].float() * 1e-38).to(c["q"].dtype)
    _attend_check(c, _attend_run(c))


def test_attend_nan_stays_with_the_rows_that_see_it():
    """A NaN value at token 40 of 45: draft rows that end before it are as without it."""
    import torch

    c = _attend_case(23, [45], [8], 4, 2, 128, 16)
    clean = _attend_run(c)
    off = 16 * (128 // 2) + (40 % 16) * 8 + 5  # the V scale of token 40, channels 80..95, of both heads
    page = c["table"][0, 40 // 16].item()
    c["cache"][page, :, 16 * 72 + off] = 0x7F
    err = _err()
    out = rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], _i(c["cu"]), 8, err=err)
    got = _np(out)
    seen = np.arange(8) + 45 - 8 + 1 > 40
    assert np.array_equal(got[~seen], clean[~seen])
    assert np.isnan(got[seen][:, :, 80:96]).all()
    rest = np.delete(got[seen], np.arange(80, 96), axis=2)
    assert np.array_equal(rest, np.delete(clean[seen], np.arange(80, 96), axis=2))
    # a NaN key takes the rows that see it whole
    c["cache"][page, :, 16 * 72 + off] = 0x38
    c["cache"][page, :, off] = 0x7F
    got = _np(rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], _i(c["cu"]), 8, err=err))
    assert np.isnan(got[seen]).all() and np.array_equal(got[~seen], clean[~seen])
    # and so does a NaN in the query
    c["cache"][page, :, off] = 0x38
    c["q"][2, 1, 7] = float("nan")
    got = _np(rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], _i(c["cu"]), 8, err=err))
    assert np.isnan(got[2, 1]).all() and np.isfinite(np.delete(got.reshape(32, 128), 9, axis=0)).all()
    assert torch.equal(err, _err())


@pytest.mark.parametrize("D,ps", [(128, 16), (64, 48), (128, 256)])
def test_attend_prompt_chunks_with_nan_bad_pages_and_rows_that_see_nothing(D, ps):
    """The same with enough rows for the tiles of 128: a NaN value and a NaN key at token 150 stay with the rows behind
    it, a page that is not there is left out, more rows than cached tokens leave the first ones 0."""
    lens, news = [200, 30, 300], [150, 40, 129]
    c = _attend_case(D + ps, lens, news, 16, 1, D, ps, pad=3, first=2)
    clean = _attend_run(c)
    _attend_check(c, clean)
    assert not clean[152:162].any()  # the second request's first rows
    row0, g = c["cu"][0], 16
    page, off = c["table"][0, 150 // ps].item(), 150 % ps
    rows = np.arange(150)
    seen = rows + 200 - 150 + 1 > 150
    for is_v in (True, False):
        at = (ps * D * 9 // 16 if is_v else 0) + ps * D // 2 + off * (D // 16) + 2
        kept = c["cache"][page, 0, at].item()
        c["cache"][page, 0, at] = 0x7F
        err = _err()
        got = _np(rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], _i(c["cu"]), c["max_q"], err=err, **c["kw"]))
        c["cache"][page, 0, at] = kept
        assert err.tolist() == [0, 0, 0, 0]
        mine, ref = got[row0:row0 + 150], clean[row0:row0 + 150]
        assert np.array_equal(mine[~seen], ref[~seen])
        assert np.isnan(mine[seen][:, :, 32:48] if is_v else mine[seen]).all()
        if is_v:
            assert np.array_equal(np.delete(mine[seen], np.arange(32, 48), 2), np.delete(ref[seen], np.arange(32, 48), 2))
        assert np.array_equal(got[row0 + 150:c["cu"][-1]], clean[row0 + 150:c["cu"][-1]])
    table = c["table"].clone()
    table[2, 0] = c["cache"].shape[0]
    err = _err()
    got = _np(rssm.kv4_attend(c["q"], c["cache"], table, c["lens"], _i(c["cu"]), c["max_q"], err=err, **c["kw"]))
    assert err[:2].tolist() == [rssm.RSSM_DEV_BAD_PAGE, 2]
    assert np.array_equal(got[row0:c["cu"][2]], clean[row0:c["cu"][2]])
    q, cut = c["q"][c["cu"][2]:c["cu"][3]], min(ps, 300)
    want = []
    for i in range(129):  # row by row: what is left out lies before what is seen
        n = 300 - 129 + i + 1
        want.append(packed.attend(_np(q[i:i + 1]), [c["K"][2][cut:n]], [c["V"][2][cut:n]], [0, 1], D ** -0.5)[0][0])
    far = np.abs(got[c["cu"][2]:c["cu"][3]] - np.array(want))
    assert far.max() <= 2.0 ** -7 * np.abs(c["V"][2]).max()  # bf16 output and fp16 weights, in the largest value
    assert g == 16


def test_attend_bad_lengths_and_pages_are_reported():
    import torch

    c = _attend_case(31, [40, 50, 60], [2, 2, 2], 8, 2, 64, 16)
    clean = _attend_run(c)

    def run(cu=None, lens=None, table=None, max_q=2, **kw):
        err, out = _err(), torch.full_like(c["q"], 7.25)
        rssm.kv4_attend(c["q"], c["cache"], c["table"] if table is None else table,
                        c["lens"] if lens is None else _i(lens), _i(c["cu"] if cu is None else cu), max_q, out=out,
                        err=err, **c["kw"], **kw)
        return _np(out), err.tolist()

    wide = c["table"].shape[1] * 16
    for kw in (dict(lens=[40, -1, 60]), dict(lens=[40, wide + 1, 60]), dict(lens=[40, 2 ** 31 - 1, 60]),
               dict(cu=[0, 2, 5, 6]), dict(lens=[40, 55, 60], max_seq=54)):
        got, err = run(**kw)
        assert err[0] == rssm.RSSM_DEV_BAD_LENGTHS, kw
        assert np.array_equal(got[:2], clean[:2]), kw
        assert (got[2:4] == 7.25).all(), kw
    got, err = run(cu=[0, 2, 4, 7])
    assert err[:2] == [rssm.RSSM_DEV_BAD_LENGTHS, 2] and (got[4:] == 7.25).all() and np.array_equal(got[:4], clean[:4])
    for page in (-1, c["cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        table = c["table"].clone()
        table[1, 1] = page
        got, err = run(table=table)
        assert err[:2] == [rssm.RSSM_DEV_BAD_PAGE, 1]
        assert np.array_equal(got[[0, 1, 4, 5]], clean[[0, 1, 4, 5]])
        # the tokens of that page are left out as if masked
        d = dict(c, K=[c["K"][1][np.r_[0:16, 32:50]]], V=[c["V"][1][np.r_[0:16, 32:50]]], q=c["q"][2:4], cu=[0, 2])
        _attend_check(d, got[2:4])


def test_attend_offsets_past_32_bits():
    """A cache of more than 4 GiB with its last pages in use."""
    import torch

    Hk, D, ps = 8, 128, 256
    pages = (4 << 30) // (Hk * ps * D * 9 // 8) + 20
    cache = torch.empty((pages, Hk, ps * D * 9 // 8), dtype=torch.uint8, device="cuda")
    r = np.random.default_rng(5)
    L = 700
    table = np.array([[pages - 1, pages - 3, pages - 2]])
    slots = np.array([table[0, t // ps] * ps + t % ps for t in range(L)])
    k, v = _kv(r, L, Hk, D), _kv(r, L, Hk, D)
    rssm.kv4_append(k, v, _i(slots), cache)
    hk, hv = rssm.kv4_export(_i(slots), cache, D)
    assert np.array_equal(_np(hk), packed.hold(_np(k), 1.0))
    c = dict(q=_t(r.normal(size=(1, 16, D)), "bfloat16"), cache=cache, table=_i(table), lens=_i([L]), cu=[0, 1],
             K=[_np(hk)], V=[_np(hv)], kw={}, max_q=1)
    _attend_check(c, _attend_run(c))


def test_sizes_that_would_wrap_are_refused():
    import torch

    one, table = _i([1]), torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for kw in (dict(page_size=2 ** 32 + 16), dict(max_tokens=2 ** 32 + 1), dict(max_tokens=0), dict(page_size=-16)):
        with pytest.raises(ValueError):
            rssm.build_tables(one, one, _i([0, 1]), _i([0]), table, **{**dict(page_size=16, max_tokens=1), **kw})
    assert not table.any()
    cache = rssm.kv4_cache(2, 1, 16, 64)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(max_q=2 ** 32 + 1), dict(max_q=1, max_seq=2 ** 32 + 1)):
        with pytest.raises(ValueError):
            rssm.kv4_attend(q, cache, table, one, _i([0, 1]), **kw)
    with pytest.raises(ValueError):
        rssm.kv4_attend(q[:, :, :0].contiguous(), cache, table, one, _i([0, 1]), 1)
