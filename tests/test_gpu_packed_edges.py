"""Operators on packed requests at the edges of what their documentation allows: sizes at a limit, inputs that are not
finite, offsets that spoil one request and must spoil no other, mixed batches, loops that run long enough to reuse
every buffer.  Oracles and tolerances are those of test_gpu_packed.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from checkpoint_input_replay_rssm_b200 import rssm
from checkpoint_input_replay_rssm_b200.hybrid import HybridShape, HybridStack
from oracle import packed
from tests.test_gpu_packed import _attend_case, _attend_check, _attend_run, _close, _err, _gdn_inputs, _gdn_ref, _gdn_run, _i, _np, _t, _tables_case, _tables_run

pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


# ---------------------------------------------------------------- block tables
def _tables_equal(B):
    case = _tables_case(B, B, 16, 40, 2, 0)
    tab, out, err = _tables_run(case)
    want = packed.tables(*case)
    assert err == [0, 0, 0, 0] and tab == want[0] and out[4] == [want[5]]
    for got, w in zip(out, want[1:5]):
        assert got == w


@pytest.mark.parametrize("B", [6015, 6016, 6110, 6111, 6143, 6144])
def test_tables_of_batches_around_the_shared_memory_that_needs_no_permission(B):
    """In a process of its own: a larger batch before it would leave the kernel with the permission."""
    code = f"from tests.test_gpu_packed_edges import _tables_equal; _tables_equal({B})"
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# ---------------------------------------------------------------- gated delta rule
def _offsets(what):
    """Offsets of requests some of which are bad, and their number of rows."""
    if what == "too large among many":
        cu = list(range(0, 6500, 100))
        cu[2] = 10 ** 6
        return cu, 6400
    if what == "negative in the middle":
        return [0, 100, -100000, 300, 400], 400
    if what == "descending to rows of their own":
        return [100, 200, 0, 100, 50, 50], 200  # requests 0 and 2 are whole and share no row, 1 and 3 are bad
    cu = list(range(0, 26 * 41, 26))
    for b in range(3, 41, 7):
        cu[b] = (-5, 2 ** 31 - 1, -2 ** 31, 10 ** 5, 2000, -1)[b % 6]
    return cu, 26 * 40


@pytest.mark.parametrize("what", ["too large among many", "negative in the middle", "descending to rows of their own",
                                  "several among many"])
def test_gdn_a_bad_offset_spoils_no_other_request(what):
    import torch

    cu, T = _offsets(what)
    B, H, P = len(cu) - 1, 2, 64
    d, _, _ = _gdn_inputs([T], H, 128, P, "bfloat16", 31, state=False)
    S0 = _t(0.1 * np.random.default_rng(32).normal(size=(B, H, P, 128)))
    good = [b for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= T]
    assert 0 < len(good) < B
    err, y, So = _err(), torch.full((T, H, P), 7.25, device="cuda"), torch.full_like(S0, 7.25)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where operands are missing
    rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], _i(cu), S0, y=y, S_out=So, err=err, workspace=ws)
    assert err[0].item() == rssm.RSSM_DEV_BAD_LENGTHS and err[1].item() not in good
    owned = np.zeros(T, bool)
    for b in range(B):
        if b not in good:
            assert (So[b] == 7.25).all(), b
            continue
        rows = slice(cu[b], cu[b + 1])
        want, Sw = packed.gdn(*(_np(d[n])[rows] for n in ("q", "k", "v", "alpha", "beta")), [0, cu[b + 1] - cu[b]], _np(S0)[b:b + 1])
        _close(_np(y)[rows], want, b)
        _close(_np(So)[b:b + 1], Sw, b)
        owned[rows] = True
    assert (y[_t(~owned, "bool")] == 7.25).all(), "rows of no request were written"


def test_gdn_requests_that_overlap_past_all_room_are_reported():
    """Six requests that each claim all rows (every second offset goes back to 0) ask for more chunks than these rows
    can have; the call ends at once and says so."""
    import time

    import torch

    cu = [0, 600] * 6
    d, _, _ = _gdn_inputs([600], 2, 128, 64, "bfloat16", 33, state=False)
    err = _err()
    torch.cuda.synchronize()
    t0 = time.monotonic()
    rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], _i(cu), err=err)
    assert err[0].item() == rssm.RSSM_DEV_BAD_LENGTHS and time.monotonic() - t0 < 1.0
    y, S = _gdn_run(d, [0, 600], None)
    want, Sw = _gdn_ref(d, [0, 600], None)
    _close(y, want, "the next call")
    _close(S, Sw, "the next call")


def test_gdn_more_requests_than_one_round_of_the_search():
    lens = [(7 * b) % 90 for b in range(70)] + [200, 0, 0, 65]
    d, cu, S0 = _gdn_inputs(lens, 2, 128, 64, "bfloat16", 34, first=2, pad=70)
    y, S = _gdn_run(d, cu, S0)
    want, Sw = _gdn_ref(d, cu, S0)
    _close(y, want, "y")
    _close(S, Sw, "state")


@pytest.mark.parametrize("lens", [[1] * 40 + [300] + [2] * 9 + [12, 13, 0], [500] + [1] * 3, [64, 12, 13, 128]])
def test_gdn_a_request_is_served_the_same_whatever_it_is_packed_with(lens):
    """Bit for bit, in arrays with and without rows behind the requests: which form serves a request goes by its length."""
    import torch

    H, P = 2, 128
    d, cu, S0 = _gdn_inputs(lens, H, 128, P, "bfloat16", 35, pad=100)
    y, S = _gdn_run(d, cu, S0)
    want, Sw = _gdn_ref(d, cu, S0)
    _close(y, want, "y")
    _close(S, Sw, "state")
    cut = {n: t[:cu[-1]].contiguous() for n, t in d.items()}
    y2, S2 = _gdn_run(cut, cu, S0)
    assert np.array_equal(y2, y[:cu[-1]]) and np.array_equal(S2, S)
    for b in sorted({lens.index(n) for n in lens if n}):
        alone = {n: t[cu[b]:cu[b + 1]].contiguous() for n, t in d.items()}
        y1, S1 = _gdn_run(alone, [0, lens[b]], S0[b:b + 1].contiguous())
        assert np.array_equal(y1, y[cu[b]:cu[b + 1]]) and np.array_equal(S1[0], S[b]), lens[b]
    short = [b for b in range(len(lens)) if 0 < lens[b] <= 12]
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in short]) if short else np.zeros(0, int)
    if len(rows):  # fp32 throughout: 2^-24 of the sums' terms, a few dozen of them
        assert np.abs(y[rows] - want[rows]).max() <= 1e-6 * np.abs(want[rows]).max()
    assert torch.is_tensor(S0)


def test_gdn_long_prompts_beside_single_tokens_are_not_served_token_by_token():
    """A prompt of 2048 tokens with 255 single tokens takes about as long as the two apart: token by token it would be
    three times as long."""
    import torch

    def run(lens):
        d, cu, S0 = _gdn_inputs(lens, 4, 128, 128, "bfloat16", 36)
        cud, y, S = _i(cu), torch.empty_like(d["v"], dtype=torch.float32), torch.empty_like(S0)
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        best = float("inf")
        for _ in range(6):
            e[0].record()
            rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], cud, S0, y=y, S_out=S)
            e[1].record()
            e[1].synchronize()
            best = min(best, e[0].elapsed_time(e[1]))
        return best

    apart = run([2048]) + run([1] * 255)
    assert run([1] * 255 + [2048]) < 1.6 * apart


@pytest.mark.parametrize("lens", [[300, 1, 0, 65], [700]])
def test_gdn_in_fp32_on_request(lens):
    """bf16 prompts that are served in chunks otherwise.  The recurrence rounds each of a token's sums to 2^-24 of itself; over
    700 tokens whose decays and writes forget, a few dozen such roundings are alive: 1e-6 of the result in the 2-norm is room
    for all of them at their worst, and a sixth of what chunks leave."""
    d, cu, S0 = _gdn_inputs(lens, 2, 128, 128, "bfloat16", 41)
    want, Sw = _gdn_ref(d, cu, S0)
    y, S = _gdn_run(d, cu, S0, fp32=True)
    for got, w in ((y, want), (S, Sw)):
        assert np.sqrt(((got - w) ** 2).sum()) <= 1e-6 * np.sqrt((w ** 2).sum())


def _same_where_finite(got, want, what):
    """Not finite at the same places, and the tolerance elsewhere."""
    lost = ~np.isfinite(want)
    assert np.array_equal(~np.isfinite(got), lost), (what, np.argwhere(~np.isfinite(got) != lost)[:5])
    _close(got[~lost], want[~lost], what)


@pytest.mark.parametrize("lens", [[150, 20, 40], [9, 20, 40]])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "alpha", "beta"])
def test_gdn_what_is_not_finite_reaches_no_earlier_output(name, value, lens):
    """One value at token 70 (or 5, and at the first one of the next request): outputs before it, of the other heads, of
    other requests and (in v) of the other channels are what they are without it.  In chunks and by the recurrence."""
    H, P = 2, 72
    d, cu, S0 = _gdn_inputs(lens, H, 128, P, "bfloat16", 37)
    for t, h in ((70 if lens[0] > 70 else 5, 1), (cu[1], 0)):
        d[name][(t, h) if d[name].dim() == 2 else (t, h, 40)] = value
    with np.errstate(invalid="ignore"):
        want, Sw = _gdn_ref(d, cu, S0)
    y, S = _gdn_run(d, cu, S0)
    _same_where_finite(y, want, "y")
    _same_where_finite(S, Sw, "state")
    assert np.isfinite(y[:5]).all() and np.isfinite(y[cu[2]:]).all() and not np.isfinite(y).all()


@pytest.mark.parametrize("first", [0, 15, 16, 17, 31, 47, 63])
def test_gdn_a_nan_key_anywhere_in_a_chunk(first):
    """At every place where the triangular system is put together from blocks."""
    d, cu, S0 = _gdn_inputs([130], 1, 128, 64, "bfloat16", 38)
    d["k"][64 + first, 0, 3] = float("nan")
    with np.errstate(invalid="ignore"):
        want, Sw = _gdn_ref(d, cu, S0)
    y, S = _gdn_run(d, cu, S0)
    _same_where_finite(y, want, "y")
    assert np.isfinite(y[:64 + first]).all() and np.isnan(y[64 + first:]).all() and np.isnan(S).all()


def test_gdn_a_state_that_outgrows_fp32_leaves_earlier_outputs():
    """One key of length 3 throughout, full strength: the state grows eightfold a token, past fp32 at about the 43rd.  The
    outputs of the tokens before are sums of terms eight times the next smaller one, so that each keeps 4 * 2^-18 of itself
    times 8 / 7 from the geometric sum of the terms, twice for the two products: below 1e-4; with fp32's last 2 binades left out."""
    import torch

    d, cu, S0 = _gdn_inputs([64], 1, 128, 64, "bfloat16", 39)
    k = torch.zeros_like(d["k"])
    k[:, :, 3] = 3.0
    d["k"], d["q"], d["alpha"], d["beta"] = k, k.clone(), torch.ones_like(d["alpha"]), torch.ones_like(d["beta"])
    want, _ = _gdn_ref(d, cu, S0)
    y, S = _gdn_run(d, cu, S0)
    size = np.sqrt((want ** 2).mean((1, 2)))
    fits = np.abs(want).max((1, 2)) < 2.0 ** 120
    assert 30 < fits.sum() < 50
    far = np.sqrt(((y - want)[fits] ** 2).mean((1, 2)))
    assert (far <= 1e-4 * size[fits]).all(), (far / size[fits]).max()
    assert not np.isfinite(y[-1]).any() and not np.isfinite(S[0, 0, :, 3]).any()



# ---------------------------------------------------------------- attention over the 4-bit cache
@pytest.mark.parametrize("lens,news,Hq,Hk", [([5, 30], [8, 1], 4, 2), ([200, 30, 300], [150, 40, 129], 16, 1), ([4000, 30], [1, 40], 8, 2)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_attend_an_infinite_query_is_nan_where_it_sees_and_zero_where_it_sees_nothing(lens, news, Hq, Hk, sign):
    """One visible token, whose score is -inf or +inf: exp(s - max) is that of inf - inf.  The other rows are as without it."""
    c = _attend_case(51 + Hq, lens, news, Hq, Hk, 128, 16)
    b = int(np.argmax(np.array(news) > np.array(lens)))  # a request whose first rows see nothing
    clean = _attend_run(c)
    one, none = c["cu"][b] + news[b] - lens[b], c["cu"][b] + news[b] - lens[b] - 1
    key = c["K"][b][0, 1 // (Hq // Hk)]
    d = int(np.argmax(np.abs(key)))
    for row in (one, none):
        c["q"][row, 1, d] = sign * float(np.sign(key[d])) * float("inf")
    got = _attend_run(c)
    assert np.isnan(got[one, 1]).all() and not got[none].any()
    got[one, 1] = clean[one, 1] = 0
    assert np.array_equal(got, clean)


# ---------------------------------------------------------------- the hybrid stack on the 4-bit cache
def _stack(**kw):
    shape = HybridShape(batch=3, blocks=1, ssm_per_block=1, d_model=256, nheads=4, headdim=32, dstate=64, ngroups=2, window=4,
                        n_q_heads=8, n_kv_heads=2, head_dim=64, context=61)
    return HybridStack(shape, seed=7, max_steps=20, kv_cache="fp4", page_size=16, **kw)


def test_hybrid_stack_says_when_its_cache_refused_a_step():
    import torch

    st = _stack()
    x = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        st.step(x)
        st.check_cache()
    st.cached_len = st.cached_len - 1000  # the device refuses lengths below 0
    st.step(x)
    with pytest.raises(rssm.RssmError, match="device error 4, request 0") as e:
        st.check_cache()
    assert e.value.status == rssm.RSSM_EDEVICE
    with pytest.raises(rssm.RssmError, match="device error 4"):  # without being asked, by the step after the next at the latest
        for _ in range(3):
            torch.cuda.synchronize()
            st.step(x)
    full = HybridStack(st.s, seed=7, max_steps=4)
    full.step(x)
    full.check_cache()  # nothing to check


# ---------------------------------------------------------------- attention: single tokens and prompt chunks in one batch
MIXED = [
    # news, Hq, Hk, D: most requests single tokens (tiles numbered through), or most of them chunks (a grid row each)
    ([1] * 20 + [70, 9, 0, 2], 16, 1, 128),
    ([1] * 9 + [0, 150] + [1] * 6, 16, 2, 64),
    ([70, 1, 64, 80, 66, 1, 77, 0, 3], 16, 1, 128),
    ([1] * 30 + [40, 1, 5], 20, 1, 64),     # 20 rows a token: the split kernel has tiles of 32
    ([1] * 12 + [33, 1, 20], 40, 1, 128),   # 40 rows a token: none
]


@pytest.mark.parametrize("news,Hq,Hk,D", MIXED)
def test_attend_single_tokens_beside_chunks(news, Hq, Hk, D):
    r = np.random.default_rng(len(news) + Hq)
    lens = [int(n + r.integers(0, 700 if n == 1 else 150)) for n in news]
    lens[0], lens[1] = 1500, 0 if news[1] == 1 else lens[1]  # a long context of its own; a row that sees nothing
    c = _attend_case(53 + Hq, lens, news, Hq, Hk, D, 32, first=2, pad=4)
    _attend_check(c, _attend_run(c))


@pytest.mark.parametrize("bad", ["offsets", "length", "overlap"])
def test_attend_a_bad_request_in_a_mixed_batch_spoils_no_other(bad):
    import torch

    news = [1] * 20 + [70, 9, 1, 2]
    c = _attend_case(54, [n + 300 for n in news], news, 16, 1, 128, 32)
    clean = _attend_run(c)
    cu, lens = list(c["cu"]), [n + 300 for n in news]
    if bad == "offsets":
        cu[7] = 10 ** 6  # requests 6 and 7
        spoilt = {6, 7}
    elif bad == "length":
        lens[20] = -1
        spoilt = {20}
    else:  # every second request claims all rows up to its own: more tiles than the rows can make
        cu = [0, 102] * 12 + [0]
        spoilt = set(range(24))
    err, out = _err(), torch.full_like(c["q"], 7.25)
    rssm.kv4_attend(c["q"], c["cache"], c["table"], _i(lens), _i(cu), 102, out=out, err=err, **c["kw"])
    assert err[0].item() == rssm.RSSM_DEV_BAD_LENGTHS and (err[1].item() in spoilt or err[1].item() == -1)
    got = _np(out)
    for b in set(range(24)) - spoilt:
        rows = slice(c["cu"][b], c["cu"][b + 1])
        assert np.abs(got[rows] - clean[rows]).max() <= 2.0 ** -7 * np.abs(c["V"][b]).max(), b
    if bad != "overlap":
        for b in spoilt:
            assert (got[c["cu"][b]:c["cu"][b + 1]] == 7.25).all()


def test_attend_a_mixed_step_takes_about_as_long_as_its_parts():
    """15 tokens over 8192 and a chunk of 256: served by one kernel, each token would be one CTA's for its whole context."""
    import torch

    def run(lens, news):
        c = _attend_case(55, lens, news, 16, 1, 128, 64)
        out, cu = torch.empty_like(c["q"]), _i(c["cu"])
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        best = float("inf")
        for _ in range(6):
            e[0].record()
            rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], cu, c["max_q"], out=out, **c["kw"])
            e[1].record()
            e[1].synchronize()
            best = min(best, e[0].elapsed_time(e[1]))
        return best

    apart = run([8192] * 15, [1] * 15) + run([512], [256])
    assert run([8192] * 15 + [512], [1] * 15 + [256]) < 1.6 * apart


@pytest.mark.parametrize("D,ps,n", [(128, 64, 1500), (64, 16, 1300), (128, 256, 2600)])
def test_attend_tiles_over_many_tiles_of_tokens(D, ps, n):
    """10 to 21 tiles of tokens a row tile: every barrier and page word of the 128-row kernel in use several times over; scores that
    grow along the context, so that the running maximum moves in the last tiles too, and ones that do not; a page that
    is not there in the 6th."""
    c = _attend_case(56 + D, [n, n - 200, 40], [9, 64, 8], 16, 4, D, ps)
    got = _attend_run(c)
    _attend_check(c, got)
    rise = dict(c, q=(c["q"].float() * 6).to(c["q"].dtype))
    _attend_check(rise, _attend_run(rise))
    table = c["table"].clone()
    at = 700 // ps
    table[0, at] = -1
    err = _err()
    gone = _np(rssm.kv4_attend(c["q"], c["cache"], table, c["lens"], _i(c["cu"]), c["max_q"], err=err, **c["kw"]))
    assert err[:2].tolist() == [rssm.RSSM_DEV_BAD_PAGE, 0]
    assert np.array_equal(gone[c["cu"][1]:], got[c["cu"][1]:])
    keep = np.r_[0:at * ps, min(n, (at + 1) * ps):n]
    d = dict(c, K=[c["K"][0][keep]], V=[c["V"][0][keep]], q=c["q"][:9], cu=[0, 9])
    _attend_check(d, gone[:9])


# ---------------------------------------------------------------- writing the 4-bit cache
@pytest.mark.parametrize("T,Hk,D,ps", [(37, 2, 128, 16), (129, 8, 128, 256), (300, 3, 64, 48)])
def test_append_leaves_every_byte_of_other_slots(T, Hk, D, ps):
    """A cache full of some bytes: behind a write of some slots, and one that skips half of them, every byte that belongs to
    another slot is as it was; the others are those of a write into a cache of zeros."""
    import torch

    r = np.random.default_rng(T)
    pages = -(-T // ps) + 1
    slots = r.permutation(pages * ps)[:T]
    k, v = (_t(r.normal(size=(T, Hk, D)), "bfloat16") for _ in range(2))

    def of_slots(some):
        """Bool [pages, Hk, bytes]: the bytes that belong to these slots."""
        m = np.zeros((pages, 2, ps, D // 2 + D // 16), bool)  # keys and values: codes and scales of a token
        m[np.asarray(some) // ps, :, np.asarray(some) % ps] = True
        codes, scales = m[..., :D // 2].reshape(pages, 2, -1), m[..., D // 2:].reshape(pages, 2, -1)
        page = np.concatenate([codes[:, 0], scales[:, 0], codes[:, 1], scales[:, 1]], 1)
        return np.broadcast_to(page[:, None], (pages, Hk, page.shape[1]))

    for used in (np.arange(T), np.arange(T)[::2]):
        named = np.full(T, -1)
        named[used] = slots[used]
        cache, zeros = (torch.full((pages, Hk, ps * D * 9 // 8), fill, dtype=torch.uint8, device="cuda") for fill in (0xA5, 0))
        for c in (cache, zeros):
            rssm.kv4_append(k, v, _i(named), c, k_scale=0.25, v_scale=0.5)
        got, mine = cache.cpu().numpy(), of_slots(slots[used])
        assert (got[~mine] == 0xA5).all()
        assert np.array_equal(got[mine], zeros.cpu().numpy()[mine])


def test_operators_repeat_themselves_bit_for_bit():
    """The same call twice, and once more beside other work: no result hangs on the order in which CTAs end."""
    import torch

    c = _attend_case(57, [3000, 700, 40, 900], [1, 3, 1, 40], 16, 1, 128, 64)
    d, cu, S0 = _gdn_inputs([1, 300, 12, 70, 0, 5], 4, 128, 128, "bfloat16", 58)
    first = None
    for n in range(3):
        if n == 2:
            noise = torch.randn(2048, 2048, device="cuda")
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    noise = noise @ noise * 1e-2
        got = [_attend_run(c), *_gdn_run(d, cu, S0)]
        first = first or got
        for a, b in zip(got, first):
            assert np.array_equal(a, b)


# ---------------------------------------------------------------- calls that follow one another closely, and at once
def test_calls_back_to_back_in_one_workspace_and_at_once_on_three_streams():
    """The delta rule and the attention launch kernels that start before the one in front has ended.  Call after call in the
    same workspace and outputs, on one stream and on three at once (each with its own), every result is bit for bit that
    of the call alone."""
    import torch

    sets = []
    for seed in (71, 72, 73):
        r = np.random.default_rng(seed)
        lens = [int(n) for n in np.where(r.random(20) < 0.6, r.integers(0, 13, 20), r.integers(13, 260, 20))]
        d, cu, S0 = _gdn_inputs(lens, 4, 128, 128, "bfloat16", seed, pad=int(r.integers(0, 200)))
        news = [1] * 18 + [40, 70, 0, 3]
        c = _attend_case(seed, [n + int(r.integers(0, 600)) for n in news], news, 16, 1, 128, 32)
        sets.append((d, _i(cu), S0, c, _i(c["cu"])))

    def run(s, y, S, out, ws):
        d, cu, S0, c, cuq = s
        rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], cu, S0, y=y, S_out=S, workspace=ws)
        rssm.kv4_attend(c["q"], c["cache"], c["table"], c["lens"], cuq, c["max_q"], out=out, workspace=ws, **c["kw"])

    def outputs(s):
        return [torch.zeros((s[0]["q"].shape[0], 4, 128), device="cuda"), torch.zeros_like(s[2]), torch.zeros_like(s[3]["q"]),
                torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")]

    want = []
    for s in sets:
        o = outputs(s)
        run(s, *o)
        torch.cuda.synchronize()
        want.append([t.clone() for t in o[:3]])
    # one stream, one workspace, the sets in turn
    outs = [outputs(s) for s in sets]
    for o in outs[1:]:
        o[3] = outs[0][3]
    for _ in range(30):
        for s, o in zip(sets, outs):
            run(s, *o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o[:3], w))
    # three streams at once
    outs = [outputs(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for n in range(30):
        for s, o, st in zip(sets, outs, streams):
            with torch.cuda.stream(st):
                run(s, *o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o[:3], w))
