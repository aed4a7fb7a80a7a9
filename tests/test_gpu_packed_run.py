"""The operators on packed requests as they are used together: requests of different lengths served in steps
(block tables, delta-rule prefill into a decode layer, attention over the 4-bit cache), captured in graphs, on
streams of their own, and inside the hybrid stack."""
import numpy as np
import pytest

from checkpoint_input_replay_rssm_b200 import rssm
from checkpoint_input_replay_rssm_b200.hybrid import HybridShape, HybridStack
from oracle import packed
from tests.test_gpu_packed import _attend_check, _close, _cu, _err, _gdn_inputs, _gdn_ref, _i, _np, _t

pytestmark = pytest.mark.gpu


def test_serving_steps_of_ragged_requests():
    """Four requests: prompts in two packed steps of their own lengths (one has nothing in the first, one in the
    second), padded to a fixed capacity, then three decode steps.  Every step's outputs are the oracle's: the
    gated-delta layer's from prefill into replay decode, the attention's over what the cache holds."""
    import torch

    B, H, N, P, Hq, Hk, D, ps, cap = 4, 2, 128, 64, 8, 2, 64, 16, 300
    steps = [[70, 0, 33, 129], [5, 64, 100, 0]] + [[1] * B] * 3
    r = np.random.default_rng(41)
    table, free, head = torch.full((B, 20), -1, dtype=torch.int32, device="cuda"), _i(r.permutation(64)), _i([0])
    cache = rssm.kv4_cache(64, Hk, ps, D)
    cached, err = _i([0] * B), _err()
    S = _t(0.1 * r.normal(size=(B, H, P, N)))
    So = _np(S)
    K, V = [np.zeros((0, Hk, D))] * B, [np.zeros((0, Hk, D))] * B
    layer = None
    for n, lens in enumerate(steps):
        mt = cap if n < 2 else B
        cu, seq_len, slots, pos, head = rssm.build_tables(cached, _i(lens), free, head, table, ps, mt, err=err)
        cuh, T = _cu(lens), sum(lens)
        assert cu.tolist() == cuh and pos.tolist()[:T] == [k.shape[0] + t for k, m in zip(K, lens) for t in range(m)]
        # delta-rule layer, all rows of the capacity present, those behind the requests holding NaN
        d, _, _ = _gdn_inputs([mt], H, N, P, "bfloat16", 50 + n)
        for t in d.values():
            t[T:] = float("nan")
        if n < 2:
            y, S = rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], cu, S, err=err)
            if n == 1:
                layer = rssm.Layer(rssm.make_config(kind="gdn", state_dtype="f32", batch=B, nheads=H, headdim=P, dstate=N, window=2))
                layer.import_state(S)
        else:
            y = layer.decode({k: v.unsqueeze(1) for k, v in d.items()})[:, 0]
        want, So = packed.gdn(*(_np(d[k])[:T] for k in ("q", "k", "v", "alpha", "beta")), cuh, So)
        _close(_np(y)[:T], want, n)
        # attention layer
        k, v, q = (_t(r.normal(size=(mt, hd, D)), "bfloat16") for hd in (Hk, Hk, Hq))
        rssm.kv4_append(k, v, slots, cache, k_scale=0.25, v_scale=0.25, err=err)
        hk, hv = packed.hold(_np(k), 0.25), packed.hold(_np(v), 0.25)
        K = [np.concatenate([x, hk[a:b]]) for x, a, b in zip(K, cuh, cuh[1:])]
        V = [np.concatenate([x, hv[a:b]]) for x, a, b in zip(V, cuh, cuh[1:])]
        out = torch.full_like(q, 7.25)
        rssm.kv4_attend(q, cache, table, seq_len, cu, max(lens), k_scale=0.25, v_scale=0.25, out=out, err=err)
        _attend_check(dict(q=q, K=K, V=V, cu=cuh), _np(out))
        assert (out[T:] == 7.25).all()
        cached = seq_len
    assert err.tolist() == [0, 0, 0, 0]
    _close(_np(layer.export_state()), So, "state")


def test_a_step_captured_once_serves_growing_requests():
    """Tables, append and attention of a decode step in one graph, replayed over lengths that grow past pages and
    past the first split; the graph's own copies move the lengths and the free list's head on."""
    import torch

    B, Hq, Hk, D, ps, width = 3, 8, 2, 128, 16, 40
    r = np.random.default_rng(42)
    lens = [1, 255, 500]
    free = _i(r.permutation(B * width + 5))
    table, head, err = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), _i([0]), _err()
    cache = rssm.kv4_cache(B * width + 5, Hk, ps, D)
    cu, cached, slots, _, nh = rssm.build_tables(_i([0] * B), _i(lens), free, head, table, ps, sum(lens))
    head.copy_(nh)
    cached = cached.clone()
    k, v = _t(r.normal(size=(sum(lens), Hk, D)), "bfloat16"), _t(r.normal(size=(sum(lens), Hk, D)), "bfloat16")
    rssm.kv4_append(k, v, slots, cache)
    K, V = ([packed.hold(_np(x), 1.0)[a:b] for a, b in zip(_cu(lens), _cu(lens)[1:])] for x in (k, v))
    sk, sv, sq = torch.zeros(B, Hk, D, device="cuda", dtype=torch.bfloat16), None, torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    sv = torch.zeros_like(sk)
    one = _i([1] * B)
    keep = [t.clone() for t in (table, head, cached, cache)]

    def step():
        cu, seq, slots, _, nh = rssm.build_tables(cached, one, free, head, table, ps, B, err=err)
        rssm.kv4_append(sk, sv, slots, cache, err=err)
        o = rssm.kv4_attend(sq, cache, table, seq, cu, 1, err=err)
        head.copy_(nh)
        cached.copy_(seq)
        return o

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t, s in zip((table, head, cached, cache), keep):
        t.copy_(s)
    for _ in range(20):
        for t, hd in ((sk, Hk), (sv, Hk), (sq, Hq)):
            t.copy_(_t(r.normal(size=(B, hd, D)), "bfloat16"))
        g.replay()
        K = [np.concatenate([a, b[None]]) for a, b in zip(K, packed.hold(_np(sk), 1.0))]
        V = [np.concatenate([a, b[None]]) for a, b in zip(V, packed.hold(_np(sv), 1.0))]
        _attend_check(dict(q=sq, K=K, V=V, cu=list(range(B + 1))), _np(out))
    assert err.tolist() == [0, 0, 0, 0]


def test_two_graphs_of_a_prefill_with_workspaces_of_their_own():
    """The same operator captured twice, replayed at once on two streams, each with its own workspace."""
    import torch

    runs = []
    for seed in (61, 62):
        d, cu, S0 = _gdn_inputs([300, 7, 150], 4, 128, 128, "bfloat16", seed)
        args = (d["q"], d["k"], d["v"], d["alpha"], d["beta"], _i(cu), S0)
        rssm.gdn_prefill(*args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = rssm.gdn_prefill(*args)
        runs.append((g, out, _gdn_ref(d, cu, S0), torch.cuda.Stream(), args))  # the graph reads the inputs where they are
    torch.cuda.synchronize()
    for _ in range(5):
        for g, out, _, st, _ in runs:
            with torch.cuda.stream(st):
                for o in out:
                    o.fill_(7.25)
                g.replay()
    torch.cuda.synchronize()
    for _, (y, S), (yw, Sw), _, _ in runs:
        _close(_np(y), yw, "y")
        _close(_np(S), Sw, "state")


def test_calls_on_a_stream_that_is_not_the_current_one():
    import torch

    st = torch.cuda.Stream()
    d, cu, S0 = _gdn_inputs([100, 3], 2, 128, 64, "bfloat16", 71)
    cud = _i(cu)
    torch.cuda.synchronize()
    y, S = rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], cud, S0, stream=st)
    z = torch.empty_like(y).fill_(3.0)  # the current stream's allocations do not meet the call's workspace
    st.synchronize()
    yw, Sw = _gdn_ref(d, cu, S0)
    _close(_np(y), yw, "y")
    _close(_np(S), Sw, "state")
    assert (z == 3.0).all()
    with pytest.raises(ValueError, match="expected a contiguous"):
        rssm.gdn_prefill(d["q"].transpose(0, 1), d["k"], d["v"], d["alpha"], d["beta"], cud, S0)
    with pytest.raises(ValueError, match="float32"):
        rssm.gdn_prefill(d["q"], d["k"], d["v"], d["alpha"].double(), d["beta"], cud, S0)


SHAPE = HybridShape(batch=3, blocks=2, ssm_per_block=1, d_model=256, nheads=4, headdim=32, dstate=64, ngroups=2, window=4,
                    n_q_heads=8, n_kv_heads=2, head_dim=64, context=61)


@pytest.mark.parametrize("context,page", [(61, 16), (0, 64)])
def test_hybrid_stack_with_a_4bit_cache(context, page):
    """Every attention layer's output over what its cache holds (an oracle of its own per layer and step), from an
    empty cache and from one whose last page is part full.  The layer adds the bf16 attention output times wo to its
    input: the product rounds to bf16 (2^-8 of it), its sum (2^-8 again), and the attention output is within the
    attention test's tolerance, for which 2^-7 of sum_j p_j |v_j| is room enough here (scores below 30)."""
    import dataclasses

    import torch

    shape = dataclasses.replace(SHAPE, context=context)
    st = HybridStack(shape, seed=7, max_steps=20, kv_cache="fp4", page_size=page)
    plain = HybridStack(shape, seed=7, max_steps=20)
    s, g, seen = shape, torch.Generator(device="cuda").manual_seed(3), []
    attn = st._attn
    st._attn = lambda x, p: seen.append((x, p, attn(x, p))) or seen[-1][2]
    for n in range(20):
        x = torch.randn((s.batch, s.d_model), generator=g, device="cuda").to(torch.bfloat16)
        seen.clear()
        st.step(x)
        assert len(seen) == s.blocks
        for x_in, p, x_out in seen:
            L = context + n + 1
            t = np.arange(L)
            tab = st.block_table.cpu().numpy()
            slots = tab[:, t // page] * page + t % page
            k, v = rssm.kv4_export(_i(slots.reshape(-1)), p["cache"], s.head_dim, k_scale=st.KV_SCALE, v_scale=st.KV_SCALE)
            K, V = (list(_np(y).reshape(s.batch, L, s.n_kv_heads, s.head_dim)) for y in (k, v))
            xn = st._norm(x_in)
            kn = _np((xn @ p["wk"]).reshape(s.batch, s.n_kv_heads, s.head_dim))
            assert np.array_equal(np.stack(K)[:, -1], packed.hold(kn, st.KV_SCALE)), "the new token's keys"
            q = _np((xn @ p["wq"]).reshape(s.batch, s.n_q_heads, s.head_dim))
            o, mean, big, _ = packed.attend(q, K, V, list(range(s.batch + 1)), s.head_dim ** -0.5)
            assert big.max() < 30
            w, flat = _np(p["wo"]), (s.batch, s.n_q_heads * s.head_dim)
            add = o.reshape(flat) @ w
            tol = (2.0 ** -7 * mean).reshape(flat) @ np.abs(w) + 2.0 ** -8 * np.abs(add) + 2.0 ** -7 * np.abs(_np(x_out)) + 1e-6
            assert (np.abs(_np(x_out) - _np(x_in) - add) <= tol).all()
    assert st.kv_err.tolist() == [0, 0, 0, 0] and st.cached_len.tolist() == [context + 20] * s.batch
    with pytest.raises(RuntimeError):
        st.step(x)
    with pytest.raises(ValueError, match="kv_cache"):
        HybridStack(shape, kv_cache="fp8")
    assert torch.equal(plain.layers[1][1]["wq"], st.layers[1][1]["wq"])


def test_hybrid_stack_with_a_4bit_cache_refuses_capture(monkeypatch):
    import torch

    st = HybridStack(SHAPE, seed=7, max_steps=4, kv_cache="fp4")
    x = torch.zeros((SHAPE.batch, SHAPE.d_model), dtype=torch.bfloat16, device="cuda")
    before = st.cached_len.tolist()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="replayed graph"):
            st.step(x)
    assert st.cached_len.tolist() == before and st.pos == SHAPE.context
    st.step(x)
    assert st.cached_len.tolist() == [n + 1 for n in before]
