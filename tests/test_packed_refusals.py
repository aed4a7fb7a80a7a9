"""Operators on packed requests: their fp64 oracle is pinned, and calls that cannot be served are
refused before anything is enqueued (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from checkpoint_input_replay_rssm_b200 import rssm
from oracle import packed, quant

P16 = 0x1000  # a 256-byte aligned address that no refused call touches


# ---------------------------------------------------------------- pins of the oracle
def test_gdn_oracle_is_the_closed_form_and_keeps_requests_apart():
    r = np.random.default_rng(1)
    T, H, N, P, cu = 7, 2, 4, 3, [0, 3, 3, 7]
    q, k, v = r.normal(size=(T, H, N)), r.normal(size=(T, H, N)), r.normal(size=(T, H, P))
    a, b, S0 = r.uniform(0.2, 1, (T, H)), r.uniform(0, 1, (T, H)), r.normal(size=(3, H, P, N))
    y, S = packed.gdn(q, k, v, a, b, cu, S0)
    assert np.array_equal(S[1], S0[1])
    for i in (0, 2):
        for h in range(H):
            X = S0[i, h]
            for t in range(cu[i], cu[i + 1]):
                kk = np.outer(k[t, h], k[t, h])
                X = a[t, h] * X @ (np.eye(N) - b[t, h] * kk) + b[t, h] * np.outer(v[t, h], k[t, h])
                np.testing.assert_allclose(y[t, h], X @ q[t, h], rtol=0, atol=1e-12)
            np.testing.assert_allclose(S[i, h], X, rtol=0, atol=1e-12)


def test_held_values_are_the_formats_casts():
    import torch

    assert np.array_equal(packed.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    r = np.random.default_rng(2)
    x = np.abs(r.normal(size=4000)) * np.exp2(r.integers(-12, 10, 4000))
    x = np.concatenate([x, packed.E4M3, (packed.E4M3[1:] + packed.E4M3[:-1]) / 2]).astype(np.float32)
    want = quant.e4m3_rne(x)
    assert np.array_equal(packed.E4M3[packed.nearest(x.astype(np.float64), packed.E4M3)], want)
    # ties of the code go to the even one, and past 6 to 6
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0])
    assert packed.E2M1[packed.nearest(ties, packed.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


def test_tables_oracle_by_hand():
    got = packed.tables([0, 17, 16], [3, 0, 2], [9, 8, 7], 1, [[-1, -1], [4, 5], [6, -1]], 16, 7)
    assert got == ([[8, -1], [4, 5], [6, 7]], [0, 3, 3, 5], [3, 17, 18],
                   [128, 129, 130, 112, 113, -1, -1], [0, 1, 2, 16, 17, -1, -1], 3)
    assert packed.tables([0], [33], [1, 2, 3], 0, [[-1, -1]], 16, 64) is None  # longer than its row
    assert packed.tables([0], [33], [1, 2], 0, [[-1] * 3], 16, 64) is None     # no third page
    assert packed.tables([0], [33], [1, 2, 3], 0, [[-1] * 3], 16, 32) is None  # no room in the map


def test_attend_oracle_sees_itself_and_no_later_row():
    q = np.array([[[1.0]], [[1.0]]])
    K, V = [np.array([[[0.0]], [[np.log(3.0)]], [[50.0]]])], [np.array([[[1.0]], [[5.0]], [[9.0]]])]
    out = packed.attend(q, K, V, [0, 2], 1.0)[0]
    assert out[0, 0, 0] == pytest.approx(4.0, abs=1e-12) and out[1, 0, 0] == pytest.approx(9.0, abs=1e-6)
    assert packed.attend(q, [K[0][:0]], [V[0][:0]], [0, 2], 1.0)[0].tolist() == [[[0.0]], [[0.0]]]


# ---------------------------------------------------------------- refusals
def _gdn(lib, ws=P16, ws_bytes=1 << 40, drop=(), S0=None, S_out=P16, y=P16, **kw):
    c = dict(batch=2, nheads=4, headdim=128, dstate=128, input_dtype=rssm.RSSM_BF16, tokens=10) | kw
    cfg = rssm.rssm_gdn_prefill_config(*c.values())
    ins = rssm.rssm_inputs(**{n: P16 for n in ("q", "k", "v", "alpha", "beta") if n not in drop})
    return lib.rssm_gdn_prefill(ctypes.byref(cfg), S0, ctypes.byref(ins), None if "cu" in drop else P16, y, S_out, ws,
                                ws_bytes, None, None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(nheads=0), dict(nheads=65536), dict(headdim=0), dict(headdim=12),
    dict(headdim=264), dict(dstate=48), dict(dstate=256), dict(input_dtype=rssm.RSSM_FP8E4M3), dict(tokens=0),
    dict(tokens=-1), dict(drop=("q",)), dict(drop=("k",)), dict(drop=("v",)), dict(drop=("alpha",)),
    dict(drop=("beta",)), dict(drop=("cu",)), dict(y=None), dict(y=P16 + 4), dict(S_out=None), dict(S_out=P16 + 8),
    dict(S0=P16), dict(S0=2 * P16 + 4)])
def test_gdn_prefill_refuses(kw):
    assert _gdn(rssm.load(), **kw) == rssm.RSSM_EINVAL


def test_gdn_prefill_refuses_a_missing_or_small_workspace():
    lib = rssm.load()
    cfg = rssm.rssm_gdn_prefill_config(2, 4, 128, 128, rssm.RSSM_BF16, 10)
    need = lib.rssm_gdn_prefill_workspace_bytes(ctypes.byref(cfg))
    if need:
        for ws, nb in ((None, need), (P16, need - 1), (P16 + 128, need)):
            assert _gdn(lib, ws=ws, ws_bytes=nb) == rssm.RSSM_EINVAL
    cfg.dstate = 48
    assert lib.rssm_gdn_prefill_workspace_bytes(ctypes.byref(cfg)) == 0
    assert lib.rssm_gdn_prefill_workspace_bytes(None) == 0


TAB = ("cached_len", "new_len", "free_pages", "free_head", "block_table", "cu_new", "seq_len", "slot_map", "position",
       "next_free")


def _tables(drop=(), alias=None, **kw):
    c = dict(batch=2, page_size=16, max_pages=4, num_free=8, max_tokens=32) | kw
    p = [None if n in drop else P16 * (i + 1) for i, n in enumerate(TAB)]
    if alias:
        p[TAB.index(alias[0])] = p[TAB.index(alias[1])]
    cfg = rssm.rssm_tables_config(*c.values())
    return rssm.load().rssm_build_tables(ctypes.byref(cfg), *p, None, None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=16385), dict(page_size=0), dict(page_size=65537), dict(max_pages=0), dict(num_free=-1),
    dict(num_free=(1 << 30) + 1), dict(max_tokens=0), dict(max_tokens=(1 << 30) + 1), dict(alias=("next_free", "free_head")),
    dict(alias=("seq_len", "cached_len")), dict(alias=("seq_len", "new_len")),
    dict(max_pages=1 << 20, page_size=4096)] + [dict(drop=(n,)) for n in TAB])
def test_build_tables_refuses(kw):
    assert _tables(**kw) == rssm.RSSM_EINVAL


def _kv(**kw):
    c = dict(n_kv_heads=2, head_dim=128, page_size=16, num_pages=4, k_scale=1.0, v_scale=0.25) | kw
    return rssm.rssm_kv4_config(*c.values())


BAD_KV = [dict(n_kv_heads=0), dict(n_kv_heads=65536), dict(head_dim=96), dict(head_dim=256), dict(page_size=0),
          dict(page_size=8), dict(page_size=24), dict(page_size=272), dict(num_pages=0),
          dict(num_pages=1 << 28), dict(k_scale=0.0), dict(k_scale=-1.0), dict(v_scale=3.0), dict(k_scale=float("nan")),
          dict(v_scale=float("inf")), dict(k_scale=2.0 ** -65), dict(v_scale=2.0 ** 65)]


@pytest.mark.parametrize("kw", BAD_KV)
def test_cache_configs_refused(kw):
    lib, cfg = rssm.load(), _kv(**kw)
    assert lib.rssm_kv4_cache_bytes(ctypes.byref(cfg)) == 0
    for f in (lib.rssm_kv4_append, lib.rssm_kv4_export):
        assert f(ctypes.byref(cfg), 3, P16, P16, P16, P16, None, None) == rssm.RSSM_EINVAL
    assert _attend(cfg) == rssm.RSSM_EINVAL


def test_cache_bytes():
    lib = rssm.load()
    assert lib.rssm_kv4_cache_bytes(ctypes.byref(_kv())) == 4 * 2 * 16 * (64 + 8) * 2
    assert lib.rssm_kv4_cache_bytes(ctypes.byref(_kv(num_pages=1 << 26, head_dim=64))) == (1 << 26) * 2 * 16 * 72
    assert lib.rssm_kv4_cache_bytes(None) == 0


@pytest.mark.parametrize("name", ["rssm_kv4_append", "rssm_kv4_export"])
def test_append_and_export_refuse(name):
    f, cfg = getattr(rssm.load(), name), _kv()
    assert f(ctypes.byref(cfg), 0, P16, P16, P16, P16, None, None) == rssm.RSSM_EINVAL
    for i in range(4):
        p = [P16] * 4
        p[i] = None
        assert f(ctypes.byref(cfg), 3, *p, None, None) == rssm.RSSM_EINVAL
    # k, v and the cache lie on 16-byte boundaries
    wide = (0, 1, 3) if name == "rssm_kv4_append" else (1, 2, 3)
    for i in wide:
        p = [P16] * 4
        p[i] += 8
        assert f(ctypes.byref(cfg), 3, *p, None, None) == rssm.RSSM_EINVAL


def _attend(cfg=None, null=None, off=None, ws=P16, ws_bytes=1 << 40, **kw):
    a = dict(batch=2, n_q_heads=8, tokens=5, max_pages=4, max_q=3, max_seq=64, sm_scale=0.1) | kw
    att = rssm.rssm_attend_config(*a.values())
    p = [P16] * 6  # q, cache, block_table, seq_len, cu_q, out
    if null is not None:
        p[null] = None
    if off is not None:
        p[off] += 8
    cfg = cfg or _kv()
    return rssm.load().rssm_kv4_attend(ctypes.byref(cfg), ctypes.byref(att), *p, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(n_q_heads=0), dict(n_q_heads=7), dict(n_q_heads=65536), dict(tokens=0),
    dict(max_pages=0), dict(max_q=0), dict(max_seq=0), dict(max_pages=1 << 27, max_seq=(1 << 30) + 1), dict(sm_scale=float("nan")), dict(sm_scale=float("inf"))]
    + [dict(null=i) for i in range(6)] + [dict(off=i) for i in (0, 1, 5)])
def test_attend_refuses(kw):
    assert _attend(**kw) == rssm.RSSM_EINVAL


def test_attend_refuses_a_missing_or_small_workspace():
    lib = rssm.load()
    cfg, att = _kv(num_pages=1 << 16), rssm.rssm_attend_config(1, 8, 1, 1 << 16, 1, 1 << 20, 0.1)
    need = lib.rssm_kv4_attend_workspace_bytes(ctypes.byref(cfg), ctypes.byref(att))
    kw = dict(batch=1, tokens=1, max_pages=1 << 16, max_q=1, max_seq=1 << 20)
    if need:
        for ws, nb in ((None, need), (P16, need - 1), (P16 + 128, need)):
            assert _attend(cfg, ws=ws, ws_bytes=nb, **kw) == rssm.RSSM_EINVAL
    att.n_q_heads = 7
    assert lib.rssm_kv4_attend_workspace_bytes(ctypes.byref(cfg), ctypes.byref(att)) == 0


def test_torch_wrappers_refuse_host_tensors_and_wrong_shapes():
    import torch

    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)  # noqa: E731
    i32, bf, u8 = torch.int32, torch.bfloat16, torch.uint8
    with pytest.raises(ValueError, match="CUDA"):
        rssm.gdn_prefill(z(3, 2, 16), z(3, 2, 16), z(3, 2, 8), z(3, 2), z(3, 2), z(2, t=i32))
    with pytest.raises(ValueError, match="CUDA"):
        rssm.build_tables(z(2, t=i32), z(2, t=i32), z(4, t=i32), z(1, t=i32), z(2, 3, t=i32), 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        rssm.kv4_append(z(3, 2, 64, t=bf), z(3, 2, 64, t=bf), z(3, t=i32), z(2, 2, 16 * 72, t=u8))
    with pytest.raises(ValueError, match="CUDA"):
        rssm.kv4_export(z(3, t=i32), z(2, 2, 16 * 72, t=u8), 64)
    with pytest.raises(ValueError, match="CUDA"):
        rssm.kv4_attend(z(3, 4, 64, t=bf), z(2, 2, 16 * 72, t=u8), z(1, 2, t=i32), z(1, t=i32), z(2, t=i32), 3)
    with pytest.raises(rssm.RssmError):
        rssm.kv4_cache(4, 2, 24, 128, device="cpu")
    assert rssm.kv4_cache(4, 2, 16, 128, device="cpu").shape == (4, 2, 16 * 144)
