"""What the operators on packed requests ask for before a launch: workspaces by the sizes of the call alone, and calls without
them refused (no GPU needed)."""
import ctypes

import pytest

from checkpoint_input_replay_rssm_b200 import rssm

P16 = 0x1000  # a 256-byte aligned address that no refused call touches


def _gdn_bytes(batch, tokens, **kw):
    c = dict(batch=batch, nheads=4, headdim=128, dstate=128, input_dtype=rssm.RSSM_BF16, tokens=tokens) | kw
    return rssm.load().rssm_gdn_prefill_workspace_bytes(ctypes.byref(rssm.rssm_gdn_prefill_config(*c.values())))


def test_gdn_workspace_goes_by_what_the_rows_can_hold():
    assert _gdn_bytes(64, 12) == 0  # no request of more than 12 tokens fits
    assert _gdn_bytes(1, 13) > 0 and _gdn_bytes(64, 13) > 0
    # one prompt and many single tokens may be in any batch of so many rows
    assert _gdn_bytes(256, 2303) >= 36 * 4 * 2 * 128 * 64 * 2
    assert _gdn_bytes(1, 10 ** 5) > _gdn_bytes(1, 10 ** 4) and _gdn_bytes(100, 10 ** 4) >= _gdn_bytes(1, 10 ** 4)
    for kw in (dict(dstate=64), dict(input_dtype=rssm.RSSM_F32), dict(input_dtype=rssm.RSSM_BF16 + rssm.RSSM_GDN_FP32)):
        assert _gdn_bytes(4, 1000, **kw) == 0


@pytest.mark.parametrize("kind", [rssm.RSSM_FP8E4M3 + rssm.RSSM_GDN_FP32, 512, -1, 3])
def test_gdn_input_types_refused(kind):
    cfg = rssm.rssm_gdn_prefill_config(1, 4, 128, 128, kind, 10)
    ins = rssm.rssm_inputs(**{n: P16 for n in ("q", "k", "v", "alpha", "beta")})
    assert rssm.load().rssm_gdn_prefill(ctypes.byref(cfg), None, ctypes.byref(ins), P16, P16, P16, P16, 1 << 40, None, None) == rssm.RSSM_EINVAL


def _attend_bytes(batch, Hq, tokens, max_pages, max_q, max_seq, Hk=2):
    kv = rssm.rssm_kv4_config(Hk, 128, 64, 1 << 12, 1.0, 1.0)
    att = rssm.rssm_attend_config(batch, Hq, tokens, max_pages, max_q, max_seq, 0.1)
    return rssm.load().rssm_kv4_attend_workspace_bytes(ctypes.byref(kv), ctypes.byref(att)), kv, att


def test_attend_workspace_of_a_mixed_batch_is_that_of_its_single_tokens():
    decode, _, _ = _attend_bytes(64, 32, 64, 512, 1, 1 << 15)
    mixed, kv, att = _attend_bytes(64, 32, 575, 512, 512, 1 << 15)
    assert mixed == decode > 0
    lib = rssm.load()
    for ws, nb in ((None, mixed), (P16, mixed - 1), (P16 + 128, mixed)):
        assert lib.rssm_kv4_attend(ctypes.byref(kv), ctypes.byref(att), *[P16] * 6, ws, nb, None, None) == rssm.RSSM_EINVAL
    assert _attend_bytes(64, 128, 575, 512, 512, 1 << 15)[0] == 0  # 64 rows a token: tiles of 128 rows alone


@pytest.mark.parametrize("batch,max_q", [(1, 1), (3, 4), (256, 1), (8, 600)])
def test_attend_workspace_does_not_shrink_with_the_context(batch, max_q):
    sizes = [_attend_bytes(batch, 32, batch * max_q, 1 << 12, max_q, n)[0] for n in (1, 256, 4096, 1 << 16, 1 << 18)]
    assert sizes == sorted(sizes)
