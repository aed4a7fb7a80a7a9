"""ctypes binding of librssm (include/rssm.h): argument marshalling only.

The module-level functions carry the C names and signatures; ``Layer`` is a
convenience owner of one handle whose workspace and outputs are torch CUDA
tensors, passing raw device pointers and ``torch.cuda.current_stream()``.
Every step of the decode path runs in librssm's kernels; there is no fallback:
loading fails loudly when the library is missing, and calls fail when no CUDA
device is present.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librssm.so")

RSSM_OK, RSSM_EINVAL, RSSM_ESTATE, RSSM_ECUDA, RSSM_EDEVICE = range(5)
RSSM_MAMBA2, RSSM_GDN, RSSM_KDA = 0, 1, 2
RSSM_REPLAY, RSSM_EAGER = 0, 1
RSSM_F32, RSSM_BF16, RSSM_FP8E4M3 = 0, 1, 2
RSSM_GDN_FP32 = 256
RSSM_DEV_BAD_ACCEPT, RSSM_DEV_BAD_COUNTERS, RSSM_DEV_PIPE_TIMEOUT = 1, 2, 3
RSSM_DEV_BAD_LENGTHS, RSSM_DEV_NO_PAGES, RSSM_DEV_BAD_PAGE = 4, 5, 6
DTYPES = {"f32": RSSM_F32, "bf16": RSSM_BF16, "fp8": RSSM_FP8E4M3}
KINDS = {"mamba2": RSSM_MAMBA2, "gdn": RSSM_GDN, "kda": RSSM_KDA}
MODES = {"replay": RSSM_REPLAY, "eager": RSSM_EAGER}


class rssm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "kind", "mode", "state_dtype", "input_dtype", "batch", "nheads", "headdim", "dstate",
        "ngroups", "window", "max_draft", "dt_scales_input")]


class rssm_workspace_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "error_off", "seq_pos_off", "ckpt_pos_off", "pending_off", "flush_count_off", "arrive_off",
        "A_off", "D_off", "ckpt_off", "ckpt_bytes", "rc_off", "rc_bytes", "rc_scale_off",
        "rc_scale_bytes", "ring", "ring_stride", "xbuf_off", "xbuf_bytes", "bbuf_off", "bbuf_bytes", "sbuf_off",
        "sbuf_bytes", "tbuf_off", "tbuf_bytes", "snap_off", "snap_bytes", "tq_max", "seqinfo_off",
        "seqinfo_bytes", "dec_off", "dec_bytes", "coef_off", "coef_bytes", "query_off", "query_bytes",
        "total_bytes")]


class rssm_inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "dt", "Bm", "Cm", "q", "k", "v", "alpha", "beta")]


class rssm_prefill_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "nheads", "headdim", "dstate", "ngroups", "T", "dt_scales_input")]


class rssm_gdn_prefill_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "nheads", "headdim", "dstate", "input_dtype", "tokens")]


class rssm_tables_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "page_size", "max_pages", "num_free", "max_tokens")]


class rssm_kv4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_kv_heads", "head_dim", "page_size", "num_pages")] + \
               [(n, ctypes.c_float) for n in ("k_scale", "v_scale")]


class rssm_attend_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_q_heads", "tokens", "max_pages", "max_q", "max_seq")] + \
               [("sm_scale", ctypes.c_float)]


# C declarations: name -> (restype, argtypes)
_VP, _I32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_CFGP, _LAYP, _INP = ctypes.POINTER(rssm_config), ctypes.POINTER(rssm_workspace_layout), ctypes.POINTER(rssm_inputs)
_PCFGP = ctypes.POINTER(rssm_prefill_config)
_GCFGP, _TCFGP = ctypes.POINTER(rssm_gdn_prefill_config), ctypes.POINTER(rssm_tables_config)
_KCFGP, _ACFGP = ctypes.POINTER(rssm_kv4_config), ctypes.POINTER(rssm_attend_config)
SIGNATURES = {
    "rssm_workspace_bytes": (_SZ, [_CFGP]),
    "rssm_workspace_layout_of": (ctypes.c_int, [_CFGP, _LAYP]),
    "rssm_create": (ctypes.c_int, [_CFGP, _VP, _SZ, _VP, ctypes.POINTER(_VP)]),
    "rssm_destroy": (ctypes.c_int, [_VP]),
    "rssm_set_stream": (ctypes.c_int, [_VP, _VP]),
    "rssm_set_params": (ctypes.c_int, [_VP, _VP, _VP]),
    "rssm_import_state": (ctypes.c_int, [_VP, _VP]),
    "rssm_export_state": (ctypes.c_int, [_VP, _VP]),
    "rssm_decode": (ctypes.c_int, [_VP, _INP, _VP]),
    "rssm_decode_static_scratch": (ctypes.c_int, [_VP, _INP, _VP]),
    "rssm_verify": (ctypes.c_int, [_VP, _I32, _INP, _VP]),
    "rssm_commit": (ctypes.c_int, [_VP, _VP]),
    "rssm_flush": (ctypes.c_int, [_VP]),
    "rssm_read_counters": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP]),
    "rssm_status_word": (ctypes.c_int, [_VP, _VP]),
    "rssm_clear_status": (ctypes.c_int, [_VP]),
    "rssm_set_split_event": (ctypes.c_int, [_VP, _VP]),
    "rssm_launch_count": (ctypes.c_int64, [_VP]),
    "rssm_last_error": (ctypes.c_char_p, [_VP]),
    "rssm_mamba2_prefill": (ctypes.c_int, [_PCFGP, _VP, _VP, _VP, _INP, _VP, _VP, _VP, _VP]),
    "rssm_gdn_prefill_workspace_bytes": (_SZ, [_GCFGP]),
    "rssm_gdn_prefill": (ctypes.c_int, [_GCFGP, _VP, _INP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "rssm_build_tables": (ctypes.c_int, [_TCFGP] + [_VP] * 12),
    "rssm_kv4_cache_bytes": (_SZ, [_KCFGP]),
    "rssm_kv4_append": (ctypes.c_int, [_KCFGP, _I32] + [_VP] * 6),
    "rssm_kv4_export": (ctypes.c_int, [_KCFGP, _I32] + [_VP] * 6),
    "rssm_kv4_attend_workspace_bytes": (_SZ, [_KCFGP, _ACFGP]),
    "rssm_kv4_attend": (ctypes.c_int, [_KCFGP, _ACFGP] + [_VP] * 7 + [_SZ, _VP, _VP]),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load librssm.so (built by checkpoint_input_replay_rssm_b200.build); no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"librssm.so not found at {path}: build it with "
                               "`python -m checkpoint_input_replay_rssm_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


class RssmError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"rssm status {status}: {msg}")
        self.status = status


def _check(st: int, h=None):
    if st != RSSM_OK:
        msg = load().rssm_last_error(h)
        raise RssmError(st, msg.decode() if msg else "")


def make_config(kind="mamba2", mode="replay", state_dtype="bf16", input_dtype="bf16", batch=1,
                nheads=1, headdim=64, dstate=128, ngroups=1, window=16, max_draft=1,
                dt_scales_input=False) -> rssm_config:
    return rssm_config(KINDS[kind], MODES[mode], DTYPES[state_dtype], DTYPES[input_dtype], batch,
                       nheads, headdim, dstate, ngroups if kind == "mamba2" else nheads, window,
                       max_draft, int(bool(dt_scales_input)))


# ---------------------------------------------------------------- C names
def rssm_workspace_bytes(cfg: rssm_config) -> int:
    return int(load().rssm_workspace_bytes(ctypes.byref(cfg)))


def rssm_workspace_layout_of(cfg: rssm_config) -> rssm_workspace_layout:
    lay = rssm_workspace_layout()
    _check(load().rssm_workspace_layout_of(ctypes.byref(cfg), ctypes.byref(lay)))
    return lay


def rssm_create(cfg: rssm_config, workspace_ptr: int, nbytes: int, stream_ptr: int):
    h = _VP()
    _check(load().rssm_create(ctypes.byref(cfg), workspace_ptr, nbytes, stream_ptr, ctypes.byref(h)))
    return h


def rssm_destroy(h):
    _check(load().rssm_destroy(h))


def rssm_set_stream(h, stream_ptr: int):
    _check(load().rssm_set_stream(h, stream_ptr), h)


def rssm_set_params(h, A_ptr: int, D_ptr: int):
    _check(load().rssm_set_params(h, A_ptr, D_ptr), h)


def rssm_import_state(h, S_ptr: int):
    _check(load().rssm_import_state(h, S_ptr), h)


def rssm_export_state(h, S_ptr: int):
    _check(load().rssm_export_state(h, S_ptr), h)


def rssm_decode(h, inputs: rssm_inputs, y_ptr: int):
    _check(load().rssm_decode(h, ctypes.byref(inputs), y_ptr), h)


def rssm_decode_static_scratch(h, inputs: rssm_inputs, y_ptr: int):
    _check(load().rssm_decode_static_scratch(h, ctypes.byref(inputs), y_ptr), h)


def rssm_verify(h, K: int, inputs: rssm_inputs, y_ptr: int):
    _check(load().rssm_verify(h, K, ctypes.byref(inputs), y_ptr), h)


def rssm_commit(h, accept_ptr: int):
    _check(load().rssm_commit(h, accept_ptr), h)


def rssm_flush(h):
    _check(load().rssm_flush(h), h)


def rssm_read_counters(h, seq_pos, ckpt_pos, pending, flush_count):
    """Host numpy arrays (int64, int64, int32, int32) of length batch, filled in place."""
    p = lambda a: None if a is None else a.ctypes.data_as(_VP)
    _check(load().rssm_read_counters(h, p(seq_pos), p(ckpt_pos), p(pending), p(flush_count)), h)


def rssm_status_word(h):
    """Returns (status, [code, sequence, head, value])."""
    info = (ctypes.c_int32 * 4)()
    st = load().rssm_status_word(h, ctypes.cast(info, _VP))
    return st, list(info)


def rssm_clear_status(h):
    _check(load().rssm_clear_status(h), h)


def rssm_set_split_event(h, event_ptr):
    _check(load().rssm_set_split_event(h, event_ptr), h)


def rssm_launch_count(h) -> int:
    return int(load().rssm_launch_count(h))


def rssm_last_error(h=None) -> str:
    m = load().rssm_last_error(h)
    return m.decode() if m else ""


def rssm_mamba2_prefill(cfg: rssm_prefill_config, A_ptr: int, D_ptr: int, S0_ptr, inputs: rssm_inputs,
                        y_ptr: int, S_out_ptr: int, err_ptr, stream_ptr):
    st = load().rssm_mamba2_prefill(ctypes.byref(cfg), A_ptr, D_ptr, S0_ptr, ctypes.byref(inputs), y_ptr,
                                    S_out_ptr, err_ptr, stream_ptr)
    if st != RSSM_OK:
        raise RssmError(st, "rssm_mamba2_prefill refused its arguments" if st == RSSM_EINVAL
                        else "rssm_mamba2_prefill launch failed")


def prefill(x, dt, Bm, Cm, A, D, S0=None, dt_scales_input=False, y=None, S_out=None, err=None, stream=None):
    """Torch convenience over rssm_mamba2_prefill: x [B,T,H,P] bf16, dt [B,T,H] fp32,
    Bm/Cm [B,T,G,N] bf16, A/D [H] fp32, S0 [B,H,P,N] fp32 or None.  Returns (y, S_out)."""
    import torch

    Bn, T, H, P = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    for t, dty in ((x, torch.bfloat16), (Bm, torch.bfloat16), (Cm, torch.bfloat16), (dt, torch.float32),
                   (A, torch.float32), (D, torch.float32)):
        assert t.is_cuda and t.is_contiguous() and t.dtype == dty
    y = y if y is not None else torch.empty((Bn, T, H, P), dtype=torch.float32, device=x.device)
    S_out = S_out if S_out is not None else torch.empty((Bn, H, P, N), dtype=torch.float32, device=x.device)
    cfg = rssm_prefill_config(Bn, H, P, N, G, T, int(bool(dt_scales_input)))
    ins = rssm_inputs(x=x.data_ptr(), dt=dt.data_ptr(), Bm=Bm.data_ptr(), Cm=Cm.data_ptr())
    st = stream if stream is not None else torch.cuda.current_stream(x.device)
    rssm_mamba2_prefill(cfg, A.data_ptr(), D.data_ptr(), None if S0 is None else S0.data_ptr(), ins,
                        y.data_ptr(), S_out.data_ptr(), None if err is None else err.data_ptr(), st.cuda_stream)
    return y, S_out


# ---------------------------------------------------------------- packed requests
# These calls are a few microseconds of GPU work where they serve single tokens, so what surrounds a launch is kept short.
class _OnStream:
    """The tensors' device is current inside; with a stream given, what is allocated inside belongs to it and the
    tensors used there are not handed out again before it is done with them."""

    def __init__(self, idx, stream, tensors):
        import torch

        if stream is not None and stream.device_index != idx:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{idx}")
        self.ctx = [torch.cuda.device(idx)] + ([torch.cuda.stream(stream)] if stream is not None else [])
        if stream is not None and stream != torch.cuda.current_stream(idx):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *a):
        for c in reversed(self.ctx):
            c.__exit__(*a)


def _run(call, idx, stream, tensors):
    """call(stream pointer) on the tensors' device, on ``stream`` or the device's current one."""
    import torch

    if stream is None and torch._C._cuda_getDevice() == idx:
        return call(torch._C._cuda_getCurrentRawStream(idx))
    with _OnStream(idx, stream, tensors):
        return call(torch._C._cuda_getCurrentRawStream(idx))


def _want(name, t, dtype, shape, idx):
    """Pointer of a dense CUDA tensor of the given dtype, shape and device index."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != idx or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{idx}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _opt(name, t, dtype, shape, idx):
    return None if t is None else _want(name, t, dtype, shape, idx)


def _workspace(t, need, idx, like):
    """(tensor, pointer, bytes) of the caller's workspace or of a new one."""
    import torch

    if t is None:
        if not need:
            return None, None, 0
        t = like.new_empty(need, dtype=torch.uint8)
    return t, _want("workspace", t, torch.uint8, (t.numel(),), idx), t.numel()


def _cuda_index(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return t.get_device()


def _int(name, v):
    """A size that reaches the library as int32, where a larger one would wrap."""
    if not 0 <= v <= 0x7fffffff:
        raise ValueError(f"{name}: expected a size below 2^31, got {v}")
    return v


def _ok(st, what):
    if st != RSSM_OK:
        raise RssmError(st, f"{what} refused its arguments" if st == RSSM_EINVAL else f"{what}: launch failed")


def gdn_prefill(q, k, v, alpha, beta, cu_seqlens, S0=None, y=None, S_out=None, workspace=None, err=None,
                stream=None, fp32=False):
    """Torch convenience over rssm_gdn_prefill: the gated delta rule over packed prompts.

    q, k [tokens, H, N], v [tokens, H, P] bf16 or fp32; alpha, beta [tokens, H] fp32; cu_seqlens
    [B + 1] int32 row offsets of the prompts; S0 [B, H, P, N] fp32 or None (zero).  Returns
    (y [tokens, H, P] fp32, S_out [B, H, P, N] fp32); S_out goes to ``Layer.import_state`` of a GDN
    layer.  ``err`` (int32 [4], zeroed by the caller) receives device-side inconsistencies.  Results are within
    6e-6 (2-norm) for bf16 prompts of more than 12 tokens with N = 128, which are served in chunks, and 1e-7 otherwise;
    ``fp32=True`` has all of them served by the fp32 recurrence, at a third of a microsecond a token.
    """
    import torch

    dev = _cuda_index(q, "q")
    if q.dim() != 3 or v.dim() != 3 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("expected q, k, v of shape [tokens, heads, dim] and cu_seqlens of [requests + 1]")
    T, H, N = q.shape
    P, Bn, dt, f32, i32 = v.shape[2], cu_seqlens.shape[0] - 1, q.dtype, torch.float32, torch.int32
    if dt is not torch.bfloat16 and dt is not f32:
        raise ValueError(f"q: expected bfloat16 or float32, got {dt}")

    def call(st):
        nonlocal y, S_out
        y = q.new_empty((T, H, P), dtype=f32) if y is None else y
        S_out = q.new_empty((Bn, H, P, N), dtype=f32) if S_out is None else S_out
        lib = load()
        kind = (RSSM_BF16 if dt is torch.bfloat16 else RSSM_F32) + (RSSM_GDN_FP32 if fp32 else 0)
        cfg = ctypes.byref(rssm_gdn_prefill_config(Bn, H, P, N, kind, T))
        _, ws, nb = _workspace(workspace, lib.rssm_gdn_prefill_workspace_bytes(cfg), dev, q)
        ins = rssm_inputs(q=_want("q", q, dt, (T, H, N), dev), k=_want("k", k, dt, (T, H, N), dev),
                          v=_want("v", v, dt, (T, H, P), dev), alpha=_want("alpha", alpha, f32, (T, H), dev),
                          beta=_want("beta", beta, f32, (T, H), dev))
        return lib.rssm_gdn_prefill(
            cfg, _opt("S0", S0, f32, (Bn, H, P, N), dev), ctypes.byref(ins),
            _want("cu_seqlens", cu_seqlens, i32, (Bn + 1,), dev), _want("y", y, f32, (T, H, P), dev),
            _want("S_out", S_out, f32, (Bn, H, P, N), dev), ws, nb, _opt("err", err, i32, (4,), dev), st)

    _ok(_run(call, dev, stream, (q, k, v, alpha, beta, cu_seqlens, S0, y, S_out, workspace, err)), "rssm_gdn_prefill")
    return y, S_out


def build_tables(cached_len, new_len, free_pages, free_head, block_table, page_size, max_tokens, err=None,
                 stream=None):
    """Torch convenience over rssm_build_tables (all int32): block_table [B, max_pages] is updated in
    place with pages of free_pages from entry free_head [1] on; returns (cu_new [B + 1], seq_len [B],
    slot_map [max_tokens], position [max_tokens], next_free [1])."""
    import torch

    dev, i32 = _cuda_index(cached_len, "cached_len"), torch.int32
    if cached_len.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("expected cached_len [requests], block_table [requests, pages] and free_pages [pages]")
    Bn, width = block_table.shape
    if max_tokens < 1 or max_tokens > 2 ** 30:
        raise ValueError(f"max_tokens: expected 1 to 2^30, got {max_tokens}")
    sizes, out = (Bn + 1, Bn, max_tokens, max_tokens, 1), None

    def call(st):
        nonlocal out
        out = cached_len.new_empty(2 * Bn + 2 * max_tokens + 2, dtype=i32).split_with_sizes(sizes)  # one allocation
        base = out[0].data_ptr()
        cfg = rssm_tables_config(Bn, _int("page_size", page_size), width, _int("free_pages", free_pages.shape[0]), max_tokens)
        return load().rssm_build_tables(
            ctypes.byref(cfg), _want("cached_len", cached_len, i32, (Bn,), dev), _want("new_len", new_len, i32, (Bn,), dev),
            _want("free_pages", free_pages, i32, (free_pages.shape[0],), dev), _want("free_head", free_head, i32, (1,), dev),
            _want("block_table", block_table, i32, (Bn, width), dev), base, base + 4 * (Bn + 1), base + 4 * (2 * Bn + 1),
            base + 4 * (2 * Bn + 1 + max_tokens), base + 4 * (2 * Bn + 1 + 2 * max_tokens), _opt("err", err, i32, (4,), dev), st)

    _ok(_run(call, dev, stream, (cached_len, new_len, free_pages, free_head, block_table, err)), "rssm_build_tables")
    return out


def kv4_cache(num_pages, n_kv_heads, page_size, head_dim, device="cuda"):
    """A zeroed paged 4-bit key/value cache: uint8 [num_pages, n_kv_heads, page_size * head_dim * 9 / 8]."""
    import torch

    cfg = rssm_kv4_config(n_kv_heads, head_dim, page_size, num_pages, 1.0, 1.0)
    if not load().rssm_kv4_cache_bytes(ctypes.byref(cfg)):
        raise RssmError(RSSM_EINVAL, "no 4-bit cache of these sizes: head_dim is 64 or 128, page_size a multiple of "
                                     "16 up to 256, num_pages * page_size < 2^31")
    return torch.zeros((num_pages, n_kv_heads, page_size * head_dim * 9 // 8), dtype=torch.uint8, device=device)


def _kv4_config(cache, head_dim, k_scale, v_scale, idx):
    """(config, pointer) of a cache on the given device."""
    import torch

    if cache.dtype is not torch.uint8 or cache.dim() != 3 or cache.get_device() != idx or not cache.is_contiguous():
        raise ValueError(f"cache: expected a contiguous uint8 tensor [pages, kv heads, page bytes] on cuda:{idx}")
    pages, heads, nb = cache.shape
    if head_dim < 1:
        raise ValueError(f"head_dim: expected 64 or 128, got {head_dim}")
    ps = nb * 8 // (9 * head_dim)
    if ps * 9 * head_dim != nb * 8:
        raise ValueError(f"cache: {nb} bytes a page and head are no whole number of tokens of {head_dim} channels")
    return rssm_kv4_config(heads, head_dim, ps, pages, k_scale, v_scale), cache.data_ptr()


def kv4_append(k, v, slot_map, cache, k_scale=1.0, v_scale=1.0, err=None, stream=None):
    """Torch convenience over rssm_kv4_append: write k, v [tokens, kv heads, head_dim] bf16 to the
    slots slot_map [tokens] int32 (negative: skipped) of ``cache`` (``kv4_cache``), in place."""
    import torch

    if k.dim() != 3 or cache.dim() != 3:
        raise ValueError("expected k of shape [tokens, kv heads, head_dim] and cache of [pages, kv heads, bytes]")
    dev, (T, _, D), bf = _cuda_index(k, "k"), k.shape, torch.bfloat16
    cfg, held = _kv4_config(cache, D, k_scale, v_scale, dev)
    sh = (T, cache.shape[1], D)

    def call(st):
        return load().rssm_kv4_append(
            ctypes.byref(cfg), T, _want("k", k, bf, sh, dev), _want("v", v, bf, sh, dev),
            _want("slot_map", slot_map, torch.int32, (T,), dev), held,
            _opt("err", err, torch.int32, (4,), dev), st)

    _ok(_run(call, dev, stream, (k, v, slot_map, cache, err)), "rssm_kv4_append")


def kv4_export(slot_map, cache, head_dim, k_scale=1.0, v_scale=1.0, k=None, v=None, err=None, stream=None):
    """Torch convenience over rssm_kv4_export: the values held at slot_map [tokens] as bf16
    (k, v) [tokens, kv heads, head_dim]."""
    import torch

    dev, bf = _cuda_index(slot_map, "slot_map"), torch.bfloat16
    if cache.dim() != 3 or slot_map.dim() != 1:
        raise ValueError("expected slot_map of shape [tokens] and cache of [pages, kv heads, bytes]")
    cfg, held = _kv4_config(cache, head_dim, k_scale, v_scale, dev)
    T = slot_map.shape[0]
    sh = (T, cache.shape[1], head_dim)

    def call(st):
        nonlocal k, v
        k = cache.new_empty(sh, dtype=bf) if k is None else k
        v = cache.new_empty(sh, dtype=bf) if v is None else v
        return load().rssm_kv4_export(
            ctypes.byref(cfg), T, _want("slot_map", slot_map, torch.int32, (T,), dev),
            held, _want("k", k, bf, sh, dev),
            _want("v", v, bf, sh, dev), _opt("err", err, torch.int32, (4,), dev), st)

    _ok(_run(call, dev, stream, (slot_map, cache, k, v, err)), "rssm_kv4_export")
    return k, v


def kv4_attend(q, cache, block_table, seq_len, cu_q, max_q, k_scale=1.0, v_scale=1.0, sm_scale=None, max_seq=None,
               out=None, workspace=None, err=None, stream=None):
    """Torch convenience over rssm_kv4_attend: causal attention of q [tokens, query heads, head_dim]
    bf16 over the cached tokens of each request (its own appended first), the requests packed by
    cu_q [B + 1] int32 with at most max_q rows each, seq_len [B] int32 cached tokens found through
    block_table [B, max_pages] int32.  sm_scale defaults to head_dim ** -0.5, max_seq (a bound of
    seq_len that sizes the launch) to max_pages * page_size.  Returns out [tokens, query heads,
    head_dim] bf16."""
    import torch

    if q.dim() != 3 or cache.dim() != 3 or block_table.dim() != 2 or seq_len.dim() != 1:
        raise ValueError("expected q [tokens, heads, head_dim], cache [pages, kv heads, bytes], block_table "
                         "[requests, pages] and seq_len [requests]")
    dev, (T, Hq, D), bf, i32 = _cuda_index(q, "q"), q.shape, torch.bfloat16, torch.int32
    cfg, held = _kv4_config(cache, D, k_scale, v_scale, dev)
    Bn, width = block_table.shape

    def call(st):
        nonlocal out
        out = q.new_empty((T, Hq, D), dtype=bf) if out is None else out
        lib, kv = load(), ctypes.byref(cfg)
        att = ctypes.byref(rssm_attend_config(Bn, Hq, T, width, _int("max_q", max_q),
                                              _int("max_seq", width * cfg.page_size if max_seq is None else max_seq),
                                              D ** -0.5 if sm_scale is None else sm_scale))
        _, ws, nb = _workspace(workspace, lib.rssm_kv4_attend_workspace_bytes(kv, att), dev, q)
        return lib.rssm_kv4_attend(
            kv, att, _want("q", q, bf, (T, Hq, D), dev), held,
            _want("block_table", block_table, i32, (Bn, width), dev), _want("seq_len", seq_len, i32, (Bn,), dev),
            _want("cu_q", cu_q, i32, (Bn + 1,), dev), _want("out", out, bf, (T, Hq, D), dev), ws, nb,
            _opt("err", err, i32, (4,), dev), st)

    _ok(_run(call, dev, stream, (q, cache, block_table, seq_len, cu_q, out, workspace, err)), "rssm_kv4_attend")
    return out


# ---------------------------------------------------------------- torch owner
class Layer:
    """One SSM layer's decode state on the current CUDA device.

    The workspace is a torch uint8 CUDA tensor owned here; inputs are torch CUDA
    tensors in the configured dtypes (x/B/C or q/k/v in ``input_dtype``; dt,
    alpha, beta fp32), laid out [B, T, ...] as include/rssm.h states.
    """

    def __init__(self, cfg: rssm_config, device=None, stream=None):
        import torch

        if not torch.cuda.is_available():
            raise RuntimeError("librssm needs a CUDA device; none is visible")
        self.torch = torch
        self.cfg = cfg
        self.device = torch.device(device or "cuda")
        self.layout = rssm_workspace_layout_of(cfg)
        self.nbytes = int(self.layout.total_bytes)
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
            self.stream = stream or torch.cuda.current_stream(self.device)
            self.h = rssm_create(cfg, self.workspace.data_ptr(), self.nbytes, self.stream.cuda_stream)
        self.B, self.H, self.P, self.N = cfg.batch, cfg.nheads, cfg.headdim, cfg.dstate
        self.T_last = 0

    def close(self):
        if getattr(self, "h", None):
            rssm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- marshalling helpers
    def _ptr(self, t, dtype=None):
        if t is None:
            return None
        assert t.is_cuda and t.is_contiguous(), "inputs must be contiguous CUDA tensors"
        if dtype is not None:
            assert t.dtype == dtype, f"expected {dtype}, got {t.dtype}"
        return t.data_ptr()

    def _inputs(self, d: dict) -> rssm_inputs:
        torch = self.torch
        wide = torch.bfloat16 if self.cfg.input_dtype == RSSM_BF16 else torch.float32
        f32 = torch.float32
        spec = {"x": wide, "dt": f32, "B": wide, "C": wide, "q": wide, "k": wide, "v": wide,
                "alpha": f32, "beta": f32}
        cname = {"B": "Bm", "C": "Cm"}
        kw = {cname.get(k, k): self._ptr(v, spec[k]) for k, v in d.items()}
        return rssm_inputs(**kw)

    def set_params(self, A, D):
        rssm_set_params(self.h, self._ptr(A, self.torch.float32), self._ptr(D, self.torch.float32))

    def import_state(self, S):
        rssm_import_state(self.h, self._ptr(S, self.torch.float32))

    def export_state(self, out=None):
        out = out if out is not None else self.torch.empty((self.B, self.H, self.P, self.N),
                                                           dtype=self.torch.float32, device=self.device)
        rssm_export_state(self.h, self._ptr(out))
        return out

    def decode(self, inputs: dict, y=None):
        y = y if y is not None else self.torch.empty((self.B, 1, self.H, self.P),
                                                     dtype=self.torch.float32, device=self.device)
        rssm_decode(self.h, self._inputs(inputs), self._ptr(y))
        return y

    def decode_static_scratch(self, inputs: dict, y=None):
        y = y if y is not None else self.torch.empty((self.B, 1, self.H, self.P),
                                                     dtype=self.torch.float32, device=self.device)
        rssm_decode_static_scratch(self.h, self._inputs(inputs), self._ptr(y))
        return y

    def verify(self, K: int, inputs: dict, y=None):
        y = y if y is not None else self.torch.empty((self.B, K, self.H, self.P),
                                                     dtype=self.torch.float32, device=self.device)
        rssm_verify(self.h, K, self._inputs(inputs), self._ptr(y))
        return y

    def commit(self, accept_len):
        rssm_commit(self.h, self._ptr(accept_len, self.torch.int32))

    def flush(self):
        rssm_flush(self.h)

    def counters(self):
        import numpy as np

        sp = np.zeros(self.B, np.int64)
        ck = np.zeros(self.B, np.int64)
        pe = np.zeros(self.B, np.int32)
        fc = np.zeros(self.B, np.int32)
        rssm_read_counters(self.h, sp, ck, pe, fc)
        return sp, ck, pe, fc

    def status(self):
        return rssm_status_word(self.h)

    def clear_status(self):
        rssm_clear_status(self.h)

    def launches(self) -> int:
        return rssm_launch_count(self.h)

    def region(self, off_name: str, bytes_name: str, dtype):
        """A torch view of one workspace region (for inspection in tests)."""
        off = getattr(self.layout, off_name)
        n = getattr(self.layout, bytes_name)
        return self.workspace[off:off + n].view(dtype)
