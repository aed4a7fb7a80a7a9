"""A synthetic hybrid decode step: where the SSM-layer saving lands in a step.

The hybrid models the ReplaySSM reports measure interleave about five SSM
layers per attention layer (blog.thibaultmonteiro.fr, "La fiche qu'on reecrit a
chaque token"), and the reports quote the whole decode step next to the SSM
kernel alone (irisproject.cloud, "Des chiffres").  This stand-in builds such a
stack with random weights (there is no trained model here): each block is
``ssm_per_block`` Mamba-2 layers decoded by librssm (replay or the eager
baseline) and one attention layer.  Every layer projects the hidden state in
and out with plain bf16 GEMMs (torch.matmul) after an RMS normalisation of its
input (pre-norm residual blocks, as in the hybrid models); the attention layer
appends the token's key and value to a bf16 cache and attends over it with
torch.nn.functional.scaled_dot_product_attention (grouped-query: the query heads
of a key/value head stacked as its query rows; flash or memory-efficient kernel), or, with
``kv_cache="fp4"``, keeps and reads its keys and values in the library's paged 4-bit cache
(rssm_build_tables once a step, rssm_kv4_append and rssm_kv4_attend per layer).  The Mamba-2
layer's short convolution and output gate are left out: they carry no decode
state that the method changes.

Only the SSM layers' state handling differs between the two modes, so the step
time difference is the SSM saving as it shows in a step.  Nothing here is on
the SSM decode path itself, which runs entirely in librssm's kernels.
"""
from __future__ import annotations

import dataclasses


@dataclasses.dataclass(frozen=True)
class HybridShape:
    batch: int = 256
    blocks: int = 1
    ssm_per_block: int = 5
    d_model: int = 4096
    nheads: int = 128     # Mamba-2 heads
    headdim: int = 64
    dstate: int = 128
    ngroups: int = 8
    window: int = 16
    n_q_heads: int = 32   # attention
    n_kv_heads: int = 2
    head_dim: int = 128
    context: int = 4096   # cached tokens per sequence before the first step

    @property
    def ssm_in(self) -> int:  # x, dt, B, C
        return self.nheads * self.headdim + self.nheads + 2 * self.ngroups * self.dstate


class HybridStack:
    """``blocks`` x (``ssm_per_block`` Mamba-2 layers + 1 attention layer) on one GPU.

    ssm_mode: "replay" (checkpoint + read copy ``read_dtype`` + buffer) or "eager"
    (fp32 state rewritten every token).  kv_cache: "bf16" (a dense cache, torch attention)
    or "fp4" (the paged 4-bit cache and its attention, pages of ``page_size`` tokens; what the device
    refuses there raises ``rssm.RssmError`` from ``check_cache``, or from a later ``step``).
    Weights, initial states and the cached keys/values come from a seeded torch generator.
    """

    KV_SCALE = 2.0 ** -4  # tensor scale of the 4-bit cache: block maxima around 1 lie mid-range of its e4m3 scales

    def __init__(self, shape: HybridShape, ssm_mode: str = "replay", read_dtype: str = "bf16", seed: int = 0,
                 device="cuda", max_steps: int = 512, kv_cache: str = "bf16", page_size: int = 64):
        import torch

        from . import rssm

        if kv_cache not in ("bf16", "fp4"):
            raise ValueError(f"kv_cache must be 'bf16' or 'fp4', got {kv_cache!r}")
        self.rssm, self.kv_cache, self.page_size = rssm, kv_cache, page_size
        self.s = s = shape
        self.torch = torch
        self.device = torch.device(device)
        g = torch.Generator(device=self.device).manual_seed(seed)
        bf = torch.bfloat16
        rnd = lambda *sh, scale: (torch.randn(sh, generator=g, device=self.device) * scale)
        self.layers = []
        for _blk in range(s.blocks):
            for _ in range(s.ssm_per_block):
                cfg = rssm.make_config(kind="mamba2", mode=ssm_mode,
                                       state_dtype=read_dtype if ssm_mode == "replay" else "f32",
                                       input_dtype="bf16", batch=s.batch, nheads=s.nheads, headdim=s.headdim,
                                       dstate=s.dstate, ngroups=s.ngroups, window=s.window, max_draft=1)
                L = rssm.Layer(cfg, device=self.device)
                A = -torch.exp(torch.rand(s.nheads, generator=g, device=self.device))
                D = torch.randn(s.nheads, generator=g, device=self.device)
                L.set_params(A.contiguous(), D.contiguous())
                L.import_state(rnd(s.batch, s.nheads, s.headdim, s.dstate, scale=0.1).contiguous())
                self.layers.append(("ssm", {
                    "layer": L,
                    "w_in": rnd(s.d_model, s.ssm_in, scale=s.d_model ** -0.5).to(bf),
                    "dt_bias": torch.full((s.nheads,), -2.0, device=self.device),
                    "w_out": rnd(s.nheads * s.headdim, s.d_model, scale=(s.nheads * s.headdim) ** -0.5).to(bf),
                    "y": torch.empty((s.batch, 1, s.nheads, s.headdim), dtype=torch.float32, device=self.device),
                }))
            qd, kvd = s.n_q_heads * s.head_dim, s.n_kv_heads * s.head_dim
            cap = s.context + max_steps
            self.layers.append(("attn", {
                "wq": rnd(s.d_model, qd, scale=s.d_model ** -0.5).to(bf),
                "wk": rnd(s.d_model, kvd, scale=s.d_model ** -0.5).to(bf),
                "wv": rnd(s.d_model, kvd, scale=s.d_model ** -0.5).to(bf),
                "wo": rnd(qd, s.d_model, scale=qd ** -0.5).to(bf),
                "k": rnd(s.batch, s.n_kv_heads, cap, s.head_dim, scale=1.0).to(bf),
                "v": rnd(s.batch, s.n_kv_heads, cap, s.head_dim, scale=1.0).to(bf),
            }))
        # torch's SDPA is held to its flash and memory-efficient kernels: its
        # default dispatch may pick a backend that builds an execution plan per
        # new sequence length, which a decode meets every step (tens of
        # milliseconds of host time per new length).
        from torch.nn.attention import SDPBackend, sdpa_kernel

        if kv_cache == "fp4":
            self._to_fp4(max_steps)

        self._sdpa_backends = lambda: sdpa_kernel([SDPBackend.FLASH_ATTENTION, SDPBackend.EFFICIENT_ATTENTION])
        self.pos = s.context  # next cache position
        self.cap = s.context + max_steps
        self.ssm_events = None  # a list here records CUDA events around every SSM decode call

    def _to_fp4(self, max_steps):
        """Move every attention layer's cached tokens into a paged 4-bit cache; the layers share one block table."""
        torch, s, rssm, ps = self.torch, self.s, self.rssm, self.page_size
        i32 = dict(dtype=torch.int32, device=self.device)
        width = -(-(s.context + max_steps) // ps)
        self.block_table = torch.full((s.batch, width), -1, **i32)
        self.free_pages = torch.arange(s.batch * width, **i32)
        self.free_head, self.cached_len = torch.zeros(1, **i32), torch.zeros(s.batch, **i32)
        self.one_new = torch.ones(s.batch, **i32)
        self.kv_err = torch.zeros(4, **i32)
        self.kv_seen = torch.zeros(4, dtype=torch.int32, pin_memory=True)  # kv_err after some step
        self.kv_event = torch.cuda.Event()
        slots = None
        if s.context:
            slots = self._tables(torch.full((s.batch,), s.context, **i32), s.batch * s.context)[2]
            self._advance()
        for kind, p in self.layers:
            if kind == "attn":
                k, v = (p.pop(n)[:, :, :s.context].transpose(1, 2).reshape(-1, s.n_kv_heads, s.head_dim) for n in "kv")
                p["cache"] = rssm.kv4_cache(s.batch * width, s.n_kv_heads, ps, s.head_dim, device=self.device)
                if slots is not None:
                    rssm.kv4_append(k, v, slots, p["cache"], k_scale=self.KV_SCALE, v_scale=self.KV_SCALE, err=self.kv_err)
        self.check_cache()

    def check_cache(self):
        """Wait for the steps so far and raise where one of the 4-bit cache's operators was refused on the device."""
        if self.kv_cache == "fp4":
            self._raise_if(self.kv_err)

    def _raise_if(self, err):
        code, b, h, value = err.tolist()
        if code:
            raise self.rssm.RssmError(self.rssm.RSSM_EDEVICE, f"4-bit attention cache: device error {code}, request {b}, "
                                                              f"head {h}, value {value}")

    def _watch(self):
        """The error word as far as it has come to the host, without waiting: a refused step does not pass for long."""
        if self.kv_event.query():
            self._raise_if(self.kv_seen)
            self.kv_seen.copy_(self.kv_err, non_blocking=True)
            self.kv_event.record()

    def _tables(self, new_len, max_tokens):
        self.tables = self.rssm.build_tables(self.cached_len, new_len, self.free_pages, self.free_head, self.block_table,
                                             self.page_size, max_tokens, err=self.kv_err)
        return self.tables

    def _advance(self):
        self.cached_len, self.free_head = self.tables[1], self.tables[4]

    def _norm(self, x):
        xf = x.float()
        return (xf * self.torch.rsqrt(xf.pow(2).mean(dim=-1, keepdim=True) + 1e-6)).to(self.torch.bfloat16)

    def _ssm(self, x, p):
        torch, s = self.torch, self.s
        u = self._norm(x) @ p["w_in"]
        HP, H, GN = s.nheads * s.headdim, s.nheads, s.ngroups * s.dstate
        inputs = {
            "x": u[:, :HP].reshape(s.batch, 1, H, s.headdim).contiguous(),
            "dt": torch.nn.functional.softplus(u[:, HP:HP + H].float() + p["dt_bias"]).reshape(s.batch, 1, H)
                  .contiguous(),
            "B": u[:, HP + H:HP + H + GN].reshape(s.batch, 1, s.ngroups, s.dstate).contiguous(),
            "C": u[:, HP + H + GN:].reshape(s.batch, 1, s.ngroups, s.dstate).contiguous(),
        }
        if self.ssm_events is not None:
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            p["layer"].decode(inputs, y=p["y"])
            e1.record()
            self.ssm_events.append((e0, e1))
        else:
            p["layer"].decode(inputs, y=p["y"])
        return x + p["y"].reshape(s.batch, HP).to(torch.bfloat16) @ p["w_out"]

    def _attn(self, x, p):
        torch, s = self.torch, self.s
        xn = self._norm(x)
        if self.kv_cache == "fp4":
            cu, seq_len, slots, _, _ = self.tables
            heads = lambda w, n: (xn @ w).reshape(s.batch, n, s.head_dim)  # noqa: E731
            sc = dict(k_scale=self.KV_SCALE, v_scale=self.KV_SCALE, err=self.kv_err)
            self.rssm.kv4_append(heads(p["wk"], s.n_kv_heads), heads(p["wv"], s.n_kv_heads), slots, p["cache"], **sc)
            o = self.rssm.kv4_attend(heads(p["wq"], s.n_q_heads), p["cache"], self.block_table, seq_len, cu, 1,
                                     max_seq=self.cap, **sc)
            return x + o.reshape(s.batch, s.n_q_heads * s.head_dim) @ p["wo"]
        # One decode token: the query heads that share a key/value head attend to
        # the same cache, so they are stacked as that head's query rows
        # ([batch, kv heads, query heads per kv head, head_dim]); query head j
        # uses key/value head j // (n_q_heads / n_kv_heads), as in grouped-query
        # attention, and no mask applies.
        q = (xn @ p["wq"]).reshape(s.batch, s.n_kv_heads, s.n_q_heads // s.n_kv_heads, s.head_dim)
        p["k"][:, :, self.pos] = (xn @ p["wk"]).reshape(s.batch, s.n_kv_heads, s.head_dim)
        p["v"][:, :, self.pos] = (xn @ p["wv"]).reshape(s.batch, s.n_kv_heads, s.head_dim)
        n = self.pos + 1
        with self._sdpa_backends():
            o = torch.nn.functional.scaled_dot_product_attention(q, p["k"][:, :, :n], p["v"][:, :, :n])
        return x + o.reshape(s.batch, s.n_q_heads * s.head_dim) @ p["wo"]

    def step(self, x):
        """One decode token for every sequence: hidden state x [batch, d_model] bf16 -> the next."""
        if self.pos >= self.cap:
            raise RuntimeError("the attention cache is full; build the stack with a larger max_steps")
        if self.kv_cache == "fp4":
            if self.torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a step of the stack advances counters on the host, which a replayed graph would not")
            self._watch()
            self._tables(self.one_new, self.s.batch)
        for kind, p in self.layers:
            x = self._ssm(x, p) if kind == "ssm" else self._attn(x, p)
        self.pos += 1
        if self.kv_cache == "fp4":
            self._advance()
        return x

    def ssm_layers(self):
        return [p["layer"] for kind, p in self.layers if kind == "ssm"]
