"""Stacked BitLinear layers through the C ABI.

One layer, as the BitNet pages describe the model around BitLinear: the
linear layers of attention and FFN are BitLinear (int8 activations), and in
BitNet v2 the O and down projections are H-BitLinear (Hadamard + int4).
Per layer, with fp32 residuals:

    q, k, v = BitLinear(x)                      (one int8 quantisation of x,
                                                 one launch for the three)
    o = H-BitLinear(attention(q, k, v))         (rotary embedding, key/value
                                                 cache, causal softmax; without
                                                 a cache, a one-token context,
                                                 which returns V)
    h = x + o
    up, gate = BitLinear(h)                     (one int8 quantisation of h,
                                                 one launch for the two)
    a = relu(gate)^2 * up                       (squared-ReLU gated unit)
    x' = h + H-BitLinear(a)                     (down projection)

Every step is a kernel of libbitnet.so; this module only sequences the calls
and owns the activation buffers (allocated once per batch size).  The
element-wise steps run inside the quantiser that consumes them: h = x + o in
the quantisation of h, a in the Hadamard quantisation of a, and x' = h + d
in the next layer's first quantisation (a final add after the last layer).
"""
from __future__ import annotations

import torch

from . import api

PROJ = ("q", "k", "v", "o", "up", "gate", "down")
H_BITS = {"o": 4, "down": 4}


def quantize_layer(weights: dict, stream=None) -> dict:
    """fp32/bf16 device weights {name: [N, K]} -> {name: (packed, s_w)}."""
    return {name: api.bitnet_quantize_weights(weights[name].contiguous(), stream=stream) for name in PROJ}


class BitLinearChain:
    """Runs a list of quantised layers on a batch of M tokens of width `hidden`.

    attention=None: the attention core over a one-token context (O's input is V).
    attention=dict(B=..., L=..., T_cap=..., heads=...): the M = B*L rows are B
    sequences of L tokens each; every layer keeps a key/value cache
    [B, T_cap, hidden] (allocated here) and runs rotary embedding, the cache
    append and causal softmax attention; forward(x, t0) places the step's
    tokens at positions t0 .. t0+L-1.  More keys of the dict:
      kv_bits    32 (default) or 4: the caches are then held in 4 bits (kv4, one
                 api.KV4Cache a layer) and read by the attention as they are;
      qk_norm    RMSNorm of every query and key head before the rotation, with
                 gamma_q / gamma_k ([d] fp32 a layer, a list) or ones;
      hadamard   (kv_bits 4; default True) Hadamard transform of the query and
                 key heads before the keys are held in 4 bits;
      kv_heads   (kv_bits 4; default heads) key heads, each shared by
                 heads / kv_heads query heads;
      window, sinks  (kv_bits 4) sliding window and first tokens that stay visible;
                 keys behind the window keep their place, positions stay below T_cap."""

    def __init__(self, layers: list, M: int, hidden: int, ffn: int, device, eps: float = 1e-6, attention=None):
        self.layers = layers
        self.M, self.hidden, self.ffn, self.eps = M, hidden, ffn, eps
        self.attention = attention
        if attention is not None:
            B, L, T_cap = attention["B"], attention["L"], attention["T_cap"]
            assert B * L == M and L <= T_cap
            self.heads = attention.get("heads", 16)
            self.rope_base = attention.get("base", 10000.0)
            self.kv_bits = attention.get("kv_bits", 32)
            self.kv_heads = attention.get("kv_heads", self.heads)
            self.qk_norm = attention.get("qk_norm", False)
            self.gamma_q, self.gamma_k = (attention.get(g) or [None] * len(layers) for g in ("gamma_q", "gamma_k"))
            self.hadamard = attention.get("hadamard", True)
            self.window, self.sinks = attention.get("window", 0), attention.get("sinks", 0)
            if self.kv_bits == 4:
                self.kv4 = [api.bitnet_kv4_cache(B, T_cap, self.kv_heads, hidden // self.heads, device) for _ in layers]
                self.att = torch.zeros((M, hidden), dtype=torch.float32, device=device)
            elif self.kv_bits == 32:
                if self.kv_heads != self.heads or self.window or self.sinks:
                    raise ValueError("shared key heads and a sliding window need kv_bits=4")
                self.kc = [torch.empty((B, T_cap, hidden), dtype=torch.float32, device=device) for _ in layers]
                self.vc = [torch.empty((B, T_cap, hidden), dtype=torch.float32, device=device) for _ in layers]
                self.att = torch.empty((M, hidden), dtype=torch.float32, device=device)
            else:
                raise ValueError("kv_bits is 32 or 4")
        self.t0 = 0
        self.pos = self.lens = self.t_max = None
        f32 = dict(dtype=torch.float32, device=device)
        e = lambda *shape: torch.empty(shape, **f32)
        self.x = [e(M, hidden), e(M, hidden)]          # layer input, chain output
        self.xq = torch.empty((M, hidden), dtype=torch.int8, device=device)
        self.sx = e(M)
        self.q, self.o, self.h, self.d = (e(M, hidden) for _ in range(4))
        kv_width = hidden if attention is None else hidden // self.heads * self.kv_heads
        self.k, self.v = e(M, kv_width), e(M, kv_width)
        self.v4 = torch.empty((M, hidden // 2), dtype=torch.uint8, device=device)
        self.sv = e(M)
        self.hq = torch.empty((M, hidden), dtype=torch.int8, device=device)
        self.sh = e(M)
        self.up, self.gate = e(M, ffn), e(M, ffn)
        self.a4 = torch.empty((M, ffn // 2), dtype=torch.uint8, device=device)
        self.sa = e(M)

    def layer(self, x_parts, w: dict, stream=None, index: int = 0):
        """One layer.  x_parts: (x,) or (h_prev, d_prev), whose sum is the
        layer input.  Returns (h, d), whose sum is the layer output.  Buffers
        are reused from layer to layer: every kernel waits for the one before
        it, so a buffer is rewritten only after its last reader has finished."""
        A, s = api, stream
        if len(x_parts) == 1:
            x = x_parts[0]
            A.bitnet_quant_act(x, None, self.eps, Xq=self.xq, s_x=self.sx, stream=s)
        else:
            x = self.x[0]
            A.bitnet_add_quant_act(x_parts[0], x_parts[1], None, self.eps, H=x, Xq=self.xq, s_x=self.sx, stream=s)
        A.bitnet_linear_group(self.xq, 8, self.sx, [w["q"], w["k"], w["v"]], Ys=[self.q, self.k, self.v], stream=s)
        if self.attention is None:
            att = self.v                                   # a one-token context returns V
        else:
            att = self.attend(index, s)
        A.bitnet_hadamard_quant_act(att, None, self.eps, 0, Xq4=self.v4, s_x=self.sv, stream=s)
        A.bitnet_linear(self.v4, 4, self.sv, *w["o"], Y=self.o, stream=s)
        A.bitnet_add_quant_act(x, self.o, None, self.eps, H=self.h, Xq=self.hq, s_x=self.sh, stream=s)
        A.bitnet_linear_group(self.hq, 8, self.sh, [w["up"], w["gate"]], Ys=[self.up, self.gate], stream=s)
        A.bitnet_glu_hadamard_quant_act(self.gate, self.up, None, self.eps, 0, Xq4=self.a4, s_x=self.sa, stream=s)
        A.bitnet_linear(self.a4, 4, self.sa, *w["down"], Y=self.d, stream=s)
        return self.h, self.d

    def attend(self, index: int, stream=None):
        """Rotation (and norm), cache append and attention of layer `index`, from
        the projections in q, k, v."""
        A, s = api, stream
        B, L = self.attention["B"], self.attention["L"]
        norm = dict(gamma_q=self.gamma_q[index], gamma_k=self.gamma_k[index], eps=self.eps, base=self.rope_base)
        if self.kv_bits == 4:
            at = dict(pos=self.pos, lens=self.lens, stream=s)
            A.bitnet_kv4_append(self.q, self.k, self.v, self.kv4[index], B, L, self.t0, self.heads, norm=self.qk_norm,
                                hadamard=self.hadamard, Qo=self.q, **norm, **at)
            return A.bitnet_kv4_attention(self.q, self.kv4[index], B, L, self.t0, self.heads, self.window, self.sinks,
                                          t_max=self.t_max, A=self.att, **at)
        if self.qk_norm:
            A.bitnet_qk_norm_rope_append(self.q, self.k, self.v, self.kc[index], self.vc[index], B, L, self.t0,
                                         self.heads, Qo=self.q, stream=s, **norm)
        else:
            A.bitnet_rope_append(self.q, self.k, self.v, self.kc[index], self.vc[index], B, L, self.t0, self.heads,
                                 self.rope_base, stream=s)
        return A.bitnet_attention(self.q, self.kc[index], self.vc[index], B, L, self.t0, self.heads, A=self.att,
                                  stream=s)

    def forward(self, x: torch.Tensor, stream=None, t0: int = 0, pos=None, lens=None, t_max=None) -> torch.Tensor:
        """x: [M, hidden] fp32 on the device; returns the last layer's output
        (one of the chain's own buffers).  t0: position of each sequence's first
        token in this step (with attention).  With kv_bits 4, pos and lens ([B] int32
        on the device) place each sequence's tokens at t0 + pos[b] on and mark the rows
        behind its first lens[b] as padding; a captured forward reads them at replay.
        t_max: a bound on the positions in use plus one (api.bitnet_kv4_attention), for
        which the attention's kernels are chosen; with pos and without it that is T_cap."""
        if not (pos is None and lens is None and t_max is None) and (self.attention is None or self.kv_bits != 4):
            raise ValueError("pos, lens and t_max need attention with kv_bits=4")
        self.t0, self.pos, self.lens, self.t_max = t0, pos, lens, t_max
        parts = (x,)
        for i, w in enumerate(self.layers):
            parts = self.layer(parts, w, stream, i)
        api.bitnet_add(parts[0], parts[1], out=self.x[1], stream=stream)
        return self.x[1]

    # kernels launched per forward: per layer 2 int8 quantisers (the second, and
    # from the second layer on the first, with the residual add folded in), 4
    # linear launches (Q/K/V in one, O, up/gate in one, down), 2 Hadamard
    # quantisers (one with the gated unit folded in); one residual add after
    # the last layer.  With attention the append and the attention's kernels: one,
    # or over a 4-bit cache what the library launches for the last forward's step
    @property
    def launches(self) -> int:
        attention = 0
        if self.attention is not None:
            attention = 2
            if self.kv_bits == 4 and self.layers:
                B, L, cache = self.attention["B"], self.attention["L"], self.kv4[0].kc
                T, d = cache.shape[2], 2 * cache.shape[3]
                attention = 1 + api.bitnet_kv4_attention_launches(
                    torch.float32, B, L, self.heads, self.kv_heads, d, T, self.window, self.sinks,
                    api._position_bound(T, self.t0, L, self.pos, self.t_max))
        return (8 + attention) * len(self.layers) + 1

    def packed_bytes(self) -> int:
        return sum(pk.numel() for w in self.layers for pk, _ in w.values())
