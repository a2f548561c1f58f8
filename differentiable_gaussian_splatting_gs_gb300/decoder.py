"""A Gaussian decoder: predicts a scene's Gaussians from image tokens and trains through the rasterizer.

One query vector per Gaussian is normalised (gs_layer_norm_fwd), reads the encoder's normalised tokens
(gs_cross_attention_fwd: the queries and the tokens have lengths of their own, shorter views are masked) and is turned
into the Gaussian's parameters by a linear head:

    h = norm(x), t = norm(tokens);  a = attention(h Wq, t Wk, t Wv);  x' = x + a Wo;  out = norm(x') Wh + bh

The gradients of these parameters, as step.train_step leaves them (gs_preprocess_bwd), come back through
backward(): written out by hand from the two operators' own backward calls, with plain matrix products between.
Weights and their gradients are float32; activations have the decoder's dtype.
"""
from __future__ import annotations

import torch

from . import api, step

# columns of the head's output
PARTS = {"mean3d": (0, 3), "log_scale": (3, 6), "quat": (6, 10), "opacity_logit": (10, 11), "sh": (11, 14)}


class GaussianDecoder:
    """n Gaussians of SH degree 0 from tokens [1, length, token_channels].

    base: the Gaussians that a zero head stands for: mean3d [n, 3], log_scale [n, 3], quat [n, 4], opacity_logit [n]
    and sh [n, 1, 3]; the head predicts offsets from them."""

    def __init__(self, base: dict, token_channels: int, channels: int = 128, heads: int = 4, kv_heads: int | None = None,
                 head_dim: int = 32, dtype=torch.float32, seed: int = 0):
        self.base, self.dtype = base, dtype
        self.n, self.heads, self.kv_heads, self.head_dim = int(base["mean3d"].shape[0]), heads, kv_heads or heads, head_dim
        dev = base["mean3d"].device
        gen = torch.Generator(device=dev).manual_seed(seed)

        def random(rows, cols):
            return torch.randn(rows, cols, device=dev, generator=gen) * rows ** -0.5

        inner, inner_kv = heads * head_dim, self.kv_heads * head_dim
        w = {"queries": random(self.n, channels) * self.n ** 0.5, "wq": random(channels, inner),
             "wk": random(token_channels, inner_kv), "wv": random(token_channels, inner_kv), "wo": random(inner, channels),
             "wh": random(channels, 14) * 0.1, "bh": torch.zeros(14, device=dev)}
        for name, size in (("q", channels), ("t", token_channels), ("x", channels)):
            w["norm_" + name + "_weight"] = torch.ones(size, device=dev)
            w["norm_" + name + "_bias"] = torch.zeros(size, device=dev)
        self.weights = w
        self.grads = {k: torch.zeros_like(v) for k, v in w.items()}
        self._saved = None

    def _norm(self, x, name: str):
        return api.gs_layer_norm_fwd(x, self.weights[f"norm_{name}_weight"], self.weights[f"norm_{name}_bias"])

    def _norm_bwd(self, dy, x, stats, name: str):
        w = self.weights[f"norm_{name}_weight"]
        out = (torch.empty_like(x), self.grads[f"norm_{name}_weight"], self.grads[f"norm_{name}_bias"])
        return api.gs_layer_norm_bwd(dy, x, *stats, w, out=out)[0]

    def forward(self, tokens, k_len=None, key_mask=None) -> dict:
        """The Gaussians' parameters (float32, as gs_preprocess takes them) from one scene's tokens [1, length,
        token_channels]; k_len [1], key_mask [1, length] as gs_cross_attention_fwd's."""
        if tokens.dim() != 3 or tokens.shape[0] != 1 or tokens.shape[2] != self.weights["wk"].shape[0]:
            raise ValueError(f"tokens must be [1, length, {self.weights['wk'].shape[0]}] (one scene), got {tuple(tokens.shape)}")
        w = {k: v.to(self.dtype) for k, v in self.weights.items()}
        x, tokens = w["queries"], tokens[0].to(self.dtype)
        h, *stats_q = self._norm(x, "q")
        t, *stats_t = self._norm(tokens, "t")
        q = (h @ w["wq"]).view(1, self.n, self.heads, self.head_dim)
        k = (t @ w["wk"]).view(1, t.shape[0], self.kv_heads, self.head_dim)
        v = (t @ w["wv"]).view(1, t.shape[0], self.kv_heads, self.head_dim)
        a, lse = api.gs_cross_attention_fwd(q, k, v, k_len=k_len, key_mask=key_mask)
        x2 = x + a.view(self.n, -1) @ w["wo"]
        y, *stats_x = self._norm(x2, "x")
        out = (y @ w["wh"]).float() + self.weights["bh"]
        self._saved = (w, x, tokens, h, stats_q, t, stats_t, q, k, v, a, lse, x2, y, stats_x, k_len, key_mask)
        return {name: (self.base[name] + out[:, lo:hi].reshape(self.base[name].shape)).contiguous()
                for name, (lo, hi) in PARTS.items()}

    def backward(self, grads: dict):
        """Leaves the weights' gradients in self.grads, from the parameters' (names as forward's); returns that of the tokens."""
        w, x, tokens, h, stats_q, t, stats_t, q, k, v, a, lse, x2, y, stats_x, k_len, key_mask = self._saved
        g = self.grads
        dout32 = torch.cat([grads[name].reshape(self.n, -1) for name in PARTS], 1)
        dout = dout32.to(self.dtype)
        torch.sum(dout32, 0, out=g["bh"])
        g["wh"].copy_(y.t() @ dout)
        dx2 = self._norm_bwd(dout @ w["wh"].t(), x2, stats_x, "x")
        g["wo"].copy_(a.view(self.n, -1).t() @ dx2)
        da = (dx2 @ w["wo"].t()).view_as(a)
        dq, dk, dv = api.gs_cross_attention_bwd(da, q, k, v, a, lse, k_len=k_len, key_mask=key_mask)
        dq, dk, dv = (x.flatten(2)[0] for x in (dq, dk, dv))
        g["wq"].copy_(h.t() @ dq)
        g["wk"].copy_(t.t() @ dk)
        g["wv"].copy_(t.t() @ dv)
        dtokens = self._norm_bwd(dk @ w["wk"].t() + dv @ w["wv"].t(), tokens, stats_t, "t")
        g["queries"].copy_(dx2 + self._norm_bwd(dq @ w["wq"].t(), x, stats_q, "q"))
        return dtokens[None]


class DecoderTrainer:
    """Trains a GaussianDecoder on views of one scene: forward, step.train_step over the views (squared-error loss),
    backward, and Adam on the decoder's weights."""

    def __init__(self, decoder: GaussianDecoder, lr: float = 2e-3, beta1: float = 0.9, beta2: float = 0.999):
        self.decoder, self.lr, self.beta1, self.beta2, self.t = decoder, lr, beta1, beta2, 0
        self.buffers = step.StepBuffers(decoder.n, decoder.base["mean3d"].device)
        self.opt = api.make_options(0)
        self.moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in decoder.weights.items()}
        self.param_grads = api.alloc_param_grads(decoder.base)

    def step(self, tokens, cameras, targets, k_len=None, key_mask=None) -> torch.Tensor:
        """One step; returns the last view's image before it (a reused buffer)."""
        d = self.decoder
        params = d.forward(tokens, k_len=k_len, key_mask=key_mask)
        image = step.train_step(params, cameras, targets, self.opt, self.param_grads, self.buffers)["image"]
        d.backward(self.param_grads)
        self.t += 1
        for name, w in d.weights.items():
            m, v = self.moments[name]
            g = d.grads[name]
            m.lerp_(g, 1 - self.beta1)
            v.lerp_(g * g, 1 - self.beta2)
            w -= self.lr * (m / (1 - self.beta1 ** self.t)) / ((v / (1 - self.beta2 ** self.t)).sqrt() + 1e-12)
        return image
