"""A Gaussian decoder: predicts a scene's Gaussians from image tokens and trains through the rasterizer.

One query vector per Gaussian is normalised (gs_layer_norm_fwd, or gs_rms_norm_fwd with norm="rms"), reads the encoder's
normalised tokens (gs_cross_attention_fwd: the queries and the tokens have lengths of their own, shorter views are masked) and
is turned into the Gaussian's parameters by a linear head:

    h = norm(x), t = norm(tokens);  a = attention(h Wq, t Wk, t Wv);  x' = x + a Wo;  out = norm(x') Wh + bh

With fp8=True the products with Wq, Wk, Wv and Wo, and those of their gradients, are 8-bit (gs_quantize_fp8, gs_matmul_fp8);
serve() runs the forward in 8 bits with weights laid out once, which is faster than bfloat16's forward (16,384 Gaussians of 4,346
tokens, 1,024 channels: 370 us, 420); a training step is not (1,770 us, 1,615), for the quantizing. The gradients of these
parameters, as step.train_step leaves them (gs_preprocess_bwd), come back through backward(): written out by hand from the operators'
own backward calls, with matrix products between. Weights and their gradients are float32; activations have the decoder's dtype.
"""
from __future__ import annotations

import torch

from . import api, step

# columns of the head's output
PARTS = {"mean3d": (0, 3), "log_scale": (3, 6), "quat": (6, 10), "opacity_logit": (10, 11), "sh": (11, 14)}


class GaussianDecoder:
    """n Gaussians of SH degree 0 from tokens [1, length, token_channels].

    base: the Gaussians that a zero head stands for: mean3d [n, 3], log_scale [n, 3], quat [n, 4], opacity_logit [n]
    and sh [n, 1, 3]; the head predicts offsets from them. norm: "layer" (with weight and bias) or "rms" (with weight)."""

    def __init__(self, base: dict, token_channels: int, channels: int = 128, heads: int = 4, kv_heads: int | None = None,
                 head_dim: int = 32, dtype=torch.float32, seed: int = 0, norm: str = "layer", fp8: bool = False):
        if norm not in ("layer", "rms"):
            raise ValueError(f'norm must be "layer" or "rms", not {norm!r}')
        self.base, self.dtype, self.rms, self.fp8 = base, dtype, norm == "rms", bool(fp8)
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
            if not self.rms:
                w["norm_" + name + "_bias"] = torch.zeros(size, device=dev)
        self.weights = w
        self.grads = {k: torch.zeros_like(v) for k, v in w.items()}
        self._saved = None

    def _norm(self, x, name: str, residual=None):
        """(norm of x + residual, that sum, what the backward needs)."""
        if self.rms:
            y, h, rstd = api.gs_rms_norm_fwd(x, self.weights[f"norm_{name}_weight"], residual)
            return y, h, (rstd,)
        if residual is not None:
            x = residual + x
        y, *stats = api.gs_layer_norm_fwd(x, self.weights[f"norm_{name}_weight"], self.weights[f"norm_{name}_bias"])
        return y, x, stats

    def _norm_bwd(self, dy, x, stats, name: str, dx=None):
        """The gradient of x, plus dx, what came back to it by other ways."""
        w, out = self.weights[f"norm_{name}_weight"], (torch.empty_like(x), self.grads[f"norm_{name}_weight"])
        if self.rms:
            return api.gs_rms_norm_bwd(dy, x, *stats, w, dx, out=out)[0]
        got = api.gs_layer_norm_bwd(dy, x, *stats, w, out=out + (self.grads[f"norm_{name}_bias"],))[0]
        return got if dx is None else dx + got

    def _norm8(self, x, name: str):
        """The norm of x in 8 bits."""
        if self.rms:
            return api.gs_rms_norm_fp8(x, self.weights[f"norm_{name}_weight"])[:2]
        return api.gs_quantize_fp8(self._norm(x, name)[0])

    def _weights8(self, backward: bool = False) -> dict:
        """The projections' weights in 8 bits, as the second operand of a product: [outputs, inputs], backward [inputs, outputs]."""
        return {name: api.gs_quantize_fp8(self.weights[name] if backward else self.weights[name].t(), 128) for name in ("wq", "wk", "wv", "wo")}

    def _project(self, x, name: str, w: dict):
        if self.fp8:
            return api.gs_matmul_fp8(*api.gs_quantize_fp8(x), *w["8bit"][name], dtype=self.dtype)
        return x @ w[name]

    def _project_bwd(self, dy, x, name: str, w: dict):
        """Leaves the weight's gradient in self.grads; returns that of x."""
        if not self.fp8:
            self.grads[name].copy_(x.t() @ dy)
            return dy @ w[name].t()
        api.gs_matmul_fp8(*api.gs_quantize_fp8(x.t()), *api.gs_quantize_fp8(dy.t()), out=self.grads[name])
        return api.gs_matmul_fp8(*api.gs_quantize_fp8(dy), *w["8bit_bwd"][name], dtype=self.dtype)

    def _scene(self, tokens):
        if tokens.dim() != 3 or tokens.shape[0] != 1 or tokens.shape[2] != self.weights["wk"].shape[0]:
            raise ValueError(f"tokens must be [1, length, {self.weights['wk'].shape[0]}] (one scene), got {tuple(tokens.shape)}")
        return tokens[0].to(self.dtype)

    def _gaussians(self, y, wh) -> dict:
        out = (y @ wh).float() + self.weights["bh"]
        return {name: (self.base[name] + out[:, lo:hi].reshape(self.base[name].shape)).contiguous()
                for name, (lo, hi) in PARTS.items()}

    def forward(self, tokens, k_len=None, key_mask=None) -> dict:
        """The Gaussians' parameters (float32, as gs_preprocess takes them) from one scene's tokens [1, length,
        token_channels]; k_len [1], key_mask [1, length] as gs_cross_attention_fwd's."""
        tokens = self._scene(tokens)
        w = {k: v.to(self.dtype) for k, v in self.weights.items()}
        if self.fp8:
            w["8bit"], w["8bit_bwd"] = self._weights8(), self._weights8(backward=True)  # the backward's are the forward's too
        x = w["queries"]
        h, _, stats_q = self._norm(x, "q")
        t, _, stats_t = self._norm(tokens, "t")
        q = self._project(h, "wq", w).view(1, self.n, self.heads, self.head_dim)
        k = self._project(t, "wk", w).view(1, t.shape[0], self.kv_heads, self.head_dim)
        v = self._project(t, "wv", w).view(1, t.shape[0], self.kv_heads, self.head_dim)
        a, lse = api.gs_cross_attention_fwd(q, k, v, k_len=k_len, key_mask=key_mask)
        y, x2, stats_x = self._norm(self._project(a.view(self.n, -1), "wo", w), "x", residual=x)
        self._saved = (w, x, tokens, h, stats_q, t, stats_t, q, k, v, a, lse, x2, y, stats_x, k_len, key_mask)
        return self._gaussians(y, w["wh"])

    def backward(self, grads: dict):
        """Leaves the weights' gradients in self.grads, from the parameters' (names as forward's); returns that of the tokens. Of the
        last forward, whose weights must not have changed since (8-bit projections are kept, the others may be read again)."""
        w, x, tokens, h, stats_q, t, stats_t, q, k, v, a, lse, x2, y, stats_x, k_len, key_mask = self._saved
        g = self.grads
        dout32 = torch.cat([grads[name].reshape(self.n, -1) for name in PARTS], 1)
        dout = dout32.to(self.dtype)
        torch.sum(dout32, 0, out=g["bh"])
        g["wh"].copy_(y.t() @ dout)
        dx2 = self._norm_bwd(dout @ w["wh"].t(), x2, stats_x, "x")
        da = self._project_bwd(dx2, a.view(self.n, -1), "wo", w).view_as(a)
        dq, dk, dv = api.gs_cross_attention_bwd(da, q, k, v, a, lse, k_len=k_len, key_mask=key_mask)
        dq, dk, dv = (x.flatten(2)[0] for x in (dq, dk, dv))
        dh = self._project_bwd(dq, h, "wq", w)
        dt = self._project_bwd(dk, t, "wk", w) + self._project_bwd(dv, t, "wv", w)
        dtokens = self._norm_bwd(dt, tokens, stats_t, "t")
        g["queries"].copy_(self._norm_bwd(dh, x, stats_q, "q", dx=dx2))
        return dtokens[None]

    def serving(self) -> dict:
        """What serve() needs of the weights, laid out once (again after they change): 8-bit projections, and the queries'
        own, which no scene changes."""
        w8 = self._weights8()
        x = self.weights["queries"].to(self.dtype)
        q = api.gs_matmul_fp8(*self._norm8(x, "q"), *w8["wq"], dtype=self.dtype)
        return {"w8": w8, "x": x, "q": q.view(1, self.n, self.heads, self.head_dim), "wh": self.weights["wh"].to(self.dtype)}

    def serve(self, tokens, state: dict, k_len=None, key_mask=None) -> dict:
        """The Gaussians as forward's, with 8-bit projections and nothing kept for a backward; state: serving()'s."""
        tokens = self._scene(tokens)
        t8, w8 = self._norm8(tokens, "t"), state["w8"]
        k, v = (api.gs_matmul_fp8(*t8, *w8[name], dtype=self.dtype).view(1, tokens.shape[0], self.kv_heads, self.head_dim)
                for name in ("wk", "wv"))
        a, _ = api.gs_cross_attention_fwd(state["q"], k, v, k_len=k_len, key_mask=key_mask)
        o = api.gs_matmul_fp8(*api.gs_quantize_fp8(a.view(self.n, -1)), *w8["wo"], dtype=self.dtype)
        return self._gaussians(self._norm(o, "x", residual=state["x"])[0], state["wh"])


class DecoderTrainer:
    """Trains a GaussianDecoder on views of one scene: forward, step.train_step over the views (squared-error loss),
    backward, with max_norm the clipping of all weights' gradients by their global norm (gs_clip_grads; the last
    step's is `grad_norm`), and Adam on the decoder's weights."""

    def __init__(self, decoder: GaussianDecoder, lr: float = 2e-3, beta1: float = 0.9, beta2: float = 0.999,
                 max_norm: float | None = None):
        self.decoder, self.lr, self.beta1, self.beta2, self.t = decoder, lr, beta1, beta2, 0
        self.max_norm, self.grad_norm = max_norm, None
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
        if self.max_norm is not None:
            self.grad_norm = api.gs_clip_grads(list(d.grads.values()), self.max_norm)
        self.t += 1
        for name, w in d.weights.items():
            m, v = self.moments[name]
            g = d.grads[name]
            m.lerp_(g, 1 - self.beta1)
            v.lerp_(g * g, 1 - self.beta2)
            w -= self.lr * (m / (1 - self.beta1 ** self.t)) / ((v / (1 - self.beta2 ** self.t)).sqrt() + 1e-12)
        return image
