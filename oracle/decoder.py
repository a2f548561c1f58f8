"""Float64 layer norm and cross attention (numpy), with the magnitudes that rounding errors scale with.

Layer norm over rows of x [R, C]; cross attention of q [B, Lq, H, D] over k, v [B, Lk, Hk, D], H a
multiple of Hk, with valid [B, Lk] truth values. Independent of the CUDA library.
"""
import numpy as np


def layer_norm_fwd(x, w, b, eps):
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = xhat if w is None else xhat * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_bwd(dy, x, w, eps):
    _, mean, rstd = layer_norm_fwd(x, None, None, eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _spread(t, heads):
    """[B, L, n, D] -> [B, heads, L, D]: every head's own copy of the shared one it reads."""
    return np.repeat(t.transpose(0, 2, 1, 3), heads // t.shape[2], axis=1)


def _gather(t, kv_heads):
    """[B, H, L, D] -> [B, L, kv_heads, D]: summed over the heads that share."""
    b, h, length, d = t.shape
    return t.reshape(b, kv_heads, h // kv_heads, length, d).sum(2).transpose(0, 2, 1, 3)


def _clean(t, valid):
    """What masked keys hold takes no part."""
    return np.where(valid[:, :, None, None], t, 0.0)


def attention_fwd(q, k, v, valid, scale):
    """dict: out [B, Lq, H, D], lse [B, H, Lq]; mag: sum_j P_j |v_j| (layout of out); size: the largest
    scale sum |q| |k| of each query [B, H, Lq]."""
    h = q.shape[2]
    k, v = _clean(k, valid), _clean(v, valid)
    qh, kh, vh = _spread(q, h), _spread(k, h), _spread(v, h)
    s = np.where(valid[:, None, None, :], scale * qh @ kh.swapaxes(2, 3), -np.inf)
    top = s.max(3, initial=-np.inf, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(3, keepdims=True)
    p = e / np.where(total == 0, 1.0, total)
    with np.errstate(divide="ignore"):
        lse = np.where(total == 0, -np.inf, np.log(total) + np.where(np.isfinite(top), top, 0.0))[..., 0]
    return {"out": (p @ vh).transpose(0, 2, 1, 3), "lse": lse, "p": p, "mag": (p @ np.abs(vh)).transpose(0, 2, 1, 3),
            "size": (scale * np.abs(qh) @ np.abs(kh).swapaxes(2, 3)).max(3, initial=0.0)}


def attention_bwd(dout, q, k, v, valid, scale, rounding=0.0, accumulate=0.0):
    """dict: dq, dk, dv, and for each a bound `<name>_tol` of its error when probabilities and score gradients
    are rounded to a relative `rounding` (also `out`, from which delta is formed) and products are accumulated
    to `accumulate` of the sum of their magnitudes (see tests)."""
    h, hk = q.shape[2], k.shape[2]
    f = attention_fwd(q, k, v, valid, scale)
    k, v = _clean(k, valid), _clean(v, valid)
    qh, kh, vh, do = _spread(q, h), _spread(k, h), _spread(v, h), _spread(dout, h)
    out, p = _spread(f["out"], h), f["p"]
    delta = (do * out).sum(3, keepdims=True)
    dp = do @ vh.swapaxes(2, 3)
    ds = scale * p * (dp - delta)
    r = {"dq": (ds @ kh).transpose(0, 2, 1, 3), "dk": _gather(ds.swapaxes(2, 3) @ qh, hk),
         "dv": _gather(p.swapaxes(2, 3) @ do, hk), "lse": f["lse"], "out": f["out"]}
    # a probability is off by a relative `rounding` plus the absolute error of its score (and of lse)
    ep = 2 * rounding + accumulate + 2 * accumulate * f["size"][..., None]
    err = scale * p * (ep * (np.abs(dp) + np.abs(delta)) + accumulate * (np.abs(do) @ np.abs(vh).swapaxes(2, 3)) +
                       rounding * (np.abs(do) * np.abs(out)).sum(3, keepdims=True))
    r["dq_tol"] = (err @ np.abs(kh)).transpose(0, 2, 1, 3) + 2 * rounding * np.abs(r["dq"])
    r["dk_tol"] = _gather(err.swapaxes(2, 3) @ np.abs(qh), hk) + 2 * rounding * np.abs(r["dk"])
    r["dv_tol"] = _gather((p * ep).swapaxes(2, 3) @ np.abs(do), hk) + 2 * rounding * np.abs(r["dv"])
    return r
