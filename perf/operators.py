"""The measured cases of the Gaussian decoder's operators: layer norm and cross attention.

A decoder that predicts a scene's Gaussians from images keeps one query vector per Gaussian (or per
group of Gaussians), normalises them (layer norm) and lets them read the image encoder's tokens
(cross attention: the queries and the tokens have lengths of their own); the loss's gradient comes
back from the rasterizer through both. A case names one pass through one operator:

    op          "layer_norm_fwd", "layer_norm_bwd", "attention_fwd" or "attention_bwd"
    dtype       "float32", "bfloat16" or "float16"
    rows, cols  layer norm: normalised rows and their length
    affine      layer norm: with a weight and a bias
    batch, heads, kv_heads, len_q, len_k, head_dim
                attention: heads of the queries and of the keys and values (heads // kv_heads query
                heads share one of these), queries and encoder tokens per batch entry
    mask        attention: "none"; "len": a valid length for each batch entry, the first of them 0;
                "keys": one truth value for each token

`own` selects the library's calls; otherwise the same operators run as elementary torch operations
in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-5


def listed():
    def ln(name, op, dtype, rows, cols, affine=True):
        return {"name": name, "op": op, "dtype": dtype, "rows": rows, "cols": cols, "affine": affine}

    def at(name, op, dtype, batch, heads, kv_heads, len_q, len_k, head_dim, mask="none"):
        return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads,
                "len_q": len_q, "len_k": len_k, "head_dim": head_dim, "mask": mask}

    return [
        # one query per Gaussian of the 2,000-Gaussian scene: the smallest call, where latency counts
        ln("norm fwd 2000x256 f32", "layer_norm_fwd", "float32", 2000, 256),
        # eight views of 1297x840, one token per 16x16 tile (82 x 53 of them), four at a time
        ln("norm fwd 139072x1024 bf16", "layer_norm_fwd", "bfloat16", 139072, 1024),
        # the 2,000 queries' way back
        ln("norm bwd 2000x256 f32", "layer_norm_bwd", "float32", 2000, 256),
        # the tokens' way back, the weight's gradient summed over all of them
        ln("norm bwd 139072x1024 bf16", "layer_norm_bwd", "bfloat16", 139072, 1024),
        # rows of an odd length, which no vector load divides
        ln("norm bwd 20001x333 f16", "layer_norm_bwd", "float16", 20001, 333),
        # one query reads one view's tokens: a Gaussian added to a served scene
        at("attn fwd 1 query bf16", "attention_fwd", "bfloat16", 1, 16, 16, 1, 4346, 64),
        # queries of a large scene's groups read one view's tokens, two scenes at a time
        at("attn fwd 16384x4346 bf16", "attention_fwd", "bfloat16", 2, 16, 16, 16384, 4346, 64),
        # 5,000 queries, shared key heads, tokens outside the object's silhouette masked
        at("attn fwd keys d128 f16", "attention_fwd", "float16", 3, 16, 4, 5000, 2500, 128, "keys"),
        # the rasterizer's own type: 5,000 queries read an 800x800 view's tokens
        at("attn fwd 5000x2500 f32", "attention_fwd", "float32", 2, 8, 8, 5000, 2500, 64),
        # the way back of a large scene's groups
        at("attn bwd 16384x4346 bf16", "attention_bwd", "bfloat16", 1, 16, 16, 16384, 4346, 64),
        # shared key heads, views of different sizes padded to one length, one of them empty
        at("attn bwd len d128 f16", "attention_bwd", "float16", 3, 16, 4, 2000, 2500, 128, "len"),
        # the rasterizer's own type: the 2,000-Gaussian scene and a 320x320 view's tokens
        at("attn bwd 2000x400 f32", "attention_bwd", "float32", 1, 8, 8, 2000, 400, 32),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer_norm_fwd", "layer_norm_bwd", "attention_fwd", "attention_bwd"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    if op.startswith("layer_norm"):
        cols = _log_uniform(rng, 32, 4096)
        rows = _log_uniform(rng, 1, min(200000, (64 << 20) // cols))
        return {"op": op, "dtype": dtype, "rows": rows, "cols": cols, "affine": rng.random() < 0.8}
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 4]) if kv_heads < 16 else kv_heads
    head_dim = rng.choice([16, 32, 40, 64, 64, 80, 96, 128])
    batch = rng.choice([1, 1, 2, 3, 4])
    len_k = _log_uniform(rng, 16, 8192)
    most = 2.5e10 if dtype != "float32" else 1e10  # pairs x head_dim: below the largest listed case
    most_q = int(min(16384, max(1, most // (batch * heads * len_k * head_dim))))
    len_q = _log_uniform(rng, 1, most_q)
    return {"op": op, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads, "len_q": len_q,
            "len_k": len_k, "head_dim": head_dim, "mask": rng.choice(["none", "none", "len", "keys"])}


# ---- inputs ------------------------------------------------------------------------------------

def _norm_inputs(case, gen):
    dtype, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
    # tokens of a trained network: every channel has its own mean and spread, a few are far out
    spread = 0.5 + torch.rand(cols, device="cuda", generator=gen) * 2
    shift = torch.randn(cols, device="cuda", generator=gen)
    shift[torch.rand(cols, device="cuda", generator=gen) < 0.01] *= 12
    x = (torch.randn(rows, cols, device="cuda", generator=gen) * spread + shift).to(dtype)
    s = {"x": x, "weight": None, "bias": None}
    if case["affine"]:
        s["weight"] = (1 + 0.2 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)
        s["bias"] = (0.2 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)
    if case["op"] == "layer_norm_bwd":
        s["dy"] = torch.randn(rows, cols, device="cuda", generator=gen).to(dtype)
        _, s["mean"], s["rstd"] = _plain_norm_fwd(s)
    return s


def _attention_inputs(case, gen):
    dtype = DTYPES[case["dtype"]]
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]

    def rand(length, n, factor):  # a projection's output: [batch, length, heads, head_dim]
        return (factor * torch.randn(b, length, n, d, device="cuda", generator=gen)).to(dtype)

    s = {"q": rand(case["len_q"], h, 1.5), "k": rand(case["len_k"], hk, 1.0), "v": rand(case["len_k"], hk, 1.0),
         "k_len": None, "key_mask": None}
    if case["mask"] == "len":
        n = torch.randint(1, case["len_k"] + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
        if b > 1:
            n[0] = 0
        s["k_len"] = n
    elif case["mask"] == "keys":
        s["key_mask"] = torch.rand(b, case["len_k"], device="cuda", generator=gen) < 0.6
    if case["op"] == "attention_bwd":
        s["dout"] = rand(case["len_q"], h, 1.0)
        s["out"], s["lse"] = _plain_attention_fwd(s)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = (_norm_inputs if case["op"].startswith("layer_norm") else _attention_inputs)(case, gen)
    s["op"] = case["op"]
    return s


# ---- the operators as elementary operations, in 32 bits ------------------------------------------

def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy if s["weight"] is None else dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    dx = dx.to(s["x"].dtype)
    if s["weight"] is None:
        return dx, None, None
    return dx, (dy * xhat).sum(0).to(s["x"].dtype), dy.sum(0).to(s["x"].dtype)


def _valid(s):
    """[batch, len_k] truth values: the keys that take part."""
    b, n = s["k"].shape[:2]
    if s["k_len"] is not None:
        return torch.arange(n, device="cuda")[None, :] < s["k_len"][:, None]
    if s["key_mask"] is not None:
        return s["key_mask"]
    return torch.ones(b, n, device="cuda", dtype=torch.bool)


def _by_head(t, heads):
    """[batch, length, n, d] in any type -> [batch, heads, length, d] in 32 bits, shared heads repeated."""
    t = t.float().transpose(1, 2)
    b, n, length, d = t.shape
    return t[:, :, None].expand(b, n, heads // n, length, d).reshape(b, heads, length, d)


def _shared(t, kv_heads):
    """Gradient per query head [batch, heads, length, d] -> summed over sharing heads [batch, length, kv_heads, d]."""
    b, h, length, d = t.shape
    return t.reshape(b, kv_heads, h // kv_heads, length, d).sum(2).transpose(1, 2).contiguous()


def _scores(s):
    q, k = s["q"], s["k"]
    h = q.shape[2]
    scores = torch.matmul(_by_head(q, h), _by_head(k, h).transpose(2, 3)) * (1 / math.sqrt(q.shape[3]))
    return scores.masked_fill_(~_valid(s)[:, None, None, :], -math.inf)


def _plain_attention_fwd(s):
    q = s["q"]
    scores = _scores(s)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)  # a row without keys: exp(-inf - 0) = 0
    p = torch.exp_(scores.sub_(top))
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, _by_head(s["v"], q.shape[2])) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top)[..., 0]
    return out.transpose(1, 2).to(q.dtype).contiguous(), lse.contiguous()


def _plain_attention_bwd(s):
    q, hk = s["q"], s["k"].shape[2]
    h, scale = q.shape[2], 1 / math.sqrt(q.shape[3])
    lse = torch.where(s["lse"] == -math.inf, torch.zeros_like(s["lse"]), s["lse"])
    p = torch.exp_(_scores(s).sub_(lse[..., None]))
    do = _by_head(s["dout"], h)
    dv = _shared(torch.matmul(p.transpose(2, 3), do), hk)
    delta = (do * _by_head(s["out"], h)).sum(3, keepdim=True)
    ds = p.mul_(torch.matmul(do, _by_head(s["v"], h).transpose(2, 3)).sub_(delta)).mul_(scale)
    dq = torch.matmul(ds, _by_head(s["k"], h)).transpose(1, 2).contiguous()
    dk = _shared(torch.matmul(ds.transpose(2, 3), _by_head(q, h)), hk)
    return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)


# ---- one pass ------------------------------------------------------------------------------------

NAMES = {"layer_norm_fwd": ("y", "mean", "rstd"), "layer_norm_bwd": ("dx", "dweight", "dbias"),
         "attention_fwd": ("out", "lse"), "attention_bwd": ("dq", "dk", "dv")}


def run(state):
    op = state["op"]
    if own:
        from differentiable_gaussian_splatting_gs_gb300 import api
        if op == "layer_norm_fwd":
            got = api.gs_layer_norm_fwd(state["x"], state["weight"], state["bias"], eps=EPS)
        elif op == "layer_norm_bwd":
            got = api.gs_layer_norm_bwd(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
        elif op == "attention_fwd":
            got = api.gs_cross_attention_fwd(state["q"], state["k"], state["v"], k_len=state["k_len"],
                                             key_mask=state["key_mask"])
        else:
            got = api.gs_cross_attention_bwd(state["dout"], state["q"], state["k"], state["v"], state["out"],
                                             state["lse"], k_len=state["k_len"], key_mask=state["key_mask"])
    else:
        got = {"layer_norm_fwd": _plain_norm_fwd, "layer_norm_bwd": _plain_norm_bwd,
               "attention_fwd": _plain_attention_fwd, "attention_bwd": _plain_attention_bwd}[op](state)
    return {name: t for name, t in zip(NAMES[op], got) if t is not None}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"].startswith("layer_norm"):
        n, c = case["rows"] * case["cols"], case["cols"] if case["affine"] else 0
        if case["op"] == "layer_norm_fwd":
            return {"bytes": 2 * n * size + 8 * case["rows"] + 2 * c * size, "flops": 8 * n}
        return {"bytes": 3 * n * size + 8 * case["rows"] + 3 * c * size, "flops": 13 * n}
    b, h, hk, lq, lk, d = (case[k] for k in ("batch", "heads", "kv_heads", "len_q", "len_k", "head_dim"))
    # the share of the keys that takes part, as the inputs are drawn
    share = {"none": 1.0, "keys": 0.6, "len": 0.5 * (b - 1) / b if b > 1 else 0.5}[case["mask"]]
    queries, keys = b * h * lq * d * size, int(b * hk * lk * d * size * share)
    whole = b * hk * lk * d * size
    pairs = int(b * h * lq * lk * share) * d
    if case["op"] == "attention_fwd":
        return {"bytes": 2 * queries + 2 * keys + 4 * b * h * lq, "flops": 4 * pairs}
    return {"bytes": 4 * queries + 2 * keys + 2 * whole + 4 * b * h * lq, "flops": 10 * pairs}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_norm(case, s):
    x = s["x"].double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    w = s["weight"].double() if s["weight"] is not None else x.new_ones(case["cols"])
    if case["op"] == "layer_norm_fwd":
        b = s["bias"].double() if s["bias"] is not None else 0.0
        return {"y": (x - mean) * rstd * w + b, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    # by the chain rule through the variance and the mean
    dy, n = s["dy"].double(), case["cols"]
    dxhat = dy * w
    dvar = (dxhat * (x - mean)).sum(1, keepdim=True) * -0.5 * rstd ** 3
    dmean = -(dxhat * rstd).sum(1, keepdim=True)
    got = {"dx": dxhat * rstd + dvar * 2 * (x - mean) / n + dmean / n}
    if s["weight"] is not None:
        got["dweight"] = torch.einsum("rc,rc->c", dy, (x - mean) * rstd)
        got["dbias"] = dy.sum(0)
    return got


def _exact_attention(case, s):
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    b, lq, h, d = q.shape
    share = h // k.shape[2]
    fwd = case["op"] == "attention_fwd"
    if fwd:
        out, lse = torch.zeros_like(q), q.new_full((b, h, lq), -math.inf)
    else:
        do, dq, dk, dv = s["dout"].double(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(b):
        if s["k_len"] is not None:
            at = torch.arange(int(s["k_len"][i]), device="cuda")
        elif s["key_mask"] is not None:
            at = s["key_mask"][i].nonzero()[:, 0]
        else:
            at = torch.arange(k.shape[1], device="cuda")
        if at.numel() == 0:
            continue
        for j in range(h):
            kk, vv = k[i, at, j // share], v[i, at, j // share]
            z = torch.einsum("qd,kd->qk", q[i, :, j], kk) / d ** 0.5
            if fwd:
                lse[i, j] = torch.logsumexp(z, 1)
                out[i, :, j] = torch.softmax(z, 1) @ vv
                continue
            p = torch.softmax(z, 1)
            dv[i, at, j // share] += p.T @ do[i, :, j]
            dp = torch.einsum("qd,kd->qk", do[i, :, j], vv)
            dz = p * (dp - (p * dp).sum(1, keepdim=True)) / d ** 0.5
            dq[i, :, j] = dz @ kk
            dk[i, at, j // share] += dz.T @ q[i, :, j]
    return {"out": out, "lse": lse} if fwd else {"dq": dq, "dk": dk, "dv": dv}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_norm if case["op"].startswith("layer_norm") else _exact_attention)(case, s)
