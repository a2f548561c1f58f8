"""The measured cases of the 8-bit decoder's operators: the root-mean-square norm with the residual's addition, 8-bit
values with a scale for each block of 128, the matrix product of such values, and the gradients' global norm and clipping.

A case names one pass through one operator:

    op          "rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "quantize_fp8", "matmul_fp8" or "clip_grads"
    dtype       "float32", "bfloat16" or "float16"; of a matrix product: its result's; "mixed" gradients: float32 and bfloat16
    rows, cols  norm, quantize: rows and their length
    residual    norm: x + residual is normalised, and comes back as h; the backward: h has a gradient of its own
    affine      norm: with a weight
    block       quantize: rows that share a scale (1 or 128); product: the same of its second operand
    transposed  quantize: x is the transpose of rows in memory
    m, n, k     product: out[m, n] = a[m, k] b[n, k]^T
    tensors, elements, clipped
                gradients: how many tensors, their elements in all, and whether their norm is above the bound

`own` selects the library's calls; otherwise the same operators run as elementary torch operations
in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 value
LEAST = 2.0 ** -126  # a scale below it is 1
EPS = 1e-6
BLOCK = 128


def listed():
    def norm(name, op, dtype, rows, cols, residual):
        return {"name": name, "op": op, "dtype": dtype, "rows": rows, "cols": cols, "residual": residual, "affine": True}

    def quantize(name, dtype, rows, cols, block, transposed=False):
        return {"name": name, "op": "quantize_fp8", "dtype": dtype, "rows": rows, "cols": cols, "block": block, "transposed": transposed}

    def product(name, dtype, m, n, k, block=BLOCK):
        return {"name": name, "op": "matmul_fp8", "dtype": dtype, "m": m, "n": n, "k": k, "block": block}

    def clip(name, dtype, tensors, elements, clipped=True):
        return {"name": name, "op": "clip_grads", "dtype": dtype, "tensors": tensors, "elements": elements, "clipped": clipped}

    return [
        # one query of a served scene between two blocks of the decoder: the smallest call, where latency counts
        norm("norm fwd 1x1024 bf16", "rms_norm_fwd", "bfloat16", 1, 1024, True),
        # the tokens of eight views of 1297x840 (82 x 53 tiles), four scenes at a time, on their way into 8-bit projections
        norm("norm fp8 139072x1024 bf16", "rms_norm_fp8", "bfloat16", 139072, 1024, True),
        # the same tokens' way back, the weight's gradient summed over all of them
        norm("norm bwd 139072x1024 bf16", "rms_norm_bwd", "bfloat16", 139072, 1024, True),
        # rows of an odd length, which no vector load divides
        norm("norm bwd 20001x333 f16", "rms_norm_bwd", "float16", 20001, 333, False),
        # an updated weight, laid out for the products
        quantize("quantize 4096x1024 f32 tiles", "float32", 4096, 1024, BLOCK),
        # the output gradient of four views' tokens along the tokens, for the weight's gradient
        quantize("quantize 4096x17384 bf16 T", "bfloat16", 4096, 17384, 1, True),
        # one served query through a projection
        product("matmul 1x4096x1024 bf16", "bfloat16", 1, 4096, 1024),
        # four views' tokens (4346 each) through a projection
        product("matmul 17384x4096x1024 bf16", "bfloat16", 17384, 4096, 1024),
        # the queries of a large scene's groups through a square one: the largest
        product("matmul 16384x4096x4096 bf16", "bfloat16", 16384, 4096, 4096),
        # a weight's gradient: scales along the tokens on both sides, float32 as the master weights
        product("matmul 4096x1024x17384 f32", "float32", 4096, 1024, 17384, 1),
        # the decoder's own gradients, after every step
        clip("clip 14 tensors 1.1M f32", "float32", 14, 1_100_000),
        # the gradients of 1.6 million Gaussians of SH degree 3 (59 floats each)
        clip("clip 5 tensors 94.4M f32", "float32", 5, 94_400_000),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "quantize_fp8", "matmul_fp8", "matmul_fp8", "clip_grads"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    if op.startswith("rms_norm"):
        cols = _log_uniform(rng, 32, 8192)
        rows = _log_uniform(rng, 1, min(200000, (64 << 20) // cols))
        return {"op": op, "dtype": dtype, "rows": rows, "cols": cols, "residual": rng.random() < 0.6, "affine": rng.random() < 0.8}
    if op == "quantize_fp8":
        cols = _log_uniform(rng, 32, 17384)
        rows = _log_uniform(rng, 1, min(140000, (64 << 20) // cols))
        return {"op": op, "dtype": dtype, "rows": rows, "cols": cols, "block": rng.choice([1, BLOCK]), "transposed": rng.random() < 0.4}
    if op == "matmul_fp8":
        n, k = _log_uniform(rng, 14, 8192), _log_uniform(rng, 32, 8192)
        m = _log_uniform(rng, 1, min(17384, int(2.5e11 // (n * k))))
        return {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "block": rng.choice([BLOCK, BLOCK, 1])}
    return {"op": op, "dtype": rng.choice(["float32", "bfloat16", "mixed"]), "tensors": _log_uniform(rng, 1, 60),
            "elements": _log_uniform(rng, 1000, 90_000_000), "clipped": rng.random() < 0.8}


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _tokens(rows, cols, gen):
    """Tokens of a trained network: every channel has its own spread, a few are far out."""
    spread = 0.5 + torch.rand(cols, device="cuda", generator=gen) * 2
    spread[torch.rand(cols, device="cuda", generator=gen) < 0.01] *= 12
    return torch.randn(rows, cols, device="cuda", generator=gen) * spread


def _norm_inputs(case, gen):
    dtype, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
    s = {"x": _tokens(rows, cols, gen).to(dtype), "residual": None, "weight": None, "dh": None}
    if case["affine"]:
        s["weight"] = (1 + 0.2 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)
    if case["residual"]:
        s["residual"] = _tokens(rows, cols, gen).to(dtype)
    if case["op"] == "rms_norm_bwd":
        s["h"] = s.pop("x") if s["residual"] is None else (s.pop("x").float() + s["residual"].float()).to(dtype)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = torch.randn(rows, cols, device="cuda", generator=gen).to(dtype)
        if case["residual"]:
            s["dh"] = torch.randn(rows, cols, device="cuda", generator=gen).to(dtype)
        s["residual"] = None
    return s


def _quantize_inputs(case, gen):
    rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
    x = _tokens(cols, rows, gen).to(dtype).t() if case["transposed"] else _tokens(rows, cols, gen).to(dtype)
    return {"x": x, "block": case["block"]}


def _padded(q):
    """The same values in rows that start 16 bytes apart, as the library lays them out."""
    rows, cols = q.shape
    if cols % 16 == 0:
        return q.contiguous()
    wide = torch.zeros(rows, (cols + 15) // 16 * 16, device="cuda", dtype=torch.uint8)
    wide[:, :cols] = q.view(torch.uint8)
    return wide.view(E4M3)[:, :cols]


def _product_inputs(case, gen):
    s = {"dtype": DTYPES[case["dtype"]]}
    for name, rows, block in (("a", case["m"], 1), ("b", case["n"], case["block"])):
        q, scale = _plain_quantize(_tokens(rows, case["k"], gen), block)
        s[name] = _padded(q)
        s[name + "_scale"] = scale.t().contiguous().t()  # consecutive rows' scales lie together
    return s


def _sizes(case):
    """Elements of each gradient: a few large ones and many small ones, of all alignments' lengths."""
    rng = random.Random(case["tensors"] * 1_000_003 + case["elements"])
    if case["tensors"] == 5 and case["elements"] % 59 == 0:  # mean3d, log_scale, quat, opacity_logit, sh
        return [case["elements"] // 59 * w for w in (3, 3, 4, 1, 48)]
    share = [math.exp(rng.gauss(0, 1.5)) for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * x / sum(share))) for x in share]


def _clip_inputs(case, gen):
    grads, square = [], 0.0
    for i, n in enumerate(_sizes(case)):
        dtype = DTYPES["bfloat16" if case["dtype"] == "mixed" and i % 2 else "float32" if case["dtype"] == "mixed" else case["dtype"]]
        spread = 10.0 ** (-4 + 3 * (i % 4) / 3)  # the parameters' gradients are of different sizes
        grads.append((torch.randn(n, device="cuda", generator=gen) * spread).to(dtype))
        square += n * spread * spread
    return {"grads": grads, "max_norm": math.sqrt(square) * (0.3 if case["clipped"] else 3.0), "out": [torch.empty_like(g) for g in grads]}


INPUTS = {"quantize_fp8": _quantize_inputs, "matmul_fp8": _product_inputs, "clip_grads": _clip_inputs}


def prepare(case, seed):
    s = INPUTS.get(case["op"], _norm_inputs)(case, _gen(seed))
    s["op"] = case["op"]
    return s


# ---- the operators as elementary operations, in 32 bits ------------------------------------------

def _blocks(x, block):
    """x [rows, cols] with zeros up to whole blocks: [rows / block, block, cols / 128, 128]."""
    rows, cols = x.shape
    up, across = -(-rows // block), -(-cols // BLOCK)
    if (up * block, across * BLOCK) != (rows, cols):
        x = torch.nn.functional.pad(x, (0, across * BLOCK - cols, 0, up * block - rows))
    return x.reshape(up, block, across, BLOCK)


def _plain_quantize(x, block):
    rows, cols = x.shape
    t = _blocks(x.float(), block)
    scale = t.abs().amax((1, 3)) / TOP
    scale = torch.where(scale < LEAST, torch.ones_like(scale), scale)
    q = (t / scale[:, None, :, None]).reshape(t.shape[0] * block, -1)[:rows, :cols]
    return q.to(E4M3), scale


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["residual"] is None else (x + s["residual"].float()).to(s["x"].dtype).float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"].float()
    return y, None if s["residual"] is None else h.to(s["x"].dtype), rstd


def _plain_norm_fwd(s):
    y, h, rstd = _plain_norm(s)
    return y.to(s["x"].dtype), h, rstd


def _plain_norm_fp8(s):
    y, h, rstd = _plain_norm(s)
    return (*_plain_quantize(y, 1), h, rstd)


def _plain_norm_bwd(s):
    dy, hhat = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy if s["weight"] is None else dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - hhat * (g * hhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), None if s["weight"] is None else (dy * hhat).sum(0).to(s["weight"].dtype)


def _values(q, scale, block):
    """What 8-bit values with their scales stand for."""
    rows, cols = q.shape
    t = _blocks(q.float(), block) * scale[:, None, :, None]
    return t.reshape(t.shape[0] * block, -1)[:rows, :cols]


def _plain_product(s):
    block = 1 if s["b_scale"].shape[0] == s["b"].shape[0] else BLOCK
    out = torch.matmul(_values(s["a"], s["a_scale"], 1), _values(s["b"], s["b_scale"], block).t())
    return (out.to(s["dtype"]),)


def _plain_clip(s):
    squares = [g.double().square().sum() for g in s["grads"]]  # a long sum
    norm = torch.stack(squares).sum().sqrt()
    factor = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0).float()
    return norm.float(), [torch.mul(g.float(), factor).to(g.dtype) for g in s["grads"]]


# ---- one pass ------------------------------------------------------------------------------------

NAMES = {"rms_norm_fwd": ("y", "h", "rstd"), "rms_norm_fp8": ("q", "scale", "h", "rstd"), "rms_norm_bwd": ("dx", "dweight"),
         "quantize_fp8": ("q", "scale"), "matmul_fp8": ("out",), "clip_grads": ("norm", "grads")}


def run(state):
    s, op = state, state["op"]
    if own:
        from differentiable_gaussian_splatting_gs_gb300 import api
        if op == "rms_norm_fwd":
            got = api.gs_rms_norm_fwd(s["x"], s["weight"], s["residual"], eps=EPS)
        elif op == "rms_norm_fp8":
            got = api.gs_rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
        elif op == "rms_norm_bwd":
            got = api.gs_rms_norm_bwd(s["dy"], s["h"], s["rstd"], s["weight"], s["dh"])
        elif op == "quantize_fp8":
            got = api.gs_quantize_fp8(s["x"], block_rows=s["block"])
        elif op == "matmul_fp8":
            got = (api.gs_matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], dtype=s["dtype"]),)
        else:
            got = (api.gs_clip_grads(s["grads"], s["max_norm"], eps=EPS, out=s["out"]), s["out"])
        if op in ("rms_norm_fwd", "rms_norm_fp8") and s["residual"] is None:
            got = (*got[:-2], None, got[-1])  # h is x itself
    else:
        got = {"rms_norm_fwd": _plain_norm_fwd, "rms_norm_fp8": _plain_norm_fp8, "rms_norm_bwd": _plain_norm_bwd,
               "quantize_fp8": lambda s: _plain_quantize(s["x"], s["block"]), "matmul_fp8": _plain_product,
               "clip_grads": _plain_clip}[op](s)
    return {name: t for name, t in zip(NAMES[op], got) if t is not None}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    op = case["op"]
    if op == "matmul_fp8":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * -(-k // BLOCK) * (m + -(-n // case["block"]))
        return {"bytes": m * k + n * k + m * n * size + scales, "flops": 2 * m * n * k}
    if op == "clip_grads":
        count = _sizes(case)
        bits = sum(c * (2 if case["dtype"] == "mixed" and i % 2 else 4 if case["dtype"] == "mixed" else size) for i, c in enumerate(count))
        return {"bytes": 2 * bits, "flops": 3 * sum(count)}
    rows, cols = case["rows"], case["cols"]
    n, across = rows * cols, -(-cols // BLOCK)
    if op == "quantize_fp8":
        return {"bytes": n * size + n + 4 * across * -(-rows // case["block"]), "flops": 2 * n}
    weights = cols * size if case["affine"] else 0
    if op == "rms_norm_bwd":
        return {"bytes": (4 if case["residual"] else 3) * n * size + 4 * rows + 2 * weights, "flops": 9 * n}
    written = n * size if op == "rms_norm_fwd" else n + 4 * rows * across
    return {"bytes": (3 if case["residual"] else 1) * n * size + written + 4 * rows + weights, "flops": 6 * n}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_quantize(x, block):
    """The quotients before their rounding, and the scales."""
    q, scale = torch.empty_like(x), []
    for j in range(0, x.shape[1], BLOCK):
        part = x[:, j:j + BLOCK]
        top = part.abs().max(1).values
        if block > 1:
            top = torch.stack([t.max() for t in top.split(block)])
        one = torch.where(top / TOP < LEAST, 1.0, top / TOP)
        scale.append(one)
        q[:, j:j + BLOCK] = part / one.repeat_interleave(block)[:x.shape[0], None]
    return q, torch.stack(scale, 1)


def _exact_norm(case, s):
    w = s["weight"].double() if s["weight"] is not None else 1.0
    if case["op"] == "rms_norm_bwd":
        h, dy = s["h"].double(), s["dy"].double()
        rstd = (torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS) ** -0.5
        # through the mean square: d rstd = -rstd^3 / cols * h dh
        dhhat = dy * w
        dsquare = -0.5 * rstd ** 3 * torch.einsum("rc,rc->r", dhhat, h)
        dx = dhhat * rstd[:, None] + 2 * dsquare[:, None] * h / case["cols"]
        got = {"dx": dx if s["dh"] is None else dx + s["dh"].double()}
        if s["weight"] is not None:
            got["dweight"] = torch.einsum("rc,rc,r->c", dy, h, rstd)
        return got
    h = s["x"].double()
    got = {}
    if s["residual"] is not None:
        got["h"] = h = (h + s["residual"].double()).to(s["x"].dtype).double()
    got["rstd"] = (torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS) ** -0.5
    y = h * got["rstd"][:, None] * w
    if case["op"] == "rms_norm_fwd":
        return {"y": y, **got}
    q, scale = _exact_quantize(y, 1)
    return {"q": q, "scale": scale, **got}


def _exact_product(case, s):
    out = torch.zeros(case["m"], case["n"], device="cuda", dtype=torch.float64)
    sb = s["b_scale"].double().repeat_interleave(case["block"], 0)[:case["n"]]
    for j in range(s["a_scale"].shape[1]):
        at = slice(j * BLOCK, (j + 1) * BLOCK)
        out += (s["a"][:, at].double() * s["a_scale"][:, j, None].double()) @ (s["b"][:, at].double() * sb[:, j, None]).T
    return {"out": out}


def _exact_clip(s):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
    factor = min(1.0, s["max_norm"] / (norm + EPS))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [g.double() * factor for g in s["grads"]]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize_fp8":
        q, scale = _exact_quantize(s["x"].double(), case["block"])
        return {"q": q, "scale": scale}
    if case["op"] == "matmul_fp8":
        return _exact_product(case, s)
    return _exact_clip(s) if case["op"] == "clip_grads" else _exact_norm(case, s)
