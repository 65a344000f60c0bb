"""What the operators around the 8-bit products are measured on: the 8-bit integer
quantiser (a scale for each row), the integer product with a scale for each
token and channel, the linear layer made of both, layer norm's forward and
backward, and the gradients' global norm with clipping, in the sizes the
library's benchmark uses (256 to 4097) and in the ranges around them.

`own` says which side `run` computes: the plain form in elementary torch
operations (False), or the library's entry points (True).
"""

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
AMAX_FLOOR = 2.0 ** -100
NORM_EPS = 1e-5
CLIP_EPS = 1e-6


def listed():
    return [
        # the activations of 16 sequences that decode one token each: latency is all
        dict(name="quantize decode 16x1024", op="quantize", rows=16, cols=1024, type="bf16"),
        # a long batch's activations
        dict(name="quantize batch 8192x8192", op="quantize", rows=8192, cols=8192, type="bf16"),
        # one token through a layer: the weight is read once, and nothing else matters
        dict(name="gemm token 1x4096x4096", op="gemm", m=1, n=4096, k=4096, type="bf16", bias="none"),
        # a prompt, ragged in every direction, to logits in float
        dict(name="gemm ragged 4097", op="gemm", m=4097, n=4097, k=4097, type="f32", bias="f32"),
        # the largest product
        dict(name="gemm batch 8192", op="gemm", m=8192, n=8192, k=8192, type="bf16", bias="none"),
        # a small layer on a short prompt, quantiser and product in one call
        dict(name="linear 256x1024x1024", op="linear", tokens=256, inputs=1024, outputs=1024, type="bf16", bias="bf16"),
        # the norm before a layer while 16 sequences decode
        dict(name="norm decode 16x1024", op="norm", rows=16, cols=1024, type="bf16", params="f32", train=False),
        # forward and backward of fp32 tokens, sizes that no vector divides
        dict(name="norm train 4097x2049", op="norm", rows=4097, cols=2049, type="f32", params="f32", train=True),
        # forward and backward of a long batch
        dict(name="norm train 8192x4096", op="norm", rows=8192, cols=4096, type="bf16", params="f32", train=True),
        # a small network's gradients, copied into the flat buffer that the optimiser reads
        dict(name="clip 4 tensors 1M", op="clip", tensors=4, elements=1 << 20, types="f32", over=True),
        # most steps of a run: the norm is within its limit and nothing has to be written
        dict(name="clip 200 tensors 64M within", op="clip", tensors=200, elements=1 << 26, types="mixed", over=False),
        # a large network's fp32 gradients, over the limit
        dict(name="clip 48 tensors 256M", op="clip", tensors=48, elements=1 << 28, types="f32", over=True),
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of [low, high]; multiples of 128, of 8 and odd ones in turn."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    step = rng.choice((1, 1, 8, 128))
    v = v // step * step if v >= step else v
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "linear", "norm", "clip"))
    kind = rng.choice(tuple(TYPES))
    bias = rng.choice(("none", "f32", kind))
    if op == "quantize":
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 64, 8192), type=kind)
    if op == "gemm":
        return dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 64, 8192), k=_size(rng, 64, 8192), type=kind, bias=bias)
    if op == "linear":
        return dict(op=op, tokens=_size(rng, 1, 4096), inputs=_size(rng, 64, 4096), outputs=_size(rng, 64, 4096), type=kind, bias=bias)
    if op == "norm":
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 64, 8192), type=kind, params=rng.choice(("f32", kind)), train=rng.random() < 0.7)
    tensors = _size(rng, 1, 200)
    return dict(op=op, tensors=tensors, elements=_size(rng, 64 * tensors, 1 << 27), types=rng.choice((*TYPES, "mixed")), over=rng.random() < 0.6)


def _tensors(case):
    """(elements, type) of each tensor of a clip case: matrices that share the elements, and a vector after each."""
    rng = random.Random("%d tensors, %d elements" % (case["tensors"], case["elements"]))
    share = [math.exp(rng.uniform(-1, 1)) for _ in range(-(-case["tensors"] // 2))]
    kinds = ("f32", "bf16") if case["types"] == "mixed" else (case["types"],)
    out = []
    for i in range(case["tensors"]):
        n = max(1, int(case["elements"] * share[i // 2] / sum(share)))
        out.append((n if i % 2 == 0 else math.isqrt(n), kinds[i // 2 % len(kinds)]))
    return out


# ---------------------------------------------------------------- plain form

def _quantize(x):
    """(codes, scales) of a matrix; the quotients in 64 bits, since many lie next to a border between two codes."""
    s = (x.abs().amax(dim=1).double().clamp(min=AMAX_FLOOR) / 127).float()
    return torch.round(x.double() / s.double()[:, None]).to(torch.int8), s


def _product(a, sa, b, sb, bias, kind):
    d = (a.float() @ b.float().T) * sa[:, None] * sb
    return (d if bias is None else d + bias.float()).to(kind)


def _plain(state):
    c = state["case"]
    if c["op"] == "quantize":
        return list(_quantize(state["x"]))
    if c["op"] == "gemm":
        return _product(*state["a"], *state["b"], state["bias"], TYPES[c["type"]])
    if c["op"] == "linear":
        return _product(*_quantize(state["x"]), *state["w"], state["bias"], TYPES[c["type"]])
    if c["op"] == "norm":
        kind, x, w, b = TYPES[c["type"]], state["x"].float(), state["w"].float(), state["b"].float()
        mean = x.mean(dim=1, keepdim=True)
        rstd = 1 / torch.sqrt((x - mean).square().mean(dim=1, keepdim=True) + NORM_EPS)
        h = (x - mean) * rstd
        y = (h * w + b).to(kind)
        if not c["train"]:
            return [y]
        dy = state["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - h * (g * h).mean(dim=1, keepdim=True))
        return [y, dx.to(kind), (dy * h).sum(dim=0), dy.sum(dim=0)]
    flat = torch.cat([g.reshape(-1).float() for g in state["grads"]])
    norm = torch.sqrt(flat.double().square().sum())
    flat = flat * torch.clamp(state["limit"] / (norm + CLIP_EPS), max=1.0).float()
    parts = flat.split([g.numel() for g in state["grads"]])
    return [norm.float()] + [torch.cat([p for p, g in zip(parts, state["grads"]) if g.dtype == kind]).to(kind) for kind in state["flat"]]


# ------------------------------------------------------------ the library's

def _library(state):
    from dense_fp32_matrix_row_amd import gradients, int8, layernorm

    c = state["case"]
    if c["op"] == "quantize":
        o = int8.quantize(state["x"])
        return [o.q, o.s]
    if c["op"] == "gemm":
        return int8.gemm(int8.Int8(*state["a"]), int8.Int8(*state["b"]), bias=state["bias"], out_dtype=TYPES[c["type"]])
    if c["op"] == "linear":
        return int8.linear(state["x"], int8.Int8(*state["w"]), bias=state["bias"])
    if c["op"] == "norm":
        if not c["train"]:
            return [layernorm.layer_norm(state["x"], state["w"], state["b"], eps=NORM_EPS)]
        y, stats = layernorm.layer_norm_forward(state["x"], state["w"], state["b"], eps=NORM_EPS)
        dx, dw, db = layernorm.layer_norm_backward(state["dy"], state["x"], stats, state["w"])
        return [y, dx, dw, db]
    # over the limit: into views of the flat buffers; within it: in place
    norm, _ = gradients.clip_grad_norm(state["grads"], state["limit"], eps=CLIP_EPS, out=state["out"])
    return [norm] + list(state["flat"].values())


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _kept(g, rows):
    """Which rows are tokens: now and then one is padding."""
    return (torch.rand(rows, 1, generator=g, device="cuda") > 1 / 64).float()


def _activations(g, rows, cols, kind):
    """Normal values off zero, some channels far larger than others, padding zero."""
    x = (_normal(g, rows, cols) + 0.5) * torch.exp(_normal(g, 1, cols))
    return (x * _kept(g, rows)).to(kind)


def _rows16(q):
    """The codes in rows of a multiple of 16 bytes, as the quantiser lays them out."""
    wide = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=torch.int8, device=q.device)
    wide[:, : q.shape[1]] = q
    return wide[:, : q.shape[1]]


def _operand(x):
    q, s = _quantize(x)
    return _rows16(q), s


def _bias(g, case, n):
    return None if case["bias"] == "none" else _normal(g, n).to(TYPES[case["bias"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "quantize":
        state["x"] = _activations(g, case["rows"], case["cols"], TYPES[case["type"]])
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        state["a"] = _operand(_activations(g, m, k, torch.bfloat16))
        state["b"] = _operand(_normal(g, n, k) / math.sqrt(k))
        state["bias"] = _bias(g, case, n)
    elif case["op"] == "linear":
        i, o = case["inputs"], case["outputs"]
        state["x"] = _activations(g, case["tokens"], i, TYPES[case["type"]])
        state["w"] = _operand(_normal(g, o, i) / math.sqrt(i))
        state["bias"] = _bias(g, case, o)
    elif case["op"] == "norm":
        rows, cols, kind = case["rows"], case["cols"], TYPES[case["type"]]
        kept = _kept(g, rows)  # padding has neither values nor gradients
        state["x"] = ((_normal(g, rows, cols) + _normal(g, rows, 1)) * torch.exp(_normal(g, 1, cols)) * kept).to(kind)
        state["w"], state["b"] = (1 + _normal(g, cols) / 4).to(TYPES[case["params"]]), (_normal(g, cols) / 4).to(TYPES[case["params"]])
        if case["train"]:
            state["dy"] = (_normal(g, rows, cols) * torch.exp(_normal(g, rows, 1)) * 1e-3 * kept).to(kind)
    else:
        sizes = _tensors(case)
        flat = {TYPES[k]: torch.zeros(sum(n for n, t in sizes if t == k), dtype=TYPES[k], device="cuda") for k in TYPES if any(t == k for _, t in sizes)}
        views, at = [], dict.fromkeys(flat, 0)
        for n, t in sizes:
            kind = TYPES[t]
            views.append(flat[kind][at[kind]:at[kind] + n])
            at[kind] += n
        values = [(_normal(g, n) * math.exp(2 * random.Random("%d %d" % (seed, i)).random() - 1) * 1e-2).to(TYPES[t]) for i, (n, t) in enumerate(sizes)]
        norm = math.sqrt(sum(float(v.double().square().sum()) for v in values))
        state["flat"], state["limit"] = flat, norm / 3 if case["over"] else norm * 3
        if not case["over"]:  # the gradients lie in the flat buffers and stay there
            for view, v in zip(views, values):
                view.copy_(v)
            values = views
        state["grads"], state["out"] = values, views
    return state


# --------------------------------------------------------------------- work

def _bytes(kind):
    return 0 if kind == "none" else 4 if kind == "f32" else 2


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (_bytes(case["type"]) + 1) + 4 * r, "flops": 2 * r * c}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + n * _bytes(case["bias"]) + m * n * _bytes(case["type"]), "flops": 2 * m * n * k}
    if case["op"] == "linear":
        t, i, o = case["tokens"], case["inputs"], case["outputs"]
        return {"bytes": (t * i + t * o) * _bytes(case["type"]) + o * i + 4 * o + o * _bytes(case["bias"]), "flops": 2 * t * i * o}
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        size, params = r * c * _bytes(case["type"]), c * _bytes(case["params"])
        if not case["train"]:
            return {"bytes": 2 * size + 2 * params, "flops": 8 * r * c}
        return {"bytes": 4 * size + 2 * params + 8 * c, "flops": 24 * r * c}
    sizes = _tensors(case)
    read = sum(n * _bytes(t) for n, t in sizes)
    return {"bytes": 2 * read if case["over"] else read, "flops": (3 if case["over"] else 2) * sum(n for n, _ in sizes)}


# -------------------------------------------------------------------- exact

def _codes64(x):
    """(codes, scales) from the definition: a code is the number of borders between codes that |x| / s lies beyond."""
    size = x.double().abs()
    top = size.max(dim=1, keepdim=True).values
    s = (torch.where(top < AMAX_FLOOR, torch.full_like(top, AMAX_FLOOR), top) / 127.0).to(torch.float32)
    borders = torch.arange(127, dtype=torch.float64, device=x.device) + 0.5
    t = (size / s.double()).contiguous()
    low, high = torch.searchsorted(borders, t), torch.searchsorted(borders, t, right=True)  # they differ on a border
    k = torch.where(low % 2 == 0, low, high)
    return torch.where(x < 0, -k, k).to(torch.int8), s[:, 0]


def _exact_product(a, sa, b, sb, bias):
    d = torch.mm(a.double() * sa.double()[:, None], (b.double() * sb.double()[:, None]).T.contiguous())
    return d if bias is None else d + bias.double()


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return list(_codes64(state["x"]))
    if case["op"] == "gemm":
        return _exact_product(*state["a"], *state["b"], state["bias"])
    if case["op"] == "linear":
        return _exact_product(*_codes64(state["x"]), *state["w"], state["bias"])
    if case["op"] == "norm":  # the gradients by differentiating the forward pass
        x, w, b = (state[k].double().requires_grad_(case["train"]) for k in ("x", "w", "b"))
        centred = x - x.sum(dim=1, keepdim=True) / x.shape[1]
        y = centred * torch.rsqrt((centred * centred).sum(dim=1, keepdim=True) / x.shape[1] + NORM_EPS) * w + b
        if not case["train"]:
            return [y]
        return [y.detach(), *torch.autograd.grad(y, (x, w, b), state["dy"].double())]
    total = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in state["grads"]))
    factor = min(1.0, state["limit"] / (total + CLIP_EPS))
    out = [torch.cat([g.double() * factor for g in state["grads"] if g.dtype == kind]) for kind in state["flat"]]
    return [torch.tensor(total, dtype=torch.float64), *out]
