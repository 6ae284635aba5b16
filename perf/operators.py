"""Performance cases of the operators of a quantized layer's training and serving.

The operators, by the functions of ``differentiable_bcjr_amd`` that compute them:

* ``fp8_block_quantize``: a matrix in 8-bit floating point (e4m3) with one float32 scale for each block of 128;
* ``fp8_block_matmul``: a b^T of two such matrices;
* ``fp8_linear`` and ``fp8_linear_quantized``: a linear layer on that product, trained (forward and both gradients) or
  served with weights that were quantized once;
* ``orthogonalize``: an update of a weight matrix, orthogonalized by Newton-Schulz products.

``run`` computes a case by its plain form (``own`` false) or by the package's calls (``own`` true).  Matrices stand for
the projections of a transformer block of width 2048 with a hidden width of 8192 and key and value widths of 512.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
BLOCK = 128
NS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # activations of 8192 tokens on their way into a projection, rows alone (serving a prompt)
        {"name": "quantize_activations", "op": "quantize", "rows": 8192, "cols": 2048, "type": "bf16", "block_rows": 1,
         "transposed": False},
        # a float32 soft codeword of the largest projection: square blocks, with the transpose that the backward reads
        {"name": "quantize_weights", "op": "quantize", "rows": 8192, "cols": 2048, "type": "fp32", "block_rows": 128,
         "transposed": True},
        # a ragged batch of tokens, both orientations in one pass (training), sizes that fill no block
        {"name": "quantize_ragged_both", "op": "quantize", "rows": 1237, "cols": 2041, "type": "bf16", "block_rows": 1,
         "transposed": True},
        # one token against the largest projection: latency and the weights' bytes
        {"name": "matmul_one_token", "op": "matmul", "m": 1, "n": 8192, "k": 2048, "out": "bf16", "b_rows": 128},
        # a few hundred ragged rows with an odd reduction length and a scale for each row of both sides
        {"name": "matmul_ragged", "op": "matmul", "m": 517, "n": 2000, "k": 1931, "out": "fp32", "b_rows": 1},
        # a whole prompt against the largest projection: the matrix cores' rate
        {"name": "matmul_prompt", "op": "matmul", "m": 8192, "n": 8192, "k": 2048, "out": "bf16", "b_rows": 128},
        # decoding one token through the narrow projection, quantizing the token on the way
        {"name": "linear_one_token", "op": "serve", "m": 1, "n": 512, "k": 2048, "type": "bf16"},
        # decoding a batch of 16 tokens through the widest projection
        {"name": "linear_16_tokens", "op": "serve", "m": 16, "n": 2048, "k": 8192, "type": "bf16"},
        # a training step of the largest projection
        {"name": "linear_train", "op": "train", "m": 8192, "n": 8192, "k": 2048, "type": "bf16"},
        # a training step of a narrow projection on a ragged batch
        {"name": "linear_train_ragged", "op": "train", "m": 1000, "n": 512, "k": 2048, "type": "bf16"},
        # the float32 update of the largest projection
        {"name": "orthogonalize_large", "op": "orthogonalize", "batch": 1, "rows": 8192, "cols": 2048, "type": "fp32"},
        # a stack of bfloat16 updates of the narrow projection, one for each of four layers
        {"name": "orthogonalize_stack", "op": "orthogonalize", "batch": 4, "rows": 512, "cols": 2048, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "matmul", "matmul", "serve", "train", "orthogonalize", "orthogonalize"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 16, 2048), "type": rng.choice(list(TYPES)),
                "block_rows": rng.choice([1, 128]), "transposed": rng.random() < 0.5}
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 8192), "k": _log(rng, 64, 2048),
                "out": rng.choice(list(TYPES)), "b_rows": rng.choice([1, 128])}
    if op == "serve":
        return {"op": op, "m": _log(rng, 1, 64), "n": _log(rng, 256, 8192), "k": _log(rng, 256, 8192),
                "type": rng.choice(list(TYPES))}
    if op == "train":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 8192), "k": _log(rng, 64, 2048),
                "type": rng.choice(list(TYPES))}
    batch = rng.choice([1, 1, 2, 3])
    rows, cols = _log(rng, 16, 8192 // batch), _log(rng, 16, 2048)
    if rng.random() < 0.5:
        rows, cols = cols, rows
    return {"op": op, "batch": batch, "rows": rows, "cols": cols, "type": rng.choice(list(TYPES))}


# ---------------------------------------------------------------- inputs


def _activations(g, rows, cols):
    """Activations: token rows of different sizes, and a few channels far above the rest."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
    loud = torch.rand(cols, generator=g, device=DEV) < 0.005
    return x * torch.where(loud, 20.0, 1.0)


def _weights(g, rows, cols):
    return torch.randn(rows, cols, generator=g, device=DEV) / math.sqrt(cols)


def _gradients(g, rows, cols):
    """Upstream gradients: small, each token's with its own size."""
    y = torch.randn(rows, cols, generator=g, device=DEV) * 1e-3
    return y * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))


def _update(g, batch, rows, cols):
    """A momentum buffer: a few strong directions over noise."""
    r = max(1, min(rows, cols) // 16)
    u = torch.randn(batch, rows, r, generator=g, device=DEV)
    v = torch.randn(batch, r, cols, generator=g, device=DEV)
    low = torch.stack([u[i] @ v[i] for i in range(batch)])
    return 1e-3 * (low / math.sqrt(r) + torch.randn(batch, rows, cols, generator=g, device=DEV))


def _held(q, scale):
    """Codes and scales as the package hands them out: the codes' rows on 16-byte boundaries, the scales block by
    block."""
    rows, cols = q.shape
    room = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=q.device)
    room[:, :cols] = q.view(torch.uint8)
    return room.view(E4M3)[:, :cols], scale.t().contiguous().t()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        make = _weights if case["block_rows"] == 128 else _activations
        s["x"] = make(g, case["rows"], case["cols"]).to(TYPES[case["type"]])
    elif op == "matmul":
        s["a"] = _held(*_codes(_activations(g, case["m"], case["k"]), 1))
        s["b"] = _held(*_codes(_weights(g, case["n"], case["k"]), case["b_rows"]))
    elif op == "serve":
        s["x"] = _activations(g, case["m"], case["k"]).to(TYPES[case["type"]])
        s["w"] = _held(*_codes(_weights(g, case["n"], case["k"]), 128))
    elif op == "train":
        t = TYPES[case["type"]]
        s["x"] = _activations(g, case["m"], case["k"]).to(t).requires_grad_(True)
        s["w"] = _weights(g, case["n"], case["k"]).requires_grad_(True)
        s["dy"] = _gradients(g, case["m"], case["n"]).to(t)
    else:
        s["g"] = _update(g, case["batch"], case["rows"], case["cols"]).to(TYPES[case["type"]])
    return s


# ---------------------------------------------------------------- plain forms


def _blocks(x, block_rows):
    """x [rows, cols] zero-padded to whole blocks, as [row blocks, block_rows, column blocks, 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block_rows))
    return x.view(x.shape[0] // block_rows, block_rows, x.shape[1] // BLOCK, BLOCK)


def _codes(x, block_rows):
    """(codes [rows, cols], scales [row blocks, column blocks]): scale = max(amax / 448, 2^-126), code = x / scale."""
    rows, cols = x.shape
    b = _blocks(x.float(), block_rows)
    scale = (b.abs().amax(dim=(1, 3)) * (1.0 / 448.0)).clamp_min(2.0 ** -126)
    q = (b * (1.0 / scale)[:, None, :, None]).to(E4M3)
    return q.view(torch.uint8).view(b.shape[0] * block_rows, -1)[:rows, :cols].contiguous().view(E4M3), scale


def _values(q, scale, block_rows):
    """The float32 values that codes and scales stand for."""
    rows, cols = q.shape
    v = q.float() * scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    return v


def _rounded(x, block_rows):
    return _values(*_codes(x, block_rows), block_rows)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        x, r = s["x"], case["block_rows"]
        out = list(_codes(x, r))
        if case["transposed"]:
            out += list(_codes(x.t(), r))
        return out
    if op == "matmul":
        a, b = _values(*s["a"], 1), _values(*s["b"], case["b_rows"])
        return (a @ b.t()).to(TYPES[case["out"]])
    if op == "serve":
        return (_rounded(s["x"], 1) @ _values(*s["w"], 128).t()).to(s["x"].dtype)
    if op == "train":
        x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
        wq = _rounded(w, 128)
        y = _rounded(x, 1) @ wq.t()
        dx = _rounded(dy, 1) @ wq
        dw = _rounded(dy.t(), 1) @ _rounded(x.t(), 1).t()
        return y.to(x.dtype), dx.to(x.dtype), dw
    g = s["g"]
    a, b, c = NS
    x = g.float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / (x.double().square().sum((-2, -1), keepdim=True).sqrt() + EPS).float()
    x = x.contiguous()
    for _ in range(5):
        gram = torch.bmm(x, x.transpose(-1, -2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return (x.transpose(-1, -2) if tall else x).to(g.dtype)


def run(s):
    if not own:
        return _plain(s)
    import differentiable_bcjr_amd as dba

    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        return dba.fp8_block_quantize(s["x"], block_rows=case["block_rows"], transposed=case["transposed"])
    if op == "matmul":
        return dba.fp8_block_matmul(*s["a"], *s["b"], out_dtype=TYPES[case["out"]])
    if op == "serve":
        return dba.fp8_linear_quantized(s["x"], *s["w"])
    if op == "train":
        y = dba.fp8_linear(s["x"], s["w"])
        dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
        return y, dx, dw
    return dba.orthogonalize(s["g"], steps=5, coefficients=NS, eps=EPS)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    up = lambda v: -(-v // BLOCK)  # noqa: E731
    if op == "quantize":
        m, k, r = case["rows"], case["cols"], case["block_rows"]
        sides = 2 if case["transposed"] else 1
        scales = (-(-m // r)) * up(k) + (up(m) * (-(-k // r)) if case["transposed"] else 0)
        return {"bytes": m * k * (BYTES[case["type"]] + sides) + 4 * scales, "flops": 2 * m * k}
    if op == "orthogonalize":
        m, n = sorted((case["rows"], case["cols"]))
        # the two symmetric products need half of their entries
        return {"bytes": 2 * case["batch"] * m * n * BYTES[case["type"]],
                "flops": case["batch"] * 5 * (m * m * n + m ** 3 + 2 * m * m * n)}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "matmul":
        scales = m * up(k) + (-(-n // case["b_rows"])) * up(k)
        return {"bytes": m * k + n * k + 4 * scales + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    e = BYTES[case["type"]]
    if op == "serve":
        return {"bytes": m * k * e + n * k + 4 * up(n) * up(k) + m * n * e, "flops": 2 * m * n * k}
    return {"bytes": 2 * m * k * e + 2 * m * n * e + 2 * n * k * 4, "flops": 6 * m * n * k}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_codes(x, block_rows):
    """Codes and scales by their definition: scales and quotients are float32 by definition, so each is rounded there;
    the rounding to e4m3 is done on its grid of steps, 2^-9 below 2^-6 and an eighth of the binade above."""
    x = x.detach().double()
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    full = x.new_zeros(rb * block_rows, cb * BLOCK)
    full[:rows, :cols] = x
    top = full.abs().reshape(rb, block_rows, cb, BLOCK).permute(0, 2, 1, 3).reshape(rb, cb, -1).max(-1).values
    part = torch.tensor(1.0 / 448.0, dtype=torch.float32, device=x.device).double()
    scale = torch.maximum((top * part).float().double(), torch.full_like(top, 2.0 ** -126))
    inverse = (1.0 / scale).float().double()
    spread = lambda t: t.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]  # noqa: E731
    v = (x * spread(inverse)).float().double()
    e = torch.frexp(v.abs())[1] - 1
    step = ((e.clamp_min(-6) - 3 + 1023).long() << 52).view(torch.float64)   # 2^(exponent - 3), by its bits
    return torch.round(v / step) * step, scale, spread(scale)


def _exact_rounded(x, block_rows):
    q, _, s = _exact_codes(x, block_rows)
    return q * s


def _exact_held(q, scale, block_rows):
    rows, cols = q.shape
    r = torch.arange(rows, device=q.device) // block_rows
    c = torch.arange(cols, device=q.device) // BLOCK
    return q.float().double() * scale.double()[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, r = s["x"], case["block_rows"]
        out = list(_exact_codes(x, r)[:2])
        if case["transposed"]:
            out += list(_exact_codes(x.t(), r)[:2])
        return out
    if op == "matmul":
        return torch.matmul(_exact_held(*s["a"], 1), _exact_held(*s["b"], case["b_rows"]).t())
    if op == "serve":
        return torch.matmul(_exact_rounded(s["x"], 1), _exact_held(*s["w"], 128).t())
    if op == "train":
        w = _exact_rounded(s["w"], 128)
        y = torch.matmul(_exact_rounded(s["x"], 1), w.t())
        dx = torch.matmul(_exact_rounded(s["dy"], 1), w)
        dw = torch.matmul(_exact_rounded(s["dy"].t(), 1), _exact_rounded(s["x"].t(), 1).t())
        return y, dx, dw
    a, b, c = NS
    found = []
    for g in s["g"].double():
        x = g if g.shape[0] <= g.shape[1] else g.t()
        x = x / (x.pow(2).sum().sqrt() + EPS)
        for _ in range(5):
            square = torch.matmul(x, x.t())
            x = a * x + b * torch.matmul(square, x) + c * torch.matmul(square, torch.matmul(square, x))
        found.append(x if g.shape[0] <= g.shape[1] else x.t())
    return torch.stack(found)
