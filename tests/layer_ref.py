"""The quantized layer's operators in 64 bits, elementary and slow, for the tests (CPU tensors)."""
import torch

E4M3 = torch.float8_e4m3fn
BLOCK = 128


def quantize(x, block_rows):
    """(q as e4m3, scale float32) by the definition: scale = max(fl(amax fl(1/448)), 2^-126), q = e4m3(fl(x fl(1/scale))).
    The product of two float32 numbers is exact in 64 bits, so rounding it there gives the float32 product."""
    x = x.double()
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    part = torch.tensor(1.0 / 448.0, dtype=torch.float32).double()
    pad = torch.zeros(rb * block_rows, cb * BLOCK, dtype=torch.float64)
    pad[:rows, :cols] = x
    top = pad.view(rb, block_rows, cb, BLOCK).abs().amax(dim=(1, 3))
    scale = (top * part).float()
    scale = torch.where(scale < 2.0 ** -126, torch.full_like(scale, 2.0 ** -126), scale)
    inv = (1.0 / scale.double()).float().double()
    spread = inv.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    return (x * spread).float().to(E4M3), scale


def values(q, scale, block_rows):
    rows, cols = q.shape
    return q.float().double() * scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def matmul_bound(av, bv, out_dtype):
    """(a b^T in 64 bits, the largest error of each entry).

    A block of 128 is summed in float32 (at most 128 roundings, taken as a whole unit 2^-23 each, as if they cut), then
    scaled and added (three roundings a block), then rounded once to the result's type.  A 16-bit result comes from the
    8-bit matrix instruction, which aligns the products of 8 neighbouring codes to the one with the largest exponent and
    cuts each 13 bits below that exponent: at most 2^-13 of the group's largest product for each of its 8 (the groups
    are cut where the kernel may cut them, so every run of 16 codes is taken as two groups with its largest)."""
    k = av.shape[1]
    ref = av @ bv.t()
    size = av.abs() @ bv.abs().t()
    blocks = -(-k // BLOCK)
    # numbers under the type's smallest normal are spaced by tiny * eps
    bound = (128 + 3 * blocks) * 2.0 ** -23 * size + torch.finfo(out_dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -8) + \
        torch.finfo(out_dtype).tiny * torch.finfo(out_dtype).eps
    if out_dtype != torch.float32:
        for k0 in range(0, k, 16):
            top = torch.zeros_like(ref)
            for i in range(k0, min(k0 + 16, k)):
                top = torch.maximum(top, av[:, i:i + 1].abs() * bv[:, i].abs())
            bound += 16 * 2.0 ** -13 * top
    return ref, bound


def newton_schulz(g, steps, coefficients, eps):
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        s = x @ x.t()
        x = a * x + (b * s + c * s @ s) @ x
    return x.t() if tall else x


def newton_schulz_rounded(g, steps, coefficients, eps, split):
    """The iteration with float32 products of operands rounded as the library documents: to the sum of two halves
    (split), or to one half with X itself kept as the sum of two and b + c taken off B's diagonal in the last step."""
    a, b, c = coefficients

    def half(v):
        return v.half().float()

    def two(v):
        return half(v) + half(v - half(v))

    op = two if split else half
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = two((x / (x.square().sum().sqrt() + eps)).float() * 1024)
    for i in range(steps):
        s = op(op(x) @ op(x).t() * (256 / 1024 ** 2))
        mu = 0.0 if split or i + 1 < steps else b + c
        p = op(b * s + s @ s * (c / 256) - mu * 256 * torch.eye(s.shape[0]))
        x = (a + mu) * x + p @ op(x) * (1 / 256)
        x = two(x) if i + 1 < steps else x
    x = x / 1024
    return x.t() if tall else x
