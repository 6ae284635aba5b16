"""A linear layer with quantized weights, and the update of its weights.

The soft codeword (while training) and the hard code (at the end) are the weights of a linear layer.  The functions here
run that layer on the 8-bit matrix cores and turn the gradient of the weights into an update:

* ``fp8_block_quantize``   -- a matrix as e4m3 codes with a float32 scale for each block of 128, and its transpose;
* ``fp8_block_matmul``     -- a b^T of two such matrices;
* ``fp8_linear``           -- y = x w^T on that product as a differentiable function of x and w;
* ``fp8_linear_quantized`` -- the same for weights that were quantized once (serving);
* ``orthogonalize``        -- Newton-Schulz orthogonalization of an update (the direction the Muon optimizer takes).

They marshal arguments for the entry points of ``include/bcjr.h``: tensors are checked, inputs that do not lie as the
library reads them are copied, and outputs and workspaces come from torch on the inputs' device and current stream.
"""
from __future__ import annotations

import torch

from . import BCJRError, _check, _ptr, abi   # noqa: F401  (BCJRError: what _check raises)

__all__ = ["fp8_block_quantize", "fp8_block_matmul", "fp8_linear", "fp8_linear_quantized", "orthogonalize"]

BLOCK = 128
CODES = torch.float8_e4m3fn
_TYPES = {torch.float32: abi.BCJR_TYPE_F32, torch.bfloat16: abi.BCJR_TYPE_BF16, torch.float16: abi.BCJR_TYPE_F16}


def _type(dtype, name: str) -> int:
    if dtype not in _TYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {dtype}")
    return _TYPES[dtype]


def _matrix(x, name: str) -> torch.Tensor:
    """A float matrix whose rows lie one after the other (any distance apart); copied where they do not."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    _type(x.dtype, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if x.shape[1] > 1 and x.stride(1) != 1 or x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        x = x.contiguous()
    return x


def _row_distance(x: torch.Tensor) -> int:
    return x.stride(-2) if x.shape[-2] > 1 else max(x.shape[-1], 1)


def _up(v: int, of: int) -> int:
    return -(-v // of)


def _call(entry, device, *args) -> None:
    """An entry point of the library on `device`'s current stream, with `device` current."""
    index = device.index
    if index == torch.cuda.current_device():
        _check(entry(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(device):
            _check(entry(*args, torch._C._cuda_getCurrentRawStream(index)))


def _new_codes(rows: int, cols: int, device) -> torch.Tensor:
    """[rows, cols] codes whose rows start on 16-byte boundaries."""
    if cols % 16 == 0:
        return torch.empty((rows, cols), dtype=CODES, device=device)
    return torch.empty((rows, _up(cols, 16) * 16), dtype=CODES, device=device)[:, :cols]


def _new_scales(row_blocks: int, col_blocks: int, device) -> torch.Tensor:
    """[row_blocks, col_blocks] scales that lie column by column: a step of a product reads one column."""
    return torch.empty((col_blocks, row_blocks), dtype=torch.float32, device=device).t()


def _quantize(x: torch.Tensor, block_rows: int, transposed: bool):
    rows, cols = x.shape
    dev = x.device
    q, s = _new_codes(rows, cols, dev), _new_scales(_up(rows, block_rows), _up(cols, BLOCK), dev)
    q_t = s_t = None
    if transposed:
        q_t, s_t = _new_codes(cols, rows, dev), _new_scales(_up(cols, block_rows), _up(rows, BLOCK), dev)
    _call(abi.load().fp8_block_quantize, dev, x.data_ptr(), _TYPES[x.dtype], rows, cols, _row_distance(x), block_rows,
          q.data_ptr(), _up(cols, 16) * 16, s.data_ptr(), _ptr(q_t), _up(rows, 16) * 16, _ptr(s_t))
    return (q, s, q_t, s_t) if transposed else (q, s)


def fp8_block_quantize(x: torch.Tensor, *, block_rows: int = 1, transposed: bool = False):
    """(q, scale) of a matrix x [M, K] (float32, bfloat16 or float16): e4m3 codes q [M, K] and float32 scales
    [ceil(M / block_rows), ceil(K / 128)], one for each block of 128 columns of one row (``block_rows=1``, activations
    and gradients) or of 128 rows (``block_rows=128``, weights).  q scale stands for x, with scale = amax / 448 (at
    least 2^-126).  With ``transposed`` also (q_t [K, M], scale_t [ceil(K / block_rows), ceil(M / 128)]) of the
    transpose, from the same pass over x.  An Inf or NaN makes the values of its block NaN."""
    x = _matrix(x, "x")
    if block_rows not in (1, BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    return _quantize(x, block_rows, transposed)


def _codes(q, name: str) -> torch.Tensor:
    """Codes whose rows lie on 16-byte boundaries; copied where they do not."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype != CODES:
        raise TypeError(f"{name} must be a float8_e4m3fn CUDA (HIP) tensor")
    if q.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, cols = q.shape
    if (cols > 1 and q.stride(1) != 1 or q.data_ptr() % 16
            or rows > 1 and (q.stride(0) % 16 or q.stride(0) < cols)):
        q = _new_codes(rows, cols, q.device).copy_(q)
    return q


def _code_distance(q: torch.Tensor) -> int:
    return q.stride(0) if q.shape[0] > 1 else _up(max(q.shape[1], 1), 16) * 16


def _scales(s, q: torch.Tensor, block_rows: int, name: str) -> torch.Tensor:
    shape = (_up(q.shape[0], block_rows), _up(q.shape[1], BLOCK))
    if not isinstance(s, torch.Tensor) or not s.is_cuda or s.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 CUDA (HIP) tensor")
    if s.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(s.shape)}")
    if (shape[0] == 1 or s.stride(0) == 1) and (shape[1] == 1 or s.stride(1) == shape[0]):
        return s
    return s.t().contiguous().t()


def _weight_block(q, s, name: str) -> int:
    """128 or 1, by which of the two shapes of scales `s` has for the codes `q`."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or not isinstance(s, torch.Tensor) or s.dim() != 2:
        raise TypeError(f"{name} and its scale must be matrices")
    return BLOCK if s.shape[0] == _up(q.shape[0], BLOCK) else 1


def _same_device(first, *others) -> None:
    for t in others:
        if t.device != first.device:
            raise ValueError(f"tensors must be on one device, not {first.device} and {t.device}")


def _matmul(a, a_scale, b, b_scale, b_rows: int, out_dtype) -> torch.Tensor:
    (m, k), n = a.shape, b.shape[0]
    out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _call(abi.load().fp8_block_matmul, a.device, a.data_ptr(), _code_distance(a), a_scale.data_ptr(), b.data_ptr(),
          _code_distance(b), b_scale.data_ptr(), b_rows, m, n, k, out.data_ptr(), _TYPES[out_dtype], max(n, 1))
    return out


def fp8_block_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, *,
                     out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a b^T [M, N] of two block-quantized matrices a [M, K] and b [N, K] (see ``fp8_block_quantize``).  a_scale is
    [M, ceil(K / 128)]; b_scale is [ceil(N / 128), ceil(K / 128)] or [N, ceil(K / 128)].  Blocks are summed in float32
    and joined in float32."""
    _type(out_dtype, "out_dtype")
    a, b_rows, b = _codes(a, "a"), _weight_block(b, b_scale, "b"), _codes(b, "b")
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"a and b must have rows of one length, not {a.shape[1]} and {b.shape[1]}")
    a_scale, b_scale = _scales(a_scale, a, 1, "a_scale"), _scales(b_scale, b, b_rows, "b_scale")
    _same_device(a, a_scale, b, b_scale)
    return _matmul(a, a_scale, b, b_scale, b_rows, out_dtype)


def _tokens(x, k: int) -> torch.Tensor:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA (HIP) tensor")
    if x.dim() < 1 or x.shape[-1] != k:
        raise ValueError(f"x must be [..., {k}], not {tuple(x.shape)}")
    if x.dim() != 2:
        x = x.reshape(x.shape[:-1].numel(), k)
    return _matrix(x, "x")


def fp8_linear_quantized(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor) -> torch.Tensor:
    """y [..., N] = x w^T in x's type, for weights w [N, K] quantized before (``fp8_block_quantize(weights,
    block_rows=128)``); x [..., K] is quantized on the way, a scale for each 128 of a row."""
    b_rows, w = _weight_block(w, w_scale, "w"), _codes(w, "w")
    w_scale = _scales(w_scale, w, b_rows, "w_scale")
    n, k = w.shape
    rows = _tokens(x, k)
    _same_device(x, w, w_scale)
    m, dev, lib = rows.shape[0], x.device, abi.load()
    y = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=dev)
    need = lib.fp8_linear_quantized_workspace_bytes(m, k)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(lib.fp8_linear_quantized, dev, rows.data_ptr(), _TYPES[x.dtype], m, _row_distance(rows), w.data_ptr(),
          _code_distance(w), w_scale.data_ptr(), b_rows, n, k, y.data_ptr(), max(n, 1), _ptr(ws), need)
    return y


def _bytes(n: int, device) -> torch.Tensor | None:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _linear_forward(x, w, grads: int):
    """(y, what the backward of `grads` needs): x [..., K] and w [N, K]."""
    n, k = w.shape
    rows = _tokens(x, k)
    m, dev, lib = rows.shape[0], x.device, abi.load()
    y = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=dev)
    keep, need = lib.fp8_linear_saved_bytes(m, n, k, grads), lib.fp8_linear_workspace_bytes(m, n, k)
    saved, ws = _bytes(keep, dev), _bytes(need, dev)
    _call(lib.fp8_linear_forward, dev, rows.data_ptr(), _TYPES[x.dtype], m, _row_distance(rows), w.data_ptr(),
          _TYPES[w.dtype], n, _row_distance(w), k, grads, y.data_ptr(), max(n, 1), _ptr(saved), keep, _ptr(ws), need)
    return y, saved


class _Fp8Linear(torch.autograd.Function):
    """y = Q(x) Q(w)^T; dx = Q(dy) Q(w), dw = Q(dy^T) Q(x^T)^T.  Only codes and scales are kept for the backward."""

    @staticmethod
    def forward(ctx, x, w):
        need_x, need_w = ctx.needs_input_grad
        grads = (abi.BCJR_GRAD_X if need_x else 0) | (abi.BCJR_GRAD_W if need_w else 0)
        y, saved = _linear_forward(x, w, grads)
        ctx.save_for_backward(saved)
        ctx.like = x.shape, x.dtype, w.shape, w.dtype, grads
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (saved,) = ctx.saved_tensors
        x_shape, x_type, (n, k), w_type, grads = ctx.like
        rows, dev, lib = _tokens(dy, n), dy.device, abi.load()
        m = rows.shape[0]
        dx = torch.empty(x_shape, dtype=x_type, device=dev) if grads & abi.BCJR_GRAD_X else None
        dw = torch.empty((n, k), dtype=w_type, device=dev) if grads & abi.BCJR_GRAD_W else None
        need = lib.fp8_linear_workspace_bytes(m, n, k)
        ws = _bytes(need, dev)
        _call(lib.fp8_linear_backward, dev, rows.data_ptr(), _TYPES[x_type], m, _row_distance(rows), n, k, grads,
              _ptr(saved), 0 if saved is None else saved.numel(), _ptr(dx), max(k, 1), _ptr(dw), _TYPES[w_type],
              max(k, 1), _ptr(ws), need)
        return dx, dw


def fp8_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """y [..., N] = x w^T in x's type as a differentiable function of x [..., K] and w [N, K], every product in 8 bits:
    x and the upstream gradient are quantized with a scale for each 128 along the sum they enter, w with one for each
    128 x 128.  dx has x's type and dw has w's.  w may be the soft codeword (``soft_quantize``) of a layer's weights."""
    w = _matrix(w, "w")
    _tokens(x, w.shape[1])
    _same_device(x, w)
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return _Fp8Linear.apply(x, w)
    return _linear_forward(x, w, 0)[0]


def orthogonalize(g: torch.Tensor, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """The matrices of g [..., rows, cols] with their singular values brought near 1, by ``steps`` Newton-Schulz steps
    X <- a X + (b A + c A A) X, A = X X^T, from X = g / (|g|_F + eps) (on the transpose where rows > cols).  The result
    has g's type or ``out_dtype``: float32 and float16 are computed like float32 products, bfloat16 with operands
    rounded to 11 bits."""
    if not isinstance(g, torch.Tensor) or not g.is_cuda:
        raise TypeError("g must be a CUDA (HIP) tensor")
    in_type, out_dtype = _type(g.dtype, "g"), out_dtype or g.dtype
    out_type = _type(out_dtype, "out_dtype")
    if g.dim() < 2:
        raise ValueError("g must have at least two dimensions")
    a, b, c = (float(v) for v in coefficients)
    out = torch.empty(g.shape, dtype=out_dtype, device=g.device)
    if out.numel() == 0:
        return out
    rows, cols = g.shape[-2:]
    g3 = g if g.dim() == 3 else g.reshape(-1, rows, cols)
    if (cols > 1 and g3.stride(2) != 1 or rows > 1 and g3.stride(1) < cols
            or g3.shape[0] > 1 and g3.stride(0) < 0):
        g3 = g3.contiguous()
    batch = g3.shape[0]
    need = abi.load().orthogonalize_workspace_bytes(batch, rows, cols, out_type)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=g.device)
    _call(abi.load().orthogonalize, g.device, g3.data_ptr(), in_type, batch, rows, cols, _row_distance(g3),
          g3.stride(0) if batch > 1 else 0, int(steps), a, b, c, float(eps), out.data_ptr(), out_type, ws.data_ptr(),
          need)
    return out
