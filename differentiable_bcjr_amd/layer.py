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


_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_lib = None


def _entry():
    global _lib
    if _lib is None:
        _lib = abi.load()
    return _lib


def _call(entry, index: int, *args) -> None:
    """An entry point of the library on device `index`'s current stream, with that device current."""
    if index == _device():
        status = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = entry(*args, _raw_stream(index))
    if status:
        _check(status)


def _type(dtype, name: str) -> int:
    if dtype not in _TYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {dtype}")
    return _TYPES[dtype]


def _up(v: int, of: int) -> int:
    return -(-v // of)


def _matrix(x, name: str):
    """(x, type, rows, columns, distance of rows) of a float matrix whose rows lie one after the other, any distance
    apart; a copy where they do not."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    t = _TYPES.get(x.dtype)
    if t is None:
        _type(x.dtype, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    (rows, cols), (ld, step) = x.shape, x.stride()
    if rows <= 1:
        ld = max(cols, 1)
    if cols > 1 and step != 1 or ld < cols:
        x, ld = x.contiguous(), max(cols, 1)
    return x, t, rows, cols, ld


def _new_codes(rows: int, cols: int, device):
    """[rows, cols] codes whose rows start on 16-byte boundaries, and their distance."""
    ld = (cols + 15) // 16 * 16 or 16
    return torch.empty_strided((rows, cols), (ld, 1), dtype=CODES, device=device), ld


def _new_scales(rows: int, cols: int, block_rows: int, device) -> torch.Tensor:
    """Scales of a matrix, column by column: a step of a product reads one column."""
    blocks = rows if block_rows == 1 else _up(rows, block_rows)
    return torch.empty_strided((blocks, (cols + 127) // 128), (1, blocks or 1), dtype=torch.float32, device=device)


def fp8_block_quantize(x: torch.Tensor, *, block_rows: int = 1, transposed: bool = False):
    """(q, scale) of a matrix x [M, K] (float32, bfloat16 or float16): e4m3 codes q [M, K] and float32 scales
    [ceil(M / block_rows), ceil(K / 128)], one for each block of 128 columns of one row (``block_rows=1``, activations
    and gradients) or of 128 rows (``block_rows=128``, weights).  q scale stands for x, with scale = amax / 448 (at
    least 2^-126).  With ``transposed`` also (q_t [K, M], scale_t [ceil(K / block_rows), ceil(M / 128)]) of the
    transpose, from the same pass over x.  An Inf or NaN makes the values of its block NaN.  Neither
    the codes nor the scales carry a gradient."""
    x, x_type, rows, cols, ld = _matrix(x, "x")
    if block_rows not in (1, BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    dev = x.device
    q, ld_q = _new_codes(rows, cols, dev)
    s = _new_scales(rows, cols, block_rows, dev)
    if not transposed:
        _call(_entry().fp8_block_quantize, dev.index, x.data_ptr(), x_type, rows, cols, ld, block_rows, q.data_ptr(),
              ld_q, s.data_ptr(), None, 0, None)
        return q, s
    q_t, ld_qt = _new_codes(cols, rows, dev)
    s_t = _new_scales(cols, rows, block_rows, dev)
    _call(_entry().fp8_block_quantize, dev.index, x.data_ptr(), x_type, rows, cols, ld, block_rows, q.data_ptr(), ld_q,
          s.data_ptr(), q_t.data_ptr(), ld_qt, s_t.data_ptr())
    return q, s, q_t, s_t


def _codes(q, name: str):
    """(q, rows, columns, distance of rows) of a matrix of codes whose rows lie on 16-byte boundaries; a copy where
    they do not."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype is not CODES:
        raise TypeError(f"{name} must be a float8_e4m3fn CUDA (HIP) tensor")
    if q.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    (rows, cols), (ld, step) = q.shape, q.stride()
    if rows <= 1:
        ld = (cols + 15) // 16 * 16 or 16
    if cols > 1 and step != 1 or ld % 16 or ld < cols or q.data_ptr() % 16:
        packed, ld = _new_codes(rows, cols, q.device)
        q = packed.copy_(q)
    return q, rows, cols, ld


def _scales(s, row_blocks: int, col_blocks: int, like: torch.Tensor, name: str) -> torch.Tensor:
    """The scales of a matrix on `like`'s device, column by column; a copy where they lie otherwise."""
    if not isinstance(s, torch.Tensor) or s.dtype is not torch.float32:
        raise TypeError(f"{name} must be a float32 CUDA (HIP) tensor")
    if s.device != like.device:
        raise ValueError(f"tensors must be on one device, not {like.device} and {s.device}")
    if s.shape != (row_blocks, col_blocks):
        raise ValueError(f"{name} must have shape {(row_blocks, col_blocks)}, not {tuple(s.shape)}")
    along, across = s.stride()
    if (row_blocks > 1 and along != 1) or (col_blocks > 1 and across != row_blocks):
        s = s.t().contiguous().t()
    return s


def _weights(q, s, name: str):
    """(q, rows, columns, distance of rows, scales, rows of a block) of a product's second operand: its scales' shape
    says whether a block is 128 rows or one."""
    q, rows, cols, ld = _codes(q, name)
    if not isinstance(s, torch.Tensor) or s.dim() != 2:
        raise TypeError(f"{name}_scale must be a float32 CUDA (HIP) matrix")
    square = (rows + 127) // 128
    if s.shape[0] == square:
        return q, rows, cols, ld, _scales(s, square, (cols + 127) // 128, q, name + "_scale"), BLOCK
    return q, rows, cols, ld, _scales(s, rows, (cols + 127) // 128, q, name + "_scale"), 1


def fp8_block_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, *,
                     out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a b^T [M, N] of two block-quantized matrices a [M, K] and b [N, K] (see ``fp8_block_quantize``).  a_scale is
    [M, ceil(K / 128)]; b_scale is [ceil(N / 128), ceil(K / 128)] or [N, ceil(K / 128)].  A float32 result comes from
    exact products summed in float32; for a 16-bit result the 8-bit matrix instruction sums the products of a block, with
    an error under the result's own rounding."""
    out_type = _type(out_dtype, "out_dtype")
    a, m, k, ld_a = _codes(a, "a")
    b, n, k_b, ld_b, b_scale, b_rows = _weights(b, b_scale, "b")
    if k != k_b:
        raise ValueError(f"a and b must have rows of one length, not {k} and {k_b}")
    a_scale = _scales(a_scale, m, (k + 127) // 128, a, "a_scale")
    dev = a.device
    if b.device != dev:
        raise ValueError(f"tensors must be on one device, not {dev} and {b.device}")
    out = torch.empty((m, n), dtype=out_dtype, device=dev)
    _call(_entry().fp8_block_matmul, dev.index, a.data_ptr(), ld_a, a_scale.data_ptr(), b.data_ptr(), ld_b,
          b_scale.data_ptr(), b_rows, m, n, k, out.data_ptr(), out_type, n or 1)
    return out


def _tokens(x, k: int, w: torch.Tensor):
    """_matrix of x [..., k] as rows, on w's device."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA (HIP) tensor")
    if x.dim() < 1 or x.shape[-1] != k:
        raise ValueError(f"x must be [..., {k}], not {tuple(x.shape)}")
    if x.device != w.device:
        raise ValueError(f"tensors must be on one device, not {x.device} and {w.device}")
    return _matrix(x if x.dim() == 2 else x.reshape(x.shape[:-1].numel(), k), "x")


def fp8_linear_quantized(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor) -> torch.Tensor:
    """y [..., N] = x w^T in x's type, for weights w [N, K] quantized before (``fp8_block_quantize(weights,
    block_rows=128)``); x [..., K] is quantized on the way, a scale for each 128 of a row.  It has no gradient (``fp8_linear`` has): an x that asks for
    one is refused unless gradients are off."""
    w, n, k, ld_w, w_scale, b_rows = _weights(w, w_scale, "w")
    rows, x_type, m, _, ld_x = _tokens(x, k, w)
    _no_gradient(x, "fp8_linear_quantized")
    dev, lib = w.device, _entry()
    y = torch.empty((m, n) if x.dim() == 2 else (*x.shape[:-1], n), dtype=x.dtype, device=dev)
    need = lib.fp8_linear_quantized_workspace_bytes(m, k)
    ws = _bytes(need, dev)
    _call(lib.fp8_linear_quantized, dev.index, rows.data_ptr(), x_type, m, ld_x, w.data_ptr(), ld_w, w_scale.data_ptr(),
          b_rows, n, k, y.data_ptr(), n or 1, _ptr(ws), need)
    return y


def _no_gradient(x, name: str) -> None:
    if x.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no gradient: call it under torch.no_grad() or on a detached tensor")


def _bytes(n: int, device) -> torch.Tensor | None:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _linear_forward(x, w, grads: int):
    """(y, what the backward of `grads` needs): x [..., K] and w [N, K]."""
    w, w_type, n, k, ld_w = _matrix(w, "w")
    rows, x_type, m, _, ld_x = _tokens(x, k, w)
    dev, lib = w.device, _entry()
    y = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=dev)
    keep, need = lib.fp8_linear_saved_bytes(m, n, k, grads), lib.fp8_linear_workspace_bytes(m, n, k)
    saved, ws = _bytes(keep, dev), _bytes(need, dev)
    _call(lib.fp8_linear_forward, dev.index, rows.data_ptr(), x_type, m, ld_x, w.data_ptr(), w_type, n, ld_w, k, grads,
          y.data_ptr(), n or 1, _ptr(saved), keep, _ptr(ws), need)
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
        rows, dy_type, m, _, ld_dy = _tokens(dy, n, dy)
        dev, lib = dy.device, _entry()
        dx = torch.empty(x_shape, dtype=x_type, device=dev) if grads & abi.BCJR_GRAD_X else None
        dw = torch.empty((n, k), dtype=w_type, device=dev) if grads & abi.BCJR_GRAD_W else None
        need = lib.fp8_linear_workspace_bytes(m, n, k)
        ws = _bytes(need, dev)
        _call(lib.fp8_linear_backward, dev.index, rows.data_ptr(), dy_type, m, ld_dy, n, k, grads, _ptr(saved),
              0 if saved is None else saved.numel(), _ptr(dx), k or 1, _ptr(dw), _TYPES[w_type], k or 1, _ptr(ws),
              need)
        return dx, dw


def fp8_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """y [..., N] = x w^T in x's type as a differentiable function of x [..., K] and w [N, K], every product in 8 bits:
    x and the upstream gradient are quantized with a scale for each 128 along the sum they enter, w with one for each
    128 x 128.  dx has x's type and dw has w's.  w may be the soft codeword (``soft_quantize``) of a layer's weights."""
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise TypeError("x and w must be CUDA (HIP) tensors")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return _Fp8Linear.apply(x, w)
    return _linear_forward(x, w, 0)[0]


def orthogonalize(g: torch.Tensor, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """The matrices of g [..., rows, cols] with their singular values brought near 1, by ``steps`` Newton-Schulz steps
    X <- a X + (b A + c A A) X, A = X X^T, from X = g / (|g|_F + eps) (on the transpose where rows > cols).  The result
    has g's type or ``out_dtype``: float32 and float16 are computed like float32 products, bfloat16 of more than 256 rows
    and columns with operands rounded to 11 bits.  It has no gradient: a g that asks for one is refused unless gradients
    are off."""
    if not isinstance(g, torch.Tensor) or not g.is_cuda:
        raise TypeError("g must be a CUDA (HIP) tensor")
    in_type, out_dtype = _type(g.dtype, "g"), out_dtype or g.dtype
    out_type = _type(out_dtype, "out_dtype")
    if g.dim() < 2:
        raise ValueError("g must have at least two dimensions")
    _no_gradient(g, "orthogonalize")
    a, b, c = (float(v) for v in coefficients)
    out = torch.empty(g.shape, dtype=out_dtype, device=g.device)
    if out.numel() == 0:
        return out
    rows, cols = g.shape[-2:]
    g3 = g if g.dim() == 3 else g.reshape(-1, rows, cols)
    if (cols > 1 and g3.stride(2) != 1 or rows > 1 and g3.stride(1) < cols
            or g3.shape[0] > 1 and g3.stride(0) < 0):
        g3 = g3.contiguous()
    batch, (_, ld, _) = g3.shape[0], g3.stride()
    dev, lib = g.device, _entry()
    need = lib.orthogonalize_workspace_bytes(batch, rows, cols, out_type)
    ws = _bytes(need, dev)
    _call(lib.orthogonalize, dev.index, g3.data_ptr(), in_type, batch, rows, cols, ld if rows > 1 else cols,
          g3.stride(0) if batch > 1 else 0, int(steps), a, b, c, float(eps), out.data_ptr(), out_type, _ptr(ws), need)
    return out
