"""Host-side checks of the quantized layer's C-ABI and Python entry points: every refusal comes before any HIP call, so
none of this needs a GPU."""
import pytest
import torch

import differentiable_bcjr_amd as dba
import layer_ref as ref
from differentiable_bcjr_amd import abi

P = 0x100000   # a 16-byte aligned non-NULL value; every call below fails a host check before it could be used
BIG = (1 << 30) + 1


def quantize(x=P, type=0, rows=8, cols=8, ld=8, block=1, q=P, ld_q=16, s=P, q_t=None, ld_qt=16, s_t=None):
    return abi.fp8_block_quantize(x, type, rows, cols, ld, block, q, ld_q, s, q_t, ld_qt, s_t, None)


def matmul(a=P, ld_a=16, a_s=P, b=P, ld_b=16, b_s=P, b_rows=1, m=8, n=8, k=8, out=P, type=0, ld_out=8):
    return abi.fp8_block_matmul(a, ld_a, a_s, b, ld_b, b_s, b_rows, m, n, k, out, type, ld_out, None)


def served(x=P, type=0, m=32, ld_x=16, w=P, ld_w=16, w_s=P, w_rows=128, n=8, k=16, out=P, ld_out=8, ws=P,
           size=1 << 30):
    return abi.fp8_linear_quantized(x, type, m, ld_x, w, ld_w, w_s, w_rows, n, k, out, ld_out, ws, size, None)


def forward(x=P, type=0, m=8, ld_x=16, w=P, w_type=0, n=8, ld_w=16, k=16, grads=3, out=P, ld_out=8, saved=P,
            keep=1 << 30, ws=P, size=1 << 30):
    return abi.fp8_linear_forward(x, type, m, ld_x, w, w_type, n, ld_w, k, grads, out, ld_out, saved, keep, ws, size,
                                  None)


def backward(dy=P, type=0, m=8, ld_dy=8, n=8, k=16, grads=3, saved=P, keep=1 << 30, dx=P, ld_dx=16, dw=P, dw_type=0,
             ld_dw=16, ws=P, size=1 << 30):
    return abi.fp8_linear_backward(dy, type, m, ld_dy, n, k, grads, saved, keep, dx, ld_dx, dw, dw_type, ld_dw, ws,
                                   size, None)


def ortho(g=P, type=0, batch=1, rows=8, cols=8, ld=8, batch_g=64, steps=5, a=1.0, b=1.0, c=1.0, eps=0.0, out=P,
          out_type=0, ws=P, size=1 << 40):
    return abi.orthogonalize(g, type, batch, rows, cols, ld, batch_g, steps, a, b, c, eps, out, out_type, ws, size, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), abi.BCJR_ERR_NULL), (dict(q=None), abi.BCJR_ERR_NULL), (dict(s=None), abi.BCJR_ERR_NULL),
    (dict(q_t=P), abi.BCJR_ERR_NULL), (dict(s_t=P), abi.BCJR_ERR_NULL), (dict(type=3), abi.BCJR_ERR_SIZE),
    (dict(type=-1), abi.BCJR_ERR_SIZE), (dict(block=64), abi.BCJR_ERR_SIZE), (dict(rows=-1), abi.BCJR_ERR_SIZE),
    (dict(cols=BIG), abi.BCJR_ERR_SIZE), (dict(ld=7), abi.BCJR_ERR_LAYOUT), (dict(q=P + 8), abi.BCJR_ERR_LAYOUT),
    (dict(ld_q=24), abi.BCJR_ERR_LAYOUT), (dict(cols=17, ld=17), abi.BCJR_ERR_LAYOUT),
    (dict(q_t=P + 1, s_t=P), abi.BCJR_ERR_LAYOUT), (dict(q_t=P, s_t=P, rows=17), abi.BCJR_ERR_LAYOUT),
    (dict(rows=1 << 30, cols=1 << 13, ld=1 << 13, ld_q=1 << 13), abi.BCJR_ERR_SIZE),
    (dict(rows=(1 << 23) + 1), abi.BCJR_ERR_SIZE),
    (dict(rows=1 << 23, cols=(1 << 11) + 1, ld=1 << 12, ld_q=1 << 12), abi.BCJR_ERR_SIZE),
    (dict(rows=0), abi.BCJR_OK), (dict(cols=0, ld=0, x=None), abi.BCJR_OK)])
def test_quantize_refusals(change, status):
    assert quantize(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(a=None), abi.BCJR_ERR_NULL), (dict(a_s=None), abi.BCJR_ERR_NULL), (dict(b=None), abi.BCJR_ERR_NULL),
    (dict(b_s=None), abi.BCJR_ERR_NULL), (dict(out=None), abi.BCJR_ERR_NULL), (dict(type=9), abi.BCJR_ERR_SIZE),
    (dict(b_rows=2), abi.BCJR_ERR_SIZE), (dict(m=-1), abi.BCJR_ERR_SIZE), (dict(k=BIG), abi.BCJR_ERR_SIZE),
    (dict(a=P + 4), abi.BCJR_ERR_LAYOUT), (dict(ld_b=40), abi.BCJR_ERR_LAYOUT), (dict(k=17), abi.BCJR_ERR_LAYOUT),
    (dict(ld_out=7), abi.BCJR_ERR_LAYOUT), (dict(ld_a=1 << 31), abi.BCJR_ERR_LAYOUT),
    (dict(m=1 << 30, n=1 << 30, ld_out=1 << 30), abi.BCJR_ERR_SIZE),
    (dict(m=1 << 23, n=(1 << 14) + 1, ld_out=1 << 15), abi.BCJR_ERR_SIZE),
    (dict(k=16, ld_a=(1 << 23) + 16), abi.BCJR_ERR_LAYOUT), (dict(m=0), abi.BCJR_OK), (dict(n=0), abi.BCJR_OK)])
def test_matmul_refusals(change, status):
    assert matmul(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), abi.BCJR_ERR_NULL), (dict(w=None), abi.BCJR_ERR_NULL), (dict(w_s=None), abi.BCJR_ERR_NULL),
    (dict(out=None), abi.BCJR_ERR_NULL), (dict(type=7), abi.BCJR_ERR_SIZE), (dict(w_rows=16), abi.BCJR_ERR_SIZE),
    (dict(m=-1), abi.BCJR_ERR_SIZE), (dict(ld_x=15), abi.BCJR_ERR_LAYOUT), (dict(w=P + 2), abi.BCJR_ERR_LAYOUT),
    (dict(ld_w=17), abi.BCJR_ERR_LAYOUT), (dict(ld_out=7), abi.BCJR_ERR_LAYOUT), (dict(ws=None), abi.BCJR_ERR_WORKSPACE),
    (dict(ws=P + 16), abi.BCJR_ERR_WORKSPACE), (dict(size=100), abi.BCJR_ERR_WORKSPACE), (dict(m=0), abi.BCJR_OK),
    (dict(n=0), abi.BCJR_OK)])
def test_linear_quantized_refusals(change, status):
    assert served(**change) == status


@pytest.mark.parametrize("call,change,status", [
    (forward, dict(x=None), abi.BCJR_ERR_NULL), (forward, dict(w=None), abi.BCJR_ERR_NULL),
    (forward, dict(out=None), abi.BCJR_ERR_NULL), (forward, dict(type=4), abi.BCJR_ERR_SIZE),
    (forward, dict(w_type=4), abi.BCJR_ERR_SIZE), (forward, dict(grads=4), abi.BCJR_ERR_SIZE),
    (forward, dict(k=BIG), abi.BCJR_ERR_SIZE), (forward, dict(ld_x=8), abi.BCJR_ERR_LAYOUT),
    (forward, dict(ld_w=8), abi.BCJR_ERR_LAYOUT), (forward, dict(ld_out=7), abi.BCJR_ERR_LAYOUT),
    (forward, dict(saved=None), abi.BCJR_ERR_WORKSPACE), (forward, dict(keep=16), abi.BCJR_ERR_WORKSPACE),
    (forward, dict(saved=P + 16), abi.BCJR_ERR_WORKSPACE), (forward, dict(ws=None), abi.BCJR_ERR_WORKSPACE),
    (forward, dict(size=16), abi.BCJR_ERR_WORKSPACE), (backward, dict(dy=None), abi.BCJR_ERR_NULL),
    (backward, dict(dx=None), abi.BCJR_ERR_NULL), (backward, dict(dw=None), abi.BCJR_ERR_NULL),
    (backward, dict(type=-1), abi.BCJR_ERR_SIZE), (backward, dict(dw_type=5), abi.BCJR_ERR_SIZE),
    (backward, dict(grads=-1), abi.BCJR_ERR_SIZE), (backward, dict(ld_dy=7), abi.BCJR_ERR_LAYOUT),
    (backward, dict(ld_dx=15), abi.BCJR_ERR_LAYOUT), (backward, dict(ld_dw=15), abi.BCJR_ERR_LAYOUT),
    (backward, dict(keep=16), abi.BCJR_ERR_WORKSPACE), (backward, dict(ws=P + 64), abi.BCJR_ERR_WORKSPACE),
    (backward, dict(size=16), abi.BCJR_ERR_WORKSPACE)])
def test_linear_refusals(call, change, status):
    assert call(**change) == status


def test_linear_buffers():
    saved, ws = abi.fp8_linear_saved_bytes, abi.fp8_linear_workspace_bytes
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    m, n, k = 100, 60, 40
    # x^T [k, m] with a scale for each row and 128 of m, w^T [k, n] with one for each 128 x 128; rows on 16 bytes
    x_t, w_t = up(k * 112) + up(k * 4), up(k * 64) + up(4)
    assert [saved(m, n, k, g) for g in range(4)] == [0, w_t, x_t, x_t + w_t]
    forward_ws = up(m * 48) + up(m * 4) + up(n * 48) + up(4)
    backward_ws = up(m * 64) + up(m * 4) + up(n * 112) + up(n * 4)
    assert ws(m, n, k) == max(forward_ws, backward_ws)
    assert abi.fp8_linear_quantized_workspace_bytes(4, 8192) == abi.fp8_linear_quantized_workspace_bytes(1, 32768) == 0
    assert abi.fp8_linear_quantized_workspace_bytes(4, 8193) == up(4 * 8208) + up(4 * 65 * 4)
    assert abi.fp8_linear_quantized_workspace_bytes(16, 2048) == 0
    assert abi.fp8_linear_quantized_workspace_bytes(17, k) == up(17 * 48) + up(17 * 4)
    assert abi.fp8_linear_quantized_workspace_bytes(m, k) == up(m * 48) + up(m * 4)
    assert saved(-1, n, k, 3) == ws(m, BIG, k) == abi.fp8_linear_quantized_workspace_bytes(-1, k) == 0


@pytest.mark.parametrize("change,status", [
    (dict(g=None), abi.BCJR_ERR_NULL), (dict(out=None), abi.BCJR_ERR_NULL), (dict(type=3), abi.BCJR_ERR_SIZE),
    (dict(out_type=3), abi.BCJR_ERR_SIZE), (dict(batch=0), abi.BCJR_ERR_SIZE), (dict(batch=65536), abi.BCJR_ERR_SIZE),
    (dict(rows=0), abi.BCJR_ERR_SIZE), (dict(cols=65537, ld=65537), abi.BCJR_ERR_SIZE),
    (dict(steps=0), abi.BCJR_ERR_SIZE), (dict(steps=1001), abi.BCJR_ERR_SIZE),
    (dict(a=float("nan")), abi.BCJR_ERR_SIZE), (dict(b=float("inf")), abi.BCJR_ERR_SIZE),
    (dict(eps=-1.0), abi.BCJR_ERR_SIZE), (dict(ld=7), abi.BCJR_ERR_LAYOUT),
    (dict(batch=2, batch_g=-1), abi.BCJR_ERR_LAYOUT), (dict(ws=None), abi.BCJR_ERR_WORKSPACE),
    (dict(ws=P + 16), abi.BCJR_ERR_WORKSPACE), (dict(size=1000), abi.BCJR_ERR_WORKSPACE)])
def test_orthogonalize_refusals(change, status):
    assert ortho(**change) == status


def test_orthogonalize_workspace():
    size = abi.orthogonalize_workspace_bytes
    # X as two halves and its transpose twice, A and B; up to 256 rows and for a float32 result both halves of all
    x, s = 320 * 448 * 2, 320 * 320 * 2
    assert size(1, 300, 400, abi.BCJR_TYPE_BF16) == 256 * 8 + 4 * x + 2 * s
    assert size(1, 300, 400, abi.BCJR_TYPE_F32) == 256 * 8 + 6 * x + 4 * s
    x, s = 128 * 192 * 2, 128 * 128 * 2
    assert size(1, 100, 150, abi.BCJR_TYPE_BF16) == size(1, 100, 150, abi.BCJR_TYPE_F32) == 256 * 8 + 6 * x + 4 * s
    assert size(1, 150, 100, abi.BCJR_TYPE_F32) == size(1, 100, 150, abi.BCJR_TYPE_F32)
    assert size(3, 64, 64, abi.BCJR_TYPE_F16) == 3 * size(1, 64, 64, abi.BCJR_TYPE_F32)
    for bad in ((0, 8, 8, 0), (1, 0, 8, 0), (1, 8, 65537, 0), (1, 8, 8, 3)):
        assert size(*bad) == 0


def test_status_strings():
    for code in (abi.BCJR_ERR_LAYOUT, abi.BCJR_ERR_SIZE):
        assert abi.bcjr_status_string(code).startswith("BCJR_ERR")


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64)
    q = x.to(torch.float8_e4m3fn)
    s = torch.ones(4, 1)
    for call in (lambda: dba.fp8_block_quantize(x), lambda: dba.fp8_block_matmul(q, s, q, s),
                 lambda: dba.fp8_linear(x, x), lambda: dba.fp8_linear_quantized(x, q, s), lambda: dba.orthogonalize(x)):
        with pytest.raises(TypeError):
            call()


def test_reference_rounds_to_the_nearest_code():
    """The tests' own quantizer against the table of all codes."""
    codes = torch.arange(0, 0x7f, dtype=torch.uint8).view(ref.E4M3).double()
    x = torch.randn(50, 300, generator=torch.Generator().manual_seed(1))
    q, s = ref.quantize(x, 1)
    spread = s.double().repeat_interleave(128, 1)[:, :300]
    v = (x.double() / spread).abs()
    nearest = (v[..., None] - codes).abs().min(-1).values
    # the code's distance is the smallest one, up to the float32 roundings of the scale and the quotient
    assert ((q.float().double().abs() - v).abs() <= nearest + v * 3 * 2.0 ** -24).all()
