"""The quantized layer on the GPU: block quantization, the 8-bit product, the linear layer and its gradients, against
64-bit references."""
import math

import pytest
import torch

import differentiable_bcjr_amd as dba
import layer_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [(1, 1), (1, 128), (1, 5000), (3, 129), (16, 16), (127, 255), (128, 128), (130, 300), (257, 1000), (1000, 24)]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda:0")


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _same_codes(q, r):
    assert q.shape == r.shape
    a, b = q.cpu().view(torch.uint8), r.view(torch.uint8)
    nan = (a & 0x7f) == 0x7f
    assert torch.equal(nan, (b & 0x7f) == 0x7f)
    assert torch.equal(a[~nan], b[~nan])


def _same_scales(s, r):
    assert s.shape == r.shape
    torch.testing.assert_close(s.cpu(), r, rtol=0, atol=0, equal_nan=True)


def _check_quantize(x, dev, block_rows, transposed):
    got = dba.fp8_block_quantize(x, block_rows=block_rows, transposed=transposed)
    host = x.cpu().float()
    q, s = ref.quantize(host, block_rows)
    _same_codes(got[0], q)
    _same_scales(got[1], s)
    if transposed:
        q, s = ref.quantize(host.t(), block_rows)
        _same_codes(got[2], q)
        _same_scales(got[3], s)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_is_the_definition(dev, shape, dtype, block_rows, transposed):
    x = _randn(*shape, seed=shape[0] * 7 + shape[1])
    x = x * torch.exp(2 * _randn(shape[0], 1, seed=5))
    _check_quantize(x.to(dtype).to(dev), dev, block_rows, transposed)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_rounds_every_tie_to_even(dev, block_rows):
    """Every e4m3 number, every midpoint of two neighbours and the float32 numbers next to it, in blocks whose largest
    entry is 448 (so the scale is 1: fl(448 fl(1/448)) = 1)."""
    codes = torch.arange(0, 0x7f, dtype=torch.uint8).view(ref.E4M3).float()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, torch.nextafter(mid, torch.zeros(())), torch.nextafter(mid, torch.full((), 1e9))])
    v = torch.cat([v, -v])
    v = torch.cat([v, torch.zeros(-len(v) % 127)]).view(-1, 127)
    x = torch.cat([v, torch.full((v.shape[0], 1), 448.0)], 1)
    assert torch.equal(ref.quantize(x, 1)[1], torch.ones(x.shape[0], 1))
    _check_quantize(x.to(dev), dev, block_rows, True)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_blocks(dev, block_rows, transposed):
    """Zeros, numbers at the bottom of float32, Inf and NaN: each stays in its own blocks."""
    x = _randn(300, 600, seed=3)
    x[0:128, 0:128] = 0
    x[5, 128:256] = 1e-42
    x[130:256, 256:384] = torch.finfo(torch.float32).tiny * _randn(126, 128, seed=4)
    x[140, 10] = math.inf
    x[141, 200] = -math.inf
    x[142, 300] = math.nan
    x[143, 400], x[143, 401] = math.nan, math.inf
    x[299, 599] = 3e38
    _check_quantize(x.to(dev), dev, block_rows, transposed)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_reads_strided_rows(dev, dtype):
    """Rows further apart than they are long, rows off the 16-byte boundaries, columns apart, broadcast rows."""
    room = _randn(70, 400, seed=6).to(dtype).to(dev)
    for x in (room[:, :300], room[3:, 1:300], room[:, ::2], room.t(), room[:1].expand(40, 400), room[5:6, 7:8]):
        for transposed in (False, True):
            _check_quantize(x, dev, 1, transposed)


def test_quantize_writes_its_rows_alone(dev):
    """Bytes between a row's end and the next row, and behind the last row, keep what they hold."""
    abi = dba.abi
    rows, cols, ld, ld_t = 37, 141, 160, 64
    x = _randn(rows, cols, seed=8).to(dev)
    q = torch.full((rows + 3, ld), 0xa5, dtype=torch.uint8, device=dev)
    q_t = torch.full((cols + 3, ld_t), 0xa5, dtype=torch.uint8, device=dev)
    s = torch.full((2 * rows + 9,), -1.0, device=dev)
    s_t = torch.full((1 * cols + 9,), -1.0, device=dev)
    rc = abi.fp8_block_quantize(x.data_ptr(), abi.BCJR_TYPE_F32, rows, cols, cols, 1, q.data_ptr(), ld, s.data_ptr(),
                                q_t.data_ptr(), ld_t, s_t.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == abi.BCJR_OK
    torch.cuda.synchronize()
    r, rs = ref.quantize(x.cpu(), 1)
    assert torch.equal(q[:rows, :cols].cpu(), r.view(torch.uint8)) and torch.equal(s[:2 * rows].cpu().view(2, rows).t(), rs)
    assert (q[:rows, cols:] == 0xa5).all() and (q[rows:] == 0xa5).all() and (s[2 * rows:] == -1).all()
    assert (q_t[:cols, rows:] == 0xa5).all() and (q_t[cols:] == 0xa5).all() and (s_t[cols:] == -1).all()


def test_quantize_nothing(dev):
    for shape in ((0, 5), (5, 0), (0, 0)):
        q, s, q_t, s_t = dba.fp8_block_quantize(torch.empty(shape, device=dev), transposed=True)
        assert q.shape == shape and q_t.shape == shape[::-1]
        assert s.shape == (shape[0], -(-shape[1] // 128)) and s_t.shape == (shape[1], -(-shape[0] // 128))


# ------------------------------------------------------------------------------------------------ product

PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 300, 2048), (3, 5, 7), (2, 130, 17), (16, 64, 500), (17, 65, 129), (64, 300, 16),
            (129, 130, 131), (128, 128, 128), (257, 64, 1000), (300, 520, 385), (33, 1000, 4096)]


def _operand(rows, k, block_rows, seed, poison=True):
    """Codes and scales as fp8_block_quantize lays them out; the bytes behind each row hold NaN codes."""
    x = _randn(rows, k, seed=seed) * torch.exp(_randn(rows, 1, seed=seed + 1))
    q, s = ref.quantize(x, block_rows)
    room = torch.full((rows, -(-k // 16) * 16), 0x7f, dtype=torch.uint8)
    room[:, :k] = q.view(torch.uint8)
    return q, s, room.cuda().view(ref.E4M3)[:, :k], s.t().contiguous().cuda().t()


def _check_product(got, av, bv, dtype):
    r, bound = ref.matmul_bound(av, bv, dtype)
    err = (got.cpu().double() - r).abs()
    assert got.dtype == dtype and got.shape == r.shape
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(dev, m, n, k, b_rows, dtype):
    aq, as_, a, a_s = _operand(m, k, 1, m + 3 * k)
    bq, bs, b, b_s = _operand(n, k, b_rows, n + 5 * k)
    _check_product(dba.fp8_block_matmul(a, a_s, b, b_s, out_dtype=dtype), ref.values(aq, as_, 1),
                   ref.values(bq, bs, b_rows), dtype)


def test_matmul_copies_other_layouts(dev):
    """Codes and scales in any strides give what packed ones give."""
    m, n, k = 40, 50, 300
    _, _, a, a_s = _operand(m, k, 1, 1)
    _, _, b, b_s = _operand(n, k, 128, 2)
    want = dba.fp8_block_matmul(a, a_s, b, b_s, out_dtype=torch.float32)
    odd = torch.empty(m, k + 1, dtype=torch.uint8, device=dev).view(ref.E4M3)[:, 1:]
    odd.copy_(a)
    turned = b.contiguous().t().contiguous().t()
    got = dba.fp8_block_matmul(odd, a_s.contiguous(), turned, b_s.contiguous(), out_dtype=torch.float32)
    assert torch.equal(got, want)


def test_matmul_nothing(dev):
    a, a_s = dba.fp8_block_quantize(torch.empty(0, 64, device=dev))
    b, b_s = dba.fp8_block_quantize(torch.randn(9, 64, device=dev), block_rows=128)
    assert dba.fp8_block_matmul(a, a_s, b, b_s).shape == (0, 9)
    a, a_s = dba.fp8_block_quantize(torch.empty(4, 0, device=dev))
    b, b_s = dba.fp8_block_quantize(torch.empty(9, 0, device=dev), block_rows=128)
    assert torch.equal(dba.fp8_block_matmul(a, a_s, b, b_s), torch.zeros(4, 9, dtype=torch.bfloat16, device=dev))


def test_matmul_keeps_rows_apart(dev):
    """A NaN or Inf of one row of a (one of b) reaches that row's (column's) results and no other."""
    m, n, k = 40, 300, 400
    x, w = _randn(m, k, seed=1).to(dev), _randn(n, k, seed=2).to(dev)
    x[7, 399], x[9, 3] = math.nan, math.inf
    a, a_s = dba.fp8_block_quantize(x)
    for block_rows in (1, 128):
        b, b_s = dba.fp8_block_quantize(w, block_rows=block_rows)
        y = dba.fp8_block_matmul(a, a_s, b, b_s)
        bad = torch.zeros(m, dtype=torch.bool, device=dev)
        bad[[7, 9]] = True
        assert torch.equal(y.isnan(), bad[:, None].expand(m, n))


def test_matmul_writes_its_entries_alone(dev):
    abi = dba.abi
    m, n, k, ld = 37, 141, 200, 150
    aq, as_, a, a_s = _operand(m, k, 1, 11)
    bq, bs, b, b_s = _operand(n, k, 128, 12)
    for dtype, code in ((torch.float32, 0), (torch.bfloat16, 1), (torch.float16, 2)):
        out = torch.full((m + 2, ld), -7.0, dtype=dtype, device=dev)
        rc = abi.fp8_block_matmul(a.data_ptr(), a.stride(0), a_s.data_ptr(), b.data_ptr(), b.stride(0), b_s.data_ptr(),
                                  128, m, n, k, out.data_ptr(), code, ld, torch.cuda.current_stream().cuda_stream)
        assert rc == abi.BCJR_OK
        _check_product(out[:m, :n], ref.values(aq, as_, 1), ref.values(bq, bs, 128), dtype)
        assert (out[:m, n:] == -7).all() and (out[m:] == -7).all()


# ------------------------------------------------------------------------------------------------ linear layer


def _linear_case(m, n, k, dtype, seed=0):
    x = (_randn(m, k, seed=seed) * torch.exp(0.5 * _randn(m, 1, seed=seed + 1))).to(dtype)
    w = _randn(n, k, seed=seed + 2) / math.sqrt(k)
    dy = (_randn(m, n, seed=seed + 3) * 1e-2).to(dtype)
    return x, w, dy


LINEAR = [(1, 16, 16), (1, 512, 2048), (5, 100, 70), (16, 300, 1000), (64, 256, 384), (200, 130, 257), (515, 129, 640)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear_and_gradients_are_the_formulas(dev, m, n, k, dtype):
    x, w, dy = _linear_case(m, n, k, dtype, seed=m + n + k)
    xg, wg = x.to(dev).requires_grad_(True), w.to(dev).requires_grad_(True)
    y = dba.fp8_linear(xg, wg)
    dx, dw = torch.autograd.grad(y, (xg, wg), dy.to(dev))
    val = lambda t, r: ref.values(*ref.quantize(t.float(), r), r)  # noqa: E731
    wv = val(w, 128)
    _check_product(y.detach(), val(x, 1), wv, dtype)
    _check_product(dx, val(dy, 1), wv.t(), dtype)
    _check_product(dw, val(dy.t(), 1), val(x.t(), 1), torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", LINEAR + [(2, 2048, 512), (33, 70, 8192), (40, 64, 100), (4, 40, 8192),
                                           (3, 4200, 1000), (4, 50, 8300), (1, 33, 33000), (16, 100, 2048),
                                           (15, 4200, 2100), (16, 60, 2050), (9, 20, 3500)])
def test_linear_quantized_is_quantize_then_matmul(dev, m, n, k, dtype):
    x, w, _ = _linear_case(m, n, k, dtype, seed=m + n + k)
    for block_rows in (1, 128):
        q, s = dba.fp8_block_quantize(w.to(dev), block_rows=block_rows)
        y = dba.fp8_linear_quantized(x.to(dev), q, s)
        _check_product(y, ref.values(*ref.quantize(x.float(), 1), 1),
                       ref.values(*ref.quantize(w, block_rows), block_rows), dtype)


def test_linear_keeps_leading_dimensions_and_skips_what_is_not_asked(dev):
    x, w, _ = _linear_case(30, 40, 50, torch.bfloat16)
    x, w = x.view(2, 3, 5, 50).to(dev), w.to(dev)
    want = dba.fp8_linear(x, w)
    assert want.shape == (2, 3, 5, 40) and want.dtype == torch.bfloat16 and not want.requires_grad
    assert torch.equal(want.view(30, 40), dba.fp8_linear(x.view(30, 50), w))
    up = torch.randn_like(want)
    xg, wg = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    both = torch.autograd.grad(dba.fp8_linear(xg, wg), (xg, wg), up)
    assert torch.equal(torch.autograd.grad(dba.fp8_linear(xg, w), xg, up)[0], both[0])
    assert torch.equal(torch.autograd.grad(dba.fp8_linear(x, wg), wg, up)[0], both[1])
    q, s = dba.fp8_block_quantize(w, block_rows=128)
    assert torch.equal(dba.fp8_linear_quantized(x, q, s), want)


def test_linear_takes_one_token_an_empty_sum_and_a_broadcast_gradient(dev):
    x, w, _ = _linear_case(6, 40, 50, torch.float32)
    x, w = x.to(dev), w.to(dev)
    q, s = dba.fp8_block_quantize(w, block_rows=128)
    one = dba.fp8_linear(x[0], w)
    assert one.shape == (40,) and torch.equal(one, dba.fp8_linear(x[:1], w)[0])
    one = dba.fp8_linear_quantized(x[0], q, s)
    assert one.shape == (40,) and torch.equal(one, dba.fp8_linear_quantized(x[:1], q, s)[0])
    for rows in (1, 30):   # k = 0
        nothing = dba.fp8_block_quantize(w[:, :0], block_rows=128)
        assert torch.equal(dba.fp8_linear_quantized(x.new_empty(rows, 0), *nothing), torch.zeros(rows, 40, device=dev))
    xg, wg = x.view(2, 3, 50).clone().requires_grad_(True), w.clone().requires_grad_(True)
    dba.fp8_linear(xg, wg).sum().backward()   # an upstream gradient of one number with strides of 0
    want = torch.autograd.grad(dba.fp8_linear(xg, wg), (xg, wg), torch.ones(2, 3, 40, device=dev))
    assert torch.equal(xg.grad, want[0]) and torch.equal(wg.grad, want[1])
    y = dba.fp8_linear(xg, wg)
    (first,) = torch.autograd.grad(y.square().sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError):   # the gradient has none of its own
        first.sum().backward()


def test_calls_without_a_gradient_refuse_to_lose_one(dev):
    g = _randn(20, 40, seed=1).to(dev)
    q = dba.fp8_block_quantize(g, block_rows=128)
    for call in (lambda x: dba.fp8_linear_quantized(x, *q), dba.orthogonalize):
        want = call(g)
        asks = g.clone().requires_grad_(True)
        with pytest.raises(RuntimeError, match="no gradient"):
            call(asks)
        with torch.no_grad():
            assert torch.equal(call(asks), want)


def test_linear_step_in_a_graph(dev):
    """Forward and both gradients captured together and replayed on new inputs, against the eager step."""
    x, w, dy = (t.to(dev) for t in _linear_case(70, 140, 150, torch.bfloat16))
    xs, ws = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(dba.fp8_linear(xs, ws), (xs, ws), dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dba.fp8_linear(xs, ws)
        dx, dw = torch.autograd.grad(y, (xs, ws), dy)
    y = y.detach()
    for seed in (31, 32, 33):
        nx, nw, ndy = (t.to(dev) for t in _linear_case(70, 140, 150, torch.bfloat16, seed=seed))
        with torch.no_grad():
            xs.copy_(nx)
            ws.copy_(nw)
            dy.copy_(ndy)
        graph.replay()
        torch.cuda.synchronize()
        a, b = nx.requires_grad_(True), nw.requires_grad_(True)
        want = dba.fp8_linear(a, b)
        grads = torch.autograd.grad(want, (a, b), ndy)
        assert torch.equal(y, want) and torch.equal(dx, grads[0]) and torch.equal(dw, grads[1])


def test_linear_without_tokens(dev):
    w = torch.randn(8, 32, device=dev, requires_grad=True)
    x = torch.empty(0, 32, device=dev, requires_grad=True)
    y = dba.fp8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.empty(0, 8, device=dev))
    assert y.shape == (0, 8) and dx.shape == (0, 32) and torch.equal(dw, torch.zeros(8, 32, device=dev))


def test_linear_gradients_follow_differences(dev):
    """The gradient of the quantized product stands for that of x w^T: along a direction it meets the difference quotient
    of the exact product up to the codes' error.  Each code is off by at most 2^-4 of its value (or 2^-10 of the scale,
    amax / 448, which is less than 2^-18 of the block's largest), the two factors' errors are independent, so the
    relative error of an inner product of random terms stays under 2 * 2^-4."""
    m, n, k = 96, 160, 224
    x, w, dy = _linear_case(m, n, k, torch.float32)
    xg, wg = x.to(dev).requires_grad_(True), w.to(dev).requires_grad_(True)
    dx, dw = torch.autograd.grad(dba.fp8_linear(xg, wg), (xg, wg), dy.to(dev))
    f = lambda x_, w_: float((x_ @ w_.t() * dy.double()).sum())  # noqa: E731
    x, w = x.double(), w.double()
    for got, size, shift in ((dx, x, lambda h, d: f(x + h * d, w) - f(x - h * d, w)),
                             (dw, w, lambda h, d: f(x, w + h * d) - f(x, w - h * d))):
        d = got.cpu().double().sign()   # along its own signs, so that nothing cancels
        quotient = shift(1e-3, d) / 2e-3
        along = float((got.cpu().double() * d).sum())
        assert abs(along - quotient) <= 2 * 2.0 ** -4 * abs(quotient)


def test_layer_on_another_stream_and_in_a_graph(dev):
    """Eager calls on a side stream, then the same calls captured and replayed on new inputs, each replay against the
    eager result."""
    x, w, dy = (t.to(dev) for t in _linear_case(130, 140, 150, torch.bfloat16))
    want = dba.fp8_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dba.fp8_linear(x, w)
        up = dba.orthogonalize(w)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(up, dba.orthogonalize(w))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq = dba.fp8_block_quantize(x, transposed=True)
        wq = dba.fp8_block_quantize(w, block_rows=128, transposed=True)
        y = dba.fp8_block_matmul(*xq[:2], *wq[:2])
        served = dba.fp8_linear_quantized(x[:1], *wq[:2])
        o = dba.orthogonalize(w)
    for seed in (20, 21, 22):
        nx, nw, _ = (t.to(dev) for t in _linear_case(130, 140, 150, torch.bfloat16, seed=seed))
        x.copy_(nx)
        w.copy_(nw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, dba.fp8_linear(nx, nw))
        assert torch.equal(served, dba.fp8_linear_quantized(nx[:1], *dba.fp8_block_quantize(nw, block_rows=128)))
        assert torch.equal(o, dba.orthogonalize(nw))


def test_layer_refusals(dev):
    x, w = torch.randn(4, 64, device=dev), torch.randn(8, 64, device=dev)
    q, s = dba.fp8_block_quantize(w, block_rows=128)
    with pytest.raises(TypeError):
        dba.fp8_block_quantize(x.double())
    with pytest.raises(TypeError):
        dba.fp8_block_quantize(x.cpu())
    with pytest.raises(ValueError):
        dba.fp8_block_quantize(x[0])
    with pytest.raises(ValueError):
        dba.fp8_block_quantize(x, block_rows=64)
    with pytest.raises(TypeError):
        dba.fp8_block_matmul(x, s, q, s)
    with pytest.raises(ValueError):
        dba.fp8_block_matmul(*dba.fp8_block_quantize(x[:, :63]), q, s)
    with pytest.raises(ValueError):
        dba.fp8_block_matmul(*dba.fp8_block_quantize(x), q, s[:, :0])
    with pytest.raises(TypeError):
        dba.fp8_block_matmul(*dba.fp8_block_quantize(x), q, s, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        dba.fp8_linear(x[:, :63], w)
    with pytest.raises(ValueError):
        dba.fp8_linear_quantized(x[:, :63], q, s)
    with pytest.raises(TypeError):
        dba.orthogonalize(w.double())
    with pytest.raises(ValueError):
        dba.orthogonalize(w[0])
    with pytest.raises(dba.BCJRError):
        dba.orthogonalize(w, steps=0)


# ------------------------------------------------------------------------------------------------ orthogonalized update

USUAL = (3.4445, -4.7750, 2.0315)
CONVERGING = (1.875, -1.25, 0.375)


def _update(kind, rows, cols, seed):
    g = _randn(rows, cols, seed=seed)
    if kind == "low-rank":
        r = max(1, min(rows, cols) // 16)
        g = _randn(rows, r, seed=seed + 1) @ _randn(r, cols, seed=seed + 2) / math.sqrt(r) + 0.05 * g
    elif kind == "one-entry":
        g = 1e-3 * g
        g[rows // 2, cols // 3] = 10.0
    elif kind == "small":
        g = 1e-30 * g
    elif kind == "large":
        g = 1e30 * g
    return g


def _check_orthogonal(got, g, steps, coefficients, eps, out_dtype):
    """Against 64 bits.  The bound is four times what the documented roundings alone make of this matrix (emulated on
    the CPU with float32 products), and the rounding of the result."""
    r = ref.newton_schulz(g, steps, coefficients, eps)
    split = out_dtype != torch.bfloat16 or min(g.shape) <= 256
    emulated = ref.newton_schulz_rounded(g, steps, coefficients, eps, split).double()
    off, norm = float((emulated - r).norm()), float(r.norm())
    err = float((got.cpu().double() - r).norm())
    tiny = torch.finfo(out_dtype).tiny * torch.finfo(out_dtype).eps * math.sqrt(r.numel())
    assert got.dtype == out_dtype and got.shape == r.shape
    assert err <= 4 * off + torch.finfo(out_dtype).eps / 2 * norm + tiny, (err / norm, off / norm)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (7, 5), (16, 16), (64, 64), (65, 130), (128, 128),
                                       (200, 100), (129, 1000), (520, 300), (260, 257), (400, 1100), (50, 4200), (8300, 60), (130, 4100)])
def test_orthogonalize_sizes(dev, rows, cols, dtype):
    g = _update("plain", rows, cols, rows + cols).to(dtype)
    _check_orthogonal(dba.orthogonalize(g.to(dev)), g.float(), 5, USUAL, 1e-7, dtype)


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("kind", ["low-rank", "one-entry", "large"])
@pytest.mark.parametrize("rows,cols", [(96, 200), (257, 130), (300, 420)])
def test_orthogonalize_kinds(dev, rows, cols, kind, out_dtype):
    g = _update(kind, rows, cols, 9)
    _check_orthogonal(dba.orthogonalize(g.to(dev), out_dtype=out_dtype), g, 5, USUAL, 1e-7, out_dtype)


@pytest.mark.parametrize("steps", [1, 2, 10])
def test_orthogonalize_steps_and_coefficients(dev, steps):
    g = _update("low-rank", 70, 150, 3)
    _check_orthogonal(dba.orthogonalize(g.to(dev), steps=steps, coefficients=CONVERGING, eps=1e-3), g, steps,
                      CONVERGING, 1e-3, torch.float32)
    small = _update("small", 70, 150, 3)
    _check_orthogonal(dba.orthogonalize(small.to(dev), steps=steps, eps=0.0), small, steps, USUAL, 0.0, torch.float32)


def test_orthogonalize_makes_rows_orthonormal(dev):
    g = _update("plain", 100, 300, 4)
    x = dba.orthogonalize(g.to(dev), steps=20, coefficients=CONVERGING).cpu().double()
    # at the fixed point the error left is that of holding X to 22 bits and A to 22: far under 1e-4
    assert float((x @ x.t() - torch.eye(100, dtype=torch.float64)).abs().max()) < 1e-4


def test_orthogonalize_zero_nan_inf_stay_in_their_matrix(dev):
    g = torch.stack([_update("plain", 40, 70, s) for s in range(4)])
    want = dba.orthogonalize(g.to(dev))
    g[0] = 0
    g[1, 39, 69] = math.nan
    g[3, 0, 5] = math.inf
    got = dba.orthogonalize(g.to(dev))
    assert (got[0] == 0).all() and got[1].isnan().all() and got[3].isnan().all()
    assert torch.equal(got[2], want[2])


@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** -149])
def test_orthogonalize_over_the_range_of_float32(dev, scale):
    """A power of two changes nothing without eps, also where |g|_F is beyond float32 or the entries are subnormal."""
    g = (_update("plain", 300, 420, 5) * 30).round()
    want = dba.orthogonalize(g.to(dev), eps=0.0)
    _check_orthogonal(want, g, 5, USUAL, 0.0, torch.float32)
    scaled = (g.double() * scale).float()
    assert torch.equal(scaled.double(), g.double() * scale)
    assert scale < 1 or scaled.norm().isinf()
    assert torch.equal(dba.orthogonalize(scaled.to(dev), eps=0.0), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_stacks_and_strides(dev, dtype):
    """A stack gives each matrix what it gets alone, in whatever strides it lies."""
    g = torch.stack([_update("plain", 150, 90, s) for s in range(6)]).to(dtype).to(dev)
    alone = torch.stack([dba.orthogonalize(m) for m in g])
    assert torch.equal(dba.orthogonalize(g), alone)
    assert torch.equal(dba.orthogonalize(g.view(2, 3, 150, 90)), alone.view(2, 3, 150, 90))
    room = torch.zeros(6, 150, 101, dtype=dtype, device=dev)
    room[:, :, 3:93] = g
    assert torch.equal(dba.orthogonalize(room[:, :, 3:93]), alone)
    turned = g.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(dba.orthogonalize(turned), alone)
    one = g[0].expand(3, 150, 90)
    assert torch.equal(dba.orthogonalize(one), alone[:1].expand(3, 150, 90))
    assert dba.orthogonalize(g[:0]).shape == (0, 150, 90) and dba.orthogonalize(g[:, :0]).shape == (6, 0, 90)


@pytest.mark.parametrize("batch,rows,cols", [(130, 64, 64), (130, 20, 100), (40, 64, 520), (260, 16, 40), (20, 200, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_many_small(dev, batch, rows, cols, dtype):
    """Stacks that fill the card with matrices of one or few k steps each."""
    g = torch.stack([_update("plain", rows, cols, s) for s in range(3)]).to(dtype)
    got = dba.orthogonalize(g[torch.arange(batch) % 3].to(dev))
    for i in (0, 1, 2):
        _check_orthogonal(got[i], g[i].float(), 5, USUAL, 1e-7, dtype)
        same = got[torch.arange(batch) % 3 == i]
        assert torch.equal(same, got[i].expand_as(same))


# ------------------------------------------------------------------------------------------------ together


def test_training_step_of_a_soft_quantized_layer(dev):
    """The operators as a training step runs them: the weights' soft codeword, the 8-bit layer on it, the exact gradient
    back to the weights' pre-image, its orthogonalized update; then the hard code, quantized and served."""
    L, k, T, n_in, n_out, seq = 8, 2, 0.1, 96, 64, 32
    gen = torch.Generator().manual_seed(5)
    code = torch.randn(1 << L, generator=gen)
    code = (code / code.std()).to(dev)
    w = torch.randn(n_out, n_in, generator=gen).to(dev).requires_grad_(True)
    x = torch.randn(40, n_in, generator=gen).to(dev)
    dy = (1e-2 * torch.randn(40, n_out, generator=gen)).to(dev)

    soft = dba.soft_quantize(w.view(-1, seq), code, L, k, T)
    y = dba.fp8_linear(x, soft.view(n_out, n_in))
    (grad,) = torch.autograd.grad(y, w, dy)
    step = dba.orthogonalize(grad)

    sv = dba.soft_codeword(w.detach().view(-1, seq), code, L, k, T).view(n_out, n_in).cpu()
    val = lambda t, r: ref.values(*ref.quantize(t, r), r)  # noqa: E731
    _check_product(y.detach(), val(x.cpu(), 1), val(sv, 128), torch.float32)
    # the gradient kernel, linear in its input, on the formula's gradient of the soft codeword
    dsoft = val(dy.cpu().t(), 1) @ val(x.cpu().t(), 1).t()
    want = dba.soft_codeword_grad(w.detach().view(-1, seq), code, dsoft.float().to(dev).view(-1, seq), L, k, T)
    assert float((grad.view(-1, seq) - want).norm() / want.norm()) < 1e-4
    _check_orthogonal(step, grad.cpu(), 5, USUAL, 1e-7, torch.float32)

    with torch.no_grad():
        w -= 0.02 * math.sqrt(max(1, n_out / n_in)) * step
    _, hard, _ = dba.viterbi_hard_code(w.detach().view(-1, seq), code, L, k)
    q, s = dba.fp8_block_quantize(hard.view(n_out, n_in), block_rows=128)
    served = dba.fp8_linear_quantized(x[:1], q, s)
    _check_product(served, val(x[:1].cpu(), 1), val(hard.view(n_out, n_in).cpu(), 128), torch.float32)
