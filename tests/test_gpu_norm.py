"""GPU parity of the RMS norm (residual, 8-bit outputs, backward) against 64-bit formulas.

Bounds, relative to the value: fp32 arithmetic has a sum of D squares, up to 32 in a thread and a tree over
the threads (at most 32 + 10 roundings of positive terms, halved by the root), rsqrt (2 units), three products: below
32 roundings of 2^-24, so F32 = 2^-19; a bf16 output adds 2^-8, e4m3 2^-4 (2^-10 absolute below 2^-6), int8 1/2 a unit."""
import pytest
import torch

from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu
F32, HALF_BF16 = 2.0 ** -19, 2.0 ** -8
SHAPES = [(1, 8), (3, 24), (33, 128), (7, 136), (64, 256), (5, 520), (9, 1000), (130, 2048), (3, 2056), (2, 4096),
          (3, 4104), (2, 8192), (2, 8200), (1, 16384)]


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(rows, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 20000 + D)
    x, r, dy, dr = (torch.randn(rows, D, generator=g).to(_dt(dtype)).cuda() for _ in range(4))
    return x, r, (1 + 0.2 * torch.randn(D, generator=g)).cuda(), dy, dr


def _norm64(r, w, eps):
    f = r.double()
    y = f / (f.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w.double()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_norm_and_residual(dtype, rows, D):
    x, res, w, _, _ = _inputs(rows, D, dtype)
    step = HALF_BF16 if dtype == "bf16" else 0.0
    y, none = kda.rms_norm(x, w, eps=1e-5)
    ref = _norm64(x, w, 1e-5)
    assert none is None and ((y.double() - ref).abs() <= (F32 + step) * ref.abs() + 1e-37).all()
    y, r = kda.rms_norm(x, None, residual=res, eps=0.0)
    assert torch.equal(r, x + res)
    ref = _norm64(r, None, 0.0)
    assert ((y.double() - ref).abs() <= (F32 + step) * ref.abs() + 1e-37).all()
    y2, r2 = kda.rms_norm(x, None, residual=res, eps=0.0, residual_out=res)
    assert r2 is res and torch.equal(y, y2) and torch.equal(r, r2)
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_bytes_and_scales(dtype, quant, group, rows, D):
    x, res, w, _, _ = _inputs(rows, D, dtype)
    x[0, : max(8, D // 2)] = 0
    y8, scale, r = kda.rms_norm_quant(x, w, residual=res if rows > 1 else None, quant=quant, group=group)
    ref = _norm64(x if r is None else r, w, 1e-6)
    g = group or D
    n = -(-D // g)
    assert scale.shape == (rows, n) and y8.shape == x.shape
    top = torch.nn.functional.pad(ref.abs(), (0, n * g - D)).reshape(rows, n, g).amax(2).clamp_min(2.0 ** -100)
    most = 448.0 if quant == "e4m3" else 127.0
    assert ((scale.double() - top / most).abs() <= 2 * F32 * top / most).all()
    sc = scale.double().repeat_interleave(g, 1)[:, :D]
    z = ref / sc
    # half a step of the byte type around the value, fp32 arithmetic (value and scale) before it
    half = (2.0 ** -4 * z.abs()).clamp_min(2.0 ** -10) if quant == "e4m3" else torch.full_like(z, 0.5)
    assert ((y8.double() - z).abs() <= half + 4 * F32 * z.abs()).all()
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
def test_zero_rows_infinities_and_nan(quant):
    x = torch.randn(6, 256, device="cuda").bfloat16()
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 2.0 ** -60
    w = torch.ones(256, device="cuda")
    y, _ = kda.rms_norm(x, w, eps=0.0)
    assert torch.isfinite(y[[0, 4, 5]]).all() and torch.isnan(y[2]).all()
    y, _ = kda.rms_norm(x, w)
    assert torch.all(y[1] == 0) and torch.all(y[3, :7] == 0) and torch.isnan(y[3, 7])
    y8, scale, _ = kda.rms_norm_quant(x, w, quant=quant, group=128)
    assert torch.all(y8[1].float() == 0) and torch.all(scale[1] > 0) and torch.isfinite(scale[[0, 1, 4, 5]]).all()
    assert torch.isnan(scale[2]).all() and torch.isnan(scale[3, 0]) and torch.all(y8[3, 128:].float() == 0)
    assert torch.isfinite(y8[[0, 1, 4, 5]].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SHAPES + [(1000, 64), (2500, 512), (0, 64)])
def test_backward(dtype, rows, D):
    x, _, w, dy, dr = _inputs(rows, D, dtype, seed=5)
    for weight, extra in ((w, dr), (None, None)):
        dx, dw = kda.rms_norm_backward(x, weight, dy, grad_residual=extra, eps=1e-5)
        f, g = x.double(), dy.double() * (1.0 if weight is None else weight.double())
        c = 1 / (f.square().mean(1, keepdim=True) + 1e-5).sqrt()
        back = f * c.pow(3) * (f * g).mean(1, keepdim=True)
        ref = c * g - back + (0.0 if extra is None else extra.double())
        # sum of the absolute values of the terms: the mean of f g is one over D signed products
        mag = c * g.abs() + f.abs() * c.pow(3) * (f * g).abs().mean(1, keepdim=True) + (0.0 if extra is None else extra.double().abs())
        step = HALF_BF16 if dtype == "bf16" else 0.0
        assert ((dx.double() - ref).abs() <= 2 * F32 * mag + step * (ref.abs() + 2 * F32 * mag) + 1e-37).all()
        # rows are added in at most rows / 592 + 64 fp32 steps
        terms = (dy.double() * f * c)
        assert ((dw.double() - terms.sum(0)).abs() <= (F32 + (rows / 592 + 64) * 2.0 ** -24) * terms.abs().sum(0) + 1e-37).all()
        again, dw2 = kda.rms_norm_backward(x, weight, dy, grad_residual=extra, eps=1e-5)
        assert torch.equal(dx, again) and torch.equal(dw, dw2)
    if rows:
        mine = dr.clone()
        dx, _ = kda.rms_norm_backward(x, w, dy, grad_residual=dr, eps=1e-5)
        into, none = kda.rms_norm_backward(x, w, dy, grad_residual=mine, eps=1e-5, grad_x=mine, want_grad_weight=False)
        assert into is mine and none is None and torch.equal(dx, mine)
    assert kda.get_device_status() == kda.KDA_OK


def test_backward_against_differences():
    """fp32: central differences of <y, dy> with step h along u are off by h^2 / 6 of the third derivative
    (below 60 max|u|^3 / rms^3 of the terms' sizes for these unit-size rows) and by rounding / h."""
    x, _, w, dy, _ = _inputs(40, 256, "f32", seed=9)
    dx, dw = kda.rms_norm_backward(x, w, dy)
    u = torch.rand(x.shape, generator=torch.Generator().manual_seed(10)).cuda() - 0.5
    h = 2.0 ** -7

    def loss(x, w):
        return (kda.rms_norm(x, w)[0].double() * dy.double()).sum()

    size = (_norm64(x, w, 1e-6) * dy.double()).abs().sum()
    diff, have = (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h), (dx.double() * u.double()).sum()
    assert abs(diff - have) <= h * h / 6 * 60 * 0.125 * size + 2 * F32 * size / h
    uw = u[0]
    diff, have = (loss(x, w + uw) - loss(x, w - uw)) / 2, (dw.double() * uw.double()).sum()
    assert abs(diff - have) <= 4 * F32 * size


def test_leading_dimensions_captured_call_and_many_rows():
    x, res, w, dy, _ = _inputs(6 * 5, 128, "bf16")
    y, r = kda.rms_norm(x.view(6, 5, 128), w, residual=res.view(6, 5, 128))
    flat, _ = kda.rms_norm(x, w, residual=res)
    assert y.shape == (6, 5, 128) and torch.equal(y.view(30, 128), flat)
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.rms_norm(x, w, y=out)
        dx, dw = kda.rms_norm_backward(x, w, dy)
    x.copy_(res)
    graph.replay()
    torch.cuda.synchronize()
    want, (wx, ww) = kda.rms_norm(x, w)[0], kda.rms_norm_backward(x, w, dy)
    assert torch.equal(out, want) and torch.equal(dx, wx) and torch.equal(dw, ww)
    # rows x D past 31 bits of bytes and elements
    rows = (1 << 31) // 1024 + 3
    big = torch.ones(rows, 1024, device="cuda", dtype=torch.bfloat16)
    big[-1, ::2] = 3.0
    y, _ = kda.rms_norm(big, None, eps=0.0, y=big.new_empty(rows, 1024))
    assert torch.all(y[:-1] == 1) and torch.equal(y[-1], kda.rms_norm(big[-1:].contiguous(), None, eps=0.0)[0][0])


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
def test_bytes_of_values_near_the_type_s_ends(quant):
    """Outputs near fp32's largest and near 2^-100: the top of each group is stored as the type's largest value."""
    top = 448.0 if quant == "e4m3" else 127.0
    x = torch.ones(3, 64, device="cuda")
    for size in (2.5e38, 1.0, 2.0 ** -99):
        y8, scale, _ = kda.rms_norm_quant(x, torch.full((64,), size, device="cuda"), eps=0.0, quant=quant, group=32)
        assert torch.all(y8.float() == top)
        assert torch.allclose(scale.double(), torch.tensor(size / top, dtype=torch.float64, device="cuda"), rtol=2.0 ** -21, atol=0.0)
