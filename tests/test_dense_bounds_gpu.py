"""Sharper bounds of the dense row operators on the GPU: exact row sums, single products, non-finite rows.

Where an answer is exact in every order of summation it is compared bit for bit. Elsewhere the tolerances count:
  - a float32 operand is split into three bfloat16 parts: truncated, rounded, and the rest. With the leading bit 1 the
    second is at most 2^-7 and the third at most 2^-16, so what the six products leave out is below 2^-22 of a
    product; the last of the six is added with one truncation (2^-23), those before it are 2^-6 of it and smaller.
    The parts add up to the operand exactly from 2^-110 up; below, to within 2^-133 (bfloat16's smallest subnormal);
  - the backward's dz of bfloat16 operands is two bfloat16 parts: within 2^-16 of it;
  - exp(-z): the argument z log2(e) is rounded (2^-24 of it) and log2(e) is off by 2^-26 of itself, so exp is off by
    1.25 |z| 2^-24 of its own size, and by 2^-22 for the approximate 2^x;
  - storing rounds by half a step (torch.finfo(t).eps / 2).
What test_dense_gpu.py asserts is wider: a float32 2-norm error of 2^-20 of the result's norm plus 2^-6 of the norm of
the elementwise slack (at 38,000 rows and more that is several hundred times 2^-20 for grad_W, so lost rows are looked
for here, on exact sums); an activation off by 2^-20 (1 + |z|), not by a fixed part of its own size; gradients of
bfloat16 layers as if dz were rounded to bfloat16.
"""
import numpy as np
import pytest
import torch

import cg_tensor_products_b200 as etp
import test_dense_gpu as base
from oracle import dense

pytestmark = pytest.mark.gpu

DTYPES = base.DTYPES
_np, _rand = base._np, base._rand


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _ints(gen, dtype, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(1, 5, 3), (515, 24, 300), (1000, 99, 37), (70001, 64, 96), (38017, 131, 257),
                                   (40000, 256, 256), (131149, 200, 128), (65537, 40, 20)])
def test_sums_over_rows_are_exact_on_small_integers(M, K, N, dtype):
    """Every row counts once: sums of small integers stay exact in float32 in any order, so grad_W and grad_bias are
    the true sums rounded once. grad_bias alone is the same."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + K + N)
    x, g = _ints(gen, dtype, M, K), _ints(gen, dtype, M, N)
    W = _ints(gen, dtype, K, N)
    gx, gW, gb = etp.linear_backward(x, W, g)
    assert torch.equal(gx, (g.double() @ W.double().T).to(dtype))
    assert torch.equal(gW, (x.double().T @ g.double()).to(dtype))
    assert torch.equal(gb, g.double().sum(0).to(dtype))
    assert torch.equal(etp.linear_backward(x, W, g, want=("bias",))[2], gb)
    out = etp.linear_forward(x, W)
    assert torch.equal(out, (x.double() @ W.double()).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(70001, 4352), (131149, 33), (300000, 1)])
def test_bias_gradient_alone(M, N, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    g = _ints(gen, dtype, M, N)
    x, W = torch.zeros(M, 1, device="cuda", dtype=dtype), torch.zeros(1, N, device="cuda", dtype=dtype)
    only = etp.linear_backward(x, W, g, want=("bias",))
    assert only[0] is None and only[1] is None and torch.equal(only[2], g.sum(0, dtype=torch.float64).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(70001, 64, 96), (40000, 256, 256), (38017, 131, 257)])
def test_sums_over_rows_through_the_activation(M, K, N, dtype):
    """The same with dz = g silu'(0) = g / 2 (silu'(0) within 8 roundings of 1/2): one lost row moves an element by
    1/2 or more, far above the tolerance in float32; in bfloat16 also the 2-norm of the rounded sums."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    x, g = _ints(gen, dtype, M, K), _ints(gen, dtype, M, N)
    _, gW, gb = etp.linear_backward(x, _ints(gen, dtype, K, N), g, torch.zeros_like(g), "silu", want=("W", "bias"))
    half = torch.finfo(dtype).eps / 2
    for got, a, b in ((gW, x, g), (gb[None], torch.ones_like(x[:, :1]), g)):
        want, size = a.double().T @ b.double() / 2, a.double().abs().T @ b.double().abs() / 2
        assert bool(((got.double() - want).abs() <= half * want.abs() + 2.0**-21 * size).all())
        assert float((got.double() - want).norm()) <= (half + 2.0**-20) * float(want.norm()) + 2.0**-21 * float(size.norm())


@pytest.mark.parametrize("M,K,N", [(300, 99, 37), (4096, 256, 256), (5000, 64, 96), (1000, 131, 515), (2, 64, 4352),
                                   (20000, 300, 128), (129, 520, 1030)])
def test_bfloat16_backward_keeps_the_activations_gradient(M, K, N):
    """dz = g silu'(z) enters the products of bfloat16 operands to 2^-16, not rounded to bfloat16 (2^-8)."""
    normal = _rand(K + N)
    bf = torch.bfloat16
    x, W = normal(M, K, dtype=bf), normal(K, N, dtype=bf, scale=K**-0.5)
    z, g = normal(M, N, dtype=bf, scale=2.0), normal(M, N, dtype=bf)
    gx, gW, gb = etp.linear_backward(x, W, g, z, "silu")
    xn, Wn, zn, gn = (_np(t) for t in (x, W, z, g))
    rx, rW, rb = dense.linear_backward(xn, Wn, gn, zn, "silu")
    # dz: two parts, the approximate exp and 1/x and six roundings; the sums: two truncated additions (2^-23) per 16
    # terms, the sums of ranges (one rounding each, below 256 of them)
    dz = np.abs(gn * dense.act_grad(zn, "silu"))
    off = 2.0**-16 * dz + 2.0**-20 * (1 + np.abs(zn)) * np.abs(gn)
    xa, Wa = np.abs(xn), np.abs(Wn)
    base._close(gx, rx, (8 + N / 8) * 2.0**-23 * (dz @ Wa.T) + off @ Wa.T, "grad_x")
    base._close(gW, rW, (8 + M / 8) * 2.0**-23 * (xa.T @ dz) + xa.T @ off, "grad_W")
    base._close(gb, rb, (8 + M / 8) * 2.0**-23 * dz.sum(0) + 2.0**-20 * ((1 + np.abs(zn)) * np.abs(gn)).sum(0), "grad_bias")
    assert etp.device_fault() == 0


def _dropped(x, w):
    """What the six part products of float32 x and w leave out (float64)."""
    def parts(v):
        p0 = (v.contiguous().view(torch.int32) & -65536).view(torch.float32)
        p1 = (v - p0).bfloat16().float()
        return p0.double(), p1.double(), (v - p0 - p1).double()

    a, b = parts(x), parts(w)
    return (a[1] * b[2] + a[2] * b[1] + a[2] * b[2]).abs()


@pytest.mark.parametrize("M,N", [(1, 1), (130, 40), (40000, 256)])
def test_float32_single_products(M, N):
    """One product per output (every other term zero), at mantissas whose dropped parts are largest: no more is
    missing than the split drops, and twice a truncation of the last addition."""
    worst = [1 + 2.0**-7 - 2.0**-23, 1 + 2.0**-7 - 2.0**-16, 1 + 2.0**-7 - 2.0**-15 + 2.0**-23, 1 + 2.0**-8 + 2.0**-16 - 2.0**-23,
             2 - 2.0**-23, 1 + 2.0**-23, 1.0, 1 + 2.0**-7 - 2.0**-15 - 2.0**-16, -(1 + 2.0**-7 - 2.0**-17 + 2.0**-22)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    pick = lambda *s: torch.tensor(worst, device="cuda")[torch.randint(0, len(worst), s, generator=gen, device="cuda")]

    def check(got, a, b):
        want, dropped = a.double() * b.double(), _dropped(a, b)
        assert bool((dropped < 2.0**-22 * want.abs()).all())
        assert bool(((got.double() - want).abs() <= dropped + (2.0**-22 + 2.0**-28) * want.abs()).all())

    x, W, g = pick(M, 1), pick(1, N), pick(M, N)
    x[0], W[0, 0], g[0, 0] = worst[0], worst[0], worst[0]
    check(etp.linear_forward(x, W), x, W)
    # grad_x: one column of grad_out that is not zero; grad_W: one row
    g1 = torch.zeros_like(g)
    g1[:, 0] = g[:, 0]
    check(etp.linear_backward(x, W, g1, want=("x",))[0], g1[:, :1], W[:, :1])
    g0 = torch.zeros_like(g)
    g0[M // 2] = g[0]
    check(etp.linear_backward(x, W, g0, want=("W",))[1], x[M // 2:M // 2 + 1], g0[M // 2:M // 2 + 1])


def test_float32_operands_of_all_magnitudes():
    """Subnormal and tiny operands against large ones: the operand to 2^-133, then the products' tolerance."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    exps = torch.arange(-149, 20, device="cuda", dtype=torch.float64)
    x = (2.0**exps * (1 + torch.rand(len(exps), generator=gen, device="cuda", dtype=torch.float64))).float()[:, None]
    x = torch.cat([x, -x, torch.tensor([[2.0**-120 * (1 + 2.0**-14)], [2.0**-126], [2.0**-149], [0.0]], device="cuda")])
    W = torch.tensor([[2.0**100, -(2.0**99) * (1 + 2.0**-7 - 2.0**-23), 1.5 * 2.0**80]], device="cuda")
    want = x.double() * W.double()
    tol = (2.0**-21 + 2.0**-28) * want.abs() + 2.0**-133 * W.double().abs()
    assert bool(((etp.linear_forward(x, W).double() - want).abs() <= tol).all())


def test_silu_of_large_pre_activations():
    """Relative to its own size: s = 1 / (1 + exp(-z)) within e = (1.25 |z| + 8) 2^-24 (argument, 2^x: 4, sum 1, 1/x:
    2), silu with one rounding more; silu' = s (1 + z (1 - s)) by the same count, and as an operand of grad_x's product
    it is split: to within 2^-133 (it falls to 2^-118 here)."""
    z = torch.cat([torch.linspace(-86, 86, 20001, device="cuda"), -torch.logspace(-6, 1.9, 5000, device="cuda")])[:, None]
    one = torch.ones(1, 1, device="cuda")
    out, zz = etp.linear_forward(z, one, None, "silu", save_z=True)
    assert torch.equal(zz, z)
    zn = _np(z)
    s, e = dense.sigmoid(zn), (1.25 * np.abs(zn) + 8) * 2.0**-24
    ref = dense.act(zn, "silu")
    assert (np.abs(_np(out) - ref) <= (e + 2.0**-24) * np.abs(ref)).all()
    gx = etp.linear_backward(z, one, torch.ones_like(z), zz, "silu", want=("x",))[0]
    q = 1 + zn * (1 - s)
    slack = s * (np.abs(zn) * (s * e + 2.0**-24 * (1 - s)) + 2.0**-23 * np.abs(q) + np.abs(q) * (e + 2.0**-22))
    assert (np.abs(_np(gx) - s * q) <= slack + 2.0**-133).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(5000, 515), (5000, 1032), (2500, 1025), (2500, 2056), (1500, 5001), (1500, 8192), (3000, 257)])
def test_layer_norm_several_rows_a_block(M, C, dtype):
    """Wide rows that a whole block takes, more of them than blocks: a block's second and later rows."""
    normal = _rand(M + C)
    x = normal(M, C, dtype=dtype, scale=2.0, shift=0.7)
    base._check_norm(x, normal(C, dtype=dtype, scale=0.2, shift=1.0), normal(C, dtype=dtype), normal(M, C, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [1, 31, 64, 515, 1024, 2056])
def test_layer_norm_statistics_of_non_finite_rows(C, dtype):
    """A row with a NaN or an infinity has no statistics: mean is not finite, rstd is NaN, gradients of it are NaN."""
    normal = _rand(C)
    x, g = normal(40, C, dtype=dtype), normal(40, C, dtype=dtype)
    want = etp.layer_norm_forward(x)
    bad = x.clone()
    bad[3, C // 2], bad[17, 0], bad[39, C - 1] = float("nan"), float("inf"), -float("inf")
    rows, rest = [3, 17, 39], [r for r in range(40) if r not in (3, 17, 39)]
    out, mean, rstd = etp.layer_norm_forward(bad)
    assert bool(out[rows].isnan().all()) and not bool(mean[rows].isfinite().any()) and bool(rstd[rows].isnan().all())
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip((out, mean, rstd), want))
    gx = etp.layer_norm_backward(bad, None, mean, rstd, g, want=("x",))[0]
    assert bool(gx[rows].isnan().all()) and bool(gx[rest].isfinite().all())


def test_layer_norm_gradients_of_rows_with_a_large_offset():
    """The backward takes the mean as it is stored, in float32: xh is off by half a step of it, 2^-24 |mean| rstd.
    Against gradients from the unrounded mean."""
    normal = _rand(2)
    C = 200
    x, g = normal(64, C, shift=1e4), normal(64, C)
    _, mean, rstd = etp.layer_norm_forward(x)
    xn, gn = _np(x), _np(g)
    _, m64, r64 = dense.layer_norm_forward(xn)
    gx, gw, gb = etp.layer_norm_backward(x, None, mean, rstd, g)
    rx, rw, rb = dense.layer_norm_backward(xn, None, m64, r64, gn)
    d = (2.0**-23 * np.abs(m64) * r64)[:, None]  # half a step of the mean, and as much for its own sum
    ga, xh = np.abs(gn), np.abs((xn - m64[:, None]) * r64[:, None])
    assert (np.abs(_np(gw) - rw) <= ((d + 2.0**-18 * xh) * ga).sum(0)).all()
    assert (np.abs(_np(gb) - rb) <= 2.0**-20 * ga.sum(0)).all()
    # r (gw - mean(gw) - xh mean(gw xh)), rstd itself within 2^-18
    gxh = (ga * xh).mean(1, keepdims=True)
    slack = r64[:, None] * (2.0**-18 * (ga + ga.mean(1, keepdims=True) + xh * gxh) + d * gxh + (xh + d) * d * ga.mean(1, keepdims=True))
    assert (np.abs(_np(gx) - rx) <= slack).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_outputs_beside_their_inputs(dtype):
    """Channels of one rank written from other channels of the same rows."""
    normal = _rand(31)
    f = normal(300, 16, 128, dtype=dtype)
    keep, W, gamma = f.clone(), normal(64, 48, dtype=dtype), normal(64, dtype=dtype)
    a, b, c = f[:, 4:9, :64], f[:, 4:9, 64:112], f[:, 4:9, 64:]
    want = etp.linear_forward(a, W)
    etp.linear_forward(a, W, out=b)
    assert torch.equal(b, want)
    f.copy_(keep)
    want = etp.layer_norm_forward(a, gamma)
    etp.layer_norm_forward(a, gamma, out=c)
    assert torch.equal(c, want[0])
    f.copy_(keep)
    gx = etp.layer_norm_backward(c, gamma, *want[1:], a, want=("x",))[0]
    etp.layer_norm_backward(c, gamma, *want[1:], f[:, 9:14, :64].copy_(a), want=("x",), grad_x=a)
    assert torch.equal(a, gx)
    rest = [d for d in range(16) if not 4 <= d < 14]
    assert torch.equal(f[:, rest], keep[:, rest])
    with pytest.raises(ValueError, match="must not overlap"):
        etp.linear_forward(a, W, out=f[:, 4:9, 63:111])


def _delay(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


def test_what_a_call_creates_belongs_to_its_stream():
    """stream=s: results that are dropped at once, blocks freed on the current stream with work still queued there,
    and results dropped while the current stream still reads them."""
    normal = _rand(37)
    M, K, N = 20000, 256, 192
    x, W, g, gamma = normal(M, K), normal(K, N), normal(M, N), normal(K)
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    out, z = etp.linear_forward(x, W, None, "silu", save_z=True)
    ln, lb = etp.layer_norm_forward(x, gamma), etp.linear_backward(x, W, g, z, "silu")
    nb = etp.layer_norm_backward(x, gamma, *ln[1:], x)
    torch.cuda.synchronize()
    # all but one result dropped while s has not begun: their memory is not the current stream's to give away
    for call, want in ((lambda: etp.layer_norm_forward(x, gamma, stream=s)[0], ln[0]),
                       (lambda: etp.linear_backward(x, W, g, z, "silu", stream=s)[1], lb[1]),
                       (lambda: etp.linear_forward(x, W, None, "silu", save_z=True, stream=s)[0], out),
                       (lambda: etp.layer_norm_backward(x, gamma, *ln[1:], x, stream=s)[2], nb[2])):
        _delay(s)
        got = call()
        fill = [torch.full(n, 7.0, device="cuda") for n in ((M,), (M,), (N,), (K,), (K, N), (M, N), (M, K)) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(bool((f == 7.0).all()) for f in fill)
        del got, fill
    # memory freed on the current stream, whose writes to it are still queued
    _delay(here)
    for _ in range(3):
        old = torch.full((M, N), 3.0, device="cuda")
        del old
    got = etp.linear_forward(x, W, None, "silu", stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    # results that the current stream reads after they were dropped
    for _ in range(2):
        got = etp.linear_forward(x, W, None, "silu", stream=s)
        here.wait_stream(s)
        _delay(here)
        later = got + 0.0
        del got
        other = etp.linear_forward(x, W, None, "none", stream=s)
        torch.cuda.synchronize()
        assert torch.equal(later, out)
        del other, later
    # a caller's own output, and a call that is already on its stream
    mine = torch.empty_like(out)
    assert etp.linear_forward(x, W, None, "silu", out=mine, stream=s) is mine
    with torch.cuda.stream(s):
        again = etp.linear_forward(x, W, None, "silu", stream=s)
    torch.cuda.synchronize()
    assert torch.equal(mine, out) and torch.equal(again, out)
