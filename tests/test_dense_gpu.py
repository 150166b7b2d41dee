"""The dense row operators on the GPU against the float64 oracle.

Tolerances, per element, with S the sum of the absolute values that the element adds up:
  - float32 products: each operand is split exactly, products dropped or rounded are below 2^-22, and at most
    four truncated (2^-23) and two rounded (2^-24) additions per 64 terms touch a partial sum, so the error is below
    (8 + T / 8) 2^-23 S for T terms; as a vector (2-norm) the errors of T random terms stay below 2^-20;
  - bfloat16 products: T / 16 truncated additions (2^-23) in one accumulator, within the same bound;
  - the activation: exp within 4 ulp of its own size and a handful of roundings, 2^-20 (1 + |z|);
  - dz = grad_out act'(z) of bfloat16 operands enters the products rounded to bfloat16, 2^-8 of each dz (not the
    bias gradient, and not without an activation, where dz is grad_out itself);
  - storing bfloat16 adds half a step, 2^-8 of the value (torch.finfo(t).eps / 2); inputs are taken as given.
"""
import numpy as np
import pytest
import torch

import cg_tensor_products_b200 as etp
import oracle
from gpu_helpers import rel_err
from oracle import dense

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rand(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    return normal


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, ref, slack, what="", random=True):
    """|got - ref| <= half a step of got's type + slack, elementwise; in float32 also 2^-20 of the 2-norm where the
    terms of a sum are random (n equal terms t round the same way at every step: up to sum_k k t 2^-24, which is
    n / 2 steps of 2^-24 of the sum and no 2^-20 for n > 32)."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    g = _np(got)
    assert np.isfinite(g).all(), what
    half = torch.finfo(got.dtype).eps / 2
    slack = np.broadcast_to(slack, ref.shape)
    off = np.abs(g - ref) - half * (np.abs(ref) + slack) - slack
    assert off.size == 0 or off.max() <= 0, (what, float(off.max()))
    norm = np.linalg.norm(ref)
    if random and got.dtype == torch.float32 and norm > 0 and ref.size >= 64:
        assert np.linalg.norm(g - ref) <= 2.0**-20 * norm + np.linalg.norm(slack) * 2.0**-6, (
            what, float(np.linalg.norm(g - ref) / norm))


def _sum_slack(a, b, terms):
    return (8 + terms / 8) * 2.0**-23 * (np.abs(a) @ np.abs(b))


def _check_linear(x, W, bias, activation, residual, grad_out, random=True):
    """Forward with z kept, then all gradients, against the oracle."""
    K, N = W.shape
    out, z = etp.linear_forward(x, W, bias, activation, residual, save_z=True)
    xn, Wn, bn, rn, gn = (_np(t) for t in (x, W, bias, residual, grad_out))
    ref, zref = dense.linear_forward(xn, Wn, bn, activation, rn)
    flat = lambda a: a.reshape(-1, a.shape[-1])
    zs = _sum_slack(flat(xn), Wn, K).reshape(zref.shape) + 2.0**-22 * (0 if bn is None else np.abs(bn))
    _close(z, zref, zs, "z")
    as_ = 1.1 * zs + 2.0**-20 * (1 + np.abs(zref)) * (activation == "silu")
    _close(out, ref, as_ + 2.0**-22 * (0 if rn is None else np.abs(rn)), "out")
    alone = etp.linear_forward(x, W, bias, activation, residual)
    assert torch.equal(alone, out)
    zk = _np(z)
    gx, gW, gb = etp.linear_backward(x, W, grad_out, z, activation)
    rx, rW, rb = dense.linear_backward(xn, Wn, gn, zk, activation)
    dz = np.abs(gn * dense.act_grad(zk, activation))
    dslack = 2.0**-20 * (1 + np.abs(zk)) * np.abs(gn) * (activation == "silu")
    operand = dslack + (2.0**-8 * dz if activation == "silu" and x.dtype == torch.bfloat16 else 0)
    _close(gx, rx, _sum_slack(flat(dz), Wn.T, N).reshape(rx.shape) + operand @ np.abs(Wn.T), "grad_x")
    xf, df, M = flat(np.abs(xn)), flat(dz), flat(xn).shape[0]
    _close(gW, rW, _sum_slack(xf.T, df, M) + xf.T @ flat(operand), "grad_W", random)
    _close(gb, rb, (8 + M / 8) * 2.0**-23 * df.sum(0) + flat(dslack).sum(0), "grad_bias", random)
    again = etp.linear_backward(x, W, grad_out, z, activation)
    assert all(torch.equal(a, b) for a, b in zip(again, (gx, gW, gb)))
    assert etp.device_fault() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N,activation", [
    (1, 1, 1, "silu"), (1, 128, 128, "silu"), (2, 3, 5, "none"), (7, 64, 1, "silu"), (127, 8, 64, "silu"),
    (128, 64, 128, "none"), (129, 65, 129, "silu"), (300, 99, 37, "silu"), (64, 500, 20, "silu"),
    (1000, 128, 128, "silu"), (515, 24, 300, "none"), (33, 1030, 130, "silu"), (5000, 16, 16, "silu"),
    (2, 128, 4352, "none"), (777, 256, 512, "silu")])
def test_linear(M, K, N, activation, dtype):
    normal = _rand(M + 31 * K + 7 * N)
    x, W = normal(M, K, dtype=dtype), normal(K, N, dtype=dtype, scale=K**-0.5)
    _check_linear(x, W, normal(N, dtype=dtype), activation, normal(M, N, dtype=dtype), normal(M, N, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nodes,L,l,K,N", [(50, 3, 0, 128, 128), (61, 3, 2, 128, 64), (40, 2, 1, 12, 20),
                                           (1, 3, 3, 64, 64), (129, 1, 1, 7, 9)])
def test_linear_on_blocks_of_features(nodes, L, l, K, N, dtype):
    """One rank's rows read and written in place inside feature tensors; the other ranks stay as they were."""
    normal = _rand(nodes + l)
    D, block = (L + 1) ** 2, slice(l * l, (l + 1) ** 2)
    feats, res = normal(nodes, D, K, dtype=dtype), normal(nodes, D, N, dtype=dtype)
    W, g = normal(K, N, dtype=dtype, scale=K**-0.5), normal(nodes, D, N, dtype=dtype)
    _check_linear(feats[:, block], W, None, "none", res[:, block], g[:, block])
    keep = res.clone()
    want = etp.linear_forward(feats[:, block], W, None, "silu", res[:, block])
    etp.linear_forward(feats[:, block], W, None, "silu", res[:, block], out=res[:, block])  # in place
    assert torch.equal(res[:, block], want)
    gx = torch.full_like(feats, 7.0)
    ref = etp.linear_backward(feats[:, block], W, g[:, block], want=("x",))[0]
    etp.linear_backward(feats[:, block], W, g[:, block], want=("x",), grad_x=gx[:, block])
    assert torch.equal(gx[:, block], ref)
    rest = [d for d in range(D) if not block.start <= d < block.stop]
    assert torch.equal(res[:, rest], keep[:, rest]) and bool((gx[:, rest] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_strides_and_broadcasts(dtype):
    """Rows at an odd pitch, an unaligned base, one row used for all, groups of one and one group."""
    normal = _rand(5)
    buf = normal(200, 77, dtype=dtype)
    W, b = normal(64, 40, dtype=dtype, scale=0.125), normal(40, dtype=dtype)
    g = normal(200, 40, dtype=dtype)
    _check_linear(buf[:, 3:67], W, b, "silu", normal(1, 40, dtype=dtype).expand(200, 40), g)
    _check_linear(buf[:1, 1:65].expand(200, 64), W, b, "silu", None, normal(1, 40, dtype=dtype).expand(200, 40),
                  random=False)
    _check_linear(normal(1, 150, 64, dtype=dtype), W, b, "silu", None, normal(1, 150, 40, dtype=dtype))
    wide = normal(30, 5, 128, dtype=dtype)
    _check_linear(wide[:, ::2, 64:], W, b, "silu", None, normal(30, 3, 40, dtype=dtype))
    _check_linear(wide.transpose(0, 1)[..., :64], W, b, "none", None, normal(5, 30, 40, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(70001, 64, 96), (30001, 48, 600), (38001, 200, 264), (40000, 256, 256), (38017, 131, 257)])
def test_linear_many_rows(M, K, N, dtype):
    """More rows than one pass of the GPU takes, with the weight gradients summed over all of them."""
    normal = _rand(9 + K)
    x, W = normal(M, K, dtype=dtype), normal(K, N, dtype=dtype, scale=K**-0.5)
    _check_linear(x, W, normal(N, dtype=dtype), "silu", normal(M, N, dtype=dtype), normal(M, N, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_partial_wants_and_empty(dtype):
    normal = _rand(3)
    x, W, g = normal(300, 48, dtype=dtype), normal(48, 80, dtype=dtype), normal(300, 80, dtype=dtype)
    gx, gW, gb = etp.linear_backward(x, W, g)
    assert torch.equal(etp.linear_backward(x, W, g, want=("x",))[0], gx)
    assert torch.equal(etp.linear_backward(x, W, g, want=("W",))[1], gW)
    only = etp.linear_backward(x, W, g, want=("bias",))
    assert only[0] is None and only[1] is None and torch.equal(only[2], gb)
    for shape in ((0, 48), (0, 3, 48), (5, 0, 48)):
        e, ge = torch.empty(shape, device="cuda", dtype=dtype), torch.empty((*shape[:-1], 80), device="cuda", dtype=dtype)
        assert etp.linear_forward(e, W).shape == ge.shape
        gx, gW, gb = etp.linear_backward(e, W, ge)
        assert gx.shape == e.shape and not gW.any() and not gb.any()


def test_linear_values_at_the_edges():
    """Large negative and positive pre-activations, subnormal and large operands, and non-finite rows that
    stay in their own outputs."""
    z = torch.tensor([[-1e4, -90.0, -40.0, 0.0, 40.0, 1e4, 3e38, 1e-30]], device="cuda").t().contiguous()
    one = torch.ones(1, 1, device="cuda")
    out, zz = etp.linear_forward(z, one, None, "silu", save_z=True)
    assert torch.equal(zz, z)
    assert np.allclose(_np(out), dense.act(_np(z), "silu"), rtol=2.0**-20, atol=1e-36)
    gx = etp.linear_backward(z, one, torch.ones_like(z), zz, "silu", want=("x",))[0]
    assert np.allclose(_np(gx), dense.act_grad(_np(z), "silu"), rtol=2.0**-20, atol=1e-15)
    for dtype in DTYPES:
        normal = _rand(4)
        x, W = normal(200, 70, dtype=dtype), normal(70, 50, dtype=dtype)
        want = etp.linear_forward(x, W)
        bad = x.clone()
        bad[17, 3], bad[150, 69], bad[199, 0] = float("nan"), float("inf"), -float("inf")
        got = etp.linear_forward(bad, W)
        rest = [r for r in range(200) if r not in (17, 150, 199)]
        assert torch.equal(got[rest], want[rest]) and not bool(torch.isfinite(got[[17, 150, 199]]).any())


def _check_norm(x, weight, bias, grad_out, eps=1e-5):
    out, mean, rstd = etp.layer_norm_forward(x, weight, bias, eps)
    xn, wn, bn, gn = (_np(t) for t in (x, weight, bias, grad_out))
    C = xn.shape[-1]
    ref, mref, rref = dense.layer_norm_forward(xn, wn, bn, eps)
    sum_eps = (4 + np.log2(C) + C / 256) * 2.0**-24  # additions in a chain: per lane, then over the lanes
    size = np.abs(xn).mean(-1)
    _close(mean, mref, sum_eps * size, "mean")
    rs = 4 * sum_eps + 2 * (sum_eps * size * rref) ** 2
    assert np.max(np.abs(_np(rstd) - rref) / rref, initial=0) <= rs.max(initial=0), "rstd"
    wa = 1.0 if wn is None else np.abs(wn)
    xh = np.abs((xn - mref[..., None]) * rref[..., None])
    slack = wa * (xh * (rs[..., None] + 2.0**-22) + (sum_eps * size * rref)[..., None] + 2.0**-23)
    _close(out, ref, slack + 2.0**-23 * (0 if bn is None else np.abs(bn)), "out")
    gx, gw, gb = etp.layer_norm_backward(x, weight, mean, rstd, grad_out)
    rx, rw, rb = dense.layer_norm_backward(xn, weight if wn is None else wn, _np(mean), _np(rstd), gn)
    r = _np(rstd)[..., None]
    ga = wa * np.abs(gn)
    gmean, gxh = ga.mean(-1, keepdims=True), (ga * xh).mean(-1, keepdims=True)
    _close(gx, rx, r * (2.0**-22 * ga + (sum_eps + 2.0**-22) * (gmean + (1 + xh) * gxh)), "grad_x")
    M = max(1, int(np.prod(xn.shape[:-1])))
    chain = (8 + M / 64) * 2.0**-24
    flat = lambda a: a.reshape(-1, C)
    _close(gw, rw, (chain + 2.0**-22) * flat(np.abs(gn) * (xh + 2.0**-22)).sum(0), "grad_weight")
    _close(gb, rb, chain * flat(np.abs(gn)).sum(0), "grad_bias")
    again = etp.layer_norm_backward(x, weight, mean, rstd, grad_out)
    assert all(torch.equal(a, b) for a, b in zip(again, (gx, gw, gb)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(1, 1), (3, 2), (1, 128), (37, 4), (1000, 8), (129, 31), (50, 64), (300, 100),
                                 (64, 257), (40, 515), (30, 1000), (20, 1024), (9, 1025), (12, 1028), (6, 4096),
                                 (3, 5001), (2, 8192), (20011, 128), (5000, 7)])
def test_layer_norm(M, C, dtype):
    normal = _rand(M + 13 * C)
    x = normal(M, C, dtype=dtype, scale=2.0, shift=0.7)
    _check_norm(x, normal(C, dtype=dtype, scale=0.2, shift=1.0), normal(C, dtype=dtype), normal(M, C, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_strides_in_place_and_optional_parts(dtype):
    normal = _rand(8)
    feats, g = normal(70, 16, 128, dtype=dtype), normal(70, 16, 128, dtype=dtype)
    w, b = normal(128, dtype=dtype, shift=1.0), normal(128, dtype=dtype)
    _check_norm(feats[:, :1], w, b, g[:, :1])
    _check_norm(feats[:, 1:4], w, None, g[:, 1:4])
    _check_norm(feats[:, 4:9, 1:100], None, b[:99].clone(), g[:, 4:9, 3:102])
    _check_norm(feats[:, 5], None, None, g[:, 0])
    _check_norm(normal(1, 128, dtype=dtype).expand(90, 128), w, b, normal(1, 128, dtype=dtype).expand(90, 128))
    keep = feats.clone()
    want, mean, rstd = etp.layer_norm_forward(feats[:, :1], w, b)
    ref = etp.layer_norm_backward(feats[:, :1], w, mean, rstd, g[:, :1])
    got = etp.layer_norm_backward(feats[:, :1], w, mean, rstd, g[:, :1], want=("x",))
    assert torch.equal(got[0], ref[0]) and got[1] is None and got[2] is None
    got = etp.layer_norm_backward(feats[:, :1], w, mean, rstd, g[:, :1], want=("weight",))
    assert torch.equal(got[1], ref[1]) and got[0] is None and got[2] is None
    gcopy = g.clone()
    etp.layer_norm_backward(feats[:, :1], w, mean, rstd, gcopy[:, :1], grad_x=gcopy[:, :1])
    assert torch.equal(gcopy[:, :1], ref[0]) and torch.equal(gcopy[:, 1:], g[:, 1:])
    etp.layer_norm_forward(feats[:, :1], w, b, out=feats[:, :1])
    assert torch.equal(feats[:, :1], want) and torch.equal(feats[:, 1:], keep[:, 1:])


def test_layer_norm_rows_that_stand_alone():
    """Constant rows, a large offset, non-finite rows that stay in their own outputs, no rows at all."""
    x = torch.full((5, 96), 3.25, device="cuda")
    out, mean, rstd = etp.layer_norm_forward(x, eps=1e-5)
    assert not out.any() and torch.equal(mean, x[:, 0]) and np.allclose(_np(rstd), 1e-5**-0.5, rtol=2.0**-22)
    normal = _rand(2)
    x = normal(64, 200, shift=1e4)
    g = normal(64, 200)
    _check_norm(x, None, None, g)
    want = etp.layer_norm_forward(x)
    bad = x.clone()
    bad[3, 7], bad[40, 0] = float("nan"), float("inf")
    got = etp.layer_norm_forward(bad)
    rest = [r for r in range(64) if r not in (3, 40)]
    assert torch.equal(got[0][rest], want[0][rest]) and bool(got[0][[3, 40]].isnan().all())
    gx = etp.layer_norm_backward(bad, None, got[1], got[2], g)[0]
    assert torch.equal(gx[rest], etp.layer_norm_backward(x, None, want[1], want[2], g)[0][rest])
    e = torch.empty((0, 32), device="cuda")
    out, mean, rstd = etp.layer_norm_forward(e)
    gx, gw, gb = etp.layer_norm_backward(e, None, mean, rstd, e)
    assert out.shape == e.shape and not gw.any() and not gb.any()


def test_streams_and_captured_graphs():
    """A side stream, and two captured graphs replayed in turn on new inputs."""
    normal = _rand(6)
    x, W, b, g = normal(3000, 64), normal(64, 64, scale=0.125), normal(64), normal(3000, 64)

    def block(x, g):
        h, mean, rstd = etp.layer_norm_forward(x, b, None)
        out, z = etp.linear_forward(h, W, b, "silu", x, save_z=True)
        gh, gW, gb = etp.linear_backward(h, W, g, z, "silu")
        return (out, *etp.layer_norm_backward(x, b, mean, rstd, gh), gW, gb)

    want = block(x, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = block(x, g)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, c) for a, c in zip(side, want))
    xs, gs = [torch.zeros_like(x) for _ in range(2)], [torch.zeros_like(g) for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(block(xs[i], gs[i]))
        graphs.append(graph)
    for i in (0, 1, 0):
        xs[i].copy_(x if i == 0 else g)
        gs[i].copy_(g if i == 0 else x)
        graphs[i].replay()
        ref = want if i == 0 else block(g, x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs[i], ref))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(1, 64, 40000), (100, 130, 19999), (129, 200, 38016), (1000, 96, 9480)])
def test_linear_few_rows_many_columns(M, K, N, dtype):
    """Several column tiles a CTA, with W converted by it and ahead of it; the transposed sizes have grad_x do the same."""
    normal = _rand(17)
    for k, n in ((K, N), (N, K)):
        x, W, b, g = (normal(*s, dtype=dtype) for s in ((M, k), (k, n), (n,), (M, n)))
        _check_linear(x, W, b, "silu", None, g)


def test_linear_largest_matrix():
    """W and grad_W of the most channels: offsets up to 2^32 elements."""
    n, dtype = 65536, torch.bfloat16
    normal = _rand(23)
    x, g = normal(2, n, dtype=dtype), normal(2, n, dtype=dtype)
    W = torch.zeros(n, n, device="cuda", dtype=dtype)
    rows, cols = [0, 1, 32767, 32768, 65534, 65535], [0, 63, 32768, 65535]
    W[rows] = normal(len(rows), n, dtype=dtype)
    out = etp.linear_forward(x, W)
    want = x[:, rows].double() @ W[rows].double()
    slack = x[:, rows].double().abs() @ W[rows].double().abs()
    assert bool(((out.double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-20 * slack).all())
    gx, gW, _ = etp.linear_backward(x, W, g, want=("x", "W"))
    want, slack = g.double() @ W[rows].double().T, g.double().abs() @ W[rows].double().abs().T
    # 65536 terms in float32 accumulators that truncate: a relative 2^-23 of the sum of magnitudes for each 16 terms
    assert bool(((gx[:, rows].double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-11 * slack).all())
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert not bool(gx[:, rest].any())
    for a, b in ((rows, slice(None)), (slice(None), cols)):
        want = x.double().T[a] @ g.double()[:, b]
        slack = x.double().T[a].abs() @ g.double()[:, b].abs()
        assert bool(((gW[a, b].double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-20 * slack).all())
    assert etp.device_fault() == 0


def test_own_workspace_on_another_stream():
    """The workspace that a call allocates for another stream is not handed to the current one while the call runs."""
    normal = _rand(19)
    x, W, g = normal(20000, 256), normal(256, 256), normal(20000, 256)
    gamma = normal(256)
    _, mean, rstd = etp.layer_norm_forward(x, gamma)
    want = (etp.linear_forward(x, W), *etp.linear_backward(x, W, g), *etp.layer_norm_backward(x, gamma, mean, rstd, g))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    need = [etp.linear_workspace_size(20000, 256, 256, "float32", b) for b in (False, True)]
    need.append(etp.layer_norm_workspace_size(20000, 256))
    runs = [lambda: (etp.linear_forward(x, W, stream=s),), lambda: etp.linear_backward(x, W, g, stream=s),
            lambda: etp.layer_norm_backward(x, gamma, mean, rstd, g, stream=s)]
    got = []
    for run, n in zip(runs, need):
        assert n > 0
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        got += run()
        junk = [torch.full((n,), 0xFF, device="cuda", dtype=torch.uint8) for _ in range(3)]
        torch.cuda.synchronize()
        del junk
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        etp.linear_workspace_size(4, 4, 4, "float16")
    assert etp.linear_workspace_size(20000, 256, 256, device="cuda") == need[0]


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_rows_and_many_rows(dtype):
    """Rows whose offsets pass 2^32 elements, and the most rows that a call takes (one row used for all of them)."""
    normal = _rand(13)
    stride = (1 << 31) - 64
    big = torch.empty(2 * stride + 128, device="cuda", dtype=dtype)
    far = big.as_strided((3, 64), (stride, 1))
    x = normal(3, 64, dtype=dtype)
    far.copy_(x)
    W = normal(64, 48, dtype=dtype)
    assert torch.equal(etp.linear_forward(far, W), etp.linear_forward(x, W))
    assert torch.equal(etp.layer_norm_forward(far)[0], etp.layer_norm_forward(x)[0])
    g = normal(3, 48, dtype=dtype)
    assert torch.equal(etp.linear_backward(far, W, g)[1], etp.linear_backward(x, W, g)[1])
    etp.linear_backward(x, W, g, want=("x",), grad_x=far)
    assert torch.equal(far, etp.linear_backward(x, W, g, want=("x",))[0])
    del big, far
    # sums of ones are exact in each range (below 2^24 terms each); joining at most 512 ranges rounds 512 times by
    # 2^-24 of a sum that never exceeds the last
    M = (1 << 31) - 129
    one = torch.ones(1, 4, device="cuda", dtype=dtype).expand(M, 4)
    _, gW, gb = etp.linear_backward(one, torch.ones(4, 4, device="cuda", dtype=dtype), one, want=("W", "bias"))
    tol = 2.0**-15 + torch.finfo(dtype).eps / 2
    assert bool(((gW.double() / M - 1).abs() <= tol).all()) and bool(((gb.double() / M - 1).abs() <= tol).all())
    assert etp.device_fault() == 0
    with pytest.raises(etp.EtpError):
        etp.linear_backward(one[:1].expand(M + 1, 4), torch.ones(4, 4, device="cuda", dtype=dtype),
                            one[:1].expand(M + 1, 4), want=("W",))


def test_two_calls_at_once():
    """Calls on two streams that overlap on the GPU, each with its own workspace."""
    normal = _rand(12)
    x, W, g = normal(50000, 96), normal(96, 160, scale=0.1), normal(50000, 160)
    want = (etp.linear_forward(x, W), *etp.linear_backward(x, W, g), *etp.layer_norm_forward(x))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((etp.linear_forward(x, W), *etp.linear_backward(x, W, g), *etp.layer_norm_forward(x)))
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    ws = torch.empty(etp.linear_workspace_size(50000, 96, 160, backward=True), dtype=torch.uint8, device="cuda")
    mine = etp.linear_backward(x, W, g, workspace=ws, stream=streams[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(mine, want[1:4]))
    with pytest.raises(etp.EtpError, match="workspace"):
        etp.linear_backward(x, W, g, workspace=ws[:16])
    assert etp.device_fault() == 0


def test_update_block_with_the_edge_tensor_product():
    """Norm and linear layers around the edge tensor product, as a model's interaction block runs them, with the
    whole VJP; against the same chain in the float64 oracle."""
    import workloads

    oracle.build()
    wl = workloads.random_graph(np.random.default_rng(0), 60, 700, 2, 16, 15)
    normal = _rand(1)
    C, D, plan = wl.C, 9, etp.Plan("0..2", 2, "0..2", wl.C)
    t = {k: torch.from_numpy(np.ascontiguousarray(getattr(wl, k))).cuda() for k in ("row_ptr", "src", "r", "x", "w", "g")}
    gamma, beta, bias = normal(C, shift=1.0, scale=0.1), normal(C), normal(C)
    Ws = [normal(C, C, scale=C**-0.5) for _ in range(3)]
    rev = etp.build_reverse_csr(wl.N, t["row_ptr"], t["src"])
    blocks = [slice(l * l, (l + 1) ** 2) for l in range(3)]

    # forward: scalars normed in place, every rank mixed, message passing, scalars updated with a residual
    h = t["x"].clone()
    _, mean, rstd = etp.layer_norm_forward(t["x"][:, :1], gamma, beta, out=h[:, :1])
    m = torch.empty_like(h)
    for b, W in zip(blocks, Ws):
        etp.linear_forward(h[:, b], W, out=m[:, b])
    a = etp.forward(plan, t["row_ptr"], t["src"], t["r"], m, t["w"])
    y = a.clone()
    s = a[:, :1].contiguous()
    _, z = etp.linear_forward(s, Ws[0], bias, "silu", a[:, :1], out=y[:, :1], save_z=True)
    # backward
    ga = t["g"].clone()
    gs, gU, gbias = etp.linear_backward(s, Ws[0], t["g"][:, :1], z, "silu")
    ga[:, :1] += gs
    gm, gw, gr = etp.backward(plan, t["row_ptr"], t["src"], *rev, t["r"], m, t["w"], ga)
    gh, gWs = torch.empty_like(h), []
    for b, W in zip(blocks, Ws):
        gWs.append(etp.linear_backward(h[:, b], W, gm[:, b], want=("x", "W"), grad_x=gh[:, b])[1])
    gx0, ggamma, gbeta = etp.layer_norm_backward(t["x"][:, :1], gamma, mean, rstd, gh[:, :1], grad_x=gh[:, :1])

    tp = oracle.OracleTP("0..2", 2, "0..2", C)
    g64 = wl.g.astype(np.float64)
    h64 = wl.x.astype(np.float64)
    h64[:, :1], mu, rs = dense.layer_norm_forward(wl.x[:, :1], _np(gamma), _np(beta))
    m64 = np.concatenate([dense.linear_forward(h64[:, b], _np(W))[0] for b, W in zip(blocks, Ws)], 1)
    a64 = tp.forward(wl.row_ptr, wl.src, wl.r, m64, wl.w.astype(np.float64))
    y64 = a64.copy()
    y64[:, :1], z64 = dense.linear_forward(a64[:, :1], _np(Ws[0]), _np(bias), "silu", a64[:, :1])
    gs64, gU64, gbias64 = dense.linear_backward(a64[:, :1], _np(Ws[0]), g64[:, :1], z64, "silu")
    ga64 = g64.copy()
    ga64[:, :1] += gs64
    ref = tp.backward(wl.row_ptr, wl.src, wl.r, m64, wl.w.astype(np.float64), ga64)
    back = [dense.linear_backward(h64[:, b], _np(W), ref["grad_x"][:, b]) for b, W in zip(blocks, Ws)]
    gh64 = np.concatenate([q[0] for q in back], 1)
    gh64[:, :1], ggamma64, gbeta64 = dense.layer_norm_backward(wl.x[:, :1], _np(gamma), mu, rs, gh64[:, :1])
    pairs = {"y": (y, y64), "grad_U": (gU, gU64), "grad_bias": (gbias, gbias64), "grad_w": (gw, ref["grad_w"]),
             "grad_r": (gr, ref["grad_r"]), "grad_x": (gh, gh64), "grad_gamma": (ggamma, ggamma64),
             "grad_beta": (gbeta, gbeta64), **{f"grad_W{l}": (gWs[l], back[l][1]) for l in range(3)}}
    errs = {k: rel_err(v, w) for k, (v, w) in pairs.items()}
    assert gx0.data_ptr() == gh.data_ptr()
    assert errs.pop("y") <= 1e-5 and max(errs.values()) <= 1e-4, errs  # the tensor product's own tolerances
