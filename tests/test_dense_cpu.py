"""Host-side checks of the dense row operators (no GPU): every declared symbol is exported, and the C ABI and
the binding refuse bad arguments before any launch. Every call that passes pointers is built to fail a check."""
import ctypes
import os
import subprocess

import pytest
import torch

import cg_tensor_products_b200 as etp
from cg_tensor_products_b200 import build as etp_build

OK, BAD, UNSUP, WS, LARGE = (etp.ETP_OK, etp.ETP_ERR_INVALID_ARG, etp.ETP_ERR_UNSUPPORTED, etp.ETP_ERR_WORKSPACE,
                             etp.ETP_ERR_TOO_LARGE)
PTR = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    etp_build.build()
    return etp._load()


def test_header_is_plain_c(tmp_path):
    """etp_dense.h compiles as C and its calls link and refuse bad arguments from a C program."""
    src = tmp_path / "dense.c"
    src.write_text("""
#include <etp_dense.h>
int main(void) {
    etp_rows x = {0, 128, 0};
    size_t n = 0;
    if (etp_linear_workspace_size(ETP_F32, 1000, 1, 64, 64, 1, &n) != ETP_OK || n == 0) return 1;
    if (etp_layer_norm_workspace_size(ETP_BF16, 1000, 3, 64, &n) != ETP_OK || n == 0) return 2;
    if (etp_linear_forward(ETP_F32, 4, 1, 64, 64, &x, 0, 0, ETP_ACT_SILU, 0, 0, &x, 0, 0, 0) != ETP_ERR_INVALID_ARG) return 3;
    if (etp_linear_backward(ETP_F32, 4, 1, 64, 64, &x, 0, ETP_ACT_NONE, 0, &x, 0, 0, 0, 0, 0, 0) != ETP_OK) return 4;
    if (etp_layer_norm_forward(ETP_F32, 4, 1, 64, 1e-5f, &x, 0, 0, &x, 0, 0, 0) != ETP_ERR_INVALID_ARG) return 5;
    if (etp_layer_norm_backward(ETP_F32, 4, 1, 64, &x, 0, 0, 0, &x, &x, 0, 0, 0, 0, 0) != ETP_ERR_INVALID_ARG) return 6;
    return 0;
}
""")
    etp_build.build()
    libdir, exe = os.path.dirname(etp.LIB_PATH), str(tmp_path / "dense")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.dirname(etp.DENSE_HEADER_PATH), str(src), "-L",
                    libdir, "-letp", f"-Wl,-rpath,{libdir}", "-o", exe], check=True, capture_output=True, text=True)
    assert subprocess.run([exe], timeout=60).returncode == 0


def rows(data=PTR, gs=64, rs=8):
    return ctypes.byref(etp._Rows(data, gs, rs))


def test_exports_every_declared_symbol(lib):
    names = etp.declared_symbols(etp.DENSE_HEADER_PATH)
    assert len(names) == 6
    for n in names:
        assert hasattr(lib, n), n


def test_linear_forward_refusals(lib):
    p = ctypes.c_void_p(PTR)

    def call(dtype=0, groups=4, per=2, K=8, N=8, x=rows(), W=p, bias=p, act=1, res=rows(), z=rows(), out=rows(), ws=p,
             n=1 << 40):
        return lib.etp_linear_forward(dtype, groups, per, K, N, x, W, bias, act, res, z, out, ws, n, None)

    assert call(groups=-1) == call(per=-1) == call(K=0) == call(N=0) == BAD
    assert call(K=etp.LINEAR_MAX_CHANNELS + 1) == call(N=etp.LINEAR_MAX_CHANNELS + 1) == BAD
    assert call(dtype=2) == call(dtype=-1) == call(act=2) == call(act=-1) == UNSUP
    assert call(groups=1 << 20, per=1 << 11) == LARGE
    assert call(x=None) == call(W=None) == call(out=None) == call(x=rows(0)) == BAD
    for name in ("x", "res", "z", "out"):  # misaligned for the type, negative or absurd strides
        assert call(**{name: rows(PTR + 2)}) == BAD
        assert call(**{name: rows(gs=-64)}) == call(**{name: rows(rs=-64)}) == BAD
        assert call(**{name: rows(gs=1 << 31)}) == BAD
    assert call(W=ctypes.c_void_p(PTR + 1)) == call(bias=ctypes.c_void_p(PTR + 2)) == BAD
    assert call(dtype=1, x=rows(PTR + 1)) == BAD
    for name in ("z", "out"):  # output rows that overlap
        assert call(**{name: rows(gs=64, rs=7)}) == BAD
        assert call(**{name: rows(gs=7, rs=64)}) == BAD
        assert call(**{name: rows(gs=12, rs=8)}) == BAD
        assert call(**{name: rows(gs=0, rs=8)}) == BAD
    big = dict(groups=1 << 20, per=1)  # sizes that need a workspace
    assert call(**big, ws=None) == call(**big, ws=ctypes.c_void_p(PTR + 8)) == BAD
    assert call(**big, n=0) == WS
    assert call(groups=0, x=None, out=None, W=None) == OK  # nothing to do
    assert call(per=0, x=None, out=None, W=None) == OK


def test_linear_backward_refusals(lib):
    p = ctypes.c_void_p(PTR)
    size = ctypes.c_size_t()
    f = lib.etp_linear_workspace_size
    assert f(0, 4, 2, 8, 8, 0, ctypes.byref(size)) == OK
    assert f(0, 4, 2, 8, 8, 1, ctypes.byref(size)) == OK and size.value > 0
    need = size.value
    assert f(0, 4, 2, 8, 8, 1, None) == f(0, -1, 2, 8, 8, 1, ctypes.byref(size)) == BAD
    assert f(0, 4, 2, 8, 8, 2, ctypes.byref(size)) == BAD
    assert f(0, 4, 2, 0, 8, 0, ctypes.byref(size)) == f(0, 4, 2, 8, 0, 1, ctypes.byref(size)) == BAD
    assert f(5, 4, 2, 8, 8, 0, ctypes.byref(size)) == UNSUP
    assert f(0, 1 << 20, 1 << 11, 8, 8, 0, ctypes.byref(size)) == LARGE

    for dtype in (0, 1):  # the most rows that a call takes: sizes that do not wrap around
        assert f(dtype, (1 << 31) - 129, 1, 4, 4, 1, ctypes.byref(size)) == OK and 0 < size.value < 1 << 30
        assert f(dtype, (1 << 31) - 128, 1, 4, 4, 1, ctypes.byref(size)) == LARGE

    def call(dtype=0, groups=4, per=2, K=8, N=8, x=rows(), W=p, act=1, z=rows(), g=rows(), gx=rows(), gW=p, gb=p,
             ws=p, n=1 << 40):
        return lib.etp_linear_backward(dtype, groups, per, K, N, x, W, act, z, g, gx, gW, gb, ws, n, None)

    assert call(groups=-1) == call(K=0) == call(N=-3) == call(g=None) == call(z=None) == BAD
    assert call(x=None) == call(W=None) == BAD  # needed for grad_W and for grad_x
    assert call(dtype=7) == call(act=9) == UNSUP
    assert call(gx=rows(rs=7)) == call(gx=rows(PTR + 2)) == BAD
    assert call(gW=ctypes.c_void_p(PTR + 2)) == call(gb=ctypes.c_void_p(PTR + 1)) == BAD
    assert call(ws=None) == call(ws=ctypes.c_void_p(PTR + 4)) == BAD
    assert call(n=0) == call(n=need - 1) == WS
    assert call(gx=None, gW=None, gb=None, x=None, W=None, z=None, g=None) == OK  # nothing wanted
    assert call(groups=1 << 20, per=1 << 11) == LARGE


def test_layer_norm_refusals(lib):
    p = ctypes.c_void_p(PTR)
    nan, inf = float("nan"), float("inf")

    def fwd(dtype=0, groups=4, per=2, C=8, eps=1e-5, x=rows(), w=p, b=p, out=rows(), mean=p, rstd=p):
        return lib.etp_layer_norm_forward(dtype, groups, per, C, eps, x, w, b, out, mean, rstd, None)

    assert fwd(groups=-1) == fwd(per=-2) == fwd(C=0) == fwd(eps=-1.0) == fwd(eps=nan) == fwd(eps=inf) == BAD
    assert fwd(dtype=3) == fwd(C=etp.NORM_MAX_CHANNELS + 1) == UNSUP
    assert fwd(x=None) == fwd(out=None) == fwd(out=rows(rs=4)) == fwd(x=rows(gs=-1)) == BAD
    assert fwd(w=ctypes.c_void_p(PTR + 2)) == fwd(mean=ctypes.c_void_p(PTR + 2)) == BAD
    assert fwd(groups=1 << 16, per=1 << 15) == LARGE
    assert fwd(groups=0, x=None, out=None) == OK
    size = ctypes.c_size_t()
    f = lib.etp_layer_norm_workspace_size
    assert f(0, 4, 2, 8, ctypes.byref(size)) == OK and size.value >= 64
    assert f(0, 4, 2, 8, None) == f(0, 4, 2, 0, ctypes.byref(size)) == BAD
    assert f(0, 4, 2, etp.NORM_MAX_CHANNELS + 1, ctypes.byref(size)) == UNSUP

    def bwd(dtype=0, groups=4, per=2, C=8, x=rows(), w=p, mean=p, rstd=p, g=rows(), gx=rows(), gw=p, gb=p, ws=p,
            n=1 << 40):
        return lib.etp_layer_norm_backward(dtype, groups, per, C, x, w, mean, rstd, g, gx, gw, gb, ws, n, None)

    assert bwd(groups=-1) == bwd(C=-1) == bwd(x=None) == bwd(g=None) == bwd(mean=None) == bwd(rstd=None) == BAD
    assert bwd(dtype=3) == bwd(C=etp.NORM_MAX_CHANNELS + 1) == UNSUP
    assert bwd(ws=None) == bwd(ws=ctypes.c_void_p(PTR + 4)) == BAD
    assert bwd(n=0) == bwd(n=size.value - 1) == WS
    assert bwd(gx=rows(rs=2)) == bwd(gw=ctypes.c_void_p(PTR + 3)) == BAD
    assert bwd(gx=None, gw=None, gb=None, x=None, g=None, mean=None, rstd=None) == OK


def test_binding_refusals(lib):
    x, W = torch.zeros(6, 4), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="no CPU path"):
        etp.linear_forward(x, W)
    with pytest.raises(ValueError, match="no CPU path"):
        etp.layer_norm_forward(x)
    for bad, text in [(lambda: etp.linear_forward(x.double(), W), "float32 or bfloat16"),
                      (lambda: etp.linear_forward(x, W.bfloat16()), "W: expected"),
                      (lambda: etp.linear_forward(x, torch.zeros(5, 8)), "x: expected 5 channels"),
                      (lambda: etp.linear_forward(x[0], W), r"x: expected \[rows, channels\]"),
                      (lambda: etp.linear_forward(x.t().contiguous().t(), W), "channels must be contiguous"),
                      (lambda: etp.linear_forward(x, W, activation="relu"), "activation"),
                      (lambda: etp.linear_forward(x, W, bias=torch.zeros(7)), "bias: expected"),
                      (lambda: etp.linear_forward(x, W, residual=torch.zeros(5, 8)), "residual: expected leading"),
                      (lambda: etp.linear_forward(x, W, residual=torch.zeros(6, 8).bfloat16()), "residual: expected"),
                      (lambda: etp.linear_forward(x, torch.zeros(8, 4).t()), "W: must be contiguous"),
                      (lambda: etp.linear_forward(torch.zeros(2, 0), torch.zeros(0, 8)), "1 <= K"),
                      (lambda: etp.linear_forward(x, torch.zeros(4, 4), out=x), "out must not overlap x"),
                      (lambda: etp.linear_backward(x, W, torch.zeros(6, 8), activation="silu"), "z: the forward"),
                      (lambda: etp.linear_backward(x, W, torch.zeros(6, 7)), "grad_out: expected 8 channels"),
                      (lambda: etp.linear_backward(x, W, torch.zeros(6, 8), grad_x=x), "grad_x must not overlap x"),
                      (lambda: etp.layer_norm_forward(x, weight=torch.zeros(5)), "weight: expected"),
                      (lambda: etp.layer_norm_backward(x, None, torch.zeros(5), torch.zeros(6), x), "mean: expected"),
                      (lambda: etp.layer_norm_forward(x, out=x.view(-1)[1:21].view(5, 4)), "out must not overlap x")]:
        with pytest.raises(ValueError, match=text):
            bad()


def test_blocks_of_one_feature_tensor_do_not_overlap():
    f = torch.zeros(5, 16, 8)
    assert not etp._overlap(f[:, :1], f[:, 1:4]) and not etp._overlap(f[:, 9:], f[:, 4:9])
    assert etp._overlap(f[:, :4], f[:, 3:6]) and etp._overlap(f[:, :1], f[:, :1])
    assert not etp._overlap(f[:2], f[2:]) and etp._overlap(f[:3], f[2:])
    assert not etp._overlap(f[:0], f) and not etp._overlap(f[:, 0, :4], f[:, 0, 4:])
    assert etp._overlap(f[:, 0, :5], f[:, 0, 4:])


def test_sizes_beyond_an_int_are_refused(lib):
    """Sizes that the C call's ints do not hold are refused, not taken modulo 2^32."""
    W, one, many = torch.zeros(4, 8), torch.zeros(1, 4), (1 << 32) + 3
    for call in (lambda: etp.linear_forward(one.expand(many, 4), W), lambda: etp.linear_forward(one.expand(2, many, 4), W),
                 lambda: etp.linear_backward(one.expand(many, 4), W, torch.zeros(1, 8).expand(many, 8), want=("bias",)),
                 lambda: etp.layer_norm_forward(one.expand(many, 4)),
                 lambda: etp.layer_norm_forward(torch.zeros(1, 1).expand(2, many)),
                 lambda: etp.layer_norm_backward(one.expand(many, 4), None, None, None, one.expand(many, 4)),
                 lambda: etp.linear_workspace_size(many, 4, 8, device="cuda:0"),
                 lambda: etp.linear_workspace_size(4, 4, many, device="cuda:0"),
                 lambda: etp.layer_norm_workspace_size(4, many, device="cuda:0")):
        with pytest.raises(etp.EtpError) as e:
            call()
        assert e.value.status == LARGE


def test_unknown_gradients_are_refused(lib):
    x, W, g, m = torch.zeros(6, 4), torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(6)
    for want in (("x", "w"), ("weight",), "bais", ("bias", None), "xW"):
        with pytest.raises(ValueError, match="want: expected some of"):
            etp.linear_backward(x, W, g, want=want)
    for want in (("x", "W"), "gamma", ("weights",)):
        with pytest.raises(ValueError, match="want: expected some of"):
            etp.layer_norm_backward(x, None, m, m, x, want=want)
    for want in (("x",), "bias", ["W", "bias"], ()):  # these get as far as the device check
        with pytest.raises(ValueError, match="no CPU path"):
            etp.linear_backward(x, W, g, want=want)


def test_overlap_is_told_from_interleaving():
    """Views of one buffer share an element exactly where the brute force finds one; other strides are only refused."""
    f = torch.zeros(5, 16, 8)
    assert not etp._overlap(f[:, 1:4, :4], f[:, 1:4, 4:]) and not etp._overlap(f[:, 1:4, 4:], f[:, 2:9, :4])
    assert etp._overlap(f[:, 1:4, :5], f[:, 3:9, 4:]) and not etp._overlap(f[1:2, 1:4], f[1:2, 4:9])
    gen = torch.Generator().manual_seed(0)
    r = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=gen))
    buf = torch.zeros(400)
    for _ in range(4000):
        rs = r(1, 9)
        gs = rs * r(1, 6) + (r(0, 3) if r(0, 2) else 0)
        views = [(r(0, 120), (r(1, 5), r(1, 5), r(1, 9))) for _ in range(2)]
        a, b = (buf[o:].as_strided(n, (gs, rs, 1)) for o, n in views)
        els = lambda o, n: {o + i * gs + j * rs + c for i in range(n[0]) for j in range(n[1]) for c in range(n[2])}
        sets = [els(o, n) for o, n in views]
        nested = all(n[2] <= rs and (n[1] - 1) * rs + n[2] <= gs for _, n in views)
        flat = els(views[0][0], (views[0][1][0], 1, views[0][1][2]))
        for got, meet in ((etp._overlap(a, b), bool(sets[0] & sets[1])), (etp._overlap(a[:, 0], b), bool(flat & sets[1])),
                          (etp._overlap(b.transpose(0, 1), a.transpose(0, 1)), bool(sets[0] & sets[1]))):
            assert got == meet if nested else got >= meet
