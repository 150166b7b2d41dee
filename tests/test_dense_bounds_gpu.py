"""Sharper bounds of the dense row operators on the GPU: single products, non-finite rows.

The tolerances count:
  - the backward's dz of bfloat16 operands is two bfloat16 parts: within 2^-16 of it;
  - storing rounds by half a step (torch.finfo(t).eps / 2).
"""
import numpy as np
import pytest
import torch

import cg_tensor_products_b200 as etp
import test_dense_gpu as base
from oracle import dense

pytestmark = pytest.mark.gpu

_np, _rand = base._np, base._rand


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


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
