"""Dense row operators in float64: linear layers with an epilogue, layer norm, and their VJPs.

Rows are the leading axes of every argument, channels the last one; the formulas are written out as the
library's header states them.
"""
import numpy as np


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def act(z, name):
    return z * sigmoid(z) if name == "silu" else z


def act_grad(z, name):
    if name != "silu":
        return np.ones_like(z)
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def linear_forward(x, W, bias=None, activation="none", residual=None):
    """(out, z): z = x W + bias, out = act(z) + residual."""
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    z = x @ W
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    out = act(z, activation)
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
    return out, z


def linear_backward(x, W, grad_out, z=None, activation="none"):
    """(grad_x, grad_W, grad_bias) for the cotangent grad_out at the pre-activation z."""
    x, W, g = (np.asarray(a, np.float64) for a in (x, W, grad_out))
    dz = g if activation == "none" else g * act_grad(np.asarray(z, np.float64), activation)
    rows = dz.reshape(-1, dz.shape[-1])
    return dz @ W.T, x.reshape(-1, x.shape[-1]).T @ rows, rows.sum(0)


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5):
    """(out, mean, rstd) over the last axis."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    out = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        out = out * np.asarray(weight, np.float64)
    if bias is not None:
        out = out + np.asarray(bias, np.float64)
    return out, mean, rstd


def layer_norm_backward(x, weight, mean, rstd, grad_out):
    """(grad_x, grad_weight, grad_bias) for the cotangent grad_out."""
    x, g = np.asarray(x, np.float64), np.asarray(grad_out, np.float64)
    rstd = np.asarray(rstd, np.float64)[..., None]
    xh = (x - np.asarray(mean, np.float64)[..., None]) * rstd
    gw = g if weight is None else g * np.asarray(weight, np.float64)
    gx = rstd * (gw - gw.mean(-1, keepdims=True) - xh * (gw * xh).mean(-1, keepdims=True))
    C = x.shape[-1]
    return gx, (g * xh).reshape(-1, C).sum(0), g.reshape(-1, C).sum(0)
