"""Float64 definitions of the atom-wise dense operators and their gradients.

    norm    s = x + residual,  rstd = (mean_j s_j^2 + eps)^(-1/2),  y = s rstd w
    linear  z = x w^T + bias,  y = act(z) + residual

and, with gy the gradient of y,

    norm    a = gy w,  xhat = s rstd,  gx = rstd (a - xhat mean_j(a xhat)) + gsum,
            gw = sum_rows gy xhat
    linear  gz = gy act'(z),  gx = gz w,  gw = gz^T x,  gbias = sum_rows gz
"""
import numpy as np
from scipy.special import erf

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def norm(x, weight=None, residual=None, eps=1e-6):
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    y = s * rstd[:, None]
    return dict(sum=s, rstd=rstd, y=y if weight is None else y * weight)


def norm_backward(gy, s, weight, rstd, gsum=None):
    a = gy if weight is None else gy * weight
    xhat = s * rstd[:, None]
    gx = rstd[:, None] * (a - xhat * (a * xhat).mean(axis=1, keepdims=True))
    return dict(gx=gx if gsum is None else gx + gsum, gweight=(gy * xhat).sum(axis=0))


def e4m3_scale(y):
    return np.maximum(np.abs(y).max(axis=1), AMAX_FLOOR) / E4M3_MAX


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + erf(z / np.sqrt(2.0)))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = sigmoid(z)
        return p + z * p * (1.0 - p)
    if name == "gelu":
        return 0.5 * (1.0 + erf(z / np.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    return np.ones_like(z)


def linear(x, w, bias=None, act_name="none", residual=None):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, act_name)
    return dict(preact=z, y=y if residual is None else y + residual)


def linear_backward(gy, x, w, z, act_name="none"):
    gz = gy if act_name == "none" else gy * act_slope(z, act_name)
    return dict(gz=gz, gx=gz @ w, gw=gz.T @ x, gbias=gz.sum(axis=0))
