"""A layer's product with its epilogue, and its gradients (TEST INFRASTRUCTURE
ONLY): pre = X W^T + bias, out = act(pre) + residual, in fp64.
"""
import numpy as np
from scipy.special import erf, expit


def act(x, name):
    """(value, derivative) of an activation."""
    x = np.asarray(x, np.float64)
    if name is None:
        return x, np.ones_like(x)
    if name == "relu":
        return np.where(x > 0, x, 0.0), (x > 0).astype(np.float64)
    if name == "silu":
        s = expit(x)
        return x * s, s + x * s * expit(-x)
    if name == "gelu":
        c = 0.5 * (1 + erf(x / np.sqrt(2)))
        return x * c, c + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
    assert name == "gelu_tanh"
    a, b = np.sqrt(2 / np.pi), 0.044715
    t = np.tanh(a * (x + b * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * a * (1 + 3 * b * x * x)


def forward(X, W, bias=None, name=None, residual=None):
    """(out, pre)."""
    pre = X @ W.T + (0 if bias is None else bias)
    return act(pre, name)[0] + (0 if residual is None else residual), pre


def backward_act(d_out, pre=None, name=None):
    """(dY, d_bias)."""
    dY = d_out * (1.0 if name is None else act(pre, name)[1])
    return dY, dY.sum(0)
