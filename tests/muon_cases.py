"""Definitions in 64 bits of the Muon step's operators and of the RMS norm, for the tests.

Tolerances count roundings. A rounding to nearest is off by at most half a step:
2^-8 of the value in bf16, 2^-11 in fp16, 2^-24 in fp32, 2^-4 in e4m3."""

import numpy as np
import torch

BF16, F16, F32, E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4
COEFFS = (3.4445, -4.7750, 2.0315)


def polar(g, steps=5, coeffs=COEFFS, eps=1e-7):
    """X_0 = g / (|g| + eps); X <- (a I + b S + c S S) X with S = X X^T, on the smaller side."""
    x = g.double().cpu()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.norm() + eps)
    a, b, c = coeffs
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def polar_tolerance(steps):
    """In the 2-norm: the output's bf16 rounding, and one fp16 rounding each of X_0 and of every
    step's S, P and X; these are independent and add as squares."""
    return BF16 + F16 * (3 * steps + 1) ** 0.5


def mean_rows(rows, scale):
    return sum(r.double() for r in rows) * scale


def norm_forward(x, w, eps):
    """y and rstd of rows x (64 bits)."""
    rstd = 1.0 / torch.sqrt(x.pow(2).mean(1, keepdim=True) + eps)
    return x * rstd * w, rstd


def norm_backward(dy, x, w, rstd):
    """dx, dweight of norm_forward, as formulas."""
    xhat = x * rstd
    g = dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0)


def bits(t):
    t = t.detach().cpu()
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t.contiguous().view(view).numpy()


def same_bits(a, b):
    return np.array_equal(bits(a), bits(b))
