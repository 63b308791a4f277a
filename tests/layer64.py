"""The layer with its epilogues in 64 bits, with the error each part of the
kernels may add, for the tests of paro_linear_act and paro_linear_gated.

The sums are taken from X' as paro_rotate returns it (the kernels round X' to
fp16, and its own tests hold it to the oracle), so that what is left is:
  * the fp32 accumulation of in products on the tensor cores, 16 at a time:
    (in / 16 + 20) 2^-23 of A = sum |x'| |w_hat| + |b| covers a rounding toward
    zero of every partial sum and the joining of the partial results;
  * the activation: its slope is at most 1.13 (GELU; SiLU 1.1), and its own
    arithmetic (fast exponential and quotient) is good to 2^-18 relative;
  * one rounding to fp16: 2^-11 relative, 2^-25 absolute below the normal range.
"""
import math

import torch

SLOPE, ARITH = 1.13, 2.0 ** -18


def w_hat(q, s, z, group):
    """fp16((q - z) s) as float64 [out][in] (the product fits 16 bits: one rounding)."""
    n_out, n_in = q.shape
    d = q.double().view(n_out, n_in // group, group) - z.double()[:, :, None]
    return (d * s.double()[:, :, None]).half().double().view(n_out, n_in)


def sums(xr, w, bias=None):
    """(s, es): X' w_hat^T + b and the bound of the kernel's error of it."""
    x, n_in = xr.double(), xr.shape[1]
    s, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        s, mag = s + bias.double(), mag + bias.double().abs()
    return s, (n_in / 16 + 20) * 2.0 ** -23 * mag


def act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def rounding(y, e):
    """Bound of the fp16 result of a value y known to e."""
    return e + 2.0 ** -11 * (y.abs() + e) + 2.0 ** -25


def linear_act(xr, w, act, bias=None, residual=None):
    s, es = sums(xr, w, bias)
    y = act64(s, act)
    e = SLOPE * es + ARITH * y.abs() + 2.0 ** -24 * s.abs()
    if residual is not None:
        y = y + residual.double()
        e = e + 2.0 ** -24 * y.abs()
    return y, rounding(y, e)


def gated(xr, w, act, bias=None):
    s, es = sums(xr, w, bias)
    n = w.shape[0] // 2
    g, u, eg, eu = s[:, :n], s[:, n:], es[:, :n], es[:, n:]
    a = act64(g, act)
    ea = SLOPE * eg + ARITH * a.abs() + 2.0 ** -24 * g.abs()
    h = a * u
    return h, rounding(h, ea * u.abs() + a.abs() * eu + ea * eu + 2.0 ** -23 * h.abs())
