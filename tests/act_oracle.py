"""Epilogues in binary64, and how far fp32 may be from them.

u = 2^-24.  Errors of the activations as they are evaluated, relative to the
result unless said:
  * e^x: the argument's product with log2 e is carried exactly, 2^h within an
    ulp, one fused multiply-add: 4 u; z / (1 + z): 4 u more; times x: 9 u in
    all, 16 are allowed for silu.
  * gelu: erfc by a polynomial of degree 8 in t = 1 / (1 + a |x|), the
    coefficients' magnitudes adding up to 1.9 of its value at worst (t = 1):
    18 u 1.9 by Horner, 3 u of t through a slope of at most 9: 62 u, with e^x
    and the products 72: 80.
  * gelu_tanh: its argument t within 6 u: 6 |t| u of the logistic, and silu's.
  * e^x below 2^-126 may be 0: results below 2^-118 may be, and a slope may lack
    2^-126 of what its logistic or density is multiplied by.
Values that are rounded to bf16 next are formed in fewer operations (`brief`):
  * e^x = 2^(x c), c = fp32(log2 e) (off by 0.25 u): the product's rounding and
    c's move the argument by 1.25 u |x| log2 e, the result by 1.25 |x| u; 2 |x| u
    are allowed.  Where it passes 2^126, so that its reciprocal may be 0, the
    value is below 89 2^-126 < 2^-118.
  * gelu: a polynomial fitted within 1.22e-5, its terms adding up to 1.6 of its
    value: the 80 u above hold for its evaluation; x^2 and its two products with
    constants' roundings: 4 u of x^2 / 2 at most.  1.3e-5 + 80 u + 2 x^2 u.
  * gelu_tanh: its argument within 6 u + 2 u, times |t|: 8 |t| u, as above.
Slopes alike, of the magnitudes of their two terms.  No activation is steeper
than 1.13.
"""
import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -118
GONE = 2.0 ** -126
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
C = 2 * math.sqrt(2 / math.pi)


def _phi(x):
    return torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)


def act(x, name):
    if name == "relu":
        return torch.where(x < 0, 0.0, x)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * 0.5 * torch.erfc(-x / math.sqrt(2))
    if name == "gelu_tanh":
        return x * torch.sigmoid(C * (x + 0.044715 * x ** 3))
    return x


def evaluation(x, name, brief=False):
    """Relative error of an activation."""
    if name == "silu":
        return 16 * U + (2 * U * x.abs() if brief else torch.zeros_like(x))
    if name == "gelu":
        return 80 * U + (1.3e-5 + 2 * U * x * x if brief else torch.zeros_like(x))
    if name == "gelu_tanh":
        return (24 + 8 * (C * (x + 0.044715 * x ** 3)).abs()) * U
    return torch.zeros_like(x)


def slope(x, name):
    """(the slope, its error)"""
    if name == "relu":
        return (x > 0).to(x.dtype), torch.zeros_like(x)
    if name == "silu":
        p, q = torch.sigmoid(x), torch.sigmoid(-x)
        return p * (1 + x * q), 16 * U * p * (1 + x.abs() * q) + GONE * (1 + x.abs())
    if name == "gelu":
        p = 0.5 * torch.erfc(-x / math.sqrt(2))
        return p + x * _phi(x), 96 * U * (p + x.abs() * _phi(x)) + GONE * (1 + x.abs())
    if name == "gelu_tanh":
        t = C * (x + 0.044715 * x ** 3)
        p, q, d = torch.sigmoid(t), torch.sigmoid(-t), C * (1 + 3 * 0.044715 * x * x)
        return p * (1 + x * q * d), (40 + 16 * t.abs()) * U * p * (1 + x.abs() * q * d) + GONE * (1 + x.abs() * d)
    return torch.ones_like(x), torch.zeros_like(x)


def epilogue(x, ex, name, gated, residual=None, brief=False):
    """(y, its error before the output's rounding) for x within ex; brief: the
    output is bf16."""
    if gated:
        n = x.shape[1] // 2
        g, u, eg, eu = x[:, :n], x[:, n:], ex[:, :n], ex[:, n:]
        a = act(g, name)
        ea = 1.2 * eg + evaluation(g, name, brief) * a.abs() + TINY
        y, e = a * u, ea * (u.abs() + eu) + a.abs() * eu + U * (a * u).abs()
    else:
        y = act(x, name)
        e = 1.2 * ex + evaluation(x, name, brief) * y.abs() + TINY
    if residual is not None:
        y = y + residual
        e = e + U * (y.abs() + e)
    return y, e


def grad(dy, x, name, gated):
    """(dpre, its error before rounding)"""
    if gated:
        n = x.shape[1] // 2
        g, u = x[:, :n], x[:, n:]
        s, es = slope(g, name)
        a = act(g, name)
        d = torch.cat([dy * s * u, dy * a], 1)
        e = torch.cat([(dy * u).abs() * (es + 2 * U * s.abs()),
                       dy.abs() * (evaluation(g, name) * a.abs() + TINY + U * a.abs())], 1)
    else:
        s, es = slope(x, name)
        d, e = dy * s, dy.abs() * (es + U * s.abs())
    return d, e + TINY
