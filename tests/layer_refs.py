"""References of the norm with quantisation and of the gated feed-forward
block, in plain numpy from their definitions in include/w4a8.h.

The norm is defined operation by operation (float32 each, float64 sums), so
``norm`` returns the very bits; ``norm64`` is the same formula in float64 with
a bound that counts the float32 roundings.  ``ffn`` is in float64 with a bound.
u = 2^-24 is half a unit in the last place of float32.
"""
import math

import numpy as np
import torch

import oracle
from selection_refs import U, rounding

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
f32 = np.float32


def _mean(v):
    """Row means of float32 values, summed exactly enough in float64."""
    return v.astype(np.float64).sum(1, keepdims=True) / v.shape[1]


def _norm(v, w, c, layer, eps):
    if layer:
        v = v - _mean(v).astype(f32)
    r = (1.0 / np.sqrt((v.astype(np.float64) ** 2).sum(1, keepdims=True) / v.shape[1]
                       + np.float64(f32(eps)))).astype(f32)
    n = (v * r) * w
    return n if c is None else n + c


def _gate_rows(gate, ids, M):
    """Factor [M][K], 1 where no gate is selected."""
    if ids is None:
        return np.broadcast_to(gate, (M, gate.shape[1]))
    out = np.ones((M, gate.shape[1]), gate.dtype)
    for m, g in enumerate(ids):
        if 0 <= g < len(gate):
            out[m] = gate[g]
    return out


def codes(n, kind):
    """(int8 codes or e4m3 bytes, float32 scales) of float32 rows."""
    fin = np.isfinite(n).all(1)
    z = np.where(fin[:, None], n, f32(0))
    if kind == "int8":
        q, s = oracle.quant_sym_rows(np.ascontiguousarray(z), 127)
    else:
        q, s = oracle.quant_rows_e4m3(np.ascontiguousarray(z))
    s = np.where(fin, s, f32(np.nan)).astype(f32)
    q = np.where(fin[:, None], q, np.zeros((), q.dtype))
    return q, s


def norm(x, y=None, y_weight=None, y_bias=None, gate=None, ids=None, x_scale=1.0, y_scale=1.0,
         weight=None, bias=None, layer=False, eps=1e-5):
    """(x', n) in float32, bit for bit; inputs float32 arrays (exact values)."""
    with np.errstate(all="ignore"):
        v = x * f32(x_scale)
        if y is not None:
            b = y
            if y_weight is not None:
                b = _norm(b, y_weight, y_bias, layer, eps)
            if gate is not None:
                b = b * _gate_rows(gate, ids, len(x))
            v = v + b * f32(y_scale)
        n = v if weight is None else _norm(v, weight, bias, layer, eps)
    return v, n


def _norm64(v, tv, w, c, layer, eps):
    """float64 norm of v, whose float32 form is within tv of it, and its bound."""
    K = v.shape[1]
    if layer:
        mu = v.mean(1, keepdims=True)
        tmu = tv.mean(1, keepdims=True) + U * np.abs(mu)
        v, tv = v - mu, tv + tmu + U * np.abs(v - mu)
    ms = (v * v).mean(1, keepdims=True) + float(f32(eps))
    r = 1.0 / np.sqrt(ms)
    # d(r) = r^3 mean(|v| dv); then the rounding of r (and a term in dv^2 that
    # stays far below them)
    tr = r ** 3 * (np.abs(v) * tv + tv * tv).mean(1, keepdims=True) + U * r
    n = v * r * w
    tn = np.abs(w) * (tv * r + np.abs(v) * tr + tv * tr) + 2.01 * U * np.abs(n)
    if c is not None:
        n = n + c
        tn = tn + U * (np.abs(n) + tn)
    return n, tn


def norm64(x, y=None, y_weight=None, y_bias=None, gate=None, ids=None, x_scale=1.0, y_scale=1.0,
           weight=None, bias=None, layer=False, eps=1e-5):
    """(x', bound, n, bound) in float64."""
    d = np.float64
    v = x.astype(d) * float(f32(x_scale))
    t = U * np.abs(v)
    if y is not None:
        b, tb = y.astype(d), np.zeros(y.shape)
        if y_weight is not None:
            b, tb = _norm64(b, tb, y_weight.astype(d),
                            None if y_bias is None else y_bias.astype(d), layer, eps)
        if gate is not None:
            f = _gate_rows(gate, ids, len(x)).astype(d)
            b, tb = b * f, tb * np.abs(f) + U * (np.abs(b * f) + tb * np.abs(f))
        s = float(f32(y_scale))
        b, tb = b * s, tb * abs(s)
        tb = tb + U * (np.abs(b) + tb)
        v, t = v + b, t + tb
        t = t + U * (np.abs(v) + t)
    if weight is None:
        return v, t, v, t
    n, tn = _norm64(v, t, weight.astype(d), None if bias is None else bias.astype(d), layer, eps)
    return v, t, n, tn


# -------------------------------------------------------------------- ffn ---

GELU_C = 2.0 * math.sqrt(2.0 / math.pi)


def ffn(Xq, sx, W13, sw13, W2, sw2, act, dt):
    """Xq int8 [M][H], sx float32 [M]; W13 [2F][H], W2 [H][F] int8 decoded
    weights; (Y float64 [M][H], tolerance).

    float32 evaluation moves h by a few u, so a code whose quotient h / sh lies
    that close to a half may fall on either side: such a code adds one step
    sh |w2| to the bound.  The other terms are the relative errors of the scales
    and products."""
    F = W2.shape[1]
    acc = oracle.gemm_i32(Xq, W13).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        gu = acc * sx[:, None].astype(np.float64) * sw13.astype(np.float64)
        g, u = gu[:, :F], gu[:, F:]
        # exp(-z) as a power of two: z's own error, and the rounded product
        # z log2(e), which moves the power by |z| u
        if act == "gelu":
            z = GELU_C * g * (1.0 + 0.044715 * g * g)
            # z: g's three roundings counted up to three times (its cube), six
            # of its own operations and the two constants'
            dz = np.abs(z) * (9 + 8 + 1) * U
        else:
            z, dz = g, np.abs(g) * (3 + 1) * U
        h = g / (1.0 + np.exp(-z)) * u
        # g and u three roundings each; the power one unit in the last place
        # (2 u) and dz, of which 1 / (1 + power) feels at most all; the sum u,
        # the reciprocal one unit (2 u), the two products u each
        rel = 6 * U + dz + 7 * U
    fin = np.isfinite(sx) & (np.abs(h) < 3.4e38).all(1)
    h = np.where(fin[:, None], h, 0.0)
    rel = np.where(fin[:, None], rel, 0.0)
    # the exponential's subnormal range: h's last bits there are absolute
    ah = np.abs(h) * rel + 2.0 ** -120 * (1.0 + np.abs(np.where(fin[:, None], u, 0.0)))
    amax = np.abs(h).max(1, keepdims=True)
    at = np.argmax(np.abs(h), 1)
    erel = np.where(amax > 0, ah[np.arange(len(h)), at][:, None] / np.maximum(amax, 1e-300), 0.0)
    # another element may be the float32 maximum: it is then within both bounds
    erel = erel + np.where(amax > 0, (np.abs(h) + ah).max(1, keepdims=True)
                           / np.maximum(amax, 1e-300) - 1.0, 0.0) + 2 * U
    sh = np.where(amax > 0, (amax / 127.0).astype(f32).astype(np.float64), 1.0)
    sh = np.where(sh > 0, sh, 1.0)
    q = h / sh
    qi = np.clip(np.rint(q), -127, 127)
    near = np.abs(np.abs(q - np.floor(q)) - 0.5) <= ah / sh + np.abs(q) * (erel + 2 * U) + 1e-30
    W = W2.astype(np.float64)
    s2 = sw2.astype(np.float64)
    y = (qi @ W.T) * sh * s2
    ty = (near.astype(np.float64) @ np.abs(W).T) * sh * s2 * (1 + 1e-6) + np.abs(y) * (erel + 4 * U)
    # what is rounded at the end lies anywhere within ty of y, so its rounding is
    # that of |y| + ty at most: where a code fell on the other side of a half,
    # y = -0.00106 became -0.00256 (ty = 0.00150), whose rounding to bfloat16 is
    # up to 2^-8 x 0.00256 = 1.0e-5, not 2^-8 x 0.00106 = 4.1e-6
    tol = ty + rounding(np.where(fin[:, None], np.abs(y) + ty, 0.0), dt)
    return np.where(fin[:, None], y, np.nan), tol
