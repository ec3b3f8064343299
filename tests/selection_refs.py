"""64-bit references of the operators whose rows choose their own weights
(routing, the few-token mixture-of-experts layer, low-rank adapters), in
plain numpy from their definitions in include/w4a8.h, with the error bounds
the tests use.

u = 2^-24 is half a unit in the last place of float32; the bounds count the
roundings of a float32 evaluation, and for outputs of fewer bits half a unit
of that type.
"""
import numpy as np

import oracle

U = 2.0 ** -24
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# half the spacing of the smallest (subnormal) values
HALF_MIN = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def decode_weights(wq, s_panels, a_panels, N, K, g):
    """int8 weights [N][K] that packed LiquidQuant arrays stand for."""
    codes = oracle.unpack_nibbles(wq, N, K)
    s = oracle.params_from_panels(s_panels, N, K // g)
    a = oracle.params_from_panels(a_panels, N, K // g)
    return oracle.lqq_decode(codes, s, a, g)


def rounding(y, dt):
    """Most that rounding y to type dt can move it."""
    return np.abs(y) * HALF_ULP[dt] + HALF_MIN[dt]


# ------------------------------------------------------------------ route ---

def route(x, k, renorm):
    """x: float64 [T][E].  (ids, weights, tolerance, offsets, rows)."""
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    tol = np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-x[t, e], e))
        order = [e for e in order if x[t, e] > -np.inf]
        if not order:
            continue
        top = x[t, order[0]]
        e_of = {e: 1.0 if x[t, e] == top else np.exp(x[t, e] - top) for e in order}
        chosen = order[:k]
        total = sum(e_of[e] for e in (chosen if renorm else order))
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w[t, j] = e_of[e] / total
            # x - top rounds once (|x - top| u in the exponential), expf is
            # within 2 units of the last place (4 u), the sum of at most E
            # terms adds E u (and its terms' own 4 u + |x - top| u, largest
            # where the term is smallest: |d| exp(d) <= 0.37, so at most
            # 0.37 E u in all), the quotient u
            d = 0.0 if x[t, e] == top else abs(x[t, e] - top)
            if d == np.inf:  # below an infinite logit: exactly 0
                continue
            tol[t, j] = w[t, j] * (d + 4 + 4 + 1.37 * E + 2) * U + 2.0 ** -149
    flat = ids.reshape(-1)
    rows = np.full(T * k, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    p = 0
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        rows[p:p + len(slots)] = slots
        p += len(slots)
        offsets[e + 1] = p
    return ids, w, tol, offsets, rows


# -------------------------------------------------------------------- moe ---

def _quant(x):
    """The definition's INT8 codes (float32 arithmetic) and float32 scale."""
    return oracle.quant_sym_rows(np.ascontiguousarray(x, np.float32), 127)


def moe(X, ids, weights, W13, sw13, W2, sw2, dt):
    """X float32 [T][H]; W13 [E][2F][H], W2 [E][H][F] int8 decoded weights;
    (Y float64 [T][H], tolerance).

    float32 evaluation moves h by a few u, so a code whose quotient h / sh
    lies that close to a half may fall on either side: such a code adds one
    step sh |w2| to the bound.  The other terms are the relative errors of
    the scales and products."""
    T, H = X.shape
    E, F2, _ = W13.shape
    F = F2 // 2
    Y = np.zeros((T, H))
    tol = np.zeros((T, H))
    fin = np.isfinite(X).all(1)
    Xq, sx = _quant(np.where(fin[:, None], X, 0.0))
    for t in range(T):
        for j in range(ids.shape[1]):
            e, w = ids[t, j], float(weights[t, j])
            if e < 0 or e >= E or w == 0.0:
                continue
            if not fin[t]:
                Y[t] = np.nan
                continue
            acc = W13[e].astype(np.int64) @ Xq[t].astype(np.int64)
            gu = acc * float(sx[t]) * sw13[e].astype(np.float64)
            g, u = gu[:F], gu[F:]
            with np.errstate(over="ignore"):
                h = u * g / (1.0 + np.exp(-g))
            # g, u: three roundings each; silu multiplies g's by at most
            # 1 + |g|; exp 4 u, sum, quotient and product u each
            rel = (3 * (1 + np.abs(g)) + 3 + 4 + 3) * U
            amax = np.abs(h).max()
            sh = np.float64(np.float32(amax / 127.0)) if amax > 0 else 1.0
            if sh == 0.0:
                sh = 1.0
            erel = rel.max() + 2 * U   # of the scale
            q = h / sh
            qi = np.clip(np.rint(q), -127, 127)
            near = np.abs(np.abs(q - np.floor(q)) - 0.5) <= np.abs(q) * (rel + erel + U) + 1e-30
            s2 = sw2[e].astype(np.float64)
            Wf = W2[e].astype(np.float64)
            y = (Wf @ qi) * sh * s2
            ty = (np.abs(Wf) @ near.astype(np.float64)) * sh * s2
            Y[t] += w * y
            tol[t] += abs(w) * (ty + np.abs(y) * (erel + 4 * U)) + np.abs(w * y) * 17 * U
    return Y, tol + rounding(Y, dt)


# ------------------------------------------------------------------- lora ---

def gemm_lora(X, W, sw, A, B, scale, adapter):
    """X float32 [M][K] (exact values of the stored type), W int8 [N][K];
    (Y float64 [M][N], tolerance for an fp16 output)."""
    M, K = X.shape
    n, R, _ = A.shape if A.size else (0, 8, K)
    Xq, sx = _quant(X)
    base = (oracle.gemm_i32(Xq, W).astype(np.float64) * sx[:, None].astype(np.float64)
            * sw.astype(np.float64))
    Y = base.copy()
    tol = 3 * U * np.abs(base)
    for a in range(n):
        m = np.nonzero(adapter == a)[0]
        if not len(m):
            continue
        V = X[m].astype(np.float64) @ A[a].T.astype(np.float64) * float(scale[a])
        D = V @ B[a].T.astype(np.float64)
        absV = np.abs(X[m]).astype(np.float64) @ np.abs(A[a]).T.astype(np.float64)
        absV *= abs(float(scale[a]))
        absB = np.abs(B[a]).T.astype(np.float64)
        Y[m] += D
        # a float32 sum of K products whose longest chain has at most K / 8
        # additions (plus the joining of 64 partial sums), the inner product
        # kept to 16 bits, the outer sum of R products onto the projection
        tol[m] += (K / 8 + 64) * U * (absV @ absB) + 2.0 ** -16 * (np.abs(V) @ absB)
        tol[m] += (2 * R + 4) * U * (np.abs(V) @ absB + np.abs(base[m]))
    return Y, tol + rounding(Y, "f16")
