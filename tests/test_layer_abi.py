"""Argument checks of w4a8_norm_quant and w4a8_ffn (no GPU: every case below is
refused, or has nothing to do, before any HIP call), of their Python wrappers,
and the references' own agreement."""
import numpy as np
import pytest

import layer_refs as ref

w4 = pytest.importorskip("w4a8_quantized_gemm_amd")
torch = pytest.importorskip("torch")
lib = w4.lib

OK, NULL, SHAPE, ALIGN, WS, UNSUP, HIP = range(7)
A = 0x10000  # a 16-byte-aligned fake device address, never dereferenced
BIG = 1 << 40


def norm(X=A, xt=2, Y=A, yt=1, yw=A, yb=A, gate=A, rows=4, ids=A, xs=1.0, ys=1.0, w=A, b=A,
         kind=0, eps=1e-5, Xout=A, out=A, ot=3, sx=A, M=4, K=256):
    return lib.w4a8_norm_quant(X, xt, Y, yt, yw, yb, gate, rows, ids, xs, ys, w, b, kind, eps, Xout,
                               out, ot, sx, M, K, None)


def test_norm_refusals():
    inf, nan = float("inf"), float("nan")
    for bad in (dict(xt=3), dict(xt=-1), dict(yt=3), dict(kind=2), dict(kind=-1), dict(ot=5),
                dict(ot=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
                dict(xs=inf), dict(xs=nan), dict(ys=nan), dict(ys=-inf)):
        assert norm(**bad) == UNSUP, bad
    for bad in (dict(M=-1), dict(M=1 << 22), dict(K=0), dict(K=-16), dict(K=24), dict(rows=0),
                dict(rows=-1),
                dict(rows=3, ids=None), dict(rows=5, ids=None)):
        assert norm(**bad) == SHAPE, bad
    assert norm(M=0, X=None, Y=None, yw=None, yb=None, gate=None, ids=None, Xout=None, out=None,
                sx=None) == OK  # empty: nothing is read
    assert norm(M=0, rows=1, ids=None) == OK
    for p in ("X", "out", "Xout", "sx"):
        assert norm(**{p: None}) == NULL, p
    assert norm(Y=None) == NULL  # a norm and a gate of nothing
    assert norm(Y=None, yw=None, yb=None) == NULL
    assert norm(Y=None, gate=None, ids=None) == NULL
    assert norm(yw=None) == NULL and norm(w=None) == NULL  # a bias without its weight
    assert norm(gate=None) == NULL                         # ids without a gate
    for p in ("X", "Y", "gate", "Xout", "out"):
        assert norm(**{p: A + 8}) == ALIGN, p
    for p in ("yw", "yb", "ids", "w", "b", "sx"):
        assert norm(**{p: A + 2}) == ALIGN, p


def ffn(Xq=A, sx=A, wq13=A, s13=A, a13=A, sw13=A, wq2=A, s2=A, a2=A, sw2=A, act=0, Y=A, ot=1, M=4,
        H=256, F=384, g=128, ws=A, wsb=BIG):
    return lib.w4a8_ffn(Xq, sx, wq13, s13, a13, sw13, wq2, s2, a2, sw2, act, Y, ot, M, H, F, g, ws,
                        wsb, None)


def test_ffn_refusals():
    for bad in (dict(ot=0), dict(ot=3), dict(ot=-1), dict(act=2), dict(act=-1)):
        assert ffn(**bad) == UNSUP, bad
    for bad in (dict(M=-1), dict(H=192), dict(H=0), dict(H=-128), dict(F=64), dict(F=0),
                dict(F=-128), dict(g=32), dict(H=1 << 18), dict(F=1 << 18),
                dict(H=65536, F=65536 // 2), dict(M=1 << 23), dict(M=(1 << 31) // 384 + 1)):
        assert ffn(**bad) == SHAPE, bad
    assert ffn(M=0, Xq=None, Y=None, ws=None, wsb=0) == OK  # empty: nothing is read
    assert ffn(M=0, H=100) == SHAPE
    for p in ("Xq", "sx", "wq13", "s13", "a13", "sw13", "wq2", "s2", "a2", "sw2", "Y"):
        assert ffn(**{p: None}) == NULL, p
    for p in ("Xq", "Y", "wq13", "s13", "a13", "wq2", "s2", "a2"):
        assert ffn(**{p: A + 8}) == ALIGN, p
    for p in ("sx", "sw13", "sw2"):
        assert ffn(**{p: A + 2}) == ALIGN, p
    need = lib.w4a8_ffn_workspace_size(4, 256, 384)
    assert need > 0
    assert ffn(wsb=need - 1) == WS
    assert ffn(ws=None) == NULL
    assert ffn(ws=A + 8) == ALIGN


def test_ffn_workspace_size():
    size = lib.w4a8_ffn_workspace_size
    assert size(0, 256, 384) == 0 and size(-1, 256, 384) == 0
    assert size(4, 200, 384) == 0 and size(4, 256, 64) == 0
    assert size(1 << 23, 256, 384) == 0
    for M, H, F in ((1, 128, 128), (16, 8192, 28672), (4096, 8192, 28672), (65, 4096, 11008)):
        # at least the INT8 rows and their scales
        assert size(M, H, F) >= M * F + 4 * M


def test_wrappers_refuse_before_the_library():
    """Types, shapes and places are named by the wrappers (CPU tensors here, so
    nothing could run)."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        w4.norm_quant(x)
    with pytest.raises(TypeError):
        w4.norm_quant(x.to(torch.int8))
    with pytest.raises(TypeError):
        w4.norm_quant([[0.0]])
    with pytest.raises(ValueError, match="GPU"):
        w4.ffn(x.to(torch.int8), None, {}, {})
    with pytest.raises(TypeError):
        w4.ffn([[0]], None, {}, {})


@pytest.mark.parametrize("layer", [False, True])
def test_definition_lies_within_the_64_bit_bound(layer):
    """The operation-by-operation definition against the formula in float64."""
    rng = np.random.default_rng(5)
    for M, K in ((1, 16), (3, 64), (5, 1040), (2, 8192)):
        a = dict(y=rng.standard_normal((M, K)).astype(np.float32),
                 y_weight=rng.standard_normal(K).astype(np.float32),
                 y_bias=rng.standard_normal(K).astype(np.float32),
                 gate=rng.standard_normal((2, K)).astype(np.float32),
                 ids=rng.integers(-1, 3, M), x_scale=0.7, y_scale=1.3,
                 weight=rng.standard_normal(K).astype(np.float32),
                 bias=rng.standard_normal(K).astype(np.float32), layer=layer, eps=1e-6)
        x = (10 * rng.standard_normal((M, K)) + 3).astype(np.float32)
        v, n = ref.norm(x, **a)
        v64, tv, n64, tn = ref.norm64(x, **a)
        assert (np.abs(v - v64) <= tv).all()
        assert (np.abs(n - n64) <= tn).all()
        assert tn.max() < 1e-3
