"""Argument checks of w4a8_route, w4a8_moe and w4a8_gemm_lora (no GPU: every
case below is refused, or has nothing to do, before any HIP call) and of
their Python wrappers."""
import pytest

w4 = pytest.importorskip("w4a8_quantized_gemm_amd")
torch = pytest.importorskip("torch")
lib = w4.lib

OK, NULL, SHAPE, ALIGN, WS, UNSUP, HIP = range(7)
A = 0x10000  # a 16-byte-aligned fake device address, never dereferenced
BIG = 1 << 40


def route(x=A, it=0, T=4, E=8, k=2, rn=1, ids=A, w=A, off=A, rows=A, ws=A, wsb=BIG):
    return lib.w4a8_route(x, it, T, E, k, rn, ids, w, off, rows, ws, wsb, None)


def test_route_refusals():
    assert route(it=3) == UNSUP and route(it=-1) == UNSUP
    assert route(rn=2) == UNSUP
    for bad in (dict(T=-1), dict(E=0), dict(E=513), dict(k=0), dict(k=9), dict(E=64, k=17),
                dict(T=1 << 28, E=8)):
        assert route(**bad) == SHAPE, bad
    for p in ("x", "ids", "w", "off", "rows"):
        assert route(**{p: None}) == NULL, p
    assert route(T=0, off=None) == NULL
    assert route(x=A + 2) == ALIGN and route(x=A + 1, it=1) == ALIGN
    assert route(x=A + 1, it=2) == ALIGN
    for p in ("ids", "w", "off", "rows"):
        assert route(**{p: A + 2}) == ALIGN, p
    need = lib.w4a8_route_workspace_size(1000, 64, 6)
    assert need > 0
    assert route(T=1000, E=64, k=6, wsb=need - 1) == WS
    assert route(T=1000, E=64, k=6, ws=None) == NULL
    assert route(T=1000, E=64, k=6, ws=A + 4) == ALIGN


def test_route_workspace_size():
    size = lib.w4a8_route_workspace_size
    assert size(0, 8, 2) == 0 and size(1, 8, 2) == 0 and size(16, 512, 16) == 0
    assert size(-1, 8, 2) == 0 and size(1000, 0, 1) == 0 and size(1000, 8, 9) == 0
    for T in (65, 1000, 16384, 16385, 100000, (1 << 31) // 64 - 1):
        assert 0 < size(T, 64, 6) <= 512 * 64 * 4


def moe(X=A, it=1, ids=A, w=A, T=4, E=8, k=2, wq13=A, s13=A, a13=A, sw13=A, wq2=A, s2=A, a2=A,
        sw2=A, Y=A, ot=1, H=256, F=384, g=128, ws=A, wsb=BIG):
    return lib.w4a8_moe(X, it, ids, w, T, E, k, wq13, s13, a13, sw13, wq2, s2, a2, sw2, Y, ot, H,
                        F, g, ws, wsb, None)


def test_moe_refusals():
    assert moe(it=3) == UNSUP and moe(ot=-1) == UNSUP
    for bad in (dict(T=-1), dict(T=257), dict(E=0), dict(E=513), dict(k=0), dict(k=17),
                dict(H=192), dict(H=0), dict(F=64), dict(F=0), dict(F=-128), dict(g=32),
                dict(H=1 << 19), dict(F=1 << 19), dict(H=65536, F=65536 // 2)):
        assert moe(**bad) == SHAPE, bad
    assert moe(T=0, X=None, Y=None, ws=None, wsb=0) == OK  # empty: nothing is read
    assert moe(T=0, H=100) == SHAPE
    for p in ("X", "ids", "w", "wq13", "s13", "a13", "sw13", "wq2", "s2", "a2", "sw2", "Y"):
        assert moe(**{p: None}) == NULL, p
    for p in ("X", "Y", "wq13", "s13", "a13", "wq2", "s2", "a2"):
        assert moe(**{p: A + 8}) == ALIGN, p
    for p in ("ids", "w", "sw13", "sw2"):
        assert moe(**{p: A + 2}) == ALIGN, p
    need = lib.w4a8_moe_workspace_size(4, 8, 2, 256, 384)
    assert need > 0
    assert moe(wsb=need - 1) == WS
    assert moe(ws=None) == NULL
    assert moe(ws=A + 8) == ALIGN
    assert lib.w4a8_moe_workspace_size(0, 8, 2, 256, 384) == 0
    assert lib.w4a8_moe_workspace_size(257, 8, 2, 256, 384) == 0


def lora(X=A, it=1, wq=A, s=A, a=A, sw=A, la=A, lb=A, sc=A, n=4, R=16, ad=A, Y=A, M=16, N=64,
         K=256, g=64, ws=A, wsb=BIG):
    return lib.w4a8_gemm_lora(X, it, wq, s, a, sw, la, lb, sc, n, R, ad, Y, M, N, K, g, ws, wsb,
                              None)


def test_lora_refusals():
    assert lora(it=0) == UNSUP and lora(it=3) == UNSUP
    for bad in (dict(M=-1), dict(N=40), dict(K=200), dict(K=0), dict(g=32), dict(R=0),
                dict(R=12), dict(R=136), dict(n=-1), dict(M=1 << 24)):
        assert lora(**bad) == SHAPE, bad
    assert lora(M=0, X=None, Y=None, ws=None, wsb=0) == OK
    assert lora(N=0, X=None, Y=None, ws=None, wsb=0) == OK
    for p in ("X", "wq", "s", "a", "sw", "ad", "Y", "la", "lb", "sc"):
        assert lora(**{p: None}) == NULL, p
    for p in ("X", "wq", "s", "a", "Y", "la", "lb"):
        assert lora(**{p: A + 8}) == ALIGN, p
    for p in ("sw", "sc", "ad"):
        assert lora(**{p: A + 2}) == ALIGN, p
    need = lib.w4a8_gemm_lora_workspace_size(16, 64, 256, 16)
    assert need > 0
    assert lora(wsb=need - 1) == WS
    assert lora(ws=None) == NULL
    assert lora(ws=A + 8) == ALIGN
    assert lib.w4a8_gemm_lora_workspace_size(0, 64, 256, 16) == 0
    assert lib.w4a8_gemm_lora_workspace_size(16, 64, 256, 12) == 0


def test_wrappers_refuse_before_the_library():
    """Types, shapes and places are named by the wrappers (CPU tensors here,
    so nothing could run)."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        w4.route(x, 2)
    with pytest.raises(TypeError):
        w4.route(x.double(), 2)
    with pytest.raises(TypeError):
        w4.route([[0.0]], 1)
    X = torch.zeros(4, 256, dtype=torch.float16)
    w13 = {"N": 512, "K": 256, "group": 64, "E": 2}
    w2 = {"N": 256, "K": 256, "group": 64, "E": 2}
    with pytest.raises(ValueError, match="GPU"):
        w4.moe(X, None, None, w13, w2)
    with pytest.raises(TypeError):
        w4.moe(X.to(torch.int8), None, None, w13, w2)
    with pytest.raises(TypeError):
        w4.gemm_lora(X.float(), {"N": 64, "K": 256, "group": 64}, {}, None)
    with pytest.raises(ValueError, match="GPU"):
        w4.gemm_lora(X, {"N": 64, "K": 256, "group": 64}, {}, None)
