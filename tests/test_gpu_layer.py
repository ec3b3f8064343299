"""The norm with quantisation and the gated feed-forward block on the GPU
against their references (layer_refs.py states bits and bounds), together as a
layer runs them, and their behaviour in serving: captured graphs, other
streams, empty and odd calls, refusals."""
import numpy as np
import pytest

import layer_refs as ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_amd as w4  # noqa: E402
from test_gpu_selection import DEV, TYPES, experts, f64, host, poison, say, within  # noqa: E402

OUT = {"f32": w4.NORM_OUT_F32, "f16": w4.NORM_OUT_F16, "bf16": w4.NORM_OUT_BF16,
       "int8": w4.NORM_OUT_INT8, "e4m3": w4.NORM_OUT_E4M3}


def typed(a, dt):
    """numpy values -> (device tensor of the type, its values as float32)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TYPES[dt])
    return t.to(DEV), t.float().numpy()


def norm_case(M, K, xt, yt, post=False, gate="none", bias=False, seed=0):
    """(wrapper arguments on the device, reference arguments)."""
    rng = np.random.default_rng(1000 + seed + M + K)

    def rows(m, scale=1.0):
        return scale * rng.standard_normal((m, K)).astype(np.float32)
    x = rows(M)
    x[:, rng.random(K) < 0.02] *= 20
    if M > 3:
        x[M - 1] = 0.0
    dx, rx = typed(x, xt)
    d, r = dict(x=dx), dict(x=rx)
    if yt:
        y = rows(M, 0.3)
        if M > 3:
            y[M - 1] = 0.0
        d["y"], r["y"] = typed(y, yt)
        if gate != "none":
            n = {"all": 1, "row": M, "ids": 1 + M // 3}[gate]
            d["gate"], r["gate"] = typed(rows(n), yt)
            if gate == "ids":
                ids = rng.integers(-1, n + 1, M).astype(np.int32)
                ids[0] = -(1 << 31)
                d["gate_ids"], r["ids"] = torch.from_numpy(ids).to(DEV), ids
    for name in ("weight", "bias") + (("y_weight", "y_bias") if post else ()):
        if name.endswith("bias") and not bias:
            continue
        v = rng.standard_normal(K).astype(np.float32)
        d[name], r[name] = torch.from_numpy(v).to(DEV), v
    return d, r


def out_for(M, K, out, xt, has_y, x):
    q = {"int8": torch.int8, "e4m3": torch.uint8}.get(out)
    return {"out": poison((M, K), q or TYPES[out]), "sx": poison(M, torch.float32) if q else None,
            "x": poison((M, K), TYPES[xt]) if has_y else x}


def same_bits(t, want):
    """want: numpy, the very bits (any NaN equals any NaN)."""
    got = host(t.view(torch.int16) if t.dtype == torch.bfloat16 else t)
    if want.dtype.kind == "f":
        ok = (got == want) | (np.isnan(got) & np.isnan(want))
    else:
        ok = got == want
    assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])


def as_type(v, dt):
    """float32 values rounded to a type, as numpy of the same bits."""
    t = torch.from_numpy(np.ascontiguousarray(v)).to(TYPES[dt])
    return (t.view(torch.int16) if dt == "bf16" else t).numpy()


def nan_free_bf16(t, want, values):
    keep = ~np.isnan(values)
    got = host(t.view(torch.int16))
    assert (got[keep] == want[keep]).all()
    assert torch.isnan(t.cpu())[torch.from_numpy(~keep)].all()


def check_norm(d, r, out, layer, **kw):
    x, has_y = d["x"], "y" in d
    M, K = x.shape
    xt = {v: k for k, v in TYPES.items()}[x.dtype]
    dst = out_for(M, K, out, xt, has_y, x)
    res = w4.norm_quant(**d, kind=w4.NORM_LAYER if layer else w4.NORM_RMS, out_type=OUT[out],
                        out=dst, **kw)
    assert res is dst
    v, n = ref.norm(**r, layer=layer, **kw)

    def floats(t, values, dt):
        if dt == "bf16":
            nan_free_bf16(t, as_type(values, dt), values)
        else:
            same_bits(t, as_type(values, dt))
    if has_y:
        floats(res["x"], v, xt)
    if out in ("int8", "e4m3"):
        q, s = ref.codes(n, out)
        same_bits(res["sx"], s)
        same_bits(res["out"], q)
    else:
        floats(res["out"], n, out)
    return res, v, n


NORM = [  # M, K, x, y, post, gate, bias, layer, out
    (1, 16, "bf16", None, False, "none", False, False, "int8"),
    (1, 4096, "bf16", None, False, "none", False, False, "int8"),
    (1, 8192, "f16", "f16", True, "row", True, True, "int8"),
    (2, 32, "f32", "bf16", True, "all", True, True, "e4m3"),
    (3, 48, "f16", "f32", False, "ids", False, False, "f32"),
    (5, 1040, "f32", "f32", True, "ids", True, False, "int8"),
    (7, 2048, "bf16", "bf16", False, "all", False, True, "bf16"),
    (7, 2064, "bf16", "f16", True, "none", False, False, "e4m3"),
    (16, 8208, "f16", "bf16", True, "row", True, False, "int8"),
    (4, 16384, "f32", "f16", False, "none", True, True, "f16"),
    (3, 16400, "bf16", "f16", True, "row", True, True, "int8"),
    (2, 32768, "f32", "f32", True, "row", True, True, "e4m3"),
    # rows that the registers do not hold
    (2, 32784, "bf16", "f16", True, "ids", True, True, "int8"),
    (1, 131072, "f32", "f32", False, "all", False, False, "e4m3"),
    (3, 40000, "f16", None, False, "none", True, True, "bf16"),
    # many rows
    (511, 2080, "bf16", "f16", True, "ids", True, False, "int8"),
    (512, 2080, "bf16", "f16", True, "ids", True, False, "int8"),
    (600, 512, "f16", "f32", False, "row", False, True, "e4m3"),
    (700, 4096, "bf16", "f16", False, "none", False, False, "int8"),
    # both sides of every row width's limit
    (259, 16, "bf16", "f16", True, "row", True, True, "int8"),
    (257, 1024, "f16", "bf16", True, "ids", True, True, "int8"),
    (258, 1040, "bf16", "f16", True, "row", False, False, "e4m3"),
    (260, 2048, "f32", "f16", True, "none", True, True, "int8"),
    (261, 2064, "bf16", None, False, "none", False, False, "int8"),
    (300, 4112, "bf16", "f16", True, "row", True, True, "bf16"),
    (257, 6144, "f16", "f32", True, "all", True, False, "int8"),
    (257, 6160, "bf16", "f16", True, "row", False, True, "e4m3"),
    (256, 8192, "bf16", "f16", True, "row", True, True, "int8"),
    (257, 8208, "f32", "f32", True, "row", True, True, "int8"),
    (258, 12288, "bf16", "f16", True, "row", False, False, "int8"),
    (257, 12304, "f16", "f16", True, "ids", True, True, "f16"),
    (257, 32768, "f32", "f32", True, "row", True, True, "e4m3"),
    (257, 32784, "bf16", "f16", False, "none", False, False, "int8"),
    (513, 5136, "f32", "bf16", True, "all", True, True, "f16"),
    (520, 8192, "f16", "f16", True, "row", False, False, "int8"),
    (515, 16384, "bf16", "bf16", False, "ids", True, True, "bf16"),
    (514, 16400, "f32", "f32", True, "none", True, False, "int8"),
]


@pytest.mark.parametrize("M,K,xt,yt,post,gate,bias,layer,out", NORM)
def test_norm(M, K, xt, yt, post, gate, bias, layer, out):
    say(f"norm M={M} K={K} x={xt} y={yt} post={post} gate={gate} layer={layer} {out}")
    d, r = norm_case(M, K, xt, yt, post, gate, bias)
    kw = dict(y_scale=0.3, x_scale=0.9, eps=1e-6) if yt else dict(x_scale=1.5)
    res, v, n = check_norm(d, r, out, layer, **kw)
    # and against the formula in float64
    v64, tv, n64, tn = ref.norm64(**r, layer=layer, **kw)
    within(v.astype(np.float64), v64, tv)
    if out in ("f32", "f16", "bf16"):
        within(f64(res["out"]), n64, tn + ref.rounding(np.abs(n64) + tn, out))
    elif out == "int8":
        got = f64(res["out"]) * f64(res["sx"])[:, None]
        within(got, n64, tn + 0.5001 * f64(res["sx"])[:, None])


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("yt", [None, "f32", "f16", "bf16"])
def test_norm_every_type(xt, yt):
    for M, K in ((2, 272), (530, 272)):
        d, r = norm_case(M, K, xt, yt, bool(yt), "row" if yt else "none", True)
        for out in OUT:
            for layer in (False, True):
                say(f"norm types x={xt} y={yt} {out} layer={layer} M={M}")
                check_norm(d, r, out, layer)


def test_norm_without_weights():
    """No norm before the projection (post-norm layers), nor after the block."""
    for M, K in ((3, 4112), (3, 33000 // 16 * 16)):
        for out in ("int8", "e4m3", "bf16"):
            d, r = norm_case(M, K, "bf16", "f16", True, "all", True)
            for name in ("weight", "bias"):
                del d[name], r[name]
            check_norm(d, r, out, True)
            for name in ("y_weight", "y_bias"):
                del d[name], r[name]
            check_norm(d, r, out, False, y_scale=-2.0)


@pytest.mark.parametrize("K", [64, 5008, 33024])
def test_norm_rows_that_are_not_finite(K):
    """NaN and infinities stay in their rows; sums, squares and scales that
    overflow or vanish follow the definition."""
    d, r = norm_case(12, K, "f32", "f32", True, "all", True)
    x, y = r["x"].copy(), r["y"].copy()
    x[0, K // 2] = np.nan
    x[1, 3] = np.inf
    y[2, K - 1] = -np.inf
    x[3] = 3e38           # squares leave float32, not float64
    y[4] = 3e38
    x[5] = 1e-42          # subnormal
    y[5] = 0
    x[6, ::2], x[6, 1::2] = 2e-45, -2e-45
    y[6] = 1e-44
    x[7] = 0
    y[7] = 0
    x[8] = 1.0            # no spread: a layer norm divides by sqrt(eps)
    y[8] = -7.5
    y[9, 0] = 3e38
    r["x"], r["y"] = x, y
    d["x"], d["y"] = typed(x, "f32")[0], typed(y, "f32")[0]
    for layer in (False, True):
        for out in ("int8", "e4m3", "f32", "f16", "bf16"):
            say(f"norm special K={K} layer={layer} {out}")
            check_norm(d, r, out, layer, eps=1e-30)
            check_norm(d, r, out, layer, x_scale=2.0, y_scale=3.0)


def test_norm_in_place_and_parts_of_a_batch():
    """The new stream over the old one; rows behind the last are left alone."""
    for M, K, xt in ((5, 4096, "bf16"), (600, 1040, "f16"), (2, 40000, "f32")):
        d, r = norm_case(M, K, xt, "f16", True, "row", False)
        v, n = ref.norm(**r)
        big = {"out": poison((M + 2, K), torch.int8), "sx": poison(M + 2, torch.float32)}
        x = poison((M + 2, K), TYPES[xt])
        x[:M] = d["x"]
        tail = [t[M:].clone() for t in (big["out"], big["sx"], x)]
        dst = {"out": big["out"][:M], "sx": big["sx"][:M], "x": x[:M]}
        w4.norm_quant(**dict(d, x=x[:M]), out=dst)
        q, s = ref.codes(n, "int8")
        same_bits(dst["out"], q)
        same_bits(dst["sx"], s)
        same_bits(dst["x"], as_type(v, xt))
        for t, want in zip((big["out"], big["sx"], x), tail):
            assert torch.equal(t[M:].view(torch.uint8), want.view(torch.uint8))


def test_norm_feeds_the_gemms_as_the_quantisers_do():
    """Codes of a float32 result equal quant_act's and quant_act_fp8's of it."""
    for M in (9, 700):
        d, _ = norm_case(M, 1024, "bf16", "f16", False, "none", False)
        n = w4.norm_quant(**d, out_type=w4.NORM_OUT_F32)["out"]
        for out, quant in ((w4.NORM_OUT_INT8, w4.quant_act), (w4.NORM_OUT_E4M3, w4.quant_act_fp8)):
            r = w4.norm_quant(**d, out_type=out)
            q, s = quant(n)
            assert torch.equal(r["out"], q) and torch.equal(r["sx"], s)


def test_norm_past_4_gib():
    """Rows whose offsets pass 32 bits, in elements and in bytes."""
    M, K = 140000, 16400
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    x[:3].normal_()
    x[-3:].normal_()
    x[3:-3].fill_(1.0)
    y = torch.ones((M, K), dtype=torch.float16, device=DEV)
    w = torch.ones(K, device=DEV)
    assert M * K > 1 << 31
    r = w4.norm_quant(x, w, y=y, out_type=w4.NORM_OUT_INT8)
    for part in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        v, n = ref.norm(x[part].float().cpu().numpy(), y[part].float().cpu().numpy(),
                        weight=np.ones(K, np.float32))
        q, s = ref.codes(n, "int8")
        same_bits(r["out"][part], q)
        same_bits(r["sx"][part], s)
        same_bits(r["x"][part], as_type(v, "bf16"))
    assert bool((r["out"][3:-3] == 127).all())


def test_norm_empty_and_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((4, 64), dtype=torch.float16, device=DEV)
    w = torch.ones(64, device=DEV)
    r = w4.norm_quant(x[:0], w, y=y[:0])
    assert r["out"].shape == (0, 64) and r["sx"].shape == (0,) and r["x"].shape == (0, 64)
    assert w4.norm_quant(x, w)["x"] is x
    for bad in (dict(weight=w[:32]), dict(bias=w, weight=None), dict(y=y[:3]), dict(y_weight=w),
                dict(gate=y), dict(y=y, gate=y[:2]), dict(y=y, gate=y[0]), dict(y=y, y_bias=w),
                dict(y=y, gate_ids=torch.zeros(4, dtype=torch.int32, device=DEV)),
                dict(x=x.t()), dict(x=x[0]), dict(weight=w.cpu()), dict(out_type=5),
                dict(y=y, gate=y[:2], gate_ids=torch.zeros(3, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            w4.norm_quant(**dict(dict(x=x, weight=w), **bad))
    for bad in (dict(weight=w.half()), dict(y=y.to(torch.int8)), dict(y=y, gate=y.float()),
                dict(y=y, gate=y, gate_ids=torch.zeros(4, dtype=torch.int64, device=DEV))):
        with pytest.raises(TypeError):
            w4.norm_quant(**dict(dict(x=x, weight=w), **bad))
    out = w4.norm_quant(x, w, y=y)
    with pytest.raises(TypeError):
        w4.norm_quant(x, w, y=y, out_type=w4.NORM_OUT_E4M3, out=out)
    with pytest.raises(TypeError):
        w4.norm_quant(x, w, y=y, out=dict(out, x=out["x"].float()))
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(x_scale=float("inf")), dict(kind=2)):
        with pytest.raises(w4.W4A8Error) as e:
            w4.norm_quant(x, w, **bad)
        assert e.value.status == 5
    with pytest.raises(w4.W4A8Error) as e:  # K % 16
        w4.norm_quant(torch.zeros((4, 72), dtype=torch.bfloat16, device=DEV))
    assert e.value.status == 2
    with pytest.raises(w4.W4A8Error) as e:  # a row that starts between 16-byte pieces
        w4.norm_quant(torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64))
    assert e.value.status == 3


# -------------------------------------------------------------------- ffn ---

def block(H, F, g, seed):
    """Packed weights of a block and their decoded values."""
    w13, W13, sw13 = experts(1, 2 * F, H, g, 6000 + seed)
    w2, W2, sw2 = experts(1, H, F, g, 7000 + seed)
    return w13, w2, (W13[0], sw13[0], W2[0], sw2[0])


def rows(M, H, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, H)).astype(np.float32)
    x[:, rng.random(H) < 0.02] *= 20
    q, s = oracle.quant_sym_rows(x, 127)
    return q, s


def run_ffn(q, s, w13, w2, act, dt, ws_fill=0xAB):
    M, H = q.shape
    F = w2["K"]
    Y = poison((M, H), TYPES[dt])
    ws = torch.empty(w4.ffn_workspace_size(M, H, F), dtype=torch.uint8, device=DEV).fill_(ws_fill)
    w4.ffn(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), w13, w2,
           act=w4.ACT_GELU if act == "gelu" else w4.ACT_SILU, out=Y, workspace=ws)
    return Y


FFN = [
    (1, 128, 128, 64, "silu", "f16"),        # one K-tile in each product
    (1, 4096, 1408, 128, "gelu", "bf16"),
    (1, 256, 11008, 64, "silu", "f16"),
    (2, 384, 640, 128, "silu", "bf16"),
    # from three rows on h is quantised by a kernel of its own
    (3, 1152, 384, 64, "silu", "f16"),
    (4, 4096, 1408, 128, "gelu", "bf16"),
    (4, 8192, 5504, 64, "silu", "bf16"),
    (5, 1152, 384, 64, "silu", "f16"),
    # group parameters of the longest rows do not fit in LDS
    (2, 128, 131072, 64, "silu", "bf16"),
    (20, 128, 131072, 64, "silu", "f16"),
    (70, 128, 131072, 128, "gelu", "f16"),
    (3, 131072, 128, 64, "silu", "f16"),
    (40, 131072, 128, 64, "gelu", "bf16"),
    (15, 512, 384, 64, "gelu", "f16"),
    (16, 1024, 2688, 128, "silu", "bf16"),
    (17, 640, 896, 64, "silu", "f16"),
    (31, 256, 1280, 128, "gelu", "bf16"),
    (33, 512, 11008, 64, "silu", "f16"),
    (47, 4096, 2688, 128, "gelu", "f16"),
    (63, 384, 8192, 128, "silu", "bf16"),
    (64, 512, 384, 128, "silu", "f16"),      # streamed, two row blocks
    (65, 384, 640, 64, "gelu", "bf16"),      # H not a multiple of 256
    (100, 2048, 1408, 64, "gelu", "f16"),
    (128, 1024, 4096, 128, "silu", "bf16"),
    (129, 8192, 128, 64, "silu", "f16"),
    (133, 128, 8320, 128, "gelu", "bf16"),
    (257, 1024, 1152, 64, "silu", "bf16"),
    (300, 256, 28672, 128, "silu", "f16"),
    (513, 4096, 384, 128, "gelu", "bf16"),
    (1000, 512, 5504, 64, "silu", "f16"),
    (2050, 256, 4224, 128, "silu", "bf16"),
    # (test_ffn_plan.py compares the plans' forms with these sizes and ffn_cases.py)
    # 64-row tiles of 128 channels of each half; 128-row tiles of many rows
    (300, 256, 11008, 64, "gelu", "f16"),
    (4296, 128, 8320, 128, "silu", "f16"),
    # down: 64-row tiles with their K split, and where 256 does not divide H
    (64, 8192, 6400, 128, "silu", "bf16"),
    (50, 8192, 8320, 64, "silu", "f16"),
    (3000, 384, 1408, 64, "gelu", "bf16"),
    # down: the GEMM's own plans (two K parts, 32 x 32, 128- and 256-row tiles)
    (300, 8192, 2048, 128, "silu", "bf16"),
    (300, 8192, 16640, 128, "silu", "bf16"),
    (2048, 8192, 128, 64, "gelu", "bf16"),
    (2048, 8192, 8320, 128, "silu", "bf16"),
]


@pytest.mark.parametrize("M,H,F,g,act,dt", FFN)
def test_ffn(M, H, F, g, act, dt):
    say(f"ffn M={M} H={H} F={F} g={g} {act} {dt}")
    w13, w2, dec = block(H, F, g, 1)
    q, s = rows(M, H, M + H)
    Y = run_ffn(q, s, w13, w2, act, dt)
    want, tol = ref.ffn(q, s, *dec, act, dt)
    within(f64(Y), want, tol)


@pytest.mark.parametrize("M", [3, 40, 200, 600])
def test_ffn_odd_rows(M):
    """All-zero rows, rows with a scale that is not finite (NaN out, the others
    unaffected), tiny and huge scales, and three calls with the same bits
    whatever the workspace held."""
    H, F, g = 512, 640, 64
    w13, w2, dec = block(H, F, g, 2)
    q, s = rows(M, H, 5)
    q[1] = 0
    s[0], s[2] = np.nan, np.inf
    if M > 10:
        s[4], s[5], s[6], s[7] = 1e-30, 1e18, 3e38, -s[7]
        q[8] = -127
        q[9] = 127
    outs = [run_ffn(q, s, w13, w2, "silu", "bf16", fill) for fill in (0, 0xAB, 0xFF)]
    want, tol = ref.ffn(q, s, *dec, "silu", "bf16")
    got = f64(outs[0])
    assert np.isnan(got[0]).all() and np.isnan(got[2]).all() and (got[1] == 0).all()
    ok = np.ones(M, bool)
    if M > 10:
        # gate and up of 1e18 x 127 x ... leave the range where rounding is
        # relative in act(g) u; only finiteness of the neighbours is at stake
        ok[[5, 6]] = False
        assert np.isnan(got[6]).all()
    within(got[ok], want[ok], tol[ok])
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


def test_ffn_part_of_a_batch():
    """Rows behind the last are left as they were."""
    H, F, g = 256, 384, 64
    w13, w2, dec = block(H, F, g, 3)
    for M in (1, 20, 64, 130, 300):
        q, s = rows(M, H, 9)
        big = poison((M + 3, H), torch.float16)
        tail = big[M:].clone()
        w4.ffn(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), w13, w2, out=big[:M])
        want, tol = ref.ffn(q, s, *dec, "silu", "f16")
        within(f64(big[:M]), want, tol)
        assert torch.equal(big[M:].view(torch.int16), tail.view(torch.int16))


def test_ffn_as_one_expert():
    """The block is the expert layer of one expert with weight 1 on the same
    rows (which there are quantised inside)."""
    H, F, g = 512, 896, 128
    w13, w2, _ = block(H, F, g, 4)
    for T in (1, 9, 70, 200):
        X = torch.randn(T, H, device=DEV, dtype=torch.bfloat16)
        q, s = w4.quant_act(X)
        a = w4.ffn(q, s, w13, w2, dtype=torch.bfloat16).float()
        one = torch.ones((T, 1), device=DEV)
        b = w4.moe(X, torch.zeros((T, 1), dtype=torch.int32, device=DEV), one, w13, w2).float()
        # the same definition: codes of h next to a half may differ
        err = (a - b).norm() / b.norm()
        assert err < 2.0 ** -8, err


def test_ffn_refusals():
    w13, w2, _ = block(256, 384, 64, 5)
    q = torch.zeros((4, 256), dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    assert w4.ffn(q, s, w13, w2).shape == (4, 256)
    assert w4.ffn(q[:0], s[:0], w13, w2).shape == (0, 256)
    for bad in (dict(Xq=q[:, :128]), dict(Xq=q.t()), dict(Xq=q[0]), dict(sx=s[:3]),
                dict(sx=s.cpu()), dict(w13=dict(w13, N=384)), dict(w2=dict(w2, group=128)),
                dict(w2=dict(w2, wq=w2["wq"][:-16])), dict(out=torch.empty(3, 256, device=DEV,
                                                                          dtype=torch.float16))):
        a = dict(dict(Xq=q, sx=s, w13=w13, w2=w2), **bad)
        with pytest.raises(ValueError):
            w4.ffn(**a)
    for bad in (dict(Xq=q.to(torch.uint8)), dict(sx=s.half()), dict(dtype=torch.float32),
                dict(out=torch.empty(4, 256, device=DEV))):
        with pytest.raises(TypeError):
            w4.ffn(**dict(dict(Xq=q, sx=s, w13=w13, w2=w2), **bad))
    with pytest.raises(w4.W4A8Error) as e:
        w4.ffn(q, s, w13, w2, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4
    with pytest.raises(w4.W4A8Error) as e:
        w4.ffn(q, s, w13, w2, act=2)
    assert e.value.status == 5


# --------------------------------------------------------------- together ---

class Layer:
    """The feed-forward half of a layer with norms before and after the block:
    x += gate norm(ffn(norm(x))), and the next projection's rows."""

    def __init__(self, M, H, F, g):
        self.w13, self.w2, self.dec = block(H, F, g, 6)
        rng = np.random.default_rng(8)
        self.w = [rng.standard_normal(H).astype(np.float32) for _ in range(3)]
        self.gate = rng.random((1, H)).astype(np.float32)
        self.dw = [torch.from_numpy(w).to(DEV) for w in self.w]
        self.dgate = torch.from_numpy(self.gate).to(DEV, torch.bfloat16)
        i8, f4 = torch.int8, torch.float32
        self.a = {"out": poison((M, H), i8), "sx": poison(M, f4), "x": None}
        self.y = poison((M, H), torch.bfloat16)
        self.b = {"out": poison((M, H), i8), "sx": poison(M, f4)}
        self.ws = torch.empty(w4.ffn_workspace_size(M, H, F), dtype=torch.uint8, device=DEV)

    def run(self, x, stream=None):
        w4.norm_quant(x, self.dw[0], out=self.a, stream=stream)
        w4.ffn(self.a["out"], self.a["sx"], self.w13, self.w2, out=self.y, workspace=self.ws,
               stream=stream)
        w4.norm_quant(x, self.dw[2], y=self.y, y_weight=self.dw[1], gate=self.dgate, y_scale=0.5,
                      out=dict(self.b, x=x), stream=stream)

    def check(self, x0, x):
        """Every step against its reference on the values it was given."""
        q, s = ref.codes(ref.norm(x0, weight=self.w[0])[1], "int8")
        same_bits(self.a["out"], q)
        same_bits(self.a["sx"], s)
        want, tol = ref.ffn(q, s, *self.dec, "silu", "bf16")
        within(f64(self.y), want, tol)
        v, n = ref.norm(x0, self.y.float().cpu().numpy(), y_weight=self.w[1], weight=self.w[2],
                        gate=self.dgate.float().cpu().numpy(), y_scale=0.5)
        same_bits(x, as_type(v, "bf16"))
        q, s = ref.codes(n, "int8")
        same_bits(self.b["out"], q)
        same_bits(self.b["sx"], s)


def stream_values(M, H, seed):
    t = torch.from_numpy(np.random.default_rng(seed).standard_normal((M, H)).astype(np.float32))
    t = t.to(torch.bfloat16)
    return t.to(DEV), t.float().numpy()


@pytest.mark.parametrize("M", [1, 24, 96, 640])
def test_layer_eager_and_captured(M):
    """norm_quant, ffn and norm_quant as a layer runs them: eagerly, on another
    stream, and captured once and replayed with new values between eager calls
    that share the buffers."""
    H, F = 512, 1152
    lay = Layer(M, H, F, 64)
    x, x0 = stream_values(M, H, 1)
    lay.run(x)
    lay.check(x0, x)
    side = torch.cuda.Stream()
    x, x0 = stream_values(M, H, 2)
    side.wait_stream(torch.cuda.current_stream())
    lay.run(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    lay.check(x0, x)

    g = torch.cuda.CUDAGraph()
    x, _ = stream_values(M, H, 3)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lay.run(x)
    for seed in (4, 5, 6):
        new, x0 = stream_values(M, H, seed)
        x.copy_(new)
        lay.ws.fill_(seed)
        g.replay()
        lay.check(x0, x)
        other, other0 = stream_values(M, H, 50 + seed)
        lay.run(other)
        lay.check(other0, other)


def test_two_layers_with_their_own_workspaces_overlap():
    """Calls on two streams at once, each with its own buffers."""
    M, H, F = 96, 512, 1152
    lays = [Layer(M, H, F, 64), Layer(M, H, F, 64)]
    xs = [stream_values(M, H, 20 + i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (x, x0), st in zip(xs, streams):
            with torch.cuda.stream(st):
                x.copy_(torch.from_numpy(x0).to(DEV, torch.bfloat16))
        for lay, (x, _), st in zip(lays, xs, streams):
            lay.run(x, stream=st)
        torch.cuda.synchronize()
        for lay, (x, x0) in zip(lays, xs):
            lay.check(x0, x)
