"""Values, sizes and kernels at the borders of the norm with quantisation and of
the gated feed-forward block, on the GPU (references: layer_refs.py)."""
import math
from fractions import Fraction

import numpy as np
import pytest

import layer_refs as ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_amd as w4  # noqa: E402
from ffn_cases import CASES  # noqa: E402
from test_gpu_layer import (as_type, block, check_norm, norm_case, rows, run_ffn,  # noqa: E402
                            same_bits)
from selection_refs import decode_weights  # noqa: E402
from test_gpu_selection import DEV, TYPES, f64, host, say, within  # noqa: E402


def subnormal_rows(K):
    """Rows of subnormal float32 values: the largest is m smallest subnormals, so
    the scale is a whole number of them and max / scale is not the codes' top
    (667 / 1 against 448, 190 / 1 against 127)."""
    tops = [1, 3, 63, 64, 190, 191, 224, 225, 465, 600, 667, 671, 672, 928, 929, 1000, 1119, 1121,
            2500, 5000, 100003, 8000009]
    rng = np.random.default_rng(K)
    x = np.zeros((len(tops), K), np.int32)
    for i, m in enumerate(tops):
        x[i] = rng.integers(-m, m + 1, K)
        x[i, rng.integers(K)] = m * (-1) ** i
    return np.copysign(np.abs(x).view(np.float32), x.astype(np.float32))


@pytest.mark.parametrize("K", [48, 5008, 33024])
def test_subnormal_rows(K):
    """Quotients past the codes' range saturate: no code of a finite row is NaN."""
    x = subnormal_rows(K)
    dx = torch.from_numpy(x).to(DEV)
    for many in (False, True):
        reps = 20 if many else 1
        d, r = dx.repeat(reps, 1), np.tile(x, (reps, 1))
        for out, quant in (("int8", w4.quant_act), ("e4m3", w4.quant_act_fp8)):
            say(f"subnormal rows K={K} {out} x{reps}")
            q, s = ref.codes(r, out)
            got = w4.norm_quant(d, out_type=getattr(w4, "NORM_OUT_" + out.upper()))
            same_bits(got["sx"], s)
            same_bits(got["out"], q)
            codes, scales = quant(d)
            same_bits(scales, s)
            same_bits(codes, q)
            if out == "e4m3":
                assert np.abs(oracle.e4m3_decode(q)).max() == 448.0


def squares(S, K):
    """K integers below 2^24 whose squares add up to S < 2^53 (so every sum of
    some of them is exact in float64, in any order)."""
    x = [math.isqrt(S // 40)] * 40
    S -= 40 * x[0] ** 2
    while S:
        x.append(math.isqrt(S))
        S -= x[-1] ** 2
    assert len(x) <= K and x[0] < 1 << 24
    return np.array(x + [0] * (K - len(x)), np.float32)


@pytest.mark.parametrize("K", [64, 80, 5008, 33024])
def test_inverse_root_next_to_a_rounding_border(K):
    """1 / sqrt(mean + eps) within some 2^-52 of the middle between two float32
    numbers: the definition's float64 operations decide on which side it falls."""
    rng = np.random.default_rng(K)
    M = 3000 if K < 100 else 120
    x = []
    for i in range(M):
        m = (1 << 24) + int(rng.integers(1 << 24))             # 25 bits, odd: a middle
        b = (2 * (m // 2) + 1) / float(1 << 24)                # in [1, 2)
        b *= 2.0 ** math.floor(math.log2(math.sqrt(K / 2.0 ** 53)) + 1)
        S = int(round(Fraction(K) / (Fraction(b) * Fraction(b)))) + i % 7 - 3
        while S >= 1 << 53:
            S >>= 2                                            # (the same middle, doubled)
        x.append(squares(S, K))
    x = np.stack(x)
    w = np.ones(K, np.float32)
    say(f"inverse root K={K}")
    _, n = ref.norm(x, weight=w, eps=1e-30)
    d = dict(weight=torch.from_numpy(w).to(DEV), eps=1e-30, out_type=w4.NORM_OUT_F32)
    got = w4.norm_quant(torch.from_numpy(x).to(DEV), **d)
    same_bits(got["out"], n)


# (widths of which a product with the rounded 1 / K misses some of these quotients)
@pytest.mark.parametrize("K", [784, 1968, 5152, 38576])
def test_mean_next_to_a_rounding_border(K):
    """Rows of two neighbouring float32 numbers, half each: the mean is exactly the
    middle between them, and rounds to the even one."""
    rng = np.random.default_rng(K)
    M = 400 if K < 1000 else 40
    lo = rng.uniform(1.0, 2.0, (M, 1)).astype(np.float32) * 2.0 ** rng.integers(-30, 30, (M, 1))
    lo = lo.astype(np.float32)
    hi = np.nextafter(lo, np.float32(np.inf))
    x = np.where(rng.permuted(np.tile(np.arange(K) % 2, (M, 1)), axis=1) == 0, lo, hi)
    x *= np.where(np.arange(M) % 2, 1, -1).astype(np.float32)[:, None]
    w = np.ones(K, np.float32)
    say(f"mean K={K}")
    _, n = ref.norm(x, weight=w, layer=True, eps=1e-30)
    d = dict(weight=torch.from_numpy(w).to(DEV), eps=1e-30, kind=w4.NORM_LAYER,
             out_type=w4.NORM_OUT_F32)
    got = w4.norm_quant(torch.from_numpy(x).to(DEV), **d)
    same_bits(got["out"], n)


@pytest.mark.parametrize("K", [512, 1024, 2048, 4096, 5120, 8192, 16384, 33024])
@pytest.mark.parametrize("layer", [False, True])
def test_rows_do_not_depend_on_their_batch(K, layer):
    """The same rows alone, in a small and in a large batch: the same bits, also
    where sums cancel (values of both signs far above the others), whose result
    is a matter of the order of the additions."""
    rng = np.random.default_rng(K)
    M = 300
    x = rng.standard_normal((M, K)).astype(np.float32)
    for i in range(0, M, 2):
        at = rng.permutation(K)[:K // 8]
        big = np.exp2(rng.uniform(20, 90, len(at) // 2)).astype(np.float32)
        x[i, at[:len(big)]], x[i, at[len(big):2 * len(big)]] = big, -big
    w = np.ones(K, np.float32)
    d = dict(weight=torch.from_numpy(w).to(DEV), out_type=w4.NORM_OUT_F32,
             kind=w4.NORM_LAYER if layer else w4.NORM_RMS)
    dx = torch.from_numpy(x).to(DEV)
    say(f"rows alone and in a batch K={K} layer={layer}")
    want = host(w4.norm_quant(dx, **d)["out"])
    for m in (1, 7, 256):
        for at in (0, M - m):
            got = host(w4.norm_quant(dx[at:at + m].contiguous(), **d)["out"])
            assert np.array_equal(got, want[at:at + m]), (m, at)


def test_empty_batch_with_its_gates():
    """No rows, and so no gate of a row: nothing to do, as in the C entry."""
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    ids = torch.zeros(0, dtype=torch.int32, device=DEV)
    for gate in (x, torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)):
        for more in ({}, dict(gate_ids=ids)):
            r = w4.norm_quant(x, w, y=x, gate=gate, **more)
            assert r["out"].shape == (0, 64) and r["sx"].shape == (0,)
    one = torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)
    for more in ({}, dict(gate_ids=torch.zeros(1, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError, match="rows"):
            w4.norm_quant(one, w, y=one, gate=x, **more)


def test_result_names_every_output():
    """out, sx and x are there whatever the caller's dict holds: x itself without
    y, no scales for floating types; the dict is not changed."""
    x = torch.randn((4, 64), device=DEV).to(torch.bfloat16)
    w = torch.ones(64, device=DEV)
    plain = w4.norm_quant(x, w)
    old = torch.empty_like(x)
    for into in ({"out": torch.empty((4, 64), dtype=torch.int8, device=DEV),
                  "sx": torch.empty(4, device=DEV)},
                 {"out": torch.empty((4, 64), dtype=torch.int8, device=DEV),
                  "sx": torch.empty(4, device=DEV), "x": old}):
        keys = dict(into)
        r = w4.norm_quant(x, w, out=into)
        assert r["x"] is x and r["out"] is into["out"] and r["sx"] is into["sx"]
        assert torch.equal(r["out"], plain["out"]) and torch.equal(r["sx"], plain["sx"])
        assert into == keys
    for into in ({"out": old}, {"out": old, "sx": torch.empty(4, device=DEV), "x": x}):
        r = w4.norm_quant(x, w, out_type=w4.NORM_OUT_BF16, out=into)
        assert r["x"] is x and r["sx"] is None and r["out"] is old
    full = {"out": old, "sx": None, "x": x}
    assert w4.norm_quant(x, w, out_type=w4.NORM_OUT_BF16, out=full) is full


def test_one_gate_by_ids():
    """A single gate row that some rows name and others do not."""
    M, K = 9, 272
    d, r = norm_case(M, K, "bf16", "f16", True, "all", True)
    ids = np.array([0, 1, -1, 0, 2, 0, -(1 << 31), (1 << 31) - 1, 0], np.int32)
    d["gate_ids"], r["ids"] = torch.from_numpy(ids).to(DEV), ids
    check_norm(d, r, "int8", False)
    check_norm(d, r, "f32", True)


@pytest.mark.parametrize("K", [16, 2064])
def test_norm_of_the_most_rows(K):
    """2^22 - 1 rows with an odd period: all against the first ones, and those
    against the definition."""
    M, P = (1 << 22) - 1, 1021
    d, r = norm_case(P, K, "bf16", "f16", False, "none", True)
    at = torch.arange(M, device=DEV) % P
    out = w4.norm_quant(**dict(d, x=d["x"][at], y=d["y"][at]))
    v, n = ref.norm(**r)
    q, s = ref.codes(n, "int8")
    same_bits(out["x"][:P], as_type(v, "bf16"))
    same_bits(out["out"][:P], q)
    same_bits(out["sx"][:P], s)
    for t in (out["x"].view(torch.int16), out["out"], out["sx"].view(M, 1)):
        whole = M // P
        for i in range(0, whole, 256):
            k = min(256, whole - i)
            assert bool((t[i * P:(i + k) * P].view(k, P, -1) == t[:P]).all()), i
        assert torch.equal(t[whole * P:], t[:M - whole * P])


# -------------------------------------------------------------------- ffn ---

def packed(W, g):
    """Packed weights of W, their decoded INT8 values and channel scales."""
    N, K = W.shape
    p = w4.pack(torch.from_numpy(W).to(DEV), group=g)
    W8 = decode_weights(host(p["wq"]).ravel(), host(p["s_u8"]).ravel(), host(p["a_u8"]).ravel(),
                        N, K, g)
    return p, W8, host(p["sw"])


def selection(n, g):
    """Packed [n][n] weights of one nonzero INT8 weight a row, on the diagonal, and
    that weight: the product is then each channel's own code."""
    p, W8, _ = packed(np.eye(n, dtype=np.float32), g)
    w = int(W8[0, 0])
    assert w > 0 and (W8 == w * np.eye(n, dtype=W8.dtype)).all()
    return p, w


@pytest.mark.parametrize("M", [1, 2, 15, 64, 300, 1300])
def test_ffn_codes_of_small_activations(M):
    """Codes of h where every gate lies between -40 and -75.

    exp(-g) evaluated to one unit in the last place (2 u, u = 2^-24), the sum, the
    quotient and the product (u each) put h within 5 u of its value, the row's
    largest |h| likewise, and the scale and a code's quotient add u each: a code may
    differ from that of the float64 quotient q only where q lies within 12 u |q|
    of a half.  A power of the rounded product g log2(e) would be off by up to
    |g| u = 75 u alone."""
    n, g = 2048, 64
    say(f"ffn small activations M={M}")
    rng = np.random.default_rng(M)
    w = rng.random((2 * n, n), dtype=np.float32)
    w[:n] = -0.5 - 0.5 * w[:n]                     # gate: sums of one sign
    w[n:] = w[n:] - 0.5                            # up: any
    w13, W13, sw13 = packed(w, g)
    w2, one = selection(n, g)
    q = rng.integers(60, 128, (M, n)).astype(np.int8)
    acc = (torch.from_numpy(q).double() @ torch.from_numpy(W13).double().t()).numpy()
    scale = np.float32(55.0 / np.abs((acc[:, :n] * sw13[:n]).mean()))
    s = (scale * rng.uniform(0.9, 1.1, M)).astype(np.float32)
    gu = (acc.astype(np.float32) * s[:, None]) * sw13
    assert gu.dtype == np.float32
    a, b = gu[:, :n].astype(np.float64), gu[:, n:].astype(np.float64)
    assert -75 < a.min() and a.max() < -40
    h = a / (1.0 + np.exp(-a)) * b
    sh = np.abs(h).max(1, keepdims=True) / 127.0
    quot = h / sh
    # (the down product's channel scale only brings the outputs near the codes)
    by = 1.0 / (one * sh.mean())
    w2["sw"] = torch.full((n,), by, dtype=torch.float32, device=DEV)
    Y = w4.ffn(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), w13, w2)
    got = f64(Y) / (one * sh * float(np.float32(by)))
    code = np.rint(got)
    assert bool(np.abs(got - code).max() < 0.07)   # fp16: 127 x 2^-11
    near = np.abs(np.abs(quot - np.floor(quot)) - 0.5) <= 12 * 2.0 ** -24 * np.abs(quot)
    assert bool(near.mean() < 1e-3)
    bad = (code != np.rint(quot)) & ~near
    assert not bad.any(), (int(bad.sum()), quot[bad][:5], code[bad][:5])


@pytest.mark.parametrize("M,H,F,g,act,dt", CASES)
def test_ffn_forms(M, H, F, g, act, dt):
    """Every kernel that a plan can choose (ffn_cases.py)."""
    say(f"ffn form M={M} H={H} F={F} g={g} {act} {dt} {w4.ffn_plan(M, H, F)}")
    w13, w2, dec = block(H, F, g, 1)
    q, s = rows(M, H, M + H)
    Y = run_ffn(q, s, w13, w2, act, dt)
    want, tol = ref.ffn(q, s, *dec, act, dt)
    within(f64(Y), want, tol)


def test_ffn_refuses_packed_arrays_that_are_not_1d():
    """As gemm_lora and moe do."""
    rng = np.random.default_rng(1)
    w13 = packed(rng.random((768, 256), dtype=np.float32), 64)[0]
    w2 = packed(rng.random((256, 384), dtype=np.float32), 64)[0]
    q = torch.zeros((4, 256), dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    assert w4.ffn(q, s, w13, w2).shape == (4, 256)
    for name in ("wq", "s_u8", "a_u8", "sw"):
        for which, p in (("w13", w13), ("w2", w2)):
            a = dict(w13=w13, w2=w2)
            a[which] = dict(p, **{name: p[name].view(2, -1)})
            with pytest.raises(ValueError, match=which):
                w4.ffn(q, s, **a)


@pytest.mark.parametrize("H,F,g,dt", [(128, 1024, 64, "bf16"), (8192, 128, 128, "f16"),
                                      (128, 128, 128, "f16")])
def test_ffn_at_the_limit_of_its_rows(H, F, g, dt):
    """M H or M F just below 2^31: h of 8 GiB, rows and results of up to 4.  The
    batch repeats its first rows with an odd period, so every row is checked: the
    first ones and the last against the reference, all against the first."""
    M, P = ((1 << 31) - 1) // max(H, F), 4099
    say(f"ffn limit M={M} H={H} F={F} {w4.ffn_plan(M, H, F)}")
    assert w4.ffn_workspace_size(M + 1, H, F) == 0
    w13, w2, dec = block(H, F, g, 7)
    q, s = rows(P, H, 3)
    at = torch.arange(M, device=DEV) % P
    Xq = torch.from_numpy(q).to(DEV)[at]
    sx = torch.from_numpy(s).to(DEV)[at]
    Y = w4.ffn(Xq, sx, w13, w2, dtype=TYPES[dt])
    want, tol = ref.ffn(q, s, *dec, "silu", dt)
    within(f64(Y[:P]), want, tol)
    last = at[M - 300:].cpu().numpy()
    within(f64(Y[M - 300:]), want[last], tol[last])
    bits = Y.view(torch.int16)
    whole = M // P
    for i in range(0, whole, 64):
        n = min(64, whole - i)
        part = bits[i * P:(i + n) * P].view(n, P, H)
        assert bool((part == bits[:P]).all()), i
    assert torch.equal(bits[whole * P:], bits[:M - whole * P])


@pytest.mark.parametrize("H,F", [(512, 640), (5120, 384)])
def test_ffn_two_rows_do_not_touch_each_other(H, F):
    """The down product quantises both rows in one workgroup: one that is not
    finite is NaN, the other's results are those of the row alone."""
    w13, w2, _ = block(H, F, 64, 8)
    q, s = rows(2, H, 5)

    def run(q, s):
        return w4.ffn(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), w13, w2,
                      dtype=torch.bfloat16)
    alone = [run(q[i:i + 1], s[i:i + 1])[0] for i in range(2)]
    both = run(q, s)
    assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])
    for bad in (np.nan, np.inf, -np.inf, 3e38):
        for i in range(2):
            t = s.copy()
            t[i] = bad
            Y = run(q, t)
            assert bool(torch.isnan(Y[i]).all()), (bad, i)
            assert torch.equal(Y[1 - i], alone[1 - i]), (bad, i)
    z = q.copy()
    z[0] = 0
    Y = run(z, s)
    assert bool((Y[0] == 0).all()) and torch.equal(Y[1], alone[1])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 2, 40, 300])
def test_ffn_of_large_gates(act, M):
    """Gates from 1e3 to 1e13 of either sign (GELU's cube leaves float32): act(g) u
    is g u or 0, and codes and scale follow."""
    n, g = 512, 128
    rng = np.random.default_rng(M)
    w = rng.standard_normal((2 * n, n)).astype(np.float32)
    w[:n] = (0.5 + 0.5 * rng.random((n, n), dtype=np.float32)) * np.where(
        rng.random((n, 1)) < 0.5, -1, 1).astype(np.float32)
    w13, W13, sw13 = packed(w, g)
    w2, one = selection(n, g)
    q = rng.integers(60, 128, (M, n)).astype(np.int8)
    acc = (torch.from_numpy(q).double() @ torch.from_numpy(W13).double().t()).numpy()
    s = (10.0 ** rng.uniform(2, 12, M) / np.abs(acc[:, :n] * sw13[:n]).mean(1) * 10).astype(
        np.float32)
    gu = (acc.astype(np.float32) * s[:, None]) * sw13
    a, b = gu[:, :n].astype(np.float64), gu[:, n:].astype(np.float64)
    assert np.abs(a).min() > 700
    h = np.where(a > 0, a * b, 0.0)
    sh = np.abs(h).max(1, keepdims=True) / 127.0
    by = (1.0 / (one * sh)).astype(np.float32)
    for m in range(M):  # a channel scale for each row: results near the codes
        if m and m % 40:
            continue
        w2["sw"] = torch.full((n,), float(by[m, 0]), dtype=torch.float32, device=DEV)
        Y = w4.ffn(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), w13, w2,
                   act=w4.ACT_GELU if act == "gelu" else w4.ACT_SILU)
        got = f64(Y[m]) / (one * sh[m] * float(by[m, 0]))
        # half a code, and the fp16 rounding of one
        assert bool((np.abs(got - h[m] / sh[m]) <= 0.5 + 0.07).all())
