"""Edges of routing, the few-token mixture-of-experts layer and the
low-rank-adapter projection on the GPU: uneven routing, precision of the
adapters' products, values that are not finite."""
import numpy as np
import pytest

import selection_refs as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_amd as w4  # noqa: E402
from test_gpu_selection import DEV, TYPES, experts, f64, poison, say, tokens, within  # noqa: E402


# -------------------------------------------------------------------- moe ---
HOT = [  # more rows on one expert than its workgroups take in one pass
    # distinct ids: one row block, up to 64 rows at once
    (200, 64, 2, 512, 256, 64, "f16", True),
    (256, 64, 1, 256, 1152, 128, "bf16", True),
    # two row blocks, up to 128 rows
    (256, 16, 2, 384, 512, 128, "bf16", True),
    (150, 8, 2, 1152, 256, 64, "f32", True),
    # the same expert for every slot: one, two and four row blocks
    (16, 64, 5, 512, 384, 64, "bf16", False),
    (60, 4, 2, 256, 512, 128, "f16", False),
    (256, 2, 2, 512, 256, 64, "f16", False),
]


@pytest.mark.parametrize("T,E,k,H,F,g,dt,distinct", HOT)
def test_moe_hot_expert(T, E, k, H, F, g, dt, distinct):
    """Every token chooses one popular expert, whose rows are walked in
    several passes; three calls give the same bits."""
    say(f"moe hot T={T} E={E} k={k} H={H} F={F} g={g} {dt} distinct={distinct}")
    rng = np.random.default_rng(T + E + k)
    hot = E // 2
    w13, W13, sw13 = experts(E, 2 * F, H, g, 3600)
    w2, W2, sw2 = experts(E, H, F, g, 4600)
    X, Xf = tokens(T, H, dt, 52 + T)
    ids = np.full((T, k), hot, np.int32)
    if distinct:
        others = np.array([e for e in range(E) if e != hot])
        for t in range(T):
            ids[t, 1:] = rng.permutation(others)[:k - 1]
            ids[t] = rng.permutation(ids[t])
    w = rng.random((T, k)).astype(np.float32)
    dids, dw = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    outs = []
    for _ in range(3):
        Y = poison((T, H), TYPES[dt])
        w4.moe(X, dids, dw, w13, w2, out=Y)
        outs.append(Y)
    want, tol = ref.moe(Xf, ids, w, W13, sw13, W2, sw2, dt)
    within(f64(outs[0]), want, tol)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


# ------------------------------------------------------------------- lora ---
# streamed (one and several row blocks), K split, 128- and 256-row tiles with
# one, two and four sets of 32 ranks
PATHS = [(5, 320, 256, 8), (40, 512, 384, 16), (100, 192, 256, 40), (128, 512, 4096, 40),
         (130, 768, 256, 72), (300, 768, 640, 16), (2100, 4096, 512, 40), (2100, 4096, 512, 104)]


def bare(M, N, K, R, n, dt, seed):
    """A projection of zero weights (its sums are exactly 0), adapter choices
    and empty rows and adapters to fill in."""
    p = w4.pack(torch.zeros((N, K), device=DEV), group=64)
    rng = np.random.default_rng(seed)
    ad = rng.integers(-1, n, M).astype(np.int32)
    X, A, B = np.zeros((M, K)), np.zeros((n, R, K)), np.zeros((n, N, R))
    return p, rng, ad, X, A, B


def adapters(p, X, A, B, ad, dt):
    """gemm_lora of float64 arrays whose values the type holds exactly."""
    def dev(a):
        t = torch.from_numpy(a).to(TYPES[dt])
        same = t.double().numpy()
        assert np.array_equal(same, a, equal_nan=True)
        return t.to(DEV)
    lora = {"A": dev(A), "B": dev(B), "scale": torch.ones(len(A), device=DEV)}
    return f64(w4.gemm_lora(dev(X), p, lora, torch.from_numpy(ad).to(DEV)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,R", PATHS)
def test_lora_inner_product_is_kept_in_float32(M, N, K, R, dt):
    """Inner products of 24 significant bits that cancel in the outer one.

    Each is a sum of three 8-bit numbers 2^-8 apart, so every float32 sum that
    forms it is exact; a channel takes the difference of two that agree in
    their first 16 bits, next to one 2^26 times as large that it does not
    take.  What is left are the roundings of the outer sum, of two products of
    at most three parts each (six additions of u, and 2 u for parts that fall
    short of the number by one unit in its last place), and the output's."""
    say(f"lora bits M={M} N={N} K={K} R={R} {dt}")
    n = 3
    p, rng, ad, X, A, B = bare(M, N, K, R, n, dt, M + R)
    X[:, :4] = [2.0 ** 12, 2.0 ** -2, 2.0 ** -6, 2.0 ** -10]

    def eight(*shape):
        return rng.integers(128, 256, shape) / 128.0
    A[:, :, 1] = np.repeat(eight(n, R // 2), 2, axis=1)
    A[:, :, 2] = np.repeat(eight(n, R // 2), 2, axis=1) * 2.0 ** -4
    A[:, :, 3] = eight(n, R) * 2.0 ** -8
    A[:, ::32, 0] = 2.0 ** 12
    pairs = np.array([r for r in range(0, R, 2) if r % 32])
    first = pairs[np.arange(N) % len(pairs)]
    for a in range(n):
        B[a, np.arange(N), first] = 2.0 ** 10
        B[a, np.arange(N), first + 1] = -2.0 ** 10
    got = adapters(p, X, A, B, ad, dt)
    want, size = np.zeros((M, N)), np.zeros((M, N))
    for a in range(n):
        V = X @ A[a].T
        m = ad == a
        want[m] = V[m] @ B[a].T
        size[m] = np.abs(V[m]) @ np.abs(B[a]).T
    within(got, want, 8 * ref.U * size + ref.rounding(want, "f16"))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,R", PATHS)
def test_lora_infinities(M, N, K, R, dt):
    """Infinite elements of B (and of A) give the infinity, or the NaN, that
    the products of the definition give: a positive or negative infinity
    where the infinite terms agree, NaN where they do not or where the inner
    product is zero; in the rows of that adapter only."""
    say(f"lora inf M={M} N={N} K={K} R={R} {dt}")
    n = 4
    inf = float("inf")
    p, rng, ad, X, A, B = bare(M, N, K, R, n, dt, M + R + 1)
    ad[:5] = [0, 1, 2, 3, -1]
    eight = rng.integers(128, 256, (M, 2)) / 128.0
    X[:, 0] = eight[:, 0] * rng.choice([-1, 1], M)
    X[:, 1] = eight[:, 1] * 2.0 ** -8
    X[:, 2] = 1.0
    if M > 64:
        X[M // 2] = 0.0          # inner products of exactly 0
    A[:, :, 0] = rng.choice([-1, 1], (n, R))
    A[:, :, 1] = 1.0
    A[1, :, 1] = 0.0             # 8 significant bits: nothing behind the first part
    A[0, R - 1, 2] = 2.0 ** 14   # next to it the others are small ...
    A[0, R - 2] = 0.0
    A[0, R - 2, 2] = 2.0 ** -14  # ... and this one tiny
    A[3, 2, 2] = inf             # an infinite inner product
    B[:] = rng.choice([-1, 1], (n, N, R)) * 2.0 ** -10
    B[0, 3::7, R - 2] = -inf
    B[0, 4::7, 1] = inf
    B[1, 5::7, 0] = inf
    B[1, 6::7, 0] = inf
    B[1, 6::7, 3] = -inf
    B[2, ::5, R - 1] = -inf
    B[3, ::3, 2] = 0.0
    got = adapters(p, X, A, B, ad, dt)
    want, size = np.zeros((M, N)), np.zeros((M, N))
    with np.errstate(invalid="ignore"):
        for a in range(n):
            m = ad == a
            # (a column of A that is infinite: 0 x inf only where X is 0)
            V = np.where(X[m][:, None, :] == 0, np.where(np.isinf(A[a])[None], np.nan, 0.0),
                         X[m][:, None, :] * A[a][None]).sum(2)
            for c0 in range(0, N, 256):
                c = slice(c0, min(N, c0 + 256))
                terms = V[:, None, :] * B[a, c][None]
                want[m, c] = terms.sum(2)
                size[m, c] = np.abs(terms).sum(2)
    for f in (np.isnan, np.isposinf, np.isneginf):
        bad = f(got) != f(want)
        assert not bad.any(), (f.__name__, int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5],
                               want[bad][:5])
    ok = np.isfinite(want)
    # V of at most 24 + 14 bits: two float32 sums of R and a few terms
    within(got[ok], want[ok], (2 * R + 12) * ref.U * size[ok] + ref.rounding(want[ok], "f16"))


def test_lora_largest_inner_product():
    """An inner product next to float32's largest value, whose first part of
    bfloat16 rounds to an infinity, times a tiny B."""
    M, N, K, R = 6, 128, 256, 8
    p, rng, ad, X, A, B = bare(M, N, K, R, 2, "bf16", 3)
    ad[:] = [0, 1, -1, 0, 1, 1]
    X[:, :3] = [1.0, 2.0 ** -8, 2.0 ** -16]
    A[:, 3, :3] = 255 / 128 * 2.0 ** 127   # 24 ones: float32's largest
    A[1] *= -1
    B[:, :, 3] = 2.0 ** -120
    B[:, ::2, 5] = float("inf")            # (times an inner product of 0)
    got = adapters(p, X, A, B, ad, "bf16")
    want = np.zeros((M, N))
    want[ad == 0], want[ad == 1] = 256.0, -256.0   # (2^128 - 2^104) 2^-120 in fp16
    want[ad >= 0, ::2] = np.nan
    within(got, want, 0.0)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("H,F", [(w4.EXACT_MAX_K, 128), (128, w4.EXACT_MAX_K)])
def test_moe_longest_rows(T, H, F):
    """The longest rows with the largest codes: int32 sums 1.6 % below the
    wrap."""
    say(f"moe longest T={T} H={H} F={F}")
    g = 128
    up, down = 0.7 / H, 0.3 / F
    w13 = w4.pack_experts(torch.full((1, 2 * F, H), up, device=DEV), group=g)
    w2 = w4.pack_experts(torch.full((1, H, F), down, device=DEV), group=g)
    W13, W2 = np.full((1, 2 * F, H), 127, np.int8), np.full((1, H, F), 127, np.int8)
    for p, W in ((w13, W13), (w2, W2)):
        part = slice(0, 64 * W.shape[2] // 2)
        np.testing.assert_array_equal(
            ref.decode_weights(p["wq"][part].cpu().numpy(),
                               p["s_u8"][:64 * W.shape[2] // g].cpu().numpy(),
                               p["a_u8"][:64 * W.shape[2] // g].cpu().numpy(), 64, W.shape[2], g),
            W[0, :64])
    X = torch.ones((T, H), dtype=torch.float16, device=DEV)
    ids, w = np.zeros((T, 1), np.int32), np.full((T, 1), 1.5, np.float32)
    Y = poison((T, H), torch.float32)
    w4.moe(X, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), w13, w2, out=Y)
    one = slice(0, 1)  # every token is the same
    want, tol = ref.moe(X[one].float().cpu().numpy(), ids[one], w[one], W13,
                        w13["sw"].cpu().numpy()[None], W2, w2["sw"].cpu().numpy()[None], "f32")
    within(f64(Y), np.repeat(want, T, 0), np.repeat(tol, T, 0))


# ------------------------------------------------------------------ route ---
@pytest.mark.parametrize("T,E,k", [(2 ** 31 - 1, 1, 1), ((2 ** 31 - 1) // 3, 3, 2)])
def test_route_largest_batches(T, E, k):
    """T * E next to 2^31: outputs past 4 GiB, slots up to 2^31 - 2."""
    say(f"route largest T={T} E={E} k={k}")
    x = torch.zeros((T, E), dtype=torch.bfloat16, device=DEV)
    x[T // 2, E - 1] = 1.0
    x[T - 1] = float("-inf")
    r = w4.route(x, k)
    offsets, ids, rows = r["offsets"].tolist(), r["ids"], r["rows"]
    # ties: the first k experts, but for one token, and the last has none
    assert offsets[0] == 0 and offsets[E] == (T - 1) * k
    assert ids[T // 2, 0].item() == E - 1 and (ids[T - 1] == -1).all()
    assert (rows[(T - 1) * k:] == -1).all()
    for e in range(E):
        for lo in range(offsets[e], offsets[e + 1], 1 << 26):
            part = rows[lo:min(offsets[e + 1], lo + (1 << 26))].long()
            assert (part[1:] > part[:-1]).all() and (ids.view(-1)[part] == e).all()
    del x, r, ids, rows
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,R", PATHS)
def test_lora_rows_that_are_not_numbers(M, N, K, R, dt):
    """Every third row holds a NaN: NaN throughout where it selects an
    adapter, and the other rows keep their bits."""
    say(f"lora NaN rows M={M} N={N} K={K} R={R} {dt}")
    n = 3
    p, rng, ad, X, A, B = bare(M, N, K, R, n, dt, M + R + 2)
    X[:] = rng.integers(-8, 9, X.shape) / 8.0
    A[:] = rng.integers(-8, 9, A.shape) / 64.0
    B[:] = rng.integers(-8, 9, B.shape) / 64.0
    good = adapters(p, X, A, B, ad, dt)
    X[1::3, K // 2] = np.nan
    got = adapters(p, X, A, B, ad, dt)
    bad = np.zeros(M, bool)
    bad[1::3] = True
    assert np.isfinite(good).all()
    assert np.isnan(got[bad & (ad >= 0)]).all()
    np.testing.assert_array_equal(got[~bad], good[~bad])
