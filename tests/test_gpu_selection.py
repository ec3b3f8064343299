"""Routing, the few-token mixture-of-experts layer and the low-rank-adapter
projection on the GPU against 64-bit references (selection_refs.py states
the tolerances), and their behaviour in serving: captured graphs, other
streams, empty and odd calls, refusals."""
import numpy as np
import pytest

import oracle
import workloads as wl
import selection_refs as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_amd as w4  # noqa: E402

DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def f64(t):
    torch.cuda.synchronize()
    return t.cpu().to(torch.float64).numpy()


def poison(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    if t.numel():
        t.view(torch.uint8).fill_(0xAB)
    return t


def within(got, want, tol):
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want))
            | ((got == want) & np.isinf(want)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5],
                           np.broadcast_to(tol, want.shape)[bad][:5])


# ------------------------------------------------------------------ route ---
ROUTE = [  # one workgroup: 16 lanes a token, then a wave a token
    (1, 1, 1), (1, 8, 2), (3, 16, 16), (256, 16, 16), (5, 17, 4), (61, 128, 8), (64, 64, 6),
    (33, 256, 8), (7, 512, 16), (2, 300, 3),
    # blocks of tokens: both lane layouts, uneven last blocks
    (257, 8, 2), (65, 64, 6), (1000, 128, 8), (130, 512, 16), (4099, 9, 3), (17000, 8, 2)]


def route_logits(T, E, dt, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)).astype(np.float32)
    x = np.round(x * 8) / 8 if seed % 2 else x  # ties
    x[rng.random((T, E)) < 0.05] = -np.inf
    if T > 2:
        x[1] = -np.inf            # no expert is available
        x[T - 1] = np.nan
        x[2, E // 2] = np.inf
        x[0] = np.where(np.arange(E) % 2, 0.0, -0.0)
    if T > 16:
        x[3] = np.inf             # all infinite: equal shares
        x[4, 0] = np.nan
        x[5] = -np.inf
        x[5, E - 1] = -3.0
        x[6] = 3e38 if dt != "f16" else 65504.0
        x[7] = np.linspace(-200, 0, E)  # weights down to underflow
    return torch.from_numpy(x).to(TYPES[dt])


@pytest.mark.parametrize("dt,renorm", [("f32", True), ("f16", False), ("bf16", True)])
@pytest.mark.parametrize("T,E,k", ROUTE)
def test_route(T, E, k, dt, renorm):
    say(f"route T={T} E={E} k={k} {dt}")
    x = route_logits(T, E, dt, T + E + k)
    out = {"ids": poison((T, k), torch.int32), "weights": poison((T, k), torch.float32),
           "offsets": poison(E + 1, torch.int32), "rows": poison(T * k, torch.int32)}
    w4.route(x.to(DEV), k, renormalize=renorm, out=out)
    ids, w, tol, offsets, rows = ref.route(x.to(torch.float64).numpy(), k, renorm)
    np.testing.assert_array_equal(host(out["ids"]), ids)
    np.testing.assert_array_equal(host(out["offsets"]), offsets)
    np.testing.assert_array_equal(host(out["rows"]), rows)
    within(f64(out["weights"]), w, tol)


@pytest.mark.parametrize("T,E,dt", [(5, 7, "bf16"), (100, 33, "f16"), (9, 5, "f32")])
def test_route_part_of_a_batch(T, E, dt):
    """Rows of a larger batch: logits aligned to an element only."""
    x = route_logits(T + 1, E, dt, 77)
    out = w4.route(x.to(DEV)[1:], 3)
    ids, w, tol, offsets, rows = ref.route(x[1:].to(torch.float64).numpy(), 3, True)
    np.testing.assert_array_equal(host(out["ids"]), ids)
    np.testing.assert_array_equal(host(out["rows"]), rows)
    np.testing.assert_array_equal(host(out["offsets"]), offsets)
    within(f64(out["weights"]), w, tol)


def test_route_no_tokens():
    out = w4.route(torch.empty((0, 8), device=DEV), 2)
    assert host(out["offsets"]).tolist() == [0] * 9
    assert out["ids"].shape == (0, 2) and out["rows"].numel() == 0


def test_route_refusals():
    x = torch.zeros((4, 8), device=DEV)
    for k in (0, 9, 2.0):
        with pytest.raises(ValueError):
            w4.route(x, k)
    with pytest.raises(ValueError, match="contiguous"):
        w4.route(torch.zeros((8, 4), device=DEV).t(), 2)
    with pytest.raises(ValueError, match="2-D"):
        w4.route(torch.zeros(8, device=DEV), 2)
    out = w4.route(x, 2)
    with pytest.raises(ValueError, match="ids"):
        w4.route(x, 3, out=out)
    with pytest.raises(TypeError, match="weights"):
        w4.route(x, 2, out=dict(out, weights=out["weights"].half()))
    with pytest.raises(w4.W4A8Error) as e:  # a workspace too small
        w4.route(torch.zeros((1000, 64), device=DEV), 6,
                 workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4


# -------------------------------------------------------------------- moe ---

def experts(E, N, K, g, seed):
    """Packed experts on the device and their decoded int8 weights."""
    Ws = np.stack([wl.gen_weights(N, K, seed + e) for e in range(E)])
    p = w4.pack_experts(torch.from_numpy(Ws).to(DEV), group=g)
    wq, s, a = (host(p[n]).reshape(E, -1) for n in ("wq", "s_u8", "a_u8"))
    W = np.stack([ref.decode_weights(wq[e], s[e], a[e], N, K, g) for e in range(E)])
    return p, W, host(p["sw"]).reshape(E, N)


def tokens(T, H, dt, seed):
    """Values of the type, and the same as float32."""
    x = torch.from_numpy(wl.gen_activations(T, H, seed, seed + 1)).to(TYPES[dt])
    return x.to(DEV), x.to(torch.float32).numpy()


MOE = [
    (1, 4, 2, 256, 384, 64, "f16"),
    (1, 1, 1, 128, 128, 128, "f32"),      # one K-tile in each product
    (2, 3, 3, 128, 640, 64, "bf16"),
    (5, 8, 2, 512, 256, 128, "bf16"),
    (16, 8, 2, 384, 896, 128, "f16"),
    (7, 64, 6, 256, 128, 64, "f16"),
    (17, 2, 1, 256, 384, 128, "bf16"),    # up to 17 rows of one expert
    (33, 2, 2, 640, 256, 64, "f16"),      # 33 rows of each
    (70, 3, 2, 256, 384, 128, "bf16"),
    (130, 2, 2, 384, 256, 64, "f16"),     # 130 rows of each
    (256, 512, 16, 128, 128, 128, "f16"),  # the most experts, choices and tokens
    # one token in two launches: the most choices, and rows that fill the LDS
    (1, 512, 16, 256, 256, 64, "bf16"),
    (1, 16, 8, 128, 16384, 128, "f16"),
    (1, 16, 9, 128, 16384, 128, "f16"),   # one more does not fit
    # up to 64 slots, rows quantised by the products' workgroups
    (2, 8, 2, 4096, 512, 128, "f32"),
    (8, 8, 8, 128, 256, 64, "f16"),
    (4, 2, 2, 1024, 8192, 128, "bf16"),
    (64, 64, 1, 256, 128, 64, "f16"),
    (65, 64, 1, 256, 128, 64, "f16"),     # 65 slots: prepared rows
]


@pytest.mark.parametrize("T,E,k,H,F,g,dt", MOE)
def test_moe(T, E, k, H, F, g, dt):
    say(f"moe T={T} E={E} k={k} H={H} F={F} g={g} {dt}")
    rng = np.random.default_rng(T * E + k)
    w13, W13, sw13 = experts(E, 2 * F, H, g, 3000)
    w2, W2, sw2 = experts(E, H, F, g, 4000)
    X, Xf = tokens(T, H, dt, 50 + T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    Y = poison((T, H), TYPES[dt])
    w4.moe(X, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), w13, w2, out=Y)
    want, tol = ref.moe(Xf, ids, w, W13, sw13, W2, sw2, dt)
    within(f64(Y), want, tol)


def test_moe_odd_ids_and_rows():
    """Ids outside the experts, the same expert twice, zero weights, tokens
    without an expert, an all-zero token, and tokens with NaN or infinity
    (their rows are NaN, the others unaffected); float32 out of fp16 in."""
    T, E, k, H, F, g = 24, 4, 3, 256, 384, 64
    rng = np.random.default_rng(5)
    w13, W13, sw13 = experts(E, 2 * F, H, g, 3100)
    w2, W2, sw2 = experts(E, H, F, g, 4100)
    X, _ = tokens(T, H, "f16", 60)
    X[3] = 0
    X[4, 7] = float("nan")
    X[5, 8] = float("inf")
    Xf = X.float().cpu().numpy()
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[0] = -1
    ids[1] = [E, 2, 1 << 30]
    ids[2] = [1, 1, 1]
    ids[6] = [-(1 << 31), 3, 3]
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[7] = 0.0
    w[8, 1] = 0.0
    Y = poison((T, H), torch.float32)
    w4.moe(X, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), w13, w2, out=Y)
    want, tol = ref.moe(Xf, ids, w, W13, sw13, W2, sw2, "f32")
    got = f64(Y)
    assert (got[0] == 0).all() and (got[7] == 0).all() and (got[3] == 0).all()
    assert np.isnan(got[4]).all() and np.isnan(got[5]).all()
    within(got, want, tol)
    # every slot without an expert
    none = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w4.moe(X, none, torch.from_numpy(w).to(DEV), w13, w2, out=Y)
    assert (f64(Y) == 0).all()


@pytest.mark.parametrize("T,k", [(1, 6), (1, 16), (5, 4), (8, 8), (16, 4), (100, 3)])
def test_moe_odd_ids_at_every_form(T, k):
    """One token, few slots, many: ids outside the experts, an expert many
    times over (more rows than a stream serves at once), zero and negative
    weights, tokens that are not finite, calls without any expert."""
    E, H, F, g = 12, 256, 384, 64
    rng = np.random.default_rng(40 + T + k)
    w13, W13, sw13 = experts(E, 2 * F, H, g, 3500)
    w2, W2, sw2 = experts(E, H, F, g, 4500)
    cases = [np.full((T, k), 7), rng.integers(-2, E + 2, (T, k)), np.full((T, k), -1),
             rng.integers(0, 2, (T, k)) * 9, np.where(rng.random((T, k)) < 0.7, 3, 1 << 30)]
    for i, ids in enumerate(cases):
        say(f"moe ids T={T} k={k} case {i}")
        ids = ids.astype(np.int32)
        X, _ = tokens(T, H, "bf16", 60 + i)
        if i == 3:
            X[T - 1, 5] = float("inf")
        if i == 4:
            X[0, 9] = float("nan")
        w = rng.standard_normal((T, k)).astype(np.float32)
        w[:, k // 2] = 0.0
        Y = poison((T, H), torch.float16)
        w4.moe(X, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), w13, w2, out=Y)
        want, tol = ref.moe(X.float().cpu().numpy(), ids, w, W13, sw13, W2, sw2, "f16")
        within(f64(Y), want, tol)


def test_moe_same_as_its_steps():
    """Routing, the layer and the same layer step by step through the grouped
    GEMM (fp16 between the steps), as a decode step runs them."""
    T, E, k, H, F, g = 12, 8, 2, 512, 640, 128
    w13, W13, sw13 = experts(E, 2 * F, H, g, 3200)
    w2, W2, sw2 = experts(E, H, F, g, 4200)
    X, Xf = tokens(T, H, "f16", 70)
    logits = torch.from_numpy(np.random.default_rng(9).standard_normal((T, E)).astype(np.float32))
    r = w4.route(logits.to(DEV), k)
    Y = w4.moe(X, r["ids"], r["weights"], w13, w2)
    want, tol = ref.moe(Xf, host(r["ids"]), host(r["weights"]), W13, sw13, W2, sw2, "f16")
    within(f64(Y), want, tol)
    rows = r["rows"].long()
    Xq, sx = w4.quant_act(X[rows // k].contiguous())
    gu = w4.gemm_grouped(Xq, sx, r["offsets"], w13, T).float()
    h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
    hq, sh = w4.quant_act(h.contiguous())
    y = w4.gemm_grouped(hq, sh, r["offsets"], w2, T).float()
    steps = torch.zeros((T, H), device=DEV)
    steps.index_add_(0, rows // k, y * r["weights"].view(-1)[rows][:, None])
    err = (Y.float() - steps).norm() / steps.norm()
    # fp16 rounds g, u and y once more (2^-11 each at most) and may move a
    # code of h by one step: far less than the codes' own 1 / 254
    assert err < 1 / 254, err


def test_moe_experts_past_4_gib():
    """The last of many experts: its weights lie more than 2^32 bytes into
    the packed array."""
    E, H, F, g = 400, 2048, 12288 // 2, 128
    w13 = {"N": 2 * F, "K": H, "group": g, "E": E}
    w2 = {"N": H, "K": F, "group": g, "E": E}
    one13, W13, sw13 = experts(1, 2 * F, H, g, 3300)
    one2, W2, sw2 = experts(1, H, F, g, 4300)
    for w, one in ((w13, one13), (w2, one2)):
        for n in ("wq", "s_u8", "a_u8", "sw"):
            full = torch.zeros(E * one[n].numel(), dtype=one[n].dtype, device=DEV)
            full[-one[n].numel():] = one[n]
            w[n] = full
    assert w13["wq"].numel() > 1 << 32
    X, Xf = tokens(3, H, "bf16", 80)
    ids = np.full((3, 2), E - 1, np.int32)
    ids[:, 1] = -1
    w = np.ones((3, 2), np.float32)
    Y = w4.moe(X, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), w13, w2)
    ids[:, 0] = 0
    want, tol = ref.moe(Xf, ids, w, W13, sw13, W2, sw2, "bf16")
    within(f64(Y), want, tol)


def test_moe_refusals():
    w13, _, _ = experts(2, 512, 256, 64, 3400)
    w2, _, _ = experts(2, 256, 256, 64, 4400)
    X = torch.zeros((4, 256), dtype=torch.float16, device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    w = torch.ones((4, 2), device=DEV)
    assert w4.moe(X, ids, w, w13, w2).shape == (4, 256)
    assert w4.moe(X[:0], ids[:0], w[:0], w13, w2).shape == (0, 256)
    for bad in (dict(X=X[:, :128]), dict(X=X.t()), dict(ids=ids[:3]), dict(ids=ids[0]),
                dict(w=w[:, :1]), dict(w2=dict(w2, E=1)), dict(w13=dict(w13, N=256)),
                dict(w2=dict(w2, wq=w2["wq"][:-16])), dict(ids=ids.cpu())):
        a = dict(X=X, ids=ids, w=w, w13=w13, w2=w2)
        a.update(bad)
        with pytest.raises(ValueError):
            w4.moe(a["X"], a["ids"], a["w"], a["w13"], a["w2"])
    with pytest.raises(TypeError):
        w4.moe(X, ids.long(), w, w13, w2)
    with pytest.raises(TypeError):
        w4.moe(X, ids, w.half(), w13, w2)
    with pytest.raises(w4.W4A8Error) as e:  # too many tokens
        w4.moe(X[:1].expand(257, 256).contiguous(), ids[:1].expand(257, 2).contiguous(),
               w[:1].expand(257, 2).contiguous(), w13, w2)
    assert e.value.status == 2


# ------------------------------------------------------------------- lora ---

def lora_case(M, N, K, R, n, g, dt, pattern, seed):
    rng = np.random.default_rng(seed)
    p, W, sw = experts(1, N, K, g, 5000 + seed)
    X, Xf = tokens(M, K, dt, 90 + seed)
    A = torch.from_numpy(rng.standard_normal((n, R, K)).astype(np.float32) * 0.02).to(TYPES[dt])
    B = torch.from_numpy(rng.standard_normal((n, N, R)).astype(np.float32) * 0.05).to(TYPES[dt])
    scale = (0.5 + rng.random(n)).astype(np.float32)
    if pattern == "runs":
        ad = np.sort(rng.integers(-1, n, M))
    elif pattern == "one":
        ad = np.full(M, n - 1)
    elif pattern == "none":
        ad = np.full(M, -1)
    else:  # any, and values that name no adapter
        ad = rng.integers(-2, n + 2, M)
        ad[rng.random(M) < 0.1] = 1 << 30
    ad = ad.astype(np.int32)
    lora = {"A": A.to(DEV), "B": B.to(DEV), "scale": torch.from_numpy(scale).to(DEV)}
    want, tol = ref.gemm_lora(Xf, W[0], sw[0], A.float().numpy(), B.float().numpy(), scale, ad)
    return X, p, lora, torch.from_numpy(ad).to(DEV), want, tol


LORA = [
    (1, 64, 128, 8, 1, 64, "bf16", "one"),
    (1, 1024, 2048, 16, 8, 64, "f16", "any"),
    (16, 512, 1024, 16, 40, 128, "f16", "any"),     # every row its own adapter
    (16, 512, 1024, 24, 3, 64, "bf16", "none"),
    (17, 320, 896, 40, 5, 128, "bf16", "any"),
    (47, 704, 640, 64, 5, 64, "bf16", "any"),
    (63, 256, 512, 128, 4, 128, "f16", "any"),
    (64, 256, 512, 8, 4, 64, "f16", "any"),         # tile kernels from here on
    (100, 192, 512, 16, 4, 64, "bf16", "any"),      # N not a multiple of 256
    (128, 512, 4096, 16, 7, 128, "bf16", "any"),    # K split
    (129, 512, 1024, 32, 3, 64, "f16", "runs"),
    (300, 768, 1280, 128, 9, 128, "bf16", "runs"),
    (300, 768, 1280, 48, 30, 64, "f16", "any"),
    (1037, 1280, 640, 16, 5, 64, "bf16", "runs"),
    (520, 256, 16384, 16, 3, 128, "f16", "runs"),   # long K
    (2100, 4096, 512, 32, 3, 128, "bf16", "runs"),
    # rows longer than the quantising kernels hold in registers; group
    # parameters that do not fit in the streamed kernel's LDS
    (5, 64, 33024, 8, 2, 64, "f16", "any"),
    (513, 64, 16640, 24, 3, 128, "bf16", "any"),
    (512, 256, 2048, 96, 6, 64, "f16", "any"),
]


@pytest.mark.parametrize("M,N,K,R,n,g,dt,pattern", LORA)
def test_gemm_lora(M, N, K, R, n, g, dt, pattern):
    say(f"lora M={M} N={N} K={K} R={R} n={n} {dt} {pattern}")
    X, p, lora, ad, want, tol = lora_case(M, N, K, R, n, g, dt, pattern, M + R)
    Y = poison((M, N), torch.float16)
    w4.gemm_lora(X, p, lora, ad, out=Y)
    within(f64(Y), want, tol)


@pytest.mark.parametrize("M", [5, 150])
def test_gemm_lora_without_adapters(M):
    """No adapters at all, and no row with one: the shared projection's bits."""
    X, p, lora, ad, _, _ = lora_case(M, 512, 1024, 16, 3, 64, "f16", "none", 7)
    Xq, sx = w4.quant_act(X)
    want = w4.gemm(Xq, sx, p)
    assert torch.equal(w4.gemm_lora(X, p, lora, ad), want)
    empty = {"A": lora["A"][:0], "B": lora["B"][:0], "scale": lora["scale"][:0]}
    assert torch.equal(w4.gemm_lora(X, p, empty, ad + 1), want)


@pytest.mark.parametrize("M", [9, 200])
def test_gemm_lora_extreme_values(M):
    """Large and tiny adapter values: the inner product may lie far outside
    fp16's range while the result does not; rows of zeros; a row that
    overflows fp16 becomes an infinity of the right sign."""
    X, p, lora, ad, _, _ = lora_case(M, 256, 512, 16, 3, 64, "f16", "any", 11)
    X[0] = 0
    ad[0] = 1
    ad[1], ad[2], ad[3], ad[4] = 0, 1, 2, 2
    lora["A"][0] *= 2.0 ** 20      # up to about 2^18 per element sum ...
    lora["A"][0].clamp_(-60000, 60000)
    lora["B"][0] *= 2.0 ** -20     # ... against fp16 subnormals
    lora["A"][1] *= 2.0 ** -12
    lora["B"][1] *= 2.0 ** 12
    lora["scale"][2] = 3e6         # beyond fp16
    W = ref.decode_weights(host(p["wq"]), host(p["s_u8"]), host(p["a_u8"]), 256, 512, 64)
    want, tol = ref.gemm_lora(X.float().cpu().numpy(), W, host(p["sw"]),
                              lora["A"].float().cpu().numpy(), lora["B"].float().cpu().numpy(),
                              host(lora["scale"]), host(ad))
    got = f64(w4.gemm_lora(X, p, lora, ad))
    # at and beyond the overflow border (65520) both are infinite, of one sign
    big = np.abs(want) > 65520 + tol
    assert np.isinf(got[big]).all() and (np.sign(got[big]) == np.sign(want[big])).all()
    sure = np.abs(want) < 65504 - tol
    within(got[sure], want[sure], tol[sure])


@pytest.mark.parametrize("M,N", [(7, 512), (40, 512), (200, 512), (128, 256)])
def test_gemm_lora_alignment(M, N):
    """Vectors need 4-byte boundaries only: channel scales, adapter scales
    and ids one element into their storage."""
    X, p, lora, ad, want, tol = lora_case(M, N, 4096, 24, 5, 64, "f16", "any", 17)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        s.copy_(t)
        return s
    got = w4.gemm_lora(X, dict(p, sw=shifted(p["sw"])), dict(lora, scale=shifted(lora["scale"])),
                       shifted(ad))
    within(f64(got), want, tol)


@pytest.mark.parametrize("M", [16, 40, 300])
def test_gemm_lora_rows_do_not_mix(M):
    """An adapter with infinities and NaN, and rows that are not finite, leave
    the rows of other adapters (in the same blocks) alone."""
    X, p, lora, ad, _, _ = lora_case(M, 512, 512, 16, 4, 64, "bf16", "any", 19)
    ad.copy_(torch.arange(M, device=DEV, dtype=torch.int32) % 5 - 1)
    good = w4.gemm_lora(X, p, lora, ad)
    assert torch.isfinite(good).all()
    lora["A"][2, 3, 7] = float("inf")
    lora["B"][2, 9] = float("nan")
    lora["B"][1, 11, 2] = float("inf")
    X[5] = float("nan")
    bad = w4.gemm_lora(X, p, lora, ad)
    ok = (ad != 2) & (ad != 1)
    ok[5] = False
    assert torch.equal(bad[ok], good[ok])
    assert not torch.isfinite(bad[ad == 1][:, 11]).any()
    assert not torch.isfinite(bad[ad == 2]).all(dim=1).any()


def test_gemm_lora_adapters_past_4_gib():
    """The last of many adapters, whose values lie past 2^32 bytes."""
    n, R, K, N, M = 600, 128, 32768, 64, 3
    rng = np.random.default_rng(3)
    p, W, sw = experts(1, N, K, 128, 5600)
    X, Xf = tokens(M, K, "bf16", 95)
    A = torch.zeros((n, R, K), dtype=torch.bfloat16, device=DEV)
    assert A.numel() * 2 > 1 << 32
    B = torch.zeros((n, N, R), dtype=torch.bfloat16, device=DEV)
    A1 = torch.from_numpy(rng.standard_normal((R, K)).astype(np.float32) * 0.02).bfloat16()
    B1 = torch.from_numpy(rng.standard_normal((N, R)).astype(np.float32) * 0.05).bfloat16()
    A[-1], B[-1] = A1.to(DEV), B1.to(DEV)
    scale = np.ones(n, np.float32)
    ad = np.array([n - 1, 0, n - 1], np.int32)
    got = w4.gemm_lora(X, p, {"A": A, "B": B, "scale": torch.from_numpy(scale).to(DEV)},
                       torch.from_numpy(ad).to(DEV))
    one = np.where(ad == n - 1, 0, -1)
    want, tol = ref.gemm_lora(Xf, W[0], sw[0], A1.float().numpy()[None],
                              B1.float().numpy()[None], scale[:1], one)
    within(f64(got), want, tol)


def test_gemm_lora_refusals():
    X, p, lora, ad, _, _ = lora_case(8, 128, 256, 16, 3, 64, "f16", "any", 13)
    assert w4.gemm_lora(X[:0], p, lora, ad[:0]).shape == (0, 128)
    for bad in (dict(X=X[:, :128]), dict(ad=ad[:4]), dict(ad=ad.cpu()), dict(X=X.t()),
                dict(lora=dict(lora, A=lora["A"][:, :8])),
                dict(lora=dict(lora, B=lora["B"][:2])),
                dict(lora=dict(lora, scale=lora["scale"][:2])),
                dict(p=dict(p, wq=p["wq"][16:]))):
        a = dict(X=X, p=p, lora=lora, ad=ad)
        a.update(bad)
        with pytest.raises(ValueError):
            w4.gemm_lora(a["X"], a["p"], a["lora"], a["ad"])
    with pytest.raises(TypeError):
        w4.gemm_lora(X.bfloat16(), p, lora, ad)
    with pytest.raises(TypeError):
        w4.gemm_lora(X, p, lora, ad.long())
    odd = {"A": lora["A"][:, :12].contiguous(), "B": lora["B"][:, :, :12].contiguous(),
           "scale": lora["scale"]}
    with pytest.raises(w4.W4A8Error) as e:  # a rank that is no multiple of 8
        w4.gemm_lora(X, p, odd, ad)
    assert e.value.status == 2


# ------------------------------------------------- a decode step as served ---

class Step:
    """Route, expert layer and an adapter projection of its output, with
    every buffer given, as a serving loop captures it."""

    def __init__(self, T=9, E=8, k=2, H=512, F=384, g=128, seed=1):
        self.k = k
        self.w13, self.W13, self.sw13 = experts(E, 2 * F, H, g, 6000 + seed)
        self.w2, self.W2, self.sw2 = experts(E, H, F, g, 7000 + seed)
        (self.Xl, self.p, self.lora, self.ad, self.want_l, self.tol_l) = lora_case(
            T, 320, H, 16, 4, 64, "f16", "any", 20 + seed)
        rng = np.random.default_rng(seed)
        self.X, self.Xf = tokens(T, H, "f16", 30 + seed)
        self.logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
        self.r = {"ids": poison((T, k), torch.int32), "weights": poison((T, k), torch.float32),
                  "offsets": poison(E + 1, torch.int32), "rows": poison(T * k, torch.int32)}
        self.Y = poison((T, H), torch.float16)
        self.Z = poison((T, 320), torch.float16)
        self.ws = torch.empty(max(w4.moe_workspace_size(T, E, k, H, F),
                                  w4.gemm_lora_workspace_size(T, 320, H, 16)),
                              dtype=torch.uint8, device=DEV)

    def __call__(self, stream=None):
        w4.route(self.logits, self.k, out=self.r, stream=stream)
        w4.moe(self.X, self.r["ids"], self.r["weights"], self.w13, self.w2, out=self.Y,
               workspace=self.ws, stream=stream)
        w4.gemm_lora(self.Y, self.p, self.lora, self.ad, out=self.Z, workspace=self.ws,
                     stream=stream)

    def outs(self):
        return list(self.r.values()) + [self.Y, self.Z]

    def blank(self, byte):
        for o in self.outs():
            o.view(torch.uint8).fill_(byte)
        self.ws.fill_(byte)

    def check(self):
        ids, w, tol, offsets, rows = ref.route(f64(self.logits), self.k, True)
        np.testing.assert_array_equal(host(self.r["ids"]), ids)
        np.testing.assert_array_equal(host(self.r["rows"]), rows)
        want, tol = ref.moe(self.Xf, ids, host(self.r["weights"]), self.W13, self.sw13, self.W2,
                            self.sw2, "f16")
        within(f64(self.Y), want, tol)
        W = ref.decode_weights(host(self.p["wq"]), host(self.p["s_u8"]), host(self.p["a_u8"]),
                               320, self.X.shape[1], 64)
        want, tol = ref.gemm_lora(self.Y.float().cpu().numpy(), W, host(self.p["sw"]),
                                  self.lora["A"].float().cpu().numpy(),
                                  self.lora["B"].float().cpu().numpy(),
                                  host(self.lora["scale"]), host(self.ad))
        within(f64(self.Z), want, tol)


def test_step_eager_and_repeatable():
    s = Step()
    s()
    s.check()
    first = [o.clone() for o in s.outs()]
    for byte in (0, 0x7F, 0xFF):  # whatever the workspace held before
        s.blank(byte)
        s()
        torch.cuda.synchronize()
        for a, b in zip(s.outs(), first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_step_captured_follows_its_inputs():
    """A captured step replayed with new logits, ids and adapters gives what
    an eager call gives on them."""
    s = Step(seed=2)
    s()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s()
    for rep in range(4):
        s.blank(0xA5 + rep)
        s.logits.copy_(torch.randn(s.logits.shape, generator=torch.Generator().manual_seed(rep)))
        s.ad.copy_(torch.roll(s.ad, rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in s.outs()]
        s.check()
        s.blank(0x11)
        s()
        torch.cuda.synchronize()
        for a, b in zip(got, s.outs()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


def test_steps_on_two_streams():
    """Two steps with workspaces of their own, enqueued on two streams at
    once, give their serial results; the stream argument selects the stream."""
    steps = [Step(seed=3), Step(T=16, seed=4)]
    for s in steps:
        s()
    torch.cuda.synchronize()
    want = [[o.clone() for o in s.outs()] for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for s in steps:
            s.blank(0x33 + rep)
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            s(stream=st)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for a, b in zip(s.outs(), w):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_allocated_outputs_belong_to_the_stream():
    """Without out and workspace the call's tensors come from its stream."""
    s = Step(seed=5)
    s()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r = w4.route(s.logits, s.k, stream=st)
    Y = w4.moe(s.X, r["ids"], r["weights"], s.w13, s.w2, stream=st)
    Z = w4.gemm_lora(Y, s.p, s.lora, s.ad, stream=st)
    st.synchronize()
    assert torch.equal(Y, s.Y) and torch.equal(Z, s.Z)
