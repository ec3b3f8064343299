"""Workloads of the operators whose rows choose their own weights.

Three operators of a served model layer on W4A8 weights:

* ``route``      top-k gating of router logits and the grouping of the chosen
                 (token, expert) slots by expert;
* ``moe``        a whole mixture-of-experts layer for a few tokens: gate and up
                 products, SiLU, down product and the weighted sum;
* ``gemm_lora``  a shared W4A8 projection plus the low-rank adapter that each
                 row selects.

``run`` computes them in elementary torch operations, or, with ``own`` set, by
the package's kernels.  Packed weights are held in the library's documented
layout in both cases; the plain form unpacks them within the call.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the gate of one decoded token of an 8-expert model
        dict(name="route_token", op="route", T=1, E=8, k=2, dtype="f32", renorm=True),
        # a decode batch through a layer of many small experts
        dict(name="route_batch", op="route", T=61, E=128, k=8, dtype="bf16", renorm=True),
        # a prefill chunk, for the grouped GEMM
        dict(name="route_prefill", op="route", T=8192, E=64, k=6, dtype="f32", renorm=False),
        # one token through an 8-expert layer (14336 x 4096 experts)
        dict(name="moe_token", op="moe", T=1, E=8, k=2, H=4096, F=14336, group=128,
             dtype="f16"),
        # sixteen requests decoding: every expert is chosen by some
        dict(name="moe_decode", op="moe", T=16, E=8, k=2, H=4096, F=14336, group=128,
             dtype="bf16"),
        # seven tokens over many small experts of an odd width
        dict(name="moe_small_experts", op="moe", T=7, E=64, k=6, H=2048, F=1408, group=64,
             dtype="f16"),
        # a large decode batch, more than one block of rows for most experts
        dict(name="moe_batch", op="moe", T=131, E=16, k=2, H=4096, F=6400, group=128,
             dtype="bf16"),
        # one token through an attention projection, adapter of rank 16
        dict(name="lora_token", op="lora", M=1, N=4096, K=4096, R=16, n=8, group=64,
             dtype="bf16", runs=False),
        # sixteen requests, each with an adapter of its own choice
        dict(name="lora_decode", op="lora", M=16, N=28672, K=8192, R=16, n=32, group=128,
             dtype="f16", runs=False),
        # an odd batch of draft tokens, wide adapters
        dict(name="lora_batch", op="lora", M=47, N=11008, K=4096, R=64, n=5, group=64,
             dtype="bf16", runs=False),
        # prompts of a few requests packed into one chunk
        dict(name="lora_prefill", op="lora", M=2048, N=11008, K=4096, R=32, n=6, group=64,
             dtype="f16", runs=True),
        # a long prompt chunk through the largest projection
        dict(name="lora_long", op="lora", M=4096, N=28672, K=8192, R=16, n=4, group=128,
             dtype="bf16", runs=True),
    ]


def _logi(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "lora"])
    if op == "route":
        E = _logi(rng, 2, 256)
        return dict(op="route", T=_logi(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 8)),
                    dtype=rng.choice(["f32", "f16", "bf16"]), renorm=rng.random() < 0.5)
    if op == "moe":
        E = _logi(rng, 2, 64)
        H = 128 * _logi(rng, 4, 32)
        # experts of one layer hold at most what an 8-expert layer's do
        F = 128 * _logi(rng, 2, max(2, min(112, 8 * 112 * 32 // (E * (H // 128)))))
        return dict(op="moe", T=_logi(rng, 1, 256), E=E, k=rng.randint(1, min(E, 8)), H=H,
                    F=F, group=rng.choice([64, 128]), dtype=rng.choice(["f16", "bf16"]))
    return dict(op="lora", M=_logi(rng, 1, 4096), N=64 * _logi(rng, 8, 256),
                K=128 * _logi(rng, 4, 64), R=8 * _logi(rng, 1, 8), n=rng.randint(1, 32),
                group=rng.choice([64, 128]), dtype=rng.choice(["f16", "bf16"]),
                runs=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs ---

def _pack(W, group):
    """LiquidQuant codes of W [N][K] in the packed layout of include/w4a8.h:
    per-channel INT8, then per group a UINT4 code with an integer scale and
    offset."""
    N, K = W.shape
    sw = W.abs().amax(1) / 127.0
    sw = torch.where(sw > 0, sw, torch.ones_like(sw))
    Q = torch.clamp(torch.round(W / sw[:, None]), -127, 127).to(torch.int32)
    Q = Q.view(N, K // group, group)
    m = Q.amin(2, keepdim=True)
    s = torch.clamp((Q.amax(2, keepdim=True) - m + 14) // 15, min=1)
    q = torch.minimum((2 * (Q - m) + s) // (2 * s), (127 - m) // s)
    q = q.to(torch.uint8).view(N // 16, 16, K // 128, 4, 4, 2, 4)   # n, r, kt, G, d, half, b
    q = q.permute(0, 2, 3, 1, 4, 6, 5)                              # n, kt, G, r, d, b, half
    wq = (q[..., 0] | (q[..., 1] << 4)).reshape(-1).contiguous()

    def panels(p):  # [N][groups] -> panels of 64 channels, channel n at 4 (n % 16) + (n % 64) / 16
        return (p.to(torch.uint8).view(N // 64, 4, 16, K // group).permute(0, 3, 2, 1)
                .reshape(-1).contiguous())
    return wq, panels(s.squeeze(2)), panels((128 + m).squeeze(2)), sw


def _packed_experts(E, N, K, group, gen):
    """E packed matrices of weights ~ Normal(0, 0.02), laid end to end."""
    parts = [_pack(torch.randn(N, K, generator=gen, device=DEV) * 0.02, group)
             for _ in range(E)]
    out = {name: torch.cat([p[i] for p in parts])
           for i, name in enumerate(("wq", "s_u8", "a_u8", "sw"))}
    out.update(N=N, K=K, group=group, E=E)
    return out


def _activations(M, K, dtype, gen):
    """Normal(0, 1) with one channel in a hundred twenty times as large."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    big = torch.rand(K, generator=gen, device=DEV) < 0.01
    return (x * torch.where(big, 20.0, 1.0)).to(_TYPES[dtype])


def _logits(T, E, gen):
    """Router logits: some experts are more popular than others."""
    return (torch.randn(T, E, generator=gen, device=DEV)
            + 0.5 * torch.randn(E, generator=gen, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    if own:
        import w4a8_quantized_gemm_amd as w4
        st["w4"] = w4
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _logits(T, E, gen)
        # a few experts are switched off for some tokens
        x = torch.where(torch.rand(T, E, generator=gen, device=DEV) < 0.02, -math.inf, x)
        st["logits"] = x.to(_TYPES[case["dtype"]])
        if own:
            i32 = dict(dtype=torch.int32, device=DEV)
            st["out"] = {"ids": torch.empty((T, k), **i32),
                         "weights": torch.empty((T, k), dtype=torch.float32, device=DEV),
                         "offsets": torch.empty(E + 1, **i32),
                         "rows": torch.empty(T * k, **i32)}
            need = w4.route_workspace_size(T, E, k)
            st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    elif case["op"] == "moe":
        T, E, k, H, F, g = (case[x] for x in ("T", "E", "k", "H", "F", "group"))
        st["w13"] = _packed_experts(E, 2 * F, H, g, gen)
        st["w2"] = _packed_experts(E, H, F, g, gen)
        st["X"] = _activations(T, H, case["dtype"], gen)
        top, ids = torch.topk(_logits(T, E, gen), k, dim=1)
        st["ids"] = ids.to(torch.int32)
        st["weights"] = torch.softmax(top, dim=1)
        if own:
            st["out"] = torch.empty((T, H), dtype=_TYPES[case["dtype"]], device=DEV)
            st["workspace"] = torch.empty(w4.moe_workspace_size(T, E, k, H, F),
                                          dtype=torch.uint8, device=DEV)
    else:
        M, N, K, R, n = (case[x] for x in ("M", "N", "K", "R", "n"))
        dt = _TYPES[case["dtype"]]
        st["packed"] = _packed_experts(1, N, K, case["group"], gen)
        st["X"] = _activations(M, K, case["dtype"], gen)
        A = (torch.randn(n, R, K, generator=gen, device=DEV) * 0.02).to(dt)
        B = (torch.randn(n, N, R, generator=gen, device=DEV) * 0.02).to(dt)
        scale = 0.5 + 1.5 * torch.rand(n, generator=gen, device=DEV)
        st["lora"] = {"A": A, "B": B, "scale": scale}
        # -1: a request of the base model
        if case["runs"]:  # each request's rows lie together
            requests = torch.randint(-1, n, (max(1, M // 300) + 1,), generator=gen, device=DEV)
            ends = torch.rand(M, generator=gen, device=DEV) < 1.0 / 300
            idx = torch.clamp(torch.cumsum(ends, 0), max=len(requests) - 1)
            st["adapter"] = requests[idx].to(torch.int32)
        else:
            st["adapter"] = torch.randint(-1, n, (M,), generator=gen, device=DEV,
                                          dtype=torch.int32)
        if own:
            st["out"] = torch.empty((M, N), dtype=torch.float16, device=DEV)
            need = w4.gemm_lora_workspace_size(M, N, K, R)
            st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------- plain form ---

def _unpack(p, e=0):
    """Signed INT8 weights [N][K] of expert e, as float64 (their products and
    sums are then exact)."""
    N, K, g = p["N"], p["K"], p["group"]
    wq = p["wq"].view(-1, N * K // 2)[e].view(N // 16, K // 128, 4, 16, 4, 4)
    q = torch.stack([wq & 15, wq >> 4], -1)           # n, kt, G, r, d, b, half
    q = q.permute(0, 3, 1, 2, 4, 6, 5).reshape(N, K // g, g).to(torch.int16)

    def param(x):
        x = x.view(-1, N * K // g)[e].view(N // 64, K // g, 16, 4)
        return x.permute(0, 3, 2, 1).reshape(N, K // g, 1).to(torch.int16)
    return (q * param(p["s_u8"]) + param(p["a_u8"]) - 128).view(N, K).to(torch.float64)


def _quant(x):
    """Per-row INT8 codes (float64 values) and float32 scales of float32 x."""
    s = x.abs().amax(1) / 127.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return torch.clamp(torch.round(x / s[:, None]), -127, 127).to(torch.float64), s


def _scaled(acc, s, sw):
    return (acc.to(torch.float32) * s[:, None]) * sw


def _route_plain(st):
    x = st["logits"].to(torch.float32)
    T, E, k = st["T"], st["E"], st["k"]
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(1, keepdim=True)
    e = torch.where(x == top, 1.0, torch.exp(x - top))
    e = torch.where(x == -math.inf, 0.0, e)
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    chosen = torch.gather(e, 1, order)
    total = (chosen if st["renorm"] else e).sum(1, keepdim=True)
    weights = torch.where(total > 0, chosen / total, 0.0)
    ids = torch.where(torch.gather(x, 1, order) == -math.inf, -1, order)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    rows = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[rows], torch.arange(E + 1, device=DEV))
    rows = torch.where(key[rows] == E, -1, rows)
    return {"ids": ids.to(torch.int32), "weights": weights,
            "offsets": offsets.to(torch.int32), "rows": rows.to(torch.int32)}


def _moe_plain(st):
    w13, w2, ids = st["w13"], st["w2"], st["ids"]
    F = st["F"]
    Xq, sx = _quant(st["X"].to(torch.float32))
    Y = torch.zeros((st["T"], st["H"]), dtype=torch.float32, device=DEV)
    for e in range(st["E"]):
        share = torch.where(ids == e, st["weights"], 0.0).sum(1)
        gu = _scaled(Xq @ _unpack(w13, e).t(), sx, w13["sw"].view(-1, 2 * F)[e])
        g, u = gu[:, :F], gu[:, F:]
        hq, sh = _quant(g / (1.0 + torch.exp(-g)) * u)
        y = _scaled(hq @ _unpack(w2, e).t(), sh, w2["sw"].view(-1, st["H"])[e])
        Y += torch.where(share[:, None] != 0, share[:, None] * y, 0.0)
    return Y.to(st["X"].dtype)


def _lora_plain(st):
    p, lora, ids = st["packed"], st["lora"], st["adapter"]
    Xf = st["X"].to(torch.float32)
    Xq, sx = _quant(Xf)
    Y = _scaled(Xq @ _unpack(p).t(), sx, p["sw"])
    for a in range(st["n"]):
        V = (Xf @ lora["A"][a].to(torch.float32).t()) * lora["scale"][a]
        V = torch.where((ids == a)[:, None], V, 0.0)
        Y += V @ lora["B"][a].to(torch.float32).t()
    return Y.to(torch.float16)


def run(st):
    if not own:
        return {"route": _route_plain, "moe": _moe_plain, "lora": _lora_plain}[st["op"]](st)
    w4 = st["w4"]
    if st["op"] == "route":
        return w4.route(st["logits"], st["k"], renormalize=st["renorm"], out=st["out"],
                        workspace=st["workspace"])
    if st["op"] == "moe":
        return w4.moe(st["X"], st["ids"], st["weights"], st["w13"], st["w2"], out=st["out"],
                      workspace=st["workspace"])
    return w4.gemm_lora(st["X"], st["packed"], st["lora"], st["adapter"], out=st["out"],
                        workspace=st["workspace"])


# ------------------------------------------------------------------- work ---

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size + 12 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if case["op"] == "moe":
        T, E, k, H, F, g = (case[x] for x in ("T", "E", "k", "H", "F", "group"))
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens choose, on average
        weights = 3 * F * H // 2 + 2 * (3 * F * H // g) + 4 * (2 * F + H)
        return {"bytes": int(active * weights) + 2 * T * H * size + 8 * T * k,
                "flops": 6 * T * k * H * F}
    M, N, K, R, n, g = (case[x] for x in ("M", "N", "K", "R", "n", "group"))
    used = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** (max(1, M // 300) if case["runs"] else M))
    return {"bytes": N * K // 2 + 2 * (N * K // g) + 4 * N + M * K * size + 4 * M
            + int(used * R * (N + K) * size) + 2 * M * N,
            "flops": 2 * M * N * K + 2 * M * R * (N + K)}


# ------------------------------------------------------------------ exact ---

def _weights64(p, e):
    """Decoded weights times their channel scale, [N][K] float64, from the
    byte positions of the documented layout."""
    N, K, g = p["N"], p["K"], p["group"]
    n = torch.arange(N, device=DEV)[:, None]
    kk = torch.arange(K, device=DEV)[None, :]
    c = kk % 128
    pos = 1024 * ((n // 16) * (K // 128) + kk // 128) + 16 * (16 * (c // 32) + n % 16)
    pos = pos + 4 * (c % 32 // 8) + c % 4
    code = p["wq"][e * (N * K // 2):(e + 1) * (N * K // 2)][pos]
    del pos
    code = torch.where(c % 8 >= 4, code >> 4, code & 15).to(torch.float64)
    j = torch.arange(K // g, device=DEV)[None, :]
    at = e * (N * K // g) + 64 * ((n // 64) * (K // g) + j) + 4 * (n % 16) + n % 64 // 16
    code = code.view(N, K // g, g)
    code.mul_(p["s_u8"][at].to(torch.float64)[:, :, None])
    code.add_(p["a_u8"][at].to(torch.float64)[:, :, None] - 128.0)
    return code.view(N, K).mul_(p["sw"][e * N:(e + 1) * N].to(torch.float64)[:, None])


def _int8_64(x):
    """The values that per-row INT8 codes of x stand for.  The operators
    define scale and code by float32 arithmetic (whole numbers, so a quotient
    next to a half has to fall on the definition's side); the values are
    float64."""
    x32 = x.to(torch.float32)
    s = x32.abs().max(dim=1).values.div(127.0)
    s = s.masked_fill(s == 0, 1.0)[:, None]
    return x32.div(s).round().clamp(-127, 127).double() * s.double()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        x = st["logits"].double()
        on = x > -math.inf
        p = torch.exp(x - x.masked_fill(~on, -1e300).max(1, keepdim=True).values)
        p = p.masked_fill(~on, 0.0)
        # position of every expert in its token's order: how many come before it
        T, E, k = case["T"], case["E"], case["k"]
        rank = torch.zeros((T, E), dtype=torch.int64, device=DEV)
        col = torch.arange(E, device=DEV)
        for e in range(E):
            o = x[:, e:e + 1]
            rank += ((o > x) | ((o == x) & (e < col))).long()
        ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        weights = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        t, e = torch.nonzero((rank < k) & on, as_tuple=True)
        ids[t, rank[t, e]] = e.int()
        weights[t, rank[t, e]] = p[t, e]
        total = (weights if case["renorm"] else p).sum(1, keepdim=True)
        weights = weights / total.masked_fill(total == 0, 1.0)
        flat = ids.view(-1)
        groups = [torch.nonzero(flat == e).view(-1) for e in range(E)]
        rows = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        found = torch.cat(groups)
        rows[:len(found)] = found.int()
        offsets = torch.tensor([0] + [len(gr) for gr in groups], device=DEV).cumsum(0).int()
        return {"ids": ids, "weights": weights, "offsets": offsets, "rows": rows}
    if case["op"] == "moe":
        F = case["F"]
        X = _int8_64(st["X"].double())
        Y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
        for e in st["ids"].unique().tolist():
            t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            gu = X[t] @ _weights64(st["w13"], e).t()
            h = torch.sigmoid(gu[:, :F]) * gu[:, :F] * gu[:, F:]
            y = _int8_64(h) @ _weights64(st["w2"], e).t()
            Y.index_add_(0, t, y * st["weights"][t, j].double()[:, None])
        return Y
    Y = _int8_64(st["X"].double()) @ _weights64(st["packed"], 0).t()
    for a in st["adapter"].unique().tolist():
        if a >= 0:
            m = torch.nonzero(st["adapter"] == a).view(-1)
            V = st["X"][m].double() @ st["lora"]["A"][a].double().t()
            Y[m] += (V @ st["lora"]["B"][a].double().t()) * st["lora"]["scale"][a].double()
    return Y
