"""Workloads of the operators between and around a layer's projections.

Two operators of a served model layer on W4A8 weights:

* ``norm``  what lies between two projections: the block's output is normed,
            gated, scaled and added to the residual stream, and the sum is
            normed and quantised for the next projection;
* ``ffn``   a gated feed-forward block: gate and up products, activation,
            per-token INT8 of their product, down product.

``run`` computes them in elementary torch operations, or, with ``own`` set, by
the package's kernels.  The norms' integer codes are part of their definition
(every float32 operation is rounded by itself, the sums are taken in 64 bits),
so both sides return equal ones; e4m3 codes are returned as the float8 values
that they are.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}


# ------------------------------------------------------------------ cases ---

def _norm_case(name, M, K, x="bf16", y="f16", out="int8", kind="rms", post=False, gate="none",
               scale=1.0, pad=0):
    """x, y: types of the residual stream and of the block's output ("none":
    no block, the first norm of a model); post: the block's output is normed
    too; gate: "none", "row" (one for each token), "all" (one for the batch)
    or "ids" (each request's own); pad: rows of zeros behind the last token."""
    return dict(name=name, op="norm", M=M, K=K, x=x, y=y, out=out, kind=kind, post=post, gate=gate,
                scale=scale, pad=pad)


def _ffn_case(name, M, H, F, group=128, act="silu", dtype="f16"):
    return dict(name=name, op="ffn", M=M, H=H, F=F, group=group, act=act, dtype=dtype)


def listed():
    return [
        # one decoded token in front of its first attention projection
        _norm_case("norm_token", 1, 4096, y="none"),
        # sixteen requests decoding, residual sum and norm in front of the FFN
        _norm_case("norm_decode", 16, 8192, x="f16"),
        # an odd padded batch with layer norms, float32 stream, FP8 projections
        _norm_case("norm_odd", 61, 2064, x="f32", y="bf16", out="e4m3", kind="layer", pad=5),
        # norms before and after the block, gate of each request, rows for adapters
        _norm_case("norm_requests", 1000, 5120, y="bf16", out="bf16", post=True, gate="ids",
                   scale=0.22),
        # a prompt chunk, sandwich norms and a gate for every token
        _norm_case("norm_gated", 2048, 4096, post=True, gate="row"),
        # a long prompt chunk between the largest projections
        _norm_case("norm_long", 8192, 8192),
        # one decoded token of a 7B-sized layer
        _ffn_case("ffn_token", 1, 4096, 11008, group=64),
        # sixteen requests decoding in a 70B-sized layer
        _ffn_case("ffn_decode", 16, 8192, 28672, dtype="bf16"),
        # an odd batch of draft tokens
        _ffn_case("ffn_batch", 47, 4096, 11008, dtype="bf16"),
        # a small shared block beside a layer's experts, an odd width, GELU
        _ffn_case("ffn_small", 133, 2048, 1408, group=64, act="gelu"),
        # prompts of a few requests packed into one chunk
        _ffn_case("ffn_prefill", 2048, 4096, 11008, group=64),
        # a long prompt chunk through a 70B-sized layer
        _ffn_case("ffn_long", 4096, 8192, 28672, dtype="bf16"),
    ]


def _logi(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        K = 16 * _logi(rng, 16, 1792)
        M = _logi(rng, 1, min(8192, 8192 * 8192 // K))
        y = rng.choice(["none", "f32", "f16", "bf16"])
        case = _norm_case("", M, K, x=rng.choice(["f32", "f16", "bf16"]), y=y,
                          out=rng.choice(["int8", "int8", "e4m3", "f16", "bf16"]),
                          kind=rng.choice(["rms", "layer"]),
                          post=y != "none" and rng.random() < 0.5,
                          gate="none" if y == "none" else rng.choice(["none", "row", "all", "ids"]),
                          scale=rng.choice([1.0, 0.22, 0.5]), pad=rng.choice([0, 0, M // 8]))
    else:
        case = _ffn_case("", _logi(rng, 1, 4096), 128 * _logi(rng, 4, 64), 128 * _logi(rng, 4, 224),
                         group=rng.choice([64, 128]), act=rng.choice(["silu", "gelu"]),
                         dtype=rng.choice(["f16", "bf16"]))
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs ---

def _pack(W, group):
    """LiquidQuant codes of W [N][K] in the packed layout of include/w4a8.h:
    per-channel INT8, then per group a UINT4 code with an integer scale and
    offset."""
    N, K = W.shape
    sw = W.abs().amax(1) / 127.0
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
    return {"wq": wq, "s_u8": panels(s.squeeze(2)), "a_u8": panels((128 + m).squeeze(2)), "sw": sw,
            "N": N, "K": K, "group": group}


def _stream_rows(M, K, dtype, pad, gen):
    """A residual stream: Normal(0, 1), one channel in a hundred twenty times
    as large, rows of zeros at the end."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    big = torch.rand(K, generator=gen, device=DEV) < 0.01
    x = x * torch.where(big, 20.0, 1.0)
    x[M - pad:] = 0.0
    return x.to(_TYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    M = case["M"]
    if own:
        import w4a8_quantized_gemm_amd as w4
        st["w4"] = w4
    if case["op"] == "norm":
        K, pad = case["K"], case["pad"]

        def vector(mean, spread):
            return mean + spread * torch.randn(K, generator=gen, device=DEV)
        layer = case["kind"] == "layer"
        st["eps"] = 1e-5
        st["x"] = _stream_rows(M, K, case["x"], pad, gen)
        st["weight"] = vector(1.0, 0.2)
        st["bias"] = vector(0.0, 0.1) if layer else None
        for name in ("y", "y_weight", "y_bias", "gate", "gate_ids"):
            st[name] = None
        if case["y"] != "none":
            dt = _TYPES[case["y"]]
            y = 0.3 * torch.randn(M, K, generator=gen, device=DEV)
            y[M - pad:] = 0.0
            st["y"] = y.to(dt)
            if case["post"]:
                st["y_weight"] = vector(0.5, 0.1)
                st["y_bias"] = vector(0.0, 0.1) if layer else None
            if case["gate"] != "none":
                rows = {"row": M, "all": 1, "ids": 1 + M // 100}[case["gate"]]
                st["gate"] = torch.sigmoid(torch.randn(rows, K, generator=gen, device=DEV)).to(dt)
            if case["gate"] == "ids":  # requests lie together; -1: a request without a gate
                requests = torch.randint(-1, rows, (M // 100 + 1,), generator=gen, device=DEV)
                ends = torch.rand(M, generator=gen, device=DEV) < 0.01
                idx = torch.clamp(torch.cumsum(ends, 0), max=len(requests) - 1)
                st["gate_ids"] = requests[idx].to(torch.int32)
        if own:
            st["kw"] = dict(kind=w4.NORM_LAYER if layer else w4.NORM_RMS,
                            out_type={"f32": w4.NORM_OUT_F32, "f16": w4.NORM_OUT_F16,
                                      "bf16": w4.NORM_OUT_BF16, "int8": w4.NORM_OUT_INT8,
                                      "e4m3": w4.NORM_OUT_E4M3}[case["out"]])
            dt = {"int8": torch.int8, "e4m3": torch.uint8}.get(case["out"])
            st["into"] = {"out": torch.empty((M, K), dtype=dt or _TYPES[case["out"]], device=DEV),
                          "sx": torch.empty(M, device=DEV) if dt else None,
                          "x": torch.empty_like(st["x"]) if st["y"] is not None else st["x"]}
    else:
        H, F, g = case["H"], case["F"], case["group"]
        for name, N, K in (("w13", 2 * F, H), ("w2", H, F)):
            st[name] = _pack(torch.randn(N, K, generator=gen, device=DEV) * 0.02, g)
        x = _stream_rows(M, H, "f32", 0, gen)
        st["sx"] = x.abs().amax(1) / 127.0
        st["Xq"] = torch.clamp(torch.round(x / st["sx"][:, None]), -127, 127).to(torch.int8)
        if own:
            st["kw"] = dict(act=w4.ACT_GELU if case["act"] == "gelu" else w4.ACT_SILU)
            st["into"] = torch.empty((M, H), dtype=_TYPES[case["dtype"]], device=DEV)
            st["workspace"] = torch.empty(max(w4.ffn_workspace_size(M, H, F), 16),
                                          dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------- plain form ---

def _over(a, b):
    """a / b rounded to float32, through 64 bits (a quotient next to a border
    falls on the right side; 53 bits hold a float32 quotient's rounding)."""
    return (a.double() / b).to(torch.float32)


def _quant(x, top):
    """Per-row scale of float32 x, max|x| / top, and x over it."""
    m = x.abs().amax(1, keepdim=True)
    s = _over(m, top)
    s = torch.where(s > 0, s, torch.ones_like(s))
    return _over(x, s.double()), s.squeeze(1)


def _normed(x, kind, weight, bias, eps):
    if kind == "layer":
        x = x - x.double().mean(1, keepdim=True).to(torch.float32)
    r = (1.0 / torch.sqrt(x.double().square().mean(1, keepdim=True) + eps)).to(torch.float32)
    n = (x * r) * weight
    return n if bias is None else n + bias


def _norm_plain(st):
    x = st["x"].to(torch.float32)
    out = {}
    eps = float(torch.tensor(st["eps"], dtype=torch.float32))
    if st["y"] is not None:
        b = st["y"].to(torch.float32)
        if st["y_weight"] is not None:
            b = _normed(b, st["kind"], st["y_weight"], st["y_bias"], eps)
        if st["gate"] is not None:
            gate, ids = st["gate"].to(torch.float32), st["gate_ids"]
            if ids is None:
                b = b * gate
            else:
                on = ((ids >= 0) & (ids < len(gate)))[:, None]
                b = torch.where(on, b * gate[torch.clamp(ids, 0, len(gate) - 1).long()], b)
        x = x + b * st["scale"]
        out["x"] = x.to(st["x"].dtype)
    n = _normed(x, st["kind"], st["weight"], st["bias"], eps)
    if st["out"] == "int8":
        q, s = _quant(n, 127.0)
        return {**out, "out": torch.clamp(torch.round(q), -127, 127).to(torch.int8), "sx": s}
    if st["out"] == "e4m3":
        q, s = _quant(n, 448.0)
        # nearest multiple of the step of the value's binade, ties to even
        step = torch.ldexp(torch.ones_like(q), torch.clamp(torch.frexp(q).exponent - 1, min=-6) - 3)
        q = torch.clamp(torch.round(q / step) * step, -448.0, 448.0)
        return {**out, "out": torch.copysign(q, n).to(torch.float8_e4m3fn), "sx": s}
    return {**out, "out": n.to(_TYPES[st["out"]])}


def _unpack(p):
    """Signed INT8 weights [N][K] as float64 (their products and sums are then
    exact)."""
    N, K, g = p["N"], p["K"], p["group"]
    wq = p["wq"].view(N // 16, K // 128, 4, 16, 4, 4)
    q = torch.stack([wq & 15, wq >> 4], -1)           # n, kt, G, r, d, b, half
    q = q.permute(0, 3, 1, 2, 4, 6, 5).reshape(N, K // g, g).to(torch.int16)

    def param(x):
        x = x.view(N // 64, K // g, 16, 4)
        return x.permute(0, 3, 2, 1).reshape(N, K // g, 1).to(torch.int16)
    return (q * param(p["s_u8"]) + param(p["a_u8"]) - 128).view(N, K).to(torch.float64)


def _product(codes, s, p):
    return ((codes.to(torch.float64) @ _unpack(p).t()).to(torch.float32) * s[:, None]) * p["sw"]


def _ffn_plain(st):
    gu = _product(st["Xq"], st["sx"], st["w13"])
    g, u = gu[:, :st["F"]], gu[:, st["F"]:]
    z = g
    if st["act"] == "gelu":
        z = g * (2.0 * math.sqrt(2.0 / math.pi)) * (1.0 + 0.044715 * g * g)
    q, s = _quant(g / (1.0 + torch.exp(-z)) * u, 127.0)
    y = _product(torch.clamp(torch.round(q), -127, 127), s, st["w2"])
    return y.to(_TYPES[st["dtype"]])


def run(st):
    if not own:
        return _norm_plain(st) if st["op"] == "norm" else _ffn_plain(st)
    w4 = st["w4"]
    if st["op"] == "norm":
        r = w4.norm_quant(st["x"], st["weight"], st["bias"], y=st["y"], y_weight=st["y_weight"],
                          y_bias=st["y_bias"], gate=st["gate"], gate_ids=st["gate_ids"],
                          y_scale=st["scale"], eps=st["eps"], out=st["into"], **st["kw"])
        q = r["out"]
        if q.dtype == torch.uint8:
            q = q.view(torch.float8_e4m3fn)
        kept = {"x": r["x"]} if st["y"] is not None else {}
        return {**kept, "out": q} if r["sx"] is None else {**kept, "out": q, "sx": r["sx"]}
    return w4.ffn(st["Xq"], st["sx"], st["w13"], st["w2"], out=st["into"],
                  workspace=st["workspace"], **st["kw"])


# ------------------------------------------------------------------- work ---

def work(case):
    M = case["M"]
    if case["op"] == "norm":
        K, layer = case["K"], case["kind"] == "layer"
        per = _SIZE[case["x"]] + _SIZE[case["out"]]
        vectors = 1 + layer
        total = 0
        flops = 4 + 4 * layer
        if case["y"] != "none":
            per += _SIZE[case["x"]] + _SIZE[case["y"]]
            flops += 3
            if case["post"]:
                vectors += 1 + layer
                flops += 4 + 4 * layer
            if case["gate"] != "none":
                rows = {"row": M, "all": 1, "ids": 1 + M // 100}[case["gate"]]
                total += rows * K * _SIZE[case["y"]] + (4 * M if case["gate"] == "ids" else 0)
                flops += 1
        quantised = case["out"] in ("int8", "e4m3")
        total += M * K * per + 4 * K * vectors + (4 * M if quantised else 0)
        return {"bytes": total, "flops": M * K * (flops + 3 * quantised)}
    H, F, g = case["H"], case["F"], case["group"]
    weights = 3 * F * H // 2 + 2 * (3 * F * H // g) + 4 * (2 * F + H)
    return {"bytes": weights + M * H + 4 * M + 2 * M * H, "flops": 6 * M * H * F}


# ------------------------------------------------------------------ exact ---

def _weights64(p):
    """Decoded weights times their channel scale, [N][K] float64, from the
    byte positions of the documented layout."""
    N, K, g = p["N"], p["K"], p["group"]
    n = torch.arange(N, device=DEV)[:, None]
    kk = torch.arange(K, device=DEV)[None, :]
    c = kk % 128
    pos = 1024 * ((n // 16) * (K // 128) + kk // 128) + 16 * (16 * (c // 32) + n % 16)
    pos = pos + 4 * (c % 32 // 8) + c % 4
    code = p["wq"][pos]
    del pos
    code = torch.where(c % 8 >= 4, code >> 4, code & 15).to(torch.float64)
    j = torch.arange(K // g, device=DEV)[None, :]
    at = 64 * ((n // 64) * (K // g) + j) + 4 * (n % 16) + n % 64 // 16
    code = code.view(N, K // g, g)
    code.mul_(p["s_u8"][at].to(torch.float64)[:, :, None])
    code.add_(p["a_u8"][at].to(torch.float64)[:, :, None] - 128.0)
    return code.view(N, K).mul_(p["sw"].to(torch.float64)[:, None])


def _int8_64(x):
    """The values that per-row INT8 codes of x stand for.  Scale and code are
    defined by float32 arithmetic (whole numbers, so a quotient next to a half
    has to fall on the definition's side); the values are float64."""
    x32 = x.to(torch.float32).double()
    s = x32.abs().max(dim=1, keepdim=True).values.div(127.0).float().double()
    s = s.masked_fill(s == 0, 1.0)
    return x32.div(s).float().round().clamp(-127, 127).double() * s


def _standard64(x, layer, w, b, eps):
    if layer:
        x = x - x.sum(1, keepdim=True) / x.shape[1]
    v = (x * x).sum(1, keepdim=True) / x.shape[1]
    x = x * (v + eps).rsqrt() * w.double()
    return x + b.double() if b is not None else x


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        layer = case["kind"] == "layer"
        x, kept = st["x"].double(), {}
        if st["y"] is not None:
            b = st["y"].double()
            if st["y_weight"] is not None:
                b = _standard64(b, layer, st["y_weight"], st["y_bias"], st["eps"])
            if st["gate"] is not None:
                factor = st["gate"].double()
                if st["gate_ids"] is not None:
                    # a row of ones behind the gates, for requests without one
                    more = torch.cat([st["gate"].double(),
                                      torch.ones(1, case["K"], device=DEV).double()])
                    factor = more[st["gate_ids"].long()]
                b = b * factor
            kept["x"] = x = x + case["scale"] * b
        n = _standard64(x, layer, st["weight"], st["bias"], st["eps"])
        if case["out"] in ("f32", "f16", "bf16"):
            return {**kept, "out": n}
        s = n.abs().max(dim=1).values / (127.0 if case["out"] == "int8" else 448.0)
        s = s.masked_fill(s == 0, 1.0)
        # codes are whole numbers by float32 arithmetic; e4m3's quotients are computed numbers
        return {**kept, "out": None if case["out"] == "int8" else n / s[:, None], "sx": s}
    F = case["F"]
    gu = (st["Xq"].double() * st["sx"].double()[:, None]) @ _weights64(st["w13"]).t()
    g, u = gu[:, :F], gu[:, F:]
    if case["act"] == "gelu":
        h = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u
    else:
        h = torch.sigmoid(g) * g * u
    return _int8_64(h) @ _weights64(st["w2"]).t()
