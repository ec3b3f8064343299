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
