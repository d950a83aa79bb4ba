"""Infinite and NaN activations, and infinite Q4_K scales, in the routed products: outputs
are what the definition sum (weight * activation) gives, infinities with their sign
and NaN where it has one; other tokens' outputs keep their bits."""
import numpy as np
import pytest
import torch

import oracle
from dequant_gemv_amd import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
UNIT = {"q4k": 256, "nvfp4": 64, "tq1": 256}


@pytest.fixture(scope="module")
def q():
    from dequant_gemv_amd import qgemv

    return qgemv


def _products(q, fmt, w, xt, ids, E, M, K, mapped):
    T = len(ids)
    order, position = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, q.qroute_workspace_bytes(T, E)), dtype=torch.uint8, device=DEV)
    q.qroute_sort(torch.from_numpy(ids).to(DEV), T, E, order, position, offsets, ws)
    src = order.cpu().long()
    y = torch.full((T, M), -9.0, device=DEV)
    wd = torch.from_numpy(np.concatenate([v.reshape(-1) for v in w])).to(DEV)
    q.GEMM_ROUTED[fmt](wd, (xt if mapped else xt[src]).to(DEV), order if mapped else None, offsets, y, T, 1, E, M, K)
    out = torch.empty(T, M)
    out[src] = y.cpu()
    return out.numpy()


def _want(x, w):
    """sum of w * x over the last axis, infinities and NaN as IEEE gives them"""
    with np.errstate(invalid="ignore"):
        return (w * x).sum(1)


# few rows (K in parts and whole), many rows
@pytest.mark.parametrize("mapped", [True, False])
@pytest.mark.parametrize("fmt", list(UNIT))
@pytest.mark.parametrize("T,E,M,units", [(1, 1, 5, 1), (7, 2, 70, 8), (20, 2, 9001, 2), (130, 1, 1000, 4), (600, 3, 900, 2)])
def test_infinite_activations(q, fmt, T, E, M, units, mapped):
    K = UNIT[fmt] * units
    rng = np.random.Generator(np.random.PCG64(T * 31 + M))
    ids = rng.integers(0, E, T).astype(np.int32)
    w = [synth.weights(fmt, M, K, 5000 + e) for e in range(E)]
    if fmt == "q4k":  # some weights that are zero: q = 0 and min = 0 in the first block of every other row
        w[0].reshape(M, -1)[::2, 4:16] = 0
    dt = torch.bfloat16 if fmt == "nvfp4" else torch.float16
    bits = np.stack([synth.activations(fmt, K, 5100 + i) for i in range(T)])
    clean = torch.from_numpy(bits.view(np.int16)).view(dt)
    x = clean.clone()
    inf, at = float("inf"), rng.integers(0, K, (T, 2))
    kinds = {0: "plus", 3: "minus", 6: "both", 9: "twice", 12: "nan", T - 1: "plus"}
    for t, kind in kinds.items():
        if t >= T:
            continue
        a, b = at[t, 0], (at[t, 0] + 1 + at[t, 1] % (K - 1)) % K
        x[t, a] = -inf if kind == "minus" else inf
        if kind != "plus" and kind != "minus":
            x[t, b] = {"both": -inf, "twice": inf, "nan": float("nan")}[kind]
    got = _products(q, fmt, w, x, ids, E, M, K, mapped)
    base = _products(q, fmt, w, clean, ids, E, M, K, mapped)
    touched = [t for t in kinds if t < T]
    rest = np.setdiff1d(np.arange(T), touched)
    assert np.array_equal(got[rest], base[rest])
    exact = [oracle.dequant(fmt, v, M, K) for v in w]
    for t in touched:
        want = _want(x[t].double().numpy(), exact[ids[t]])
        assert not np.isfinite(want).any()
        assert np.array_equal(got[t], want.astype(np.float32), equal_nan=True), (t, kinds[t])


@pytest.mark.parametrize("T,M", [(3, 40), (200, 700), (1100, 300)])
@pytest.mark.parametrize("fmt", ["q4k", "tq1"])
def test_infinite_scales(q, fmt, T, M):
    """Blocks with an infinite d or dmin, in rows of their own."""
    K = 512
    w = synth.weights(fmt, M, K, 5200)
    x = torch.from_numpy(np.stack([synth.activations(fmt, K, 5300 + i) for i in range(T)]).view(np.int16)).view(torch.float16)
    x[0] = x[0].abs() + 1            # one token whose activations are all above zero
    if fmt == "q4k":
        rows = w.reshape(M, 2, 144)
        rows[1, 0, 0:2] = (0x00, 0x7C)   # d = inf: weights inf, NaN where scale * q is 0
        rows[2, 1, 2:4] = (0x00, 0x7C)   # dmin = inf: weights -inf, NaN where min is 0
        rows[3, 0, 0:2] = (0x00, 0xFC)
        rows[3, 0, 4:16] = 0xFF          # d = -inf, scales and mins 63
        rows[3, 0, 16:] |= 0x11          # and no q of 0: every weight is -inf
    else:
        rows = w.reshape(M, 2, 54)
        rows[1, 0, 52:54] = (0x00, 0x7C)  # weights inf, -inf and NaN
        rows[2, 1, 52:54] = (0x00, 0xFC)
        rows[3, 0, 52:54] = (0x00, 0xFC)
        rows[3, 0, :52] = 0               # every digit 0, every weight -inf * -1
    got = _products(q, fmt, [w], x, np.zeros(T, dtype=np.int32), 1, M, K, True)
    with np.errstate(invalid="ignore"):
        exact = oracle.dequant(fmt, w, M, K)
    for t in range(T):
        want = _want(x[t].double().numpy(), exact)
        assert np.isfinite(want[4:]).all() and not np.isfinite(want[1:4]).any()
        assert np.array_equal(got[t, 1:4], want[1:4].astype(np.float32), equal_nan=True), t
        assert np.isfinite(got[t, 0]) and np.isfinite(got[t, 4:]).all()
    assert got[0, 3] == (-np.inf if fmt == "q4k" else np.inf)
