"""Q4_K weights in the routed products are not rounded, with few rows or many.

Activations of one power of two and zeros: an output is one weight times that
power of two.  d * scale * q and dmin * min are each exact in fp32 (11 + 10 and
11 + 6 bits), all other terms are zero, and one fused multiply-add rounds their
difference, so the only right answer is the exact weight rounded once to fp32.
An fp16 weight would be off by up to 2^-12 of itself."""
import numpy as np
import pytest
import torch

import oracle
from dequant_gemv_amd import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def q():
    from dequant_gemv_amd import qgemv

    return qgemv


# (T, E, M, K): one weight set's worth of tiles and several, short last tiles of
# tokens and of weight rows, few and many workgroups
CASES = [(3, 2, 33, 256), (40, 1, 300, 512), (65, 1, 257, 768), (200, 1, 1025, 256), (300, 3, 129, 1280),
         (520, 1, 128, 1280), (700, 2, 513, 1792), (1024, 2, 1700, 512), (1333, 40, 896, 256), (4099, 3, 1537, 768)]


@pytest.mark.parametrize("mapped", [True, False])
@pytest.mark.parametrize("T,E,M,K", CASES)
def test_q4k_weights_are_not_rounded(q, T, E, M, K, mapped):
    rng = np.random.Generator(np.random.PCG64(T + M))
    ids = rng.integers(0, E, T).astype(np.int32)
    w = [synth.weights("q4k", M, K, 3000 + e) for e in range(E)]
    at, power = rng.integers(0, K, T), rng.integers(-6, 7, T)
    x = np.zeros((T, K), dtype=np.float16)
    x[np.arange(T), at] = 2.0 ** power
    t = torch.from_numpy(ids).to(DEV)
    order, position = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, q.qroute_workspace_bytes(T, E)), dtype=torch.uint8, device=DEV)
    q.qroute_sort(t, T, E, order, position, offsets, ws)
    y = torch.full((T, M), -9.0, device=DEV)
    src = order.cpu().numpy()
    xd = torch.from_numpy(x if mapped else x[src]).to(DEV)
    wd = torch.from_numpy(np.concatenate([v.reshape(-1) for v in w])).to(DEV)
    q.qgemm_q4k_routed(wd, xd, order if mapped else None, offsets, y, T, 1, E, M, K)
    got, exact = y.cpu().numpy(), [oracle.dequant("q4k", v, M, K).astype(np.float64) for v in w]
    for p in range(T):
        s = src[p]
        want = (exact[ids[s]][:, at[s]] * 2.0 ** power[s]).astype(np.float32)
        assert np.array_equal(got[p], want), (p, float(np.max(np.abs(got[p] / want - 1))))
