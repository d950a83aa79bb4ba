"""TQ1_0 matrices whose last dword holds two bytes that are not theirs: the last block's
scale sits in it, the bytes after it are garbage (NaN codes), and every tile's last
row takes its scale from where the tile ends.  Exact inputs (scales of 1,
activations -1, 0, 1): one right result."""
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


# (T, E, M, units): M * units * E odd, so the matrices end in the middle of a dword; one
# and several parts of K, workgroups of 32 and 64 rows, rows 1 .. 16 of a wave's last tile
@pytest.mark.parametrize("T,E,M,units", [(1, 1, 1, 1), (3, 1, 17, 3), (2, 1, 15, 5), (20, 3, 33, 7), (50, 1, 1025, 1),
                                         (300, 7, 129, 3), (900, 9, 515, 1), (30, 1, 4099, 35)])
def test_tq1_last_scale(q, T, E, M, units):
    K = 256 * units
    rng = np.random.Generator(np.random.PCG64(M))
    w = [synth.weights_exact("tq1", M, K, 40 + e) for e in range(E)]
    packed = np.concatenate([v.reshape(-1) for v in w])
    assert packed.size % 4 == 2
    guarded = np.full(packed.size + 62, 0x7E, dtype=np.uint8)
    guarded[:packed.size] = packed
    wd = torch.from_numpy(guarded).to(DEV)
    ids = rng.integers(0, E, T).astype(np.int32)
    x = np.stack([synth.x_ternary("tq1", K, 70 + i) for i in range(T)])
    order, position = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, q.qroute_workspace_bytes(T, E)), dtype=torch.uint8, device=DEV)
    q.qroute_sort(torch.from_numpy(ids).to(DEV), T, E, order, position, offsets, ws)
    y = torch.full((T, M), -9.0, device=DEV)
    q.qgemm_tq1_routed(wd, torch.from_numpy(x.view(np.int16)).to(DEV), order, offsets, y, T, 1, E, M, K)
    got, src = y.cpu().numpy(), order.cpu().numpy()
    xv = torch.from_numpy(x.view(np.int16)).view(torch.float16).double().numpy()
    for e in range(E):
        p = np.nonzero(ids[src] == e)[0]
        want = xv[src[p]] @ oracle.dequant("tq1", w[e], M, K).T
        assert np.array_equal(got[p], want.astype(np.float32)), e
