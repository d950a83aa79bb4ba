"""Products and adapters over hundreds of weight sets, most of them unnamed, a few with most
of the rows, with the references and tolerances of their own tests."""
import numpy as np
import pytest
import test_gpu_lora as lora
import test_gpu_routed as routed

pytestmark = pytest.mark.gpu

q = routed.q


def _skewed(T, k, E, seed):
    """Router ids: different weight sets a token, popularity falling as 1 / rank, the first
    and the last set among the named ones, some slots naming none."""
    rng = np.random.Generator(np.random.PCG64(seed))
    p = 1.0 / np.arange(1, E + 1)
    p /= p.sum()
    rank = rng.permutation(E)
    ids = np.stack([rank[rng.choice(E, k, replace=False, p=p)] for _ in range(T)]).astype(np.int32)
    ids[0, 0], ids[T - 1, k - 1] = 0, E - 1
    if T > 8:
        ids[3] = -1
        ids[5, 0] = E
    return ids


@pytest.mark.parametrize("mapped", [True, False])
@pytest.mark.parametrize("fmt", list(routed.UNIT))
@pytest.mark.parametrize("T,k,E,M,units", [(5, 2, 1024, 17, 1), (300, 2, 257, 33, 2), (900, 4, 129, 70, 1), (1500, 2, 1000, 16, 1)])
def test_products(q, T, k, E, M, units, fmt, mapped):
    K = routed.UNIT[fmt] * units
    got = routed._run(q, fmt, _skewed(T, k, E, T + E), k, E, M, K, 7000, "f32", mapped)
    routed._check(fmt, *got, k, M, K, "f32", mapped)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,E,r,M,K", [(7, 1024, 16, 40, 64), (500, 300, 64, 1100, 72), (900, 1000, 128, 33, 136)])
def test_adapters(q, T, E, r, M, K, dt):
    ids = _skewed(T, 1, E, T + E)[:, 0].tolist()
    x, a, b, scale, c = lora._inputs(T, E, r, M, K, dt, "f32", T)
    order, offsets = lora._plan(q, ids, E)
    y = lora.torch.full((T, M), float("nan"), device=lora.DEV)
    q.QLORA[dt](*(v.to(lora.DEV) for v in (x, a, b, scale)), order, offsets, c.to(lora.DEV), y, T, E, r, M, K,
                lora._ws(q, T, E, r, M, K))
    lora._check(y, ids, E, r, K, x, a, b, scale, c, "f32")
