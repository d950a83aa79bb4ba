"""Adapters whose inner product v = A_e x has components of very different sizes.

Column m of an output takes component m % r alone (B has one nonzero a row), so
every component is checked by its own size.  v_j is summed in fp32 by at most
K / 32 accumulations of 32 products and 4 waves and 16 parts, each off by at most
2^-23 of what it adds up; scale * v_j rounds once and is kept bit for bit down to
2^-39 of the token's largest component (fp16; to 2^-63 of it below) or to 24 bits
(bf16); the products of its terms with B and their sum pass through r + 4
additions of at most 2^-23 each:
    |dy| <= |s B| ((K / 32 + 52) 2^-23 sum_i |A_ji x_i| + (r + 6) 2^-23 |v_j| + 2^-62 max |v|)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    from dequant_gemv_amd import qgemv

    return qgemv


# (T, E, r, M, K): one launch (r <= 32, or A small and few columns), two launches
# with B ahead in registers or not, tiles of 16 and of 32 tokens
CASES = [(5, 1, 16, 48, 256), (20, 2, 32, 160, 512), (9, 1, 128, 256, 264), (40, 1, 64, 1100, 264),
         (70, 1, 40, 1200, 1024), (24, 3, 72, 1216, 520), (33, 1, 256, 1300, 264), (130, 2, 128, 1090, 96)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,E,r,M,K", CASES)
def test_every_component_by_its_own_size(q, T, E, r, M, K, dt):
    g = torch.Generator().manual_seed(T + r)
    x = torch.randn(T, K, generator=g).to(DT[dt])
    # rows of A from 2^14 down to 2^-14 (their own rounding is part of the input)
    down = torch.linspace(14, -14, r)[torch.randperm(r, generator=g)].round()
    a = (torch.randn(E, r, K, generator=g) * 2.0 ** down[:, None]).clamp(-60000, 60000).to(DT[dt])
    b = torch.zeros(E, M, r)
    cols = torch.arange(M)
    b[:, cols, cols % r] = torch.rand(E, M, generator=g) + 0.5
    b = b.to(DT[dt])
    scale = torch.rand(E, generator=g) + 0.5
    ids = torch.randint(0, E, (T,), generator=g).int()
    order, position = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    q.qroute_sort(ids.to(DEV), T, E, order, position, offsets)
    ws = torch.empty(q.qlora_workspace_bytes(T, E, r, M, K), dtype=torch.uint8, device=DEV)
    y = torch.full((T, M), float("nan"), device=DEV)
    q.QLORA[dt](*(v.to(DEV) for v in (x, a, b, scale)), order, offsets, None, y, T, E, r, M, K, ws)
    got = y.cpu().double().numpy()
    for t in range(T):
        e = int(ids[t])
        A, xv = a[e].double().numpy(), x[t].double().numpy()
        v, sums = A @ xv, np.abs(A) @ np.abs(xv)
        sb = float(scale[e]) * b[e].double().numpy()[np.arange(M), np.arange(M) % r]
        at = np.arange(M) % r
        bound = (K / 32 + 52) * 2.0 ** -23 * sums + (r + 6) * 2.0 ** -23 * np.abs(v) + 2.0 ** -62 * np.abs(v).max()
        err = np.abs(got[t] - sb * v[at])
        assert np.all(err <= sb * bound[at]), (t, float(np.max(err / (sb * bound[at]))))
