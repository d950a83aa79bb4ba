"""The combine's gradient with the most tokens: rows of more than 1024 elements, for which
four waves a token would be 2^32 work items."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_combine_grad_of_the_most_tokens():
    from dequant_gemv_amd import qgemv as q

    T, C = 2 ** 24, 1032  # 35 GB each of dy, rows and drows
    rows = torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    rows.view(-1, 4, C).copy_(torch.arange(4, device=DEV)[None, :, None].expand(T // 4, 4, C))
    dy = torch.full((T, C), 2.0, dtype=torch.bfloat16, device=DEV)
    drows = torch.full((T, C), -9.0, dtype=torch.bfloat16, device=DEV)
    position = torch.arange(T, dtype=torch.int32, device=DEV).flip(0)
    weights = torch.full((T, 1), 0.25, device=DEV)
    dweights = torch.full((T, 1), -9.0, device=DEV)
    q.qroute_combine_grad(dy, rows, position, weights, drows, dweights, T, 1, C)
    want = (2.0 * C) * (position % 4).float()  # every sum exact
    assert torch.equal(dweights[:, 0], want)
    assert int(drows.view(torch.int16).max()) == int(drows.view(torch.int16).min())
    assert float(drows[T - 1, C - 1]) == 0.5
    del rows, dy, drows
    torch.cuda.empty_cache()
