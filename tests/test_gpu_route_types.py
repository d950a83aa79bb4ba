"""The row movers and the adapters for the pairs of element types that their own tests
leave out, with those tests' references and tolerances."""
import pytest
import test_gpu_lora as lora
import test_gpu_route as route

pytestmark = pytest.mark.gpu

q = route.q
TYPES = ("f32", "f16", "bf16")
# one wave a token and four, whole pieces and rows of odd lengths
SHAPES = [(5, 3, 4, 250), (33, 4, 9, 1022), (70, 6, 8, 2051), (37, 2, 8, 2048)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dt,yt", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,k,E,C", SHAPES)
def test_combine(q, T, k, E, C, dt, yt, weighted):
    route.test_combine(q, T, k, E, C, weighted, dt, yt)


@pytest.mark.parametrize("dt,yt", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,k,E,C", SHAPES)
def test_combine_grad(q, T, k, E, C, dt, yt):
    route.test_combine_grad(q, T, k, E, C, dt, yt)


# one launch and two, B in registers and not, tiles of 16 and 32 tokens, rows of y of whole
# dwords and not
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("dt,yt", [("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("T,E,r,M,K", [(17, 4, 32, 4, 4096), (5, 2, 24, 37, 136), (50, 4, 64, 1091, 264),
                                       (300, 5, 40, 1260, 96), (33, 2, 256, 66, 264), (200, 3, 128, 515, 2048)])
def test_lora(q, T, E, r, M, K, dt, yt, kind):
    lora.test_lora(q, T, E, r, M, K, dt, yt, kind)
