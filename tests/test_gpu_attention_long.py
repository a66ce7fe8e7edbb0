"""attention over very many keys: what the sums of a row lose on the way.  Scores are chosen so that everything but the sum
under test is exact or bounded by a few roundings.

The roundings that the bounds count, with u half a step of the type (finfo.eps / 2): the output's u; the weights' own 2^-20
(their exponents' one rounded product and the exponential); the row's sum, FP32: weights of a tile of 128 keys are added to
one another (in two halves of 64), tiles' sums to the row's, 2^-24 of the sum for every addition one after another.
"""
import math

import pytest
import torch

from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF, HF = torch.bfloat16, torch.float16
KERNELS = [(1, 1), (1, 4), (2, 1), (3, 1), (3, 4)]        # kernel, CTAs that share keys
N = 2 ** 22


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gap", [0.3, 0.55, 0.7])
def test_sum_of_equal_weights(kernel, dtype, gap):
    """The first of every 128 keys has the largest score, all others lie `gap` powers of two below it: weights that are no
    power of two.  Only key 0 has a value, so the output is that value times its weight (exact) over the row's sum."""
    import rotated_w4a8_int8_gb300 as cr
    q = torch.ones(20, 1, 64, dtype=dtype, device=DEV)
    k, v = (torch.zeros(N, 1, 64, dtype=dtype, device=DEV) for _ in range(2))
    k[::128, 0, 0] = 1.0
    v[0] = 2.0 ** 15
    scale = float(torch.tensor(gap * math.log(2), dtype=torch.float32))
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel, scale=scale)
    torch.cuda.synchronize()
    want = 2.0 ** 15 / (N // 128 + (N - N // 128) * math.exp(-scale))
    bound = torch.finfo(dtype).eps / 2 + 2.0 ** -20 + (64 + N // 128) * 2.0 ** -24
    assert float((out.double() / want - 1).abs().max()) <= bound
