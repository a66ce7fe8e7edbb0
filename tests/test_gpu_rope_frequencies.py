"""qk_norm_rope with frequencies that are Inf or NaN: their pairs become NaN, whatever the position, and no other value
changes.  Very large and very small finite frequencies keep their turn."""
import math

import pytest
import torch

from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def rotate(x, pos, freq, interleaved):
    import rotated_w4a8_int8_gb300 as cr
    y = torch.empty_like(x)
    cr.qk_norm_rope(x, None, pos, torch.tensor(freq, dtype=torch.float64, device=DEV), [len(freq)], y, None,
                    interleaved=interleaved)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,P", [(128, 64), (128, 32), (24, 12), (14, 7)])      # runs of eight, of four, single elements
def test_frequencies_without_an_angle(D, P, interleaved):
    ensure_built()
    g = torch.Generator().manual_seed(D + P)
    x = torch.randn(5, 3, D, generator=g).to(DEV)
    pos = torch.tensor([[0], [1], [-7], [20000], [2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    freq = [10000.0 ** (-i / P) for i in range(P)]
    want = rotate(x, pos, freq, interleaved)
    bad = {0: math.nan, 2: math.inf, P - 1: -math.inf}
    got = rotate(x, pos, [bad.get(i, f) for i, f in enumerate(freq)], interleaved)
    lost = torch.zeros(D, dtype=torch.bool)
    for i in bad:
        lost[[2 * i, 2 * i + 1] if interleaved else [i, i + P]] = True
    lost = lost.to(DEV)
    assert bool(got[:, :, lost].isnan().all())
    assert torch.equal(got[:, :, ~lost], want[:, :, ~lost])


@pytest.mark.parametrize("freq", [2.0 ** 60, 1e300, 1.7976931348623157e308, 5e-324, 1e-30, 0.0])
def test_extreme_finite_frequencies(freq):
    ensure_built()
    x = torch.randn(2, 1, 16, generator=torch.Generator().manual_seed(3)).to(DEV)
    pos = torch.tensor([[0], [3]], dtype=torch.int32, device=DEV)
    y = rotate(x, pos, [freq] * 8, False)
    assert torch.equal(y[0], x[0])                                      # position 0 does not turn
    length = torch.hypot(x[:, 0, :8], x[:, 0, 8:])
    assert torch.allclose(torch.hypot(y[:, 0, :8], y[:, 0, 8:]), length, rtol=2e-6, atol=0)
    if freq < 1e-20:
        assert torch.equal(y, x)
