"""gemm_fused's activations over their whole range, tails included: products of zero codes leave act(bias).

Tolerances, relative to the value, in units of 2^-23.  FP32 outputs: SiLU's exponential (2), sum (1/2), reciprocal (1) and
product (1/2) are 4, 2^-21; GELU's polynomial (2 1/2), its variable's reciprocal (1), exponential and its correction
(2 1/2) and three products (1 1/2) are less than 8, 2^-20; the tanh form's cubic argument v is rounded four times, which
its exponential turns into |v| 2^-22 of the value, beside SiLU's 2^-21.
16-bit outputs: 3e-5 of the value, as the header states, and half a unit of the type.  Values below 2^-120 leave the
normal numbers within the functions: 2^-120 is allowed as an absolute error.
"""
import math

import pytest
import torch

from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def grid():
    near = torch.linspace(-20, 20, 16001, dtype=torch.float64)
    far = torch.linspace(-100, 100, 4001, dtype=torch.float64)
    small = torch.logspace(-30, 0, 301, dtype=torch.float64)
    x = torch.cat([near, far, small, -small, torch.tensor([0.0], dtype=torch.float64)]).float()
    return x[:x.numel() // 4 * 4]


def exact(act, x):
    x = x.double()
    if act == "SILU":
        return x * torch.sigmoid(x)
    if act == "GELU":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
    v = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return x * torch.sigmoid(v)


@pytest.mark.parametrize("act", ["SILU", "GELU", "GELU_TANH"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M", [2, 65])                    # the few-token kernel and the other one
def test_functions_over_their_range(act, out, M):
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    x = grid()
    N, z = x.numel(), dict(dtype=torch.float16, device=DEV)
    y = torch.empty(M, N, dtype=TORCH_DT[out], device=DEV)
    cr.gemm_fused(torch.zeros(M, 256, **z), torch.ones(M, device=DEV), torch.zeros(N, 256, **z),
                  torch.ones(N, device=DEV), y, bias=x.to(DEV), act=getattr(cr, "ACT_" + act))
    torch.cuda.synchronize()
    assert bool((y == y[0]).all())
    got, want = y[0].double().cpu(), exact(act, x)
    if out == "fp32":
        v = 2 * math.sqrt(2 / math.pi) * (x.double() + 0.044715 * x.double() ** 3)
        rel = {"SILU": 2.0 ** -21, "GELU": 2.0 ** -20, "GELU_TANH": 2.0 ** -21 + 2.0 ** -22 * v.abs()}[act]
        lim = rel * want.abs() + 2.0 ** -120
    else:
        lim = (3e-5 + HALF_ULP[out]) * want.abs() + (2.0 ** -25 if out == "fp16" else 2.0 ** -120)
    worst = ((got - want).abs() / lim).argmax()
    assert bool(((got - want).abs() <= lim).all()), (float(x[worst]), float(got[worst]), float(want[worst]))


@pytest.mark.parametrize("M", [2, 65])
def test_infinite_and_undefined_inputs(M):
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    x = torch.tensor([math.inf, math.nan, 1e30, -1e30, 3e38, -3e38, 0.0, 1.0])
    z = dict(dtype=torch.float16, device=DEV)
    for out in ("bf16", "fp32"):
        for act in ("SILU", "GELU", "GELU_TANH"):
            y = torch.empty(M, 8, dtype=TORCH_DT[out], device=DEV)
            cr.gemm_fused(torch.zeros(M, 256, **z), torch.ones(M, device=DEV), torch.zeros(8, 256, **z),
                          torch.ones(8, device=DEV), y, bias=x.to(DEV), act=getattr(cr, "ACT_" + act))
            got = y[M - 1].float().cpu()
            assert got[0] == math.inf and math.isnan(got[1])
            assert torch.equal(got[[2, 4]], x[[2, 4]].to(TORCH_DT[out]).float())
            assert bool((got[[3, 5, 6]] == 0).all())
