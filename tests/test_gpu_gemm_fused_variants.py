"""Every tile width and K split of gemm_fused's many-token kernel, forced one by one, over several waves of tiles, uneven
chunks of K and ragged edges; the dispatch of 17 to 64 tokens with large weights; and its bounded waits.

Without an activation the epilogue is FP32 operations in a stated order, so outputs are equal bit for bit to the same
operations on the exact product (FP64 sums of integers)."""
import math
import time

import pytest
import torch

from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def cr():
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    return cr


def problem(M, N, Kp, out, seed, residual=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    codes = lambda rows: (rand(rows, Kp) * 40).round().clamp(-127, 127).half()
    return dict(a=codes(M), w=codes(N), sa=0.02 + 0.01 * rand(M).abs(), sw=(0.02 + 0.01 * rand(N).abs()) / math.sqrt(Kp),
                bias=rand(N), gate=rand(N), residual=(2 * rand(M, N)).to(TORCH_DT[out]) if residual else None)


def exact(p, out):
    acc = p["a"].double() @ p["w"].double().t()
    y = (acc.float() * p["sa"][:, None] * p["sw"] + p["bias"]) * p["gate"]
    if p["residual"] is not None:
        y = y + p["residual"].float()
    return y.to(TORCH_DT[out])


def forced(cr, p, y, tile, slices, **kw):
    cr.gemm_fused_selftest(p["a"], p["sa"], p["w"], p["sw"], y, tile, slices, bias=p["bias"], gate=p["gate"],
                           residual=p["residual"], **kw)
    return y


VARIANTS = [(128, 1), (256, 1), (128, 2), (128, 3), (128, 4), (192, 2), (192, 3), (192, 4), (256, 2), (256, 3), (256, 4)]
# K_p: whole tiles in chunks of 16 steps of 64 (84 = 16, ..., 16, 4; 36 = 16, 16, 4; 32; 20), slices of unequal lengths
SHAPES = [(2305, 2600, 5376), (2305, 2600, 2304), (513, 700, 2048), (700, 513, 5376), (40, 1000, 3840), (257, 130, 20480)]


@pytest.mark.parametrize("tile,slices", VARIANTS)
@pytest.mark.parametrize("M,N,Kp", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_variant_bit_for_bit(cr, tile, slices, M, N, Kp, out):
    # 2305 x 2600 in whole tiles: 110 (256 wide) and 210 (128 wide) of them, more than the GPU has CTA pairs (76)
    p = problem(M, N, Kp, out, M + N + Kp)
    y = torch.full((M, N), 9.0, dtype=TORCH_DT[out], device=DEV)
    forced(cr, p, y, tile, slices)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    assert torch.equal(y, exact(p, out))


@pytest.mark.parametrize("tile,slices", VARIANTS)
def test_variant_with_unaligned_rows_in_place(cr, tile, slices):
    # rows that start on no 16-byte boundary (an odd width), the residual read from the output itself
    M, N, Kp = 1030, 777, 2304
    p = problem(M, N, Kp, "fp16", tile + slices)
    want = exact(p, "fp16")
    y = p["residual"]
    forced(cr, p, y, tile, slices)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("tile,slices", VARIANTS)
@pytest.mark.parametrize("act", ["SILU", "GELU_TANH"])
def test_activation_does_not_depend_on_the_variant(cr, tile, slices, act):
    M, N, Kp = 300, 600, 2304
    p = problem(M, N, Kp, "fp32", 3)
    code = getattr(cr, "ACT_" + act)
    y = torch.empty(M, N, device=DEV)
    forced(cr, p, y, tile, slices, act=code)
    want = torch.empty_like(y)
    cr.gemm_fused(p["a"], p["sa"], p["w"], p["sw"], want, bias=p["bias"], act=code, gate=p["gate"], residual=p["residual"])
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [17, 33, 64])
@pytest.mark.parametrize("N,Kp", [(1700, 5376), (5376, 2048), (300, 30720)])     # more than 16 MiB of FP16-held weights
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_few_tokens_with_large_weights(cr, M, N, Kp, out):
    assert N * Kp * 2 > 16 << 20
    p = problem(M, N, Kp, out, M)
    y = torch.empty(M, N, dtype=TORCH_DT[out], device=DEV)
    cr.gemm_fused(p["a"], p["sa"], p["w"], p["sw"], y, bias=p["bias"], gate=p["gate"], residual=p["residual"])
    torch.cuda.synchronize()
    assert torch.equal(y, exact(p, out))


def test_refusals(cr):
    p = problem(20, 64, 768, "bf16", 1)
    y = torch.empty(20, 64, dtype=torch.bfloat16, device=DEV)
    for tile, slices in [(0, 1), (64, 1), (192, 1), (128, 0), (128, 5), (256, 2)]:        # 768 is less than 2 x 512
        with pytest.raises(cr.ConvRotError) as e:
            forced(cr, p, y, tile, slices)
        assert e.value.status == 1


@pytest.mark.parametrize("tile,slices,M,N,out", [(256, 1, 3000, 3000, "bf16"), (128, 1, 200, 300, "fp32"),
                                                 (192, 2, 300, 600, "fp16"), (256, 4, 300, 600, "bf16")])
def test_waits_run_out_and_the_context_survives(cr, tile, slices, M, N, out):
    # the producer is off: every role has to leave its loop, meet at the cluster's barriers (split tiles have two more)
    # and land the residual boxes it asked for; then the kernel returns, and the next launch is right
    p = problem(M, N, 2048, out, 5)
    y = torch.zeros(M, N, dtype=TORCH_DT[out], device=DEV)
    forced(cr, p, y, tile, slices)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    t0 = time.time()
    forced(cr, p, y, tile, slices, starve=True)
    code = cr.device_error()                          # synchronises
    waited = time.time() - t0
    assert code != 0 and 1.0 < waited < 30.0
    assert cr.device_error() == 0                     # reading clears the word
    forced(cr, p, y, tile, slices)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    assert torch.equal(y, exact(p, out))
