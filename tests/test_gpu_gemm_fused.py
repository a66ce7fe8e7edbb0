"""gemm_fused (the integer product with bias, activation, channel gate and
residual in its epilogue) against exact integers and 64-bit formulas.

Without an activation every step of the epilogue is one FP32 operation in a
stated order, so the output has to be equal bit for bit.  With one, the
tolerance is 3e-6 of the terms (products, bias and the functions at a few
units of 2^-24 each; the functions' slopes are at most 1.13) times the gate,
plus half a unit in the last place of the output type.
"""
import math

import pytest
import torch

from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
ACTS = ["NONE", "RELU", "SILU", "GELU", "GELU_TANH"]


@pytest.fixture(scope="module")
def cr():
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    return cr


def codes(rows, Kp, g, full=False):
    if full:
        return torch.full((rows, Kp), 127.0)
    return (torch.randn(rows, Kp, generator=g) * 40).round().clamp(-127, 127)


def problem(M, N, Kp, out, seed, bias=True, gate=True, residual=True, full=False):
    g = torch.Generator().manual_seed(seed)
    a, w = codes(M, Kp, g, full), codes(N, Kp, g, full)
    return dict(a=a, w=w, sa=0.01 + 0.02 * torch.rand(M, generator=g),
                sw=(0.01 + 0.02 * torch.rand(N, generator=g)) / math.sqrt(Kp),
                bias=torch.randn(N, generator=g) if bias else None,
                gate=torch.randn(N, generator=g) if gate else None,
                residual=(2 * torch.randn(M, N, generator=g)).to(TORCH_DT[out]) if residual else None)


def product(p):
    # exact: integers below 2^53 in FP64
    return (p["a"].double().to(DEV) @ p["w"].double().to(DEV).t()).cpu()


def run(cr, p, out, fmt=torch.float16, act=0, y=None, residual="own"):
    M, N = p["a"].shape[0], p["w"].shape[0]
    y = torch.full((M, N), 9.0, dtype=TORCH_DT[out], device=DEV) if y is None else y
    dev = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    cr.gemm_fused(dev["a"].to(fmt), dev["sa"], dev["w"].to(fmt), dev["sw"], y, bias=dev["bias"], act=act,
                  gate=dev["gate"], residual=dev["residual"] if residual == "own" else residual)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    return y


def exact_f32(p, out):
    """No activation: the epilogue's FP32 operations one by one."""
    y = product(p).float() * p["sa"][:, None] * p["sw"]
    if p["bias"] is not None:
        y = y + p["bias"]
    if p["gate"] is not None:
        y = y * p["gate"]
    if p["residual"] is not None:
        y = y + p["residual"].float()
    return y.to(TORCH_DT[out])


def check_act(got, p, act, out):
    lin = product(p) * p["sa"].double()[:, None] * p["sw"].double()
    bias = 0.0 if p["bias"] is None else p["bias"].double()
    gate = 1.0 if p["gate"] is None else p["gate"].double()
    res = torch.zeros(()).double() if p["residual"] is None else p["residual"].double()
    x = lin + bias
    f = {"NONE": x, "RELU": x.clamp(min=0), "SILU": x * torch.sigmoid(x), "GELU": x * torch.special.ndtr(x),
         "GELU_TANH": 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))}[act]
    y = f * gate + res
    size = (lin.abs() + torch.as_tensor(bias).abs()) * torch.as_tensor(gate).abs() + res.abs()
    lim = 3e-6 * size + HALF_ULP[out] * (y.abs() + 3e-6 * size) + (2.0 ** -25 if out == "fp16" else 0)
    err = (got.double().cpu() - y).abs()
    assert torch.all(err <= lim), float((err / lim).max())


SIZES = [(1, 1, 256), (1, 300, 5376), (2, 7, 512), (3, 16, 768), (5, 100, 2304), (8, 257, 1024), (9, 129, 256),
         (15, 64, 1280), (16, 1000, 2048), (17, 33, 512), (24, 300, 1536), (32, 512, 1024), (33, 65, 2560),
         (48, 200, 768), (63, 130, 256), (64, 384, 5376), (65, 40, 256), (100, 700, 512), (128, 256, 1024),
         (130, 257, 2304), (256, 512, 5376), (257, 100, 20480), (300, 1500, 1024), (513, 260, 3584), (700, 513, 256)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,Kp", SIZES)
def test_without_activation_bit_for_bit(cr, M, N, Kp, out):
    p = problem(M, N, Kp, out, M + N + Kp)
    want = exact_f32(p, out)
    assert torch.equal(run(cr, p, out).cpu(), want)
    if M <= cr.FEW_TOKENS:
        assert torch.equal(run(cr, p, out, torch.int8).cpu(), want)
    # residual read from the output itself
    y = p["residual"].to(DEV)
    assert torch.equal(run(cr, p, out, y=y, residual=y).cpu(), want)


@pytest.mark.parametrize("bias,gate,residual", [(False, False, False), (True, False, False), (False, True, False),
                                                (False, False, True)])
@pytest.mark.parametrize("M,N,Kp", [(4, 300, 512), (40, 90, 512), (200, 300, 768)])
def test_each_option_alone(cr, M, N, Kp, bias, gate, residual):
    p = problem(M, N, Kp, "bf16", 5, bias, gate, residual)
    got = run(cr, p, "bf16").cpu()
    assert torch.equal(got, exact_f32(p, "bf16"))
    if not gate and not residual:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        cr.gemm(p["a"].half().to(DEV), p["sa"].to(DEV), p["w"].half().to(DEV), p["sw"].to(DEV), y,
                bias=p["bias"].to(DEV) if bias else None)
        torch.cuda.synchronize()
        assert torch.equal(got, y.cpu())


@pytest.mark.parametrize("M,Kp", [(1, 65536), (16, 5376), (64, 16384), (96, 20480), (300, 65536)])
def test_extreme_codes_stay_exact(cr, M, Kp):
    # all codes 127: partial sums far above 2^24 overall, odd totals from one changed code
    N = 70
    p = problem(M, N, Kp, "fp32", 9, False, False, False, full=True)
    p["a"][:, 5] = 126.0
    p["w"][::2] *= -1
    p["w"][:, 9] = torch.arange(N).float() - 35
    want = exact_f32(p, "fp32")
    assert torch.equal(run(cr, p, "fp32").cpu(), want)
    if M <= cr.FEW_TOKENS:
        assert torch.equal(run(cr, p, "fp32", torch.int8).cpu(), want)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,Kp", [(3, 130, 512), (50, 77, 768), (150, 300, 1024)])
def test_activations(cr, act, out, M, N, Kp):
    p = problem(M, N, Kp, out, 11)
    p["bias"][:4] = torch.tensor([-200.0, 200.0, -20.0, 20.0])      # far ends of the functions
    code = getattr(cr, "ACT_" + act)
    check_act(run(cr, p, out, act=code), p, act, out)
    if M <= cr.FEW_TOKENS:
        check_act(run(cr, p, out, torch.int8, act=code), p, act, out)


@pytest.mark.parametrize("M", [2, 40, 200])
@pytest.mark.parametrize("out,off,pitch,roff,rpitch", [("bf16", 1, 333, 0, 304), ("bf16", 4, 308, 3, 401),
                                                       ("fp32", 1, 301, 2, 306), ("fp16", 0, 302, 4, 304)])
def test_strides_and_neighbours(cr, M, out, off, pitch, roff, rpitch):
    N, Kp = 300, 512
    p = problem(M, N, Kp, out, 21)
    dt = TORCH_DT[out]
    ob = torch.full((off + M * pitch + 8,), 9.0, dtype=dt, device=DEV)
    ov = ob[off:off + M * pitch].view(M, pitch)[:, :N]
    rb = torch.zeros(roff + M * rpitch, dtype=dt, device=DEV)
    rv = rb[roff:].view(M, rpitch)[:, :N]
    rv.copy_(p["residual"])
    a = torch.full((M, Kp + 64), 100.0, dtype=torch.float16, device=DEV)
    w = torch.full((N, Kp + 128), 100.0, dtype=torch.float16, device=DEV)
    a[:, :Kp], w[:, :Kp] = p["a"].to(DEV), p["w"].to(DEV)
    dev = {k: p[k].to(DEV) for k in ("sa", "sw", "bias", "gate")}
    for fmt in [torch.float16] + ([torch.int8] if M <= cr.FEW_TOKENS else []):
        ov.fill_(9.0)
        cr.gemm_fused(a.to(fmt), dev["sa"], w.to(fmt), dev["sw"], ov, K_p=Kp, bias=dev["bias"], gate=dev["gate"], residual=rv)
        torch.cuda.synchronize()
        assert torch.equal(ov.cpu(), exact_f32(p, out))
        ov.fill_(9.0)
        assert torch.all(ob == 9)


@pytest.mark.parametrize("M,fmt,pitch", [(3, torch.int8, 2 ** 30 + 8), (3, torch.float16, 2 ** 30 + 3),
                                         (70, torch.float16, 2 ** 25 + 8), (70, torch.float16, 2 ** 25 + 5)])
def test_offsets_past_32_bits(cr, M, fmt, pitch):
    # output and residual (the same matrix) span more than 2^31 elements; aligned rows and odd ones
    N, Kp = 130, 512
    p = problem(M, N, Kp, "bf16", 51)
    big = torch.empty((M - 1) * pitch + N, dtype=torch.bfloat16, device=DEV)
    y = big.as_strided((M, N), (pitch, 1))
    y.copy_(p["residual"])
    assert torch.equal(run(cr, p, "bf16", fmt, y=y, residual=y).cpu(), exact_f32(p, "bf16"))


def test_many_tiles_and_full_waves(cr):
    # more tiles than CTA pairs, a ragged last strip and column
    p = problem(2305, 2600, 512, "bf16", 31)
    got = run(cr, p, "bf16", act=cr.ACT_NONE).cpu()
    assert torch.equal(got, exact_f32(p, "bf16"))


def test_runs_repeat_bit_for_bit(cr):
    for M in (7, 64, 256, 600):
        p = problem(M, 900, 4096, "bf16", M)
        a = run(cr, p, "bf16", act=cr.ACT_GELU)
        b = run(cr, p, "bf16", act=cr.ACT_GELU)
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,fmt", [(1, torch.int8), (16, torch.float16), (200, torch.float16)])
def test_other_stream_and_graph(cr, M, fmt):
    p = problem(M, 600, 1024, "bf16", 41)
    want = run(cr, p, "bf16", fmt)
    dev = {k: v.to(DEV) for k, v in p.items()}
    a, w = dev["a"].to(fmt), dev["w"].to(fmt)
    y = torch.zeros_like(want)
    kw = dict(bias=dev["bias"], gate=dev["gate"], residual=dev["residual"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cr.gemm_fused(a, dev["sa"], w, dev["sw"], y, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.gemm_fused(a, dev["sa"], w, dev["sw"], y, **kw)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_empty_calls(cr):
    z = lambda *s, **k: torch.empty(*s, device=DEV, **k)
    h = dict(dtype=torch.float16)
    cr.gemm_fused(z(0, 256, **h), z(0), z(8, 256, **h), z(8), z(0, 8))
    cr.gemm_fused(z(3, 256, **h), z(3), z(0, 256, **h), z(0), z(3, 0))
