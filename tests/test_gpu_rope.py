"""qk_norm_rope (per-head RMS norm and rotary positions with several axes)
against the formula in 64 bits.

Tolerances.  FP32 errors relative to the pair's length: the angle (a 24-bit
fraction of half a turn: 2e-7 radians), sine and cosine (2^-23), three
products and a sum (2^-24 each), the norm's factor (5e-7) stay below 2e-6
together.  The output's own rounding adds half a unit in the last place.
"""
import math

import pytest
import torch

from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
SMALLEST = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}


@pytest.fixture(scope="module")
def cr():
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    return cr


def reference(x, w, pos, pairs, theta, eps, interleaved):
    """x [M, H, D] on the CPU; returns the 64-bit result and each value's pair length."""
    u = x.double()
    if w is not None:
        u = u / (u.square().mean(2, keepdim=True) + eps).sqrt() * w.double()
    P = sum(pairs)
    y, size = u.clone(), u.abs().clone()
    i = 0
    for a, n in enumerate(pairs):
        for j in range(n):
            phi = pos[:, a].double() * theta ** (-j / n)
            c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
            e, o = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
            ue, uo = u[:, :, e], u[:, :, o]
            y[:, :, e], y[:, :, o] = ue * c - uo * s, uo * c + ue * s
            size[:, :, e] = size[:, :, o] = torch.hypot(ue, uo)
            i += 1
    return y, size


def check(got, ref, dtype):
    y, size = ref
    err = (got.double().cpu() - y).abs()
    lim = 2e-6 * size + HALF_ULP[dtype] * (y.abs() + 2e-6 * size) + SMALLEST[dtype]
    assert torch.all(err <= lim), float((err / lim.clamp_min(1e-300)).max())


CASES = [  # M, heads q, heads k, D, pairs of each axis, interleaved, norm
    (1, 1, 1, 2, [1], False, True),
    (3, 2, 1, 6, [1, 1], True, True),
    (17, 5, 5, 64, [32], False, False),
    (9, 56, 56, 128, [16, 24, 24], False, True),
    (9, 56, 56, 128, [16, 24, 24], True, True),
    (33, 32, 8, 96, [20, 20], True, False),
    (12, 7, 1, 96, [8, 0, 40], False, True),
    (5, 4, 4, 80, [20, 20], False, True),
    (5, 4, 4, 80, [10, 10], True, True),
    (4, 3, 3, 128, [16, 16], False, True),          # half of the head turns
    (4, 3, 2, 128, [16, 16], True, False),
    (4, 6, 3, 256, [32, 32, 32, 32], False, True),
    (6, 3, 3, 72, [12, 12, 12], False, True),
    (6, 3, 3, 67, [15, 7], True, True),             # odd width, a value left over
    (130, 2, 2, 128, [64], False, True),
    (2, 2, 1, 1024, [200, 312], False, True),
    (3, 4, 2, 48, [24], False, True),
    (3, 2, 2, 64, [0], False, True),                # the norm alone
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,Hq,Hk,D,pairs,interleaved,norm", CASES)
def test_against_64_bits(cr, dtype, M, Hq, Hk, D, pairs, interleaved, norm):
    g = torch.Generator().manual_seed(M + 3 * D + Hq)
    dt = TORCH_DT[dtype]
    qkv = torch.randn(M, (Hq + 2 * Hk) * D, generator=g).to(dt)
    pos = torch.randint(0, 4000, (M, len(pairs)), generator=g, dtype=torch.int32)
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g) if norm else None for _ in range(2))
    freq = cr.rope_inv_freq(pairs, 10000.0)
    dev = qkv.to(DEV)
    q = dev[:, :Hq * D].unflatten(1, (Hq, D))
    k = dev[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    qo = torch.full((M, Hq, D), 7.0, dtype=dt, device=DEV)
    ko = torch.full((M, Hk, D), 7.0, dtype=dt, device=DEV)
    args = dict(q_weight=None if wq is None else wq.to(DEV), k_weight=None if wk is None else wk.to(DEV),
                eps=1e-6, interleaved=interleaved)
    fd = torch.tensor(freq, dtype=torch.float64, device=DEV)
    cr.qk_norm_rope(q, k, pos.to(DEV), fd, pairs, qo, ko, **args)
    torch.cuda.synchronize()
    ref_q = reference(qkv[:, :Hq * D].unflatten(1, (Hq, D)), wq, pos, pairs, 10000.0, 1e-6, interleaved)
    ref_k = reference(qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)), wk, pos, pairs, 10000.0, 1e-6, interleaved)
    check(qo, ref_q, dtype)
    check(ko, ref_k, dtype)
    assert torch.equal(dev.cpu(), qkv)
    # in place, in the packed buffer: v stays
    cr.qk_norm_rope(q, k, pos.to(DEV), fd, pairs, q, k, **args)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(dev[:, (Hq + Hk) * D:].cpu(), qkv[:, (Hq + Hk) * D:])


@pytest.mark.parametrize("off,head,tok", [(0, 128, 1024), (1, 130, 1027), (8, 136, 1040), (4, 132, 1060), (0, 1000, 128)])
def test_strides_and_alignment(cr, off, head, tok):
    # heads and tokens apart, at odd places, and head-major storage ([H, M, D]: tok < head)
    M, H, D, pairs = 7, 6, 128, [20, 22, 22]
    g = torch.Generator().manual_seed(off + head)
    n = off + (M - 1) * tok + (H - 1) * head + D + 64
    buf = torch.randn(n, generator=g).to(torch.bfloat16).to(DEV)
    q = buf.as_strided((M, H, D), (tok, head, 1), off)
    out = torch.full((n,), 3.0, dtype=torch.bfloat16, device=DEV)
    qo = out.as_strided((M, H, D), (tok, head, 1), off)
    pos = torch.randint(-50, 50, (M, 5), generator=g, dtype=torch.int32)
    w = 1 + 0.3 * torch.randn(D, generator=g)
    fd = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    cr.qk_norm_rope(q, None, pos.to(DEV)[:, 1:4], fd, pairs, qo, None, q_weight=w.to(DEV))
    torch.cuda.synchronize()
    check(qo, reference(q.cpu(), w, pos[:, 1:4], pairs, 10000.0, 1e-6, False), "bf16")
    qo.fill_(3.0)
    assert torch.all(out == 3)


def test_offsets_past_32_bits(cr):
    M, H, D, pairs, tok = 2, 3, 128, [64], 2 ** 31 + 512
    g = torch.Generator().manual_seed(8)
    x = torch.randn(M, H, D, generator=g).to(torch.bfloat16)
    buf = torch.empty(tok + H * D, dtype=torch.bfloat16, device=DEV)
    q = buf.as_strided((M, H, D), (tok, D, 1))
    q.copy_(x)
    pos = torch.tensor([[3], [11]], dtype=torch.int32)
    fd = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    w = 1 + 0.3 * torch.randn(D, generator=g)
    cr.qk_norm_rope(q, None, pos.to(DEV), fd, pairs, q, None, q_weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, reference(x, w, pos, pairs, 10000.0, 1e-6, False), "bf16")


def test_large_and_negative_positions(cr):
    # FP32 products of position and frequency would be off by up to 60 radians here
    D, pairs = 64, [16, 16]
    pos = torch.tensor([[0, 0], [1, -1], [131071, -131072], [2 ** 30, -2 ** 30], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    x = torch.randn(5, 3, D, generator=torch.Generator().manual_seed(2))
    out = torch.empty(5, 3, D, device=DEV)
    fd = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    cr.qk_norm_rope(x.to(DEV), None, pos.to(DEV), fd, pairs, out, None)
    torch.cuda.synchronize()
    # the reference's own angle, one rounding of a 64-bit product, is off by 2^31 * 2^-53 = 2.4e-7
    y, size = reference(x, None, pos, pairs, 10000.0, 1e-6, False)
    check(out, (y, 1.25 * size), "fp32")


def test_position_zero_is_the_identity_and_lengths_are_kept(cr):
    D = 128
    x = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(3)).to(DEV)
    out = torch.empty_like(x)
    fd = torch.tensor(cr.rope_inv_freq([64]), dtype=torch.float64, device=DEV)
    cr.qk_norm_rope(x, None, torch.zeros(4, 1, dtype=torch.int32, device=DEV), fd, [64], out, None)
    torch.cuda.synchronize()
    assert torch.equal(out, x)
    pos = torch.tensor([[3], [70], [500], [9999]], dtype=torch.int32, device=DEV)
    cr.qk_norm_rope(x, None, pos, fd, [64], out, None)
    torch.cuda.synchronize()
    assert torch.allclose(out.double().norm(dim=2), x.double().norm(dim=2), rtol=4e-6)


def test_scores_depend_on_relative_positions(cr):
    # <rope(q, a), rope(k, b)> is a function of a - b, axis by axis
    D, pairs = 96, [16, 16, 16]
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(1, 1, D, generator=g).expand(2, 1, D).contiguous().to(DEV) for _ in range(2))
    a = torch.tensor([[5, 9, 2], [105, 59, 32]], dtype=torch.int32, device=DEV)
    b = torch.tensor([[1, 4, 30], [101, 54, 60]], dtype=torch.int32, device=DEV)
    fd = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    cr.qk_norm_rope(q, None, a, fd, pairs, qo, None)
    cr.qk_norm_rope(k, None, b, fd, pairs, ko, None)
    torch.cuda.synchronize()
    s = (qo.double() * ko.double()).sum(2).flatten()
    assert abs(float(s[0] - s[1])) <= 2 * 2e-6 * float(q.double().norm() * k.double().norm())


def test_zero_head_and_bad_values(cr):
    D = 128
    x = torch.randn(3, 2, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[0, 0] = 0
    x[1, 1, 7] = float("inf")
    x[2, 0, 3] = float("nan")
    w = torch.ones(D, device=DEV)
    out = torch.empty(3, 2, D, dtype=torch.bfloat16, device=DEV)
    pos = torch.ones(3, 1, dtype=torch.int32, device=DEV)
    fd = torch.tensor(cr.rope_inv_freq([64]), dtype=torch.float64, device=DEV)
    cr.qk_norm_rope(x.to(DEV), None, pos, fd, [64], out, None, q_weight=w)
    torch.cuda.synchronize()
    assert torch.all(out[0, 0] == 0)
    ref = reference(x, w.cpu(), pos.cpu(), [64], 10000.0, 1e-6, False)
    for m, h in ((0, 1), (1, 0), (2, 1)):
        check(out[m:m + 1, h:h + 1], tuple(t[m:m + 1, h:h + 1] for t in ref), "bf16")


def test_other_stream_and_graph(cr):
    M, H, D, pairs = 40, 8, 128, [16, 24, 24]
    x = torch.randn(M, H, D, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    pos = torch.arange(3 * M, dtype=torch.int32, device=DEV).view(M, 3)
    fd = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    cr.qk_norm_rope(x, None, pos, fd, pairs, a, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cr.qk_norm_rope(x, None, pos, fd, pairs, b, None, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.qk_norm_rope(x, None, pos, fd, pairs, b, None)
    b.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_frequencies(cr):
    got = cr.rope_inv_freq([3, 0, 2], 500.0)
    want = [500.0 ** (-j / 3) for j in range(3)] + [500.0 ** (-j / 2) for j in range(2)]
    assert len(got) == 5 and all(math.isclose(a, b, rel_tol=1e-15) for a, b in zip(got, want))
