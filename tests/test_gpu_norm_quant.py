"""rms_norm_quant (residual addition, RMS norm, ConvRot256 rotation, row S8)
against the same formula in 64 bits.

Tolerances.  The kernel's FP32 errors relative to a row's own values: the sum
of squares (chains of at most 64 additions, half of it reaches the factor),
the reciprocal square root (2 ulp), the weight product and eight butterfly
stages (each at most 2^-24 of a partial sum, and partial sums are at most
about four times the row's largest rotated value) stay below 4e-6 together.
The scale is held to that.  A code moves by at most one where its value lies
that near to a half: at a mean code of 30 to 40, below 4e-4 of the codes;
0.999 equal is asked for, and single codes where a case has few.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def cr():
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    return cr


def make(M, K, dtype, seed, residual):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randint(0, K, (max(1, K // 50),), generator=g)] *= 20.0
    r = (2 * torch.randn(M, K, generator=g)).to(TORCH_DT[dtype]) if residual else None
    w = 1 + 0.2 * torch.randn(K, generator=g)
    return x.to(TORCH_DT[dtype]), r, w


def reference(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h64 = h.double().numpy()
    u = h64 / np.sqrt(np.mean(h64 * h64, axis=1, keepdims=True) + eps)
    if w is not None:
        u = u * w.double().numpy()
    K = u.shape[1]
    pad = np.zeros((u.shape[0], oracle.padded_k(K)))
    pad[:, :K] = u
    v = oracle.rotate_blocks(pad)
    s = np.abs(v).max(axis=1) / 127.0
    q = np.zeros_like(v)
    q[s > 0] = np.rint(v[s > 0] / s[s > 0, None])
    return h, q, s


def check(q, s, qr, sr):
    got, ref = q.float().cpu().numpy(), qr
    d = np.abs(got - ref)
    assert d.max(initial=0) <= 1
    assert np.sum(d > 0) <= max(2, 1e-3 * d.size)
    s = s.cpu().numpy().astype(np.float64)
    assert np.all((s == 0) == (sr == 0))
    assert np.all(np.abs(s - sr) <= 4e-6 * sr)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,residual", [
    (1, 1, False), (3, 31, True), (2, 255, False), (5, 256, True), (4, 257, True), (7, 1000, False),
    (33, 5000, True), (64, 5376, True), (3, 16384, False), (2, 16385, True), (3, 20480, True), (2, 32768, False),
    (2, 33025, True), (1, 65536, False)])
def test_against_64_bits(cr, dtype, M, K, residual):
    x, r, w = make(M, K, dtype, 7 * M + K, residual)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)
    Kp = cr.padded_k(K)
    for fmt in (torch.float16, torch.int8):
        q = torch.full((M, Kp), 99, dtype=fmt, device=DEV)
        s = torch.full((M,), -1.0, device=DEV)
        h = torch.zeros(M, K, dtype=x.dtype, device=DEV)
        n = torch.empty(M, device=DEV)
        cr.rms_norm_quant(x.to(DEV), K, q, s, residual=None if r is None else r.to(DEV), h=h, weight=w.to(DEV), a_norm=n)
        torch.cuda.synchronize()
        check(q, s, q_ref, s_ref)
        assert torch.equal(h.cpu(), h_ref)
        true = q.double().norm(dim=1)
        assert torch.all(n.double() >= true)
        assert torch.all(n.double() <= 1.002 * true + 1.01 * Kp ** 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("off,pitch", [(0, 640), (1, 603), (8, 608), (3, 600)])
def test_strided_rows_and_neighbours(cr, dtype, off, pitch):
    # rows inside wider buffers, aligned and not; what lies beside them is not touched
    M, K, Kp = 9, 590, 768
    x, r, w = make(M, K, dtype, off + pitch, True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-5)

    def wide(t):
        b = torch.full((M * pitch + 32,), 5.0, dtype=t.dtype, device=DEV)
        v = b[off:off + M * pitch].view(M, pitch)[:, :K]
        v.copy_(t)
        return b, v
    (_, xv), (_, rv), (hb, hv) = wide(x), wide(r), wide(torch.zeros_like(x))
    hv.fill_(5.0)
    qb = torch.full((M, Kp + 6), 77.0, dtype=torch.float16, device=DEV)
    s = torch.empty(M, device=DEV)
    cr.rms_norm_quant(xv, K, qb[:, :Kp], s, residual=rv, h=hv, weight=w.to(DEV), eps=1e-5)
    torch.cuda.synchronize()
    check(qb[:, :Kp], s, q_ref, s_ref)
    assert torch.equal(hv.cpu(), h_ref)
    assert torch.all(qb[:, Kp:] == 77)
    hv.fill_(5.0)
    assert torch.all(hb == 5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [590, 5001, 20483, 33025])
@pytest.mark.parametrize("starts,pads", [((0, 1, 3), (0, 0, 0)), ((5, 5, 5), (1, 9, 17)), ((2, 2, 2), (0, 3, 0)),
                                         ((8, 0, 16), (8, 16, 0))])
def test_operands_that_lie_differently(cr, dtype, K, starts, pads):
    # x, residual and h each with its own start and pitch; one-byte codes from an odd multiple of two
    M, Kp = 6, cr.padded_k(K)
    x, r, w = make(M, K, dtype, K + starts[1] + pads[1], True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)

    def wide(t, start, pad):
        b = torch.full((start + M * (K + pad) + 8,), 5.0, dtype=t.dtype, device=DEV)
        v = b[start:start + M * (K + pad)].view(M, K + pad)[:, :K]
        v.copy_(t)
        return b, v
    (_, xv), (_, rv), (hb, hv) = (wide(t, a, b) for t, a, b in zip((x, r, torch.full_like(x, 5.0)), starts, pads))
    qb = torch.full((M, Kp + 10), 77, dtype=torch.int8, device=DEV)
    s = torch.empty(M, device=DEV)
    cr.rms_norm_quant(xv, K, qb[:, 2:2 + Kp], s, residual=rv, h=hv, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(qb[:, 2:2 + Kp], s, q_ref, s_ref)
    assert torch.equal(hv.cpu(), h_ref)
    assert torch.all(qb[:, :2] == 77) and torch.all(qb[:, 2 + Kp:] == 77)
    hv.fill_(5.0)
    assert torch.all(hb == 5)


@pytest.mark.parametrize("K", [1001, 5377, 20483, 40001])
def test_in_place_odd_widths(cr, K):
    # vectors that two rows, or two CTAs of a row, share
    M = 50
    x, r, w = make(M, K, "bf16", K, True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)
    xd = x.to(DEV)
    q = torch.empty(M, cr.padded_k(K), dtype=torch.float16, device=DEV)
    s = torch.empty(M, device=DEV)
    cr.rms_norm_quant(xd, K, q, s, residual=r.to(DEV), h=xd, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, s, q_ref, s_ref)
    assert torch.equal(xd.cpu(), h_ref)


@pytest.mark.parametrize("M,K", [(700, 512), (700, 768), (700, 1024), (700, 333), (400, 40000)])
def test_many_rows(cr, M, K):
    x, r, w = make(M, K, "bf16", M + K, True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)
    q = torch.empty(M, cr.padded_k(K), dtype=torch.float16, device=DEV)
    s = torch.empty(M, device=DEV)
    h = torch.empty_like(x, device=DEV)
    cr.rms_norm_quant(x.to(DEV), K, q, s, residual=r.to(DEV), h=h, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, s, q_ref, s_ref)
    assert torch.equal(h.cpu(), h_ref)


@pytest.mark.parametrize("K", [1000, 5376, 20480])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(cr, which, K):
    M = 50
    x, r, w = make(M, K, "bf16", K, True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)
    xd, rd = x.to(DEV), r.to(DEV)
    q = torch.empty(M, cr.padded_k(K), dtype=torch.float16, device=DEV)
    s = torch.empty(M, device=DEV)
    cr.rms_norm_quant(xd, K, q, s, residual=rd, h=xd if which == "x" else rd, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, s, q_ref, s_ref)
    assert torch.equal((xd if which == "x" else rd).cpu(), h_ref)


def test_zero_tiny_and_large_rows(cr):
    K = 600
    x, _, w = make(8, K, "fp32", 3, False)
    x[0] = 0.0
    x[1] *= 1e-30              # the squares vanish beside eps
    x[2] *= 1e-5
    x[3] *= 1e12
    x[4] = 0.0
    x[4, 17] = -3.0            # a single value: every code of its block is +-127
    h_ref, q_ref, s_ref = reference(x, None, w, 1e-6)
    q = torch.empty(8, 768, dtype=torch.float16, device=DEV)
    s = torch.empty(8, device=DEV)
    cr.rms_norm_quant(x.to(DEV), K, q, s, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, s, q_ref, s_ref)
    assert float(s[0]) == 0 and torch.all(q[0] == 0)
    assert torch.all(q[4, :256].abs() == 127) and torch.all(q[4, 256:] == 0)


def test_residual_that_cancels_leaves_zero_codes(cr):
    x, _, w = make(3, 512, "bf16", 4, False)
    q = torch.full((3, 512), 9.0, dtype=torch.float16, device=DEV)
    s = torch.full((3,), 9.0, device=DEV)
    cr.rms_norm_quant(x.to(DEV), 512, q, s, residual=(-x).to(DEV), weight=w.to(DEV))
    torch.cuda.synchronize()
    assert torch.all(q == 0) and torch.all(s == 0)


def test_without_weight_and_a_bad_row_leaves_the_others(cr):
    M, K = 6, 1024
    x, _, _ = make(M, K, "fp16", 5, False)
    _, q_ref, s_ref = reference(x, None, None, 1e-6)
    bad = x.clone()
    bad[2, 5], bad[4, 9] = float("nan"), float("inf")
    q = torch.empty(M, K, dtype=torch.float16, device=DEV)
    s = torch.empty(M, device=DEV)
    cr.rms_norm_quant(bad.to(DEV), K, q, s)
    torch.cuda.synchronize()
    good = [0, 1, 3, 5]
    check(q[good], s[good], q_ref[good], s_ref[good])


def test_matches_quant_act_on_a_unit_norm_row(cr):
    # mean square 1 and a vanishing eps: the norm changes nothing, and the codes are the layer's own
    K = 2048
    x = torch.where(torch.rand(16, K, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0)
    qa, qb = (torch.empty(16, K, dtype=torch.int8, device=DEV) for _ in range(2))
    sa, sb = (torch.empty(16, device=DEV) for _ in range(2))
    cr.rms_norm_quant(x.to(DEV), K, qa, sa, eps=1e-30)
    cr.quant_act(x.to(DEV), K, qb, sb)
    torch.cuda.synchronize()
    assert torch.equal(qa, qb) and torch.equal(sa, sb)


def test_other_stream_and_graph(cr):
    M, K = 20, 5376
    x, r, w = make(M, K, "bf16", 6, True)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    q, q2 = (torch.empty(M, K, dtype=torch.float16, device=DEV) for _ in range(2))
    s, s2 = (torch.empty(M, device=DEV) for _ in range(2))
    cr.rms_norm_quant(xd, K, q, s, residual=rd, weight=wd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cr.rms_norm_quant(xd, K, q2, s2, residual=rd, weight=wd, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.rms_norm_quant(xd, K, q2, s2, residual=rd, weight=wd)
    q2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_offsets_past_32_bits(cr):
    # two rows more than 2^31 elements apart
    K, pitch = 1000, 2 ** 31 + 24
    x, r, w = make(2, K, "bf16", 9, True)
    h_ref, q_ref, s_ref = reference(x, r, w, 1e-6)
    big = torch.empty(pitch + K, dtype=torch.bfloat16, device=DEV)
    xv = big.as_strided((2, K), (pitch, 1))
    xv.copy_(x)
    q = torch.empty(2, 1024, dtype=torch.float16, device=DEV)
    s = torch.empty(2, device=DEV)
    cr.rms_norm_quant(xv, K, q, s, residual=r.to(DEV), h=xv, weight=w.to(DEV))
    torch.cuda.synchronize()
    check(q, s, q_ref, s_ref)
    assert torch.equal(xv.cpu(), h_ref)


def test_empty_call(cr):
    x = torch.empty(0, 300, device=DEV)
    cr.rms_norm_quant(x, 300, torch.empty(0, 512, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV))
