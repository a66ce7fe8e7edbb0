"""rms_norm_quant and qk_norm_rope with many rows: CTAs that hold several tokens (rotary, from 1824 and 7296 tokens on)
or several short rows (the norm, from 153 rows on), in every type, with the last CTA part full.  Tolerances are those
of test_gpu_rope.py and test_gpu_norm_quant.py."""
import pytest
import torch

import test_gpu_norm_quant as norm
import test_gpu_rope as rope
from gpu_util import DEV, TORCH_DT, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def cr():
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    return cr


# one, two and four tokens per CTA, with every remainder
@pytest.mark.parametrize("M", [1823, 1824, 1825, 7295, 7296, 7297, 7298, 7299])
@pytest.mark.parametrize("dtype,D,Hq,Hk,pairs,interleaved,normed", [
    ("bf16", 128, 3, 2, [16, 24, 24], False, True),          # runs of eight
    ("fp16", 64, 5, 1, [8, 8], True, True),
    ("fp32", 96, 2, 2, [20, 28], False, False),              # runs of four
    ("bf16", 24, 9, 3, [4, 8], True, True),
    ("fp16", 14, 2, 1, [3, 2], False, True),                 # single elements
])
def test_rotary(cr, M, dtype, D, Hq, Hk, pairs, interleaved, normed):
    g = torch.Generator().manual_seed(M + D)
    q = torch.randn(M, Hq, D, generator=g).to(TORCH_DT[dtype])
    k = torch.randn(M, Hk, D, generator=g).to(TORCH_DT[dtype])
    pos = torch.stack([torch.randperm(M, generator=g) - M // 2 for _ in pairs], 1).to(torch.int32)   # no two alike
    w = [(1 + 0.2 * torch.randn(D, generator=g)) if normed else None for _ in range(2)]
    freq = torch.tensor(cr.rope_inv_freq(pairs), dtype=torch.float64, device=DEV)
    yq, yk = torch.empty(M, Hq, D, dtype=q.dtype, device=DEV), torch.empty(M, Hk, D, dtype=q.dtype, device=DEV)
    cr.qk_norm_rope(q.to(DEV), k.to(DEV), pos.to(DEV), freq, pairs, yq, yk,
                    q_weight=None if w[0] is None else w[0].to(DEV), k_weight=None if w[1] is None else w[1].to(DEV),
                    interleaved=interleaved)
    torch.cuda.synchronize()
    rope.check(yq, rope.reference(q, w[0], pos, pairs, 10000.0, 1e-6, interleaved), dtype)
    rope.check(yk, rope.reference(k, w[1], pos, pairs, 10000.0, 1e-6, interleaved), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", [(153, 256), (700, 200), (701, 512), (163, 333), (407, 768), (402, 600), (509, 1024), (305, 1001)])
def test_short_rows(cr, dtype, residual, M, K):
    x, r, w = norm.make(M, K, dtype, M + K, residual)
    h_ref, q_ref, s_ref = norm.reference(x, r, w, 1e-6)
    for fmt in (torch.float16, torch.int8):
        q = torch.full((M, cr.padded_k(K)), 99, dtype=fmt, device=DEV)
        s = torch.full((M,), -1.0, device=DEV)
        h = torch.zeros(M, K, dtype=x.dtype, device=DEV)
        n = torch.empty(M, device=DEV)
        cr.rms_norm_quant(x.to(DEV), K, q, s, residual=None if r is None else r.to(DEV), h=h, weight=w.to(DEV), a_norm=n)
        torch.cuda.synchronize()
        norm.check(q, s, q_ref, s_ref)
        assert torch.equal(h.cpu(), h_ref)
        true = q.double().norm(dim=1)
        assert torch.all(n.double() >= true) and torch.all(n.double() <= 1.002 * true + 1.01 * cr.padded_k(K) ** 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(160, 1280), (310, 1281), (320, 5376), (306, 20480), (153, 40000)])
def test_longer_rows_without_residual(cr, dtype, M, K):
    x, _, w = norm.make(M, K, dtype, M + K, False)
    _, q_ref, s_ref = norm.reference(x, None, w, 1e-6)
    q, s = torch.empty(M, cr.padded_k(K), dtype=torch.float16, device=DEV), torch.empty(M, device=DEV)
    cr.rms_norm_quant(x.to(DEV), K, q, s, weight=w.to(DEV))
    torch.cuda.synchronize()
    norm.check(q, s, q_ref, s_ref)
