"""rms_norm_quant, qk_norm_rope and gemm_fused in a row on shared buffers, each launched while the one before it still
runs: a captured chain has to give what the same calls give with a synchronisation after each.  Every step reads what
the step before has just written (codes, scales, the stream, channel gates and norm weights that a one-token product
computes) and overwrites what earlier steps read; the results are exact functions of their inputs, so they are equal
bit for bit."""
import math

import pytest
import torch

from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

LAYERS, D, PAIRS = 12, 64, [8, 12, 12]


class Chain:
    def __init__(self, cr, M, K, fmt, dt):
        g = torch.Generator(device=DEV).manual_seed(M + K)
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
        codes = lambda n: (40 * rand(n, K)).round().clamp(-127, 127)
        self.cr, self.M, self.K = cr, M, K
        self.start = rand(M, K).to(dt)
        self.stream = self.start.clone()
        self.w = [codes(K).to(fmt) for _ in range(3)]
        self.sw = [(0.5 + torch.rand(K, generator=g, device=DEV)) / (40 * math.sqrt(K)) for _ in range(3)]
        self.aq = torch.empty(M, K, dtype=fmt, device=DEV)
        self.sa = torch.empty(M, device=DEV)
        self.y = torch.empty(M, K, dtype=dt, device=DEV)
        # one token's codes, from which the channel vectors come
        self.cond = [(codes(1).to(fmt), 0.02 * (1 + i) * torch.ones(1, device=DEV)) for i in range(3)]
        self.vec = torch.empty(1, K, device=DEV)
        self.norm = torch.empty(K, device=DEV)
        self.pos = torch.randint(-500, 500, (M, 3), generator=g, device=DEV, dtype=torch.int32)
        self.freq = torch.tensor(cr.rope_inv_freq(PAIRS), dtype=torch.float64, device=DEV)
        self.qw = 1 + 0.1 * rand(D)

    def run(self, after=lambda: None):
        cr, M, K = self.cr, self.M, self.K
        self.stream.copy_(self.start)
        after()
        for i in range(LAYERS):
            c, s = self.cond[i % 3]
            w, sw = self.w[i % 3], self.sw[i % 3]
            cr.gemm_fused(c, s, w, sw, self.vec, act=cr.ACT_SILU)                        # the layer's channel vector
            after()
            cr.rms_norm_quant(self.stream, K, self.aq, self.sa, weight=self.vec[0])      # read by the norm,
            after()
            cr.gemm_fused(self.aq, self.sa, w, sw, self.y, bias=self.vec[0])             # as the bias,
            after()
            q = self.y.view(M, K // D, D)
            cr.qk_norm_rope(q, None, self.pos, self.freq, PAIRS, q, None, q_weight=self.qw)
            after()
            cr.rms_norm_quant(self.y, K, self.aq, self.sa)
            after()
            cr.gemm_fused(self.aq, self.sa, w, sw, self.stream, gate=self.vec[0], residual=self.stream)   # and the gate
            after()
        return self.stream


@pytest.mark.parametrize("M,K,fmt,dt", [
    (1, 512, torch.int8, torch.bfloat16), (5, 1024, torch.float16, torch.float16), (40, 512, torch.int8, torch.float32),
    (40, 512, torch.float16, torch.bfloat16), (200, 512, torch.float16, torch.bfloat16),
    (700, 768, torch.float16, torch.bfloat16), (300, 5376, torch.float16, torch.bfloat16)])
def test_chain_equals_synchronised_calls(M, K, fmt, dt):
    ensure_built()
    import rotated_w4a8_int8_gb300 as cr
    c = Chain(cr, M, K, fmt, dt)
    want = c.run(torch.cuda.synchronize).clone()
    assert bool(torch.isfinite(want.float()).all()) and not torch.equal(want, c.start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.stream, want)
    for _ in range(3):
        graph.replay()                               # and back to back
    torch.cuda.synchronize()
    assert torch.equal(c.stream, want)
    assert cr.device_error() == 0
