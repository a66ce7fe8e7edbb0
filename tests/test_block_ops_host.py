"""Host-side refusals of rms_norm_quant, qk_norm_rope and gemm_fused: every
bad argument is turned away before anything reaches the GPU."""
import ctypes
import math

import pytest
import torch

import rotated_w4a8_int8_gb300 as cr

P = 1 << 20        # fake address, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return cr.load_library()


def test_rms_norm_quant_rejects_bad_arguments(lib):
    ok = dict(x=P, dt=0, ldx=512, r=P, ldr=512, h=P, ldh=512, w=P, eps=1e-6, M=4, K=512, q=P, fmt=1, ldq=512, s=P, n=None)

    def call(**kw):
        a = {**ok, **kw}
        return lib.convrot_rms_norm_quant(a["x"], a["dt"], a["ldx"], a["r"], a["ldr"], a["h"], a["ldh"], a["w"], a["eps"],
                                          a["M"], a["K"], a["q"], a["fmt"], a["ldq"], a["s"], a["n"], None)
    assert call(K=0) == 1 and call(M=-1) == 1
    assert call(dt=5) == 3 and call(fmt=2) == 3
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == 1
    assert call(ldx=511) == 1 and call(ldr=511) == 1 and call(ldh=511) == 1
    assert call(K=300, ldq=511) == 1                                  # ld_aq < K_p
    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1
    assert call(x=P + 1) == 2 and call(r=P + 1) == 2 and call(h=P + 1) == 2
    assert call(dt=2, r=P + 2) == 2
    assert call(q=P + 2) == 2 and call(ldq=513) == 2 and call(fmt=0, q=P + 1) == 2
    assert call(w=P + 4) == 2 and call(s=P + 2) == 2 and call(n=P + 2) == 2
    big = dict(ldx=1 << 30, ldr=1 << 30, ldh=1 << 30, ldq=1 << 31)
    assert call(K=65537, **big) == 3 and call(K=(1 << 30) - 1, **big) == 3
    assert call(M=0) == 0


def test_qk_norm_rope_rejects_bad_arguments(lib):
    def pairs(*n):
        return (ctypes.c_int * len(n))(*n)
    ok = dict(q=P, qt=1024, qh=128, qo=P, qot=1024, qoh=128, hq=8, qw=P, k=P, kt=256, kh=128, ko=P, kot=256, koh=128, hk=2,
              kw=None, dt=0, M=5, D=128, pos=P, ldp=3, ap=pairs(16, 24, 24), na=3, f=P, eps=1e-6, il=0)

    def call(**kw):
        a = {**ok, **kw}
        return lib.convrot_qk_norm_rope(*[a[n] for n in ("q", "qt", "qh", "qo", "qot", "qoh", "hq", "qw", "k", "kt", "kh",
                                                         "ko", "kot", "koh", "hk", "kw", "dt", "M", "D", "pos", "ldp", "ap",
                                                         "na", "f", "eps", "il")], None)
    assert call(dt=3) == 3
    assert call(M=-1) == 1 and call(D=0) == 1 and call(hq=-1) == 1 and call(hk=-1) == 1
    assert call(D=1025) == 3
    assert call(ap=pairs(16, 24, 25)) == 1                            # 2P > D
    assert call(ap=pairs(16, -1, 24)) == 1
    assert call(ap=pairs(2 ** 30, 2 ** 30, 2 ** 30)) == 3             # the sum does not wrap
    assert call(ap=None) == 1 and call(na=0) == 1 and call(na=5, ap=pairs(1, 1, 1, 1, 1), ldp=5) == 1
    assert call(ldp=2) == 1
    assert call(q=None) == 1 and call(qo=None) == 1 and call(k=None) == 1 and call(ko=None) == 1
    assert call(pos=None) == 1 and call(f=None) == 1
    assert call(qt=-1) == 1 and call(qh=-128) == 1
    assert call(qoh=127) == 1                                         # heads of the output overlap
    assert call(qot=1023) == 1                                        # tokens of the output overlap
    assert call(q=P + 1) == 2 and call(ko=P + 1) == 2 and call(qw=P + 2) == 2
    assert call(pos=P + 2) == 2 and call(f=P + 4) == 2
    assert call(eps=0.0) == 1 and call(eps=float("nan")) == 1
    assert call(M=0) == 0 and call(hq=0, hk=0) == 0


def test_rope_inv_freq_rejects_bad_arguments(lib):
    out = (ctypes.c_double * 4)()
    two = (ctypes.c_int * 2)(2, 2)
    f = lib.convrot_rope_inv_freq
    assert f(two, 2, 1e4, out) == 0 and out[0] == 1.0 and out[2] == 1.0 and out[1] == pytest.approx(0.01)
    assert f(two, 0, 1e4, out) == 1 and f(two, 5, 1e4, out) == 1 and f(None, 2, 1e4, out) == 1
    assert f(two, 2, 0.0, out) == 1 and f(two, 2, float("nan"), out) == 1 and f(two, 2, float("inf"), out) == 1
    assert f(two, 2, 1e4, None) == 1
    assert f((ctypes.c_int * 1)(-1), 1, 1e4, out) == 1 and f((ctypes.c_int * 1)(513), 1, 1e4, out) == 3


def test_gemm_fused_rejects_bad_arguments(lib):
    ok = dict(a=P, lda=512, sa=P, w=P, ldw=512, sw=P, fmt=1, b=P, act=0, g=P, r=P, ldr=8, M=4, N=8, K=512, o=P, dt=0, ldo=8)

    def call(**kw):
        a = {**ok, **kw}
        return lib.convrot_gemm_fused(a["a"], a["lda"], a["sa"], a["w"], a["ldw"], a["sw"], a["fmt"], a["b"], a["act"],
                                      a["g"], a["r"], a["ldr"], a["M"], a["N"], a["K"], a["o"], a["dt"], a["ldo"], None)
    assert call(K=500) == 1 and call(K=0) == 1 and call(M=-1) == 1 and call(N=-1) == 1
    assert call(K=65536 + 256, lda=70000, ldw=70000) == 3
    assert call(dt=3) == 3 and call(fmt=2) == 3 and call(act=5) == 3 and call(act=-1) == 3
    assert call(lda=256) == 1 and call(ldw=256) == 1 and call(ldo=7) == 1 and call(ldr=7) == 1
    assert call(fmt=0, M=65) == 3                                     # one-byte codes: few tokens only
    for name in ("a", "w", "sa", "sw", "o"):
        assert call(**{name: None}) == 1
    assert call(a=P + 8) == 2 and call(w=P + 8) == 2 and call(lda=516) == 2 and call(ldw=516) == 2
    assert call(fmt=0, lda=520) == 2
    assert call(o=P + 1) == 2 and call(r=P + 1) == 2 and call(sa=P + 2) == 2
    assert call(sw=P + 4) == 2 and call(b=P + 4) == 2 and call(g=P + 4) == 2
    assert call(M=0) == 0 and call(N=0, ldo=0, ldr=0) == 0


def test_binding_refuses_wrong_tensors(lib):
    f32, f16, i32 = torch.float32, torch.float16, torch.int32
    s4 = _Fake((4,), f32)
    x, q = _Fake((4, 300), f32), _Fake((4, 512), f16)
    for bad in (_Fake((4, 299), f32), _Fake((3, 300), f32), _Fake((4, 300), f32, (1, 4)), _Fake((4, 300), f16),
                _Fake((4, 300), f32, cuda=False), _Fake((300,), f32)):
        with pytest.raises(ValueError, match="residual must be"):
            cr.rms_norm_quant(x, 300, q, s4, residual=bad)
    with pytest.raises(ValueError, match="a_scale must be"):
        cr.rms_norm_quant(x, 300, q, _Fake((5,), f32))
    with pytest.raises(ValueError, match="a_q must be"):
        cr.rms_norm_quant(x, 300, _Fake((4, 512), f32), s4)
    with pytest.raises(ValueError, match="w_q must be"):          # one kind of codes for both operands
        cr.gemm_fused(_Fake((4, 256), f16), s4, _Fake((8, 256), torch.int8), _Fake((8,), f32), _Fake((4, 8), f32))
    with pytest.raises(ValueError, match="bias must be"):
        cr.gemm_fused(_Fake((4, 256), f16), s4, _Fake((8, 256), f16), _Fake((8,), f32), _Fake((4, 8), f32),
                      bias=_Fake((8,), f16))
    pos, freq = _Fake((4, 1), i32), _Fake((4,), torch.float64)
    h = _Fake((4, 2, 8), f16)
    with pytest.raises(ValueError, match="q_out must be"):
        cr.qk_norm_rope(h, None, pos, freq, [4], _Fake((4, 2, 9), f16), None)
    with pytest.raises(ValueError, match="pos must be"):
        cr.qk_norm_rope(h, None, _Fake((4, 1), torch.int64), freq, [4], h, None)
    with pytest.raises(ValueError, match="inv_freq must be"):
        cr.qk_norm_rope(h, None, pos, _Fake((4,), f32), [4], h, None)
    with pytest.raises(ValueError, match="belong together"):
        cr.qk_norm_rope(h, h, pos, freq, [4], h, None)


class _Fake:
    """What a CUDA tensor says of itself; no call below gets past the checks."""

    def __init__(self, shape, dtype, strides=None, cuda=True):
        self.shape, self.dtype, self.is_cuda, self.device = shape, dtype, cuda, "cuda:0" if cuda else "cpu"
        self.strides = strides or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))

    def stride(self):
        return self.strides

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self.strides == tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def data_ptr(self):
        return P

    def get_device(self):
        return 0
