"""Refusals of attention, paged_attention and cache_write, by the C ABI and by the binding, before anything is launched
(CPU only)."""
import ctypes

import pytest
import torch

import rotated_w4a8_int8_gb300 as cr
from test_block_ops_binding import COUNTING_ABI, WAITING_ABI, bind, compiled, on
from test_block_ops_host import _Fake

P = 1 << 20                             # aligned fake device address: no call below reaches the GPU


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rows_call(**kw):
    a = dict(q=P, qr=512, qh=64, k=P, kr=128, kh=64, v=P, vr=128, vh=64, o=2 * P, orow=512, oh=64, dt=0, rows=0, keys=5, hq=8,
             hk=2, D=64, seqs=None, B=1, scale=0.125, causal=0)
    a.update(kw)
    return cr.load_library().convrot_attention(
        a["q"], a["qr"], a["qh"], a["k"], a["kr"], a["kh"], a["v"], a["vr"], a["vh"], a["o"], a["orow"], a["oh"], a["dt"],
        a["rows"], a["keys"], a["hq"], a["hk"], a["D"], a["seqs"], a["B"], a["scale"], a["causal"], None)


def test_largest_scale():
    """scale * log2(e), which the kernels use, is finite too."""
    assert rows_call(rows=4, scale=2.0 ** 127) == 1 and rows_call(rows=4, scale=3.4e38) == 1
    assert rows_call(rows=4, seqs=P + 8, scale=2.0 ** 126) == 2       # (refused for an address that is looked at after it)


def test_attention_arguments():
    assert rows_call() == 0                                   # no rows: nothing to do
    assert rows_call(rows=4, seqs=P, B=0) == 0                # no sequences
    assert rows_call(rows=4, seqs=None, B=0) == 0             # (an empty tensor has no address)
    assert rows_call(dt=2) == 3 and rows_call(dt=7) == 3      # FP32 is not taken
    assert rows_call(rows=-1) == 1 and rows_call(keys=-1) == 1 and rows_call(B=-1) == 1
    assert rows_call(hq=0) == 1 and rows_call(hk=0) == 1 and rows_call(hq=7) == 1
    assert rows_call(D=0) == 1 and rows_call(D=68) == 3 and rows_call(D=136) == 3
    assert rows_call(rows=(1 << 30) + 1) == 3 and rows_call(keys=(1 << 26) + 1) == 3 and rows_call(B=65536) == 3
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert rows_call(rows=4, scale=scale) == 1
    for name in ("q", "k", "v", "o"):
        assert rows_call(rows=4, **{name: None}) == 1
        assert rows_call(rows=4, **{name: P + 8}) == 2
    for name in ("qr", "qh", "kr", "kh", "vr", "vh", "orow", "oh"):
        assert rows_call(rows=4, **{name: 56}) == 1           # below D
        assert rows_call(rows=4, **{name: -512}) == 1
        assert rows_call(rows=4, **{name: 1028}) == 2         # no whole 16-byte pieces
        assert rows_call(rows=4, **{name: 1 << 39}) == 3
    for name in ("q", "k", "v"):
        assert rows_call(rows=4, **{n: P + (1 << 20) * (n == name) for n in ("q", "k", "v")}, o=P + (1 << 20)) == 1   # in place
    assert rows_call(rows=4, orow=64, oh=64) == 1             # outputs overlap
    assert rows_call(rows=4, orow=128, oh=64) == 1
    assert rows_call(rows=4, seqs=P + 4) == 2


def pages_call(fn="paged", **kw):
    a = dict(q=P, qr=512, qh=64, k=P, kp=2048, kr=128, kh=64, v=P, vp=2048, vr=128, vh=64, o=2 * P, orow=512, oh=64, dt=1,
             rows=4, hq=8, hk=2, D=64, n=9, size=16, t=P, ld=5, per=5, seqs=P, B=3, scale=0.125, causal=0)
    a.update(kw)
    lib = cr.load_library()
    if fn == "write":
        return lib.convrot_cache_write(a["q"], a["qr"], a["qh"], a["o"], a["orow"], a["oh"], a["k"], a["kp"], a["kr"], a["kh"],
                                       a["v"], a["vp"], a["vr"], a["vh"], a["dt"], a["rows"], a["hk"], a["D"], a["n"], a["size"],
                                       a["t"], a["ld"], a["per"], a["seqs"], a["B"], None)
    return lib.convrot_paged_attention(a["q"], a["qr"], a["qh"], a["k"], a["kp"], a["kr"], a["kh"], a["v"], a["vp"], a["vr"],
                                       a["vh"], a["o"], a["orow"], a["oh"], a["dt"], a["rows"], a["hq"], a["hk"], a["D"], a["n"],
                                       a["size"], a["t"], a["ld"], a["per"], a["seqs"], a["B"], a["scale"], a["causal"], None)


@pytest.mark.parametrize("fn", ["paged", "write"])
def test_paged_arguments(fn):
    call = lambda **kw: pages_call(fn, **kw)
    assert call(rows=0) == 0 and call(B=0) == 0
    assert call(dt=2) == 3 and call(D=12) == 3 and call(D=200) == 3
    for size in (8, 24, 0, -16, 131072):
        assert call(size=size) == (1 if size <= 0 else 3)
    assert call(n=-1) == 1 and call(per=-1) == 1
    assert call(t=None) == 1 and call(t=P + 2) == 2 and call(ld=4) == 1
    assert call(seqs=None) == 1 and call(seqs=P + 8) == 2
    for name in ("q", "k", "v", "o"):
        assert call(**{name: None}) == 1
        assert call(**{name: P + 2}) == 2
    for name in ("kp", "kr", "kh", "vp", "vr", "vh", "qr", "orow"):
        assert call(**{name: 60}) == 1
        assert call(**{name: (1 << 16) + 4}) == 2
    if fn == "write":
        assert call(kp=1024) == 1 and call(vr=64) == 1        # what is written does not overlap


def test_caches_are_written_once():
    """The same memory as both caches, or as a cache and an input, is refused."""
    lib, at = cr.load_library(), [P * n for n in (1, 2, 3, 4)]

    def call(k, v, kc, vc):
        return lib.convrot_cache_write(k, 512, 64, v, 512, 64, kc, 2048, 128, 64, vc, 2048, 128, 64, 0, 4, 2, 64, 9, 16, P, 5, 5,
                                       P, 3, None)
    for same in ((0, 1, 2, 2), (0, 1, 0, 2), (0, 1, 1, 2), (0, 1, 2, 0), (0, 1, 2, 1)):
        assert call(*(at[i] for i in same)) == 1


def test_selftest_arguments():
    lib = cr.load_library()

    def call(kernel, slices, starve=0):
        return lib.convrot_attention_selftest(P, 512, 64, P, 0, 128, 64, P, 0, 128, 64, 2 * P, 512, 64, 0, 0, 8, 2, 64, 5, 0, 0,
                                              None, 0, 0, None, 1, 0.125, 0, kernel, slices, starve, None)
    assert call(1, 16) == 0 and call(1, 3, 1) == 0 and call(2, 1) == 0 and call(3, 7, 1) == 0
    for kernel, slices, starve in ((0, 1, 0), (4, 1, 0), (1, 0, 0), (1, 17, 0), (2, 2, 0), (3, 9, 0)):
        assert call(kernel, slices, starve) == 1


F16, BF, I32 = torch.float16, torch.bfloat16, torch.int32


def heads_args(**kw):
    a = dict(q=_Fake((6, 4, 64), BF), k=_Fake((9, 2, 64), BF), v=_Fake((9, 2, 64), BF), out=_Fake((6, 4, 64), BF),
             seqs=_Fake((3, 4), I32))
    a.update(kw)
    return a["q"], a["k"], a["v"], a["out"], a["seqs"]


@pytest.mark.parametrize("name,bad", [
    ("q", _Fake((6, 4), BF)), ("q", _Fake((6, 4, 64), torch.float32)), ("k", _Fake((9, 2, 32), BF)), ("k", _Fake((9, 2, 64), F16)),
    ("v", _Fake((8, 2, 64), BF)), ("v", _Fake((9, 4, 64), BF)), ("v", _Fake((9, 2, 64), BF, (128, 1, 2))),
    ("out", _Fake((6, 2, 64), BF)), ("out", _Fake((5, 4, 64), BF)), ("seqs", _Fake((3, 3), I32)), ("seqs", _Fake((3, 4), torch.int8)),
    ("seqs", _Fake((12,), I32))])
def test_attention_tensors(name, bad):
    with pytest.raises(ValueError, match=f"attention: {name} must be"):
        cr.attention(*heads_args(**{name: bad}))


def test_missing_tensors():
    with pytest.raises(ValueError):
        cr.attention(*heads_args(v=None))
    with pytest.raises(ValueError):
        cr.attention(*heads_args(out=None))
    with pytest.raises(ValueError, match="seqs is needed"):
        cr.paged_attention(*paged_args(seqs=None))


def paged_args(**kw):
    a = dict(q=_Fake((6, 4, 64), BF), k=_Fake((9, 16, 2, 64), BF), v=_Fake((9, 16, 2, 64), BF), pages=_Fake((3, 5), I32),
             seqs=_Fake((3, 4), I32), out=_Fake((6, 4, 64), BF))
    a.update(kw)
    return a["q"], a["k"], a["v"], a["pages"], a["seqs"], a["out"]


@pytest.mark.parametrize("name,key,bad", [
    ("k_cache", "k", _Fake((9, 16, 2, 32), BF)), ("k_cache", "k", _Fake((9, 16, 2, 64), F16)), ("k_cache", "k", _Fake((144, 2, 64), BF)),
    ("v_cache", "v", _Fake((8, 16, 2, 64), BF)), ("v_cache", "v", _Fake((9, 32, 2, 64), BF)), ("v_cache", "v", _Fake((9, 16, 1, 64), BF)),
    ("pages", "pages", _Fake((2, 5), I32)), ("pages", "pages", _Fake((3, 5), torch.float32)), ("pages", "pages", _Fake((15,), I32)),
    ("seqs", "seqs", _Fake((3, 5), I32)), ("out", "out", _Fake((6, 4, 32), BF))])
def test_paged_tensors(name, key, bad):
    with pytest.raises(ValueError, match=f"paged_attention: {name} must be"):
        cr.paged_attention(*paged_args(**{key: bad}))


@pytest.mark.parametrize("name,at,bad", [
    ("k", 0, _Fake((6, 2, 64), torch.float32)), ("v", 1, _Fake((6, 1, 64), BF)), ("v", 1, _Fake((5, 2, 64), BF)),
    ("k_cache", 2, _Fake((9, 16, 2, 64), F16)), ("v_cache", 3, _Fake((9, 16, 4, 64), BF)), ("pages", 4, _Fake((4, 5), I32)),
    ("seqs", 5, _Fake((3, 2), I32))])
def test_write_tensors(name, at, bad):
    args = [_Fake((6, 2, 64), BF), _Fake((6, 2, 64), BF), *paged_args()[1:5]]
    args[at] = bad
    with pytest.raises(ValueError, match=f"cache_write: {name} must be"):
        cr.cache_write(*args)


def test_write_needs_the_caches_heads():
    with pytest.raises(ValueError, match="with k's 1 heads"):
        cr.cache_write(_Fake((6, 1, 64), BF), _Fake((6, 1, 64), BF), *paged_args()[1:5])


def attention_call(m, d):
    shapes = [((6, 4, 64), BF), ((9, 2, 64), BF), ((9, 2, 64), BF), ((6, 4, 64), BF), ((3, 4), I32)]
    return m.attention(*(on(i, *sh) for i, sh in zip(d, shapes)), 0.125, False, None)


def paged_call(m, d):
    shapes = [((6, 4, 64), BF), ((9, 16, 2, 64), BF), ((9, 16, 2, 64), BF), ((3, 5), I32), ((3, 4), I32), ((6, 4, 64), BF)]
    return m.paged_attention(*(on(i, *sh) for i, sh in zip(d, shapes)), 0.125, True, None)


def write_call(m, d):
    shapes = [((6, 2, 64), BF), ((6, 2, 64), BF), ((9, 16, 2, 64), BF), ((9, 16, 2, 64), BF), ((3, 5), I32), ((3, 4), I32)]
    return m.cache_write(*(on(i, *sh) for i, sh in zip(d, shapes)), None)


CALLS = [(attention_call, ("q", "k", "v", "out", "seqs")), (paged_call, ("q", "k_cache", "v_cache", "pages", "seqs", "out")),
         (write_call, ("k", "v", "k_cache", "v_cache", "pages", "seqs"))]


@pytest.fixture
def marshal():
    m = cr._operators()
    yield m
    cr._block_ops = None                 # the next call binds the library's own entries again


@pytest.mark.parametrize("call,names", CALLS)
def test_tensors_lie_on_the_current_device(marshal, tmp_path, call, names):
    abi = compiled(tmp_path, COUNTING_ABI)
    calls, address = ctypes.c_int.in_dll(abi, "calls"), ctypes.cast(abi.count, ctypes.c_void_p).value
    marshal.bind_attention(address, address, address)
    bind(marshal, abi.count, 1)
    assert call(marshal, [1] * len(names)) == 0 and calls.value == 1
    for i, name in enumerate(names[1:], 1):
        with pytest.raises(ValueError, match=f"{name} must be on cuda:1"):
            call(marshal, [1] * i + [0] + [1] * (len(names) - i - 1))
    bind(marshal, abi.count, 0)
    with pytest.raises(ValueError, match=f"{names[0]} must be on the current device"):
        call(marshal, [1] * len(names))
    assert calls.value == 1


@pytest.mark.parametrize("call,names", CALLS)
def test_other_threads_run_while_a_call_waits(marshal, tmp_path, call, names):
    import threading
    import time
    abi = compiled(tmp_path, WAITING_ABI)
    flag, address = ctypes.c_int.in_dll(abi, "flag"), ctypes.cast(abi.wait_for_flag, ctypes.c_void_p).value
    marshal.bind_attention(address, address, address)
    bind(marshal, abi.wait_for_flag, 0)

    def later():
        time.sleep(0.05)
        flag.value = 1
    t = threading.Thread(target=later)
    t.start()
    assert call(marshal, [0] * len(names)) == 0
    t.join()


CHOICE = """
#include "attention_choice.h"
extern "C" int few_slices(long long units, long long tiles, int sms, int largest) {
  return cratt::few_slices(units, tiles, sms, largest);
}
"""


def test_ctas_that_share_keys(tmp_path):
    """As many as were chosen for 152 SMs when that was written into the code; never a larger cluster than the device
    takes, and fewer on fewer SMs."""
    import os
    import subprocess
    src, so = tmp_path / "choice.cpp", tmp_path / "choice.so"
    src.write_text(CHOICE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(cr.LIB_PATH), "csrc"),
                    str(src), "-o", str(so)], check=True)
    slices = ctypes.CDLL(str(so)).few_slices
    slices.argtypes = [ctypes.c_longlong] * 2 + [ctypes.c_int] * 2

    def as_before(units, tiles):
        n, most = 304 // units, tiles // 2
        if n < 2:
            n, most = 4, tiles // 32
        if n > 8:
            n = max(152 // units, 8)
        return max(1, min(n, most, 16))
    for units in (1, 2, 7, 8, 9, 16, 17, 19, 20, 30, 38, 56, 76, 150, 152, 153, 304, 305, 4096, 65535 * 8):
        for tiles in (0, 1, 2, 3, 17, 31, 32, 64, 129, 313, 1 << 20):
            want = as_before(units, tiles)
            assert slices(units, tiles, 152, 16) == want
            for largest in (1, 8, 11):
                assert slices(units, tiles, 152, largest) == min(want, largest)
            assert slices(units, tiles, 19, 16) <= max(8, 19 // units)
    assert slices(2, 1 << 20, 19, 16) == 9 and slices(1, 1 << 20, 8, 16) == 8


def test_frame_cache_refuses_what_it_cannot_hold():
    """A frame longer than the window, or one past the table, is refused, and the cache is as before."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import dit_block
    cache = dit_block.FrameCache(tokens=64, window=40, heads=1, head_dim=8, page=16, device="cpu")
    with pytest.raises(ValueError, match="window"):
        cache.extend(41)
    assert cache.extend(40).tolist() == [[0, 40, 0, 40]]
    assert cache.extend(24).tolist() == [[0, 24, 24, 40]]
    with pytest.raises(ValueError, match="table"):
        cache.extend(1)
    assert cache.length == 64 and sorted(cache.held) == [1, 2, 3]
