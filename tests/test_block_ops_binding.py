"""The binding of rms_norm_quant, qk_norm_rope and gemm_fused (csrc/marshal.c), with a C ABI that only counts its
calls: what it checks of memory written past a tensor's logical columns, and of devices, and that other Python threads run
while a call waits."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import rotated_w4a8_int8_gb300 as cr
from test_block_ops_host import _Fake


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


COUNTING_ABI = """
int calls;
int count() { ++calls; return 0; }
"""


def compiled(tmp_path, source):
    c, so = tmp_path / "abi.c", tmp_path / "abi.so"
    c.write_text(source)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-w", str(c), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def bind(m, entry, device, gpus=2):
    """Binds the marshalling module to `entry` for all three calls; `device` is the current one of `gpus`."""
    address = ctypes.cast(entry, ctypes.c_void_p).value
    m.bind(address, address, address, gpus, cr._refuse, lambda d: 100 + d, lambda: device, torch.bfloat16, torch.float16,
           torch.float32, torch.float64, torch.int8, torch.int32)


@pytest.fixture
def marshal():
    m = cr._operators()
    yield m
    cr._block_ops = None                 # the next call binds the library's own entries again


def on(device, shape, dtype):
    t = _Fake(shape, dtype)
    t.get_device = lambda: device
    return t


def norm_call(m, devices):
    f32 = torch.float32
    shapes = [((4, 256), f32), ((4, 256), torch.float16), ((4,), f32), ((4, 256), f32), ((4, 256), f32), ((256,), f32), ((4,), f32)]
    x, q, s, r, h, w, n = (on(d, *sh) for d, sh in zip(devices, shapes))
    return m.rms_norm_quant(x, 256, q, s, r, h, w, 1e-6, n, None)


def rope_call(m, devices):
    f16, f32 = torch.float16, torch.float32
    shapes = [((4, 2, 8), f16), ((4, 2, 8), f16), ((4, 1), torch.int32), ((4,), torch.float64), ((4, 2, 8), f16),
              ((4, 2, 8), f16), ((8,), f32), ((8,), f32)]
    q, k, pos, freq, qo, ko, qw, kw = (on(d, *sh) for d, sh in zip(devices, shapes))
    return m.qk_norm_rope(q, k, pos, freq, [4], qo, ko, qw, kw, 1e-6, False, None)


def gemm_call(m, devices):
    f16, f32 = torch.float16, torch.float32
    shapes = [((4, 256), f16), ((4,), f32), ((8, 256), f16), ((8,), f32), ((4, 8), f32), ((8,), f32), ((8,), f32), ((4, 8), f32)]
    a, sa, w, sw, out, b, g, r = (on(d, *sh) for d, sh in zip(devices, shapes))
    return m.gemm_fused(a, sa, w, sw, out, None, b, 0, g, r, None)


CALLS = [(norm_call, ("x", "a_q", "a_scale", "residual", "h", "weight", "a_norm")),
         (rope_call, ("q", "k", "pos", "inv_freq", "q_out", "k_out", "q_weight", "k_weight")),
         (gemm_call, ("a_q", "a_scale", "w_q", "w_scale", "out", "bias", "gate", "residual"))]


@pytest.mark.parametrize("call,names", CALLS)
def test_tensors_lie_on_the_current_device(marshal, tmp_path, call, names):
    abi = compiled(tmp_path, COUNTING_ABI)
    calls = ctypes.c_int.in_dll(abi, "calls")
    bind(marshal, abi.count, 1)
    assert call(marshal, [1] * len(names)) == 0 and calls.value == 1
    for i, name in enumerate(names[1:], 1):
        with pytest.raises(ValueError, match=f"{name} must be on cuda:1"):
            call(marshal, [1] * i + [0] + [1] * (len(names) - i - 1))
    bind(marshal, abi.count, 0)
    with pytest.raises(ValueError, match=f"{names[0]} must be on the current device"):
        call(marshal, [1] * len(names))
    assert calls.value == 1
    bind(marshal, abi.count, None, gpus=1)           # with one GPU neither tensors nor the runtime are asked
    assert call(marshal, [None] * len(names)) == 0 and calls.value == 2


# a launch that waits, 2 s at most, for something that a Python thread does
WAITING_ABI = """
#include <unistd.h>
volatile int flag;
int wait_for_flag() { for (int i = 0; i < 2000 && !flag; ++i) usleep(1000); return flag ? 0 : 7; }
"""


@pytest.mark.parametrize("call,names", CALLS)
def test_other_threads_run_while_a_call_waits(marshal, tmp_path, call, names):
    abi = compiled(tmp_path, WAITING_ABI)
    flag = ctypes.c_int.in_dll(abi, "flag")
    bind(marshal, abi.wait_for_flag, 0)

    def later():
        time.sleep(0.05)
        flag.value = 1
    t = threading.Thread(target=later)
    t.start()
    assert call(marshal, [0] * len(names)) == 0
    t.join()


@pytest.mark.parametrize("K,shape,strides", [
    (300, (4, 300), (512, 1)),           # rows of K_p codes fit the pitch, but reach past the view
    (300, (4, 511), (1024, 1)),
    (1, (4, 1), (512, 2)),               # one logical column: K_p contiguous codes are written all the same
    (1, (4, 256), (512, 2)),
    (257, (1, 300), (4096, 1)),
])
def test_codes_need_all_padded_columns(K, shape, strides):
    M = shape[0]
    x, s = _Fake((M, K), torch.float32), _Fake((M,), torch.float32)
    with pytest.raises(ValueError, match="a_q must be"):
        cr.rms_norm_quant(x, K, _Fake(shape, torch.float16, strides), s)
