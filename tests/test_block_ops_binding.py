"""Host side of rms_norm_quant, qk_norm_rope and gemm_fused, beyond the plain refusals: what the binding checks of
memory that a call writes past its tensors' logical columns."""
import pytest
import torch

import rotated_w4a8_int8_gb300 as cr
from test_block_ops_host import _Fake


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


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
