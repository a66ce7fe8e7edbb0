"""attention and paged_attention against 64 bits: every kernel and split, head widths, shared heads, ragged and empty
sequences, causal masks, pages, windows, strides, and what may not have a say (keys and rows outside the sequences).
The bound is derived in attention_util.py."""
import math

import pytest
import torch

from attention_util import check, paged, reference
from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF, HF = torch.bfloat16, torch.float16
FEW, WHOLE, SHARED = 1, 2, 3
KERNELS = [(FEW, 1), (FEW, 3), (FEW, 8), (FEW, 16), (WHOLE, 1), (SHARED, 1), (SHARED, 2), (SHARED, 5), (SHARED, 8)]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def inputs(rows, keys, heads_q, heads_k, D, dtype, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    q, k, v = rand(rows, heads_q, D) * std, rand(keys, heads_k, D) * std, rand(keys, heads_k, D)
    return q.to(dtype), k.to(dtype), v.to(dtype)


def run(q, k, v, seqs, kernel=None, causal=False, page=0, window=0, scale=None, out=None):
    import rotated_w4a8_int8_gb300 as cr
    out = torch.full_like(q, 9.0) if out is None else out
    want, bound = reference(q, k, v, seqs, q.shape[2] ** -0.5 if scale is None else scale, causal, out)
    table, where = None, torch.tensor(seqs, dtype=torch.int32, device=DEV)
    if page:
        k, v, table, where = paged(k, v, seqs, page, window)
    if kernel:
        cr.attention_selftest(q, k, v, out, *kernel, pages=table, seqs=where, scale=scale, causal=causal)
    elif page:
        cr.paged_attention(q, k, v, table, where, out, scale=scale, causal=causal)
    else:
        cr.attention(q, k, v, out, seqs=where, scale=scale, causal=causal)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    check(out, want, bound)
    return out


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("q_len,k_len", [(1, 1), (1, 300), (2, 129), (128, 128), (129, 127), (300, 1000)])
def test_one_sequence(kernel, q_len, k_len):
    q, k, v = inputs(q_len, k_len, 2, 2, 128, BF)
    run(q, k, v, [(0, q_len, 0, k_len)], kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype,heads_q,heads_k", [(64, HF, 4, 2), (8, BF, 3, 3), (72, HF, 7, 1), (96, BF, 8, 2), (128, HF, 2, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_sequences(kernel, D, dtype, heads_q, heads_k, causal):
    # rows 0 .. 2 and the last ones lie in no sequence, and keys between the sequences are NaN
    lens = [(5, 140), (0, 9), (130, 130), (3, 0), (1, 257), (40, 20), (260, 300)]
    seqs, a, f = [], 3, 2
    for n, m in lens:
        seqs.append((a, n, f, m))
        a, f = a + n, f + m + 3
    q, k, v = inputs(a + 4, f, heads_q, heads_k, D, dtype, seed=D)
    used = torch.zeros(f, dtype=torch.bool, device=DEV)
    for _, _, s, m in seqs:
        used[s:s + m] = True
    k[~used], v[~used] = math.nan, math.inf
    run(q, k, v, seqs, kernel, causal)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page,window", [(16, 0), (64, 0), (256, 0), (16, 37), (128, 200), (1024, 700)])
@pytest.mark.parametrize("causal", [False, True])
def test_pages(kernel, page, window, causal):
    lens = [(7, 140), (1, 16), (130, 300), (2, 0), (1, 129)]
    seqs, a, f = [], 0, 0
    for n, m in lens:
        seqs.append((a, n, f, m))
        a, f = a + n, f + m
    q, k, v = inputs(a, f, 4, 2, 80, BF, seed=page)
    run(q, k, v, seqs, kernel, causal, page, window)


@pytest.mark.parametrize("kernel", KERNELS)
def test_growing_scores(kernel):
    # the largest scores come last, far above the first ones: the reference moves again and again
    q, k, v = inputs(150, 900, 2, 1, 64, BF)
    k *= torch.linspace(0, 12, 900, device=DEV)[:, None, None].to(BF)
    run(q, k, v, [(0, 150, 0, 900)], kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_scale_and_large_scores(kernel, dtype):
    q, k, v = inputs(140, 333, 2, 2, 128, dtype, std=3.0)
    run(q, k, v, [(0, 140, 0, 333)], kernel, scale=0.5)


@pytest.mark.parametrize("kernel", KERNELS)
def test_views_of_a_packed_product(kernel):
    H, Hk, D, M = 6, 2, 96, 200
    qkv, _, _ = inputs(M, 1, H + 2 * Hk, 1, D, BF)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    wide = torch.full((M, H + 1, 128), 4.0, dtype=BF, device=DEV)
    out = wide[:, :H, :D]
    run(q, k, v, [(0, M, 0, M)], kernel, True, out=out)
    assert bool((wide[:, H] == 4).all()) and bool((wide[:, :, D:] == 4).all())


@pytest.mark.parametrize("rows,keys,heads_q,heads_k,D", [(1, 77, 56, 56, 128), (3, 4097, 8, 2, 128), (200, 512, 8, 8, 64),
                                                         (64, 5000, 32, 8, 96), (1000, 1000, 4, 4, 128), (5, 0, 4, 4, 64)])
def test_chosen_kernels(rows, keys, heads_q, heads_k, D):
    q, k, v = inputs(rows, keys, heads_q, heads_k, D, BF, seed=rows)
    run(q, k, v, [(0, rows, 0, keys)])


def test_all_rows_and_keys_without_sequences():
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = inputs(300, 200, 4, 2, 64, HF)
    out = torch.empty_like(q)
    cr.attention(q, k, v, out)
    torch.cuda.synchronize()
    check(out, *reference(q, k, v, [(0, 300, 0, 200)], 0.125, False, out))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype", [(104, BF), (112, HF), (120, BF)])
@pytest.mark.parametrize("page", [0, 32])
def test_widths_below_the_widest(kernel, D, dtype, page):
    # computed as 128 columns; the next head's and the next row's values lie right behind
    seqs = [(0, 3, 0, 130), (3, 140, 130, 300)]
    q, k, v = inputs(143, 430, 4, 2, D, dtype, seed=D)
    run(q, k, v, seqs, kernel, True, page, 21 if page else 0)
