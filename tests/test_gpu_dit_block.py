"""A DiT block composed from rms_norm_quant, qk_norm_rope, gemm_fused and the
layer's own calls (examples/dit_block.py), against the same chain in 64 bits
with the roundings of its stored tensors: BF16 between the operators, S8 codes
for the products' operands.

Tolerance: the chain's stored tensors agree to about half a BF16 unit (2^-9)
where FP32 and 64-bit values round apart, and such a step moves S8 codes by
one (1/127 of a row's largest at rows of K codes: 1e-2 / sqrt(K) of a product).
Six such tensors in a row stay well below 1e-2 of the output's norm.
"""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import DEV, ensure_built

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

HID, HEADS, D, FFN, PAIRS, EPS = 512, 4, 128, 768, [16, 24, 24], 1e-6


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def quantised(u):
    pad = np.zeros((u.shape[0], oracle.padded_k(u.shape[1])))
    pad[:, :u.shape[1]] = u
    v = oracle.rotate_blocks(pad)
    s = np.abs(v).max(axis=1) / 127
    return np.rint(v / s[:, None]), s


def rms(x, w):
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + EPS) * w


def rope(x, pos):
    y = x.copy()
    i, P = 0, sum(PAIRS)
    for a, n in enumerate(PAIRS):
        for j in range(n):
            phi = pos[:, a].astype(np.float64) * 10000.0 ** (-j / n)
            c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
            e, o = x[:, :, i], x[:, :, i + P]
            y[:, :, i], y[:, :, i + P] = e * c - o * s, o * c + e * s
            i += 1
    return y


def linears(codes):
    import dit_block
    made, raw = {}, {}
    for seed, (name, N, K) in enumerate([("qkv", 3 * HEADS * D, HID), ("out", HID, HEADS * D), ("up", 2 * FFN, HID),
                                         ("up_gelu", FFN, HID), ("down", HID, FFN)]):
        wl = synth.Workload(name, 1, K, N, "bf16", "bf16", False, 0.0, 1.0, 60 + seed)
        packed, scales, t = synth.make_nvfp4_weight(wl, std=1 / np.sqrt(K))
        raw[name] = oracle.prepare_weight(packed, scales, t, K)
        made[name] = dit_block.Linear(torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV),
                                      torch.tensor([float(t)], device=DEV), K, codes)
    return made, raw


def product(q, s, raw):
    qw, sw = raw
    return (q @ qw.astype(np.float64).T) * s[:, None] * sw.astype(np.float64)


@pytest.mark.parametrize("M,codes,ffn", [(150, torch.float16, "swiglu"), (300, torch.float16, "gelu"),
                                         (7, torch.int8, "swiglu"), (1, torch.int8, "gelu")])
def test_block_against_64_bits(M, codes, ffn):
    ensure_built()
    import dit_block
    import rotated_w4a8_int8_gb300 as cr
    made, raw = linears(codes)
    if ffn == "gelu":
        made["up"], raw["up"] = made["up_gelu"], raw["up_gelu"]
    g = torch.Generator().manual_seed(M)
    vec = {n: (m + s * torch.randn(k, generator=g)) for n, k, m, s in
           [("norm1", HID, 1, .1), ("norm2", HID, 1, .1), ("q_norm", D, 1, .1), ("k_norm", D, 1, .1),
            ("qkv_bias", 3 * HEADS * D, 0, .1), ("up_bias", made["up"].N, 0, .1), ("gate1", HID, .5, .2), ("gate2", HID, .5, .2)]}
    h = torch.randn(M, HID, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 60, (M, 3), generator=g, dtype=torch.int32)
    block = dit_block.Block({**made, **{n: v.to(DEV) for n, v in vec.items()}}, HEADS, D, PAIRS, ffn, EPS)
    got = block(h.to(DEV), pos.to(DEV)).double().cpu().numpy()
    assert cr.device_error() == 0

    v = {n: t.double().numpy() for n, t in vec.items()}
    h0, p = h.double().numpy(), pos.numpy()
    qkv = bf(product(*quantised(rms(h0, v["norm1"])), raw["qkv"]) + v["qkv_bias"])
    q, k, val = (qkv[:, i * HEADS * D:(i + 1) * HEADS * D].reshape(M, HEADS, D) for i in range(3))
    q, k = bf(rope(rms(q, v["q_norm"]), p)), bf(rope(rms(k, v["k_norm"]), p))
    sc = np.einsum("mhd,nhd->hmn", q, k) / np.sqrt(D)
    sc = np.exp(sc - sc.max(axis=2, keepdims=True))
    att = bf(np.einsum("hmn,nhd->mhd", sc / sc.sum(axis=2, keepdims=True), val).reshape(M, HEADS * D))
    mid = bf(bf(product(*quantised(att), raw["out"]) * v["gate1"]) + h0)
    up = product(*quantised(rms(mid, v["norm2"])), raw["up"]) + v["up_bias"]
    if ffn == "swiglu":
        up = bf(up)
        act = up[:, :FFN] / (1 + np.exp(-up[:, :FFN])) * up[:, FFN:]
    else:
        act = bf(0.5 * up * (1 + np.tanh(np.sqrt(2 / np.pi) * (up + 0.044715 * up ** 3))))
    want = product(*quantised(act), raw["down"]) * v["gate2"] + mid
    assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)
