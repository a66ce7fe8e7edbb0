"""The DiT block of examples/dit_block.py frame by frame over its cache, with cross attention, against the same chain in
64 bits with the roundings of its stored tensors.  Tolerance as in test_gpu_dit_block.py: a stored BF16 tensor that rounds
apart moves S8 codes by one (1/127 of a row's largest at rows of K codes: 1e-2 / sqrt(K) of a product); ten such tensors
in a row stay below 2e-2 of the output's norm."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import DEV, ensure_built
from test_gpu_dit_block import D, EPS, FFN, HEADS, HID, PAIRS, bf, product, quantised, rms, rope

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

CTX = 320


def block_and_weights(codes):
    import dit_block
    made, raw = {}, {}
    for seed, (name, N, K) in enumerate([("qkv", 3 * HEADS * D, HID), ("out", HID, HEADS * D), ("up", 2 * FFN, HID),
                                         ("down", HID, FFN), ("cross_q", HEADS * D, HID), ("cross_kv", 2 * HEADS * D, CTX),
                                         ("cross_out", HID, HEADS * D)]):
        wl = synth.Workload(name, 1, K, N, "bf16", "bf16", False, 0.0, 1.0, 160 + seed)
        packed, scales, t = synth.make_nvfp4_weight(wl, std=1 / np.sqrt(K))
        raw[name] = oracle.prepare_weight(packed, scales, t, K)
        made[name] = dit_block.Linear(torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV),
                                      torch.tensor([float(t)], device=DEV), K, codes)
    g = torch.Generator().manual_seed(9)
    vec = {n: (m + s * torch.randn(k, generator=g)) for n, k, m, s in
           [("norm1", HID, 1, .1), ("norm2", HID, 1, .1), ("norm3", HID, 1, .1), ("q_norm", D, 1, .1), ("k_norm", D, 1, .1),
            ("qkv_bias", 3 * HEADS * D, 0, .1), ("up_bias", 2 * FFN, 0, .1), ("gate1", HID, .5, .2), ("gate2", HID, .5, .2)]}
    block = dit_block.Block({**made, **{n: v.to(DEV) for n, v in vec.items()}}, HEADS, D, PAIRS, "swiglu", EPS)
    return block, raw, {n: t.double().numpy() for n, t in vec.items()}


def attend(q, k, v):
    s = np.einsum("mhd,nhd->hmn", q, k) / math.sqrt(D)
    s = np.exp(s - s.max(axis=2, keepdims=True))
    return bf(np.einsum("hmn,nhd->mhd", s / s.sum(axis=2, keepdims=True), v).reshape(q.shape[0], HEADS * D))


@pytest.mark.parametrize("frames,window,codes", [((150, 150, 70), 10 ** 4, torch.float16), ((40, 40, 40, 33, 40), 100, torch.float16),
                                                 ((7, 1, 1, 1), 9, torch.int8)])
def test_frames_over_a_cache(frames, window, codes):
    ensure_built()
    import dit_block
    import rotated_w4a8_int8_gb300 as cr
    block, raw, v = block_and_weights(codes)
    g = torch.Generator().manual_seed(len(frames))
    states = torch.randn(70 if codes == torch.float16 else 50, CTX, generator=g).to(torch.bfloat16)
    cross = block.cross_keys(states.to(DEV))
    kv = bf(product(*quantised(states.double().numpy()), raw["cross_kv"])).reshape(-1, 2, HEADS, D)
    cache = dit_block.FrameCache(sum(frames), min(window, sum(frames)), HEADS, D, page=16)
    keys, values = np.zeros((0, HEADS, D)), np.zeros((0, HEADS, D))
    for M in frames:
        h = torch.randn(M, HID, generator=g).to(torch.bfloat16)
        pos = torch.randint(0, 60, (M, 3), generator=g, dtype=torch.int32)
        got = block(h.to(DEV), pos.to(DEV), cache, cross).double().cpu().numpy()
        assert cr.device_error() == 0
        h0, p = h.double().numpy(), pos.numpy()
        qkv = bf(product(*quantised(rms(h0, v["norm1"])), raw["qkv"]) + v["qkv_bias"])
        q, k, val = (qkv[:, i * HEADS * D:(i + 1) * HEADS * D].reshape(M, HEADS, D) for i in range(3))
        q, k = bf(rope(rms(q, v["q_norm"]), p)), bf(rope(rms(k, v["k_norm"]), p))
        keys, values = (np.concatenate([a, b])[-window:] for a, b in ((keys, k), (values, val)))
        att = attend(q, keys, values)
        mid = bf(bf(product(*quantised(att), raw["out"]) * v["gate1"]) + h0)
        q = bf(product(*quantised(rms(mid, v["norm3"])), raw["cross_q"])).reshape(M, HEADS, D)
        att = attend(q, kv[:, 0], kv[:, 1])
        mid = bf(bf(product(*quantised(att), raw["cross_out"])) + mid)
        up = bf(product(*quantised(rms(mid, v["norm2"])), raw["up"]) + v["up_bias"])
        act = up[:, :FFN] / (1 + np.exp(-up[:, :FFN])) * up[:, FFN:]
        want = product(*quantised(act), raw["down"]) * v["gate2"] + mid
        assert np.linalg.norm(got - want) <= 2e-2 * np.linalg.norm(want)
