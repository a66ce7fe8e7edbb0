"""One block of a video DiT on the library's operators.

    h  -> rms_norm_quant -> qkv product (bias) -> qk_norm_rope (in place, time x height x width)
       -> attention -> quant_act -> out product (channel gate)
       -> rms_norm_quant (adds the residual stream, writes the sum)
       -> FFN up, either SwiGLU (gemm_fused, then quant_act with its SwiGLU) or GELU in the product's epilogue
       -> quant_act -> FFN down (channel gate, plus the residual stream in place)

The weights are NVFP4 and become rotated S8 codes once, at two bytes per code (FP16-held, for prompts) or one (for at
most FEW_TOKENS tokens).  The attention between q, k and v is torch's: the library has none.  Run as a script it times
a block of random weights:

    python examples/dit_block.py --tokens 4096
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rotated_w4a8_int8_gb300 as cr  # noqa: E402


class Linear:
    """A prepared weight: rotated codes and row scales of an NVFP4 weight [N, K]."""

    def __init__(self, packed, block_scales, tensor_scale, K: int, codes: torch.dtype):
        N = packed.shape[0]
        self.K, self.N = K, N
        self.codes = torch.empty(N, cr.padded_k(K), dtype=codes, device=packed.device)
        self.scale = torch.empty(N, device=packed.device)
        cr.prepare_weight(packed, block_scales, tensor_scale, K, self.codes, self.scale)


class Block:
    """`weights`: qkv, out, up, down (Linear); norm1, norm2, q_norm, k_norm, qkv_bias, up_bias (or None), gate1,
    gate2 (FP32 vectors).  `axis_pairs` spans the head width over the position axes."""

    def __init__(self, weights: dict, heads: int, head_dim: int, axis_pairs, ffn: str = "swiglu", eps: float = 1e-6):
        self.w, self.heads, self.head_dim, self.ffn, self.eps = weights, heads, head_dim, ffn, eps
        self.axis_pairs = list(axis_pairs)
        dev = weights["norm1"].device
        self.inv_freq = torch.tensor(cr.rope_inv_freq(self.axis_pairs), dtype=torch.float64, device=dev)
        self.codes = weights["qkv"].codes.dtype

    def _quantised(self, x, K, **kw):
        a = torch.empty(x.shape[0], cr.padded_k(K), dtype=self.codes, device=x.device)
        s = torch.empty(x.shape[0], device=x.device)
        cr.quant_act(x, K, a, s, **kw)
        return a, s

    def _normed(self, x, weight, **kw):
        K = x.shape[1]
        a = torch.empty(x.shape[0], cr.padded_k(K), dtype=self.codes, device=x.device)
        s = torch.empty(x.shape[0], device=x.device)
        cr.rms_norm_quant(x, K, a, s, weight=weight, eps=self.eps, **kw)
        return a, s

    def _product(self, a, s, lin: Linear, like, **kw):
        out = torch.empty(a.shape[0], lin.N, dtype=like.dtype, device=like.device)
        cr.gemm_fused(a, s, lin.codes, lin.scale, out, **kw)
        return out

    def __call__(self, h, pos):
        """h [tokens, hidden] (bf16 or fp16), pos int32 [tokens, axes]; returns the block's output, h unchanged."""
        w, H, D = self.w, self.heads, self.head_dim
        M = h.shape[0]
        qkv = self._product(*self._normed(h, w["norm1"]), w["qkv"], h, bias=w["qkv_bias"])
        q, k, v = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
        cr.qk_norm_rope(q, k, pos, self.inv_freq, self.axis_pairs, q, k, q_weight=w["q_norm"], k_weight=w["k_norm"],
                        eps=self.eps)
        att = torch.nn.functional.scaled_dot_product_attention(*(t.transpose(0, 1)[None] for t in (q, k, v)))
        att = att[0].transpose(0, 1).reshape(M, H * D)
        proj = self._product(*self._quantised(att, H * D), w["out"], h, gate=w["gate1"])
        mid = torch.empty_like(h)
        a, s = self._normed(proj, w["norm2"], residual=h, h=mid)
        if self.ffn == "swiglu":
            up = self._product(a, s, w["up"], h, bias=w["up_bias"])
            a, s = self._quantised(up, w["down"].K, swiglu=True)
        else:
            up = self._product(a, s, w["up"], h, bias=w["up_bias"], act=cr.ACT_GELU_TANH)
            a, s = self._quantised(up, w["down"].K)
        cr.gemm_fused(a, s, w["down"].codes, w["down"].scale, mid, gate=w["gate2"], residual=mid)
        return mid


def grid_positions(frames: int, height: int, width: int, device) -> torch.Tensor:
    """int32 [frames * height * width, 3]: time, height and width of every token."""
    axes = torch.meshgrid(*(torch.arange(n, dtype=torch.int32, device=device) for n in (frames, height, width)),
                          indexing="ij")
    return torch.stack([a.flatten() for a in axes], 1).contiguous()


def random_block(hidden: int, heads: int, head_dim: int, ffn_width: int, axis_pairs, codes=torch.float16,
                 ffn: str = "swiglu", seed: int = 0, device="cuda") -> Block:
    g = torch.Generator(device=device).manual_seed(seed)

    def linear(N, K):
        packed = torch.randint(0, 256, (N, -(-K // 16) * 8), generator=g, device=device, dtype=torch.uint8)
        scales = torch.randint(0x30, 0x39, (N, -(-K // 16)), generator=g, device=device, dtype=torch.uint8)
        t = torch.tensor([0.25 / K ** 0.5], device=device)
        return Linear(packed, scales, t, K, codes)

    def vec(n, mean, std):
        return mean + std * torch.randn(n, generator=g, device=device)
    up = 2 * ffn_width if ffn == "swiglu" else ffn_width
    return Block(dict(qkv=linear(3 * heads * head_dim, hidden), out=linear(hidden, heads * head_dim),
                      up=linear(up, hidden), down=linear(hidden, ffn_width), norm1=vec(hidden, 1, 0.1),
                      norm2=vec(hidden, 1, 0.1), q_norm=vec(head_dim, 1, 0.1), k_norm=vec(head_dim, 1, 0.1),
                      qkv_bias=vec(3 * heads * head_dim, 0, 0.1), up_bias=vec(up, 0, 0.1), gate1=vec(hidden, 0.5, 0.1),
                      gate2=vec(hidden, 0.5, 0.1)), heads, head_dim, axis_pairs, ffn)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--ffn", choices=("swiglu", "gelu"), default="swiglu")
    a = ap.parse_args()
    codes = torch.int8 if a.tokens <= cr.FEW_TOKENS else torch.float16
    block = random_block(5376, 56, 128, 14336, (16, 24, 24), codes, a.ffn)
    pos = grid_positions(-(-a.tokens // 2304), 36, 64, "cuda")[:a.tokens].contiguous()
    h = torch.randn(a.tokens, 5376, device="cuda").bfloat16()
    for _ in range(3):
        block(h, pos)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(5):
        out = block(h, pos)
    end.record()
    torch.cuda.synchronize()
    if cr.device_error():
        raise RuntimeError("a kernel timed out")
    print(f"{a.tokens} tokens, {a.ffn}: {begin.elapsed_time(end) / 5:.3f} ms per block, output rms "
          f"{out.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
