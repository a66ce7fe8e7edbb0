"""One block of a video DiT on the library's operators.

    h  -> rms_norm_quant -> qkv product (bias) -> qk_norm_rope (in place, time x height x width)
       -> attention, to the call's own tokens or, frame by frame, to a cache of those before (cache_write,
       paged_attention) -> quant_act -> out product (channel gate)
       -> if the block has the weights: rms_norm_quant -> q product -> attention to an encoder's states, whose k and v
       are a product of their own -> quant_act -> out product (added to the stream)
       -> rms_norm_quant (adds the residual stream, writes the sum)
       -> FFN up, either SwiGLU (gemm_fused, then quant_act with its SwiGLU) or GELU in the product's epilogue
       -> quant_act -> FFN down (channel gate, plus the residual stream in place)

The weights are NVFP4 and become rotated S8 codes once, at two bytes per code (FP16-held, for prompts) or one (for at
most FEW_TOKENS tokens).  Run as a script it times a block of random weights:

    python examples/dit_block.py --tokens 4096
    python examples/dit_block.py --tokens 2304 --cached 19989 --context 512
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


class FrameCache:
    """Keys and values of the tokens before, in pages.  `window` bounds the tokens that a frame sees, its own among
    them; pages that lie before it are used again.  A frame is at most as long as the window."""

    def __init__(self, tokens: int, window: int, heads: int, head_dim: int, page: int = 64, dtype=torch.bfloat16,
                 device="cuda"):
        # the window, the frame's last page and a first one that is left in part
        self.k, self.v = (torch.zeros(-(-window // page) + 2, page, heads, head_dim, dtype=dtype, device=device)
                          for _ in range(2))
        self.table = torch.zeros(1, -(-tokens // page), dtype=torch.int32, device=device)
        self.free = list(range(self.k.shape[0]))
        self.held: dict[int, int] = {}            # index in the table -> page
        self.window, self.page, self.length = window, page, 0

    def extend(self, n: int) -> torch.Tensor:
        """Room for n more tokens; the call's seqs: every token in the window, the new ones at the end."""
        if n > self.window or self.length + n > self.table.shape[1] * self.page:
            raise ValueError(f"{n} tokens after {self.length}: more than the window ({self.window}) or the table "
                             f"({self.table.shape[1] * self.page}) holds")
        self.length += n
        first = max(0, self.length - self.window)
        for i in [i for i in self.held if (i + 1) * self.page <= first]:
            self.free.append(self.held.pop(i))
        new = [i for i in range(first // self.page, -(-self.length // self.page)) if i not in self.held]
        for i in new:
            self.held[i] = self.free.pop()
        if new:                                   # the last ones of the table, in a row
            self.table[0, new[0]:new[-1] + 1] = torch.tensor([self.held[i] for i in new], dtype=torch.int32)
        return torch.tensor([[0, n, first, self.length - first]], dtype=torch.int32, device=self.table.device)


class Block:
    """`weights`: qkv, out, up, down (Linear); norm1, norm2, q_norm, k_norm, qkv_bias, up_bias (or None), gate1,
    gate2 (FP32 vectors); with cross attention also cross_q, cross_kv, cross_out (Linear) and norm3.  `axis_pairs` spans
    the head width over the position axes."""

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

    def cross_keys(self, context):
        """k and v [states, heads, head_dim] of an encoder's states [states, width]: once per prompt."""
        kv = self._product(*self._quantised(context, context.shape[1]), self.w["cross_kv"], context)
        return kv.unflatten(1, (2, self.heads, self.head_dim)).unbind(1)

    def __call__(self, h, pos, cache: FrameCache | None = None, cross=None, cross_seqs=None):
        """h [tokens, hidden] (bf16 or fp16), pos int32 [tokens, axes]; returns the block's output, h unchanged.  cache:
        the tokens are a frame after those in it.  cross: an encoder's k and v (cross_keys); cross_seqs: attention's
        seqs where it is a batch."""
        w, H, D = self.w, self.heads, self.head_dim
        M = h.shape[0]
        qkv = self._product(*self._normed(h, w["norm1"]), w["qkv"], h, bias=w["qkv_bias"])
        q, k, v = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
        cr.qk_norm_rope(q, k, pos, self.inv_freq, self.axis_pairs, q, k, q_weight=w["q_norm"], k_weight=w["k_norm"],
                        eps=self.eps)
        att = torch.empty(M, H, D, dtype=h.dtype, device=h.device)
        if cache is None:
            cr.attention(q, k, v, att)
        else:
            seqs = cache.extend(M)
            cr.cache_write(k, v, cache.k, cache.v, cache.table, seqs)
            cr.paged_attention(q, cache.k, cache.v, cache.table, seqs, att)
        proj = self._product(*self._quantised(att.flatten(1), H * D), w["out"], h, gate=w["gate1"])
        mid = torch.empty_like(h)
        if cross is not None:
            q = self._product(*self._normed(proj, w["norm3"], residual=h, h=mid), w["cross_q"], h).unflatten(1, (H, D))
            cr.attention(q, *cross, att, seqs=cross_seqs)
            proj, h = self._product(*self._quantised(att.flatten(1), H * D), w["cross_out"], h), mid
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
                 ffn: str = "swiglu", seed: int = 0, device="cuda", context_width: int = 0) -> Block:
    g = torch.Generator(device=device).manual_seed(seed)

    def linear(N, K):
        packed = torch.randint(0, 256, (N, -(-K // 16) * 8), generator=g, device=device, dtype=torch.uint8)
        scales = torch.randint(0x30, 0x39, (N, -(-K // 16)), generator=g, device=device, dtype=torch.uint8)
        t = torch.tensor([0.25 / K ** 0.5], device=device)
        return Linear(packed, scales, t, K, codes)

    def vec(n, mean, std):
        return mean + std * torch.randn(n, generator=g, device=device)
    up = 2 * ffn_width if ffn == "swiglu" else ffn_width
    width = heads * head_dim
    cross = dict(cross_q=linear(width, hidden), cross_kv=linear(2 * width, context_width), cross_out=linear(hidden, width),
                 norm3=vec(hidden, 1, 0.1)) if context_width else {}
    return Block(dict(qkv=linear(3 * heads * head_dim, hidden), out=linear(hidden, heads * head_dim),
                      up=linear(up, hidden), down=linear(hidden, ffn_width), norm1=vec(hidden, 1, 0.1),
                      norm2=vec(hidden, 1, 0.1), q_norm=vec(head_dim, 1, 0.1), k_norm=vec(head_dim, 1, 0.1),
                      qkv_bias=vec(3 * heads * head_dim, 0, 0.1), up_bias=vec(up, 0, 0.1), gate1=vec(hidden, 0.5, 0.1),
                      gate2=vec(hidden, 0.5, 0.1), **cross), heads, head_dim, axis_pairs, ffn)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--ffn", choices=("swiglu", "gelu"), default="swiglu")
    ap.add_argument("--cached", type=int, default=0, help="the tokens are a frame after this many in a cache")
    ap.add_argument("--context", type=int, default=0, help="cross attention to this many states of an encoder")
    a = ap.parse_args()
    codes = torch.int8 if a.tokens <= cr.FEW_TOKENS else torch.float16
    block = random_block(5376, 56, 128, 14336, (16, 24, 24), codes, a.ffn, context_width=4096 if a.context else 0)
    pos = grid_positions(-(-a.tokens // 2304), 36, 64, "cuda")[:a.tokens].contiguous()
    h = torch.randn(a.tokens, 5376, device="cuda").bfloat16()
    cross = block.cross_keys(torch.randn(a.context, 4096, device="cuda").bfloat16()) if a.context else None
    cache = None
    if a.cached:
        cache = FrameCache(a.cached + 8 * a.tokens, a.cached + a.tokens, 56, 128)
        cache.extend(a.cached)
    for _ in range(3):
        block(h, pos, cache, cross)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(5):
        out = block(h, pos, cache, cross)
    end.record()
    torch.cuda.synchronize()
    if cr.device_error():
        raise RuntimeError("a kernel timed out")
    print(f"{a.tokens} tokens, {a.ffn}: {begin.elapsed_time(end) / 5:.3f} ms per block, output rms "
          f"{out.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
