"""Attention in 64 bits, and how far a kernel's result may be from it.

Bound of an output element, with u half a step of the operands' type (finfo.eps / 2), p_j the weights and
A = sum_j p_j |v_j| (both from 64 bits):

    u A          the weights' rounding for their product with v
  + u |out|      the output's rounding
  + 2 e A        the weights' own error e (numerator and sum): a score's FP32 sum of D products (D 2^-23 of the sum of
                 their absolute values), its scaling and the exponential (2^-20 of the largest score, and 2^-20)
  + n 2^-30 V    FP16 only: weights below 2^-20 of the largest are subnormal (n keys, V = max |v|; a step is 2^-24 where
                 the largest weight is at least 2^6)
  + a subnormal step of the output.
"""
import math

import torch


def reference(q, k, v, seqs, scale, causal, out):
    """(expected, bound) in float64; rows in no sequence keep `out` with bound 0.  k, v: one [keys, heads_k, D] tensor
    each, or a function of a sequence's number that gives its keys."""
    u = torch.finfo(q.dtype).eps / 2
    D, group = q.shape[2], q.shape[1] // (k[0] if isinstance(k, list) else k).shape[1]
    want, bound = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64, device=out.device)
    for b, (a, n, f, m) in enumerate(seqs):
        if n == 0:
            continue
        kk, vv = (k[b], v[b]) if isinstance(k, list) else (k[f:f + m], v[f:f + m])
        kk, vv = (t.double().repeat_interleave(group, 1).transpose(0, 1) for t in (kk, vv))
        qq = q[a:a + n].double().transpose(0, 1)
        see = torch.full((n,), m, device=q.device)
        if causal:
            see = (m - n + 1 + torch.arange(n, device=q.device)).clamp(max=m)
        hidden = torch.arange(m, device=q.device)[None, :] >= see[:, None]
        s = torch.matmul(qq, kk.transpose(1, 2)) * scale
        size = (torch.matmul(qq.abs(), kk.abs().transpose(1, 2)) * scale).masked_fill(hidden, 0.0)
        s = s.masked_fill(hidden, -math.inf)
        p = torch.softmax(s, 2) if m else s
        p = torch.where((see <= 0)[None, :, None], torch.zeros_like(p), p)
        y, A = torch.matmul(p, vv), torch.matmul(p, vv.abs())
        e = torch.zeros(p.shape[:2], dtype=torch.float64, device=q.device)
        top = 0.0
        if m:
            e = size.amax(2) * (D * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -20
            top = float(vv.abs().max())
        lim = u * (A + y.abs()) + 2 * e[:, :, None] * A + torch.finfo(q.dtype).tiny * u
        if q.dtype == torch.float16:
            lim = lim + m * 2.0 ** -30 * top
        want[a:a + n], bound[a:a + n] = y.transpose(0, 1), lim.transpose(0, 1)
        bound[a:a + n][see <= 0] = 0.0
    return want, bound


def check(got, want, bound):
    assert bool(torch.isfinite(got).all())
    over = (got.double() - want).abs() - bound
    assert float(over.max()) <= 0, (float(over.max()), float(((got.double() - want).abs() / (bound + 1e-300)).max()),
                                    int((over > 0).sum()))


def paged(k, v, seqs, page, window=0, spare=2, seed=0):
    """Caches, table and seqs that hold each sequence's keys at positions window, window + 1, ...  Places that hold none
    are NaN; entries of the table that are not needed are out of range."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(window + m) // page) for _, _, _, m in seqs]
    lead = window // page
    total = sum(n - lead for n in need if n > lead) + spare
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(seqs), max(need) + 1), -7, dtype=torch.int32)
    caches = [torch.full((total, page, *t.shape[1:]), math.nan, dtype=t.dtype, device=t.device) for t in (k, v)]
    for b, (_, _, f, m) in enumerate(seqs):
        for i in range(lead, need[b]):
            table[b, i] = order.pop()
        pos = torch.arange(window, window + m)
        at = (table[b].long()[pos // page].to(k.device), (pos % page).to(k.device)) if m else None
        for c, t in zip(caches, (k, v)):
            if m:
                c[at] = t[f:f + m]
    where = torch.tensor([(a, n, window, m) for a, n, _, m in seqs], dtype=torch.int32, device=k.device)
    return caches[0], caches[1], table.to(k.device), where
