"""Cases of the block's attention and of the cache that it reads, and their plain forms.

Three operators:

- "attend": attention of packed sequences of q to k and v of other lengths (attention): a video's tokens to a text
  encoder's states or to themselves;
- "paged": attention of a chunk of new tokens, or of single ones, over a cache in pages (paged_attention);
- "write": the chunk's keys and values into the cache's pages (cache_write).

`own` False computes them in elementary torch operations in 32 bits, `own` True calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# the video's token count and heads that this library's layers run at, and one latent frame of 36 x 64 tokens
TOKENS, HEADS, FRAME = 19989, 56, 36 * 64
MOST = 4 * TOKENS * TOKENS * HEADS * 128          # operations of the largest listed case


def listed():
    return [
        # a video's tokens to one prompt's encoder states
        {"name": "attend text", "op": "attend", "B": 1, "q": TOKENS, "k": 512, "heads_q": HEADS, "heads_k": HEADS,
         "D": 128, "dtype": "bf16", "causal": False, "empty": False},
        # the block's self attention over a whole video
        {"name": "attend video", "op": "attend", "B": 1, "q": TOKENS, "k": TOKENS, "heads_q": HEADS, "heads_k": HEADS,
         "D": 128, "dtype": "bf16", "causal": False, "empty": False},
        # images of several sizes in one call, prompts of ragged length in a padded batch, one of them empty (the
        # unconditional branch), shared k heads
        {"name": "attend ragged", "op": "attend", "B": 5, "q": 4097, "k": 333, "heads_q": 32, "heads_k": 8, "D": 96,
         "dtype": "fp16", "causal": False, "empty": True},
        # one conditioning token to a prompt: latency
        {"name": "attend one token", "op": "attend", "B": 1, "q": 1, "k": 77, "heads_q": HEADS, "heads_k": HEADS,
         "D": 128, "dtype": "bf16", "causal": False, "empty": False},
        # the encoder's own layers: causal prompts of ragged length
        {"name": "attend prompts", "op": "attend", "B": 8, "q": 1000, "k": 1000, "heads_q": 32, "heads_k": 8, "D": 64,
         "dtype": "bf16", "causal": True, "empty": False},
        # frame by frame: a latent frame's tokens to the cached video and themselves
        {"name": "paged frame", "op": "paged", "B": 1, "q": FRAME, "k": TOKENS, "heads_q": HEADS, "heads_k": HEADS,
         "D": 128, "dtype": "bf16", "page": 256, "causal": False, "first": 0},
        # one token over a long cache
        {"name": "paged one token", "op": "paged", "B": 1, "q": 1, "k": TOKENS, "heads_q": HEADS, "heads_k": HEADS,
         "D": 128, "dtype": "bf16", "page": 64, "causal": False, "first": 0},
        # a batch of single tokens, ragged lengths, shared k heads
        {"name": "paged batch", "op": "paged", "B": 64, "q": 1, "k": 8191, "heads_q": 32, "heads_k": 8, "D": 128,
         "dtype": "fp16", "page": 16, "causal": True, "first": 0},
        # chunks of prompts, ragged, over a window of the cache that begins inside a page
        {"name": "paged chunks", "op": "paged", "B": 5, "q": 700, "k": 4097, "heads_q": 32, "heads_k": 8, "D": 80,
         "dtype": "bf16", "page": 32, "causal": True, "first": 1001},
        # a latent frame into the cache
        {"name": "write frame", "op": "write", "B": 1, "q": FRAME, "k": 3 * FRAME, "heads_k": HEADS, "D": 128,
         "dtype": "bf16", "page": 256, "first": 0},
        # a batch of single tokens: latency
        {"name": "write tokens", "op": "write", "B": 16, "q": 1, "k": 257, "heads_k": 8, "D": 128, "dtype": "bf16",
         "page": 16, "first": 0},
        # ragged chunks
        {"name": "write chunks", "op": "write", "B": 9, "q": 1500, "k": 2049, "heads_k": 8, "D": 80, "dtype": "fp16",
         "page": 32, "first": 77},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "paged", "paged", "write"])
    heads_k = _log(rng, 1, HEADS)
    shared = rng.choice([1, 1, 2, 4, 7])
    while heads_k * shared > HEADS:
        shared = max(1, shared // 2)
    c = {"op": op, "D": rng.choice([64, 72, 80, 96, 128, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "attend":
        same = rng.random() < 0.4                          # self attention, or an encoder's states
        q = _log(rng, 1, TOKENS)
        c.update(B=_log(rng, 1, 8), q=q, k=q if same else _log(rng, 1, 2048), heads_q=heads_k * shared, heads_k=heads_k,
                 causal=same and rng.random() < 0.4, empty=not same and rng.random() < 0.3)
    elif op == "paged":
        q = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        c.update(B=_log(rng, 1, 64), q=q, k=max(q, _log(rng, 1, 32768)), heads_q=heads_k * shared, heads_k=heads_k,
                 page=rng.choice([16, 32, 64, 128, 256]), causal=rng.random() < 0.5,
                 first=_log(rng, 1, 1000) if rng.random() < 0.3 else 0)
    else:
        q = _log(rng, 1, 4096)
        c.update(B=_log(rng, 1, 64), q=q, k=q + rng.randrange(2048), heads_k=heads_k, page=rng.choice([16, 32, 64, 128, 256]),
                 first=_log(rng, 1, 1000) if rng.random() < 0.3 else 0)
    while c["B"] > 1 and (c["B"] * max(c["q"], c["k"]) * heads_k > TOKENS * HEADS or work(c)["flops"] > MOST // 4):
        c["B"] = max(1, c["B"] // 2)
    return c


# ---------------------------------------------------------------- sequences
def _ragged(longest, B):
    """Lengths of B sequences: the longest first, then spread from a quarter of it up."""
    return [longest] + [max(1, int(longest * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(1, B)]


def _lengths(c):
    """(q lengths, k lengths) of the case's sequences."""
    B = c["B"]
    q = _ragged(c["q"], B)
    if c["op"] == "attend":
        k = list(q) if c["causal"] or c["q"] == c["k"] else _ragged(c["k"], B)
        if c["empty"]:
            k[-1] = 0
        return q, k
    return q, [max(a, b) for a, b in zip(q, _ragged(c["k"], B))]


def _pairs(c):
    """Visible (row, key) pairs."""
    n = 0
    for q, k in zip(*_lengths(c)):
        n += q * k - q * (q - 1) // 2 if c["causal"] else q * k
    return n


def work(c):
    q, k = _lengths(c)
    D = c["D"]
    if c["op"] == "write":
        return {"bytes": 8 * sum(q) * c["heads_k"] * D, "flops": 0}
    return {"bytes": 4 * D * (sum(q) * c["heads_q"] + sum(k) * c["heads_k"]), "flops": 4 * _pairs(c) * c["heads_q"] * D}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    D, Hk = case["D"], case["heads_k"]
    q_len, k_len = _lengths(case)

    def rand(*shape, std=1.0):
        # heads after their norm: unit values, a few channels larger
        x = torch.randn(*shape, generator=g, device=dev)
        x[..., :: max(8, D // 8)] *= 2.0
        return x.mul_(std).to(dt)

    s = {"case": case, "q_len": q_len, "k_len": k_len}
    q_start = [sum(q_len[:i]) for i in range(len(q_len))]
    rows = sum(q_len) + (5 if case["B"] > 1 else 0)            # rows behind the last sequence stay as they are
    s["q_start"] = q_start
    if case["op"] == "attend":
        most = max(k_len)
        k_start = [i * most for i in range(case["B"])]         # the encoder's padded batch
        s["k"], s["v"] = rand(max(1, case["B"] * most), Hk, D), rand(max(1, case["B"] * most), Hk, D)
    else:
        page, first = case["page"], case["first"]
        k_start = [first] * case["B"]
        need = [-(-(first + k) // page) for k in k_len]
        lead = first // page                                   # pages before the window are free again
        used = sum(n - lead for n in need)
        order = torch.randperm(used + 3, generator=g, device=dev).to(torch.int32)
        table = torch.full((case["B"], max(need) + 1), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, lead:n] = order[at:at + n - lead]
            at += n - lead
        s["pages"] = table
        s["k_cache"], s["v_cache"] = rand(used + 3, page, Hk, D), rand(used + 3, page, Hk, D)
        if case["op"] == "write":
            qkv = rand(rows, 3 * Hk, D)                        # the packed product's output
            s["k"], s["v"] = qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
        # where every key of a sequence lies, for the plain form's gather
        s["where"] = []
        for b, k in enumerate(k_len):
            p = torch.arange(first, first + k, device=dev)
            s["where"].append((table[b, p // page].long(), p % page))
    s["k_start"] = k_start
    s["seqs"] = torch.tensor(list(zip(q_start, q_len, k_start, k_len)), dtype=torch.int32, device=dev)
    if case["op"] != "write":
        s["q"] = rand(rows, case["heads_q"], D)
        s["out"] = torch.zeros(rows, case["heads_q"], D, dtype=dt, device=dev)
    return s


def run(s):
    if own:
        return {"attend": _own_attend, "paged": _own_paged, "write": _own_write}[s["case"]["op"]](s)
    return _plain_write(s) if s["case"]["op"] == "write" else _plain_attention(s)


# ---------------------------------------------------------------- the library's calls
def _own_attend(s):
    import rotated_w4a8_int8_gb300 as cr
    cr.attention(s["q"], s["k"], s["v"], s["out"], seqs=s["seqs"], causal=s["case"]["causal"])
    return s["out"]


def _own_paged(s):
    import rotated_w4a8_int8_gb300 as cr
    cr.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["seqs"], s["out"], causal=s["case"]["causal"])
    return s["out"]


def _own_write(s):
    import rotated_w4a8_int8_gb300 as cr
    cr.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["seqs"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


# ---------------------------------------------------------------- plain forms
def _keys(s, b):
    """k and v [heads_k, keys, D] of sequence b."""
    if s["case"]["op"] == "attend":
        a, n = s["k_start"][b], s["k_len"][b]
        k, v = s["k"][a:a + n], s["v"][a:a + n]
    else:
        page, row = s["where"][b]
        k, v = s["k_cache"][page, row], s["v_cache"][page, row]
    return k.transpose(0, 1), v.transpose(0, 1)


def _plain_attention(s):
    c, out = s["case"], s["out"]
    scale, group = c["D"] ** -0.5, c["heads_q"] // c["heads_k"]
    for b, (n, m) in enumerate(zip(s["q_len"], s["k_len"])):
        a = s["q_start"][b]
        if m == 0:
            out[a:a + n] = 0
            continue
        k, v = _keys(s, b)
        hidden = None
        if c["causal"] and n > 1:
            i = torch.arange(n, device=out.device)
            hidden = torch.arange(m, device=out.device)[None, :] > (m - n + i)[:, None]
        # as many heads at a time as keep the scores under 2 GB
        step = max(1, min(c["heads_k"], (1 << 29) // (group * n * m)))
        for h in range(0, c["heads_k"], step):
            x = s["q"][a:a + n, h * group:(h + step) * group].transpose(0, 1).float()
            x = x.reshape(-1, group * n, c["D"])
            p = torch.matmul(x, k[h:h + step].float().transpose(1, 2)).mul_(scale)
            if hidden is not None:
                p.view(-1, group, n, m).masked_fill_(hidden, float("-inf"))
            p.sub_(p.amax(2, keepdim=True)).exp_()
            y = torch.matmul(p, v[h:h + step].float()) / p.sum(2, keepdim=True)
            out[a:a + n, h * group:(h + step) * group] = y.view(-1, n, c["D"]).transpose(0, 1)
    return out


def _plain_write(s):
    for b, (n, m) in enumerate(zip(s["q_len"], s["k_len"])):
        page, row = s["where"][b]
        a = s["q_start"][b]
        s["k_cache"].index_put_((page[m - n:], row[m - n:]), s["k"][a:a + n])
        s["v_cache"].index_put_((page[m - n:], row[m - n:]), s["v"][a:a + n])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def exact(case, seed):
    if case["op"] != "write" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "write":
        for which in ("k", "v"):                     # row by row of the flattened cache
            flat = s[which + "_cache"].view(-1, case["heads_k"], case["D"])
            for b, (a, n, f, m) in enumerate(s["seqs"].tolist()):
                pos = torch.arange(f + m - n, f + m, device=flat.device)
                flat[s["pages"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]] = s[which][a:a + n]
        return {"k": s["k_cache"].double(), "v": s["v_cache"].double()}
    f64 = torch.float64
    D, group = case["D"], case["heads_q"] // case["heads_k"]
    out = s["out"].to(f64)
    for b, (a, n, f, m) in enumerate(s["seqs"].tolist()):
        if m == 0:
            continue
        if case["op"] == "attend":
            rows = torch.arange(f, f + m, device=out.device)
            ks, vs = s["k"], s["v"]
        else:
            pos = torch.arange(f, f + m, device=out.device)
            rows = s["pages"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]
            ks, vs = (s[w].view(-1, case["heads_k"], D) for w in ("k_cache", "v_cache"))
        for h in range(case["heads_q"]):
            k, v = ks[rows, h // group].to(f64), vs[rows, h // group].to(f64)
            for i in range(0, n, 2048):              # blocks of rows: log of the sum, then weights
                e = min(n, i + 2048)
                z = s["q"][a + i:a + e, h].to(f64) @ k.t() / math.sqrt(D)
                if case["causal"]:
                    see = m - n + torch.arange(i, e, device=out.device)
                    z = z.where(torch.arange(m, device=out.device) <= see[:, None], -math.inf)
                out[a + i:a + e, h] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v
    return out
