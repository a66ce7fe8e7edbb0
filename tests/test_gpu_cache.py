"""cache_write: every token's keys and values in their place, everything else in the caches untouched, and the chunk's
attention over what was written."""
import pytest
import torch

from attention_util import check, reference
from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def setup(seqs, heads, D, page, dtype, seed=0, spare=3):
    """q, k, v of the rows, caches of random contents, a table that holds the sequences' positions."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = max(a + n for a, n, _, _ in seqs) + 2
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)
    need = [-(-(f + m) // page) for _, _, f, m in seqs]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(seqs), max(need) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    qkv = rand(rows, 3 * heads, D)
    caches = [rand(sum(need) + spare, page, heads, D) for _ in range(2)]
    return qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:], caches, table.to(DEV)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("heads,D,dtype", [(1, 8, torch.float16), (3, 72, torch.bfloat16), (56, 128, torch.bfloat16)])
@pytest.mark.parametrize("seqs", [[(0, 1, 0, 1)], [(0, 300, 0, 300)], [(2, 7, 0, 40), (9, 0, 3, 5), (12, 130, 21, 131), (150, 1, 0, 17)]])
def test_places(page, heads, D, dtype, seqs):
    import rotated_w4a8_int8_gb300 as cr
    _, k, v, caches, table = setup(seqs, heads, D, page, dtype)
    want = [c.clone() for c in caches]
    for b, (a, n, f, m) in enumerate(seqs):
        for i in range(n):
            pos = f + m - n + i
            for c, t in zip(want, (k, v)):
                c[table[b, pos // page], pos % page] = t[a + i]
    cr.cache_write(k, v, *caches, table, torch.tensor(seqs, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    assert all(torch.equal(c, w) for c, w in zip(caches, want))


def test_caches_of_other_strides():
    # heads outermost, rows within them: [heads, pages, rows, D] seen as [pages, rows, heads, D]
    import rotated_w4a8_int8_gb300 as cr
    seqs = [(0, 33, 0, 50), (33, 20, 0, 20)]
    _, k, v, caches, table = setup(seqs, 4, 64, 16, torch.bfloat16)
    other = [c.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for c in caches]
    where = torch.tensor(seqs, dtype=torch.int32, device=DEV)
    cr.cache_write(k, v, *caches, table, where)
    cr.cache_write(k, v, *other, table, where)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(caches, other))


@pytest.mark.parametrize("causal", [False, True])
def test_chunks_written_and_attended_to(causal):
    """Three chunks of two sequences, each written and then attended to; the second sequence drops what lies before a
    window from its second chunk on."""
    import rotated_w4a8_int8_gb300 as cr
    heads, D, page, scale = 4, 96, 32, 96 ** -0.5
    g = torch.Generator(device=DEV).manual_seed(5)
    chunks = [(40, 17), (1, 100), (130, 1)]
    total = [sum(c[i] for c in chunks) for i in range(2)]
    order = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.stack([order[:10], order[10:]]).to(DEV)
    assert max(total) <= 320
    caches = [torch.full((20, page, heads, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kept = [[], []]
    done = [0, 0]
    for step, lens in enumerate(chunks):
        qkv = torch.randn(sum(lens), 3 * heads, D, generator=g, device=DEV).to(torch.bfloat16)
        q, k, v = qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
        first = [0, 11 if step else 0]
        done = [d + n for d, n in zip(done, lens)]
        seqs = [(0, lens[0], first[0], done[0] - first[0]), (lens[0], lens[1], first[1], done[1] - first[1])]
        where = torch.tensor(seqs, dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        cr.cache_write(k, v, *caches, table, where)
        cr.paged_attention(q, *caches, table, where, out, causal=causal)
        torch.cuda.synchronize()
        assert cr.device_error() == 0
        for b in range(2):
            a, n = seqs[b][:2]
            kept[b].append((k[a:a + n], v[a:a + n]))
        keys = [torch.cat([x[0] for x in kept[b]])[first[b]:] for b in range(2)]
        values = [torch.cat([x[1] for x in kept[b]])[first[b]:] for b in range(2)]
        check(out, *reference(q, keys, values, seqs, scale, causal, out))


def test_bad_sequences_and_pages_are_left_out_and_reported():
    """Refused by the kernels' own bounds: nothing outside the tensors is touched, the rest of the call is done."""
    import rotated_w4a8_int8_gb300 as cr
    seqs = [(0, 20, 0, 20), (20, 20, 0, 40), (40, 5, 0, 5)]
    q, k, v, caches, table = setup(seqs, 2, 64, 16, torch.float16)
    before = [c.clone() for c in caches]

    def write(bad, tab=table):
        for c, w in zip(caches, before):
            c.copy_(w)
        rows = [list(s) for s in seqs]
        rows[1] = bad
        cr.cache_write(k, v, *caches, tab, torch.tensor(rows, dtype=torch.int32, device=DEV))
        return cr.device_error()

    for bad in ([20, 20, 0, 4000], [-1, 3, 0, 9], [20, 2 ** 30, 0, 2 ** 30], [20, 9, 0, 8], [20, 9, -3, 12], [2 ** 31 - 1, 1, 0, 1]):
        assert write(bad) == 16
        where = (table[0, 0].long(), 0)
        assert torch.equal(caches[0][where], k[0]) and torch.equal(caches[0][table[2, 0].long(), 4], k[44])
        assert all(torch.equal(c[table[1, :3].long()], w[table[1, :3].long()]) for c, w in zip(caches, before))
    for entry in (-1, caches[0].shape[0], 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 2] = entry
        assert write([20, 20, 0, 40], tab) == 17
        assert torch.equal(caches[0][table[1, 1].long(), 4], k[20])
    assert cr.device_error() == 0


@pytest.mark.parametrize("kernel", [(1, 2), (2, 1), (3, 2)])
def test_attention_reports_bad_sequences_and_pages(kernel):
    import rotated_w4a8_int8_gb300 as cr
    seqs = [(0, 20, 0, 20), (20, 20, 0, 40), (40, 5, 0, 5)]
    q, k, v, caches, table = setup(seqs, 2, 64, 16, torch.float16)
    where = torch.tensor(seqs, dtype=torch.int32, device=DEV)
    want = torch.full_like(q, 2.0)
    cr.attention_selftest(q, *caches, want, *kernel, pages=table, seqs=where)
    assert cr.device_error() == 0
    for bad in ([20, 20, 0, 4000], [-1, 3, 0, 9], [20, 2 ** 30, 0, 2 ** 30], [20, 9, -3, 12], [2 ** 31 - 1, 1, 0, 1]):
        where[1] = torch.tensor(bad, dtype=torch.int32)
        out = torch.full_like(q, 2.0)
        cr.attention_selftest(q, *caches, out, *kernel, pages=table, seqs=where)
        assert cr.device_error() == 16
        assert torch.equal(out[:20], want[:20]) and torch.equal(out[40:], want[40:]) and bool((out[20:40] == 2).all())
        out.fill_(2.0)
        cr.attention_selftest(q, k, v, out, *kernel, seqs=where)
        assert cr.device_error() == 16 and bool((out[20:40] == 2).all())
    where[1] = torch.tensor(seqs[1], dtype=torch.int32)
    for entry in (-1, caches[0].shape[0], 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 2] = entry
        out = torch.full_like(q, 2.0)
        cr.attention_selftest(q, *caches, out, *kernel, pages=tab, seqs=where)
        assert cr.device_error() == 17
        assert torch.equal(out[:20], want[:20]) and torch.equal(out[40:], want[40:])
    assert cr.device_error() == 0
