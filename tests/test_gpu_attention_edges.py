"""attention, paged_attention and cache_write where calls meet: captured and replayed on new lengths, on other streams and
two at once, one launched while the one before still runs; offsets past 2^31 elements, many sequences, values that are no
numbers, waits that run out.  The bound is derived in attention_util.py."""
import math
import time

import pytest
import torch

from attention_util import check, paged, reference
from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF, HF = torch.bfloat16, torch.float16
EACH = [(1, 1), (1, 4), (2, 1), (3, 1), (3, 4)]        # kernel, CTAs that share keys


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def rand(*shape, seed=0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def i32(rows):
    return torch.tensor(rows, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows,heads_q,heads_k", [(3, 4, 2), (200, 4, 4), (700, 2, 1)])
def test_captured_and_replayed_on_new_lengths(rows, heads_q, heads_k):
    """The graph holds no length: seqs, tables and contents are read at each replay."""
    import rotated_w4a8_int8_gb300 as cr
    D, page = 64, 32
    q, k, v = rand(rows, heads_q, D), rand(900, heads_k, D, seed=1), rand(900, heads_k, D, seed=2)
    kc, vc = (torch.full((64, page, heads_k, D), math.nan, dtype=BF, device=DEV) for _ in range(2))
    table, seqs, out = torch.zeros(2, 30, dtype=torch.int32, device=DEV), torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros_like(q)
    run = lambda: cr.paged_attention(q, kc, vc, table, seqs, out, causal=True)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens, window in [(((1, 1), (rows - 1, rows)), 0), (((rows - 2, rows + 100), (2, 800 - rows)), 0), (((0, 0), (rows, 777)), 45)]:
        where, a, f = [], 0, 0
        for n, m in lens:
            where.append((a, n, f, m))
            a, f = a + n, f + max(m, 0)
        nk, nv, t, w = paged(k, v, where, page, window)
        kc[:nk.shape[0]], vc[:nv.shape[0]] = nk, nv
        table.zero_()
        table[:, :t.shape[1]] = t
        seqs.copy_(w)
        out.fill_(3.0)
        want = reference(q, k, v, where, D ** -0.5, True, out)
        graph.replay()
        torch.cuda.synchronize()
        assert cr.device_error() == 0
        check(out, *want)


def test_streams():
    """The given stream is used, and two calls may run at once."""
    import rotated_w4a8_int8_gb300 as cr
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    sets = [(rand(300, 4, 128, seed=s), rand(2000, 4, 128, seed=s + 10), rand(2000, 4, 128, seed=s + 20)) for s in range(2)]
    small = [(rand(1, 4, 128, seed=s), k, v) for s, (_, k, v) in enumerate(sets)]
    outs = [torch.zeros_like(q) for q, _, _ in sets + small]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (q, k, v) in enumerate(sets + small):
            cr.attention(q, k, v, outs[i], stream=(a, b)[i % 2])
    torch.cuda.synchronize()
    for o, (q, k, v) in zip(outs, sets + small):
        check(o, *reference(q, k, v, [(0, q.shape[0], 0, 2000)], 128 ** -0.5, False, o))


@pytest.mark.parametrize("rows,page", [(1, 16), (40, 64), (300, 64)])
def test_chain_equals_synchronised_calls(rows, page):
    """Every call is launched while the one before it still runs, reads what that one writes and overwrites what it
    reads: rotary positions in place, keys and values into the cache, attention over them, whose output is the next
    layer's input."""
    import rotated_w4a8_int8_gb300 as cr
    H, D, layers = 4, 64, 10
    x0 = rand(rows, H, D)
    x, y, out = (torch.empty_like(x0) for _ in range(3))
    caches = [torch.empty(60, page, H, D, dtype=BF, device=DEV) for _ in range(2)]
    start = [rand(60, page, H, D, seed=s) for s in (3, 4)]
    table = torch.arange(59, -1, -1, dtype=torch.int32, device=DEV).view(1, 60)
    seqs = [i32([(0, rows, 0, 100 + rows * (i + 1))]) for i in range(2)]
    pos = torch.arange(rows, dtype=torch.int32, device=DEV).view(-1, 1)
    freq = torch.tensor(cr.rope_inv_freq([32]), dtype=torch.float64, device=DEV)

    def run(after=lambda: None):
        x.copy_(x0)
        for c, s in zip(caches, start):
            c.copy_(s)
        after()
        for i in range(layers):
            cr.qk_norm_rope(x, x, pos, freq, [32], y, out)
            after()
            cr.cache_write(out, x, *caches, table, seqs[i % 2])
            after()
            cr.paged_attention(y, *caches, table, seqs[i % 2], x, scale=0.02)
            after()
            cr.attention(y, out, x, out2, scale=1.0)
            after()
            x.copy_(out2)
        return x

    out2 = torch.empty_like(x0)
    want = run(torch.cuda.synchronize).clone()
    assert bool(torch.isfinite(want.float()).all()) and not torch.equal(want, x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want) and cr.device_error() == 0


@pytest.mark.parametrize("kernel", EACH)
def test_runs_agree_bit_for_bit(kernel):
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = rand(150, 8, 96, dtype=HF), rand(1500, 2, 96, seed=1, dtype=HF), rand(1500, 2, 96, seed=2, dtype=HF)
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        cr.attention_selftest(q, k, v, o, *kernel)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("kernel", EACH)
def test_offsets_past_32_bits(kernel):
    """Pages 2^30 elements apart and rows 2^24: the last ones lie more than 2^31 elements behind the first."""
    import rotated_w4a8_int8_gb300 as cr
    D, H, page = 64, 2, 64
    far = torch.empty(7 * 2 ** 29 + 2 ** 14, dtype=BF, device=DEV)
    pages = far.as_strided((4, page, H, D), (2 ** 30, H * D, D, 1))
    vpages = far.as_strided((4, page, H, D), (2 ** 30, H * D, D, 1), 2 ** 13)      # after the keys of the same page
    k, v = rand(4 * page, H, D, seed=1), rand(4 * page, H, D, seed=2)
    rows = far.as_strided((200, H, D), (2 ** 24, D, 1), 2 ** 15)
    q = rand(200, H, D)
    rows.copy_(q)
    out = far.as_strided((200, H, D), (2 ** 24, D, 1), 2 ** 16)
    out.fill_(7.0)
    table, seqs = i32([[2, 0, 3, 1]]), i32([(0, 200, 0, 4 * page)])
    cr.cache_write(k[56:], v[56:], pages, vpages, table, seqs)           # the last 200 tokens
    cr.cache_write(k[:56], v[:56], pages, vpages, table, i32([(0, 56, 0, 56)]))
    cr.attention_selftest(rows, pages, vpages, out, *kernel, pages=table, seqs=seqs)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    for i, p in enumerate([2, 0, 3, 1]):
        assert torch.equal(pages[p], k[i * page:(i + 1) * page]) and torch.equal(vpages[p], v[i * page:(i + 1) * page])
    check(out, *reference(q, k, v, [(0, 200, 0, 4 * page)], D ** -0.5, False, out))
    # the same rows as keys and values
    cr.attention_selftest(rows[:5], rows, rows, out[:5], *kernel)
    torch.cuda.synchronize()
    check(out[:5], *reference(q[:5], q, q, [(0, 5, 0, 200)], D ** -0.5, False, out[:5]))


@pytest.mark.parametrize("kernel", [(1, 2), (2, 1), (3, 2), None])
def test_many_sequences(kernel):
    import rotated_w4a8_int8_gb300 as cr
    g = torch.Generator().manual_seed(4)
    lens = [(int(n), int(m)) for n, m in zip(torch.randint(0, 9, (500,), generator=g), torch.randint(0, 70, (500,), generator=g))]
    lens[77] = (300, 400)
    order = torch.randperm(500, generator=g).tolist()      # rows of the sequences in no order
    at, seqs, f = 0, [None] * 500, 0
    for b in order:
        n, m = lens[b]
        seqs[b] = (at, n, f, m)
        at, f = at + n, f + m
    q, k, v = rand(at, 2, 64), rand(f, 1, 64, seed=1), rand(f, 1, 64, seed=2)
    out = torch.empty_like(q)
    if kernel:
        cr.attention_selftest(q, k, v, out, *kernel, seqs=i32(seqs), causal=True)
    else:
        cr.attention(q, k, v, out, seqs=i32(seqs), causal=True)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    check(out, *reference(q, k, v, seqs, 0.125, True, out))


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads_q", [2, 6])
def test_rows_behind_a_sequence_have_no_say(kernel, dtype, heads_q):
    """The same bits whatever the next sequence's rows, and rows in no sequence, hold: they lie in the same tiles."""
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = rand(300, heads_q, 64, dtype=dtype), rand(900, 2, 64, seed=1, dtype=dtype), rand(900, 2, 64, seed=2, dtype=dtype)
    k = (k * torch.linspace(0.5, 1.5, 900, device=DEV)[:, None, None]).to(dtype)
    seqs, outs = [(0, 21, 0, 600), (21, 137, 600, 300), (170, 100, 0, 900)], []
    for factor in (1.0, 30.0, -1000.0, math.inf, math.nan):
        x = q.clone()
        for a, n in ((21, 137), (158, 12), (270, 30)):
            x[a:a + n] *= factor
        out = torch.zeros_like(q)
        cr.attention_selftest(x, k, v, out, *kernel, seqs=i32(seqs))
        outs.append(torch.cat([out[:21], out[170:270]]))
    torch.cuda.synchronize()
    assert cr.device_error() == 0 and bool(torch.isfinite(outs[0]).all()) and all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("kernel", [(1, 1), (1, 2), (2, 1), (3, 2), None])
def test_most_sequences(kernel):
    """As many sequences as a call takes, their rows in no order: a page each, written and attended to."""
    import rotated_w4a8_int8_gb300 as cr
    B, n, m, D, page = 65535, 3, 5, 64, 16
    order = torch.randperm(B, generator=torch.Generator().manual_seed(8)).to(DEV)
    q, k, v = rand(B * n, 1, D), rand(B * n, 1, D, seed=1), rand(B * n, 1, D, seed=2)
    kc, vc = rand(B, page, 1, D, seed=3), rand(B, page, 1, D, seed=4)
    table = torch.arange(B - 1, -1, -1, dtype=torch.int32, device=DEV).view(B, 1)
    seqs = torch.stack([order * n, torch.full_like(order, n), order % 11, torch.full_like(order, m)], 1).to(torch.int32)
    want_k, want_v = kc.clone(), vc.clone()
    where = (table[:, :1].long(), (order % 11)[:, None] + m - n + torch.arange(n, device=DEV))
    rows = order[:, None] * n + torch.arange(n, device=DEV)
    want_k[where], want_v[where] = k[rows], v[rows]
    cr.cache_write(k, v, kc, vc, table, seqs)
    out = torch.empty_like(q)
    if kernel:
        cr.attention_selftest(q, kc, vc, out, *kernel, pages=table, seqs=seqs, causal=True)
    else:
        cr.paged_attention(q, kc, vc, table, seqs, out, causal=True)
    torch.cuda.synchronize()
    assert cr.device_error() == 0 and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    keys = (table[:, :1].long(), (order % 11)[:, None] + torch.arange(m, device=DEV))
    kk, vv, qq = want_k[keys][:, :, 0].double(), want_v[keys][:, :, 0].double(), q[rows][:, :, 0].double()
    s, size = torch.matmul(qq, kk.transpose(1, 2)) / 8, torch.matmul(qq.abs(), kk.abs().transpose(1, 2)) / 8
    hidden = torch.arange(m, device=DEV) > m - n + torch.arange(n, device=DEV)[:, None]
    p = torch.softmax(s.masked_fill(hidden, -math.inf), 2)
    y, A, u = p @ vv, p @ vv.abs(), torch.finfo(BF).eps / 2
    e = size.amax(2, keepdim=True) * (D * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -20
    check(out[rows][:, :, 0], y, u * (A + y.abs()) + 2 * e * A + torch.finfo(BF).tiny * u)


@pytest.mark.parametrize("kernel", EACH)
def test_values_that_are_no_numbers(kernel):
    """A row of q that is NaN stays alone; an Inf or NaN among the values shows in its column of every row that sees the
    key, a NaN key in every row."""
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = rand(40, 2, 64), rand(300, 2, 64, seed=1), rand(300, 2, 64, seed=2)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    cr.attention_selftest(q, k, v, clean, *kernel)
    bad = q.clone()
    bad[7, 1, 3] = math.nan
    cr.attention_selftest(bad, k, v, out, *kernel)
    torch.cuda.synchronize()
    assert bool(out[7, 1].isnan().all())
    out[7, 1] = clean[7, 1]
    assert torch.equal(out, clean)
    bad = v.clone()
    bad[123, 0, 5], bad[299, 1, 6] = math.inf, math.nan
    cr.attention_selftest(q, k, bad, out, *kernel)
    torch.cuda.synchronize()
    assert bool((out[:, 0, 5] == math.inf).all()) and bool(out[:, 1, 6].isnan().all())
    out[:, 0, 5], out[:, 1, 6] = clean[:, 0, 5], clean[:, 1, 6]
    assert torch.equal(out, clean)
    bad = k.clone()
    bad[200, 1, 0] = math.nan
    cr.attention_selftest(q, bad, v, out, *kernel)
    torch.cuda.synchronize()
    assert bool(out[:, 1].isnan().all()) and torch.equal(out[:, 0], clean[:, 0])


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page", [0, 16])
def test_scores_of_minus_infinity(kernel, dtype, page):
    """Keys with such a score have no weight; a row with no other key is 0 / 0, a row that sees no key zeros."""
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = (rand(n, h, 64, seed=n + h, dtype=dtype) for n, h in ((50, 4), (400, 2), (400, 2)))
    q[:, :, 0] = 1.0
    k[:200, :, 0], k[200:300, :, 0] = -math.inf, -math.inf             # all of the first 200, 100 of the others
    seqs = [(0, 20, 0, 200), (20, 10, 200, 200), (30, 0, 5, 5), (30, 20, 390, 10)]
    table, where, kk, vv = None, i32(seqs), k, v
    if page:
        kk, vv, table, where = paged(k, v, seqs, page, 5)
    out = torch.full_like(q, 3.0)
    cr.attention_selftest(q, kk, vv, out, *kernel, pages=table, seqs=where, causal=True)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    assert bool(out[:20].isnan().all()) and bool((out[30:40] == 0).all())
    finite = [(20, 10, 300, 100), (30, 20, 390, 10)]
    want, bound = reference(q, k, v, finite, 0.125, True, torch.zeros_like(out))
    check(out[20:], want[20:], bound[20:])


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_infinite_values_of_light_keys(kernel, dtype):
    """Weights down to 2^-22 of the largest one: an infinite value stays the infinity that it is."""
    import rotated_w4a8_int8_gb300 as cr
    n, D = 320, 64
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k = torch.zeros(20, 1, D, dtype=dtype, device=DEV), torch.zeros(n, 1, D, dtype=dtype, device=DEV)
    q[:, 0, :3] = 1.0
    q[:, 0, 3] = torch.arange(20, device=DEV).to(dtype) / 20
    k[:, 0, 0] = -(torch.rand(n, generator=g, device=DEV) * 14).to(dtype)            # exp(-15.25) = 2^-22
    k[:, 0, 3] = -torch.rand(n, generator=g, device=DEV).to(dtype)
    k[0] = 0.0
    out = torch.empty_like(q)
    for first in range(0, n, D):
        v, d = torch.ones(n, 1, D, dtype=dtype, device=DEV), torch.arange(D, device=DEV)
        v[first + d, 0, d] = torch.where(d % 2 == 0, math.inf, -math.inf).to(dtype)
        cr.attention_selftest(q, k, v, out, *kernel, scale=1.0)
        torch.cuda.synchronize()
        assert bool((out[:, 0, 0::2] == math.inf).all()) and bool((out[:, 0, 1::2] == -math.inf).all())


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_equal_weights_of_many_keys(kernel, dtype):
    """All scores zero: every weight is 1 / n, the smallest that n keys can share."""
    import rotated_w4a8_int8_gb300 as cr
    n = 30000
    q, k, v = torch.zeros(130, 1, 64, dtype=dtype, device=DEV), rand(n, 1, 64, dtype=dtype), rand(n, 1, 64, seed=1, dtype=dtype) + 1
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel)
    torch.cuda.synchronize()
    check(out, *reference(q, k, v, [(0, 130, 0, n)], 0.125, False, out))


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [4, 150])
def test_large_scores(kernel, dtype, rows):
    """Scores up to 2^37, whose FP32 sums are exact (whole numbers below 2^14, times a power of two): what is left is the
    weights of the largest ones, equal where there are several.  Rows past the first half have ordinary scores."""
    import rotated_w4a8_int8_gb300 as cr
    g = torch.Generator(device=DEV).manual_seed(rows)
    whole = lambda *shape: torch.randint(-8, 9, shape, generator=g, device=DEV).to(dtype)
    q, k, v = whole(rows, 2, 128) * 2.0 ** 12, whole(700, 2, 128) * 2.0 ** 12, rand(700, 2, 128, seed=1, dtype=dtype)
    q[rows // 2:] *= 2.0 ** -25 if dtype == BF else 2.0 ** -24
    assert bool((k * 2.0 ** -12 == (k * 2.0 ** -12).round()).all()) and float(q[:rows // 2].abs().max()) == 2.0 ** 15
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel, scale=0.125)
    torch.cuda.synchronize()
    want, bound = reference(q, k, v, [(0, rows, 0, 700)], 0.125, False, out)
    # exact scores: only the weights' and the output's rounding (and, for FP32 sums and the exponential, 2^-18 of both)
    p_v = reference(q, k, v.abs(), [(0, rows, 0, 700)], 0.125, False, out)[0]
    u, half = torch.finfo(dtype).eps / 2, rows // 2
    tight = (u + 2.0 ** -18) * (p_v + want.abs())
    bound[:half] = tight[:half]
    check(out, want, bound)


@pytest.mark.parametrize("kernel", EACH)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_references_of_one_row_agree(kernel, dtype):
    """Weights of one row are taken from several references: of the slots and CTAs that share its keys, and before and
    after one has moved.  Scores are whole numbers (times a power of two) of 2^13 to 2^16 powers of two, that grow by
    less than one from tile to tile while every 32nd row's growth moves its warp's references; the values' signs alternate
    with the tiles, so that what is left shows a factor between them.  The bound has only roundings: of the weights and the
    output, and 2^-18 for sums and the exponential."""
    import rotated_w4a8_int8_gb300 as cr
    rows, n, D = 130, 1024, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    r, j = torch.arange(rows, device=DEV), torch.arange(n, device=DEV)
    q, k = torch.zeros(rows, 1, D, device=DEV), torch.zeros(n, 1, D, device=DEV)
    base = (45000 + 2000 * r + 77 * r * r) % 300000 + 46000                   # 0.18 powers of two each
    q[:, 0, 0], q[:, 0, 1], q[:, 0, 2] = base // 4096, base % 4096 // 16, base % 16
    q[:, 0, 3], q[:, 0, 4] = torch.where(r % 32 == 0, 64.0, 0.0), 1.0
    k[:, 0, 0], k[:, 0, 1], k[:, 0, 2], k[:, 0, 3], k[:, 0, 4] = 4096.0, 16.0, 1.0, (j // 128).float(), (j // 128 + j % 3).float()
    v = torch.randn(n, 1, D, generator=g, device=DEV).abs() * torch.where(j // 128 % 2 == 0, 1.0, -1.0)[:, None, None]
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel, scale=0.125)
    torch.cuda.synchronize()
    want = reference(q, k, v, [(0, rows, 0, n)], 0.125, False, out)[0]
    p_v = reference(q, k, v.abs(), [(0, rows, 0, n)], 0.125, False, out)[0]
    check(out, want, (torch.finfo(dtype).eps / 2 + 2.0 ** -18) * (p_v + want.abs()))


@pytest.mark.parametrize("kernel", [(1, 2), (2, 1), (3, 2)])
def test_wait_that_runs_out_is_reported(kernel):
    import rotated_w4a8_int8_gb300 as cr
    assert cr.device_error() == 0
    q, k, v = rand(9, 2, 64), rand(300, 2, 64, seed=1), rand(300, 2, 64, seed=2)
    out = torch.empty_like(q)
    t0 = time.time()
    cr.attention_selftest(q, k, v, out, *kernel, starve=True)
    code = cr.device_error()              # synchronises
    assert code not in (0, 16, 17) and 1.0 < time.time() - t0 < 30.0
    assert cr.device_error() == 0         # reading clears the word
    cr.attention_selftest(q, k, v, out, *kernel)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    check(out, *reference(q, k, v, [(0, 9, 0, 300)], 0.125, False, out))


def test_heads_outermost():
    """[heads, rows, D] tensors, seen as [rows, heads, D]."""
    import rotated_w4a8_int8_gb300 as cr
    q, k, v = (rand(4, n, 72, seed=n).transpose(0, 1) for n in (150, 333, 333))
    out = torch.empty(4, 150, 72, dtype=BF, device=DEV).transpose(0, 1)
    for rows in (150, 2):
        cr.attention(q[:rows], k, v, out[:rows])
        torch.cuda.synchronize()
        check(out[:rows], *reference(q[:rows], k, v, [(0, rows, 0, 333)], 72 ** -0.5, False, out[:rows]))


def test_errors_leave_outputs():
    import rotated_w4a8_int8_gb300 as cr
    q, k = rand(4, 2, 64), rand(8, 2, 64)
    out = torch.full_like(q, 5.0)
    for bad in (rand(4, 2, 65)[:, :, 1:], rand(4, 2, 68)[:, :, :64]):          # rows off 16 bytes
        with pytest.raises(cr.ConvRotError, match="misaligned"):
            cr.attention(bad, k, k, out)
    with pytest.raises(cr.ConvRotError, match="unsupported"):
        cr.attention(rand(4, 2, 144), rand(8, 2, 144), rand(8, 2, 144), rand(4, 2, 144))
    with pytest.raises(cr.ConvRotError, match="invalid"):
        cr.attention(q, rand(8, 2, 64)[:, :1].expand(8, 2, 64), k, out)        # heads on top of each other
    torch.cuda.synchronize()
    assert bool((out == 5).all())


def test_nothing_to_attend_to():
    """No pages, no table, no sequences: rows without keys become zeros, a sequence that has some is reported, rows in
    no sequence stay."""
    import rotated_w4a8_int8_gb300 as cr
    q = rand(6, 2, 64)
    none = torch.empty(0, 16, 2, 64, dtype=BF, device=DEV)
    for caches, table in (((none, none), torch.zeros(2, 3, dtype=torch.int32, device=DEV)),
                          ([rand(4, 16, 2, 64)] * 2, torch.zeros(2, 0, dtype=torch.int32, device=DEV))):
        out = torch.full_like(q, 5.0)
        cr.paged_attention(q, *caches, table, i32([(0, 2, 0, 0), (2, 3, 0, 7)]), out)
        assert cr.device_error() == 16
        assert bool((out[:2] == 0).all()) and bool((out[2:] == 5).all())
    k = rand(4, 2, 64)
    cr.cache_write(k, k, none, none, torch.zeros(1, 3, dtype=torch.int32, device=DEV), i32([(0, 4, 0, 4)]))
    assert cr.device_error() == 17
    out = torch.full_like(q, 5.0)
    cr.attention(q, k, k, out, seqs=torch.empty(0, 4, dtype=torch.int32, device=DEV))
    cr.attention(q[:0], k, k, out[:0])
    torch.cuda.synchronize()
    assert cr.device_error() == 0 and bool((out == 5).all())


def test_a_call_longer_than_a_wait_may_last():
    """2^18 rows by 2^18 keys, 128 heads: more than the two seconds after which a wait is given up.  No tile is ragged, so
    the warp that looks after those waits all the time."""
    import rotated_w4a8_int8_gb300 as cr
    n, H, D = 2 ** 18, 128, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.empty(n, H, D, dtype=BF, device=DEV).normal_(generator=g) for _ in range(3))
    out = torch.empty_like(q)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    cr.attention(q, k, v, out)
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) > 2100
    assert cr.device_error() == 0
    for row, head in ((0, 0), (n // 2 + 77, 63), (n - 1, H - 1)):
        at = slice(row, row + 1), slice(head, head + 1)
        check(out[at], *reference(q[at], k[:, at[1]], v[:, at[1]], [(0, 1, 0, n)], D ** -0.5, False, out[at]))


@pytest.mark.parametrize("D,causal,page", [(128, False, 0), (128, True, 64), (64, False, 0), (96, True, 0)])
@pytest.mark.parametrize("q_len", [2048, 2000, 1500, 300])
def test_items_left_to_a_second_launch(D, causal, page, q_len):
    """2048 rows of 20 heads are 160 items of 256 rows, eight more than the SMs: with many keys these are shared.  The
    sequence may have fewer rows than the host counted on."""
    import rotated_w4a8_int8_gb300 as cr
    m = 6001
    q, k, v = rand(2048, 20, D), rand(m, 4, D, seed=1), rand(m, 4, D, seed=2)
    seqs, out = [(5, q_len, 0, m)] if q_len < 2048 else [(0, q_len, 0, m)], torch.full_like(q, 3.0)
    want = reference(q, k, v, seqs, D ** -0.5, causal, out)
    if page:
        kc, vc, table, where = paged(k, v, seqs, page, 9)
        cr.paged_attention(q, kc, vc, table, where, out, causal=causal)
    else:
        cr.attention(q, k, v, out, seqs=i32(seqs), causal=causal)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    check(out, *want)
