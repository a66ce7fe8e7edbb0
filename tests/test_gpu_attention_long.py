"""attention over very many keys: what the sums of a row lose on the way.  Scores are chosen so that everything but the sum
under test is exact or bounded by a few roundings.

The roundings that the bounds count, with u half a step of the type (finfo.eps / 2): the output's u; the weights' own 2^-20
(their exponents' one rounded product and the exponential); the row's sum, FP32: weights of a tile of 128 keys are added to
one another (in two halves of 64), tiles' sums to the row's, 2^-24 of the sum for every addition one after another; the
tensor core's accumulators, which are cut towards zero: at most 2^-26 of a sum that grows evenly for every key (four cuts
for 16 keys, each less than 2^-23 of what has been summed by then) until it is added to FP32 sums after 2^15 keys in FP16, 2^17
in BF16: u (kernel 1, which has two products for each key: 2 u); and those sums, 2^-24 for each addition.
"""
import math

import pytest
import torch

from attention_util import check, paged, reference
from gpu_util import DEV, ensure_built

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF, HF = torch.bfloat16, torch.float16
KERNELS = [(1, 1), (1, 4), (2, 1), (3, 1), (3, 4)]        # kernel, CTAs that share keys
N = 2 ** 22


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gap", [0.3, 0.55, 0.7])
def test_sum_of_equal_weights(kernel, dtype, gap):
    """The first of every 128 keys has the largest score, all others lie `gap` powers of two below it: weights that are no
    power of two.  Only key 0 has a value, so the output is that value times its weight (exact) over the row's sum."""
    import rotated_w4a8_int8_gb300 as cr
    q = torch.ones(20, 1, 64, dtype=dtype, device=DEV)
    k, v = (torch.zeros(N, 1, 64, dtype=dtype, device=DEV) for _ in range(2))
    k[::128, 0, 0] = 1.0
    v[0] = 2.0 ** 15
    scale = float(torch.tensor(gap * math.log(2), dtype=torch.float32))
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel, scale=scale)
    torch.cuda.synchronize()
    want = 2.0 ** 15 / (N // 128 + (N - N // 128) * math.exp(-scale))
    bound = torch.finfo(dtype).eps / 2 + 2.0 ** -20 + (64 + N // 128) * 2.0 ** -24
    assert float((out.double() / want - 1).abs().max()) <= bound


@pytest.fixture(scope="module")
def values():
    """Values in [1, 2) of 2^24 keys, and their mean in 64 bits."""
    made = {}

    def of(dtype):
        if dtype not in made:
            made.clear()
            n, g = 2 ** 24, torch.Generator(device=DEV).manual_seed(1)
            v, mean = torch.empty(n, 1, 64, dtype=dtype, device=DEV), torch.zeros(1, 64, dtype=torch.float64, device=DEV)
            for part in v.split(2 ** 20):
                part.copy_(torch.rand(part.shape, generator=g, device=DEV) * 0.875 + 1)
                mean += part.double().sum(0)
            made[dtype] = v, mean / n
        return made[dtype]
    yield of
    made.clear()


@pytest.mark.parametrize("dtype,kernel", [(t, k) for t in (BF, HF) for k in KERNELS])
def test_sum_of_values(values, dtype, kernel):
    """All scores zero: the weights and their sum are exact, the output is the values' mean."""
    import rotated_w4a8_int8_gb300 as cr
    v, want = values(dtype)
    q = torch.zeros(20, 1, 64, dtype=dtype, device=DEV)
    out = torch.empty_like(q)
    cr.attention_selftest(q, v, v, out, *kernel)
    torch.cuda.synchronize()
    u, held = torch.finfo(dtype).eps / 2, 2 ** 24 // (2 ** 14 if dtype == HF else 2 ** 17)
    assert float((out.double() / want - 1).abs().max()) <= (3 if kernel[0] == 1 else 2) * u + held * 2.0 ** -24


def within(q, k, v, seqs, causal, out, got, cuts=1):
    """check() with the accumulators' term: `cuts` u times the sum of p |v|."""
    want, bound = reference(q, k, v, seqs, q.shape[2] ** -0.5, causal, out)
    check(got, want, bound + cuts * torch.finfo(q.dtype).eps / 2 * reference(q, k, v.abs(), seqs, q.shape[2] ** -0.5, causal, out)[0])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal,grows", [(False, False), (True, True), (False, True)])
def test_references_that_move(kernel, dtype, causal, grows):
    """Keys enough for several rounds of sums (where two slots or the CTAs share them too), whose largest scores come
    last, far above the first ones, or not; heads of 72 columns, rows that see no key."""
    import rotated_w4a8_int8_gb300 as cr
    n, g = 150001, torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(m, h, 72, generator=g, device=DEV) for m, h in ((140, 2), (n, 1), (n, 1)))
    if grows:
        k *= torch.linspace(0.1, 5, n, device=DEV)[:, None, None]
    q, k, v = q.to(dtype), k.to(dtype), (v + 1).to(dtype)
    seqs = [(0, 10, 0, 3), (12, 128, 3, n - 3)]
    out = torch.full_like(q, 7.0)
    before = out.clone()
    kc, vc, table, where = paged(k, v, seqs, 256, 300)
    cr.attention_selftest(q, kc, vc, out, *kernel, pages=table, seqs=where, causal=causal)
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    within(q, k, v, seqs, causal, before, out, 2 if kernel[0] == 1 else 1)


def test_long_and_short_items_in_turn():
    """More items than CTAs, long ones and short ones after one another on the same CTA."""
    import rotated_w4a8_int8_gb300 as cr
    lens, g = [33000, 90, 40000], torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.randn(m, h, 64, generator=g, device=DEV).to(HF) for m, h in ((120, 160), (sum(lens), 1), (sum(lens), 1)))
    seqs = [(40 * i, 40, sum(lens[:i]), n) for i, n in enumerate(lens)]
    out = torch.zeros_like(q)
    cr.attention_selftest(q, k, v, out, 2, 1, seqs=torch.tensor(seqs, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert cr.device_error() == 0
    for h in range(0, 160, 40):
        part = slice(h, h + 40)
        within(q[:, part], k, v, seqs, False, torch.zeros_like(q[:, part]), out[:, part])


@pytest.mark.parametrize("rows,dtype,keys", [(4, HF, 300000), (4, BF, 2200000), (200, HF, 70000), (400, BF, 140000)])
def test_captured_and_at_once(rows, dtype, keys):
    """Long keys through the chosen kernels: on two streams at once and replayed from two graphs, the same bits as one
    call alone."""
    import rotated_w4a8_int8_gb300 as cr
    g = torch.Generator(device=DEV).manual_seed(rows)
    sets = [[torch.randn(n, h, 64, generator=g, device=DEV).to(dtype) for n, h in ((rows, 8), (keys, 2), (keys, 2))] for _ in range(2)]
    want, out = ([torch.zeros_like(q) for q, _, _ in sets] for _ in range(2))
    for o, s in zip(want, sets):
        cr.attention(*s, o)
        torch.cuda.synchronize()
    part = slice(0, 4)
    within(sets[0][0][part], *sets[0][1:], [(0, 4, 0, keys)], False, torch.zeros_like(want[0][part]), want[0][part], 2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for st, o, s in zip(streams, out, sets):
            cr.attention(*s, o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, o, s in zip(graphs, out, sets):
        o.zero_()
        with torch.cuda.graph(graph):
            cr.attention(*s, o)
            cr.attention(*s, o)
    for st, graph in zip(streams, graphs):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    assert cr.device_error() == 0 and all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("light", [28.5, 29.51, 31.2])
def test_many_light_keys(kernel, light):
    """2^22 keys, each of 2^-light of the weight of the first, whose value is zero, in FP16: steps of its subnormals are
    2^-24, the largest weight is at least 2^12, so a key's weight is off by at most 2^-37.  (The exponent: one product, FP32,
    of up to 32.)"""
    import rotated_w4a8_int8_gb300 as cr
    q = torch.ones(20, 1, 64, dtype=HF, device=DEV)
    k, v = torch.zeros(N, 1, 64, dtype=HF, device=DEV), torch.ones(N, 1, 64, dtype=HF, device=DEV)
    k[1:, 0, 0] = -1.0
    v[0] = 0.0
    scale = float(torch.tensor(light * math.log(2), dtype=torch.float32))
    out = torch.empty_like(q)
    cr.attention_selftest(q, k, v, out, *kernel, scale=scale)
    torch.cuda.synchronize()
    mass = (N - 1) * math.exp(-scale)
    want = mass / (1 + mass)
    assert float((out.double() - want).abs().max()) <= (N - 1) * 2.0 ** -37 + want * (3 * torch.finfo(HF).eps / 2 + 2.0 ** -18)
