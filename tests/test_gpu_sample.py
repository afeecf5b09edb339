"""The draw of the next token on the GPU against the definition in 64 bits: filters alone and
together, ties, masks, odd sizes, borders between tokens, rows that have no answer, streams, graphs."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
INF, NAN = math.inf, math.nan
BELOW_ONE = float(np.nextafter(np.float32(1), np.float32(0)))


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


def reference(logits, u, t, k, p, m):
    """{token: logs of its probability} of a row in 64 bits: one of each, or two where the draw or the
    nucleus lies within 2^-34 of the total of a border, as the call allows."""
    l = logits.double().cpu().numpy().copy()
    if np.isnan(l).any() or l.max() == -INF or not (t >= 0) or t == INF:
        return {-1: [NAN]}
    if t < 2.0**-100:
        return {int(np.argmax(l)): [0.0]}
    if l.max() == INF:
        l = np.where(l == INF, 0.0, -INF)
    top = l.max()
    w = np.exp((l - top) / t)
    order = np.argsort(-l, kind="stable")
    nk = k if 0 < k < len(l) else len(l)
    cum = np.cumsum(w[order][:nk])
    found = {}
    for near in (1 - 2.0**-34, 1.0, 1 + 2.0**-34):
        n = nk
        if p < 1:
            n = min(n, int((cum < p * cum[-1] * near).sum()) + 1)
        if m > 0:
            n = min(n, int((w >= m).sum()))
        kept = np.zeros(len(l), bool)
        kept[order[:max(n, 1)]] = True
        c = np.cumsum(np.where(kept, w, 0.0))
        for close in (-2.0**-34, 0.0, 2.0**-34):
            goal = (min(max(u, 0.0), 1.0) if u == u else 0.0) * c[-1] + close * c[-1]
            at = min(int((c <= max(goal, 0.0)).sum()), int(np.nonzero(kept & (w > 0))[0][-1]))
            found.setdefault(at, set()).add(math.log(w[at] / c[-1]) if w[at] > 0 else -INF)
    return found


def draw(tq, logits, u, t=None, k=None, p=None, m=None, logp=True, stream=None):
    n = logits.shape[0]

    def arg(v, dtype):
        return None if v is None else torch.tensor(v, dtype=dtype, device="cuda")
    tokens = torch.full((n,), -77, dtype=I32, device="cuda")
    out = torch.full((n,), 7.0, device="cuda") if logp else None
    u = u if isinstance(u, torch.Tensor) else arg(u, F32)
    tq.tq_sample(logits, u, tokens, arg(t, F32), arg(k, I32), arg(p, F32), arg(m, F32), out, stream)
    return tokens, out


def check(tq, logits, u, t=None, k=None, p=None, m=None):
    n = logits.shape[0]
    tokens, logp = draw(tq, logits, u, t, k, p, m)
    f = lambda v, d: [d] * n if v is None else [np.float32(x) for x in v]   # noqa: E731
    kk = [0] * n if k is None else k
    bare = 0
    for i, (a, ti, ki, pi, mi) in enumerate(zip(tokens.tolist(), f(t, 1.0), kk, f(p, 1.0), f(m, 0.0))):
        want = reference(logits[i], float(np.float32(u[i])), float(ti), int(ki), float(pi), float(mi))
        assert a in want, (i, a, want, u[i], ti, ki, pi, mi)
        bare += len(want) > 1
        got = logp[i].item()
        if a == -1:
            assert math.isnan(got)
        else:
            # the logarithm rounded to 32 bits, of sums good to 2^-35: half a step, and 2^-30 of leeway
            assert any(abs(got - v) <= abs(v) * 2.0**-24 + 2.0**-30 for v in want[a]), (i, a, got, want)
    return bare


def rand_u(n, seed):
    return np.random.RandomState(seed).uniform(size=n).astype(np.float32).tolist()


VOCABS = [1, 2, 3, 31, 32, 33, 127, 1000, 1025, 4096, 5003, 16384, 50021]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("vocab", VOCABS)
def test_all_filters(tq, vocab, dtype):
    """Rows of all settings, in logits that 16 bits round to many equal ones."""
    n = 24
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(n, vocab, generator=g) * 2.5).to(dtype).cuda()
    r = np.random.RandomState(vocab)
    t = r.choice([0.0, 0.3, 0.7, 1.0, 1.5, 8.0], n).tolist()
    k = r.choice([0, 0, 1, 2, 5, 40, 1000, vocab, vocab + 1, -3], n).tolist()
    p = r.choice([1.0, 1.0, 0.0, 1e-6, 0.3, 0.9, 0.999, 2.0, NAN], n).tolist()
    m = r.choice([0.0, 0.0, 1e-4, 0.05, 0.5, 1.0, 3.0, -1.0, NAN], n).tolist()
    check(tq, x, rand_u(n, vocab + 1), t, k, p, m)


@pytest.mark.parametrize("vocab", [7, 1000, 40000, 262144])
@pytest.mark.parametrize("one", ["plain", "k", "p", "m", "all"])
def test_each_filter(tq, vocab, one):
    n = 5
    g = torch.Generator().manual_seed(vocab + 7)
    x = (torch.randn(n, vocab, generator=g) * 3).cuda()
    kw = dict(plain={}, k=dict(k=[1, 2, 50, 300, vocab - 1]), p=dict(p=[0.05, 0.5, 0.9, 0.99, 0.9999]),
              m=dict(m=[0.5, 0.1, 0.01, 1e-3, 1e-6]),
              all=dict(t=[0.5, 0.8, 1.0, 1.2, 2.0], k=[3, 20, 50, 5000, 0], p=[0.9, 0.5, 0.95, 0.8, 0.999],
                       m=[0.1, 0.01, 0.05, 1e-3, 1e-4]))[one]
    check(tq, x, rand_u(n, 3), **kw)


@pytest.mark.parametrize("vocab", [2, 65, 3000, 131072])
def test_equal_logits(tq, vocab):
    """One value, and two: order and cuts go by the index alone."""
    x = torch.full((6, vocab), -3.25, device="cuda")
    x[3:, ::2] = 1.5
    check(tq, x, [0.0, 0.5, BELOW_ONE] * 2, p=[0.5, 0.999, 1.0] * 2, k=[vocab // 2 + 1, 0, vocab - 1] * 2)
    check(tq, x, [0.25, 0.75, 0.999] * 2, p=[0.25, 0.5, 0.75] * 2)
    check(tq, x, [0.25, 0.75, 0.999] * 2, m=[1.0, 0.5, 0.001] * 2)
    check(tq, x, [0.9] * 6, t=[0.0] * 6)


@pytest.mark.parametrize("vocab", [1, 40, 3000, 70000])
def test_min_p_above_one(tq, vocab):
    """No weight is that large: one token is kept, the first of the order, also of equal largest ones."""
    g = torch.Generator().manual_seed(vocab)
    l = torch.randint(0, 5, (6, vocab), generator=g).float().cuda()
    l[5] = INF
    m = [1.0000001, 1.5, INF, 2.0, 1.0, 3.0]
    check(tq, l, [0.0, 0.5, 0.99, 0.7, 0.9, 0.6], [1.0, 0.5, 2.0, 1.0, 1.0, 1.0], m=m)
    check(tq, l, [0.0, 0.5, 0.99, 0.7, 0.9, 0.6], [1.0, 0.5, 2.0, 1.0, 1.0, 1.0], [3, 0, 9, 2, 5, 1],
          [0.5, 0.9, 1.0, 0.3, 0.8, 0.5], m)


def test_masked(tq):
    """Minus infinity and the type's lowest value are never drawn beside others, whatever u is."""
    for dtype in (F32, F16, BF16):
        for low in (-INF, torch.finfo(dtype).min):
            x = torch.full((8, 999), low, dtype=dtype, device="cuda")
            x[:, 500] = 1.0
            x[4:, 501] = 1.0
            x[4:, 3] = -2.0
            us = [0.0, 0.3, 0.999, BELOW_ONE] * 2
            check(tq, x, us)
            check(tq, x, us, k=[5, 1, 0, 600] * 2, p=[1.0, 0.9, 0.5, 0.9999] * 2, m=[0.0, 0.1, 0.0, 1e-9] * 2)
            check(tq, x, us, t=[2.0, 0.5, 1e-3, 1e3] * 2)
    x = torch.full((2, 64), torch.finfo(F32).min, device="cuda")   # nothing else: all are alike
    check(tq, x, [0.0, 0.77])


def test_rows_without_an_answer(tq):
    x = torch.randn(9, 300, generator=torch.Generator().manual_seed(2)).cuda()
    x[0, 17] = NAN
    x[1] = -INF
    x[2, 299] = -NAN
    x[3, 4] = INF
    x[4, [5, 250]] = INF
    x[4, 6] = NAN
    x[5, [5, 250]] = INF
    u = [0.5] * 9
    check(tq, x, u, t=[1, 1, 1, 1, 1, 1, -1.0, INF, NAN])
    check(tq, x, [0.9] * 9, k=[7] * 9, p=[0.9] * 9, m=[0.1] * 9)
    tokens, logp = draw(tq, x, u, t=[1, 1, 1, 1, 1, 1, -1.0, INF, NAN])
    assert tokens.tolist()[:3] == [-1] * 3 and tokens.tolist()[6:] == [-1] * 3
    assert tokens.tolist()[3] == 4 and tokens.tolist()[4] == -1 and tokens.tolist()[5] in (5, 250)
    one = torch.full((2, 1), -INF, device="cuda")
    one[1] = NAN
    assert draw(tq, one, [0.1, 0.1])[0].tolist() == [-1, -1]


def test_uniform_numbers_out_of_range(tq):
    x = torch.randn(7, 50, generator=torch.Generator().manual_seed(3)).cuda()
    x[:, 0] = x[:, 49] = -INF
    tokens, _ = draw(tq, x, [-0.5, NAN, -INF, 0.0, 1.0, 7.5, INF])
    assert tokens.tolist() == [1, 1, 1, 1, 48, 48, 48]


@pytest.mark.parametrize("temperature", [1e-30, 1e-8, 1e-3, 0.05, 30.0, 1e6, 1e30])
def test_temperatures(tq, temperature):
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(6, 2000, generator=g) * 4).cuda()
    x[1:3] += 1000.0      # large logits of small differences
    x[3] *= 1e-6
    x[4] *= 1e30
    check(tq, x, rand_u(6, 5), t=[temperature] * 6)
    check(tq, x, rand_u(6, 6), t=[temperature] * 6, p=[0.9] * 6, k=[100] * 6)


def test_below_the_least_temperature_is_greedy(tq):
    x = torch.randn(3, 100, generator=torch.Generator().manual_seed(5)).cuda()
    x[:, 70] = x[:, 30] = 9.0
    tokens, logp = draw(tq, x, [0.9] * 3, t=[0.0, 1e-31, 1e-38])
    assert tokens.tolist() == [30] * 3 and logp.tolist() == [0.0] * 3


def test_borders(tq):
    """u on both sides of borders that are near 0, where 32 bits have room for them: a border is
    within 2^-35 of the total of where exact sums have it."""
    r = np.random.RandomState(8)
    for vocab, lead in ((300, 12.0), (5000, 14.0), (100000, 17.0)):
        l = r.normal(size=vocab).astype(np.float32) * 2
        l[:3] = l.max() - lead          # light tokens in front
        l[3] = l.max()
        x = torch.from_numpy(np.tile(l, (6, 1))).cuda()
        w = np.exp(l.astype(np.float64) - l.max())
        c = np.cumsum(w) / w.sum()
        us = []
        for j in range(3):
            us += [c[j] - 2.0**-34, c[j] + 2.0**-34]
        assert all(0 < a < 1e-4 for a in us)
        tokens, _ = draw(tq, x, us)
        assert tokens.tolist() == [0, 1, 1, 2, 2, 3]


def test_distribution(tq):
    """Evenly spread u draw each token as often as its probability says, to one draw."""
    n, vocab = 4096, 37
    l = torch.randn(vocab, generator=torch.Generator().manual_seed(9)) * 1.5
    u = ((torch.arange(n) + 0.5) / n).cuda()
    tokens, logp = draw(tq, l.cuda().expand(n, vocab).contiguous(), u, t=[0.8] * n)
    prob = torch.softmax(l.double() / 0.8, 0)
    counts = torch.bincount(tokens.cpu(), minlength=vocab).double()
    assert (counts - prob * n).abs().max() <= 1.0 + 1e-6
    assert (logp.cpu().double() - prob.log()[tokens.cpu().long()]).abs().max() < 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("stride,offset", [(1003, 0), (1003, 1), (1024, 3), (1001, 7), (1008, 8)])
def test_strides_and_offsets(tq, dtype, stride, offset):
    n, vocab = 9, 1000
    flat = torch.full((n * stride + 16,), NAN, dtype=dtype, device="cuda")
    x = flat.as_strided((n, vocab), (stride, 1), offset)
    x.copy_((torch.randn(n, vocab, generator=torch.Generator().manual_seed(10)) * 3).to(dtype))
    check(tq, x, rand_u(n, 11), p=[0.9] * n, k=[0, 100, 0] * 3)
    want = draw(tq, x.contiguous(), rand_u(n, 11))
    got = draw(tq, x, rand_u(n, 11))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_without_logp_and_settings(tq):
    x = torch.randn(5, 700, generator=torch.Generator().manual_seed(12)).cuda()
    u = rand_u(5, 13)
    assert torch.equal(draw(tq, x, u, logp=False)[0], draw(tq, x, u, [1.0] * 5, [0] * 5, [1.0] * 5, [0.0] * 5)[0])


def test_many_rows(tq):
    """More rows than run at once, every one with the same answer as alone."""
    n, vocab = 3000, 600
    x = (torch.randn(n, vocab, generator=torch.Generator().manual_seed(14)) * 2).cuda()
    u = rand_u(n, 15)
    tokens, logp = draw(tq, x, u, p=[0.8] * n)
    for i in range(0, n, 171):
        a, b = draw(tq, x[i:i + 1], u[i:i + 1], p=[0.8])
        assert a.item() == tokens[i].item() and b.item() == logp[i].item()


def test_graph_and_streams(tq):
    n, vocab = 16, 20000
    g = torch.Generator().manual_seed(16)
    x = (torch.randn(n, vocab, generator=g) * 2).cuda()
    u, t = torch.rand(n, generator=g).cuda(), torch.ones(n, device="cuda")
    k, p = torch.zeros(n, dtype=I32, device="cuda"), torch.ones(n, device="cuda")
    tokens, logp = torch.empty(n, dtype=I32, device="cuda"), torch.empty(n, device="cuda")
    tq.tq_sample(x, u, tokens, t, k, p, None, logp)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        tq.tq_sample(x, u, tokens, t, k, p, None, logp)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(torch.randn(n, vocab, generator=g) * (1 + i))
        u.copy_(torch.rand(n, generator=g))
        t.copy_(torch.rand(n, generator=g) + 0.2)
        k.copy_(torch.randint(0, 60, (n,), generator=g, dtype=I32))
        p.copy_(torch.rand(n, generator=g))
        graph.replay()
        a, b = tokens.clone(), logp.clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            c, e = draw(tq, x, u, t.tolist(), k.tolist(), p.tolist())
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(b, e)
        for j in range(n):
            want = reference(x[j], u[j].item(), t[j].item(), k[j].item(), p[j].item(), 0.0)
            assert a[j].item() in want


def test_rows_past_32_bits(tq):
    """Rows that start past 2^31 and 2^32 values from the first."""
    vocab, stride = 1000, (1 << 31) + 24
    flat = torch.empty(2 * stride + vocab, dtype=F16, device="cuda")
    x = flat.as_strided((3, vocab), (stride, 1))
    x.copy_((torch.randn(3, vocab, generator=torch.Generator().manual_seed(17)) * 2).to(F16))
    check(tq, x, [0.1, 0.5, 0.9], p=[0.9] * 3)


def test_shapes_refused(tq):
    x, u = torch.zeros(3, 10, device="cuda"), torch.zeros(3, device="cuda")
    tokens = torch.zeros(3, dtype=I32, device="cuda")
    for args, code in (((x, u[:2], tokens), tq.TQ_ERR_SHAPE), ((x, u, tokens[:2]), tq.TQ_ERR_SHAPE),
                       ((x, u, u), tq.TQ_ERR_TYPE), ((x[0], u, tokens), tq.TQ_ERR_SHAPE),
                       ((x, u.double(), tokens), tq.TQ_ERR_TYPE)):
        with pytest.raises(tq.TQError) as e:
            tq.tq_sample(*args)
        assert e.value.code == code
    with pytest.raises(ValueError):
        tq.tq_sample(torch.zeros(3, 20, device="cuda")[:, ::2], u, tokens)


def span(l, u, t, k, p, m, delta):
    """The lowest and the highest token of a row's draw in 64 bits, if the borders of the nucleus and of the
    draw lie up to delta of the total beside the exact ones."""
    l = l.double().cpu().numpy()
    w = np.exp((l - l.max()) / t)
    order = np.argsort(-l, kind="stable")
    nk = k if 0 < k < len(l) else len(l)
    cum = np.cumsum(w[order][:nk])
    found = []
    for near in (-delta, 0.0, delta):
        n = min(nk, int((cum < (p + near) * cum[-1]).sum()) + 1) if p < 1 else nk
        if m > 0:
            n = min(n, int((w >= m).sum()))
        kept = np.zeros(len(l), bool)
        kept[order[:max(n, 1)]] = True
        c = np.cumsum(np.where(kept, w, 0.0))
        for close in (-delta, 0.0, delta):
            at = int((c <= max(u + close, 0.0) * c[-1]).sum())
            found.append(min(at, int(np.nonzero(kept)[0][-1])))
    return min(found) - 1, max(found) + 1


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("vocab", [262144, 70001])
def test_light_tokens_weigh_together(tq, rows, vocab):
    """A leader and many tokens whose weights are a few units of 2^-45 of its own, or less: what one of them
    is off by counts that many times. The header's 2^-32 of the total is up to 50,000 of them here."""
    x = torch.empty(rows, vocab)
    f = lambda v: float(np.float32(v))   # noqa: E731
    wrong = []
    for drop, lead, base, u, k, p, m in [
            # below the leader; where that is; what both are above; then, as parts of all light tokens' share:
            # u from 0 on (or from 1 down), top-k, top-p from 1 down; min-p
            (30.49, -1, 0.0, 0.7, 0.0, 0.0, 1e-14), (32.0, -1, 0.0, 0.6, 0.0, 0.0, 1e-16),
            (30.49, vocab // 2, 0.0, 0.3, 0.0, 0.0, 1e-14), (22.0, 0, 0.0, -0.2, 0.0, 0.6, 0.0),
            (21.5, 0, -1.0, -0.3, 0.0, 0.3, 0.0), (28.0, -1, 0.0, 0.4, 0.99, 0.0, 0.0),
            (26.0, -1, 2.0, 0.2, 0.75, 0.5, 1e-13), (20.0, 5, 0.0, -0.1, 0.0, 0.25, 0.0),
            (30.5, -1, 9000.0, 0.7, 0.0, 0.0, 1e-14), (30.49, -1, 0.0, 0.7, 0.0, 0.0, 0.0)]:
        x.fill_(base - drop)
        x[:, lead] = base
        share = (vocab - 1) * math.exp(-drop)
        u, k, p = f(u * share if u > 0 else 1 + u * share), int(k * vocab), f(1 - p * share)
        kw = dict(k=[k] * rows, p=[p] * rows, m=[m] * rows) if (k, p, m) != (0, 1.0, 0.0) else {}
        tokens, _ = draw(tq, x.cuda(), [u] * rows, **kw)
        lo, hi = span(x[0], u, 1.0, k, p, f(m), 2.0**-32)
        assert 0 < lo and hi < vocab - 1 and hi - lo < 0.6 * vocab      # (the case says something)
        wrong += [(drop, lead, u, k, p, m, a, lo, hi) for a in tokens.tolist() if not lo <= a <= hi]
    assert not wrong, wrong


@pytest.mark.parametrize("vocab", [2, 6, 256, 512, 1000, 4096, 262144])
@pytest.mark.parametrize("value", [0.0, -3.25, 7.7, 5000.0])
def test_shares_of_equal_logits_are_exact(tq, vocab, value):
    """A half and a quarter of equal weights are met by just that many of them, whatever a weight is in units:
    u just below 1 draws the last of them."""
    x = torch.full((4, vocab), value)
    x[2:, vocab // 2:] = -INF
    tokens, _ = draw(tq, x.cuda(), [BELOW_ONE] * 4, p=[0.5, 0.25, 0.5, 0.25])
    halves = [vocab] * 2 + [vocab // 2] * 2
    assert tokens.tolist() == [max(1, math.ceil(n * p)) - 1 for n, p in zip(halves, [0.5, 0.25] * 2)]


def blocks_of(rows, vocab, size):
    """What the call takes for these sizes: thread blocks a row (twice as many as before while at most 608 are
    in the call and a block has more than 2048 tokens), and whether their slices stay in shared memory (up to
    64 KB)."""
    cluster = 1
    while cluster < 16 and 2 * rows * cluster <= 608 and vocab > cluster * 2048:
        cluster *= 2
    return cluster, ((vocab + cluster - 1) // cluster + 31) // 32 * 32 * size <= 65536


def check_rows(tq, x, u, t, k, p, m, rows):
    """Some rows of a draw of many against the definition; every row's draw is made."""
    tokens, logp = draw(tq, x, u, t, k, p, m)
    f = lambda v: float(np.float32(v))   # noqa: E731
    for i in rows:
        want = reference(x[i], f(u[i]), f(t[i]), int(k[i]), f(p[i]), f(m[i]))
        a, got = tokens[i].item(), logp[i].item()
        assert a in want, (i, a, want, u[i], t[i], k[i], p[i], m[i])
        assert math.isnan(got) if a == -1 else any(abs(got - v) <= abs(v) * 2.0**-24 + 2.0**-30 for v in want[a]), i


@pytest.mark.parametrize("n,vocab,dtype,blocks,pad,offset", [
    (320, 32771, F32, 1, 5, 0), (320, 40001, F16, 1, 0, 3), (320, 40001, BF16, 1, 6, 1), (305, 16400, F32, 1, 0, 1),
    (200, 128001, F16, 2, 7, 0), (150, 131073, F32, 4, 2, 2), (76, 140001, F32, 8, 0, 0), (310, 262144, BF16, 1, 0, 0)],
    ids=str)
def test_slices_that_stay_in_memory(tq, n, vocab, dtype, blocks, pad, offset):
    """Rows whose slices are too large for shared memory: filters of their own, at any address."""
    assert blocks_of(n, vocab, dtype.itemsize) == (blocks, False)
    stride = vocab + pad
    flat = torch.full((n * stride + 16,), NAN, dtype=dtype, device="cuda")
    x = flat.as_strided((n, vocab), (stride, 1), offset)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x.copy_(torch.randn(n, vocab, generator=g, device="cuda") * 2.5)
    x[1::7].masked_fill_(torch.rand(x[1::7].shape, generator=g, device="cuda") < 0.9, -INF)
    x[2, vocab // 2], x[3, 7], x[4] = INF, NAN, -INF
    r = np.random.RandomState(n)
    t = r.choice([0.0, 0.3, 0.7, 1.0, 1.5, 8.0], n).tolist()
    k = r.choice([0, 0, 1, 5, 40, 700, 1000, vocab // 2, vocab], n).tolist()
    p = r.choice([1.0, 1.0, 1e-6, 0.3, 0.9, 0.999], n).tolist()
    m = r.choice([0.0, 0.0, 1e-4, 0.05, 0.5, 3.0], n).tolist()
    check_rows(tq, x, rand_u(n, vocab + 1), t, k, p, m, list(range(14)) + list(range(20, n, max(1, n // 24))))
    assert torch.isnan(flat[offset + n * stride:]).all()


@pytest.mark.parametrize("n,vocab,dtype,blocks", [(320, 32800, F32, 1), (320, 262144, F32, 1), (200, 128001, F16, 2)],
                         ids=str)
def test_equal_logits_that_stay_in_memory(tq, n, vocab, dtype, blocks):
    """One value, two and four in such rows: cuts among equal logits, the sums of all of them."""
    assert blocks_of(n, vocab, dtype.itemsize) == (blocks, False)
    x = torch.full((n, vocab), -3.25, dtype=dtype, device="cuda")
    x[3::6, ::2] = 1.5
    x[4::6] = (torch.arange(vocab, device="cuda") % 4).to(dtype)
    x[5::6, 1:] = -12.5
    t = [1.0, 0.7, 2.0, 1.0, 0.5, 1.0] * n
    k = [vocab // 2 + 1, 0, vocab - 1, 0, vocab // 3, 0] * n
    p = [0.5, 0.999, 1.0, 0.25, 0.75, 0.99] * n
    m = [0.0, 0.5, 0.0, 0.001, 0.0, 1e-9] * n
    check_rows(tq, x, rand_u(n, 21), t[:n], k[:n], p[:n], m[:n], range(12))
    check_rows(tq, x, [BELOW_ONE, 0.0] * (n // 2), t[1:n + 1], [0] * n, p[:n], m[2:n + 2], range(n - 12, n))
    check_rows(tq, x, [0.5] * n, [0.0] * n, [0] * n, [1.0] * n, [0.0] * n, range(6))


def test_light_tokens_that_stay_in_memory(tq):
    """The sums of many light tokens in rows of one thread block each."""
    n, vocab, drop = 320, 262144, 30.49
    assert blocks_of(n, vocab, 4) == (1, False)
    x = torch.full((n, vocab), -drop, device="cuda")
    x[:, -1] = 0.0
    share = (vocab - 1) * math.exp(-drop)
    parts = [0.1, 0.35, 0.7, 0.9]
    us = [float(np.float32(v * share)) for v in parts] * (n // 4)
    for m in (1e-14, 0.0):
        tokens, _ = draw(tq, x, us, m=[m] * n)
        for j in range(4):
            lo, hi = span(x[0], us[j], 1.0, 0, 1.0, float(np.float32(m)), 2.0**-32)
            assert lo <= tokens[j::4].min() and tokens[j::4].max() <= hi, (m, us[j], tokens[j].item(), lo, hi)
