"""Paged attention on the GPU against the 64-bit form: single tokens to long chunks, ragged batches,
shared heads, windows, rows that see nothing, pages that end inside tiles, strides, splits."""
import math

import pytest
import torch

from attn_util import assert_within, attention

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


def problem(lens, hq, hk, dim, page, dtype, seed=0, order="hnd", peak=2.0, poison=True, window=0):
    """Inputs on the CPU and the GPU for sequences of (total, new) tokens. Every slot that no new
    token sees holds NaN, and table entries of pages no token sees are out of range."""
    g = torch.Generator().manual_seed(seed + 31 * len(lens) + dim)
    need = [-(-n // page) for n, _ in lens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1]) + 2), -1, dtype=torch.int32)
    k = torch.randn(pages, hk, page, dim, generator=g).to(dtype)
    v = torch.randn(pages, hk, page, dim, generator=g).to(dtype)
    seen = torch.zeros(pages, page, dtype=torch.bool)
    for b, (n, q) in enumerate(lens):
        lo = max(0, n - q - window + 1) if window else 0
        for i in range(need[b]):
            table[b, i] = perm.pop()
            at = i * page
            seen[table[b, i], max(0, lo - at):max(0, n - at)] = q > 0
            if at + page <= lo:
                table[b, i] = 10**8    # a page before the window: freed
    if poison:
        for c in (k, v):
            c.transpose(1, 2)[~seen] = float("nan")
    ntok = sum(q for _, q in lens)
    Q = (torch.randn(ntok, hq, dim, generator=g) * peak).to(dtype)
    q_start = torch.tensor([0] + [q for _, q in lens], dtype=torch.int32).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([n for n, _ in lens], dtype=torch.int32)
    kd, vd = k.cuda(), v.cuda()
    if order == "nhd":
        kd, vd = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kd, vd))
    elif order == "both":
        both = torch.stack([kd, vd], 1)
        kd, vd = both[:, 0], both[:, 1]
    return Q, k, v, table, q_start, kv_len, kd, vd


def call(tq, prob, out, window=0, scale=None, max_q=None, max_kv=None, lse=True):
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    ntok, hq, dim = Q.shape
    nseq = len(kv_len)
    mq = max_q if max_q is not None else int((q_start[1:] - q_start[:-1]).max())
    mk = max_kv if max_kv is not None else int(kv_len.max())
    O = torch.full((ntok, hq, dim), float("nan"), dtype=out, device="cuda")
    L = torch.full((ntok, hq), float("nan"), device="cuda") if lse else None
    need = tq.tq_paged_attention_workspace_bytes(nseq, ntok, hq, k.shape[1], dim, mq, mk, window)
    ws = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    tq.tq_paged_attention(Q.cuda(), tq.PagedKV(kd, vd, table.cuda()), q_start.cuda(), kv_len.cuda(),
                          O, mq, mk, scale if scale is not None else dim ** -0.5, ws, window, L)
    return O, L


def check(tq, prob, out, window=0, **kw):
    Q, k, v, table, q_start, kv_len, _, _ = prob
    scale = kw.get("scale", Q.shape[2] ** -0.5)
    o, lse, tol, tol_lse = attention(Q, k, v, table, q_start, kv_len, scale, window, out)
    O, L = call(tq, prob, out, window, **kw)
    assert_within(O, o, tol, "o")
    L = L.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(L[none], lse[none])
    assert (O.cpu()[none] == 0).all()
    assert_within(L[~none], lse[~none], tol_lse[~none], "lse")
    return O


CASES = [
    # (total, new) of each sequence, q heads, kv heads, dim, page, type, out, window, order
    ([(1, 1)], 1, 1, 128, 16, F16, F16, 0, "hnd"),
    ([(333, 1)], 40, 40, 128, 16, F16, F16, 0, "hnd"),
    ([(64, 1), (65, 1), (1, 1), (63, 1), (129, 1)], 10, 2, 128, 16, BF16, BF16, 0, "nhd"),
    ([(5000, 1)], 8, 1, 128, 64, BF16, F32, 0, "hnd"),
    ([(5000, 1), (17, 1), (2500, 1)], 6, 2, 64, 32, F16, F32, 0, "both"),
    ([(700, 5), (0, 0), (5, 5), (90, 1)], 8, 4, 64, 8, F16, F16, 0, "hnd"),
    ([(400, 5), (31, 5), (300, 3)], 15, 3, 80, 48, BF16, BF16, 100, "nhd"),
    ([(3000, 1), (20, 1)], 8, 2, 96, 24, F16, F16, 256, "hnd"),
    ([(3000, 7)], 4, 4, 128, 256, BF16, BF16, 1, "hnd"),
    ([(17, 17)], 2, 2, 8, 8, F16, F32, 0, "hnd"),
    ([(40, 40), (33, 2)], 3, 1, 40, 16, BF16, BF16, 7, "hnd"),
    ([(300, 300)], 5, 1, 128, 16, BF16, BF16, 0, "hnd"),
    ([(513, 200), (100, 100), (1, 1)], 4, 2, 128, 32, F16, F16, 0, "nhd"),
    ([(1500, 129), (140, 128)], 8, 8, 64, 64, BF16, BF16, 64, "both"),
    ([(900, 260), (2100, 1), (64, 64)], 12, 4, 96, 48, BF16, F32, 0, "hnd"),
    ([(700, 333)], 16, 2, 80, 40, F16, F16, 500, "hnd"),
    ([(4100, 40)], 8, 2, 128, 128, BF16, BF16, 0, "hnd"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(tq, case):
    lens, hq, hk, dim, page, dtype, out, window, order = case
    check(tq, problem(lens, hq, hk, dim, page, dtype, order=order, window=window), out, window)


@pytest.mark.parametrize("nseq,most", [(49, 60), (70, 40), (420, 25)])
def test_many_sequences_of_many_rows(tq, nseq, most):
    """More sequences than the lengths kept in shared memory, and more row tiles than threads; some
    sequences empty, some without new tokens, some of one token among chunks."""
    g = torch.Generator().manual_seed(nseq)
    lens = []
    for b in range(nseq):
        q = int(torch.randint(0, most, (1,), generator=g)) if b % 7 else b % 2
        lens.append((q + int(torch.randint(0, 200, (1,), generator=g)) if b % 11 else q, q))
    lens[3] = (150, most)
    check(tq, problem(lens, 8, 2, 64, 16, BF16), BF16)


@pytest.mark.parametrize("lens,hq,hk", [([(257, 256)], 1, 1), ([(3000, 128)], 1, 1), ([(3000, 129)], 1, 1),
                                        ([(2600, 1), (1300, 300)], 7, 1), ([(128, 128)] * 40, 8, 8),
                                        ([(6000, 70)], 2, 1), ([(130, 3)] * 3, 64, 1)])
def test_row_tile_edges(tq, lens, hq, hk):
    """Row tiles of exactly 128, 129 and 256 rows, groups that do not divide them, a row tile cut
    into many pieces, several row tiles a block."""
    for dim in (64, 128):
        check(tq, problem(lens, hq, hk, dim, 32, F16), F32)


@pytest.mark.parametrize("new", [1, 3, 300])
def test_tokens_that_see_nothing(tq, new):
    """A kv_len below the number of new tokens: the first ones stand before position 0."""
    prob = problem([(50, 50), (40, 40)], 4, 2, 64, 16, F16)
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    g = torch.Generator().manual_seed(1)
    Q = torch.randn(new + 2, 4, 64, generator=g).to(F16)
    q_start, kv_len = torch.tensor([0, new, new + 2]).int(), torch.tensor([new // 2, 40]).int()
    if new // 2 > 50:
        prob = problem([(150, 150), (40, 40)], 4, 2, 64, 16, F16)
        k, v, table, kd, vd = prob[1], prob[2], prob[3], prob[6], prob[7]
    check(tq, (Q, k, v, table, q_start, kv_len, kd, vd), F32)


def test_rows_past_the_last_sequence_are_not_written(tq):
    for n, max_q in ((200, 1), (40, 300)):    # one split or several, both kernels
        prob = list(problem([(n, 1), (n, 2)], 4, 2, 64, 16, F16))
        prob[0] = torch.cat([prob[0], prob[0]])
        O, L = call(tq, tuple(prob), F16, max_q=max(max_q, 2), max_kv=100 * n)
        assert torch.isnan(O[3:]).all() and torch.isnan(L[3:]).all()
        assert not torch.isnan(O[:3]).any()


@pytest.mark.parametrize("new", [1, 40, 300])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_scores(tq, new, dtype):
    """Scores of hundreds, growing and falling along the keys: the running maximum moves every tile,
    and weights far below it vanish without a NaN."""
    prob = problem([(1300, new)], 4, 1, 128, 16, dtype, poison=False)
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    up = torch.linspace(0.2, 4.0, 1300).to(dtype)
    for j in range(1300):
        k[table[0, j // 16], 0, j % 16] = up[j if new != 40 else 1299 - j] * (1 if j % 7 else -1)
    Q = (torch.ones_like(Q) * (torch.arange(4)[None, :, None] - 1.5)).to(dtype)
    check(tq, (Q, k, v, table, q_start, kv_len, k.cuda(), v.cuda()), F32)


@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scale(tq, scale):
    for new in (2, 200):
        check(tq, problem([(400, new)], 4, 2, 64, 16, F16, peak=1.0), F32, scale=scale)


def test_constant_values_come_back(tq):
    """With every value 1 the output is the sum of the weights over itself, whatever the scores."""
    for new in (1, 150):
        prob = problem([(1000, new)], 8, 2, 128, 16, BF16, poison=False)
        Q, k, v, table, q_start, kv_len, kd, vd = prob
        vd.fill_(1.0)
        O, _ = call(tq, prob, F32)
        assert (O - 1).abs().max().item() <= 2.0**-8 + 2.0**-12


@pytest.mark.parametrize("max_kv,new", [(100, 1), (64, 1), (3000, 1), (100000, 1), (1, 200), (10**6, 200)])
def test_bounds_that_are_not_tight(tq, max_kv, new):
    """max_kv only plans: too large or too small, the result is that of the exact one."""
    check(tq, problem([(1900, new), (300, min(new, 100))], 4, 2, 64, 16, F16), F32, max_kv=max_kv)


def test_split_count_changes_only_roundings(tq):
    prob = problem([(8000, 1)], 8, 1, 128, 16, BF16)
    a, la = call(tq, prob, F32)
    b, lb = call(tq, prob, F32, max_kv=64)     # planned as one split
    assert (a - b).abs().max().item() <= 2 * 2.0**-8 * 1.0
    assert (la - lb).abs().max().item() <= 1e-5


def test_same_inputs_same_bits(tq):
    for lens in ([(3000, 1)] * 3, [(700, 300), (200, 5)]):
        prob = problem(lens, 8, 2, 128, 16, BF16)
        a, la = call(tq, prob, BF16)
        for _ in range(3):
            b, lb = call(tq, prob, BF16)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_pages_and_lengths_are_reported(tq):
    for new in (1, 200):
        prob = list(problem([(300, new)], 4, 2, 64, 16, F16))
        for entry in (-1, prob[1].shape[0], 2**31 - 1):
            bad = prob[3].clone()
            bad[0, 5] = entry
            call(tq, tuple(prob[:3] + [bad] + prob[4:]), F16)
            assert tq.tq_device_status() == tq.TQ_ERR_INDEX, (new, entry)
        long = prob[:5] + [torch.tensor([100000]).int()] + prob[6:]
        call(tq, tuple(long), F16, max_kv=300)
        assert tq.tq_device_status() == tq.TQ_ERR_INDEX
        call(tq, tuple(prob), F16, max_q=1 if new > 1 else 0)
        assert tq.tq_device_status() == tq.TQ_ERR_INDEX
        call(tq, tuple(prob), F16)
        assert tq.tq_device_status() == tq.TQ_OK


@pytest.mark.parametrize("starts", [[0, 90, 40, 130], [30, 60, 100, 130], [-7, 60, 100, 1 << 30]])
def test_starts_out_of_order_stay_in_bounds(tq, starts):
    """q_start that is not what it should be: whatever comes out, the call ends, stays within its
    buffers (here between rows that are checked), and the next one is right."""
    for new in ([1, 1, 1], [50, 40, 40]):
        prob = list(problem([(200, n) for n in new], 8, 2, 64, 16, F16))
        want, _ = call(tq, tuple(prob), F16)
        good, ntok = prob[4], prob[0].shape[0]
        prob[4] = torch.tensor([min(s, 2 * ntok) if s > 0 else s for s in starts], dtype=torch.int32)
        call(tq, tuple(prob), F16, max_q=max(new))
        tq.tq_device_status()
        prob[4] = good
        again, _ = call(tq, tuple(prob), F16)
        assert torch.equal(want, again)


def test_strided_queries_and_output(tq):
    prob = problem([(300, 3), (64, 1)], 4, 2, 64, 16, F16)
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    want, _ = call(tq, prob, F16)
    wide = torch.zeros(4, 4 * 64 + 24, dtype=F16, device="cuda")
    Qs = torch.as_strided(wide, (4, 4, 64), (4 * 64 + 24, 64, 1), 8)
    Qs.copy_(Q)
    out = torch.zeros(4, 4 * 64 + 3, device="cuda", dtype=F16)
    O = torch.as_strided(out, (4, 4, 64), (4 * 64 + 3, 64, 1), 1)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    tq.tq_paged_attention(Qs, tq.PagedKV(kd, vd, table.cuda()), q_start.cuda(), kv_len.cuda(), O, 3,
                          300, 64 ** -0.5, ws)
    assert torch.equal(O, want)
    assert (out[:, :1] == 0).all() and (out[:, 257:] == 0).all()


def test_long_cache_offsets_pass_32_bits(tq):
    """Pages whose byte and element offsets pass 2^32, in a cache of which only those are used."""
    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 9       # 2^32 elements and a little more
    k = torch.empty(pages, heads, page, dim, dtype=F16, device="cuda")
    v = torch.empty_like(k)
    for new in (1, 150):
        n = 5 * page - 3
        table = torch.tensor([[pages - 1, pages - 3, 0, pages - 2, pages // 2 + 1]], dtype=torch.int32)
        g = torch.Generator().manual_seed(9)
        kc, vc = torch.zeros(5, heads, page, dim, dtype=F16), torch.zeros(5, heads, page, dim, dtype=F16)
        small = torch.arange(5, dtype=torch.int32)[None]
        for i in range(5):
            kc[i] = torch.randn(heads, page, dim, generator=g)
            vc[i] = torch.randn(heads, page, dim, generator=g)
            k[table[0, i]], v[table[0, i]] = kc[i].cuda(), vc[i].cuda()
        Q = torch.randn(new, 16, dim, generator=g).to(F16)
        q_start, kv_len = torch.tensor([0, new]).int(), torch.tensor([n]).int()
        o, _, tol, _ = attention(Q, kc, vc, small, q_start, kv_len, dim ** -0.5, 0, F16)
        O, _ = call(tq, (Q, k, v, table, q_start, kv_len, k, v), F16)
        assert_within(O, o, tol, "o")
        # and the append to them
        X = torch.randn(1, 2 * heads, dim, device="cuda")
        tq.tq_kv_append(None, X[:, :heads], X[:, heads:], None, tq.PagedKV(k, v, table.cuda()),
                        torch.zeros(1, dtype=torch.int32, device="cuda"),
                        torch.full((1,), 5 * page - 3, dtype=torch.int32, device="cuda"))
        assert torch.equal(v[pages // 2 + 1, :, page - 3], X[0, heads:].half())


def test_append_then_attend(tq):
    """The two calls in a row, in a graph, as a decode step runs them: the second sees what the
    first wrote."""
    from attn_util import frequencies, norm_rope
    g = torch.Generator().manual_seed(4)
    hq, hk, dim, page, lens = 8, 2, 128, 16, [200, 33, 1]
    Q, k, v, table, q_start, kv_len, kd, vd = problem([(n, 1) for n in lens], hq, hk, dim, page, BF16)
    X = torch.randn(3, hq + 2 * hk, dim, generator=g)
    w = torch.rand(dim, generator=g) + 0.5
    pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32)
    turns, _ = tq.tq_rope_turns(dim, 1e4)
    rope, kv = tq.Rope(turns.cuda()), tq.PagedKV(kd, vd, table.cuda())
    Xd, Yq = X.cuda(), torch.empty(3, hq, dim, dtype=BF16, device="cuda")
    O = torch.empty(3, hq, dim, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    dev = [t.cuda() for t in (torch.arange(3, dtype=torch.int32), pos, q_start, kv_len, w)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            tq.tq_kv_append(Xd[:, :hq], Xd[:, hq:hq + hk], Xd[:, hq + hk:], Yq, kv, dev[0], dev[1],
                            rope, dev[4], dev[4])
            tq.tq_paged_attention(Yq, kv, dev[2], dev[3], O, 1, 256, dim ** -0.5, ws)
    graph.replay()
    torch.cuda.synchronize()
    # the queries and keys as the call rounded them, within its own bound of the definition
    wantq, boundq = norm_rope(X[:, :hq], w, 1e-6, frequencies(dim), False, 1.0, pos, BF16)
    assert_within(Yq, wantq, boundq, "q")
    o, _, tol, _ = attention(Yq.cpu(), kd.cpu(), vd.cpu(), table, q_start, kv_len, dim ** -0.5, 0, F32)
    assert_within(O, o, tol, "o")


@pytest.mark.parametrize("lens,hq,hk", [([(300, 1)], 4, 4), ([(20000, 1)], 2, 1), ([(900, 200)], 4, 1),
                                        ([(900, 40), (500, 300)] * 5, 8, 8), ([(70, 40)] * 200, 8, 2)])
def test_timeout_reported_then_cleared(tq, lens, hq, hk):
    """A first block whose tiles never arrive gives up after a short limit, says so once, and the
    next call is right: one block of the few-row kernel, a cluster, many splits, the many-row one."""
    import time
    for dim in (64, 128):
        prob = problem(lens, hq, hk, dim, 16, F16)
        want, _ = call(tq, prob, F16)
        torch.cuda.synchronize()
        tq.tq_debug_stall_next_launch(200_000)
        try:
            t = time.perf_counter()
            call(tq, prob, F16)
            torch.cuda.synchronize()
            t = time.perf_counter() - t
        finally:
            tq.tq_debug_stall_next_launch(0)
        assert tq.tq_device_status() == tq.TQ_ERR_TIMEOUT
        assert t < 0.8 and tq.tq_device_status() == tq.TQ_OK
        again, _ = call(tq, prob, F16)
        assert torch.equal(want, again)


def test_no_work(tq):
    prob = problem([(0, 0), (20, 0)], 2, 2, 64, 16, F16)
    O, L = call(tq, prob, F16, max_q=1)
    assert O.numel() == 0
    assert math.isfinite(float(tq.tq_device_status()))


def many_rows(tq, prob, max_kv, window=0):
    """Whether the plan takes the kernel for many rows: its workspace has a fixed size, the partial
    results of two row tiles of 256 rows for each of 152 blocks and a few words a block."""
    Q, k, _, _, q_start, kv_len, _, _ = prob
    mq = int((q_start[1:] - q_start[:-1]).max())
    need = tq.tq_paged_attention_workspace_bytes(len(kv_len), Q.shape[0], Q.shape[1], k.shape[1], Q.shape[2],
                                                 mq, max_kv, window)
    part = 2 * 152 * 256 * (Q.shape[2] + 1) * 4
    return part <= need <= part + 152 * 64


BOTH = [([(300, 300)], 5, 1, 128, 16, BF16, BF16, "hnd"),
        ([(513, 200), (100, 100), (1, 1)], 4, 2, 128, 32, F16, F16, "nhd"),
        ([(900, 260), (2100, 1), (64, 64)], 12, 4, 96, 48, BF16, F32, "hnd"),
        ([(4100, 40)], 8, 2, 128, 128, BF16, BF16, "hnd"),
        ([(400, 300), (0, 0), (31, 5), (300, 3)], 15, 3, 80, 8, F16, F16, "both"),
        ([(257, 256)], 1, 1, 64, 32, F16, F32, "hnd"), ([(3000, 129)], 1, 1, 128, 32, F16, F32, "hnd"),
        ([(2600, 1), (1300, 300)], 7, 1, 64, 16, BF16, BF16, "nhd"),
        ([(128, 128)] * 40, 8, 8, 64, 64, F16, F16, "hnd"), ([(6000, 70)], 2, 1, 64, 24, F16, F32, "hnd"),
        ([(130, 3)] * 3, 64, 1, 128, 16, F16, F16, "hnd"), ([(130, 130), (70, 7)], 24, 3, 40, 40, F16, F16, "hnd"),
        ([(70, 40)] * 60, 8, 2, 8, 8, BF16, BF16, "hnd")]


@pytest.mark.parametrize("case", BOTH, ids=str)
def test_both_kernels(tq, case):
    """max_kv only plans: a small one takes the kernel for few rows, a large one that for many, and
    both are right. A large max_kv also makes splits that no key falls into."""
    lens, hq, hk, dim, page, dtype, out, order = case
    prob = problem(lens, hq, hk, dim, page, dtype, order=order)
    assert not many_rows(tq, prob, 1) and many_rows(tq, prob, 10**8)
    a = check(tq, prob, out, max_kv=1)
    b = check(tq, prob, out, max_kv=10**8)
    assert a.shape == b.shape


@pytest.mark.parametrize("lens,hq,hk,dim,page,window", [([(1500, 1000)] * 8, 8, 8, 64, 64, 700),
                                                        ([(2500, 1000), (40, 40)] * 3, 16, 2, 128, 16, 600),
                                                        ([(900, 700)] * 12, 12, 4, 80, 48, 65)])
def test_windows_of_many_rows(tq, lens, hq, hk, dim, page, window):
    prob = problem(lens, hq, hk, dim, page, BF16, window=window)
    assert many_rows(tq, prob, max(n for n, _ in lens), window)
    check(tq, prob, BF16, window)


@pytest.mark.parametrize("lens,hq,hk", [([(900, 200)], 4, 1), ([(70, 40)] * 200, 8, 2)])
@pytest.mark.parametrize("max_kv", [1, 10**8])
def test_timeout_in_both_kernels(tq, lens, hq, hk, max_kv):
    for dim in (64, 128):
        prob = problem(lens, hq, hk, dim, 16, F16)
        want, _ = call(tq, prob, F16, max_kv=max_kv)
        torch.cuda.synchronize()
        tq.tq_debug_stall_next_launch(200_000)
        try:
            call(tq, prob, F16, max_kv=max_kv)
            torch.cuda.synchronize()
        finally:
            tq.tq_debug_stall_next_launch(0)
        assert tq.tq_device_status() == tq.TQ_ERR_TIMEOUT
        again, _ = call(tq, prob, F16, max_kv=max_kv)
        assert torch.equal(want, again) and tq.tq_device_status() == tq.TQ_OK


@pytest.mark.parametrize("starts", [[0, 90, 40, 130], [30, 60, 100, 130], [-7, 60, 100, 1 << 30]])
@pytest.mark.parametrize("max_kv", [1, 10**8])
def test_starts_out_of_order_in_both_kernels(tq, starts, max_kv):
    prob = list(problem([(200, n) for n in (50, 40, 40)], 8, 2, 64, 16, F16))
    want, _ = call(tq, tuple(prob), F16, max_kv=max_kv)
    good, ntok = prob[4], prob[0].shape[0]
    prob[4] = torch.tensor([min(s, 2 * ntok) for s in starts], dtype=torch.int32)
    call(tq, tuple(prob), F16, max_q=50, max_kv=max_kv)
    tq.tq_device_status()
    prob[4] = good
    again, _ = call(tq, tuple(prob), F16, max_kv=max_kv)
    assert torch.equal(want, again)


@pytest.mark.parametrize("max_kv", [1, 10**8])
def test_bad_pages_in_both_kernels(tq, max_kv):
    prob = list(problem([(300, 200)], 4, 2, 64, 16, F16))
    for entry in (-1, prob[1].shape[0], 2**31 - 1):
        bad = prob[3].clone()
        bad[0, 5] = entry
        call(tq, tuple(prob[:3] + [bad] + prob[4:]), F16, max_kv=max_kv)
        assert tq.tq_device_status() == tq.TQ_ERR_INDEX, entry
    long = prob[:5] + [torch.tensor([100000]).int()] + prob[6:]
    call(tq, tuple(long), F16, max_kv=max_kv)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    call(tq, tuple(prob), F16, max_q=1, max_kv=max_kv)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    check(tq, tuple(prob), F16, max_kv=max_kv)


@pytest.mark.parametrize("max_kv", [1, 10**8])
def test_large_scores_and_negative_scales_in_both_kernels(tq, max_kv):
    prob = problem([(1300, 300)], 4, 1, 128, 16, BF16, poison=False)
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    up = torch.linspace(0.2, 4.0, 1300).to(BF16)
    for j in range(1300):
        k[table[0, j // 16], 0, j % 16] = up[j] * (1 if j % 7 else -1)
    Q = (torch.ones_like(Q) * (torch.arange(4)[None, :, None] - 1.5)).to(BF16)
    check(tq, (Q, k, v, table, q_start, kv_len, k.cuda(), v.cuda()), F32, max_kv=max_kv)
    for scale in (0.0, -0.7, 3.0):
        check(tq, problem([(400, 200)], 4, 2, 64, 16, F16, peak=1.0), F32, scale=scale, max_kv=max_kv)


@pytest.mark.parametrize("max_kv", [1, 10**8])
def test_tokens_that_see_nothing_in_both_kernels(tq, max_kv):
    prob = problem([(150, 150), (40, 40)], 4, 2, 64, 16, F16)
    g = torch.Generator().manual_seed(1)
    Q = torch.randn(302, 4, 64, generator=g).to(F16)
    q_start, kv_len = torch.tensor([0, 300, 302]).int(), torch.tensor([150, 40]).int()
    check(tq, (Q,) + prob[1:4] + (q_start, kv_len) + prob[6:], F32, max_kv=max_kv)
