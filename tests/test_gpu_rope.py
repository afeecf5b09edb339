"""Norm and rotation of heads, and the append to the paged cache, on the GPU against the 64-bit
form: types, layouts, parts of a head, odd sizes, strides, alignment, padding, bad indices."""
import itertools

import pytest
import torch

from attn_util import assert_within, frequencies, norm_rope

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


def rope_of(tq, rot, inter, amplitude=1.0, base=1e4):
    turns, _ = tq.tq_rope_turns(rot, base)
    return tq.Rope(turns.cuda(), inter, amplitude)


def rand(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype)


CASES = [
    # ntok, q heads, k heads, dim, rot, interleaved, norm, in, out
    (1, 40, 40, 128, 128, False, True, F32, BF16),
    (1, 1, 0, 2, 2, True, True, F32, F32),
    (7, 3, 1, 80, 40, True, True, F32, F16),
    (33, 5, 2, 64, 64, False, False, F16, F16),
    (9, 4, 4, 96, 32, False, True, BF16, BF16),
    (5, 2, 2, 256, 256, False, True, F32, F32),
    (5, 2, 2, 256, 64, True, True, F16, F32),
    (6, 3, 3, 66, 18, True, True, F32, BF16),      # 9 pairs: one value at a time
    (6, 3, 3, 66, 66, False, True, BF16, F32),
    (4, 2, 1, 100, 60, False, True, F16, BF16),    # 30 pairs: two at a time
    (4, 2, 1, 254, 254, True, False, F32, F16),
    (3, 2, 2, 128, 0, False, True, F32, BF16),     # norm only
    (700, 9, 4, 128, 128, False, True, F32, BF16), # four heads a group
    (1500, 2, 5, 64, 32, True, True, BF16, F16),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope(tq, case):
    ntok, hq, hk, dim, rot, inter, norm, tin, tout = case
    g = torch.Generator().manual_seed(hash(case[:6]) & 0xFFFF)
    X = (rand(g, ntok, hq + hk, dim) * 3).to(tin)
    pos = torch.randint(0, 200000, (ntok,), generator=g, dtype=torch.int32)
    pos[0] = 0 if ntok > 1 else 131071
    wq, wk = (rand(g, dim) * 0.3 + 1, rand(g, dim) * 0.3 + 1) if norm else (None, None)
    Xd = X.cuda()
    Yq = torch.full((ntok, hq, dim), float("nan"), dtype=tout, device="cuda")
    Yk = torch.full((ntok, hk, dim), float("nan"), dtype=tout, device="cuda")
    tq.tq_qk_norm_rope(Xd[:, :hq], Xd[:, hq:] if hk else None, Yq, Yk if hk else None, pos.cuda(),
                       rope_of(tq, rot, inter, 1.25), None if wq is None else wq.cuda(),
                       None if wk is None else wk.cuda(), 1e-5)
    for x, y, w in ((X[:, :hq], Yq, wq), (X[:, hq:], Yk, wk)):
        if y.numel():
            want, bound = norm_rope(x, w, 1e-5, frequencies(rot), inter, 1.25, pos, tout)
            assert_within(y, want, bound, "y")


@pytest.mark.parametrize("kind", range(5))
def test_long_positions_and_scaled_tables(tq, kind):
    """Positions of up to 2^31 - 1 and negative ones: the angle is exact modulo one turn."""
    turns, amp = tq.tq_rope_turns(64, 5e5, kind, 8.0, 4096.0, 1.0, 4.0)
    pos = torch.tensor([0, 1, 65535, 131072, 2**24 + 1, 2**31 - 1, -1, -70000], dtype=torch.int32)
    X = rand(torch.Generator().manual_seed(3), 8, 2, 64)
    Y = torch.empty(8, 2, 64, device="cuda")
    tq.tq_qk_norm_rope(X.cuda(), None, Y, None, pos.cuda(), tq.Rope(turns.cuda(), False, amp))
    # the table's own fractions of a turn, multiplied exactly
    ang = [[(int(p) * (int(t) % (1 << 64))) % (1 << 64) / 2.0**64 * 2 * torch.pi for t in turns]
           for p in pos]
    c, s = torch.tensor(ang).double().cos() * amp, torch.tensor(ang).double().sin() * amp
    a, b = X.double()[..., :32], X.double()[..., 32:]
    c, s = c[:, None], s[:, None]
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    bound = 40 * 2.0**-24 * amp * (a.abs() + b.abs()).repeat(1, 1, 2)
    assert_within(Y, want, bound, "y")


def test_strides_alignment_and_in_place(tq):
    """Rows of a wider buffer, starts that are not 16-byte aligned, and results over the inputs: the
    values are those of the aligned call, bit for bit."""
    g = torch.Generator().manual_seed(5)
    n, h, d = 11, 3, 128
    X, w, pos = rand(g, n, h, d).cuda(), (rand(g, d) + 1).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    rope = rope_of(tq, d, False)
    base = torch.empty(n, h, d, device="cuda")
    tq.tq_qk_norm_rope(X, None, base, None, pos, rope, w)
    for shift, pad in itertools.product((1, 2, 4), (1, 6, 8)):
        wide = torch.empty(n * (h * d + pad) + 8, device="cuda")
        Xs = torch.as_strided(wide, (n, h, d), (h * d + pad, d, 1), shift)
        Xs.copy_(X)
        out = torch.zeros(n * (h * d + pad) + 8, device="cuda")
        Y = torch.as_strided(out, (n, h, d), (h * d + pad, d, 1), shift)
        tq.tq_qk_norm_rope(Xs, None, Y, None, pos, rope, w)
        assert_within(Y, base.double().cpu(), 8 * 2.0**-24 * (1 + base.abs().double().cpu()), "strided")
        assert out.sum().item() == pytest.approx(Y.sum().item(), rel=1e-3, abs=1e-2)
        gap = torch.ones_like(out, dtype=torch.bool)
        torch.as_strided(gap, (n, h, d), (h * d + pad, d, 1), shift).fill_(False)
        assert (out[gap] == 0).all()
        tq.tq_qk_norm_rope(Xs, None, Xs, None, pos, rope, w)
        assert torch.equal(Xs, Y)


def test_values_that_pass_keep_their_bits(tq):
    """Values past rot_dim, with no norm and the same type, are copied: infinities, -0, subnormals
    (and a NaN as a NaN), and they do not reach the rotated ones."""
    X = torch.zeros(2, 1, 64, dtype=F16, device="cuda")
    X[0, 0, 32:36] = torch.tensor([float("inf"), float("nan"), -0.0, 6e-8], dtype=F16)
    Y = torch.empty_like(X)
    tq.tq_qk_norm_rope(X, None, Y, None, torch.tensor([5, 6], dtype=torch.int32).cuda(),
                       rope_of(tq, 32, True))
    assert torch.isnan(Y[0, 0, 33]) and (Y[..., :32] == 0).all()
    X[0, 0, 33] = Y[0, 0, 33] = 0
    assert torch.equal(X[..., 32:].view(torch.int16), Y[..., 32:].view(torch.int16))


def test_zero_rows(tq):
    """A head of zeros stays zero under the norm (eps keeps the root finite)."""
    X = torch.zeros(3, 2, 128, device="cuda")
    Y = torch.full((3, 2, 128), 7.0, device="cuda")
    tq.tq_qk_norm_rope(X, None, Y, None, None, None, torch.ones(128, device="cuda"))
    assert (Y == 0).all()


APPEND = [
    # lens (total, new) of the sequences, q heads, kv heads, dim, rot, inter, page, in, cache, order
    ([(1, 1)], 4, 4, 128, 128, False, 16, F32, BF16, "hnd"),
    ([(37, 1), (16, 1), (17, 1), (1, 1)], 10, 2, 128, 64, False, 16, F32, F16, "nhd"),
    ([(50, 50), (9, 3), (0, 0), (700, 1)], 3, 3, 80, 40, True, 48, F32, BF16, "hnd"),
    ([(300, 299), (33, 32)], 0, 5, 96, 96, False, 8, BF16, BF16, "nhd"),
    ([(1024, 1000)], 8, 8, 64, 64, True, 128, F16, F16, "both"),
    ([(90, 90)], 2, 1, 8, 8, False, 24, F32, F16, "hnd"),
]


def make_cache(order, pages, heads, page, dim, dtype):
    """k, v [pages][heads][page][dim] views of a cache in some order, filled with a marker."""
    mk = lambda *s: torch.full(s, -77.0, dtype=dtype, device="cuda")   # noqa: E731
    if order == "hnd":
        return mk(pages, heads, page, dim), mk(pages, heads, page, dim)
    if order == "nhd":
        return mk(pages, page, heads, dim).transpose(1, 2), mk(pages, page, heads, dim).transpose(1, 2)
    both = mk(pages, 2, heads, page, dim)     # keys and values of a page side by side
    return both[:, 0], both[:, 1]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(tq, case):
    lens, hq, hk, dim, rot, inter, page, tin, tc, order = case
    g = torch.Generator().manual_seed(len(lens) * dim + page)
    need = [-(-n // page) for n, _ in lens]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = perm.pop()
    seq = torch.tensor([b for b, (n, q) in enumerate(lens) for _ in range(q)], dtype=torch.int32)
    pos = torch.tensor([n - q + i for n, q in lens for i in range(q)], dtype=torch.int32)
    # two padding tokens among the others
    seq = torch.cat([seq[:1], torch.tensor([0, 10**6], dtype=torch.int32), seq[1:]])
    pos = torch.cat([pos[:1], torch.tensor([-1, -5], dtype=torch.int32), pos[1:]])
    ntok = len(pos)
    X = (rand(g, ntok, hq + 2 * hk, dim) * 2).to(tin)
    wq, wk = rand(g, dim) * 0.3 + 1, rand(g, dim) * 0.3 + 1
    k, v = make_cache(order, pages, hk, page, dim, tc)
    kv = tq.PagedKV(k, v, table.cuda())
    Yq = torch.full((ntok, hq, dim), -55.0, dtype=tc, device="cuda") if hq else None
    Xd = X.cuda()
    tq.tq_kv_append(Xd[:, :hq] if hq else None, Xd[:, hq:hq + hk], Xd[:, hq + hk:], Yq, kv,
                    seq.cuda(), pos.cuda(), rope_of(tq, rot, inter), wq.cuda(), wk.cuda(), 1e-6)
    real = pos >= 0
    if hq:
        want, bound = norm_rope(X[:, :hq], wq, 1e-6, frequencies(rot), inter, 1.0, pos, tc)
        assert_within(Yq[real.cuda()], want[real], bound[real], "q")
        assert (Yq[~real.cuda()] == -55).all()
    wantk, boundk = norm_rope(X[:, hq:hq + hk], wk, 1e-6, frequencies(rot), inter, 1.0, pos, tc)
    wantv = X[:, hq + hk:].to(tc).double()
    k, v = k.cpu(), v.cpu()
    written = torch.zeros(pages, page, dtype=torch.bool)
    for t in range(ntok):
        if pos[t] < 0:
            continue
        at, slot = int(table[seq[t], pos[t] // page]), int(pos[t]) % page
        assert_within(k[at, :, slot], wantk[t], boundk[t], f"k of token {t}")
        assert torch.equal(v[at, :, slot].double(), wantv[t])
        written[at, slot] = True
    for c in (k, v):
        assert (c.transpose(1, 2)[~written] == -77).all(), "slots that are not the call's changed"


def test_append_bad_indices_are_skipped_and_reported(tq):
    k, v = make_cache("hnd", 4, 1, 16, 64, BF16)
    table = torch.tensor([[0, 9], [-3, 1]], dtype=torch.int32, device="cuda")
    kv = tq.PagedKV(k, v, table)
    X = torch.randn(1, 3, 64, device="cuda")
    Y = torch.zeros(1, 1, 64, dtype=BF16, device="cuda")
    for seq, pos in ((0, 16), (1, 3), (2, 0), (-1, 0), (0, 32), (0, 2**31 - 1)):
        tq.tq_kv_append(X[:, :1], X[:, 1:2], X[:, 2:], Y, kv,
                        torch.tensor([seq], dtype=torch.int32, device="cuda"),
                        torch.tensor([pos], dtype=torch.int32, device="cuda"))
        assert tq.tq_device_status() == tq.TQ_ERR_INDEX, (seq, pos)
        assert (k == -77).all() and (v == -77).all()
    tq.tq_kv_append(X[:, :1], X[:, 1:2], X[:, 2:], Y, kv,
                    torch.tensor([1], dtype=torch.int32, device="cuda"),
                    torch.tensor([16], dtype=torch.int32, device="cuda"))
    assert tq.tq_device_status() == tq.TQ_OK
    assert torch.equal(v[1, 0, 0], X[0, 2].to(BF16))


def test_other_stream_and_graph(tq):
    """The call runs on the caller's stream, and in a captured graph, without a copy or a wait."""
    X = torch.randn(5, 4, 128, device="cuda")
    Y, Z = torch.zeros_like(X), torch.zeros_like(X)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    rope = rope_of(tq, 128, False)
    tq.tq_qk_norm_rope(X, None, Y, None, pos, rope)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tq.tq_qk_norm_rope(X, None, Z, None, pos, rope)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, Z)
