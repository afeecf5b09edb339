"""Low-rank adapters beside a product, on the GPU against the 64-bit form: types, ranks, odd sizes,
strides, tokens in any order, padding that holds anything, bad indexes, streams and graphs."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
INF = float("inf")


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


def scratch(tq, ntok, adapters):
    n = tq.tq_lora_add_workspace_bytes(ntok, adapters)
    return torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda") if n else None


def make(ntok, cols, rows, adapters, top, xt=F32, wt=BF16, yt=F32, seed=0, bare=0.1, ragged=True, pad=0):
    """Inputs on the GPU; slots of A and B past an adapter's rank hold NaN."""
    g = torch.Generator().manual_seed(seed)
    rank = torch.randint(0 if ragged else top, top + 1, (adapters,), generator=g, dtype=I32)
    if adapters:
        rank[0] = top
    a = torch.randn(adapters, top, cols, generator=g).mul_(cols ** -0.5).to(wt)
    brs = top + pad
    b = torch.randn(adapters, rows, brs, generator=g).to(wt)
    for i, r in enumerate(rank.tolist()):
        a[i, r:] = float("nan")
        b[i, :, r:] = float("nan")
    ids = torch.randint(0, adapters, (ntok,), generator=g, dtype=I32) if adapters else torch.full((ntok,), -1, dtype=I32)
    ids[torch.rand(ntok, generator=g) < bare] = -1
    x = torch.randn(ntok, cols, generator=g).to(xt)
    z = torch.randn(ntok, rows, generator=g).to(yt)
    scale = torch.rand(adapters, generator=g) + 0.5
    return {"a": a.cuda(), "b": b.cuda()[:, :, :top], "ids": ids.cuda(), "rank": rank.cuda(),
            "scale": scale.cuda(), "x": x.cuda(), "z": z.cuda()}


def reference(d, z=True):
    """(Y, the sum of the magnitudes of Y's terms, the adapters' part) in 64 bits."""
    n, rows = d["z"].shape
    y = d["z"].double().clone() if z else torch.zeros(n, rows, dtype=torch.float64, device="cuda")
    mag, part = y.abs(), torch.zeros_like(y)
    for i in range(d["a"].shape[0]):
        at = (d["ids"] == i).nonzero()[:, 0]
        r = int(d["rank"][i])
        if len(at) == 0 or r == 0:
            continue
        a, b, s = d["a"][i, :r].double(), d["b"][i, :, :r].double(), float(d["scale"][i])
        x = d["x"][at].double()
        part[at] = s * (x @ a.T) @ b.T
        mag[at] += s * (x.abs() @ a.abs().T) @ b.abs().T
    return y + part, mag, part


def check(d, got, z=True):
    want, mag, part = reference(d, z)
    got64 = got.double()
    assert torch.isfinite(got64).all()
    # Rounding Y to its type: half a step, which is the same for all values below the least normal one
    # (f16: 2^-25 below 2^-14). Products: 2^-21 of each (three operations of it, doubled
    # for their second order). Sums in 32 bits: at most cols / 16 + rank + 32 additions one after
    # another, each off by 2^-24 of a partial sum, which the sum of the magnitudes bounds.
    cols, top = d["a"].shape[2], d["a"].shape[1]
    step = torch.finfo(got.dtype).eps / 2
    bound = want.abs().clamp(min=torch.finfo(got.dtype).tiny) * step + mag * (2.0**-19 + (cols / 16 + top + 32) * 2.0**-24) + 1e-30
    worst = ((got64 - want).abs() / bound).max().item()
    assert worst <= 1.0, worst
    # The same errors as independent ones: rms of a product 2^-21, of a sum of n steps sqrt(n) 2^-24
    # (n <= 1500 here: 2.3e-6), against the rms of the adapters' part; a product to only 11 bits
    # (2^-12) would show.
    off = (got64 - want).pow(2).mean().sqrt()
    limit = part.pow(2).mean().sqrt() * (2.0**-20 + 2.5e-6) + want.pow(2).mean().sqrt() * step
    assert off <= limit, (off.item(), limit.item())


def run(tq, d, yt=None, stream=None):
    y = torch.full_like(d["z"], float("nan"))
    lora = tq.Lora(d["a"], d["b"], d["rank"], d["scale"])
    tq.tq_lora_add(d["x"], lora, d["ids"], y, d["z"], scratch(tq, len(d["ids"]), d["a"].shape[0]), stream)
    return y


SHAPES = [
    # ntok, cols, rows, adapters, max rank
    (1, 256, 64, 1, 8), (1, 5120, 5120, 4, 16), (2, 8, 1, 1, 1), (3, 264, 33, 2, 3), (5, 1024, 1000, 5, 12),
    (16, 512, 512, 1, 16), (17, 512, 519, 1, 17), (31, 2048, 257, 40, 64), (33, 640, 96, 3, 33),
    (64, 5120, 1031, 64, 8), (100, 136, 2000, 7, 100), (255, 256, 256, 9, 16), (256, 1288, 300, 300, 20),
    (257, 1288, 300, 300, 20), (300, 17408, 100, 3, 256), (1000, 512, 777, 11, 64), (2100, 256, 512, 1, 128),
    (513, 96, 40, 513, 5),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("types", [(F32, BF16, F32), (F32, F16, F32), (BF16, BF16, BF16), (F16, F16, F16),
                                   (F32, BF16, F16), (BF16, BF16, F32)], ids=str)
def test_against_64_bits(tq, shape, types):
    ntok, cols, rows, adapters, top = shape
    xt, wt, yt = types
    d = make(ntok, cols, rows, adapters, top, xt, wt, yt, seed=ntok + rows)
    check(d, run(tq, d))


# many tokens an adapter. From 4096 tokens (2048 above rank 112), 512 an adapter and rank 33 on, tiles of 128,
# their last ones short, in passes of 64 ranks; rows in 16-byte pieces (others go the way of few tokens), and
# fewer columns than thread blocks share
MANY = [(600, 640, 512, 2, 64), (513, 96, 8, 3, 5), (900, 17408, 256, 2, 48),
        (4096, 256, 136, 1, 64), (4100, 640, 512, 8, 33), (5000, 264, 40, 5, 48), (4096, 96, 8, 3, 64),
        (4200, 1288, 2048, 4, 40), (4097, 17408, 72, 2, 64), (6000, 8, 1032, 2, 64), (4500, 520, 777, 2, 50),
        (4096, 256, 136, 9, 64), (4096, 256, 136, 4, 65), (4200, 520, 264, 3, 130), (4100, 1032, 520, 2, 200),
        (4300, 264, 128, 1, 51), (4100, 264, 132, 1, 40), (2048, 136, 264, 4, 113), (2060, 136, 264, 1, 112)]


@pytest.mark.parametrize("shape", MANY, ids=str)
@pytest.mark.parametrize("types", [(F32, BF16, F32), (F32, F16, F32), (BF16, BF16, BF16), (F16, F16, F32),
                                   (F32, BF16, F16)], ids=str)
def test_many_tokens_of_few_adapters(tq, shape, types):
    ntok, cols, rows, adapters, top = shape
    xt, wt, yt = types
    d = make(ntok, cols, rows, adapters, top, xt, wt, yt, seed=ntok + rows)
    got = run(tq, d)
    check(d, got)
    lora, ws = tq.Lora(d["a"], d["b"], d["rank"], d["scale"]), scratch(tq, ntok, adapters)
    y = d["z"].clone()
    tq.tq_lora_add(d["x"], lora, d["ids"], y, y, ws)
    assert torch.equal(y, got)
    none = torch.full_like(y, float("nan"))
    tq.tq_lora_add(d["x"], lora, d["ids"], none, workspace=ws)
    check(d, none, z=False)


def test_many_tokens_order_and_strides(tq):
    """Tokens in another order, and rows of wider tensors, give the same bits."""
    d = make(4500, 520, 264, 6, 40, seed=50)
    want = run(tq, d)
    p = torch.randperm(4500, generator=torch.Generator().manual_seed(1)).cuda()
    e = dict(d, x=d["x"][p].contiguous(), z=d["z"][p].contiguous(), ids=d["ids"][p].contiguous())
    assert torch.equal(run(tq, e), want[p])
    wide = torch.full((4500, 1000), float("nan"), device="cuda")
    x, y, z = wide[:, 4:524], wide[:, 528:792], torch.full((4500, 272), float("nan"), device="cuda")[:, 4:268]
    x.copy_(d["x"])
    z.copy_(d["z"])
    before = wide.clone()
    tq.tq_lora_add(x, tq.Lora(d["a"], d["b"], d["rank"], d["scale"]), d["ids"], y, z, scratch(tq, 4500, 6))
    assert torch.equal(y, want)
    left = torch.ones_like(wide, dtype=torch.bool)
    left[:, 528:792] = False
    assert torch.equal(wide.view(I32)[left], before.view(I32)[left])


@pytest.mark.parametrize("top", [40, 100])
def test_many_tokens_graph_and_streams(tq, top):
    """From a graph with other adapters each time, and on two streams at once; in one pass and in two."""
    ntok, cols, rows, adapters = 4200, 264, 136, 4
    ds = [make(ntok, cols, rows, adapters, top, seed=60 + s, bare=0.3 * s) for s in range(3)]
    want = [run(tq, d) for d in ds]
    for d, y in zip(ds, want):
        check(d, y)
        assert torch.equal(y[d["ids"] < 0], d["z"][d["ids"] < 0])
    e = {n: t.clone() for n, t in ds[0].items()}
    lora = tq.Lora(e["a"], e["b"], e["rank"], e["scale"])
    y, ws = torch.empty_like(e["z"]), scratch(tq, ntok, adapters)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        tq.tq_lora_add(e["x"], lora, e["ids"], y, e["z"], ws)
    torch.cuda.synchronize()
    for d, w in list(zip(ds, want))[::-1]:
        for n in e:
            e[n].copy_(d[n])
        y.fill_(float("nan"))
        graph.replay()
        assert torch.equal(y, w)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ds], [[], [], []]
    for _ in range(4):
        for i, (d, s) in enumerate(zip(ds, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(tq, d))
    torch.cuda.synchronize()
    for i in range(3):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("top", [40, 51, 100])
def test_many_tokens_weights_at_any_address(tq, top):
    """Rows of B 2 bytes off, and of an odd stride, give the bits of those at 8-byte addresses."""
    d = make(4100, 264, 136, 3, top, seed=70, pad=-top % 4)
    want = run(tq, d)
    b = torch.full((3, 140, top + 3 - top % 2), float("nan"), device="cuda", dtype=BF16)[:, 3:139, 1:top + 1]
    b.copy_(d["b"])
    assert torch.equal(run(tq, dict(d, b=b)), want)


def test_many_tokens_not_finite_and_bad(tq):
    d = make(4300, 256, 64, 2, 48, seed=51, bare=0.0, ragged=False)
    clean = run(tq, d)
    d["x"][3, 5], d["x"][4200, 9] = float("inf"), float("nan")
    got = run(tq, d)
    touched = torch.zeros(4300, dtype=torch.bool, device="cuda")
    touched[[3, 4200]] = True
    assert torch.equal(got[~touched], clean[~touched]) and not torch.isfinite(got[touched]).any()
    d["ids"][::3] = 9
    got = run(tq, d)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    assert torch.equal(got[::3], d["z"][::3])


@pytest.mark.parametrize("ntok", [1, 16, 40, 300, 700, 5000])
def test_exact_on_small_integers(tq, ntok):
    """Sums of integers below 2^24 have no rounding in any order: the result is equal to the bit."""
    g = torch.Generator().manual_seed(ntok)

    def ints(hi, *shape):
        return torch.randint(-hi, hi + 1, shape, generator=g).float()
    for top, cols, rows in ((5, 72, 31), (16, 512, 300), (64, 1024, 136)):
        d = {"a": ints(2, 3, top, cols).bfloat16().cuda(), "b": ints(2, 3, rows, top).bfloat16().cuda(),
             "x": ints(3, ntok, cols).cuda(), "z": ints(100, ntok, rows).cuda(),
             "ids": torch.randint(-1, 3, (ntok,), generator=g, dtype=I32).cuda(),
             "rank": torch.tensor([top, 1, top // 2], dtype=I32).cuda(), "scale": torch.tensor([1.0, 2.0, -1.0]).cuda()}
        want = reference(d)[0]
        assert want.abs().max() < 2**24
        assert torch.equal(run(tq, d).double(), want)


@pytest.mark.parametrize("ntok", [3, 40, 400])
def test_in_place_and_without_base(tq, ntok):
    d = make(ntok, 520, 203, 4, 24, seed=5, bare=0.3)
    want = run(tq, d)
    lora = tq.Lora(d["a"], d["b"], d["rank"], d["scale"])
    y = d["z"].clone()
    tq.tq_lora_add(d["x"], lora, d["ids"], y, y, scratch(tq, ntok, 4))
    assert torch.equal(y, want)
    none = torch.full_like(y, float("nan"))
    tq.tq_lora_add(d["x"], lora, d["ids"], none, workspace=scratch(tq, ntok, 4))
    check(d, none, z=False)
    assert (none[d["ids"] < 0] == 0).all()


@pytest.mark.parametrize("ntok", [4, 300])
def test_rows_without_adapter_keep_their_bits(tq, ntok):
    """In place nothing of them is written; beside it they are copied, NaN and all."""
    d = make(ntok, 256, 100, 2, 8, seed=6)
    d["ids"][::2] = -5
    d["z"][::2, ::3] = float("nan")
    lora = tq.Lora(d["a"], d["b"], d["rank"], d["scale"])
    y = d["z"].clone()
    tq.tq_lora_add(d["x"], lora, d["ids"], y, y, scratch(tq, ntok, 2))
    out = run(tq, d)
    for got in (y, out):
        assert torch.equal(got[::2].view(I32), d["z"][::2].view(I32))


@pytest.mark.parametrize("ntok", [5, 300])
def test_strides_and_offsets(tq, ntok):
    """Views of larger tensors, rows of a fused projection, an adapter cut out of a wider stack."""
    d = make(ntok, 264, 131, 3, 10, seed=7, pad=3)
    want = run(tq, d)
    wide = torch.full((ntok, 900), float("nan"), device="cuda")
    x = wide[:, 12:12 + 264]
    x.copy_(d["x"])
    y = wide[:, 301:301 + 131]      # in the same rows as x
    z = torch.full((ntok, 140), float("nan"), device="cuda")[:, 5:136]
    z.copy_(d["z"])
    a = torch.full((3, 12, 280), float("nan"), device="cuda", dtype=BF16)[:, :10, 8:272]
    a.copy_(d["a"])
    b = torch.full((3, 140, 13), float("nan"), device="cuda", dtype=BF16)[:, 7:138, 1:11]
    b.copy_(d["b"])
    before = wide.clone()
    tq.tq_lora_add(x, tq.Lora(a, b, d["rank"], d["scale"]), d["ids"], y, z, scratch(tq, ntok, 3))
    check(d, y)
    assert (y - want).abs().max() <= 1e-4   # other loads, the same products
    left = torch.ones_like(wide, dtype=torch.bool)
    left[:, 301:432] = False
    assert torch.equal(wide.view(I32)[left], before.view(I32)[left])


def test_defaults_of_rank_and_scale(tq):
    d = make(9, 256, 70, 3, 8, seed=8, ragged=False)
    d["scale"].fill_(1.0)
    y = torch.empty_like(d["z"])
    tq.tq_lora_add(d["x"], tq.Lora(d["a"], d["b"]), d["ids"], y, d["z"])
    check(d, y)


@pytest.mark.parametrize("ntok", [24, 500])
def test_order_of_the_tokens_does_not_matter(tq, ntok):
    d = make(ntok, 1024, 333, 6, 16, seed=9)
    want = run(tq, d)
    p = torch.randperm(ntok, generator=torch.Generator().manual_seed(1)).cuda()
    e = dict(d, x=d["x"][p].contiguous(), z=d["z"][p].contiguous(), ids=d["ids"][p].contiguous())
    assert torch.equal(run(tq, e), want[p])
    assert torch.equal(run(tq, d), want)    # and the same call twice gives the same bits


@pytest.mark.parametrize("ntok", [20, 400])
def test_values_that_are_not_finite_stay_in_their_row(tq, ntok):
    d = make(ntok, 256, 64, 2, 16, seed=10, bare=0.0)
    clean = run(tq, d)
    for t, v in ((3, float("inf")), (7, float("nan")), (11, -float("inf"))):
        d["x"][t, 5] = v
    got = run(tq, d)
    touched = torch.zeros(ntok, dtype=torch.bool, device="cuda")
    touched[[3, 7, 11]] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert not torch.isfinite(got[touched]).any() or (d["rank"][d["ids"][touched].long()] == 0).any()


def test_large_values_of_x(tq):
    """Near the largest 32-bit float, and an infinity that the formula gives: the split in two parts
    overflows nowhere on its own."""
    d = make(8, 256, 40, 1, 4, seed=11, bare=0.0, ragged=False)
    d["x"].zero_()
    d["a"].fill_(1.0)
    d["b"].fill_(1.0)
    d["scale"].fill_(2.0**-4)
    d["z"].zero_()
    d["x"][0, 3] = 3.4e38
    d["x"][1, 3] = float("inf")
    d["x"][2, 3] = 2.0**-126
    got = run(tq, d)
    assert torch.allclose(got[0], torch.full_like(got[0], 3.4e38 / 4), rtol=2.0**-20)
    assert (got[1] == float("inf")).all()
    assert torch.allclose(got[2], torch.full_like(got[2], 2.0**-128), rtol=2.0**-9, atol=0)


@pytest.mark.parametrize("ntok", [12, 600])
def test_bad_indexes_are_reported_and_get_the_base(tq, ntok):
    d = make(ntok, 256, 90, 3, 8, seed=12, bare=0.0, ragged=False)
    d["rank"][1] = 9            # above max_rank
    d["ids"][::4] = 3           # no such adapter
    d["ids"][1::4] = 1
    d["ids"][2] = 0x7FFFFFFF
    got = run(tq, d)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    bad = (d["ids"] == 1) | (d["ids"] >= 3)
    assert torch.equal(got[bad], d["z"][bad])
    e = {k: v.clone() for k, v in d.items()}
    e["rank"][1] = 0
    e["ids"][bad] = -1
    check(e, got)
    d["rank"][1] = -1
    got = run(tq, d)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    assert torch.equal(got[bad], d["z"][bad])


def test_nothing_to_add(tq):
    x, z = torch.randn(3, 16, device="cuda"), torch.randn(3, 5, device="cuda")
    for adapters, top in ((0, 4), (2, 0)):
        lora = tq.Lora(torch.empty(adapters, top, 16, dtype=F16, device="cuda"),
                       torch.empty(adapters, 5, top, dtype=F16, device="cuda"))
        y = torch.full_like(z, float("nan"))
        tq.tq_lora_add(x, lora, torch.full((3,), -1, dtype=I32, device="cuda"), y, z)
        assert torch.equal(y, z)
    tq.tq_lora_add(x[:0], lora, torch.empty(0, dtype=I32, device="cuda"), z[:0], z[:0])


@pytest.mark.parametrize("ntok", [8, 500])
def test_graph_with_other_adapters_each_time(tq, ntok):
    d = make(ntok, 512, 200, 5, 16, seed=13)
    lora = tq.Lora(d["a"], d["b"], d["rank"], d["scale"])
    y, ws = torch.empty_like(d["z"]), scratch(tq, ntok, 5)
    tq.tq_lora_add(d["x"], lora, d["ids"], y, d["z"], ws)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        tq.tq_lora_add(d["x"], lora, d["ids"], y, d["z"], ws)
    torch.cuda.synchronize()
    for seed in range(4):
        e = make(ntok, 512, 200, 5, 16, seed=20 + seed, bare=0.2 * seed)
        for n in ("x", "z", "ids", "a", "b", "rank", "scale"):
            d[n].copy_(e[n])
        y.fill_(float("nan"))
        graph.replay()
        check(d, y)


@pytest.mark.parametrize("ntok", [8, 500])
def test_two_streams(tq, ntok):
    """Calls on two streams at once, each with a workspace of its own."""
    ds = [make(ntok, 1024, 600, 5, 16, seed=s) for s in (30, 31)]
    want = [run(tq, d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[], []]
    for _ in range(5):
        for i, (d, s) in enumerate(zip(ds, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(tq, d))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_offsets_past_32_bits(tq):
    """Adapters, activations and outputs that lie past 2^31 and 2^32 values from their start."""
    step = (1 << 31) + 64
    flat = torch.zeros(2 * step + 4096, dtype=F16, device="cuda")
    cols, rows, top = 64, 40, 8
    a = flat.as_strided((3, top, cols), (step, cols, 1))
    b = flat.as_strided((3, rows, top), (step, top, 1), 2048)
    d = make(4, cols, rows, 3, top, F32, F16, F32, seed=14, bare=0.0, ragged=False)
    a.copy_(d["a"])
    b.copy_(d["b"])
    d["ids"].copy_(torch.tensor([2, 0, 1, 2], dtype=I32))
    big = torch.empty(3 * ((1 << 30) + 64) + 4096, dtype=F32, device="cuda")
    y = big.as_strided((4, rows), ((1 << 30) + 64, 1))
    z = big.as_strided((4, rows), ((1 << 30) + 64, 1), 64)
    x = big.as_strided((4, cols), ((1 << 30) + 64, 1), 128)
    z.copy_(d["z"])
    x.copy_(d["x"])
    tq.tq_lora_add(x, tq.Lora(a, b, d["rank"], d["scale"]), d["ids"], y, z)
    check(d, y.contiguous())


def test_workspace_refused(tq):
    d = make(300, 256, 64, 2, 8, seed=15)
    lora, y = tq.Lora(d["a"], d["b"], d["rank"], d["scale"]), torch.empty_like(d["z"])
    n = tq.tq_lora_add_workspace_bytes(300, 2)
    if n:
        for ws, code in ((None, tq.TQ_ERR_NULL), (torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
                                                   tq.TQ_ERR_WORKSPACE)):
            with pytest.raises(tq.TQError) as e:
                tq.tq_lora_add(d["x"], lora, d["ids"], y, d["z"], ws)
            assert e.value.code == code
    for bad in (dict(Z=d["z"][:, :63]), dict(Y=y[:5]), dict(ids=d["ids"][:7])):
        args = dict(X=d["x"], lora=lora, ids=d["ids"], Y=y, Z=d["z"])
        args.update(bad)
        with pytest.raises(tq.TQError) as e:
            tq.tq_lora_add(**args)
        assert e.value.code == tq.TQ_ERR_SHAPE


@pytest.mark.parametrize("ntok,top", [(3, 8), (40, 20), (300, 20), (4200, 40)])
def test_without_columns(tq, ntok, top):
    """A product over nothing is zero: Y is Z, X and A may be missing."""
    d = make(ntok, 8, 264, 2, top, seed=80, ragged=False)
    lora = tq.Lora(d["a"], d["b"], None, d["scale"])
    s = lora.struct
    s.a, s.cols, s.a_stride, s.a_row_stride = None, 0, 0, 0
    y = torch.full_like(d["z"], float("nan"))
    ws = scratch(tq, ntok, 2)
    rc = tq.library().tq_lora_add(None, 0, tq.TQ_F32, lora.ref, d["ids"].data_ptr(), d["z"].data_ptr(), 264,
                                  y.data_ptr(), 264, tq.TQ_F32, ntok, ws.data_ptr() if ws is not None else None,
                                  ws.numel() if ws is not None else 0, torch.cuda.current_stream().cuda_stream)
    assert rc == tq.TQ_OK
    assert torch.equal(y, d["z"])


@pytest.mark.parametrize("shape", [(4200, 264, 136, 1, 40), (6000, 8, 1032, 2, 64), (4097, 5120, 2048, 2, 64),
                                   (4200, 520, 264, 3, 130)], ids=str)
def test_timeout_reported_then_cleared(tq, shape):
    """A first block of the kernel for long batches that hands nothing to the tensor cores (columns of x, or,
    where it has none, rows of B): its waits run out, once, the other tiles are right, the next call is. In
    one pass of ranks and in three."""
    ntok, cols, rows, adapters, top = shape
    d = make(ntok, cols, rows, adapters, top, seed=90)
    want = run(tq, d)
    assert tq.tq_device_status() == tq.TQ_OK
    torch.cuda.synchronize()
    tq.tq_debug_stall_next_launch(200_000)
    try:
        t = time.perf_counter()
        got = run(tq, d)
        torch.cuda.synchronize()
        t = time.perf_counter() - t
    finally:
        tq.tq_debug_stall_next_launch(0)
    assert tq.tq_device_status() == tq.TQ_ERR_TIMEOUT
    assert t < 0.8 and tq.tq_device_status() == tq.TQ_OK
    assert ((got != want).any(dim=1).sum() <= 128)      # the tokens of one tile
    assert torch.equal(run(tq, d), want)


@pytest.mark.parametrize("ntok", [4096, 300])
def test_many_columns_of_one_sign(tq, ntok):
    """Sums on the tensor cores are cut, which leans one way: they may not grow with the columns. 2^20 columns of
    positive values, far more than any chain of them."""
    cols, rows, top = 1 << 20, 8, 40
    g = torch.Generator(device="cuda").manual_seed(ntok)
    x = torch.rand(ntok, cols, generator=g, device="cuda")
    a = (torch.rand(1, top, cols, generator=g, device="cuda") + 0.5).to(BF16)
    b = torch.zeros(1, rows, top, device="cuda", dtype=BF16)
    pick = torch.arange(rows) * 5
    b[0, torch.arange(rows), pick] = 1.0                       # Y's rows are values of h
    y = torch.empty(ntok, rows, device="cuda")
    tq.tq_lora_add(x, tq.Lora(a, b), torch.zeros(ntok, dtype=I32, device="cuda"), y, None, scratch(tq, ntok, 1))
    at = torch.arange(0, ntok, ntok // 48, device="cuda")
    want = x[at].double() @ a[0, pick.cuda()].double().T
    # A step on the tensor cores adds eight products to a sum, each of the nine cut by less than a unit of 2^-23
    # of it, and a chain of 128 steps (16 chunks, four steps of both parts) grows evenly, so half of that on
    # average: 128 / 2 * 9 * 2^-23. These are joined by at most 64 * 8 + 4 additions, growing too: 258 * 2^-24.
    # Products: 2^-21.
    bound = 64 * 9 * 2.0**-23 + 258 * 2.0**-24 + 2.0**-21
    worst = ((y[at].double() - want).abs() / want).max().item()
    print("off by", worst)
    assert worst <= bound, (worst, bound)


@pytest.mark.parametrize("types", [(F32, BF16, F32), (F32, F16, F32), (BF16, BF16, F32), (F32, BF16, BF16)], ids=str)
@pytest.mark.parametrize("ntok,top,rows", [(5, 5, 31), (9, 40, 136), (40, 16, 136), (40, 64, 31), (300, 20, 136),
                                           (300, 100, 33), (5000, 40, 136), (4200, 130, 136)])
def test_infinite_weights(tq, ntok, top, rows, types):
    """What the formula gives: infinity, and NaN where zero meets it or two of them. Small integers, whose
    second part is zero in every split, also beside each infinity."""
    xt, wt, yt = types
    g = torch.Generator().manual_seed(ntok + top)
    cols = 72

    def ints(hi, *shape):
        return torch.randint(-hi, hi + 1, shape, generator=g).float()
    a, b = ints(2, 3, top, cols), ints(2, 3, rows, top)
    a[0, 3, 7], a[0, top - 1, 71], b[1, 4, 2], b[1, rows - 1, top - 1] = INF, -INF, -INF, INF
    a[2, 0, 0], b[2, 5, 1], b[2, 6, 0] = INF, INF, float("nan")
    d = {"a": a.to(wt).cuda(), "b": b.to(wt).cuda(), "x": ints(3, ntok, cols).to(xt).cuda(),
         "z": ints(100, ntok, rows).to(yt).cuda(), "ids": torch.randint(-1, 3, (ntok,), generator=g, dtype=I32).cuda(),
         "rank": torch.full((3,), top, dtype=I32).cuda(), "scale": torch.tensor([1.0, 2.0, -1.0]).cuda()}
    d["x"][::5, 3] = INF
    want = d["z"].double()
    for i in range(3):
        at = (d["ids"] == i).nonzero()[:, 0]
        for t in at.split(256):      # (products term by term: no library's way with infinities)
            h = (d["x"][t].double()[:, None] * d["a"][i].double()).sum(2) * d["scale"][i].double()
            want[t] += (h[:, None] * d["b"][i].double()).sum(2)
    got, want = run(tq, d), want.to(yt)
    assert torch.isnan(want).any() and torch.isinf(want).any() and torch.isfinite(want).any()
    wrong = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not wrong.any(), (wrong.sum().item(), got[wrong][:8], want[wrong][:8], wrong.nonzero()[:8])
