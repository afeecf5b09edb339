"""Host side of the norm/rotation, append and attention calls: rotation tables against their
formulas, and refusals, which return before any CUDA call (fake addresses are safe)."""
import ctypes
import math

import pytest
import torch

A, B, C, D, E, G, H = (0x7F0000000000 + i * 0x10000000 for i in range(7))
FLOAT = ctypes.c_float


@pytest.fixture(scope="module")
def tq():
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    return bit_matvec_gb300


def turn(t):
    return (int(t) % (1 << 64)) / 2.0**64


@pytest.mark.parametrize("rot,base", [(2, 1e4), (64, 1e4), (128, 5e5), (20, 10.0)])
def test_plain_turns(tq, rot, base):
    t, amp = tq.tq_rope_turns(rot, base)
    assert t.numel() == rot // 2 and amp == 1.0
    for i, x in enumerate(t):
        f = base ** (-2.0 * i / rot)
        assert turn(x) == pytest.approx(f / (2 * math.pi), rel=1e-15)


def test_scaled_turns(tq):
    rot, base, factor, length = 128, 1e4, 4.0, 4096.0
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    got = [turn(x) * 2 * math.pi for x in tq.tq_rope_turns(rot, base, tq.ROPE_LINEAR, factor)[0]]
    assert got == pytest.approx([x / factor for x in f], rel=1e-14)
    nb = base * factor ** (rot / (rot - 2))
    got = [turn(x) * 2 * math.pi for x in tq.tq_rope_turns(rot, base, tq.ROPE_BASE, factor)[0]]
    assert got == pytest.approx([nb ** (-2.0 * i / rot) for i in range(rot // 2)], rel=1e-14)
    assert got[-1] == pytest.approx(f[-1] / factor, rel=1e-12)   # what that base is chosen for
    t, amp = tq.tq_rope_turns(rot, base, tq.ROPE_BANDS, factor, length, 1.0, 4.0)
    assert amp == 1.0
    for i, x in enumerate(t):
        n = length * f[i] / (2 * math.pi)
        keep = min(max((n - 1.0) / 3.0, 0.0), 1.0)
        assert turn(x) * 2 * math.pi == pytest.approx(f[i] * keep + f[i] / factor * (1 - keep), rel=1e-14)
    t, amp = tq.tq_rope_turns(rot, base, tq.ROPE_RAMP, factor, length, 1.0, 32.0)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-7)
    at = [64 * math.log(length / (n * 2 * math.pi)) / math.log(base) for n in (32.0, 1.0)]
    first, last = math.floor(at[0]), math.ceil(at[1])
    assert 0 < first < last < 64
    for i, x in enumerate(t):
        keep = 1 - min(max((i - first) / (last - first), 0.0), 1.0)
        assert turn(x) * 2 * math.pi == pytest.approx(f[i] * keep + f[i] / factor * (1 - keep), rel=1e-14)


@pytest.mark.parametrize("args", [(3, 1e4), (-2, 1e4), (64, 0.0), (64, -1.0), (64, 1e4, 9),
                                  (64, 1e4, 1, 0.5), (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0.0),
                                  (64, 1e4, 4, 2.0, 4096.0, 4.0, 4.0), (64, math.inf),
                                  (64, 1e4, 3, 2.0, 4096.0, 0.0, 4.0), (64, 1e4, 1, math.nan),
                                  (64, 1.0, 3, 2.0, 4096.0)])
def test_turns_refusals(tq, args):
    with pytest.raises(tq.TQError) as e:
        tq.tq_rope_turns(*args)
    assert e.value.code == tq.TQ_ERR_SHAPE


def rope(tq, turns=H, rot=64, amp=1.0):
    r = tq.Rope._Struct(turns, rot, 0, amp)
    return r, ctypes.addressof(r)


def qk(tq, **over):
    a = dict(xq=A, xqs=512, xk=A + 1024, xks=512, xt=0, yq=B, yqs=256, yk=C, yks=256, yt=2, n=3, hq=4,
             hk=4, d=64, qw=D, kw=E, eps=1e-6, rope=None, pos=G)
    a.update(over)
    keep, ref = a["rope"] or rope(tq)
    return tq.library().tq_qk_norm_rope(a["xq"], a["xqs"], a["xk"], a["xks"], a["xt"], a["yq"], a["yqs"],
                                        a["yk"], a["yks"], a["yt"], a["n"], a["hq"], a["hk"], a["d"],
                                        a["qw"], a["kw"], a["eps"], ref, a["pos"], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), "SHAPE"), (dict(hq=-1), "SHAPE"), (dict(d=0), "SHAPE"), (dict(d=65), "SHAPE"),
    (dict(d=258), "SHAPE"), (dict(xqs=200), "SHAPE"), (dict(yks=255), "SHAPE"), (dict(xqs=-512), "SHAPE"),
    (dict(eps=-1.0), "SHAPE"), (dict(eps=math.nan), "SHAPE"), (dict(xt=3), "TYPE"), (dict(yt=-1), "TYPE"),
    (dict(xq=None), "NULL"), (dict(yk=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(xq=A + 2), "ALIGN"), (dict(yq=B + 1), "ALIGN"), (dict(qw=D + 2), "ALIGN"), (dict(pos=G + 1), "ALIGN"),
    (dict(yq=A, yqs=512), "ALIAS"), (dict(yq=A + 4, yqs=512, yt=0), "ALIAS"), (dict(yk=B), "ALIAS"),
    (dict(yq=D), "ALIAS"), (dict(yq=G), "ALIAS"), (dict(yq=H), "ALIAS"),
])
def test_qk_refusals(tq, over, code):
    assert qk(tq, **over) == getattr(tq, "TQ_ERR_" + code)


def test_qk_rope_refusals(tq):
    assert qk(tq, rope=rope(tq, rot=66)) == tq.TQ_ERR_SHAPE
    assert qk(tq, rope=rope(tq, rot=33)) == tq.TQ_ERR_SHAPE
    assert qk(tq, rope=rope(tq, rot=-2)) == tq.TQ_ERR_SHAPE
    assert qk(tq, rope=rope(tq, amp=math.inf)) == tq.TQ_ERR_SHAPE
    assert qk(tq, rope=rope(tq, turns=None)) == tq.TQ_ERR_NULL
    assert qk(tq, rope=rope(tq, turns=H + 4)) == tq.TQ_ERR_ALIGN


def test_qk_nothing_to_do(tq):
    assert qk(tq, n=0, xq=None, yq=None, xk=None, yk=None) == tq.TQ_OK
    assert qk(tq, hq=0, hk=0) == tq.TQ_OK


def cache(tq, **over):
    a = dict(k=A, v=B, table=C, nseq=2, width=4, tstride=4, pages=8, page=16, heads=2, dim=64,
             ps=2048, hs=1024, ss=64, type=2)
    a.update(over)
    s = tq.PagedKV._Struct(a["k"], a["v"], a["table"], a["nseq"], a["width"], a["tstride"], a["pages"],
                           a["page"], a["heads"], a["dim"], a["ps"], a["hs"], a["ss"], a["type"], 0)
    return s, ctypes.addressof(s)


def append(tq, kv=None, **over):
    a = dict(xq=D, xqs=512, xk=D + 1024, xks=512, xv=D + 1536, xvs=512, xt=0, yq=E, yqs=256, seq=G,
             pos=G + 4096, n=3, hq=4, qw=H, kw=H + 4096, eps=1e-6)
    a.update(over)
    keep = kv or cache(tq)
    return tq.library().tq_kv_append(a["xq"], a["xqs"], a["xk"], a["xks"], a["xv"], a["xvs"], a["xt"],
                                     a["yq"], a["yqs"], keep[1], a["seq"], a["pos"], a["n"], a["hq"],
                                     a["qw"], a["kw"], a["eps"], None, None)


BAD_CACHES = [(dict(page=12), "SHAPE"), (dict(page=0), "SHAPE"), (dict(dim=60), "SHAPE"),
              (dict(dim=136, hs=4096, ps=8192, ss=136), "SHAPE"), (dict(heads=0), "SHAPE"),
              (dict(pages=0), "SHAPE"), (dict(nseq=-1), "SHAPE"), (dict(nseq=(1 << 30) + 1), "SHAPE"), (dict(tstride=3), "SHAPE"),
              (dict(ss=68), "SHAPE"), (dict(ss=56), "SHAPE"), (dict(hs=8), "SHAPE"), (dict(ps=-8), "SHAPE"),
              (dict(type=0), "TYPE"), (dict(type=7), "TYPE"), (dict(k=None), "NULL"),
              (dict(table=None), "NULL"), (dict(k=A + 8), "ALIGN"), (dict(table=C + 2), "ALIGN")]


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_cache_refusals(tq, over, code):
    kv = cache(tq, **over)
    assert append(tq, kv=kv) == getattr(tq, "TQ_ERR_" + code)
    hq = 2 * max(over.get("heads", 2), 1)
    assert attend(tq, kv=kv, hq=hq) == getattr(tq, "TQ_ERR_" + code)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), "SHAPE"), (dict(xks=100), "SHAPE"), (dict(xvs=64), "SHAPE"), (dict(yqs=64), "SHAPE"),
    (dict(xt=5), "TYPE"), (dict(xk=None), "NULL"), (dict(seq=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(yq=None), "NULL"), (dict(xv=D + 1538), "ALIGN"), (dict(seq=G + 2), "ALIGN"),
    (dict(yq=A), "ALIAS"), (dict(yq=D), "ALIAS"), (dict(xk=A), "ALIAS"), (dict(seq=B), "ALIAS"),
])
def test_append_refusals(tq, over, code):
    assert append(tq, **over) == getattr(tq, "TQ_ERR_" + code)


def test_append_one_buffer_for_keys_and_values_refused(tq):
    assert append(tq, kv=cache(tq, v=A)) == tq.TQ_ERR_ALIAS
    assert append(tq, n=0, xk=None, xv=None, seq=None, pos=None) == tq.TQ_OK


def attend(tq, kv=None, **over):
    a = dict(q=D, qs=256, start=G, lens=G + 4096, o=E, os=256, ot=0, lse=E + 65536, n=3, hq=4, mq=2,
             mkv=64, scale=0.125, window=0, ws=H, wsb=1 << 24)
    a.update(over)
    keep = kv or cache(tq)
    return tq.library().tq_paged_attention(a["q"], a["qs"], keep[1], a["start"], a["lens"], a["o"], a["os"],
                                           a["ot"], a["lse"], a["n"], a["hq"], a["mq"], a["mkv"],
                                           a["scale"], a["window"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(hq=3), "SHAPE"), (dict(hq=0), "SHAPE"), (dict(n=-1), "SHAPE"), (dict(mq=-1), "SHAPE"),
    (dict(mkv=-1), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(scale=math.nan), "SHAPE"),
    (dict(scale=math.inf), "SHAPE"), (dict(qs=250), "SHAPE"), (dict(qs=260), "SHAPE"), (dict(os=255), "SHAPE"),
    (dict(n=1 << 29), "SHAPE"), (dict(ot=4), "TYPE"), (dict(q=None), "NULL"), (dict(o=None), "NULL"), (dict(start=None), "NULL"),
    (dict(lens=None), "NULL"), (dict(q=D + 8), "ALIGN"), (dict(o=E + 2), "ALIGN"), (dict(lse=E + 65537), "ALIGN"),
    (dict(o=D), "ALIAS"), (dict(o=A), "ALIAS"), (dict(lse=G), "ALIAS"), (dict(o=E, lse=E + 64), "ALIAS"),
])
def test_attention_refusals(tq, over, code):
    assert attend(tq, **over) == getattr(tq, "TQ_ERR_" + code)


def test_attention_workspace(tq):
    n = tq.tq_paged_attention_workspace_bytes(2, 3, 4, 2, 64, 2, 100000)
    assert n > 0
    assert attend(tq, mkv=100000, wsb=n - 1) == tq.TQ_ERR_WORKSPACE
    assert attend(tq, mkv=100000, ws=None) == tq.TQ_ERR_NULL
    assert attend(tq, mkv=100000, ws=H + 8) == tq.TQ_ERR_ALIGN
    assert attend(tq, mkv=100000, ws=E) == tq.TQ_ERR_ALIAS
    assert attend(tq, n=0, q=None, o=None) == tq.TQ_OK
    assert attend(tq, kv=cache(tq, nseq=0)) == tq.TQ_OK
    with pytest.raises(tq.TQError):
        tq.tq_paged_attention_workspace_bytes(2, 3, 5, 2, 64, 2, 100)
    # scratch stays within a small multiple of the output however long the cache is
    for nseq, new, hq, hk, kv in ((1, 1, 64, 8, 1 << 20), (64, 1, 40, 8, 8192), (1, 4096, 40, 8, 1 << 17),
                                  (512, 1, 32, 32, 1 << 17), (4, 300, 8, 1, 30000)):
        ntok = nseq * new
        assert tq.tq_paged_attention_workspace_bytes(nseq, ntok, hq, hk, 128, new, kv) <= 96 << 20


def test_binding_checks(tq):
    t = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        tq.PagedKV(torch.zeros(1, 1, 8, 8), torch.zeros(1, 1, 8, 8), torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(t, None, t, None)
    with pytest.raises(ValueError):
        tq.Rope(torch.zeros(4))
    with pytest.raises(tq.TQError):
        tq.tq_qk_norm_rope(t, None, torch.zeros(2, 2, 32), None)


def test_marshalling_module(tq):
    """What the C marshalling refuses before it looks for a GPU."""
    calls = __import__("bit_matvec_gb300.binding", fromlist=["_calls"])._calls()
    x = torch.zeros(3, 2, 64)
    for bad in ([], [x] * 3, [None] * 11):
        with pytest.raises(TypeError):
            calls.qk_norm_rope(*bad)
    with pytest.raises(AttributeError):
        tq.tq_qk_norm_rope(5, None, x, None)
    for other in (torch.zeros(3, 2, 32), torch.zeros(3, 128), torch.zeros(2, 2, 64)):
        with pytest.raises(tq.TQError) as e:
            tq.tq_qk_norm_rope(x, None, other, None)
        assert e.value.code == tq.TQ_ERR_SHAPE
    with pytest.raises(tq.TQError) as e:
        tq.tq_qk_norm_rope(x.double(), None, x, None)
    assert e.value.code == tq.TQ_ERR_TYPE


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1, 1 << 62, (1 << 63) - 1])
def test_windows_as_long_as_any_sequence_plan_as_none(tq, window):
    """The workspace, a function of the plan alone, is that of no window."""
    for sizes in ((1, 1, 64, 8, 128, 1, 131072), (1, 5, 32, 4, 64, 5, 9001), (16, 80, 32, 4, 64, 5, 9001),
                  (64, 64, 40, 8, 128, 1, 8192), (8, 2000, 40, 8, 128, 512, 4096), (3, 3, 8, 8, 64, 1, 100)):
        assert tq.tq_paged_attention_workspace_bytes(*sizes, window) == \
            tq.tq_paged_attention_workspace_bytes(*sizes, 0), sizes


def ramp_rule(rot, base, factor, length, low, high):
    """Frequencies of the ramp from its definition: kept at `high` turns and more over `length`, divided
    by factor at `low` and fewer, between them linear in the pair's number."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    at = [0.5 * rot * math.log(length / (n * 2 * math.pi)) / math.log(base) for n in (high, low)]
    first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    out = []
    for i, x in enumerate(f):
        n = length * x / (2 * math.pi)
        keep = 1.0 if n >= high else 0.0 if n <= low else 1 - (i - first) / (last - first)
        out.append(x * keep + x / factor * (1 - keep))
    return out


@pytest.mark.parametrize("rot,base,length,low,high,what", [
    (8, 10.0, 65536.0, 1.0, 32.0, "kept"),          # 1854 to 10430 turns, all above high
    (128, 1e4, 1e9, 1.0, 32.0, "kept"),
    (64, 1e6, 2.0, 1.0, 32.0, "divided"),           # under a third of a turn
    (8, 10.0, 3.0, 1.0, 2.0, "divided"),
    (2, 1e4, 4096.0, 1.0, 32.0, "kept"), (2, 1e4, 5.0, 1.0, 32.0, "divided"), (2, 1e4, 60.0, 1.0, 32.0, "mixed"),
    (128, 1e4, 4096.0, 1.0, 32.0, "mixed"), (64, 5e5, 8192.0, 1.0, 4.0, "mixed"), (20, 10.0, 300.0, 8.0, 32.0, "mixed"),
    (128, 1e4, 60.0, 1.0, 32.0, "mixed"),           # the ramp begins before the first pair
    (16, 3.0, 300.0, 1.0, 32.0, "mixed"),           # and ends past the last one
])
def test_ramp_ends(tq, rot, base, length, low, high, what):
    factor = 4.0
    got = [turn(x) * 2 * math.pi for x in tq.tq_rope_turns(rot, base, tq.ROPE_RAMP, factor, length, low, high)[0]]
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if what == "kept":
        assert got == pytest.approx(f, rel=1e-14)
    elif what == "divided":
        assert got == pytest.approx([x / factor for x in f], rel=1e-14)
    else:
        assert got == pytest.approx(ramp_rule(rot, base, factor, length, low, high), rel=1e-13)


def test_spans_past_64_bits_refused(tq):
    """Counts and strides that are each allowed, and buffers of more than 2^58 values that their product
    would be (which the tests for overlap could not compute)."""
    most = 1 << 40
    assert qk(tq, n=(1 << 31) - 1, xqs=most) == tq.TQ_ERR_SHAPE
    assert qk(tq, n=(1 << 31) - 1, yks=most) == tq.TQ_ERR_SHAPE
    assert append(tq, n=(1 << 31) - 1, xvs=most) == tq.TQ_ERR_SHAPE
    assert attend(tq, n=1 << 28, qs=most) == tq.TQ_ERR_SHAPE
    assert attend(tq, n=1 << 28, os=most) == tq.TQ_ERR_SHAPE
    for over in (dict(nseq=1 << 30, tstride=most), dict(pages=0x7ffffffe, ps=(1 << 39) - 8),
                 dict(page=1 << 24, ss=(1 << 39) - 8)):
        assert append(tq, kv=cache(tq, **over)) == tq.TQ_ERR_SHAPE
        assert attend(tq, kv=cache(tq, **over)) == tq.TQ_ERR_SHAPE


def test_workspace_error_names_no_other_call(tq):
    with_call = str(tq.TQError(tq.TQ_ERR_WORKSPACE, "tq_paged_attention"))
    assert "workspace" in with_call and "matmul" not in with_call
