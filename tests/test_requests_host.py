"""Host side of the adapter and sampling calls: workspace sizes and refusals, which return before any
CUDA call (fake addresses are safe)."""
import ctypes
import math

import pytest
import torch

A, B, C, D, E, G, H, W = (0x7F0000000000 + i * 0x10000000 for i in range(8))
BIG = 1 << 40


@pytest.fixture(scope="module")
def tq():
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    return bit_matvec_gb300


def lora(tq, **over):
    a = dict(a=A, b=B, rank=C, scale=C + 4096, adapters=4, top=16, rows=100, cols=64, as_=1024, ars=64,
             bs=1600, brs=16, type=2)
    a.update(over)
    s = tq.Lora._Struct(a["a"], a["b"], a["rank"], a["scale"], a["adapters"], a["top"], a["rows"],
                        a["cols"], a["as_"], a["ars"], a["bs"], a["brs"], a["type"], 0)
    return s, ctypes.addressof(s)


def add(tq, struct=None, **over):
    a = dict(x=D, xs=64, xt=0, ids=E, z=G, zs=100, y=H, ys=100, yt=0, n=3, ws=W, wsb=1 << 20)
    a.update(over)
    keep, ref = struct or lora(tq)
    return tq.library().tq_lora_add(a["x"], a["xs"], a["xt"], ref, a["ids"], a["z"], a["zs"], a["y"],
                                    a["ys"], a["yt"], a["n"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(adapters=-1), "SHAPE"), (dict(adapters=32769), "SHAPE"), (dict(top=-1), "SHAPE"),
    (dict(top=257, brs=257), "SHAPE"), (dict(rows=-1), "SHAPE"), (dict(rows=(1 << 24) + 1), "SHAPE"),
    (dict(cols=60), "SHAPE"), (dict(cols=-8), "SHAPE"), (dict(cols=1 << 25), "SHAPE"),
    (dict(as_=-8), "SHAPE"), (dict(as_=1028), "SHAPE"), (dict(ars=68), "SHAPE"), (dict(ars=56), "SHAPE"),
    (dict(brs=15), "SHAPE"), (dict(bs=-1), "SHAPE"), (dict(as_=2 * BIG), "SHAPE"),
    (dict(adapters=32768, bs=BIG), "OK"), (dict(rows=1 << 24, brs=BIG), "SHAPE"),
    (dict(type=0), "TYPE"), (dict(type=3), "TYPE"), (dict(a=None), "NULL"), (dict(b=None), "NULL"),
    (dict(a=A + 8), "ALIGN"), (dict(b=B + 1), "ALIGN"), (dict(rank=C + 2), "ALIGN"),
    (dict(scale=C + 1), "ALIGN"),
])
def test_lora_description_refusals(tq, over, code):
    # (no tokens: what is allowed enqueues nothing)
    want = getattr(tq, "TQ_" + code if code == "OK" else "TQ_ERR_" + code)
    assert add(tq, struct=lora(tq, **over), **(dict(n=0) if code == "OK" else {})) == want


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), "SHAPE"), (dict(n=1 << 31), "SHAPE"), (dict(xs=56), "SHAPE"), (dict(xs=66), "SHAPE"),
    (dict(ys=99), "SHAPE"), (dict(zs=99), "SHAPE"), (dict(xs=-64), "SHAPE"), (dict(ys=2 * BIG), "SHAPE"),
    (dict(n=(1 << 31) - 1, ys=BIG), "SHAPE"), (dict(xt=1), "TYPE"), (dict(xt=5), "TYPE"),
    (dict(yt=3), "TYPE"), (dict(yt=-1), "TYPE"), (dict(x=None), "NULL"), (dict(ids=None), "NULL"),
    (dict(y=None), "NULL"), (dict(x=D + 8), "ALIGN"), (dict(ids=E + 2), "ALIGN"), (dict(y=H + 2), "ALIGN"),
    (dict(z=G + 1), "ALIGN"), (dict(y=D), "ALIAS"), (dict(y=A), "ALIAS"), (dict(y=B + 64), "ALIAS"),
    (dict(y=C), "ALIAS"), (dict(y=C + 4096), "ALIAS"), (dict(y=E), "ALIAS"), (dict(y=G + 4), "ALIAS"),
    (dict(y=G, ys=104), "ALIAS"), (dict(y=G + 100 * 4), "ALIAS"),
])
def test_lora_refusals(tq, over, code):
    assert add(tq, **over) == getattr(tq, "TQ_ERR_" + code)


def test_lora_nothing_to_do(tq):
    assert add(tq, n=0, x=None, y=None, ids=None) == tq.TQ_OK
    assert add(tq, struct=lora(tq, rows=0)) == tq.TQ_OK
    assert tq.library().tq_lora_add(D, 64, 0, None, E, G, 100, H, 100, 0, 3, W, 1 << 20,
                                    None) == tq.TQ_ERR_NULL


def test_lora_without_columns(tq):
    """h is zeros then, and B is read all the same: it may not be missing where there is a rank."""
    without = dict(cols=0, a=None, as_=0, ars=0)
    for over in ({}, dict(top=1, brs=1), dict(adapters=1)):
        assert add(tq, struct=lora(tq, b=None, **without, **over), x=None, xs=0) == tq.TQ_ERR_NULL


def test_lora_workspace(tq):
    assert tq.tq_lora_add_workspace_bytes(0, 0) == tq.tq_lora_add_workspace_bytes(256, 32768) == 0
    sizes = [tq.tq_lora_add_workspace_bytes(n, 64) for n in (257, 1000, 8192, 1 << 20)]
    assert sizes == sorted(sizes)
    # some bytes a token and an adapter
    assert tq.tq_lora_add_workspace_bytes(1 << 20, 32768) <= 32 * ((1 << 20) + 32768)
    for bad in ((-1, 4), (5, -1), (1 << 31, 4), (5, 32769)):
        with pytest.raises(tq.TQError):
            tq.tq_lora_add_workspace_bytes(*bad)


def test_lora_class(tq):
    a, b = torch.zeros(2, 4, 8, dtype=torch.float16), torch.zeros(2, 5, 4, dtype=torch.float16)
    for bad in ((a, b), (a[0], b), (a, b.bfloat16()), (a, b[:, :, :3]), (a[:1], b)):
        with pytest.raises(ValueError):   # the first: not on a GPU
            tq.Lora(*bad)


def test_lora_rank_and_scale_in_one_piece(tq):
    """Their addresses alone are kept: views with gaps, or of one value for all, would be read
    beside what they show."""
    a, b = torch.zeros(2, 4, 8, dtype=torch.float16), torch.zeros(2, 5, 4, dtype=torch.float16)
    rank, scale = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2)
    for kw in (dict(rank=rank[::2]), dict(rank=rank[:1].expand(2)), dict(scale=scale[:, 1]),
               dict(scale=torch.ones(1).expand(2)), dict(rank=rank[:2], scale=scale[:, 0])):
        with pytest.raises(ValueError, match="contiguous"):
            tq.Lora(a, b, **kw)
    with pytest.raises(ValueError, match="CUDA"):   # what is left to refuse here
        tq.Lora(a, b, rank[2:], scale[1])


def draw(tq, **over):
    a = dict(x=A, stride=1000, type=0, n=3, vocab=1000, u=B, t=C, k=C + 4096, p=C + 8192, m=C + 12288,
             tokens=D, logp=E)
    a.update(over)
    return tq.library().tq_sample(a["x"], a["stride"], a["type"], a["n"], a["vocab"], a["u"], a["t"],
                                  a["k"], a["p"], a["m"], a["tokens"], a["logp"], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), "SHAPE"), (dict(n=1 << 31), "SHAPE"), (dict(vocab=0), "SHAPE"),
    (dict(vocab=262145, stride=262145), "SHAPE"), (dict(stride=999), "SHAPE"), (dict(stride=-1), "SHAPE"),
    (dict(stride=2 * BIG), "SHAPE"), (dict(n=(1 << 31) - 1, stride=BIG), "SHAPE"), (dict(type=3), "TYPE"),
    (dict(x=None), "NULL"), (dict(u=None), "NULL"), (dict(tokens=None), "NULL"), (dict(x=A + 2), "ALIGN"),
    (dict(x=A + 1, type=1), "ALIGN"), (dict(u=B + 1), "ALIGN"), (dict(t=C + 2), "ALIGN"),
    (dict(k=C + 2), "ALIGN"), (dict(p=C + 3), "ALIGN"), (dict(m=C + 1), "ALIGN"),
    (dict(tokens=D + 2), "ALIGN"), (dict(logp=E + 2), "ALIGN"), (dict(tokens=A + 8), "ALIAS"),
    (dict(logp=B), "ALIAS"), (dict(tokens=E), "ALIAS"), (dict(logp=C + 8196), "ALIAS"),
])
def test_sample_refusals(tq, over, code):
    assert draw(tq, **over) == getattr(tq, "TQ_ERR_" + code)


def test_sample_nothing_to_do(tq):
    assert draw(tq, n=0, x=None, u=None, tokens=None) == tq.TQ_OK


def test_marshalling(tq):
    """What the C marshalling refuses before it looks for a GPU."""
    calls = __import__("bit_matvec_gb300.binding", fromlist=["_calls"])._calls()
    x = torch.zeros(3, 64)
    for bad in ([], [x] * 3, [None] * 11):
        with pytest.raises(TypeError):
            calls.lora_add(*bad)
        with pytest.raises(TypeError):
            calls.sample(*bad)
    with pytest.raises(ValueError):   # not on a GPU
        tq.tq_sample(x, x, x)
    with pytest.raises(tq.TQError) as e:
        tq.tq_sample(torch.zeros(3, 2, 64), x, x)
    assert e.value.code == tq.TQ_ERR_SHAPE
    with pytest.raises(tq.TQError) as e:
        tq.tq_sample(x.double(), x, x)
    assert e.value.code == tq.TQ_ERR_TYPE


class Placed:
    """What the marshalling asks a tensor for, of one that would lie on GPU `device`."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0, at=A):
        self.shape, self.dtype, self.device, self.at = torch.Size(shape), dtype, device, at

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.at

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize


def test_tensors_of_several_devices(tq):
    """Each tensor of a call in turn on another GPU than the others, and the description's: refused
    before anything is asked of a GPU."""
    calls = __import__("bit_matvec_gb300.binding", fromlist=["_calls"])._calls()
    f32, i32, bf16 = torch.float32, torch.int32, torch.bfloat16
    rope = tq.Rope._Struct(A, 32, 0, 1.0)
    cache = tq.PagedKV._Struct(A, B, C, 2, 8, 8, 16, 16, 2, 64, 2048, 1024, 64, 2, 0)
    low = tq.Lora._Struct(A, B, None, None, 4, 16, 100, 64, 1024, 64, 1600, 16, 2, 0)
    every = {
        "lora_add": ((3, 64), low, ("i", 3), (3, 100), (3, 100), ("b", 64), None),
        "sample": ((3, 50), ("f", 3), ("i", 3), ("f", 3), ("i", 3), ("f", 3), ("f", 3), ("f", 3), None),
        "paged_attention": (("q", 3, 4, 64), cache, ("i", 3), ("i", 2), ("q", 3, 4, 64), 2, 100, 0.125, ("b", 64),
                            0, ("f", 12), None),
        "kv_append": ((3, 4, 64), (3, 2, 64), (3, 2, 64), ("q", 3, 4, 64), cache, ("i", 3), ("i", 3), rope,
                      ("f", 64), ("f", 64), 1e-6, None),
        "qk_norm_rope": ((3, 4, 64), (3, 2, 64), (3, 4, 64), (3, 2, 64), ("i", 3), rope, ("f", 64), ("f", 64),
                         1e-6, None),
    }
    for name, form in every.items():
        movable = [i for i, f in enumerate(form) if isinstance(f, (tuple, ctypes.Structure))]
        for away in movable:
            args = []
            for i, f in enumerate(form):
                device = 1 if i == away else 0
                if isinstance(f, ctypes.Structure):
                    f.device = device
                    f = ctypes.addressof(f)
                elif isinstance(f, tuple):
                    kind = f[0] if isinstance(f[0], str) else "f"
                    dtype = {"f": f32, "i": i32, "b": torch.uint8, "q": bf16}[kind]
                    f = Placed(f[1:] if isinstance(f[0], str) else f, dtype, device)
                args.append(f)
            with pytest.raises(ValueError, match="one device"):
                getattr(calls, name)(*args)
