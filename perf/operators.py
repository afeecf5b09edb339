"""The operators around the attention of a decode step, as cases to be measured.

Between the fused query/key/value projection (tq_quantize_matmul, whose rows
are f32 [q heads | k heads | v heads]) and the output projection, a serving
program normalises and rotates the queries and keys, appends the keys and
values to a paged cache, and attends from the new tokens to that cache. The
three kinds of case are these three calls:

  qk      tq_qk_norm_rope     queries and keys: RMS norm of each head with a
                              learned weight, then the rotation, one pass
  append  tq_kv_append        the same, with keys and values written to their
                              slots of the paged cache and the queries beside
  attend  tq_paged_attention  causal attention of each sequence's new tokens
                              over its pages, from one token to long chunks

run() computes the plain form in elementary 32-bit torch operations, or, where
`own` is true, calls the library as a user does.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
SCRATCH = 96 << 20   # the one scratch buffer that a serving program keeps for its attention calls


# ---------------------------------------------------------------- cases

def listed():
    """Smallest calls, ordinary ones and large ones of each operator; 5120 = 40 heads x 128 is
    the width of this repository's 15360 x 5120 fused projection."""
    return [
        # the queries and keys of one token of a decode step, as many key heads as query heads
        dict(name="qk 1 token", kind="qk", ntok=1, hq=40, hk=40, dim=128, rot=128, inter=False,
             norm=True, base=1e4, factor=1.0, maxpos=5000, tin="f32", tout="bf16"),
        # a ragged prompt, a part of an 80-wide head rotated in interleaved pairs
        dict(name="qk 509 tokens", kind="qk", ntok=509, hq=20, hk=4, dim=80, rot=40, inter=True,
             norm=True, base=1e4, factor=4.0, maxpos=16000, tin="f32", tout="f16"),
        # a large prefill step at positions of a long context
        dict(name="qk 8192 tokens", kind="qk", ntok=8192, hq=40, hk=8, dim=128, rot=128,
             inter=False, norm=True, base=1e6, factor=8.0, maxpos=131072, tin="f32", tout="bf16"),
        # one new token of each of 64 sequences, a decode step of a batch
        dict(name="append 64 tokens", kind="append", nseq=64, maxq=1, maxkv=4096, hq=40, hk=8,
             dim=128, rot=128, inter=False, norm=True, base=1e6, factor=1.0, page=16, tin="f32",
             tout="bf16"),
        # ragged chunks of a few sequences, no norm, part of a 96-wide head, pages of 48
        dict(name="append 6 chunks", kind="append", nseq=6, maxq=301, maxkv=700, hq=12, hk=12,
             dim=96, rot=64, inter=True, norm=False, base=1e4, factor=2.0, page=48, tin="f16",
             tout="f16"),
        # the chunks of a large prefill step
        dict(name="append 2 x 4096", kind="append", nseq=2, maxq=4096, maxkv=4608, hq=40, hk=8,
             dim=128, rot=128, inter=False, norm=True, base=1e6, factor=8.0, page=64, tin="f32",
             tout="bf16"),
        # the smallest call: one token over a short context
        dict(name="attend 1 token", kind="attend", nseq=1, maxq=1, maxkv=333, hq=40, hk=40,
             dim=128, page=16, window=0, ragged=False, type="f16"),
        # a decode step of a batch, ragged lengths, five query heads to a key head
        dict(name="attend 64 tokens", kind="attend", nseq=64, maxq=1, maxkv=8192, hq=40, hk=8,
             dim=128, page=16, window=0, ragged=True, type="bf16"),
        # one long context
        dict(name="attend 131072", kind="attend", nseq=1, maxq=1, maxkv=131072, hq=64, hk=8,
             dim=128, page=64, window=0, ragged=False, type="bf16"),
        # drafts of 5 tokens checked at once, sliding window
        dict(name="attend 16 x 5", kind="attend", nseq=16, maxq=5, maxkv=9001, hq=32, hk=4,
             dim=64, page=32, window=4096, ragged=True, type="f16"),
        # chunks of several sequences in one step, of ragged lengths
        dict(name="attend 8 chunks", kind="attend", nseq=8, maxq=512, maxkv=4096, hq=40, hk=8,
             dim=128, page=32, window=0, ragged=True, type="bf16"),
        # a large chunk over a long prefix
        dict(name="attend 4096", kind="attend", nseq=1, maxq=4096, maxkv=20480, hq=40, hk=8,
             dim=128, page=64, window=0, ragged=False, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("qk", "append", "attend", "attend"))
    dim = rng.choice((64, 80, 96, 128, 128))
    hk = rng.choice((1, 2, 4, 5, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 8))
    page = rng.choice((8, 16, 32, 48, 64, 128))
    if kind != "attend":
        rot = rng.choice((dim, dim, dim // 2))
        case = dict(kind=kind, hq=hk * group, hk=hk, dim=dim, rot=rot, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.7, base=rng.choice((1e4, 5e5, 1e6)),
                    factor=rng.choice((1.0, 2.0, 8.0)), tin=rng.choice(("f32", "f32", "bf16", "f16")),
                    tout=rng.choice(("bf16", "f16")))
        if kind == "qk":
            case.update(ntok=_log(rng, 1, 8192), maxpos=_log(rng, 9000, 131072))
        else:
            nseq = _log(rng, 1, 64)
            maxq = _log(rng, 1, max(1, 8192 // nseq))
            case.update(nseq=nseq, maxq=maxq, maxkv=maxq + _log(rng, 1, 4096), page=page)
        return case
    case = dict(kind=kind, hq=hk * group, hk=hk, dim=dim, page=page,
                window=rng.choice((0, 0, 0, _log(rng, 16, 4096))), ragged=rng.random() < 0.7,
                type=rng.choice(("bf16", "f16")))
    maxq = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 2048)))
    nseq = _log(rng, 1, 64 if maxq <= 16 else 8)
    # at most 2^30 values of the scores, and a quarter of a million cached tokens
    most = min((1 << 30) // (case["hq"] * maxq * nseq), (1 << 18) // nseq)
    case.update(nseq=nseq, maxq=maxq, maxkv=max(maxq, _log(rng, min(most, max(maxq, 16)), max(most, 16))))
    return case


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """(new tokens, total tokens) of each sequence, the same for every seed: the largest of each is
    there."""
    r = np.random.RandomState(1000003 * case["nseq"] + 1009 * case["maxq"] + case["maxkv"])
    n, mq, mk = case["nseq"], case["maxq"], case["maxkv"]
    if not case.get("ragged", True):
        return np.full(n, mq), np.full(n, mk)
    q = np.maximum(1, np.round(mq * r.uniform(0.3, 1.0, n)).astype(int))
    kv = np.round(mk * r.uniform(0.1, 1.0, n)).astype(int)
    q[0], kv[0] = mq, mk
    return q, np.maximum(q, kv)


def _frequencies(case):
    """Radians per position of each pair: base^(-2i/rot), the low frequencies stretched by
    `factor` (those of fewer than one turn over 4096 positions, blended up to 32 turns)."""
    f = case["base"] ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
    if case["factor"] == 1.0:
        return f
    keep = np.clip((f * 4096 / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
    return f * keep + f / case["factor"] * (1.0 - keep)


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0


def _turns(case):
    """The frequencies as 64-bit fractions of a turn per position, two's complement."""
    t = [int(round(float(f) / (2 * math.pi) * 2.0**64)) % (1 << 64) for f in _frequencies(case)]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in t], dtype=torch.int64)


def _randn(g, shape, dtype, mul=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return x.mul_(mul) if mul != 1.0 else x


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _cache(g, r, pages_of, page, hk, dim, dtype):
    """Key and value pages [pages][head][slot][dim], all slots holding something (stale values where
    nothing was written yet), and the table of each sequence's pages, in no order."""
    width = int(pages_of.max())
    total = int(pages_of.sum()) + 3
    order = r.permutation(total)
    table = np.zeros((len(pages_of), width), dtype=np.int32)
    at = 0
    for b, n in enumerate(pages_of):
        table[b, :n] = order[at:at + n]
        at += n
    k = _randn(g, (total, hk, page, dim), dtype)
    v = _randn(g, (total, hk, page, dim), dtype)
    return k, v, _i32(table)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.RandomState((seed * 7919 + 13) % (1 << 31))
    s = {"case": case, "seed": seed}
    dim = case["dim"]
    if case["kind"] == "attend":
        t = TYPES[case["type"]]
        q, kv = _lengths(case)
        k, v, table = _cache(g, r, -(-kv // case["page"]), case["page"], case["hk"], dim, t)
        ntok = int(q.sum())
        s.update(k=k, v=v, table=table, q_start=_i32(np.concatenate([[0], np.cumsum(q)])),
                 kv_len=_i32(kv), seq=_i32(np.repeat(np.arange(len(q)), q)),
                 pos=_i32(np.concatenate([np.arange(b - a, b) for a, b in zip(q, kv)])),
                 row=_i32(np.concatenate([np.arange(a) for a in q])),
                 Q=_randn(g, (ntok, case["hq"], dim), t, 2.0),
                 O=torch.empty((ntok, case["hq"], dim), dtype=t, device=DEV),
                 scratch=torch.empty(SCRATCH, dtype=torch.uint8, device=DEV),
                 max_q=int(q.max()), max_kv=int(kv.max()), scale=dim ** -0.5)
        return s
    tin, tout = TYPES[case["tin"]], TYPES[case["tout"]]
    hq, hk = case["hq"], case["hk"]
    s.update(turns=_turns(case).to(DEV), amp=_amplitude(case))
    if case["norm"]:
        s.update(wq=_randn(g, (dim,), torch.float32, 0.2) + 1.0,
                 wk=_randn(g, (dim,), torch.float32, 0.2) + 1.0)
    if case["kind"] == "qk":
        ntok = case["ntok"]
        X = _randn(g, (ntok, hq + hk, dim), tin, 1.7)
        start = r.randint(0, case["maxpos"] - ntok + 1)
        s.update(Xq=X[:, :hq], Xk=X[:, hq:], pos=_i32(np.arange(start, start + ntok)),
                 Yq=torch.empty((ntok, hq, dim), dtype=tout, device=DEV),
                 Yk=torch.empty((ntok, hk, dim), dtype=tout, device=DEV))
        return s
    q, kv = _lengths(case)
    # as many pages as the step touches, with a few that it does not
    first = (kv - q) // case["page"]
    k, v, short = _cache(g, r, -(-kv // case["page"]) - first, case["page"], hk, dim, tout)
    table = np.full((len(q), int((-(-kv // case["page"])).max())), 0, dtype=np.int32)
    short = short.cpu().numpy()
    for b in range(len(q)):
        n = -(-int(kv[b]) // case["page"]) - int(first[b])
        table[b, first[b]:first[b] + n] = short[b, :n]
    ntok = int(q.sum())
    X = _randn(g, (ntok, hq + 2 * hk, dim), tin, 1.7)
    s.update(Xq=X[:, :hq], Xk=X[:, hq:hq + hk], Xv=X[:, hq + hk:], k=k, v=v, table=_i32(table),
             seq=_i32(np.repeat(np.arange(len(q)), q)),
             pos=_i32(np.concatenate([np.arange(b - a, b) for a, b in zip(q, kv)])),
             Yq=torch.empty((ntok, hq, dim), dtype=tout, device=DEV))
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_norm_rope(x, w, s):
    """x [ntok][heads][dim] -> f32, normalised by head and rotated."""
    case = s["case"]
    rot, inter = case["rot"], case["inter"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    # the product wraps at 2^64, which drops whole turns
    turn = (s["pos"].long()[:, None] * s["turns"]).float() * 2.0**-64
    c = (torch.cos(turn * (2 * math.pi)) * s["amp"])[:, None]
    n = (torch.sin(turn * (2 * math.pi)) * s["amp"])[:, None]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    t, page = s["k"].dtype, s["case"]["page"]
    pos = s["pos"].long()
    at = s["table"].long()[s["seq"].long(), pos // page]
    s["k"][at, :, pos % page] = _plain_norm_rope(s["Xk"], s.get("wk"), s).to(t)
    s["v"][at, :, pos % page] = s["Xv"].to(t)
    return {"q": _plain_norm_rope(s["Xq"], s.get("wq"), s).to(t), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    case = s["case"]
    hk, dim, n = case["hk"], case["dim"], case["nseq"]
    group = case["hq"] // hk
    seq, row = s["seq"].long(), s["row"].long()
    mq = s["max_q"]
    keys = s["table"].shape[1] * case["page"]
    k = s["k"][s["table"].long()].transpose(1, 2).reshape(n, hk, keys, dim).float()
    v = s["v"][s["table"].long()].transpose(1, 2).reshape(n, hk, keys, dim).float()
    q = torch.zeros((n, mq, hk, group, dim), device=DEV)
    q[seq, row] = s["Q"].view(-1, hk, group, dim).float() * s["scale"]
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hk, mq * group, dim)
    w = torch.matmul(q, k.transpose(-1, -2)).view(n, hk, mq, group, keys)
    pos = torch.full((n, mq), -1, dtype=torch.long, device=DEV)
    pos[seq, row] = s["pos"].long()
    at = torch.arange(keys, device=DEV)
    seen = at <= pos[..., None]
    if case["window"]:
        seen &= at > pos[..., None] - case["window"]
    w.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(n, hk, mq * group, keys), v).view(n, hk, mq, group, dim)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4)[seq, row].reshape(-1, case["hq"], dim).to(s["Q"].dtype)


def run(s):
    kind = s["case"]["kind"]
    if own:
        import bit_matvec_gb300 as tq
        if kind == "attend":
            kv = s.get("kv") or s.setdefault("kv", tq.PagedKV(s["k"], s["v"], s["table"]))
            tq.tq_paged_attention(s["Q"], kv, s["q_start"], s["kv_len"], s["O"], s["max_q"],
                                  s["max_kv"], s["scale"], s["scratch"],
                                  window=s["case"]["window"])
            return s["O"]
        rope = s.get("rope") or s.setdefault("rope", tq.Rope(s["turns"], s["case"]["inter"],
                                                             s["amp"]))
        if kind == "qk":
            tq.tq_qk_norm_rope(s["Xq"], s["Xk"], s["Yq"], s["Yk"], s["pos"], rope, s.get("wq"),
                               s.get("wk"), EPS)
            return {"q": s["Yq"], "k": s["Yk"]}
        kv = s.get("kv") or s.setdefault("kv", tq.PagedKV(s["k"], s["v"], s["table"]))
        tq.tq_kv_append(s["Xq"], s["Xk"], s["Xv"], s["Yq"], kv, s["seq"], s["pos"], rope,
                        s.get("wq"), s.get("wk"), EPS)
        return {"q": s["Yq"], "k": s["k"], "v": s["v"]}
    if kind == "attend":
        return _plain_attend(s)
    if kind == "qk":
        t = s["Yq"].dtype
        return {"q": _plain_norm_rope(s["Xq"], s.get("wq"), s).to(t),
                "k": _plain_norm_rope(s["Xk"], s.get("wk"), s).to(t)}
    return _plain_append(s)


# ---------------------------------------------------------------- cost and truth

def _seen_pairs(q, kv, window):
    """Pairs of a new token and a key it sees, and keys that some new token sees."""
    pairs = keys = 0
    for a, b in zip(q.tolist(), kv.tolist()):
        p = np.arange(b - a, b, dtype=np.int64) + 1
        pairs += int(np.minimum(p, window).sum() if window else p.sum())
        keys += min(b, a + window - 1) if window else b
    return pairs, keys


def work(case):
    dim, hq, hk = case["dim"], case["hq"], case["hk"]
    if case["kind"] == "qk":
        n = case["ntok"] * (hq + hk) * dim
        return {"bytes": n * (SIZE[case["tin"]] + SIZE[case["tout"]]) + 4 * case["ntok"], "flops": 7 * n}
    q, kv = _lengths(case)
    ntok = int(q.sum())
    if case["kind"] == "append":
        n = ntok * (hq + 2 * hk) * dim
        return {"bytes": n * (SIZE[case["tin"]] + SIZE[case["tout"]]) + 8 * ntok, "flops": 7 * n}
    pairs, keys = _seen_pairs(q, kv, case["window"])
    return {"bytes": SIZE[case["type"]] * dim * (2 * keys * hk + 2 * ntok * hq),
            "flops": 4 * pairs * hq * dim}


def _exact_head(x, w, case, pos):
    """The definition for rows x [ntok][heads][dim], in 64 bits, from the frequencies themselves."""
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    f = torch.from_numpy(_frequencies(case)).to(DEV)
    z = _amplitude(case) * torch.exp(1j * (pos.double()[:, None] * f))[:, None, :]
    half = case["rot"] // 2
    first = torch.arange(half, device=DEV) * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)
    turned = torch.complex(x[..., first], x[..., second]) * z
    y = x.clone()
    y[..., first], y[..., second] = turned.real, turned.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "qk":
        return {n: _exact_head(s["X" + n], s.get("w" + n), case, s["pos"]) for n in ("q", "k")}
    if case["kind"] == "append":
        k, v = s["k"].double(), s["v"].double()
        newk = _exact_head(s["Xk"], s.get("wk"), case, s["pos"])
        pos = s["pos"].long()
        where = s["table"].long()[s["seq"].long(), torch.div(pos, case["page"], rounding_mode="floor")]
        slot = torch.remainder(pos, case["page"])
        for h in range(case["hk"]):
            k[where, h, slot] = newk[:, h]
            v[where, h, slot] = s["Xv"][:, h].double()
        return {"q": _exact_head(s["Xq"], s.get("wq"), case, s["pos"]), "k": k, "v": v}
    q, kv = _lengths(case)
    o = torch.zeros(s["Q"].shape, dtype=torch.float64, device=DEV)
    group, at = case["hq"] // case["hk"], 0
    for b in range(case["nseq"]):
        a, n = int(q[b]), int(kv[b])
        pages = s["table"][b, :-(-n // case["page"])].long()
        p = torch.arange(n - a, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hidden = (j > p) | ((j <= p - case["window"]) if case["window"] else torch.zeros_like(j > p))
        for h in range(case["hk"]):
            kk = s["k"][pages, h].reshape(-1, case["dim"])[:n].double()
            vv = s["v"][pages, h].reshape(-1, case["dim"])[:n].double()
            for g in range(group):
                z = s["Q"][at:at + a, h * group + g].double() @ kk.T / math.sqrt(case["dim"])
                z[hidden] = -math.inf
                o[at:at + a, h * group + g] = torch.softmax(z, -1) @ vv
        at += a
    return o
