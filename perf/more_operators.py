"""What differs from request to request in one batched step, as cases to be measured.

A serving program multiplies the activations of all its requests by one shared
ternary matrix (tq_quantize_matmul, which leaves f32 rows). Each request may
bring a fine-tune of that matrix, as a low-rank adapter beside it, and after
the last matrix its own way of drawing the next token. The two kinds of case:

  lora    tq_lora_add   Y[t] = Z[t] + scale B (A x[t]) with the adapter of each
                        token's request: from one token to a large prefill,
                        many adapters of several ranks at once, tokens in any
                        order, some without an adapter
  sample  tq_sample     the next token of each row of logits, with the row's own
                        temperature, top-k, top-p and min-p, from one given
                        uniform number a row, and the log of the probability
                        it was drawn with

run() computes the plain form in elementary torch operations, or, where `own`
is true, calls the library as a user does.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
SCRATCH = 1 << 20   # the one scratch buffer that a serving program keeps for its adapter calls


# ---------------------------------------------------------------- cases

def listed():
    """Smallest calls, ordinary ones and large ones of each operator, on the matrices of this
    repository's decode step (15360, 17408 and 5120 rows or columns)."""
    return [
        # one request's token beside the output projection
        dict(name="lora 1 token", kind="lora", ntok=1, cols=5120, rows=5120, adapters=4, rank=16,
             ragged=False, bare=0.0, sorted=True, x="f32", w="bf16", y="f32"),
        # a decode step of 48 requests of 32 fine-tunes, one in ten of the base model
        dict(name="lora 48 tokens", kind="lora", ntok=48, cols=5120, rows=17408, adapters=32,
             rank=16, ragged=True, bare=0.1, sorted=False, x="f32", w="bf16", y="f32"),
        # a large decode batch of many fine-tunes of higher rank
        dict(name="lora 256 tokens", kind="lora", ntok=256, cols=17408, rows=5120, adapters=100,
             rank=64, ragged=True, bare=0.0, sorted=False, x="f32", w="f16", y="f32"),
        # odd sizes, 16-bit activations, a mixed step of prompts and single tokens
        dict(name="lora 777 tokens", kind="lora", ntok=777, cols=4104, rows=5003, adapters=9,
             rank=20, ragged=True, bare=0.2, sorted=False, x="bf16", w="bf16", y="bf16"),
        # a prefill step of one fine-tune
        dict(name="lora 4096 tokens", kind="lora", ntok=4096, cols=5120, rows=15360, adapters=2,
             rank=64, ragged=False, bare=0.0, sorted=True, x="f32", w="bf16", y="f32"),
        # a large prefill step, prompts of several fine-tunes and of the base model
        dict(name="lora 8192 tokens", kind="lora", ntok=8192, cols=5120, rows=17408, adapters=16,
             rank=32, ragged=True, bare=0.1, sorted=True, x="f32", w="bf16", y="f32"),
        # one request's next token, the usual filters together
        dict(name="sample 1 row", kind="sample", ntok=1, vocab=131072, mode="all", spread=2.5,
             masked=0.0, type="f32", pad=0),
        # few requests, 16-bit logits of an odd vocabulary in padded rows, nucleus only
        dict(name="sample 7 rows", kind="sample", ntok=7, vocab=50021, mode="top_p", spread=3.0,
             masked=0.0, type="bf16", pad=3),
        # a batch in which every request has settings of its own
        dict(name="sample 64 rows", kind="sample", ntok=64, vocab=131072, mode="mixed", spread=2.5,
             masked=0.0, type="f32", pad=0),
        # many requests on a small vocabulary, a fifth of it forbidden by a grammar
        dict(name="sample 512 rows", kind="sample", ntok=512, vocab=32768, mode="mixed", spread=3.0,
             masked=0.2, type="f32", pad=0),
        # many requests, half precision, the most likely tokens only
        dict(name="sample 200 rows", kind="sample", ntok=200, vocab=128001, mode="top_k", spread=2.0,
             masked=0.0, type="f16", pad=7),
        # the largest batch and vocabulary, drawn from all of it: samples for training on
        dict(name="sample 256 rows", kind="sample", ntok=256, vocab=262144, mode="plain", spread=2.5,
             masked=0.0, type="f32", pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        x, w = rng.choice((("f32", "bf16"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"),
                           ("f16", "f16")))
        cols, rows = 8 * _log(rng, 32, 2176), _log(rng, 256, 17408)
        case = dict(kind="lora", ntok=_log(rng, 1, min(8192, (1 << 28) // (cols + 2 * rows))),
                    cols=cols, rows=rows, rank=_log(rng, 1, 128),
                    ragged=rng.random() < 0.6, bare=rng.choice((0.0, 0.0, 0.1, 0.5)),
                    sorted=rng.random() < 0.5, x=x, w=w,
                    y=rng.choice(("f32", "f32", w)))
        # at most 2^13 rows of A in all, and fewer where tokens are many
        most = max(1, min(256, (1 << 13) // case["rank"], (1 << 22) // (case["ntok"] * case["rank"])))
        case["adapters"] = _log(rng, 1, most)
        return case
    ntok = _log(rng, 1, 512)
    return dict(kind="sample", ntok=ntok, vocab=_log(rng, 1000, min(262144, (1 << 26) // ntok)),
                mode=rng.choice(("plain", "greedy", "top_k", "top_p", "min_p", "all", "mixed", "mixed")),
                spread=rng.choice((1.0, 2.0, 3.0, 4.0)), masked=rng.choice((0.0, 0.0, 0.3, 0.9)),
                type=rng.choice(("f32", "f32", "bf16", "f16")), pad=rng.choice((0, 0, 1, 5, 8)))


# ---------------------------------------------------------------- inputs

def _ids(case):
    """The adapter of each token (-1: none) and the rank of each adapter, the same for every
    seed."""
    n, count = case["ntok"], case["adapters"]
    r = np.random.RandomState(7001 * n + 31 * count + case["rank"])
    ids = r.randint(0, count, n)
    ids[r.uniform(size=n) < case["bare"]] = -1
    if case["sorted"]:
        ids.sort()
    top = case["rank"]
    rank = r.choice([max(1, top // 4), max(1, top // 2), top], count) if case["ragged"] else np.full(count, top)
    return ids, rank


def _randn(g, shape, dtype, mul=1.0):
    x = torch.randn(shape, generator=g, device=DEV)
    return x.mul_(mul).to(dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _settings(case, seed):
    """temperature, top_k, top_p, min_p of each row; 1, 0, 1, 0 where a filter is off."""
    n, mode = case["ntok"], case["mode"]
    r = np.random.RandomState((seed * 7919 + 101) % (1 << 31))
    t = r.uniform(0.6, 1.3, n).astype(np.float32)
    k = np.minimum(case["vocab"], np.exp(r.uniform(np.log(5), np.log(300), n)).astype(np.int32))
    p = r.uniform(0.5, 0.99, n).astype(np.float32)
    m = np.exp(r.uniform(np.log(0.002), np.log(0.2), n)).astype(np.float32)
    what = r.randint(0, 6, n) if mode == "mixed" else np.full(
        n, ("plain", "greedy", "top_k", "top_p", "min_p", "all").index(mode))
    t[what == 1] = 0.0
    k[(what != 2) & (what != 5)] = 0
    p[(what != 3) & (what != 5)] = 1.0
    m[(what != 4) & (what != 5)] = 0.0
    return t, k, p, m


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case, "seed": seed}
    n = case["ntok"]
    if case["kind"] == "lora":
        ids, rank = _ids(case)
        w, count, top = TYPES[case["w"]], case["adapters"], case["rank"]
        r = np.random.RandomState((seed * 6007 + 17) % (1 << 31))
        s.update(ids=_i32(ids), rank=_i32(rank),
                 scale=torch.from_numpy(r.uniform(0.25, 2.0, count).astype(np.float32)).to(DEV),
                 a=_randn(g, (count, top, case["cols"]), w, case["cols"] ** -0.5),
                 b=_randn(g, (count, case["rows"], top), w, top ** -0.5),
                 X=_randn(g, (n, case["cols"]), TYPES[case["x"]]),
                 Z=_randn(g, (n, case["rows"]), TYPES[case["y"]]),
                 Y=torch.empty((n, case["rows"]), dtype=TYPES[case["y"]], device=DEV),
                 scratch=torch.empty(SCRATCH, dtype=torch.uint8, device=DEV))
        return s
    vocab = case["vocab"]
    # a bell with a heavy upper end: a few tokens that the context asks for
    x = torch.randn((n, vocab + case["pad"]), generator=g, device=DEV).mul_(case["spread"])
    likely = torch.randint(0, vocab, (n, 40), generator=g, device=DEV)
    more = torch.empty((n, 40), device=DEV).exponential_(0.25, generator=g)
    x.scatter_add_(1, likely, more + case["spread"])
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < case["masked"], -math.inf)
    t, k, p, m = _settings(case, seed)
    s.update(logits=x.to(TYPES[case["type"]])[:, :vocab],
             u=torch.rand(n, generator=g, device=DEV),
             temperature=torch.from_numpy(t).to(DEV), top_k=_i32(k), top_p=torch.from_numpy(p).to(DEV),
             min_p=torch.from_numpy(m).to(DEV), tokens=torch.empty(n, dtype=torch.int32, device=DEV),
             logp=torch.empty(n, device=DEV))
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_lora(s):
    """Every token against every adapter, those of others masked out between the two products."""
    count, top, cols = s["a"].shape
    h = torch.matmul(s["X"].float(), s["a"].reshape(count * top, cols).float().T)
    mine = s["ids"][:, None] == torch.arange(count, device=DEV)
    used = torch.arange(top, device=DEV) < s["rank"][:, None]
    h = h.view(-1, count, top) * s["scale"][:, None]
    h = torch.where(mine[:, :, None] & used, h, torch.zeros_like(h))
    b = s["b"].permute(0, 2, 1).reshape(count * top, -1).float()
    return (s["Z"].float() + torch.matmul(h.view(-1, count * top), b)).to(s["Y"].dtype)


def _plain_sample(s):
    """Weights and their sums in 64 bits: the draw and the nucleus compare sums with borders that
    lie as near as one weight of a quarter million."""
    x = s["logits"].float()
    vocab = x.shape[1]
    top = x.amax(1, keepdim=True)
    cold = s["temperature"][:, None] == 0
    t = torch.where(cold, torch.ones_like(top), s["temperature"][:, None]).double()
    w = torch.exp((x.double() - top.double()) / t)
    # equal logits in the order of their indexes; the filters keep a beginning of this order
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ordered = torch.gather(w, 1, order)
    place = torch.arange(vocab, device=DEV)
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], vocab))[:, None]
    ordered = torch.where(place < k, ordered, torch.zeros_like(ordered))
    before = torch.cumsum(ordered, 1) - ordered
    p = torch.where(s["top_p"] < 1, s["top_p"], torch.full_like(s["top_p"], 2.0))[:, None].double()
    keep = (place < k) & (before < p * ordered.sum(1, keepdim=True)) & (ordered >= s["min_p"][:, None].double())
    keep[:, 0] = True
    kept = torch.where(torch.zeros_like(keep).scatter(1, order, keep), w, torch.zeros_like(w))
    total = kept.sum(1, keepdim=True)
    passed = (torch.cumsum(kept, 1) <= s["u"][:, None].double() * total).sum(1, keepdim=True)
    token = torch.where(cold, order[:, :1], passed.clamp(max=vocab - 1))
    logp = torch.log(torch.gather(w, 1, token) / total)
    return {"tokens": token[:, 0].int(),
            "logp": torch.where(cold, torch.zeros_like(logp), logp)[:, 0].float()}


def run(s):
    if own:
        import bit_matvec_gb300 as tq
        if s["case"]["kind"] == "lora":
            lora = s.get("lora") or s.setdefault("lora", tq.Lora(s["a"], s["b"], s["rank"], s["scale"]))
            tq.tq_lora_add(s["X"], lora, s["ids"], s["Y"], s["Z"], s["scratch"])
            return s["Y"]
        tq.tq_sample(s["logits"], s["u"], s["tokens"], s["temperature"], s["top_k"], s["top_p"],
                     s["min_p"], s["logp"])
        return {"tokens": s["tokens"], "logp": s["logp"]}
    if s["case"]["kind"] == "lora":
        return _plain_lora(s)
    return _plain_sample(s)


# ---------------------------------------------------------------- cost and truth

def work(case):
    n = case["ntok"]
    if case["kind"] == "sample":
        return {"bytes": n * case["vocab"] * SIZE[case["type"]] + 28 * n, "flops": 4 * n * case["vocab"]}
    ids, rank = _ids(case)
    wide = case["cols"] + case["rows"]
    here = ids[ids >= 0]
    weights = int(rank[np.unique(here)].sum()) * wide * SIZE[case["w"]]
    return {"bytes": weights + len(here) * case["cols"] * SIZE[case["x"]] +
            2 * n * case["rows"] * SIZE[case["y"]] + 4 * n,
            "flops": 2 * int(rank[here].sum()) * wide}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "lora":
        ids, rank = _ids(case)
        y = s["Z"].double()
        for i in np.unique(ids[ids >= 0]):
            at, r = torch.from_numpy(np.nonzero(ids == i)[0]).to(DEV), int(rank[i])
            delta = s["b"][i, :, :r].double() @ (s["a"][i, :r].double() @ s["X"][at].double().T)
            y[at] += float(s["scale"][i]) * delta.T
        return y
    t, k, p, m = _settings(case, seed)
    logp = np.zeros(case["ntok"])
    u = s["u"].double().cpu().numpy()
    for i in range(case["ntok"]):
        if t[i] == 0:
            continue
        # the row's tokens from the most likely on, in logarithms
        z = s["logits"][i].double() / float(t[i])
        z, where = torch.sort(z, descending=True, stable=True)
        if k[i] > 0:
            z, where = z[:int(k[i])], where[:int(k[i])]
        z = z - torch.logsumexp(z, 0)
        n = len(z)
        if p[i] < 1:
            n = int((torch.cumsum(z.exp(), 0) < float(p[i])).sum()) + 1
        if m[i] > 0:
            n = min(n, max(1, int((z - z[0] >= math.log(float(m[i]))).sum())))
        z, where = z[:n] - torch.logsumexp(z[:n], 0), where[:n]
        by_index = torch.argsort(where)
        at = int((torch.cumsum(z[by_index].exp(), 0) <= u[i]).sum())
        logp[i] = float(z[by_index][min(at, n - 1)])
    return {"tokens": None, "logp": torch.from_numpy(logp).to(DEV)}
