"""Plain 64-bit forms of the norm/rotation, append and attention operators, with the error bounds
of the 32-bit ones, on the CPU."""
import math

import torch

U = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}   # half an ulp of 1
TINY = {torch.float32: 1e-40, torch.float16: 2.0**-25, torch.bfloat16: 1e-40}


def frequencies(rot, base=1e4):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else torch.zeros(0).double()


def norm_rope(x, w, eps, freq, inter, amplitude, pos, out):
    """(value, bound) in 64 bits for x [tokens][heads][dim] and an output of type `out`.

    The bound: a norm's sum of dim squares in 32 bits (16 roundings on the longest path of the
    lanes' sums, halved by the root), root, quotient, two products, the angle (2^-25 of a turn),
    sine and cosine (2 ulp), amplitude, two products and a sum: under 40 roundings of 2^-24, on
    |a| + |b|; then the output's own rounding."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs()
    half = freq.numel()
    if half:
        first = torch.arange(half) * (2 if inter else 1)
        second = first + (1 if inter else half)
        ang = pos.double()[:, None] * freq
        c, s = (amplitude * torch.cos(ang))[:, None], (amplitude * torch.sin(ang))[:, None]
        a, b = x[..., first], x[..., second]
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        both = (a.abs() + b.abs()) * abs(amplitude)
        mag = mag.clone()
        mag[..., first], mag[..., second] = both, both
    return y, 40 * 2.0**-24 * mag + U[out] * y.abs() + TINY[out]


def gather(cache, table, n):
    """Keys 0 .. n-1 of one sequence: [heads][n][dim] in 64 bits."""
    page = cache.shape[2]
    pages = table[:-(-n // page)].long()
    pages = torch.where(pages < cache.shape[0], pages, 0)   # pages no token sees may be anything
    return cache[pages].transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n].double()


def attention(q, k, v, table, q_start, kv_len, scale, window, out):
    """(o, lse, bound of o, bound of lse) in 64 bits, all on the CPU.

    With weights p_j = exp(s_j - max): each is off by the 32-bit score's error (dim + 2 roundings
    of scale sum |q||k|, doubled for the chain's arithmetic), the exponential's (2^-21), and its
    rounding to the cache's type (and, in f16, 2^-25 where it is subnormal); the sums of n products
    by n roundings."""
    heads, dim = k.shape[1], k.shape[3]
    group = q.shape[1] // heads
    o = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(kv_len)):
        at, end, n = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if end == at:
            continue
        pos = torch.arange(n - (end - at), n)
        if n == 0:
            continue
        kk, vv = gather(k, table[b], n), gather(v, table[b], n)
        j = torch.arange(n)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(heads):
            qq = q[at:end, h * group:(h + 1) * group].double()          # [rows][group][dim]
            keys, vals = kk[h], vv[h]
            used = seen.any(0)
            keys, vals = torch.where(used[:, None], keys, 0.0), torch.where(used[:, None], vals, 0.0)
            s = torch.einsum("rgd,nd->rgn", qq, keys) * scale
            sa = torch.einsum("rgd,nd->rgn", qq.abs(), keys.abs()) * abs(scale)
            s = s.masked_fill(~seen[:, None], -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(top == -math.inf, 0.0, top)) * seen[:, None]
            total = p.sum(-1, keepdim=True)
            safe = torch.where(total == 0, 1.0, total)
            oo = torch.einsum("rgn,nd->rgd", p, vals) / safe
            mass = torch.einsum("rgn,nd->rgd", p, vals.abs()) / safe
            sub = vals.abs().sum(0) * 2.0**-25 / safe
            score = (sa * seen[:, None]).amax(-1, keepdim=True)
            rel = (dim + 2) * 2.0**-23 * score + 2.0**-20 + n * 2.0**-23
            o[at:end, h * group:(h + 1) * group] = oo
            lse[at:end, h * group:(h + 1) * group] = (top + torch.log(total))[..., 0]
            tol[at:end, h * group:(h + 1) * group] = mass * (2 * rel + U[k.dtype]) + sub + \
                U[out] * oo.abs() + TINY[out]
            tol_lse[at:end, h * group:(h + 1) * group] = (rel + 2.0**-22 * (1 + lse[at:end, h * group:(h + 1) * group, None].abs().nan_to_num(posinf=0.0)))[..., 0]
    return o, lse, tol, tol_lse


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} not finite"
    off = (got - want).abs() > bound
    if off.any():
        at = tuple(int(i) for i in off.nonzero()[0])
        raise AssertionError(f"{what}: {int(off.sum())} of {off.numel()} outside, first {at}: got "
                             f"{float(got[at])}, want {float(want[at])} +- {float(bound[at])}")
