"""Norm and rotation of many heads on the GPU, where a group of lanes takes up to eight heads of a token
(from 24,576 heads on), against the 64-bit form: types, widths, heads that eight do not divide, in
place, padding, and just below and above the border."""
import pytest
import torch

from attn_util import assert_within, frequencies, norm_rope
from test_gpu_rope import BF16, F16, F32, make_cache, rope_of

pytestmark = pytest.mark.gpu
BORDER = 24576


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


# ntok, q heads, k heads, dim, rot, interleaved, norm, in, out
CASES = [(1900, 9, 4, 128, 128, False, True, tin, tout) for tin in (F32, F16, BF16) for tout in (F32, F16, BF16)]
CASES += [
    (4100, 5, 1, 64, 32, True, True, F32, BF16),      # 8 lanes a head; 5 and 1 heads
    (4100, 5, 1, 64, 64, False, False, BF16, F16),
    (1500, 15, 2, 256, 128, False, True, F16, F32),   # 32 lanes a head
    (1500, 1, 16, 200, 200, True, True, BF16, BF16),  # lanes past the head
    (631, 40, 8, 80, 40, True, True, F32, F16),
    (600, 41, 0, 96, 64, False, True, F16, BF16),     # queries only, six batches and one head
    (3100, 0, 8, 128, 0, False, True, F32, BF16),     # keys only, no rotation
    (BORDER // 12, 8, 4, 128, 64, False, True, F32, BF16), (BORDER // 12 - 1, 8, 4, 128, 64, False, True, F32, BF16),
    (2731, 8, 1, 64, 64, False, True, BF16, BF16), (2730, 8, 1, 64, 64, False, True, BF16, BF16),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope(tq, case):
    ntok, hq, hk, dim, rot, inter, norm, tin, tout = case
    g = torch.Generator().manual_seed(ntok + dim)
    X = (torch.randn(ntok, hq + hk, dim, generator=g) * 3).to(tin)
    pos = torch.randint(0, 200000, (ntok,), generator=g, dtype=torch.int32)
    wq, wk = ((torch.randn(dim, generator=g) * 0.3 + 1) for _ in range(2)) if norm else (None, None)
    Xd = X.cuda()
    Yq = torch.full((ntok, hq, dim), float("nan"), dtype=tout, device="cuda")
    Yk = torch.full((ntok, hk, dim), float("nan"), dtype=tout, device="cuda")
    wqd, wkd = (None if w is None else w.cuda() for w in (wq, wk))
    if hq:
        tq.tq_qk_norm_rope(Xd[:, :hq], Xd[:, hq:] if hk else None, Yq, Yk if hk else None, pos.cuda(),
                           rope_of(tq, rot, inter, 1.25), wqd, wkd, 1e-5)
    else:
        tq.tq_qk_norm_rope(Xd, None, Yk, None, pos.cuda(), rope_of(tq, rot, inter, 1.25), wkd, None, 1e-5)
    for x, y, w in ((X[:, :hq], Yq, wq), (X[:, hq:], Yk, wk)):
        if y.numel():
            want, bound = norm_rope(x, w, 1e-5, frequencies(rot), inter, 1.25, pos, tout)
            assert_within(y, want, bound, "y")


@pytest.mark.parametrize("hq,hk,dtype", [(9, 4, F32), (40, 8, BF16), (3, 17, F16)])
def test_in_place(tq, hq, hk, dtype):
    """Over the inputs, in one wide buffer: the bits of a call with outputs of its own."""
    ntok, dim = BORDER // (hq + hk) + 1, 128
    X = torch.randn(ntok, hq + hk, dim, device="cuda").to(dtype)
    w, pos = torch.rand(dim, device="cuda") + 0.5, torch.arange(ntok, dtype=torch.int32, device="cuda")
    rope = rope_of(tq, dim, False)
    Y = torch.empty_like(X)
    tq.tq_qk_norm_rope(X[:, :hq], X[:, hq:], Y[:, :hq], Y[:, hq:], pos, rope, w, w)
    wide = torch.full((ntok, (hq + hk) * dim + 8), 7.0, device="cuda", dtype=dtype)
    Z = torch.as_strided(wide, (ntok, hq + hk, dim), ((hq + hk) * dim + 8, dim, 1))
    Z.copy_(X)
    tq.tq_qk_norm_rope(Z[:, :hq], Z[:, hq:], Z[:, :hq], Z[:, hq:], pos, rope, w, w)
    assert torch.equal(Z, Y)
    assert (wide[:, (hq + hk) * dim:] == 7).all()


@pytest.mark.parametrize("tin,tc,order", [(F32, BF16, "hnd"), (F32, F16, "nhd"), (BF16, BF16, "both"),
                                          (F16, F16, "nhd"), (BF16, F16, "hnd"), (F16, BF16, "hnd")])
@pytest.mark.parametrize("hq,hk,dim,rot,inter,page", [(9, 5, 128, 128, False, 16), (0, 12, 64, 32, True, 48),
                                                      (40, 8, 96, 96, False, 64)])
def test_append(tq, hq, hk, dim, rot, inter, page, tin, tc, order):
    """Ragged chunks with padding tokens among the others; slots that are not the call's stay."""
    g = torch.Generator().manual_seed(hq * dim + page)
    total = BORDER // (hq + 2 * hk) + 9
    new = [total // 2, 1, total - total // 2 - 1]
    kv = [new[0], new[1] + 70, new[2] + 33]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g)
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    seq = torch.cat([torch.full((q,), b, dtype=torch.int32) for b, q in enumerate(new)])
    pos = torch.cat([torch.arange(n - q, n, dtype=torch.int32) for n, q in zip(kv, new)])
    pad = torch.rand(total, generator=g) < 0.05
    pos[pad], seq[pad] = -1, 10**6
    X = (torch.randn(total, hq + 2 * hk, dim, generator=g) * 2).to(tin)
    wq, wk = torch.randn(dim, generator=g) * 0.3 + 1, torch.randn(dim, generator=g) * 0.3 + 1
    k, v = make_cache(order, pages, hk, page, dim, tc)
    Yq = torch.full((total, hq, dim), -55.0, dtype=tc, device="cuda") if hq else None
    Xd = X.cuda()
    tq.tq_kv_append(Xd[:, :hq] if hq else None, Xd[:, hq:hq + hk], Xd[:, hq + hk:], Yq,
                    tq.PagedKV(k, v, table.cuda()), seq.cuda(), pos.cuda(), rope_of(tq, rot, inter), wq.cuda(),
                    wk.cuda(), 1e-6)
    real = ~pad
    if hq:
        want, bound = norm_rope(X[real][:, :hq], wq, 1e-6, frequencies(rot), inter, 1.0, pos[real], tc)
        Yq = Yq.cpu()
        assert_within(Yq[real], want, bound, "q")
        assert (Yq[pad] == -55).all()
    wantk, boundk = norm_rope(X[real][:, hq:hq + hk], wk, 1e-6, frequencies(rot), inter, 1.0, pos[real], tc)
    where = table[seq[real].long(), pos[real].long() // page].long()
    slot = pos[real].long() % page
    k, v = k.cpu().transpose(1, 2), v.cpu().transpose(1, 2)     # [pages][page][heads][dim]
    assert_within(k[where, slot], wantk, boundk, "k")
    assert torch.equal(v[where, slot], X[real][:, hq + hk:].to(tc))
    other = torch.ones(pages, page, dtype=torch.bool)
    other[where, slot] = False
    assert (k[other] == -77).all() and (v[other] == -77).all()
