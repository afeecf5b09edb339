"""Paged attention on the GPU where its inputs are not what they should be, or at the edges of what a
type holds. max_kv only plans: 1 takes the kernel for few rows, 10^8 that for many."""
import pytest
import torch

from attn_util import U, assert_within, attention, gather
from test_gpu_attention import BF16, BOTH, F16, F32, call, many_rows, problem

pytestmark = pytest.mark.gpu
BOTH_KERNELS = pytest.mark.parametrize("max_kv", [1, 10**8])


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


def call_fenced(tq, prob, max_kv, max_q=None, fence=4096):
    """call() with O, lse and the workspace inside wider buffers; whether what is beside them stayed."""
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    ntok, hq, dim = Q.shape
    mq = max_q if max_q is not None else int((q_start[1:] - q_start[:-1]).max())
    need = tq.tq_paged_attention_workspace_bytes(len(kv_len), ntok, hq, k.shape[1], dim, mq, max_kv)

    def fenced(n, dtype, fill):
        whole = torch.full((n + 2 * fence,), fill, dtype=dtype, device="cuda")
        return whole, whole[fence:fence + n]

    o, O = fenced(ntok * hq * dim, F32, -3.0)
    lse, L = fenced(ntok * hq, F32, -3.0)
    ws, W = fenced(max(need, 16), torch.uint8, 0xA5)
    O = O.view(ntok, hq, dim)
    tq.tq_paged_attention(Q.cuda(), tq.PagedKV(kd, vd, table.cuda()), q_start.cuda(), kv_len.cuda(), O,
                          mq, max_kv, dim ** -0.5, W, 0, L)
    kept = all(bool((x[:fence] == f).all() and (x[-fence:] == f).all())
               for x, f in ((o, -3.0), (lse, -3.0), (ws, 0xA5)))
    return O, L, kept


@BOTH_KERNELS
@pytest.mark.parametrize("starts", [[0, 90, 40, 130], [-1, 60, 100, 130], [0, 60, 100, 131], [0, 0, -5, 130],
                                    [130, 100, 60, 0], [0, 2**31 - 1, 60, 130]])
def test_starts_out_of_order_are_reported(tq, starts, max_kv):
    """A q_start that decreases or leaves the call's tokens is said so, and nothing beside the outputs
    and the workspace is written; the next call is right."""
    prob = list(problem([(200, n) for n in (50, 40, 40)], 8, 2, 64, 16, F16))
    want, _ = call(tq, tuple(prob), F32, max_kv=max_kv)
    good = prob[4]
    prob[4] = torch.tensor(starts, dtype=torch.int64).to(torch.int32)
    _, _, kept = call_fenced(tq, prob, max_kv, max_q=130)
    assert tq.tq_device_status() == tq.TQ_ERR_INDEX
    assert kept
    prob[4] = good
    again, L, kept = call_fenced(tq, prob, max_kv)
    assert kept and torch.equal(want, again)
    assert tq.tq_device_status() == tq.TQ_OK


def test_more_row_tiles_than_19_bits_count(tq):
    """A token of each of 530,000 sequences, 200 query heads to a key/value head: with one position
    each, a row is the value at that position, whatever the query."""
    nseq, hq, dim = 530000, 200, 8
    v = torch.randn(64, 1, 8, dim, device="cuda", dtype=F16)
    table = torch.randint(0, 64, (nseq, 1), device="cuda", dtype=torch.int32)
    Q = torch.randn(nseq, hq, dim, device="cuda", dtype=F16)
    O = torch.full_like(Q, float("nan"))
    need = tq.tq_paged_attention_workspace_bytes(nseq, nseq, hq, 1, dim, 1, 1)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    tq.tq_paged_attention(Q, tq.PagedKV(torch.randn_like(v), v, table),
                          torch.arange(nseq + 1, device="cuda", dtype=torch.int32),
                          torch.ones(nseq, device="cuda", dtype=torch.int32), O, 1, 1, 0.3, ws)
    assert need == 2 * 152 * 256 * (dim + 1) * 4 + 152 * 32      # the kernel for many rows
    want = v[table[:, 0].long(), 0, 0]
    assert tq.tq_device_status() == tq.TQ_OK
    assert torch.equal(O, want[:, None].expand_as(O))


@pytest.mark.parametrize("lens,hq,hk", [([(5000, 1)], 8, 1), ([(900, 5)] * 3, 8, 2), ([(900, 300), (40, 40)], 8, 2)])
def test_windows_as_long_as_any_sequence(tq, lens, hq, hk):
    prob = problem(lens, hq, hk, 64, 16, BF16)
    want, want_lse = call(tq, prob, F32)
    for window in (1 << 30, (1 << 31) - 1, (1 << 63) - 1):
        got, lse = call(tq, prob, F32, window)
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


# a few rows: one block, a cluster, ranges joined through the workspace, rows of several fragments; many
# rows: whole row tiles, alternate key tiles, cut row tiles
PLANS = [([(60, 1)], 4, 4, 1), ([(2000, 1)], 8, 8, None), ([(20000, 1)], 2, 1, None), ([(900, 9)] * 40, 8, 2, 1),
         ([(900, 260), (300, 20)], 4, 1, 10**8), ([(3000, 100)], 2, 2, 10**8), ([(700, 600)] * 6, 8, 8, 10**8)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_queries_that_are_not_finite_are_not_hidden(tq, plan, dtype, bad):
    """A NaN in a query is NaN in its row and its lse, an infinity too (it makes scores of both signs),
    however the keys are split; the other rows are what they were, but for roundings."""
    lens, hq, hk, max_kv = plan
    prob = list(problem(lens, hq, hk, 64, 16, dtype))
    Q, k, v, table, q_start, kv_len, _, _ = prob
    o, want_lse, tol, tol_lse = attention(Q, k, v, table, q_start, kv_len, 64 ** -0.5, 0, F32)
    g = torch.Generator().manual_seed(3)
    Q = prob[0] = prob[0].clone()
    hit = torch.zeros(Q.shape[:2], dtype=torch.bool)
    for _ in range(max(1, hit.numel() // 20)):
        hit.view(-1)[torch.randint(0, hit.numel(), (1,), generator=g)] = True
    # not the first positions, whose few scores may all have one sign
    pos = torch.cat([torch.arange(n - q, n) for n, q in lens])
    hit &= (pos >= 40)[:, None]
    assert hit.any()
    Q[..., 7][hit] = bad
    got, lse = call(tq, tuple(prob), F32, max_kv=max_kv)
    got, lse = got.cpu(), lse.cpu()
    assert torch.isnan(got[hit]).all()
    assert torch.isnan(lse[hit]).all()
    assert_within(got[~hit], o[~hit], tol[~hit], "o")
    assert_within(lse[~hit], want_lse[~hit], tol_lse[~hit], "lse")


@pytest.mark.parametrize("above", [8, 14, 16, 18, 20])
@pytest.mark.parametrize("every", [128, 20000])
@pytest.mark.parametrize("new,max_kv", [(1, None), (1, 1), (20, 1), (200, 10**8)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_small_weights_beside_a_large_one(tq, dtype, new, max_kv, every, above):
    """One key `above` the others in its score, with a value of zero, and 20,000 others: what comes out
    is the others' part alone, which an f16 weight below 2^-25 would not have. With one such key every
    128, whatever share of the keys a block takes has one.

    The bound is that of the 64-bit form with a weight's subnormal rounding at 2^-32 of the largest
    weight's instead of 2^-25: f16 weights are kept 2^7 or more above one."""
    n, dim = 20000, 64
    Q, k, v, table, q_start, kv_len, _, _ = problem([(n, new)], 2, 1, dim, 16, dtype, poison=False)
    Q = torch.ones_like(Q)
    k *= 0.05
    v = (v * 0.1 + 1).to(dtype)
    for j in range(0, n, every):
        k[table[0, j // 16], 0, j % 16] = above / dim ** 0.5   # times dim and the scale dim^-1/2: above
        v[table[0, j // 16], 0, j % 16] = 0
    # o in 64 bits; roundings as in attention(): scores, exponentials and sums in 32 bits, weights in dtype
    kk, vv = gather(k, table[0], n)[0], gather(v, table[0], n)[0]
    score = torch.einsum("rhd,nd->rhn", Q.double(), kk) * dim ** -0.5
    size = torch.einsum("rhd,nd->rhn", Q.double().abs(), kk.abs()).amax(-1, keepdim=True) * dim ** -0.5
    seen = torch.arange(n)[None] <= torch.arange(n - new, n)[:, None]
    p = torch.exp(score - score.amax(-1, keepdim=True)) * seen[:, None]
    total = p.sum(-1, keepdim=True)
    want, mass = p @ vv / total, p @ vv.abs() / total
    rel = (dim + 2) * 2.0**-23 * size + 2.0**-20 + n * 2.0**-23
    bound = mass * (2 * rel + U[dtype]) + vv.abs().sum(0) * 2.0**-32 / total
    O, _ = call(tq, (Q, k, v, table, q_start, kv_len, k.cuda(), v.cuda()), F32, max_kv=max_kv)
    assert_within(O, want, bound, "o")


THREADS = """
import ctypes, threading, torch
import bit_matvec_gb300 as tq
lib = tq.library()
dev = dict(device="cuda")
k, v = (torch.randn(8, 2, 16, 64, **dev).half() for _ in range(2))
table = torch.arange(8, dtype=torch.int32, **dev)[None]
kv = tq.PagedKV(k, v, table)
q = torch.randn(1, 4, 64, **dev).half()
starts, lens = torch.tensor([0, 1], dtype=torch.int32, **dev), torch.tensor([100], dtype=torch.int32, **dev)
out = [torch.zeros(1, 4, 64, **dev) for _ in range(8)]
streams = [torch.cuda.Stream() for _ in out]
need = tq.tq_paged_attention_workspace_bytes(1, 1, 4, 2, 64, 1, 100)
ws = [torch.empty(max(need, 16), dtype=torch.uint8, **dev) for _ in out]
torch.cuda.synchronize()
gate, codes = threading.Barrier(len(out)), [None] * len(out)
def first_call(i):
    gate.wait()     # ctypes lets go of the interpreter's lock: the calls do run side by side
    codes[i] = lib.tq_paged_attention(q.data_ptr(), 256, kv.ref, starts.data_ptr(), lens.data_ptr(),
                                      out[i].data_ptr(), 256, tq.TQ_F32, None, 1, 4, 1, 100, 0.125, 0,
                                      ws[i].data_ptr(), need, streams[i].cuda_stream)
threads = [threading.Thread(target=first_call, args=(i,)) for i in range(len(out))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert codes == [tq.TQ_OK] * len(out), codes
assert all(torch.equal(o, out[0]) for o in out) and out[0].abs().max() > 0
assert tq.tq_device_status() == tq.TQ_OK
"""


def test_first_calls_of_several_host_threads(tq):
    """A fresh process whose first attention calls come from eight threads at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(2):
        subprocess.run([sys.executable, "-c", THREADS], cwd=root, check=True, timeout=300)


@pytest.mark.parametrize("max_kv", [100, 10**8])
def test_first_cuda_call_of_a_host_thread(tq, max_kv):
    """A thread that never made a CUDA call, on tensors of another one: both kernels."""
    import threading
    prob = problem([(100, 70)], 4, 2, 64, 16, F16)
    want, want_lse = call(tq, prob, F32, max_kv=max_kv)
    Q, k, v, table, q_start, kv_len, kd, vd = prob
    need = tq.tq_paged_attention_workspace_bytes(1, 70, 4, 2, 64, 70, max_kv)
    args = (Q.cuda(), tq.PagedKV(kd, vd, table.cuda()), q_start.cuda(), kv_len.cuda())
    O, L = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    stream, errors = torch.cuda.current_stream(), []
    torch.cuda.synchronize()

    def work():
        try:
            tq.tq_paged_attention(*args, O, 70, max_kv, 64 ** -0.5, ws, 0, L, stream=stream)
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(O, want) and torch.equal(L, want_lse)


@pytest.mark.parametrize("nseq,max_kv", [(1, 1), (5, 1), (1, 10**8), (5, 10**8), (60, 10**8)])
def test_no_new_tokens_in_any_sequence(tq, nseq, max_kv):
    """Tokens of no sequence beside sequences of no new tokens: nothing is written, nothing reported."""
    prob = list(problem([(20 * b, 0) for b in range(nseq)], 16, 1, 64, 16, F16))
    prob[0] = torch.randn(300, 16, 64).to(F16)
    assert many_rows(tq, prob[:4] + [torch.tensor([0, 300])] + prob[5:], max_kv) == (max_kv > 1)
    O, L = call(tq, tuple(prob), F32, max_q=300, max_kv=max_kv)
    assert torch.isnan(O).all() and torch.isnan(L).all()
    assert tq.tq_device_status() == tq.TQ_OK


@pytest.mark.parametrize("case", BOTH, ids=str)
def test_both_kernels_give_the_same(tq, case):
    """The same call planned for the kernel for few rows and for that for many: within the sum of their
    bounds of one another, and the same rows see nothing."""
    lens, hq, hk, dim, page, dtype, out, order = case
    prob = problem(lens, hq, hk, dim, page, dtype, order=order)
    assert not many_rows(tq, prob, 1) and many_rows(tq, prob, 10**8)
    _, _, tol, tol_lse = attention(*prob[:6], dim ** -0.5, 0, out)
    a, la = call(tq, prob, out, max_kv=1)
    b, lb = call(tq, prob, out, max_kv=10**8)
    assert ((a - b).double().abs().cpu() <= 2 * tol).all()
    none = torch.isinf(la)
    assert torch.equal(none, torch.isinf(lb))
    assert ((la - lb).double().abs().cpu() <= 2 * tol_lse)[~none.cpu()].all()
    assert tq.tq_device_status() == tq.TQ_OK
