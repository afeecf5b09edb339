"""A step of several requests as a server makes it: the shared ternary product, the adapters of each
request beside it, the draw of each request's next token; eager, and from one captured graph whose
requests change from replay to replay."""
import importlib.util
import os

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    import bit_matvec_gb300
    yield bit_matvec_gb300
    assert bit_matvec_gb300.tq_device_status() == bit_matvec_gb300.TQ_OK


@pytest.mark.parametrize("ntok,vocab,cols", [(1, 1000, 512), (5, 4000, 1024), (12, 2048, 512), (300, 777, 256)])
def test_product_adapters_draw(tq, ntok, vocab, cols):
    from test_gpu_lora import check, make, scratch
    from test_gpu_sample import reference
    w = torch.from_numpy(synth.pq2_0_weights(vocab, cols, 3)).cuda()
    laid = tq.repacked_empty(vocab, cols)
    tq.tq_repack(w, laid, vocab, cols)
    d = make(ntok, cols, vocab, 4, 8, seed=40)
    lora = tq.Lora(d["a"], d["b"], d["rank"], d["scale"])
    g = torch.Generator().manual_seed(41)
    x, u = d["x"], torch.empty(ntok, device="cuda")
    t, p = torch.empty(ntok, device="cuda"), torch.empty(ntok, device="cuda")
    k = torch.empty(ntok, dtype=torch.int32, device="cuda")
    xq, ws = tq.q8K_empty(ntok, cols), tq.workspace_empty(vocab, cols, ntok)
    lws = scratch(tq, ntok, 4)
    base, y = torch.empty(ntok, vocab, device="cuda"), torch.empty(ntok, vocab, device="cuda")
    tokens, logp = torch.empty(ntok, dtype=torch.int32, device="cuda"), torch.empty(ntok, device="cuda")

    def step():
        tq.tq_quantize_matmul(laid, x, xq, y, vocab, cols, ntok, ws)
        tq.tq_lora_add(x, lora, d["ids"], y, y, lws)
        tq.tq_sample(y, u, tokens, t, k, p, None, logp)

    def request(i):
        x.copy_(torch.randn(ntok, cols, generator=g))
        d["ids"].copy_(torch.randint(-1, 4, (ntok,), generator=g, dtype=torch.int32))
        u.copy_(torch.rand(ntok, generator=g))
        t.copy_(torch.rand(ntok, generator=g) * (i % 3))
        k.copy_(torch.randint(0, 30, (ntok,), generator=g, dtype=torch.int32))
        p.copy_(torch.rand(ntok, generator=g) * 0.5 + 0.5)

    def inspect():
        tq.tq_quantize_matmul(laid, x, xq, base, vocab, cols, ntok, ws)
        d["z"] = base
        check(d, y)
        for i in range(0, ntok, max(1, ntok // 20)):
            want = reference(y[i], u[i].item(), t[i].item(), k[i].item(), p[i].item(), 0.0)
            assert tokens[i].item() in want

    request(1)
    step()
    inspect()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(4):
        request(i)
        y.fill_(float("nan"))
        tokens.fill_(-9)
        graph.replay()
        inspect()
    # many replays of one request with nothing between them: the same tokens every time
    want = tokens.clone()
    for _ in range(20):
        graph.replay()
    assert torch.equal(tokens, want)
