"""One attention block of a decoder on the library: ternary projections, head norms and rotation,
the paged key/value cache, causal attention, ternary output projection.

    python examples/attention_block.py [--seqs 4] [--prompt 300] [--steps 16]

The prompts of all sequences go in as one ragged chunk; then one token of every sequence a step,
captured once in a CUDA graph and replayed (the lengths and positions are device arrays, so the
graph serves every step). The outputs are compared with those of taking each whole sequence as one
chunk: the same tokens through the other kernels. Weights and inputs are random.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_matvec_gb300 as tq  # noqa: E402
import synth  # noqa: E402

I32 = torch.int32


class AttentionBlock:
    """y = x + Wo attention(Wqkv x), with the weights laid out once and the workspaces kept. shapes:
    the (tokens, most tokens of a sequence) of the calls to come."""

    def __init__(self, width, q_heads, kv_heads, head_dim, shapes, max_kv, nseq, device="cuda"):
        self.width, self.hq, self.hk, self.dim = width, q_heads, kv_heads, head_dim
        self.rows = (q_heads + 2 * kv_heads) * head_dim
        self.out_cols = q_heads * head_dim
        self.max_kv, self.device = max_kv, device
        self.wqkv = self._weights(self.rows, width, 11)
        self.wo = self._weights(width, self.out_cols, 12)
        ones = torch.ones(head_dim, device=device)
        self.q_norm, self.k_norm = ones.clone(), ones.clone()
        # a context four times as long as the 4096 positions the rotation was made for
        turns, amplitude = tq.tq_rope_turns(head_dim, 1e6, tq.ROPE_RAMP, 4.0, 4096.0, 1.0, 32.0)
        self.rope = tq.Rope(turns.to(device), False, amplitude)
        # buffers for the largest call, and one workspace for all of them (fewer tokens may need more)
        n = max(t for t, _ in shapes)
        empty = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        self.qkv, self.att = empty(n, self.rows), empty(n, self.out_cols)
        self.q, self.y = empty(n, q_heads, head_dim, dtype=torch.bfloat16), empty(n, width)
        self.xq, self.aq = tq.q8K_empty(n, width, device), tq.q8K_empty(n, self.out_cols, device)
        need = max([tq.tq_paged_attention_workspace_bytes(nseq, t, q_heads, kv_heads, head_dim, m, max_kv)
                    for t, m in shapes] +
                   [tq.tq_matmul_workspace_bytes(r, c, t) for r, c in
                    ((self.rows, width), (width, self.out_cols)) for t, _ in shapes])
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)

    def _weights(self, rows, cols, seed):
        packed = torch.from_numpy(synth.pq2_0_weights(rows, cols, seed)).to(self.device)
        laid = tq.repacked_empty(rows, cols, self.device)
        tq.tq_repack(packed, laid, rows, cols)
        return laid

    def cache(self, pages, page_size, table):
        shape = (pages, self.hk, page_size, self.dim)
        k = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        return tq.PagedKV(k, torch.zeros_like(k), table)

    def forward(self, x, kv, seq_ids, positions, q_start, kv_len, max_q):
        """x [tokens][width] f32; the tokens' keys and values are added to kv. Returns a view of
        this block's output buffer."""
        n = x.shape[0]
        qkv, att, y = self.qkv[:n], self.att[:n], self.y[:n]
        tq.tq_quantize_matmul(self.wqkv, x, self.xq, qkv, self.rows, self.width, n, self.ws)
        heads = qkv.view(n, self.hq + 2 * self.hk, self.dim)
        tq.tq_kv_append(heads[:, :self.hq], heads[:, self.hq:self.hq + self.hk],
                        heads[:, self.hq + self.hk:], self.q[:n], kv, seq_ids, positions, self.rope,
                        self.q_norm, self.k_norm)
        tq.tq_paged_attention(self.q[:n], kv, q_start, kv_len, att.view(n, self.hq, self.dim), max_q,
                              self.max_kv, self.dim ** -0.5, self.ws)
        tq.tq_quantize_matmul(self.wo, att, self.aq, y, self.width, self.out_cols, n, self.ws)
        return y.add_(x)


def page_table(lengths, page_size, seed, device):
    need = [-(-n // page_size) for n in lengths]
    order = np.random.RandomState(seed).permutation(sum(need))
    table = np.zeros((len(need), max(need)), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).to(device), sum(need)


def chunk_args(before, new, device):
    """Device arrays of a step that adds new[b] tokens to before[b]."""
    t = lambda a: torch.tensor(a, dtype=I32, device=device)   # noqa: E731
    seq = [b for b, n in enumerate(new) for _ in range(n)]
    pos = [before[b] + i for b, n in enumerate(new) for i in range(n)]
    return (t(seq), t(pos), t([0] + list(np.cumsum(new))), t([a + n for a, n in zip(before, new)]), max(new))


def run(seqs=4, prompt=300, steps=16, width=5120, q_heads=40, kv_heads=8, head_dim=128, page_size=16,
        seed=7):
    """The largest difference between stepwise and whole outputs, over their rms."""
    dev = "cuda"
    r = np.random.RandomState(seed)
    prompts = [max(1, int(prompt * f)) for f in r.uniform(0.2, 1.0, seqs)]
    total = [n + steps for n in prompts]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = [torch.randn(n, width, generator=g, device=dev) for n in total]
    shapes = [(sum(prompts), max(prompts)), (seqs, 1), (sum(total), max(total))]
    block = AttentionBlock(width, q_heads, kv_heads, head_dim, shapes, max(total), seqs)
    table, pages = page_table(total, page_size, seed, dev)

    # the prompts, then a token of every sequence at a time
    kv = block.cache(pages, page_size, table)
    first = block.forward(torch.cat([a[:n] for a, n in zip(x, prompts)]), kv,
                          *chunk_args([0] * seqs, prompts, dev)).clone()
    out = [[c] for c in first.split(prompts)]
    seq_ids, pos, q_start, kv_len, _ = chunk_args(prompts, [1] * seqs, dev)
    step_x = torch.empty(seqs, width, device=dev)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step_y = block.forward(step_x, kv, seq_ids, pos, q_start, kv_len, 1)
            pos.add_(1)      # the next step's positions and lengths
            kv_len.add_(1)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for i in range(steps):
        step_x.copy_(torch.stack([a[n + i] for a, n in zip(x, prompts)]))
        graph.replay()
        for b, row in enumerate(step_y.clone()):
            out[b].append(row[None])
    end.record()
    stepwise = torch.cat([torch.cat(o) for o in out])

    # every sequence whole, as one chunk
    whole = block.forward(torch.cat(x), block.cache(pages, page_size, table),
                          *chunk_args([0] * seqs, total, dev))
    if tq.tq_device_status() != tq.TQ_OK:
        raise RuntimeError("a kernel reported an error")
    off = ((stepwise - whole).abs().max() / whole.pow(2).mean().sqrt()).item()
    return off, start.elapsed_time(end) / max(steps, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("seqs", 4), ("prompt", 300), ("steps", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    off, ms = run(a.seqs, a.prompt, a.steps)
    print(f"{a.seqs} sequences, {a.steps} steps: {ms * 1e3:.0f} us a step with its copies, "
          f"stepwise and whole outputs differ by at most {off:.4f} of their rms")
