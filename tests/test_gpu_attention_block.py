"""The attention block example: prompts in one chunk, then decode steps from a graph, against whole
sequences in one chunk."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(seqs=3, prompt=70, steps=5, width=1024, q_heads=8, kv_heads=2),
                                dict(seqs=1, prompt=1, steps=3, width=512, q_heads=4, kv_heads=4),
                                dict(seqs=5, prompt=200, steps=4, width=768, q_heads=12, kv_heads=3,
                                     head_dim=64, page_size=32)], ids=str)
def test_steps_equal_whole_chunks(kw):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_matvec_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("attention_block",
                                                  os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, _ = m.run(**kw)
    # Attention of the two ways differs by bf16 roundings of the weights (2^-8 of the values' mean
    # magnitude at most), and a value that lands on the other side of an int8 step moves by 1/127
    # of its block's largest: errors of a few percent of the rms of a sum over such values.
    assert off < 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(seqs=5, prompt=300, steps=64, width=1024, q_heads=8, kv_heads=2),
                                dict(seqs=3, prompt=600, steps=16, width=512, q_heads=4, kv_heads=4),
                                dict(seqs=8, prompt=2, steps=3, width=512, q_heads=4, kv_heads=4)], ids=str)
def test_workspace_of_every_call(kw):
    """Batches whose prompts, or steps, need a larger workspace than all their tokens at once do."""
    test_steps_equal_whole_chunks(kw)
