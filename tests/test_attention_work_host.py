"""How the many-row attention kernel deals its work to thread blocks, on the host: the kernel's own
arithmetic (csrc/tq_attn_work.cuh) in a model of all blocks and threads (attn_work_model.cc)."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    """check(q_start, kv_len, ntok, group, heads, window, max_positions, grid, sound): '' or what is
    wrong."""
    cc = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cc:
        pytest.skip("no C++ compiler")
    lib = str(tmp_path_factory.mktemp("work") / "model.so")
    subprocess.run([cc, "-O2", "-std=c++17", "-Wall", "-Wextra", "-fPIC", "-shared",
                    os.path.join(HERE, "attn_work_model.cc"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).attn_work_check
    i = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, i, ctypes.c_int64, i, i, i, i, i, i, ctypes.c_char_p]

    def call(q_start, kv_len, ntok, group, heads, window=0, max_positions=1 << 30, grid=152, sound=True):
        q = np.asarray(q_start, dtype=np.int32)
        k = np.asarray(kv_len, dtype=np.int32)
        why = ctypes.create_string_buffer(256)
        ok = fn(q.ctypes.data, k.ctypes.data, len(k), ntok, group, heads, window, max_positions, grid,
                int(sound), why)
        assert ok == (why.value == b"")
        return why.value.decode()

    return call


def batch(r):
    """New tokens and lengths of a well-formed batch: ragged, some sequences empty or shorter than their
    new tokens."""
    nseq = r.choice((1, 1, 2, 3, 8, 40, 70))
    most = r.choice((1, 3, 40, 300, 2000))
    new = [r.choice((0, 1, most, r.randint(0, most))) for _ in range(nseq)]
    new[r.randrange(nseq)] = most
    kv = [max(0, n + r.choice((0, 0, -n // 2, r.randint(0, 3000), r.randint(0, 30)))) for n in new]
    return new, kv


@pytest.mark.parametrize("seed", range(6))
def test_every_key_tile_once(check, seed):
    r = random.Random(seed)
    for _ in range(60):
        new, kv = batch(r)
        group, heads = r.choice((1, 2, 3, 5, 8, 40)), r.choice((1, 2, 8))
        q_start = np.concatenate([[0], np.cumsum(new)])
        args = (q_start, kv, int(q_start[-1]) + r.choice((0, 0, 5)), group, heads, r.choice((0, 0, 1, 100, 700)),
                r.choice((1 << 30, 1024)), r.choice((152, 152, 148, 7)))
        assert check(*args) == "", args


@pytest.mark.parametrize("seed", range(4))
def test_starts_out_of_order_stay_in_bounds(check, seed):
    """Whatever q_start holds: no head, token or partial result past the last one, and an end."""
    r = random.Random(100 + seed)
    for _ in range(1500):
        nseq, ntok = r.randint(1, 9), r.randint(1, 3000)
        q_start = [r.choice((r.randint(-10, ntok + 10), r.randint(0, ntok), -2**31, 2**31 - 1))
                   if r.random() < 0.1 else r.randint(0, ntok) for _ in range(nseq + 1)]
        args = (q_start, [r.randint(0, 4000) for _ in range(nseq)], ntok, r.choice((1, 2, 8)), r.choice((1, 8)))
        assert check(*args, sound=False) == "", args


@pytest.mark.parametrize("nseq,new,kv,group,heads", [
    (530000, 1, 1, 200, 1), (4097, 2048, 2048, 16, 1), (2, 1 << 24, 1 << 20, 8, 1), (700000, 1, 300, 130, 3)])
def test_more_row_tiles_than_19_bits_count(check, nseq, new, kv, group, heads):
    """Row tiles by the half million, which single tokens of many sequences, or long chunks, can be."""
    q_start = np.arange(nseq + 1, dtype=np.int64) * new
    kv_len = np.full(nseq, kv)
    kv_len[::7] += 129
    assert nseq * -(-new * group // 256) > 1 << 19
    assert check(q_start, kv_len, nseq * new, group, heads) == ""


def test_no_work(check):
    """No new tokens at all, in few sequences and in more than are counted."""
    for nseq in (1, 40, 1 << 19):
        for ntok in (0, 5):
            assert check(np.zeros(nseq + 1), np.full(nseq, 100), ntok, 4, 2) == ""
