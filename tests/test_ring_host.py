"""What a thread block that gave up waits for before it leaves: the last copies of each stage of its
ring (csrc/tq_ring.cuh), in a model of the stages' barriers."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def last_phase(tmp_path_factory):
    cc = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cc:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("ring")
    src = d / "ring.cc"
    src.write_text(f'#include "{HERE}/../bit_matvec_gb300/csrc/tq_ring.cuh"\n'
                   'extern "C" int last_phase(int n, int s, int k) { return tq::last_phase(n, s, k); }\n')
    subprocess.run([cc, "-O1", "-std=c++17", "-fPIC", "-shared", str(src), "-o", str(d / "ring.so")], check=True)
    return ctypes.CDLL(str(d / "ring.so")).last_phase


class Barrier:
    """An mbarrier of one arrival: a wait for a parity passes unless the current phase has it."""

    def __init__(self):
        self.phase = 0

    def landed(self):
        self.phase += 1

    def passes(self, parity):
        return self.phase % 2 != parity


@pytest.mark.parametrize("stages", [3, 5, 8])
def test_no_block_leaves_before_its_copies_have_landed(last_phase, stages):
    """A producer stops after any number of items, with the last one of a stage still in flight: the
    wait holds until it lands, and passes then."""
    for issued in range(0, 4 * stages + 2):
        for stage in range(stages):
            items = list(range(stage, issued, stages))
            parity = last_phase(issued, stage, stages)
            if not items:
                assert parity == -1
                continue
            bar = Barrier()
            for _ in items[:-1]:
                bar.landed()     # a stage is only refilled when its last item was used
            assert not bar.passes(parity), (issued, stage)
            bar.landed()
            assert bar.passes(parity), (issued, stage)


def test_the_items_a_range_has_are_not_those_issued(last_phase):
    """Why the count has to be of items issued: with three of four items issued, the parity of the
    fourth passes on stage 0 while the first one is in flight."""
    bar = Barrier()
    assert bar.passes(last_phase(4, 0, 3)) and not bar.passes(last_phase(3, 0, 3))
