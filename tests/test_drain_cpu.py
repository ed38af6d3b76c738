"""How a block that gave up a wait ends the phases of its barriers (csrc/drain.cuh), on a model of a barrier that
counts arrivals and announced bytes."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_rejection_spec_gb300", "csrc")


class Drain(ctypes.Structure):
    _fields_ = [("begun", ctypes.c_bool), ("missing", ctypes.c_uint32), ("parity", ctypes.c_uint32)]


@pytest.fixture(scope="module")
def drain_of(tmp_path_factory):
    where = tmp_path_factory.mktemp("drain")
    source, library = where / "drain.cpp", where / "drain.so"
    source.write_text('#include "drain.cuh"\nextern "C" specrej::Drain drain_of(uint32_t a, uint32_t n) '
                      '{ return specrej::drain_of(a, n); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-w", "-I", CSRC, str(source), "-o", str(library)])
    f = ctypes.CDLL(str(library)).drain_of
    f.restype, f.argtypes = Drain, [ctypes.c_uint32, ctypes.c_uint32]
    return f


class Barrier:
    """Phases of `count` arrivals; a phase also waits for the bytes announced in it."""

    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phase = count, count, 0, 0

    def _turn(self):
        assert self.pending >= 0
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, announced=0):
        self.bytes += announced
        self.pending -= 1
        self._turn()

    def land(self, n):
        self.bytes -= n
        self._turn()

    def done(self, parity):
        return (self.phase - 1) % 2 == parity


@pytest.mark.parametrize("count", [2, 3])
def test_what_is_in_flight_is_waited_for_and_nothing_else(drain_of, count):
    rng = random.Random(count)
    for _ in range(3000):
        bar, arrivals, flying = Barrier(count), 0, []
        last = rng.randrange(7)
        for phase in range(last + 1):
            made = count if phase < last else rng.randrange(count + 1)  # the last may stop anywhere
            for _ in range(made):
                n = rng.choice([0, 16, 48])
                bar.arrive(n)
                arrivals += 1
                if n:
                    flying.append(n)
            while phase < last and flying:  # the next begins when this one is over
                bar.land(flying.pop())
        for _ in range(rng.randrange(len(flying) + 1)):
            bar.land(flying.pop())
        d = drain_of(arrivals, count)
        assert d.begun == (arrivals > 0) and 0 <= d.missing < count
        for _ in range(d.missing):
            bar.arrive()
        assert d.begun or not flying
        while flying:
            assert not bar.done(d.parity)
            bar.land(flying.pop())
        assert not d.begun or bar.done(d.parity)


def test_both_parities_are_never_done():
    """Why the wait needs the parity of the last phase: of the two, one is always over and one never."""
    bar = Barrier(2)
    for _ in range(5):
        assert bar.done(0) != bar.done(1)
        bar.arrive(16)
        assert bar.done(0) != bar.done(1)
        bar.arrive()
        bar.land(16)
