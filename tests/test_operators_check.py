"""check_operators() with a stand-in for the library: every device's record is
read and cleared, whatever the others hold.  No GPU."""
from __future__ import annotations

import pytest

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators


class FakeLibrary:
    def __init__(self, records, broken=()):
        self.records, self.broken, self.read = dict(records), broken, []

    def gemm_ops_check(self, handle, status, detail):
        self.read.append(handle)
        if handle in self.broken:
            return sg.GEMM_ERR_CUDA
        status._obj.value, detail._obj.value = self.records[handle]
        self.records[handle] = (0, 0)
        return 0


@pytest.fixture
def fake(monkeypatch):
    def install(records, broken=()):
        lib = FakeLibrary(records, broken)
        monkeypatch.setattr(operators, "_handles", {n: h for n, h in enumerate(records)})
        monkeypatch.setattr(operators, "_lib", lambda: lib)
        return lib
    return install


def test_every_record_is_read_and_the_first_error_raised(fake):
    lib = fake({11: (0, 0), 12: (sg.GEMM_ERR_TIMEOUT, (1 << 16) | 1), 13: (sg.GEMM_ERR_BOUNDS, 0), 14: (0, 0)})
    with pytest.raises(sg.GemmError) as e:
        sg.check_operators()
    assert e.value.status == sg.GEMM_ERR_TIMEOUT and lib.read == [11, 12, 13, 14]
    sg.check_operators()         # all cleared


def test_a_failing_check_does_not_hide_the_others(fake):
    lib = fake({21: (0, 0), 22: (sg.GEMM_ERR_TIMEOUT, 0)}, broken=(21,))
    with pytest.raises(sg.GemmError) as e:
        sg.check_operators()
    assert e.value.status == sg.GEMM_ERR_CUDA and lib.read == [21, 22]


def test_nothing_recorded(fake):
    fake({31: (0, 0)})
    sg.check_operators()
