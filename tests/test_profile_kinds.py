"""ssd_profile_read says how many kinds of kernels there are to a caller that asks for none, and writes no more than it is
given room for (no GPU needed)."""
import ctypes

import pytest

from state_space_sequence_ssd_gb300 import _ffi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _ffi.lib()


def test_asking_for_none_tells_how_many_there_are(lib):
    n = ctypes.c_int(-1)
    assert lib.ssd_profile_read(None, None, 0, ctypes.byref(n)) == 0
    names = [lib.ssd_kernel_name(k) for k in range(n.value)]
    assert b"chunk_scan" in names and b"layer_norm_bwd" in names and b"unknown" not in names
    assert lib.ssd_kernel_name(n.value) == b"unknown"
    ms, counts, got = (ctypes.c_float * n.value)(), (ctypes.c_int * n.value)(), ctypes.c_int(0)
    assert lib.ssd_profile_read(ms, counts, n.value, ctypes.byref(got)) == 0
    assert got.value == n.value


@pytest.mark.parametrize("room", [1, 8])
def test_no_more_is_written_than_there_is_room(lib, room):
    counts, n = (ctypes.c_int * (room + 1))(*[-7] * (room + 1)), ctypes.c_int(0)
    assert lib.ssd_profile_read(None, counts, room, ctypes.byref(n)) == 0
    assert n.value == room and counts[room] == -7 and all(counts[k] >= 0 for k in range(room))
