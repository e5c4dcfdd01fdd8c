"""Per-stage timing of the C ABI: how much of the caller's arrays is written
(no GPU needed: nothing is recorded)."""
import ctypes
import os

import pytest

from block_sparse_spatiotemporal_b200 import fvattn as F


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(F.library_path()):
        from block_sparse_spatiotemporal_b200 import build
        build.build()
    return F.lib()


def arrays(n=32):
    return (ctypes.c_double * n)(*[7.0] * n), (ctypes.c_int64 * n)(*[7] * n)


def test_profile_read_writes_the_ten_stages_it_always_had(lib):
    """A program built when there were ten stages passes arrays of ten."""
    ms, n = arrays()
    assert lib.fvattn_profile_read(ms, n) == 0
    assert list(ms) == [0.0] * 10 + [7.0] * 22 and list(n) == [0] * 10 + [7] * 22
    assert lib.fvattn_profile_read(None, None) == 0


def test_profile_read_stages_writes_as_many_as_asked(lib):
    for count in (0, 1, 10, len(F.STAGES)):
        ms, n = arrays()
        assert lib.fvattn_profile_read_stages(ms, n, count) == 0
        assert list(ms) == [0.0] * count + [7.0] * (32 - count) and list(n) == [0] * count + [7] * (32 - count)
    ms, n = arrays()
    assert lib.fvattn_profile_read_stages(ms, n, 32) == 0      # stages that do not exist: 0
    assert list(ms) == [0.0] * 32 and list(n) == [0] * 32
    assert lib.fvattn_profile_read_stages(None, None, 16) == 0
    ms, n = arrays()
    assert lib.fvattn_profile_read_stages(ms, n, -1) == -1 and list(ms) == [7.0] * 32
    assert set(F.profile_read()) == set(F.STAGES)
