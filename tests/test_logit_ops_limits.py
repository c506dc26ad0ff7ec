"""Size limits of the logit operators that are refused on the host."""

import ctypes

import pytest

from draft_model_distillation_amd import _binding as B
from tests import test_logit_ops_validation as LV


@pytest.fixture(scope="module")
def lib():
    return B.load_library(require_torch_runtime=False)


def test_history_longer_than_the_index_range(lib):
    at = dict(history=LV.P, history_len=LV.P, ld_history=1 << 31)
    assert LV._adjust(lib, **at, max_history=(1 << 29) + 1) == 2
    assert LV._adjust(lib, **at, max_history=(1 << 31) - 1) == 2
    assert "max_history" in lib.opd_last_error().decode()
    assert ctypes.sizeof(B.OpdAdjust) % 8 == 0


def test_rows_past_the_counted_range(lib):
    many = (1 << 31)
    assert LV._topk(lib, n=many) == 2 and LV._adjust(lib, n=many) == 2
    for which in ("fwd", "bwd", "fused"):
        assert LV._loss(lib, which, n=many) == 2
