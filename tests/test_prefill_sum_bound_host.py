"""The sum bound of the prefill workspaces, up to the largest number a caller
may pass for it."""
import pytest

import paged_fp8_kv_03_gb300 as pkv


def _fp4(total, *window):
    return pkv.pkv_prefill_fp4_workspace_size(3, 2, 100, 5000, total, *window)


def _fp8(total):
    return pkv.pkv_prefill_workspace_size(3, 2, 5000, total)


@pytest.mark.parametrize("size", [_fp4, _fp8, lambda total: _fp4(total, 64, 4)])
def test_large_sum_bounds_are_none(size):
    for total in (1 << 40, 2 ** 63 - 200, 2 ** 63 - 128, 2 ** 63 - 127, 2 ** 63 - 1):
        assert size(total) == size(0), total


def test_sum_bounds_count_whole_tiles():
    for size in (_fp4, _fp8):
        assert size(1) == size(127) == size(128) < size(129) == size(256) < size(257) < size(0)
