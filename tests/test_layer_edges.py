"""Sizes of the operators around the mixer at the ends of their ranges, without a GPU."""
import os

import pytest

import gated_delta_rule_64_amd as kda
from gated_delta_rule_64_amd import _layer, _lib
from tests.test_layer_abi import OK, SHAPE, ssm


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.library_path()):
        from gated_delta_rule_64_amd import build
        build.build()
    return _layer._load()


@pytest.mark.parametrize("packed", [0, 1])
@pytest.mark.parametrize("D", [1, 8, 64, 6144])
def test_conv_workspace_of_the_longest_sequences(lib, D, packed):
    """Up to 2^31 - 1 rows take about as many partial sums as 2^20: 64 to 128 rows of blocks."""
    top = 2 ** 31 - 1
    sizes = [lib.kda_conv_bwd_workspace_bytes(1, T, D, 4, 1, packed, 1) for T in (2 ** 20, top - 130, top - 65, top - 63, top - 31, top)]
    assert all(64 * 5 * D * 4 <= n <= 128 * 5 * D * 4 for n in sizes), sizes


def test_scan_rows_are_bounded(lib):
    most = 2 ** 31 - 65
    for chunk in (True, False):
        assert ssm(lib, chunk, B=1, N=1, T=most + 1) == SHAPE and "exceeds" in kda.kda_last_error()
        assert ssm(lib, chunk, cu=8, B=1, N=0, T=most) == OK
    size = lib.kda_ssm_chunk_fwd_workspace_bytes
    assert size(1, most + 1, 1, 1, 64, 64, 1, 0, 1) == 0
    # dt' and the two sums of every row at least
    assert size(1, most, 1, 1, 64, 64, 1, 0, 1) >= size(1, most - 64, 1, 1, 64, 64, 1, 0, 1) >= 12 * (most - 64)
