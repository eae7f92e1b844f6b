"""Sizes of the operators around the mixer at the ends of their ranges, without a GPU."""
import os

import pytest
import torch

import gated_delta_rule_64_amd as kda
from gated_delta_rule_64_amd import _layer, _lib
from tests.test_abi import _rec, _rec_ex
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
    """Up to 2^31 - 1 rows take about as many partial sums as 2^20: 64 to 512 rows of blocks."""
    top = 2 ** 31 - 1
    sizes = [lib.kda_conv_bwd_workspace_bytes(1, T, D, 4, 1, packed, 1) for T in (2 ** 20, top - 130, top - 65, top - 63, top - 31, top)]
    assert all(64 * 5 * D * 4 <= n <= 512 * 5 * D * 4 for n in sizes), sizes
    assert all(a <= b for a, b in zip(sizes[1:], sizes[2:])), sizes


def test_conv_backward_of_narrow_rows_fills_the_units(lib):
    """Rows of blocks of a long batch: 512 where one block is as wide as a row, 128 for wide rows."""
    for D, most in ((8, 512), (256, 512), (512, 256), (1024, 128), (6144, 128)):
        rows = lib.kda_conv_bwd_workspace_bytes(1, 1 << 20, D, 4, 1, 0, 1) / (5 * D * 4)
        assert 0.9 * most <= rows <= most or (D == 8 and rows == 128), (D, rows)   # 8 channels: 128 tiles a block


def test_scan_rows_are_bounded(lib):
    most = 2 ** 31 - 65
    for chunk in (True, False):
        assert ssm(lib, chunk, B=1, N=1, T=most + 1) == SHAPE and "exceeds" in kda.kda_last_error()
        assert ssm(lib, chunk, cu=8, B=1, N=0, T=most) == OK
    size = lib.kda_ssm_chunk_fwd_workspace_bytes
    assert size(1, most + 1, 1, 1, 64, 64, 1, 0, 1) == 0
    # dt' and the two sums of every row at least
    assert size(1, most, 1, 1, 64, 64, 1, 0, 1) >= size(1, most - 64, 1, 1, 64, 64, 1, 0, 1) >= 12 * (most - 64)


def test_grids_of_2_to_the_32_threads_are_refused(lib):
    """HIP counts a launch's threads in 32 bits and would leave the rest out."""
    for chunk, N in ((False, 2 ** 21), (True, 2 ** 20)):
        assert ssm(lib, chunk, B=N, N=N, T=1, HV=32, V=64, xs=2048, dts=32) == SHAPE and "grid" in kda.kda_last_error()


def test_decode_grids_of_2_to_the_32_threads_are_refused(lib):
    _lib.load_library()
    N = 2 ** 21
    assert _rec(lib, B=N, N=N, HV=64, V=64) == SHAPE and "grid" in kda.kda_last_error()
    assert _rec_ex(lib, B=N, N=N, HV=16, V=64, lay=1) == SHAPE and "grid" in kda.kda_last_error()   # 16 columns a wave


def test_overlap_is_by_bytes():
    """The binding's check of given outputs, on host tensors."""
    buf = torch.zeros(1000)

    def hits(out, t, rows=1, stride=1, same=()):
        try:
            _layer._apart("out", out, (("t", t, rows, stride),), same)
        except ValueError:
            return True
        return False
    t = buf[100:200]
    for a, b, want in ((0, 100, False), (0, 101, True), (199, 300, True), (200, 300, False), (150, 150, False), (0, 1000, True),
                       (120, 130, True)):
        assert hits(buf[a:b], t) is want
    assert hits(buf[100:200], t) and not hits(buf[100:200], t, same=("t",)) and hits(buf[101:201], t, same=("t",))
    assert not hits(t, None) and not hits(t, buf[150:150])
    rows = buf.as_strided((5, 10), (100, 1), 200)     # elements 200.., 300.., .. 600..609
    for a, b, want in ((0, 200, False), (0, 201, True), (210, 300, False), (209, 300, True), (210, 301, True), (610, 700, False),
                       (609, 700, True), (550, 560, False), (450, 560, True)):
        assert hits(buf[a:b], rows, 5, 100) is want, (a, b)


def test_scan_bounds_see_a_dropped_part():
    """What the bounds of the GPU tests of the scan's writes and decays are made to see: a weighted x
    cut into two bf16 instead of three, and running sums of decays without their low part."""
    eps = 2.0 ** -24
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1000, generator=g).bfloat16().float()
    v = (torch.rand(1000, generator=g) + 0.5) * x

    def cut(v, parts):
        left, total = v.clone(), torch.zeros_like(v, dtype=torch.float64)
        for _ in range(parts):
            top = (left.view(torch.int32) & -65536).view(torch.float32)
            total += top.double()
            left = left - top
        return total
    off = lambda t: ((t - v.double()).abs() / v.double().abs()).max().item()  # noqa: E731
    assert off(cut(v, 3)) == 0 and off(cut(v, 2)) > 4 * 40 * eps      # 40: the widest of test_scan_writes_are_fp32_products
    # sixteen decays of 131 log2(e), then some of 0.01: 2^(last - sum at the write) from the sums
    steps = torch.cat([torch.full((16,), 131.0), 0.001 + 0.01 * torch.rand(48, generator=g)])
    cum = torch.cumsum(steps.double() * -1.4426950408889634, 0)
    want = torch.exp2(cum[-1] - cum[16])
    hi = cum.float()
    lo = (cum - hi.double()).float()
    both = torch.exp2((hi[-1] - hi[16]).double() + (lo[-1] - lo[16]).double())
    assert abs(both - want) <= 2 * eps * want
    assert abs(torch.exp2((hi[-1] - hi[16]).double()) - want) > 4 * 16 * eps * want
