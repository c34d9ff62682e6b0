"""The largest matrices that the quantisers take, on the CPU at made-up addresses: a call
that is taken stops at the device check."""

import pytest
import torch

from muon_newton_schulz_04_amd import binding as B

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: for hosts without a GPU")


@pytest.mark.parametrize("rows,segments,taken", [
    # 512 columns of a row are a wave's, four waves a workgroup of 256 threads, and a
    # launch has fewer than 2^32 threads: 2^26 - 4 such segments, and the first beyond
    (4, (1 << 24) - 1, False),           # more columns than 2^21
    ((1 << 24) - 1, 4, True),            # 2^26 - 4
    (22369621, 3, False),                # 2^26 - 1 in more rows than 2^24
    (24573, 2731, False),                # 2^26 - 1
    (18631, 3602, False),                # 2^26 - 2
    ((1 << 23), 8, False),               # 2^26
    (1 << 20, 63, True),
])
def test_rows(rows, segments, taken):
    q = B.muon_eight(1 << 50, 1 << 51, 0, B.MUON_EIGHT_E4M3, 0)
    s = B.muon_quantize(rows, 512 * segments - 3, 0, B.MUON_TYPE_BF16, 1 << 49, q, 0)
    assert s == (B.MUON_E_NO_DEVICE if taken else B.MUON_E_SHAPE), B.muon_op_last_error()


@pytest.mark.parametrize("rows,cols,taken", [(1 << 21, 128 * 511, True), (128 * 511, 1 << 21, True),
                                             (1 << 21, 128 * 512, False), (128 * 512, 1 << 21, False)])
def test_weights(rows, cols, taken):
    q, t = (B.muon_eight(k << 50, k << 48, 0, B.MUON_EIGHT_E4M3, 0) for k in (1, 3))
    s = B.muon_quantize_weight(rows, cols, 0, B.MUON_TYPE_FP32, 5 << 50, q, t, 0)
    assert s == (B.MUON_E_NO_DEVICE if taken else B.MUON_E_SHAPE), B.muon_op_last_error()
