"""Sizes of the experts' operators that need more workgroups than one launch has in some
tile, or in all of them. On the CPU: what the entry points take and refuse, at made-up
addresses (a call that is taken stops at the device check). On the GPU: results of sizes
past 2^22 workgroups against float64. Tolerances are test_grouped_linear_gpu.py's.
"""

import pytest
import torch

from eight import close, cpu64, sum_tol
from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L

AT = [k << 50 for k in range(1, 6)]  # addresses that are only compared


def _call(op, rows, experts, fin, fout, layout):
    d = B.muon_grouped(rows, experts, fin, fout, 0, 0, 0, 0, B.MUON_TYPE_BF16, layout)
    if op == "forward":
        return B.muon_grouped_linear_forward(d, AT[0], AT[1], AT[2], None, AT[3], 0)
    if op == "grad input":
        return B.muon_grouped_linear_grad_input(d, AT[0], AT[1], AT[2], None, AT[3], 0)
    return B.muon_grouped_linear_grad_weight(d, AT[0], AT[1], AT[2], AT[3], AT[4], 0, AT[4] * 2, 1 << 40, 0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: for hosts without a GPU")
@pytest.mark.parametrize("layout", [B.MUON_WEIGHT_IN_OUT, B.MUON_WEIGHT_OUT_IN])
@pytest.mark.parametrize("op,rows,experts,fin,fout,taken", [
    # the cheapest tile has more than 2^22 workgroups
    ("forward", 131072, 16384, 64, 16384, True),
    ("forward", 1 << 20, 65536, 64, 4096, True),
    ("forward", 1 << 20, 65536, 8, 6400, True),
    ("grad input", 131072, 16384, 16384, 64, True),
    # rows off 16-byte borders have one tile, 64 x 64
    ("forward", 1 << 20, 16, 9, 16385, True),
    ("grad input", 1 << 20, 16, 16385, 9, True),
    ("grad weight", 100, 65536, 9, 3649, True),
    # the last size of it and the first beyond: 2^24 workgroups of 256 threads are 2^32
    ("forward", 64 * 1023 - 1, 1, 9, 64 * 16384 - 1, True),
    ("forward", 64 * 1023, 1, 9, 64 * 16384 - 1, False),
    ("grad weight", 100, 65536, 1023, 1023 - 64, True),
    ("grad weight", 100, 65536, 1023, 1023, False),
    # no tile is large enough
    ("forward", (1 << 24) - 1, 65536, 64, 1 << 21, False),
    ("grad input", (1 << 24) - 1, 65536, 1 << 21, 64, False),
    ("grad weight", 100, 65536, 1 << 20, 64, False),
], ids=str)
def test_sizes_are_refused_only_where_no_tile_takes_them(op, rows, experts, fin, fout, taken, layout):
    s = _call(op, rows, experts, fin, fout, layout)
    assert s == (B.MUON_E_NO_DEVICE if taken else B.MUON_E_SHAPE), B.muon_op_last_error()


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


@pytest.mark.gpu
def test_rows_past_2_22_workgroups():
    """2^20 rows of 9 features to 16385, through registers: 4.2 million tiles of 64 x 64;
    rows of each expert, those around its ends among them."""
    _room(40)
    n, i, o, e = 1 << 20, 9, 16385, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, i, generator=g, device="cuda").bfloat16()
    w = torch.randn(e, i, o, generator=g, device="cuda").bfloat16()
    at = [0] + sorted(torch.randint(0, n, (e - 1,), generator=torch.Generator().manual_seed(2)).tolist()) + [n]
    y = L.grouped_linear_forward(x, w, torch.tensor(at, dtype=torch.int32).cuda())
    for k in range(e):
        a, b = at[k], at[k + 1]
        rows = sorted({r for r in (a, a + 63, a + 64, (a + b) // 2, b - 65, b - 64, b - 1) if a <= r < b})
        if rows:
            x64, w64 = cpu64(x[rows]), cpu64(w[k])
            close(torch.stack([y[r] for r in rows]), x64 @ w64, sum_tol(x64, w64), torch.bfloat16)


@pytest.mark.gpu
def test_weight_gradients_past_2_22_workgroups():
    """65536 experts, 9 x 3649 each: 58 tiles of 64 x 64, 64 workgroups an expert."""
    _room(16)
    n, i, o, e = 300, 9, 3649, 65536
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, i, generator=g, device="cuda").bfloat16()
    dy = torch.randn(n, o, generator=g, device="cuda").bfloat16()
    # the last expert, the first and one between have all the rows
    at = torch.full((e + 1,), 200, dtype=torch.int32)
    at[0], at[1:40001], at[e] = 0, 70, n
    dw, db = L.grouped_linear_grad_weight(x, dy, at.cuda(), dw=torch.full((e, i, o), 7.0, device="cuda"), dbias=True)
    some = {0: (0, 70), 40000: (70, 200), e - 1: (200, 300)}
    for k, (a, b) in some.items():
        x64, d64 = cpu64(x[a:b]), cpu64(dy[a:b])
        close(dw[k], x64.t() @ d64, sum_tol(x64.t(), d64), torch.float32)
        ones = torch.ones(1, b - a, dtype=torch.float64)
        close(db[k], d64.sum(0), sum_tol(ones, d64)[0], torch.float32)
        dw[k] = 0
        db[k] = 0
    assert not dw.any() and not db.any()
