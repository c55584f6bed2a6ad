"""Block norms of more rows than workgroups are launched: a workgroup walks several rows, requesting the next one
while it sums and stores this one. And rows at the ends of the range in which squares are fp32."""

import numpy as np
import pytest
import torch

from gpu_util import bits, log
from test_gpu_norm import check, make, run

pytestmark = pytest.mark.gpu

# More than twice the most workgroups of each launch shape (4096 up to 4096 channels, 2048 up to 8192, 1024 past
# that), so that some take three rows and use each of the two buffers of partial sums twice; D % 8 last channels
SHAPES = [(9001, 520), (8200, 1003), (8300, 2056), (4100, 5120), (4100, 8191), (2100, 8193), (2050, 16384)]
PARTS = [(1, 1, 1, 1), (1, 1, 0, 0), (0, 0, 0, 1), (1, 0, 0, 1), (1, 0, 1, 0)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("parts", PARTS, ids=str)
def test_several_rows_per_workgroup(rows, D, parts):
    resid_bf16 = (D + sum(parts)) % 2 == 0
    log(f"norm rows={rows} D={D} parts={parts} resid_bf16={resid_bf16}")
    c = make(rows + D, rows, D, parts, resid_bf16)
    got = run(c, not resid_bf16)
    check(c, got, not resid_bf16)
    if parts[0]:
        log("in place")
        same = run(c, not resid_bf16, in_place=True)
        for x, y in zip(got, same):
            assert (x is None) == (y is None) and (x is None or np.array_equal(bits(x), bits(y)))


@pytest.mark.parametrize("rows,D", SHAPES[:1] + SHAPES[3:4] + SHAPES[5:6])
def test_a_row_does_not_depend_on_where_it_stands(rows, D):
    """The same rows in another order, other rows before and after each in its workgroup: the same bits, in place and
    with columns between the rows too."""
    c = make(rows, rows, D, (1, 1, 1, 1), True)
    order = torch.randperm(rows, generator=torch.Generator().manual_seed(D))
    log(f"norm rows={rows} D={D}, in order")
    a = run(c, True)
    for in_place, pad in ((False, 0), (True, 0), (True, 8)):
        log(f"norm rows={rows} D={D}, shuffled, in_place={in_place} pad={pad}")
        b = run({k: t[order] if t is not None and t.dim() == 2 else t for k, t in c.items()}, True, in_place=in_place,
                pad=pad)
        for x, y in zip(a, b):
            assert np.array_equal(bits(x.contiguous())[order.numpy()], bits(y.contiguous()))


@pytest.mark.parametrize("D", [64, 2051, 16384])
def test_ends_of_the_range_of_squares(D):
    """Without eps: rows of values from 2^-60 to 2^63 / sqrt(D) are normalized as any others; a row whose squares sum
    past fp32's range gives 0, one whose squares are all 0 infinities, one of zeros NaN."""
    c = make(D, 7, D, (0, 0, 0, 1), False)
    unit = c["resid"].sign() * (1 + torch.rand(7, D, generator=torch.Generator().manual_seed(1)))
    unit[unit == 0] = 1.0
    scale = torch.tensor([2.0 ** -60, 2.0 ** -30, 1.0, 2.0 ** 62 / D ** 0.5, 2.0 ** 64, 2.0 ** -80, 0.0])
    c["resid"] = unit * scale[:, None]
    log(f"norm of rows of 2^-80 to 2^64, D={D}, eps 0")
    _, y = run(c, False, eps=0.0)
    check(dict(c, resid=c["resid"][:4]), (None, y[:4]), False, eps=0.0)
    assert not y[4].any()
    assert torch.isinf(y[5]).all()
    assert torch.isnan(y[6]).all()
