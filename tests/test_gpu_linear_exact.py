"""kda_lin_prefill on inputs whose results are known to the last bit, and its bfloat16 outputs against its fp32 ones."""

import numpy as np
import pytest
import torch

from gpu_util import bits, log
from test_gpu_linear import cache_of, inputs, run_prefill, slot_table

pytestmark = pytest.mark.gpu

# Each of the ways in which the library runs a prompt: 16-column workgroups, one workgroup per head, segments
WAYS = [([70, 3, 200], 4, 2), ([70, 3, 200], 72, 8), ([1500, 40, 0, 333], 8, 4)]


@pytest.mark.parametrize("lens,H,Hk", WAYS, ids=str)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_bf16_outputs_are_the_fp32_outputs_rounded(lens, H, Hk, dk, dv):
    """A bfloat16 `out` holds, bit for bit, the fp32 outputs of the same call rounded to nearest even; states and
    checkpoints do not depend on the type of `out` at all."""
    log(f"lin prefill fp32 and bf16 out, lens={lens} H={H} dk={dk} dv={dv}")
    p = inputs(161 + H, sum(lens), H, Hk, dk, dv, True)
    slots = slot_table(6, len(lens), len(lens) + 1)
    pos = np.array([n // 2 for n in lens], np.int32)
    cache0 = cache_of(9, len(lens) + 1, H, dv, dk)
    f = run_prefill(p, lens, slots, cache0, pos=pos)
    b = run_prefill(p, lens, slots, cache0, bf16=True, pos=pos)
    assert np.array_equal(bits(f[1]), bits(b[1])) and np.array_equal(bits(f[2]), bits(b[2]))
    differ = int((bits(b[0]) != bits(f[0].bfloat16())).sum())
    assert differ == 0, f"{differ} of {b[0].numel()} outputs are not the fp32 output rounded"
