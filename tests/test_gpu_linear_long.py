"""kda_lin_prefill with segments as long as those of large calls: each wave forms the decays of a third group of chunks."""

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as K
import linear_ref as R
from gpu_util import bits, dev, log
from test_gpu_linear import cache_of, inputs, run_prefill, split

pytestmark = pytest.mark.gpu

H, HK = 256, 8  # many heads: long segments from few tokens


def segments_written(ws, H, dk, dv):
    """States that a call left in a workspace that was all 0xFF (their decays lie behind them)."""
    states = ws[: ws.numel() // (4 * H * dk * dv) * (4 * H * dk * dv)].view(torch.int32).view(-1, H * dk * dv)
    return int((states != -1).all(1).sum())


@pytest.mark.parametrize("dk,dv,chunks", [(128, 128, 36), (64, 128, 36), (128, 64, 21), (64, 64, 21)])
def test_long_segments(dk, dv, chunks):
    """A row of two segments, each longer than two groups of decays (a chunk per wave: dv / 16 of them), beside a short
    row; decays per token; checkpoints that add a partial chunk to the first segment, to the second, and at their
    border; both types of outputs. Six heads are compared with the recurrence in 64 bits, the others with themselves
    across the calls."""
    group = dv // 16
    lens = [64 * (chunks - 1) + 17, 90]
    n = sum(lens)
    p = inputs(241, n, H, HK, dk, dv, True)
    cache0 = cache_of(11, 2, H, dv, dk)
    slots = np.array([1, 0], np.int32)
    need = K.kda_lin_prefill_workspace(2, n, H, dk, dv)
    heads = torch.tensor([0, 1, 2, 3, H // 2 + 1, H - 2])
    kh = heads // (H // HK)
    q, k, v = split(p, p["x"])
    refs = {}
    for b, at in ((0, 0), (1, lens[0])):
        r = slice(at, at + lens[b])
        args = (q[r][:, kh], k[r][:, kh], v[r][:, heads], p["alpha"][r][:, heads], cache0[slots[b]][heads])
        for c in ({5 * 64 + 13, lens[0] // 64 * 64 - 5 * 64 - 1, lens[0]} if b == 0 else {33}):
            refs[b, c] = R.recur(*args, ckpt=c), R.recur(*args, absolute=True, ckpt=c)
    first = None
    for c in sorted(c for b, c in refs if b == 0):
        for bf16 in (False, True):
            log(f"lin prefill of {chunks} chunks x {H} heads, dk={dk} dv={dv} checkpoint={c} bf16={bf16}")
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev())
            out, cache, ck, err = run_prefill(p, lens, slots, cache0, bf16=bf16, pos=np.array([c, 33], np.int32), workspace=ws)
            assert err == 0
            nseg = segments_written(ws, H, dk, dv)
            assert nseg == 2 and chunks / nseg > 2 * group, (nseg, chunks)
            for b, at, pos in ((0, 0, c), (1, lens[0], 33)):
                (ref, S, atc), (A, SA, atA) = refs[b, pos]
                r = slice(at, at + lens[b])
                # the states' roundings: two per token; a bfloat16 output is the fp32 one rounded (half a step, 2^-8)
                bound = R.roundings(lens[b], dk) * R.U32 * A + (R.UB16 * 1.001 * ref.abs() if bf16 else 0) + 1e-37
                R.check(out[r][:, heads], ref, bound, f"out of row {b}")
                R.check(cache[slots[b]][heads], S, R.roundings(lens[b], 0) * R.U32 * SA + 1e-37, f"state of row {b}")
                R.check(ck[b][heads], atc, R.roundings(pos, 0) * R.U32 * atA + 1e-37, f"checkpoint of row {b}")
            if c == lens[0]:  # no chunk is cut: bfloat16 outputs and the states are those of the fp32 call
                if first is None:
                    first = out, cache, ck
                else:
                    assert np.array_equal(bits(out), bits(first[0].bfloat16()))
                    assert np.array_equal(bits(cache), bits(first[1])) and np.array_equal(bits(ck), bits(first[2]))


@pytest.mark.parametrize("dk,dv,chunks", [(128, 128, 36), (64, 64, 21)])
def test_every_decay_of_a_long_segment_counts(dk, dv, chunks):
    """Decays of 1, 1/2 and 2, one of 1/2 or 2 per chunk at a random token, differing by head; the first token writes and
    every token reads. All products are exact, so each output and the final state show a decay that is missed, taken
    twice or taken from another chunk or head."""
    n = 64 * (chunks - 1) + 17
    g = torch.Generator().manual_seed(7)
    p = inputs(251, n, H, HK, dk, dv, True, decay="ones")
    kw = HK * dk
    x = torch.zeros_like(p["x"])
    x[:, 5: kw: dk] = 1                              # q: channel 5
    x[0, kw + 5: 2 * kw: dk] = 1                     # k: channel 5, the first token only
    x[:, 2 * kw: 2 * kw + H * dv] = p["x"][:, 2 * kw: 2 * kw + H * dv]
    alpha = torch.ones(n, H)
    start = torch.randint(2, (H,), generator=g)  # 1/2 and 2 in turn, so that products stay in range
    for c in range(chunks):
        m = min(64, n - 64 * c)
        at = 64 * c + torch.randint(1 if c == 0 else 0, m, (H,), generator=g)
        alpha[at, torch.arange(H)] = torch.where((c + start) % 2 == 0, 0.5, 2.0)
    gam = alpha[1:].double().cumprod(0)
    want = torch.cat([torch.ones(1, H, dtype=torch.float64), gam])[:, :, None] * \
        x[0, 2 * kw: 2 * kw + H * dv].double().view(1, H, dv)
    need = K.kda_lin_prefill_workspace(1, n, H, dk, dv)
    for bf16 in (False, True):
        log(f"lin prefill, a decay per chunk, dk={dk} dv={dv} bf16={bf16}")
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev())
        out, cache, _, _ = run_prefill(dict(p, x=x, alpha=alpha), [n], np.array([0], np.int32), torch.zeros(1, H, dv, dk),
                                       bf16=bf16, workspace=ws)
        assert chunks / segments_written(ws, H, dk, dv) > 2 * (dv // 16)
        assert torch.equal(out.double(), want)
        state = torch.zeros(H, dv, dk, dtype=torch.float64)
        state[:, :, 5] = want[-1]
        assert torch.equal(cache[0].double(), state)
