"""kda_lin_prefill on inputs whose results are known to the last bit, and its bfloat16 outputs against its fp32 ones."""

import numpy as np
import pytest
import torch

from gpu_util import bits, log
from test_gpu_linear import cache_of, inputs, run_prefill, slot_table

pytestmark = pytest.mark.gpu

# Each of the ways in which the library runs a prompt: 16-column workgroups, one workgroup per head, segments
WAYS = [([70, 3, 200], 4, 2), ([70, 3, 200], 72, 8), ([1500, 40, 0, 333], 8, 4)]
DIMS = [(128, 128), (64, 128), (128, 64), (64, 64)]


@pytest.mark.parametrize("lens,H,Hk", WAYS, ids=str)
@pytest.mark.parametrize("dk,dv", DIMS)
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


def two_parts(x):
    """x as the sum of two bfloat16 values rounded to nearest: what an operand in 16 bits would hold."""
    hi = x.bfloat16().float()
    return hi + (x - hi).bfloat16().float()


def prompt(p, n, k=None, q=None, v=None, alpha=None):
    """p with its tokens, or parts of them, replaced (n tokens and the ones behind the last row)."""
    kw = p["Hk"] * p["dk"]
    x = p["x"].clone()
    for t, lo, w in ((q, 0, kw), (k, kw, kw), (v, 2 * kw, p["H"] * p["dv"])):
        if t is not None:
            x[:n, lo: lo + w] = t.reshape(n, w).bfloat16()
    return dict(p, x=x, alpha=p["alpha"] if alpha is None else alpha)


def one_hot(index, d):
    return torch.nn.functional.one_hot(index, d).float()


@pytest.mark.parametrize("lens,H,Hk", WAYS, ids=str)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_states_are_read_with_all_their_bits(lens, H, Hk, dk, dv):
    """Nothing decays and nothing is written; a token's q picks one channel. Then o is that channel of the state, all 24
    bits of it, and the final state and the checkpoint are the state as it was."""
    n = sum(lens)
    p = inputs(221, n, H, Hk, dk, dv, False, decay="ones")
    pick = torch.randint(dk, (n, Hk), generator=torch.Generator().manual_seed(1))
    p = prompt(p, n, k=torch.zeros(n, Hk, dk), q=one_hot(pick, dk))
    slots = slot_table(2, len(lens), len(lens) + 1)
    pos = np.array([m // 2 for m in lens], np.int32)
    cache0 = cache_of(9, len(lens) + 1, H, dv, dk)
    assert (two_parts(cache0) != cache0).float().mean() > 0.9  # 16 bits would not do
    for bf16 in (False, True):
        log(f"lin prefill reading states, lens={lens} H={H} dk={dk} dv={dv} bf16={bf16}")
        out, cache, ck, err = run_prefill(p, lens, slots, cache0, bf16=bf16, pos=pos)
        assert err == 0 and np.array_equal(bits(cache), bits(cache0))
        at = 0
        for b, m in enumerate(lens):
            assert np.array_equal(bits(ck[b]), bits(cache0[slots[b]]))
            S = cache0[slots[b]]  # [H, dv, dk]
            c = pick[at: at + m].repeat_interleave(H // Hk, 1)  # [m, H]
            want = torch.gather(S.expand(m, H, dv, dk), 3, c[:, :, None, None].expand(m, H, dv, 1))[..., 0]
            assert np.array_equal(bits(out[at: at + m]), bits(want.bfloat16() if bf16 else want)), b
            at += m


@pytest.mark.parametrize("lens,H,Hk", WAYS, ids=str)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("gap", [1, 7, 20, 50, 100])
def test_decays_reach_scores_and_states_with_all_their_bits(lens, H, Hk, dk, dv, gap):
    """One token of a row writes powers of two, every other k is 0; one later token's decay is a fraction of 24 bits, a
    few others' are 1/2, the rest are 1. Every product is then exact: inside a chunk (the decayed score) and across
    chunks (the state), an output is the value times the decays since, to the last bit, and so is the final state."""
    n = sum(lens)
    g = torch.Generator().manual_seed(gap)
    p = inputs(231, n, H, Hk, dk, dv, True, decay="ones")
    c0 = torch.randint(dk, (1, Hk), generator=g)
    q = one_hot(c0.expand(n, Hk), dk)
    k = torch.zeros(n, Hk, dk)
    v = torch.exp2(torch.randint(-3, 4, (n, H, dv), generator=g).float()) * (1 - 2 * torch.randint(2, (n, H, dv), generator=g))
    alpha = torch.where(torch.rand(n, H, generator=g) < 0.02, 0.5, 1.0)
    want = torch.zeros(n, H, dv)
    state = torch.zeros(len(lens), H, dv, dk)
    at = 0
    for b, m in enumerate(lens):
        if m:
            s = at + m // 3  # the token that writes
            k[s] = one_hot(c0[0], dk)
            if m // 3 + gap < m:
                alpha[s + gap] = 0.5 + 0.5 * torch.rand(H, generator=g)
                assert (two_parts(alpha[s + gap]) != alpha[s + gap]).any()
            x = v[s].clone()
            for t in range(s, at + m):
                if t > s:
                    x = x * alpha[t][:, None]  # exact: a 24-bit fraction once, powers of two otherwise
                want[t] = x
            state[b].scatter_(2, c0[0].repeat_interleave(H // Hk)[:, None, None].expand(H, dv, 1), x[:, :, None])
        at += m
    p = prompt(p, n, k=k, q=q, v=v, alpha=alpha)
    slots = np.arange(len(lens), dtype=np.int32)
    for bf16 in (False, True):
        log(f"lin prefill of one written token, lens={lens} H={H} dk={dk} dv={dv} gap={gap} bf16={bf16}")
        out, cache, _, err = run_prefill(p, lens, slots, torch.zeros(len(lens), H, dv, dk), bf16=bf16)
        assert err == 0
        assert torch.equal(out[:n], want.bfloat16() if bf16 else want)
        assert torch.equal(cache, state)


@pytest.mark.parametrize("H", [2, 80])
def test_small_values(H):
    """bfloat16 inputs below fp32's normal range are not flushed; states are read to 2^-133, the smallest bfloat16, and
    kept as they are."""
    n, d = 70, 128
    p = inputs(261, n, H, H, d, d, False, decay="ones")
    q = torch.zeros(n, H, d)
    e = torch.arange(n) % 10 - 133
    q[torch.arange(n), :, 5] = torch.exp2(e.double()).float()[:, None]
    log(f"lin prefill with q down to 2^-133, H={H}")
    out, cache, _, _ = run_prefill(prompt(p, n, k=torch.zeros(n, H, d), q=q), [n], np.array([0], np.int32),
                                   torch.full((1, H, d, d), 2.0 ** 100))
    assert torch.equal(out, torch.exp2(e + 100.0)[:, None, None].expand(n, H, d)) and bool((cache == 2.0 ** 100).all())
    g = torch.Generator().manual_seed(3)
    S = ((1 + torch.rand(1, H, d, d, generator=g)).double() * torch.exp2(-100.0 - torch.randint(40, (1, H, d, d), generator=g))).float()
    pick = torch.arange(n) % d
    q = one_hot(pick[:, None].expand(n, H), d)
    log(f"lin prefill with states down to 2^-139, H={H}")
    out, cache, _, _ = run_prefill(prompt(p, n, k=torch.zeros(n, H, d), q=q), [n], np.array([0], np.int32), S)
    want = S[0, :, :, pick].permute(2, 0, 1)
    assert torch.equal(cache, S)
    assert float((out.double() - want.double()).abs().max()) < 2.0 ** -133
    big = want >= 2.0 ** -109
    assert torch.equal(out[big], want[big])
