"""Linear attention with a decay per head against the plain 64-bit recurrence (linear_ref.py), at the sizes,
layouts and positions where it can go wrong."""

import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as K
import linear_ref as R
from gpu_util import SENTINEL_BITS, bits, dev, i32, log, sentinel

pytestmark = pytest.mark.gpu


def inputs(seed, n, H, Hk, dk, dv, per_token, fused=False, decay="mixed"):
    """CPU tensors of n tokens; fused: q, k, v are slices of one [n, Hk dk + Hk dk + H dv + 8] array."""
    g = torch.Generator().manual_seed(seed)
    w = 2 * Hk * dk + H * dv + 8
    x = torch.randn(n, w, generator=g)
    x[:, : 2 * Hk * dk] /= dk ** 0.5
    x = x.bfloat16()
    u = torch.rand(n, H, generator=g) if per_token else torch.rand(H, generator=g)
    if decay == "mixed":
        # one head in four keeps nearly everything, one forgets within a few tokens
        h = torch.arange(H) % 4
        a = torch.where(h == 0, 1 - 1e-4 * u, torch.where(h == 1, u, torch.where(h == 2, 0.9 + 0.1 * u, 0.5 + 0.5 * u)))
    elif decay == "zeros":
        a = torch.where(u < 0.2, torch.zeros(()), torch.where(u < 0.4, torch.full((), 1e-30), u))
    elif decay == "signed":
        a = 2 * u - 1
    else:
        a = torch.ones_like(u)
    return dict(x=x, Hk=Hk, dk=dk, dv=dv, H=H, alpha=a.float(), fused=fused)


def split(p, x):
    """(q, k, v) of the projection rows x: slices where fused, contiguous copies otherwise."""
    n, kw = x.shape[0], p["Hk"] * p["dk"]
    q = x[:, :kw].unflatten(1, (p["Hk"], p["dk"]))
    k = x[:, kw: 2 * kw].unflatten(1, (p["Hk"], p["dk"]))
    v = x[:, 2 * kw: 2 * kw + p["H"] * p["dv"]].unflatten(1, (p["H"], p["dv"]))
    return (q, k, v) if p["fused"] else (q.contiguous(), k.contiguous(), v.contiguous())


def cache_of(seed, slots, H, dv, dk):
    return torch.randn(slots, H, dv, dk, generator=torch.Generator().manual_seed(seed))


def slot_table(seed, B, slots):
    return np.random.default_rng(seed).permutation(slots)[:B].astype(np.int32)


SHAPES = [(1, 1, 1, 64, 64), (1, 32, 32, 128, 128), (3, 6, 2, 128, 64), (5, 5, 1, 64, 128), (13, 24, 8, 64, 128),
          (33, 32, 8, 128, 128)]


@pytest.mark.parametrize("B,H,Hk,dk,dv", SHAPES)
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_decode(B, H, Hk, dk, dv, per_token, bf16):
    log(f"lin decode B={B} H={H} Hk={Hk} dk={dk} dv={dv} per_token={per_token} bf16={bf16}")
    p = inputs(B + H, B, H, Hk, dk, dv, per_token, fused=bf16)
    cache0 = cache_of(7, B + 2, H, dv, dk)
    slots = slot_table(3, B, B + 2)
    if B > 2:
        slots[1] = -1
    q, k, v = split(p, p["x"])
    qd, kd, vd = split(p, p["x"].to(dev()))
    cache = cache0.to(dev())
    out = sentinel((B, H, dv)) if not bf16 else torch.full((B, H, dv), 7.0, dtype=torch.bfloat16, device=dev())
    before = bits(out)
    K.kda_lin_decode_step(cache, i32(slots), qd, kd, vd, p["alpha"].to(dev()), out)
    torch.cuda.synchronize()
    for b in range(B):
        if slots[b] < 0:
            assert np.array_equal(bits(out)[b], before[b])
            continue
        al = p["alpha"][b: b + 1] if per_token else p["alpha"]
        args = (q[b: b + 1], k[b: b + 1], v[b: b + 1], al, cache0[slots[b]])
        ref, S, _ = R.recur(*args)
        A, SA, _ = R.recur(*args, absolute=True)
        # a step rounds the decayed state and the sum (2 u), a read-out dot at most 16 times more
        R.check(out[b], ref[0], 18 * R.U32 * A[0] + (R.UB16 * 1.001 * ref[0].abs() if bf16 else 0) + 1e-37, f"out {b}")
        R.check(cache[slots[b]], S, 2 * R.U32 * SA + 1e-37, f"state {b}")
    rest = np.setdiff1d(np.arange(B + 2), slots)
    assert np.array_equal(bits(cache)[rest], cache0.numpy().view(np.uint32)[rest])


@pytest.mark.parametrize("H,Hk,dk,dv,bf16,weighted", [(4, 2, 64, 64, False, True), (3, 3, 128, 128, True, True),
                                                      (8, 1, 64, 128, True, False), (6, 2, 128, 64, False, True)])
def test_decode_gate(H, Hk, dk, dv, bf16, weighted):
    B = 4
    log(f"lin decode gated H={H} dk={dk} dv={dv} bf16={bf16}")
    p = inputs(5, B, H, Hk, dk, dv, True)
    g = torch.Generator().manual_seed(9)
    gate = (3 * torch.randn(B, H, dv, generator=g)).bfloat16()
    weight = torch.randn(dv, generator=g) if weighted else None
    cache0 = cache_of(8, B, H, dv, dk)
    slots = np.array([2, 0, 3, 1], np.int32)
    q, k, v = split(p, p["x"])
    cache = cache0.to(dev())
    out = torch.zeros(B, H, dv, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    K.kda_lin_decode_step(cache, i32(slots), q.to(dev()), k.to(dev()), v.to(dev()), p["alpha"].to(dev()), out,
                          gate=gate.to(dev()), weight=weight.to(dev()) if weighted else None, eps=1e-5)
    torch.cuda.synchronize()
    for b in range(B):
        args = (q[b: b + 1], k[b: b + 1], v[b: b + 1], p["alpha"][b: b + 1], cache0[slots[b]])
        o, S, _ = R.recur(*args)
        A, SA, _ = R.recur(*args, absolute=True)
        y = R.gated(o[0], gate[b], weight, 1e-5)
        # the error of o (18 u A) scales with y / o; the norm's relative error is that of the vector plus
        # at most 64 u of its own (a mean of dv terms, a root, a reciprocal, an exponential, products)
        f = 1 / ((o[0] ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
        eo = 18 * R.U32 * A[0]
        wg = (weight.double().abs() if weighted else 1.0) / (1 + torch.exp(-gate[b].double()))
        bound = eo * f * wg * 1.01 + (64 * R.U32 + 1.01 * (eo ** 2).mean(-1, keepdim=True).sqrt() * f) * y.abs() + 1e-37
        if bf16:
            bound = bound + R.UB16 * 1.001 * y.abs()
        R.check(out[b], y, bound, f"gated out {b}")
        R.check(cache[slots[b]], S, 2 * R.U32 * SA + 1e-37, f"state {b}")


@pytest.mark.parametrize("dk,dv,B,H", [(128, 128, 2, 3), (64, 128, 2, 3), (128, 64, 2, 3), (64, 64, 40, 32)])
def test_decode_widths_agree_bit_for_bit(dk, dv, B, H):
    p = inputs(11, B, H, H, dk, dv, True)
    cache0 = cache_of(12, B, H, dv, dk).to(dev())
    qkv = [t.to(dev()) for t in split(p, p["x"])]
    al = p["alpha"].to(dev())
    ref = None
    for w in (0, 4, 8, 16, 32, 64, 128):
        if w > dv:
            with pytest.raises(K.KdaError):
                K.kda_lin_decode_step(cache0, i32(np.arange(B)), *qkv, al, torch.empty(B, H, dv, device=dev()), tile_w=w)
            continue
        log(f"lin decode width {w} dk={dk} dv={dv}")
        cache, out = cache0.clone(), torch.empty(B, H, dv, device=dev())
        K.kda_lin_decode_step(cache, i32(np.arange(B)), *qkv, al, out, tile_w=w)
        torch.cuda.synchronize()
        got = (bits(out), bits(cache))
        if ref is None:
            ref = got
        assert all(np.array_equal(x, y) for x, y in zip(got, ref)), w


def run_prefill(p, lens, slots, cache0, *, bf16=False, pos=None, extra=0, stream=None, workspace=None):
    """(out, cache, ckpt, dev_err) on the CPU; `extra` tokens of the arrays lie behind the last row."""
    B, H, dv, dk = len(lens), p["H"], p["dv"], p["dk"]
    q, k, v = split(p, p["x"].to(dev()))
    cache = cache0.to(dev())
    n = p["x"].shape[0]
    out = torch.full((n, H, dv), 7.0, dtype=torch.bfloat16, device=dev()) if bf16 else sentinel((n, H, dv))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ck = sentinel((B, H, dv, dk)) if pos is not None else None
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    K.kda_lin_prefill(cache, i32(slots), i32(cu), q, k, v, p["alpha"].to(dev()), out,
                      ckpt_pos=i32(pos) if pos is not None else None, ckpt=ck, dev_err=err, stream=stream,
                      workspace=workspace)
    torch.cuda.synchronize()
    return out.cpu(), cache.cpu(), ck.cpu() if ck is not None else None, int(err.item())


def check_prefill(p, lens, slots, cache0, got, *, bf16=False, pos=None, skip=()):
    out, cache, ck, err = got
    q, k, v = split(p, p["x"])
    per_token = p["alpha"].dim() == 2
    cu = np.concatenate([[0], np.cumsum(lens)])
    untouched = bits(torch.full((1,), 7.0, dtype=torch.bfloat16))[0] if bf16 else SENTINEL_BITS
    for b, n in enumerate(lens):
        r = slice(int(cu[b]), int(cu[b + 1]))
        if slots[b] < 0 or b in skip:
            assert np.all(bits(out[r]) == untouched), f"out of skipped row {b}"
            if pos is not None:
                assert np.all(bits(ck[b]) == SENTINEL_BITS)
            continue
        al = p["alpha"][r] if per_token else p["alpha"]
        c = -1 if pos is None else int(pos[b])
        args = (q[r], k[r], v[r], al, cache0[slots[b]])
        ref, S, at = R.recur(*args, ckpt=c)
        A, SA, atA = R.recur(*args, absolute=True, ckpt=c)
        R.check(out[r], ref, R.out_bound(A, n, p["dk"], ref, bf16), f"out of row {b} ({n} tokens)")
        R.check(cache[slots[b]], S, R.roundings(n, 0) * R.U32 * SA + 1e-37, f"state of row {b} ({n} tokens)")
        if n == 0:
            assert torch.equal(cache[slots[b]], cache0[slots[b]])
        if pos is not None and c >= 0:
            R.check(ck[b], at, R.roundings(c, 0) * R.U32 * atA + 1e-37, f"checkpoint of row {b} (after {c} of {n})")
        elif pos is not None:
            assert np.all(bits(ck[b]) == SENTINEL_BITS)
    assert np.all(bits(out[int(cu[-1]):]) == untouched), "out behind the last row"
    live = [s for b, s in enumerate(slots) if s >= 0 and b not in skip]
    rest = np.setdiff1d(np.arange(cache0.shape[0]), live)
    assert np.array_equal(bits(cache)[rest], bits(cache0)[rest]), "slots of no row"


LENS = [[1], [0, 1, 2, 3], [15, 16, 17], [31, 32, 33], [63, 64, 65], [127, 0, 129, 1], [300], [200, 5, 64, 131]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,Hk,dk,dv,per_token,bf16", [
    (2, 2, 128, 128, True, False), (6, 2, 64, 128, False, True), (3, 1, 128, 64, True, True), (4, 4, 64, 64, False, False),
    # more than 512 (row, head, 16 columns): the kernel of whole heads
    (72, 8, 128, 128, True, True), (80, 16, 64, 128, False, False), (136, 8, 128, 64, True, False),
    (132, 132, 64, 64, True, True)])
def test_prefill(lens, H, Hk, dk, dv, per_token, bf16):
    log(f"lin prefill lens={lens} H={H} Hk={Hk} dk={dk} dv={dv} per_token={per_token} bf16={bf16}")
    p = inputs(sum(lens) + H, sum(lens) + 3, H, Hk, dk, dv, per_token, fused=bf16)
    slots = slot_table(1, len(lens), len(lens) + 2)
    cache0 = cache_of(2, len(lens) + 2, H, dv, dk)
    got = run_prefill(p, lens, slots, cache0, bf16=bf16)
    assert got[3] == 0
    check_prefill(p, lens, slots, cache0, got, bf16=bf16)


@pytest.mark.parametrize("decay", ["zeros", "signed", "ones"])
@pytest.mark.parametrize("dk,dv,H", [(128, 128, 8), (64, 64, 8), (128, 128, 24), (64, 64, 48)])
def test_prefill_decays(decay, dk, dv, H):
    """Decays that forget the state outright, underflow inside a chunk, change sign, or keep everything."""
    lens = [130, 70, 16]
    log(f"lin prefill decays={decay} dk={dk} H={H}")
    p = inputs(17, sum(lens), H, 4, dk, dv, True, decay=decay)
    slots = slot_table(1, 3, 4)
    cache0 = cache_of(2, 4, H, dv, dk)
    got = run_prefill(p, lens, slots, cache0)
    check_prefill(p, lens, slots, cache0, got)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("H", [1, 4, 24])
@pytest.mark.parametrize("long", [False, True])
def test_prefill_checkpoints(dk, dv, H, long):
    """Checkpoints before, at and after chunk edges, at both ends of a row, in empty and padding rows."""
    lens = [70, 200, 64, 128, 1, 0, 0, 333, 40, 65, 129]
    pos = np.array([1, 63, 64, 65, 1, 0, -1, 256, 0, 65, 127], np.int32)
    if not long:  # up to 640 tokens
        lens, pos = lens[:6] + [0, 40, 65], np.array([1, 63, 64, 65, 1, 0, -1, 0, 65], np.int32)
    slots = slot_table(4, len(lens), len(lens) + 1)
    slots[lens.index(40)] = -1
    log(f"lin prefill checkpoints dk={dk} H={H} {sum(lens)} tokens")
    p = inputs(23, sum(lens), H, H, dk, dv, True)
    cache0 = cache_of(2, len(lens) + 1, H, dv, dk)
    got = run_prefill(p, lens, slots, cache0, pos=pos)
    assert got[3] == 0
    check_prefill(p, lens, slots, cache0, got, pos=pos)


@pytest.mark.parametrize("lens,H,Hk,per_token,dk", [([2500], 2, 1, True, 128), ([1300, 40, 700, 0, 1], 4, 4, False, 128),
                                                    ([1800], 1, 1, False, 64), ([5, 1500], 8, 2, True, 64)])
def test_prefill_long(lens, H, Hk, per_token, dk):
    """Rows long enough to be shared by several workgroups, checkpoints in the middle of one."""
    pos = np.array([n * 24 // 25 // 32 * 32 if n > 40 else -1 for n in lens], np.int32)
    log(f"lin prefill long lens={lens} H={H} per_token={per_token} dk={dk}")
    p = inputs(31, sum(lens) + 2, H, Hk, dk, dk, per_token, fused=True)
    slots = slot_table(4, len(lens), len(lens) + 1)
    cache0 = cache_of(2, len(lens) + 1, H, dk, dk)
    got = run_prefill(p, lens, slots, cache0, pos=pos)
    assert got[3] == 0
    check_prefill(p, lens, slots, cache0, got, pos=pos)


def test_prefill_checkpoint_without_tokens():
    """n_tok = 0: every row is empty and its checkpoint is the state as it was."""
    p = inputs(1, 0, 2, 2, 64, 64, True)
    cache0 = cache_of(2, 3, 2, 64, 64)
    pos = np.array([0, -1, 0], np.int32)
    got = run_prefill(p, [0, 0, 0], np.array([1, 0, 2], np.int32), cache0, pos=pos)
    assert got[3] == 0
    check_prefill(p, [0, 0, 0], np.array([1, 0, 2], np.int32), cache0, got, pos=pos)


@pytest.mark.parametrize("H", [3, 24])
def test_prefill_row_errors_skip_the_row(H):
    """A slot past the cache, a decreasing range, one past n_tok, a checkpoint past the row: the bit is set,
    the row is skipped in full, the others are right."""
    dk, dv = 128, 128
    lens = [40, 50, 70]
    p = inputs(41, sum(lens), H, 1, dk, dv, True)
    cache0 = cache_of(2, 5, H, dv, dk)
    for slots, pos, bit in ((np.array([0, 5, 2], np.int32), np.array([3, -1, 70], np.int32), K.KDA_DEVERR_SLOT),
                            (np.array([0, 4, 2], np.int32), np.array([3, 51, 70], np.int32), K.KDA_DEVERR_CKPT)):
        log(f"lin prefill row error bit {bit}")
        got = run_prefill(p, lens, slots, cache0, pos=pos)
        assert got[3] == bit
        check_prefill(p, lens, slots, cache0, got, pos=pos, skip=(1,))
    q, k, v = split(p, p["x"].to(dev()))
    for cu in ([0, 40, 30, 160], [0, 40, 90, 161], [-1, 40, 90, 160]):
        cache, out = cache0.to(dev()), sentinel((160, H, dv))
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        log(f"lin prefill cu={cu}")
        K.kda_lin_prefill(cache, i32([0, 1, 2]), i32(cu), q, k, v, p["alpha"].to(dev()), out, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == K.KDA_DEVERR_SEQLEN
        for b in range(3):
            a0, a1 = cu[b], cu[b + 1]
            if a0 < 0 or a1 < a0 or a1 > 160:
                assert torch.equal(cache[b].cpu(), cache0[b])
                continue
            r = slice(a0, a1)
            args = (split(p, p["x"])[0][r], split(p, p["x"])[1][r], split(p, p["x"])[2][r], p["alpha"][r], cache0[b])
            _, S, _ = R.recur(*args)
            _, SA, _ = R.recur(*args, absolute=True)
            R.check(cache[b], S, R.roundings(a1 - a0, 0) * R.U32 * SA + 1e-37, f"state of row {b}")


def test_decode_row_errors():
    p = inputs(3, 3, 2, 2, 64, 64, True)
    cache0 = cache_of(2, 3, 2, 64, 64)
    q, k, v = (t.to(dev()) for t in split(p, p["x"]))
    cache, out = cache0.to(dev()), sentinel((3, 2, 64))
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    log("lin decode slot past the cache")
    K.kda_lin_decode_step(cache, i32([0, 3, -1]), q, k, v, p["alpha"].to(dev()), out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.KDA_DEVERR_SLOT
    assert np.all(bits(out)[1:] == SENTINEL_BITS) and not np.any(bits(out)[0] == SENTINEL_BITS)
    assert torch.equal(cache[1:].cpu(), cache0[1:])


@pytest.mark.parametrize("H", [4, 24])
def test_nonfinite_inputs_stay_in_their_row_and_head(H):
    """NaN and infinity in the tokens, decays and state of one row and head leave every other row and head the
    bits they have without them."""
    lens, d = [70, 66, 150], 128
    p = inputs(51, sum(lens) + 1, H, H, d, d, True)
    cache0 = cache_of(2, 4, H, d, d)
    slots = np.array([3, 1, 0], np.int32)
    clean = run_prefill(p, lens, slots, cache0)
    x, al, c = p["x"].clone(), p["alpha"].clone(), cache0.clone()
    kw = H * d
    x[75, kw + 2 * d: kw + 3 * d] = float("nan")  # k of row 1, head 2
    x[80, 2 * d] = float("inf")                   # q
    x[90, 2 * kw + 2 * d] = float("-inf")         # v
    al[100, 2] = float("nan")
    c[1, 2] = float("inf")
    x[286] = float("nan")                         # the token behind the last row
    log("lin prefill with non-finite values in row 1, head 2")
    got = run_prefill(dict(p, x=x, alpha=al), lens, slots, c)
    for b, (o, n) in enumerate(zip((0, 70, 136), lens)):
        for h in range(H):
            if (b, h) == (1, 2):
                assert not torch.isfinite(got[0][o: o + n, h]).all()
                continue
            assert np.array_equal(bits(got[0][o: o + n, h]), bits(clean[0][o: o + n, h])), (b, h)
            assert np.array_equal(bits(got[1][slots[b], h]), bits(clean[1][slots[b], h])), (b, h)


@pytest.mark.parametrize("T,H,Hk", [(150, 4, 2), (150, 72, 8), (700, 2, 2)])
def test_prefill_matches_decode_steps(T, H, Hk):
    """A prompt in one call (each of the ways in which the library runs one), and the same tokens one call each."""
    d = 128
    p = inputs(61, T, H, Hk, d, d, True)
    cache0 = cache_of(2, 2, H, d, d)
    one = run_prefill(p, [T], np.array([1], np.int32), cache0)
    q, k, v = (t.to(dev()) for t in split(p, p["x"]))
    cache, out, al = cache0.to(dev()), torch.empty(T, H, d, device=dev()), p["alpha"].to(dev())
    s = i32([1])
    log(f"lin decode, {T} steps")
    for t in range(T):
        K.kda_lin_decode_step(cache, s, q[t: t + 1], k[t: t + 1], v[t: t + 1], al[t: t + 1], out[t: t + 1])
    torch.cuda.synchronize()
    args = tuple(t.cpu() for t in (q, k, v, al)) + (cache0[1],)
    A, SA, _ = R.recur(*args, absolute=True)
    c = R.roundings(T, d) * R.U32
    R.check(out, one[0].double(), 2 * c * A, "outputs")
    R.check(cache[1], one[1][1].double(), 2 * c * SA, "state")


def test_prefill_resumes():
    """A prompt in two calls, the second from the state the first left, against one call."""
    n, cut, H, d = 300, 117, 2, 64
    p = inputs(71, n, H, H, d, d, True)
    cache0 = cache_of(2, 1, H, d, d)
    s0 = np.array([0], np.int32)
    one = run_prefill(p, [n], s0, cache0)
    a = run_prefill(dict(p, x=p["x"][:cut], alpha=p["alpha"][:cut]), [cut], s0, cache0)
    b = run_prefill(dict(p, x=p["x"][cut:], alpha=p["alpha"][cut:]), [n - cut], s0, a[1])
    q, k, v = split(p, p["x"])
    A, SA, _ = R.recur(q, k, v, p["alpha"], cache0[0], absolute=True)
    c = 2 * R.roundings(n, d) * R.U32
    R.check(torch.cat([a[0], b[0]]), one[0].double(), c * A, "outputs")
    R.check(b[1][0], one[1][0].double(), c * SA, "state")


def test_repeats_bit_for_bit_and_on_another_stream():
    lens = [1000, 3, 260]
    p = inputs(81, sum(lens), 8, 2, 128, 128, True, fused=True)
    cache0 = cache_of(2, 3, 8, 128, 128)
    slots = np.array([2, 0, 1], np.int32)
    a = run_prefill(p, lens, slots, cache0)
    b = run_prefill(p, lens, slots, cache0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    c = run_prefill(p, lens, slots, cache0, stream=side)
    for other in (b, c):
        assert np.array_equal(bits(a[0]), bits(other[0])) and np.array_equal(bits(a[1]), bits(other[1]))


def test_workspace_given_by_the_caller():
    lens = [3000, 200]
    p = inputs(91, sum(lens), 2, 2, 128, 128, False)
    cache0 = cache_of(2, 2, 2, 128, 128)
    slots = np.array([1, 0], np.int32)
    need = K.kda_lin_prefill_workspace(2, sum(lens), 2, 128, 128)
    a = run_prefill(p, lens, slots, cache0)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=dev())
    b = run_prefill(p, lens, slots, cache0, workspace=ws)
    assert np.array_equal(bits(a[0]), bits(b[0])) and np.array_equal(bits(a[1]), bits(b[1]))
    assert bool((ws[need:] == 0xFF).all())
    if need:
        with pytest.raises(K.KdaError) as e:
            run_prefill(p, lens, slots, cache0, workspace=ws[: need - 1])
        assert e.value.status == K.KDA_ERR_INVALID


def test_overlapping_rows_are_run_or_reported():
    """A table whose rows overlap (each range valid by itself) asks for more segments than the library plans for:
    every row either has its right state or is left alone and reported."""
    n, H, d, B = 2000, 2, 64, 9
    p = inputs(95, n, H, H, d, d, True)
    cache0 = cache_of(2, B, H, d, d)
    q, k, v = split(p, p["x"].to(dev()))
    cu = [0, n] * 5  # even rows [0, n), odd rows decreasing
    cache, out = cache0.to(dev()), torch.empty(n, H, d, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    log("lin prefill with overlapping rows")
    K.kda_lin_prefill(cache, i32(np.arange(B)), i32(cu), q, k, v, p["alpha"].to(dev()), out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.KDA_DEVERR_SEQLEN
    ran = 0
    for b in range(B):
        if torch.equal(cache[b].cpu(), cache0[b]):
            continue
        assert b % 2 == 0
        args = split(p, p["x"]) + (p["alpha"], cache0[b])
        _, S, _ = R.recur(*args)
        _, SA, _ = R.recur(*args, absolute=True)
        R.check(cache[b], S, R.roundings(n, 0) * R.U32 * SA + 1e-37, f"state of row {b}")
        ran += 1
    assert ran >= 1


def test_many_rows():
    """More rows than a wave has lanes: the search for a workgroup's row goes on past the first 64."""
    lens = [(7 * b) % 90 for b in range(150)]
    lens[97] = 900
    H, d = 2, 64
    pos = np.array([n // 2 if b % 3 else -1 for b, n in enumerate(lens)], np.int32)
    p = inputs(96, sum(lens), H, 1, d, d, True)
    slots = slot_table(5, len(lens), len(lens))
    cache0 = cache_of(2, len(lens), H, d, d)
    log(f"lin prefill with {len(lens)} rows")
    got = run_prefill(p, lens, slots, cache0, pos=pos)
    assert got[3] == 0
    check_prefill(p, lens, slots, cache0, got, pos=pos)


def test_offsets_past_32_bits():
    """States and tokens that start more than 2^31 elements into their arrays."""
    H, d, n = 2, 128, 70
    stride = H * d * d
    slots = (1 << 31) // stride + 2
    big = torch.empty(slots, H, d, d, device=dev())
    last = slots - 1
    p = inputs(101, n, H, 1, d, d, True)
    S0 = cache_of(2, 1, H, d, d)
    big[last] = S0[0].to(dev())
    q, k, v = (t.to(dev()) for t in split(p, p["x"]))
    out = torch.empty(n, H, d, device=dev())
    log("lin prefill and decode at a slot past 2^31 elements")
    K.kda_lin_prefill(big, i32([last]), i32([0, n]), q, k, v, p["alpha"].to(dev()), out)
    args = split(p, p["x"]) + (p["alpha"], S0[0])
    ref, S, _ = R.recur(*args)
    A, SA, _ = R.recur(*args, absolute=True)
    R.check(out, ref, R.out_bound(A, n, d, ref, False), "out")
    R.check(big[last], S, R.roundings(n, 0) * R.U32 * SA, "state")
    one = torch.empty(1, H, d, device=dev())
    K.kda_lin_decode_step(big, i32([last]), q[:1], k[:1], v[:1], p["alpha"][:1].to(dev()), one)
    ref2, _, _ = R.recur(split(p, p["x"])[0][:1], split(p, p["x"])[1][:1], split(p, p["x"])[2][:1], p["alpha"][:1], S)
    A2, _, _ = R.recur(split(p, p["x"])[0][:1], split(p, p["x"])[1][:1], split(p, p["x"])[2][:1], p["alpha"][:1], SA,
                       absolute=True)
    R.check(one, ref2, R.out_bound(A2, n + 1, d, ref2, False), "out of the step after it")
    del big
    # tokens: a skipped row of 270,000 tokens in front, 64 heads of 128: 2^31 elements of v and out before the live one
    H, lead = 64, 270000
    n = 33
    v = torch.zeros(lead + n, H, d, dtype=torch.bfloat16, device=dev())
    q = torch.zeros(lead + n, 1, d, dtype=torch.bfloat16, device=dev())
    p = inputs(102, n, H, 1, d, d, False)
    qs, ks, vs = split(p, p["x"])
    k = torch.zeros_like(q)
    q[lead:], k[lead:], v[lead:] = qs.to(dev()), ks.to(dev()), vs.to(dev())
    out = torch.zeros(lead + n, H, d, dtype=torch.bfloat16, device=dev())
    S0 = cache_of(3, 1, H, d, d)
    cache = S0.to(dev())
    log("lin prefill at tokens past 2^31 elements")
    K.kda_lin_prefill(cache, i32([-1, 0]), i32([0, lead, lead + n]), q, k, v, p["alpha"].to(dev()), out)
    ref, S, _ = R.recur(qs, ks, vs, p["alpha"], S0[0])
    A, SA, _ = R.recur(qs, ks, vs, p["alpha"], S0[0], absolute=True)
    R.check(out[lead:], ref, R.out_bound(A, n, d, ref, True), "out")
    R.check(cache[0], S, R.roundings(n, 0) * R.U32 * SA, "state")
    assert int(out[:lead].count_nonzero()) == 0


def test_state_transfer_moves_linear_states():
    """kda_state_pack / kda_state_unpack carry a linear-attention state to another cache; the next step there
    gives the same bits."""
    H, d = 4, 128
    p = inputs(111, 2, H, H, d, d, True)
    a = cache_of(2, 2, H, d, d).to(dev())
    b = torch.zeros(3, H, d, d, device=dev())
    q, k, v = (t.to(dev()) for t in split(p, p["x"]))
    al = p["alpha"].to(dev())
    buf, o1, o2 = torch.empty(1, H, d, d, device=dev()), torch.empty(1, H, d, device=dev()), torch.empty(1, H, d, device=dev())
    log("lin decode, state transfer, lin decode")
    K.kda_lin_decode_step(a, i32([1]), q[:1], k[:1], v[:1], al[:1], o1)
    K.kda_state_pack(a, i32([1]), buf)
    K.kda_state_unpack(b, i32([2]), buf)
    K.kda_lin_decode_step(a, i32([1]), q[1:], k[1:], v[1:], al[1:], o1)
    K.kda_lin_decode_step(b, i32([2]), q[1:], k[1:], v[1:], al[1:], o2)
    torch.cuda.synchronize()
    assert np.array_equal(bits(o1), bits(o2)) and np.array_equal(bits(a[1]), bits(b[2]))


def test_graph_replays_match_eager():
    """A prompt and eight steps in one HIP graph: every replay against the eager run, with eager work between."""
    H, d, T, steps = 8, 128, 1100, 8
    p = inputs(121, T + steps, H, 4, d, d, True)
    cache0 = cache_of(2, 2, H, d, d).to(dev())
    cache = cache0.clone()
    q, k, v = (t.to(dev()) for t in split(p, p["x"]))
    al = p["alpha"].to(dev())
    out = torch.zeros(T + steps, H, d, device=dev())
    cu, s = i32([0, T]), i32([1])

    def work():
        K.kda_lin_prefill(cache, s, cu, q[:T], k[:T], v[:T], al[:T], out[:T])
        for t in range(T, T + steps):
            K.kda_lin_decode_step(cache, s, q[t: t + 1], k[t: t + 1], v[t: t + 1], al[t: t + 1], out[t: t + 1])

    log("lin graph: eager")
    work()
    torch.cuda.synchronize()
    ref = (bits(out), bits(cache))
    cache.copy_(cache0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    log("lin graph: capture")
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            work()
    torch.cuda.current_stream().wait_stream(stream)
    for r in range(4):
        cache.copy_(cache0)
        out.zero_()
        torch.cuda.synchronize()
        log(f"lin graph: replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), ref[0]) and np.array_equal(bits(cache), ref[1]), f"replay {r}"
        cache.copy_(cache0)
        work()  # eager work between the replays
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), ref[0]), f"eager after replay {r}"


def test_two_threads_on_two_streams():
    """Calls of two threads at once, each on its stream with a workspace of its own, agree with the same calls alone."""
    dims = [([3000, 70], 4, 2, 128, 128), ([900, 2200], 8, 8, 64, 64)]
    jobs = []
    for i, (lens, H, Hk, dk, dv) in enumerate(dims):
        p = inputs(131 + i, sum(lens), H, Hk, dk, dv, True)
        q, k, v = (t.to(dev()) for t in split(p, p["x"]))
        cache0 = cache_of(5 + i, 2, H, dk, dv).to(dev())
        assert K.kda_lin_prefill_workspace(2, sum(lens), H, dk, dv) > 0
        jobs.append(dict(cache0=cache0, slots=i32([1, 0]), cu=i32(np.concatenate([[0], np.cumsum(lens)])), q=q, k=k, v=v,
                         al=p["alpha"].to(dev()), stream=torch.cuda.Stream(),
                         out=[torch.zeros(sum(lens), H, dv, device=dev()) for _ in range(8)],
                         cache=[cache0.clone() for _ in range(8)]))

    def run(j, r, stream=None):
        K.kda_lin_prefill(j["cache"][r], j["slots"], j["cu"], j["q"], j["k"], j["v"], j["al"], j["out"][r], stream=stream)
        K.kda_lin_decode_step(j["cache"][r], j["slots"], j["q"][:2], j["k"][:2], j["v"][:2], j["al"][:2], j["out"][r][:2],
                              stream=stream)

    for j in jobs:
        run(j, 0)
    torch.cuda.synchronize()
    log("lin: two threads")
    failures = []

    def thread(j):
        try:
            for r in range(1, 8):
                run(j, r, j["stream"])
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            failures.append(e)

    threads = [threading.Thread(target=thread, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for j in jobs:
        for r in range(1, 8):
            assert np.array_equal(bits(j["out"][r]), bits(j["out"][0])), r
            assert np.array_equal(bits(j["cache"][r]), bits(j["cache"][0])), r


def test_streams_by_handle():
    """`stream` as an integer handle, the default stream's 0 among them, with the call's own workspace."""
    lens = [2000, 3]
    p = inputs(141, sum(lens), 4, 4, 128, 64, False)
    cache0 = cache_of(6, 2, 4, 64, 128)
    slots = np.array([0, 1], np.int32)
    ref = run_prefill(p, lens, slots, cache0)
    side = torch.cuda.Stream()
    for handle in (torch.cuda.default_stream().cuda_stream, side.cuda_stream):
        torch.cuda.synchronize()
        log(f"lin: stream handle {'0' if handle == 0 else 'of a side stream'}")
        side.wait_stream(torch.cuda.current_stream())
        # the inputs are copied on the current stream: ordered before the side stream's work
        q, k, v = split(p, p["x"].to(dev()))
        cache, out = cache0.to(dev()), sentinel((sum(lens), 4, 64))
        al, s, cu = p["alpha"].to(dev()), i32(slots), i32([0, 2000, 2003])
        torch.cuda.synchronize()
        K.kda_lin_prefill(cache, s, cu, q, k, v, al, out, stream=handle)
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), bits(ref[0])) and np.array_equal(bits(cache), bits(ref[1]))


def test_two_graphs_that_share_a_memory_pool():
    """Two graphs captured into one pool, each allocating its call's workspace there, replayed in turn."""
    jobs = []
    for i, lens in enumerate(([1500, 10], [700, 900])):
        p = inputs(151 + i, sum(lens), 4, 2, 128, 128, True)
        q, k, v = (t.to(dev()) for t in split(p, p["x"]))
        cache0 = cache_of(8 + i, 2, 4, 128, 128).to(dev())
        assert K.kda_lin_prefill_workspace(2, sum(lens), 4, 128, 128) > 0
        j = dict(cache0=cache0, cache=cache0.clone(), out=torch.zeros(sum(lens), 4, 128, device=dev()),
                 args=(i32([1, 0]), i32([0, lens[0], sum(lens)]), q, k, v, p["alpha"].to(dev())))
        K.kda_lin_prefill(j["cache"], *j["args"], j["out"])
        torch.cuda.synchronize()
        j["ref"] = bits(j["out"]), bits(j["cache"])
        jobs.append(j)
    pool = torch.cuda.graph_pool_handle()
    for j in jobs:
        j["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(j["graph"], pool=pool):
            K.kda_lin_prefill(j["cache"], *j["args"], j["out"])
    for r in range(3):
        log(f"lin: shared pool, replay {r}")
        for j in jobs:
            j["cache"].copy_(j["cache0"])
            j["out"].zero_()
        for j in jobs if r % 2 else jobs[::-1]:
            j["graph"].replay()
        torch.cuda.synchronize()
        for j in jobs:
            assert np.array_equal(bits(j["out"]), j["ref"][0]) and np.array_equal(bits(j["cache"]), j["ref"][1]), r
        K.kda_lin_prefill(jobs[0]["cache"], *jobs[0]["args"], jobs[0]["out"])  # eager work between the replays
        torch.cuda.synchronize()
