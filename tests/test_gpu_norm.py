"""The norms around a block against the plain 64-bit form (linear_ref.norm_ref), and a run of a whole
linear-attention layer through the operators."""

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as K
import linear_ref as R
from gpu_util import bits, dev, i32, log

pytestmark = pytest.mark.gpu

# (z, w_post, gate, y): every combination of parts that the call allows
PARTS = [(0, 0, 0, 1), (1, 0, 0, 0), (1, 0, 0, 1), (1, 1, 0, 1), (1, 0, 1, 1), (1, 1, 1, 1), (1, 1, 1, 0)]


def make(seed, rows, D, parts, resid_bf16):
    g = torch.Generator().manual_seed(seed)
    z, post, gate, y = parts
    rt = torch.bfloat16 if resid_bf16 else torch.float32
    return dict(resid=(3 * torch.randn(rows, D, generator=g)).to(rt),
                z=torch.randn(rows, D, generator=g).bfloat16() if z else None,
                w_post=torch.randn(D, generator=g) if post else None,
                gate=(3 * torch.randn(rows, D, generator=g)).bfloat16() if gate else None,
                w_pre=torch.randn(D, generator=g) if y else None)


def run(c, y_bf16, *, scale=0.7, eps=1e-6, in_place=False, pad=0, stream=None):
    """(resid_out, y) on the CPU; pad: rows of every array are that much further apart than D."""
    rows, D = c["resid"].shape

    def put(t):
        if t is None:
            return None
        w = torch.full((rows, D + pad), -7.0, dtype=t.dtype, device=dev())
        w[:, :D] = t.to(dev())
        return w[:, :D]

    resid, z, gate = put(c["resid"]), put(c["z"]), put(c["gate"])
    ro = None
    if z is not None:
        ro = resid if in_place else put(torch.zeros_like(c["resid"]))
    y = put(torch.zeros(rows, D, dtype=torch.bfloat16 if y_bf16 else torch.float32)) if c["w_pre"] is not None else None
    K.kda_block_norm(resid, z, ro, y, w_post=None if c["w_post"] is None else c["w_post"].to(dev()), gate=gate,
                     res_scale=scale, w_pre=None if c["w_pre"] is None else c["w_pre"].to(dev()), eps=eps,
                     stream=stream)
    torch.cuda.synchronize()
    if pad:
        for t in (ro, y):
            if t is not None:
                assert bool((t._base[:, D:] == -7.0).all()), "columns between the rows"
    return ro, y


def check(c, got, y_bf16, *, scale=0.7, eps=1e-6):
    r, rb, y, yb = R.norm_ref(c["resid"], c["z"], c["w_post"], c["gate"], scale, c["w_pre"], eps)
    if got[0] is not None:
        if c["resid"].dtype == torch.bfloat16:
            rb = rb + R.UB16 * 1.001 * r.abs()
        R.check(got[0], r, rb, "resid_out")
    if got[1] is not None:
        R.check(got[1], y, yb + (R.UB16 * 1.001 * y.abs() if y_bf16 else 0), "y")


@pytest.mark.parametrize("parts", PARTS, ids=str)
@pytest.mark.parametrize("D", [1, 7, 64, 512, 520, 1000, 2051, 4096, 4104, 7168, 8193, 16384])
def test_parts_and_widths(parts, D):
    for resid_bf16 in (False, True):
        y_bf16 = resid_bf16 == (D % 2 == 0)
        log(f"norm D={D} parts={parts} resid_bf16={resid_bf16} y_bf16={y_bf16}")
        c = make(D, 3, D, parts, resid_bf16)
        check(c, run(c, y_bf16), y_bf16)


@pytest.mark.parametrize("rows", [1, 2, 63, 1000])
@pytest.mark.parametrize("D", [1024, 5120])
def test_rows(rows, D):
    log(f"norm rows={rows} D={D}")
    c = make(rows, rows, D, (1, 1, 1, 1), True)
    check(c, run(c, True), True)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("D", [96, 2048])
@pytest.mark.parametrize("resid_bf16", [False, True])
def test_strided_and_in_place(pad, D, resid_bf16):
    log(f"norm in place, pad={pad} D={D} resid_bf16={resid_bf16}")
    c = make(D + pad, 5, D, (1, 1, 1, 1), resid_bf16)
    a = run(c, True, pad=pad)
    check(c, a, True)
    b = run(c, True, pad=pad, in_place=True)
    assert np.array_equal(bits(a[0].contiguous()), bits(b[0].contiguous()))
    assert np.array_equal(bits(a[1].contiguous()), bits(b[1].contiguous()))


def test_vector_and_scalar_rows_agree():
    """The same rows 16-byte aligned and not: the sums run in another order, the values agree to the bound."""
    c = make(5, 4, 2048, (1, 1, 1, 1), False)
    check(c, run(c, False, pad=0), False)
    check(c, run(c, False, pad=3), False)


def test_zero_rows_extremes_and_scale():
    c = make(6, 6, 640, (1, 1, 1, 1), False)
    c["z"][0] = 0
    c["z"][1] = 1e-20
    c["z"][2] = 1e15
    c["gate"][3] = 200.0
    c["gate"][4] = -200.0
    c["resid"][5] = 0
    log("norm: zero rows, tiny and large values, saturated gates")
    check(c, run(c, True), True)
    check(c, run(c, False, scale=0.0), False, scale=0.0)
    check(c, run(c, False, scale=-2.5, eps=1e-3), False, scale=-2.5, eps=1e-3)


def test_nonfinite_rows_stay_alone():
    c = make(7, 4, 1000, (1, 1, 1, 1), True)
    clean = run(c, True)
    c["z"][1, 17] = float("nan")
    c["resid"][2, 999] = float("inf")
    log("norm: NaN and infinity in two rows")
    got = run(c, True)
    for row in (0, 3):
        for x, y in zip(got, clean):
            assert np.array_equal(bits(x[row].contiguous()), bits(y[row].contiguous()))
    assert torch.isnan(got[1][1].float()).all()


def test_large_strides():
    """Rows more than 2^31 elements apart."""
    D, stride = 64, (1 << 31) + 8
    z = torch.empty(stride + D, dtype=torch.bfloat16, device=dev()).as_strided((2, D), (stride, 1))
    c = make(8, 2, D, (1, 1, 0, 1), True)
    z.copy_(c["z"].to(dev()))
    resid, ro, y = c["resid"].to(dev()), torch.zeros(2, D, dtype=torch.bfloat16, device=dev()), torch.zeros(2, D, device=dev())
    log("norm: rows of z 2^31 + 8 elements apart")
    K.kda_block_norm(resid, z, ro, y, w_post=c["w_post"].to(dev()), res_scale=0.7, w_pre=c["w_pre"].to(dev()))
    torch.cuda.synchronize()
    check(c, (ro, y), False)


def test_repeats_and_graph_replays():
    c = make(9, 300, 4096, (1, 1, 1, 1), True)
    d = {k: (t.to(dev()) if t is not None else None) for k, t in c.items()}
    r0 = d["resid"].clone()
    y = torch.zeros(300, 4096, dtype=torch.bfloat16, device=dev())

    def work():
        K.kda_block_norm(d["resid"], d["z"], d["resid"], y, w_post=d["w_post"], gate=d["gate"], res_scale=0.5,
                         w_pre=d["w_pre"])

    work()
    torch.cuda.synchronize()
    ref = (bits(d["resid"]), bits(y))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    log("norm graph: capture")
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            work()
    torch.cuda.current_stream().wait_stream(stream)
    for r in range(3):
        d["resid"].copy_(r0)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(d["resid"]), ref[0]) and np.array_equal(bits(y), ref[1]), f"replay {r}"


def layer_ref(x, lens, w_in, wqkv, wo, w_post, w_next, alpha, H, Hk, d, S, scale):
    """The layer in 64 bits on the CPU, each operator's bf16 outputs rounded as the operators round them."""
    n, kw = x.shape[0], Hk * d
    _, _, h, _ = R.norm_ref(x, w_pre=w_in)
    qkv = (h.bfloat16().double() @ wqkv.double()).bfloat16()
    q, k, v = qkv[:, :kw].view(n, Hk, d), qkv[:, kw: 2 * kw].view(n, Hk, d), qkv[:, 2 * kw:].view(n, H, d)
    outs, states, at = [], [], 0
    for b, t in enumerate(lens):
        o, s, _ = R.recur(q[at: at + t], k[at: at + t], v[at: at + t], alpha, S[b])
        outs.append(o)
        states.append(s)
        at += t
    o = torch.cat(outs).reshape(n, H * d).bfloat16()
    z = (o.double() @ wo.double()).bfloat16()
    r, _, y, _ = R.norm_ref(x, z, w_post, None, scale, w_next)
    return r, y, torch.stack(states)


def test_layer_prompt_then_steps():
    """A linear-attention layer as a server runs it: norm, one projection, prompts, output projection, post-norm
    with the next block's norm; then single-token steps on the same cache. Against the layer in 64 bits: a bf16
    rounding of the normed input, the projections and the outputs moves a value by 2^-8 at most each, and the
    norms in between keep vectors of a length; four such steps and a factor 2 for their mixing give 2^-5."""
    H, Hk, d, Dm = 4, 2, 64, 256
    g = torch.Generator().manual_seed(13)
    lens = [90, 1, 33]
    wqkv = (torch.randn(Dm, (2 * Hk + H) * d, generator=g) / Dm ** 0.5).bfloat16()
    wqkv[:, : 2 * Hk * d] *= 0.25
    wo = (torch.randn(H * d, Dm, generator=g) / (H * d) ** 0.5).bfloat16()
    w_in, w_post, w_next = (1 + 0.1 * torch.randn(Dm, generator=g) for _ in range(3))
    alpha = torch.tensor([0.999, 0.97, 0.8, 0.5])
    S = torch.zeros(3, H, d, d)
    cache = torch.zeros(4, H, d, d, device=dev())
    slots = i32([2, 0, 3])
    D = {n: t.to(dev()) for n, t in dict(wqkv=wqkv, wo=wo, w_in=w_in, w_post=w_post, w_next=w_next, alpha=alpha).items()}

    def layer(x, prompt):
        n, kw = x.shape[0], Hk * d
        h = torch.empty(n, Dm, dtype=torch.bfloat16, device=dev())
        K.kda_block_norm(x, y=h, w_pre=D["w_in"])
        qkv = h @ D["wqkv"]
        q, k, v = qkv[:, :kw].view(n, Hk, d), qkv[:, kw: 2 * kw].view(n, Hk, d), qkv[:, 2 * kw:].view(n, H, d)
        out = torch.empty(n, H, d, dtype=torch.bfloat16, device=dev())
        if prompt:
            K.kda_lin_prefill(cache, slots, i32([0, 90, 91, 124]), q, k, v, D["alpha"], out)
        else:
            K.kda_lin_decode_step(cache, slots, q, k, v, D["alpha"], out)
        z = out.view(n, H * d) @ D["wo"]
        y = torch.empty(n, Dm, dtype=torch.bfloat16, device=dev())
        K.kda_block_norm(x, z, x, y, w_post=D["w_post"], res_scale=0.5, w_pre=D["w_next"])
        return x, y

    for step in range(4):
        n = sum(lens) if step == 0 else 3
        x = torch.randn(n, Dm, generator=g)
        log(f"layer: {'prompt' if step == 0 else 'step'} of {n} tokens")
        r, y = layer(x.to(dev()), step == 0)
        torch.cuda.synchronize()
        rr, yr, S = layer_ref(x, lens if step == 0 else [1, 1, 1], w_in, wqkv, wo, w_post, w_next, alpha, H, Hk, d, S, 0.5)
        for got, ref, what in ((r, rr, "residual"), (y, yr, "normed"), (cache[[2, 0, 3]], S, "state")):
            e = (got.cpu().double() - ref).norm() / ref.norm()
            assert e <= 2.0 ** -5, (step, what, float(e))
