"""Layouts of the linear-attention calls' arguments: what is taken, what is refused."""

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as K
from gpu_util import bits, dev, i32, log
from test_gpu_linear import cache_of, inputs, split

pytestmark = pytest.mark.gpu

H, D = 4, 64


def call(op, p, alpha, out=None, n=70):
    """(cache, out) of one call on its own copies."""
    q, k, v = split(p, p["x"].to(dev()))
    cache = cache_of(5, n if op == "decode" else 2, H, D, D).to(dev())
    out = torch.empty(n, H, D, device=dev()) if out is None else out
    if op == "decode":
        K.kda_lin_decode_step(cache, i32(np.arange(n)), q, k, v, alpha, out)
    else:
        K.kda_lin_prefill(cache, i32([1, 0]), i32([0, 40, n]), q, k, v, alpha, out)
    torch.cuda.synchronize()
    return bits(cache), bits(out)


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_decays_with_a_stride_between_tokens(op):
    """alpha as a slice of a wider projection, and as one row of decays expanded over the tokens."""
    p = inputs(211, 70, H, 2, D, D, True)
    ref = call(op, p, p["alpha"].to(dev()))
    wide = torch.full((70, 2 * H + 3), float("nan"), device=dev())
    wide[:, 3: 3 + H] = p["alpha"].to(dev())
    log(f"lin {op}: decays sliced out of rows of {2 * H + 3}")
    got = call(op, p, wide[:, 3: 3 + H])
    assert all(np.array_equal(x, y) for x, y in zip(got, ref))
    fixed = p["alpha"][7].to(dev())
    log(f"lin {op}: expanded decays")
    got = call(op, p, fixed.expand(70, H))
    assert all(np.array_equal(x, y) for x, y in zip(got, call(op, p, fixed)))


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_decays_refused(op):
    p = inputs(212, 70, H, 2, D, D, True)
    al = p["alpha"].to(dev())
    for bad in (al.t().contiguous().t(), al.repeat_interleave(2, 1)[:, ::2], al[0].repeat_interleave(2)[::2], al[:, :1].expand(70, H)):
        with pytest.raises(ValueError):
            call(op, p, bad)
    with pytest.raises(K.KdaError) as e:  # overlapping rows
        call(op, p, al.flatten().as_strided((70, H), (1, 1)))
    assert e.value.status == K.KDA_ERR_INVALID


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("dtype,step", [(torch.float32, 4), (torch.bfloat16, 4)], ids=["fp32", "bf16"])
def test_alignment_of_outputs(op, dtype, step):
    """out may start 16 bytes (bf16: 8) into an allocation, and nowhere in between."""
    p = inputs(213, 70, H, 2, D, D, True)
    al = p["alpha"].to(dev())
    ref = call(op, p, al, torch.empty(70, H, D, dtype=dtype, device=dev()))
    buf = torch.zeros(70 * H * D + 8, dtype=dtype, device=dev())
    for off in range(1, 9):
        out = buf[off: off + 70 * H * D].view(70, H, D)
        log(f"lin {op}: out {off} elements of {dtype} into its allocation")
        if off % step:
            with pytest.raises(K.KdaError) as e:
                call(op, p, al, out)
            assert e.value.status == K.KDA_ERR_ALIGN
        else:
            buf.zero_()
            got = call(op, p, al, out)
            assert all(np.array_equal(x, y) for x, y in zip(got, ref))
            assert not buf[:off].any() and not buf[off + 70 * H * D:].any()


def test_calls_of_nothing():
    """No rows, no tokens: nothing is written and nothing fails."""
    none = torch.zeros(0, H, D, dtype=torch.bfloat16, device=dev())
    cache = cache_of(5, 2, H, D, D).to(dev())
    before = bits(cache)
    al, out = torch.ones(H, device=dev()), torch.empty(0, H, D, device=dev())
    log("lin decode, prefill and norm of nothing")
    K.kda_lin_decode_step(cache, i32([]), none, none, none, al, out)
    K.kda_lin_decode_step(cache, i32([]), none, none, none, al.expand(0, H), out, gate=none)
    K.kda_lin_prefill(cache, i32([]), i32([0]), none, none, none, al, out)
    K.kda_lin_prefill(cache, i32([1, 0]), i32([0, 0, 0]), none, none, none, al.expand(0, H), out)
    K.kda_block_norm(torch.zeros(0, 64, device=dev()), y=torch.zeros(0, 64, device=dev()), w_pre=torch.ones(64, device=dev()))
    torch.cuda.synchronize()
    assert np.array_equal(bits(cache), before)


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_bfloat16_bits_as_integers(op):
    p = inputs(214, 70, H, 2, D, D, True)
    al = p["alpha"].to(dev())
    ref = call(op, p, al, torch.empty(70, H, D, dtype=torch.bfloat16, device=dev()))
    log(f"lin {op}: bits as int16")
    got = call(op, dict(p, x=p["x"].view(torch.int16)), al, torch.empty(70, H, D, dtype=torch.int16, device=dev()))
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


@pytest.mark.parametrize("n,heads", [(2000, 8), (70, 4)], ids=["segments", "short"])
def test_captured_with_the_stream_named(n, heads):
    """A prompt and a step captured with stream= the captured stream, its workspace allocated under the capture; every
    replay against the eager run, with eager work between."""
    p = inputs(215, n, heads, 2, D, D, True)
    q, k, v = split(p, p["x"].to(dev()))
    cache0 = cache_of(5, 1, heads, D, D).to(dev())
    cache, out = cache0.clone(), torch.empty(n, heads, D, device=dev())
    s, cu, al = i32([0]), i32([0, n]), p["alpha"].to(dev())

    def work(stream):
        K.kda_lin_prefill(cache, s, cu, q, k, v, al, out, stream=stream)
        K.kda_lin_decode_step(cache, s, q[:1], k[:1], v[:1], al[:1], out[:1], stream=stream)

    work(None)
    torch.cuda.synchronize()
    ref = bits(cache), bits(out)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    log(f"lin capture with the stream named, {n} tokens")
    with torch.cuda.graph(graph, stream=side):
        work(side)
    for r in range(3):
        cache.copy_(cache0)
        out.zero_()
        torch.cuda.synchronize()
        log(f"replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(cache), ref[0]) and np.array_equal(bits(out), ref[1]), r
        cache.copy_(cache0)
        work(0)
        torch.cuda.synchronize()
        assert np.array_equal(bits(cache), ref[0]) and np.array_equal(bits(out), ref[1]), r


@pytest.mark.parametrize("heads", [4, 72])
def test_tokens_before_the_first_row(heads):
    """cu_seqlens need not start at 0: the tokens before the first row are no row's, and their outputs stay."""
    n, lead = 210, 7
    p = inputs(216, n, heads, 2, D, D, True)
    q, k, v = split(p, p["x"].to(dev()))
    al, cache0 = p["alpha"].to(dev()), cache_of(5, 2, heads, D, D).to(dev())
    ref, rout = cache0.clone(), torch.empty(n - lead, heads, D, device=dev())
    log(f"lin prefill of rows that start at token {lead}, {heads} heads")
    K.kda_lin_prefill(ref, i32([1, 0]), i32([0, 150, n - lead]), q[lead:].contiguous(), k[lead:].contiguous(), v[lead:].contiguous(),
                      al[lead:].contiguous(), rout)
    cache, out = cache0.clone(), torch.full((n, heads, D), 7.0, device=dev())
    K.kda_lin_prefill(cache, i32([1, 0]), i32([lead, lead + 150, n]), q, k, v, al, out)
    torch.cuda.synchronize()
    assert np.array_equal(bits(cache), bits(ref)) and np.array_equal(bits(out[lead:]), bits(rout))
    assert bool((out[:lead] == 7.0).all())
