"""Workspaces of the prefill calls on the GPU: the stream they are allocated on, and one kept for
calls of several sizes."""

import contextlib

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as K
from gpu_util import bits, dev, i32, log
from test_gpu_linear import cache_of, inputs, split

pytestmark = pytest.mark.gpu


def long_prompt(seed, n=4000, H=32):
    """Arguments of a call whose workspace is too large for any other tensor's leftover block."""
    p = inputs(seed, n, H, 1, 128, 128, False)
    q, k, v = split(p, p["x"].to(dev()))
    args = (cache_of(seed, 1, H, 128, 128).to(dev()), i32([0]), i32([0, n]), q, k, v, p["alpha"].to(dev()),
            torch.empty(n, H, 128, device=dev()))
    need = K.kda_lin_prefill_workspace(1, n, H, 128, 128)
    return args, need


def streams_of_allocations(call, size):
    """The streams' handles of the allocations of at least `size` bytes that torch makes during the call."""
    torch.cuda.memory._record_memory_history(max_entries=1000, stacks="python")
    try:
        call()
        torch.cuda.synchronize()
        trace = torch.cuda.memory._snapshot()["device_traces"][0]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    return [e["stream"] for e in trace if e["action"] == "alloc" and e["size"] >= size]


@pytest.mark.parametrize("kind", ["none", "handle 0", "default stream", "current stream", "side stream", "side handle"])
def test_workspace_comes_from_the_stream_of_the_launch(kind):
    args, need = long_prompt(171)
    assert need >= 32 << 20
    side = torch.cuda.Stream()
    stream, handle = {"none": (None, 0), "handle 0": (0, 0), "default stream": (torch.cuda.default_stream(), 0),
                      "current stream": (torch.cuda.current_stream(), 0), "side stream": (side, side.cuda_stream),
                      "side handle": (side.cuda_stream, side.cuda_stream)}[kind]
    torch.cuda.synchronize()
    log(f"lin prefill on stream {kind}")
    assert streams_of_allocations(lambda: K.kda_lin_prefill(*args, stream=stream), need) == [handle]


def test_calls_on_the_default_stream_and_on_pool_streams_at_once():
    """Calls on handle 0 and on 32 streams of torch's pool, each with a workspace of the call's own, queued without a
    wait between them, agree with the calls alone."""
    args, _ = long_prompt(181, 2100, 16)
    cache0 = args[0].clone()
    K.kda_lin_prefill(*args)
    torch.cuda.synchronize()
    ref = bits(args[0]), bits(args[7])
    streams = [torch.cuda.Stream() for _ in range(32)]
    caches = [cache0.clone() for _ in range(33)]
    outs = [torch.empty_like(args[7]) for _ in range(33)]
    torch.cuda.synchronize()
    log("lin prefill on 33 streams")
    for c, o, s in zip(caches, outs, [0] + streams):
        K.kda_lin_prefill(c, *args[1:7], o, stream=s)
    torch.cuda.synchronize()
    for i, (c, o) in enumerate(zip(caches, outs)):
        assert np.array_equal(bits(c), ref[0]) and np.array_equal(bits(o), ref[1]), i


def test_chunk_prefill_workspace_comes_from_the_stream_of_the_launch():
    n, H, d = 2000, 32, 128
    need = K.kda_prefill_chunked_workspace(1, n, H, d, d)
    x = torch.full((n, H, d), 0.05, dtype=torch.bfloat16, device=dev())
    args = (torch.zeros(1, H, d, d, device=dev()), i32([0]), i32([0, n]), x, x, x, torch.full((n, H, d), 0.9, device=dev()),
            torch.full((n, H), 0.5, device=dev()), torch.empty(n, H, d, device=dev()))
    side = torch.cuda.Stream()
    for stream, handle in ((0, 0), (side, side.cuda_stream), (None, 0)):
        torch.cuda.synchronize()
        log(f"chunk prefill on stream handle {'0' if handle == 0 else 'of a side stream'}")
        assert streams_of_allocations(lambda: K.kda_prefill_chunked(*args, stream=stream), need) == [handle]


def test_one_workspace_for_calls_of_several_sizes():
    """A buffer for the largest call, full of NaN, serves the smaller ones in turn; the bits are those of the calls alone."""
    H, d = 32, 128
    sizes = [8000, 4096, 3840, 2560, 700]
    ws = torch.full((K.kda_lin_prefill_workspace(1, max(sizes), H, d, d),), 0xFF, dtype=torch.uint8, device=dev())
    p = inputs(191, max(sizes), H, 4, d, d, True)
    q, k, v = split(p, p["x"].to(dev()))
    al, cache0 = p["alpha"].to(dev()), cache_of(3, 1, H, d, d).to(dev())
    for n in sizes:
        log(f"lin prefill of {n} tokens with the workspace of the largest call")
        got = []
        for w in (None, ws):
            cache, out = cache0.clone(), torch.empty(n, H, d, device=dev())
            K.kda_lin_prefill(cache, i32([0]), i32([0, n]), q[:n], k[:n], v[:n], al[:n], out, workspace=w)
            torch.cuda.synchronize()
            got.append((bits(cache), bits(out)))
        assert all(np.array_equal(x, y) for x, y in zip(*got)), n


@pytest.mark.parametrize("kind", ["current", "handle 0", "side stream"])
def test_a_workspace_that_does_not_fit_is_torchs_out_of_memory_error(kind):
    """What a server catches around kda_prefill_chunked. The allocator is limited to what it holds already and every
    block of it that would do is taken, so that the call's workspace is refused on the host; afterwards the same call
    runs."""
    args, need = long_prompt(201)
    stream = {"current": None, "handle 0": 0, "side stream": torch.cuda.Stream()}[kind]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = bits(args[0])
    total = torch.cuda.get_device_properties(0).total_memory
    log(f"lin prefill without room for its workspace, stream {kind}")
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)
    taken = []
    try:
        with torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else contextlib.nullcontext():
            with contextlib.suppress(torch.OutOfMemoryError):
                for _ in range(torch.cuda.memory_reserved() // need + 1):
                    taken.append(torch.empty(need, dtype=torch.uint8, device=dev()))
        with pytest.raises(torch.OutOfMemoryError):
            K.kda_lin_prefill(*args, stream=stream)
    finally:
        del taken
        torch.cuda.set_per_process_memory_fraction(1.0)
    torch.cuda.synchronize()
    assert np.array_equal(bits(args[0]), before)
    K.kda_lin_prefill(*args, stream=stream)
    torch.cuda.synchronize()
    assert not np.array_equal(bits(args[0]), before)
