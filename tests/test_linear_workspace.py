"""Workspaces of the prefill calls on the host: the stream they are allocated on, and their sizes."""

import contextlib

import pytest
import torch

import gated_delta_rule_98_amd as pkg
import gated_delta_rule_98_amd.linear as linear
from gated_delta_rule_98_amd import kda


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.fixture
def cuda(monkeypatch):
    """torch.cuda's stream functions without a GPU; entered: the handles of the streams made current, in order."""
    entered = []

    def external(handle, device=None):
        assert handle != 0, "ExternalStream(0) is a stream of torch's pool, not the default stream"
        return Stream(handle)

    @contextlib.contextmanager
    def current(s):
        entered.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", current)
    return entered


@pytest.mark.parametrize("stream", [0, Stream(0), 64, Stream(64)], ids=["0", "stream 0", "64", "stream 64"])
def test_prefill_builds_no_stream_from_handle_zero(cuda, monkeypatch, stream):
    class Native:
        @staticmethod
        def lin_prefill(*args):
            return kda.KDA_OK

    monkeypatch.setattr(linear, "native", Native)
    linear.kda_lin_prefill(torch.zeros(1), *[None] * 7, stream=stream)


@pytest.mark.parametrize("stream,handle", [(0, 0), (Stream(0), 0), (64, 64), (Stream(64), 64)],
                         ids=["0", "stream 0", "64", "stream 64"])
def test_workspace_is_allocated_on_the_stream_that_uses_it(cuda, stream, handle):
    assert kda.workspace_on(24, "cpu", stream).nbytes == 24
    assert cuda == [handle]


def test_workspace_without_a_stream_stays_on_the_current_one(cuda):
    assert kda.workspace_on(24, "cpu", None).nbytes == 24
    assert cuda == []


@pytest.mark.parametrize("stream,handle", [(None, None), (0, 0), (Stream(64), 64)], ids=["none", "0", "stream 64"])
def test_chunk_prefill_allocates_on_the_stream_that_uses_it(cuda, monkeypatch, stream, handle):
    monkeypatch.setattr(kda, "_prefill_chunked_checks", lambda *a: (1, 8, 1, 64, 64, 1, 4096))
    monkeypatch.setattr(kda, "kda_prefill_chunked_workspace", lambda *a: 24)
    with pytest.raises(ValueError, match="device tensor"):  # a host workspace goes no further
        kda.kda_prefill_chunked(torch.zeros(1), *[None] * 8, stream=stream)
    assert cuda == ([] if handle is None else [handle])


@pytest.mark.parametrize("H", [1, 3, 5, 8, 16, 24, 32, 40, 64, 96, 128, 300, 512, 700])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_a_workspace_for_the_largest_call_serves_the_smaller_ones(H, dk, dv):
    """kda_lin_prefill refuses a workspace below kda_lin_prefill_workspace(), so that may not fall as a call grows.
    It stays within two states for each of 512 (segment, head) pairs and their decays."""
    rows = [1, 2, 3, 4, 5, 8, 16, 17, 33, 64, 130, 1000]
    tokens = sorted({0, 1, 63, 640, 641} | {64 * c + d for c in [*range(1, 40), *range(40, 700, 7)] for d in (0, 1)} |
                    {10 ** 5, 10 ** 6, 10 ** 7, 2 ** 31 - 1})
    need = [[pkg.kda_lin_prefill_workspace(B, n, H, dk, dv) for n in tokens] for B in rows]
    for i in range(len(rows)):
        for j in range(len(tokens)):
            assert j == 0 or need[i][j] >= need[i][j - 1], (rows[i], tokens[j - 1], tokens[j])
            assert i == 0 or need[i][j] >= need[i - 1][j], (rows[i - 1], rows[i], tokens[j])
    assert max(map(max, need)) <= 2 * 512 * (dk * dv + 1) * 4 + 16
