"""Linear attention and the block norm on the host: the headers' entry points are exported and bound, and bad
arguments are refused before anything is enqueued (fake, never dereferenced device addresses; no GPU)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import gated_delta_rule_98_amd as pkg
from gated_delta_rule_98_amd import kda as E
from gated_delta_rule_98_amd.linear import kda_lin_tokens

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="hands fake device addresses to the library")


def test_headers_library_and_binding_agree():
    names = set()
    for h in ("kda_linear.h", "kda_norm.h"):
        names |= set(re.findall(r"^int\s+(kda_\w+)\s*\(", open(os.path.join(ROOT, "include", h)).read(), flags=re.M))
    assert names == {"kda_lin_decode_step", "kda_lin_prefill", "kda_lin_prefill_workspace", "kda_block_norm"}
    lib = pkg.load_library()
    for n in names:
        assert getattr(lib, n) is not None and callable(getattr(pkg, n))


def _x(**over):
    d = dict(q=A, k=A, v=A, alpha=A, qs=256, ks=256, vs=256, as_=2, Hk=2)
    d.update(over)
    return ctypes.byref(kda_lin_tokens(*d.values()))


def _decode(**over):
    d = dict(cache=A, num_slots=8, slot_stride=2 * 128 * 128, slot_ids=A, B=4, H=2, dk=128, dv=128, x=_x(), out=A,
             epi=None, dev_err=None, opts=None, stream=None)
    d.update(over)
    return E.load_library().kda_lin_decode_step(*d.values())


def _prefill(**over):
    d = dict(cache=A, num_slots=8, slot_stride=2 * 128 * 128, slot_ids=A, cu=A, B=4, n_tok=90, H=2, dk=128, dv=128,
             x=_x(), out=A, ckpt_pos=None, ckpt=None, ws=A, ws_bytes=1 << 40, dev_err=None, opts=None, stream=None)
    d.update(over)
    return E.load_library().kda_lin_prefill(*d.values())


TOKEN_ERRORS = [
    (dict(q=None), E.KDA_ERR_INVALID), (dict(k=None), E.KDA_ERR_INVALID), (dict(v=None), E.KDA_ERR_INVALID),
    (dict(alpha=None), E.KDA_ERR_INVALID), (dict(Hk=0), E.KDA_ERR_INVALID), (dict(Hk=-1), E.KDA_ERR_INVALID),
    (dict(Hk=3), E.KDA_ERR_INVALID), (dict(qs=248), E.KDA_ERR_INVALID), (dict(ks=248), E.KDA_ERR_INVALID),
    (dict(vs=248), E.KDA_ERR_INVALID), (dict(as_=1), E.KDA_ERR_INVALID), (dict(as_=-2), E.KDA_ERR_INVALID),
    (dict(qs=260), E.KDA_ERR_ALIGN), (dict(ks=257), E.KDA_ERR_ALIGN), (dict(vs=258), E.KDA_ERR_ALIGN),
    (dict(q=A + 8), E.KDA_ERR_ALIGN), (dict(k=A + 2), E.KDA_ERR_ALIGN), (dict(v=A + 4), E.KDA_ERR_ALIGN),
    (dict(alpha=A + 2), E.KDA_ERR_ALIGN), (dict(qs=(1 << 24) + 8), E.KDA_ERR_UNSUPPORTED),
    (dict(vs=(1 << 24) + 8), E.KDA_ERR_UNSUPPORTED), (dict(as_=(1 << 24) + 1), E.KDA_ERR_UNSUPPORTED)]


@needs_no_gpu
@pytest.mark.parametrize("call", [_decode, _prefill])
def test_shared_refusals(call):
    assert call(B=0) == E.KDA_OK
    assert call(B=-1) == E.KDA_ERR_INVALID
    assert call(H=0) == E.KDA_ERR_INVALID
    assert call(dk=96) == E.KDA_ERR_UNSUPPORTED
    assert call(dv=32) == E.KDA_ERR_UNSUPPORTED
    assert call(cache=None) == E.KDA_ERR_INVALID
    assert call(cache=A + 8) == E.KDA_ERR_ALIGN
    assert call(slot_ids=None) == E.KDA_ERR_INVALID
    assert call(slot_ids=A + 2) == E.KDA_ERR_ALIGN
    assert call(num_slots=-1) == E.KDA_ERR_INVALID
    assert call(slot_stride=2 * 128 * 128 - 4) == E.KDA_ERR_INVALID
    assert call(slot_stride=2 * 128 * 128 + 2) == E.KDA_ERR_ALIGN
    assert call(x=None) == E.KDA_ERR_INVALID
    assert call(out=None) == E.KDA_ERR_INVALID
    assert call(out=A + 8) == E.KDA_ERR_ALIGN
    bf16 = ctypes.byref(E.kda_options(0, 0, E.KDA_OUT_BF16))
    assert call(out=A + 4, opts=bf16) == E.KDA_ERR_ALIGN
    assert call(dev_err=A + 1) == E.KDA_ERR_ALIGN
    for over, want in TOKEN_ERRORS:
        assert call(x=_x(**over)) == want, over
    assert call(opts=ctypes.byref(E.kda_options(0, 0, E.KDA_RAW_INPUTS))) == E.KDA_ERR_UNSUPPORTED
    assert call(opts=ctypes.byref(E.kda_options(0, 0, 8))) == E.KDA_ERR_INVALID
    assert call(opts=ctypes.byref(E.kda_options(0, 1, 0))) == E.KDA_ERR_INVALID
    dup, pad = np.array([3, 1, -1, 3], np.int32), np.array([3, -1, 1, -1], np.int32)
    chk = ctypes.byref(E.kda_options(0, 0, E.KDA_CHECK_SLOTS))
    assert call(slot_ids=dup.ctypes.data, opts=chk) == E.KDA_ERR_INVALID
    # passes every host check: only the launch itself fails without a device
    assert call(slot_ids=pad.ctypes.data, opts=chk) == E.KDA_ERR_HIP
    assert call(out=A + 8, opts=bf16) == E.KDA_ERR_HIP
    assert call(x=_x(as_=0)) == E.KDA_ERR_HIP
    assert call(x=_x(Hk=1, qs=128, ks=128)) == E.KDA_ERR_HIP


@needs_no_gpu
def test_decode_refusals():
    assert _decode(epi=ctypes.byref(E.kda_epilogue(None, None, 1e-6))) == E.KDA_ERR_INVALID
    assert _decode(epi=ctypes.byref(E.kda_epilogue(A, None, -1.0))) == E.KDA_ERR_INVALID
    assert _decode(epi=ctypes.byref(E.kda_epilogue(A + 2, None, 1e-6))) == E.KDA_ERR_ALIGN
    gate = ctypes.byref(E.kda_epilogue(A, None, 1e-6))
    assert _decode(epi=gate, opts=ctypes.byref(E.kda_options(64, 0, 0))) == E.KDA_ERR_UNSUPPORTED
    for w in (2, 3, 24, 256):
        assert _decode(opts=ctypes.byref(E.kda_options(w, 0, 0))) == E.KDA_ERR_UNSUPPORTED, w
    assert _decode(dv=64, slot_stride=2 * 128 * 128, opts=ctypes.byref(E.kda_options(128, 0, 0))) == E.KDA_ERR_UNSUPPORTED
    for w in (0, 4, 8, 16, 32, 64, 128):
        assert _decode(opts=ctypes.byref(E.kda_options(w, 0, 0))) == E.KDA_ERR_HIP, w
    assert _decode(epi=gate) == E.KDA_ERR_HIP
    assert _decode(B=1 << 30, H=32, slot_stride=32 * 128 * 128, x=_x(qs=4096, ks=4096, vs=4096, as_=32)) == \
        E.KDA_ERR_UNSUPPORTED


@needs_no_gpu
def test_prefill_refusals():
    assert _prefill(n_tok=0) == E.KDA_OK
    assert _prefill(n_tok=-1) == E.KDA_ERR_INVALID
    assert _prefill(cu=None) == E.KDA_ERR_INVALID
    assert _prefill(cu=A + 2) == E.KDA_ERR_ALIGN
    assert _prefill(ckpt_pos=A) == E.KDA_ERR_INVALID
    assert _prefill(ckpt_pos=A, ckpt=A + 8) == E.KDA_ERR_ALIGN
    assert _prefill(ckpt_pos=A + 2, ckpt=A) == E.KDA_ERR_ALIGN
    assert _prefill(opts=ctypes.byref(E.kda_options(16, 0, 0))) == E.KDA_ERR_UNSUPPORTED
    assert _prefill(n_tok=0, x=None, out=None, ckpt_pos=A, ckpt=A) == E.KDA_ERR_HIP
    n = ctypes.c_size_t(0)
    ws = E.load_library().kda_lin_prefill_workspace
    assert ws(4, 90, 2, 128, 128, None) == E.KDA_ERR_INVALID
    assert ws(-1, 90, 2, 128, 128, ctypes.byref(n)) == E.KDA_ERR_INVALID
    assert ws(4, 90, 2, 96, 128, ctypes.byref(n)) == E.KDA_ERR_UNSUPPORTED
    assert ws(1, 100000, 32, 128, 128, ctypes.byref(n)) == E.KDA_OK
    need = n.value
    big = dict(B=1, n_tok=100000, H=32, slot_stride=32 * 128 * 128, x=_x(qs=4096, ks=4096, vs=4096, as_=32, Hk=32))
    if need:
        assert _prefill(ws=None, **big) == E.KDA_ERR_INVALID
        assert _prefill(ws_bytes=need - 1, **big) == E.KDA_ERR_INVALID
        assert _prefill(ws=A + 8, **big) == E.KDA_ERR_ALIGN
    assert _prefill(ws_bytes=need, **big) == E.KDA_ERR_HIP
    assert ws(4, 0, 2, 128, 128, ctypes.byref(n)) == E.KDA_OK and n.value == 0


@needs_no_gpu
def test_grids_past_the_launch_limits_are_refused():
    def opts(w):
        return ctypes.byref(E.kda_options(w, 0, 0))

    # 2^23 rows x 2 heads x 32 tiles of 64 threads: 2^35 threads; a quarter of 2^32 is launched
    assert _decode(B=1 << 23, opts=opts(4)) == E.KDA_ERR_UNSUPPORTED
    assert _decode(B=1 << 18, opts=opts(4)) == E.KDA_ERR_HIP
    # a workgroup of 512 threads per (row, head)
    assert _prefill(B=1 << 22) == E.KDA_ERR_UNSUPPORTED
    assert _prefill(B=(1 << 22) - 4) == E.KDA_ERR_HIP
    assert _prefill(B=1 << 22, n_tok=0, ckpt_pos=A, ckpt=A) == E.KDA_ERR_UNSUPPORTED


def _norm(**over):
    d = dict(resid=A, rs=64, z=A, zs=64, ro=A, ros=64, y=A, ys=64, w_post=A, gate=A, gs=64, scale=1.0, w_pre=A,
             eps=1e-6, rows=3, D=64, flags=0, stream=None)
    d.update(over)
    return E.load_library().kda_block_norm(*d.values())


@needs_no_gpu
def test_norm_refusals():
    assert _norm(rows=0) == E.KDA_OK
    for bad in (dict(rows=-1), dict(D=0), dict(flags=4), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(scale=float("nan")), dict(scale=float("-inf")), dict(resid=None), dict(z=None),
                dict(z=None, ro=None), dict(z=None, ro=None, w_post=None), dict(z=None, ro=None, gate=None),
                dict(ro=None), dict(y=None), dict(w_pre=None), dict(z=None, ro=None, w_post=None, gate=None, y=None,
                                                                    w_pre=None),
                dict(rs=63), dict(zs=63), dict(ros=63), dict(ys=63), dict(gs=63), dict(ros=128)):
        assert _norm(**bad) == E.KDA_ERR_INVALID, bad
    assert _norm(D=16385, rs=20000, zs=20000, ros=20000, ys=20000, gs=20000) == E.KDA_ERR_UNSUPPORTED
    for bad in (dict(resid=A + 2), dict(ro=A + 2), dict(z=A + 1), dict(y=A + 2), dict(gate=A + 1), dict(w_post=A + 2),
                dict(w_pre=A + 2), dict(flags=1, resid=A + 1, ro=A + 1), dict(flags=2, y=A + 1)):
        assert _norm(**bad) == E.KDA_ERR_ALIGN, bad
    for ok in (dict(), dict(y=None, w_pre=None), dict(z=None, ro=None, w_post=None, gate=None), dict(w_post=None),
               dict(gate=None), dict(flags=3), dict(flags=1, resid=A + 2, ro=A + 2), dict(D=63), dict(ro=2 * A, ros=128)):
        assert _norm(**ok) == E.KDA_ERR_HIP, ok


def test_binding_refuses_host_tensors():
    c = torch.zeros(1, 2, 64, 64)
    t = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.kda_lin_decode_step(c, torch.zeros(1, dtype=torch.int32), t, t, t, torch.zeros(2), torch.zeros(1, 2, 64))
    with pytest.raises(ValueError):
        pkg.kda_lin_prefill(c, torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), t, t, t,
                            torch.zeros(2), torch.zeros(1, 2, 64))
    with pytest.raises(ValueError):
        pkg.kda_block_norm(torch.zeros(2, 8), y=torch.zeros(2, 8), w_pre=torch.zeros(8))
