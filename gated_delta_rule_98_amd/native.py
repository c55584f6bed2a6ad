"""The native marshalling module (kda_native.so, csrc/kda_binding.cpp), bound to libkda.so's entry points on
its first use. Like the library it is built by gated_delta_rule_98_amd/build.py; importing the package works
without it and the first call raises, naming the build command."""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from .kda import load_library, workspace_on

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kda_native.so")

_module = None


def native():
    """The bound module."""
    global _module
    if _module is None:
        lib = load_library()
        if not os.path.exists(PATH):
            raise FileNotFoundError(f"{PATH} is missing: build it with `python gated_delta_rule_98_amd/build.py`")
        loader = importlib.machinery.ExtensionFileLoader("kda_native", PATH)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("kda_native", loader))
        loader.exec_module(mod)
        # the current stream's handle without building a Stream object, where torch has it
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                   for f in ("kda_lin_decode_step", "kda_lin_prefill", "kda_lin_prefill_workspace",
                             "kda_block_norm")), stream, workspace_on)
        _module = mod
    return _module
