"""The kernels that a call of the layers on packed weights would run, from the
library's own choice (host only): tests name the kernel that a case is meant to
reach, so a change of the rule cannot move it elsewhere unseen."""
from __future__ import annotations

import ctypes

_I32, _I64 = ctypes.c_int32, ctypes.c_int64


def linear_path(lib, tokens, m, n, g, gated=False):
    """(tokens of a tile, how): 16 is the few-token kernel, "gather" or "copied"
    for where X' comes from; 32, 64, 128 the tile kernel with "whole" tiles, all
    "split" along K, or "mixed"."""
    fn = lib.gptq_internal_w4a16_linear_path
    fn.argtypes, fn.restype = [_I64, _I64, _I64, _I32, _I32, ctypes.POINTER(_I32)], ctypes.c_int
    out = (_I32 * 5)()
    assert fn(tokens, m, n, g, int(gated), out) == 1
    tile, gather, whole, parted, splits = out
    if tile == 16:
        return 16, "gather" if gather else "copied"
    assert splits > 1 or parted == 0
    return tile, "whole" if splits == 1 else "mixed" if whole else "split"


def moe_path(lib, cfg, tokens, out):
    """dict of the form of gptq_w4a16_moe: small (two launches), logits (a launch
    of their own), gate_up_lds and down_lds (rows in LDS, else read from memory),
    gate_up_pass, down_pass (tokens), slices (of down's K)."""
    fn = lib.gptq_internal_w4a16_moe_path
    fn.argtypes, fn.restype = [ctypes.c_void_p, _I64, _I32, ctypes.POINTER(_I32)], ctypes.c_int
    c, v = cfg.c(), (_I32 * 7)()
    assert fn(ctypes.byref(c), tokens, {"bf16": 0, "fp32": 1}[out], v) == 1
    return dict(zip(("small", "logits", "gate_up_lds", "gate_up_pass", "down_lds", "down_pass", "slices"), v))
