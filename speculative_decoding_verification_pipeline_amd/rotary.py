"""Rotary positions (ss_rotate in include/ss_sampler.h): queries and keys turned pair
by pair by angles that grow with their position.

The frequencies are formed once, in binary64; the angles of a call are formed and
reduced in the HIP library, also in binary64, so far positions lose nothing and no
table of sines is kept. PageCache.write takes a Rotary to turn keys as it writes
them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .sampler import (_HALF_DTYPES, SS_OK, CRotary, _check, _check_block, _check_out_heads, _empty,
                      _heads, _require, _stream_on, load_library)


def frequencies(dim, base=10000.0, scaling=None, factor=1.0, original=None, fast=32.0, slow=1.0):
    """Radians per position of the dim / 2 pairs, and the factor on the turned values.

    Pair i turns by base^(-2 i / dim). scaling, for contexts `factor` times as long:
    None; "linear": positions divided by factor; "ntk": the base raised so that the
    slowest pair is slowed down by factor and the fastest stays; "parts": pairs that
    turn over `fast` times within the `original` length stay, those below `slow`
    times are divided by factor, between them a ramp over the index, and values are
    multiplied by 0.1 ln(factor) + 1."""
    _require(dim >= 2 and dim % 2 == 0, "dim must be even and at least 2")
    _require(base > 1 and factor >= 1, "base must be above 1 and factor at least 1")
    _require(scaling in (None, "linear", "ntk", "parts"),
             "scaling must be None, 'linear', 'ntk' or 'parts'")
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "parts":
        return f, 1.0
    _require(original is not None and original > 0, "'parts' needs the original length")
    _require(fast > slow > 0, "fast must be above slow, and slow above 0")

    def pair(turns):  # the index, not rounded, of the pair that turns so often
        return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo = max(math.floor(pair(fast)), 0)
    hi = min(math.ceil(pair(slow)), dim // 2 - 1)
    out = []
    for i, x in enumerate(f):
        ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append(x * (1 - ramp) + x / factor * ramp)
    return out, 0.1 * math.log(factor) + 1.0


class Rotary:
    """The rotation of the first dim entries of a head. interleaved: entries 2 i and
    2 i + 1 are pairs, else i and i + dim / 2. base, scaling, factor, original, fast
    and slow as frequencies() takes them, or inv_freq: dim / 2 radians per position of
    the caller's. magnitude: the factor on turned values (None: frequencies')."""

    def __init__(self, dim, base=10000.0, scaling=None, factor=1.0, original=None, fast=32.0,
                 slow=1.0, interleaved=False, inv_freq=None, magnitude=None, device=None):
        if inv_freq is None:
            inv_freq, m = frequencies(dim, base, scaling, factor, original, fast, slow)
        else:
            inv_freq, m = torch.as_tensor(inv_freq, dtype=torch.float64).flatten().tolist(), 1.0
        _require(dim >= 2 and dim % 2 == 0 and len(inv_freq) == dim // 2,
                 "inv_freq must be dim / 2 frequencies")
        self.lib = load_library()
        self.dim, self.interleaved = dim, bool(interleaved)
        self.inv_freq = inv_freq
        self.magnitude = m if magnitude is None else float(magnitude)
        _require(all(map(math.isfinite, inv_freq)) and math.isfinite(self.magnitude),
                 "frequencies and magnitude must be finite")
        self.turns = torch.tensor([x / (2 * math.pi) for x in inv_freq], dtype=torch.float64,
                                  device="cuda" if device is None else device)
        _require(self.turns.is_cuda, "a Rotary lives on a GPU")
        self.device = self.turns.device.index
        self._c = CRotary(self.turns.data_ptr(), dim, int(self.interleaved), self.magnitude)

    def on(self, device):
        """The rotation as the ABI takes it, for calls on this device."""
        if device != self.device:
            raise ValueError(f"the rotary lives on cuda:{self.device}, not cuda:{device}")
        return self._c

    def rotate(self, queries, positions, keys=None, out_queries=None, out_keys=None, stream=None):
        """Turn queries [..., heads, head_dim] (bfloat16 or float16; one or two leading
        dimensions) by positions int32 of the leading shape, and keys, of their own
        number of heads, along. Outputs may be given; an input given as its own output
        is turned in place. Returns out_queries, or (out_queries, out_keys)."""
        dev = self.device
        code = _HALF_DTYPES.get(getattr(queries, "dtype", None))
        _require(code is not None and queries.dim() in (3, 4),
                 "queries must be [T, heads, dim] or [B, N, heads, dim] of bfloat16 or float16")
        lead = queries.shape[:-2]
        _require(self.dim <= queries.shape[-1], f"heads must have at least {self.dim} entries")
        pos = _check_block(positions, "positions", lead, torch.int32, dev)
        if out_queries is None:
            out_queries = _empty(tuple(queries.shape), queries, queries.dtype, stream)
        arrays = [(queries, "queries", queries), (out_queries, "out_queries", queries)]
        if keys is not None:
            _require(keys.dim() == queries.dim() and keys.shape[:-2] == lead and
                     keys.shape[-1] == queries.shape[-1],
                     "keys must match queries but for the number of heads")
            if out_keys is None:
                out_keys = _empty(tuple(keys.shape), keys, keys.dtype, stream)
            arrays += [(keys, "keys", keys), (out_keys, "out_keys", keys)]
        else:
            _require(out_keys is None, "out_keys needs keys")
        c = []
        for i, (t, name, like) in enumerate(arrays):
            _require(isinstance(t, torch.Tensor) and t.shape == like.shape,
                     f"{name} must be {list(like.shape)}")
            if t.dim() == 3:
                t = t.unsqueeze(0)
            c.append(_heads(t, name, None, queries.dtype, dev))
            if i % 2:
                _check_out_heads(t, name)
        q, oq, k, ok = [ctypes.byref(x) for x in c] + [None] * (4 - len(c))
        B, N = (1, lead[0]) if len(lead) == 1 else lead
        st = self.lib.ss_rotate(dev, ctypes.byref(self._c), code, B, N, queries.shape[-1], pos, q, oq,
                                queries.shape[-2], k, ok, 0 if keys is None else keys.shape[-2],
                                _stream_on(stream, dev))
        if st != SS_OK:
            _check("ss_rotate", st)
        return out_queries if keys is None else (out_queries, out_keys)
