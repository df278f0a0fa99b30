"""Rotary positions (ss_rotate in include/ss_sampler.h): queries and keys turned pair
by pair by angles that grow with their position.

The frequencies are formed once, in binary64; the angles of a call are formed and
reduced in the HIP library, also in binary64, so far positions lose nothing and no
table of sines is kept. PageCache.write takes a Rotary to turn keys as it writes
them.
"""
from __future__ import annotations

import math

import torch

from .sampler import (_HALF_DTYPES, SS_OK, _check, _check_block, _heads, _out_heads, _pack_rotary,
                      _require, _stream_on, load_library)


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

    # the ramp may end behind the last pair: of a long original length all turn more than `slow` times
    lo = max(math.floor(pair(fast)), 0)
    hi = min(math.ceil(pair(slow)), dim - 1)
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
        self._c = _pack_rotary(self.turns.data_ptr(), dim, int(self.interleaved), self.magnitude)

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
        if code is None or queries.dim() not in (3, 4):
            raise ValueError("queries must be [T, heads, dim] or [B, N, heads, dim] of bfloat16 or float16")
        shape, dtype = queries.shape, queries.dtype
        lead, dim = shape[:-2], shape[-1]
        if self.dim > dim:
            raise ValueError(f"heads must have at least {self.dim} entries")
        pos = _check_block(positions, "positions", lead, torch.int32, dev)
        q = _heads(queries, "queries", None, dtype, dev)
        out_queries, oq = _out_heads(out_queries, "out_queries", shape, queries, dtype, stream)
        k = ok = None
        k_heads = 0
        if keys is not None:
            k_heads = keys.shape[-2] if getattr(keys, "ndim", 0) == len(shape) else -1
            if k_heads < 0 or keys.shape != (*lead, k_heads, dim):
                raise ValueError("keys must match queries but for the number of heads")
            k = _heads(keys, "keys", None, dtype, dev)
            out_keys, ok = _out_heads(out_keys, "out_keys", keys.shape, keys, dtype, stream)
        elif out_keys is not None:
            raise ValueError("out_keys needs keys")
        B, N = lead if len(lead) == 2 else (1, lead[0])
        st = self.lib.ss_rotate(dev, self._c, code, B, N, dim, pos, q, oq, shape[-2], k, ok, k_heads,
                                _stream_on(stream, dev))
        if st != SS_OK:
            _check("ss_rotate", st)
        return out_queries if keys is None else (out_queries, out_keys)
