"""Rotary positions for the tiled attention and its cache.

``Rope`` holds the frequencies of one model's rotation and turns queries and keys::

    rope = Rope(head_dim=128, base=500000.0, scaling={"kind": "yarn", "factor": 8.0, "original_len": 8192})
    q, k = rope(q, k)                        # [B, H, N, D], positions 0 .. N - 1; differentiable
    y = sdpa.attention(q, k, v, is_causal=True)

    q = cache.append(layer, k, v, n_new, rope=rope, q=q)   # a step over a PagedKVCache

Pair i of the r = rotary_dim first dimensions (its halves i and i + r / 2, or 2 i and
2 i + 1 when interleaved) turns by position * f_i radians, f_i = base^(-2 i / r), and
is scaled by `amplitude`.  The kernels take the frequencies as 64-bit fractions of a
turn (include/rope.h), so far positions lose nothing.

Scalings for contexts longer than a model was trained on, by factor s:

* ``{"kind": "linear", "factor": s}``: f_i / s;
* ``{"kind": "ntk", "factor": s}``: the base becomes base * s^(r / (r - 2)), which leaves
  the first pair and divides the last one's frequency by s;
* ``{"kind": "yarn", "factor": s, "original_len": L}`` (optional "beta_fast" 32,
  "beta_slow" 1): pairs that turn more than beta_fast times over L positions keep
  their frequency, those that turn less than beta_slow times get f_i / s, with a ramp
  over the pairs between; the amplitude is 0.1 ln s + 1 (at
  least 1) unless given;
* ``{"kind": "bands", "factor": s, "low": a, "high": b, "original_len": L}``: as yarn, with
  a blend that is linear in the turns L f_i / (2 pi) between a and b, amplitude 1.

``inv_freq`` gives the r / 2 frequencies themselves instead.
"""
from __future__ import annotations

import math
from fractions import Fraction

from . import _lib

__all__ = ["Rope", "frequencies"]

# 1 / (2 pi), to 60 decimal places
_PER_TURN = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)


def frequencies(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None):
    """(radians per position of each of the rotary_dim / 2 pairs, amplitude)."""
    r = rotary_dim
    s = dict(scaling or {"kind": "none"})
    kind, amplitude = s.pop("kind", None), 1.0
    known = {"none": (), "linear": ("factor",), "ntk": ("factor",),
             "yarn": ("factor", "original_len", "beta_fast", "beta_slow"),
             "bands": ("factor", "low", "high", "original_len")}
    if kind not in known:
        raise ValueError(f"scaling kind {kind!r} is not one of {sorted(known)}")
    optional = {"beta_fast": 32.0, "beta_slow": 1.0}
    for name in known[kind]:
        value = s.pop(name, optional.get(name))
        if value is None or not (float(value) > 0.0 and math.isfinite(float(value))):
            raise ValueError(f"scaling {kind!r} needs a positive {name}, not {value!r}")
        optional[name] = float(value)
    if s:
        raise ValueError(f"scaling {kind!r} does not take {sorted(s)}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be above 1, not {base}")
    if kind == "ntk" and r > 2:
        base = base * optional["factor"] ** (r / (r - 2))
    freqs = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        freqs = [f / optional["factor"] for f in freqs]
    elif kind == "yarn":
        k, L = optional["factor"], optional["original_len"]
        if optional["beta_fast"] < optional["beta_slow"]:
            raise ValueError("beta_fast must not be below beta_slow")
        # the pair that turns n times over L positions
        pair = lambda n: r * math.log(L / (2 * math.pi * n)) / (2 * math.log(base))
        lo = max(math.floor(pair(optional["beta_fast"])), 0)
        hi = min(math.ceil(pair(optional["beta_slow"])), r - 1)
        for i, f in enumerate(freqs):
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            freqs[i] = f * (1 - ramp) + f / k * ramp
        amplitude = max(0.1 * math.log(k) + 1.0, 1.0)
    elif kind == "bands":
        k, a, b = optional["factor"], optional["low"], optional["high"]
        if not a < b:
            raise ValueError("low must be below high")
        for i, f in enumerate(freqs):
            blend = min(max((optional["original_len"] * f / (2 * math.pi) - a) / (b - a), 0.0), 1.0)
            freqs[i] = f / k * (1 - blend) + f * blend
    return freqs, amplitude


class Rope:
    """One model's rotation.  head_dim is 64 or 128, rotary_dim (default: head_dim)
    even; amplitude overrides the scaling's.  Call it with q [B, Hq, N, D] and
    k [B, Hk, N, D] (or q alone), fp16 or bf16 on the GPU in any strides: the results are
    contiguous, as the attention calls take them, and differentiable."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: dict | None = None, inv_freq=None,
                 amplitude: float | None = None):
        if head_dim not in (64, 128):
            raise NotImplementedError(f"head dim {head_dim} is not one of (64, 128)")
        r = head_dim if rotary_dim is None else int(rotary_dim)
        if r < 2 or r > head_dim or r % 2:
            raise ValueError(f"rotary_dim must be even and in [2, {head_dim}], not {r}")
        if inv_freq is None:
            freqs, amp = frequencies(r, float(base), scaling)
        else:
            if scaling is not None:
                raise ValueError("inv_freq already holds the scaled frequencies")
            freqs, amp = [float(f) for f in inv_freq], 1.0
            if len(freqs) != r // 2 or not all(map(math.isfinite, freqs)):
                raise ValueError(f"inv_freq must be {r // 2} finite numbers")
        amp = amp if amplitude is None else float(amplitude)
        if not (amp > 0.0 and math.isfinite(amp)):
            raise ValueError(f"amplitude must be positive, not {amp}")
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, r, bool(interleaved)
        self.inv_freq, self.amplitude = tuple(freqs), amp
        # as fractions of a turn, 64 bits (the signed view of an unsigned word)
        words = [round(Fraction(f) * _PER_TURN * 2 ** 64) % 2 ** 64 for f in freqs]
        self._words = [w - 2 ** 64 if w >= 2 ** 63 else w for w in words]
        self._turns = {}   # by device index (-1: the CPU)

    def turns(self, device):
        """The frequencies as the kernels take them (int64 [rotary_dim / 2]) on a device.  The
        first call on each device copies them there: make it before a stream capture."""
        import torch
        device = torch.device(device)
        index = -1 if device.type != "cuda" else torch.cuda.current_device() if device.index is None else device.index
        if index not in self._turns:
            if index >= 0 and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a rotation's first use on a device cannot be captured: call turns(device) before")
            with torch.inference_mode(False):   # kept for training, too: a backward pass saves it
                t = torch.tensor(self._words, dtype=torch.int64, device=device)
            try:   # inside a function transform it is a wrapper that ends with it: not to be kept
                plain = type(t) is torch.Tensor and t.data_ptr() != 0
            except RuntimeError:
                plain = False
            if not plain:
                raise RuntimeError("a rotation's first use on a device cannot be inside a function transform: call "
                                   "turns(device) before")
            self._turns[index] = (t, self.rotary_dim, self.interleaved, self.amplitude, self.head_dim)
        return self._turns[index][0]

    def for_rows(self, x):
        """What the calls take for rows x: the frequencies on its device, and the numbers."""
        a = self._turns.get(x.get_device())
        if a is None:
            self.turns(x.device)
            a = self._turns[x.get_device()]
        return a

    def __call__(self, q, k=None, positions=None, start: int = 0):
        """q, or (q, k), turned to positions (int32 [N], [1, N] or [B, N]; None: start + n)."""
        r = (_lib._bind or _lib._load_bind()).rotary(q, k, positions, start, self.for_rows(q))
        return r if type(r) is not int else _lib.rotary(q, k, self, positions, start)
