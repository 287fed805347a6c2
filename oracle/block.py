"""LayerNorm, the dense linear with its epilogue, and 8-bit checkpoints, in fp64 (oracle).

TEST INFRASTRUCTURE ONLY: see ``oracle/__init__.py``.

    layernorm   y = (x - mean) / sqrt(var + eps) * g + b           (per row)
    linear      z = x W^T + b,  y = residual + act(z)
    checkpoint  per 64 columns of a row: amax = max |x|, q = sign(x) floor(127 |x| / amax + 1/2),
                restored value bf16(q amax / 127); below 2^-118 zeros, with an inf or NaN all NaN

The checkpoint is computed in exact rational arithmetic on the bf16 bit patterns (Python integers), so it
fixes every tie.  Gradients are torch.autograd's of these forwards in float64.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

from .nf4 import bf16_round

BLOCK = 64


def layernorm(x: torch.Tensor, g: torch.Tensor, b, eps: float) -> torch.Tensor:
    c = x - x.mean(dim=-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(dim=-1, keepdim=True) + eps) * g
    return y if b is None else y + b


def act(z: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "relu":
        return z * (z > 0)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    assert kind == "none"
    return z


def linear(x, w, b, kind, residual=None):
    """-> (z, y)"""
    z = x @ w.T
    if b is not None:
        z = z + b
    y = act(z, kind)
    return z, (y if residual is None else y + residual)


def _parts(bits: int):
    """finite bf16 bits -> (sign, integer significand, exponent): value = sign * sig * 2^exp"""
    e, m = (bits >> 7) & 0xFF, bits & 0x7F
    return (-1 if bits & 0x8000 else 1), (m | 0x80 if e else m), (e if e else 1) - 134


def ckpt8_block(bits):
    """bf16 bit patterns of one block -> (amax bits, codes): the definition, in integers."""
    mags = [b & 0x7FFF for b in bits]
    top = max(mags)
    if top >= 0x7F80:
        return 0x7FC0, [0] * len(bits)
    _, ts, te = _parts(top)
    if Fraction(ts) * Fraction(2) ** te < Fraction(2) ** -118:
        return 0, [0] * len(bits)
    codes = []
    for b in bits:
        s, m, e = _parts(b)
        r = Fraction(127 * m, ts) * Fraction(2) ** (e - te)
        codes.append(s * math.floor(r + Fraction(1, 2)))
    return top, codes


def ckpt8_pack(x: torch.Tensor):
    """bf16 [rows, d] -> (codes int8 [rows, d], amax bits uint16 [rows, ceil(d / 64)])"""
    bits = x.contiguous().view(torch.int16).numpy().view(np.uint16)
    rows, d = bits.shape
    nb = -(-d // BLOCK)
    codes, amax = np.zeros((rows, d), np.int8), np.zeros((rows, nb), np.uint16)
    for r in range(rows):
        for k in range(nb):
            sl = slice(k * BLOCK, min(d, (k + 1) * BLOCK))
            amax[r, k], codes[r, sl] = ckpt8_block([int(v) for v in bits[r, sl]])
    return codes, amax


def ckpt8_unpack(codes: np.ndarray, amax: np.ndarray) -> torch.Tensor:
    """-> bf16 [rows, d]: q amax / 127 rounded to bf16 (through float64, whose rounding error of one division
    cannot reach a bf16 midpoint: those are at least 1e-5 away)"""
    d = codes.shape[1]
    a = (amax.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    v = codes.astype(np.float64) * np.repeat(a, BLOCK, axis=1)[:, :d] / 127.0
    return torch.from_numpy(bf16_round(v.astype(np.float32))).to(torch.bfloat16)


def ckpt8_roundtrip(x: torch.Tensor) -> torch.Tensor:
    return ckpt8_unpack(*ckpt8_pack(x))
