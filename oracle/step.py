"""The target's step around its cache in plain numpy (oracle side): microscaled formats, norms with the residual's
addition, linear layers, and distributions and draws out of logits.

Formats ("fp8", "fp4": blocks of 32 under a power of two; "nv4": blocks of 16 under an e4m3 scale and the tensor's
factor): every element and scale is found by looking for the nearest value of its type, ties to the even code.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

from .sampling import QBITS

BLOCK = {"fp8": 32, "fp4": 32, "nv4": 16}


def _codes(exp_bits: int, man_bits: int, bias: int, top: int) -> np.ndarray:
    """Values of the non-negative codes 0 .. top of a small float."""
    c = np.arange(top + 1)
    e, f = c >> man_bits, c & ((1 << man_bits) - 1)
    return np.where(e > 0, (1 + f / 2.0 ** man_bits) * 2.0 ** (e - bias), f / 2.0 ** man_bits * 2.0 ** (1 - bias))


E4M3 = _codes(4, 3, 7, 0x7e)             # up to 448; 0x7f is NaN
E2M1 = _codes(2, 1, 1, 7)                # up to 6


def nearest_code(values: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Code of the value nearest to |x|, ties to the even code, the largest beyond it."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def scale_layout(rows: int, blocks: int) -> np.ndarray:
    """Byte of the scale of [row, block] (blocks of a row up to the next multiple of 4)."""
    r, c = np.arange(rows)[:, None], np.arange(-(-blocks // 4) * 4)[None]
    return ((r // 128) * (-(-blocks // 4)) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4


def quantize(fmt: str, x: np.ndarray, g: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """(codes with the sign in the top bit [rows, cols], scale bytes [rows, blocks]) of finite x."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, BLOCK[fmt])
    top = np.abs(b).max(-1)
    if fmt == "nv4":
        g = np.float32(g)
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            t = (top.astype(np.float32) / (np.float32(6) * g)).astype(np.float64)
        byte = np.where(top > 0, nearest_code(E4M3, t), 0)
        d = E4M3[byte].astype(np.float32) * g
        with np.errstate(over="ignore"):
            some = d >= np.float32(2.0 ** -126)      # (elements are zeros where d is less)
            q = np.where(some[..., None], b.astype(np.float32) / np.where(some, d, np.float32(1))[..., None],
                         np.float32(0)).astype(np.float64)
    else:
        byte = np.searchsorted(2.0 ** np.arange(-127, 128), top / (448.0 if fmt == "fp8" else 6.0), side="left")
        q = b / 2.0 ** (byte - 127.0)[..., None]
    code = nearest_code(E4M3 if fmt == "fp8" else E2M1, q)
    code = code | (np.signbit(b).astype(int) << (7 if fmt == "fp8" else 3))
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def unpack_bytes(fmt: str, data: np.ndarray, scale: np.ndarray, rows: int, cols: int) -> Tuple[np.ndarray, np.ndarray]:
    """Codes and scale bytes (with those up to the multiple of 4) from a matrix's memory."""
    data = data.reshape(rows, -1)
    if fmt != "fp8":
        data = np.stack((data & 15, data >> 4), -1).reshape(rows, cols)
    return data, scale[scale_layout(rows, cols // BLOCK[fmt])]


def pack_bytes(fmt: str, code: np.ndarray, byte: np.ndarray, fill: int = 0) -> Tuple[np.ndarray, np.ndarray]:
    """A matrix's memory; `fill`: what stands for the rows behind the last in the scales."""
    rows, blocks = byte.shape
    data = code if fmt == "fp8" else code[:, 0::2] | (code[:, 1::2] << 4)
    scale = np.full(-(-rows // 128) * -(-blocks // 4) * 512, fill, dtype=np.uint8)
    at = scale_layout(rows, blocks)
    scale[at] = 0
    scale[at[:, :blocks]] = byte
    return data.astype(np.uint8), scale


def values(fmt: str, code: np.ndarray, byte: np.ndarray, g: float = 1.0) -> np.ndarray:
    """What codes and scales stand for."""
    v, sign = (E4M3[np.minimum(code & 127, 0x7e)], code >> 7) if fmt == "fp8" else (E2M1[code & 7], code >> 3)
    v = np.where(sign == 1, -v, v)
    if fmt == "nv4":
        d = (E4M3[byte].astype(np.float32) * np.float32(g)).astype(np.float64)
    else:
        d = 2.0 ** (byte.astype(np.float64) - 127.0)
    return (v.reshape(v.shape[0], -1, BLOCK[fmt]) * d[..., None]).reshape(v.shape)


def swiglu(x: np.ndarray) -> np.ndarray:
    a, b = np.split(np.asarray(x, dtype=np.float64), 2, axis=-1)
    return a / (1.0 + np.exp(-a)) * b


def add_norm(x: np.ndarray, residual: Optional[np.ndarray], gain: Optional[np.ndarray], eps: float):
    """(sum, normed)."""
    h = np.asarray(x, dtype=np.float64) + (0.0 if residual is None else np.asarray(residual, dtype=np.float64))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, y if gain is None else y * np.asarray(gain, dtype=np.float64)


def weights(z: np.ndarray, temperature: float) -> np.ndarray:
    """floor(2^40 e^((z - max) / t)); all on the first largest where t <= 0."""
    z = np.asarray(z, dtype=np.float64)
    if not temperature > 0:
        w = np.zeros(z.size, dtype=np.int64)
        w[np.flatnonzero(z == z.max())[0]] = 1 << QBITS
        return w
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        return np.floor(np.exp((z - z.max()) / max(float(temperature), 1e-30)) * 2.0 ** QBITS).astype(np.int64)


def kept(z: np.ndarray, w: np.ndarray, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0, slack: int = 0):
    """(order, fewest, most): tokens in falling order of z, the lower id first among equals, and how many of its first
    top_k and top_p keep when weights may be `slack` units in all off; min_p applies to weights afterwards."""
    z = np.asarray(z, dtype=np.float64)
    order = np.lexsort((np.arange(z.size), -z))
    n = z.size if top_k <= 0 else min(top_k, z.size)
    if not top_p < 1:
        return order, n, n
    cum = np.cumsum(w[order[:n]].astype(object))
    need = max(1, int(np.ceil(max(top_p, 0.0) * float(cum[-1]))))
    first = lambda v: int(np.searchsorted(cum.astype(np.float64), float(v))) + 1
    return order, min(first(max(need - slack, 1)), n), min(first(need + slack), n)


def distribution(z, temperature: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> np.ndarray:
    """Kept whole weights of a row."""
    w = weights(z, temperature)
    order, n, _ = kept(z, w, top_k, top_p)
    out = np.zeros_like(w)
    out[order[:n]] = w[order[:n]]
    if min_p > 0:
        out[out < min(float(min_p), 1.0) * 2.0 ** QBITS] = 0
    return out
