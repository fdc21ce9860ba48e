"""64-bit reference of the page-scaled 8-bit formats and of rotary positions (numpy),
written from the formats' definitions: used by the GPU tests and checked on the CPU by
``test_page8_host.py``."""
from __future__ import annotations

import numpy as np

PAGE = 32
I8, E4M3 = 3, 4
F16_MAX = 65504.0


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 0x7F) == 0x7F] = np.nan
    return np.where(b & 0x80, -v, v)


def e4m3_round(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to the even code) of fp64 values within +-448."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.clip(np.round(y / step) * step, -448, 448)


def clean(x: np.ndarray) -> np.ndarray:
    return np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=F16_MAX, neginf=-F16_MAX), -F16_MAX, F16_MAX)


def scale_for(fmt: int, amax: np.ndarray) -> np.ndarray:
    """Scale a page needs for a largest magnitude, in the format's fp32 arithmetic."""
    a = amax.astype(np.float32)
    if fmt == I8:
        return a / np.float32(127)
    m, e = np.frexp(a)  # a = m 2^e
    return np.where(a > 0, np.ldexp(np.float32(1), e - 9 + (m > 0.875)), np.float32(0)).astype(np.float32)


class PageCache:
    """One tensor (K or V) of a page-scaled cache: codes as values [pages, heads, 32, d]
    and fp32 scales [pages, heads]; ``append`` follows the documented fp32 steps."""

    def __init__(self, fmt, pages, heads, d):
        self.fmt = fmt
        self.codes = np.zeros((pages, heads, PAGE, d), dtype=np.float64)
        self.scale = np.zeros((pages, heads), dtype=np.float32)

    def _round(self, y32: np.ndarray) -> np.ndarray:
        y = y32.astype(np.float64)
        return np.clip(np.round(y), -127, 127) if self.fmt == I8 else e4m3_round(np.clip(y, -448, 448))

    def append(self, x: np.ndarray, slots) -> None:
        """x [n, heads, d] (any float type), slots [n]; negative slots are skipped."""
        x = clean(x)
        last = {}
        for t, s in enumerate(slots):
            if s >= 0:
                last[int(s)] = t  # the later of two tokens for one slot is kept
        pages = {}
        for s, t in last.items():
            pages.setdefault(s // PAGE, []).append((s % PAGE, t))
        for p, items in pages.items():
            at, tok = [i[0] for i in items], [i[1] for i in items]
            fresh = 0 in at
            need = scale_for(self.fmt, np.abs(x[tok]).max(axis=(0, 2)))
            old = np.zeros_like(need) if fresh else self.scale[p]
            d = np.maximum(old, need)
            if not fresh:
                ratio = np.where(d > old, old / np.where(d > 0, d, 1), 1).astype(np.float32)
                moved = self._round(self.codes[p].astype(np.float32) * ratio[:, None, None])
                self.codes[p] = np.where((d > old)[:, None, None], moved, self.codes[p])
            inv = np.where(d > 0, np.float32(1) / np.where(d > 0, d, 1), 0).astype(np.float32)
            self.codes[p][:, at] = self._round(x[tok].astype(np.float32).transpose(1, 0, 2) * inv[:, None, None])
            self.scale[p] = d

    def values(self) -> np.ndarray:
        return self.codes * self.scale.astype(np.float64)[:, :, None, None]


def raw_codes(fmt: int, plane: np.ndarray) -> np.ndarray:
    """Device code bytes -> code values."""
    return plane.view(np.int8).astype(np.float64) if fmt == I8 else e4m3_values()[plane]


def frequencies(rot, scaling="none", base=10000.0, factor=1.0, ctx=0, low=0.0, high=0.0):
    """(f_i, multiplier) written from the definitions."""
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    turns = ctx * f / (2 * np.pi)
    if scaling == "ramp":
        # pair index at which a frequency turns `n` times in ctx tokens
        def index(n):
            return rot / 2 * np.log(ctx / (2 * np.pi * n)) / np.log(base)
        lo, hi = max(np.floor(index(high)), 0), min(np.ceil(index(low)), rot - 1)
        w = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - w) + f / factor * w, 0.1 * np.log(factor) + 1
    if scaling == "bands":
        w = np.clip((turns - low) / (high - low), 0, 1)
        return f * w + f / factor * (1 - w), 1.0
    return f, 1.0


def rotate(x, positions, freq, mscale, rot, interleaved):
    """fp64 rotation of x [n, heads, d] by positions [n]."""
    x = x.astype(np.float64)
    w = positions.astype(np.float64)[:, None] * np.asarray(freq)[None, :]
    c, s = (mscale * np.cos(w))[:, None, :], (mscale * np.sin(w))[:, None, :]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def attention(q, kv, row_slots, rows, window=0):
    """fp64 attention over dequantised planes.  q [total_q, hq, d]; kv = (K, V) values
    [pages, heads, 32, d]; row_slots[r] = slots of row r's positions; rows = (seq_len, q_offset).
    Returns o and A = sum p |v| (the size against which rounding errors of p count)."""
    o, size, at = np.empty(q.shape), np.empty(q.shape), 0
    d, hkv = q.shape[2], kv[0].shape[1]
    group = q.shape[1] // hkv
    for r, (seq, off) in enumerate(rows):
        s = np.asarray(row_slots[r])
        k, v = (x[s // PAGE, :, s % PAGE] for x in kv)  # [seq, heads, d]
        nq = seq - off
        dist = np.arange(off, seq)[:, None] - np.arange(seq)[None, :]
        seen = (dist >= 0) & ((dist < window) if window else True)
        for h in range(q.shape[1]):
            x = q[at:at + nq, h].astype(np.float64) @ k[:, h // group].T / np.sqrt(d)
            x = np.where(seen, x, -np.inf)
            p = np.exp(x - x.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            o[at:at + nq, h] = p @ v[:, h // group]
            size[at:at + nq, h] = p @ np.abs(v[:, h // group])
        at += nq
    return o, size


def attention_tolerance(fmt, q, o, size, k_scale, v_scale, n_keys):
    """Element-wise bound on the kernels' error, counted rounding by rounding:
    p and o are rounded to fp16 (2^-11 each, p below 2^-14 by 2^-25 absolutely, next to a largest
    of 1 or more; chunk tiles keep the largest at 2^-4 or more, where n independent errors of
    2^-21 / sqrt(3) have a root mean square below n 2^-25 from 86 keys on); I8 scores and
    values are sums of codes + 128 whose offset is taken out again, so their fp32 accumulation
    (one rounding of at most 2^-23 a step) counts against 255 rather than the code."""
    d = q.shape[2]
    big = 255.0 if fmt == I8 else 448.0
    q_sum = np.abs(q.astype(np.float64)).sum(axis=2, keepdims=True)
    score = (d / 16 + 1) * 2.0 ** -23 * big * q_sum * float(k_scale.max()) / np.sqrt(d) + 2.0 ** -20
    steps = n_keys / 16 + 16
    value = (steps * 2.0 ** -23 * big + n_keys * 2.0 ** -25 * big) * float(v_scale.max())
    return 1.01 * 2.0 ** -11 * (size + np.abs(o)) + 2.0 ** -25 + 2.5 * score * size + value
