"""CPU oracle of the 8-bit paged cache: e4m3 codes, the scales of pages, rows written and read back; and of
rotary positions. fp64 where values are computed, fp32 where the definition says so.

Test infrastructure only; nothing of the library runs here. Codes are held as uint8.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
LARGEST = 448.0
NAN_CODE = 0x7F


def _value(c):
    sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


VALUES = np.array([_value(c) for c in range(256)])


def decode_codes(codes):
    return VALUES[codes]


def encode(x):
    """The codes nearest to x (ties to the even code; |x| <= 448 after rounding, NaN to NaN). -0 keeps its sign."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(x)
    ok = np.isfinite(x)
    safe = np.where(ok, mag, 0.0)
    assert (safe <= LARGEST).all()
    table = VALUES[:127]  # 0 .. 448, ascending with the code
    hi = np.searchsorted(table, safe, side="left")
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - safe, safe - table[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (table[hi] == safe), hi, lo)
    code = pick.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(ok, code, NAN_CODE).astype(np.uint8)


def scale_for(amax):
    """The least power of two s >= 2^-100 with amax <= 448 s, by counting up."""
    s = 2.0 ** -100
    while amax > LARGEST * s:
        s *= 2.0
    return s


def store(codes, scale, rows, slots):
    """K or V rows [T][H][D] (bf16 values) into ``codes`` [P][H][16][D] uint8 and ``scale`` [P][H] float32, in place."""
    P, H = scale.shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= P * PAGE:
            t += 1
            continue
        page, end = s // PAGE, t
        while end < len(slots) and slots[end] >= 0 and int(slots[end]) // PAGE == page:
            end += 1
        at = [int(x) % PAGE for x in slots[t:end]]
        for h in range(H):
            new = np.asarray(rows[t:end, h], dtype=np.float64)
            fin = np.abs(new[np.isfinite(new)])
            need = np.float32(scale_for(fin.max() if fin.size else 0.0))
            old = np.float32(scale[page, h])
            s_new = need if 0 in at else np.fmax(need, old)
            if 0 not in at and s_new != old:
                ratio = np.float32(old / s_new)
                rest = [r for r in range(PAGE) if r not in at]
                moved = VALUES[codes[page, h, rest]].astype(np.float32) * ratio
                codes[page, h, rest] = encode(moved)
            inv = np.float32(1.0) / s_new
            for i, r in enumerate(at):
                x = np.where(np.isfinite(new[i]), new[i], np.nan).astype(np.float32) * inv
                codes[page, h, r] = encode(x)
            scale[page, h] = s_new
        t = end


def values(codes, scale):
    """What the cache holds, in fp64."""
    return VALUES[codes] * np.asarray(scale, dtype=np.float64)[..., None, None]


def to_bf16(x):
    """fp64 values that fp32 holds exactly, rounded to bf16 (nearest even), as float32."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def load(codes, scale, table, token_start, out, first=None):
    """``out`` [T][H][D] with the requests' rows written where the definition says; error bits (page 1, length 2)."""
    out, err = np.array(out, dtype=np.float64), 0
    held = values(codes, scale)
    for t in range(min(int(token_start[-1]), len(out))):
        b = max(i for i in range(len(token_start) - 1) if token_start[i] <= t)
        pos = t - int(token_start[b]) + (0 if first is None else int(first[b]))
        if not 0 <= pos < table.shape[1] * PAGE:
            err |= 2
            continue
        page = int(table[b, pos // PAGE])
        if not 0 <= page < len(codes):
            err |= 1
            continue
        out[t] = to_bf16(held[page, :, pos % PAGE])
    return out, err


def frequencies(dim, base, scaling, factor=1.0, original=0):
    """Radians per position of every pair, and the amplitude."""
    w = []
    for i in range(dim // 2):
        b = base * factor ** (dim / (dim - 2)) if scaling == "ntk" and dim > 2 else base
        x = b ** (-2.0 * i / dim)
        if scaling == "linear":
            x /= factor
        if scaling == "yarn":
            turns = original * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - 1) / 31))
            x = g * x + (1 - g) * x / factor
        if scaling == "yarn_pairs":
            low, high = (dim * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32, 1))
            low, high = max(math.floor(low), 0), min(math.ceil(high), dim - 1)
            g = 1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            x = g * x + (1 - g) * x / factor
        w.append(x)
    return np.array(w), (0.1 * math.log(factor) + 1 if scaling.startswith("yarn") else 1.0)


def rotary(x, positions, w, offset=0, interleaved=False, inverse=False, amplitude=1.0):
    """Rows [T][H][D] turned, in fp64."""
    y = np.array(x, dtype=np.float64)
    for i, f in enumerate(w):
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + len(w))
        a = np.asarray(positions, dtype=np.float64) * f * (-1 if inverse else 1)
        z = (x[..., offset + i0] + 1j * x[..., offset + i1]) * (amplitude * np.exp(1j * a))[:, None]
        y[..., offset + i0], y[..., offset + i1] = z.real, z.imag
    return y
