"""Plain 64-bit forms of the eight-bit layer's operators (numpy), from their
definitions: heads turned by positions of several axes, E4M3 and E8M0 values,
the append to a cache with a scale per block of tokens and head, tokens in
8-bit integers and their product."""
from __future__ import annotations

import numpy as np


def turn_axes(x, w, freq, axis_of, positions, rot, inter, rot_scale, eps):
    """x: tokens x heads x size in fp64; the rows normed (with a weight) and turned, pair j by its axis's position."""
    y = np.array(x, np.float64)
    if w is not None:
        y = y * w / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    if rot:
        axes = positions.shape[0]
        at = np.where((axis_of < axes)[:, None], positions[np.minimum(axis_of, axes - 1)], 0).T.astype(np.float64)   # tokens x pairs
        angle = (at * freq.astype(np.float64))[:, None]
        c, s = rot_scale * np.cos(angle), rot_scale * np.sin(angle)
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def e4m3_values():
    """The 256 values of OCP E4M3 by its definition."""
    v = np.empty(256)
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        x = np.nan if e == 15 and m == 7 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        v[code] = -x if code & 128 else x
    return v


E4M3 = e4m3_values()


def e8m0_value(byte):
    b = np.asarray(byte).astype(np.float64)
    return np.where(b == 255, np.nan, np.exp2(b - 127))


def e4m3_code(x):
    """Nearest code, ties to even, saturating; 0x7F for what is not finite."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    spacing = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    v = np.minimum(np.round(a / spacing) * spacing, 448.0)
    codes = np.argsort(E4M3[:127], kind="stable")
    c = codes[np.searchsorted(E4M3[:127][codes], v)].astype(np.uint8)
    return np.where(np.isfinite(x), np.where(np.signbit(x), c | 0x80, c), 0x7F).astype(np.uint8)


def scale_byte(most):
    """E8M0 byte of the least 2^e, e >= -127, with most <= 448 * 2^e; 0 for 0."""
    m = np.asarray(most, np.float64)
    e = np.arange(255)
    return (m[..., None] > 448.0 * np.exp2(e - 127.0)).sum(-1).astype(np.uint8)


def append(x, cu, table, lens, cache, scales, page, block, longest):
    """The append's definition, block by block.  x: rows x heads x size; cache: slots x heads x size codes, scales:
    blocks x heads bytes; both are changed."""
    pages = cache.shape[0] // page
    capacity = table.shape[1] * page
    heads = cache.shape[1]
    for b in range(table.shape[0]):
        n = int(np.clip(lens[b], 0, capacity))
        m = min(int(cu[b + 1] - cu[b]), longest)
        p0 = n - m
        for start in range(max(p0, 0) // block * block, n, block):
            lo, hi = max(start, p0, 0), min(start + block, n)
            entry = int(table[b, start // page])
            if lo >= hi or not 0 <= entry < pages:
                continue
            slot = entry * page + start % page
            at, old = slot // block, lo - start
            new = x[cu[b] + lo - p0:cu[b] + hi - p0]
            finite = np.where(np.isfinite(new), np.abs(new), 0.0)
            for h in range(heads):
                need = int(scale_byte(finite[:, h].max()))
                was = int(scales[at, h]) if old else 0
                byte = max(need, was)
                if old and byte != was:
                    rows = cache[slot:slot + old, h]
                    v = E4M3[rows] * np.exp2(float(was - byte))
                    cache[slot:slot + old, h] = np.where(np.isnan(v), rows, e4m3_code(np.where(np.isnan(v), 0, v)) | (rows & 0x80))
                scales[at, h] = byte
                cache[slot + old:slot + hi - start, h] = e4m3_code(new[:, h] * np.exp2(127.0 - byte))


def quantize_tokens(x):
    """(codes, scales) of the rows of x (values of bf16 numbers): scale = fp32(max |row| fp32(1 / 127)), 1 where that is 0;
    the integer nearest to fp32(x / scale), ties to even; a row with a value that is not finite: zeros, NaN."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(1)
    y = np.where(bad[:, None], np.float32(0), x)
    s = np.abs(y).max(1) * (np.float32(1) / np.float32(127))
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    q = np.clip(np.rint(y / s[:, None]), -127, 127).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), s).astype(np.float32)


def product(a, s_a, w, s_w, bias=None):
    """fp64 values of (sum a w) s_a s_w + bias; the sums are exact."""
    sums = a.astype(np.float64) @ w.astype(np.float64).T
    y = sums * s_a.astype(np.float64)[:, None] * s_w.astype(np.float64)
    return y if bias is None else y + bias, sums
