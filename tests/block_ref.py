"""Plain CPU references of rotary positions and of the block-scaled cache: 64-bit
arithmetic, one block and one query at a time, straight from include/misa.h."""

from __future__ import annotations

import math

import numpy as np
import torch

from tests import serve_ref


def rope(x, pos, freq, first, pairs, amplitude):
    """y in 64 bits and how far fp32 may be from it.  Angles are products of 80 bits.

    An angle is good to 2^-50 of itself and, reduced to half a turn and rounded to
    fp32, to 2 pi 2^-25; cosine and sine to two fp32 steps (2^-22) and the
    amplitude's rounding (2^-24): together below 2^-20.  Two products and their sum
    round by 3 * 2^-24 of |a| + |b| more."""
    n = x.shape[0]
    x = x.double()
    rot = 2 * len(freq)
    angle = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(freq, dtype=np.longdouble)[None]
    full = 2 * np.longdouble("3.14159265358979323846264338327950288")
    part = (angle - np.rint(angle / full) * full).astype(np.float64)
    cos, sin = torch.from_numpy(np.cos(part))[:, None], torch.from_numpy(np.sin(part))[:, None]
    far = torch.from_numpy(np.abs(angle).astype(np.float64))[:, None] * 2.0 ** -50
    y, tol = x.clone(), torch.zeros_like(x)
    if pairs == 0:
        ia = first + torch.arange(rot // 2)
        ib = ia + rot // 2
    else:
        ia = first + 2 * torch.arange(rot // 2)
        ib = ia + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = amplitude * (a * cos - b * sin)
    y[..., ib] = amplitude * (a * sin + b * cos)
    tol[..., ia] = tol[..., ib] = abs(amplitude) * (a.abs() + b.abs()) * (2.0 ** -20 + 3 * 2.0 ** -24 + far)
    assert y.shape[0] == n
    return y, tol


def block_scale(top):
    """The smallest 2^e, e >= -100, with top <= 448 * 2^e."""
    e = -100
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def places(c, table, r, p):
    """Page and slot of position p of row r, or None."""
    if p < 0 or p >= c.row_pages * c.page_tokens:
        return None
    page = int(table[r, p // c.page_tokens])
    return (page, p % c.page_tokens) if 0 <= page < c.pages else None


def write(c, B, offsets, lengths, new, pool, scale, table):
    """pool (e4m3 codes) and scale after the call: copies."""
    bits, scale = pool.view(torch.uint8).clone(), scale.clone()
    n = new.shape[0]
    off = [min(max(int(x), 0), n) for x in offsets]
    for r in range(c.rows):
        count = off[r + 1] - off[r]
        if count <= 0:
            continue
        start = int(lengths[r]) - count
        blocks = {}
        for i in range(count):
            if places(c, table, r, start + i):
                blocks.setdefault((start + i) // B, []).append(i)
        for b, tokens in blocks.items():
            page, slot0 = places(c, table, r, b * B)
            low = start + tokens[0] - b * B
            for h in range(c.kv_heads):
                x = new[[off[r] + i for i in tokens], h].double()
                size = x.abs()
                top = torch.where(torch.isfinite(size), size, 0.0).max().item()
                unit, at = block_scale(top), (page, h, slot0 // B)
                if low > 0:
                    had = scale[at].item()
                    if had < unit:
                        old = bits[page, h, slot0:slot0 + low].view(pool.dtype).double() * (had / unit)
                        bits[page, h, slot0:slot0 + low] = old.float().to(pool.dtype).view(torch.uint8)
                    unit = max(unit, had)
                y = torch.where(torch.isfinite(x), x / unit, math.nan).float().to(pool.dtype).view(torch.uint8)
                bits[page, h, slot0 + low:slot0 + low + len(tokens)] = y
                scale[at] = unit
    return bits.view(pool.dtype), scale


def same_codes(got, want):
    """Equal codes, any NaN code for a NaN."""
    a, b = got.view(torch.uint8), want.view(torch.uint8)
    both = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
    return bool(((a == b) | both).all())


def read(c, B, offsets, first, lengths, pool, scale, table, n):
    """code, unit of each packed entry (float64, NaN codes NaN), and which entries are written."""
    code = torch.zeros(n, c.kv_heads, c.dk, dtype=torch.uint8)
    unit = torch.ones(n, c.kv_heads)
    written = torch.zeros(n, dtype=torch.bool)
    off = [min(max(int(x), 0), n) for x in offsets]
    for r in range(c.rows):
        for i in range(off[r], off[r + 1]):
            written[i] = True
            p = (0 if first is None else int(first[r])) + i - off[r]
            at = places(c, table, r, p) if p < int(lengths[r]) else None
            if at:
                code[i] = pool.view(torch.uint8)[at[0], :, at[1]]
                unit[i] = scale[at[0], :, at[1] // B]
    return code.view(pool.dtype), unit, written


def attend(misa, c, B, heads, k, scale, offsets, q, k_pages, k_scale, v_pages, v_scale, table, lengths, idx):
    """out, lse, their tolerances, and which queries are written: serve_ref.attend with a row
    for each query, whose weights are held to 2^-16.

    Tiles of queries hold a weight to 2^-11 (f16, half a step), and one that f16 holds as a
    subnormal to 2^-32 of the largest one, at most 448 loudest scales of value: what that adds
    to the tolerance comes as `wide`."""
    n = q.shape[0]
    off = [min(max(int(x), 0), n) for x in offsets]
    row, seen, written = [0] * n, [0] * n, torch.zeros(n, dtype=torch.bool)
    for r in range(c.rows):
        for i in range(off[r], off[r + 1]):
            row[i], seen[i], written[i] = r, max(0, int(lengths[r]) - (off[r + 1] - 1 - i)), True
    many = misa.cache(n, c.row_pages, c.pages, c.page_tokens, c.kv_heads, c.dk, c.dv, c.kv_dtype)
    ks, vs = (x.repeat_interleave(B, dim=2) for x in (k_scale, v_scale))
    args = (many, heads, k, scale, q, k_pages, ks)
    rest = (vs, table[torch.tensor(row)], seen, idx)
    out, lse, out_tol, lse_tol = serve_ref.attend(*args, v_pages, *rest)
    size = serve_ref.attend(*args, v_pages.float().abs().to(v_pages.dtype), *rest)[0]
    loud = torch.zeros(n, dtype=torch.float64)
    for i in range(n):
        at = [places(c, table, row[i], p) for p in range(seen[i])]
        loud[i] = max([v_scale[a[0], :, a[1] // B].max().item() for a in at if a], default=0.0)
    many_seen = torch.tensor(seen, dtype=torch.float64)
    wide = 2.0 ** -11 * size * (1 + 2.0 ** -8) + (many_seen * loud * 448 * 2.0 ** -32)[:, None, None]
    return out, lse, out_tol, lse_tol, wide, written
