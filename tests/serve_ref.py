"""Plain CPU references of the serving operators: 64-bit arithmetic and
one-entry-at-a-time bookkeeping, straight from the definitions in
include/misa.h."""

from __future__ import annotations

import math

import numpy as np
import torch

BF16_HALF, E4M3_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24  # finfo(t).eps / 2


def up(a, b):
    return -(-a // b)


def attend(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale, table, lengths, idx):
    """out, lse in 64 bits, and how far an fp32 evaluation may be from each.

    A score is a dot product of dk exact products added in fp32: off by at most
    e = scale * (dk + 4) * 2^-23 * sum |q_i k_i| (a rounding or truncation per
    addition, the scales' products in the 4), plus the rounding of its exponent
    argument, (|s| + |max|) * 2^-23.  A weight is then off by a factor of
    exp(+-2e), its two bf16 parts by 2^-16, and n of them are added: relative
    n * 2^-23 of sum p |v|.  The result's own rounding is half a bf16 step."""
    rows, dv = c.rows, c.dv
    share = heads // c.kv_heads
    out = torch.zeros(rows, heads, dv, dtype=torch.float64)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(rows):
        n = int(lengths[r])
        n = min(max(n, 0), c.row_pages * c.page_tokens)
        listed = [int(s) for s in idx[r]] if k else range(n)
        at = [(int(table[r, s // c.page_tokens]), s % c.page_tokens) for s in listed if 0 <= s < n]
        at = [(p, s) for p, s in at if 0 <= p < c.pages]
        if not at:
            continue
        page, slot = (torch.tensor(x) for x in zip(*at))
        for g in range(c.kv_heads):
            kk = k_pages[page, g, slot].double()
            if k_scale is not None:
                kk = kk * k_scale[page, g, slot].double()[:, None]
            if v_pages is None:
                vv = kk[:, :dv]
            else:
                vv = v_pages[page, g, slot].double()
                if v_scale is not None:
                    vv = vv * v_scale[page, g, slot].double()[:, None]
            for j in range(g * share, (g + 1) * share):
                qq = q[r, j].double()
                s = scale * (kk @ qq)
                e = (abs(scale) * (c.dk + 4) * 2.0 ** -23 * (kk.abs() @ qq.abs())).max()
                e = e + 2.0 ** -22 * s.abs().max()
                top = s.max()
                p = torch.exp(s - top)
                total = p.sum()
                out[r, j] = (p / total) @ vv
                lse[r, j] = top + torch.log(total)
                rel = 2 * e + 2.0 ** -16 + (len(at) + 8) * 2.0 ** -22
                out_tol[r, j] = BF16_HALF * out[r, j].abs() + (1 + BF16_HALF) * rel * ((p / total) @ vv.abs())
                lse_tol[r, j] = e + (len(at) + 8) * 2.0 ** -23 + 2.0 ** -22 * (1 + abs(lse[r, j]))
    return out, lse, out_tol, lse_tol


def e4m3_scale(x):
    """The shared scale of the last axis, in 64 bits."""
    top = x.double().abs()
    top = torch.where(torch.isnan(top), 0.0, top).amax(-1)
    return torch.where(top >= 2.0 ** -100, top / 448, 1.0)


def check_e4m3(code, scale, x, slack=0.0):
    """Codes and scales of x [..., n] (64 bits): the scale within two fp32
    roundings (its maximum's and the division's) and x's own relative slack;
    each code within half an e4m3 step (half a subnormal step, 2^-10, near zero)
    of x / scale, itself off by the product's roundings and the slack."""
    want = e4m3_scale(x)
    assert torch.all((scale.double() - want).abs() <= want * (4 * F32_HALF + slack))
    y = x.double() / scale.double()[..., None]
    got = code.double()
    finite = ~torch.isnan(y)
    assert torch.equal(torch.isnan(got), ~finite)
    off = (got - y).abs()[finite]
    y = y.abs()[finite]
    assert torch.all(off <= torch.clamp(y * E4M3_HALF, min=2.0 ** -10) + y * (8 * F32_HALF + 2 * slack))


def norm(x, residual, weight, groups, eps):
    """y and z in 64 bits, and how far fp32 may be from z: the residual's
    addition, n + 8 additions and products in the mean square (half of that in
    its root), and six more roundings."""
    y = x.double() + (residual.double() if residual is not None else 0)
    rows, n = y.shape
    part = y.view(rows, groups, -1)
    r = 1 / torch.sqrt(part.square().mean(-1, keepdim=True) + eps)
    z = (part * r * weight.double()).view(rows, n)
    # the sum's rounding moves a small y that cancels: relative to |x| + |residual|
    size = x.double().abs() + (residual.double().abs() if residual is not None else 0)
    zs = (size.view_as(part) * r * weight.double().abs()).view(rows, n)
    rel = (n / groups + 8) / 2 * F32_HALF + 8 * F32_HALF
    spread = (size.view_as(part).square().sum(-1, keepdim=True) / part.square().sum(-1, keepdim=True).clamp(min=1e-300)).sqrt()
    grow = (1 + spread).expand_as(part).reshape(rows, n)
    return y, z, z.abs() * rel * grow + zs * 2 * F32_HALF


class Book:
    """Tables, lengths and refs of a paged cache, one list entry at a time."""

    def __init__(self, c, table, lengths, refs):
        self.c = c
        self.table, self.lengths, self.refs = (np.array(x, dtype=np.int64) for x in (table, lengths, refs))

    def _page(self, p):
        return 0 <= p < self.c.pages

    def _free_ids(self):
        return [p for p in range(self.c.pages) if self.refs[p] <= 0]

    def extend(self, row, count):
        c, ok, used = self.c, [], 0
        free = self._free_ids()
        for i, (r, more) in enumerate(zip(row, count)):
            good = 0 <= r < c.rows and more >= 0 and r not in list(row[:i])
            if good:
                n = int(self.lengths[r])
                good = n >= 0 and n + more <= c.row_pages * c.page_tokens
            if good:
                a, b = up(n, c.page_tokens), up(n + more, c.page_tokens)
                good = a == b or used + b - a <= len(free)
                for s in range(a, b):
                    if good:
                        self.table[r, s] = free[used + s - a]
                        self.refs[free[used + s - a]] = 1
                used += b - a
                if good:
                    self.lengths[r] += more
            ok.append(int(good))
        return ok

    def fork(self, parent, child):
        c, ok, src, dst, used = self.c, [], [], [], 0
        free = self._free_ids()
        lengths = self.lengths.copy()
        for i, (p, h) in enumerate(zip(parent, child)):
            good = 0 <= p < c.rows and 0 <= h < c.rows and p != h and h not in list(child[:i])
            good = good and lengths[h] == 0
            a = b = -1
            if good:
                n = min(max(int(lengths[p]), 0), c.row_pages * c.page_tokens)
                whole = n // c.page_tokens
                if n % c.page_tokens and self._page(self.table[p, whole]):
                    good = used < len(free)
                    if good:
                        a, b = int(self.table[p, whole]), free[used]
                        self.refs[b] = 1
                    used += 1
            if good:
                self.table[h, :whole] = self.table[p, :whole]
                for x in self.table[p, :whole]:
                    if self._page(x):
                        self.refs[x] += 1
                if n % c.page_tokens:
                    self.table[h, whole] = b
                self.lengths[h] = n
            ok.append(int(good))
            src.append(a)
            dst.append(b)
        return src, dst, ok

    def free(self, row):
        c = self.c
        for r in row:
            if not 0 <= r < c.rows:
                continue
            held = up(min(max(int(self.lengths[r]), 0), c.row_pages * c.page_tokens), c.page_tokens)
            for s in range(held):
                if self._page(self.table[r, s]):
                    self.refs[self.table[r, s]] -= 1
                self.table[r, s] = -1
            self.lengths[r] = 0

    def compact(self):
        c = self.c
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, c.pages) if self.refs[p] > 0]
        to = {p: p for p in range(c.pages) if self.refs[p] > 0}
        to.update(zip(movers, holes))
        refs = np.zeros_like(self.refs)
        for a, b in to.items():
            refs[b] = self.refs[a]
        self.refs = refs
        self.table = np.vectorize(lambda x: to.get(int(x), -1), otypes=[np.int64])(self.table)
        half = max(1, c.pages // 2)
        pad = [-1] * (half - len(holes))
        return [to.get(p, -1) for p in range(c.pages)], live, movers + pad, holes + pad
