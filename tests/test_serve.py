"""The serving operators (include/misa.h, "serving") against the plain CPU
references of tests/serve_ref.py, and their argument checks.  The refusals run
on the CPU: they return before anything is launched."""

from __future__ import annotations

import ctypes
import math
import sys

import numpy as np
import pytest
import torch

from tests import serve_ref as ref

FAKE = 1 << 20  # an aligned non-null address; never dereferenced (calls fail validation)
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def misa():
    import long_context_pool_amd as m

    return m


def _log(msg):
    print(msg, file=sys.stderr, flush=True)


# ------------------------------------------------------------------ refusals (CPU)


def _attend(misa, c, heads=8, k=0, scale=0.1, q=FAKE, kp=FAKE, ks=None, vp=FAKE, vs=None, table=FAKE, lengths=FAKE,
            idx=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40):
    return misa.lib().misa_attend(ctypes.byref(c), heads, k, scale, q, kp, ks, vp, vs, table, lengths, idx, out, lse,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(rows=0), -1), (dict(row_pages=0), -1), (dict(pages=0), -1), (dict(page_tokens=0), -1),
    (dict(page_tokens=4097), -2), (dict(rows=1 << 16, row_pages=1 << 15), -2), (dict(pages=(1 << 24) + 1), -2),
    (dict(row_pages=1 << 20, page_tokens=4096), -2), (dict(rows=65536), -2), (dict(kv_heads=0), -1),
    (dict(kv_heads=257), -2), (dict(kv_heads=3), -1), (dict(dk=96, dv=96), -2), (dict(dk=128, dv=64), -2),
    (dict(dk=576, dv=512, kv_heads=2), -2), (dict(kv_dtype=0), -2), (dict(kv_dtype=3), -1),
])
def test_attend_refuses_caches(misa, change, expect):
    fields = dict(rows=4, row_pages=8, pages=40, page_tokens=16, kv_heads=2, dk=128, dv=128, kv_dtype=1)
    fields.update(change)
    c = misa.cache(*fields.values())
    assert _attend(misa, c) == expect
    assert misa.misa_attend_workspace_bytes(c, 8, 0) == 0


@pytest.mark.parametrize("change,expect", [
    (dict(heads=0), -1), (dict(heads=7), -1), (dict(heads=2048), -2), (dict(k=-1), -1), (dict(k=(1 << 20) + 1, idx=FAKE), -2),
    (dict(k=4), -1), (dict(idx=FAKE), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(q=None), -1), (dict(kp=None), -1), (dict(vp=None), -1), (dict(table=None), -1), (dict(lengths=None), -1),
    (dict(out=None), -1), (dict(q=FAKE + 2), -1), (dict(kp=FAKE + 8), -1), (dict(lse=FAKE + 4), -1),
    (dict(k=4, idx=FAKE + 4), -1),
])
def test_attend_refuses_arguments(misa, change, expect):
    assert _attend(misa, misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_BF16), **change) == expect


def test_attend_refuses_far_scales(misa):
    """Scales whose product with log2(e) leaves fp32's range."""
    c = misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_BF16)
    assert _attend(misa, c, scale=3e38) == -2 and _attend(misa, c, scale=-3e38) == -2
    assert _attend(misa, c, scale=2.0 ** 127, q=None) == -1  # the next check


def test_attend_refuses_missing_scales_latent_values_and_short_workspaces(misa):
    fp8 = misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_FP8_E4M3)
    assert _attend(misa, fp8, ks=None, vs=FAKE) == -1
    assert _attend(misa, fp8, ks=FAKE, vs=None) == -1
    latent = misa.cache(4, 8, 40, 16, 1, 576, 512, misa.MISA_BF16)
    assert _attend(misa, latent, vp=FAKE) == -1
    long = misa.cache(1, 4096, 5000, 64, 1, 128, 128, misa.MISA_BF16)
    need = misa.misa_attend_workspace_bytes(long, 8, 0)
    if need:
        assert _attend(misa, long, ws_bytes=need - 1) == -3
        assert _attend(misa, long, ws=None) == -3
        assert _attend(misa, long, ws=FAKE + 8) == -1


def test_write_refuses(misa):
    c = misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_BF16)
    good = dict(n=3, row=FAKE, pos=FAKE, kn=FAKE, vn=FAKE, kp=FAKE, ks=None, vp=FAKE, vs=None, table=FAKE)

    def call(c=c, **change):
        a = {**good, **change}
        return misa.lib().misa_page_write(ctypes.byref(c), *a.values(), None)

    for change in (dict(n=-1), dict(row=None), dict(pos=None), dict(kn=None), dict(vn=None), dict(kp=None),
                   dict(vp=None), dict(table=None), dict(kn=FAKE + 8), dict(row=FAKE + 4)):
        assert call(**change) == -1, change
    assert call(n=1 << 30) == -2
    assert call(n=0, row=None, pos=None, kn=None, vn=None) == 0  # nothing to do: nothing is launched
    fp8 = misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_FP8_E4M3)
    assert call(fp8) == -1 and call(fp8, ks=FAKE) == -1
    latent = misa.cache(4, 8, 40, 16, 1, 576, 512, misa.MISA_BF16)
    assert call(latent) == -1 and call(latent, vp=None) == -1


def test_bookkeeping_refuses(misa):
    lib = misa.lib()
    c = misa.cache(4, 8, 40, 16, 0, 0, 0, 0)  # only the table's half is looked at
    r = ctypes.byref(c)
    for name, args in (("misa_page_extend", 6), ("misa_page_fork", 8), ("misa_page_free", 4)):
        f = getattr(lib, name)
        assert f(r, -1, *[FAKE] * args, None) == -1
        assert f(r, 4097, *[FAKE] * args, None) == -2
        for i in range(args):
            for bad in (None, FAKE + 4):
                assert f(r, 2, *[bad if j == i else FAKE for j in range(args)], None) == -1, (name, i)
        assert f(ctypes.byref(misa.cache(0, 8, 40, 16, 0, 0, 0, 0)), 2, *[FAKE] * args, None) == -1
    ws = misa.misa_page_workspace_bytes(c)
    assert ws > 0
    assert misa.misa_page_workspace_bytes(misa.cache(4, 8, 0, 16, 0, 0, 0, 0)) == 0
    for i in range(8):
        assert lib.misa_page_compact(r, *[None if j == i else FAKE for j in range(8)], FAKE, ws, None) == -1
    assert lib.misa_page_compact(r, *[FAKE] * 8, FAKE, ws - 1, None) == -3
    assert lib.misa_page_compact(r, *[FAKE] * 8, None, ws, None) == -3


def test_copy_refuses(misa):
    lib = misa.lib()

    def call(data=FAKE, page_bytes=64, planes=2, n_buffers=1, pages=10, n=3, src=FAKE, dst=FAKE):
        b = (misa.misa_page_buffer * 9)(*[misa.misa_page_buffer(data, page_bytes, planes)] * 9)
        return lib.misa_page_copy(b, n_buffers, pages, n, src, dst, None)

    for change in (dict(data=None), dict(data=FAKE + 4), dict(page_bytes=0), dict(page_bytes=6), dict(page_bytes=-4),
                   dict(planes=0), dict(n_buffers=0), dict(pages=0), dict(n=-1), dict(src=None), dict(dst=FAKE + 4)):
        assert call(**change) == -1, change
    assert call(n_buffers=9) == -2
    assert call(page_bytes=1 << 31, planes=65536, n=4096) == -2  # more workgroups than a grid holds
    assert call(page_bytes=1 << 31, planes=65536, pages=1 << 24, n=0) == -2  # offsets beyond 64 bits
    assert call(page_bytes=1 << 31, planes=1 << 15, pages=1 << 17, n=0) == -2
    assert call(page_bytes=1 << 31, planes=1 << 14, pages=1 << 17, n=0) == 0
    assert lib.misa_page_copy(None, 1, 10, 3, FAKE, FAKE, None) == -1
    assert call(n=0, src=None, dst=None) == 0


def test_norm_refuses(misa):
    lib = misa.lib()

    def call(rows=2, n=64, groups=1, xt=1, ot=2, eps=1e-6, x=FAKE, res=None, w=FAKE, s=None, out=FAKE, scale=FAKE):
        return lib.misa_rms_norm(rows, n, groups, xt, ot, eps, x, res, w, s, out, scale, None)

    for change in (dict(rows=-1), dict(n=0), dict(groups=0), dict(groups=5), dict(xt=3), dict(ot=-1), dict(eps=-1.0),
                   dict(eps=math.nan), dict(x=None), dict(w=None), dict(out=None), dict(scale=None), dict(x=FAKE + 8),
                   dict(res=FAKE + 2), dict(s=FAKE + 4)):
        assert call(**change) == -1, change
    assert call(xt=2) == -2 and call(n=32769) == -2 and call(rows=1 << 24) == -2
    assert call(rows=0, x=None, w=None, out=None, scale=None) == 0


def test_binding_raises(misa):
    with pytest.raises(misa.MisaError, match="misa_page_free"):
        misa.misa_page_free(misa.cache(4, 8, 40, 16, 0, 0, 0, 0), -1, FAKE, FAKE, FAKE, FAKE, stream=0)


def test_binding_refuses_host_and_strided_tensors(misa):
    c = misa.cache(4, 8, 40, 16, 0, 0, 0, 0)
    host = torch.zeros(32, dtype=torch.int32)
    with pytest.raises(ValueError, match="contiguous and on the device"):
        misa.misa_page_free(c, 1, host, FAKE, FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="contiguous and on the device"):
        misa.page_buffers([(host, 1, 4)])


class Elsewhere:
    """What the binding asks of a tensor, on a device that need not be there."""

    def __init__(self, dtype, device):
        self.dtype, self.device = dtype, device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE

    def numel(self):
        return 1

    element_size = numel


def test_binding_refuses_wide_integers(misa):
    """A list of 64-bit integers would be read as twice as many."""
    c = misa.cache(4, 8, 40, 16, 2, 128, 128, misa.MISA_BF16)
    wide = Elsewhere(torch.int64, 0)
    calls = {
        "misa_attend": ([c, 8, 4, 0.1] + [FAKE] * 10 + [None], (9, 10, 11)),  # table, lengths, idx
        "misa_page_write": ([c, 1] + [FAKE] * 9, (2, 3, 10)),
        "misa_page_extend": ([c, 1] + [FAKE] * 6, (2, 3, 4, 5, 6)),
        "misa_page_fork": ([c, 1] + [FAKE] * 8, (2, 3, 4, 5, 6)),
        "misa_page_free": ([c, 1] + [FAKE] * 4, (2, 3, 4, 5)),
        "misa_page_compact": ([c] + [FAKE] * 8 + [None], (1, 2)),
    }
    for name, (args, places) in calls.items():
        for i in places:
            with pytest.raises(ValueError, match="must be torch.int32, not torch.int64"):
                getattr(misa, name)(*[wide if j == i else x for j, x in enumerate(args)], stream=0)


def test_binding_refuses_tensors_apart(misa):
    c = misa.cache(4, 8, 40, 16, 0, 0, 0, 0)
    here, there = Elsewhere(torch.int32, 0), Elsewhere(torch.int32, 1)
    with pytest.raises(ValueError, match="on the device"):
        misa.misa_page_free(c, 1, there, here, here, here, stream=0)
    with pytest.raises(ValueError, match="on the device"):
        misa.misa_page_free(c, 1, FAKE, Elsewhere(torch.int32, -1), FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="on the device"):
        misa.page_buffers([(here, 1, 4), (there, 1, 4)])


# ------------------------------------------------------------------ inputs


def _pools(c, gen, misa):
    """CPU pools, every slot NaN until _fill names it."""
    fp8 = c.kv_dtype == misa.MISA_FP8_E4M3
    shape = (c.pages, c.kv_heads, c.page_tokens)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    latent = c.dk != c.dv
    k = torch.full((*shape, c.dk), math.nan).to(dt)
    v = None if latent else torch.full((*shape, c.dv), math.nan).to(dt)
    ks = torch.full(shape, math.nan) if fp8 else None
    vs = torch.full(shape, math.nan) if fp8 and not latent else None
    return k, v, ks, vs


def _fill(pools, page, slot, gen):
    k, v, ks, vs = pools
    for pool, scale in ((k, ks), (v, vs)):
        if pool is None:
            continue
        x = torch.randn(len(page), pool.shape[1], pool.shape[3], generator=gen)
        x = (x * (60 if scale is not None else 1)).to(pool.dtype)
        if pool.dtype == torch.float8_e4m3fn:
            pool.view(torch.uint8)[page, :, slot] = x.view(torch.uint8)
        else:
            pool[page, :, slot] = x
        if scale is not None:
            scale[page, :, slot] = (0.5 + torch.rand(len(page), pool.shape[1], generator=gen)) / 60


def _table(c, lengths, gen, holes=()):
    """Random distinct pages for the rows' tokens; `holes`: (row, entry, value) put in afterwards."""
    ids = torch.randperm(c.pages, generator=gen).tolist()
    table = torch.full((c.rows, c.row_pages), -1, dtype=torch.int32)
    for r, n in enumerate(lengths):
        for s in range(ref.up(n, c.page_tokens)):
            table[r, s] = ids.pop()
    for r, s, x in holes:
        table[r, s] = x
    return table


def _cuda(*xs):
    return [x if x is None else x.cuda() for x in xs]


def _run_attend(misa, c, heads, k, scale, q, pools, table, lengths, idx, stream=None, want_lse=True):
    kp, vp, ks, vs = _cuda(*pools)
    q, table, lengths, idx = _cuda(q, table, lengths, idx)
    guard = 64  # values behind the outputs that must stay
    n_out, n_lse = c.rows * heads * c.dv, c.rows * heads
    out = torch.full((n_out + guard,), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((n_lse + guard,), 7.0, device="cuda")
    need = misa.misa_attend_workspace_bytes(c, heads, k)
    ws = torch.full((need + guard,), 0xFF, device="cuda", dtype=torch.uint8)  # NaN to whoever reads it unwritten
    misa.misa_attend(c, heads, k, scale, q, kp, ks, vp, vs, table, lengths, idx, out, lse if want_lse else None,
                     ws[:need] if need else None, stream)
    torch.cuda.synchronize()
    assert torch.all(out[n_out:] == 7) and torch.all(lse[n_lse:] == 7) and torch.all(ws[need:] == 0xFF)
    return out[:n_out].view(c.rows, heads, c.dv).cpu(), lse[:n_lse].view(c.rows, heads).cpu()


def _check_attend(misa, c, heads, k, scale, q, pools, table, lengths, idx):
    got, lse = _run_attend(misa, c, heads, k, scale, q, pools, table, lengths, idx)
    out, want_lse, out_tol, lse_tol = ref.attend(c, heads, k, scale, q, pools[0], pools[2], pools[1], pools[3], table,
                                                 lengths, idx)
    off = (got.double() - out).abs()
    assert not torch.isnan(got).any()
    assert torch.all(off <= out_tol), (off - out_tol).max()
    empty = want_lse == -math.inf
    assert torch.equal(lse.double() == -math.inf, empty)
    assert torch.all(((lse.double() - want_lse).abs() <= lse_tol)[~empty])
    return got, lse


def _attend_case(misa, dk, dv, kv_heads, heads, P, lengths, dtype, k=0, seed=0, spare=3, row_pages=None, holes=()):
    gen = torch.Generator().manual_seed(seed)
    row_pages = row_pages or max(1, max(ref.up(n, P) for n in lengths))
    pages = sum(ref.up(n, P) for n in lengths) + spare
    c = misa.cache(len(lengths), row_pages, pages, P, kv_heads, dk, dv, dtype)
    table = _table(c, lengths, gen, holes)
    pools = _pools(c, gen, misa)
    at = [(int(table[r, s // P]), s % P) for r, n in enumerate(lengths) for s in range(n)]
    at = [x for x in at if 0 <= x[0] < pages]
    if at:
        page, slot = (torch.tensor(x) for x in zip(*at))
        _fill(pools, page, slot, gen)
    q = (2 * torch.randn(len(lengths), heads, dk, generator=gen)).bfloat16()
    idx = None
    if k:  # out of order, with padding, tokens behind the row's end and far out of range
        idx = torch.full((len(lengths), k), -1, dtype=torch.int32)
        for r, n in enumerate(lengths):
            pick = torch.randperm(n, generator=gen)[:max(0, k - 2)]
            idx[r, : len(pick)] = pick.int()
            if k > 2 and len(pick) < k:
                idx[r, -1] = n
            if r % 2:
                idx[r] = idx[r][torch.randperm(k, generator=gen)]
    return c, heads, k, dk ** -0.5, q, pools, table, torch.tensor(lengths, dtype=torch.int32), idx


DIMS = [(64, 64), (128, 128), (256, 256), (576, 512)]


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("share", [1, 5, 16, 17, 40])
def test_attend_head_layouts(misa, dk, dv, share, fp8):
    """Query heads per cached head below, at and above a matrix tile's 16 rows; ragged rows, one of them empty."""
    kv = 1 if dk != dv else 3
    case = _attend_case(misa, dk, dv, kv, kv * share, 16, [77, 0, 1, 130, 16], 2 if fp8 else 1, seed=share)
    _log(f"[gpu] attend dk {dk} kv {kv} share {share} fp8 {fp8}")
    _check_attend(misa, *case)


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("P", [1, 7, 16, 24, 64, 100])
def test_attend_pages_and_lists(misa, dk, dv, P, fp8):
    """Pages of odd sizes that end inside a tile; lists out of order, longer and shorter than the row."""
    kv = 1 if dk != dv else 2
    for k in (0, 1, 50, 131):
        case = _attend_case(misa, dk, dv, kv, kv * 4, P, [200, 33, 0, 2], 2 if fp8 else 1, k=k, seed=P + k, row_pages=250)
        _log(f"[gpu] attend dk {dk} P {P} k {k} fp8 {fp8}")
        _check_attend(misa, *case)


@gpu
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
def test_attend_lengths(misa, n):
    for dk, dv, dtype in ((128, 128, 1), (128, 128, 2), (64, 64, 1), (576, 512, 1)):
        _log(f"[gpu] attend n {n} dk {dk} dtype {dtype}")
        _check_attend(misa, *_attend_case(misa, dk, dv, 1, 4, 32, [n, max(0, n - 1)], dtype, seed=n))


@gpu
@pytest.mark.parametrize("k", [0, 64])
def test_attend_missing_pages(misa, k):
    """Table entries that name no page hide their tokens; a row of them is empty."""
    holes = [(0, 0, -1), (0, 3, 1 << 20), (0, 4, -(1 << 30)), (1, 0, -1), (1, 1, -1), (1, 2, 10 ** 6), (2, 1, -7)]
    for dtype in (1, 2):
        case = _attend_case(misa, 128, 128, 2, 8, 16, [100, 40, 60], dtype, k=k, seed=3, holes=holes)
        _log(f"[gpu] attend holes k {k} dtype {dtype}")
        got, lse = _check_attend(misa, *case)
        assert torch.all(got[1] == 0) and torch.all(lse[1] == -math.inf)


@gpu
def test_attend_bad_lengths_and_lists(misa):
    """Lengths below zero and beyond the table, list entries of any value: clipped or ignored."""
    case = list(_attend_case(misa, 128, 128, 2, 8, 16, [64, 64, 64, 64], 1, seed=4))
    lengths = torch.tensor([-5, 1 << 30, 64, -(1 << 31)], dtype=torch.int32)
    case[7] = lengths
    _log("[gpu] attend bad lengths")
    _check_attend(misa, *case)
    case[2], case[8] = 8, torch.tensor([[-1, 3, -(1 << 31), (1 << 31) - 1, 64, 63, 5, 5]] * 4, dtype=torch.int32)
    _check_attend(misa, *case)  # the token listed twice counts twice


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_attend_extreme_scores(misa, fp8):
    """Scores far apart (one token takes all), all equal, and a zero scale (the plain mean)."""
    c, heads, k, scale, q, pools, table, lengths, idx = _attend_case(misa, 128, 128, 1, 8, 16, [300, 75], 2 if fp8 else 1, seed=5)
    for qq, sc in ((q * 50, scale), (q * 0, scale), (q, 0.0), (q, -scale)):
        _check_attend(misa, c, heads, k, sc, qq, pools, table, lengths, idx)
    # a visible NaN or infinity reaches its own head's result and no other
    pools[0][table[0, 0], 0, 3, 5] = math.nan
    got, lse = _run_attend(misa, c, heads, k, scale, q, pools, table, lengths, idx)
    assert torch.isnan(got[0]).all() and torch.isnan(lse[0]).all() and not torch.isnan(got[1]).any()


@gpu
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("share,k", [(4, 0), (4, 60), (20, 0), (40, 60)])
def test_attend_infinite_values(misa, dk, share, k):
    """Infinite values of visible tokens give infinities of their sign in their dimension alone, both signs NaN."""
    case = _attend_case(misa, dk, dk, 2, 2 * share, 16, [3000, 75], 1, k=k, seed=dk + share)
    c, heads, k, scale, q, pools, table, lengths, idx = case
    s, t = (int(x) for x in idx[0, :2]) if k else (5, 2100)
    for token, dim, value in ((s, 0, math.inf), (t, 1, -math.inf), (s, 2, math.inf), (t, 2, math.inf), (s, 3, math.inf),
                              (t, 3, -math.inf), (t, dk - 1, math.inf)):
        pools[1][table[0, token // 16], 1, token % 16, dim] = value
    _log(f"[gpu] attend infinite values dk {dk} share {share} k {k}")
    got, lse = _run_attend(misa, *case)
    want, want_lse, tol, lse_tol = ref.attend(c, heads, k, scale, q, pools[0], pools[2], pools[1], pools[3], table, lengths, idx)
    far = ~torch.isfinite(want)
    assert far.sum() == 5 * share
    assert torch.equal(torch.nan_to_num(got.double()[far], nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want[far], nan=7.0, posinf=8.0, neginf=9.0))
    assert torch.all((got.double() - want).abs()[~far] <= tol[~far])
    assert torch.all((lse.double() - want_lse).abs() <= lse_tol)


@gpu
def test_attend_splits_long_rows(misa):
    """One long row beside short ones: the split row joined, without lse too, twice the same bits."""
    for dk, dv, dtype, k in ((128, 128, 2, 0), (128, 128, 1, 3000), (576, 512, 1, 0)):
        kv = 1 if dk != dv else 2
        case = _attend_case(misa, dk, dv, kv, kv * 8, 64, [20011, 5, 0], dtype, k=k, seed=6)
        _log(f"[gpu] attend long dk {dk} k {k}")
        got, lse = _check_attend(misa, *case)
        again, _ = _run_attend(misa, *case, want_lse=False)
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@gpu
@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, 1), (64, 64, 2), (128, 128, 1), (128, 128, 2), (256, 256, 1), (256, 256, 2)])
def test_attend_large_caches(misa, dk, dv, dtype):
    """Caches of more than 64 MB, read with loads that are not kept; a row of a few tokens beside a long one."""
    n = (70 << 20) // (2 * (dk + dv) * (2 if dtype == 1 else 1))
    case = _attend_case(misa, dk, dv, 1, 2, 64, [n, 77], dtype, seed=8)
    _log(f"[gpu] attend large dk {dk} dtype {dtype} n {n}")
    _check_attend(misa, *case)


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dk,share", [(64, 4), (64, 20), (64, 40), (128, 4), (128, 20), (128, 40), (256, 4), (256, 20)])
def test_attend_dense_stages(misa, dk, share, fp8):
    """Whole rows of several stages of 2048 tokens, hidden tokens at their edges: one and two tiles of query heads with
    loads that are not kept, and two chunks of heads with loads that are."""
    lengths = [0] * 1024
    lengths[0], lengths[5], lengths[900], lengths[1023] = 5000, 2049, 4097, 77
    holes = [(0, 127, -1), (0, 128, -1), (0, 256, -1), (5, 128, -1), (900, 0, -1)]
    case = _attend_case(misa, dk, dk, 1, share, 16, lengths, 2 if fp8 else 1, seed=share, row_pages=313, holes=holes)
    _log(f"[gpu] dense stages {dk} share {share} fp8 {fp8}")
    _check_attend(misa, *case)


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("heads", [64, 65, 128])
def test_attend_latent_stages(misa, heads, fp8):
    """Splits of several stages of 512 tokens, whose slots are filled again while buffers change hands; hidden tokens at
    a stage's edges; one chunk of 64 query heads, a second one of a single head, two whole ones.  Many rows by the
    table, few with tokens, so that a row has few splits."""
    lengths = [0] * 64
    lengths[3], lengths[17], lengths[40], lengths[63] = 8191, 2049, 513, 1100
    holes = [(3, 31, -1), (3, 32, -1), (3, 64, -1), (3, 300, -1), (17, 33, -1), (17, 128, -1), (40, 32, -1), (63, 0, -1)]
    case = _attend_case(misa, 576, 512, 1, heads, 16, lengths, 2 if fp8 else 1, seed=heads, row_pages=512, holes=holes)
    _log(f"[gpu] latent stages {heads} fp8 {fp8}")
    _check_attend(misa, *case)


@gpu
def test_attend_far_offsets(misa):
    """Pools beyond 2^32 bytes and 2^31 elements: the rows live in the last pages."""
    P, kv, d = 64, 8, 128
    pages = (1 << 32) // (P * kv * d) + 100
    c = misa.cache(2, 4, pages, P, kv, d, d, misa.MISA_BF16)
    gen = torch.Generator().manual_seed(7)
    kp = torch.empty(pages, kv, P, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    lengths = torch.tensor([200, 70], dtype=torch.int32)
    small = misa.cache(2, 4, 6, P, kv, d, d, misa.MISA_BF16)
    table = _table(small, [200, 70], gen)
    pools = _pools(small, gen, misa)
    n = 6 * P
    _fill(pools, torch.arange(n) // P, torch.arange(n) % P, gen)
    kp[pages - 6:], vp[pages - 6:] = pools[0].cuda(), pools[1].cuda()
    q = torch.randn(2, 16, d, generator=gen).bfloat16()
    want = _run_attend(misa, small, 16, 0, 0.1, q, pools, table, lengths, None)
    far = torch.where(table >= 0, table + pages - 6, -1)
    _log("[gpu] attend far offsets")
    got = _run_attend(misa, c, 16, 0, 0.1, q, (kp, vp, None, None), far, lengths, None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and a write there
    new = torch.randn(1, kv, d, generator=gen).bfloat16().cuda()
    row, pos = _cuda(torch.tensor([1], dtype=torch.int32), torch.tensor([69], dtype=torch.int32))
    misa.misa_page_write(c, 1, row, pos, new, new, kp, None, vp, None, far.cuda())
    torch.cuda.synchronize()
    assert torch.equal(kp[far[1, 1], :, 5], new[0]) and torch.equal(vp[far[1, 1], :, 5], new[0])


# ------------------------------------------------------------------ writes


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("P,n", [(1, 1), (7, 20), (16, 33), (64, 300)])
def test_page_write(misa, dk, dv, P, n, fp8):
    """Tokens land in their slots and nowhere else; padding and impossible entries are skipped."""
    gen = torch.Generator().manual_seed(n)
    kv, rows = 1 if dk != dv else 3, 3
    row_pages = ref.up(n, P) + 1
    c = misa.cache(rows, row_pages, rows * row_pages + 2, P, kv, dk, dv, 2 if fp8 else 1)
    table = _table(c, [row_pages * P] * rows, gen, holes=[(2, 0, -1), (2, row_pages - 1, c.pages)])
    pools = _pools(c, gen, misa)
    want = [x if x is None else x.clone() for x in pools]
    row = torch.randint(-1, rows + 1, (n,), generator=gen).int()
    pos = torch.randperm(row_pages * P + 2, generator=gen)[:n].int() - 1
    if n > 5:
        row[3], pos[3], row[4], pos[4] = -(1 << 31), 0, 0, (1 << 31) - 1
    kn = torch.randn(n, kv, dk, generator=gen).bfloat16()
    kn[0] = 0
    if n > 1:
        kn[1] *= 2.0 ** -90
        kn[1, 0, :4] = torch.tensor([2.0 ** -110, -(2.0 ** -130), 0.0, -0.0])
        kn[n // 2] *= 1e30
    vn = None if dk != dv else 3 * torch.randn(n, kv, dv, generator=gen).bfloat16()
    kp, vp, ks, vs = _cuda(*pools)
    _log(f"[gpu] write dk {dk} P {P} n {n} fp8 {fp8}")
    misa.misa_page_write(c, n, *_cuda(row, pos, kn, vn), kp, ks, vp, vs, table.cuda())
    torch.cuda.synchronize()
    hit = torch.zeros(c.pages, P, dtype=torch.bool)
    got = [x if x is None else x.cpu() for x in (kp, vp, ks, vs)]
    for i in range(n):
        r, s = int(row[i]), int(pos[i])
        if not (0 <= r < rows and 0 <= s < row_pages * P):
            continue
        page, slot = int(table[r, s // P]), s % P
        if not 0 <= page < c.pages:
            continue
        hit[page, slot] = True
        for new, pool, scale in ((kn, got[0], got[2]), (vn, got[1], got[3])):
            if new is None:
                continue
            if fp8:
                ref.check_e4m3(pool[page, :, slot], scale[page, :, slot], new[i].double())
            else:
                assert torch.equal(pool[page, :, slot].view(torch.int16), new[i].view(torch.int16))
    for a, b in zip(got, want):  # every other slot as it was, bit for bit
        if a is not None:
            bits = torch.uint8 if a.dtype == torch.float8_e4m3fn else torch.int16 if a.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(a.view(bits)[~hit[:, None].expand(a.shape[:3])], b.view(bits)[~hit[:, None].expand(b.shape[:3])])


@gpu
def test_page_write_nan_and_infinity(misa):
    c = misa.cache(1, 1, 1, 4, 1, 128, 128, misa.MISA_FP8_E4M3)
    kn = torch.randn(2, 1, 128).bfloat16()
    kn[0, 0, 7], kn[1, 0, 9] = math.nan, math.inf
    pools = _cuda(*_pools(c, None, misa))
    i32 = dict(dtype=torch.int32, device="cuda")
    misa.misa_page_write(c, 2, torch.zeros(2, **i32), torch.arange(2, **i32), kn.cuda(), kn.cuda(), pools[0], pools[2],
                         pools[1], pools[3], torch.zeros(1, 1, **i32))
    code, scale = pools[0][0, 0].cpu(), pools[2][0, 0].cpu()
    ref.check_e4m3(code[0], scale[0], kn[0, 0].double())
    assert torch.isnan(code[1].float())[9] and torch.isnan(code[1].float()).sum() == 1 and torch.isinf(scale[1])


@gpu
@pytest.mark.parametrize("dk,dv", DIMS)
def test_page_write_ties(misa, dk, dv):
    """Codes are the exact quotients' (64 bits tell a bf16 quotient from a tie), ties to even."""
    gen = torch.Generator().manual_seed(dk)
    n, kv = 400, 1 if dk != dv else 3
    c = misa.cache(1, 25, 25, 16, kv, dk, dv, misa.MISA_FP8_E4M3)
    new = torch.randn(n, kv, dk, generator=gen).bfloat16()
    new[0] = torch.arange(dk).bfloat16() / 8
    new[1] *= 2.0 ** 120
    new[2] *= 2.0 ** -95
    kp, vp, ks, vs = _cuda(*_pools(c, gen, misa))
    i32 = dict(dtype=torch.int32, device="cuda")
    _log(f"[gpu] write ties {dk}")
    v = None if vp is None else -new
    misa.misa_page_write(c, n, torch.zeros(n, **i32), torch.arange(n, **i32), *_cuda(new, v), kp, ks, vp, vs,
                         torch.arange(25, **i32).view(1, 25))
    want = (new.double() * 448 / new.double().abs().amax(-1, keepdim=True)).to(torch.float8_e4m3fn).float()
    for pool, sign in ((kp, 1), (vp, -1)):
        if pool is not None:
            got = pool.cpu().float().transpose(1, 2).reshape(n, kv, dk)
            assert torch.equal(got, sign * want)


# ------------------------------------------------------------------ bookkeeping


class Device:
    """A Book's arrays on the GPU, the calls on them, and the comparison."""

    def __init__(self, misa, book):
        self.misa, self.c = misa, book.c
        self.table, self.lengths, self.refs = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                                               (book.table, book.lengths, book.refs))

    def ints(self, values):
        return torch.tensor(list(values), dtype=torch.int32, device="cuda")

    def out(self, n):
        return torch.full((n + 8,), 77, dtype=torch.int32, device="cuda")

    @staticmethod
    def taken(x, n):
        assert torch.all(x[n:] == 77)
        return x[:n].tolist()

    def extend(self, row, count):
        ok = self.out(len(row))
        self.misa.misa_page_extend(self.c, len(row), self.ints(row), self.ints(count), self.table, self.lengths,
                                   self.refs, ok)
        return self.taken(ok, len(row))

    def fork(self, parent, child):
        n = len(parent)
        outs = [self.out(n) for _ in range(3)]
        self.misa.misa_page_fork(self.c, n, self.ints(parent), self.ints(child), self.table, self.lengths, self.refs,
                                 *outs)
        return tuple(self.taken(x, n) for x in outs)

    def free(self, row):
        self.misa.misa_page_free(self.c, len(row), self.ints(row), self.table, self.lengths, self.refs)

    def compact(self, in_place):
        c, half = self.c, max(1, self.c.pages // 2)
        table = self.table if in_place else torch.full_like(self.table, 55)
        refs = self.refs if in_place else torch.full_like(self.refs, 55)
        outs = [self.out(n) for n in (c.pages, 1, half, half)]
        ws = torch.full((self.misa.misa_page_workspace_bytes(c),), 0xFF, dtype=torch.uint8, device="cuda")
        self.misa.misa_page_compact(c, self.table, self.refs, table, refs, *outs, ws)
        self.table, self.refs = table, refs
        m, live, src, dst = (self.taken(x, n) for x, n in zip(outs, (c.pages, 1, half, half)))
        return m, live[0], src, dst

    def same(self, book):
        assert self.lengths.tolist() == book.lengths.tolist()
        assert torch.equal(self.table.cpu().long(), torch.from_numpy(book.table))
        assert self.refs.tolist() == book.refs.tolist()


def _book(misa, rows, row_pages, pages, P):
    c = misa.cache(rows, row_pages, pages, P, 1, 64, 64, misa.MISA_BF16)
    return ref.Book(c, np.full((rows, row_pages), -1), np.zeros(rows), np.zeros(pages))


@gpu
@pytest.mark.parametrize("rows,row_pages,pages,P,seed", [
    (1, 1, 1, 1, 0), (6, 5, 17, 4, 1), (40, 9, 200, 16, 2), (300, 40, 6000, 3, 3), (64, 700, 9000, 1, 4),
    (20, 30, 333, 100, 5),
])
def test_bookkeeping_sequences(misa, rows, row_pages, pages, P, seed):
    """Random runs of extend, fork, free and compact, with impossible and repeated entries and a pool that runs out."""
    rng = np.random.default_rng(seed)
    book = _book(misa, rows, row_pages, pages, P)
    dev = Device(misa, book)
    for step in range(24):
        n = int(rng.integers(1, 2 * rows + 2))
        op = rng.choice(["extend", "extend", "fork", "free", "compact"])
        _log(f"[gpu] bookkeeping {rows} x {row_pages} of {pages}: step {step} {op} {n}")
        if op == "extend":
            row = rng.integers(-1, rows + 1, n).tolist()
            count = rng.integers(-1, max(2, row_pages * P // 2), n).tolist()
            assert dev.extend(row, count) == book.extend(row, count)
        elif op == "fork":
            parent, child = rng.integers(-1, rows + 1, n).tolist(), rng.integers(-1, rows + 1, n).tolist()
            assert dev.fork(parent, child) == book.fork(parent, child)
        elif op == "free":
            row = rng.integers(-1, rows + 1, max(1, n // 3)).tolist()
            dev.free(row)
            book.free(row)
        else:
            assert dev.compact(bool(step % 2)) == book.compact()
        dev.same(book)
        counted = np.bincount(book.table[book.table >= 0], minlength=pages)
        assert (counted == book.refs).all()  # the reference's own invariant


@gpu
def test_bookkeeping_long_lists(misa):
    """The largest list, pages beyond one scan's chunk, and entries that need many pages each."""
    rows, row_pages, pages, P = 4096, 12, 30000, 8
    rng = np.random.default_rng(9)
    book = _book(misa, rows, row_pages, pages, P)
    book.refs[rng.permutation(pages)[:9000]] = 3  # pages in use elsewhere
    dev = Device(misa, book)
    row, count = rng.permutation(rows).tolist(), rng.integers(0, 60, rows).tolist()
    assert dev.extend(row, count) == book.extend(row, count)
    dev.same(book)
    gone = rng.permutation(rows)[:2000].tolist()
    dev.free(gone)
    book.free(gone)
    parent = rng.integers(0, rows, 4096).tolist()
    child = (gone * 3)[:4096]
    assert dev.fork(parent, child) == book.fork(parent, child)
    dev.same(book)
    assert dev.compact(False) == book.compact()
    dev.same(book)


@gpu
@pytest.mark.parametrize("live", ["none", "all", "low", "high", "odd"])
@pytest.mark.parametrize("pages", [1, 2, 255, 257, 5000, 8192, 8193, 20481, 65536, 70001])
def test_compact_pools(misa, pages, live):
    book = _book(misa, 3, 7, pages, 4)
    at = np.arange(pages)
    use = {"none": at < 0, "all": at >= 0, "low": at < pages // 3, "high": at >= pages - pages // 3, "odd": at % 2 == 1}[live]
    book.refs[use] = 2
    book.table[:] = np.arange(21).reshape(3, 7) * 977 % max(1, pages) - 1
    dev = Device(misa, book)
    _log(f"[gpu] compact {pages} {live}")
    assert dev.compact(True) == book.compact()
    dev.same(book)


@gpu
@pytest.mark.parametrize("page_bytes", [4, 12, 64, 1000, 2004, 4096, 5004, 16384, 16400, 40012, 70000])
def test_page_copy(misa, page_bytes):
    """Pages land in every plane of every buffer; bad pairs are skipped, the rest stays."""
    gen = torch.Generator().manual_seed(page_bytes)
    pages, planes = 9, (1, 3)
    data = [torch.randint(0, 256, (p, pages, b), generator=gen, dtype=torch.uint8) for p, b in zip(planes, (page_bytes, 32))]
    src = torch.tensor([1, -1, 5, 9, 3, 7, 2], dtype=torch.int32)
    dst = torch.tensor([0, 4, 6, 8, 1 << 30, 7, -1], dtype=torch.int32)
    want = [x.clone() for x in data]
    for x in want:
        x[:, 0], x[:, 6] = x[:, 1].clone(), x[:, 5].clone()
    dev = [torch.cat([x.flatten(), torch.full((64,), 9, dtype=torch.uint8)]).cuda() for x in data]
    bufs = misa.page_buffers([(dev[0], planes[0], page_bytes), (dev[1], planes[1], 32)])
    _log(f"[gpu] copy {page_bytes}")
    misa.misa_page_copy(bufs, pages, 7, src.cuda(), dst.cuda())
    torch.cuda.synchronize()
    for x, w in zip(dev, want):
        assert torch.equal(x.cpu()[:-64], w.flatten()) and torch.all(x[-64:] == 9)


@gpu
def test_page_copy_long_lists(misa):
    """More pieces than workgroups of a grid: pairs far down the list, the others skipped."""
    pages, n = 50, 200000
    data = torch.randint(0, 256, (2, pages, 64), dtype=torch.uint8)
    src = torch.full((n,), -1, dtype=torch.int32)
    dst = src.clone()
    want = data.clone()
    for i, (a, b) in enumerate([(3, 4), (10, 0), (49, 20)]):
        src[n - 1 - 70000 * i], dst[n - 1 - 70000 * i] = a, b
        want[:, b] = data[:, a]
    dev = data.cuda()
    _log("[gpu] copy long list")
    misa.misa_page_copy(misa.page_buffers([(dev, 2, 64)]), pages, n, src.cuda(), dst.cuda())
    assert torch.equal(dev.cpu(), want)


@gpu
def test_captured_bookkeeping(misa):
    """Free, fork, copy, extend and compact in one graph, replayed with eager work between, each replay against the
    reference."""
    rng = np.random.default_rng(12)
    book = _book(misa, 24, 12, 300, 4)
    dev = Device(misa, book)
    first = list(range(12)), rng.integers(0, 40, 12).tolist()
    assert dev.extend(*first) == book.extend(*first)
    n = 8
    rows, parent, child, grow, count = (dev.ints([0] * n) for _ in range(5))
    src, dst, ok, more = (dev.ints([0] * n) for _ in range(4))
    pmap, live = dev.ints([0] * 300), dev.ints([0])
    msrc, mdst = dev.ints([0] * 150), dev.ints([0] * 150)
    ws = torch.empty(misa.misa_page_workspace_bytes(book.c), dtype=torch.uint8, device="cuda")
    data = torch.arange(300, dtype=torch.int32, device="cuda").view(300, 1).repeat(1, 4)
    bufs = misa.page_buffers([(data, 1, 16)])

    def step():
        c = book.c
        misa.misa_page_free(c, n, rows, dev.table, dev.lengths, dev.refs)
        misa.misa_page_fork(c, n, parent, child, dev.table, dev.lengths, dev.refs, src, dst, ok)
        misa.misa_page_copy(bufs, 300, n, src, dst)
        misa.misa_page_extend(c, n, grow, count, dev.table, dev.lengths, dev.refs, more)
        misa.misa_page_compact(c, dev.table, dev.refs, dev.table, dev.refs, pmap, live, msrc, mdst, ws)
        misa.misa_page_copy(bufs, 300, 150, msrc, mdst)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    state = [x.clone() for x in (dev.table, dev.lengths, dev.refs)]
    with torch.cuda.stream(side):
        step()  # all entries name row 0: a first run before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for x, y in zip((dev.table, dev.lengths, dev.refs), state):
        x.copy_(y)
    pool = np.arange(300)[:, None].repeat(4, 1)
    data.copy_(torch.from_numpy(pool.astype(np.int32)))
    for turn in range(5):
        values = [rng.integers(-1, 25, n), rng.integers(-1, 25, n), rng.integers(-1, 25, n), rng.integers(-1, 25, n),
                  rng.integers(0, 12, n)]
        for x, y in zip((rows, parent, child, grow, count), values):
            x.copy_(torch.from_numpy(y.astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        r, p, h, g, k = (v.tolist() for v in values)
        book.free(r)
        fsrc, fdst, fok = book.fork(p, h)
        for a, b in zip(fsrc, fdst):
            if a >= 0:
                pool[b] = pool[a]
        fmore = book.extend(g, k)
        wmap, wlive, csrc, cdst = book.compact()
        moved = pool.copy()
        for a, b in zip(csrc, cdst):
            if a >= 0:
                moved[b] = pool[a]
        pool = moved
        assert (src.tolist(), dst.tolist(), ok.tolist(), more.tolist()) == (fsrc, fdst, fok, fmore), turn
        assert (pmap.tolist(), live.tolist()) == (wmap, [wlive]), turn
        dev.same(book)
        assert (data.cpu().numpy() == pool).all()
        assert int(torch.ones(1000, device="cuda").sum()) == 1000  # eager work between replays


# ------------------------------------------------------------------ the norm


def _check_norm(misa, rows, n, groups, xt, ot, eps, x, residual, weight, in_place=False):
    names = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}
    dx, dr, dw = _cuda(x, residual, weight)
    total = dx if in_place else torch.full((rows * n + 64,), 5.0, device="cuda").to(xt)
    out = torch.full((rows * n + 64,), 5.0, device="cuda").to(ot)
    scale = torch.full((rows + 8,), 5.0, device="cuda")
    misa.misa_rms_norm(rows, n, groups, names[xt], names[ot], eps, dx, dr, dw, total if residual is not None else None,
                       out, scale)
    torch.cuda.synchronize()
    assert torch.all(out[rows * n:].float() == 5) and torch.all(scale[rows if ot == torch.float8_e4m3fn else 0:] == 5)
    y, z, tol = ref.norm(x, residual, weight, groups, eps)
    if residual is not None:
        got = total.flatten().cpu().double()
        assert in_place or torch.all(got[rows * n:] == 5)
        half = ref.BF16_HALF if xt == torch.bfloat16 else ref.F32_HALF
        assert torch.all((got[:rows * n].view(rows, n) - y).abs() <= y.abs() * half + (x.double().abs() + residual.double().abs()) * ref.F32_HALF)
    got = out[:rows * n].cpu().view(rows, n)
    if ot == torch.float8_e4m3fn:
        top = z.abs().amax(-1, keepdim=True).clamp(min=1e-300)
        y8 = z / scale[:rows].cpu().double()[:, None]
        want = ref.e4m3_scale(z)
        assert torch.all((scale[:rows].cpu().double() - want).abs() <= want * 8 * ref.F32_HALF + (tol / 448).amax(-1))
        room = torch.clamp(y8.abs() * ref.E4M3_HALF, min=2.0 ** -10) + 448 * tol / top * 2 + y8.abs() * 8 * ref.F32_HALF
        assert torch.all((got.double() - y8).abs() <= room)
    else:
        half = ref.BF16_HALF if ot == torch.bfloat16 else ref.F32_HALF
        assert torch.all((got.double() - z).abs() <= z.abs() * half * (1 + 2.0 ** -8) + tol * (1 + half))


@gpu
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float8_e4m3fn], ids=["f32", "bf16", "fp8"])
@pytest.mark.parametrize("rows,n,groups", [
    (1, 1, 1), (3, 17, 1), (5, 128, 1), (2, 130, 2), (7, 1000, 1), (2, 4096, 1), (3, 8192, 64), (2, 896, 8), (1, 32768, 1),
    (2, 32768, 256), (9, 512, 4), (3, 2048, 8), (4, 12, 12), (130, 64, 1), (2, 16384, 1), (2, 5120, 40), (1, 20000, 1),
    (5, 7, 1), (300, 8, 1), (33, 9, 1), (70, 127, 1), (9, 513, 1), (3, 4095, 1), (2, 8191, 1), (2, 16383, 1), (2, 32767, 1),
    (7, 1002, 1), (3, 24, 3), (2, 1120, 2), (2, 8000, 8), (40, 96, 12), (2, 30000, 2),
    (19, 200, 1), (9, 256, 2), (6, 251, 1), (5, 1024, 1), (5, 1017, 1), (3, 2048, 16), (5, 1999, 1), (3, 6000, 1), (2, 6143, 1), (3, 6144, 48),
])
def test_norm(misa, rows, n, groups, xt, ot):
    gen = torch.Generator().manual_seed(n)
    x = (torch.randn(rows, n, generator=gen) * (1 + 20 * (torch.rand(n, generator=gen) < 0.02))).to(xt)
    weight = torch.randn(n // groups, generator=gen)
    _log(f"[gpu] norm {rows} x {n} / {groups} {xt} {ot}")
    for residual in (None, (2 * torch.randn(rows, n, generator=gen)).to(xt)):
        _check_norm(misa, rows, n, groups, xt, ot, 1e-6, x, residual, weight)
    _check_norm(misa, rows, n, groups, xt, ot, 1e-6, x, residual, weight, in_place=True)


@gpu
@pytest.mark.parametrize("ot,rows,n,groups", [
    (torch.float8_e4m3fn, 4095, 4096, 1), (torch.float8_e4m3fn, 4096, 4096, 1), (torch.float8_e4m3fn, 4098, 4095, 1),
    (torch.float8_e4m3fn, 2049, 8192, 64), (torch.float8_e4m3fn, 70000, 251, 1), (torch.float8_e4m3fn, 130000, 130, 2),
    (torch.bfloat16, 2047, 4096, 1), (torch.bfloat16, 2048, 4096, 1), (torch.bfloat16, 2050, 4095, 1),
    (torch.bfloat16, 1025, 8192, 64), (torch.bfloat16, 35000, 251, 1),
])
def test_norm_large_outputs(misa, ot, rows, n, groups):
    """Outputs from just below to above 16 MB, from which on they are stored past the caches; rows of odd length, whose
    stores are aligned to an element only."""
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(rows, n, generator=gen).bfloat16()
    _log(f"[gpu] norm large {rows} x {n} / {groups} {ot}")
    _check_norm(misa, rows, n, groups, torch.bfloat16, ot, 1e-6, x, None, torch.randn(n // groups, generator=gen))


@gpu
def test_norm_zero_and_tiny_rows(misa):
    """A row of zeros gives zeros with scale 1; a part of zeros beside others; tiny values under a large eps."""
    x = torch.zeros(3, 1024)
    x[1, 128:256] = torch.randn(128)
    x[2] = 1e-18 * torch.randn(1024)
    weight = torch.ones(128)
    for ot in (torch.float32, torch.float8_e4m3fn):
        _check_norm(misa, 3, 1024, 8, torch.float32, ot, 1e-6, x, None, weight)
    out = torch.empty(1, 1024, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.empty(4, device="cuda")
    misa.misa_rms_norm(1, 1024, 1, 0, 2, 1e-6, x.cuda(), None, torch.ones(1024, device="cuda"), None, out, scale)
    assert torch.all(out.float() == 0) and scale[0] == 1


@gpu
@pytest.mark.parametrize("n,groups", [(64, 1), (1024, 8), (1001, 1), (4096, 1), (12, 4)])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float8_e4m3fn], ids=["f32", "bf16", "fp8"])
def test_norm_far_values(misa, n, groups, ot):
    """Small values with small weights, large ones with large weights: their products leave fp32's range, the result
    does not.  Ordinary rows beside the far ones."""
    gen = torch.Generator().manual_seed(n)
    for value, by in ((1e-16, 1e-25), (1e16, 1e24), (1e-16, 1.0), (1e16, 1e-20)):
        x = torch.randn(5, n, generator=gen)
        x[::2] *= value
        x[3] *= math.sqrt(value)
        _check_norm(misa, 5, n, groups, torch.float32, ot, 0.0, x, None, by * torch.randn(n // groups, generator=gen))


@gpu
@pytest.mark.parametrize("rows,n,groups", [(3, 64, 1), (2, 1024, 8), (5, 1001, 1), (2, 4096, 1), (3, 12, 4), (2, 32768, 1), (2, 30000, 2), (9, 256, 1), (2, 2048, 16)])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float8_e4m3fn], ids=["f32", "bf16", "fp8"])
def test_norm_mean_square_near_the_largest(misa, rows, n, groups, ot):
    """Mean squares up to 3e38, whose sums leave fp32's range; an ordinary row beside them."""
    gen = torch.Generator().manual_seed(n)
    x = (0.9 + 0.2 * torch.rand(rows, n, generator=gen)) * 1.5e19 * (2 * torch.randint(0, 2, (rows, n), generator=gen) - 1)
    x[-1] = torch.randn(n, generator=gen)
    weight = torch.randn(n // groups, generator=gen)
    _log(f"[gpu] norm near the largest {rows} x {n} / {groups} {ot}")
    for xt in (torch.float32, torch.bfloat16):
        _check_norm(misa, rows, n, groups, xt, ot, 1e-6, x.to(xt), None, weight)


@gpu
def test_norm_nan_row_stays_in_its_row(misa):
    x = torch.randn(4, 256)
    x[1, 3], x[2, 5] = math.nan, math.inf
    out = torch.empty(4, 256, device="cuda")
    misa.misa_rms_norm(4, 256, 1, 0, 0, 1e-6, x.cuda(), None, torch.ones(256, device="cuda"), None, out, None)
    bad = torch.isnan(out).any(1).cpu()
    assert bad.tolist() == [False, True, True, False]


# ------------------------------------------------------------------ together


def _step_state(misa, fp8, seed=11):
    """A small serving state: 9 rows, an index cache, a paged cache and one layer's weights of the norms."""
    import synth

    p = synth.small("serve", batch=9, L=600, T=1, H=32, h=8, B=64, k=96, kprime=None, dtype=synth.FP8_E4M3, needles=4, seed=seed)
    x = synth.generate(p)
    gen = torch.Generator().manual_seed(seed)
    P, kv, d, heads = 16, 2, 128, 16
    width = ref.up(p.L, P) + 2
    c = misa.cache(p.batch + 3, width, (p.batch + 3) * width, P, kv, d, d, misa.MISA_FP8_E4M3 if fp8 else misa.MISA_BF16)
    return p, x, gen, c, heads


@gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_serving_step(misa, fp8):
    """A decode step as it is used: extend, norm the hidden state into the indexer's 8-bit queries and newest key,
    pick tokens, write the new keys and values, attend; then fork, free and compact, after which the same attention
    gives the same bits."""
    p, x, gen, c, heads = _step_state(misa, fp8)
    dev, i32 = "cuda", dict(dtype=torch.int32, device="cuda")
    n = p.batch
    table = torch.full((c.rows, c.row_pages), -1, **i32)
    lengths, refs = torch.zeros(c.rows, **i32), torch.zeros(c.pages, **i32)
    kp, vp, ks, vs = (t if t is None else t.cuda() for t in _pools(c, gen, misa))
    rows = torch.arange(n, **i32)
    ok = torch.empty(n, **i32)
    # the prompts
    misa.misa_page_extend(c, n, rows, torch.full((n,), p.L - 1, **i32), table, lengths, refs, ok)
    m = n * (p.L - 1)
    row = torch.arange(n, **i32).repeat_interleave(p.L - 1)
    pos = torch.arange(p.L - 1, **i32).repeat(n)
    kn, vn = (torch.randn(m, c.kv_heads, c.dk, generator=gen).bfloat16().cuda() for _ in range(2))
    misa.misa_page_write(c, m, row, pos, kn, vn, kp, ks, vp, vs, table)
    # one new token a row
    misa.misa_page_extend(c, n, rows, torch.ones(n, **i32), table, lengths, refs, ok)
    assert torch.all(ok == 1) and torch.all(lengths[:n] == p.L) and torch.all(lengths[n:] == 0)
    hidden = torch.randn(n, p.H * p.d, generator=gen).bfloat16().cuda()
    q8 = torch.empty(n, 1, p.H, p.d, dtype=torch.float8_e4m3fn, device=dev)
    qs = torch.empty(n, 1, device=dev)
    misa.misa_rms_norm(n, p.H * p.d, p.H, misa.MISA_BF16, misa.MISA_FP8_E4M3, 1e-6, hidden, None,
                       torch.ones(p.d, device=dev), None, q8, qs)
    k8, k8s = x.k.cuda(), x.k_scale.cuda()
    new8 = torch.empty(n, p.d, dtype=torch.float8_e4m3fn, device=dev)
    new8s = torch.empty(n, device=dev)
    misa.misa_rms_norm(n, p.d, 1, misa.MISA_BF16, misa.MISA_FP8_E4M3, 1e-6, hidden[:, :p.d].contiguous(), None,
                       torch.ones(p.d, device=dev), None, new8, new8s)
    k8[:, -1] = new8
    k8s[:, -1] = new8s
    shp = misa.shape(n, p.L, 1, p.H, p.d, p.B, misa.MISA_FP8_E4M3)
    pooled = torch.empty(n, p.M, p.d, device=dev)
    misa.misa_pool_keys(shp, k8, k8s, pooled)
    sel_heads = torch.empty(n, p.h, **i32)
    # idx covers every row of the cache: the rows behind the batch hold nothing
    idx = torch.full((c.rows, p.k), -1, **i32)
    ws = torch.empty(misa.misa_workspace_bytes(shp, p.h, p.k, p.k), dtype=torch.uint8, device=dev)
    misa.misa_decode_step(shp, p.h, p.k, q8, qs, x.w.cuda(), pooled, k8, k8s, sel_heads, None, idx, None, ws)
    kn1, vn1 = (torch.randn(n, c.kv_heads, c.dk, generator=gen).bfloat16().cuda() for _ in range(2))
    misa.misa_page_write(c, n, rows, lengths[:n] - 1, kn1, vn1, kp, ks, vp, vs, table)
    q = torch.randn(c.rows, heads, c.dk, generator=gen).bfloat16()
    pools = [t if t is None else t.cpu() for t in (kp, vp, ks, vs)]
    for k, list_ in ((0, None), (p.k, idx.cpu())):
        got, lse = _check_attend(misa, c, heads, k, c.dk ** -0.5, q, pools, table.cpu(), lengths.cpu(), list_)
        assert torch.all(got[n:] == 0)
    # fork rows 0 and 1 to the spare ones, free row 0, compact: the children attend as their parents did
    parent, child = torch.tensor([0, 1], **i32), torch.tensor([n, n + 2], **i32)
    src, dst, ok2 = (torch.empty(2, **i32) for _ in range(3))
    misa.misa_page_fork(c, 2, parent, child, table, lengths, refs, src, dst, ok2)
    assert torch.all(ok2 == 1)
    triples = [(t, 1, t[0].numel() * t.element_size()) for t in (kp, vp, ks, vs) if t is not None]
    bufs = misa.page_buffers(triples)
    misa.misa_page_copy(bufs, c.pages, 2, src, dst)
    misa.misa_page_free(c, 1, parent[:1].contiguous(), table, lengths, refs)
    assert table[0].max() == -1
    pmap, live = torch.empty(c.pages, **i32), torch.empty(1, **i32)
    src, dst = (torch.empty(c.pages // 2, **i32) for _ in range(2))
    pws = torch.empty(misa.misa_page_workspace_bytes(c), dtype=torch.uint8, device=dev)
    misa.misa_page_compact(c, table, refs, table, refs, pmap, live, src, dst, pws)
    misa.misa_page_copy(bufs, c.pages, c.pages // 2, src, dst)
    assert int((refs > 0).sum()) == int(live) and torch.all(refs[:int(live)] > 0)
    pools = [t if t is None else t.cpu() for t in (kp, vp, ks, vs)]
    q2 = q.clone()
    q2[n], q2[n + 2] = q[0], q[1]
    for k, list_ in ((0, None), (p.k, idx.cpu())):
        if k:
            list_[n], list_[n + 2] = list_[0], list_[1]
            got_all, lse_all = got, lse
        again, lse2 = _run_attend(misa, c, heads, k, c.dk ** -0.5, q2, pools, table.cpu(), lengths.cpu(), list_)
        if k:
            for a, b in ((n, 0), (n + 2, 1), (1, 1), (5, 5)):
                assert torch.equal(again[a], got_all[b]) and torch.equal(lse2[a], lse_all[b])
        assert torch.all(again[0] == 0) and torch.all(lse2[0] == -math.inf)


@gpu
def test_captured_steps(misa):
    """The calls of a step captured into a graph on a side stream, replayed with eager work between, each replay
    against an eager run of the same inputs.  Two graphs share one workspace."""
    c = misa.cache(3, 40, 130, 16, 2, 128, 128, misa.MISA_FP8_E4M3)
    gen = torch.Generator().manual_seed(21)
    i32 = dict(dtype=torch.int32, device="cuda")
    heads = 8
    table = _table(c, [600, 600, 600], gen).cuda()
    pools = _cuda(*[x if x is None else torch.nan_to_num(x.float(), nan=0.5).to(x.dtype) for x in _pools(c, gen, misa)])
    kp, vp, ks, vs = pools
    q = torch.randn(3, heads, 128, generator=gen).bfloat16().cuda()
    x = torch.randn(3, 2 * 128, generator=gen).bfloat16().cuda()
    rows, pos = torch.arange(3, **i32), torch.tensor([5, 250, 599], **i32)
    lengths = pos + 1
    kn = torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    vn = torch.randn(3, 2, 128, generator=gen).bfloat16().cuda()
    weight = torch.ones(128, device="cuda")
    need = misa.misa_attend_workspace_bytes(c, heads, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(3, heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    lse = [torch.empty(3, heads, device="cuda") for _ in range(3)]

    def step(i, stream=None):
        misa.misa_rms_norm(3, 256, 2, 1, 1, 1e-6, x, None, weight, None, kn, None, stream)
        misa.misa_page_write(c, 3, rows, pos, kn, vn, kp, ks, vp, vs, table, stream)
        misa.misa_attend(c, heads, 0, 0.09, q, kp, ks, vp, vs, table, lengths, None, outs[i], lse[i], ws, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.synchronize()
    graphs = []
    for i in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(i)
        graphs.append(g)
    for turn in range(4):
        x.normal_(generator=None)
        vn.normal_()
        q.normal_()
        pos.random_(0, 600)
        torch.add(pos, 1, out=lengths)
        torch.cuda.synchronize()
        for i in (1, 2):
            graphs[i - 1].replay()
            torch.cuda.synchronize()
            step(0)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], outs[i]) and torch.equal(lse[0], lse[i]), (turn, i)
            assert not torch.isnan(outs[0]).any()


@gpu
@pytest.mark.parametrize("dt", [1, 2], ids=["bf16", "fp8"])
def test_captured_latent_rows_and_long_norms(misa, dt):
    """Attention over a latent cache in splits, and a norm whose rows need more LDS than a launch has by default:
    replays with other inputs against eager runs."""
    c, heads, k, scale, q, pools, table, lengths, idx = _attend_case(misa, 576, 512, 1, 70, 16, [2500, 0, 900], dt, seed=41)
    kp, vp, ks, vs = _cuda(*pools)
    q, table, lengths = _cuda(q, table, lengths)
    x = torch.randn(3, 30000, device="cuda").bfloat16()
    weight = torch.randn(15000, device="cuda")
    need = misa.misa_attend_workspace_bytes(c, heads, k)
    assert need > 0  # more than one split
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty(3, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, heads, device="cuda"),
             torch.empty(3, 30000, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")) for _ in range(2)]

    def step(i):
        out, lse, codes, codes_scale = outs[i]
        misa.misa_rms_norm(3, 30000, 2, 1, 2, 1e-6, x, None, weight, None, codes, codes_scale)
        misa.misa_attend(c, heads, k, scale, q, kp, ks, vp, vs, table, lengths, None, out, lse, ws)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(1)
    for turn, tokens in enumerate(([2500, 0, 900], [1300, 0, 0], [1, 0, 640])):
        x.normal_()
        q.normal_()
        lengths.copy_(torch.tensor(tokens))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(0)
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b), turn
        assert not torch.isnan(outs[0][0]).any()


@gpu
def test_two_streams(misa):
    """Calls on two streams at once, each with its own workspace, against the same calls one by one."""
    cases = [_attend_case(misa, 128, 128, 2, 16, 64, [9000, 3000], dt, seed=31 + dt) for dt in (1, 2)]
    want = [_run_attend(misa, *case) for case in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    state = []
    for case, s in zip(cases, streams):
        c, heads, k, scale, q, pools, table, lengths, idx = case
        with torch.cuda.stream(s):
            kp, vp, ks, vs = _cuda(*pools)
            out = torch.empty(c.rows, heads, c.dv, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(c.rows, heads, device="cuda")
            ws = torch.empty(max(16, misa.misa_attend_workspace_bytes(c, heads, k)), dtype=torch.uint8, device="cuda")
            state.append((q.cuda(), kp, ks, vp, vs, table.cuda(), lengths.cuda(), None, out, lse, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for case, s, args in zip(cases, streams, state):
            misa.misa_attend(*case[:4], *args, stream=s)
    torch.cuda.synchronize()
    for args, (out, lse) in zip(state, want):
        assert torch.equal(args[8].cpu(), out) and torch.equal(args[9].cpu(), lse)
