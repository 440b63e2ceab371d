"""Rotary positions and the block-scaled cache (include/misa.h) against the plain CPU
references of tests/block_ref.py, their argument checks, and their use together.  The
refusals run on the CPU: they return before anything is launched."""

from __future__ import annotations

import ctypes
import math
import sys

import pytest
import torch

from tests import block_ref as ref
from tests.serve_ref import check_e4m3

FAKE = 1 << 20  # an aligned non-null address; never dereferenced (calls fail validation)
gpu = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
MANY = 70  # new tokens of a row for which tiles of queries have their larger form, whatever the heads
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: E4M3}


@pytest.fixture(scope="module")
def misa():
    import long_context_pool_amd as m

    return m


def _log(msg):
    print(msg, file=sys.stderr, flush=True)


# ------------------------------------------------------------------ refusals (CPU)


def _spec(misa, **change):
    f = dict(heads=4, d=128, first=0, rot=64, pairs=0, x_dtype=1, out_dtype=1, x_stride=512, out_stride=512, amplitude=1.0)
    f.update(change)
    return misa.rope_spec(**f)


@pytest.mark.parametrize("change,expect", [
    (dict(heads=0), -1), (dict(d=0), -1), (dict(first=-1), -1), (dict(rot=0), -1), (dict(rot=3), -1),
    (dict(first=66), -1), (dict(rot=130), -1), (dict(pairs=2), -1), (dict(pairs=-1), -1), (dict(x_dtype=3), -1),
    (dict(x_dtype=2), -2), (dict(out_dtype=3), -1), (dict(x_stride=511), -1), (dict(out_stride=511), -1),
    (dict(amplitude=math.nan), -1), (dict(amplitude=math.inf), -1), (dict(x_stride=1 << 31), -2),
    (dict(out_stride=1 << 31), -2), (dict(out_dtype=2, out_stride=520), -1),
    (dict(heads=512, x_stride=65536, out_stride=65536), -2),
    (dict(heads=2, d=2048, rot=2048, x_stride=4096, out_stride=4096), -2),
])
def test_rope_refuses_specs(misa, change, expect):
    assert misa.lib().misa_rope(ctypes.byref(_spec(misa, **change)), 3, FAKE, FAKE, FAKE, 2 * FAKE, FAKE, None) == expect


def test_rope_refuses_arguments(misa):
    def call(n=3, x=FAKE, pos=FAKE, freq=FAKE, out=2 * FAKE, scale=FAKE, **spec):
        return misa.lib().misa_rope(ctypes.byref(_spec(misa, **spec)), n, x, pos, freq, out, scale, None)

    for change in (dict(n=-1), dict(x=None), dict(pos=None), dict(freq=None), dict(out=None), dict(x=FAKE + 2),
                   dict(out=FAKE + 8), dict(freq=FAKE + 8), dict(out_dtype=2, scale=None),
                   dict(out=FAKE, out_dtype=0), dict(out=FAKE, out_stride=520), dict(out=FAKE, out_dtype=2)):
        assert call(**change) == -1, change
    assert call(n=1 << 24) == -2
    assert call(n=0, x=None, pos=None, freq=None, out=None) == 0
    assert misa.lib().misa_rope(None, 3, FAKE, FAKE, FAKE, FAKE, None, None) == -1


def test_rope_frequencies(misa):
    rot, base = 64, 10000.0
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    freq, amplitude = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_PLAIN, rot, base))
    assert amplitude == 1 and freq == pytest.approx(plain, rel=1e-15)
    freq, amplitude = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_LINEAR, rot, base, 8.0))
    assert amplitude == 1 and freq == pytest.approx([f / 8 for f in plain], rel=1e-15)
    freq, amplitude = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_PARTS, rot, base, 40.0, 4096.0, 32.0, 1.0))
    assert amplitude == pytest.approx(1 + 0.1 * math.log(40.0), rel=2.0 ** -24)
    turns = [4096 * f / (2 * math.pi) for f in plain]
    low = max(i for i, t in enumerate(turns) if t >= 32)  # the last pair that turns 32 times and more
    high = min(i for i, t in enumerate(turns) if t <= 1)
    for i, f in enumerate(freq):
        mix = min(max((i - low) / (high - low), 0), 1)
        assert f == pytest.approx(plain[i] * (1 - mix) + plain[i] / 40 * mix, rel=1e-14), i
    # one that every pair turns often in stays as it is; the amplitude is the factor's alone
    freq, _ = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_PARTS, rot, base, 4.0, 1e9, 32.0, 1.0))
    assert freq == pytest.approx(plain, rel=1e-14)
    got = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_PARTS, 2, base, 4.0, 100.0, 2.0, 2.0))
    assert all(math.isfinite(f) for f in got[0])


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (64, 1e4, 4.0, 65536.0, 32.0, 1.0),  # the last pair turns 1.39 times: the ramp ends behind it
    (64, 1e4, 4.0, 131072.0, 32.0, 1.0),
    (128, 1e4, 4.0, 131072.0, 32.0, 1.0),
    (128, 1e4, 4.0, 65536.0, 32.0, 1.0),
    (64, 1e4, 4.0, 32768.0, 32.0, 1.0),
    (96, 5e5, 8.0, 8192.0, 4.0, 1.0),
    (64, 1e4, 40.0, 20.0, 32.0, 1.0),  # no pair turns `fast` times
    (64, 1e4, 40.0, 5.0, 2.0, 1.0),  # every pair turns fewer than `slow` times
    (2, 1e4, 4.0, 5.0, 2.0, 1.0),
    (2, 1e4, 4.0, 100.0, 32.0, 1.0),
])
def test_rope_frequencies_by_parts(misa, rot, base, factor, original, fast, slow):
    """The header's rule: pairs that turn `fast` times keep f, those that turn `slow` times and fewer have
    f / factor, and what lies between is on one line over the pairs' numbers."""
    freq, _ = misa.misa_rope_frequencies(misa.rope_scaling(misa.MISA_ROPE_PARTS, rot, base, factor, original, fast, slow))
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [original * f / (2 * math.pi) for f in plain]
    share = [(1 - f / p) / (1 - 1 / factor) for f, p in zip(freq, plain)]  # of f / factor
    ramp = []
    for i in range(rot // 2):
        if turns[i] >= fast:
            assert share[i] == pytest.approx(0, abs=1e-12), i
        elif turns[i] <= slow:
            assert share[i] == pytest.approx(1, abs=1e-12), i
        else:
            ramp.append((i, share[i]))
            assert share[i] < 1, i
    # its ends: the pairs (of any whole number) next to those that turn `fast` and `slow` times
    at = [rot * math.log(original / (2 * math.pi * x)) / (2 * math.log(base)) for x in (fast, slow)]
    low, high = max(math.floor(at[0]), 0), math.ceil(at[1])
    for i, x in ramp:
        assert x == pytest.approx((i - low) / (high - low), abs=1e-12), i


def test_rope_frequencies_refuse(misa):
    out, amplitude = (ctypes.c_double * 1024)(), ctypes.c_float()

    def call(kind=2, rot=64, base=1e4, factor=4.0, original=4096.0, fast=32.0, slow=1.0):
        s = misa.rope_scaling(kind, rot, base, factor, original, fast, slow)
        return misa.lib().misa_rope_frequencies(ctypes.byref(s), out, ctypes.byref(amplitude))

    assert call() == 0
    for change in (dict(kind=3), dict(kind=-1), dict(rot=0), dict(rot=5), dict(base=1.0), dict(base=math.nan),
                   dict(base=math.inf), dict(factor=0.5), dict(factor=math.inf), dict(factor=math.nan),
                   dict(original=0.0), dict(fast=0.5), dict(slow=0.0), dict(original=math.inf), dict(fast=math.nan)):
        assert call(**change) == -1, change
    assert call(rot=1026) == -2
    assert call(kind=0, factor=0.0, original=0.0, fast=0.0, slow=0.0) == 0
    s = misa.rope_scaling(0, 64, 1e4)
    assert misa.lib().misa_rope_frequencies(None, out, ctypes.byref(amplitude)) == -1
    assert misa.lib().misa_rope_frequencies(ctypes.byref(s), None, ctypes.byref(amplitude)) == -1
    assert misa.lib().misa_rope_frequencies(ctypes.byref(s), out, None) == -1


def test_rope_frequencies_refuse_cheaply(misa):
    """A size that is refused takes no memory first."""
    import tracemalloc

    tracemalloc.start()
    try:
        for rot in (1026, 1 << 27, (1 << 31) - 2, -4):
            with pytest.raises(misa.MisaError):
                misa.misa_rope_frequencies(misa.rope_scaling(0, rot, 1e4))
        assert tracemalloc.get_traced_memory()[1] < 1 << 20
    finally:
        tracemalloc.stop()
    assert len(misa.misa_rope_frequencies(misa.rope_scaling(0, 1024, 1e4))[0]) == 512


def _calls(misa, c, block=32):
    """The block calls with good arguments, to be changed one at a time."""
    lib, r = misa.lib(), ctypes.byref(c)

    def write(n=3, block=block, **change):
        a = dict(offsets=FAKE, lengths=FAKE, kn=FAKE, vn=FAKE, kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, table=FAKE)
        a.update(change)
        return lib.misa_block_write(r, block, n, *a.values(), None)

    def read(n=3, block=block, out_dtype=1, **change):
        a = dict(offsets=FAKE, first=None, lengths=FAKE, kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, table=FAKE, ko=FAKE,
                 kos=FAKE, vo=FAKE, vos=FAKE)
        a.update(change)
        return lib.misa_block_read(r, block, n, out_dtype, *a.values(), None)

    def attend(n=3, block=block, heads=8, most=1, k=0, scale=0.1, ws=FAKE, ws_bytes=1 << 40, **change):
        a = dict(offsets=FAKE, q=FAKE, kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, table=FAKE, lengths=FAKE, idx=None, out=FAKE,
                 lse=None)
        a.update(change)
        return lib.misa_block_attend(r, block, heads, n, most, k, scale, *a.values(), ws, ws_bytes, None)

    return write, read, attend


@pytest.mark.parametrize("change,block,expect", [
    (dict(rows=0), 32, -1), (dict(pages=0), 32, -1), (dict(kv_heads=0), 32, -1), (dict(kv_heads=257), 32, -2),
    (dict(rows=65536), 32, -2), (dict(kv_dtype=1), 32, -2), (dict(kv_dtype=0), 32, -2), (dict(kv_dtype=3), 32, -1),
    (dict(dk=96, dv=96), 32, -2), (dict(dk=576, dv=512, kv_heads=1), 32, -2), (dict(page_tokens=48), 32, -1),
    (dict(), 0, -1), (dict(), -16, -1), (dict(), 8, -2), (dict(), 48, -2), (dict(), 256, -2), (dict(), 128, -1),
])
def test_block_calls_refuse_caches(misa, change, block, expect):
    fields = dict(rows=4, row_pages=8, pages=40, page_tokens=64, kv_heads=2, dk=128, dv=128, kv_dtype=2)
    fields.update(change)
    c = misa.cache(*fields.values())
    for call in _calls(misa, c, block):
        assert call() == expect, call
    assert misa.misa_block_attend_workspace_bytes(c, block, 8, 3, 3, 0) == 0


def test_block_calls_refuse_arguments(misa):
    c = misa.cache(4, 8, 40, 64, 2, 128, 128, misa.MISA_FP8_E4M3)
    write, read, attend = _calls(misa, c)
    for call, names in ((write, "offsets lengths kn kp ks table".split()),
                        (read, "offsets lengths kp ks table ko".split()),
                        (attend, "offsets q kp ks vp vs table lengths out".split())):
        for name in names:
            for bad in (None, FAKE + 4):
                assert call(**{name: bad}) == -1, (call, name)
        assert call(n=-1) == -1
        assert call(n=0, **{x: None for x in names}) == 0
    for call, name in ((write, "vn"), (write, "vp"), (write, "vs"), (read, "vo"), (read, "vp"), (read, "vs"),
                       (attend, "vp"), (attend, "vs")):
        assert call(**{name: None}) == -1, name  # values are there, or none of their arrays
        assert call(**{name: FAKE + 8}) == -1, name
    assert attend(vp=None, vs=None) == -1
    assert write(n=1 << 25) == -2 and read(n=1 << 28) == -2
    assert read(out_dtype=3) == -1 and read(out_dtype=-1) == -1 and read(first=FAKE + 4) == -1
    assert read(out_dtype=2, kos=None) == -1 and read(out_dtype=2, vos=None) == -1
    for change in (dict(heads=0), dict(heads=7), dict(k=-1), dict(most=-1), dict(k=4), dict(idx=FAKE),
                   dict(scale=math.nan), dict(scale=math.inf), dict(lse=FAKE + 4), dict(k=4, idx=FAKE + 4)):
        assert attend(**change) == -1, change
    for change in (dict(heads=2048), dict(k=(1 << 20) + 1, idx=FAKE), dict(n=(1 << 20) + 1),
                   dict(n=1 << 20, heads=128), dict(scale=3e38)):
        assert attend(**change) == -2, change
    # More workgroups than a launch holds.
    for change in (dict(n=1 << 18, heads=64, k=4, idx=FAKE), dict(n=1 << 18, heads=64, most=1)):
        assert attend(**change) == -2, change
    many = misa.cache(65535, 8, 40, 64, 256, 128, 128, misa.MISA_FP8_E4M3)
    assert _calls(misa, many)[2](n=2, heads=256, most=2) == -2
    assert read(n=(1 << 26) + 1) == -2  # of two heads
    long = misa.cache(1, 4096, 5000, 64, 1, 128, 128, misa.MISA_FP8_E4M3)
    for most in (1, 5, 80):
        need = misa.misa_block_attend_workspace_bytes(long, 32, 8, most, most, 0)
        assert need > 0
        attend = _calls(misa, long)[2]
        assert attend(n=most, most=most, ws_bytes=need - 1) == -3 and attend(n=most, most=most, ws=None) == -3
        assert attend(n=most, most=most, ws=FAKE + 8) == -1


def test_block_workspace_follows_the_queries(misa):
    """A few queries on a table of many rows need about what they need on a table of few."""
    def need(rows, n, heads, kv, most):
        c = misa.cache(rows, 512, 4096, 64, kv, 128, 128, misa.MISA_FP8_E4M3)
        return misa.misa_block_attend_workspace_bytes(c, 32, heads, n, most, 0)

    for n, heads, kv, most in ((80, 64, 8, 5), (80, 64, 8, 80), (4, 1024, 64, 4), (2, 8, 8, 2)):
        few, many = need(32, n, heads, kv, most), need(900, n, heads, kv, most)
        # parts for all workgroups at a time, or for each unit that can have work: sums of (pairs of a query's row) x 128;
        # and 8 bytes a unit, of which the table's rows have one each
        pairs = min(128, n * heads // kv)
        working = (n * heads // kv >> 6) + n
        assert 0 < few <= many <= max(few, max(512, kv * working) * (pairs * (128 * 4 + 8) + 8)) + 900 * 8 + 1024, (n, few, many)
        assert many <= 1 << 28


# ------------------------------------------------------------------ rotary positions


ROPE = [
    # n, heads, d, first, rot, pairs, x, out, extra x elements, in place
    (1, 1, 128, 0, 128, 0, 1, 1, 0, False),
    (3, 5, 128, 0, 64, 1, 1, 2, 0, False),
    (7, 1, 128, 64, 64, 0, 0, 2, 0, False),  # 16 threads a token, the last workgroup half empty
    (5, 3, 192, 128, 64, 1, 1, 1, 3 * 192, False),  # the rest in front
    (4, 8, 128, 0, 128, 0, 1, 1, 2 * 128, True),
    (2, 40, 64, 16, 32, 1, 0, 0, 64, True),
    (3, 64, 128, 0, 64, 1, 1, 2, 0, False),
    (2, 250, 128, 32, 96, 0, 0, 2, 16, False),  # the longest rows
    (2, 16, 2048, 512, 1024, 1, 1, 0, 0, False),
    (33, 2, 64, 0, 64, 0, 0, 1, 8, False),
    # sizes and strides off the runs of 16
    (3, 3, 30, 4, 10, 0, 1, 1, 0, False),
    (3, 3, 30, 4, 10, 1, 1, 1, 7, True),
    (2, 7, 72, 0, 2, 0, 0, 2, 1, False),
    (2, 7, 72, 70, 2, 1, 1, 2, 0, False),
    (4, 2, 128, 0, 64, 0, 0, 0, 4, True),
    (1, 1, 2, 0, 2, 0, 1, 0, 0, False),
]


@gpu
@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(misa, case):
    n, heads, d, first, rot, pairs, xt, ot, extra, in_place = case
    _log(f"[gpu] rope {case}")
    g = torch.Generator().manual_seed(n * heads + d)
    row = heads * d
    wide = torch.randn(n, row + extra, generator=g).to(TYPES[xt])
    pos = torch.randint(-100, 1 << 20, (n,), generator=g).int()
    pos[0] = 0
    if n > 2:
        pos[1], pos[2] = (1 << 31) - 1, -(1 << 31)
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    amplitude = 1.25
    want, tol = ref.rope(wide[:, :row].reshape(n, heads, d), pos.numpy(), freq, first, pairs, amplitude)
    on = wide.cuda()
    x = on[:, :row]
    out_wide = on if in_place else torch.full((n, row + (0 if ot == 2 else 3 * 16)), 7, device="cuda").to(TYPES[ot])
    out = out_wide[:, :row]
    scale = torch.zeros(n, device="cuda") if ot == 2 else None
    spec = misa.rope_spec(heads, d, first, rot, pairs, xt, ot, on.stride(0), out_wide.stride(0), amplitude)
    misa.misa_rope(spec, n, x, pos.cuda(), torch.tensor(freq, dtype=torch.float64, device="cuda"), out, scale)
    got = out.cpu().reshape(n, heads, d)
    if in_place:
        assert torch.equal(on.cpu()[:, row:], wide[:, row:])
    elif ot != 2:
        assert torch.all(out_wide[:, row:].cpu() == 7)
    if ot == 2:
        # the scale's maximum is off by its value's tolerance, and so is a code
        slack = (tol.flatten(1).amax(1) / want.abs().flatten(1).amax(1)).max().item()
        top = want.abs().flatten(1).amax(1)
        assert torch.all((scale.cpu().double() - top / 448).abs() <= top / 448 * (2.0 ** -22 + slack))
        y = want / scale.cpu().double()[:, None, None]
        off = (got.double() - y).abs()
        step = torch.clamp(y.abs() * 2.0 ** -4, min=2.0 ** -10)
        assert torch.all(off <= step * (1 + 2.0 ** -8) + tol / scale.cpu().double()[:, None, None] + y.abs() * 2.0 ** -20)
    else:
        half = 2.0 ** -8 if ot == 1 else 2.0 ** -24
        assert torch.all((got.double() - want).abs() <= tol * (1 + half) + want.abs() * half)
        rest = [i for i in range(d) if not first <= i < first + rot]
        assert torch.equal(got[..., rest], wide[:, :row].reshape(n, heads, d)[..., rest].to(TYPES[ot]))


@gpu
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("d,rot", [(128, 64), (72, 36), (512, 32)])
def test_rope_codes_are_the_nearest(misa, d, rot, pairs):
    """Codes of passing values are their fp32 quotients by the token's scale, rounded to nearest even, and the
    scale is amax / 448: both to the bit, and a zero token, one with an infinity and one with NaN as well."""
    n, heads = 300, 3
    _log(f"[gpu] rope codes {d} {rot} {pairs}")
    g = torch.Generator().manual_seed(d)
    x = torch.randn(n, heads, d, generator=g).bfloat16()
    top = 16 + torch.arange(n) % 128 / 8  # exact in bf16, above every turned value
    x[:, 1, rot + 1] = top.bfloat16()
    x[40] = 0
    x[41, 0, rot] = math.inf
    x[42, 2, d - 1] = math.nan
    x[43:60] *= 2.0 ** 90
    x[60:80] *= 2.0 ** -80
    spec = misa.rope_spec(heads, d, 0, rot, pairs, 1, 2, heads * d, heads * d)
    out, scale = torch.zeros(n, heads, d, device="cuda").to(E4M3), torch.zeros(n, device="cuda")
    freq = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    misa.misa_rope(spec, n, x.cuda(), torch.arange(n).int().cuda(), freq, out, scale)
    y = x.float()
    amax = torch.where(y.isnan(), 0.0, y.abs()).flatten(1).amax(1)
    amax[42] = top[42]
    unit = torch.where(amax > 0, amax / 448, 1.0)
    assert torch.equal(scale.cpu(), unit)
    assert ref.same_codes(out.cpu()[..., rot:].contiguous(), (y / unit[:, None, None]).to(E4M3)[..., rot:].contiguous())


@gpu
def test_rope_turns_back_and_keeps_distances(misa):
    """Rotations by p and -p cancel, and q . k depends on the distance alone."""
    n, heads, d = 16, 2, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, heads, d, generator=g).expand(n, -1, -1).contiguous().cuda()
    freq = torch.tensor(misa.misa_rope_frequencies(misa.rope_scaling(0, d, 10000.0))[0], dtype=torch.float64, device="cuda")
    spec = misa.rope_spec(heads, d, 0, d, 1, 0, 0, heads * d, heads * d)
    pos = (torch.arange(n) * 70001).int().cuda()
    y, z, w = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    misa.misa_rope(spec, n, x, pos, freq, y, None)
    misa.misa_rope(spec, n, y, -pos, freq, z, None)
    misa.misa_rope(spec, n, x, pos + 9, freq, w, None)
    norm = x.double().square().sum(-1)
    # two rotations, each off by 2^-20 + 3 * 2^-24 of |a| + |b| <= sqrt(2) |(a, b)|
    assert torch.all((z - x).abs().amax(-1) <= norm.sqrt() * 2 * 2 ** 0.5 * 2.0 ** -19.6)
    dots = (y.double() * w.double()).sum(-1)
    assert torch.all((dots - dots[:1]).abs() <= norm * 4 * 2 ** 0.5 * 2.0 ** -19.6)


# ------------------------------------------------------------------ the cache


def _cells(g, *shape):
    return (100 * torch.randn(shape, generator=g)).clamp(-448, 448).to(E4M3)


def _pool(misa, g, lengths, P, B, kv, d, spare=3, width=None):
    """A cache with rows of these lengths on random pages: (cache, table, k, ks, v, vs) on the CPU."""
    rows = len(lengths)
    held = [-(-max(n, 0) // P) for n in lengths]
    width = width or max(held + [1])
    pages = sum(held) + spare
    ids = torch.randperm(pages, generator=g).int()
    table = torch.full((rows, width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    c = misa.cache(rows, width, pages, P, kv, d, d, misa.MISA_FP8_E4M3)
    k, v = _cells(g, pages, kv, P, d), _cells(g, pages, kv, P, d)
    ks, vs = (2.0 ** torch.randint(-9, -4, (pages, kv, P // B), generator=g).float() for _ in range(2))
    return c, table, k, ks, v, vs


def _offsets(counts, at=0):
    got = [at]
    for n in counts:
        got.append(got[-1] + n)
    return torch.tensor(got, dtype=torch.int32)


def _cuda(*tensors):
    return [None if t is None else t.cuda() for t in tensors]


WRITE = [
    # lengths after the write, new tokens, P, B, kv, d, padding in front and behind
    ([1], [1], 16, 16, 1, 64, 0, 0),
    ([5, 17, 32, 33], [5, 1, 3, 33], 16, 16, 2, 64, 0, 0),
    ([100, 64, 65, 0, 200], [37, 64, 1, 0, 90], 64, 64, 3, 128, 2, 3),
    ([100, 129], [100, 129], 128, 32, 2, 128, 0, 5),
    ([300, 128, 127], [300, 1, 2], 128, 128, 1, 256, 0, 0),
    ([90, 200], [64, 129], 96, 32, 5, 64, 0, 0),
    ([130, 40], [130, 40], 128, 128, 2, 64, 1, 0),
    ([31, 95], [20, 70], 32, 16, 1, 256, 0, 0),
    ([50] * 70, [1] * 70, 64, 64, 1, 64, 0, 2),  # rows beyond one look of a wave
    ([50] * 70, [0, 3] * 35, 64, 64, 1, 64, 0, 0),
]


@gpu
@pytest.mark.parametrize("case", WRITE, ids=str)
@pytest.mark.parametrize("values", [True, False])
def test_write(misa, case, values):
    lengths, counts, P, B, kv, d, front, behind = case
    _log(f"[gpu] write {case} {values}")
    g = torch.Generator().manual_seed(len(lengths) + d)
    c, table, k, ks, v, vs = _pool(misa, g, lengths, P, B, kv, d)
    offsets = _offsets(counts, front)
    n = int(offsets[-1]) + behind
    loud = 2.0 ** torch.randint(-8, 9, (n, kv, 1), generator=g)  # some blocks grow louder, some do not
    kn = (torch.randn(n, kv, d, generator=g) * loud).bfloat16()
    vn = (torch.randn(n, kv, d, generator=g) * loud.flip(0)).bfloat16()
    wk, wks = ref.write(c, B, offsets, lengths, kn, k, ks, table)
    wv, wvs = ref.write(c, B, offsets, lengths, vn, v, vs, table)
    if not values:
        vn = v = vs = None
    ln = torch.tensor(lengths, dtype=torch.int32)
    gk, gks, gv, gvs = _cuda(k, ks, v, vs)
    misa.misa_block_write(c, B, n, offsets.cuda(), ln.cuda(), kn.cuda(), None if vn is None else vn.cuda(), gk, gks, gv,
                          gvs, table.cuda())
    assert torch.equal(gks.cpu(), wks) and ref.same_codes(gk.cpu(), wk)
    if values:
        assert torch.equal(gvs.cpu(), wvs) and ref.same_codes(gv.cpu(), wv)


@gpu
def test_write_hard_values(misa):
    """Zeros, subnormals, the largest, infinities and NaN, next to ordinary values of their block; 448 * 2^e
    and its neighbours on both sides of a scale; a block that grows by 2^200."""
    B, d = 16, 64
    g = torch.Generator().manual_seed(4)
    rows = [0.0, -0.0, 2.0 ** -133, 2.0 ** -110, 2.0 ** -93, 2.0 ** -92, 448.0, 450.0, 446.0, 3.3895e38, -1.75, math.inf,
            -math.inf, math.nan]
    n = len(rows)
    c, table, k, ks, v, vs = _pool(misa, g, [20] * n, 32, B, 1, d)
    new = torch.randn(20 * n, 1, d, generator=g).mul(2.0 ** -3).bfloat16().view(n, 20, 1, d)
    for r, x in enumerate(rows):
        new[r, :, 0, 5] = x
        if r < 6:
            new[r] = x
    new = new.view(-1, 1, d)
    quiet = (new.float() * 2.0 ** -120).bfloat16()
    for kn, counts in ((new, [20] * n), (torch.cat([quiet.view(n, 20, 1, d)[:, :7].reshape(-1, 1, d)]), [7] * n),
                       (new.view(n, 20, 1, d)[:, 7:].reshape(-1, 1, d).contiguous(), [13] * n)):
        after = torch.tensor([20 if counts[0] != 7 else 7] * n, dtype=torch.int32)
        offsets = _offsets(counts)
        wk, wks = ref.write(c, B, offsets, after, kn, k, ks, table)
        gk, gks = _cuda(k, ks)
        misa.misa_block_write(c, B, kn.shape[0], offsets.cuda(), after.cuda(), kn.cuda(), None, gk, gks, None, None,
                              table.cuda())
        assert torch.equal(gks.cpu(), wks) and ref.same_codes(gk.cpu(), wk)
        k, ks = gk.cpu(), gks.cpu()


@gpu
def test_write_skips_what_is_not_there(misa):
    """No page, a table too short, more new tokens than the row has, offsets that do not ascend or pass n."""
    B, d, P = 16, 64, 16
    g = torch.Generator().manual_seed(5)
    lengths = [40, 70, 20, 33]
    c, table, k, ks, v, vs = _pool(misa, g, [40, 48, 20, 33], P, B, 2, d, width=3)
    table[0, 1], table[3, 0] = -1, c.pages + 5
    ln = torch.tensor(lengths, dtype=torch.int32)
    for offsets in (_offsets([40, 40, 25, 33]), torch.tensor([0, 30, 20, 90, 400], dtype=torch.int32),
                    torch.tensor([-7, 5, 5, 20, 30], dtype=torch.int32)):
        kn = torch.randn(138, 2, d, generator=g).bfloat16()
        wk, wks = ref.write(c, B, offsets, lengths, kn, k, ks, table)
        gk, gks = _cuda(k, ks)
        misa.misa_block_write(c, B, 138, offsets.cuda(), ln.cuda(), kn.cuda(), None, gk, gks, None, None, table.cuda())
        assert torch.equal(gks.cpu(), wks) and ref.same_codes(gk.cpu(), wk)


READ = [
    # lengths, first, tokens read, P, B, kv, d, padding in front and behind
    ([1], None, [1], 16, 16, 1, 64, 0, 0),
    ([100, 64, 0, 65], [3, 0, 0, 60], [97, 64, 0, 5], 64, 32, 2, 128, 1, 2),
    ([300], [7], [290], 96, 16, 3, 256, 0, 0),
    ([40, 50], [-3, 45], [50, 12], 16, 16, 1, 128, 0, 3),  # before and behind the row: zeros
    ([20] * 130, None, [20, 0] * 65, 32, 32, 1, 64, 0, 0),
    ([700, 3], None, [700, 3], 128, 128, 1, 128, 0, 0),
]


@gpu
@pytest.mark.parametrize("case", READ, ids=str)
@pytest.mark.parametrize("out", [0, 1, 2])
def test_read(misa, case, out):
    lengths, first, counts, P, B, kv, d, front, behind = case
    _log(f"[gpu] read {case} {out}")
    g = torch.Generator().manual_seed(len(lengths) + d)
    c, table, k, ks, v, vs = _pool(misa, g, lengths, P, B, kv, d)
    table[0, 0] = c.pages if len(lengths) == 4 else table[0, 0]
    k.view(torch.uint8)[:, :, 0, 1] = 0x7F  # a NaN code is one
    offsets = _offsets(counts, front)
    n = int(offsets[-1]) + behind
    ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    fs = None if first is None else torch.tensor(first, dtype=torch.int32).cuda()
    ko, vo = (torch.full((n, kv, d), 5.0, device="cuda").to(TYPES[out]) for _ in range(2))
    kos, vos = (torch.full((n, kv), 5.0, device="cuda") if out == 2 else None for _ in range(2))
    gk, gks, gv, gvs = _cuda(k, ks, v, vs)
    misa.misa_block_read(c, B, n, out, offsets.cuda(), fs, ln, gk, gks, gv, gvs, table.cuda(), ko, kos, vo, vos)
    for pool, scale, got, units in ((k, ks, ko, kos), (v, vs, vo, vos)):
        code, unit, written = ref.read(c, B, offsets, first, lengths, pool, scale, table, n)
        got = got.cpu()
        if out == 2:
            assert ref.same_codes(got[written], code[written])
            assert torch.equal(units.cpu()[written], unit[written]) and torch.all(units.cpu()[~written] == 5)
        else:  # a code times a power of two is exact in both types
            want = (code.float() * unit[..., None]).to(TYPES[out])
            assert torch.equal(got[written].nan_to_num(-1), want[written].nan_to_num(-1))
        assert torch.all(got[~written].float() == 5)
    ko.zero_()
    misa.misa_block_read(c, B, n, out, offsets.cuda(), fs, ln, gk, gks, None, None, table.cuda(), ko, kos, None, None)
    code, unit, written = ref.read(c, B, offsets, first, lengths, k, ks, table, n)
    if out == 2:
        assert ref.same_codes(ko.cpu()[written], code[written])


@gpu
@pytest.mark.parametrize("out", [0, 1, 2])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_of_many_tokens(misa, out, d):
    """32 MB and more, marked as not to be kept: rows that end inside a workgroup's tokens, a lost page."""
    P, B, kv = 128, 64, 4
    n = (33 << 20) // (2 * kv * d * (1 + (4, 2, 1)[out])) + 1
    lengths = [n - 7000, 5, 0, 6995]
    _log(f"[gpu] read {n} tokens {d} {out}")
    g = torch.Generator().manual_seed(54)
    c, table, k, ks, v, vs = _pool(misa, g, lengths, P, B, kv, d)
    table[3, 2] = -1
    ko, vo = (torch.zeros(n, kv, d, device="cuda").to(TYPES[out]) for _ in range(2))
    kos, vos = (torch.zeros(n, kv, device="cuda") if out == 2 else None for _ in range(2))
    misa.misa_block_read(c, B, n, out, _offsets(lengths).cuda(), None, torch.tensor(lengths).int().cuda(),
                         *_cuda(k, ks, v, vs, table), ko, kos, vo, vos)
    for pool, scale, got, units in ((k, ks, ko, kos), (v, vs, vo, vos)):
        code, unit, _ = ref.read(c, B, _offsets(lengths), None, lengths, pool, scale, table, n)
        if out == 2:
            assert ref.same_codes(got.cpu(), code) and torch.equal(units.cpu(), unit)
        else:
            assert torch.equal(got.cpu(), (code.float() * unit[..., None]).to(TYPES[out]))


# ------------------------------------------------------------------ attention


def _check_attend(misa, c, B, heads, k, scale, offsets, q, pools, table, lengths, idx, most):
    """Calls and compares; tiles of several queries hold weights to 11 bits."""
    n = q.shape[0]
    kp, ks, vp, vs = pools
    out, lse, out_tol, lse_tol, wide, written = ref.attend(misa, c, B, heads, k, scale, offsets, q, kp, ks, vp, vs, table,
                                                           lengths, idx)
    if k == 0 and most > 1:
        out_tol = out_tol + wide
    ln = torch.tensor(lengths, dtype=torch.int32)
    go = torch.full((n, heads, c.dk), 3.0, dtype=torch.bfloat16, device="cuda")
    gl = torch.full((n, heads), 3.0, device="cuda")
    need = misa.misa_block_attend_workspace_bytes(c, B, heads, n, most, k)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    misa.misa_block_attend(c, B, heads, n, most, k, scale, *_cuda(offsets, q, kp, ks, vp, vs, table, ln, idx), go, gl, ws)
    go, gl = go.cpu().double(), gl.cpu().double()
    assert torch.all(go[~written] == 3) and torch.all(gl[~written] == 3)
    go, gl, out, lse, out_tol, lse_tol = (x[written] for x in (go, gl, out, lse, out_tol, lse_tol))
    bad = torch.isnan(out)
    assert torch.equal(torch.isnan(go), bad)
    worst = ((go - out).abs() / out_tol.clamp(min=1e-30))[~bad].max().item() if (~bad).any() else 0
    _log(f"  worst {worst:.3f} of the tolerance")
    assert torch.all(((go - out).abs() <= out_tol + 1e-30) | bad)
    none, badl = lse == -math.inf, torch.isnan(lse)
    assert torch.equal(gl == -math.inf, none) and torch.equal(torch.isnan(gl), badl)
    assert torch.all(((gl - lse).abs() <= lse_tol) | none | badl)


ATTEND = [
    # lengths, new tokens, P, B, kv, heads, d, padding in front and behind
    ([1], [1], 16, 16, 1, 1, 64, 0, 0),
    ([1], [1], 16, 16, 1, 1, 128, 0, 0),
    ([3, 70, 0, 129], [1, 1, 0, 1], 64, 32, 2, 16, 128, 1, 2),
    ([3, 70, 0, 129], [3, 2, 0, 5], 64, 32, 2, 16, 128, 1, 2),
    ([200], [200], 128, 128, 1, 5, 64, 0, 0),
    ([65, 64, 63], [65, 64, 63], 32, 16, 2, 14, 64, 0, 3),
    ([150, 33], [130, 33], 64, 64, 1, 8, 128, 0, 0),
    ([257], [100], 48, 16, 1, 12, 128, 2, 0),
    ([100, 31, 90], [40, 31, 1], 96, 32, 1, 4, 256, 0, 1),
    ([70], [9], 16, 16, 3, 3, 256, 0, 0),
    ([90], [20], 16, 16, 1, 40, 128, 0, 0),
    ([40] * 66, [1, 0, 2] * 22, 64, 64, 1, 2, 64, 0, 0),
    ([2, 5], [4, 5], 16, 16, 1, 2, 64, 0, 0),  # more new tokens than the row has: they see nothing
]


@gpu
@pytest.mark.parametrize("case", ATTEND, ids=str)
@pytest.mark.parametrize("most", [1, 2, MANY])
def test_attend(misa, case, most):
    """Every kernel on every case: `most` picks one, and no result depends on it."""
    lengths, counts, P, B, kv, heads, d, front, behind = case
    _log(f"[gpu] block attend {case} {most}")
    g = torch.Generator().manual_seed(sum(lengths) + d)
    c, table, *pools = _pool(misa, g, lengths, P, B, kv, d)
    offsets = _offsets(counts, front)
    q = torch.randn(int(offsets[-1]) + behind, heads, d, generator=g).bfloat16()
    _check_attend(misa, c, B, heads, 0, d ** -0.5, offsets, q, pools, table, lengths, None, most)


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3, 3.0])
@pytest.mark.parametrize("most", [1, 3, MANY])
def test_attend_scales(misa, scale, most):
    _log(f"[gpu] block attend scale {scale} {most}")
    g = torch.Generator().manual_seed(9)
    c, table, *pools = _pool(misa, g, [90, 77], 32, 16, 2, 64)
    offsets = _offsets([6, 3])
    q = torch.randn(9, 6, 64, generator=g).bfloat16()
    _check_attend(misa, c, 16, 6, 0, scale, offsets, q, pools, table, [90, 77], None, most)


@gpu
@pytest.mark.parametrize("most", [1, 3, MANY])
def test_attend_blocks_of_far_scales(misa, most):
    """Neighbouring blocks' scales up to 2^40 apart, either way: weights follow the values' scale."""
    _log(f"[gpu] block attend far scales {most}")
    g = torch.Generator().manual_seed(10)
    n = 400
    c, table, k, ks, v, vs = _pool(misa, g, [n], 16, 16, 1, 64)
    vs = 2.0 ** torch.randint(-20, 21, vs.shape, generator=g).float()
    offsets = _offsets([5])
    q = torch.randn(5, 4, 64, generator=g).bfloat16()
    _check_attend(misa, c, 16, 4, 0, 0.05, offsets, q, (k, ks, v, vs), table, [n], None, most)
    vs[table[0, 12:].long()] *= 2.0 ** -50  # the quiet ones at the end, with all the weight
    ks[table[0, :12].long()] = 2.0 ** -60
    _check_attend(misa, c, 16, 4, 0, 4.0, offsets, q, (k, ks, v, vs), table, [n], None, most)


@gpu
@pytest.mark.parametrize("most", [1, 3, MANY])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 6])
@pytest.mark.parametrize("far", [20, 40])
def test_attend_loud_blocks_that_are_not_seen_yet(misa, most, d, heads, far):
    """New tokens over several blocks of one tile of tokens (of 32 or 64), the later blocks 2^far louder: a query
    that sees the quiet ones alone loses nothing by what is behind it."""
    _log(f"[gpu] block attend loud blocks behind {most} {d} {heads} {far}")
    g = torch.Generator().manual_seed(41)
    lengths, counts = [64, 150, 70, 200], [64, 40, 3, 32]
    c, table, k, ks, v, vs = _pool(misa, g, lengths, 16, 16, 1, d)
    vs *= 2.0 ** -20
    for r, page in ((0, 2), (0, 3), (1, 8), (1, 9), (2, 4), (3, 11)):
        vs[table[r, page].item()] *= 2.0 ** far
    q = torch.randn(sum(counts), heads, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, heads, 0, 0.05, _offsets(counts), q, (k, ks, v, vs), table, lengths, None, most)


@gpu
@pytest.mark.parametrize("most", [1, 3, MANY])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_nan_where_it_is_not_seen(misa, most, d):
    """NaN behind the row's end, in pages it lost, and at tokens that only later queries see."""
    _log(f"[gpu] block attend nan {most} {d}")
    g = torch.Generator().manual_seed(11)
    lengths, counts = [70, 45], [9, 45]
    c, table, k, ks, v, vs = _pool(misa, g, lengths, 16, 16, 2, d)
    ends = [(0, 70, 80), (1, 45, 48)]
    for r, a, b in ends:
        for p in range(a, b):
            for pool in (k, v):
                pool.view(torch.uint8)[table[r, p // 16], :, p % 16] = 0x7F
    k.view(torch.uint8)[table[0, 2].item()] = 0xFF
    v.view(torch.uint8)[table[0, 2].item()] = 0xFF
    ks[table[0, 2].item()] = vs[table[0, 2].item()] = math.nan
    table[0, 2] = -1
    offsets = _offsets(counts)
    q = torch.randn(54, 4, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 4, 0, 0.1, offsets, q, (k, ks, v, vs), table, lengths, None, most)
    # one NaN value (one dimension) and one NaN key at tokens inside the new ones
    v.view(torch.uint8)[table[1, 1], 0, 4, 7] = 0x7F  # token 20 of row 1, kv head 0
    v.view(torch.uint8)[table[0, 4], 1, 1, 3] = 0xFF  # token 65 of row 0, kv head 1
    _check_attend(misa, c, 16, 4, 0, 0.1, offsets, q, (k, ks, v, vs), table, lengths, None, most)
    k.view(torch.uint8)[table[1, 2], 1, 0, 0] = 0x7F  # token 32 of row 1, kv head 1
    _check_attend(misa, c, 16, 4, 0, 0.1, offsets, q, (k, ks, v, vs), table, lengths, None, most)


@gpu
@pytest.mark.parametrize("most", [1, 3, MANY])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lost", [1, 2])
def test_attend_nan_beside_a_lost_page(misa, most, d, lost):
    """A NaN value that every query sees, one or two pages from one that the row lost."""
    _log(f"[gpu] block attend nan beside a lost page {most} {d} {lost}")
    g = torch.Generator().manual_seed(22)
    c, table, k, ks, v, vs = _pool(misa, g, [200], 16, 16, 1, d)
    v.view(torch.uint8)[table[0, 0], 0, 5, 9] = 0x7F
    v.view(torch.uint8)[table[0, 4], 0, 2, 3] = 0xFF
    table[0, lost] = -1
    q = torch.randn(2, 2, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 2, 0, 0.1, _offsets([2]), q, (k, ks, v, vs), table, [200], None, most)


@gpu
@pytest.mark.parametrize("most", [1, 4, MANY])
def test_attend_long_rows_in_splits(misa, most):
    """Few queries, long rows: parts that are joined, some of them without tokens."""
    _log(f"[gpu] block attend splits {most}")
    g = torch.Generator().manual_seed(12)
    lengths, counts = [3000, 5], [4, 2]
    c, table, *pools = _pool(misa, g, lengths, 64, 32, 1, 64)
    offsets = _offsets(counts, 1)
    q = torch.randn(8, 2, 64, generator=g).bfloat16()
    assert misa.misa_block_attend_workspace_bytes(c, 32, 2, 8, most, 0) > 0
    _check_attend(misa, c, 32, 2, 0, 0.125, offsets, q, pools, table, lengths, None, most)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [2, 100])
@pytest.mark.parametrize("lengths,counts", [
    ([5000, 4, 0, 600, 2500, 300], [3, 4, 0, 1, 0, 2]),  # parts of one row and whole rows
    ([900, 700], [60, 9]),  # units of one row, most of them alike
    ([40, 7], [3, 5]),  # fewer tokens than a part's least
    ([0, 1, 700], [2, 3, 2]),  # queries before the first token
    ([700] * 5 + [0] * 1200, [2] * 5 + [0] * 1200),  # more rows than are shared out
    ([300] + [60 + i % 50 for i in range(279)], [1] * 280),  # more units than workgroups at a time
])
def test_attend_parts(misa, d, most, lengths, counts):
    _log(f"[gpu] block attend parts {d} {most} {lengths[:6]} {counts[:6]}")
    g = torch.Generator().manual_seed(31)
    c, table, *pools = _pool(misa, g, lengths, 32, 16, 2, d)
    q = torch.randn(sum(counts) + 3, 6, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 6, 0, 0.09, _offsets(counts), q, pools, table, lengths, None, most)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [2, MANY])
def test_attend_few_queries_of_a_table_of_many_rows(misa, d, most):
    """Parts are numbered by the queries' units of work, of which there are far fewer than rows of the table."""
    _log(f"[gpu] block attend few of many rows {d} {most}")
    g = torch.Generator().manual_seed(32)
    lengths, counts = [0] * 900, [0] * 900
    for r, length, count in ((0, 70, 0), (3, 2900, 2), (450, 5, 1), (451, 1200, 3), (899, 33, 2)):
        lengths[r], counts[r] = length, count
    c, table, *pools = _pool(misa, g, lengths, 32, 16, 2, d)
    assert misa.misa_block_attend_workspace_bytes(c, 16, 6, 8, most, 0) > 0
    q = torch.randn(8, 6, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 6, 0, 0.09, _offsets(counts), q, pools, table, lengths, None, most)


@gpu
def test_attend_rows_of_more_tiles_than_fp32_counts(misa):
    """Heads of 256, a row of 2^24 + 1 tiles of 32 tokens beside a short one: 32 parts hold all of them.  Every
    score is 0 and every value a power of two, so that sums are exact but for the logarithm and the division."""
    _log("[gpu] block attend 2^24 + 1 tiles")
    P, d = 4096, 256
    width = 1 << 18
    length = (1 << 29) + 1
    c = misa.cache(2, width, 3, P, 1, d, d, misa.MISA_FP8_E4M3)
    table = torch.zeros(2, width, dtype=torch.int32)
    table[0, length // P * 31 // 32:] = 1  # the last thirty-second and what is behind it
    table[1] = 2
    k = torch.zeros(3, 1, P, d).to(E4M3)
    v = torch.tensor([1.0, -1.0, 2.0]).view(3, 1, 1, 1).expand(3, 1, P, d).contiguous().to(E4M3)
    ks, vs = torch.ones(3, 1, P // 128), torch.ones(3, 1, P // 128)
    out, lse = torch.empty(3, 1, d, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 1, device="cuda")
    ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, 128, 1, 3, 2, 0), dtype=torch.uint8, device="cuda")
    misa.misa_block_attend(c, 128, 1, 3, 2, 0, 1.0, *_cuda(_offsets([2, 1]), torch.ones(3, 1, d).bfloat16(), k, ks, v, vs, table,
                           torch.tensor([length, 40]).int()), None, out, lse, ws)
    quiet = length // P * 31 // 32 * P
    for i, (n, mean) in enumerate([(length - 1, (2 * quiet - length + 1) / (length - 1)), (length, (2 * quiet - length) / length),
                                   (40, 2.0)]):
        assert abs(lse[i, 0].item() - math.log(n)) <= 2.0 ** -18, (i, lse[i, 0].item(), math.log(n))
        assert torch.all((out[i].cpu().double() - mean).abs() <= abs(mean) * 2.0 ** -8 * (1 + 2.0 ** -8)), i


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [2, MANY])
@pytest.mark.parametrize("lengths,counts", [
    ([9000, 0, 6200], [3, 0, 2]),  # nine and seven stages of 1024 tokens in one workgroup
    ([7169, 1024, 1025, 2049], [40, 2, 1, 3]),  # a stage's last and first token
])
def test_attend_whole_rows_of_many_stages(misa, d, most, lengths, counts):
    """More rows in the table than are shared out, so that long rows stay whole: pages and scales are looked up
    by the waves in turn, stage after stage; pages of their own scales, some of them lost."""
    _log(f"[gpu] block attend stages {d} {most} {lengths}")
    g = torch.Generator().manual_seed(51)
    idle = [0] * 1200
    lengths, counts = lengths + idle, counts + idle
    c, table, *pools = _pool(misa, g, lengths, 32, 16, 1, d)
    assert misa.misa_block_attend_workspace_bytes(c, 16, 2, sum(counts), most, 0) == 0
    table[0, 6500 // 32], table[0, 100] = -1, c.pages
    q = torch.randn(sum(counts), 2, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 2, 0, 0.09, _offsets(counts), q, pools, table, lengths, None, most)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [3, MANY])
def test_attend_most_parts(misa, d, most):
    """One row in the 32 parts that are the most, joined eight at a time."""
    _log(f"[gpu] block attend 32 parts {d} {most}")
    g = torch.Generator().manual_seed(52)
    c, table, *pools = _pool(misa, g, [20011], 32, 32, 1, d)
    table[0, 300] = -1
    q = torch.randn(3, 2, d, generator=g).bfloat16()
    _check_attend(misa, c, 32, 2, 0, 0.09, _offsets([3]), q, pools, table, [20011], None, most)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_single_tokens_of_large_caches(misa, d):
    """A table of 64 MB of tokens and more, whose loads are marked as not to be kept; the rows are shorter."""
    _log(f"[gpu] block attend large table {d}")
    g = torch.Generator().manual_seed(53)
    lengths, counts = [3000, 0, 70, 1], [1, 0, 1, 1]
    width = (64 << 20) // (3 * 32 * 2 * 2 * d) + 1
    c, table, *pools = _pool(misa, g, lengths, 32, 16, 2, d, width=width)
    q = torch.randn(3, 8, d, generator=g).bfloat16()
    _check_attend(misa, c, 16, 8, 0, 0.09, _offsets(counts), q, pools, table, lengths, None, 1)


@gpu
@pytest.mark.parametrize("d,kv,heads,k", [(64, 1, 4, 7), (128, 2, 16, 40), (128, 1, 20, 130), (256, 1, 2, 64)])
def test_attend_lists(misa, d, kv, heads, k):
    """A list per query: any order, padding, tokens it does not see yet, the same token twice."""
    _log(f"[gpu] block attend lists {d} {kv} {heads} {k}")
    g = torch.Generator().manual_seed(13)
    lengths, counts = [150, 0, 61], [20, 0, 3]
    c, table, *pools = _pool(misa, g, lengths, 32, 16, kv, d)
    offsets = _offsets(counts)
    n = 24
    q = torch.randn(n, heads, d, generator=g).bfloat16()
    idx = torch.randint(-1, 150, (n, k), generator=g).int()
    idx[3] = -1
    idx[4] = 149  # behind the query
    _check_attend(misa, c, 16, heads, k, d ** -0.5, offsets, q, pools, table, lengths, idx, 20)


@gpu
def test_attend_refused_or_unread_offsets(misa):
    """Offsets that do not ascend, or pass n: nothing outside the arrays is touched, and rows with a
    proper range are right."""
    g = torch.Generator().manual_seed(14)
    lengths = [50, 60, 70]
    c, table, *pools = _pool(misa, g, lengths, 16, 16, 1, 64)
    q = torch.randn(12, 2, 64, generator=g).bfloat16()
    for most in (1, 3, MANY):
        for offsets in ([0, 4, 4, 400], [-9, 4, 7, 12]):
            _check_attend(misa, c, 16, 2, 0, 0.1, torch.tensor(offsets, dtype=torch.int32), q, pools, table, lengths, None,
                          most)
        go = torch.zeros(12, 2, 64, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, 16, 2, 12, most, 0), dtype=torch.uint8, device="cuda")
        off = torch.tensor([8, 3, 9, 1], dtype=torch.int32)
        misa.misa_block_attend(c, 16, 2, 12, most, 0, 0.1, *_cuda(off, q, *pools, table, torch.tensor(lengths).int()), None,
                               go, None, ws)
        torch.cuda.synchronize()


@gpu
def test_far_pages(misa):
    """A pool beyond 4 GiB a buffer: pages whose byte offsets pass 32 bits."""
    P, B, kv, d = 128, 64, 8, 128
    pages = (1 << 32) // (kv * P * d) + 40  # 4.2 GiB of keys, and of values
    rows, L = 2, 300
    k, v = (torch.zeros(pages, kv, P, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.ones(pages, kv, P // B, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3, 0], [1, pages - 2, pages - 30]], dtype=torch.int32)
    c = misa.cache(rows, 3, pages, P, kv, d, d, misa.MISA_FP8_E4M3)
    g = torch.Generator().manual_seed(15)
    kn, vn = (torch.randn(rows * L, kv, d, generator=g).bfloat16().cuda() for _ in range(2))
    offsets, lengths = _offsets([L, L]).cuda(), torch.tensor([L, L], dtype=torch.int32, device="cuda")
    misa.misa_block_write(c, B, rows * L, offsets, lengths, kn, vn, k, ks, v, vs, table.cuda())
    ko, vo = torch.empty_like(kn), torch.empty_like(vn)
    misa.misa_block_read(c, B, rows * L, 1, offsets, None, lengths, k, ks, v, vs, table.cuda(), ko, None, vo, None)
    # a code is off by half a step of its value, or half a subnormal step of the block's scale (at most
    # 2^-5 for values below 448 * 2^-6 = 7)
    assert torch.all((ko.float() - kn.float()).abs() <= kn.float().abs() * 2.0 ** -4 + 2.0 ** -16)
    assert torch.all((vo.float() - vn.float()).abs() <= vn.float().abs() * 2.0 ** -4 + 2.0 ** -16)
    q = torch.randn(6, kv, d, generator=g).bfloat16()
    kc, vc = (x.cpu().float().view(rows, L, kv, d) for x in (ko, vo))
    for most in (1, 3, MANY):
        off = _offsets([3, 3]).cuda()
        out = torch.empty(6, kv, d, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, B, kv, 6, most, 0), dtype=torch.uint8, device="cuda")
        misa.misa_block_attend(c, B, kv, 6, most, 0, 0.1, off, q.cuda(), k, ks, v, vs, table.cuda(), lengths, None, out, None, ws)
        for i in range(6):
            seen = L - 2 + i % 3
            s = torch.einsum("hd,thd->ht", q[i].double(), kc[i // 3, :seen].double()) * 0.1
            p = torch.softmax(s, 1)
            want = torch.einsum("ht,thd->hd", p, vc[i // 3, :seen].double())
            size = torch.einsum("ht,thd->hd", p, vc[i // 3, :seen].double().abs())
            # the result's rounding, the weights' (2^-11), and scores of |s| < 16 to 2^-16
            assert torch.all((out[i].cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2.0 ** -15) + 1e-9)


# ------------------------------------------------------------------ together


def _step(misa, c, B, heads, kv, d, state, n, most, ws):
    """A step of a server's layer: rotate queries and keys in the fused rows, write, attend."""
    spec = misa.rope_spec(heads + kv, d, 0, d, 0, 1, 1, (heads + 2 * kv) * d, (heads + 2 * kv) * d)
    fused = state["fused"]
    misa.misa_rope(spec, n, fused[:, :(heads + kv) * d], state["pos"], state["freq"], fused[:, :(heads + kv) * d], None)
    state["q"].copy_(fused[:, :heads * d].view(n, heads, d))
    state["kn"].copy_(fused[:, heads * d:(heads + kv) * d].view(n, kv, d))
    state["vn"].copy_(fused[:, (heads + kv) * d:].view(n, kv, d))
    misa.misa_block_write(c, B, n, state["offsets"], state["lengths"], state["kn"], state["vn"], state["k"], state["ks"],
                          state["v"], state["vs"], state["table"])
    misa.misa_block_attend(c, B, heads, n, most, 0, d ** -0.5, state["offsets"], state["q"], state["k"], state["ks"],
                           state["v"], state["vs"], state["table"], state["lengths"], None, state["out"], state["lse"], ws)


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_prompt_then_tokens(misa, captured):
    """A prompt in one chunk, then single tokens, two rows, pages taken by misa_page_extend and a row forked
    on the way: every step's outputs against the 64-bit attention over what the cache reads back as, and the
    cache against the values that went in."""
    B, P, kv, heads, d, rows, width = 16, 32, 2, 6, 64, 3, 8
    pages = 30
    g = torch.Generator(device="cuda").manual_seed(16)
    c = misa.cache(rows, width, pages, P, kv, d, d, misa.MISA_FP8_E4M3)
    i32 = dict(dtype=torch.int32, device="cuda")
    state = {
        "k": torch.full((pages, kv, P, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3),
        "v": torch.full((pages, kv, P, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3),
        "ks": torch.full((pages, kv, P // B), math.nan, device="cuda"),
        "vs": torch.full((pages, kv, P // B), math.nan, device="cuda"),
        "table": torch.full((rows, width), -1, **i32), "lengths": torch.zeros(rows, **i32),
        "freq": torch.tensor(misa.misa_rope_frequencies(misa.rope_scaling(0, d, 1e4))[0], dtype=torch.float64, device="cuda"),
    }
    refs = torch.zeros(pages, **i32)
    history = [[] for _ in range(rows)]  # rotated keys and values of each row, 64 bits

    def buffers(n):
        state.update(fused=torch.empty(n, (heads + 2 * kv) * d, dtype=torch.bfloat16, device="cuda"), pos=torch.zeros(n, **i32),
                     q=torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda"),
                     kn=torch.empty(n, kv, d, dtype=torch.bfloat16, device="cuda"),
                     vn=torch.empty(n, kv, d, dtype=torch.bfloat16, device="cuda"), offsets=torch.zeros(rows + 1, **i32),
                     out=torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(n, heads, device="cuda"))

    def extend(counts):
        ok = torch.empty(rows, **i32)
        misa.misa_page_extend(c, rows, torch.arange(rows, **i32), torch.tensor(counts, **i32), state["table"],
                              state["lengths"], refs, ok)
        assert ok.tolist() == [1] * rows

    def fill(counts):
        """New fused rows and their positions, in place."""
        n = sum(counts)
        state["fused"].copy_(torch.randn(state["fused"].shape, generator=g, device="cuda"))
        pos = []
        for r, x in enumerate(counts):
            pos += range(len(history[r]), len(history[r]) + x)
        state["pos"][:n] = torch.tensor(pos, **i32)
        state["offsets"].copy_(_offsets(counts).cuda())

    def check(counts):
        i = 0
        for r, x in enumerate(counts):
            L = len(history[r]) + x
            if L == 0:
                continue
            ko, vo = (torch.empty(L, kv, d, device="cuda") for _ in range(2))
            off = torch.tensor([0] * (r + 1) + [L] * (rows - r), **i32)
            misa.misa_block_read(c, B, L, 0, off, None, state["lengths"], state["k"], state["ks"], state["v"], state["vs"],
                                 state["table"], ko, None, vo, None)
            for j in range(x):
                history[r].append((state["kn"][i + j].double(), state["vn"][i + j].double()))
            for j, cached in enumerate((ko, vo)):
                want = torch.stack([h[j] for h in history[r]])
                # a code: half a step of the value, or half a subnormal step (2^-10) of the block's scale, which is
                # below twice its largest value / 448, that of a head here below 8; twice where a block was rescaled
                assert torch.all((cached.double() - want).abs() <= want.abs() * 2.0 ** -4 + 2 * 2.0 ** -10 * 16 / 448)
            for j in range(x):
                seen = L - x + j + 1
                for h in range(heads):
                    kk, vv = ko[:seen, h // 3].double(), vo[:seen, h // 3].double()
                    s = kk @ state["q"][i + j, h].double() * d ** -0.5
                    p = torch.softmax(s, 0)
                    want, size = p @ vv, p @ vv.abs()
                    tol = want.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2.0 ** -15) + 1e-8
                    assert torch.all((state["out"][i + j, h].double() - want).abs() <= tol)
                    assert abs(state["lse"][i + j, h].item() - torch.logsumexp(s, 0).item()) < 2.0 ** -15
            i += x

    counts = [50, 33, 0]
    buffers(sum(counts))
    extend(counts)
    fill(counts)
    ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, B, heads, sum(counts), 50, 0), dtype=torch.uint8, device="cuda")
    _step(misa, c, B, heads, kv, d, state, sum(counts), 50, ws)
    check(counts)
    # row 2 becomes a copy of row 1: its partly filled last page moves with codes and scales
    src, dst, ok = (torch.empty(1, **i32) for _ in range(3))
    misa.misa_page_fork(c, 1, torch.tensor([1], **i32), torch.tensor([2], **i32), state["table"], state["lengths"], refs,
                        src, dst, ok)
    misa.misa_page_copy(misa.page_buffers([(state["k"], 1, kv * P * d), (state["ks"], 1, kv * P // B * 4),
                                           (state["v"], 1, kv * P * d), (state["vs"], 1, kv * P // B * 4)]), pages, 1, src, dst)
    history[2] = list(history[1])
    counts = [1, 1, 1]
    buffers(3)
    ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, B, heads, 3, 1, 0), dtype=torch.uint8, device="cuda")
    graph = None
    if captured:
        fill(counts)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(misa, c, B, heads, kv, d, state, 3, 1, ws)
    for _ in range(6):
        extend(counts)
        fill(counts)
        if captured:
            graph.replay()
        else:
            _step(misa, c, B, heads, kv, d, state, 3, 1, ws)
        torch.cuda.synchronize()
        check(counts)


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_indexer_keys_from_pages(misa, captured):
    """The indexer's keys kept in pages, read back into its dense layout, give the top-k that it gives for the
    same codes and scales held densely."""
    import synth

    L, T, H, h, k, P, B, batch = 300, 4, 16, 4, 40, 32, 32, 2
    g = torch.Generator().manual_seed(17)
    c, table, pool, scale, _, _ = _pool(misa, g, [L] * batch, P, B, 1, 128)
    keys = torch.randn(batch * L, 1, 128, generator=g).bfloat16()
    offsets, lengths = _offsets([L] * batch).cuda(), torch.tensor([L] * batch, dtype=torch.int32, device="cuda")
    gp, gs, gt = _cuda(pool, scale, table)
    misa.misa_block_write(c, B, batch * L, offsets, lengths, keys.cuda(), None, gp, gs, None, None, gt)
    code, unit, written = ref.read(c, B, offsets.cpu(), None, [L] * batch, *[x.cpu() for x in (gp, gs)], table, batch * L)
    dense, dense_scale = torch.zeros(batch * L, 1, 128, device="cuda").to(E4M3), torch.zeros(batch * L, 1, device="cuda")
    shp = misa.shape(batch, L, T, H, 128, 64, synth.FP8_E4M3)
    q = (50 * torch.randn(batch, T, H, 128, generator=g)).to(E4M3).cuda()
    qs, w = torch.full((batch, T), 0.02, device="cuda"), torch.randn(batch, T, H, generator=g).cuda()
    heads = torch.arange(h, dtype=torch.int32).repeat(batch, T, 1).cuda()
    ws = torch.empty(misa.misa_workspace_bytes(shp, h, k, k), dtype=torch.uint8, device="cuda")

    def top(kk, kks):
        idx, sc = torch.empty(batch, T, k, dtype=torch.int32, device="cuda"), torch.empty(batch, T, k, device="cuda")
        misa.misa_score_topk(shp, h, k, q, qs, w, kk, kks, heads, idx, sc, ws)
        return idx, sc

    def read():
        misa.misa_block_read(c, B, batch * L, 2, offsets, None, lengths, gp, gs, None, None, gt, dense, dense_scale, None, None)

    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            read()
    for _ in range(3):
        dense.view(torch.uint8).zero_()
        graph.replay() if captured else read()
        want = [x.sort(-1).values for x in top(code.cuda(), unit.cuda())]
        got = [x.sort(-1).values for x in top(dense, dense_scale)]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_calls_on_streams_of_their_own(misa):
    """Two attentions at once with workspaces of their own, beside their results one after the other."""
    g = torch.Generator().manual_seed(18)
    jobs = []
    for most, lengths, counts in ((1, [5000, 3000], [1, 1]), (30, [4000], [30])):
        c, table, *pools = _pool(misa, g, lengths, 64, 32, 2, 128)
        q = torch.randn(sum(counts), 8, 128, generator=g).bfloat16()
        on = _cuda(_offsets(counts), q, *pools, table, torch.tensor(lengths).int())
        need = misa.misa_block_attend_workspace_bytes(c, 32, 8, sum(counts), most, 0)
        jobs.append((c, most, on, [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]))

    def call(job, which, out, stream):
        c, most, on, ws = job
        misa.misa_block_attend(c, 32, 8, on[1].shape[0], most, 0, 0.1, *on, None, out, None, ws[which], stream)

    alone = []
    for job in jobs:
        out = torch.empty_like(job[2][1])
        call(job, 0, out, None)
        alone.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(jobs[i % 2][2][1]) for i in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        call(jobs[i % 2], i // 2, outs[i], streams[i])
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(outs[i], alone[i % 2])


@gpu
def test_calls_at_once_against_the_reference(misa):
    """A prompt, drafts, single tokens, lists and writes at once on streams of their own: each against what the
    reference gives for it."""
    _log("[gpu] calls at once")
    g = torch.Generator().manual_seed(61)
    jobs = []
    for most, k, lengths, counts in ((1, 0, [2500, 900], [1, 1]), (5, 0, [1500, 40], [5, 3]), (150, 0, [700], [150]),
                                     (2, 30, [300, 20], [2, 1])):
        c, table, *pools = _pool(misa, g, lengths, 32, 16, 2, 64)
        n = sum(counts)
        q = torch.randn(n, 6, 64, generator=g).bfloat16()
        idx = torch.randint(-1, 300, (n, k), generator=g).int() if k else None
        want = ref.attend(misa, c, 16, 6, k, 0.1, _offsets(counts), q, *pools, table, lengths, idx)
        on = _cuda(_offsets(counts), q, *pools, table, torch.tensor(lengths).int(), idx)
        ws = torch.empty(misa.misa_block_attend_workspace_bytes(c, 16, 6, n, most, k), dtype=torch.uint8, device="cuda")
        jobs.append((c, n, most, k, on, torch.empty_like(on[1]), torch.empty(n, 6, device="cuda"), ws, want))
    lengths, counts = [100, 64, 65, 200], [37, 64, 1, 90]
    c, table, pool, scale, _, _ = _pool(misa, g, lengths, 64, 32, 2, 128)
    new = torch.randn(sum(counts), 2, 128, generator=g).bfloat16()
    codes, units = ref.write(c, 32, _offsets(counts), lengths, new, pool, scale, table)
    writes = [_cuda(_offsets(counts), torch.tensor(lengths).int(), new, pool, scale, table) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (cc, n, most, k, on, out, lse, ws, _), stream in zip(jobs, streams):
            misa.misa_block_attend(cc, 16, 6, n, most, k, 0.1, *on, out, lse, ws, stream)
    for (off, ln, kn, kp, ks, tb), stream in zip(writes, streams[4:]):
        misa.misa_block_write(c, 32, len(new), off, ln, kn, None, kp, ks, None, None, tb, stream)
    torch.cuda.synchronize()
    for _, _, most, k, _, out, lse, _, (wo, wl, out_tol, lse_tol, wide, _) in jobs:
        tol = out_tol + wide if k == 0 and most > 1 else out_tol
        assert torch.all((out.cpu().double() - wo).abs() <= tol + 1e-30)
        empty = wl == -math.inf
        assert torch.equal(lse.cpu() == -math.inf, empty) and torch.all(((lse.cpu().double() - wl).abs() <= lse_tol) | empty)
    for _, _, _, kp, ks, _ in writes:
        assert torch.equal(ks.cpu(), units) and ref.same_codes(kp.cpu(), codes)


@gpu
def test_binding_refuses(misa):
    c = misa.cache(1, 2, 4, 16, 1, 64, 64, misa.MISA_FP8_E4M3)
    i32 = dict(dtype=torch.int32, device="cuda")
    spec = misa.rope_spec(2, 64, 0, 64, 0, 0, 0, 128, 128)
    x, pos = torch.zeros(4, 128, device="cuda"), torch.zeros(4, **i32)
    freq = torch.zeros(32, dtype=torch.float64, device="cuda")
    for bad in (dict(x=x[:, ::2]), dict(x=torch.zeros(4, 130, device="cuda")[:, :128]), dict(x=x.cpu()), dict(pos=pos.long()),
                dict(freq=freq.float()), dict(out=x.cpu()), dict(x=x.flatten()), dict(pos=pos.cpu())):
        a = {**dict(x=x, pos=pos, freq=freq, out=torch.zeros_like(x)), **bad}
        with pytest.raises(ValueError):
            misa.misa_rope(spec, 4, a["x"], a["pos"], a["freq"], a["out"], None)
    pool, scale = torch.zeros(4, 1, 16, 64, dtype=torch.uint8, device="cuda").view(E4M3), torch.ones(4, 1, 1, device="cuda")
    off, ln, table = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 2, **i32)
    new = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(off=off.long()), dict(ln=ln.long()), dict(table=table.long()), dict(new=new.cpu())):
        a = {**dict(off=off, ln=ln, table=table, new=new), **bad}
        with pytest.raises(ValueError):
            misa.misa_block_write(c, 16, 1, a["off"], a["ln"], a["new"], None, pool, scale, None, None, a["table"])
