"""The long-context operators without a GPU: the oracle against its definitions, and the entry points' refusals, each
before any launch."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int8_mqa_decode_gb300 as cai
from int8_mqa_decode_gb300 import build as cai_build
from oracle import kv4, pages
from test_kv4_host import FAKE, _arr


@pytest.fixture(scope="module")
def lib():
    cai_build.build()
    return cai.load()


# ---- the oracle

@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_equal_positions_is_the_plain_one(inter):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(7, 2, 128)).astype(np.float32)
    ang = np.arange(50)[:, None] * (1e4 ** (-np.arange(49) / 49))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = rng.integers(0, 50, 7)
    got = pages.rotate_axes(x, pos[:, None].repeat(3, 1), [i % 3 for i in range(49)], cos, sin, inter)
    assert np.array_equal(got, kv4.rotate(x, pos, cos, sin, inter))
    # One axis moves only its own pairs.
    two = pages.rotate_axes(x, np.stack([pos, pos * 0], 1), [0] * 20 + [1] * 29, cos, sin, inter)
    first = np.arange(0, 40) if inter else np.r_[0:20, 49:69]
    assert np.array_equal(two[..., first], got[..., first])
    rest = np.setdiff1d(np.arange(128), first)
    assert np.array_equal(two[..., rest], x[..., rest])


# ---- refusals

@pytest.mark.parametrize("entry", ["cai_kv_append_rope_axes", "cai_kv4_append_axes"])
def test_axes_refusals(lib, entry):
    kind = cai.cai_kv_pool if "kv4" not in entry else cai.cai_kv4_pool
    rope = cai.cai_rope(FAKE, FAKE, 100, 128, 0)

    def call(rope=rope, axis=(0,) * 64, axes=3, pos=FAKE, pools=_arr(kind), hkv=2, k=FAKE, dt=1, ks=256, q=FAKE, batch=2, n=1,
             off=None, total=0, table=FAKE, maxp=4, start=FAKE):
        r = ctypes.byref(rope) if rope is not None else None
        a = (ctypes.c_uint8 * 64)(*axis) if axis is not None else None
        return getattr(lib, entry)(pools, hkv, r, a, axes, pos, k, FAKE, dt, ks, 256, q, 1024, FAKE, 8, batch, n, off, total,
                                   table, maxp, start, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0 and call(off=FAKE, total=0) == 0
    assert call(rope=None) == 1 and call(axis=None) == 1 and call(pos=None) == 1 and call(pos=FAKE + 2) == 1
    assert call(axes=0) == 2 and call(axes=5) == 2 and call(axes=-1) == 2
    assert call(axis=(3,) + (0,) * 63) == 1 and call(axis=(0,) * 63 + (3,)) == 1
    assert call(axis=(0,) * 32 + (9,) * 32, rope=cai.cai_rope(FAKE, FAKE, 100, 64, 0), batch=0) == 0  # entries past the pairs are not read
    assert call(rope=cai.cai_rope(FAKE, FAKE, 100, 130, 0)) == 2 and call(rope=cai.cai_rope(FAKE, FAKE, 0, 64, 0)) == 1
    assert call(pools=None) == 1 and call(k=None) == 1 and call(ks=255) == 1 and call(table=None) == 1 and call(start=None) == 1


def test_summary_bounds_its_keys():
    rng = np.random.default_rng(1)
    for size in (1e-30, 1.0, 1e6):
        k = rng.normal(size=(20, 128)).astype(np.float32) * np.float32(size)
        codes, s = pages.summarize(k)
        hi, lo = codes[:128].astype(np.float64) * s, codes[128:].astype(np.float64) * s
        slack = 2.0 ** -22 * np.abs(k).max()  # of the divisions' roundings
        assert (k <= hi + slack).all() and (k >= lo - slack).all()
        assert (hi - k.max(0) <= s + slack).all() and (k.min(0) - lo <= s + slack).all()
        assert np.abs(codes).max() == 127
    codes, s = pages.summarize(np.zeros((3, 128)))
    assert s == 0 and (codes == 0).all()


def test_scores_bound_the_logits():
    rng = np.random.default_rng(2)
    k = rng.normal(size=(8, 16, 128)).astype(np.float32)
    q = kv4.bf16_round(rng.normal(size=(5, 128)).astype(np.float32))
    codes, scale = zip(*(pages.summarize(x) for x in k))
    got = pages.scores(q, np.stack(codes), np.array(scale))
    logit = np.einsum("hd,btd->bht", q.astype(np.float64), k).max((1, 2))
    # A query's channels are off by half a code, at the summary's bounds.
    slack = np.abs(np.stack(codes)).reshape(8, 2, 128).max(1).sum(-1) * np.array(scale) * (np.abs(q).max() / 127 / 2)
    assert (logit <= got + slack).all()


def test_corrected_quotients_are_the_divisions():
    """The kernel's x / t: one correction of the product with the rounded inverse, for every pair of bf16 significands."""
    f, wide = np.float32, np.longdouble
    amax = np.arange(128, 256, dtype=np.float32)[:, None]
    t = amax / f(127)
    inv = f(1) / t
    for e in range(12):  # (smaller numerators round to 0)
        x = np.arange(128, 256, dtype=np.float32)[None] * f(2.0 ** -e)
        q = x * inv
        r = (x.astype(wide) - q.astype(wide) * t.astype(wide)).astype(f)  # (exact before its rounding, as a fused product)
        q = (q.astype(wide) + r.astype(wide) * inv.astype(wide)).astype(f)
        assert np.array_equal(np.where(x <= amax, q, 0), np.where(x <= amax, x / t, 0))


@pytest.mark.parametrize("least,most", [(-99, -60), (-20, 0)])  # scales from 2^-100 to 1
def test_twice_corrected_quotients_are_the_divisions(least, most):
    """A summary's x / s: two corrections of the product with the rounded inverse, for fp32 x anywhere in [-127 s, 127 s] and
    within some ulps of whole multiples of s."""
    f, wide = np.float32, np.longdouble
    rng = np.random.default_rng(3)
    amax = (rng.uniform(64, 128, 4000) * 2.0 ** rng.integers(least, most + 1, 4000)).astype(f)[:, None]
    s = amax / f(127)
    inv = f(1) / s
    near = (rng.integers(-127, 128, (4000, 300)) * s.astype(np.float64)).astype(f)
    steps = rng.integers(-3, 4, near.shape)
    for k in range(3):
        near = np.where(np.abs(steps) > k, np.nextafter(near, np.where(steps > 0, f(np.inf), f(-np.inf))), near)
    wild = amax * np.ldexp(rng.uniform(-1, 1, (4000, 300)), -rng.integers(0, 30, (4000, 300))).astype(f)
    x = np.clip(np.concatenate([near, wild, amax, -amax], 1), -amax, amax)
    q = x * inv
    for _ in range(2):
        r = (x.astype(wide) - q.astype(wide) * s.astype(wide)).astype(f)
        q = (q.astype(wide) + r.astype(wide) * inv.astype(wide)).astype(f)
    # A remainder is a multiple of ulp(q) ulp(s), 2^-149 or more for |q| >= 2^-3 and s >= 2^-100; a smaller quotient, whose
    # remainder may be rounded, counts by its sign alone.
    whole = np.abs(x) >= s * f(2.0 ** -3)
    assert np.array_equal(q[whole], (x / s)[whole]) and np.array_equal(np.ceil(q), np.ceil(x / s))


def test_selection_takes_ends_and_ties():
    codes, scale = np.zeros((20, 256), np.int8), np.ones(20, np.float32)
    blocks, tokens = pages.select(np.ones((2, 128), np.float32), codes, scale, 19 * 16 + 3, 16, 6, 1, 2)
    assert list(blocks) == [0, 1, 2, 3, 18, 19] and tokens == 5 * 16 + 4
    codes[7, :128] = 5
    blocks, _ = pages.select(np.ones((2, 128), np.float32), codes, scale, 19 * 16 + 3, 16, 4, 1, 2)
    assert list(blocks) == [0, 7, 18, 19]
    blocks, tokens = pages.select(np.ones((2, 128), np.float32), codes, scale, 37, 16, 4, 1, 2)
    assert list(blocks) == [0, 1, 2] and tokens == 38


def _sums(n=2, **kw):
    a = dict(data=FAKE, num_pages=8, page_size=16, head_dim=128)
    a.update(kw)
    return (cai.cai_kv_summary * n)(*[cai.cai_kv_summary(a["data"], a["num_pages"], a["page_size"], a["head_dim"])] * n)


@pytest.mark.parametrize("entry", ["cai_kv_summarize", "cai_kv4_summarize"])
def test_summarize_refusals(lib, entry):
    kind = cai.cai_kv_pool if "kv4" not in entry else cai.cai_kv4_pool

    def call(pools=_arr(kind), sums=_sums(), hkv=2, batch=2, n=1, off=None, table=FAKE, maxp=4, start=FAKE):
        return getattr(lib, entry)(pools, sums, hkv, batch, n, off, table, maxp, start, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0
    assert call(pools=None) == 1 and call(sums=None) == 1 and call(hkv=0) == 2 and call(hkv=9) == 2
    assert call(sums=_sums(data=None)) == 1 and call(sums=_sums(data=FAKE + 8)) == 1 and call(sums=_sums(num_pages=7)) == 1
    assert call(sums=_sums(page_size=32)) == 1 and call(sums=_sums(page_size=24)) == 2 and call(sums=_sums(head_dim=64)) == 2
    assert call(table=None) == 1 and call(start=None) == 1 and call(maxp=0) == 1 and call(n=-1) == 1 and call(batch=-1) == 1
    assert call(batch=65536) == 2 and call(n=1 << 23) == 2 and call(maxp=(1 << 30) // 16 + 1) == 2
    assert cai.cai_kv_summary_bytes(10) == 2600 and cai.cai_kv_summary_bytes(0) == cai.cai_kv_summary_bytes(4, 0) == 0


def test_select_refusals(lib):
    need = cai.cai_kv_select_workspace_size(2, 2, 8, 2, 64)
    assert need >= 2 * 2 * 64 * 4

    def call(sums=_sums(), hkv=2, q=FAKE, batch=2, n=1, off=None, total=0, hq=8, table=FAKE, maxp=64, start=FAKE, keep=4,
             first=1, last=2, ws=FAKE, ws_bytes=need, pages_out=FAKE, len_out=FAKE):
        return lib.cai_kv_select(sums, hkv, q, batch, n, off, total, hq, table, maxp, start, keep, first, last, ws, ws_bytes,
                                 pages_out, len_out, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0 and call(off=FAKE, total=0) == 0
    assert call(sums=None) == 1 and call(hkv=0) == 2 and call(sums=_sums(page_size=8)) == 2 and call(sums=_sums(data=FAKE + 4)) == 1
    assert call(first=-1) == 1 and call(last=0) == 1 and call(first=3, last=2) == 1 and call(keep=0) == 1
    assert call(first=2147483647, last=2147483647) == 1 and call(keep=(1 << 26) + 1) == 2
    assert call(hq=7) == 2 and call(hq=0) == 2 and call(hq=2 * 129) == 2
    assert call(q=None) == 1 and call(q=FAKE + 8) == 1 and call(table=None) == 1 and call(start=None) == 1
    assert call(pages_out=None) == 1 and call(len_out=None) == 1
    assert call(ws=None) == 3 and call(ws_bytes=need - 1) == 3 and call(ws=FAKE + 64) == 3
    assert call(batch=-1) == 1 and call(n=-1) == 1 and call(off=FAKE, total=-1) == 1 and call(maxp=0) == 1 and call(batch=65536) == 2
    assert call(off=FAKE, total=1 << 30, n=1 << 22) == 2  # a block of a launch for each row and K/V head
    for bad in ((0, 2, 8, 2, 64), (2, -1, 8, 2, 64), (2, 2, 7, 2, 64), (2, 2, 8, 9, 64), (2, 2, 8, 2, 0), (65536, 2, 8, 2, 64)):
        assert cai.cai_kv_select_workspace_size(*bad) == 0


@pytest.mark.parametrize("four", [False, True])
def test_attend_refusals(lib, four):
    entry = lib.cai_kv4_attend_pages if four else lib.cai_kv_attend_pages
    size = cai.cai_kv4_attend_pages_workspace_size if four else cai.cai_kv_attend_pages_workspace_size
    kind = cai.cai_kv4_pool if four else cai.cai_kv_pool
    need = size(3, 64, 2, 100, 16, 4)

    def call(pools=_arr(kind), hkv=2, q=FAKE, rows=3, hq=64, pages=FAKE, width=100, length=FAKE, scale=0.1, splits=4, ws=FAKE,
             ws_bytes=need, out=FAKE):
        return entry(pools, hkv, q, rows, hq, pages, width, length, scale, splits, ws, ws_bytes, out, None, None, None)

    assert need > 0 and call(rows=0) == 0
    assert call(pools=None) == 1 and call(hkv=0) == 2 and call(hkv=9) == 2 and call(pools=_arr(kind, page_size=24)) == 2
    assert call(hq=0) == 2 and call(hq=63) == 2 and call(hq=2 * 129) == 2
    assert call(q=None) == 1 and call(q=FAKE + 8) == 1 and call(pages=None) == 1 and call(length=None) == 1
    assert call(out=None) == 1 and call(out=FAKE + 8) == 1
    assert call(rows=-1) == 1 and call(rows=65536) == 2 and call(width=0) == 1 and call(width=(1 << 26) + 1) == 2
    assert call(scale=float("inf")) == 1 and call(splits=-1) == 1 and call(splits=65) == 1
    assert call(ws=None) == 3 and call(ws_bytes=need - 1) == 3 and call(ws=FAKE + 128) == 3
    for bad in ((0, 64, 2, 100, 16, 0), (3, 63, 2, 100, 16, 0), (3, 64, 9, 100, 16, 0), (3, 64, 2, 0, 16, 0), (3, 64, 2, 100, 24, 0),
                (3, 64, 2, 100, 16, 65), (65536, 64, 2, 100, 16, 0), (3, 258, 2, 100, 16, 0)):
        assert size(*bad) == 0
