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
