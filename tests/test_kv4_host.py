"""The 4-bit cache and the rotated appends without a GPU: the oracle's quantizer and layout against
their definitions, and the entry points' refusals, each before any launch."""
import ctypes
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int8_mqa_decode_gb300 as cai
from int8_mqa_decode_gb300 import build as cai_build
from oracle import kv4

FAKE = 0x10000  # aligned, never dereferenced: every call here is refused (or empty) before a launch


@pytest.fixture(scope="module")
def lib():
    cai_build.build()
    return cai.load()


# ---- the oracle

def test_bf16_round_is_torchs():
    x = np.concatenate([np.random.default_rng(0).normal(size=4000).astype(np.float32) * s for s in (1e-30, 1e-5, 1, 1e5)])
    assert np.array_equal(kv4.bf16_round(x), torch.from_numpy(x).bfloat16().float().numpy())


def test_quantizer_edges():
    x = np.zeros((6, 128), np.float32)
    x[1, 0] = 7.0                               # scale 1: integers are exact
    x[1, 1:8] = [-7, 3.5, 2.5, -0.5, 0.5, 1.5, -1.5]  # ties to even
    x[2] = 1e9                                  # saturates: scale 9344
    x[3, 32:] = 1e-9                            # the scale underflows to 0: codes 0
    x[4, 40] = -2.0 ** -20                      # a subnormal fp16 scale
    x[5, 127] = 448.0                           # only its group of 32 has a scale
    c, s = kv4.quantize4(x)
    assert (c[0] == 0).all() and (s[0] == 0).all()
    assert list(c[1, :8]) == [7, -7, 4, 2, 0, 0, 2, -2] and s[1, 0] == 1
    assert (s[2] == 9344).all() and (c[2] == 7).all()
    assert (s[3] == 0).all() and (c[3] == 0).all()
    assert s[4, 1] == np.float16(2.0 ** -20 / 7) and c[4, 40] == -7 and (c[4, :32] == 0).all()
    assert s[5, 3] == 64 and c[5, 127] == 7 and (s[5, :3] == 0).all()


def test_quantizer_error_and_exact_products():
    x = np.random.default_rng(1).normal(size=(500, 128)).astype(np.float32) * np.logspace(-3, 3, 500, dtype=np.float32)[:, None]
    c, s = kv4.quantize4(x)
    v = kv4.dequantize4(c, s)
    # Half a step; the largest value may be clamped by the scale's rounding, 2^-8 of 7 steps at most.
    step = np.repeat(s.astype(np.float64), 32, -1)
    assert (np.abs(v - x) <= step * (0.5 + 7 * 2.0 ** -8)).all()
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)  # every value is an fp16 number


@pytest.mark.parametrize("page", [16, 32, 64])
def test_layout_is_a_bijection(page):
    """Every bit of a page belongs to exactly one token's code or scale."""
    pool = kv4.pool4(1, page, 0)
    for r in range(page):
        before = pool.copy()
        kv4.write4(pool, [0], r, np.full((1, 128), 7), np.full((1, 4), 1, np.float16), np.full((1, 128), 7),
                   np.full((1, 4), 1, np.float16), page)
        assert (pool & before == before).all()  # disjoint from the tokens before
    assert (pool.reshape(-1, 2304)[:, :2048] == 0xFF).all()
    assert (pool.reshape(-1, 2304)[:, 2048:].copy().view(np.float16) == 1).all()


def test_layout_round_trip():
    rng = np.random.default_rng(2)
    n, page = 90, 32
    table = rng.permutation(5)
    kc, vc = rng.integers(-7, 8, (2, n, 128)).astype(np.int8)
    ks, vs = rng.random((2, n, 4)).astype(np.float16)
    pool = kv4.pool4(5, page)
    kv4.write4(pool, table, 3, kc, ks, vc, vs, page)
    got = kv4.read4(pool, table, np.arange(3, 3 + n), page)
    for a, b in zip(got, (kc, ks, vc, vs)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [2, 98, 128])
def test_rotation(rot, inter):
    """Turns by the angle, keeps lengths, and scores depend on the distance alone."""
    rng = np.random.default_rng(3)
    ang = np.arange(50)[:, None] * (100.0 ** (-np.arange(rot // 2) / (rot // 2)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    x = rng.normal(size=(50, 2, 128)).astype(np.float32)
    y = kv4.rotate(x, np.arange(50), cos, sin, inter)
    assert np.array_equal(y[..., rot:], x[..., rot:]) and np.array_equal(y[0], x[0])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
    q, k = x[:1].repeat(50, 0), x[1:2].repeat(50, 0)
    yq, yk = (kv4.rotate(z, np.arange(50), cos, sin, inter) for z in (q, k))
    assert np.allclose((yq[7] * yk[3]).sum(-1), (yq[45] * yk[41]).sum(-1), atol=1e-4)


# ---- refusals

def _arr(kind, n=2, **kw):
    a = dict(pages=FAKE, num_pages=8, page_size=16, head_dim=128)
    a.update(kw)
    return (kind * n)(*[kind(a["pages"], a["num_pages"], a["page_size"], a["head_dim"])] * n)


def test_page_bytes(lib):
    assert [cai.cai_kv4_page_bytes(p) for p in (16, 32, 64)] == [2304, 4608, 9216]
    assert cai.cai_kv4_page_bytes(0) == cai.cai_kv4_page_bytes(24) == cai.cai_kv4_page_bytes(16, 100) == 0


@pytest.mark.parametrize("entry", ["cai_kv_append_rope", "cai_kv4_append"])
def test_append_refusals(lib, entry):
    kind = cai.cai_kv_pool if entry == "cai_kv_append_rope" else cai.cai_kv4_pool
    rope = cai.cai_rope(FAKE, FAKE, 100, 128, 0)

    def call(pools=_arr(kind), hkv=2, rope=rope, k=FAKE, v=FAKE, dt=1, ks=256, vs=256, q=FAKE, qs=1024, qo=FAKE, hq=8,
             batch=2, n=1, off=None, total=0, table=FAKE, maxp=4, start=FAKE):
        r = ctypes.byref(rope) if rope is not None else None
        return getattr(lib, entry)(pools, hkv, r, k, v, dt, ks, vs, q, qs, qo, hq, batch, n, off, total, table, maxp,
                                   start, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0 and call(off=FAKE, total=0) == 0
    assert call(pools=None) == 1
    assert call(hkv=0) == 2 and call(hkv=9) == 2
    assert call(pools=_arr(kind, page_size=24)) == 2 and call(pools=_arr(kind, head_dim=64)) == 2
    assert call(pools=_arr(kind, pages=FAKE + 8)) == 1 and call(pools=_arr(kind, num_pages=0)) == 1
    mixed = _arr(kind)
    mixed[1].page_size = 32
    assert call(pools=mixed) == 1
    for r in (cai.cai_rope(FAKE, FAKE, 100, 3, 0), cai.cai_rope(FAKE, FAKE, 100, 0, 0), cai.cai_rope(FAKE, FAKE, 100, 130, 0)):
        assert call(rope=r) == 2
    for r in (cai.cai_rope(None, FAKE, 100, 64, 0), cai.cai_rope(FAKE, FAKE, 0, 64, 0), cai.cai_rope(FAKE, FAKE + 2, 9, 64, 0)):
        assert call(rope=r) == 1
    assert call(dt=2) == 1
    assert call(ks=255) == 1 and call(vs=128) == 1 and call(ks=260) == 1  # too short, not whole 16 bytes of bf16
    assert call(dt=0, ks=258) == 1
    assert call(k=FAKE + 8) == 1 and call(v=None) == 1 and call(table=None) == 1 and call(start=None) == 1
    assert call(rope=None) == 1                    # queries without a rotation
    assert call(hq=0) == 1                         # q given, no heads
    assert call(q=None) == 1 and call(qo=None) == 1 and call(qs=1000) == 1 and call(qs=1028) == 1 and call(hq=-1) == 1
    assert call(qs=2048, q=FAKE, qo=FAKE) == 1     # in place only when contiguous
    assert call(hq=1025, qs=1 << 20) == 2
    assert call(batch=-1) == 1 and call(n=-1) == 1 and call(off=FAKE, total=-1) == 1 and call(maxp=0) == 1
    assert call(batch=65536) == 2 and call(maxp=(1 << 30) // 16 + 1) == 2 and call(n=1 << 23) == 2


@pytest.mark.parametrize("entry", ["cai_kv_read", "cai_kv4_read"])
def test_read_refusals(lib, entry):
    kind = cai.cai_kv_pool if entry == "cai_kv_read" else cai.cai_kv4_pool

    def call(pools=_arr(kind), hkv=2, k=FAKE, v=FAKE, dt=0, batch=2, n=1, off=None, total=0, table=FAKE, maxp=4, start=FAKE):
        return getattr(lib, entry)(pools, hkv, k, v, dt, batch, n, off, total, table, maxp, start, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0
    assert call(k=None, v=None) == 1 and call(k=FAKE + 4) == 1 and call(v=FAKE + 8) == 1
    assert call(dt=7) == 1 and call(hkv=0) == 2 and call(start=None) == 1 and call(table=None) == 1
    assert call(pools=None) == 1 and call(maxp=-1) == 1 and call(n=-1) == 1


def test_decode_refusals(lib):
    def call(pools=_arr(cai.cai_kv4_pool), hkv=2, q=FAKE, batch=2, hq=8, table=FAKE, maxp=64, ctx=FAKE, window=0, scale=0.1,
             splits=1, ws=None, ws_bytes=0, out=FAKE):
        return lib.cai_kv4_decode(pools, hkv, q, batch, hq, table, maxp, ctx, window, scale, splits, ws, ws_bytes, out, None,
                                  None, None)

    assert call(batch=0) == 0
    assert call(pools=None) == 1 and call(hkv=9) == 2
    assert call(hq=0) == 2 and call(hq=7) == 2 and call(hq=2 * 129) == 2
    assert call(q=None) == 1 and call(q=FAKE + 8) == 1 and call(out=FAKE + 8) == 1 and call(ctx=None) == 1
    assert call(window=-1) == 1 and call(scale=float("inf")) == 1 and call(splits=65) == 1 and call(splits=-1) == 1
    assert call(maxp=0) == 1 and call(batch=65536) == 2
    need = cai.cai_kv4_decode_workspace_size(2, 8, 2, 64, 16, 0, 4)
    assert need > 0
    assert call(splits=4) == 3 and call(splits=4, ws=FAKE, ws_bytes=need - 1) == 3
    assert call(splits=4, ws=FAKE + 128, ws_bytes=need) == 3
    assert call(splits=0) == 3
    assert cai.cai_kv4_decode_workspace_size(2, 8, 2, 64, 16, 0, 1) == 0  # one range: no partials
    for bad in ((0, 8, 2, 64, 16, 0, 0), (2, 7, 2, 64, 16, 0, 0), (2, 8, 9, 64, 16, 0, 0), (2, 8, 2, 64, 24, 0, 0),
                (2, 8, 2, 64, 16, -1, 0), (2, 8, 2, 64, 16, 0, 65)):
        assert cai.cai_kv4_decode_workspace_size(*bad) == 0


def test_prefill_refusals(lib):
    def call(pools=_arr(cai.cai_kv4_pool), hkv=2, q=FAKE, batch=2, n=4, off=None, total=0, hq=8, table=FAKE, maxp=64,
             prefix=FAKE, window=0, scale=0.1, ws=None, ws_bytes=0, out=FAKE):
        return lib.cai_kv4_prefill(pools, hkv, q, batch, n, off, total, hq, table, maxp, prefix, window, scale, ws, ws_bytes,
                                   out, None, None, None)

    assert call(batch=0) == 0 and call(n=0) == 0 and call(off=FAKE, total=0) == 0
    assert call(hq=6) == 2 and call(hq=2 * 256) == 2 and call(hq=7) == 2   # a power of two of heads per K/V head
    assert call(pools=None) == 1 and call(q=None) == 1 and call(prefix=None) == 1 and call(out=FAKE + 2) == 1
    assert call(window=-1) == 1 and call(scale=float("nan")) == 1 and call(n=-1) == 1 and call(off=FAKE, total=-1) == 1
    assert call(batch=40000) == 2 and call(maxp=(1 << 24) // 16 + 1) == 2
    need = cai.cai_kv4_prefill_workspace_size(2, 8, 2, 64, 16)
    assert need > 0 and call() == 3 and call(ws=FAKE, ws_bytes=need - 1) == 3 and call(ws=FAKE + 16, ws_bytes=need) == 3


def test_binding_refuses_what_it_can_see(lib):
    """CPU tensors, wrong types and shapes never reach the library."""
    with pytest.raises(ValueError):
        cai.KV4Pool(4, 16, pages=torch.zeros(4 * 2304, dtype=torch.uint8))  # not on a GPU
    with pytest.raises(ValueError):
        cai.Rope(torch.zeros(4, 64), torch.zeros(4, 32))
    with pytest.raises(ValueError):
        cai.Rope(torch.zeros(4, 64), torch.zeros(4, 64))
    with pytest.raises(TypeError):
        cai.cai_kv4_decode(["pool"], torch.zeros(1, 8, 128), None, None, 0, 1.0, 0, None, None)


def test_header_declares_what_the_binding_calls():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "cai.h")).read()
    for name in cai.__all__:
        if name.startswith("cai_"):
            assert re.search(r"\b%s\s*\(" % name, text), name
