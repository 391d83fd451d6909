"""Attention over the 4-bit cache at the edges of its arguments, against the 64-bit oracle.

Bounds: those of test_gpu_kv4.py, with the softmax scale's magnitude where that file has its one scale.
|out - ref| <= 2^-8 |ref| (the output's rounding to bf16) + (2^-11 + 2^-12) sum p|v| (a weight's rounding to
fp16 and its exponent's) + n 2^-25 max|v| (weights among the subnormals of fp16), the last two
rounded themselves (a factor 1 + 2^-8).  lse: 2^-20 of scale * sum |q k| and of 1 + |lse|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
from oracle import kv4  # noqa: E402
from test_gpu_kv4 import DEV, SCALE, Cache, _built, dev, flag, host, queries  # noqa: E402,F401


def check_rows(cache, out, lse, q, b, first, window, scale, where):
    """Rows out, lse, q [n][hq][128] of sequence b at positions first .. against the oracle."""
    n, g = q.shape[0], q.shape[1] // cache.hkv
    for j in range(cache.hkv):
        k, v = cache.k[j][b], cache.v[j][b]
        pos, at = np.arange(len(k))[None], first + np.arange(n)[:, None]
        seen = pos <= at
        if window:
            seen &= pos > at - window
        hs = slice(j * g, (j + 1) * g)
        ref, rl, a, big = kv4.attend_rows(q[:, hs].astype(np.float64), k, v, scale, seen)
        got, gl = out[:, hs].astype(np.float64), lse[:, hs].astype(np.float64)
        none = ~np.isfinite(rl)
        assert (gl[none] == -np.inf).all() and (got[none] == 0).all(), where
        assert np.isfinite(got).all() and np.isfinite(gl[~none]).all(), where
        soft = (2.0 ** -11 + 2.0 ** -12) * a + seen.sum(1)[:, None, None] * 2.0 ** -25 * np.abs(v).max(initial=0)
        bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * soft
        err = np.abs(got - ref)
        assert (err[~none] <= bound[~none]).all(), (where, (err - bound)[~none].max())
        off = np.abs(gl[~none] - rl[~none])
        assert (off <= 2.0 ** -20 * (big + 1 + np.abs(np.where(none, 0, rl)))[~none]).all(), (where, off.max())


def decode(pools, q, table, ctx, window=0, scale=SCALE, splits=0, page=16):
    n = cai.cai_kv4_decode_workspace_size(q.shape[0], q.shape[1], len(pools), table.shape[1], page, window, splits)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if n else None
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse, err = torch.full(q.shape[:2], float("nan"), device=DEV), flag()
    cai.cai_kv4_decode(pools, q, table, dev(np.array(ctx, np.int32)), window, scale, splits, ws, out, lse, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    return host(out), host(lse)


def prefill(pools, q, table, prefix, new, window=0, scale=SCALE, page=16, packed=True, max_new=None):
    n = cai.cai_kv4_prefill_workspace_size(len(new), q.shape[1], len(pools), table.shape[1], page)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse, err = torch.full(q.shape[:2], float("nan"), device=DEV), flag()
    pre = dev(np.array(prefix, np.int32))
    if packed:
        off = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        cai.cai_kv4_prefill(pools, q, table, pre, window, scale, ws, out, lse, err, q_offsets=off, max_new=max_new or max(new))
    else:
        sh = lambda t: t.unflatten(0, (len(new), new[0]))  # noqa: E731
        cai.cai_kv4_prefill(pools, sh(q), table, pre, window, scale, ws, sh(out), sh(lse), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    return host(out), host(lse)


# ------------------------------------------------------------------- softmax scales of any sign

LENGTHS = [1, 16, 31, 33, 0, 127, 129, 300, 1000]


@pytest.mark.parametrize("scale", [0.0, -SCALE, -3 * SCALE])
@pytest.mark.parametrize("hq", [1, 8, 12, 32, 64])
def test_decode_scales(scale, hq):
    """A masked key counts for nothing whatever the scale: contexts that end inside a step, windows that start in one."""
    cache = Cache(LENGTHS, 1, 16, seed=hq)
    q = queries(np.random.default_rng(hq), len(LENGTHS), hq)
    for window, splits in ((0, 0), (0, 3), (100, 0), (333, 2)):
        out, lse = decode(cache.pools, q, cache.table, LENGTHS, window, scale, splits)
        for b, n in enumerate(LENGTHS):
            check_rows(cache, out[b:b + 1], lse[b:b + 1], host(q[b:b + 1]), b, n - 1, window, scale, (b, n, window, splits))


@pytest.mark.parametrize("scale", [0.0, -SCALE])
@pytest.mark.parametrize("hkv,hq", [(2, 8), (1, 32)])
@pytest.mark.parametrize("window", [0, 70])
def test_prefill_scales(scale, hkv, hq, window):
    """The same in chunks, packed rows with single tokens among them, and calls of one token each."""
    prefix, new = [0, 300, 17, 129, 64], [40, 1, 3, 1, 2]
    cache = Cache([a + n for a, n in zip(prefix, new)], hkv, 16, seed=hq)
    q = queries(np.random.default_rng(hq), sum(new), hq)
    off = np.concatenate([[0], np.cumsum(new)])
    out, lse = prefill(cache.pools, q, cache.table, prefix, new, window, scale)
    for b, n in enumerate(new):
        s = slice(off[b], off[b + 1])
        check_rows(cache, out[s], lse[s], host(q[s]), b, prefix[b], window, scale, ("packed", b))
    for n in (1, 2):
        first = [a + m - n for a, m in zip(prefix, new)]
        some = [b for b in range(5) if first[b] >= 0]
        qn = queries(np.random.default_rng(n), len(some) * n, hq)
        out, lse = prefill(cache.pools, qn, cache.table[some].contiguous(), [first[b] for b in some], [n] * len(some), window,
                           scale, packed=False)
        for i, b in enumerate(some):
            s = slice(i * n, (i + 1) * n)
            check_rows(cache, out[s], lse[s], host(qn[s]), b, first[b], window, scale, (n, b))


# ------------------------------------------------------------ a heavy key beside a long flat rest

# The largest logit has a weight of 2^7 and more, which is part of the sum that divides, so a weight among the
# subnormals of fp16 is off by 2^-25 / 2^7 of the sum at most: n 2^-32 max|v| where the bound above has n 2^-25.  Long
# sums: a thread adds n / 128 weights (and 16 of a tile) in fp32, n 2^-30 of their sum at most; the products add
# n / 16 times, a bit of fp32 cut off each time, n 2^-27 of sum p|v|.
SINK_KEYS = 131072


@pytest.fixture(scope="module")
def sink():
    """One K/V head: position 0 has the only key that is not 0 and the only value that is."""
    rng = np.random.default_rng(77)
    k, v = np.zeros((SINK_KEYS, 128), np.float32), rng.normal(size=(SINK_KEYS, 128)).astype(np.float32) + 1
    k[0, 0], v[0] = 7.0, 0.0  # (its group's scale is 1: the cache has 7)
    pages = SINK_KEYS // 64
    pool = cai.KV4Pool(pages, 64)
    table = dev(rng.permutation(pages).astype(np.int32)[None])
    cai.cai_kv4_append([pool], dev(k)[None, :, None], dev(v)[None, :, None], table, torch.zeros(1, dtype=torch.int32, device=DEV))
    return pool, table, kv4.dequantize4(*kv4.quantize4(v))


def check_sink(sink, out, lse, q, n, where):
    """out, lse, q [hq][128] of a row that attends positions 0 .. n - 1."""
    v = sink[2][:n]
    z = q[:, 0].astype(np.float64) * 7.0 * SCALE
    total = np.exp(z) + (n - 1)
    ref = v.sum(0)[None] / total[:, None]
    each = 2.0 ** -11 + 2.0 ** -12 + n * (2.0 ** -27 + 2.0 ** -30)
    soft = each * np.abs(v).sum(0)[None] / total[:, None] + n * 2.0 ** -32 * np.abs(v).max()
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * soft
    err = np.abs(out.astype(np.float64) - ref)
    assert (err <= bound).all(), (where, err.max(), np.abs(ref).max())
    assert (np.abs(lse - np.log(total)) <= 2.0 ** -20 * (z + 1 + np.log(total)) + n * 2.0 ** -30).all(), where


def sink_queries(rows, hq):
    """Logits of the heavy key between 14 and 19 (20 to 27 in powers of two): the rest has up to a sixth of the weight."""
    q = np.random.default_rng(hq).normal(size=(rows, hq, 128)).astype(np.float32)
    q[..., 0] = np.linspace(14, 19, rows * hq).reshape(rows, hq) / (7 * SCALE)
    return dev(q, torch.bfloat16)


@pytest.mark.parametrize("splits", [0, 1, 7])
@pytest.mark.parametrize("hq", [8, 16, 32, 64])
def test_decode_counts_small_weights(sink, hq, splits):
    q = sink_queries(2, hq)
    ctx = [SINK_KEYS, 70001]
    out, lse = decode([sink[0]], q, sink[1].repeat(2, 1), ctx, splits=splits, page=64)
    for b, n in enumerate(ctx):
        check_sink(sink, out[b], lse[b], host(q[b]), n, (b, splits))


@pytest.mark.parametrize("packed", [False, True])
def test_prefill_counts_small_weights(sink, packed):
    prefix, n, hq = SINK_KEYS - 9, 9, 32
    q = sink_queries(n, hq)
    out, lse = prefill([sink[0]], q, sink[1], [prefix], [n], page=64, packed=packed)
    for i in range(n):
        check_sink(sink, out[i], lse[i], host(q[i]), prefix + i + 1, i)
