"""The cache operators at the edges of their arguments, against the 64-bit oracle.

Appends and fp32 reads are exact.  Bounds of the attention: those of test_gpu_kv4.py, with the softmax scale's magnitude
where that file has its one scale:
|out - ref| <= 2^-8 |ref| (the output's rounding to bf16) + (2^-11 + 2^-12) sum p|v| (a weight's rounding to
fp16 and its exponent's) + n 2^-25 max|v| (weights among the subnormals of fp16), the last two
rounded themselves (a factor 1 + 2^-8).  lse: 2^-20 of scale * sum |q k| and of 1 + |lse|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
import oracle  # noqa: E402
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


# -------------------------------------------------------------------------- page rings, long prompts

def ring_table(cache, keep_from):
    """The cache's table with -1 for the pages wholly before position keep_from[b], as a recycled local buffer has them."""
    t = cache.table_np.copy()
    for b, lo in enumerate(keep_from):
        t[b, :max(0, lo) // cache.page] = -1
    return dev(t)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hq", [8, 32, 64])
@pytest.mark.parametrize("window", [17, 128, 700])
def test_decode_of_recycled_pages(page, hq, window):
    """Pages before the window may have gone: no flag, and the same result as with them there."""
    lengths = [5, 64, 129, 700, 1500]
    cache = Cache(lengths, 1, page, seed=window)
    q = queries(np.random.default_rng(hq), len(lengths), hq)
    table = ring_table(cache, [n - window for n in lengths])
    for splits in (0, 3):
        out, lse = decode(cache.pools, q, table, lengths, window, splits=splits, page=page)
        for b, n in enumerate(lengths):
            check_rows(cache, out[b:b + 1], lse[b:b + 1], host(q[b:b + 1]), b, n - 1, window, SCALE, (b, splits))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("packed", [False, True])
def test_prefill_of_recycled_pages(page, packed):
    window, new = 100, [20, 20, 20, 20] if not packed else [20, 1, 7, 0]
    prefix = [0, 90, 131, 900]
    cache = Cache([a + n for a, n in zip(prefix, new)], 2, page, seed=page)
    q = queries(np.random.default_rng(page), sum(new), 16)
    table = ring_table(cache, [a + 1 - window for a in prefix])
    out, lse = prefill(cache.pools, q, table, prefix, new, window, page=page, packed=packed)
    off = np.concatenate([[0], np.cumsum(new)])
    for b, n in enumerate(new):
        s = slice(off[b], off[b + 1])
        if n:
            check_rows(cache, out[s], lse[s], host(q[s]), b, prefix[b], window, SCALE, b)


@pytest.mark.parametrize("window", [0, 300])
def test_prefill_of_a_first_prompt(window):
    """Nothing before it, more than a thousand tokens, and another one beside it."""
    new = [1100, 700]
    cache = Cache(new, 1, 64, seed=21)
    q = queries(np.random.default_rng(21), sum(new), 4)
    out, lse = prefill(cache.pools, q, cache.table, [0, 0], new, window, page=64)
    for b, s in enumerate((slice(0, 1100), slice(1100, 1800))):
        check_rows(cache, out[s], lse[s], host(q[s]), b, 0, window, SCALE, b)


def test_prefill_over_several_windows_of_sequences():
    """A packed call's sequences are walked 32 at a time: a window without rows, one of single tokens alone, a last one
    that is not full, and a bound on a sequence's rows far above what any brings."""
    rng = np.random.default_rng(22)
    stored = Cache([200, 170], 2, 16, seed=22)
    new = rng.integers(0, 12, 141)
    new[32:64], new[64:96], new[100], new[140] = 0, 1, 90, 33
    which = np.arange(141) % 2
    prefix = [stored.lengths[w] - int(k) for w, k in zip(which, new)]
    q = queries(rng, int(new.sum()), 16)
    table = stored.table[torch.from_numpy(which).to(DEV)].contiguous()
    off = np.concatenate([[0], np.cumsum(new)])
    for bound in (90, 4096):
        out, lse = prefill(stored.pools, q, table, prefix, new.tolist(), max_new=bound)
        for b, n in enumerate(new):
            s = slice(off[b], off[b + 1])
            if n:
                check_rows(stored, out[s], lse[s], host(q[s]), which[b], prefix[b], 0, SCALE, (b, bound))


# ------------------------------------------------------------------------------- rotated appends

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("rot,shift", [(2, 0), (8, 0), (24, 0), (98, 0), (8, 1), (128, 1), (64, 1)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("new", [[3, 0, 1], [40, 2, 17]])
def test_half_split_rotations(four, rot, shift, in_place, new):
    """Half-split pairs that are not whole vectors (rot / 2 not a multiple of 4 for K, of 8 for q), more query heads than a
    warp takes, and tables that start 4 bytes past a 16-byte boundary; exact."""
    rng = np.random.default_rng(rot + shift)
    new, start = np.array(new), np.array([5, 0, 30])
    rows, hq, hkv, page = int(new.sum()), 13, 2, 16
    q, k, v = (rng.normal(size=(rows, h, 128)).astype(np.float32) for h in (hq, hkv, hkv))
    q, k, v = (dev(x, torch.bfloat16) for x in (q, k, v))
    ang = rng.uniform(-7, 7, size=(80, rot // 2)).astype(np.float32)
    cos, sin = np.cos(ang), np.sin(ang)

    def at_offset(x):
        room = torch.empty(x.size + 4, device=DEV)
        t = room[shift:shift + x.size].view(x.shape)
        t.copy_(dev(x))
        return t

    table = rng.permutation(16).astype(np.int32)[:15].reshape(3, 5)
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    pools = [cls(16, page, pages=torch.zeros(16 * bytes_, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
    pos = np.concatenate([s + np.arange(n) for s, n in zip(start, new)])
    want = kv4.bf16_round(kv4.rotate(host(q), pos, cos, sin, False))
    kr, vr = kv4.rotate(host(k), pos, cos, sin, False), host(v)
    qo, err = q if in_place else torch.empty_like(q), flag()
    (cai.cai_kv4_append if four else cai.cai_kv_append_rope)(
        pools, k, v, dev(table), dev(start.astype(np.int32)), rope=cai.Rope(at_offset(cos), at_offset(sin)), q=q, q_out=qo,
        q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()), err_flag=err)
    assert err.item() == 0
    assert np.array_equal(host(qo), want)
    at = np.concatenate([[0], np.cumsum(new)])
    for j in range(hkv):
        ref = np.zeros(16 * bytes_, np.uint8)
        for b in range(3):
            s = slice(at[b], at[b + 1])
            if not new[b]:
                continue
            if four:
                kv4.write4(ref, table[b], int(start[b]), *kv4.quantize4(kr[s, j]), *kv4.quantize4(vr[s, j]), page)
            else:
                oracle.pool_write(ref, table[b], int(start[b]), *oracle.quantize_rows(kr[s, j]), *oracle.quantize_rows(vr[s, j]), page)
        assert np.array_equal(pools[j].pages.cpu().numpy(), ref), j


@pytest.mark.parametrize("four", [False, True])
def test_rows_under_a_loose_bound(four):
    """max_new far above every sequence's count: the same bytes and values as under the tight one."""
    rng = np.random.default_rng(31)
    new = rng.integers(0, 3, 70)
    start = rng.integers(0, 60, 70)
    rows = int(new.sum())
    k, v = (dev(rng.normal(size=(rows, 8, 128)).astype(np.float32)) for _ in range(2))
    table = dev(rng.permutation(70 * 4).astype(np.int32).reshape(70, 4))
    off, at = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), dev(start.astype(np.int32))
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    append, read = (cai.cai_kv4_append, cai.cai_kv4_read) if four else (cai.cai_kv_append_rope, cai.cai_kv_read)
    got = []
    for bound in (2, 9000):
        pools = [cls(280, 16, pages=torch.zeros(280 * bytes_, dtype=torch.uint8, device=DEV)) for _ in range(8)]
        err, ko, vo = flag(), torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
        append(pools, k, v, table, at, q_offsets=off, max_new=bound, err_flag=err)
        read(pools, ko, vo, table, at, q_offsets=off, max_new=bound, err_flag=err)
        assert err.item() == 0
        got.append((torch.stack([p.pages for p in pools]), ko, vo))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    want = kv4.dequantize4(*kv4.quantize4(host(k))).astype(np.float32) if four else None
    if four:
        assert np.array_equal(host(got[0][1]), want)


def test_packed_steps_that_follow_each_other():
    """Appends and packed attention back to back on one q buffer and one workspace: each launch starts when the one before
    allows it, and the results are those of calls that were waited for one by one."""
    rng = np.random.default_rng(41)
    hkv, hq, page, steps = 2, 16, 16, 6
    new = np.array([1, 60, 1, 1, 35, 0, 1])
    start = np.array([500, 0, 3, 1200, 77, 9, 0])
    table_np = rng.permutation(7 * 110).astype(np.int32).reshape(7, 110)
    rows = int(new.sum())
    qkv = [queries(rng, rows, hq + 2 * hkv) for _ in range(steps)]
    off, table = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), dev(table_np)
    cos, sin = (dev(f(np.outer(np.arange(1800), 1e4 ** (-np.arange(64) / 64))).astype(np.float32)) for f in (np.cos, np.sin))
    rope = cai.Rope(cos, sin)
    at = [dev((start + i * new).astype(np.int32)) for i in range(steps)]

    def run(wait):
        pools = [cai.KV4Pool(7 * 110, page, pages=torch.full((7 * 110 * 2304,), 0x99, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
        for p in pools:
            p.pages.view(-1, 2304)[:, 2048:] = 0x2C  # every slot's scale is a small number: the prefixes hold something
        ws = torch.full((cai.cai_kv4_prefill_workspace_size(7, hq, hkv, 110, page),), 0xFF, dtype=torch.uint8, device=DEV)
        qr = torch.empty(rows, hq, 128, dtype=torch.bfloat16, device=DEV)
        outs = [torch.zeros(rows, hq, 128, dtype=torch.bfloat16, device=DEV) for _ in range(steps)]
        lses, err = [torch.zeros(rows, hq, device=DEV) for _ in range(steps)], flag()
        torch.cuda.synchronize()
        for i in range(steps):
            x = qkv[i]
            cai.cai_kv4_append(pools, x[:, hq:hq + hkv], x[:, hq + hkv:], table, at[i], rope=rope, q=x[:, :hq], q_out=qr,
                               q_offsets=off, max_new=60, err_flag=err)
            if wait:
                torch.cuda.synchronize()
            cai.cai_kv4_prefill(pools, qr, table, at[i], 0, SCALE, ws, outs[i], lses[i], err, q_offsets=off, max_new=60)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert err.item() == 0
        return torch.stack(outs), torch.stack(lses), torch.stack([p.pages for p in pools])

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
