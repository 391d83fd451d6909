"""The cache operators on a GPU against the 64-bit oracle: rotated appends (bit for bit, whole pools),
reads, decode and prefill attention over the 4-bit cache, and a run of them together.

Bounds.  Appends and fp32 reads are exact.  Attention: K, V and q are exact fp16 products with fp32
sums; a weight is 2^z rounded to fp16 (2^-11 of it) with z off by the sums' rounding, at most 2^-12 of
the weight for the logits here (checked by the bound on lse), and where it falls among the
subnormals of fp16 it is off by 2^-25 of the largest at most; the output is rounded to bf16 once.
So |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-12) sum p|v| + n 2^-25 max|v|, and the last two terms are
themselves rounded (a factor 1 + 2^-8).  lse: the fp32 sums of 128 products, and of the weights:
2^-20 of scale * sum |q k| and of 1 + |lse|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
import oracle  # noqa: E402
from oracle import kv4  # noqa: E402

SCALE = 128 ** -0.5
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_mqa_decode_gb300 import build
    build.build()
    yield
    cai.cai_set_fault_injection(-1)
    cai.cai_set_wait_limit_ns(0)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if dtype is None else t.to(dtype)


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def tables(rng, lengths, page, spare=3, width=0):
    """A shuffled block table with -1 where nothing is, and the pool's pages."""
    pages = -(-np.asarray(lengths) // page)
    total = int(pages.sum()) + spare
    perm, t, at = rng.permutation(total).astype(np.int32), np.full((len(pages), max(1, width, pages.max(initial=0))), -1, np.int32), 0
    for b, n in enumerate(pages):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


class Cache:
    """hkv 4-bit pools holding random K, V of every sequence, all other bytes 0xFF (scales NaN); host values kept."""

    def __init__(self, lengths, hkv, page, seed=0, width=0, v_size=1.0):
        rng = np.random.default_rng(seed)
        self.lengths, self.page, self.hkv = list(lengths), page, hkv
        self.table_np, self.num_pages = tables(rng, lengths, page, width=width)
        self.table = dev(self.table_np)
        self.pools, self.k, self.v = [], [], []
        for _ in range(hkv):
            ks, vs, host = [], [], kv4.pool4(self.num_pages, page)
            dst = dev(host)
            pool = cai.KV4Pool(self.num_pages, page, pages=dst)
            for b, n in enumerate(lengths):
                x = rng.normal(size=(2, n, 128)).astype(np.float32)
                x[0, :, rng.integers(0, 128, 3)] *= 4
                x[1] *= v_size
                if n:  # through the append, which has tests of its own
                    cai.cai_kv4_append([pool], dev(x[0])[None, :, None], dev(x[1])[None, :, None], self.table[b:b + 1],
                                       torch.zeros(1, dtype=torch.int32, device=DEV))
                ks.append(kv4.dequantize4(*kv4.quantize4(x[0])))
                vs.append(kv4.dequantize4(*kv4.quantize4(x[1])))
            self.pools.append(pool)
            self.k.append(ks)
            self.v.append(vs)

    def check(self, out, lse, q, b, first, window, where):
        """Rows out, lse, q [n][hq][128] of sequence b at positions first .. against the oracle."""
        n, hq = q.shape[0], q.shape[1]
        g = hq // self.hkv
        for j in range(self.hkv):
            k, v = self.k[j][b], self.v[j][b]
            pos, at = np.arange(len(k))[None], first + np.arange(n)[:, None]
            seen = pos <= at
            if window:
                seen &= pos > at - window
            hs = slice(j * g, (j + 1) * g)
            ref, rl, a, big = kv4.attend_rows(q[:, hs].astype(np.float64), k, v, SCALE, seen)
            got, gl = out[:, hs].astype(np.float64), lse[:, hs].astype(np.float64)
            none = ~np.isfinite(rl)
            assert (gl[none] == -np.inf).all() and (got[none] == 0).all(), where
            soft = (2.0 ** -11 + 2.0 ** -12) * a + seen.sum(1)[:, None, None] * 2.0 ** -25 * np.abs(v).max(initial=0)
            bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * soft
            err = np.abs(got - ref)
            assert (err[~none] <= bound[~none]).all(), (where, (err - bound)[~none].max())
            lb = 2.0 ** -20 * (big + 1 + np.abs(np.where(none, 0, rl)))
            off = np.abs(gl[~none] - rl[~none])
            assert (off <= lb[~none]).all(), (where, off.max())


def queries(rng, rows, hq, size=1.0):
    return dev(rng.normal(size=(rows, hq, 128)).astype(np.float32) * size, torch.bfloat16)


def host(t):
    return t.float().cpu().numpy()


# ------------------------------------------------------------------------------------ append

APPENDS = [  # hkv, hq, page, rot, interleaved, bf16, new tokens, starts
    (1, 8, 16, 128, False, True, [1, 1, 1], [0, 15, 63]),
    (2, 6, 32, 128, True, True, [33, 0, 1, 70], [0, 5, 31, 17]),
    (8, 8, 64, 64, False, False, [1, 2, 130], [63, 62, 0]),
    (3, 0, 16, 98, False, True, [5, 40], [9, 1]),
    (1, 1, 32, 2, True, False, [16, 17, 15], [16, 15, 1]),
    (4, 0, 64, 0, False, False, [20], [44]),
]


def append_case(four, case, packed, seed=0, slices=True):
    hkv, hq, page, rot, inter, bf16, new, start = case
    rng = np.random.default_rng(seed)
    new, start = np.array(new), np.array(start)
    n = int(new.sum())
    table, num_pages = tables(rng, start + new, page)
    dt = torch.bfloat16 if bf16 else torch.float32
    qkv = dev(rng.normal(size=(n, hq + 2 * hkv, 128)).astype(np.float32) * 3, dt)
    qkv[:, -1] *= 1e-3
    q = qkv[:, :hq] if bf16 else qkv[:, :hq].bfloat16()
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not slices:
        k, v = k.contiguous(), v.contiguous()
    pos = np.concatenate([s + np.arange(m) for s, m in zip(start, new)]).astype(int) if n else np.zeros(0, int)
    ang = np.arange(300)[:, None] * (1e4 ** (-np.arange(max(1, rot // 2)) / max(1, rot // 2)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    rope = cai.Rope(dev(cos), dev(sin), inter) if rot else None
    cls, bytes_ = (cai.KV4Pool, kv4.page_bytes4(page)) if four else (cai.KVPool, oracle.page_bytes(page))
    pools = [cls(num_pages, page, pages=torch.full((num_pages * bytes_,), 0xA5, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
    err = flag()
    qo = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device=DEV) if hq else None
    f = cai.cai_kv4_append if four else cai.cai_kv_append_rope
    kw = dict(rope=rope, err_flag=err)
    if packed:
        kw.update(q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()))
        if hq:
            kw.update(q=q, q_out=qo)
        f(pools, k, v, dev(table), dev(start.astype(np.int32)), **kw)
    else:
        m = int(new[0])
        sh = lambda t: t.unflatten(0, (len(new), m))  # noqa: E731
        if hq:
            kw.update(q=sh(q), q_out=sh(qo))
        f(pools, sh(k), sh(v), dev(table), dev(start.astype(np.int32)), **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    turn = (lambda x: kv4.rotate(x, pos, cos, sin, inter)) if rot else (lambda x: x)
    if hq:
        assert np.array_equal(host(qo), kv4.bf16_round(turn(host(q))))
    kr, vr = turn(host(k)), host(v)
    at = np.concatenate([[0], np.cumsum(new)])
    for j in range(hkv):
        want = np.full(num_pages * bytes_, 0xA5, np.uint8)
        for b in range(len(new)):
            s = slice(at[b], at[b + 1])
            if four:
                (kc, ks), (vc, vs) = kv4.quantize4(kr[s, j]), kv4.quantize4(vr[s, j])
                kv4.write4(want, table[b], int(start[b]), kc, ks, vc, vs, page)
            elif new[b]:
                (kc, ks), (vc, vs) = oracle.quantize_rows(kr[s, j]), oracle.quantize_rows(vr[s, j])
                oracle.pool_write(want, table[b], int(start[b]), kc, ks, vc, vs, page)
        assert np.array_equal(pools[j].pages.cpu().numpy(), want), j
    return pools, dev(table), new, start, kr, vr


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_packed(four, i):
    append_case(four, APPENDS[i], True, seed=i, slices=i % 2 == 0)


MANY = (5, 2, 16, 128, False, True, [1 if i % 40 else 230 for i in range(300)] + [0, 17], [(i * 7) % 70 for i in range(302)])


@pytest.mark.parametrize("four", [False, True])
def test_append_and_read_of_long_beside_many_single_tokens(four):
    """A batch whose longest sequence would give every other one blocks without rows."""
    pools, table, new, start, kr, vr = append_case(four, MANY, True, seed=30)
    kw = dict(q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()))
    k, v = (torch.full(kr.shape, float("nan"), device=DEV) for _ in range(2))
    (cai.cai_kv4_read if four else cai.cai_kv_read)(pools, k, v, table, dev(start.astype(np.int32)), **kw)

    def want(x):
        if four:
            return kv4.dequantize4(*kv4.quantize4(x)).astype(np.float32)
        c, s = oracle.quantize_rows(x.reshape(-1, 128))
        return (c.astype(np.float32) * s[:, None]).reshape(x.shape)

    assert np.array_equal(host(k), want(kr)) and np.array_equal(host(v), want(vr))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n", [1, 19])
def test_append_equal_counts(four, n):
    append_case(four, (2, 4, 32, 64, False, True, [n] * 3, [0, 31, 40]), False, seed=7)


def test_append_without_rotation_is_the_plain_append():
    rng = np.random.default_rng(5)
    k, v = (dev(rng.normal(size=(3, 21, 1, 128)).astype(np.float32)) for _ in range(2))
    table, pages = tables(rng, [30, 40, 50], 16)
    start = dev(np.array([9, 19, 29], np.int32))
    a, b = (cai.KVPool(pages, 16, pages=torch.zeros(pages * 4224, dtype=torch.uint8, device=DEV)) for _ in range(2))
    cai.cai_kv_append(a, k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), dev(table), start)
    cai.cai_kv_append_rope([b], k, v, dev(table), start)
    assert torch.equal(a.pages, b.pages)


@pytest.mark.parametrize("four", [False, True])
def test_append_bad_tokens_are_left_out(four):
    """Positions past the table or the rotation, pages past the pool, offsets out of order: flagged, nothing else written."""
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    f = cai.cai_kv4_append if four else cai.cai_kv_append_rope
    rope = cai.Rope(torch.ones(40, 64, device=DEV), torch.zeros(40, 64, device=DEV))

    def run(start, table, bits, offsets=(0, 2, 4), rope=rope, n=2):
        pool = cls(4, 16, pages=torch.full((4 * bytes_,), 7, dtype=torch.uint8, device=DEV))
        x = torch.ones(4, 1, 128, device=DEV)
        err = flag()
        f([pool], x, x, dev(np.array(table, np.int32)), dev(np.array(start, np.int32)), rope=rope,
          q_offsets=dev(np.array(offsets, np.int32)), max_new=n, err_flag=err)
        assert err.item() == bits
        return (pool.pages.view(4, -1) != 7).any(1).tolist()

    assert run([0, 16], [[0, -1, -1], [-1, 3, -1]], 0) == [True, False, False, True]
    assert run([0, 47], [[0, 1, 2], [0, 1, 3]], cai.CAI_DEVERR_LENGTH) == [True, False, False, False]  # 48 is past the table, 47 past the rotation
    assert run([0, 47], [[0, 1, 2], [0, 1, 3]], cai.CAI_DEVERR_LENGTH, rope=None) == [True, False, False, True]
    assert run([-1, 16], [[0, 1, 2], [1, 1, 2]], cai.CAI_DEVERR_LENGTH) == [True, True, False, False]
    assert run([2147483647, 16], [[0, 1, 2], [1, 1, 2]], cai.CAI_DEVERR_LENGTH) == [False, True, False, False]
    assert run([0, 0], [[4, 1, 2], [1, 1, 2]], cai.CAI_DEVERR_PAGE) == [False, True, False, False]
    assert run([0, 0], [[-1, 1, 2], [1, 1, 2]], cai.CAI_DEVERR_PAGE) == [False, True, False, False]
    for off in ((0, 3, 4), (2, 0, 4), (-1, 1, 3), (0, 2, 5)):
        got = run([0, 16], [[0, 1, 2], [0, 1, 2]], cai.CAI_DEVERR_LENGTH, offsets=off)
        assert not (got[2] or got[3]) and sum(got) <= 1


def test_append_query_in_place_and_outlier_rows():
    """q_out may be q; rows with zeros, infinities' neighbours and huge values quantize as the oracle says."""
    x = np.zeros((6, 1, 128), np.float32)
    x[1] = 1e30
    x[2, 0, ::2] = 65504
    x[3, 0, 5] = 1e-38
    x[4] = np.linspace(-1e-6, 1e-6, 128)
    x[5] = np.linspace(-3e4, 6e4, 128)
    table = np.array([[1]], np.int32)
    pool = cai.KV4Pool(2, 16, pages=torch.zeros(2 * 2304, dtype=torch.uint8, device=DEV))
    cos, sin = torch.rand(20, 64, device=DEV), torch.rand(20, 64, device=DEV)
    q = torch.randn(1, 6, 4, 128, device=DEV, dtype=torch.bfloat16)
    want = kv4.bf16_round(kv4.rotate(host(q)[0], np.arange(6), cos.cpu().numpy(), sin.cpu().numpy(), False))
    one = cai.Rope(torch.ones(20, 1, device=DEV), torch.zeros(20, 1, device=DEV))
    cai.cai_kv4_append([pool], dev(x)[None], dev(x)[None], dev(table), torch.zeros(1, dtype=torch.int32, device=DEV),
                       rope=cai.Rope(cos, sin), q=q, q_out=q)
    cai.cai_kv4_append([pool], dev(x)[None], dev(x)[None], dev(table), torch.zeros(1, dtype=torch.int32, device=DEV), rope=one)
    assert np.array_equal(host(q)[0], want)
    ref = kv4.pool4(2, 16, 0)
    kv4.write4(ref, table[0], 0, *kv4.quantize4(x[:, 0]), *kv4.quantize4(x[:, 0]), 16)
    assert np.array_equal(pool.pages.cpu().numpy(), ref)


# -------------------------------------------------------------------------------------- read

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("i", [1, 2, 5])
def test_read_gives_back_what_the_cache_stands_for(four, i):
    pools, table, new, start, kr, vr = append_case(four, APPENDS[i], True, seed=20 + i)
    n, hkv = kr.shape[0], kr.shape[1]
    read = cai.cai_kv4_read if four else cai.cai_kv_read
    kw = dict(q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()))

    def want(x):
        if four:
            return kv4.dequantize4(*kv4.quantize4(x)).astype(np.float32)
        c, s = oracle.quantize_rows(x.reshape(-1, 128))
        return (c.astype(np.float32) * s[:, None]).reshape(x.shape)

    for dt in (torch.float32, torch.bfloat16):
        k, v = (torch.full((n, hkv, 128), float("nan"), dtype=dt, device=DEV) for _ in range(2))
        read(pools, k, v, table, dev(start.astype(np.int32)), **kw)
        as_dt = kv4.bf16_round if dt == torch.bfloat16 else (lambda x: x)
        assert np.array_equal(host(k), as_dt(want(kr))) and np.array_equal(host(v), as_dt(want(vr)))
        only = torch.full_like(v, float("nan"))
        read(pools, None, only, table, dev(start.astype(np.int32)), **kw)
        assert torch.equal(only, v)


def test_read_into_outputs_of_odd_alignment():
    """16-byte aligned outputs, not 32: the same values, and nothing around them."""
    pools, table, new, start, kr, _ = append_case(True, APPENDS[1], True, seed=3)
    kw = dict(q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()))
    n = kr.shape[0] * kr.shape[1] * 128
    for dt, pad in ((torch.float32, 4), (torch.bfloat16, 8)):
        room = torch.full((n + 2 * pad,), 9.0, dtype=dt, device=DEV)
        k = room[pad:-pad].view(kr.shape)
        cai.cai_kv4_read(pools, k, None, table, dev(start.astype(np.int32)), **kw)
        want = kv4.dequantize4(*kv4.quantize4(kr)).astype(np.float32)
        assert np.array_equal(host(k), want if dt == torch.float32 else kv4.bf16_round(want))
        assert (room[:pad] == 9).all() and (room[-pad:] == 9).all()


@pytest.mark.parametrize("four", [False, True])
def test_read_bad_rows_are_zero(four):
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    pool = cls(2, 16, pages=torch.full((2 * bytes_,), 0x31, dtype=torch.uint8, device=DEV))
    read = cai.cai_kv4_read if four else cai.cai_kv_read
    for table, start, bits, zero in (([[1, 5]], [14], cai.CAI_DEVERR_PAGE, [0, 0, 1, 1]), ([[1, 0]], [30], cai.CAI_DEVERR_LENGTH, [0, 0, 1, 1]),
                                     ([[1, 0]], [-2], cai.CAI_DEVERR_LENGTH, [1, 1, 0, 0])):
        k = torch.full((1, 4, 1, 128), 9.0, device=DEV)
        err = flag()
        read([pool], k, None, dev(np.array(table, np.int32)), dev(np.array(start, np.int32)), err_flag=err)
        assert err.item() == bits
        assert [bool((k[0, i] == 0).all()) for i in range(4)] == [bool(z) for z in zero]


# ------------------------------------------------------------------------------------ decode

def decode(cache, q, ctx, window=0, splits=0, err=None, ws=None):
    b, hq = q.shape[0], q.shape[1]
    n = cai.cai_kv4_decode_workspace_size(b, hq, cache.hkv, cache.table.shape[1], cache.page, window, splits)
    if ws is None:
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)  # no preparation is needed
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b, hq), float("nan"), device=DEV)
    cai.cai_kv4_decode(cache.pools, q, cache.table, dev(np.array(ctx, np.int32)), window, SCALE, splits, ws if n else None, out,
                       lse, err)
    return out, lse


def check_decode(cache, q, ctx, window=0, splits=0):
    err = flag()
    out, lse = decode(cache, q, ctx, window, splits, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    o, l, x = host(out), host(lse), host(q)
    for b, n in enumerate(ctx):
        cache.check(o[b:b + 1], l[b:b + 1], x[b:b + 1], b, n - 1, window, (b, n, window, splits))


LENGTHS = [1, 16, 17, 31, 32, 33, 0, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("hkv,hq", [(1, 1), (1, 8), (1, 12), (2, 32), (1, 24), (1, 32), (8, 8), (1, 40), (1, 64), (1, 128), (3, 15)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_heads(hkv, hq, page):
    cache = Cache(LENGTHS, hkv, page, seed=hq)
    check_decode(cache, queries(np.random.default_rng(hq), len(LENGTHS), hq), LENGTHS)


@pytest.mark.parametrize("window", [1, 15, 16, 100, 128, 333, 1000, 5000])
def test_decode_windows(window):
    cache = Cache(LENGTHS, 2, 32, seed=window)
    for hq in (8, 64):
        q = queries(np.random.default_rng(window), len(LENGTHS), hq, 2.0)
        check_decode(cache, q, LENGTHS, window)
        check_decode(cache, q, LENGTHS, window, 3)


@pytest.mark.parametrize("splits", [1, 2, 5, 64])
def test_decode_splits(splits):
    lengths = [3000, 1, 0, 1500, 129]
    cache = Cache(lengths, 1, 16, seed=splits)
    for hq in (4, 16, 48):
        check_decode(cache, queries(np.random.default_rng(hq), 5, hq), lengths, 0, splits)


def test_decode_shorter_than_written_and_unused_table():
    """ctx_len below what the pages hold; the table wider than any sequence needs."""
    cache = Cache([500, 400], 1, 32, width=200)
    for ctx in ([333, 17], [0, 0], [500, 1]):
        check_decode(cache, queries(np.random.default_rng(1), 2, 8), ctx)


@pytest.mark.parametrize("size", [8.0, 30.0])
def test_decode_sharp_logits(size):
    """Logits spread over tens of units: the references rise many times and most weights vanish."""
    lengths = [700, 2500]
    cache = Cache(lengths, 2, 64, seed=3)
    for hq in (8, 32, 64):
        check_decode(cache, queries(np.random.default_rng(hq), 2, hq, size), lengths)
        check_decode(cache, queries(np.random.default_rng(hq), 2, hq, size), lengths, 0, 4)


@pytest.mark.parametrize("v_size", [1e-3, 300.0, 9000.0])
def test_decode_value_sizes(v_size):
    lengths = [200, 900]
    cache = Cache(lengths, 1, 16, seed=4, v_size=v_size)
    check_decode(cache, queries(np.random.default_rng(0), 2, 32), lengths)


def test_decode_many_short_sequences():
    """More sequences than blocks, and more of them in a block than it lists at a time."""
    rng = np.random.default_rng(9)
    lengths = rng.integers(0, 40, 700)
    small = Cache(lengths[:40], 1, 16, seed=9)
    b = 9000  # every sequence reads one of 40 stored ones
    which = rng.integers(0, 40, b)
    ctx = np.array([small.lengths[w] for w in which], np.int32)
    q = queries(rng, b, 8)
    table = small.table[torch.from_numpy(which).to(DEV)].contiguous()
    ws = torch.empty(cai.cai_kv4_decode_workspace_size(b, 8, 1, table.shape[1], 16, 0), dtype=torch.uint8, device=DEV)
    out = torch.empty(b, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(b, 8, device=DEV)
    cai.cai_kv4_decode(small.pools, q, table, dev(ctx), 0, SCALE, 0, ws, out, lse)
    o, l, x = host(out), host(lse), host(q)
    for i in list(range(50)) + list(range(b - 50, b)) + list(rng.integers(0, b, 100)):
        small.check(o[i:i + 1], l[i:i + 1], x[i:i + 1], which[i], int(ctx[i]) - 1, 0, i)


@pytest.mark.parametrize("hq", [8, 16, 32, 64])
@pytest.mark.parametrize("width", [3, 40])
def test_decode_many_short_sequences_cut_or_whole(hq, width):
    """The same in both splits: tables of up to 512 tokens (no sequence is cut) and longer ones, and every kernel."""
    rng = np.random.default_rng(width)
    small = Cache(rng.integers(0, 45, 30), 1, 16, seed=10, width=width)
    b = 9000 if hq == 8 and width == 40 else 5200
    which = rng.integers(0, 30, b)
    ctx = np.array([small.lengths[w] for w in which], np.int32)
    q = queries(rng, b, hq)
    table = small.table[torch.from_numpy(which).to(DEV)].contiguous()
    ws = torch.empty(max(1, cai.cai_kv4_decode_workspace_size(b, hq, 1, width, 16, 0)), dtype=torch.uint8, device=DEV)
    out = torch.empty(b, hq, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(b, hq, device=DEV)
    cai.cai_kv4_decode(small.pools, q, table, dev(ctx), 0, SCALE, 0, ws, out, lse)
    for i in list(range(30)) + list(range(b - 30, b)) + list(rng.integers(0, b, 60)):
        small.check(host(out[i:i + 1]), host(lse[i:i + 1]), host(q[i:i + 1]), which[i], int(ctx[i]) - 1, 0, i)


@pytest.mark.parametrize("hq", [8, 32])
def test_decode_an_infinite_head_spoils_no_other(hq):
    """A head whose logits are all infinite or NaN leaves its neighbours alone."""
    cache = Cache([700], 1, 16, seed=11)
    q = queries(np.random.default_rng(11), 1, hq)
    want, wl = decode(cache, q, [700])
    q2 = q.clone()
    q2[0, 0] = -float("inf")
    q2[0, 5] = float("nan")
    out, lse = decode(cache, q2, [700])
    rest = [h for h in range(hq) if h not in (0, 5)]
    assert torch.equal(out[0, rest], want[0, rest]) and torch.equal(lse[0, rest], wl[0, rest])


def test_decode_bad_lengths_and_pages():
    cache = Cache([100, 200, 300], 2, 16, seed=2)
    q = queries(np.random.default_rng(2), 3, 16)
    good, good_lse = decode(cache, q, [100, 200, 300])
    for ctx, bad in (([100, -1, 300], 1), ([100, 200, 305], 2)):
        err = flag()
        out, lse = decode(cache, q, ctx, err=err)
        torch.cuda.synchronize()
        assert err.item() == cai.CAI_DEVERR_LENGTH
        assert (out[bad] == 0).all() and (lse[bad] == -float("inf")).all()
        for b in range(3):
            if b != bad:
                assert (out[b].float() - good[b].float()).abs().max() <= 2.0 ** -6
    for page in (-1, cache.num_pages, 2147483647):
        table = cache.table.clone()
        table[1, 3] = page
        err = flag()
        out, lse, keep = torch.zeros_like(q), torch.zeros(3, 16, device=DEV), cache.table
        cache.table = table
        out, lse = decode(cache, q, [100, 200, 300], err=err)
        cache.table = keep
        torch.cuda.synchronize()
        assert err.item() == cai.CAI_DEVERR_PAGE
        assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[2].float()).all()
        assert torch.isfinite(out[1].float()).all()  # that page's keys are left out


def test_decode_pages_past_two_gigabytes():
    """Byte offsets past 32 bits: the sequence's pages lie at the end of a 5 GB pool."""
    small = Cache([450], 1, 64, seed=6)
    pages = 5_000_000_000 // 9216
    big = torch.empty(pages * 9216, dtype=torch.uint8, device=DEV)
    n = small.num_pages
    big.view(pages, -1)[-n:] = small.pools[0].pages.view(n, -1)
    small.pools = [cai.KV4Pool(pages, 64, pages=big)]
    small.table = torch.where(small.table >= 0, small.table + (pages - n), small.table)
    check_decode(small, queries(np.random.default_rng(6), 1, 8), [450])
    k = torch.empty(1, 450, 1, 128, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    cai.cai_kv4_read(small.pools, k, None, small.table, zero)
    assert np.array_equal(host(k)[0, :, 0], small.k[0][0].astype(np.float32))
    x = torch.randn(1, 450, 1, 128, device=DEV)
    cai.cai_kv4_append(small.pools, x, x, small.table, zero)
    cai.cai_kv4_read(small.pools, k, None, small.table, zero)
    assert np.array_equal(host(k)[0, :, 0], kv4.dequantize4(*kv4.quantize4(host(x)[0, :, 0])).astype(np.float32))


def test_decode_is_the_same_every_time():
    """No order of arrival shows in the result."""
    cache = Cache([900, 20, 3000], 2, 32, seed=8)
    q = queries(np.random.default_rng(8), 3, 64)
    first = decode(cache, q, [900, 20, 3000])
    for _ in range(5):
        again = decode(cache, q, [900, 20, 3000])
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_graphs_and_streams():
    """Two captured graphs that share a workspace, replayed in turn; and a call on another stream."""
    cache = Cache([500, 900], 1, 16, seed=5)
    rng = np.random.default_rng(5)
    qs = [queries(rng, 2, 32) for _ in range(2)]
    ctx = dev(np.array([500, 900], np.int32))
    ws = torch.empty(cai.cai_kv4_decode_workspace_size(2, 32, 1, cache.table.shape[1], 16, 0), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(2, 32, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lses = [torch.zeros(2, 32, device=DEV) for _ in range(2)]
    call = lambda i, **kw: cai.cai_kv4_decode(cache.pools, qs[i], cache.table, ctx, 0, SCALE, 0, ws, outs[i], lses[i], **kw)  # noqa: E731
    call(0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            outs[i].zero_()
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for b, n in enumerate([500, 900]):
            cache.check(host(outs[i])[b:b + 1], host(lses[i])[b:b + 1], host(qs[i])[b:b + 1], b, n - 1, 0, (i, b))
    want = outs[0].clone()
    side = torch.cuda.Stream()
    outs[0].zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(0, stream=side)
    side.synchronize()
    assert torch.equal(outs[0], want)


@pytest.mark.parametrize("hq", [8, 16, 32, 64])
def test_decode_gives_up_then_recovers(hq):
    """A load that never comes: the launch reports the timeout and ends, and the next call is right."""
    lengths = [2000, 5000]
    cache = Cache(lengths, 1, 16, seed=1)
    q = queries(np.random.default_rng(1), 2, hq)
    cai.cai_set_wait_limit_ns(20_000_000)
    cai.cai_set_fault_injection(1)
    try:
        err = flag()
        decode(cache, q, lengths, splits=2, err=err)
        torch.cuda.synchronize()
        assert err.item() == cai.CAI_DEVERR_TIMEOUT
    finally:
        cai.cai_set_fault_injection(-1)
        cai.cai_set_wait_limit_ns(0)
    check_decode(cache, q, lengths)


# ----------------------------------------------------------------------------------- prefill

def check_prefill(cache, q, prefix, new, window=0, packed=True, max_new=None):
    hq = q.shape[1]
    err = flag()
    ws = torch.full((cai.cai_kv4_prefill_workspace_size(len(new), hq, cache.hkv, cache.table.shape[1], cache.page),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    pre = dev(np.array(prefix, np.int32))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    if packed:
        cai.cai_kv4_prefill(cache.pools, q, cache.table, pre, window, SCALE, ws, out, lse, err, q_offsets=dev(off),
                            max_new=max_new or max(new))
    else:
        sh = lambda t: t.unflatten(0, (len(new), new[0]))  # noqa: E731
        cai.cai_kv4_prefill(cache.pools, sh(q), cache.table, pre, window, SCALE, ws, sh(out), sh(lse), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    o, l, x = host(out), host(lse), host(q)
    for b, n in enumerate(new):
        s = slice(off[b], off[b + 1])
        if n:
            cache.check(o[s], l[s], x[s], b, prefix[b], window, (b, n, window))


@pytest.mark.parametrize("hkv,hq", [(1, 1), (1, 32), (2, 8), (4, 64), (8, 8), (1, 128)])
@pytest.mark.parametrize("window", [0, 70])
def test_prefill_packed(hkv, hq, window):
    prefix, new = [0, 300, 17, 5, 129, 1000, 64], [40, 1, 0, 130, 3, 1, 2]
    cache = Cache([a + n for a, n in zip(prefix, new)], hkv, 32, seed=hq)
    check_prefill(cache, queries(np.random.default_rng(hq), sum(new), hq), prefix, new, window)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n", [1, 37])
def test_prefill_equal_counts(page, n):
    prefix = [0, 111, 640]
    cache = Cache([a + n for a in prefix], 2, page, seed=n)
    q = queries(np.random.default_rng(n), 3 * n, 16, 2.0)
    check_prefill(cache, q, prefix, [n] * 3, 0, packed=False)
    check_prefill(cache, q, prefix, [n] * 3, 200, packed=False)


def test_prefill_split_last_wave():
    """Few q-tiles over long prefixes: key ranges of a q-tile are merged."""
    cache = Cache([3000, 2100], 1, 64, seed=12)
    check_prefill(cache, queries(np.random.default_rng(12), 200, 32), [2900, 2000], [100, 100], 0, packed=False)


def test_prefill_single_rows_alone_and_decode_agree():
    lengths = [77, 500, 1, 2000]
    cache = Cache(lengths, 2, 16, seed=13)
    q = queries(np.random.default_rng(13), 4, 32)
    check_prefill(cache, q, [n - 1 for n in lengths], [1] * 4, max_new=9)


def test_prefill_of_one_token_each_is_a_decode_step():
    """Without offsets, too: the same rows, flags and edges as through the decode call."""
    lengths = [77, 500, 1, 2000]
    cache = Cache(lengths, 2, 16, seed=19)
    q = queries(np.random.default_rng(19), 4, 32)
    want = decode(cache, q, lengths)
    ws = torch.full((cai.cai_kv4_prefill_workspace_size(4, 32, 2, cache.table.shape[1], 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def run(prefix):
        out = torch.full((4, 1, 32, 128), 5.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((4, 1, 32), 5.0, device=DEV)
        err = flag()
        cai.cai_kv4_prefill(cache.pools, q[:, None], cache.table, dev(np.array(prefix, np.int32)), 0, SCALE, ws, out, lse, err)
        return out[:, 0], lse[:, 0], int(err.item())

    out, lse, err = run([n - 1 for n in lengths])
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out, lse, err = run([76, -1, 0, cache.table.shape[1] * 16])
    assert err == cai.CAI_DEVERR_LENGTH
    for b in (1, 3):
        assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
    for b in (0, 2):
        assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])


def test_prefill_more_items_than_a_block_lists():
    """Past 4096 q-tiles a packed call numbers them densely."""
    rng = np.random.default_rng(16)
    one = Cache([200, 180], 8, 16, seed=16)
    b, n, hq = 64, 130, 64  # 64 sequences of 9 q-tiles for each of 8 K/V heads, over two stored ones
    which = [i % 2 for i in range(b)]
    table = one.table[torch.tensor(which, device=DEV)].contiguous()
    new = [n] * b
    new[3], new[7] = 1, 0
    prefix = [one.lengths[w] - k for w, k in zip(which, new)]
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = queries(rng, int(off[-1]), hq)
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(b, hq, 8, table.shape[1], 16), dtype=torch.uint8, device=DEV)
    out, lse, err = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV), flag()
    cai.cai_kv4_prefill(one.pools, q, table, dev(np.array(prefix, np.int32)), 0, SCALE, ws, out, lse, err, q_offsets=dev(off), max_new=n)
    assert err.item() == 0
    for i in (0, 1, 3, 30, 62, 63):
        s = slice(off[i], off[i + 1])
        one.check(host(out[s]), host(lse[s]), host(q[s]), which[i], prefix[i], 0, i)


def test_attention_into_outputs_of_odd_alignment():
    """Outputs that start 16 bytes into a sector; rows behind the last sequence stay as they were."""
    cache = Cache([300, 33], 1, 16, seed=17)
    rng = np.random.default_rng(17)
    prefix, new, rows = [150, 13], [150, 20], 180
    q = queries(rng, rows, 16)
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(2, 16, 1, cache.table.shape[1], 16), dtype=torch.uint8, device=DEV)
    room = torch.full((rows * 16 * 128 + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    lroom = torch.full((rows * 16 + 1,), 7.0, device=DEV)
    out, lse = room[8:8 + rows * 16 * 128].view(rows, 16, 128), lroom[1:].view(rows, 16)
    cai.cai_kv4_prefill(cache.pools, q, cache.table, dev(np.array(prefix, np.int32)), 0, SCALE, ws, out, lse,
                        q_offsets=dev(np.array([0, 150, 170], np.int32)), max_new=150)
    for b, s in enumerate((slice(0, 150), slice(150, 170))):
        cache.check(host(out[s]), host(lse[s]), host(q[s]), b, prefix[b], 0, b)
    assert (room[:8] == 7).all() and (room[8 + 170 * 16 * 128:] == 7).all() and (lroom[1 + 170 * 16:] == 7).all() and lroom[0] == 7
    for hq in (8, 32):
        q = queries(rng, 2, hq)
        room = torch.full((2 * hq * 128 + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
        out, lse = room[8:8 + 2 * hq * 128].view(2, hq, 128), torch.empty(2, hq, device=DEV)
        ws = torch.empty(max(1, cai.cai_kv4_decode_workspace_size(2, hq, 1, cache.table.shape[1], 16, 0)), dtype=torch.uint8, device=DEV)
        cai.cai_kv4_decode(cache.pools, q, cache.table, dev(np.array([300, 33], np.int32)), 0, SCALE, 0, ws, out, lse)
        for b, n in enumerate((300, 33)):
            cache.check(host(out[b:b + 1]), host(lse[b:b + 1]), host(q[b:b + 1]), b, n - 1, 0, (hq, b))
        assert (room[:8] == 7).all() and (room[-8:] == 7).all()


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The launch goes to the current device: with another one current, nothing is launched."""
    cache = Cache([20], 1, 16, seed=18)
    q = queries(np.random.default_rng(18), 1, 8)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.zeros(1, 1, 1, 128, device=DEV)
    before = cache.pools[0].pages.clone()
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(1, 8, 1, cache.table.shape[1], 16), dtype=torch.uint8, device=DEV)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: decode(cache, q, [20]), lambda: cai.cai_kv4_append(cache.pools, x, x, cache.table, zero),
                 lambda: cai.cai_kv4_read(cache.pools, x, None, cache.table, zero),
                 lambda: cai.cai_kv4_prefill(cache.pools, q[None], cache.table, zero, 0, SCALE, ws, torch.empty_like(q)[None])):
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert torch.equal(cache.pools[0].pages, before)


def test_prefill_bad_sequences():
    """Lengths past the table and offsets out of order: flagged, zero or untouched rows, the others right."""
    prefix, new = [10, 20, 30], [5, 1, 6]
    cache = Cache([a + n for a, n in zip(prefix, new)], 2, 16, seed=14)
    q = queries(np.random.default_rng(14), 12, 8)
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(3, 8, 2, cache.table.shape[1], 16), dtype=torch.uint8, device=DEV)

    def run(prefix, off):
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((12, 8), 5.0, device=DEV)
        err = flag()
        cai.cai_kv4_prefill(cache.pools, q, cache.table, dev(np.array(prefix, np.int32)), 0, SCALE, ws, out, lse, err,
                            q_offsets=dev(np.array(off, np.int32)), max_new=6)
        return host(out), host(lse), int(err.item())

    o, l, e = run([10, 1 << 20, 30], [0, 5, 6, 12])
    assert e == cai.CAI_DEVERR_LENGTH and (o[5] == 0).all() and (l[5] == -np.inf).all()
    cache.check(o[:5], l[:5], host(q)[:5], 0, 10, 0, "0")
    cache.check(o[6:], l[6:], host(q)[6:], 2, 30, 0, "2")
    o, l, e = run([-3, 20, 30], [0, 5, 6, 12])
    assert e == cai.CAI_DEVERR_LENGTH and (o[:5] == 0).all() and (l[:5] == -np.inf).all()
    o, l, e = run(prefix, [0, 5, 4, 12])
    assert e == cai.CAI_DEVERR_LENGTH
    cache.check(o[:4], l[:4], host(q)[:4], 0, 10, 0, "0")


def test_prefill_items_longer_than_the_wait_limit():
    """The limit is one of waits for a step, not for a work item: 900 items of 260 thousand keys under 0.3 ms."""
    n, prefix = 900, 260000
    pages = -(-(prefix + n) // 64)
    pool = cai.KV4Pool(pages, 64)
    table = torch.randperm(pages, device=DEV).to(torch.int32)[None].contiguous()
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.randn(1, prefix + n, 1, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    cai.cai_kv4_append([pool], x, x.flip(1), table, zero)
    q = torch.randn(1, n, 128, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(1, 128, 1, pages, 64), dtype=torch.uint8, device=DEV)
    at = zero + prefix
    outs = []
    for limit in (0, 300_000):
        cai.cai_set_wait_limit_ns(limit)
        try:
            err, out = flag(), torch.empty_like(q)
            cai.cai_kv4_prefill([pool], q, table, at, 0, SCALE, ws, out, None, err)
            torch.cuda.synchronize()
            assert err.item() == 0
            outs.append(out)
        finally:
            cai.cai_set_wait_limit_ns(0)
    assert torch.equal(outs[0], outs[1])


def test_prefill_gives_up_then_recovers():
    prefix, new = [900, 1500, 2000], [64, 1, 100]
    cache = Cache([a + n for a, n in zip(prefix, new)], 1, 16, seed=15)
    q = queries(np.random.default_rng(15), sum(new), 32)
    ws = torch.empty(cai.cai_kv4_prefill_workspace_size(3, 32, 1, cache.table.shape[1], 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    cai.cai_set_wait_limit_ns(20_000_000)
    cai.cai_set_fault_injection(1)
    try:
        err = flag()
        cai.cai_kv4_prefill(cache.pools, q, cache.table, dev(np.array(prefix, np.int32)), 0, SCALE, ws, out, None, err,
                            q_offsets=dev(np.array([0, 64, 65, 165], np.int32)), max_new=100)
        torch.cuda.synchronize()
        assert err.item() == cai.CAI_DEVERR_TIMEOUT
    finally:
        cai.cai_set_fault_injection(-1)
        cai.cai_set_wait_limit_ns(0)
    check_prefill(cache, q, prefix, new)


# ---------------------------------------------------------------------------------- together

def test_a_dialogue_through_all_of_them():
    """Prefill a prompt, decode three tokens, rotated, with both caches' appends, moving a dialogue from the int8
    cache to the 4-bit one by reading it back; every step captured into one graph and replayed."""
    rng = np.random.default_rng(42)
    hkv, hq, page, prompt, steps = 2, 16, 16, 45, 3
    g = hq // hkv
    total = prompt + steps
    table_np, pages = tables(rng, [total], page)
    table = dev(table_np)
    ang = np.arange(total)[:, None] * (1e4 ** (-np.arange(64) / 64))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    rope = cai.Rope(dev(cos), dev(sin))
    qkv = dev(rng.normal(size=(total, hq + 2 * hkv, 128)).astype(np.float32), torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pool8 = [cai.KVPool(pages, page, pages=torch.zeros(pages * 4224, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
    pool4 = [cai.KV4Pool(pages, page, pages=torch.zeros(pages * 2304, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
    at = [torch.full((1,), i, dtype=torch.int32, device=DEV) for i in range(total + 1)]
    qr = torch.empty(total, hq, 128, dtype=torch.bfloat16, device=DEV)
    kk, vv = (torch.empty(1, prompt, hkv, 128, device=DEV) for _ in range(2))
    out = torch.zeros(total, hq, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(total, hq, device=DEV)
    err = flag()
    ws_p = torch.empty(cai.cai_kv4_prefill_workspace_size(1, hq, hkv, table.shape[1], page), dtype=torch.uint8, device=DEV)
    ws_d = torch.empty(cai.cai_kv4_decode_workspace_size(1, hq, hkv, table.shape[1], page, 0), dtype=torch.uint8, device=DEV)

    def dialogue():
        cai.cai_kv_append_rope(pool8, k[None, :prompt], v[None, :prompt], table, at[0], rope=rope, q=q[None, :prompt],
                               q_out=qr[None, :prompt], err_flag=err)
        cai.cai_kv_read(pool8, kk, vv, table, at[0], err_flag=err)
        cai.cai_kv4_append(pool4, kk, vv, table, at[0], err_flag=err)  # rotated already
        cai.cai_kv4_prefill(pool4, qr[None, :prompt], table, at[0], 0, SCALE, ws_p, out[None, :prompt], lse[None, :prompt], err)
        for i in range(prompt, total):
            cai.cai_kv4_append(pool4, k[i:i + 1, None], v[i:i + 1, None], table, at[i], rope=rope, q=q[i:i + 1, None],
                               q_out=qr[i:i + 1, None], err_flag=err)
            cai.cai_kv4_decode(pool4, qr[i:i + 1], table, at[i + 1], 0, SCALE, 0, ws_d, out[i:i + 1], lse[i:i + 1], err)

    dialogue()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dialogue()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, first)
    pos = np.arange(total)
    kr = kv4.rotate(host(k), pos, cos, sin, False)
    vals = []
    for x in (kr, host(v)):
        c, s = oracle.quantize_rows(x[:prompt].reshape(-1, 128))
        x = x.copy()
        x[:prompt] = (c.astype(np.float32) * s[:, None]).reshape(prompt, hkv, 128)
        vals.append(kv4.dequantize4(*kv4.quantize4(x)))
    cache = Cache([0], hkv, page)
    cache.k = [[vals[0][:, j]] for j in range(hkv)]
    cache.v = [[vals[1][:, j]] for j in range(hkv)]
    cache.check(host(out), host(lse), kv4.bf16_round(kv4.rotate(host(q), pos, cos, sin, False)), 0, 0, 0, "dialogue")
    assert g * hkv == hq
