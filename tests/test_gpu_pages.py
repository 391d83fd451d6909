"""Page summaries, the selection of pages and attention over lists of pages, against the oracle.

Summaries and selections are exact: whole numbers, minima, maxima and single fp32 operations."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
import oracle  # noqa: E402
from oracle import kv4, pages  # noqa: E402
from test_gpu_kv4 import DEV, SCALE, _built, dev, flag, host, tables  # noqa: E402,F401


class Dialogues:
    """hkv pools, int8 or 4-bit, with the keys and values of every sequence, all other bytes 0xFF; host values kept."""

    def __init__(self, four, lengths, hkv, page, seed=0, width=0, size=None, fill=0xFF):
        rng = np.random.default_rng(seed)
        self.four, self.lengths, self.page, self.hkv = four, list(lengths), page, hkv
        self.table_np, self.num_pages = tables(rng, lengths, page, width=width)
        self.table = dev(self.table_np)
        bytes_ = kv4.page_bytes4(page) if four else oracle.page_bytes(page)
        cls = cai.KV4Pool if four else cai.KVPool
        self.pools = [cls(self.num_pages, page, pages=torch.full((self.num_pages * bytes_,), fill, dtype=torch.uint8, device=DEV))
                      for _ in range(hkv)]
        self.k, self.v = [[] for _ in range(hkv)], [[] for _ in range(hkv)]
        for b, n in enumerate(lengths):
            x = rng.normal(size=(2, n, hkv, 128)).astype(np.float32)
            x[0, ..., rng.integers(0, 128, 3)] *= 4
            if size is not None:
                x *= size(b, n)[None, :, None, None]
            for j in range(hkv):
                self.k[j].append(self.stored(x[0, :, j]))
                self.v[j].append(self.stored(x[1, :, j]))
            if n:
                append = cai.cai_kv4_append if four else cai.cai_kv_append_rope
                append(self.pools, dev(x[0])[None], dev(x[1])[None], self.table[b:b + 1], torch.zeros(1, dtype=torch.int32, device=DEV))

    def stored(self, x):
        """The fp32 values that cached x stands for."""
        if self.four:
            return kv4.dequantize4(*kv4.quantize4(x)).astype(np.float32)
        c, s = oracle.quantize_rows(np.ascontiguousarray(x)) if len(x) else (np.zeros(x.shape, np.int8), np.zeros(0, np.float32))
        return c.astype(np.float32) * s[:, None]

    def summaries(self, fill=0x5A):
        return [cai.KVSummary(self.num_pages, self.page, data=torch.full((self.num_pages * 260,), fill, dtype=torch.uint8, device=DEV))
                for _ in range(self.hkv)]

    def summarize(self, sums, start, n_new, offsets=None, err=None):
        f = cai.cai_kv4_summarize if self.four else cai.cai_kv_summarize
        f(self.pools, sums, self.table, dev(np.array(start, np.int32)), n_new,
          q_offsets=None if offsets is None else dev(np.array(offsets, np.int32)), err_flag=err)

    def want(self, start, new, fill=0x5A):
        """The summaries' bytes after a call on untouched buffers."""
        out = []
        for j in range(self.hkv):
            raw = np.full(self.num_pages * 260, fill, np.uint8)
            codes, scale = raw[:self.num_pages * 256].view(np.int8).reshape(-1, 256), raw[self.num_pages * 256:].view(np.float32)
            for b, (s, n) in enumerate(zip(start, new)):
                for i in range(s // self.page, -(-(s + n) // self.page) if n else 0):
                    codes[self.table_np[b, i]], scale[self.table_np[b, i]] = pages.summarize(
                        self.k[j][b][i * self.page:min((i + 1) * self.page, s + n)])
            out.append(raw)
        return out

    def full_summaries(self):
        sums = self.summaries()
        self.summarize(sums, [0] * len(self.lengths), max(self.lengths), np.concatenate([[0], np.cumsum(self.lengths)]))
        return sums


def same(sums, want):
    for s, w in zip(sums, want):
        assert np.array_equal(s.data.cpu().numpy(), w)


# ----------------------------------------------------------------------------------- summaries

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hkv,page", [(1, 16), (3, 32), (8, 64)])
def test_summaries_of_new_tokens(four, hkv, page):
    """Counts of 0, 1 and more, from and to anywhere in a page; the pages' earlier tokens count, later ones do not."""
    start = [0, 5, page - 1, page, 3 * page - 1, 7, 0]
    new = [1, 0, 1, 1, 2, 4 * page + 3, 2 * page]
    d = Dialogues(four, [s + n + 5 for s, n in zip(start, new)], hkv, page, seed=hkv)  # (tokens past the count are there, too)
    sums, err = d.summaries(), flag()
    d.summarize(sums, start, max(new), np.concatenate([[0], np.cumsum(new)]), err)
    assert err.item() == 0
    same(sums, d.want(start, new))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n", [1, 16, 50])
def test_summaries_of_equal_counts(four, n):
    start = [0, 15, 16, 33, 64]
    d = Dialogues(four, [s + n for s in start], 2, 32, seed=n)
    sums, err = d.summaries(), flag()
    d.summarize(sums, start, n, err=err)
    assert err.item() == 0
    same(sums, d.want(start, [n] * 5))


@pytest.mark.parametrize("four", [False, True])
def test_summaries_of_zeros_and_of_one_sign(four):
    """Pages of zeros (scale 0), of keys of one sign, and of sizes far apart; a loose bound on the counts."""
    rng = np.random.default_rng(9)
    d = Dialogues(four, [16, 48, 40], 1, 16, seed=4, size=lambda b, n: np.zeros(n) if b == 0 else np.logspace(-3, 3, n) if b == 1 else np.ones(n))
    sums, err = d.summaries(), flag()
    d.summarize(sums, [0] * 3, 4000, [0, 16, 64, 104], err)
    assert err.item() == 0
    same(sums, d.want([0] * 3, [16, 48, 40]))
    x = np.abs(rng.normal(size=(2, 20, 1, 128)).astype(np.float32)) + 0.1
    x[1] *= -1
    table = np.array([[1, 0], [2, 3]], np.int32)
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    pool = cls(4, 16, pages=torch.full((4 * bytes_,), 0xFF, dtype=torch.uint8, device=DEV))
    start = torch.zeros(2, dtype=torch.int32, device=DEV)
    (cai.cai_kv4_append if four else cai.cai_kv_append_rope)([pool], dev(x), dev(x), dev(table), start)
    s = cai.KVSummary(4, 16)
    (cai.cai_kv4_summarize if four else cai.cai_kv_summarize)([pool], [s], dev(table), start, 20)
    got = s.data[:4 * 256].view(torch.int8).view(4, 256).cpu().numpy()
    for b in range(2):
        for i in range(2):
            code, _ = pages.summarize(d.stored(x[b, 16 * i:16 * (i + 1), 0]))
            assert np.array_equal(got[table[b, i]], code) and ((code >= 0).all() if b == 0 else (code <= 0).all())


@pytest.mark.parametrize("size", [3e-38, 1e-33, 1e-30, 1e-3, 1e3, 1e30])
def test_summaries_of_keys_of_any_size(size):
    """int8: scales on both sides of those whose quotients are computed by products; zeros beside the smallest numbers."""
    d = Dialogues(False, [100, 7], 2, 32, seed=21, size=lambda b, n: np.where(np.arange(n) % 5 == 4, 0.0, size))
    sums, err = d.summaries(), flag()
    d.summarize(sums, [0, 0], 100, [0, 100, 107], err)
    assert err.item() == 0
    same(sums, d.want([0, 0], [100, 7]))


@pytest.mark.parametrize("four", [False, True])
def test_summaries_bad_arguments_on_the_device(four):
    """Positions outside the table, page ids outside the pool, offsets out of order: flagged, other pages done."""
    d = Dialogues(four, [40, 40], 1, 16, seed=2)
    for start, table, offsets, bits, done in (
            ([30, -3], None, [0, 4, 8], cai.CAI_DEVERR_LENGTH, [(0, 30, 34), (1, 0, 1)]),       # -3 .. 0: the page of 0 is done
            ([46, 0], None, [0, 4, 8], cai.CAI_DEVERR_LENGTH, [(0, 32, 48), (1, 0, 4)]),       # 48 is past the table
            ([2147483647, 0], None, [0, 4, 8], cai.CAI_DEVERR_LENGTH, [(1, 0, 4)]),
            ([0, 0], [[-1, 0, 1], [99, 3, 4]], [0, 4, 8], cai.CAI_DEVERR_PAGE, []),
            ([0, 16], None, [4, 0, 4], cai.CAI_DEVERR_LENGTH, [(1, 16, 20)]),
            ([0, 0], None, [-1, 1, 99], cai.CAI_DEVERR_LENGTH, [])):
        sums, err = d.summaries(), flag()
        old = d.table
        if table is not None:
            d.table = dev(np.array(table, np.int32))
        d.summarize(sums, start, 4, offsets, err)
        d.table = old
        assert err.item() == bits
        got = sums[0].data[:d.num_pages * 256].view(d.num_pages, 256)
        changed = set(torch.nonzero((got != 0x5A).any(1))[:, 0].tolist())
        assert changed == {int(d.table_np[b, p // 16]) for b, lo, hi in done for p in range(lo, hi)}


@pytest.mark.parametrize("four", [False, True])
def test_summaries_of_many_sequences_with_a_loose_bound(four):
    """The largest n_new that a call may give, beside 300 short sequences."""
    new = [int(n) for n in np.random.default_rng(5).integers(0, 40, 300)]
    d = Dialogues(four, new, 1, 16, seed=6)
    sums, err = d.summaries(), flag()
    d.summarize(sums, [0] * 300, 1 << 22, np.concatenate([[0], np.cumsum(new)]), err)
    assert err.item() == 0
    same(sums, d.want([0] * 300, new))


# ----------------------------------------------------------------------------------- selection

def random_summaries(rng, hkv, num_pages, page, ties=False):
    out, host_side = [], []
    for _ in range(hkv):
        a, b = rng.integers(-127, 128, (2, num_pages, 128))
        codes = np.concatenate([np.maximum(a, b), np.minimum(a, b)], 1).astype(np.int8)
        scale = np.exp(rng.normal(size=num_pages) * 0.5).astype(np.float32) * np.float32(0.05)
        if ties:  # few different pages
            which = rng.integers(0, 3, num_pages)
            codes, scale = codes[which], scale[which]
        raw = np.concatenate([codes.view(np.uint8).ravel(), scale.view(np.uint8)])
        out.append(cai.KVSummary(num_pages, page, data=dev(raw)))
        host_side.append((codes, scale))
    return out, host_side


def run_select(sums, q, table, start, keep, first, last, offsets=None, max_new=None, err=None):
    lead = q.shape[:-2]
    rows = int(np.prod(lead))
    size = cai.cai_kv_select_workspace_size(len(start), rows, q.shape[-2], len(sums), table.shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)  # (NaN scores)
    out = torch.full((*lead, len(sums), keep), -7, dtype=torch.int32, device=DEV)
    length = torch.full(lead, -7, dtype=torch.int32, device=DEV)
    cai.cai_kv_select(sums, q, table, dev(np.array(start, np.int32)), first, last, ws, out, length, err,
                      None if offsets is None else dev(np.array(offsets, np.int32)), max_new)
    torch.cuda.synchronize()
    return out.cpu().numpy().reshape(rows, len(sums), keep), length.cpu().numpy().reshape(rows)


def check_select(hkv, g, page, start, new, keep, first, last, seed=0, ties=False, packed=True, size=1.0):
    rng = np.random.default_rng(seed)
    start, new = np.array(start), np.array(new)
    table, num_pages = tables(rng, start + new, page)
    sums, side = random_summaries(rng, hkv, num_pages, page, ties)
    rows = int(new.sum())
    q = dev(rng.normal(size=(rows, hkv * g, 128)).astype(np.float32) * size, torch.bfloat16)
    err = flag()
    offsets = np.concatenate([[0], np.cumsum(new)])
    if packed:
        got, length = run_select(sums, q, dev(table), start, keep, first, last, offsets, int(new.max()), err)
    else:
        got, length = run_select(sums, q.unflatten(0, (len(new), int(new[0]))), dev(table), start, keep, first, last, err=err)
    assert err.item() == 0
    qh = host(q)
    for b in range(len(new)):
        for i in range(new[b]):
            r = offsets[b] + i
            for j in range(hkv):
                codes, scale = side[j]
                ids = table[b, :(start[b] + i) // page + 1]
                blocks, tokens = pages.select(qh[r, j * g:(j + 1) * g], codes[ids], scale[ids], int(start[b] + i), page, keep, first, last)
                want = np.full(keep, -1)
                want[:len(blocks)] = ids[blocks]
                assert np.array_equal(got[r, j], want), (b, i, j)
                assert length[r] == tokens


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 8, 9, 16, 33, 64, 128])
def test_select_groups(g):
    """Every padding of the columns, single rows beside chunks, contexts below and above what is taken."""
    check_select(1 if g > 64 else 2, g, 16, [0, 70, 15, 16, 333, 900, 2000], [1, 1, 3, 40, 0, 17, 1], 9, 1, 2, seed=g)


@pytest.mark.parametrize("keep,first,last", [(1, 0, 1), (3, 1, 2), (4, 1, 2), (20, 0, 1), (64, 2, 4), (300, 5, 9), (17, 16, 1)])
@pytest.mark.parametrize("page", [16, 32, 64])
def test_select_counts(keep, first, last, page):
    check_select(1, 8, page, [3, 40 * page, 299 * page + 5, 300 * page, 301 * page], [1] * 5, keep, first, last, seed=keep, packed=False)


def test_select_ties_go_to_the_lower_page():
    check_select(2, 4, 16, [3000, 700, 4100, 12000], [2, 2, 2, 2], 40, 1, 2, ties=True, packed=False)
    check_select(1, 4, 16, [3000, 700], [2, 2], 40, 0, 1, ties=True, packed=False, size=0.0)  # zero queries: all scores 0


@pytest.mark.parametrize("context", [4100, 16000, 131071, 300000])
def test_select_long_context(context):
    """A table of each kernel's range: a warp a row, a block, and contexts of any length."""
    check_select(1, 16, 16, [context, 900, context - 3], [1, 2, 1], 128, 1, 2, seed=5)
    check_select(1, 2, 16, [context, 2000], [1, 2], 33, 1, 2, seed=6, ties=True)


def test_select_extreme_queries():
    check_select(2, 2, 16, [1000, 1111], [1, 1], 12, 0, 1, seed=6, size=3e4)
    check_select(2, 2, 16, [1000, 1111], [1, 1], 12, 0, 1, seed=7, size=1e-37)


def test_select_padded_batch_and_bad_arguments():
    """Rows behind the last sequence and of bad sequences: lists of -1 and length 0; bad page ids flagged."""
    rng = np.random.default_rng(3)
    sums, _ = random_summaries(rng, 2, 64, 16)
    table = dev(rng.permutation(64)[:60].reshape(2, 30).astype(np.int32))
    q = dev(rng.normal(size=(9, 4, 128)).astype(np.float32), torch.bfloat16)

    def run(start, offsets, bits, tb=table, max_new=4, keep=5):
        err = flag()
        got, length = run_select(sums, q, tb, start, keep, 1, 1, offsets, max_new, err)
        assert err.item() == bits
        assert ((got == -1).all((1, 2)) == (length == 0)).all() and (got != -7).all()
        return (length > 0).tolist()

    assert run([100, 200], [0, 3, 6], 0) == [True] * 6 + [False] * 3
    assert run([100, 478], [0, 3, 6], cai.CAI_DEVERR_LENGTH) == [True] * 5 + [False] * 4      # 480 is past the table
    assert run([-2, 200], [0, 3, 6], cai.CAI_DEVERR_LENGTH) == [False] * 2 + [True] * 4 + [False] * 3
    assert run([100, 200], [0, 5, 6], cai.CAI_DEVERR_LENGTH) == [False] * 5 + [True] + [False] * 3  # more than max_new
    assert run([100, 200], [0, 3, 11], cai.CAI_DEVERR_LENGTH, max_new=20) == [True] * 3 + [False] * 6
    bad = table.clone()
    bad[0, 2], bad[1, 3] = 64, -1
    assert run([100, 200], [0, 3, 6], cai.CAI_DEVERR_PAGE, tb=bad) == [True] * 6 + [False] * 3
    assert run([100, 200], [0, 3, 6], cai.CAI_DEVERR_PAGE, tb=bad, keep=40) == [True] * 6 + [False] * 3


def test_select_leaves_its_neighbours_alone():
    """Outputs are written within their bounds, and no table entry past the context counts."""
    rng = np.random.default_rng(8)
    sums, _ = random_summaries(rng, 1, 40, 16)
    table = np.full((1, 500), 1 << 30, np.int32)
    table[0, :30] = rng.permutation(40)[:30]
    q = dev(rng.normal(size=(1, 1, 3, 128)).astype(np.float32), torch.bfloat16)
    room = torch.full((3, 7), -7, dtype=torch.int32, device=DEV)
    ws = torch.empty(cai.cai_kv_select_workspace_size(1, 1, 3, 1, 500), dtype=torch.uint8, device=DEV)
    err, length = flag(), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    cai.cai_kv_select(sums, q, dev(table), dev(np.array([479], np.int32)), 1, 1, ws, room[1].view(1, 1, 1, 7), length, err)
    assert err.item() == 0 and (room[0] == -7).all() and (room[2] == -7).all() and (room[1] >= 0).all()
    assert room[1, 0] == table[0, 0] and room[1, 6] == table[0, 29] and length.item() == 7 * 16


# ------------------------------------------------------------------------ attention over lists

"""Bounds of the attention.  q, K and V enter the products exactly; a weight is 2^z rounded to fp16, 2^-11 of it, with z off
by the fp32 sums' rounding, 2^-12 of the weight at most for the logits here (checked by the bound on lse); weights among
fp16's subnormals are off by 2^-32 of the largest that enters a product, so by 2^-32 max|v| of the output each; the output is
rounded to bf16 once: |out - ref| <= 2^-8 |ref| + (1 + 2^-8) ((2^-11 + 2^-12) sum p|v| + n 2^-32 max|v|).
lse: 2^-20 of scale * sum |q k|, of 1 + |lse| and, where V's scale goes through the exponent, of its logarithm."""


def attend(d, q, lists, lens, scale=SCALE, splits=0, bits=0, poison=0xFF):
    size = cai.cai_kv4_attend_pages_workspace_size if d.four else cai.cai_kv_attend_pages_workspace_size
    n = size(q.shape[0], q.shape[1], d.hkv, lists.shape[2], d.page, splits)
    ws = torch.full((n,), poison, dtype=torch.uint8, device=DEV) if n else None
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse, err = torch.full(q.shape[:2], float("nan"), device=DEV), flag()
    f = cai.cai_kv4_attend_pages if d.four else cai.cai_kv_attend_pages
    f(d.pools, q, dev(np.ascontiguousarray(lists, np.int32)), dev(np.array(lens, np.int32)), scale, splits, ws, out, lse, err)
    torch.cuda.synchronize()
    assert err.item() == bits
    return host(out), host(lse)


def page_values(d):
    """K and V float64 [hkv][pages][P][128] by page id (NaN where nothing is), and V's scales' logarithms' largest magnitude."""
    k = np.full((d.hkv, d.num_pages, d.page, 128), np.nan)
    v = np.full_like(k, np.nan)
    for j in range(d.hkv):
        for b, n in enumerate(d.lengths):
            for i in range(-(-n // d.page)):
                x = slice(i * d.page, min(n, (i + 1) * d.page))
                k[j, d.table_np[b, i], :x.stop - x.start] = d.k[j][b][x]
                v[j, d.table_np[b, i], :x.stop - x.start] = d.v[j][b][x]
    return k, v


def check_attend(d, q, lists, lens, out, lse, scale=SCALE, skip=()):
    k, v = page_values(d)
    g = q.shape[1] // d.hkv
    qh = host(q).astype(np.float64)
    for r, n in enumerate(lens):
        if r in skip:
            continue
        for j in range(d.hkv):
            ids = lists[r, j, :-(-n // d.page)]
            kk, vv = (x[j, ids].reshape(-1, 128)[:n] for x in (k, v))
            hs = slice(j * g, (j + 1) * g)
            ref, rl, a, big = kv4.attend_rows(qh[r:r + 1, hs], kk, vv, scale, np.ones((1, n), bool))
            got, gl = out[r:r + 1, hs].astype(np.float64), lse[r:r + 1, hs].astype(np.float64)
            if n == 0:
                assert (got == 0).all() and (gl == -np.inf).all(), (r, j)
                continue
            assert np.isfinite(got).all() and np.isfinite(gl).all(), (r, j)
            top = np.abs(vv).max(initial=0)
            bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((2.0 ** -11 + 2.0 ** -12) * a + n * 2.0 ** -32 * top) + 2.0 ** -133
            err = np.abs(got - ref)
            assert (err <= bound).all(), (r, j, (err - bound).max(), err.max())
            vs = np.abs(vv).max(-1) / 127  # (of int8 tokens; 2^-100 at least)
            lv = 0.0 if d.four else np.abs(np.log2(np.maximum(vs, 2.0 ** -100))).max()
            assert (np.abs(gl - rl) <= 2.0 ** -20 * (big + 1 + np.abs(rl) + lv)).all(), (r, j, np.abs(gl - rl).max())


def random_lists(rng, d, rows, width, lens):
    """For every row and K/V head pages of one sequence in any order, whole ones but the last."""
    lists = np.full((rows, d.hkv, width), -1, np.int64)
    for r, n in enumerate(lens):
        for j in range(d.hkv):
            whole = np.concatenate([d.table_np[b, :m // d.page] for b, m in enumerate(d.lengths)])
            lists[r, j, :-(-n // d.page)] = rng.choice(whole, -(-n // d.page))  # (a page may stand there twice)
    return lists


ATTEND = [  # hkv, heads of a group, page, splits
    (1, 1, 16, 0), (2, 3, 32, 0), (8, 4, 64, 0), (1, 8, 16, 3), (2, 9, 32, 0), (1, 16, 64, 1), (2, 17, 16, 0), (1, 32, 32, 0),
    (1, 33, 16, 0), (2, 40, 64, 2), (1, 64, 32, 0), (1, 65, 16, 0), (1, 128, 64, 0),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hkv,g,page,splits", ATTEND)
def test_attend_lists(four, hkv, g, page, splits):
    rng = np.random.default_rng(g)
    d = Dialogues(four, [700, 64, 333], hkv, page, seed=g)
    lens = [0, 1, page, page + 1, 127, 128, 129, 640, 255, 0, 5 * page + 3]
    width = 640 // page + 1
    lists = random_lists(rng, d, len(lens), width, lens)
    q = dev(rng.normal(size=(len(lens), hkv * g, 128)).astype(np.float32) * 1.5, torch.bfloat16)
    out, lse = attend(d, q, lists, lens, splits=splits)
    check_attend(d, q, lists, lens, out, lse)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [4, 32, 64])
def test_attend_many_rows(four, g):
    """More rows than blocks, and few long ones that are cut; the same again to the bit."""
    rng = np.random.default_rng(g)
    d = Dialogues(four, [900, 2000], 1, 16, seed=g + 1)
    for rows, width in ((400, 12), (3, 125)):
        lens = rng.integers(0, width * 16 + 1, rows)
        lens[0] = width * 16
        lists = random_lists(rng, d, rows, width, lens)
        q = dev(rng.normal(size=(rows, g, 128)).astype(np.float32), torch.bfloat16)
        out, lse = attend(d, q, lists, lens)
        check_attend(d, q, lists, lens, out, lse)
        again = attend(d, q, lists, lens, poison=0)
        assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g,rows", [(6, 430), (16, 170), (32, 170), (64, 75), (128, 30)])
def test_attend_rows_cut_anywhere_and_in_equal_pieces(four, g, rows):
    """Counts at which the blocks share all rows' tiles, and the same rows in equal pieces."""
    rng = np.random.default_rng(g + 9)
    d = Dialogues(four, [2500], 1, 16, seed=g + 2)
    width = 128
    lens = rng.integers(0, width * 16 + 1, rows)
    lens[-1] = width * 16
    lists = rng.choice(d.table_np[0, :156], (rows, 1, width))
    q = dev(rng.normal(size=(rows, g, 128)).astype(np.float32), torch.bfloat16)
    check = rng.choice(rows, 25, replace=False)
    for splits in (0, 1, 3, 7):
        out, lse = attend(d, q, lists, lens, splits=splits)
        check_attend(d, q, lists, lens, out, lse, skip=set(range(rows)) - set(check.tolist()))
        assert np.isfinite(out).all()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [6, 16, 32, 64])
@pytest.mark.parametrize("most", [300, 1500])
def test_attend_more_rows_than_the_chip_takes_at_once(four, g, most):
    """Rows of one tile and of many in turn, several to a block, cut wherever the blocks' shares end: every row against
    a plain 64-bit formulation, and the same bits again."""
    rng = np.random.default_rng(g)
    d = Dialogues(four, [2000], 1, 16, seed=g)
    rows, width = 1300, -(-most // 16)
    lens = rng.integers(1, most + 1, rows)
    lens[::3] = rng.integers(1, 200, len(lens[::3]))
    lists = rng.choice(d.table_np[0, :125], (rows, 1, width))
    q = dev(rng.normal(size=(rows, g, 128)).astype(np.float32), torch.bfloat16)
    out, lse = attend(d, q, lists, lens)
    k, v = (dev(x[0].reshape(-1, 128)) for x in page_values(d))
    k, v = (torch.nan_to_num(x) for x in (k, v))
    ids, t = dev(lists[:, 0]), torch.arange(width * 16, device=DEV)
    n = dev(lens)
    for a in range(0, rows, 100):
        r = slice(a, min(rows, a + 100))
        at = ids[r][:, t // 16] * 16 + t % 16
        kk, vv, seen = k[at], v[at], t < n[r, None]
        qd = q[r].double()
        z = torch.einsum("rhd,rtd->rht", qd, kk) * SCALE
        z = torch.where(seen[:, None], z, torch.full_like(z, -np.inf))
        p = torch.softmax(z, -1)
        ref, soft = torch.einsum("rht,rtd->rhd", p, vv), torch.einsum("rht,rtd->rhd", p, vv.abs())
        top = torch.where(seen[..., None], vv.abs(), torch.zeros_like(vv)).amax((1, 2))[:, None, None]
        bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * ((2.0 ** -11 + 2.0 ** -12) * soft + n[r, None, None] * 2.0 ** -32 * top)
        err = (dev(out[r]).double() - ref).abs()
        bad = (err > bound).any(-1).any(-1).nonzero()[:, 0].tolist()
        assert not bad, [(a + i, int(lens[a + i])) for i in bad]
        rl = torch.logsumexp(z, -1)
        big = (torch.einsum("rhd,rtd->rht", qd.abs(), kk.abs()) * SCALE * seen[:, None]).amax(-1)
        lv = 0.0 if four else 20.0  # (|log2| of V's scales here, at most)
        assert ((dev(lse[r]).double() - rl).abs() <= 2.0 ** -20 * (big + 1 + rl.abs() + lv)).all()
    again = attend(d, q, lists, lens, poison=0)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


def test_attend_whole_contexts_is_the_decode():
    """Lists of all pages of a 4-bit context give what the decode gives: both within the bounds (their sums are cut
    differently, so not to the bit)."""
    rng = np.random.default_rng(1)
    for g in (4, 24):
        d = Dialogues(True, [500, 1, 129], 1, 16, seed=g)
        q = dev(rng.normal(size=(3, g, 128)).astype(np.float32), torch.bfloat16)
        out, lse = attend(d, q, d.table_np[:, None], d.lengths)
        n = cai.cai_kv4_decode_workspace_size(3, g, 1, d.table.shape[1], 16, 0, 0)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        o2, l2 = torch.empty_like(q), torch.empty(3, g, device=DEV)
        cai.cai_kv4_decode(d.pools, q, d.table, dev(np.array(d.lengths, np.int32)), 0, SCALE, 0, ws, o2, l2)
        check_attend(d, q, d.table_np[:, None], d.lengths, out, lse)
        check_attend(d, q, d.table_np[:, None], d.lengths, host(o2), host(l2))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -24, 2.0 ** -10, 2.0 ** 12])
def test_attend_values_of_any_size(four, size):
    """Small and large values keep their precision (the 4-bit scales are fp16: 2^-14 and up), zero vectors among them."""
    if four and size < 2.0 ** -11:
        pytest.skip("fp16 scales")
    rng = np.random.default_rng(2)
    d = Dialogues(four, [400], 1, 16, seed=3)
    x = rng.normal(size=(2, 1, 400, 1, 128)).astype(np.float32)
    x[1] *= size
    x[1, 0, ::7] = 0
    append = cai.cai_kv4_append if four else cai.cai_kv_append_rope
    append(d.pools, dev(x[0]), dev(x[1]), d.table, torch.zeros(1, dtype=torch.int32, device=DEV))
    d.k, d.v = [[d.stored(x[0, 0, :, 0])]], [[d.stored(x[1, 0, :, 0])]]
    for g in (4, 32):
        q = dev(rng.normal(size=(1, g, 128)).astype(np.float32), torch.bfloat16)
        out, lse = attend(d, q, d.table_np[:, None], [400])
        check_attend(d, q, d.table_np[:, None], [400], out, lse)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("first", [True, False])
def test_attend_one_heavy_key(four, first):
    """One key far above a flat rest whose weights are small but many, at the list's start or its end."""
    rng = np.random.default_rng(4)
    n = 2048
    d = Dialogues(four, [n], 1, 32, seed=5)
    x = np.zeros((2, 1, n, 1, 128), np.float32)
    x[0, 0, 0 if first else n - 1] = 1.0
    x[1] = rng.normal(size=(1, n, 1, 128)) + 3
    append = cai.cai_kv4_append if four else cai.cai_kv_append_rope
    append(d.pools, dev(x[0]), dev(x[1]), d.table, torch.zeros(1, dtype=torch.int32, device=DEV))
    d.k, d.v = [[d.stored(x[0, 0, :, 0])]], [[d.stored(x[1, 0, :, 0])]]
    for g in (2, 20, 64):
        q = torch.full((1, g, 128), 1.0, dtype=torch.bfloat16, device=DEV)
        for scale in (5.0 / 128, 12.0 / 128, -12.0 / 128, 0.0):
            out, lse = attend(d, q, d.table_np[:, None], [n], scale=scale)
            check_attend(d, q, d.table_np[:, None], [n], out, lse, scale=scale)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [4, 32])
def test_attend_bad_arguments_on_the_device(four, g):
    """Bad lengths give zeros, bad page ids are flagged and left out; other rows do not notice."""
    rng = np.random.default_rng(6)
    d = Dialogues(four, [300], 1, 16, seed=7)
    lists = np.repeat(d.table_np[:, None, :10], 4, 0).astype(np.int64)
    q = dev(rng.normal(size=(4, g, 128)).astype(np.float32), torch.bfloat16)
    out, lse = attend(d, q, lists, [160, 161, -1, 31], bits=cai.CAI_DEVERR_LENGTH)
    for r in (1, 2):
        assert (out[r] == 0).all() and (lse[r] == -np.inf).all()
    check_attend(d, q, lists, [160, 0, 0, 31], out, lse, skip=(1, 2))
    for bad in (-1, d.num_pages, 2147483647, -2147483648):
        broken = lists.copy()
        broken[1, 0, 3] = bad
        out, lse = attend(d, q, broken, [160, 160, 16, 31], bits=cai.CAI_DEVERR_PAGE)
        without = lists.copy()
        without[1, 0, 3:9] = lists[1, 0, 4:10]
        check_attend(d, q, without, [160, 144, 16, 31], out, lse)
    broken = lists.copy()
    broken[1, 0, 3:] = 1 << 29  # behind the length: not read
    out, lse = attend(d, q, broken, [160, 48, 16, 31])
    check_attend(d, q, broken, [160, 48, 16, 31], out, lse)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g,rows", [(6, 430), (32, 170), (64, 75)])
def test_attend_bad_rows_among_many(four, g, rows):
    """Counts at which the blocks share all rows' tiles: invalid lengths, empty rows and bad page ids between the others."""
    rng = np.random.default_rng(g + 20)
    d = Dialogues(four, [2500], 1, 16, seed=g + 3)
    width = 128
    lens = rng.integers(0, width * 16 + 1, rows)
    wrong = rng.choice(rows, 40, replace=False)
    lens[wrong[:10]], lens[wrong[10:20]], lens[wrong[20:30]] = -5, width * 16 + 1, 0
    lists = rng.choice(d.table_np[0, :156], (rows, 1, width)).astype(np.int64)
    lists[wrong[30:]] = d.num_pages + 3
    lens[wrong[30:]] = np.maximum(lens[wrong[30:]], 1)
    q = dev(rng.normal(size=(rows, g, 128)).astype(np.float32), torch.bfloat16)
    out, lse = attend(d, q, lists, lens, bits=cai.CAI_DEVERR_LENGTH | cai.CAI_DEVERR_PAGE)
    assert (out[wrong] == 0).all() and (lse[wrong] == -np.inf).all()
    check = set(rng.choice(np.setdiff1d(np.arange(rows), wrong), 20, replace=False).tolist())
    check_attend(d, q, lists, lens, out, lse, skip=set(range(rows)) - check)
    assert np.isfinite(out).all()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [4, 32, 64])
def test_attend_rows_of_bad_pages_alone(four, g):
    """A row none of whose pages is in the pool has nothing to attend, in one piece or cut; its neighbours do not notice."""
    rng = np.random.default_rng(16)
    d = Dialogues(four, [3000], 1, 16, seed=17)
    lists = np.repeat(d.table_np[:, None, :180], 3, 0).astype(np.int64)
    lists[1] = d.num_pages + rng.integers(0, 9, 180)
    q = dev(rng.normal(size=(3, g, 128)).astype(np.float32), torch.bfloat16)
    for lens, splits in (([70, 90, 100], 0), ([2880, 2880, 2000], 0), ([2880, 2880, 2000], 5)):
        out, lse = attend(d, q, lists, lens, splits=splits, bits=cai.CAI_DEVERR_PAGE)
        assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
        check_attend(d, q, lists, lens, out, lse, skip=(1,))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [4, 32])
def test_attend_graphs_share_a_workspace(four, g):
    """Two captured calls of different shapes in turn on one workspace, replayed: the bits of calls on their own."""
    rng = np.random.default_rng(18)
    d = Dialogues(four, [900, 700], 2, 16, seed=19)
    size = cai.cai_kv4_attend_pages_workspace_size if four else cai.cai_kv_attend_pages_workspace_size
    f = cai.cai_kv4_attend_pages if four else cai.cai_kv_attend_pages
    calls = []
    for rows, width in ((3, 50), (200, 7)):
        lens = rng.integers(0, 16 * width + 1, rows)
        lists = random_lists(rng, d, rows, width, lens)
        q = dev(rng.normal(size=(rows, 2 * g, 128)).astype(np.float32), torch.bfloat16)
        calls.append((q, lists, lens, attend(d, q, lists, lens), size(rows, 2 * g, 2, width, 16)))
    ws = torch.full((max(c[4] for c in calls),), 0xFF, dtype=torch.uint8, device=DEV)
    graphs = []
    for q, lists, lens, _, _ in calls:
        args = [q, dev(np.ascontiguousarray(lists, np.int32)), dev(np.array(lens, np.int32))]
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        f(d.pools, *args, SCALE, 0, ws, out, lse)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            f(d.pools, *args, SCALE, 0, ws, out, lse)
        graphs.append((graph, out, lse, args))
    for _ in range(3):
        for graph, out, lse, _ in graphs:
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for (_, out, lse, _), (_, _, _, want, _) in zip(graphs, calls):
            assert np.array_equal(host(out), want[0]) and np.array_equal(host(lse), want[1])


@pytest.mark.parametrize("g", [4, 32, 64])
@pytest.mark.parametrize("stage", [0, 1, 4])
def test_attend_timeout_is_reported(g, stage):
    """A copy that never comes: the wait ends, the flag says so, and the next call is right."""
    rng = np.random.default_rng(8)
    d = Dialogues(False, [900], 1, 16, seed=9)
    q = dev(rng.normal(size=(2, g, 128)).astype(np.float32), torch.bfloat16)
    lists, lens = np.repeat(d.table_np[:, None, :56], 2, 0), [896, 896]
    cai.cai_set_wait_limit_ns(20_000_000)
    cai.cai_set_fault_injection(stage)
    try:
        attend(d, q, lists, lens, splits=1, bits=cai.CAI_DEVERR_TIMEOUT)
    finally:
        cai.cai_set_fault_injection(-1)
        cai.cai_set_wait_limit_ns(0)
    out, lse = attend(d, q, lists, lens, splits=1)
    check_attend(d, q, lists, lens, out, lse)


# ------------------------------------------------------------------------------- a run together

def sparse_step(d, sums, rope, qkv, hq, start, new, keep, first, last, ws, outs):
    """append (axes) -> summarize -> select -> attend, packed rows."""
    hkv, n = d.hkv, qkv.shape[0]
    off, pos = ws["offsets"], ws["positions"]
    append = cai.cai_kv4_append_axes if d.four else cai.cai_kv_append_rope_axes
    append(d.pools, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], d.table, start, rope, pos, q=qkv[:, :hq], q_out=outs["q"],
           q_offsets=off, max_new=new, err_flag=ws["err"])
    (cai.cai_kv4_summarize if d.four else cai.cai_kv_summarize)(d.pools, sums, d.table, start, new, q_offsets=off, err_flag=ws["err"])
    cai.cai_kv_select(sums, outs["q"], d.table, start, first, last, ws["select"], outs["pages"], outs["len"], ws["err"], off, new)
    (cai.cai_kv4_attend_pages if d.four else cai.cai_kv_attend_pages)(
        d.pools, outs["q"], outs["pages"], outs["len"], SCALE, 0, ws["attend"], outs["out"], outs["lse"], ws["err"])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hkv,g,page", [(1, 32, 16), (2, 4, 32)])
def test_sparse_steps(four, hkv, g, page):
    """A chunk, then decode steps in a padded batch, eagerly and from a captured graph: every stage against the oracle."""
    rng = np.random.default_rng(11)
    before, new, hq, keep, first, last = np.array([900, 0, 33, 1500]), np.array([40, 3, 0, 1]), hkv * g, 8, 1, 2
    d = Dialogues(four, before, hkv, page, seed=12, width=-(-1600 // page))
    # Room for the tokens to come: pages behind the pool that the dialogues use.
    bytes_ = kv4.page_bytes4(page) if four else oracle.page_bytes(page)
    cls = cai.KV4Pool if four else cai.KVPool
    used = d.num_pages
    d.pools = [cls(used + 64, page, pages=torch.cat((p.pages, torch.full((64 * bytes_,), 0xFF, dtype=torch.uint8, device=DEV)))) for p in d.pools]
    d.num_pages = used + 64
    at = 0
    for b in range(4):
        have = -(-int(before[b]) // page)
        for i in range(have, -(-(int(before[b]) + 50) // page)):
            d.table_np[b, i] = used + at
            at += 1
    d.table = dev(d.table_np)
    sums = d.summaries(fill=0xEE)
    d.summarize(sums, [0] * 4, int(before.max()), np.concatenate([[0], np.cumsum(before)]))
    half = 64
    ang = np.arange(2000)[:, None] * (1e4 ** (-np.arange(half) / half))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    axis = [i * 3 // half for i in range(half)]
    rope = cai.RopeAxes(dev(cos), dev(sin), axis)
    k, v = [[list(x) for x in d.k[j]] for j in range(hkv)], [[list(x) for x in d.v[j]] for j in range(hkv)]

    def buffers(rows):
        return (dict(offsets=torch.zeros(5, dtype=torch.int32, device=DEV), positions=torch.zeros(rows, 3, dtype=torch.int32, device=DEV),
                     err=flag(), select=torch.empty(cai.cai_kv_select_workspace_size(4, rows, hq, hkv, d.table.shape[1]), dtype=torch.uint8, device=DEV),
                     attend=torch.empty((cai.cai_kv4_attend_pages_workspace_size if four else cai.cai_kv_attend_pages_workspace_size)(
                         rows, hq, hkv, keep, page), dtype=torch.uint8, device=DEV)),
                dict(q=torch.zeros(rows, hq, 128, dtype=torch.bfloat16, device=DEV), pages=torch.full((rows, hkv, keep), -9, dtype=torch.int32, device=DEV),
                     len=torch.full((rows,), -9, dtype=torch.int32, device=DEV), out=torch.full((rows, hq, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
                     lse=torch.full((rows, hq), float("nan"), device=DEV)))

    def check(start, new, qkv, pos, outs, total):
        pos_np, q_in = pos, host(qkv)
        turned = pages.rotate_axes(q_in[:, :hq + hkv], pos_np, axis, cos, sin, False)
        off = np.concatenate([[0], np.cumsum(new)])
        for j in range(hkv):
            for b in range(4):
                r = slice(off[b], off[b + 1])
                k[j][b] += list(d.stored(turned[r, hq + j]))
                v[j][b] += list(d.stored(q_in[r, hq + hkv + j]))
        d.lengths = [int(s + n) for s, n in zip(start, new)]
        d.k, d.v = ([[np.array(x, np.float32).reshape(-1, 128) for x in y] for y in z] for z in (k, v))
        q = kv4.bf16_round(turned[:, :hq])
        n = off[-1]
        assert np.array_equal(host(outs["q"])[:n], q[:n])
        lists, length = outs["pages"].cpu().numpy(), outs["len"].cpu().numpy()
        for j in range(hkv):
            for b in range(4):
                codes, scale = zip(*(pages.summarize(d.k[j][b][i:i + page]) for i in range(0, max(1, d.lengths[b]), page))) if d.lengths[b] else ((), ())
                for i in range(new[b]):
                    blocks, tokens = pages.select(q[off[b] + i, j * g:(j + 1) * g], np.array(codes), np.array(scale), int(start[b] + i), page, keep, first, last)
                    want = np.full(keep, -1)
                    want[:len(blocks)] = d.table_np[b, blocks]
                    assert np.array_equal(lists[off[b] + i, j], want) and length[off[b] + i] == tokens
        assert (lists[n:] == -1).all() and (length[n:] == 0).all()
        check_attend(d, outs["q"], lists, length, host(outs["out"]), host(outs["lse"]))
        assert (outs["out"][n:total] == 0).all()

    # The chunk.
    rows = int(new.sum())
    ws, outs = buffers(rows)
    ws["offsets"].copy_(dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
    pos = rng.integers(0, 2000, (rows, 3)).astype(np.int32)
    ws["positions"].copy_(dev(pos))
    qkv = dev(rng.normal(size=(rows, hq + 2 * hkv, 128)).astype(np.float32) * 1.5, torch.bfloat16)
    sparse_step(d, sums, rope, qkv, hq, dev(before.astype(np.int32)), 40, keep, first, last, ws, outs)
    torch.cuda.synchronize()
    assert ws["err"].item() == 0
    check(before, new, qkv, pos, outs, rows)

    # Decode steps of three of the four sequences, a batch padded to six rows, from one graph on another stream.
    ws, outs = buffers(6)
    start = dev((before + new).astype(np.int32))
    qkv = torch.zeros(6, hq + 2 * hkv, 128, dtype=torch.bfloat16, device=DEV)
    one = np.array([1, 1, 0, 1])
    ws["offsets"].copy_(dev(np.concatenate([[0], np.cumsum(one)]).astype(np.int32)))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    keep_pages = [p.pages.clone() for p in d.pools]
    keep_sums = [s.data.clone() for s in sums]
    with torch.cuda.stream(stream):
        sparse_step(d, sums, rope, qkv, hq, start, 1, keep, first, last, ws, outs)  # (a warm-up; undone below)
        with torch.cuda.graph(graph, stream=stream):
            sparse_step(d, sums, rope, qkv, hq, start, 1, keep, first, last, ws, outs)
    torch.cuda.synchronize()
    for a, b in zip([p.pages for p in d.pools] + [s.data for s in sums], keep_pages + keep_sums):
        a.copy_(b)
    now = before + new
    for step in range(3):
        pos = rng.integers(0, 2000, (6, 3)).astype(np.int32)
        ws["positions"].copy_(dev(pos))
        qkv.copy_(dev(rng.normal(size=tuple(qkv.shape)).astype(np.float32) * 1.5, torch.bfloat16))
        start.copy_(dev(now.astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert ws["err"].item() == 0
        check(now, one, qkv, pos, outs, 6)
        now = now + one
