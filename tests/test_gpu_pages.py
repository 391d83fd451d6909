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


def test_select_long_context():
    check_select(1, 16, 16, [131071, 100000], [1, 2], 128, 1, 2, seed=5)


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
    """Outputs are written within their bounds, and no row of the table past the context is looked at."""
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
