"""The size of the workspace of attention over lists: enough for every smaller call, too."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import int8_mqa_decode_gb300 as cai
from int8_mqa_decode_gb300 import build as cai_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    cai_build.build()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hq,hkv,page", [(8, 1, 16), (32, 1, 16), (64, 1, 64), (128, 1, 32), (6, 3, 16), (64, 8, 32), (256, 2, 64)])
@pytest.mark.parametrize("splits", [0, 1, 4, 64])
def test_more_rows_or_pages_need_no_less(four, hq, hkv, page, splits):
    size = cai.cai_kv4_attend_pages_workspace_size if four else cai.cai_kv_attend_pages_workspace_size
    rows = [*range(1, 40), *range(40, 700, 7), 1000, 4096, 65535]
    widths = [1, 2, 7, 8, 9, 16, 31, 32, 33, 64, 128, 500, 8192, 1 << 20]
    sizes = {(r, w): size(r, hq, hkv, w, page, splits) for r, w in itertools.product(rows, widths)}
    for (r, w), n in sizes.items():
        before = [sizes[r2, w] for r2 in rows if r2 < r][-1:] + [sizes[r, w2] for w2 in widths if w2 < w][-1:]
        assert n >= max(before, default=0), (r, w)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hq,hkv,page,width", [(8, 1, 16, 32), (32, 1, 16, 128), (64, 1, 64, 64), (64, 8, 32, 64), (6, 3, 16, 200)])
def test_a_workspace_serves_smaller_calls(four, hq, hkv, page, width):
    """A workspace for 700 rows, calls of fewer rows and narrower lists: none is refused, and nothing behind it is written."""
    size, attend, cls = (
        (cai.cai_kv4_attend_pages_workspace_size, cai.cai_kv4_attend_pages, cai.KV4Pool) if four
        else (cai.cai_kv_attend_pages_workspace_size, cai.cai_kv_attend_pages, cai.KVPool))
    pool = [cls(4, page) for _ in range(hkv)]
    for p in pool:
        p.pages.zero_()  # codes and scales of 0
    for splits in (0, 3):
        n = size(700, hq, hkv, width, page, splits)
        room = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        for rows in (1, 3, 20, 37, 64, 75, 100, 128, 152, 153, 200, 256, 304, 305, 608, 609, 700):
            for w in (width, width - 1, width // 2, width // 4, 1):
                q = torch.zeros(rows, hq, 128, dtype=torch.bfloat16, device="cuda")
                pages = torch.zeros(rows, hkv, w, dtype=torch.int32, device="cuda")
                lengths = torch.full((rows,), w * page, dtype=torch.int32, device="cuda")
                out, lse, err = torch.full_like(q, 7), torch.zeros(rows, hq, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
                attend(pool, q, pages, lengths, 1.0, splits, room[:n], out, lse, err)
                # Keys and values of 0: out = 0, lse the logarithm of their count.
                assert err.item() == 0 and (out == 0).all()
                assert ((lse - torch.log(lengths[:1].float())).abs() <= 2.0 ** -20 * (1 + 9 + 100)).all()
        assert (room[n:] == 0xA5).all()
