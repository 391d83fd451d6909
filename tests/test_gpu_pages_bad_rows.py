"""Rows outside the table and queries that are not finite: what they touch, and what they leave alone."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
from test_gpu_kv4 import _built, dev, flag, host  # noqa: E402,F401
from test_gpu_pages import Dialogues, attend, check_attend, random_lists, random_summaries, run_select  # noqa: E402


@pytest.mark.parametrize("start", [480, 500, 2 ** 31 - 1, -2, -2 ** 31])
@pytest.mark.parametrize("packed", [True, False])
def test_select_rows_outside_the_table_flag_no_pages(start, packed):
    """A sequence without a row inside its table has no pages: entries of the table that are no page ids are not flagged."""
    rng = np.random.default_rng(1)
    sums, _ = random_summaries(rng, 2, 64, 16)
    table = np.full((3, 30), -1, np.int32)
    table[0, :20], table[2, :25] = rng.permutation(64)[:20], rng.permutation(64)[:25]
    q = dev(rng.normal(size=(6, 8, 128)).astype(np.float32), torch.bfloat16)
    at, err = [300, start, 390], flag()
    if packed:
        got, length = run_select(sums, q, dev(table), at, 7, 1, 2, [0, 2, 4, 6], 2, err)
    else:
        got, length = run_select(sums, q.unflatten(0, (3, 2)), dev(table), at, 7, 1, 2, err=err)
    assert err.item() == cai.CAI_DEVERR_LENGTH
    assert (got[2:4] == -1).all() and (length[2:4] == 0).all()
    other = run_select(sums, q[[0, 1, 4, 5]].unflatten(0, (2, 2)), dev(table[[0, 2]]), [300, 390], 7, 1, 2)
    assert np.array_equal(got[[0, 1, 4, 5]], other[0]) and np.array_equal(length[[0, 1, 4, 5]], other[1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("g", [4, 16, 32, 64])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_attend_queries_that_are_not_finite_concern_their_head_alone(four, g, what):
    rng = np.random.default_rng(2)
    d = Dialogues(four, [700], 2, 16, seed=3)
    lens = [500, 37, 0, 640]
    lists = random_lists(rng, d, 4, 40, lens)
    q = rng.normal(size=(4, 2 * g, 128)).astype(np.float32)
    bad = rng.random((4, 2 * g)) < 0.2
    bad[:, 0], bad[:, g] = True, False
    for splits in (0, 1, 3):
        clean, clean_lse = attend(d, dev(q, torch.bfloat16), lists, lens, splits=splits)
        broken = q.copy()
        broken[bad, 5] = what
        out, lse = attend(d, dev(broken, torch.bfloat16), lists, lens, splits=splits)
        # A raise of one head's reference asks for the others' weights anew: the same numbers.
        assert np.array_equal(out[~bad], clean[~bad]) and np.array_equal(lse[~bad], clean_lse[~bad])
    check_attend(d, dev(q, torch.bfloat16), lists, lens, clean, clean_lse)
