"""Waits that run out in the selection's scores and in the 4-bit attention over lists: a message never comes (the host
says which), the launch reports it and ends, and the next calls are right."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
from test_gpu_kv4 import _built, dev, flag, tables  # noqa: E402,F401
from test_gpu_pages import Dialogues, attend, check_attend, check_select, random_summaries, run_select  # noqa: E402


@pytest.fixture
def drop():
    def at(stage):
        cai.cai_set_wait_limit_ns(20_000_000)
        cai.cai_set_fault_injection(stage)
    yield at
    cai.cai_set_fault_injection(-1)
    cai.cai_set_wait_limit_ns(0)


@pytest.mark.parametrize("batch,pages,stage", [(3, 200, 0), (700, 300, 1), (700, 300, 2)])
@pytest.mark.parametrize("g", [1, 4, 12, 32])
def test_scores_give_up_then_recover(drop, batch, pages, stage, g):
    """One tile of pages a block, and several (more sequences than blocks fit the chip)."""
    rng = np.random.default_rng(g)
    start = np.full(batch, pages * 16 - 3)
    table, num_pages = tables(rng, start + 1, 16)
    sums, _ = random_summaries(rng, 1, num_pages, 16)
    q = dev(rng.normal(size=(batch, 1, g, 128)).astype(np.float32), torch.bfloat16)
    err = flag()
    drop(stage)
    got, length = run_select(sums, q, dev(table), start, 9, 1, 2, err=err)
    assert err.item() == cai.CAI_DEVERR_TIMEOUT
    assert (length == 8 * 16 + (pages * 16 - 3) % 16 + 1).all()
    for b in range(batch):  # (some pages of the row's context)
        assert set(got[b, 0]) <= set(table[b, :pages])
    drop(-1)
    cai.cai_set_wait_limit_ns(0)
    check_select(1, g, 16, [pages * 16 - 3] * 5, [1] * 5, 9, 1, 2, seed=g, packed=False)


@pytest.mark.parametrize("g", [4, 16, 32, 64])
@pytest.mark.parametrize("stage", [0, 1, 4])
def test_attend4_gives_up_then_recovers(drop, g, stage):
    rng = np.random.default_rng(8)
    d = Dialogues(True, [2100], 1, 16, seed=9)
    q = dev(rng.normal(size=(2, g, 128)).astype(np.float32), torch.bfloat16)
    lists, lens = np.repeat(d.table_np[:, None, :128], 2, 0), [2048, 2048]
    drop(stage)
    attend(d, q, lists, lens, splits=1, bits=cai.CAI_DEVERR_TIMEOUT)
    drop(-1)
    cai.cai_set_wait_limit_ns(0)
    out, lse = attend(d, q, lists, lens, splits=1)
    check_attend(d, q, lists, lens, out, lse)
