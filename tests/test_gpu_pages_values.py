"""int8 attention over lists: values of very different size, and zeros, in one list.

The bounds are those of test_gpu_pages.py: neither the sizes of the values nor their order enters them but by the
largest value and, for lse, by the logarithm of V's scales."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
from test_gpu_kv4 import DEV, _built, dev  # noqa: E402,F401
from test_gpu_pages import Dialogues, attend, check_attend  # noqa: E402


def dialogue(k, v):
    """One sequence of the given keys and values fp32 [n][128] in an int8 cache, pages of 16."""
    n = len(k)
    d = Dialogues(False, [n], 1, 16, seed=1)
    cai.cai_kv_append_rope(d.pools, dev(k)[None, :, None], dev(v)[None, :, None], d.table,
                           torch.zeros(1, dtype=torch.int32, device=DEV))
    d.k, d.v = [[d.stored(k)]], [[d.stored(v)]]
    return d


def check(k, v, g, splits=(0, 1), scale=1.0 / 128, rng=None):
    d = dialogue(k, v)
    q = np.ones((1, g, 128)) if rng is None else rng.normal(size=(1, g, 128))
    q = dev(q.astype(np.float32), torch.bfloat16)
    for s in splits:
        out, lse = attend(d, q, d.table_np[:, None], [len(k)], scale=scale, splits=s)
        check_attend(d, q, d.table_np[:, None], [len(k)], out, lse, scale=scale)


def sized(rng, n, exponents):
    """Values fp32 [n][128] whose largest is 2^e to 2^(e + 0.6) (0 for an e of -inf)."""
    v = rng.uniform(-1, 1, (n, 128))
    v /= np.abs(v).max(1, keepdims=True)
    return (v * np.exp2(exponents + rng.uniform(0, 0.6, n))[:, None]).astype(np.float32)


@pytest.mark.parametrize("g", [4, 32, 64])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("most", [10, 33.5, 50, 90, 126])
def test_zeros_beside_large_values(g, first, most):
    """Tiles of zero vectors before, or after, one large value, their logits above it, equal and below."""
    rng = np.random.default_rng(5)
    for n, at in ((129, 128), (400, 300), (400, 399)):
        e = np.full(n, -np.inf)
        e[at] = most
        for above in (-12.0, 0.0, 11.0, 60.0):  # (logits: powers of e)
            k = np.zeros((n, 128), np.float32)
            k[np.isinf(e)] = above
            v = sized(rng, n, e)
            check(*((k, v) if first else (k[::-1].copy(), v[::-1].copy())), g)


@pytest.mark.parametrize("g", [4, 32, 64])
@pytest.mark.parametrize("spread", [20, 70, 120, 210])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_values_of_every_size(g, spread, order):
    """Sizes over 2^spread, tile by tile and within tiles, some vectors zero, random logits."""
    rng = np.random.default_rng(6)
    n = 700
    e = np.linspace(-min(spread / 2, 85), spread - min(spread / 2, 85), n)
    e = e if order == "rising" else e[::-1] if order == "falling" else rng.permutation(e)
    e = np.where(rng.random(n) < 0.1, -np.inf, e)
    check(rng.normal(size=(n, 128)).astype(np.float32) * 3, sized(rng, n, e), g, splits=(0, 1, 3), scale=128 ** -0.5, rng=rng)


@pytest.mark.parametrize("g", [4, 32, 64])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -92])
def test_long_lists_of_the_smallest_values(g, size):
    """20000 tokens whose weights over V's scale, 2^-100 at least, are as large as they get: 2^7 in the first tile and
    2^7.8 times that in all others."""
    rng = np.random.default_rng(7)
    k = np.zeros((32, 128), np.float32)
    k[16:] = 5.4  # (logit: a power of e)
    d = dialogue(k, (rng.uniform(0.9, 1.0, (32, 128)) * size).astype(np.float32))
    lists = np.repeat(d.table_np[0, [0, 1]], [8, 1242])[None, None]
    q = dev(np.ones((1, g, 128), np.float32), torch.bfloat16)
    for splits in (1, 2):
        out, lse = attend(d, q, lists, [20000], scale=1.0 / 128, splits=splits)
        check_attend(d, q, lists, [20000], out, lse, scale=1.0 / 128)
