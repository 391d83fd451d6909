"""Appends rotated by positions on several axes, bit for bit against the oracle (whole pools)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int8_mqa_decode_gb300 as cai  # noqa: E402
import oracle  # noqa: E402
from oracle import kv4, pages  # noqa: E402
from test_gpu_kv4 import DEV, _built, dev, flag, host, tables  # noqa: E402,F401

CASES = [  # hkv, hq, page, rot, interleaved, axes, axis of pair i of n, bf16, new tokens, starts
    (1, 8, 16, 128, False, 3, lambda i, n: (i >= 16) + (i >= 40), True, [1, 1, 1], [0, 15, 63]),      # sections of 8s
    (2, 6, 32, 128, True, 3, lambda i, n: i % 3, True, [33, 0, 1, 70], [0, 5, 31, 17]),               # in turn
    (8, 8, 64, 64, False, 4, lambda i, n: 3 - i * 4 // n, False, [1, 2, 130], [63, 62, 0]),           # backwards
    (3, 0, 16, 98, False, 2, lambda i, n: int(i > 20), True, [5, 40], [9, 1]),                        # odd vectors
    (1, 1, 32, 2, True, 4, lambda i, n: 2, True, [16, 17, 15], [16, 15, 1]),                          # one pair
    (4, 4, 64, 128, False, 1, lambda i, n: 0, False, [20, 16], [44, 0]),
    (2, 16, 16, 128, False, 3, lambda i, n: (i * 7 // 5) % 3, False, [48, 3], [16, 2]),               # axes change inside vectors
    (1, 9, 16, 32, True, 3, lambda i, n: i * 3 // n, True, [1 if i % 40 else 230 for i in range(90)], [(i * 7) % 70 for i in range(90)]),
]


def axes_case(four, case, packed, seed=0, odd_tables=False):
    hkv, hq, page, rot, inter, axes, of, bf16, new, start = case
    rng = np.random.default_rng(seed)
    new, start = np.array(new), np.array(start)
    n, half = int(new.sum()), rot // 2
    axis = [of(i, half) for i in range(half)]
    table, num_pages = tables(rng, start + new, page)
    dt = torch.bfloat16 if bf16 else torch.float32
    qkv = dev(rng.normal(size=(n, hq + 2 * hkv, 128)).astype(np.float32) * 3, dt)
    q = qkv[:, :hq] if bf16 else qkv[:, :hq].bfloat16()
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = rng.integers(0, 300, (n, axes)).astype(np.int32)  # unrelated to the slots
    ang = np.arange(300)[:, None] * (1e4 ** (-np.arange(half) / half))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    c, s = dev(cos), dev(sin)
    if odd_tables:  # 4-byte aligned tables
        c, s = (torch.cat((x.new_zeros(1), x.flatten()))[1:].view(x.shape) for x in (c, s))
    cls, bytes_ = (cai.KV4Pool, kv4.page_bytes4(page)) if four else (cai.KVPool, oracle.page_bytes(page))
    pools = [cls(num_pages, page, pages=torch.full((num_pages * bytes_,), 0xA5, dtype=torch.uint8, device=DEV)) for _ in range(hkv)]
    err = flag()
    qo = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device=DEV) if hq else None
    f = cai.cai_kv4_append_axes if four else cai.cai_kv_append_rope_axes
    kw = dict(err_flag=err)
    sh = lambda t: t  # noqa: E731
    if packed:
        kw.update(q_offsets=dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), max_new=int(new.max()))
    else:
        sh = lambda t: t.unflatten(0, (len(new), int(new[0])))  # noqa: E731
    if hq:
        kw.update(q=sh(q), q_out=sh(qo))
    f(pools, sh(k), sh(v), dev(table), dev(start.astype(np.int32)), cai.RopeAxes(c, s, axis, inter), sh(dev(pos)), **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    turn = lambda x: pages.rotate_axes(x, pos, axis, cos, sin, inter)  # noqa: E731
    if hq:
        assert np.array_equal(host(qo), kv4.bf16_round(turn(host(q))))
    kr, vr = turn(host(k)), host(v)
    at = np.concatenate([[0], np.cumsum(new)])
    for j in range(hkv):
        want = np.full(num_pages * bytes_, 0xA5, np.uint8)
        for b in range(len(new)):
            r = slice(at[b], at[b + 1])
            if four:
                (kc, ks), (vc, vs) = kv4.quantize4(kr[r, j]), kv4.quantize4(vr[r, j])
                kv4.write4(want, table[b], int(start[b]), kc, ks, vc, vs, page)
            elif new[b]:
                (kc, ks), (vc, vs) = oracle.quantize_rows(kr[r, j]), oracle.quantize_rows(vr[r, j])
                oracle.pool_write(want, table[b], int(start[b]), kc, ks, vc, vs, page)
        assert np.array_equal(pools[j].pages.cpu().numpy(), want), j


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_axes_packed(four, i):
    axes_case(four, CASES[i], True, seed=i, odd_tables=i % 2 == 1)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n", [1, 19])
def test_axes_equal_counts(four, n):
    axes_case(four, (2, 4, 32, 64, False, 3, lambda i, m: i * 3 // m, True, [n] * 3, [0, 31, 40]), False, seed=7, odd_tables=n == 1)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_equal_positions_are_the_plain_rotation(four, n):
    rng = np.random.default_rng(3)
    table, num_pages = tables(rng, [50, 60], 16)
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    plain, axes = (cai.cai_kv4_append, cai.cai_kv4_append_axes) if four else (cai.cai_kv_append_rope, cai.cai_kv_append_rope_axes)
    k, v = (dev(rng.normal(size=(2, n, 1, 128)).astype(np.float32)) for _ in range(2))
    q = dev(rng.normal(size=(2, n, 4, 128)).astype(np.float32), torch.bfloat16)
    cos, sin = torch.rand(80, 64, device=DEV), torch.rand(80, 64, device=DEV)
    start = np.array([7, 20], np.int32)
    pos = (start[:, None] + np.arange(n))[..., None].repeat(3, -1).astype(np.int32)
    got = []
    for which in range(2):
        pool = cls(num_pages, 16, pages=torch.zeros(num_pages * bytes_, dtype=torch.uint8, device=DEV))
        qo = torch.zeros_like(q)
        if which:
            axes([pool], k, v, dev(table), dev(start), cai.RopeAxes(cos, sin, [i % 3 for i in range(64)]), dev(pos), q=q, q_out=qo)
        else:
            plain([pool], k, v, dev(table), dev(start), rope=cai.Rope(cos, sin), q=q, q_out=qo)
        got.append((pool.pages, qo))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n", [2, 32])
@pytest.mark.parametrize("bad", [-1, 40, 2147483647, -2147483648])
def test_axes_rows_past_the_tables_are_left_out(four, n, bad):
    """A position on any axis, used by a pair or not, that the tables do not have: that row alone is left out."""
    cls, bytes_ = (cai.KV4Pool, 2304) if four else (cai.KVPool, 4224)
    f = cai.cai_kv4_append_axes if four else cai.cai_kv_append_rope_axes
    rope = cai.RopeAxes(torch.ones(40, 64, device=DEV), torch.zeros(40, 64, device=DEV), [0] * 32 + [1] * 32)
    x = torch.ones(1, n, 1, 128, device=DEV)
    q = torch.ones(1, n, 2, 128, dtype=torch.bfloat16, device=DEV)
    table, start = dev(np.array([[1, 0]], np.int32)), torch.zeros(1, dtype=torch.int32, device=DEV)
    clean = cls(2, 16, pages=torch.full((2 * bytes_,), 7, dtype=torch.uint8, device=DEV))
    pos = torch.full((1, n, 3), 39, dtype=torch.int32, device=DEV)
    f([clean], x, x, table, start, rope, pos)
    row = n - 1
    without = cls(2, 16, pages=torch.full((2 * bytes_,), 7, dtype=torch.uint8, device=DEV))
    f([without], x[:, :row], x[:, :row], table, start, rope, pos[:, :row].contiguous())
    for axis in range(3):
        p2 = pos.clone()
        p2[0, row, axis] = bad
        pool = cls(2, 16, pages=torch.full((2 * bytes_,), 7, dtype=torch.uint8, device=DEV))
        err, qo = flag(), torch.full_like(q, 5)
        f([pool], x, x, table, start, rope, p2, q=q, q_out=qo, err_flag=err)
        assert err.item() == cai.CAI_DEVERR_LENGTH
        assert torch.equal(pool.pages, without.pages) and not torch.equal(pool.pages, clean.pages)
        assert (qo[0, row] == 5).all() and (qo[0, :row] == 1).all()


def test_axes_binding_refusals():
    cos = torch.ones(40, 64, device=DEV)
    pool = cai.KVPool(2, 16)
    x = torch.ones(1, 2, 1, 128, device=DEV)
    table, start = dev(np.array([[1, 0]], np.int32)), torch.zeros(1, dtype=torch.int32, device=DEV)
    rope = cai.RopeAxes(cos, cos, [2] * 64)
    pos = torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)
    for bad in (pos[..., :2].contiguous(), pos[0], pos[:, :1].contiguous(), pos.repeat(1, 1, 2)[..., ::2]):
        with pytest.raises(ValueError):
            cai.cai_kv_append_rope_axes([pool], x, x, table, start, rope, bad)
    with pytest.raises(TypeError):
        cai.cai_kv_append_rope_axes([pool], x, x, table, start, rope, pos.long())
    with pytest.raises(TypeError):
        cai.cai_kv_append_rope_axes([pool], x, x, table, start, cai.Rope(cos, cos), pos)
    with pytest.raises(TypeError):
        cai.cai_kv_append_rope([pool], x, x, table, start, rope=rope)
    with pytest.raises(ValueError):
        cai.RopeAxes(cos, cos, [0] * 63)
    with pytest.raises(ValueError):
        cai.RopeAxes(cos, cos, [4] * 64)
    with pytest.raises(cai.CaiError):
        cai.cai_kv_append_rope_axes([pool], x, x, table, start, rope, torch.zeros(1, 2, 5, dtype=torch.int32, device=DEV))
