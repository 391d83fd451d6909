"""Cases of the cache operators: rotated appends into the int8 and the 4-bit paged cache, reading
cached rows back as values, and decode and prefill attention over the 4-bit cache.

`run` computes a case in plain torch (`own = False`) or through the library (`own = True`).
The 4-bit cache's arithmetic: a token's K (and V) vector of 128 channels is four groups of 32;
a group's scale is its largest magnitude / 7, rounded to bf16 and then to fp16 (at most 9344);
a code is round-half-even(x / scale) clamped to [-7, 7], and stands for code * scale.
"""
import math

import numpy as np
import torch

own = False

D = 128            # head_dim
BLOCK = 2304       # bytes of 16 tokens in the 4-bit cache
DEV = "cuda"
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step of a small dialogue server: four sequences, MQA, bf16 projections.
        dict(name="append8_step", op="append8", batch=4, n=1, ragged=False, hq=8, hkv=1, page=16, lo=64, hi=512,
             rot=128, inter=False, bf16=True),
        # A chunk of a reused dialogue prefix, its q, k and v slices of one fused projection.
        dict(name="append8_chunk", op="append8", batch=16, n=256, ragged=False, hq=32, hkv=1, page=16, lo=8192,
             hi=8192, rot=128, inter=False, bf16=True),
        # A decode step of a full batch with grouped heads, half of the channels rotated, fp32 inputs.
        dict(name="append4_step", op="append4", batch=256, n=1, ragged=False, hq=32, hkv=8, page=16, lo=256, hi=32768,
             rot=64, inter=True, bf16=False),
        # Continuous batching: sequences bring 0 to 400 tokens each.
        dict(name="append4_ragged", op="append4", batch=48, n=400, ragged=True, hq=32, hkv=2, page=64, lo=1, hi=9000,
             rot=128, inter=False, bf16=True),
        # Dialogues leaving the int8 cache for another format.
        dict(name="read8_dialogues", op="read8", batch=16, n=4096, ragged=True, hq=1, hkv=1, page=16, lo=0, hi=512,
             bf16=False),
        # A batch's last thousand tokens for an attention the library does not have.
        dict(name="read4_batch", op="read4", batch=64, n=1024, ragged=True, hq=1, hkv=4, page=32, lo=0, hi=4000,
             bf16=True),
        # The smallest decode step, where latency counts.
        dict(name="decode4_small", op="decode4", batch=4, hq=8, hkv=1, page=16, lo=64, hi=512, spread="uniform",
             window=0),
        # The global layer of a hybrid step: lognormal contexts.
        dict(name="decode4_hybrid", op="decode4", batch=256, hq=32, hkv=1, page=16, lo=256, hi=32768,
             spread="lognormal", window=0),
        # Grouped heads, medium contexts.
        dict(name="decode4_grouped", op="decode4", batch=96, hq=64, hkv=8, page=32, lo=256, hi=16384,
             spread="uniform", window=0),
        # Long contexts, 64 heads on one K/V head.
        dict(name="decode4_long", op="decode4", batch=64, hq=64, hkv=1, page=64, lo=16384, hi=131072,
             spread="uniform", window=0),
        # New turns on a reused prefix.
        dict(name="prefill4_chunk", op="prefill4", batch=16, n=256, ragged=False, hq=32, hkv=1, page=16, lo=8192,
             hi=8192, window=0),
        # A mixed step of a local layer: decode rows beside chunks, grouped heads.
        dict(name="prefill4_mixed", op="prefill4", batch=40, n=300, ragged=True, hq=32, hkv=4, page=32, lo=0, hi=6000,
             window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "append4", "read8", "read4", "decode4", "decode4", "prefill4", "prefill4"])
    page = rng.choice([16, 32, 64])
    if op == "decode4":
        hkv = rng.choice([1, 1, 2, 4, 8])
        g = rng.choice([1, 3, 4, 5, 8, 12, 16, 24, 32, 40, 64])
        hi = _log(rng, 20, 131072)
        batch = max(1, min(_log(rng, 1, 256), 5_000_000 // (hi * hkv)))
        return dict(op=op, batch=batch, hq=g * hkv, hkv=hkv, page=page, lo=rng.randint(0, hi), hi=hi,
                    spread=rng.choice(["uniform", "lognormal"]), window=rng.choice([0, 0, 0, 1024, rng.randint(1, 2000)]))
    if op == "prefill4":
        hkv = rng.choice([1, 2, 4])
        g = rng.choice([1, 2, 4, 8, 16, 32])
        n = _log(rng, 2, 500)
        hi = _log(rng, 1, 8192)
        most = 16 * 256 * 32 * 8192  # the largest listed case's (row, key) pairs
        batch = max(1, min(_log(rng, 1, 48), most // (n * g * hkv * (hi + n))))
        return dict(op=op, batch=batch, n=n, ragged=rng.random() < 0.5, hq=g * hkv, hkv=hkv, page=page, lo=rng.randint(0, hi),
                    hi=hi, window=rng.choice([0, 0, 1024, rng.randint(1, 2000)]))
    hkv = rng.choice([1, 2, 4, 8])
    n = rng.choice([1, 1, _log(rng, 2, 1000)])
    hi = _log(rng, 1, 30000)
    batch = max(1, min(_log(rng, 1, 256), 16384 // (n * hkv)))
    case = dict(op=op, batch=batch, n=n, ragged=n > 1 and rng.random() < 0.5, hq=hkv * rng.choice([1, 4, 8]), hkv=hkv,
                page=page, lo=rng.randint(0, hi), hi=hi, bf16=rng.random() < 0.5)
    if op.startswith("append"):
        case.update(rot=rng.choice([128, 128, 64, 32, 98, 2]), inter=rng.random() < 0.5)
    return case


# ----------------------------------------------------------------------------------- inputs

def _lengths(case):
    """Context (or prefix) lengths: the case alone gives them, a seed their order."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    rng = np.random.default_rng(7)
    if case.get("spread") == "lognormal":
        x = np.exp(rng.normal(math.log(max(1.0, hi / 8)), 1.0, b))
        return np.clip(x, lo, hi).astype(np.int64)
    return rng.integers(lo, hi + 1, b).astype(np.int64)


def _new(case):
    """New tokens of every sequence, likewise."""
    b, n = case["batch"], case["n"]
    if not case["ragged"]:
        return np.full(b, n, dtype=np.int64)
    rng = np.random.default_rng(8)
    new = rng.integers(0, n + 1, b)
    new[rng.random(b) < 0.3] = 1  # decode rows beside the chunks
    new[0] = n
    return new.astype(np.int64)


def _tables(lengths, page, rng):
    """A block table [batch][max pages] over a shuffled pool; unused entries are -1."""
    pages = -(-lengths // page)
    total, most = int(pages.sum()), max(1, int(pages.max()))
    perm, table, at = rng.permutation(max(1, total)).astype(np.int32), np.full((len(lengths), most), -1, np.int32), 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += int(k)
    return torch.from_numpy(table).to(DEV), max(1, total)


def _cache4(hkv, num_pages, page, gen):
    """Filled 4-bit pools [hkv][bytes]: near-normal codes, scales of unit-size keys and values with some larger groups."""
    blocks = hkv * num_pages * (page // 16)
    pool = torch.empty(blocks, BLOCK, dtype=torch.uint8, device=DEV)
    step = 1 << 16
    for a in range(0, blocks, step):
        n = min(step, blocks - a)
        x = torch.randn(n, 2048, 2, device=DEV, generator=gen).mul_(2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        pool[a:a + n, :2048] = x[..., 0] | (x[..., 1] << 4)
        s = torch.randn(n, 128, device=DEV, generator=gen).mul_(0.35).exp_().mul_(0.3)
        pool[a:a + n, 2048:] = s.to(torch.bfloat16).to(torch.float16).view(torch.uint8)
    return pool.view(hkv, -1)


def _cache8(hkv, num_pages, page, gen):
    """Filled int8 pools [hkv][bytes]."""
    num_pages *= hkv
    pool = torch.empty(num_pages, page * 264, dtype=torch.uint8, device=DEV)
    x = torch.randn(num_pages, page * 256, device=DEV, generator=gen).mul_(40).round_().clamp_(-127, 127)
    pool[:, :page * 256] = x.to(torch.int8).view(torch.uint8)
    s = torch.randn(num_pages, page * 2, device=DEV, generator=gen).mul_(0.2).exp_().mul_(0.025)
    pool[:, page * 256:] = s.view(torch.uint8)
    return pool.view(hkv, -1)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, b, page, hq, hkv = case["op"], case["batch"], case["page"], case["hq"], case["hkv"]
    before = rng.permutation(_lengths(case))
    st = dict(case=case)
    if op == "decode4":
        st["ctx"] = before
        st["table"], pages = _tables(before, page, rng)
        st["arena"] = _cache4(hkv, pages, page, gen)  # one pool per K/V head
        st["len"] = torch.from_numpy(before.astype(np.int32)).to(DEV)
        st["q"] = (torch.randn(b, hq, D, device=DEV, generator=gen) * 1.5).to(torch.bfloat16)
        return st
    new = rng.permutation(_new(case))
    st["before"], st["new"] = before, new
    st["rows"] = int(new.sum())
    st["table"], pages = _tables(before + new, page, rng)
    st["start"] = torch.from_numpy(before.astype(np.int32)).to(DEV)
    st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
    st["arena"] = (_cache8 if op.endswith("8") else _cache4)(hkv, pages, page, gen)
    if op == "prefill4":
        st["q"] = (torch.randn(st["rows"], hq, D, device=DEV, generator=gen) * 1.5).to(torch.bfloat16)
    elif op.startswith("append"):
        # One fused projection [rows][hq + 2 hkv][128]: q, k and v are its slices; some channels are large.
        qkv = torch.randn(st["rows"], hq + 2 * hkv, D, device=DEV, generator=gen)
        qkv[:, hq:hq + hkv] *= torch.where(torch.rand(D, device=DEV, generator=gen) < 0.05, 6.0, 1.0)
        dt = torch.bfloat16 if case["bf16"] else torch.float32
        st["qkv"] = qkv.to(dt)
        st["q"] = st["qkv"][:, :hq] if case["bf16"] else qkv[:, :hq].to(torch.bfloat16).contiguous()
        st["k"], st["v"] = st["qkv"][:, hq:hq + hkv], st["qkv"][:, hq + hkv:]
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        ang = torch.arange(int((before + new).max()) + 1, device=DEV, dtype=torch.float64)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    return st


# -------------------------------------------------------------------------------- plain form

def _rows(st):
    """Sequence and position of every new row, on the device."""
    off = st["offsets"].long()
    i = torch.arange(st["rows"], device=DEV)
    seq = torch.searchsorted(off, i, right=True) - 1
    return seq, st["start"].long()[seq] + i - off[seq]


def _rotate(x, st, pos):
    """Rotation of channels [0, rot) in fp32, every product and the sum rounded on its own."""
    rot, half = st["case"]["rot"], st["case"]["rot"] // 2
    c, s = st["cos"][pos][:, None], st["sin"][pos][:, None]
    y = x.float().clone()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if st["case"]["inter"] else (y[..., :half], y[..., half:rot])
    lo, hi = a * c - b * s, b * c + a * s
    if st["case"]["inter"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = lo, hi
    else:
        y[..., :half], y[..., half:rot] = lo, hi
    return y


def _codes4(x):
    """fp32 [..., 128] -> codes (float), scales fp16 [..., 4]."""
    g = x.unflatten(-1, (4, 32))
    amax = g.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).to(torch.bfloat16).clamp(max=9344.0).to(torch.float16)
    sf = s.float()[..., None]
    c = torch.where(sf > 0, (g / torch.where(sf > 0, sf, torch.ones_like(sf))).round().clamp(-7, 7), torch.zeros_like(g))
    return c.flatten(-2), s


def _codes8(x):
    amax = x.abs().amax(-1, keepdim=True)
    s = amax / torch.full_like(amax, 127.0)
    c = torch.where(s > 0, (x / torch.where(s > 0, s, torch.ones_like(s))).round().clamp(-127, 127), torch.zeros_like(x))
    return c, s


def _write4(pools, page_id, slot, page, k, v):
    """Writes rows k, v fp32 [rows][heads][128] into their slots and returns the values they stand for."""
    heads = torch.arange(len(pools), device=DEV)
    blk, r = (page_id * (page // 16) + slot // 16)[:, None], (slot % 16)[:, None]
    t, hb, e = (r % 8) // 2, r // 8, r % 2
    kc, ks = _codes4(k)
    vc, vs = _codes4(v)
    p = pools.view(len(pools), -1, BLOCK)
    # K: word (t, j) of a token's 64 bytes holds channels 32 j + 8 t + 2 i + e at bits 4 i + 16 e.
    c = (kc + 8).to(torch.uint8).unflatten(-1, (4, 4, 4, 2)).permute(0, 1, 3, 2, 5, 4)  # [row, head, t, j, e, i]
    b = c[..., 0::2] | (c[..., 1::2] << 4)                                              # bytes [..., t, j, e, i / 2]
    p[..., :1024].unflatten(2, (16, 64))[heads, blk, r] = b.flatten(2)
    # V: a token's byte of word (h, g, t, w) holds channels 16 (4 h + w) + g and + 8.
    c = (vc + 8).to(torch.uint8).unflatten(-1, (2, 4, 2, 8))                            # [..., h, w, half, g]
    b = (c[..., 0, :] | (c[..., 1, :] << 4)).transpose(-1, -2)                          # [..., h, g, w]
    p[..., 1024:2048].unflatten(2, (2, 8, 4, 4, 4)).permute(0, 1, 4, 6, 2, 3, 5)[heads, blk, t, hb + 2 * e] = b
    sc = p[..., 2048:].view(torch.float16)
    sc[..., :64].unflatten(2, (16, 4))[heads, blk, r] = ks
    sc[..., 64:].unflatten(2, (4, 2, 4, 2)).permute(0, 1, 2, 3, 5, 4)[heads, blk, t, hb, e] = vs
    up = lambda c, s: (c.unflatten(-1, (4, 32)) * s.float()[..., None]).flatten(-2)  # noqa: E731
    return up(kc, ks), up(vc, vs)


def _write8(pools, page_id, slot, page, k, v):
    heads = torch.arange(len(pools), device=DEV)
    page_id, slot = page_id[:, None], slot[:, None]
    kc, ks = _codes8(k)
    vc, vs = _codes8(v)
    p = pools.view(len(pools), -1, page * 264)
    p[..., :page * D].unflatten(2, (page, D))[heads, page_id, slot] = kc.to(torch.int8).view(torch.uint8)
    p[..., page * D:page * 256].unflatten(2, (D, page)).transpose(2, 3)[heads, page_id, slot] = vc.to(torch.int8).view(torch.uint8)
    sc = p[..., page * 256:].view(torch.float32)
    sc[heads, page_id, slot] = ks[..., 0]
    sc[heads, page_id, page + slot] = vs[..., 0]
    return kc * ks, vc * vs


def _values4(blocks):
    """4-bit blocks uint8 [..., 2304] -> the K and V values fp32 [..., 16, 128] that they stand for."""
    shape, blocks = blocks.shape[:-1], blocks.reshape(-1, BLOCK)
    n = blocks.shape[0]
    sc = blocks[:, 2048:].contiguous().view(torch.float16).float()
    kb = blocks[:, :1024].reshape(n, 16, 4, 4, 2, 2)                   # [row, t, j, e, i / 2]
    k = torch.stack((kb & 15, kb >> 4), -1).float() - 8                # [..., e, i / 2, i % 2]
    k = k.flatten(5).permute(0, 1, 3, 2, 5, 4).reshape(n, 16, 4, 32)   # [row, j, t, i, e]
    k = k * sc[:, :64].view(n, 16, 4, 1)
    vb = blocks[:, 1024:2048].reshape(n, 2, 8, 4, 4, 2, 2)             # [h, g, t, w, e, hb]
    v = torch.stack((vb & 15, vb >> 4), -1).float() - 8                # [..., half]
    v = v.permute(0, 6, 3, 5, 1, 4, 7, 2).reshape(n, 2, 4, 2, 4, 32)   # [hb, t, e, h w half g]: group = channel / 32
    v = v * sc[:, 64:].view(n, 4, 2, 4, 2).permute(0, 2, 1, 4, 3)[..., None]
    return k.reshape(*shape, 16, D), v.reshape(*shape, 16, D)


def _attend(c, q, k, v, pos, live, rows_pos):
    """Attention of q [B][n][hq][128] over k, v [B][hkv][S][128] at positions pos [B][S] (live: which exist)."""
    b, n, hq, hkv = q.shape[0], q.shape[1], c["hq"], c["hkv"]
    ok = live[:, None] & (pos[:, None] <= rows_pos[..., None])
    if c["window"]:
        ok &= pos[:, None] > rows_pos[..., None] - c["window"]
    qg = q.float().view(b, n, hkv, hq // hkv, D).transpose(1, 2).flatten(2, 3)
    z = (qg @ k.transpose(2, 3)).mul_(SCALE).unflatten(2, (n, hq // hkv))
    z.masked_fill_(~ok[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    z.sub_(m).exp_()
    s = z.sum(-1, keepdim=True)
    o = (z.flatten(2, 3) @ v).view(b, hkv, n, hq // hkv, D) / torch.where(s > 0, s, torch.ones_like(s))
    lse = (m + s.log())[..., 0]
    return o.transpose(1, 2).reshape(b, n, hq, D).to(torch.bfloat16), lse.transpose(1, 2).reshape(b, n, hq)


def _gather4(st, first, count):
    """K and V of cache blocks [first, first + count) of every sequence, [B][hkv][count * 16][128]."""
    per = st["case"]["page"] // 16
    blk = first[:, None] + torch.arange(count, device=DEV)
    pages = st["table"].long().gather(1, (blk // per).clamp(max=st["table"].shape[1] - 1)).clamp(min=0)
    arena = st["arena"].view(len(st["arena"]), -1, BLOCK)
    heads = torch.arange(len(arena), device=DEV)[:, None]
    k, v = _values4(arena[heads, (pages * per + blk % per)[:, None]])  # [B][hkv][count][2304]
    return k.flatten(2, 3), v.flatten(2, 3)


def _plain(st):
    c = st["case"]
    op, page = c["op"], c["page"]
    if op == "decode4":
        length = st["len"].long()
        first = (length - c["window"]).clamp(min=0) // 16 if c["window"] else torch.zeros_like(length)
        most = int(min(c["window"] + 31, st["ctx"].max()) if c["window"] else st["ctx"].max())
        count = max(1, -(-most // 16))
        pos = first[:, None] * 16 + torch.arange(count * 16, device=DEV)
        k, v = _gather4(st, first, count)
        out, lse = _attend(c, st["q"][:, None], k, v, pos, pos < length[:, None], length[:, None] - 1)
        return {"out": out[:, 0], "lse": lse[:, 0]}
    seq, at = _rows(st)
    page_id, slot = st["table"].long()[seq, at // page], at % page
    if op == "prefill4":
        n = int(st["new"].max())
        i = at - st["start"].long()[seq]
        q = torch.zeros(c["batch"], n, c["hq"], D, device=DEV, dtype=torch.bfloat16)
        q[seq, i] = st["q"]
        end = st["start"].long() + (st["offsets"][1:] - st["offsets"][:-1])
        count = max(1, -(-int((st["before"] + st["new"]).max()) // 16))
        pos = torch.arange(count * 16, device=DEV).expand(c["batch"], -1)
        k, v = _gather4(st, torch.zeros_like(end), count)
        out, lse = _attend(c, q, k, v, pos, pos < end[:, None], st["start"].long()[:, None] + torch.arange(n, device=DEV))
        return {"out": out[seq, i], "lse": lse[seq, i]}
    arena = st["arena"]
    heads = torch.arange(len(arena), device=DEV)
    if op.startswith("read"):
        page_id, slot = page_id[:, None], slot[:, None]
        if op == "read4":
            k, v = _values4(arena.view(len(arena), -1, BLOCK)[heads, page_id * (page // 16) + slot // 16])
            r = (slot % 16)[..., None, None].expand(-1, len(arena), 1, D)
            k, v = k.gather(2, r)[:, :, 0], v.gather(2, r)[:, :, 0]
        else:
            p = arena.view(len(arena), -1, page * 264)
            sc = p[..., page * 256:].view(torch.float32)
            k = p[..., :page * D].view(torch.int8).unflatten(2, (page, D))[heads, page_id, slot].float()
            v = p[..., page * D:page * 256].view(torch.int8).unflatten(2, (D, page)).transpose(2, 3)[heads, page_id, slot].float()
            k, v = k * sc[heads, page_id, slot][..., None], v * sc[heads, page_id, page + slot][..., None]
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        return {"k": k.to(dt), "v": v.to(dt)}
    write = _write4 if op == "append4" else _write8
    k, v = write(arena, page_id, slot, page, _rotate(st["k"], st, at), st["v"].float())
    return {"q": _rotate(st["q"], st, at).to(torch.bfloat16), "k": k, "v": v}


# --------------------------------------------------------------------------- the library's calls

def _own(st):
    import int8_mqa_decode_gb300 as cai
    c = st["case"]
    op, b = c["op"], c["batch"]
    if "handles" not in st:  # what a program keeps: pool handles, the rotation's tables, a workspace
        pool = cai.KVPool if op.endswith("8") else cai.KV4Pool
        bytes_ = cai.cai_page_bytes(c["page"]) if op.endswith("8") else cai.cai_kv4_page_bytes(c["page"])
        st["handles"] = [pool(p.numel() // bytes_, c["page"], pages=p) for p in st["arena"]]
        most = st["table"].shape[1]
        if op.startswith("append"):
            st["rope"] = cai.Rope(st["cos"], st["sin"], interleaved=c["inter"])
        elif op == "decode4":
            st["ws"] = torch.empty(cai.cai_kv4_decode_workspace_size(b, c["hq"], c["hkv"], most, c["page"], c["window"]),
                                   dtype=torch.uint8, device=DEV)
        elif op == "prefill4":
            st["ws"] = torch.empty(cai.cai_kv4_prefill_workspace_size(b, c["hq"], c["hkv"], most, c["page"]),
                                   dtype=torch.uint8, device=DEV)
    pools = st["handles"]
    if op == "decode4":
        out = torch.empty(b, c["hq"], D, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(b, c["hq"], dtype=torch.float32, device=DEV)
        cai.cai_kv4_decode(pools, st["q"], st["table"], st["len"], c["window"], SCALE, 0, st["ws"], out, lse)
        return {"out": out, "lse": lse}
    n = st["rows"]
    if c["ragged"]:
        packed = dict(q_offsets=st["offsets"], max_new=c["n"])
        shape = lambda x: x  # noqa: E731
    else:
        packed = {}
        shape = lambda x: x.unflatten(0, (b, c["n"]))  # noqa: E731
    if op == "prefill4":
        out = torch.empty(n, c["hq"], D, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(n, c["hq"], dtype=torch.float32, device=DEV)
        cai.cai_kv4_prefill(pools, shape(st["q"]), st["table"], st["start"], c["window"], SCALE, st["ws"], shape(out),
                            shape(lse), **packed)
        return {"out": out, "lse": lse}
    read = cai.cai_kv_read if op.endswith("8") else cai.cai_kv4_read
    dt = torch.bfloat16 if c["bf16"] and op.startswith("read") else torch.float32
    k = torch.empty(n, c["hkv"], D, dtype=dt, device=DEV)
    v = torch.empty_like(k)
    if op.startswith("read"):
        read(pools, shape(k), shape(v), st["table"], st["start"], **packed)
        return {"k": k, "v": v}
    append = cai.cai_kv_append_rope if op == "append8" else cai.cai_kv4_append
    q = torch.empty(n, c["hq"], D, dtype=torch.bfloat16, device=DEV)
    append(pools, shape(st["k"]), shape(st["v"]), st["table"], st["start"], rope=st["rope"], q=shape(st["q"]),
           q_out=shape(q), **packed)
    read(pools, shape(k), shape(v), st["table"], st["start"], **packed)  # what the cache now stands for
    return {"q": q, "k": k, "v": v}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: cached tokens, inputs and block-table entries read once, outputs written once."""
    c, op, page, hkv, hq = case, case["op"], case["page"], case["hkv"], case["hq"]
    token = 264 if op.endswith("8") else 144
    before = _lengths(c)
    if op == "decode4":
        keys = float((np.minimum(before, c["window"]) if c["window"] else before).sum())
        io = c["batch"] * hq * (2 * D + 2 * D + 4) + 4 * keys / page
        return {"bytes": keys * hkv * token + io, "flops": 4 * D * keys * hq}
    new = _new(c)
    rows = float(new.sum())
    if op == "prefill4":
        # Every row attends its prefix and the chunk up to itself, at most the window.
        seen = [np.arange(p + 1, p + n + 1) for p, n in zip(before, new)]
        pairs = float(sum((np.minimum(x, c["window"]) if c["window"] else x).sum() for x in seen))
        keys = float(sum(min(p + n, c["window"] + n - 1) if c["window"] else p + n for p, n in zip(before, new) if n))
        io = rows * hq * (2 * D + 2 * D + 4) + 4 * keys / page
        return {"bytes": keys * hkv * token + io, "flops": 4 * D * pairs * hq}
    wide = 2 if c["bf16"] else 4
    if op.startswith("read"):
        return {"bytes": rows * (hkv * (token + 2 * D * wide) + 4 / page), "flops": rows * hkv * 2 * D}
    # k, v in; cache bytes and the values they stand for out; q in and out; a row of each table.
    bytes_ = rows * (hkv * (2 * D * wide + token + 2 * D * 4) + hq * D * 4 + c["rot"] * 4)
    return {"bytes": bytes_, "flops": rows * (hkv * 8 * D + hq * 3 * D)}


# ------------------------------------------------------------------------------------ exact

def _exact_rotation(x, pos, cos, sin, inter, rounded):
    """x float64 [rows][heads][128]; `rounded`: every product and sum to fp32, as the operator is defined."""
    f = (lambda a: a.astype(np.float32).astype(np.float64)) if rounded else (lambda a: a)
    y = x.copy()
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, s = cos[pos, i][:, None], sin[pos, i][:, None]
        y[:, :, a] = f(f(x[:, :, a] * c) - f(x[:, :, b] * s))
        y[:, :, b] = f(f(x[:, :, b] * c) + f(x[:, :, a] * s))
    return y


def _exact_values(x, bits):
    """What the cache stands for after an append of x float64 [rows][heads][128]."""
    f32 = lambda a: a.astype(np.float32)  # noqa: E731
    top, size = (7, 32) if bits == 4 else (127, D)
    out = np.zeros_like(x)
    for a in range(0, D, size):
        g = x[..., a:a + size]
        s = f32(np.abs(g).max(-1) / top)
        if bits == 4:
            s = torch.from_numpy(np.ascontiguousarray(s)).bfloat16().float().numpy()
            s = np.minimum(s, 9344.0).astype(np.float16)
        s = s.astype(np.float64)[..., None]
        code = np.clip(np.rint(f32(np.divide(g, s, out=np.zeros_like(g), where=s > 0))), -top, top)
        out[..., a:a + size] = code * s
    return out


def _exact_cached(pool, page, page_id, slot, bits):
    """K, V float64 [rows][128] of single tokens, by the byte that each code stands in."""
    ch = torch.arange(D, device=DEV)
    base = page_id.long()[:, None] * (page * (264 if bits == 8 else 144))
    slot = slot[:, None]
    if bits == 8:
        k, v = pool[base + slot * D + ch].view(torch.int8), pool[base + page * D + ch * page + slot].view(torch.int8)
        words = pool.view(torch.float32)
        at = base // 4 + page * 64 + slot
        return k.double() * words[at].double(), v.double() * words[at + page].double()
    base = base + (slot // 16) * BLOCK
    r = slot % 16
    bit = 4 * (ch % 8 // 2) + 16 * (ch % 2)
    k = (pool[base + r * 64 + (ch % 32 // 8) * 16 + (ch // 32) * 4 + bit // 8] >> (bit % 8)) & 15
    m, g, up = ch // 16, ch % 8, ch % 16 // 8
    t, hb, e = r % 8 // 2, r // 8, r % 2
    v = (pool[base + 1024 + (((m // 4) * 32 + g * 4 + t) * 4 + m % 4) * 4 + hb + 2 * e] >> (4 * up)) & 15
    half = pool.view(torch.float16)
    ks = half[(base + 2048) // 2 + r * 4 + ch // 32]
    vs = half[(base + 2176) // 2 + t * 16 + hb * 8 + (ch // 32) * 2 + e]
    return (k.double() - 8) * ks.double(), (v.double() - 8) * vs.double()


def exact(case, seed):
    st = prepare(case, seed)
    c, op, page, hkv, hq = case, case["op"], case["page"], case["hkv"], case["hq"]
    bits = 8 if op.endswith("8") else 4
    table = st["table"]
    if op in ("decode4", "prefill4"):
        start = st["ctx"] - 1 if op == "decode4" else st["before"]  # position of the first query row
        new = np.ones(c["batch"], np.int64) if op == "decode4" else st["new"]
        out = torch.zeros(int(new.sum()), hq, D, dtype=torch.float64, device=DEV)
        lse = torch.full((len(out), hq), -math.inf, dtype=torch.float64, device=DEV)
        q, row = st["q"].double(), 0
        for b in range(c["batch"]):
            n, p0 = int(new[b]), int(start[b])
            rows, row = slice(row, row + n), row + n
            if n == 0 or p0 < 0:
                continue
            lo = max(0, p0 + 1 - c["window"]) if c["window"] else 0
            key = torch.arange(lo, p0 + n, device=DEV)
            at = torch.arange(p0, p0 + n, device=DEV)[:, None]
            seen = key <= at
            if c["window"]:
                seen = seen & (key > at - c["window"])
            for j in range(hkv):
                k, v = _exact_cached(st["arena"][j], page, table[b, key // page], key % page, 4)
                step = max(1, 200_000_000 // (n * len(key)))
                for h in range(j * hq // hkv, (j + 1) * hq // hkv, step):
                    hs = slice(h, min(h + step, (j + 1) * hq // hkv))
                    s = torch.einsum("nhd,kd->hnk", q[rows, hs], k) * SCALE
                    s = torch.where(seen, s, torch.full((), -math.inf, dtype=torch.float64, device=DEV))
                    lse[rows, hs] = torch.logsumexp(s, -1).T
                    out[rows, hs] = torch.einsum("hnk,kd->nhd", torch.softmax(s, -1), v)
        return {"out": out, "lse": lse}
    seq = np.repeat(np.arange(c["batch"]), st["new"])
    pos = np.concatenate([p + np.arange(n) for p, n in zip(st["before"], st["new"])])
    if op.startswith("read"):
        at = torch.from_numpy(pos).to(DEV)
        pid = table[torch.from_numpy(seq).to(DEV), at // page]
        kv = [_exact_cached(p, page, pid, at % page, bits) for p in st["arena"]]
        return {"k": torch.stack([x for x, _ in kv], 1), "v": torch.stack([x for _, x in kv], 1)}
    cos, sin = (st[x].cpu().numpy().astype(np.float64) for x in ("cos", "sin"))
    wide = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    return {"q": _exact_rotation(wide(st["q"]), pos, cos, sin, c["inter"], False),
            "k": _exact_values(_exact_rotation(wide(st["k"]), pos, cos, sin, c["inter"], True), bits),
            "v": _exact_values(wide(st["v"]), bits)}
