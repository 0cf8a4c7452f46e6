"""The block-scaled cache on the GPU: the producer bit for bit against its fp32 definition, reading back exactly, decode
and chunk attention per element against fp64 within derived bounds (tests/block_helpers.py)."""
import numpy as np
import pytest
import torch

import int8_kv_cache_token_gb300 as i8
from tests.block_helpers import BS, Cache, attend, bf16, tables

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(a):
    return dev(np.asarray(a, np.float32)).to(torch.bfloat16)


def upload(c):
    return dict(k_cache=dev(c.paged("k")), v_cache=dev(c.paged("v")), k_scale=dev(c.scale["k"]), v_scale=dev(c.scale["v"]))


def same_cache(g, c):
    for w in "kv":
        assert np.array_equal(g[w + "_scale"].cpu().numpy(), c.scale[w])
        assert np.array_equal(g[w + "_cache"].cpu().numpy(), c.paged(w))


def cu_of(news):
    return dev(np.cumsum([0] + list(news)).astype(np.int32))


def close(out, ref, err, is16):
    out = out.float().cpu().numpy().astype(np.float64)
    tol = err + (2.0 ** -8 if is16 else 2.0 ** -24) * np.abs(ref) + 1e-30
    worst = (np.abs(out - ref) / tol).max()
    assert np.isfinite(out).all() and worst <= 1, f"{worst:.3g} times the bound, max-abs {np.abs(out - ref).max():.3g}"


# ------------------------------------------------------------------------------------------------- producer
@pytest.mark.parametrize("D, Hkv", [(64, 3), (128, 8), (256, 4)])
@pytest.mark.parametrize("lens, news", [
    ([1], [1]), ([16], [16]), ([17, 33, 5], [17, 2, 5]), ([40, 31, 64, 100], [7, 31, 16, 1]), ([50, 20], [0, 20]),
    ([300], [290]), ([15, 16, 17, 18], [2, 2, 2, 2])])
def test_write_bit_exact(D, Hkv, lens, news):
    rng = np.random.default_rng(D + sum(lens))
    table, nb = tables(rng, lens)
    c = Cache(nb, Hkv, D).random(rng)
    T = sum(news)
    x = {w: bf16(rng.standard_normal((T, Hkv, D)) * np.exp2(rng.integers(-6, 7, (T, Hkv, 1)))) for w in "kv"}
    x["k"][0, 0] = 0
    g = upload(c)
    i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), dev(np.int32(lens)), dev(table), **g, cu_tokens=cu_of(news))
    c.write(x, lens, news, table)
    same_cache(g, c)
    assert i8.device_error() == 0


@pytest.mark.parametrize("D", [64, 256])
def test_write_token_by_token(D):
    """A sequence grown one token a call: every step equals the definition; zeros, growing and falling magnitudes."""
    rng = np.random.default_rng(D)
    lens0, Hkv = [0, 14, 31], 2
    table, nb = tables(rng, [60, 60, 60])
    c = Cache(nb, Hkv, D).random(rng)
    g = upload(c)
    bt = dev(table)
    for step in range(20):
        lens = [L + step + 1 for L in lens0]
        x = {w: bf16(rng.standard_normal((3, Hkv, D)) * np.exp2(rng.integers(-9, 9, (3, Hkv, 1)))) for w in "kv"}
        if step % 5 == 0:
            x["k"][:] = 0
        i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), dev(np.int32(lens)), bt, **g)
        c.write(x, lens, [1, 1, 1], table)
        same_cache(g, c)
    assert i8.device_error() == 0


def test_write_all_zero_tiny_and_huge():
    table, nb = np.array([[0, 1, 2]], np.int32), 3
    for v in (0.0, 2.0 ** -133, 2.0 ** -120, 3.3e38):
        c = Cache(nb, 1, 64)
        x = {w: bf16(np.full((48, 1, 64), v, np.float32) * np.where(np.arange(64) % 3, 1, -0.5)) for w in "kv"}
        g = upload(c)
        i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), dev(np.int32([48])), dev(table), **g, cu_tokens=cu_of([48]))
        c.write(x, [48], [48], table)
        same_cache(g, c)


def test_write_padding_strides_and_many_sequences():
    rng = np.random.default_rng(3)
    B, Hkv, D = 300, 2, 64
    lens = [int(x) for x in rng.integers(0, 40, B)]
    news = [int(rng.integers(0, L + 1)) for L in lens]
    table, nb = tables(rng, lens)
    c = Cache(nb, Hkv, D).random(rng)
    T = sum(news)
    rows = T + 13  # rows of no sequence behind the last
    fused = torch.full((rows, 3 * Hkv * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = {w: bf16(rng.standard_normal((T, Hkv, D))) for w in "kv"}
    k, v = (fused[:, i * Hkv * D:(i + 1) * Hkv * D].unflatten(1, (Hkv, D)) for i in (0, 2))
    k[:T], v[:T] = dev_bf16(x["k"]), dev_bf16(x["v"])
    g = upload(c)
    i8.block_kv_write(k, v, dev(np.int32(lens)), dev(table), **g, cu_tokens=cu_of(news))
    c.write(x, lens, news, table)
    same_cache(g, c)
    # one row a sequence, some of them unused
    lens = [0 if b % 3 == 0 else L for b, L in enumerate(lens)]
    x = {w: bf16(rng.standard_normal((B, Hkv, D))) for w in "kv"}
    i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), dev(np.int32(lens)), dev(table), **g)
    has = [b for b in range(B) if lens[b]]
    c.write({w: x[w][has] for w in "kv"}, [lens[b] for b in has], [1] * len(has), table[has])
    same_cache(g, c)
    assert i8.device_error() == 0


def test_write_bad_tables_and_counts():
    """Entries and counts out of range: nothing of them is written, and error 2 is recorded."""
    rng = np.random.default_rng(4)
    table, nb = tables(rng, [40, 40])
    c = Cache(nb, 2, 64).random(rng)
    x = dev_bf16(rng.standard_normal((80, 2, 64)))
    for lens, cu, tb in (([40, 40], [0, 40, 80], np.full_like(table, nb)), ([40, 40], [0, 40, 80], np.full_like(table, -1)),
                         ([40, 5000], [0, 0, 40], table), ([30, 40], [0, 40, 40], table), ([40, 40], [0, 0, 81], table),
                         ([40, 40], [50, 30, 30], table), ([40, 40], [-16, -16, 3], table)):
        g = upload(c)
        i8.block_kv_write(x, x, dev(np.int32(lens)), dev(tb), **g, cu_tokens=dev(np.int32(cu)))
        same_cache(g, c)
        assert i8.device_error() == 2


# ------------------------------------------------------------------------------------------------- reading back
@pytest.mark.parametrize("D, Hkv", [(64, 5), (128, 2), (256, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_exact(D, Hkv, dtype):
    rng = np.random.default_rng(D)
    lens, news = [33, 16, 1, 70], [33, 3, 1, 20]
    table, nb = tables(rng, lens)
    c = Cache(nb, Hkv, D).random(rng)
    T = sum(news)
    k = torch.full((T + 5, Hkv, D), 7.0, dtype=dtype, device="cuda")
    v = k.clone()
    i8.block_kv_read(k, v, dev(np.int32(lens)), dev(table), **upload(c), cu_tokens=cu_of(news))
    for w, t in (("k", k), ("v", v)):
        ref = np.concatenate([c.history(table[b], L, w)[L - n:] for b, (L, n) in enumerate(zip(lens, news))])
        ref = bf16(ref) if dtype is torch.bfloat16 else ref
        assert np.array_equal(t[:T].float().cpu().numpy(), ref)
        assert (t[T:] == 7).all()  # rows of no sequence
    assert i8.device_error() == 0


# ------------------------------------------------------------------------------------------------- decode
def _decode(D, Hq, Hkv, lens, dtype=torch.bfloat16, cap=0.0, window=0, slopes=False, begin=None, seed=0, scale=0.0, zero=0.0,
            spread=1.0, qmul=2.0, mb=0, **kw):
    rng = np.random.default_rng(seed)
    table, nb = tables(rng, lens)
    if mb:  # a wider table, its rest outside the pool
        table = np.concatenate([table, np.full((len(lens), mb - table.shape[1]), nb + 5, np.int32)], 1)
    c = Cache(nb, Hkv, D).random(rng, zero, spread)
    q = bf16(rng.standard_normal((len(lens), Hq, D)) * qmul)
    sl = np.exp2(-rng.uniform(0, 8, Hq)).astype(np.float32) if slopes else None
    out = torch.full((len(lens), Hq, D), float("nan"), dtype=dtype, device="cuda")
    i8.block_decode_attn(out, dev_bf16(q), **upload(c), block_tables=dev(table), seq_lens=dev(np.int32(lens)), softmax_scale=scale,
                         softcap=cap, window=window, key_begin=None if begin is None else dev(np.int32(begin)),
                         alibi_slopes=None if sl is None else dev(sl), **kw)
    assert i8.device_error() == 0
    for b, L in enumerate(lens):
        lo = max(0, begin[b] if begin is not None else 0, L - window if window else 0)
        ref, err = attend(q[b:b + 1], c, table[b], L, [lo], [L], [L - 1],
                          scale or D ** -0.5, cap, sl, dtype is torch.bfloat16)
        close(out[b:b + 1], ref, err, dtype is torch.bfloat16)
    return out


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 6, 2), (64, 5, 5), (128, 32, 8), (128, 12, 1), (256, 24, 4), (256, 17, 1)])
@pytest.mark.parametrize("lens", [[1], [16, 17], [300, 0, 5, 1]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode(D, Hq, Hkv, lens, dtype):
    _decode(D, Hq, Hkv, lens, dtype, seed=D + Hq)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(cap=30.0), dict(cap=0.5), dict(window=1), dict(window=33), dict(slopes=True),
                                dict(begin=[16, 7, 400, 0]), dict(cap=50.0, window=100, slopes=True, begin=[3, -5, 250, 1]),
                                dict(scale=0.7), dict(zero=0.5), dict(spread=12.0)])
def test_decode_variants(D, kw):
    for dtype in (torch.float32, torch.bfloat16):
        _decode(D, 8, 2, [170, 40, 400, 1], dtype, seed=D, **kw)


def test_decode_long_and_ragged():
    _decode(128, 8, 2, [5000, 3, 1200, 0, 90], seed=1)
    _decode(256, 6, 1, [9001], torch.float32, seed=2)
    _decode(64, 2, 2, [int(x) for x in np.random.default_rng(0).integers(0, 40, 300)], seed=3)  # more sequences than threads


def test_decode_work_split():
    """A cluster per pair (narrow tables) and the evenly cut list (wide ones) on the same sequences, and clusters of which
    some CTAs or warps have no block."""
    rng = np.random.default_rng(11)
    for D, Hq, Hkv, lens in ((256, 12, 2, [500, 3]), (128, 8, 2, [700, 0, 1, 260]), (64, 3, 1, [129]), (128, 40, 20, [90, 33, 5])):
        table, nb = tables(rng, lens)
        c = Cache(nb, Hkv, D).random(rng)
        q = bf16(rng.standard_normal((len(lens), Hq, D)))
        for mb in (table.shape[1], 40, 100, 400, 4000):
            if mb < table.shape[1]:
                continue
            wide = np.full((len(lens), mb), nb + 5, np.int32)
            wide[:, :table.shape[1]] = table
            for dtype in (torch.float32, torch.bfloat16):
                out = torch.full((len(lens), Hq, D), float("nan"), dtype=dtype, device="cuda")
                i8.block_decode_attn(out, dev_bf16(q), **upload(c), block_tables=dev(wide), seq_lens=dev(np.int32(lens)))
                for b, L in enumerate(lens):
                    ref, err = attend(q[b:b + 1], c, table[b], L, [0], [L], [L - 1], D ** -0.5, 0.0, None, dtype is torch.bfloat16)
                    close(out[b:b + 1], ref, err, dtype is torch.bfloat16)
    assert i8.device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [9, 16, 20, 33])
@pytest.mark.parametrize("kw", [dict(), dict(cap=1.5), dict(slopes=True, window=150, begin=[5, 0, 900, 60, 0, 0])])
def test_decode_many_heads_per_kv_head(D, G, kw):
    """More than eight query heads per KV head, in narrow tables (passes of eight rows) and wide ones (sixteen): full passes and
    parts of one, CTAs with several segments, more sequences than a warp looks at together."""
    for dtype in (torch.float32, torch.bfloat16):
        _decode(D, 3 * G, 3, [400, 40, 1003, 77, 0, 1], dtype, seed=D + G, **kw)
        _decode(D, 3 * G, 3, [400, 40, 1003, 77, 0, 1], dtype, seed=D + G, mb=2000, **kw)
    _decode(D, G, 1, [90], seed=G, **{**kw, "begin": [3]})
    if not kw:
        _decode(D, 2 * G, 2, [900, 3], seed=G, mb=300, qmul=30.0)
        _decode(D, G, 1, [int(x) for x in np.random.default_rng(G).integers(0, 60, 200)], seed=G, mb=500)


def test_decode_extremes():
    """Scores far apart, and rows of q at the ends of bf16's range."""
    _decode(128, 4, 2, [200], torch.float32, seed=5, qmul=200.0)
    _decode(128, 4, 2, [200], torch.float32, seed=6, qmul=0.0)
    _decode(64, 4, 2, [50], torch.float32, seed=7, qmul=2.0 ** -60)
    _decode(64, 4, 2, [50], torch.float32, seed=8, qmul=2.0 ** 60, scale=2.0 ** -63)


def test_decode_hidden_values_do_not_count():
    """NaN scales of blocks that no row sees, and any codes behind the last token, change nothing."""
    rng = np.random.default_rng(9)
    lens = [70, 37]
    table, nb = tables(rng, lens)
    c = Cache(nb, 2, 128).random(rng)
    q = dev_bf16(rng.standard_normal((2, 8, 128)))
    args = dict(block_tables=dev(table), seq_lens=dev(np.int32(lens)), window=20)
    outs = []
    for spoil in (False, True):
        if spoil:
            for b, L in enumerate(lens):
                first = (L - 20) // BS
                for w in "kv":
                    c.scale[w][table[b, :first]] = np.nan
                    c.codes[w][table[b, (L - 1) // BS], :, L % BS or BS:] = -128
            used = set(table[0, :5]) | set(table[1, :3])
            for w in "kv":
                c.scale[w][[i for i in range(nb) if i not in used]] = np.inf
        out = torch.empty((2, 8, 128), dtype=torch.float32, device="cuda")
        i8.block_decode_attn(out, q, **upload(c), **args)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and i8.device_error() == 0


def test_decode_bad_tables_and_lengths():
    """A table entry outside the pool and a length above the table are recorded; nothing outside is read."""
    rng = np.random.default_rng(10)
    table, nb = tables(rng, [40])
    c = Cache(nb, 2, 64).random(rng)
    q = dev_bf16(rng.standard_normal((1, 4, 64)))
    out = torch.empty((1, 4, 64), dtype=torch.float32, device="cuda")
    for bad in (nb, -3, 1 << 30):
        t = table.copy()
        t[0, 1] = bad
        i8.block_decode_attn(out, q, **upload(c), block_tables=dev(t), seq_lens=dev(np.int32([40])))
        assert i8.device_error() == 2
    i8.block_decode_attn(out, q, **upload(c), block_tables=dev(table), seq_lens=dev(np.int32([4000])))
    assert i8.device_error() == 2
    i8.block_decode_attn(out, q, **upload(c), block_tables=dev(table), seq_lens=dev(np.int32([-7])))
    assert i8.device_error() == 0 and (out == 0).all()


# ------------------------------------------------------------------------------------------------- chunk
def _chunk(D, Hq, Hkv, H, C, dtype=torch.bfloat16, cap=0.0, window=0, slopes=False, begin=None, end=None, seed=0, zero=0.0,
           spread=1.0, sample=None, **kw):
    rng = np.random.default_rng(seed)
    n = H + C
    table, nb = tables(rng, [n])
    c = Cache(nb, Hkv, D).random(rng, zero, spread)
    q = bf16(rng.standard_normal((C, Hq, D)) * 2)
    sl = np.exp2(-rng.uniform(0, 8, Hq)).astype(np.float32) if slopes else None
    pos = np.arange(H, n)
    kb = None if begin is None else np.int32(begin(rng, pos))
    ke = None if end is None else np.int32(end(rng, pos))
    out = torch.full((C, Hq, D), float("nan"), dtype=dtype, device="cuda")
    i8.block_prefix_attn(out, dev_bf16(q), **upload(c), block_table=dev(table[0]), history_len=H, softcap=cap, window=window,
                         key_begin=None if kb is None else dev(kb), key_end=None if ke is None else dev(ke),
                         alibi_slopes=None if sl is None else dev(sl), **kw)
    assert i8.device_error() == 0
    lo = np.zeros(C, np.int64) if kb is None else kb.astype(np.int64)
    if window:
        lo = np.maximum(lo, pos - window + 1)
    hi = pos + 1 if ke is None else np.minimum(ke, n)
    rows = np.arange(C) if sample is None or sample >= C else np.unique(np.r_[0, C - 1, rng.integers(0, C, sample)])
    ref, err = attend(q[rows], c, table[0], n, lo[rows], hi[rows], pos[rows], D ** -0.5, cap,
                      sl, dtype is torch.bfloat16)
    close(out[torch.from_numpy(rows).cuda()], ref, err, dtype is torch.bfloat16)


def docs(rng, pos):
    """Packed documents: the first key of each row's document."""
    cut = np.where(rng.random(pos.size) < 0.15, pos, 0)
    return np.maximum.accumulate(cut)


def holes(rng, pos):
    """Some rows see nothing: they begin behind their own position."""
    return np.where(rng.random(pos.size) < 0.4, pos + 5, pos // 2)


def prefix(rng, pos):
    return np.maximum(pos + 1, pos[0] + pos.size // 2)


def anywhere(rng, pos):
    return rng.integers(-5, pos[-1] + 40, pos.size)


VARIANTS = [dict(), dict(cap=30.0), dict(cap=2.0, slopes=True), dict(window=1), dict(window=50), dict(slopes=True),
            dict(begin=docs), dict(begin=holes), dict(end=prefix), dict(end=prefix, slopes=True, cap=20.0),
            dict(begin=anywhere, end=anywhere), dict(begin=docs, window=9), dict(zero=0.5), dict(spread=12.0)]


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 6, 2), (128, 8, 1), (256, 5, 5), (256, 12, 2)])
@pytest.mark.parametrize("H, C", [(0, 1), (5, 3), (0, 50), (83, 33)])
def test_chunk_small(D, Hq, Hkv, H, C):
    for dtype in (torch.float32, torch.bfloat16):
        _chunk(D, Hq, Hkv, H, C, dtype, seed=H + C)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", VARIANTS)
def test_chunk_variants(D, kw):
    _chunk(D, 6, 2, 70, 41, seed=D, **kw)
    _chunk(D, 4, 4, 0, 130, seed=D + 1, **kw)
    _chunk(D, 12, 2, 150, 41, seed=D + 2, **kw)
    _chunk(D, 3, 1, 0, 150, torch.float32, seed=D + 3, **kw)


@pytest.mark.parametrize("D, Hq, Hkv, H, C", [(64, 16, 2, 2900, 701), (128, 8, 4, 40, 2100), (256, 24, 4, 1000, 1300), (128, 32, 8, 9000, 33)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=40.0, begin=docs), dict(window=300, slopes=True), dict(begin=holes, dtype=torch.float32),
                                dict(end=prefix, slopes=True, dtype=torch.float32, cap=15.0)])
def test_chunk_long(D, Hq, Hkv, H, C, kw):
    """Many row blocks and tiles: row blocks cut over CTAs, CTAs with several row blocks."""
    _chunk(D, Hq, Hkv, H, C, seed=D + C, sample=10, **kw)


def test_chunk_hidden_blocks_and_bad_tables():
    """Blocks that no row sees may have any table entry and any scale; an entry outside the pool that a row sees is recorded."""
    rng = np.random.default_rng(30)
    H, C, Hq, Hkv, D = 400, 100, 8, 2, 128
    table, nb = tables(rng, [H + C])
    c = Cache(nb, Hkv, D).random(rng)
    q = dev_bf16(rng.standard_normal((C, Hq, D)))
    outs = []
    begin = dev(np.full(C, 200, np.int32))
    for spoil in (False, True):
        t = table[0].copy()
        if spoil:
            for w in "kv":
                c.scale[w][t[:12]] = np.nan
                c.scale[w][[i for i in range(nb) if i not in set(t)]] = np.inf
            t[:6] = -1
            t[6:9] = nb + 100
        out = torch.empty((C, Hq, D), dtype=torch.float32, device="cuda")
        i8.block_prefix_attn(out, q, **upload(c), block_table=dev(t), history_len=H, key_begin=begin)
        outs.append(out)
        assert i8.device_error() == 0
    assert torch.equal(outs[0], outs[1])
    for C2 in (100, 3):
        t = table[0].copy()
        t[20] = nb
        i8.block_prefix_attn(outs[0][:C2], q[:C2], **upload(c), block_table=dev(t), history_len=H, key_begin=begin[:C2])
        assert i8.device_error() == 2


def test_chunk_intervals_at_the_ends_of_their_type():
    """Begins and ends anywhere in 32 bits: cut to the keys there are."""
    big = 2 ** 31 - 1

    def begin(rng, pos):
        return rng.choice([-big - 1, -1, 0, 7, big], pos.size)

    def end(rng, pos):
        return rng.choice([-big - 1, -1, 0, 20, big], pos.size)

    for D, C in ((64, 5), (64, 130), (256, 130)):
        _chunk(D, 4, 2, 60, C, torch.float32, seed=C, begin=begin, end=end)
        _chunk(D, 4, 2, 60, C, seed=C, end=end, window=30, slopes=True)


def test_chunk_many_row_blocks():
    """More row blocks than the threads that lay out the work."""
    _chunk(64, 8, 1, 100, 12400, seed=3, window=64, sample=12)


def test_pool_beyond_32_bits():
    """Blocks whose codes lie past 2^32 bytes of the pool."""
    rng = np.random.default_rng(40)
    Hq, Hkv, D, C = 8, 8, 256, 40
    NB = (1 << 32) // (Hkv * D * BS) + 50
    small, _ = tables(rng, [C], extra=0)
    n = small.shape[1]
    c = Cache(n, Hkv, D)  # zeros, like the pool
    g = dict(k_cache=torch.zeros((NB, Hkv, D // 16, 16, 16), dtype=torch.int8, device="cuda"),
             v_cache=torch.zeros((NB, Hkv, D, 16), dtype=torch.int8, device="cuda"),
             k_scale=torch.zeros((NB, Hkv), device="cuda"), v_scale=torch.zeros((NB, Hkv), device="cuda"))
    table = np.int32(NB - 40 + small)
    x = {w: bf16(rng.standard_normal((C, Hkv, D))) for w in "kv"}
    q = bf16(rng.standard_normal((C, Hq, D)))
    i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), dev(np.int32([C])), dev(table), **g, cu_tokens=cu_of([C]))
    c.write(x, [C], [C], small)
    for name, part in upload(c).items():
        assert torch.equal(g[name][NB - 40:NB - 40 + n], part)
    k = torch.empty((C, Hkv, D), device="cuda")
    v = torch.empty_like(k)
    i8.block_kv_read(k, v, dev(np.int32([C])), dev(table), **g, cu_tokens=cu_of([C]))
    assert np.array_equal(k.cpu().numpy(), c.history(small[0], C, "k"))
    for rows in (1, C):  # the decode, and a chunk of as many rows on either route
        pos = np.arange(C - rows, C)
        ref, err = attend(q[C - rows:], c, small[0], C, 0 * pos, pos + 1, pos, D ** -0.5, 0.0, None, False)
        out = torch.empty((rows, Hq, D), device="cuda")
        i8.block_prefix_attn(out, dev_bf16(q[C - rows:]), **g, block_table=dev(table[0]), history_len=C - rows)
        close(out, ref, err, False)
    out = torch.empty((1, Hq, D), device="cuda")
    i8.block_decode_attn(out, dev_bf16(q[C - 1:]), **g, block_tables=dev(table), seq_lens=dev(np.int32([C])))
    ref, err = attend(q[C - 1:], c, small[0], C, [0], [C], [C - 1], D ** -0.5, 0.0, None, False)
    close(out, ref, err, False)
    assert i8.device_error() == 0


def test_chunk_rows_at_the_limits_of_both_routes():
    """Numbers of (token, head) rows around the change of route and around a row block."""
    for C in (63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257):
        _chunk(64, 1, 1, 77, C, torch.float32, seed=C, sample=40)
    # the same rows on either side of the rule on rows and keys, with and without a window
    for H in (200, 3000):
        for window in (0, 90):
            _chunk(128, 8, 4, H, 40, seed=H, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sixteen_rows_strided_and_replayed(D):
    """Passes of sixteen rows on a strided q, captured and replayed with other values: the bits of an eager call."""
    rng = np.random.default_rng(D)
    lens, Hq, Hkv = [700, 90, 0, 333], 24, 2
    table, nb = tables(rng, lens)
    wide = np.concatenate([table, np.full((len(lens), 1000), nb, np.int32)], 1)
    c, table = upload(Cache(nb, Hkv, D).random(rng)), dev(wide)
    fused = torch.zeros((len(lens), (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    q, sl = fused[:, :Hq * D].view(len(lens), Hq, D), dev(np.int32([16, 16, 0, 16]))  # the third has no page
    ws = i8.block_decode_workspace(len(lens), Hq, Hkv, D, wide.shape[1])
    out, again = (torch.empty((len(lens), Hq, D), dtype=torch.float32, device="cuda") for _ in range(2))
    i8.block_decode_attn(out, q, **c, block_tables=table, seq_lens=sl, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i8.block_decode_attn(out, q, **c, block_tables=table, seq_lens=sl, workspace=ws)
    for n in (lens, [33, 1, 0, 330], lens):
        q.copy_(dev_bf16(rng.standard_normal((len(lens), Hq, D))))
        sl.copy_(dev(np.int32(n)))
        g.replay()
        i8.block_decode_attn(again, q.contiguous(), **c, block_tables=table, seq_lens=sl)
        assert torch.equal(out, again) and out.abs().sum() > 0
    assert i8.device_error() == 0


def test_sixteen_rows_bad_tables_are_recorded():
    """Passes of sixteen rows: a table entry outside the pool of a visible block, in a decode and in a chunk."""
    rng = np.random.default_rng(16)
    H, C, Hq, Hkv, D = 11000, 25, 32, 2, 64
    table, nb = tables(rng, [H + C])
    c = Cache(nb, Hkv, D).random(rng)
    q = dev_bf16(rng.standard_normal((C, Hq, D)))
    out = torch.empty((C, Hq, D), dtype=torch.bfloat16, device="cuda")
    wide = np.concatenate([table, np.zeros((1, 4000), np.int32)], 1)  # enough blocks for sixteen rows per pass
    for bad in (None, nb, -1):
        t, w = table.copy(), wide.copy()
        if bad is not None:
            t[0, 300] = w[0, 300] = bad
        i8.block_decode_attn(out[:1], q[:1], **upload(c), block_tables=dev(w), seq_lens=dev(np.int32([H])))
        assert i8.device_error() == (0 if bad is None else 2)
        i8.block_prefix_attn(out[:5], q[:5], **upload(c), block_table=dev(t[0]), history_len=H)
        assert i8.device_error() == (0 if bad is None else 2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 33, 64])
def test_chunk_few_rows(D, rows):
    """Around the numbers of rows that fill a pass of eight or sixteen, over short and long histories."""
    for i, H in enumerate((0, 30, 2500, 41000)):
        _chunk(D, 2, 2, H, rows, torch.float32 if i % 2 else torch.bfloat16, cap=3.0 if i else 0.0, begin=docs if i == 1 else None,
               seed=D + rows, sample=6)
        _chunk(D, 6, 2, H, (rows + 2) // 3, seed=D + rows, slopes=i == 2, begin=holes if i == 0 else None, sample=6)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_workspace_at_sixteen_bytes(D):
    """A workspace on a 16-byte boundary that is no 32-byte boundary gives the same bits."""
    rng = np.random.default_rng(D)
    H, C, Hq, Hkv = 300, 260, 4, 2
    table, nb = tables(rng, [H + C])
    c, q = Cache(nb, Hkv, D).random(rng), dev_bf16(rng.standard_normal((C, Hq, D)))
    n = i8.block_prefix_workspace(H, C, Hq, Hkv, D).numel()
    room = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
    outs = []
    for shift in (0, 16):
        at = -room.data_ptr() % 32 + shift
        out = torch.full((C, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        i8.block_prefix_attn(out, q, **upload(c), block_table=dev(table[0]), history_len=H, workspace=room[at:at + n])
        outs.append(out)
    assert torch.equal(*outs) and i8.device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", VARIANTS)
def test_chunk_row_groups_of_sixteen(D, kw):
    """A CTA per (group, KV head), and the evenly cut list of long histories."""
    for dtype in (torch.float32, torch.bfloat16):
        _chunk(D, 8, 8, 100, 235, dtype, seed=D, sample=40, **kw)
        _chunk(D, 8, 4, 11000, 25, dtype, seed=D + 1, sample=10, **kw)


# ------------------------------------------------------------------------------------------------- together
def test_prefill_then_decode():
    """As a server uses them: two sequences prefilled in chunks, then decoded token by token; the decode of the newest
    token equals the chunk call of that one token within the bounds, and what is read back is what was attended to."""
    rng = np.random.default_rng(20)
    Hq, Hkv, D, B = 8, 2, 128, 2
    table, nb = tables(rng, [200, 200])
    c = Cache(nb, Hkv, D)
    g = {k: torch.zeros_like(t) for k, t in upload(c).items()}
    bt = dev(table)
    lens = [0, 0]
    for news in ([60, 45], [33, 0], [1, 1], [1, 1], [1, 1]):
        lens = [L + n for L, n in zip(lens, news)]
        x = {w: bf16(rng.standard_normal((sum(news), Hkv, D))) for w in "kv"}
        q = bf16(rng.standard_normal((sum(news), Hq, D)))
        sl = dev(np.int32(lens))
        one = news == [1, 1]
        i8.block_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), sl, bt, **g, cu_tokens=None if one else cu_of(news))
        c.write(x, lens, news, table)
        same_cache(g, c)
        at = 0
        if one:
            out = torch.empty((B, Hq, D), dtype=torch.float32, device="cuda")
            i8.block_decode_attn(out, dev_bf16(q), **g, block_tables=bt, seq_lens=sl, softcap=25.0)
        for b, (L, n) in enumerate(zip(lens, news)):
            if not n:
                continue
            pos = np.arange(L - n, L)
            ref, err = attend(q[at:at + n], c, table[b], L, 0 * pos, pos + 1, pos, D ** -0.5, 25.0, None, False)
            got = torch.empty((n, Hq, D), dtype=torch.float32, device="cuda")
            i8.block_prefix_attn(got, dev_bf16(q[at:at + n]), **g, block_table=bt[b], history_len=L - n, softcap=25.0)
            if n == 1:
                close(got, ref, err, False)
                close(out[b:b + 1], ref, err, False)
            else:  # a chunk's weights may be rounded to f16
                close(got, ref, attend(q[at:at + n], c, table[b], L, 0 * pos, pos + 1, pos, D ** -0.5, 25.0, None, True)[1], False)
            at += n
    assert i8.device_error() == 0


def test_graph_replay_and_streams():
    """Write, read, decode and chunk captured in one graph and replayed on new values; another stream; own workspaces."""
    rng = np.random.default_rng(21)
    Hq, Hkv, D = 8, 2, 128
    lens = [90, 33]
    table, nb = tables(rng, lens)
    c = Cache(nb, Hkv, D).random(rng)
    g = upload(c)
    bt, sl = dev(table), dev(np.int32(lens))
    k, v, q = (torch.zeros((2, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    ws = [i8.block_decode_workspace(2, Hq, Hkv, D, table.shape[1]) for _ in range(2)]
    wp = i8.block_prefix_workspace(89, 1, Hq, Hkv, D)
    outs = [torch.zeros((2, Hq, D), dtype=torch.float32, device="cuda") for _ in range(2)]
    oc = torch.zeros((1, Hq, D), dtype=torch.float32, device="cuda")

    def step(i):
        i8.block_kv_write(k, v, sl, bt, **g)
        i8.block_decode_attn(outs[i], q, **g, block_tables=bt, seq_lens=sl, workspace=ws[i])
        i8.block_prefix_attn(oc, q[:1], **g, block_table=bt[0], history_len=89, workspace=wp)

    def check(i, x, qn):
        c.write(x, lens, [1, 1], table)
        same_cache(g, c)
        for b, L in enumerate(lens):
            ref, err = attend(qn[b:b + 1], c, table[b], L, [0], [L], [L - 1], D ** -0.5, 0.0, None, False)
            close(outs[i][b:b + 1], ref, err, False)
            if b == 0:
                close(oc, ref, err, False)

    def new():
        x = {w: bf16(rng.standard_normal((2, Hkv, D)) * 3) for w in "kv"}
        qn = bf16(rng.standard_normal((2, Hq, D)))
        k.copy_(dev_bf16(x["k"]))
        v.copy_(dev_bf16(x["v"]))
        q.copy_(dev_bf16(qn))
        return x, qn

    step(0)  # modules loaded, shared memory opted in
    torch.cuda.synchronize()
    g2 = upload(c)
    for n in g:
        g[n].copy_(g2[n])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(0)
    for _ in range(3):
        x, qn = new()
        graph.replay()
        torch.cuda.synchronize()
        check(0, x, qn)
    x, qn = new()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1)
    side.synchronize()
    check(1, x, qn)
    # a stream given by hand, the workspace allocated by the call
    x, qn = new()
    side.wait_stream(torch.cuda.current_stream())
    i8.block_kv_write(k, v, sl, bt, **g, stream=side)
    i8.block_decode_attn(outs[1], q, **g, block_tables=bt, seq_lens=sl, stream=side)
    i8.block_prefix_attn(oc, q[:1], **g, block_table=bt[0], history_len=89, stream=side)
    side.synchronize()
    check(1, x, qn)
    assert i8.device_error() == 0


def test_strided_rows_of_q():
    rng = np.random.default_rng(22)
    lens = [60, 21, 7]
    table, nb = tables(rng, lens)
    c = Cache(nb, 2, 64).random(rng)
    g = upload(c)
    fused = dev_bf16(rng.standard_normal((3, 10, 64)))
    q = fused[:, 2:8]
    a, b = (torch.empty((3, 6, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    args = dict(block_tables=dev(table), seq_lens=dev(np.int32(lens)))
    i8.block_decode_attn(a, q, **g, **args)
    i8.block_decode_attn(b, q.contiguous(), **g, **args)
    assert torch.equal(a, b)
    i8.block_prefix_attn(a, q, **g, block_table=dev(table[0]), history_len=57)
    i8.block_prefix_attn(b, q.contiguous(), **g, block_table=dev(table[0]), history_len=57)
    assert torch.equal(a, b)
    with pytest.raises(i8.I8KVError, match="contiguous"):
        i8.block_decode_attn(a, fused[:, 2:8].transpose(1, 2).contiguous().transpose(1, 2), **g, **args)


def test_binding_refusals_on_device():
    c = i8.alloc_block_cache(4, 2, 64)
    bt, sl = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((1, 4, 64), device="cuda")
    with pytest.raises(i8.I8KVError, match="bfloat16"):
        i8.block_kv_write(k.float(), k, sl, bt, **c)
    with pytest.raises(i8.I8KVError, match="cu_tokens"):
        i8.block_kv_write(k.expand(2, 2, 64).contiguous(), k.expand(2, 2, 64).contiguous(), sl, bt, **c)
    with pytest.raises(i8.I8KVError, match="seq_lens"):
        i8.block_decode_attn(out, q, **c, block_tables=bt, seq_lens=sl.long())
    with pytest.raises(i8.I8KVError, match="v_scale"):
        i8.block_decode_attn(out, q, **{**c, "v_scale": c["v_scale"][:2]}, block_tables=bt, seq_lens=sl)
    with pytest.raises(i8.I8KVError, match="out"):
        i8.block_decode_attn(out.half(), q, **c, block_tables=bt, seq_lens=sl)
    with pytest.raises(i8.I8KVError, match="cover"):
        i8.block_prefix_attn(out, q, **c, block_table=bt[0], history_len=64)
    n = 400  # more pairs than SMs: a call with a workspace
    with pytest.raises(i8.I8KVError, match="workspace"):
        i8.block_decode_attn(out.expand(n, 4, 64).contiguous(), q.expand(n, 4, 64), **c, block_tables=bt.expand(n, 4).contiguous(),
                             seq_lens=sl.expand(n).contiguous(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
