"""Cases of the block-scaled 8-bit KV cache: writing it, reading it back, and the decode and chunk attention over it.

The cache holds int8 codes in pages of 16 tokens (K [NB, Hkv, D/16, 16, 16], V [NB, Hkv, D, 16]) and one fp32 scale per
(block, KV head) for K and for V.  Scores may be capped by a tanh, biased by distance (a slope per query head) and
limited by a sliding window or by each row's own interval of visible keys."""
import math

import torch

own = False
BS = 16


def listed():
    return [
        # one sequence takes its next token: pure latency
        dict(name="write-step-1", op="write", B=1, L=4096, n=1, ragged=False, Hkv=4, D=256),
        # a decode batch: one token a sequence, at every offset of its block
        dict(name="write-step-64", op="write", B=64, L=900, n=1, ragged=True, Hkv=8, D=128),
        # prefill: ragged chunks of several sequences, 8192 tokens together at most
        dict(name="write-chunk", op="write", B=4, L=5000, n=2048, ragged=True, Hkv=8, D=128),
        # a short sequence leaves the cache
        dict(name="read-1", op="read", B=1, L=517, n=517, ragged=False, Hkv=4, D=256, f32=True),
        # a batch is swapped out: its whole history in bf16
        dict(name="read-batch", op="read", B=16, L=8192, n=8192, ragged=True, Hkv=8, D=128, f32=False),
        # interactive use: one sequence, a middling history
        dict(name="decode-1", op="decode", B=1, L=4096, ragged=False, Hq=24, Hkv=4, D=256, cap=0.0, window=0, slopes=False,
             begin=False, f32=False),
        # a few short sequences with capped scores, fp32 result
        dict(name="decode-cap-f32", op="decode", B=5, L=777, ragged=True, Hq=8, Hkv=8, D=64, cap=30.0, window=0,
             slopes=False, begin=True, f32=True),
        # a served batch at long histories
        dict(name="decode-16", op="decode", B=16, L=32768, ragged=False, Hq=32, Hkv=8, D=128, cap=50.0, window=0,
             slopes=False, begin=False, f32=False),
        # a large ragged batch with distance biases
        dict(name="decode-64-bias", op="decode", B=64, L=32768, ragged=True, Hq=24, Hkv=4, D=256, cap=0.0, window=0,
             slopes=True, begin=False, f32=False),
        # a few tokens to verify after a long history
        dict(name="chunk-16", op="chunk", C=16, H=8192, Hq=24, Hkv=4, D=256, cap=50.0, window=0, slopes=False, docs=0,
             prefix=0, f32=False),
        # packed documents of a first chunk, each with its own mask, within a sliding window
        dict(name="chunk-docs", op="chunk", C=4096, H=0, Hq=32, Hkv=8, D=128, cap=0.0, window=1024, slopes=False, docs=7,
             prefix=0, f32=False),
        # a prefill chunk over a long history, capped scores
        dict(name="chunk-2048", op="chunk", C=2048, H=16384, Hq=24, Hkv=4, D=256, cap=50.0, window=0, slopes=False, docs=0,
             prefix=0, f32=False),
    ]


HEADS = [(24, 4), (32, 8), (8, 8), (16, 2), (12, 1), (5, 5)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "chunk", "chunk"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 256])
    if op in ("write", "read"):
        B = _log(rng, 1, 64)
        room = 8192 if op == "write" else 65536
        n = 1 if op == "write" and rng.random() < 0.5 else _log(rng, 1, max(1, room // B))
        c = dict(op=op, B=B, L=n + _log(rng, 1, 4096), n=n, ragged=rng.random() < 0.7, Hkv=Hkv, D=D)
        if op == "read":
            c["f32"] = rng.random() < 0.5
        return c
    cap = rng.choice([0.0, 0.0, 20.0, 30.0, 50.0])
    slopes = rng.random() < 0.3
    window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    if op == "decode":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, L=_log(rng, 1, min(32768, 524288 // B)), ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, D=D, cap=cap,
                    window=window, slopes=slopes, begin=rng.random() < 0.3, f32=rng.random() < 0.3)
    C = _log(rng, 1, 2048)
    docs = rng.choice([0, 0, _log(rng, 1, 8)])
    H = rng.choice([0, _log(rng, 1, 16384)])
    prefix = 0 if docs or rng.random() < 0.7 else _log(rng, 1, H + C)
    return dict(op=op, C=C, H=H, Hq=Hq, Hkv=Hkv, D=D, cap=cap, window=window, slopes=slopes, docs=docs, prefix=prefix, f32=False)


# ------------------------------------------------------------------------------------------------- sizes and inputs
def _lengths(case):
    """Sequence lengths and numbers of new (or read) tokens, fixed by the case: the largest first, then spread below it."""
    B, L, ragged = case["B"], case["L"], case["ragged"]
    n = case.get("n", 1)
    lens, news = [], []
    for b in range(B):
        part = 1.0 if not ragged else ((b * 0.6180339887498949) % 1.0 if b else 1.0)
        m = max(1, int(n * part)) if n > 1 else 1
        lens.append(max(m, int(max(1, L * (part if part > 1 / 32 else 1 / 32)))))
        news.append(m)
    if case["op"] == "read":
        news = [min(m, x) for m, x in zip(news, lens)]
    return lens, news


def _slopes(Hq, gen, dev):
    return torch.exp2(-8.0 * (torch.arange(Hq, device=dev, dtype=torch.float32) + 1) / Hq) * (0.9 + 0.2 * torch.rand(Hq, device=dev, generator=gen))


def _values(shape, gen, dev, outliers=0.0):
    x = torch.randn(shape, device=dev, generator=gen)
    if outliers:
        x *= torch.where(torch.rand(shape[:-1] + (1,), device=dev, generator=gen) < outliers, 6.0, 1.0)
    return x.to(torch.bfloat16)


def _quantized(NB, Hkv, D, gen, dev, channel):
    """Codes [NB, Hkv, 16 tokens, D] and scales [NB, Hkv] of N(0,1) values, some channels of which stand out (keys)."""
    codes = torch.empty((NB, Hkv, BS, D), dtype=torch.int8, device=dev)
    scale = torch.empty((NB, Hkv), device=dev)
    gain = torch.where(torch.rand(Hkv, 1, D, device=dev, generator=gen) < 0.02, channel, 1.0)
    step = max(1, (1 << 26) // (Hkv * BS * D))
    for a in range(0, NB, step):
        x = torch.randn((min(step, NB - a), Hkv, BS, D), device=dev, generator=gen) * gain
        s = x.abs().amax((-1, -2)) / 127
        codes[a:a + step] = torch.clamp(torch.round(x / s[..., None, None]), -127, 127).to(torch.int8)
        scale[a:a + step] = s
    return codes, scale


def _paged(codes, keys):
    NB, Hkv, _, D = codes.shape
    if keys:
        return codes.view(NB, Hkv, BS, D // 16, 16).permute(0, 1, 3, 2, 4).contiguous()
    return codes.permute(0, 1, 3, 2).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    Hkv, D, op = case["Hkv"], case["D"], case["op"]
    s = dict(case=case)
    if op == "chunk":
        lens, news = [case["H"] + case["C"]], [case["C"]]
    else:
        lens, news = _lengths(case)
    nblk = [(x + BS - 1) // BS for x in lens]
    NB, mb = sum(nblk), max(nblk)
    codes, s["k_scale"] = _quantized(NB, Hkv, D, gen, dev, 4.0)
    s["k_cache"] = _paged(codes, True)
    codes, s["v_scale"] = _quantized(NB, Hkv, D, gen, dev, 1.0)
    s["v_cache"] = _paged(codes, False)
    del codes
    # a shared pool: the blocks of a sequence lie anywhere in it; unused entries of a table row are 0
    perm = torch.randperm(NB, device=dev, generator=gen).to(torch.int32)
    n = torch.tensor(nblk, device=dev)
    col = torch.arange(mb, device=dev)
    at = (torch.cumsum(n, 0) - n)[:, None] + col
    s["block_tables"] = torch.where(col < n[:, None], perm[at.clamp(max=NB - 1)], 0).to(torch.int32)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if op in ("write", "read"):
        cu = [0]
        for m in news:
            cu.append(cu[-1] + m)
        s["cu_tokens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["T"] = cu[-1]
        if op == "write":
            s["k"] = _values((cu[-1], Hkv, D), gen, dev, 0.05)
            s["v"] = _values((cu[-1], Hkv, D), gen, dev, 0.05)
            # the tokens of the blocks that the call changes, which are read back
            back = [x - (x - m) // BS * BS for x, m in zip(lens, news)]
            cub = [0]
            for m in back:
                cub.append(cub[-1] + m)
            s["cu_back"] = torch.tensor(cub, dtype=torch.int32, device=dev)
            s["T_back"] = cub[-1]
        return s
    rows = case["C"] if op == "chunk" else case["B"]
    s["q"] = (_values((rows, case["Hq"], D), gen, dev).float() * 1.5).to(torch.bfloat16)
    s["slopes"] = _slopes(case["Hq"], gen, dev) if case["slopes"] else None
    s["key_begin"] = s["key_end"] = None
    if op == "decode" and case["begin"]:  # padding on the left: a part of each history is not visible
        s["key_begin"] = (torch.rand(rows, device=dev, generator=gen) * 0.4 * s["seq_lens"]).to(torch.int32)
    if op == "chunk":
        C, H = case["C"], case["H"]
        pos = torch.arange(H, H + C, device=dev, dtype=torch.int32)
        if case["docs"]:  # the chunk's tokens belong to several documents; the first goes on from the history
            cut = (torch.rand(C, device=dev, generator=gen) < case["docs"] / C)
            s["key_begin"] = torch.cummax(torch.where(cut, pos, torch.zeros_like(pos)), 0)[0].to(torch.int32)
        if case["prefix"]:  # the first positions are visible to every row
            s["key_end"] = torch.clamp(pos + 1, min=case["prefix"]).to(torch.int32)
    return s


def work(case):
    Hkv, D, op = case["Hkv"], case["D"], case["op"]
    if op in ("write", "read"):
        lens, news = _lengths(case)
        T = sum(news)
        if op == "read":
            return dict(bytes=2 * T * Hkv * D * (1 + (4 if case["f32"] else 2)), flops=2 * T * Hkv * D)
        back = sum(x - (x - m) // BS * BS for x, m in zip(lens, news))
        # the new tokens in bf16, their codes, and the changed blocks' values read back in bf16
        return dict(bytes=2 * T * Hkv * D * 3 + 2 * back * Hkv * D * 3, flops=4 * T * Hkv * D)
    Hq = case["Hq"]
    w = case["window"]
    if op == "decode":
        lens, _ = _lengths(case)
        seen = sum(min(x, w) if w else x for x in lens)
        if case["begin"]:
            seen = int(0.8 * seen)
        return dict(bytes=2 * seen * Hkv * D + len(lens) * Hq * D * (2 + (4 if case["f32"] else 2)), flops=4 * seen * Hq * D)
    C, H = case["C"], case["H"]
    pairs = sum(min(H + j + 1, w) if w else H + j + 1 for j in range(C))
    if case["docs"]:
        d = max(1, C // (case["docs"] + 1))
        pairs = min(pairs, sum(min(j % d + 1 + (H if j < d else 0), w or 1 << 30) for j in range(C)))
    if case["prefix"]:
        pairs += sum(max(0, case["prefix"] - (H + j + 1)) for j in range(C))
    keys = min(H + C, C + w) if w else H + C
    return dict(bytes=2 * keys * Hkv * D + C * Hq * D * 4, flops=4 * pairs * Hq * D)


# ------------------------------------------------------------------------------------------------- the plain form
def _dense(s, b_rows, positions, want):
    """Values code x scale [rows, positions, Hkv, D] in fp32 of the given positions of the block-table rows."""
    cache, scale = s[want + "_cache"], s[want + "_scale"]
    blk = torch.gather(s["block_tables"].long()[b_rows], 1, positions // BS)
    off = positions % BS
    if want == "k":
        codes = cache[blk, :, :, off].flatten(-2)
    else:
        codes = cache[blk, :, :, off]
    return codes.float() * scale[blk][..., None]


def _ragged(s, cu, T):
    """Sequence and position of each of the T tokens of a ragged call."""
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, s["seq_lens"].long()[b] - cu[1:].long()[b] + t


def _plain_write(s):
    b, pos = _ragged(s, s["cu_tokens"], s["T"])
    off = pos % BS
    blk = s["block_tables"].long()[b, pos // BS]
    NB, Hkv = s["k_scale"].shape
    # the offset of each block's first new token; blocks without one keep everything
    first = torch.full((NB,), BS, device=blk.device).scatter_reduce(0, blk, off, "amin")
    written = torch.zeros((NB, BS), dtype=torch.bool, device=blk.device)
    written[blk, off] = True
    for x, cache, scale, keys in ((s["k"], s["k_cache"], s["k_scale"], True), (s["v"], s["v_cache"], s["v_scale"], False)):
        x = x.float()
        amax = torch.zeros((NB, Hkv), device=x.device).scatter_reduce(0, blk[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        old = torch.where(first[:, None] == 0, 0.0, scale)
        new = torch.where(first[:, None] == BS, scale, torch.maximum(old, amax / 127))
        touched = torch.unique(blk)
        ratio = torch.where(new > 0, old / new, 0.0)[touched][:, :, None, None]
        codes = cache[touched]
        codes = codes.permute(0, 1, 3, 2, 4).flatten(-2) if keys else codes.permute(0, 1, 3, 2)
        before = (torch.arange(BS, device=x.device) < first[touched][:, None])[:, None, :, None]
        codes = torch.where(before, torch.round(codes.float() * ratio), codes.float())
        s_tok = new[blk][..., None]
        q = torch.clamp(torch.round(torch.where(s_tok > 0, x / s_tok, 0.0)), -127, 127)
        codes[torch.searchsorted(touched, blk), :, off] = q
        codes = codes.to(torch.int8)
        cache[touched] = _paged(codes, keys)
        scale.copy_(new)


def _plain_read(s, cu, T, dtype):
    b, pos = _ragged(s, cu, T)
    return [_dense(s, b, pos[:, None], w)[:, 0].to(dtype) for w in ("k", "v")]


def _scores(x, case, s, dist):
    """Scores after the cap and the distance bias; x [..., Hq, rows, keys], dist [..., rows, keys] broadcast over heads."""
    x = x * case["D"] ** -0.5
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * dist
    return x


def _softmax(x, visible):
    """Rows without a visible key are zero."""
    x = torch.where(visible, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(s):
    case = s["case"]
    B, Hq, D = s["q"].shape
    Hkv, L = case["Hkv"], s["seq_lens"].long()
    pos = torch.arange(s["block_tables"].shape[1] * BS, device=L.device)
    lo = torch.zeros_like(L)
    if case["window"]:
        lo = (L - case["window"]).clamp(min=0)
    if s["key_begin"] is not None:
        lo = torch.maximum(lo, s["key_begin"].long())
    visible = ((pos >= lo[:, None]) & (pos < L[:, None]))[:, None, None]
    rows, every = torch.arange(B, device=L.device), pos.expand(B, -1)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, _dense(s, rows, every, "k").permute(0, 2, 3, 1)).view(B, Hq, 1, -1)
    dist = (L[:, None] - 1 - pos).abs().float()[:, None, None]
    p = _softmax(_scores(x, case, s, dist), visible).view(B, Hkv, Hq // Hkv, -1)
    o = torch.matmul(p, _dense(s, rows, every, "v").permute(0, 2, 1, 3)).view(B, Hq, D)
    return o.to(torch.float32 if case["f32"] else torch.bfloat16)


def _interval(s):
    """First and last + 1 visible key of each row of a chunk."""
    case = s["case"]
    C, H = case["C"], case["H"]
    pos = torch.arange(H, H + C, device=s["q"].device)
    lo = torch.zeros_like(pos) if s["key_begin"] is None else s["key_begin"].long()
    hi = pos + 1 if s["key_end"] is None else s["key_end"].long()
    if case["window"]:
        lo = torch.maximum(lo, pos - case["window"] + 1)
    return pos, lo, hi.clamp(max=H + C)


def _plain_chunk(s):
    case = s["case"]
    C, Hq, D = s["q"].shape
    Hkv, G = case["Hkv"], Hq // case["Hkv"]
    n = case["H"] + C
    key = torch.arange(n, device=s["q"].device)
    pos, lo, hi = _interval(s)
    one = torch.zeros(1, dtype=torch.long, device=key.device)
    k, v = (_dense(s, one, key[None], w)[0].permute(1, 0, 2) for w in ("k", "v"))
    q = s["q"].float().view(C, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * C, D)
    x = torch.matmul(q, k.transpose(1, 2)).view(Hq, C, n)
    visible = (key >= lo[:, None]) & (key < hi[:, None])
    p = _softmax(_scores(x, case, s, (pos[:, None] - key).abs().float()), visible)
    o = torch.matmul(p.view(Hkv, G * C, n), v).view(Hq, C, D).permute(1, 0, 2)
    return o.to(torch.float32 if case["f32"] else torch.bfloat16).contiguous()


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import int8_kv_cache_token_gb300 as i8
        cache = dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op in ("write", "read"):
            if op == "write":
                i8.block_kv_write(s["k"], s["v"], s["seq_lens"], s["block_tables"], **cache, cu_tokens=s["cu_tokens"])
            cu, T = (s["cu_back"], s["T_back"]) if op == "write" else (s["cu_tokens"], s["T"])
            dtype = torch.float32 if case.get("f32") else torch.bfloat16
            k = torch.empty((T, case["Hkv"], case["D"]), dtype=dtype, device=cu.device)
            v = torch.empty_like(k)
            i8.block_kv_read(k, v, s["seq_lens"], s["block_tables"], **cache, cu_tokens=cu)
            return [k, v] if op == "read" else [k, v, s["k_scale"], s["v_scale"]]
        out = torch.empty(s["q"].shape, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=s["q"].device)
        if op == "decode":
            i8.block_decode_attn(out, s["q"], **cache, block_tables=s["block_tables"], seq_lens=s["seq_lens"],
                                 softcap=case["cap"], window=case["window"], key_begin=s["key_begin"], alibi_slopes=s["slopes"])
        else:
            i8.block_prefix_attn(out, s["q"], **cache, block_table=s["block_tables"][0], history_len=case["H"],
                                 softcap=case["cap"], window=case["window"], key_begin=s["key_begin"], key_end=s["key_end"],
                                 alibi_slopes=s["slopes"])
        return out
    if op == "write":
        _plain_write(s)
        return _plain_read(s, s["cu_back"], s["T_back"], torch.bfloat16) + [s["k_scale"], s["v_scale"]]
    if op == "read":
        return _plain_read(s, s["cu_tokens"], s["T"], torch.float32 if case["f32"] else torch.bfloat16)
    return _plain_decode(s) if op == "decode" else _plain_chunk(s)


# ------------------------------------------------------------------------------------------------- 64 bits
def _history(s, b, n, want):
    """The first n tokens of sequence b as float64 [n, Hkv, D], page by page."""
    blocks = s["block_tables"][b, : (n + BS - 1) // BS].long()
    codes = s[want + "_cache"][blocks].double()
    codes = codes.permute(0, 3, 1, 2, 4).flatten(3) if want == "k" else codes.permute(0, 3, 1, 2)
    return (codes * s[want + "_scale"][blocks].double()[:, None, :, None]).flatten(0, 1)[:n]


def _attend(q, k, v, lo, hi, pos, case, slopes):
    """One sequence's rows q [rows, Hq, D] over keys [n, Hkv, D] in 64 bits, head by head."""
    rows, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device=q.device)
    t = torch.arange(k.shape[0], device=q.device)
    hidden = (t < lo[:, None]) | (t >= hi[:, None])
    for h in range(Hq):
        x = q[:, h].double() @ k[:, h // G].T / math.sqrt(D)
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        if slopes is not None:
            x = x - slopes[h].double() * (pos[:, None] - t).abs()
        x = x.masked_fill(hidden, -1e300)
        e = torch.exp(x - x.max(-1, keepdim=True).values).masked_fill(hidden, 0.0)
        out[:, h] = (e @ v[:, h // G]) / e.sum(-1, keepdim=True).clamp(min=1e-300)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "read":
        lens, news = _lengths(case)
        return [torch.cat([_history(s, b, n, w)[n - m:] for b, (n, m) in enumerate(zip(lens, news))]) for w in ("k", "v")]
    if op == "write":
        lens, news = _lengths(case)
        outs, scales, at = {"k": [], "v": []}, {"k": s["k_scale"].double(), "v": s["v_scale"].double()}, 0
        for b, (n, m) in enumerate(zip(lens, news)):
            start = (n - m) // BS * BS
            for w in ("k", "v"):
                old = _history(s, b, n, w)[start:]
                new = s[w][at: at + m].double()
                for p in range(start, n, BS):
                    blk = int(s["block_tables"][b, p // BS])
                    f, e = max(0, n - m - p), min(BS, n - p)
                    fresh = new[p + f - (n - m): p + e - (n - m)]
                    was = scales[w][blk].clone() if f else torch.zeros_like(scales[w][blk])
                    sc = torch.maximum(was, (fresh.abs().amax((0, 2)) / 127).float().double())
                    scales[w][blk] = sc
                    sc = sc.clamp(min=1e-300)[:, None]
                    kept = torch.round(old[p - start: p - start + f] / sc) * sc
                    outs[w].append(torch.cat([kept, torch.clamp(torch.round(fresh / sc), -127, 127) * sc]))
            at += m
        return [torch.cat(outs["k"]), torch.cat(outs["v"]), scales["k"], scales["v"]]
    if op == "decode":
        lens, _ = _lengths(case)
        got = []
        for b, n in enumerate(lens):
            lo = max(n - case["window"], 0) if case["window"] else 0
            if s["key_begin"] is not None:
                lo = max(lo, int(s["key_begin"][b]))
            one = torch.ones(1, dtype=torch.long, device=s["q"].device)
            got.append(_attend(s["q"][b: b + 1], _history(s, b, n, "k"), _history(s, b, n, "v"), one * lo, one * n, one * (n - 1), case,
                               s["slopes"]))
        return torch.cat(got)
    n = case["H"] + case["C"]
    pos, lo, hi = _interval(s)
    return _attend(s["q"], _history(s, 0, n, "k"), _history(s, 0, n, "v"), lo, hi, pos, case, s["slopes"])
