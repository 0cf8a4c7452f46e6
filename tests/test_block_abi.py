"""Refusals of the block-scaled cache's entry points: answered on the host, before anything is launched."""
import ctypes

import pytest
import torch

import int8_kv_cache_token_gb300 as i8
from int8_kv_cache_token_gb300 import binding, build

P = ctypes.c_void_p
A = P(16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _reason():
    return i8.last_error()


def _write(lib, k=A, v=A, ks=1024, vs=1024, T=4, cu=A, sl=A, bt=A, B=2, Hkv=4, D=256, bs=16, mb=8, nb=10, kc=A, vc=A, sk=A, sv=A):
    return lib.i8kv_block_kv_write(k, v, ks, vs, T, cu, sl, bt, B, Hkv, D, bs, mb, nb, kc, vc, sk, sv, None)


@pytest.mark.parametrize("kw, status, word", [
    (dict(bs=8), 2, "block_size"), (dict(D=96), 2, "head_dim"), (dict(Hkv=0), 1, "Hkv"), (dict(Hkv=300), 2, "Hkv"),
    (dict(nb=0), 1, "num_blocks"), (dict(T=-1), 1, "T=-1"), (dict(B=-1), 1, "B=-1"), (dict(cu=None), 1, "cu_tokens"),
    (dict(sl=None), 1, "seq_lens"), (dict(bt=None), 1, "block_tables"), (dict(mb=0), 1, "max_blocks"),
    (dict(k=None), 1, "k is NULL"), (dict(v=P(24)), 1, "v must be 16-byte"), (dict(ks=1020), 1, "k_stride"),
    (dict(vs=-8), 1, "v_stride"), (dict(kc=None), 1, "cache"), (dict(sv=P(20)), 1, "aligned"),
    (dict(T=1 << 30, B=1 << 29), 2, "too large")])
def test_write_refusals(lib, kw, status, word):
    assert _write(lib, **kw) == status
    assert word in _reason()


def test_write_nothing(lib):
    assert _write(lib, T=0, k=None, v=None, cu=None) == 0
    assert _write(lib, B=0, T=0) == 0


def _read(lib, k=A, v=A, dt=1, T=4, cu=A, sl=A, bt=A, B=2, Hkv=4, D=256, bs=16, mb=8, nb=10, kc=A, vc=A, sk=A, sv=A):
    return lib.i8kv_block_kv_read(k, v, dt, T, cu, sl, bt, B, Hkv, D, bs, mb, nb, kc, vc, sk, sv, None)


@pytest.mark.parametrize("kw, status, word", [
    (dict(dt=2), 1, "out_dtype"), (dict(k=None), 1, "out is NULL"), (dict(v=P(8)), 1, "aligned"), (dict(D=32), 2, "head_dim"),
    (dict(cu=None), 1, "cu_tokens"), (dict(vc=P(17)), 1, "aligned"), (dict(T=-4), 1, "T=-4")])
def test_read_refusals(lib, kw, status, word):
    assert _read(lib, **kw) == status
    assert word in _reason()


def _decode(lib, out=A, dt=0, q=A, qs=24 * 256, kc=A, vc=A, sk=A, sv=A, bt=A, sl=A, kb=None, al=None, B=1, Hq=24, Hkv=4, D=256,
            bs=16, mb=8, nb=10, scale=0.0, cap=0.0, win=0, ws=A, n=1 << 30):
    return lib.i8kv_block_decode_attn(out, dt, q, qs, kc, vc, sk, sv, bt, sl, kb, al, B, Hq, Hkv, D, bs, mb, nb, scale, cap, win,
                                      ws, n, None)


ATTN = [(dict(dt=3), 1, "out_dtype"), (dict(out=None), 1, "out is NULL"), (dict(q=None), 1, "q is NULL"),
        (dict(qs=4), 1, "q_stride"), (dict(Hq=10), 1, "multiple"), (dict(Hq=0), 1, "multiple"), (dict(D=80), 2, "head_dim"),
        (dict(bs=32), 2, "block_size"), (dict(cap=-1.0), 1, "softcap"), (dict(cap=float("nan")), 1, "softcap"),
        (dict(cap=1e-5), 1, "softcap"), (dict(cap=float("inf")), 1, "softcap"), (dict(win=-1), 1, "window"),
        (dict(kc=None), 1, "cache"), (dict(nb=0), 1, "num_blocks"), (dict(Hq=8192), 2, "Hq")]
# calls that need a workspace on every device
BIG_DECODE = dict(B=1 << 16)
BIG_CHUNK = dict(C=5000)


@pytest.mark.parametrize("kw, status, word", ATTN + [
    (dict(sl=None), 1, "seq_lens"), (dict(mb=0), 1, "max_blocks"), (dict(B=-1), 1, "B="), (dict(B=1 << 28, mb=1 << 20), 2, "31 bits"),
    (dict(BIG_DECODE, ws=None), 3, "workspace"), (dict(BIG_DECODE, n=64), 3, "workspace"), (dict(BIG_DECODE, ws=P(24)), 1, "aligned")])
def test_decode_refusals(lib, kw, status, word):
    assert _decode(lib, **kw) == status
    assert word in _reason()


def _chunk(lib, out=A, dt=0, q=A, qs=24 * 256, kc=A, vc=A, sk=A, sv=A, bt=A, H=100, C=5, kb=None, ke=None, al=None, Hq=24, Hkv=4,
           D=256, bs=16, nb=10, scale=0.0, cap=0.0, win=0, ws=A, n=1 << 30):
    return lib.i8kv_block_prefix_attn(out, dt, q, qs, kc, vc, sk, sv, bt, H, C, kb, ke, al, Hq, Hkv, D, bs, nb, scale, cap, win, ws,
                                      n, None)


@pytest.mark.parametrize("kw, status, word", ATTN + [(dict(bt=None), 1, "block_table"), (dict(H=-1), 1, "history_len"),
                                                     (dict(C=-2), 1, "chunk_len"), (dict(H=1 << 30), 2, "history_len"),
                                                     (dict(BIG_CHUNK, ws=None), 3, "workspace"),
                                                     (dict(BIG_CHUNK, n=64), 3, "workspace"),
                                                     (dict(BIG_CHUNK, ws=P(24)), 1, "aligned")])
def test_chunk_refusals(lib, kw, status, word):
    assert _chunk(lib, **kw) == status
    assert word in _reason()


def test_empty_calls_and_workspace_sizes(lib):
    assert _decode(lib, B=0, ws=None) == 0 and _chunk(lib, C=0, ws=None, bt=None) == 0
    for D in (64, 128, 256):
        assert lib.i8kv_block_decode_workspace_bytes(1 << 16, 24, 4, D, 100) > 0
        assert lib.i8kv_block_prefix_workspace_bytes(0, 5000, 24, 4, D) > 0
        # few rows over so many keys that their list of blocks would pass 31 bits: as 128-row blocks, on 16-bit tiles
        assert lib.i8kv_block_prefix_workspace_bytes((1 << 30) - 64, 8, 64, 64, D) > (1 << 30) * 64 * D * 4
    assert lib.i8kv_block_decode_workspace_bytes(1, 24, 4, 96, 100) == 0
    assert lib.i8kv_block_decode_workspace_bytes(1, 23, 4, 128, 100) == 0
    assert lib.i8kv_block_prefix_workspace_bytes(-1, 5, 24, 4, 128) == 0


def test_binding_refuses_host_tensors():
    c = i8.alloc_block_cache(4, 2, 64, device="cpu")
    bt, sl = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(i8.I8KVError, match="CUDA"):
        i8.block_kv_write(k, k, sl, bt, **c)
    with pytest.raises(i8.I8KVError, match="CUDA"):
        i8.block_decode_attn(torch.zeros(1, 2, 64), k, **c, block_tables=bt, seq_lens=sl)
