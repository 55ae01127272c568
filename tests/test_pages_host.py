"""Block pool owners and compaction, and the refusals of the prompt, window and
page calls (CPU: arguments are checked before anything is launched)."""
import ctypes

import pytest

from decode_step_gb300 import _lib
from decode_step_gb300 import binding as bd
from decode_step_gb300._lib import KVCacheDesc, LatentCacheDesc, TTSError, lib

A = 0x10000  # an aligned address that nothing reads: every call here is refused


def test_shared_blocks_are_free_once_every_owner_has_freed_them():
    pool = bd.BlockPool(6)
    ids = pool.alloc(4)
    pool.share(ids[:2])
    pool.share(ids[1:2])
    assert [pool.owners(i) for i in range(6)] == [2, 3, 1, 1, 0, 0]
    pool.free(ids)
    assert [pool.owners(i) for i in range(6)] == [1, 2, 0, 0, 0, 0] and pool.num_free == 4
    pool.free([0, 1])
    assert pool.num_free == 5
    pool.free([1])
    assert pool.num_free == 6
    assert pool.alloc(1) == [1]  # last freed, first out


@pytest.mark.parametrize("ids", [[4], [0, 0], [-1], [6], [0, 1, 5]])
def test_share_and_free_are_all_or_nothing(ids):
    pool = bd.BlockPool(6)
    pool.alloc(2)
    pool.share([0])
    for call in (pool.share, pool.free):
        with pytest.raises(TTSError) as e:
            call(ids)
        assert e.value.code == -1
    assert [pool.owners(i) for i in range(6)] == [2, 1, 0, 0, 0, 0] and pool.num_free == 4
    for i in (-1, 6):
        with pytest.raises(TTSError):
            pool.owners(i)


def test_compaction_closes_the_gaps():
    pool = bd.BlockPool(10)
    pool.alloc(10)
    pool.free([8, 1, 0, 5, 3])
    pool.share([9, 4])
    assert pool.compact() == [0, 1, 2, 3, 4, 5, 0, 1, 8, 3]   # 2, 4, 6, 7, 9 in use
    assert [pool.owners(i) for i in range(10)] == [1, 1, 1, 2, 2, 0, 0, 0, 0, 0]
    assert pool.compact() == list(range(10))
    assert pool.alloc(3) == [5, 6, 7] and pool.num_free == 2
    pool.free([0])
    assert pool.num_free == 3


def test_compaction_of_full_and_empty_pools():
    pool = bd.BlockPool(3)
    assert pool.compact() == [0, 1, 2] and pool.alloc(3) == [0, 1, 2]
    assert pool.compact() == [0, 1, 2] and pool.num_free == 0
    assert lib().tts_block_pool_compact(None, (ctypes.c_int32 * 3)()) == -1
    assert lib().tts_block_pool_share(None, (ctypes.c_int32 * 3)(), 1) == -1
    assert lib().tts_block_pool_owners(None, 0) == -1


def kv(**kw):
    d = dict(num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, dtype=_lib.TTS_BF16, k_pool=A, v_pool=A)
    d.update(kw)
    return KVCacheDesc(*d.values())


BAD_CACHES = [(dict(num_blocks=0), -1), (dict(block_size=32), -2), (dict(k_pool=None), -1), (dict(v_pool=None), -1),
              (dict(k_pool=A + 8), -1), (dict(dtype=7), -2)]


def moves(cache, n=1, B=1, blocks=4, src=A, table=A):
    """Status of the three page moves."""
    r, L = ctypes.byref(cache), lib()
    return [L.tts_kv_copy_blocks(r, src, A, n, None, None),
            L.tts_kv_fork(r, table, blocks, A, B, src, A, A, n, None, None),
            L.tts_kv_compact(r, src, table, blocks, B, None, None)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_page_moves_refuse_bad_caches(kw, code):
    assert moves(kv(**kw)) == [code] * 3


def test_page_moves_refuse_bad_arguments():
    c = kv()
    assert moves(c, n=-1)[:2] == [-1, -1]
    assert moves(c, src=None) == [-1, -1, -1]
    assert moves(c, table=None)[1:] == [-1, -1]
    assert moves(c, blocks=0)[1:] == [-1, -1]
    assert moves(c, blocks=(1 << 20) + 1)[1:] == [-1, -1]
    assert moves(c, B=-1)[1:] == [-1, -1]
    r = ctypes.byref(c)
    assert lib().tts_kv_copy_blocks(r, None, None, 0, None, None) == 0   # nothing to copy
    assert lib().tts_kv_copy_blocks(None, A, A, 1, None, None) == -1
    lat = LatentCacheDesc(8, 16, 100, 64, _lib.TTS_BF16, A)
    assert lib().tts_latent_copy_blocks(ctypes.byref(lat), A, A, 1, None, None) == -2
    assert lib().tts_latent_compact(ctypes.byref(lat), A, A, 4, 1, None, None) == -2
    assert lib().tts_latent_fork(None, A, 4, A, 1, A, A, A, 1, None, None) == -1


def packed(cache, B=2, start=A, rows=5, Hq=4, base=0.0, q=None, q_out=None, k=A):
    return lib().tts_kv_append_packed(ctypes.byref(cache), A, 4, A, B, start, rows, Hq, base, q, q_out, k, A, None, None)


def test_packed_append_refusals():
    c = kv()
    assert packed(c, start=None) == -1
    assert packed(c, B=-1) == -1 and packed(c, B=(1 << 20) + 1) == -1
    assert packed(c, rows=-1) == -1
    assert packed(c, k=None) == -1 and packed(c, k=A + 2) == -1
    assert packed(c, base=10000.0) == -1                      # no queries
    assert packed(c, base=10000.0, q=A) == -1                 # nowhere to put them
    assert packed(c, base=10000.0, q=A, q_out=A + 4) == -1
    assert packed(c, base=0.5, q=A, q_out=A) == -1
    assert packed(c, base=10000.0, q=A, q_out=A, Hq=3) == -1
    assert packed(kv(dtype=_lib.TTS_F32, head_dim=64), base=10000.0, q=A, q_out=A) == -2
    assert packed(c, B=0) == 0 and packed(c, rows=0) == 0     # nothing to append


def window(cache, window=8, sinks=0, B=1, q_len=1, Hq=4, max_ctx=64, scale=0.1, ws=1 << 30):
    return lib().tts_window_decode_attn(ctypes.byref(cache), A, 4, A, max_ctx, B, q_len, Hq, scale, 0, window, sinks, A, A,
                                        A, ws, None, None)


def test_window_refusals():
    c = kv()
    assert window(c, window=0) == -1 and window(c, sinks=-1) == -1
    assert window(c, Hq=3) == -1 and window(c, scale=0.0) == -1
    assert window(c, q_len=9) == -2                            # 18 rows a KV head
    assert window(c, ws=16) == -3
    assert window(kv(head_dim=64)) == -2
    assert window(c, B=0) == 0


def prompt(cache, B=2, start=A, rows=5, Hq=4, scale=0.1, win=0, sinks=0, q=A, ws=1 << 30, ws_at=A, blocks=4):
    return lib().tts_prompt_attn(ctypes.byref(cache), A, blocks, A, B, start, rows, Hq, scale, win, sinks, q, A, ws_at, ws,
                                 None, None)


def test_prompt_refusals():
    c = kv()
    assert prompt(c, start=None) == -1 and prompt(c, q=None) == -1 and prompt(c, q=A + 8) == -1
    assert prompt(c, B=-1) == -1 and prompt(c, rows=-1) == -1
    assert prompt(c, win=-1) == -1 and prompt(c, sinks=-1) == -1
    assert prompt(c, scale=0.0) == -1 and prompt(c, scale=float("nan")) == -1 and prompt(c, scale=float("inf")) == -1
    assert prompt(c, Hq=3) == -1 and prompt(c, Hq=0) == -1
    assert prompt(c, blocks=0) == -1 and prompt(c, blocks=(1 << 20) + 1) == -1
    assert prompt(kv(dtype=_lib.TTS_F32, head_dim=64)) == -2 and prompt(kv(head_dim=64)) == -2
    assert prompt(c, Hq=258) == -2 and prompt(c, B=4097) == -2
    assert prompt(kv(num_blocks=1 << 27)) == -2                # 2^32 rows of keys
    assert prompt(c, ws=1000) == -3 and prompt(c, ws_at=None) == -3 and prompt(c, ws_at=A + 16) == -3
    assert prompt(c, blocks=1 << 20, rows=1 << 24, Hq=256) == -2   # tiles past 2^30
    assert prompt(c, B=0) == 0 and prompt(c, rows=0) == 0
    size = lib().tts_prompt_attn_workspace_size
    assert size(1, 1, 4, 2, 128) == size(4096, 10 ** 6, 128, 1, 128) > 0
    assert size(1, 1, 3, 2, 128) == 0 and size(1, 1, 4, 2, 64) == 0 and size(4097, 1, 4, 2, 128) == 0
    assert size(-1, 1, 4, 2, 128) == 0 and size(1, 1, 129, 1, 128) == 0
