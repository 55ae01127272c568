"""Calls without rows or streams take empty tensors, whose address is null, and
still refuse everything else (CPU: nothing is launched)."""
import ctypes

import pytest

from decode_step_gb300 import _lib
from decode_step_gb300._lib import KVCacheDesc, lib

A = 0x10000  # an aligned address that nothing reads


def kv(**kw):
    d = dict(num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, dtype=_lib.TTS_BF16, k_pool=A, v_pool=A)
    d.update(kw)
    return KVCacheDesc(*d.values())


def append(cache, B, rows, rope=10000.0, start=A, row=None, table=None, Hq=4):
    ref = None if cache is None else ctypes.byref(cache)
    return lib().tts_kv_append_packed(ref, table, 4, table, B, start, rows, Hq, rope, row, row, row, row, None, None)


def prompt(cache, B, rows, start=A, row=None, table=None, win=0, Hq=4):
    ref = None if cache is None else ctypes.byref(cache)
    return lib().tts_prompt_attn(ref, table, 4, table, B, start, rows, Hq, 0.1, win, 0, row, row, None, 0, None, None)


@pytest.mark.parametrize("dtype", [_lib.TTS_BF16, _lib.TTS_FP8_E4M3])
def test_nothing_to_do(dtype):
    c = kv(dtype=dtype)
    for call in (append, prompt):
        assert call(c, 2, 0, table=A) == 0 and call(c, 0, 0) == 0 and call(c, 0, 5, row=A) == 0
    assert append(c, 2, 0, rope=0.0, table=A) == 0


def test_what_is_missing_is_refused():
    c = kv()
    for call in (append, prompt):
        assert call(c, 2, 5, table=A) == -1 and call(c, 2, 5, row=A) == -1   # rows without tensors, or tables
        assert call(c, 2, 0, start=None) == -1 and call(None, 0, 0) == -1
        assert call(kv(k_pool=None), 2, 0) == -1 and call(kv(block_size=32), 2, 0) == -2
        assert call(c, 2, 0, Hq=3) == -1 and call(c, -1, 0) == -1 and call(c, 2, -1) == -1
        assert call(c, 2, 0, row=A + 8, table=A) == -1
    assert append(c, 2, 0, rope=0.5) == -1 and prompt(c, 2, 0, win=-1) == -1
