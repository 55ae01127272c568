"""Limits of the latent-cache calls on the host (CPU only)."""
import ctypes

import pytest

import decode_step_gb300 as pkg
from decode_step_gb300 import _lib
from decode_step_gb300.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return pkg.lib()


def test_latent_stalls_are_modes(L):
    for what in (_lib.TEST_STALL_LATENT_DECODE, _lib.TEST_STALL_LATENT_PREFILL):
        assert L.tts_test_set_stall(what, 10_000) == 0
    for what in (-1, 3, 6):
        assert L.tts_test_set_stall(what, 10_000) == -1
    assert L.tts_test_set_stall(_lib.TEST_STALL_NONE, 2_000_000_000) == 0


def test_rows_that_are_too_many(L):
    """B * q_len up to 2^20 for the decode attention, B for prompts; num_q_heads
    * q_len up to 1024."""
    ws = L.tts_latent_decode_attn_workspace_size
    assert ws(1 << 20, 1, 2, 64, 64, 64, 16) > 0 and ws((1 << 20) + 1, 1, 2, 64, 64, 64, 16) == 0
    assert ws(1 << 18, 4, 2, 64, 64, 64, 16) > 0 and ws((1 << 18) + 1, 4, 2, 64, 64, 64, 16) == 0
    fake = ctypes.c_void_p(0x10000)    # never dereferenced: the calls fail validation first
    cache = _lib.LatentCacheDesc(8, 16, 64, 64, 1, fake)

    def decode(B, q_len, Hq):
        return L.tts_latent_decode_attn(ctypes.byref(cache), fake, 4, fake, 16, B, q_len, Hq, 64, 64, 0.1, 0, fake, fake, fake,
                                        fake, fake, fake, 0, None, None)

    assert decode(1 << 20, 1, 2) == -3 and decode((1 << 20) + 1, 1, 2) == -2       # too little workspace; too many rows
    assert decode(1, 512, 2) == -3 and decode(1, 513, 2) == -2
    pws = L.tts_latent_prefill_attn_workspace_size
    assert pws(1 << 20, 8, 2, 64, 64, 64, 16) > 0 and pws((1 << 20) + 1, 8, 2, 64, 64, 64, 16) == 0
