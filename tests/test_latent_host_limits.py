"""Limits of the latent-cache calls on the host (CPU only)."""
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
