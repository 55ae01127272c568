"""The latent attentions' bounded waits give up, flag TTS_ERRBIT_TIMEOUT and
return.

A test-only stall (tts_test_set_stall) makes the first tile of every CTA expect
16 bytes more than its copies deliver.  With a short wait limit the kernels
must finish, flag the timeout, and leave the context usable: the same call
without the stall is then right.  Nothing here faults, traps or hangs: every
wait is bounded and the stall only withholds a completion."""
from __future__ import annotations

import pytest
import torch

import latent_ref as ref
from test_gpu_latent import check, run_decode, run_prefill, up

pytestmark = pytest.mark.gpu

LIMIT = 200_000  # SM clock cycles per wait, about 0.1 ms


@pytest.fixture
def bd():
    from decode_step_gb300 import binding
    yield binding
    binding.tts_test_set_stall(binding._lib.TEST_STALL_NONE)


def stalled_then_right(bd, what, call, want, tol):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.tts_test_set_stall(what, LIMIT)
    call(err)
    torch.cuda.synchronize()           # the kernels returned
    assert int(err) & bd._lib.ERRBIT_TIMEOUT
    bd.tts_test_set_stall(bd._lib.TEST_STALL_NONE)
    err.zero_()
    out = call(err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(out.view(want.shape), want, tol)


@pytest.mark.parametrize("q_len,Hq", [(1, 16), (3, 16), (4, 16)])     # 16, 48 and 64 rows a group
def test_decode_wait_times_out(bd, q_len, Hq):
    s = ref.make([q_len] * 6, [20, 900, 64, 3, 400, 130], Hq, 512, 128, 128, 301)
    d = up(s)
    want, tol = ref.attend_all(s, True, True)
    stalled_then_right(bd, bd._lib.TEST_STALL_LATENT_DECODE, lambda err: run_decode(bd, s, d, q_len, True, err), want, tol)


@pytest.mark.parametrize("nope,v", [(64, 64), (128, 128)])
def test_prefill_wait_times_out(bd, nope, v):
    s = ref.make([300, 7, 130], [0, 400, 5], 4, 256, nope, v, 302)
    d = up(s)
    want, tol = ref.attend_all(s, True, False)
    stalled_then_right(bd, bd._lib.TEST_STALL_LATENT_PREFILL, lambda err: run_prefill(bd, s, d, err), want, tol)
