"""LatentStep on more than one CUDA stream: whose memory a prompt's output is
(GPU)."""
from __future__ import annotations

import pytest
import torch

import latent_ref as ref
from test_gpu_latent import NAN, check, up

pytestmark = pytest.mark.gpu

HQ, LAT, V, CODES = 8, 128, 64, 300
PAUSE = 40_000_000        # SM clock cycles, some 20 ms


@pytest.fixture
def setup():
    from decode_step_gb300 import binding as bd
    from decode_step_gb300.step import LatentStep
    s = ref.make([60, 33], [0, 0], HQ, LAT, 64, V, 201, max_blocks=12, spare=60)
    s["table"] = torch.randperm(s["pool"].shape[0], generator=torch.Generator().manual_seed(7))[:24].to(torch.int32).view(2, 12).contiguous()
    s["pool"].fill_(NAN)
    d = up(s)
    W = (torch.randn(CODES, HQ * V, generator=torch.Generator().manual_seed(8)) * 0.2).to(torch.bfloat16).cuda()
    step = LatentStep(bd.LatentCache(d["pool"], LAT), d["w_uk"], d["w_uv"], W, 2, 160, prompt_rows=100, prompt_ctx=200)
    args = (d["table"], d["ctx_before"], d["ctx_lens"], d["row_start"], d["q_nope"], d["q_rope"], d["c_new"], d["kr_new"])
    # (the first call of a process loads the kernels, which waits for the GPU)
    step.prompt(*args)
    step(*token(d, s)[0])
    torch.cuda.synchronize()
    return s, d, step, args


def token(d, s):
    e = ref.make([1] * 2, s["ctx"], HQ, LAT, 64, V, 202)
    u = up(e)
    return (d["table"], u["ctx_before"], u["ctx_lens"], u["q_nope"].view(2, 1, HQ, 64), u["q_rope"].view(2, 1, HQ, 64),
            u["c_new"], u["kr_new"]), e


def test_prompt_output_belongs_to_its_stream(setup):
    """Memory freed on the current stream with work still to run on it is not
    the output of a prompt on another stream."""
    s, d, step, args = setup
    side = torch.cuda.Stream()
    want = step.prompt(*args)
    torch.cuda.synchronize()
    n = want.numel()
    held = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    torch.cuda._sleep(PAUSE)
    held.fill_(7.0)
    del held
    out = step.prompt(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
