"""LatentStep on more than one CUDA stream: whose memory a prompt's output is,
and calls that would otherwise share buffers (GPU)."""
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


def rotated(s):
    """The prompt rows' rotated queries, to half a step of bf16."""
    pos = torch.cat([torch.arange(n) for n in s["new"]])
    return ref.rotate(s["q_rope"], pos[:, None], 10000.0).to(torch.bfloat16)


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


def test_prompt_and_step_have_buffers_of_their_own(setup):
    """A prompt beside running steps: neither's queries nor workspace are the
    other's."""
    s, d, step, args = setup
    step.prompt(*args)
    prompt_q = step.q[:93]
    prompt_bits = prompt_q.clone()
    step(*token(d, s)[0])
    torch.cuda.synchronize()
    assert torch.equal(prompt_q, prompt_bits)


def test_prompt_beside_steps(setup):
    """Prompts of one stream and steps of another, overlapping, into separate
    blocks: each call's result is that of the call alone."""
    from decode_step_gb300 import binding as bd
    s, d, step, args = setup
    # the prompts' streams have blocks of their own
    other = torch.tensor([i for i in range(s["pool"].shape[0]) if i not in s["table"].flatten().tolist()][:24], dtype=torch.int32).view(2, 12).cuda()
    pargs = (other,) + args[1:]
    targs, _ = token(d, s)
    want_out = step.prompt(*pargs).clone()
    step(*targs)
    torch.cuda.synchronize()
    want_step, want_ids = step.out.clone(), step.ids.clone()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for _ in range(30):
        outs = []
        for _ in range(10):
            outs.append(step.prompt(*pargs, stream=side))
            step(*targs, stream=main)
        torch.cuda.synchronize()
        assert torch.equal(step.out, want_step) and torch.equal(step.ids, want_ids)
        for o in outs:
            assert torch.equal(o, want_out)
    assert int(step.err) == 0


@pytest.mark.parametrize("kind", ["prompt", "step"])
def test_calls_of_one_kind_follow_one_another(setup, kind):
    """Two prompts (or steps) on two streams use the same buffers: the second
    waits for the first."""
    s, d, step, args = setup
    targs, _ = token(d, s)
    call = (lambda st: step.prompt(*args, stream=st)) if kind == "prompt" else (lambda st: step(*targs, stream=st))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(PAUSE)
    call(a)
    after_a, after_b = torch.cuda.Event(), torch.cuda.Event()
    after_a.record(a)
    call(b)
    after_b.record(b)
    after_b.synchronize()
    assert after_a.query()


def test_a_step_is_captured_after_calls_on_other_streams(setup):
    """Inside a capture there is no waiting for work before it."""
    s, d, step, args = setup
    targs, e = token(d, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(*targs, stream=side)
    step.prompt(*args, stream=side)
    torch.cuda.synchronize()
    want = step.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*targs)
    step.out.fill_(NAN)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, want)
    step(*targs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(step.out, want)
    t = dict(s, pool=d["pool"].cpu(), q_rope=rotated(s))
    want, tol = ref.attend_all(t, True, False)
    out = step.prompt(*args)
    # (the reference's rotated queries may be rounded the other way: half a step of each of 64, a score's size)
    check(out, want, tol + 2.0 ** -8 * want.abs().amax(), "prompt")
