"""Prompts that are refused beside prompts that are not (GPU)."""
from __future__ import annotations

import pytest
import torch

import latent_ref as ref
from test_gpu_latent import CTX_LEN, NAN, check, poisoned, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    from decode_step_gb300 import binding
    return binding


def test_a_refused_long_prompt_does_not_hold_up_the_others(bd):
    """Its rows get zeros in no more than a few times what attending over them
    would take, and the other stream's are right."""
    Hq, L, v, rows = 16, 64, 128, 8191
    s = ref.make([40, rows, 30], [0, 0, 9], Hq, L, 64, v, 71, garbage=0.0)
    d = up(s)
    cache = bd.LatentCache(d["pool"], L)
    total = sum(s["ctx"])
    ws = poisoned(bd.tts_latent_prefill_attn_workspace_size(3, s["T"], Hq, L, 64, v, total))
    out = torch.full((s["T"], Hq, v), NAN, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = s["ctx_lens"].clone()
    bad[1] = rows - 1                                     # fewer than its rows
    bad = bad.cuda()

    def ms(lens):
        best = 1e9
        for _ in range(4):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            bd.tts_latent_prefill_attn(cache, d["table"], lens, total, d["row_start"], d["q_nope"], d["q_rope"], d["w_uk"],
                                       d["w_uv"], out, ws, s["scale"], err=err)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    served = ms(d["ctx_lens"])
    assert int(err) == 0
    out.fill_(NAN)
    refused = ms(bad)
    assert int(err) == CTX_LEN
    assert (out[40:40 + rows] == 0).all()
    for b, at in ((0, 0), (2, 40 + rows)):
        want, tol = ref.attend(s, b, True, False)
        check(out[at:at + s["new"][b]], want, tol, f"stream {b}")
    assert refused < 2 * served, f"{refused:.3f} ms with the prompt refused, {served:.3f} ms with it served"


@pytest.mark.parametrize("B", [3, 40, 500])
def test_many_refused_streams(bd, B):
    Hq, L, v = 3, 64, 64
    new = [1 + (7 * i) % 11 for i in range(B)]
    s = ref.make(new, [2] * B, Hq, L, 64, v, 72, garbage=0.0)
    lens = s["ctx_lens"].clone()
    refused = [b for b in range(B) if b % 3 == 1]
    for b in refused:
        lens[b] = new[b] - 1 if b % 2 else 16 * s["table"].shape[1] + 1
    d = up(s)
    total = sum(s["ctx"])
    ws = poisoned(bd.tts_latent_prefill_attn_workspace_size(B, s["T"], Hq, L, 64, v, total))
    out = torch.full((s["T"] + 5, Hq, v), NAN, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.tts_latent_prefill_attn(bd.LatentCache(d["pool"], L), d["table"], lens.cuda(), total, d["row_start"], d["q_nope"],
                               d["q_rope"], d["w_uk"], d["w_uv"], out[:s["T"]], ws, s["scale"], err=err)
    want, tol = ref.attend_all(s, True, False, skip=refused)
    check(out[:s["T"]], want, tol)
    assert torch.isnan(out[s["T"]:].float()).all() and int(err) == CTX_LEN
