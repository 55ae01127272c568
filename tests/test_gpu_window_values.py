"""tts_window_decode_attn: values that are not finite in fp32 caches, and scores
far below zero."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd

NAN, INF = float("nan"), float("inf")


def attend(s, q_len, window=None):
    """tts_window_decode_attn's output; with window 0 tts_decode_attn's."""
    pools = tuple(None if p is None else p.cuda() for p in s["pools"])
    cache, table, lens = bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda()
    B, top = len(s["new"]), max(s["ctx"])
    q = s["q"].cuda().view(B, q_len, s["Hq"], s["D"])
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(B, q_len, s["Hq"], s["Hkv"], s["D"], top), dtype=torch.uint8,
                     device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    window = s["window"] if window is None else window
    if window:
        bd.tts_window_decode_attn(cache, table, lens, top, q, out, ws, s["scale"], window, s["sinks"], causal=s["causal"],
                                  err=err)
    else:
        bd.tts_decode_attn(cache, table, lens, top, q, out, ws, s["scale"], s["causal"], err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.view(-1, s["Hq"], s["D"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("low", [False, True])
def test_values_that_are_not_finite_show_whatever_their_weight(dtype, value, low):
    """Token 40 leaves the windows of rows 1 and 2, token 59 is seen by row 2 alone, token 3 is a
    sink that all see, 4 and 20 are seen by none.  `low`: the scores of 3, 40 and 59 lie so far
    below the others that their weights are zero, and zero times an infinity is no number."""
    s = pr.make([3], [57], 4, 2, dtype, 18, 4, True, seed=3, hide=False)
    s["q"] = s["q"].abs() + 0.5
    for t, d in ((40, 5), (59, 33), (3, 60), (4, 9), (20, 11)):
        b = int(s["table"][0, t // 16])
        s["v_pool"][b, 1, t % 16, d] = value
        if t in (4, 20):
            s["k_pool"][b, 1, t % 16, d] = value
        elif low:
            s["k_pool"][b, 1, t % 16] = -200.0
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    assert torch.isfinite(ref[:, :2]).all() and torch.isfinite(ref[:, 2:, 9]).all()
    got = attend(s, 3).cpu()
    bad = ~torch.isfinite(ref)
    assert [int(bad[r].sum()) for r in range(3)] == [4, 2, 4]
    assert torch.equal(~torch.isfinite(got.double()), bad)
    if not (low and dtype == "bf16"):
        pr.check(got, ref, tol)
    else:
        # (bf16: values of tiles at an edge are given to their rows as they are)
        ref, got, tol = (x.masked_fill(bad, 0.0) for x in (ref, got, tol))
        pr.check(got, ref, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("size", [1e27, 1e30, 1e34])
def test_scores_far_below_zero_have_weights(dtype, window, size):
    """Keys that point away from the queries, in steps of which the first takes it all: scores of
    -1e28 to -2e35, in one part and in parts of several warps.  Without a window the plain decode."""
    s = pr.make([2, 2], [3, 5000], 4, 2, dtype, window, 4 if window else 0, True, seed=61)
    s["q"] = torch.ones_like(s["q"])
    steps = torch.where(torch.rand(s["k_pool"].shape[:3], generator=torch.Generator().manual_seed(62)) < 0.25, 1.0, 2.0)
    k = (-size * steps)[..., None].expand(s["k_pool"].shape)
    s["k_pool"] = torch.where(torch.isfinite(s["k_pool"]), k.to(s["k_pool"].dtype), s["k_pool"])
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    assert torch.isfinite(ref).all() and bool((ref.abs().amax(-1) > 0.01).all())
    pr.check(attend(s, 2, window), ref, tol)
