"""tts_window_decode_attn against the 64-bit reference: windows, sinks and
their edges, types, head groups, causal rows, blocks given back, values that
are not finite, refused streams, streams of work, captured calls."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd


def upload(s):
    pools = tuple(None if p is None else p.cuda() for p in s["pools"])
    return bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda()


def run(s, q_len, err=None, max_ctx=None, window=None, ws=None):
    cache, table, lens = upload(s)
    B, top = len(s["new"]), max_ctx or max(max(s["ctx"]), q_len)
    q = s["q"].cuda().view(B, q_len, s["Hq"], s["D"])
    out = torch.full_like(q, 7.0)
    if ws is None:
        ws = torch.zeros(bd.tts_decode_attn_workspace_size(B, q_len, s["Hq"], s["Hkv"], s["D"], top), dtype=torch.uint8,
                         device="cuda")
    bd.tts_window_decode_attn(cache, table, lens, top, q, out, ws, s["scale"], s["window"] if window is None else window,
                              s["sinks"], causal=s["causal"], err=err)
    torch.cuda.synchronize()
    return out.view(-1, s["Hq"], s["D"])


CTX = [1, 15, 16, 17, 40, 255, 256, 257, 700]


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (15, 4), (16, 16), (17, 37), (100, 0), (256, 4), (5000, 4), (33, 640),
                                          (2, 5000)])
def test_windows(dtype, window, sinks):
    s = pr.make([1] * len(CTX), [c - 1 for c in CTX], 4, 2, dtype, window, sinks, causal=False, seed=window + sinks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, 1, err)
    assert int(err.item()) == 0
    pr.check(out, *pr.attend_all(s))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("q_len,Hq,Hkv", [(5, 4, 2), (2, 16, 2), (5, 3, 1), (16, 1, 1), (1, 16, 1), (3, 20, 4), (1, 8, 8)])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_and_groups(dtype, q_len, Hq, Hkv, causal):
    ctx = [q_len, q_len + 1, 31 + q_len, 48 + q_len, 300]
    s = pr.make([q_len] * len(ctx), [c - q_len for c in ctx], Hq, Hkv, dtype, 21, 5, causal, seed=q_len * Hq)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, q_len, err)
    assert int(err.item()) == 0
    pr.check(out, *pr.attend_all(s))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_a_window_past_every_context_changes_nothing(dtype):
    s = pr.make([3] * 4, [0, 30, 61, 900], 4, 2, dtype, 0, 0, True, seed=9)
    out = run(s, 3, window=2 ** 31 - 1)
    cache, table, lens = upload(s)
    q = s["q"].cuda().view(4, 3, 4, s["D"])
    ref = torch.empty_like(q)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(4, 3, 4, 2, s["D"], 903), dtype=torch.uint8, device="cuda")
    bd.tts_decode_attn(cache, table, lens, 903, q, ref, ws, s["scale"], True)
    assert torch.equal(out, ref.view_as(out))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(dtype, value):
    """Token 40 leaves the windows of rows 1 and 2, token 59 is seen by row 2
    alone, token 3 is a sink that all see, and 4 and 20 are seen by none."""
    s = pr.make([3], [57], 4, 2, dtype, 18, 4, True, seed=3, hide=False)
    vis = pr.visible(s, 0)
    assert vis[:, 40].tolist() == [True, False, False] and vis[:, 59].tolist() == [False, False, True]
    for t, d in ((40, 5), (59, 127), (3, 64), (4, 9), (20, 11)):
        if dtype == "fp8":
            if value == value:
                pytest.skip("codes hold no infinities")
            b = int(s["table"][0, t // 16])
            rec = s["pools"][0][b, 1]
            rec[2048 + 16 * d + 4 * (t % 8 // 2) + t % 2 + 2 * (t % 16 // 8)] = 0xFF
            s["v_val"][b, 1, t % 16, d] = value
        else:
            b = int(s["table"][0, t // 16])
            s["v_pool"][b, 1, t % 16, d] = value
            s["k_pool"][b, 1, t % 16, d] = value if t in (4, 20) else s["k_pool"][b, 1, t % 16, d]
    if dtype != "fp8":
        pr.finish(s)
    ref, tol = pr.attend_all(s)
    assert not torch.isfinite(ref).all() and torch.isfinite(ref[:, 2:, 9]).all()
    pr.check(run(s, 3), ref, tol)


def test_refused_streams_and_bad_blocks():
    s = pr.make([2] * 5, [20, 30, 98, 55, 200], 4, 2, "bf16", 40, 4, True, seed=5, max_blocks=13)
    s["ctx_lens"][1] = 1              # fewer than its rows
    s["ctx_lens"][2] = 13 * 16 + 1    # past the table
    s["table"][3, 2] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, 2, err, max_ctx=400)
    assert int(err.item()) == _lib.ERRBIT_CTX_LEN | _lib.ERRBIT_BLOCK_ID
    pr.check(out, *pr.attend_all(s, skip=(1, 2)))


def test_rows_whose_blocks_are_all_gone_get_zeros():
    s = pr.make([1, 1], [39, 39], 4, 2, "bf16", 8, 0, False, seed=6)
    s["table"][1] = -1
    out = run(s, 1)
    pr.check(out, *pr.attend_all(s))
    assert not out[1].any()


def test_long_context_split_over_many_warps():
    s = pr.make([1], [30000], 4, 1, "bf16", 20000, 100, False, seed=8)
    pr.check(run(s, 1), *pr.attend_all(s))


def test_captured_and_replayed_with_new_lengths():
    s = pr.make([1] * 3, [50, 300, 700], 4, 2, "bf16", 64, 4, False, seed=11, hide=False, garbage=0.0)
    cache, table, lens = upload(s)
    q = s["q"].cuda().view(3, 1, 4, 128)
    out = torch.empty_like(q)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(3, 1, 4, 2, 128, 701), dtype=torch.uint8, device="cuda")

    def call():
        bd.tts_window_decode_attn(cache, table, lens, 701, q, out, ws, s["scale"], 64, 4)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for lengths in ([51, 301, 701], [1, 17, 400]):
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        direct = torch.empty_like(q)
        bd.tts_window_decode_attn(cache, table, lens, 701, q, direct, ws, s["scale"], 64, 4)
        assert torch.equal(out, direct)
        s["ctx"] = lengths
        s["before"] = [c - 1 for c in lengths]
        ref, tol = pr.attend_all(s)
        # (tokens that the first lengths hid hold zeros: values like others)
        pr.check(out.view(3, 4, 128), ref, tol)


def test_refusals():
    s = pr.make([1], [20], 4, 2, "bf16", 8, 0, False)
    cache, table, lens = upload(s)
    q = s["q"].cuda().view(1, 1, 4, 128)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(1, 1, 4, 2, 128, 21), dtype=torch.uint8, device="cuda")
    for kw, code in ((dict(window=0), -1), (dict(window=-4), -1), (dict(window=4, sinks=-1), -1)):
        with pytest.raises(bd.TTSError) as e:
            bd.tts_window_decode_attn(cache, table, lens, 21, q, torch.empty_like(q), ws, 0.1, **kw)
        assert e.value.code == code
    with pytest.raises(bd.TTSError) as e:
        bd.tts_window_decode_attn(cache, table, lens, 21, q, torch.empty_like(q), ws[:64], 0.1, 8)
    assert e.value.code == -3
    with pytest.raises(ValueError):
        bd.tts_window_decode_attn(cache, table, lens, 21, q.float(), torch.empty_like(q), ws, 0.1, 8)
    with pytest.raises(ValueError):
        bd.tts_window_decode_attn(cache, table.cpu(), lens, 21, q, torch.empty_like(q), ws, 0.1, 8)
