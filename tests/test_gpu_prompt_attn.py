"""tts_prompt_attn against the 64-bit reference: lengths from one row to many,
head groups, windows, sinks and their edges, ragged and refused streams, values
that are not finite, work split over CTAs, captured calls."""
from __future__ import annotations

import math

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd

DTYPES = ["bf16", "fp8"]


def upload(s):
    pools = tuple(None if p is None else p.cuda() for p in s["pools"])
    return bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda(), s["row_start"].cuda()


def workspace(s):
    n = bd.tts_prompt_attn_workspace_size(len(s["new"]), s["T"], s["Hq"], s["Hkv"], s["D"])
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def run(s, err=None, ws=None, q=None):
    cache, table, lens, start = upload(s)
    q = s["q"].cuda() if q is None else q
    out = torch.full_like(q, 7.0)
    ws = workspace(s) if ws is None else ws
    bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"], s["window"], s["sinks"], err=err)
    torch.cuda.synchronize()
    # the tickets are zero again
    assert not ws[-8 * 152:].any()
    return out


def good(s, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, err, **kw)
    assert int(err.item()) == 0
    pr.check(out, *pr.attend_all(s))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,before", [([1], [0]), ([1], [127]), ([1], [128]), ([64], [0]), ([65], [63]), ([128], [0]),
                                        ([129], [128]), ([127], [1]), ([333], [0]), ([17], [700]), ([256], [255])])
def test_one_stream(dtype, new, before):
    good(pr.make(new, before, 4, 2, dtype, seed=new[0] + before[0]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ragged_streams(dtype):
    good(pr.make([1, 0, 200, 33, 64, 5, 129], [0, 40, 0, 333, 64, 1000, 127], 4, 2, dtype, seed=2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (3, 1), (16, 2), (20, 4), (12, 4), (128, 1), (100, 1)])
def test_head_groups(dtype, Hq, Hkv):
    good(pr.make([150, 7, 40], [0, 100, 3], Hq, Hkv, dtype, seed=Hq))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 130), (100, 0), (128, 128), (200, 4), (300, 37),
                                          (129, 300), (5000, 4), (2 ** 31 - 1, 7)])
def test_windows(dtype, window, sinks):
    good(pr.make([1, 130, 300, 64], [600, 500, 0, 1000], 4, 2, dtype, window, sinks, seed=window % 1000 + sinks))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,before,window,sinks", [([61], [20000], 0, 0), ([5], [9000], 0, 0), ([130, 1], [3000, 9000], 0, 0),
                                                     ([1500], [0], 0, 0), ([700, 900, 40], [100, 0, 5000], 2000, 20)])
def test_segments_split_over_ctas(dtype, new, before, window, sinks):
    """Twice on one workspace, and alike bit for bit: parts are joined in the order of the CTAs."""
    s = pr.make(new, before, 4, 2, dtype, window, sinks, seed=new[0])
    ws = workspace(s)
    first = run(s, ws=ws)
    pr.check(first, *pr.attend_all(s))
    for _ in range(3):
        assert torch.equal(run(s, ws=ws), first)


@pytest.mark.parametrize("gain", [0.0, 30.0])
def test_flat_and_peaked_weights(gain):
    """All weights alike, and one token that takes nearly all (scores of +-300: their fp32 rounding is 2^-15 there)."""
    s = pr.make([200], [100], 4, 2, "bf16", seed=4, q_gain=gain)
    ref, tol = pr.attend_all(s)
    _, val = ref, tol
    v = torch.stack([pr.cached(s, 0, g)[1].abs().amax(0) for g in range(2)]).repeat_interleave(2, 0)
    # (an error e of a score moves out by at most e times the spread of the values)
    pr.check(run(s), ref, tol + gain * 2.0 ** -18 * 300 * v[None])


def test_scores_far_below_zero():
    """Keys that all point away from the queries: the maximum is what counts."""
    s = pr.make([70], [200], 4, 2, "bf16", seed=5)
    s["q"] = torch.full_like(s["q"], 8.0)
    k = s["k_pool"]
    k[torch.isfinite(k)] = -8.0
    pr.finish(s)
    pr.check(run(s), *pr.attend_all(s))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(value):
    """One in a token that late rows do not see any more, one that early rows do
    not see yet, one in a sink, and some that no row sees."""
    s = pr.make([90], [300], 4, 2, "bf16", 100, 4, seed=6, hide=False)
    vis = pr.visible(s, 0)
    for t, d in ((250, 5), (340, 127), (389, 66), (3, 64), (100, 9), (5, 11)):
        b = int(s["table"][0, t // 16])
        s["v_pool"][b, 1, t % 16, d] = value
        if not vis[:, t].any():
            s["k_pool"][b, 1, t % 16, d] = value
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    assert torch.isfinite(ref[:, :2]).all() and torch.isfinite(ref[:, 2:, 9]).all()
    for d in (5, 127, 66):
        bad = ~torch.isfinite(ref[:, 2, d])
        assert bad.any() and not bad.all()
    pr.check(run(s), ref, tol)


def test_fp8_values_that_are_not_numbers_reach_the_rows_that_see_them():
    s = pr.make([90], [300], 4, 2, "fp8", 100, 4, seed=6, hide=False)
    vis = pr.visible(s, 0)
    for t, d in ((250, 5), (340, 127), (389, 66), (3, 64), (100, 9), (5, 11)):
        b, slot = int(s["table"][0, t // 16]), t % 16
        s["pools"][0][b, 1, 2048 + 16 * d + 4 * (slot % 8 // 2) + slot % 2 + 2 * (slot // 8)] = 0xFF
        s["v_val"][b, 1, slot, d] = float("nan")
    assert not vis[:, 100].any() and not vis[:, 5].any()
    ref, tol = pr.attend_all(s)
    assert torch.isfinite(ref[:, :2]).all() and torch.isfinite(ref[:, 2:, 9]).all()
    for d in (5, 127, 66):
        bad = ~torch.isfinite(ref[:, 2, d])
        assert bad.any() and not bad.all()
    pr.check(run(s), ref, tol)


def test_fp8_scales_of_any_size():
    """Values from 2^-20 to 50,000: scales times 2^8 from 2^-21 to 28,571.  A weight times that is a
    subnormal of f16 below 2^-14, off by 2^-25: 2^-33 of a code of at most 448, a token."""
    s = pr.make([70, 40], [0, 200], 4, 2, "fp8", seed=21)
    g = torch.Generator().manual_seed(22)
    k, v = s["k_pool"], s["v_pool"]
    size = torch.exp(torch.rand(v.shape[:3], generator=g) * (math.log(5e4) - math.log(2.0 ** -20)) + math.log(2.0 ** -20))
    top = v.float().abs().amax(-1)
    s["v_pool"] = (v.float() / top[..., None] * size[..., None]).to(torch.bfloat16)
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    pr.check(run(s), ref, tol + 270 * 2.0 ** -33 * 448)


def test_values_that_are_not_finite_in_split_segments():
    s = pr.make([60], [6000], 2, 1, "bf16", seed=7)
    for t, d in ((6030, 5), (6059, 100), (3000, 7)):
        s["v_pool"][int(s["table"][0, t // 16]), 0, t % 16, d] = float("inf")
    pr.finish(s)
    pr.check(run(s), *pr.attend_all(s))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_keys_that_are_not_finite_act_through_their_scores(value):
    s = pr.make([90], [100], 4, 2, "bf16", seed=8)
    s["q"] = s["q"].abs() + 0.1
    s["k_pool"][int(s["table"][0, 150 // 16]), 0, 150 % 16] = value
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    if value == float("-inf"):
        assert torch.isfinite(ref).all()
    else:  # (a weight of infinity over infinity)
        ref[50:, :2] = float("nan")
    pr.check(run(s), ref, tol)


def test_refused_streams_and_bad_blocks():
    s = pr.make([20, 30, 40, 50, 60], [20, 30, 98, 155, 200], 4, 2, "bf16", seed=9, max_blocks=17)
    s["ctx_lens"][1] = 29              # fewer than its rows
    s["ctx_lens"][2] = 17 * 16 + 1     # past the table
    s["table"][3, 2] = 10 ** 6
    s["table"][4, :] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, err)
    assert int(err.item()) == _lib.ERRBIT_CTX_LEN | _lib.ERRBIT_BLOCK_ID
    pr.check(out, *pr.attend_all(s, skip=(1, 2)))
    assert not out[140:].any()


def test_row_starts_out_of_range():
    s = pr.make([20, 30, 40], [20, 30, 40], 4, 2, "bf16", seed=10)
    s["row_start"] = torch.tensor([0, 20, 10, 400], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, err)
    assert int(err.item()) == _lib.ERRBIT_CTX_LEN
    ref, tol = pr.attend(s, 0)
    # stream 2's rows lie past the end: those that exist are zero (rows 10 to 19
    # are stream 0's as well: either's)
    pr.check(out[:10], ref[:10], tol[:10])
    assert not out[20:].any()


def test_rows_of_no_stream_are_left_alone():
    s = pr.make([20, 30], [20, 300], 4, 2, "bf16", seed=11)
    q = torch.cat((s["q"], s["q"][:9])).cuda()
    s["row_start"] = s["row_start"] + 0
    out = run(s, q=q)
    pr.check(out[:50], *pr.attend_all(s))
    assert bool((out[50:] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seed", range(6))
def test_segments_of_all_kinds_in_every_cta(dtype, seed):
    """Several segments a CTA: whole and split, rows for both halves and for one that both work on in turns,
    after one another in every order."""
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(1, 700, (10,), generator=g).tolist()
    before = torch.randint(0, 1500, (10,), generator=g).tolist()
    s = pr.make(new, before, 8, 4, dtype, 1000 if seed % 2 else 0, 4, seed=seed)
    first = run(s)
    pr.check(first, *pr.attend_all(s))
    assert torch.equal(run(s), first)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_streams_bits_do_not_depend_on_its_neighbours(dtype):
    """The rows next to a stream's last in a tile are the next stream's, and with three heads a
    group two are no query at all: neither may move what the stream's own rows are rounded by."""
    s = pr.make([85, 70, 130], [700, 500, 0], 6, 2, dtype, seed=31)
    first = run(s)
    loud = s["q"].clone()
    loud[85:] *= 64.0
    mixed = run(s, q=loud.cuda())
    assert torch.equal(first[:85], mixed[:85])
    run(s, q=(s["q"] * 64.0).cuda())
    assert torch.equal(first, run(s))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [0.25, float("nan")])
def test_blocks_past_32_bit_offsets(dtype, value):
    """The last of 65,600 blocks (33 KB or 32 KB of 8 heads) lie past 2^31 bytes."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    s = pr.make([70, 3], [200, 90], 16, 8, dtype, 60, 4, seed=41)
    if dtype == "bf16":
        s["pools"][1][:, 3, 5, 17] = value  # (values that are not finite are looked up by address)
    want = run(s)
    q = s["q"][:4].cuda().view(2, 2, 16, 128)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(2, 2, 16, 8, 128, 400), dtype=torch.uint8, device="cuda")
    outs = []
    for far in (False, True):
        if far:
            small = s["pools"][0].shape[0]
            big = []
            for p in s["pools"]:
                big.append(p if p is None else torch.zeros(65600, *p.shape[1:], dtype=p.dtype, device="cuda"))
                if p is not None:
                    big[-1][65600 - small:] = p.cuda()
            s["pools"] = tuple(big)
            s["table"] = torch.where(s["table"] >= 0, s["table"] + 65600 - small, s["table"])
        cache, table, lens, _ = upload(s)
        out = torch.empty_like(q)
        bd.tts_window_decode_attn(cache, table, lens, 400, q, out, ws, s["scale"], 60, 4, causal=True)
        torch.cuda.synchronize()
        outs.append(out)
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert same(run(s), want) and same(*outs)


def test_many_streams():
    new = [(7 * i) % 5 for i in range(700)]
    good(pr.make(new, [(13 * i) % 90 for i in range(700)], 2, 1, "bf16", seed=12))


def test_captured_and_replayed_with_new_lengths():
    s = pr.make([40, 70], [300, 10], 4, 2, "bf16", seed=13, max_blocks=30)
    cache, table, lens, start = upload(s)
    q = s["q"].cuda()
    out = torch.empty_like(q)
    ws = workspace(s)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"])
    for new, ctx in (([40, 70], [340, 80]), ([100, 10], [120, 77]), ([1, 109], [333, 80])):
        if new[1] > ctx[1]:
            ctx[1] = new[1]
            table[1] = table[0]
            s["table"][1] = s["table"][0]
        s.update(new=new, ctx=ctx, before=[c - n for c, n in zip(ctx, new)],
                 row_start=torch.tensor([0, new[0], 110], dtype=torch.int32))
        lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        start.copy_(s["row_start"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        pr.check(out, *pr.attend_all(s))


def test_programmatic_launches():
    """A chain of append and attention whose kernels start early."""
    s = pr.make([100, 33], [64, 300], 4, 2, "bf16", seed=14)
    cache, table, lens, start = upload(s)
    q = s["q"].cuda()
    ref = run(s)
    k = torch.stack([cache.k_pool[table[b].long()[t // 16], :, t % 16] for b in range(2)
                     for t in range(s["before"][b], s["ctx"][b])])
    v = torch.stack([cache.v_pool[table[b].long()[t // 16], :, t % 16] for b in range(2)
                     for t in range(s["before"][b], s["ctx"][b])])
    pos = s["ctx_before"].cuda()
    ws = workspace(s)
    outs = [torch.empty_like(q) for _ in range(20)]
    flags = bd.tts_set_launch_flags(_lib.LAUNCH_PROGRAMMATIC)
    try:
        for out in outs:
            bd.tts_kv_append_packed(cache, table, pos, start, k, v)
            bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"])
    finally:
        bd.tts_set_launch_flags(flags)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, ref)


def test_a_wait_that_runs_out_is_reported():
    s = pr.make([300], [100], 4, 2, "bf16", seed=15)
    ws = workspace(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, table, lens, start = upload(s)
    q = s["q"].cuda()
    out = torch.empty_like(q)
    assert _lib.lib().tts_test_set_stall(_lib.TEST_STALL_PROMPT, 2_000_000) == 0
    try:
        bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"], err=err)
        torch.cuda.synchronize()
    finally:
        _lib.lib().tts_test_set_stall(_lib.TEST_STALL_NONE, 2_000_000_000)
    assert int(err.item()) == _lib.ERRBIT_TIMEOUT
    good(s)


def test_two_streams_with_workspaces_of_their_own():
    cases = [pr.make([150, 20], [0, 3000], 4, 2, "bf16", seed=16), pr.make([90], [4000], 4, 2, "bf16", 1000, 4, seed=17)]
    refs = [run(s) for s in cases]
    up = [upload(s) + (s["q"].cuda(), workspace(s), torch.cuda.Stream()) for s in cases]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (s, (cache, table, lens, start, q, ws, stream)) in enumerate(zip(cases, up)):
            out = torch.empty_like(q)
            outs[i].append(out)
            stream.wait_stream(torch.cuda.current_stream())
            bd.tts_prompt_attn(cache, table, lens, start, q, out, ws, s["scale"], s["window"], s["sinks"], stream=stream)
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        for out in got:
            assert torch.equal(out, ref)


def test_refusals():
    s = pr.make([20], [20], 4, 2, "bf16")
    cache, table, lens, start = upload(s)
    q, ws = s["q"].cuda(), workspace(s)
    for kw, code in ((dict(window=-1), -1), (dict(sinks=-1), -1)):
        with pytest.raises(bd.TTSError) as e:
            bd.tts_prompt_attn(cache, table, lens, start, q, torch.empty_like(q), ws, 0.1, **kw)
        assert e.value.code == code
    with pytest.raises(bd.TTSError) as e:
        bd.tts_prompt_attn(cache, table, lens, start, q, torch.empty_like(q), ws[:-256], 0.1)
    assert e.value.code == -3
    for bad in (dict(q=q.float()), dict(start=start[:1].contiguous()), dict(lens=lens.cpu()), dict(q=q[:, :3])):
        with pytest.raises((ValueError, bd.TTSError)):
            bd.tts_prompt_attn(cache, table, bad.get("lens", lens), bad.get("start", start), bad.get("q", q),
                               torch.empty_like(q), ws, 0.1)
