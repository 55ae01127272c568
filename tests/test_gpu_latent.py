"""The latent cache on the GPU: append, absorbed decode attention and expanded
prompt attention against a 64-bit reference, at the sizes and masks where they
can go wrong.  Tolerances are those derived in latent_ref."""
from __future__ import annotations

import math
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]
NAN = float("nan")
CTX_LEN, BLOCK_ID = 2, 1        # error bits


@pytest.fixture(scope="module")
def bd():
    from decode_step_gb300 import binding
    return binding


def up(s):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in s.items()}


def poisoned(n):
    """A workspace whose every float and bf16 word is NaN."""
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values are not finite"
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst error over tolerance "
                           f"{((got - want).abs() / tol.clamp(min=1e-30)).max():.2f}, max error {(got - want).abs().max():.2e}")


# ------------------------------------------------------------------- append

BASE = 10000.0


def run_append(bd, s, d, ragged, inplace=False, err=None, row_start=None):
    cache = bd.LatentCache(d["pool"], s["L"])
    q_out = d["q_rope"] if inplace else torch.full_like(d["q_rope"], NAN)
    bd.tts_latent_append(cache, d["table"], d["ctx_before"], d["c_new"], d["kr_new"], d["q_rope"], q_out, BASE,
                         row_start=(d["row_start"] if row_start is None else row_start) if ragged else None, err=err)
    return q_out


def check_rotated(got, x, pos):
    """Within half a step of the exact rotation plus fp32 arithmetic: cos and
    sin to 2^-22, three fp32 roundings (2^-24) of terms up to |x1| + |x2|."""
    want = ref.rotate(x, pos, BASE)
    mag = x.double().abs()
    mag = mag[..., :32] + mag[..., 32:]
    tol = ref.U * want.abs() + 2.0 ** -20 * torch.cat((mag, mag), -1) + 1e-38
    check(got, want, tol, "rotation")


APPENDS = [
    # new tokens, cached before, Hq, latent
    ([1], [0], 16, 512),
    ([1, 1, 1, 1], [0, 15, 16, 4095], 16, 512),
    ([5, 5, 5], [14, 11, 250], 4, 128),
    ([1, 1], [31, 7], 1, 64),
    ([3] * 40, list(range(40)), 33, 320),
]


@pytest.mark.parametrize("new,before,Hq,L", APPENDS)
@pytest.mark.parametrize("inplace", [False, True])
def test_append_uniform(bd, new, before, Hq, L, inplace):
    s = ref.make(new, before, Hq, L, 64, 64, seed=1, garbage=7.0)
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run_append(bd, s, d, False, inplace, err)
    _check_append(s, d, q_out)
    assert int(err) == 0


def _check_append(s, d, q_out, skip_rows=()):
    pool = d["pool"].cpu()
    want = s["pool"].clone()
    rows, pos, r = [], [], 0
    for b, n in enumerate(s["new"]):
        for j in range(n):
            p = s["before"][b] + j
            if r not in skip_rows:
                blk = int(s["table"][b, p // 16])
                rows.append((r, blk, p % 16))
                pos.append(p)
            r += 1
    pos = torch.tensor(pos)
    idx = torch.tensor([x[0] for x in rows])
    blk, slot = torch.tensor([x[1] for x in rows]), torch.tensor([x[2] for x in rows])
    got = pool[blk, slot]
    assert torch.equal(got[:, :s["L"]], s["c_new"][idx])
    check_rotated(got[:, s["L"]:], s["kr_new"][idx], pos)
    check_rotated(q_out.cpu()[idx], s["q_rope"][idx], pos[:, None])
    want[blk, slot] = got
    assert torch.equal(pool, want), "slots of other tokens changed"


@pytest.mark.parametrize("new", [[7], [0, 3, 0, 130, 1, 0], [1] * 70, [0, 0, 2] + [0] * 40 + [5]])
def test_append_ragged(bd, new):
    before = [(7 * i) % 50 for i in range(len(new))]
    s = ref.make(new, before, 8, 256, 64, 64, seed=2, garbage=3.0)
    d = up(s)
    _check_append(s, d, run_append(bd, s, d, True))


def test_append_ragged_leaves_rows_of_no_stream(bd):
    """Rows before the first and behind the last stream are not read into the
    pool, and their query rows are left alone."""
    s = ref.make([4, 6], [10, 20], 8, 128, 64, 64, seed=3, garbage=0.0)
    d = up(s)
    shifted = torch.tensor([2, 2 + 3, 2 + 3 + 2], dtype=torch.int32).cuda()     # rows 2..4 and 5..6 of 10
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run_append(bd, s, d, True, err=err, row_start=shifted)
    assert int(err) == 0
    q = q_out.cpu()
    keep = torch.tensor([0, 1, 7, 8, 9])
    assert torch.isnan(q[keep].float()).all()
    pos = torch.tensor([10, 11, 12, 20, 21])
    check_rotated(q[2:7], s["q_rope"][2:7], pos[:, None])
    pool = d["pool"].cpu()
    want = s["pool"].clone()
    for r, (b, p) in zip(range(2, 7), [(0, 10), (0, 11), (0, 12), (1, 20), (1, 21)]):
        blk = int(s["table"][b, p // 16])
        assert torch.equal(pool[blk, p % 16, :128], s["c_new"][r])
        want[blk, p % 16] = pool[blk, p % 16]
    assert torch.equal(pool, want)


def test_append_skips_bad_slots(bd):
    """A position outside the table, a negative one and a bad block id skip
    their rows and set their bits; the others are written."""
    s = ref.make([2, 2, 2, 2], [30, 5, 0, 8], 4, 128, 64, 64, seed=4, garbage=1.0)
    s["ctx_before"][1] = -1
    s["table"][2, 0] = s["pool"].shape[0]
    s["ctx_before"][0] = 16 * s["table"].shape[1] - 1     # its second token is past the table
    s["before"][0] = 16 * s["table"].shape[1] - 1
    s["table"][0, -1] = s["table"][0, 0]
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run_append(bd, s, d, False, err=err)
    assert int(err) == CTX_LEN | BLOCK_ID
    skipped = (1, 2, 3, 4, 5)
    assert torch.isnan(q_out.cpu()[list(skipped)].float()).all()
    s["new"], s["before"] = s["new"], [s["before"][0], 5, 0, 8]
    _check_append(s, d, q_out, skip_rows=skipped)


def test_append_bad_row_start_writes_nothing_else(bd):
    """A decreasing row_start: rows it gives to no stream are skipped."""
    s = ref.make([4, 4, 4], [0, 0, 0], 4, 128, 64, 64, seed=5, garbage=1.0)
    d = up(s)
    start = torch.tensor([0, 4, -100, 1 << 30], dtype=torch.int32).cuda()
    q_out = run_append(bd, s, d, True, row_start=start).cpu()
    check_rotated(q_out[:4], s["q_rope"][:4], torch.arange(4)[:, None])


def test_append_without_queries(bd):
    s = ref.make([2, 2], [3, 4], 4, 128, 64, 64, seed=6, garbage=1.0)
    d = up(s)
    bd.tts_latent_append(bd.LatentCache(d["pool"], 128), d["table"], d["ctx_before"], d["c_new"], d["kr_new"], rope_base=BASE)
    blk = int(s["table"][1, 0])
    assert torch.equal(d["pool"].cpu()[blk, 5, :128], s["c_new"][3])


# ------------------------------------------------------------------- decode

def run_decode(bd, s, d, q_len, causal, err=None, max_ctx=None, ws=None, out=None):
    B, Hq = len(s["new"]), s["Hq"]
    max_ctx = max(1, max(s["ctx"])) if max_ctx is None else max_ctx
    if ws is None:
        ws = poisoned(bd.tts_latent_decode_attn_workspace_size(B, q_len, Hq, s["L"], s["nope"], s["v"], max_ctx))
    if out is None:
        out = torch.full((B, q_len, Hq, s["v"]), NAN, dtype=torch.bfloat16, device="cuda")
    bd.tts_latent_decode_attn(bd.LatentCache(d["pool"], s["L"]), d["table"], d["ctx_lens"], max_ctx,
                              d["q_nope"].view(B, q_len, Hq, -1), d["q_rope"].view(B, q_len, Hq, -1), d["w_uk"],
                              d["w_uv"], out, ws, s["scale"], causal=causal, err=err)
    return out


def decode_case(bd, ctx, q_len, Hq, L, nope, v, causal, seed=11, **kw):
    s = ref.make([q_len] * len(ctx), [c - q_len for c in ctx], Hq, L, nope, v, seed, **kw)
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_decode(bd, s, d, q_len, causal, err)
    want, tol = ref.attend_all(s, causal, True)
    check(out.view(s["T"], Hq, v), want, tol, f"decode {ctx} {q_len} {Hq} {L}")
    assert int(err) == 0


@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
def test_decode_lengths(bd, ctx):
    decode_case(bd, [ctx], 1, 16, 512, 128, 128, False)


@pytest.mark.parametrize("Hq", [1, 2, 3, 7, 8, 15, 17, 24, 32, 48, 63, 64, 65, 80, 128])
def test_decode_heads(bd, Hq):
    decode_case(bd, [70, 3], 1, Hq, 128, 64, 64, False)


@pytest.mark.parametrize("L", [64, 128, 192, 256, 320, 384, 448, 512])
@pytest.mark.parametrize("nope,v", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_decode_widths(bd, L, nope, v):
    decode_case(bd, [130, 77, 16], 1, 4, L, nope, v, False)


@pytest.mark.parametrize("q_len", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq", [4, 16])
def test_decode_query_rows(bd, q_len, causal, Hq):
    decode_case(bd, [q_len, q_len + 1, 64, 65, 67, 200], q_len, Hq, 256, 128, 128, causal)


@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("q_len,ctx,Hq", [(5, 71, 16), (5, 66, 4), (3, 64, 16), (70, 200, 2)])
def test_decode_later_tokens_not_finite(bd, what, q_len, ctx, Hq):
    """A row's own token (and what follows) does not reach the rows before it."""
    s = ref.make([q_len] * 2, [ctx - q_len] * 2, Hq, 192, 128, 64, 12)
    want, tol = ref.attend_all(s, True, True)
    first = q_len // 2                        # the row whose token is spoilt
    t = ctx - q_len + first
    s["pool"][s["table"][0, t // 16].long(), t % 16, 5:40] = what
    s["pool"][s["table"][0, t // 16].long(), t % 16, 192 + 7] = what
    out = run_decode(bd, s, up(s), q_len, True).view(2, q_len, Hq, 64)
    want, tol = want.view(out.shape), tol.view(out.shape)
    check(out[1], want[1], tol[1], "the other stream")
    check(out[0, :first], want[0, :first], tol[0, :first], "rows before")
    if what != what:
        assert torch.isnan(out[0, first:].float()).all()


def test_decode_many_rows(bd):
    decode_case(bd, [300, 128], 8, 128, 128, 64, 64, True)       # 1024 query rows a stream


@pytest.mark.parametrize("B,q_len,Hq,L,nope,v", [(42, 2, 152, 512, 64, 128), (85, 8, 20, 192, 128, 64), (30, 2, 152, 64, 64, 64)])
def test_decode_many_rows_per_head(bd, B, q_len, Hq, L, nope, v):
    """So many rows a head that the output product takes them in rounds."""
    decode_case(bd, [q_len + (5 * i) % 23 for i in range(B)], q_len, Hq, L, nope, v, True)


def test_decode_ragged_batch(bd):
    ctx = [1 + (37 * i * i) % 700 for i in range(70)]
    decode_case(bd, ctx, 1, 8, 256, 64, 64, False)


def test_decode_many_streams(bd):
    decode_case(bd, [1 + (13 * i) % 40 for i in range(400)], 1, 2, 64, 64, 64, False)


def test_decode_long_context(bd):
    decode_case(bd, [20011, 3, 9000], 1, 4, 128, 64, 64, False)


def test_decode_split_verify(bd):
    decode_case(bd, [5003, 1200], 5, 16, 512, 128, 128, True)


@pytest.mark.parametrize("gain", [8.0, 40.0])
def test_decode_sharp_scores(bd, gain):
    """Scores of size tens: the running maximum moves often and by much."""
    s = ref.make([1, 1], [900, 300], 16, 256, 64, 64, 17, q_gain=gain)
    s["scale"] /= 4 if gain > 10 else 1
    d = up(s)
    out = run_decode(bd, s, d, 1, False)
    want, tol = ref.attend_all(s, False, True)
    check(out.view(s["T"], 16, 64), want, tol + 2.0 ** -14 * gain, "sharp")


@pytest.mark.parametrize("rising", [True, False])
def test_decode_monotone_scores(bd, rising):
    """Every token's score above (or below) all earlier ones, over a range of
    some hundreds: each tile raises the maximum (or adds nothing)."""
    n = 700
    s = ref.make([1], [n - 1], 16, 128, 64, 64, 18)
    ramp = torch.linspace(0, 1, n) if rising else torch.linspace(1, 0, n)
    rows = torch.zeros(-(-n // 16) * 16, 192, dtype=torch.bfloat16)
    rows[:n, :128] = torch.randn(n, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    rows[:n, 128] = (ramp * 64).to(torch.bfloat16)
    s["pool"][s["table"][0].long()] = rows.view(-1, 16, 192)
    s["q_rope"].zero_()
    s["q_rope"][..., 0] = 64.0
    s["q_nope"] *= 0.125
    d = up(s)
    out = run_decode(bd, s, d, 1, False)
    want, tol = ref.attend_all(s, False, True)
    # scores reach 64 * 64 * scale = 362: fp32 keeps them to 362 * 2^-23 each way
    check(out.view(1, 16, 64), want, tol + 2.0 ** -13 * want.abs().amax(), "monotone")


def test_decode_bad_lengths_give_zeros(bd):
    s = ref.make([2] * 6, [30, 40, 0, 60, 20, 9], 4, 128, 64, 64, 19)
    d = up(s)
    max_ctx = 50
    lens = s["ctx_lens"].clone()
    lens[0], lens[2], lens[4] = 0, 1, -7          # empty, fewer than its rows, negative; stream 3 has 62 > 50
    d["ctx_lens"] = lens.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_decode(bd, s, d, 2, True, err, max_ctx=max_ctx).view(s["T"], 4, 64)
    assert int(err) == CTX_LEN
    want, tol = ref.attend_all(s, True, True, skip=(0, 2, 3, 4))
    check(out, want, tol, "bad lengths")
    for b in (0, 2, 3, 4):
        assert (out[2 * b:2 * b + 2] == 0).all()


def test_decode_length_past_the_table(bd):
    s = ref.make([1, 1], [30, 20], 4, 128, 64, 64, 20)
    d = up(s)
    lens = s["ctx_lens"].clone()
    lens[0] = 16 * s["table"].shape[1] + 1
    d["ctx_lens"] = lens.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_decode(bd, s, d, 1, False, err, max_ctx=1000).view(2, 4, 64)
    want, tol = ref.attend_all(s, False, True, skip=(0,))
    check(out, want, tol, "past the table")
    assert int(err) == CTX_LEN


def test_decode_bad_blocks_are_left_out(bd):
    s = ref.make([1, 1, 1], [200, 40, 100], 16, 256, 64, 128, 21)
    nb = s["pool"].shape[0]
    s["table"][0, 0], s["table"][0, 3], s["table"][0, 12] = -1, nb, 1 << 30
    s["table"][1, :] = -5                           # every token left out: zeros
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_decode(bd, s, d, 1, False, err).view(3, 16, 128)
    want, tol = ref.attend_all(s, False, True)
    check(out, want, tol, "bad blocks")
    assert (out[1] == 0).all()
    assert int(err) == BLOCK_ID


def test_decode_row_masked_by_bad_blocks(bd):
    """Causal rows of which the first see only tokens in an invalid block."""
    s = ref.make([4], [14], 8, 128, 64, 64, 22)      # rows at 14..17, block 0 invalid
    s["table"][0, 0] = -1
    d = up(s)
    out = run_decode(bd, s, d, 4, True).view(4, 8, 64)
    want, tol = ref.attend_all(s, True, True)
    check(out, want, tol, "masked rows")
    assert (out[:2] == 0).all() and (out[2:] != 0).any()


def test_decode_writes_only_its_outputs(bd):
    s = ref.make([1] * 3, [20, 90, 5], 5, 128, 64, 64, 23)
    d = up(s)
    big = torch.full((3 * 5 * 64 + 512,), 5.0, dtype=torch.bfloat16, device="cuda")
    n = bd.tts_latent_decode_attn_workspace_size(3, 1, 5, 128, 64, 64, 91)
    ws = poisoned(n + 4096)
    pool = d["pool"].clone()
    run_decode(bd, s, d, 1, False, ws=ws[:n], out=big[256:256 + 960].view(3, 1, 5, 64))
    assert (big[:256] == 5).all() and (big[256 + 960:] == 5).all()
    assert (ws[n:] == 0xFF).all()
    assert torch.equal(pool.view(torch.int16), d["pool"].view(torch.int16))
    want, tol = ref.attend_all(s, False, True)
    check(big[256:256 + 960].view(3, 5, 64), want, tol)


def test_decode_repeats_exactly_and_reuses_a_workspace(bd):
    """The same call gives the same bits, whatever an earlier call left in the
    workspace."""
    s = ref.make([1] * 9, [10, 700, 3, 64, 128, 999, 31, 0, 55], 16, 512, 128, 128, 24)
    t = ref.make([5] * 4, [100, 2000, 50, 7], 16, 512, 128, 128, 25)
    d, e = up(s), up(t)
    n = max(bd.tts_latent_decode_attn_workspace_size(9, 1, 16, 512, 128, 128, 1000),
            bd.tts_latent_decode_attn_workspace_size(4, 5, 16, 512, 128, 128, 2005))
    ws = poisoned(n)
    first = run_decode(bd, s, d, 1, False, ws=ws).clone()
    other = run_decode(bd, t, e, 5, True, ws=ws)
    again = run_decode(bd, s, d, 1, False, ws=ws)
    assert torch.equal(first, again)
    want, tol = ref.attend_all(t, True, True)
    check(other.view(t["T"], 16, 128), want, tol)


# ------------------------------------------------------------------ prefill

def run_prefill(bd, s, d, err=None, total=None, row_start=None, out=None, ws=None, T=None):
    B, Hq = len(s["new"]), s["Hq"]
    total = sum(c for c, n in zip(s["ctx"], s["new"]) if n) if total is None else total
    T = d["q_nope"].shape[0]
    if ws is None:
        ws = poisoned(bd.tts_latent_prefill_attn_workspace_size(B, T, Hq, s["L"], s["nope"], s["v"], total))
    if out is None:
        out = torch.full((T, Hq, s["v"]), NAN, dtype=torch.bfloat16, device="cuda")
    bd.tts_latent_prefill_attn(bd.LatentCache(d["pool"], s["L"]), d["table"], d["ctx_lens"], total,
                               d["row_start"] if row_start is None else row_start, d["q_nope"], d["q_rope"], d["w_uk"],
                               d["w_uv"], out, ws, s["scale"], err=err)
    return out


def prefill_case(bd, new, before, Hq, L, nope, v, seed=31, **kw):
    s = ref.make(new, before, Hq, L, nope, v, seed, **kw)
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(bd, s, d, err)
    want, tol = ref.attend_all(s, True, False)
    check(out, want, tol, f"prefill {new} {before}")
    assert int(err) == 0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
def test_prefill_lengths(bd, n):
    prefill_case(bd, [n], [0], 2, 512, 128, 128)


@pytest.mark.parametrize("before", [1, 15, 64, 127, 128, 129, 500])
def test_prefill_after_a_prefix(bd, before):
    prefill_case(bd, [130, 3], [before, before], 2, 128, 64, 64)


@pytest.mark.parametrize("Hq", [1, 3, 16, 33])
def test_prefill_heads(bd, Hq):
    prefill_case(bd, [70, 129], [5, 0], Hq, 128, 64, 64)


@pytest.mark.parametrize("L", [64, 128, 192, 256, 320, 384, 448, 512])
@pytest.mark.parametrize("nope,v", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_prefill_widths(bd, L, nope, v):
    prefill_case(bd, [140], [20], 2, L, nope, v)


@pytest.mark.parametrize("new", [[0, 5, 0, 300, 1, 0], [1] * 40, [17] * 20, [0, 0, 200], [129, 0, 0]])
def test_prefill_ragged(bd, new):
    prefill_case(bd, new, [(11 * i) % 40 for i in range(len(new))], 3, 128, 64, 128)


def test_prefill_longer(bd):
    prefill_case(bd, [1500, 700], [77, 0], 2, 256, 128, 128)


@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("n,before,spoilt", [(140, 20, 100), (300, 3, 200), (7, 0, 1), (20, 125, 4)])
def test_prefill_later_tokens_not_finite(bd, what, n, before, spoilt):
    s = ref.make([n, 9], [before, 2], 2, 128, 64, 128, 33)
    want, tol = ref.attend_all(s, True, False)
    t = before + spoilt
    s["pool"][s["table"][0, t // 16].long(), t % 16, 5:40] = what
    s["pool"][s["table"][0, t // 16].long(), t % 16, 128 + 7] = what
    out = run_prefill(bd, s, up(s))
    check(out[n:], want[n:], tol[n:], "the other stream")
    check(out[:spoilt], want[:spoilt], tol[:spoilt], "rows before")
    if what != what:
        assert torch.isnan(out[spoilt:n].float()).all()


@pytest.mark.parametrize("gain", [8.0])
def test_prefill_sharp_scores(bd, gain):
    s = ref.make([600], [100], 4, 128, 64, 64, 32, q_gain=gain)
    d = up(s)
    out = run_prefill(bd, s, d)
    want, tol = ref.attend_all(s, True, False)
    check(out, want, tol + 2.0 ** -14 * gain, "sharp")


def test_prefill_leaves_rows_of_no_stream(bd):
    s = ref.make([40, 30], [0, 9], 4, 128, 64, 64, 33)
    pad = 50
    for k in ("q_nope", "q_rope"):
        x = s[k]
        s[k] = torch.cat((torch.full((pad, *x.shape[1:]), NAN, dtype=x.dtype), x,
                          torch.full((pad, *x.shape[1:]), NAN, dtype=x.dtype)))
    d = up(s)
    out = torch.full((70 + 2 * pad, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(bd, s, d, err, row_start=(s["row_start"] + pad).cuda(), out=out)
    assert (out[:pad] == 9).all() and (out[70 + pad:] == 9).all() and int(err) == 0
    s["q_nope"], s["q_rope"] = s["q_nope"][pad:-pad], s["q_rope"][pad:-pad]
    want, tol = ref.attend_all(s, True, False)
    check(out[pad:-pad], want, tol)


def test_prefill_bad_streams_give_zeros(bd):
    """Context shorter than the rows, negative, past the table; the others are
    unaffected."""
    s = ref.make([20, 30, 10, 5, 6], [0, 3, 40, 2, 1], 4, 128, 64, 64, 34)
    d = up(s)
    lens = s["ctx_lens"].clone()
    lens[0], lens[2], lens[3] = 19, -1, 16 * s["table"].shape[1] + 1
    d["ctx_lens"] = lens.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(bd, s, d, err, total=1000)
    assert int(err) == CTX_LEN
    want, tol = ref.attend_all(s, True, False, skip=(0, 2, 3))
    check(out, want, tol)
    at = s["row_start"]
    for b in (0, 2, 3):
        assert (out[int(at[b]):int(at[b + 1])] == 0).all()


def test_prefill_total_exceeded(bd):
    """Streams that take the sum of contexts past max_total_ctx get zeros."""
    s = ref.make([20, 30, 10], [0, 100, 4], 4, 128, 64, 64, 35)
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(bd, s, d, err, total=20 + 130 - 1)
    assert int(err) == CTX_LEN
    want, tol = ref.attend_all(s, True, False, skip=(1, 2))
    check(out, want, tol)


def test_prefill_bad_rows(bd):
    """row_start outside [0, num_rows]: that stream's rows inside get zeros."""
    s = ref.make([20, 30], [0, 0], 4, 128, 64, 64, 36)
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(bd, s, d, err, row_start=torch.tensor([0, 20, 51], dtype=torch.int32).cuda())
    assert int(err) == CTX_LEN
    want, tol = ref.attend_all(s, True, False, skip=(1,))
    check(out, want, tol)
    assert (out[20:] == 0).all()


def test_prefill_overlapping_rows_stay_in_the_workspace(bd):
    """Streams that claim the same rows have more query tiles than the
    workspace is sized for; those past its end are left out."""
    Hq, L, T, B = 2, 64, 700, 9
    s = ref.make([T], [0], Hq, L, 64, 64, 63)
    d = up(s)
    d["table"] = s["table"].expand(B, -1).contiguous().cuda()
    d["ctx_lens"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, T] * 5, dtype=torch.int32, device="cuda")      # streams 0, 2, 4, ...: all the rows
    n = bd.tts_latent_prefill_attn_workspace_size(B, T, Hq, L, 64, 64, 5 * T)
    ws = poisoned(n + 4096)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty((T, Hq, 64), dtype=torch.bfloat16, device="cuda")
    bd.tts_latent_prefill_attn(bd.LatentCache(d["pool"], L), d["table"], d["ctx_lens"], 5 * T, rows, d["q_nope"],
                               d["q_rope"], d["w_uk"], d["w_uv"], out, ws[:n], s["scale"], err=err)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xFF).all()
    assert int(err) == CTX_LEN


def test_prefill_bad_blocks(bd):
    s = ref.make([150, 20, 40], [30, 0, 0], 4, 128, 64, 64, 37)
    nb = s["pool"].shape[0]
    s["table"][0, 1], s["table"][0, 7] = -1, nb
    s["table"][1, :] = -1
    s["table"][2, 0] = nb + 5                        # its first 16 rows see nothing
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(bd, s, d, err)
    assert int(err) == BLOCK_ID
    want, tol = ref.attend_all(s, True, False)
    check(out, want, tol)
    at = s["row_start"]
    assert (out[int(at[1]):int(at[2])] == 0).all() and (out[int(at[2]):int(at[2]) + 16] == 0).all()


def test_prefill_repeats_exactly(bd):
    s = ref.make([300, 5, 129], [10, 0, 200], 4, 256, 128, 128, 38)
    d = up(s)
    n = bd.tts_latent_prefill_attn_workspace_size(3, s["T"], 4, 256, 128, 128, sum(s["ctx"]))
    ws = poisoned(n + 4096)
    first = run_prefill(bd, s, d, ws=ws[:n]).clone()
    again = run_prefill(bd, s, d, ws=ws[:n])
    assert torch.equal(first, again)
    assert (ws[n:] == 0xFF).all()


# ------------------------------------------------------- streams and graphs

def test_calls_on_another_stream_and_captured(bd):
    """Both attentions and the append on a side stream, then captured in one
    graph that is replayed with new inputs."""
    s = ref.make([1] * 5, [30, 200, 64, 1, 500], 16, 256, 128, 64, 41)
    t = ref.make([1] * 5, [30, 200, 64, 1, 500], 16, 256, 128, 64, 42)
    d = up(s)
    side = torch.cuda.Stream()
    n = bd.tts_latent_decode_attn_workspace_size(5, 1, 16, 256, 128, 64, 501)
    ws = poisoned(n)
    out = torch.full((5, 1, 16, 64), NAN, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run_decode(bd, s, d, 1, False, ws=ws, out=out)
    side.synchronize()
    want, tol = ref.attend_all(s, False, True)
    check(out.view(5, 16, 64), want, tol)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_decode(bd, s, d, 1, False, ws=ws, out=out)
    u = up(t)
    for k in ("pool", "table", "q_nope", "q_rope", "w_uk", "w_uv"):
        d[k].copy_(u[k])
    g.replay()
    torch.cuda.synchronize()
    want, tol = ref.attend_all(t, False, True)
    check(out.view(5, 16, 64), want, tol)


def test_prefill_captured(bd):
    s = ref.make([100, 40], [0, 30], 4, 128, 64, 64, 43)
    t = ref.make([100, 40], [0, 30], 4, 128, 64, 64, 44)
    d = up(s)
    ws = poisoned(bd.tts_latent_prefill_attn_workspace_size(2, 140, 4, 128, 64, 64, 170))
    out = torch.full((140, 4, 64), NAN, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    run_prefill(bd, s, d, ws=ws, out=out)
    with torch.cuda.graph(g):
        run_prefill(bd, s, d, ws=ws, out=out)
    u = up(t)
    for k in ("pool", "table", "q_nope", "q_rope", "w_uk", "w_uv"):
        d[k].copy_(u[k])
    g.replay()
    torch.cuda.synchronize()
    want, tol = ref.attend_all(t, True, False)
    check(out, want, tol)


def test_a_stream_from_prompt_to_tokens(bd):
    """The operators as a serving loop uses them: two prompts appended and
    attended in one ragged call, then three single-token steps and a causal
    five-token step on the same cache, against the reference that keeps its own
    copy of the cache."""
    Hq, L, nope, v = 8, 256, 64, 64
    s = ref.make([37, 150], [0, 0], Hq, L, nope, v, 51, garbage=NAN, max_blocks=12, spare=30)
    ids = torch.randperm(s["pool"].shape[0], generator=torch.Generator().manual_seed(3))[:24].to(torch.int32)
    s["table"] = ids.view(2, 12).contiguous()
    s["pool"].fill_(NAN)
    pool = s["pool"].clone().cuda()
    w_uk, w_uv = s["w_uk"].cuda(), s["w_uv"].cuda()
    cache = bd.LatentCache(pool, L)
    ws = poisoned(max(bd.tts_latent_prefill_attn_workspace_size(2, 187, Hq, L, nope, v, 187),
                      bd.tts_latent_decode_attn_workspace_size(2, 5, Hq, L, nope, v, 192)))
    table = s["table"].cuda()
    lens = [0, 0]
    for step, new in enumerate([[37, 150], [1, 1], [1, 1], [1, 1], [5, 5]]):
        t = ref.make(new, lens, Hq, L, nope, v, 60 + step)
        t["table"], t["w_uk"], t["w_uv"] = s["table"], s["w_uk"], s["w_uv"]
        d = up(t)
        q = torch.empty_like(d["q_rope"])
        bd.tts_latent_append(cache, table, d["ctx_before"], d["c_new"], d["kr_new"], d["q_rope"], q, BASE,
                             row_start=d["row_start"] if step == 0 else None)
        out = torch.full((sum(new), Hq, v), NAN, dtype=torch.bfloat16, device="cuda")
        if step == 0:
            bd.tts_latent_prefill_attn(cache, table, d["ctx_lens"], sum(t["ctx"]), d["row_start"], d["q_nope"], q, w_uk,
                                       w_uv, out, ws, t["scale"])
        else:
            n = new[0]
            bd.tts_latent_decode_attn(cache, table, d["ctx_lens"], 192, d["q_nope"].view(2, n, Hq, nope),
                                      q.view(2, n, Hq, 64), w_uk, w_uv, out.view(2, n, Hq, v), ws, t["scale"], causal=True)
        torch.cuda.synchronize()
        t["q_rope"], t["pool"] = q.cpu(), pool.cpu()     # rotation and rows as stored: checked by the append's tests
        rows = torch.cat([torch.arange(p, p + n) for n, p in zip(new, lens)])
        which = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
        assert torch.equal(t["pool"][t["table"][which, rows // 16].long(), rows % 16][:, :L], t["c_new"])
        want, tol = ref.attend_all(t, True, step != 0)
        check(out, want, tol, f"step {step}")
        lens = t["ctx"]


def test_append_far_positions(bd):
    """Angles of positions past a million tokens."""
    s = ref.make([2, 1], [0, 0], 4, 128, 64, 64, 7, garbage=1.0)
    s["before"] = [1_000_003, 7_654_321]
    s["ctx_before"] = torch.tensor(s["before"], dtype=torch.int32)
    s["table"] = torch.full((2, 500_000), -1, dtype=torch.int32)
    s["table"][0, 1_000_003 // 16], s["table"][1, 7_654_321 // 16] = 0, 1
    d = up(s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run_append(bd, s, d, True, err=err)
    assert int(err) == 0
    _check_append(s, d, q_out)


def test_blocks_beyond_32_bits(bd):
    """Blocks whose values lie past 2^31 elements and 2^32 bytes of the pool."""
    L, Hq, nblocks = 512, 4, 240_000                      # 2.2e9 elements, 4.4 GB
    s = ref.make([9, 33], [70, 0], Hq, L, 128, 128, 61)
    pool = torch.empty((nblocks, 16, L + 64), dtype=torch.bfloat16, device="cuda")
    used = s["pool"].shape[0]
    ids = torch.where(torch.arange(used) % 3 == 0, torch.arange(used), nblocks - 1 - torch.arange(used))
    pool[ids.cuda()] = s["pool"].cuda()
    d = up(s)
    d["table"] = torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0).long()].int(), s["table"]).cuda()
    d["pool"] = pool
    q = run_append(bd, s, d, ragged=True)
    t = dict(s, pool=pool[ids.cuda()].cpu(), q_rope=q.cpu())
    at = 0
    for b, (n, before) in enumerate(zip(s["new"], s["before"])):
        for j in range(n):
            got = t["pool"][s["table"][b, (before + j) // 16].long(), (before + j) % 16]
            assert torch.equal(got[:L], s["c_new"][at + j])
            check_rotated(got[None, L:], s["kr_new"][at + j][None], torch.tensor([before + j]))
        at += n
    d["q_rope"] = q
    want, tol = ref.attend_all(t, True, False)
    check(run_prefill(bd, s, d), want, tol, "prompt")
    u = ref.make([1, 1], [78, 32], Hq, L, 128, 128, 62)
    t.update(new=[1, 1], T=2, row_start=u["row_start"], q_nope=u["q_nope"], q_rope=u["q_rope"])
    e = dict(d, q_nope=u["q_nope"].cuda(), q_rope=u["q_rope"].cuda())
    want, tol = ref.attend_all(t, False, True)
    out = run_decode(bd, t, e, 1, False)
    check(out.view(2, Hq, 128), want, tol, "step")


def test_append_many_rows(bd):
    """More rows than CTAs run at once: four rows a CTA, the last CTA partly filled."""
    new = [701, 0, 1200, 1, 600]
    s = ref.make(new, [3, 0, 90, 15, 1], 2, 64, 64, 64, 8, garbage=1.0)
    d = up(s)
    _check_append(s, d, run_append(bd, s, d, True))
    s = ref.make([2447], [5], 2, 64, 64, 64, 9, garbage=1.0)
    d = up(s)
    _check_append(s, d, run_append(bd, s, d, False))


def test_shared_prefix_blocks(bd):
    """Streams whose tables name the same blocks (a shared voice prompt)."""
    s = ref.make([3, 3, 3], [61, 61, 61], 8, 128, 64, 64, 81)
    s["table"][1, :2] = s["table"][0, :2]
    s["table"][2, 1] = s["table"][0, 1]
    d = up(s)
    want, tol = ref.attend_all(s, True, True)
    check(run_decode(bd, s, d, 3, True).view(9, 8, 64), want, tol, "decode")
    want, tol = ref.attend_all(s, True, False)
    check(run_prefill(bd, s, d), want, tol, "prefill")


def test_two_streams_at_once(bd):
    """Calls that overlap, each with its own workspace."""
    cases, outs = [], []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(3):
        s = ref.make([2] * 20, [50 * i + 7 * k for k in range(20)], 16, 256, 64, 64, 90 + i)
        d = up(s)
        ws = [poisoned(bd.tts_latent_decode_attn_workspace_size(20, 2, 16, 256, 64, 64, max(s["ctx"]))),
              poisoned(bd.tts_latent_prefill_attn_workspace_size(20, s["T"], 16, 256, 64, 64, sum(s["ctx"])))]
        out = [torch.full((20, 2, 16, 64), NAN, dtype=torch.bfloat16, device="cuda"),
               torch.full((40, 16, 64), NAN, dtype=torch.bfloat16, device="cuda")]
        cases.append((s, d, ws, out))
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (s, d, ws, out) in zip(streams, cases):
            with torch.cuda.stream(st):
                run_decode(bd, s, d, 2, True, ws=ws[0], out=out[0])
                run_prefill(bd, s, d, ws=ws[1], out=out[1])
    torch.cuda.synchronize()
    for s, d, ws, out in cases:
        want, tol = ref.attend_all(s, True, True)
        check(out[0].view(40, 16, 64), want, tol, "decode")
        want, tol = ref.attend_all(s, True, False)
        check(out[1], want, tol, "prefill")


def test_two_graphs_share_a_workspace(bd):
    """A decode and a prompt call captured with one workspace, replayed in turn."""
    s = ref.make([1] * 6, [40 * k + 3 for k in range(6)], 16, 256, 64, 64, 95)
    t = ref.make([50, 7, 130], [0, 20, 3], 16, 256, 64, 64, 96)
    d, e = up(s), up(t)
    ws = poisoned(max(bd.tts_latent_decode_attn_workspace_size(6, 1, 16, 256, 64, 64, max(s["ctx"])),
                      bd.tts_latent_prefill_attn_workspace_size(3, t["T"], 16, 256, 64, 64, sum(t["ctx"]))))
    out = [torch.full((6, 1, 16, 64), NAN, dtype=torch.bfloat16, device="cuda"),
           torch.full((t["T"], 16, 64), NAN, dtype=torch.bfloat16, device="cuda")]
    graphs = []
    for run in (lambda: run_decode(bd, s, d, 1, False, ws=ws, out=out[0]), lambda: run_prefill(bd, t, e, ws=ws, out=out[1])):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for o in out:
        o.fill_(NAN)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    want, tol = ref.attend_all(s, False, True)
    check(out[0].view(6, 16, 64), want, tol, "decode")
    want, tol = ref.attend_all(t, True, False)
    check(out[1], want, tol, "prefill")


def test_programmatic_launches(bd):
    """Append, attention, append, attention, .. with programmatic launches: each
    call sees what the one before wrote."""
    from decode_step_gb300 import _lib
    Hq, L = 16, 512
    s = ref.make([1] * 30, [20 + 9 * i for i in range(30)], Hq, L, 128, 128, 97)
    d = up(s)
    cache = bd.LatentCache(d["pool"], L)
    ws = poisoned(bd.tts_latent_decode_attn_workspace_size(30, 1, Hq, L, 128, 128, 400))
    prev = bd.tts_set_launch_flags(_lib.LAUNCH_PROGRAMMATIC)
    try:
        outs, qs, steps = [], [], []
        for i in range(4):
            t = ref.make([1] * 30, s["before"], Hq, L, 128, 128, 100 + i)
            e = up(t)
            q = torch.empty_like(e["q_rope"])
            out = torch.empty((30, 1, Hq, 128), dtype=torch.bfloat16, device="cuda")
            steps.append((t, e))
            qs.append(q)
            outs.append(out)
        torch.cuda.synchronize()
        for (t, e), q, out in zip(steps, qs, outs):     # the same slots again and again
            bd.tts_latent_append(cache, d["table"], d["ctx_before"], e["c_new"], e["kr_new"], e["q_rope"], q, BASE)
            bd.tts_latent_decode_attn(cache, d["table"], d["ctx_lens"], 400, e["q_nope"].view(30, 1, Hq, 128),
                                      q.view(30, 1, Hq, 64), d["w_uk"], d["w_uv"], out, ws, s["scale"])
    finally:
        bd.tts_set_launch_flags(prev)
    torch.cuda.synchronize()
    pool = s["pool"]
    for (t, e), q, out in zip(steps, qs, outs):
        for b in range(30):
            p = s["before"][b]
            pool[int(s["table"][b, p // 16]), p % 16] = torch.cat(
                (t["c_new"][b], ref.rotate(t["kr_new"][b], torch.tensor(p), BASE).to(torch.bfloat16)))
        u = dict(s, pool=pool, q_nope=t["q_nope"], q_rope=q.cpu())
        want, tol = ref.attend_all(u, False, True)
        # a value of the new token's stored key part may be rounded the other way than here: a step (2^-7) of
        # a value near 1, times a query value near 1 and the scale 0.072, times its weight, at most 1 / 20
        check(out.view(30, Hq, 128), want, tol + 2.0 ** -7 * 0.072 * 4 / 20, "step")


def test_latent_step(bd):
    """LatentStep: prompts, then steps that pick tokens, eagerly and captured."""
    from decode_step_gb300.step import LatentStep
    Hq, L, nope, v, V = 8, 128, 64, 64, 600
    s = ref.make([40, 1, 77], [0, 0, 0], Hq, L, nope, v, 98, max_blocks=10, spare=40)
    s["table"] = torch.randperm(s["pool"].shape[0], generator=torch.Generator().manual_seed(5))[:30].to(torch.int32).view(3, 10).contiguous()
    s["pool"].fill_(NAN)
    d = up(s)
    W = (torch.randn(V, Hq * v, generator=torch.Generator().manual_seed(6)) * 0.2).to(torch.bfloat16).cuda()
    cache = bd.LatentCache(d["pool"], L)
    step = LatentStep(cache, d["w_uk"], d["w_uv"], W, 3, 160, prompt_rows=128, prompt_ctx=200)
    out = step.prompt(d["table"], d["ctx_before"], d["ctx_lens"], d["row_start"], d["q_nope"], d["q_rope"], d["c_new"], d["kr_new"])
    torch.cuda.synchronize()
    t = dict(s, pool=d["pool"].cpu(), q_rope=step.q[:118].cpu())
    want, tol = ref.attend_all(t, True, False)
    check(out, want, tol, "prompt")
    with pytest.raises(ValueError, match="prompt rows"):
        step.prompt(d["table"], d["ctx_before"], d["ctx_lens"], d["row_start"], d["q_nope"], d["q_rope"],
                    torch.zeros(129, L, dtype=torch.bfloat16, device="cuda"), d["kr_new"])
    e = up(ref.make([1] * 3, s["ctx"], Hq, L, nope, v, 99))
    args = (d["table"], e["ctx_before"], e["ctx_lens"], e["q_nope"].view(3, 1, Hq, nope), e["q_rope"].view(3, 1, Hq, 64),
            e["c_new"], e["kr_new"])

    def check_step():
        torch.cuda.synchronize()
        u = dict(s, new=[1] * 3, ctx=[c + 1 for c in s["ctx"]], T=3, row_start=torch.arange(4), pool=d["pool"].cpu(),
                 q_nope=e["q_nope"].cpu(), q_rope=step.q[:3].cpu())
        want, tol = ref.attend_all(u, False, True)
        check(step.out.view(3, Hq, v), want, tol, "step")
        logits = step.out.view(3, -1).double() @ W.double().t()
        top = logits.topk(2, 1)
        clear = (top.values[:, 0] - top.values[:, 1] > 1e-3).cpu()
        assert clear.any() and torch.equal(step.ids.cpu()[clear], top.indices[:, 0].int().cpu()[clear])
        assert int(step.err) == 0

    step(*args)
    check_step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*args)
    step.out.fill_(NAN)
    step.ids.fill_(-1)
    g.replay()
    check_step()


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("L,nope,v", [(64, 64, 64), (128, 64, 128), (256, 64, 64), (512, 128, 128)])
def test_first_call_of_a_process(op, L, nope, v):
    """A shape's launch does not rest on what another shape's set up before."""
    code = f"""
import sys; sys.path[:0] = {[str(ROOT), str(ROOT / "tests")]!r}
import torch, latent_ref as ref, test_gpu_latent as t
from decode_step_gb300 import binding as bd
s = ref.make([5], [20], 4, {L}, {nope}, {v}, 5)
out = t.run_decode(bd, s, t.up(s), 5, True) if {op == "decode"} else t.run_prefill(bd, s, t.up(s))
want, tol = ref.attend_all(s, True, {op == "decode"})
t.check(out.view(5, 4, {v}), want, tol)
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_tensor_checks(bd):
    s = ref.make([1, 1], [20, 30], 4, 128, 64, 64, 71)
    d = up(s)
    with pytest.raises(ValueError):
        run_decode(bd, s, {**d, "q_nope": d["q_nope"].float()}, 1, False)
    with pytest.raises(ValueError):
        run_decode(bd, s, {**d, "w_uk": d["w_uk"][:, :, :64]}, 1, False)
    with pytest.raises(ValueError):
        run_decode(bd, s, {**d, "ctx_lens": d["ctx_lens"].long()}, 1, False)
    with pytest.raises(ValueError):
        run_prefill(bd, s, {**d, "row_start": d["row_start"][:2]})
    with pytest.raises(bd.TTSError):
        run_decode(bd, s, d, 1, False, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert math.isfinite(s["scale"])
