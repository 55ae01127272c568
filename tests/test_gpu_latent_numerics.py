"""Latents that are not finite, weights that are not finite, scores and values
far from one, and the inner roundings of the latent cache's attentions, against
the 64-bit definition (decode and prompt calls on the GPU)."""
from __future__ import annotations

import math

import pytest
import torch

import latent_ref as ref
from test_gpu_latent import NAN, check, run_decode, run_prefill, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    from decode_step_gb300 import binding
    return binding


def spoil(s, b, t, l, what):
    """Element l of token t of stream b."""
    s["pool"][s["table"][b, t // 16].long(), t % 16, l] = what


def not_finite(x):
    return ~torch.isfinite(x.float())


# ------------------------------------------------- latents that are not finite

@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("q_len,ctx,Hq,first", [(5, 71, 16, 2), (5, 66, 4, 1), (3, 64, 16, 0), (8, 130, 20, 7), (70, 200, 2, 30)])
def test_decode_rows_that_see_an_infinite_latent(bd, what, q_len, ctx, Hq, first):
    """One element of a late token's latent: its score is minus infinity for
    the heads whose q~ has the other sign there, so that its weight is zero;
    in the definition the value times that zero is still not a number.  Rows
    before the token do not see it."""
    s = ref.make([q_len] * 2, [ctx - q_len] * 2, Hq, 192, 128, 64, 12)
    want, tol = ref.attend_all(s, True, True)
    spoil(s, 0, ctx - q_len + first, 11, what)
    out = run_decode(bd, s, up(s), q_len, True).view(2, q_len, Hq, 64)
    want, tol = want.view(out.shape), tol.view(out.shape)
    check(out[1], want[1], tol[1], "the other stream")
    if first:
        check(out[0, :first], want[0, :first], tol[0, :first], "rows before")
    assert not_finite(out[0, first:]).all()


@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
def test_decode_an_infinite_latent_that_all_rows_see(bd, what):
    s = ref.make([5] * 2, [100, 60], 16, 192, 128, 64, 13)
    want, tol = ref.attend_all(s, True, True)
    spoil(s, 0, 17, 191, what)
    out = run_decode(bd, s, up(s), 5, True).view(10, 16, 64)
    check(out[5:], want[5:], tol[5:], "the other stream")
    assert not_finite(out[:5]).all()


@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("n,before,spoilt", [(140, 20, 100), (300, 3, 200), (7, 0, 1), (20, 125, 3)])
def test_prefill_rows_that_see_an_infinite_latent(bd, what, n, before, spoilt):
    """Queries and key weights of one sign, so that every head's score of the
    token is an infinity of the latent's sign (minus: weight zero)."""
    s = ref.make([n, 9], [before, 2], 2, 128, 64, 128, 33)
    s["q_nope"], s["w_uk"] = s["q_nope"].abs(), s["w_uk"].abs()
    want, tol = ref.attend_all(s, True, False)
    spoil(s, 0, before + spoilt, 40, what)
    out = run_prefill(bd, s, up(s))
    check(out[n:], want[n:], tol[n:], "the other stream")
    check(out[:spoilt], want[:spoilt], tol[:spoilt], "rows before")
    assert not_finite(out[spoilt:n]).all()


# ------------------------------------------------- weights that are not finite

@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("v", [64, 128])
def test_value_weights_that_are_not_finite(bd, what, form, v):
    """An element of w_uv makes its output dimension of its head not finite in
    every row, and no other."""
    n = 3 if form == "decode" else 150
    s = ref.make([n, n], [40, 3], 3, 128, 64, v, 35)
    want, tol = ref.attend_all(s, True, form == "decode")
    s["w_uv"][1, 5, 77] = what
    s["w_uv"][2, v - 1, 0] = what
    d = up(s)
    out = (run_decode(bd, s, d, n, True) if form == "decode" else run_prefill(bd, s, d)).view(2 * n, 3, v).cpu()
    for h, dim in ((1, 5), (2, v - 1)):
        assert not_finite(out[:, h, dim]).all()
        out[:, h, dim] = 0
        want[:, h, dim] = 0
    check(out, want, tol + 1e-30, form)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("which", ["w_uk", "w_uv"])
def test_a_head_whose_weights_are_nan(bd, form, which):
    n = 3 if form == "decode" else 150
    s = ref.make([n, n], [40, 3], 3, 128, 64, 64, 36)
    want, tol = ref.attend_all(s, True, form == "decode")
    s[which][1] = NAN
    d = up(s)
    out = (run_decode(bd, s, d, n, True) if form == "decode" else run_prefill(bd, s, d)).view(2 * n, 3, 64)
    assert torch.isnan(out[:, 1].float()).all()
    for h in (0, 2):
        check(out[:, h], want[:, h], tol[:, h], f"head {h}")


@pytest.mark.parametrize("what", [NAN, math.inf])
@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("which", ["q_nope", "q_rope"])
def test_queries_that_are_not_finite(bd, what, form, which):
    """A query of one row and head reaches that row's output of that head."""
    n = 5 if form == "decode" else 150
    s = ref.make([n, n], [40, 3], 3, 128, 64, 64, 42)
    want, tol = ref.attend_all(s, True, form == "decode")
    s[which][n + 2, 1, 9] = what
    d = up(s)
    out = (run_decode(bd, s, d, n, True) if form == "decode" else run_prefill(bd, s, d)).view(2 * n, 3, 64).cpu()
    assert not_finite(out[n + 2, 1]).all()
    out[n + 2, 1] = want[n + 2, 1].to(torch.bfloat16)
    check(out, want, tol, form)


# --------------------------------------------------------- values far from one

@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("v", [64, 128])
@pytest.mark.parametrize("exps", [(-22, -22, -22), (-40, -40, -40), (20, 20, 20), (90, 90, 90), (0, -22, 24), (-60, 0, 17)])
def test_values_of_any_size(bd, form, v, exps):
    """Value weights times powers of two, head by head: the outputs scale
    exactly, so each is within the same relative tolerance."""
    n = 4 if form == "decode" else 150
    s = ref.make([n, n], [40, 3], 3, 128, 64, v, 37)
    want, tol = ref.attend_all(s, True, form == "decode")
    size = torch.tensor([2.0 ** e for e in exps], dtype=torch.float64).view(1, 3, 1)
    s["w_uv"] = (s["w_uv"].double() * size.view(3, 1, 1)).to(torch.bfloat16)
    d = up(s)
    out = (run_decode(bd, s, d, n, True) if form == "decode" else run_prefill(bd, s, d)).view(2 * n, 3, v)
    check(out.double().cpu() / size, want, tol, f"{form} {exps}")


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("small,large", [(1.0, 2.0 ** 20), (1.0, 2.0 ** 60), (2.0 ** -30, 1.0), (2.0 ** -24, 2.0 ** 30)])
def test_a_later_token_of_another_size(bd, form, small, large):
    """The first tokens' latents times `small`, a later one's times `large`:
    rows before it have outputs of the small size, rows that see it are right
    too.  (The keys are kept apart: q_nope is zero, the scores are the rotated
    parts'.)"""
    n, before = (8, 50) if form == "decode" else (200, 10)
    s = ref.make([n, 5 if form == "prefill" else n], [before, 2], 2, 128, 64, 64, 38)
    s["q_nope"].zero_()
    ids, spoilt = s["table"][0, :-(-s["ctx"][0] // 16)].long(), n // 2
    rows = s["pool"][ids].view(-1, 192)
    rows[:s["ctx"][0], :128] = (rows[:s["ctx"][0], :128].double() * small).to(torch.bfloat16)
    t = before + spoilt
    rows[t, :128] = (rows[t, :128].double() / small * large).to(torch.bfloat16)
    s["pool"][ids] = rows.view(-1, 16, 192)
    want, tol = ref.attend_all(s, True, form == "decode")
    d = up(s)
    out = run_decode(bd, s, d, n, True).view(2 * n, 2, 64) if form == "decode" else run_prefill(bd, s, d)
    check(out[n:], want[n:], tol[n:], "the other stream")
    check(out[:spoilt], want[:spoilt], tol[:spoilt], "rows before")
    check(out[spoilt:n], want[spoilt:n], tol[spoilt:n], "rows that see it")


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -12, 1.0, 2.0 ** 40])
def test_prompt_tokens_without_values(bd, size):
    """The first 130 tokens' latents are zero, the others of one size: the
    zeros have their weights and add nothing."""
    s = ref.make([170], [60], 2, 128, 64, 64, 41)
    s["q_nope"].zero_()
    ids = s["table"][0, :-(-s["ctx"][0] // 16)].long()
    rows = s["pool"][ids].view(-1, 192)
    rows[:130, :128] = 0
    rows[130:230, :128] = (rows[130:230, :128].double() * size).to(torch.bfloat16)
    s["pool"][ids] = rows.view(-1, 16, 192)
    want, tol = ref.attend_all(s, True, False)
    out = run_prefill(bd, s, up(s))
    check(out, want, tol)
    assert (out[:70] == 0).all() and (out[70:] != 0).any()


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_scores_far_below_zero(bd, form):
    """Every score of a row at -1.2e32 or (the first tokens') twice that: the
    softmax is over the others, evenly."""
    n = 2 if form == "decode" else 140
    s = ref.make([n], [90], 2, 128, 64, 64, 39)
    s["q_nope"].zero_()
    s["q_rope"].zero_()
    s["q_rope"][..., 3] = -2.0 ** 55
    ids = s["table"][0, :-(-s["ctx"][0] // 16)].long()
    rows = s["pool"][ids].view(-1, 192)
    rows[:, 128:] = 0
    rows[:, 128 + 3] = 2.0 ** 55
    rows[:70, 128 + 3] = 2.0 ** 56
    s["pool"][ids] = rows.view(-1, 16, 192)
    want, tol = ref.attend_all(s, True, form == "decode")
    assert (want != 0).all()
    d = up(s)
    out = run_decode(bd, s, d, n, True).view(n, 2, 64) if form == "decode" else run_prefill(bd, s, d)
    check(out, want, tol, form)


# --------------------------------------------------------- the inner roundings
#
# q_nope is zero, so q~ and the expanded keys do not matter and the scores are
# the rotated parts' (fp32).  A head's w_uv takes two latent dimensions in the
# proportion in which its row's attended latent cancels, so that the output is
# some 2^-9 of its terms and its own rounding some 2^-17 of them: what is left
# is the roundings inside.  In units of the terms, with half steps h (bf16 2^-8,
# f16 2^-11) and softmax weights p_t:
#   decode  weights and attended latents each as a rounding and the rounding of
#           its remainder: off by at most h^2 = 2^-16 each
#   prompt  weights and values to f16: independent, each of variance at most
#           h^2 / 3 = 2^-22 / 3 of its square
# plus 2^-18 of the terms for fp32 (scores up to 16 to 2^-23 of themselves, the
# hardware exponential, sums of some hundred terms) and half a step of the output.

def cancelling(s):
    """w_uv so that the last row's outputs cancel; returns, per head and output
    dimension, the definition's output, the sum of the terms' sizes over tokens
    and over latent dimensions, and the root of the sum of their squares."""
    Hq, L, v = s["Hq"], s["L"], s["v"]
    s["q_nope"].zero_()
    rows, _ = ref.cached_rows(s, 0)
    c, kr = rows[:, :L], rows[:, L:]
    sc = s["scale"] * (s["q_rope"][s["new"][0] - 1].double() @ kr.t())
    assert float(sc.abs().max()) < 16
    p = torch.softmax(sc, 1)                                   # [Hq][ctx]
    lat = p @ c
    s["w_uv"].zero_()
    for h in range(Hq):
        for d in range(v):
            i, j = d, v + (5 * d + 3 * h) % (L - v)
            k = math.frexp(max(abs(float(lat[h, i])), abs(float(lat[h, j]))))[1]
            s["w_uv"][h, d, i] = math.ldexp(float(lat[h, j]), -k)
            s["w_uv"][h, d, j] = -math.ldexp(float(lat[h, i]), -k)
    w = s["w_uv"].double()
    val = torch.einsum("hdl,tl->htd", w, c)
    out = torch.einsum("ht,htd->hd", p, val)
    assert (ref.attend(s, 0, True, False)[0][-1] - out).abs().max() < 1e-12
    return dict(p=p, c=c, w=w, val=val, out=out,
                tokens=torch.einsum("ht,hdl,tl->hd", p, w.abs(), c.abs()), latents=torch.einsum("hl,hdl->hd", lat.abs(), w.abs()),
                squares=torch.einsum("ht,htd->hd", p * p, val * val).sqrt(),
                values=torch.einsum("ht,htd->hd", p, val.abs()))


def decode_tol(x):
    return 2.0 ** -8 * x["out"].abs() + 2.0 ** -16 * (x["tokens"] + x["latents"]) + 2.0 ** -18 * x["tokens"]


def prefill_tol(x):
    # eight standard deviations of 2 squares' worth of roundings
    return 2.0 ** -8 * x["out"].abs() + 8 * 2.0 ** -11 * x["squares"] * (2 / 3) ** 0.5 + 2.0 ** -18 * x["tokens"]


def decode_inputs(Hq, ctx):
    return ref.make([1], [ctx - 1], Hq, 192, 64, 64, 40 + Hq, q_gain=3.0)


def prefill_inputs(v):
    return ref.make([150], [60], 16, 256, 64, v, 50 + v, q_gain=3.0)


@pytest.mark.parametrize("Hq", [16, 32, 48, 64, 128])
@pytest.mark.parametrize("ctx", [60, 500])
def test_decode_inner_roundings(bd, Hq, ctx):
    s = decode_inputs(Hq, ctx)
    x = cancelling(s)
    out = run_decode(bd, s, up(s), 1, False)
    check(out.view(Hq, 64), x["out"], decode_tol(x), "decode")


@pytest.mark.parametrize("v", [64, 128])
def test_prefill_inner_roundings(bd, v):
    s = prefill_inputs(v)
    x = cancelling(s)
    out = run_prefill(bd, s, up(s))
    check(out[-1], x["out"], prefill_tol(x), "prefill")
