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
