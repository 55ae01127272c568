"""The tolerances of the latent cache's inner roundings are tight enough to see
a coarser one: the definition with that rounding planted in it fails them."""
import pytest
import torch

from test_gpu_latent_numerics import cancelling, decode_inputs, decode_tol, prefill_inputs, prefill_tol


def bf(x):
    return x.to(torch.bfloat16).double()


def f16(x):
    return x.to(torch.float16).double()


def two(x):
    return bf(x) + bf(x - bf(x))


@pytest.mark.parametrize("Hq", [16, 32, 48, 64, 128])
@pytest.mark.parametrize("ctx", [60, 500])
def test_decode_tolerance_sees_a_lost_remainder(Hq, ctx):
    x = cancelling(decode_inputs(Hq, ctx))
    tol = decode_tol(x)
    # (relative to the largest weight, as the kernel has them)
    top = x["p"].amax(1, keepdim=True)
    p = x["p"] / top

    def out(p, weights, latents):
        lat = latents((weights(p) @ x["c"]) / p.sum(1, keepdim=True))
        return bf(torch.einsum("hl,hdl->hd", lat, x["w"]))

    assert ((out(p, two, two) - x["out"]).abs() <= tol).all()
    assert ((out(p, bf, two) - x["out"]).abs() > tol).any(1).all(), "weights without their remainders, in every head"
    assert ((out(p, two, bf) - x["out"]).abs() > tol).any(1).all(), "latents without their remainders, in every head"


@pytest.mark.parametrize("v", [64, 128])
def test_prefill_tolerance_sees_bf16(v):
    x = cancelling(prefill_inputs(v))
    tol = prefill_tol(x)
    p = x["p"] / x["p"].amax(1, keepdim=True)

    def out(weights, values):
        return bf(torch.einsum("ht,htd->hd", weights(p), values(x["val"])) / p.sum(1, keepdim=True))

    assert ((out(f16, f16) - x["out"]).abs() <= tol).all()
    assert ((out(bf, f16) - x["out"]).abs() > tol).any()
    assert ((out(f16, bf) - x["out"]).abs() > tol).any()
