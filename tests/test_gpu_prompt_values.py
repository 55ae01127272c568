"""tts_prompt_attn: values that are not finite in the places where the kernel
looks them up by a part's note, in tiles beside blocks outside the pool, and in
parts whose rows have no weights."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd

NAN = float("nan")


def run(s, err=None):
    pools = tuple(None if p is None else p.cuda() for p in s["pools"])
    q = s["q"].cuda()
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(bd.tts_prompt_attn_workspace_size(len(s["new"]), s["T"], s["Hq"], s["Hkv"], s["D"]), dtype=torch.uint8,
                     device="cuda")
    bd.tts_prompt_attn(bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda(), s["row_start"].cuda(), q, out, ws,
                       s["scale"], s["window"], s["sinks"], err=err)
    torch.cuda.synchronize()
    return out


def put(s, b, t, g, d, value):
    """Value (token t, KV head g, dimension d) of stream b; NaN in an FP8 cache."""
    block, slot = int(s["table"][b, t // 16]), t % 16
    if s["dtype"] == "fp8":
        assert value != value
        s["pools"][0][block, g, 2048 + 16 * d + 4 * (slot % 8 // 2) + slot % 2 + 2 * (slot // 8)] = 0x7F
    else:
        s["pools"][1][block, g, slot, d] = value
    s["v_val"][block, g, slot, d] = value


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_value_looked_up_while_short_segments_follow(dtype):
    """A stream with rows for both halves of a query tile, whose last rows see values that are
    not finite in the last KV head; the CTA goes on with some twenty segments of one tile and one
    half, whose notes must not take the place of the note that the other half still reads."""
    s = pr.make([100] + [1 + i % 30 for i in range(600)], [0] + [i % 20 for i in range(600)], 16, 8, dtype, seed=51)
    for d in (5, 40, 70, 127):
        put(s, 0, 98, 7, d, NAN)
    put(s, 0, 66, 7, 33, NAN)
    ref, tol = pr.attend_all(s)
    assert int(torch.isnan(ref).sum()) == 2 * (2 * 4 + 34)
    for _ in range(5):
        pr.check(run(s), ref, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_value_beside_a_block_outside_the_pool(dtype):
    """In a tile that every row sees whole but for one block: the value reaches every row. In the
    bad block's place nothing does, whatever an earlier tile left there."""
    s = pr.make([40], [400], 4, 2, dtype, seed=52)
    s["table"][0, 7] = s["k_pool"].shape[0]        # tokens 112..127, in the tile of 80..159
    s["table"][0, 20] = -5                         # tokens 320..335, in the tile of 320..399
    put(s, 0, 100, 1, 5, NAN)
    put(s, 0, 390, 0, 77, NAN)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref, tol = pr.attend_all(s)
    assert int(torch.isnan(ref).sum()) == 2 * 2 * 40
    pr.check(run(s, err), ref, tol)
    assert int(err.item()) == _lib.ERRBIT_BLOCK_ID


@pytest.mark.parametrize("new", [5, 100])
def test_a_value_in_a_part_without_weights(new):
    """Keys of -inf in the last 1,500 tokens: the last CTAs' parts of a segment have no weights
    (one half's rows in turns, and both halves'), and a value in them that is no number still
    reaches the rows that see it."""
    s = pr.make([new], [9000], 4, 2, "bf16", seed=53)
    s["q"] = s["q"].abs() + 0.1
    for t in range(9000 + new - 1500, 9000 + new):
        s["k_pool"][int(s["table"][0, t // 16]), :, t % 16] = float("-inf")
    pr.finish(s)
    put(s, 0, 9000 + new - 2, 1, 5, NAN)
    put(s, 0, 9000 + new - 1, 0, 99, NAN)
    ref, tol = pr.attend_all(s)
    assert int(torch.isnan(ref).sum()) == 2 * 2 + 2 * 1
    pr.check(run(s), ref, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [3, 100])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("size", [1e5, 1e8, 1e11, 1e30, 1e34])
def test_scores_of_any_size(dtype, new, sign, size):
    """Keys in steps of which one takes it all, scores from 1e6 to 2e35 on either side of zero; the
    first tokens see all of one step, so that the maximum moves on the way."""
    s = pr.make([new, 7], [5000, 0], 4, 2, dtype, seed=61)
    s["q"] = torch.ones_like(s["q"])
    far = torch.rand(s["k_pool"].shape[:3], generator=torch.Generator().manual_seed(62)) < 0.25
    for t in range(700):
        far[int(s["table"][0, t // 16]), :, t % 16] = sign < 0
    k = (sign * size * torch.where(far, 2.0, 1.0))[..., None].expand(s["k_pool"].shape)
    s["k_pool"] = torch.where(torch.isfinite(s["k_pool"]), k.to(s["k_pool"].dtype), s["k_pool"])
    pr.finish(s)
    ref, tol = pr.attend_all(s)
    assert torch.isfinite(ref).all() and bool((ref.abs().amax(-1) > 0.01).all())
    pr.check(run(s), ref, tol)
