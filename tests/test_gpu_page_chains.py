"""Page moves, appends and attention in chains whose kernels start while the one
before still runs: each reads what the one before, and the one before that,
wrote.  Compared bit for bit with the same calls one at a time."""
from __future__ import annotations

import contextlib

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd

ROUNDS, B, L = 24, 3, 77  # streams 0 and 2 hold L tokens


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t if t.dtype == torch.uint8 else t.view(torch.int16 if t.element_size() == 2 else torch.int32)


@contextlib.contextmanager
def launches(flags):
    before = bd.tts_set_launch_flags(flags)
    try:
        yield
    finally:
        bd.tts_set_launch_flags(before)


def state(dtype, seed):
    """Two streams of L tokens in blocks 0-4 and 5-9 of 24, stream 1 empty, and new tokens for every round."""
    g = torch.Generator().manual_seed(seed)
    D, elem = pr.dim(dtype), torch.float32 if dtype == "f32" else torch.bfloat16
    k, v = (torch.randn(24, 2, 16, D, generator=g).to(elem) for _ in range(2))
    if dtype == "fp8":
        pools = (pr.records(*pr.quantise(k), *pr.quantise(v)).cuda(), None)
    else:
        pools = (k.cuda(), v.cuda())
    rows = [torch.randn(ROUNDS + 1, 1, h, D, generator=g).to(elem).cuda() for h in (2, 2, 4)]
    q = torch.randn(ROUNDS, B, 1, 4, D, generator=g).to(elem).cuda()
    table = torch.full((B, 8), -1, dtype=torch.int32)
    table[0, :5], table[2, :5] = torch.arange(5), torch.arange(5, 10)
    return bd.KVCache(*pools), pools, table.cuda(), rows, q


def decode(cache, table, lens, q, window, ws):
    out = torch.empty_like(q)
    scale = q.shape[-1] ** -0.5
    if window:
        bd.tts_window_decode_attn(cache, table, lens, 128, q, out, ws, scale, window, 4)
    else:
        bd.tts_decode_attn(cache, table, lens, 128, q, out, ws, scale)
    return out


def forks(dtype, window, flags):
    """Stream 1 forked from 0 and 2 in turns into one of two blocks, a token appended, a step of all three."""
    cache, pools, table, (k, v, _), q = state(dtype, 71)
    pos, lens, start = i32(L, 0, L), i32(L, L + 1, L), i32(0, 0, 1, 1)
    parent, child, fresh = (i32(0), i32(2)), i32(1), (i32(20), i32(21), i32(22))
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(B, 1, 4, 2, q.shape[-1], 128), dtype=torch.uint8, device="cuda")
    outs = []
    torch.cuda.synchronize()
    with launches(flags):
        for i in range(ROUNDS):
            bd.tts_kv_fork(cache, table, pos, parent[i % 2], child, fresh[i % 3])
            bd.tts_kv_append_packed(cache, table, pos, start, k[i], v[i])
            outs.append(decode(cache, table, lens, q[i], window, ws))
            if not flags:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    return outs, [table, pos] + [p for p in pools if p is not None]


def moves(dtype, window, flags):
    """The blocks of streams 0 and 2 moved to others and back, the last token of both written anew, a step."""
    cache, pools, table, (k, v, _), q = state(dtype, 72)
    there, back = list(range(24)), list(range(24))
    for i in range(10):
        there[i], back[12 + i] = 12 + i, i
    maps = i32(*there), i32(*back)
    pos, lens, start = i32(L - 1, 0, L - 1), i32(L, 0, L), i32(0, 1, 1, 2)
    ws = torch.zeros(bd.tts_decode_attn_workspace_size(B, 1, 4, 2, q.shape[-1], 128), dtype=torch.uint8, device="cuda")
    outs = []
    torch.cuda.synchronize()
    with launches(flags):
        for i in range(ROUNDS):
            bd.tts_kv_compact(cache, maps[i % 2], table)
            bd.tts_kv_append_packed(cache, table, pos, start, k[i:i + 2].view(2, 2, -1), v[i:i + 2].view(2, 2, -1))
            outs.append(decode(cache, table, lens, q[i], window, ws))
            if not flags:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    return outs, [table] + [p for p in pools if p is not None]


def same(run, *args):
    (want, kept), (got, now) = run(*args, 0), run(*args, _lib.LAUNCH_PROGRAMMATIC)
    for i, (x, y) in enumerate(zip(want, got)):
        assert torch.equal(bits(x), bits(y)), i
    assert not torch.equal(bits(want[0]), bits(want[1]))
    for x, y in zip(kept, now):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [0, 30])
def test_fork_append_decode(dtype, window):
    same(forks, dtype, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [0, 30])
def test_compact_append_decode(dtype, window):
    same(moves, dtype, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("before", [0, 2000])
def test_append_and_prompt(dtype, before):
    """New tokens and queries in every round, rotated on the way: keys, values and queries all come
    from the kernel before.  The prompt is long enough, with 2,000 tokens before it, for parts."""
    new = [100, 33]
    s = pr.make(new, [before, 300], 4, 2, dtype, seed=73, garbage=0.0, hide=False)
    pools = tuple(None if p is None else p.cuda() for p in s["pools"])
    cache, table, lens, start = bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda(), s["row_start"].cuda()
    pos = s["ctx_before"].cuda()
    g = torch.Generator().manual_seed(74)
    k, v, q = (torch.randn(8, 133, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (2, 2, 4))
    ws = torch.zeros(bd.tts_prompt_attn_workspace_size(2, 133, 4, 2, 128), dtype=torch.uint8, device="cuda")
    turned = torch.empty_like(q[0])
    runs = []
    for flags in (0, _lib.LAUNCH_PROGRAMMATIC):
        outs = [torch.empty_like(q[0]) for _ in range(8)]
        torch.cuda.synchronize()
        with launches(flags):
            for i, out in enumerate(outs):
                bd.tts_kv_append_packed(cache, table, pos, start, k[i], v[i], q[i], turned, 10000.0)
                bd.tts_prompt_attn(cache, table, lens, start, turned, out, ws, s["scale"])
                if not flags:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        runs.append(outs)
    for i, (x, y) in enumerate(zip(*runs)):
        assert torch.equal(x, y), i
        assert i == 0 or not torch.equal(x, runs[0][i - 1])


def test_every_ticket_is_zero_again():
    """Long segments split over a few CTAs from the first one on, joined by the last of them: the
    tickets, at the workspace's end, are all zero afterwards."""
    s = pr.make([130, 5], [700, 900], 4, 2, "bf16", seed=75)
    pools = tuple(p.cuda() for p in s["pools"])
    q = s["q"].cuda()
    out = torch.empty_like(q)
    ws = torch.zeros(bd.tts_prompt_attn_workspace_size(2, s["T"], 4, 2, 128), dtype=torch.uint8, device="cuda")
    tickets = -(-8 * torch.cuda.get_device_properties(0).multi_processor_count // 256) * 256
    for _ in range(3):
        bd.tts_prompt_attn(bd.KVCache(*pools), s["table"].cuda(), s["ctx_lens"].cuda(), s["row_start"].cuda(), q, out, ws,
                           s["scale"])
        torch.cuda.synchronize()
        assert ws[:-tickets].any() and not ws[-tickets:].any()
    pr.check(out, *pr.attend_all(s))
