"""Steps and prompts with tokens that the append skips, and without any rows."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd
    from decode_step_gb300.step import LatentStep, WindowStep

HQ, HKV, D, V = 4, 2, 128, 300


def rand(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def window_step(window=40, rope=10000.0, dtype="bf16"):
    g = torch.Generator().manual_seed(1)
    pools = [rand(g, 20, HKV, 16, D) for _ in range(2)]
    W = (torch.randn(V, HQ * D, generator=g) * 0.05).to(torch.bfloat16).cuda()
    return WindowStep(bd.KVCache(*pools), W, HQ, 2, 160, window, 3, rope_base=rope, prompt_rows=60), g


@pytest.mark.parametrize("window", [0, 40])
def test_window_step_of_skipped_tokens_knows_no_earlier_call(window):
    """Stream 1's block is outside the pool in the second call: its rows are answered alike
    whatever the first call's queries were, and its tokens' queries are zeros."""
    for prompt in (False, True):
        outs = []
        for first in (1.0, -30.0, None):
            step, g = window_step(window)
            table = torch.arange(20, dtype=torch.int32).view(2, 10).cuda()
            n = 25 if prompt else 1
            T = 2 * n
            q, k, v = rand(g, T, HQ, D), rand(g, T, HKV, D), rand(g, T, HKV, D)

            def call(q, table):
                pos, lens = i32(40, 40), i32(40 + n, 40 + n)
                if prompt:
                    return step.prompt(table, pos, lens, i32(0, n, T), q, k, v)
                step(table, pos, lens, q.view(2, 1, HQ, D), k.view(2, 1, HKV, D), v.view(2, 1, HKV, D))
                return step.out.view(T, HQ, D)

            if first is not None:
                call(q * first, table)
            bad = table.clone()
            bad[1, 3 if prompt else 2:] = 999
            outs.append((call(q, bad).clone(), step.ids.clone()))
            assert int(step.err.item()) == _lib.ERRBIT_BLOCK_ID
            skipped = slice(n + (8 if prompt else 0), T)  # (40 + 8 tokens fill stream 1's good blocks)
            assert not step.q[skipped].any() and step.q[:n].any()
        for out, ids in outs[1:]:
            assert torch.equal(out, outs[0][0])
            assert prompt or torch.equal(ids, outs[0][1])


@pytest.mark.parametrize("prompt", [False, True])
def test_latent_step_of_skipped_tokens_knows_no_earlier_call(prompt):
    heads, lat, nope, vd = 8, 128, 64, 64
    n = 25 if prompt else 1
    T = 2 * n
    outs = []
    for first in (1.0, -30.0, None):
        g = torch.Generator().manual_seed(2)
        pool = rand(g, 20, 16, lat + 64)
        W = (torch.randn(V, heads * vd, generator=g) * 0.05).to(torch.bfloat16).cuda()
        step = LatentStep(bd.LatentCache(pool, lat), rand(g, heads, nope, lat), rand(g, heads, vd, lat), W, 2, 160,
                          prompt_rows=60, prompt_ctx=200)
        table = torch.arange(20, dtype=torch.int32).view(2, 10).cuda()
        qn, qr, c, kr = rand(g, T, heads, nope), rand(g, T, heads, 64), rand(g, T, lat), rand(g, T, 64)
        pos, lens = i32(40, 40), i32(40 + n, 40 + n)

        def call(qr, table):
            if prompt:
                return step.prompt(table, pos, lens, i32(0, n, T), qn, qr, c, kr)
            step(table, pos, lens, qn.view(2, 1, heads, nope), qr.view(2, 1, heads, 64), c, kr)
            return step.out.view(T, heads, vd)

        if first is not None:
            call(qr * first, table)
        bad = table.clone()
        bad[1, 3 if prompt else 2:] = 999
        outs.append((call(qr, bad).clone(), step.ids.clone()))
        assert int(step.err.item()) == _lib.ERRBIT_BLOCK_ID
        assert not step.q[n + (8 if prompt else 0):T].any() and step.q[:n].any()
    for out, ids in outs[1:]:
        assert torch.equal(out, outs[0][0])
        assert prompt or torch.equal(ids, outs[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rope", [0.0, 10000.0])
@pytest.mark.parametrize("streams", [0, 1, 2])
def test_no_rows(dtype, rope, streams):
    """An empty prompt, alone and through the object: nothing is done and nothing refused."""
    if dtype == "fp8":
        cache = bd.KVCache(torch.zeros(4, HKV, 4224, dtype=torch.uint8, device="cuda"))
    else:
        cache = bd.KVCache(*(torch.zeros(4, HKV, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = torch.zeros(streams, 2, dtype=torch.int32, device="cuda")
    lens, start = i32(*[0] * streams), i32(*[0] * (streams + 1))
    q, kv = (torch.zeros(0, h, D, dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV))
    err = i32(0)
    if rope:
        bd.tts_kv_append_packed(cache, table, lens, start, kv, kv, q, torch.empty_like(q), rope, err=err)
    else:
        bd.tts_kv_append_packed(cache, table, lens, start, kv, kv, err=err)
    ws = torch.zeros(bd.tts_prompt_attn_workspace_size(streams, 0, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    bd.tts_prompt_attn(cache, table, lens, start, q, torch.empty_like(q), ws, 0.1, err=err)
    if streams:
        W = torch.zeros(V, HQ * D, dtype=torch.bfloat16, device="cuda")
        step = WindowStep(cache, W, HQ, streams, 32, 8, 3, rope_base=rope, prompt_rows=4)
        out = step.prompt(table, lens, lens, start, q, kv, kv)
        assert out.shape == (0, HQ, D) and int(step.err.item()) == 0
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not cache.k_pool.any()


def test_a_float32_cache_has_steps_and_no_prompts():
    g = torch.Generator().manual_seed(4)
    pools = [torch.randn(20, HKV, 16, 64, generator=g).cuda() for _ in range(2)]
    cache = bd.KVCache(*pools)
    W = torch.randn(V, HQ * 64, generator=g).cuda()
    for bad in (dict(), dict(rope_base=0.0, prompt_rows=4), dict(rope_base=10000.0)):
        with pytest.raises(ValueError, match="float32"):
            WindowStep(cache, W, HQ, 2, 160, 40, 3, **bad)
    table = torch.arange(20, dtype=torch.int32).view(2, 10)
    for window in (0, 40):
        step = WindowStep(cache, W, HQ, 2, 160, window, 3, rope_base=0.0)
        q, k, v = (torch.randn(2, 1, h, 64, generator=g) for h in (HQ, HKV, HKV))
        step(table.cuda(), i32(100, 7), i32(101, 8), q.cuda(), k.cuda(), v.cuda())
        torch.cuda.synchronize()
        assert int(step.err.item()) == 0
        for b, p in ((0, 100), (1, 7)):
            assert all(torch.equal(x[int(table[b, p // 16]), :, p % 16].cpu(), y[b, 0]) for x, y in zip(pools, (k, v)))
        s = dict(new=[1, 1], before=[100, 7], ctx=[101, 8], Hq=HQ, Hkv=HKV, D=64, dtype="f32", window=window, sinks=3,
                 causal=False, scale=step.scale, table=table, k_val=pools[0].cpu().double(), v_val=pools[1].cpu().double(),
                 T=2, q=q.view(2, HQ, 64), row_start=torch.tensor([0, 1, 2]))
        pr.check(step.out.view(2, HQ, 64), *pr.attend_all(s))


def test_captured_prompt_and_steps_follow_their_inputs():
    """A prompt and two steps in one graph, zeros and appends among them, replayed with other tokens,
    and with a block outside the pool: as the same calls one after another."""
    step, g = window_step()
    other, _ = window_step()
    table = torch.arange(20, dtype=torch.int32).view(2, 10).cuda()
    q, k, v = (torch.empty(54, h, D, dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
    at = [i32(0, 30), i32(25, 55), i32(26, 56), i32(27, 57)]
    start = i32(0, 25, 50)

    def calls(step):
        out = [step.prompt(table, at[0], at[1], start, q[:50], k[:50], v[:50]).clone()]
        for i in range(2):
            rows = slice(50 + 2 * i, 52 + 2 * i)
            step(table, at[1 + i], at[2 + i], q[rows].view(2, 1, HQ, D), k[rows].view(2, 1, HKV, D),
                 v[rows].view(2, 1, HKV, D))
            out += [step.out.clone(), step.ids.clone()]
        return out

    for x in (q, k, v):
        x.copy_(rand(g, *x.shape))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        calls(step)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = calls(step)
    for bad in (False, True, False):
        for x in (q, k, v):
            x.copy_(rand(g, *x.shape))
        table[1, 3] = 999 if bad else 13
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = calls(other)
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)
        assert all(torch.equal(a, b) for a, b in zip((step.cache.k_pool, step.cache.v_pool),
                                                     (other.cache.k_pool, other.cache.v_pool)))
    assert int(step.err.item()) == int(other.err.item()) == _lib.ERRBIT_BLOCK_ID
