"""WindowStep as a server uses it: prompts of several lengths, token steps whose
contexts leave the window, blocks given back and taken again, a fork with its
shared and copied blocks, a compaction in between; every output against the
64-bit reference on the cache as stored."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import binding as bd
    from decode_step_gb300.step import WindowStep

HQ, HKV, D, V = 4, 2, 128, 300


class Server:
    """Streams with their blocks, on the host; tables and pools on the device."""

    def __init__(self, dtype, B, window, sinks, blocks, width, seed, rope=10000.0):
        self.g = torch.Generator().manual_seed(seed)
        if dtype == "fp8":
            pool = torch.full((blocks, HKV, 4224), 0x7F, dtype=torch.uint8, device="cuda")   # NaN codes and scales
            self.cache = bd.KVCache(pool)
        else:
            pools = [torch.full((blocks, HKV, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            self.cache = bd.KVCache(*pools)
        self.dtype, self.B, self.window, self.sinks = dtype, B, window, sinks
        self.W = (torch.randn(V, HQ * D, generator=self.g) * 0.05).to(torch.bfloat16).cuda()
        self.step = WindowStep(self.cache, self.W, HQ, B, 16 * width, window, sinks, rope_base=rope, prompt_rows=900)
        self.pool = bd.BlockPool(blocks)
        self.table = [[-1] * width for _ in range(B)]
        self.ctx = [0] * B

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16).cuda()

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def grow(self, b, n):
        """Blocks for n more tokens; one that others share is copied first."""
        src, dst = [], []
        last = self.ctx[b] // 16
        if self.ctx[b] % 16 and self.pool.owners(self.table[b][last]) > 1:
            src.append(self.table[b][last])
            dst += self.pool.alloc(1)
            self.pool.free(src)
            self.table[b][last] = dst[0]
        for i in range(-(-self.ctx[b] // 16), -(-(self.ctx[b] + n) // 16)):
            self.table[b][i] = self.pool.alloc(1)[0]
        if src:
            bd.tts_kv_copy_blocks(self.cache, self.i32(src), self.i32(dst))

    def give_back(self, b):
        for i in self.step.gone(self.ctx[b]):
            if self.table[b][i] >= 0:
                self.pool.free([self.table[b][i]])
                self.table[b][i] = -1

    def values(self):
        """Keys and values [blocks][HKV][16][D] as stored, in 64 bits."""
        if self.dtype != "fp8":
            return self.cache.k_pool.cpu().double(), self.cache.v_pool.cpu().double()
        rec = self.cache.k_pool.cpu()
        k = torch.empty(rec.shape[0], HKV, 16, D, dtype=torch.uint8)
        v = torch.empty_like(k)
        for s in range(16):
            for c in range(8):
                at = 128 * s + 16 * (c ^ (s % 8))
                k[:, :, s, 16 * c:16 * c + 16] = rec[:, :, at:at + 16]
            v[:, :, s] = rec[:, :, 2048 + 4 * (s % 8 // 2) + s % 2 + 2 * (s // 8):4096:16]
        ks, vs = (rec[:, :, at:at + 64].contiguous().view(torch.float32).double()[..., None] for at in (4096, 4160))
        return k.view(torch.float8_e4m3fn).double() * ks, v.view(torch.float8_e4m3fn).double() * vs

    def check(self, new, out, rows):
        """out [T][HQ][D] of the rows, the last new[b] tokens of each stream."""
        k, v = self.values()
        before = [c - n for c, n in zip(self.ctx, new)]
        s = dict(new=new, before=before, ctx=list(self.ctx), Hq=HQ, Hkv=HKV, D=D, dtype=self.dtype, window=self.window,
                 sinks=self.sinks, causal=True, scale=self.step.scale, table=torch.tensor(self.table), k_val=k, v_val=v,
                 T=sum(new), q=rows.cpu(), row_start=torch.tensor([sum(new[:b]) for b in range(self.B + 1)]))
        # (what no row sees may be anything: the reference's products would not be)
        for x in (k, v):
            x[~torch.isfinite(x)] = 0
        pr.check(out.view(-1, HQ, D), *pr.attend_all(s))
        assert int(self.step.err.item()) == 0

    def prompt(self, new):
        for b, n in enumerate(new):
            self.grow(b, n)
        before = self.i32(self.ctx)
        self.ctx = [c + n for c, n in zip(self.ctx, new)]
        T = sum(new)
        q, k, v = self.rand(T, HQ, D), self.rand(T, HKV, D), self.rand(T, HKV, D)
        start = self.i32([sum(new[:b]) for b in range(self.B + 1)])
        out = self.step.prompt(self.i32(self.table), before, self.i32(self.ctx), start, q, k, v)
        self.check(new, out, self.step.q)
        for b in range(self.B):
            self.give_back(b)

    def token(self):
        for b in range(self.B):
            self.grow(b, 1)
        before = self.i32(self.ctx)
        self.ctx = [c + 1 for c in self.ctx]
        q, k, v = self.rand(self.B, 1, HQ, D), self.rand(self.B, 1, HKV, D), self.rand(self.B, 1, HKV, D)
        ids = self.step(self.i32(self.table), before, self.i32(self.ctx), q, k, v)
        self.check([1] * self.B, self.step.out, self.step.q)
        logits = self.step.out.view(self.B, -1).double() @ self.W.double().t()
        top = logits.topk(2, 1)
        clear = top.values[:, 0] - top.values[:, 1] > 1e-2
        assert torch.equal(ids[clear].long(), top.indices[clear, 0])
        for b in range(self.B):
            self.give_back(b)

    def fork(self, parent, child):
        for b in child:
            self.pool.free([i for i in self.table[b] if i >= 0])
            self.table[b] = [-1] * len(self.table[b])
            self.ctx[b] = 0
        table, ctx = self.i32(self.table), self.i32(self.ctx)
        fresh = []
        for p, c in zip(parent, child):
            full = self.ctx[p] // 16
            shared = [i for i in self.table[p][:full] if i >= 0]
            self.pool.share(shared)
            fresh.append(self.pool.alloc(1)[0] if self.ctx[p] % 16 else -1)
            self.table[c][:full] = self.table[p][:full]
            if self.ctx[p] % 16:
                self.table[c][full] = fresh[-1]
            self.ctx[c] = self.ctx[p]
        self.step.fork(table, ctx, self.i32(parent), self.i32(child), self.i32(fresh))
        assert ctx.tolist() == self.ctx
        got = table.tolist()
        for c in child:
            n = -(-self.ctx[c] // 16)
            assert got[c][:n] == self.table[c][:n]

    def compact(self):
        table = self.i32(self.table)
        block_map = self.pool.compact()
        self.step.compact(self.i32(block_map), table)
        self.table = [[block_map[i] if i >= 0 else i for i in row] for row in self.table]
        assert table.tolist() == self.table
        used = {i for row in self.table for i in row if i >= 0}
        assert max(used) < len(used) == self.cache.num_blocks - self.pool.num_free


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window,sinks", [(100, 20), (64, 0), (0, 0)])
def test_a_server(dtype, window, sinks):
    s = Server(dtype, 4, window, sinks, 160 if not window else 90, 30, seed=window + 1)
    s.prompt([70, 33, 1, 160])
    for _ in range(3):
        s.token()
    s.prompt([5, 0, 200, 17])           # pieces join two of the streams and two others' prompts
    s.fork([0, 3], [1, 2])              # streams 1 and 2 begin anew as continuations
    s.compact()
    for _ in range(20):                 # past blocks' ends, each its own way
        s.token()
    s.compact()
    s.prompt([40, 3, 0, 60])
    s.token()
    for b in range(4):
        s.pool.free([i for i in s.table[b] if i >= 0])
    assert s.pool.num_free == s.cache.num_blocks
    if window:
        assert all(sum(i >= 0 for i in row) <= (window + 15) // 16 + -(-sinks // 16) + 2 for row in s.table)


def test_without_rotation_and_with_more_rows():
    """q_len 3, causal, no rotary embedding: q is read as it is."""
    g = torch.Generator().manual_seed(3)
    pools = [torch.zeros(20, HKV, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = bd.KVCache(*pools)
    W = (torch.randn(V, HQ * D, generator=g) * 0.05).to(torch.bfloat16).cuda()
    step = WindowStep(cache, W, HQ, 2, 160, 40, 3, q_len=3, causal=True, rope_base=0.0, prompt_rows=120)
    table = torch.randperm(20, generator=g).to(torch.int32).view(2, 10).cuda()

    def rand(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    ctx = [0, 0]
    for new in ([70, 21], [3, 3], [3, 3]):
        T = sum(new)
        q, k, v = rand(T, HQ, D), rand(T, HKV, D), rand(T, HKV, D)
        before = list(ctx)
        ctx = [c + n for c, n in zip(ctx, new)]
        if T > 6:
            out = step.prompt(table, i32(*before), i32(*ctx), i32(0, new[0], T), q, k, v)
        else:
            step(table, i32(*before), i32(*ctx), q.view(2, 3, HQ, D), k.view(2, 3, HKV, D), v.view(2, 3, HKV, D))
            out = step.out.view(T, HQ, D)
        s = dict(new=new, before=before, ctx=ctx, Hq=HQ, Hkv=HKV, D=D, dtype="bf16", window=40, sinks=3, causal=True,
                 scale=step.scale, table=table.cpu(), k_val=pools[0].cpu().double(), v_val=pools[1].cpu().double(), T=T,
                 q=q.cpu(), row_start=torch.tensor([0, new[0], T]))
        pr.check(out, *pr.attend_all(s))
    assert int(step.err.item()) == 0


def test_refused_shapes():
    pools = [torch.zeros(4, HKV, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = bd.KVCache(*pools)
    W = torch.zeros(V, HQ * D, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(window=-1), dict(sinks=-1), dict(q_len=9)):
        with pytest.raises(ValueError):
            WindowStep(cache, W, HQ, 2, 64, **bad)
    with pytest.raises(ValueError):
        WindowStep(cache, W[:, :-1].contiguous(), HQ, 2, 64)
    step = WindowStep(cache, W, HQ, 2, 64, 16, prompt_rows=4)
    z = torch.zeros(5, HQ, D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        step.prompt(t, t[:, 0].contiguous(), t[:, 0].contiguous(), t[0, :3].contiguous(), z, z[:, :HKV], z[:, :HKV])
    assert step.gone(10) == range(0, 0) and step.gone(31) == range(0, 1) and step.gone(47) == range(0, 2)
