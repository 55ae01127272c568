"""Page moves (tts_kv_copy_blocks, tts_kv_fork, tts_kv_compact, also for a
latent cache) and the packed append: bytes as they should be, everything else
as it was."""
from __future__ import annotations

import pytest
import torch

import paged_ref as pr

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_step_gb300 import _lib
    from decode_step_gb300 import binding as bd

KINDS = ["bf16", "fp8", "f32", "latent"]


def make_cache(kind, nb, Hkv=3, seed=0):
    """A cache of random bytes and its pools."""
    g = torch.Generator().manual_seed(seed)
    if kind == "latent":
        pool = torch.randint(0, 2 ** 15, (nb, 16, 128 + 64), generator=g).to(torch.int16).view(torch.bfloat16).cuda()
        return bd.LatentCache(pool, 128), [pool]
    if kind == "fp8":
        pool = torch.randint(0, 256, (nb, Hkv, 4224), generator=g).to(torch.uint8).cuda()
        return bd.KVCache(pool), [pool]
    if kind == "f32":
        pools = [torch.randn(nb, Hkv, 16, 64, generator=g).cuda() for _ in range(2)]
    else:
        pools = [torch.randn(nb, Hkv, 16, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    return bd.KVCache(*pools), pools


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.uint8 else t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nb,n,Hkv", [(2, 1, 1), (40, 17, 3), (700, 333, 8), (9, 0, 2)])
def test_copies(kind, nb, n, Hkv):
    cache, pools = make_cache(kind, nb, Hkv)
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(1))
    src, dst = perm[:n], perm[n:2 * n]
    want = [bits(p).clone() for p in pools]
    for w in want:
        w[dst.cuda()] = w[src.cuda()]
    err = i32([0])
    bd.tts_kv_copy_blocks(cache, i32(src.tolist()), i32(dst.tolist()), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


def test_one_block_to_many_and_bad_ids():
    cache, pools = make_cache("bf16", 12)
    want = [bits(p).clone() for p in pools]
    for w in want:
        w[[1, 2, 5]] = w[7].clone()
    err = i32([0])
    bd.tts_kv_copy_blocks(cache, i32([7, 7, 7, 12, 7, -1]), i32([1, 2, 5, 3, 99, 4]), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _lib.ERRBIT_BLOCK_ID
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 100, 8000])
def test_forks(kind, ctx):
    full, part = ctx // 16, ctx % 16 != 0
    need = full + part
    nb = need + 20
    cache, pools = make_cache(kind, nb)
    g = torch.Generator().manual_seed(2)
    perm = torch.randperm(nb, generator=g).tolist()
    B, width = 9, need + 2
    table = torch.full((B, width), -7, dtype=torch.int32)
    table[4, :need] = torch.tensor(perm[:need], dtype=torch.int32)
    table[2, :1] = perm[need + 10]
    lens = torch.tensor([3] * B, dtype=torch.int32)
    lens[4], lens[2] = ctx, 5
    parent, child, fresh = [4, 4, 2], [0, 8, 5], [perm[need], perm[need + 1], perm[need + 2]]
    want = [bits(p).clone() for p in pools]
    want_table, want_lens = table.clone(), lens.clone()
    for p, c, f in zip(parent, child, fresh):
        L = int(lens[p])
        want_lens[c] = L
        want_table[c, :L // 16] = table[p, :L // 16]
        if L % 16:
            want_table[c, L // 16] = f
            for w in want:
                w[f] = w[int(table[p, L // 16])]
    table, lens, err = table.cuda(), lens.cuda(), i32([0])
    bd.tts_kv_fork(cache, table, lens, i32(parent), i32(child), i32(fresh), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(table.cpu(), want_table) and torch.equal(lens.cpu(), want_lens)
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


@pytest.mark.parametrize("parent,child,fresh,lens,bit", [
    (3, 1, 5, 20, 16), (-1, 1, 5, 20, 16), (0, 3, 5, 20, 16), (0, -2, 5, 20, 16), (0, 0, 5, 20, 16),
    (0, 1, 5, 49, 2), (0, 1, 5, -1, 2), (0, 1, 8, 20, 1), (0, 1, -1, 20, 1), (0, 1, 5, 40, 1)])
def test_skipped_forks(parent, child, fresh, lens, bit):
    """Nothing is written; the good fork beside them is made."""
    cache, pools = make_cache("bf16", 8)
    table, ctx = i32([[0, 1, -1], [-1, -1, -1], [-1, -1, -1]]), i32([lens, 4, 4])
    err = i32([0])
    want = [bits(p).clone() for p in pools]
    before = table.clone(), ctx.clone()
    bd.tts_kv_fork(cache, table, ctx, i32([parent]), i32([child]), i32([fresh]), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bit
    assert torch.equal(table, before[0]) and torch.equal(ctx, before[1])
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nb,live", [(1, 1), (30, 7), (30, 29), (700, 400)])
def test_compaction_of_a_pool(kind, nb, live):
    cache, pools = make_cache(kind, nb)
    pool = bd.BlockPool(nb)
    ids = pool.alloc(nb)
    g = torch.Generator().manual_seed(nb + live)
    gone = [ids[i] for i in torch.randperm(nb, generator=g)[:nb - live].tolist()]
    pool.free(gone)
    held = [i for i in ids if i not in set(gone)]
    held = [held[i] for i in torch.randperm(live, generator=g).tolist()]
    width = live // 3 + 2
    table = torch.full((3, width), -1, dtype=torch.int32)
    for i, x in enumerate(held):
        table[i % 3, i // 3] = x
    contents = [[bits(p)[int(e)].clone() if e >= 0 else None for e in table.flatten()] for p in pools]
    old = table.clone()
    table = table.cuda()
    err = i32([0])
    block_map = pool.compact()
    bd.tts_kv_compact(cache, i32(block_map), table, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    new = table.cpu()
    assert torch.equal(new < 0, old < 0) and sorted(new[new >= 0].tolist()) == list(range(live))
    for p, c in zip(pools, contents):
        for e, want in zip(new.flatten().tolist(), c):
            assert e < 0 or torch.equal(bits(p)[e], want)
    assert pool.num_free == nb - live and all(pool.owners(i) == (i < live) for i in range(nb))


def test_bad_destinations_stay():
    cache, pools = make_cache("bf16", 8)
    want = [bits(p).clone() for p in pools]
    for w in want:
        w[1] = w[6].clone()
    err = i32([0])
    table = i32([[6, 5, 4, 3, -1, 8]])
    # 6 moves to 1; 5 to a block outside, 4 to one that moves itself
    bd.tts_kv_compact(cache, i32([0, 1, 2, 3, 6, 9, 1, 7]), table, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _lib.ERRBIT_BLOCK_ID
    assert table.cpu().tolist() == [[1, 5, 4, 3, -1, 8]]
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


def test_blocks_past_32_bit_offsets():
    """65,600 blocks of 32 KB of keys: the last ones lie past 2^31 bytes."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    nb = 65600
    pools = [torch.zeros(nb, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i, p in enumerate(pools):
        p[nb - 1] = 3.0 + i
    bd.tts_kv_copy_blocks(bd.KVCache(*pools), i32([nb - 1]), i32([nb - 2]))
    torch.cuda.synchronize()
    for i, p in enumerate(pools):
        assert bool((p[nb - 2] == 3.0 + i).all()) and not p[nb - 3].any()


# ------------------------------------------------------------- packed append

def append_case(kind, new, before, Hkv=2, Hq=4, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    D = pr.dim(kind)
    elem = torch.float32 if kind == "f32" else torch.bfloat16
    need = [-(-(n + p) // 16) for n, p in zip(new, before)]
    nb = sum(need) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(new), max([1] + need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    T = sum(new) + extra
    rows = [torch.randn(T, h, D, generator=g).to(elem) for h in (Hkv, Hkv, Hq)]
    start = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    return table, start, torch.tensor(before, dtype=torch.int32), rows, nb


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("rope", [0.0, 10000.0])
@pytest.mark.parametrize("new,before", [([1], [0]), ([17, 0, 1, 40], [0, 5, 31, 700]), ([3] * 70, list(range(70))),
                                        ([700], [65000])])
def test_packed_append_gives_what_each_stream_alone_gives(kind, rope, new, before):
    """Bit for bit the results of the unpacked append, a stream at a time."""
    if kind == "f32" and rope:
        pytest.skip("no rotary append of fp32 caches")
    table, start, pos, (k, v, q), nb = append_case(kind, new, before, extra=3)
    cache, pools = make_cache(kind, nb, 2)
    other, want = make_cache(kind, nb, 2)
    table, start, pos, k, v, q = (x.cuda() for x in (table, start, pos, k, v, q))
    q_out, q_in = torch.full_like(q, 5.0), q.clone()
    err = i32([0])
    if rope:
        bd.tts_kv_append_packed(cache, table, pos, start, k, v, q, q_out, rope_base=rope, err=err)
    else:
        bd.tts_kv_append_packed(cache, table, pos, start, k, v, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for b, n in enumerate(new):
        if not n:
            continue
        at = slice(int(start[b]), int(start[b]) + n)
        qb = q[at][None].clone()
        if rope:
            bd.tts_kv_append_rope(other, table[b:b + 1].contiguous(), pos[b:b + 1].contiguous(), qb, k[at][None].contiguous(), v[at][None].contiguous(),
                                  rope_base=rope)
            assert torch.equal(q_out[at], qb[0])
        else:
            bd.tts_kv_append(other, table[b:b + 1].contiguous(), pos[b:b + 1].contiguous(), k[at][None].contiguous(), v[at][None].contiguous())
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), bits(w))
    assert torch.equal(q, q_in)
    assert bool((q_out[sum(new):] == 5.0).all())
    if rope:
        # in place
        bd.tts_kv_append_packed(cache, table, pos, start, k, v, q, rope_base=rope)
        assert torch.equal(q[:sum(new)], q_out[:sum(new)]) and torch.equal(q[sum(new):], q_in[sum(new):])
        # the rotation itself (one rounding, and fp32 arithmetic)
        at = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
        where = torch.cat([torch.arange(p, p + n) for n, p in zip(new, before)])
        ref = pr.rotate(q_in[:sum(new)].cpu(), where[:, None], rope)
        assert len(at) == sum(new)
        assert ((q_out[:sum(new)].cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20).all()


def test_packed_append_skips_what_does_not_fit():
    table, start, pos, (k, v, q), nb = append_case("bf16", [20, 20, 20], [0, 0, 0])
    cache, pools = make_cache("bf16", nb, 2)
    before = [bits(p).clone() for p in pools]
    table[1, 1] = nb                    # tokens 16..19 of stream 1 have no block
    pos[2] = 30                         # past the table from token 2 on
    q_out = torch.full_like(q, 5.0).cuda()
    err = i32([0])
    bd.tts_kv_append_packed(cache, table.cuda(), pos.cuda(), start.cuda(), k.cuda(), v.cuda(), q.cuda(), q_out, 10000.0,
                            err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _lib.ERRBIT_BLOCK_ID | _lib.ERRBIT_CTX_LEN
    same = (q_out == 5.0).flatten(1).all(1).cpu()
    assert same.tolist() == [False] * 36 + [True] * 4 + [False] * 2 + [True] * 18
    # streams 0 and 1 wrote their first blocks, and the rest of the pool is as it was
    touched = {int(table[0, 0]), int(table[0, 1]), int(table[1, 0]), int(table[2, 1])}
    for p, w in zip(pools, before):
        assert all(torch.equal(bits(p)[i], w[i]) for i in range(nb) if i not in touched)


def test_page_refusals():
    cache, _ = make_cache("bf16", 4)
    table = i32([[0, 1]])
    with pytest.raises(ValueError):
        bd.tts_kv_copy_blocks(cache, i32([0]), i32([1, 2]))
    with pytest.raises(ValueError):
        bd.tts_kv_copy_blocks(cache, torch.tensor([0], dtype=torch.int64, device="cuda"), i32([1]))
    with pytest.raises(ValueError):
        bd.tts_kv_compact(cache, i32([0, 1, 2]), table)
    with pytest.raises(ValueError):
        bd.tts_kv_fork(cache, table, i32([3, 4]), i32([0]), i32([1]), i32([2]))
    with pytest.raises(ValueError):
        bd.tts_kv_copy_blocks(cache, torch.tensor([0], dtype=torch.int32), i32([1]))
