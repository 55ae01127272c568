"""Prompts, sliding windows and page moves over the paged KV cache, as cases to measure.

The cache is a pool of blocks of 16 tokens, [num_blocks][Hkv][16][D] for keys
and for values (or one FP8 record per block and KV head); a table gives each
stream's blocks.  Operators:

  append  the new tokens of prompts of different lengths, packed row after row,
          go to their slots; queries and keys are rotated at their positions.
  prompt  the packed rows of chunks of new tokens attend, causally, over what
          their streams have cached (their own tokens among it).
  decode  a few query rows a stream attend over the last `window` tokens and
          the first `sinks` ones.
  copy    blocks are copied to others (a stream that is about to write into a
          block that others share takes a copy first).
  fork    streams begin as continuations of others: they share the full blocks
          and get a copy of the last, partly filled one.
  compact the blocks in use move to the front of the pool, tables follow.

With a window, prompt rows too see only the `window` last tokens up to their
own, and the first `sinks`.  Blocks that no row sees any more have gone back to
the pool: their table entries are -1.

`run` computes them with elementary torch operations in 32 bits, or, with
`own` set, by the library's calls.  `exact` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16            # tokens a block
ROPE_BASE = 10000.0


# -------------------------------------------------------------------- cases

def _append(name, B, new, prefix=(0, 0), Hq=16, Hkv=8, rope=True, lens=1):
    return {"name": name, "op": "append", "dtype": "bf16", "B": B, "new_lo": new[0], "new_hi": new[1], "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "Hq": Hq, "Hkv": Hkv, "rope": rope, "lens": lens}


def _prompt(name, B, new, prefix=(0, 0), Hq=16, Hkv=8, dtype="bf16", window=0, sinks=0, lens=1):
    return {"name": name, "op": "prompt", "dtype": dtype, "B": B, "new_lo": new[0], "new_hi": new[1], "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "Hq": Hq, "Hkv": Hkv, "window": window, "sinks": sinks, "lens": lens}


def _decode(name, B, ctx, window, sinks, q_len=1, Hq=16, Hkv=8, dtype="bf16", causal=False, lens=1):
    return {"name": name, "op": "decode", "dtype": dtype, "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "q_len": q_len, "Hq": Hq,
            "Hkv": Hkv, "window": window, "sinks": sinks, "causal": causal, "lens": lens}


def _pages(name, op, blocks, moved, B, ctx, Hkv=8, dtype="bf16", lens=1):
    return {"name": name, "op": op, "dtype": dtype, "blocks": blocks, "moved": moved, "B": B, "ctx": ctx, "Hkv": Hkv, "lens": lens}


def listed():
    """The cases.  Heads, batches and context ranges are the decode step's own
    workloads (semantic, acoustic, sampled, speculative verify)."""
    return [
        # voice prompts and text of 12 new streams, written in one call
        _append("append-prompts-b12", 12, (37, 1500)),
        # the next piece of a text that a caller streams in: latency only
        _append("append-piece", 1, (17, 17), prefix=(700, 700)),
        # one new stream's text and voice prompt: time to the first token
        _prompt("prompt-one", 1, (333, 333)),
        # chunks of 8 streams that keep a bounded context in an FP8 cache
        _prompt("prompt-window-fp8-b8", 8, (61, 700), prefix=(0, 2000), dtype="fp8", window=1000, sinks=4),
        # a long script read in whole: 8,191 rows, after 700 cached tokens of the voice
        _prompt("prompt-script", 1, (8191, 8191), prefix=(700, 700)),
        # a short piece of text joins hours of dialogue: few rows, a long cache
        _prompt("prompt-piece-long", 1, (61, 61), prefix=(65472, 65472)),
        # a stream's first steps: all of a short, odd context inside the window
        _decode("decode-first-b1", 1, (17, 17), window=1024, sinks=4),
        # 64 streams of long dialogues that keep the last 1,500 tokens
        _decode("decode-dialogue-b64", 64, (1500, 60000), window=1500, sinks=4),
        # speculative verify over an FP8 cache: five causal rows a stream, more than a block of voice kept
        _decode("decode-verify-fp8-b64", 64, (256, 8000), window=1001, sinks=37, q_len=5, dtype="fp8", causal=True),
        # 48 streams about to write into a last block that they share with others
        _pages("copy-shared-b48", "copy", 200, 48, 48, 400),
        # 64 continuations of one voice prompt
        _pages("fork-voice-b64", "fork", 170, 64, 65, 1500),
        # a pool of 4,096 blocks, a third of them free, closes up
        _pages("compact-pool", "compact", 4096, 2700, 60, 700),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["append", "prompt", "prompt", "decode", "decode", "copy", "fork", "compact"])
    Hq, Hkv = rng.choice([(16, 8), (16, 8), (16, 4), (8, 8), (12, 4), (20, 4), (16, 2), (4, 1)])
    lens = rng.randrange(1, 1 << 20)
    if op == "append":
        B = _log_int(rng, 1, 32)
        c = _append("", B, (1, _log_int(rng, 1, 16000 // B)), (0, rng.choice([0, 55, 1000])), Hq, Hkv, rng.random() < 0.7, lens)
    elif op == "prompt":
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, min(8191, 9000 // B))
        prefix = rng.choice([0, 0, 300, 3000, 30000])
        while prefix and B * hi * (hi + prefix) > 32 << 20:
            prefix //= 2
        window = rng.choice([0, 0, _log_int(rng, 16, 5000)])
        c = _prompt("", B, (_log_int(rng, 1, hi), hi), (0, prefix), Hq, Hkv, rng.choice(["bf16", "bf16", "fp8"]), window,
                    rng.choice([0, 1, 4, 37]) if window else 0, lens)
    elif op == "decode":
        B = _log_int(rng, 1, 128)
        window = _log_int(rng, 1, 120000 // B if B > 32 else 4000)
        dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
        q_len = rng.choice([q for q in (1, 1, 2, 3, 5) if q * (Hq // Hkv) <= 16])
        lo = _log_int(rng, q_len, 4000)
        c = _decode("", B, (lo, _log_int(rng, lo, 60000)), window, rng.choice([0, 1, 4, 16, 37]), q_len, Hq, Hkv, dtype,
                    rng.random() < 0.5, lens)
    else:
        blocks = _log_int(rng, 40, 4096)
        ctx = _log_int(rng, 1, 1500)
        if op == "copy":
            c = _pages("", op, blocks, _log_int(rng, 1, blocks // 2), 1, 1, Hkv, rng.choice(["bf16", "f32"]), lens)
        elif op == "fork":
            n = _log_int(rng, 1, 128)
            c = _pages("", op, -(-ctx // BLOCK) + n + 7, n, n + 1, ctx, Hkv, rng.choice(["bf16", "f32"]), lens)
        else:
            live = _log_int(rng, blocks // 4, blocks)
            B = _log_int(rng, 1, min(64, live))
            c = _pages("", op, blocks, live, B, max(1, min(ctx, live // B * BLOCK)), Hkv, rng.choice(["bf16", "f32"]), lens)
    del c["name"]
    return c


def _dim(case):
    return 64 if case["dtype"] == "f32" else 128


def _lengths(case):
    """(new tokens, tokens cached before them) of each stream, from the case alone."""
    rng = random.Random(case["lens"])
    B = case["B"]
    if case["op"] == "decode":
        q = case["q_len"]
        return [q] * B, [max(rng.randint(case["ctx_lo"], case["ctx_hi"]), q) - q for _ in range(B)]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    return new, [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(B)]


def _seen(case, n, p):
    """The (low, high) ranges of tokens that some of a stream's n rows after p tokens see."""
    window, sinks, ctx = case.get("window", 0), case.get("sinks", 0), n + p
    first = ctx if case["op"] == "decode" and not case["causal"] else p + 1     # tokens up to the first row's own
    low = max(0, first - window) if window else 0
    if low <= sinks:
        return [(0, ctx)]
    return [(0, sinks), (low, ctx)] if sinks else [(low, ctx)]


def _pairs(case, n, p):
    """Pairs of a row and a token that it sees."""
    window, sinks = case.get("window", 0) or 1 << 30, case.get("sinks", 0)
    if case["op"] == "decode" and not case["causal"]:
        ctx = n + p
        return n * (min(ctx, window) + min(sinks, max(0, ctx - window)))
    return sum(min(t, window) + min(sinks, max(0, t - window)) for t in range(p + 1, p + n + 1))


def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once."""
    Hkv, D = case["Hkv"], _dim(case)
    elem = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("copy", "fork", "compact"):
        block = 2 * Hkv * BLOCK * D * elem
        if case["op"] == "copy":
            return {"bytes": case["moved"] * (2 * block + 8), "flops": 0}
        if case["op"] == "fork":
            n, full = case["moved"], case["ctx"] // BLOCK
            return {"bytes": n * (4 * full + 16 + (2 * block if case["ctx"] % BLOCK else 0)) + 4 * full, "flops": 0}
        old = _live(case)
        return {"bytes": 2 * block * sum(i >= len(old) for i in old) + 4 * case["blocks"] + 8 * case["B"] * -(-case["ctx"] // BLOCK),
                "flops": 0}
    new, before = _lengths(case)
    Hq, T = case["Hq"], sum(new)
    if case["op"] == "append":
        row = (2 * Hkv + (Hq if case["rope"] else 0)) * D * elem
        return {"bytes": 2 * T * row + 4 * (2 * case["B"] + 1), "flops": 3 * T * D * (Hq + Hkv) if case["rope"] else 0}
    token = 2 * Hkv * (D + 4) if case["dtype"] == "fp8" else 2 * Hkv * D * elem
    tokens = sum(hi - lo for n, p in zip(new, before) for lo, hi in _seen(case, n, p))
    return {"bytes": 2 * T * Hq * D * elem + token * tokens,
            "flops": 4 * Hq * D * sum(_pairs(case, n, p) for n, p in zip(new, before))}


# ------------------------------------------------------------------- inputs

def _swizzle(dev):
    """Place of chunk c (16 bytes) of slot s's key codes: c ^ (s % 8)."""
    s = torch.arange(BLOCK, device=dev)[:, None]
    return torch.arange(8, device=dev)[None] ^ (s % 8)


def _slot_order(dev):
    """Place of slot s among a dimension's 16 value codes."""
    s = torch.arange(BLOCK, device=dev)
    return 4 * (s % 8 // 2) + s % 2 + 2 * (s // 8)


def _records(k, v):
    """FP8 records [n][Hkv][4224] of key and value blocks [n][Hkv][16][128]."""
    out = torch.empty(*k.shape[:2], 4224, dtype=torch.uint8, device=k.device)
    codes = []
    for at, x in ((4096, k), (4160, v)):
        scale = x.float().abs().amax(-1) / 448
        codes.append((x.float() / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))
        out[..., at:at + 64] = scale.contiguous().view(torch.uint8)
    at = _swizzle(k.device)
    keys = out[..., :2048].view(*k.shape[:2], BLOCK, 8, 16)
    keys.scatter_(3, at[None, None, :, :, None].expand_as(keys), codes[0].view(*k.shape[:3], 8, 16))
    values = out[..., 2048:4096].view(*k.shape[:2], 128, BLOCK)
    values[..., _slot_order(k.device)] = codes[1].transpose(2, 3)
    return out


def _values(records, dtype):
    """Keys and values [n][Hkv][16][128] of FP8 records, as `dtype`."""
    n = records.shape[:2]
    at = _swizzle(records.device)
    keys = records[..., :2048].reshape(*n, BLOCK, 8, 16)
    keys = keys.gather(3, at[None, None, :, :, None].expand_as(keys)).reshape(*n, BLOCK, 128)
    values = records[..., 2048:4096].reshape(*n, 128, BLOCK)[..., _slot_order(records.device)].transpose(2, 3)
    scale = records[..., 4096:].contiguous().view(torch.float32).view(*n, 2, BLOCK, 1).to(dtype)
    return (keys.contiguous().view(torch.float8_e4m3fn).to(dtype) * scale[:, :, 0],
            values.contiguous().view(torch.float8_e4m3fn).to(dtype) * scale[:, :, 1])


def _live(case):
    """Blocks in use before a compaction, in the order of the streams that hold them."""
    rng = random.Random(case["lens"])
    return rng.sample(range(case["blocks"]), case["moved"])


def _inputs(case, seed):
    """Tensors of one case, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    B, Hkv, D = case["B"], case["Hkv"], _dim(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    s = {"case": case}
    if case["op"] in ("copy", "fork", "compact"):
        nb, n, ctx = case["blocks"], case["moved"], case["ctx"]
        s["k_pool"], s["v_pool"] = normal(nb, Hkv, BLOCK, D), normal(nb, Hkv, BLOCK, D)
        need = -(-ctx // BLOCK)
        if case["op"] == "copy":
            perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
            s["src"], s["dst"] = perm[:n].clone(), perm[n:2 * n].clone()
        elif case["op"] == "fork":
            perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
            s["table"] = torch.full((B, need + 3), -1, dtype=torch.int32, device=dev)
            s["table"][0, :need] = perm[:need]
            s["ctx"] = ints([ctx] + [0] * (B - 1))
            s["parent"], s["child"] = ints([0] * n), ints(range(1, n + 1))
            s["new_block"] = perm[need:need + n].clone()
        else:
            old = _live(case)
            s["table"] = torch.full((B, need + 3), -1, dtype=torch.int32, device=dev)
            s["table"][:, :need] = ints(old[:B * need]).view(B, need)
            # blocks behind the first len(old) go to the free ones before them, in order
            to = list(range(nb))
            free = sorted(set(range(len(old))) - set(old))
            for i, j in zip(sorted(i for i in old if i >= len(old)), free):
                to[i] = j
            s["map"] = ints(to)
        return s
    new, before = _lengths(case)
    T, Hq = sum(new), case["Hq"]
    ctx = [n + p for n, p in zip(new, before)]
    blocks = [sorted({t for lo, hi in _seen(case, n, p) for t in range(lo // BLOCK, -(-hi // BLOCK))})
              for n, p in zip(new, before)]
    num_blocks = sum(map(len, blocks)) + 7
    # blocks of the pool in random order; entries of blocks without a visible token are -1
    perm = torch.randperm(num_blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(-(-c // BLOCK) for c in ctx)), -1, dtype=torch.int32, device=dev)
    table[ints([b for b, x in enumerate(blocks) for _ in x]).long(), ints([i for x in blocks for i in x]).long()] = \
        perm[:num_blocks - 7]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    # slots without a token hold what an earlier stream left
    k, v = normal(num_blocks, Hkv, BLOCK, D), normal(num_blocks, Hkv, BLOCK, D)
    if case["dtype"] == "fp8":
        k, v = _records(k, v), None
    s.update(new=new, before_list=before, table=table, before=ints(before), ctx=ints(ctx), row_start=ints(start),
             max_ctx=max(ctx), T=T, k_pool=k, v_pool=v, q=normal(T, Hq, D))
    if case["op"] == "append":
        s["k_new"], s["v_new"] = normal(T, Hkv, D), normal(T, Hkv, D)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = D ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from decode_step_gb300 import binding as bd
        s["cache"] = bd.KVCache(s["k_pool"], s["v_pool"])
        if case["op"] == "prompt":
            n = bd.tts_prompt_attn_workspace_size(case["B"], s["T"], case["Hq"], case["Hkv"], _dim(case))
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        elif case["op"] == "decode":
            n = bd.tts_decode_attn_workspace_size(case["B"], case["q_len"], case["Hq"], case["Hkv"], _dim(case), s["max_ctx"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------- run

def run(s):
    """One pass through the case's operator."""
    return (_run_own if own else _run_plain)(s)


def _outputs(s):
    op = s["case"]["op"]
    if op in ("prompt", "decode"):
        return s["out"]
    pools = s["k_pool"], s["v_pool"]
    return pools + {"append": (s["out"],) if s["case"].get("rope") else (), "copy": (), "fork": (s.get("table"), s.get("ctx")),
                    "compact": (s.get("table"),)}[op]


def _run_own(s):
    from decode_step_gb300 import binding as bd
    c = s["case"]
    if c["op"] == "append":
        if c["rope"]:
            bd.tts_kv_append_packed(s["cache"], s["table"], s["before"], s["row_start"], s["k_new"], s["v_new"], s["q"],
                                    s["out"], rope_base=ROPE_BASE)
        else:
            bd.tts_kv_append_packed(s["cache"], s["table"], s["before"], s["row_start"], s["k_new"], s["v_new"])
    elif c["op"] == "prompt":
        bd.tts_prompt_attn(s["cache"], s["table"], s["ctx"], s["row_start"], s["q"], s["out"], s["ws"], s["scale"],
                           window=c["window"], sinks=c["sinks"])
    elif c["op"] == "decode":
        shape = (c["B"], c["q_len"]) + s["q"].shape[1:]
        bd.tts_window_decode_attn(s["cache"], s["table"], s["ctx"], s["max_ctx"], s["q"].view(shape), s["out"].view(shape),
                                  s["ws"], s["scale"], window=c["window"], sinks=c["sinks"], causal=c["causal"])
    elif c["op"] == "copy":
        bd.tts_kv_copy_blocks(s["cache"], s["src"], s["dst"])
    elif c["op"] == "fork":
        bd.tts_kv_fork(s["cache"], s["table"], s["ctx"], s["parent"], s["child"], s["new_block"])
    else:
        bd.tts_kv_compact(s["cache"], s["map"], s["table"])
    return _outputs(s)


def _rotate(x, angle):
    """Rotate-half of x [..., D] by `angle` (64-bit, D / 2 values a row)."""
    half = x.shape[-1] // 2
    cos, sin = angle.cos().float(), angle.sin().float()
    x1, x2 = x[..., :half].float(), x[..., half:].float()
    return torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "append":
        rows = torch.arange(s["T"], device="cuda")
        stream = (rows[:, None] >= s["row_start"][None, 1:]).sum(1)
        pos = s["before"][stream] + rows - s["row_start"][stream]
        k = s["k_new"]
        if c["rope"]:
            D = k.shape[-1]
            angle = pos.double()[:, None] * ROPE_BASE ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
            k = _rotate(k, angle[:, None]).to(k.dtype)
            s["out"].copy_(_rotate(s["q"], angle[:, None]))
        block = s["table"][stream, pos // BLOCK].long()
        s["k_pool"][block, :, pos % BLOCK] = k
        s["v_pool"][block, :, pos % BLOCK] = s["v_new"]
    elif c["op"] == "copy":
        for pool in (s["k_pool"], s["v_pool"]):
            pool[s["dst"].long()] = pool[s["src"].long()]
    elif c["op"] == "fork":
        full, child, parent = c["ctx"] // BLOCK, s["child"].long(), s["parent"].long()
        s["table"][child, :full] = s["table"][parent, :full]
        if c["ctx"] % BLOCK:
            for pool in (s["k_pool"], s["v_pool"]):
                pool[s["new_block"].long()] = pool[s["table"][parent, full].long()]
            s["table"][child, full] = s["new_block"]
        s["ctx"][child] = s["ctx"][parent]
    elif c["op"] == "compact":
        to = s["map"].long()
        moved = (to != torch.arange(c["blocks"], device="cuda")).nonzero()[:, 0]
        for pool in (s["k_pool"], s["v_pool"]):
            pool[to[moved]] = pool[moved]
        s["table"].copy_(torch.where(s["table"] >= 0, s["map"][s["table"].clamp(min=0).long()], s["table"]))
    elif c["op"] == "decode":
        _plain_decode(s)
    else:
        _plain_prompt(s)
    return _outputs(s)


def _cached(s, block, slot):
    """Keys and values [..., Hkv, D] of tokens, in 32 bits."""
    if s["case"]["dtype"] == "fp8":
        k, v = _values(s["k_pool"], torch.float32)
    else:
        k, v = s["k_pool"], s["v_pool"]
    return k[block, :, slot].float(), v[block, :, slot].float()


def _plain_decode(s):
    c = s["case"]
    B, q, Hq, Hkv, D, window, sinks = c["B"], c["q_len"], c["Hq"], c["Hkv"], _dim(c), c["window"], c["sinks"]
    rows = torch.arange(q, device="cuda")
    limit = s["ctx"].long().view(B, 1) - ((q - 1 - rows) if c["causal"] else 0 * rows)       # [B][q]
    # the first tokens, and the span of the windows
    low = (limit[:, 0] - window).clamp(min=sinks)
    span = min(window + q - 1, s["max_ctx"])
    pos = torch.cat((torch.arange(sinks, device="cuda").expand(B, -1), low[:, None] + torch.arange(span, device="cuda")), 1)
    at = torch.minimum(pos, s["ctx"].long()[:, None] - 1)
    block = s["table"].gather(1, at // BLOCK).long().clamp(min=0)
    k, v = _cached(s, block, at % BLOCK)                                                       # [B][tokens][Hkv][D]
    p = pos[:, None]
    seen = (p < limit[..., None]) & ((p < sinks) | (p >= limit[..., None] - window))           # [B][q][tokens]
    qh = s["q"].float().view(B, q, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(qh, k.permute(0, 2, 3, 1)) * s["scale"]                               # [B][Hkv][q group][tokens]
    score = score.view(B, Hkv, q, Hq // Hkv, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = (w / w.sum(-1, keepdim=True)).view(B, Hkv, q * Hq // Hkv, -1)
    o = torch.matmul(w, v.permute(0, 2, 1, 3)).view(B, Hkv, q, Hq // Hkv, D).permute(0, 2, 1, 3, 4)
    s["out"].view(B, q, Hkv, Hq // Hkv, D).copy_(o)


def _plain_prompt(s):
    """A stream at a time, up to 2,048 rows of one KV head at a time."""
    c = s["case"]
    Hkv, group, D, window, sinks = c["Hkv"], c["Hq"] // c["Hkv"], _dim(c), c["window"], c["sinks"]
    q, out = s["q"].view(-1, Hkv, group, D), s["out"].view(-1, Hkv, group, D)
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
        pos = torch.cat([torch.arange(lo, hi, device="cuda") for lo, hi in _seen(c, n, p)])
        k, v = _cached(s, s["table"][b, pos // BLOCK].long(), pos % BLOCK)
        for r in range(0, n, 2048):
            m = min(2048, n - r)
            own_pos = torch.arange(p + r, p + r + m, device="cuda")[:, None]
            hidden = pos > own_pos
            if window:
                hidden |= (pos <= own_pos - window) & (pos >= sinks)
            hidden = hidden[:, None].expand(-1, group, -1).reshape(m * group, -1)
            for h in range(Hkv):
                x = q[at + r:at + r + m, h].reshape(m * group, D).float()
                score = (torch.matmul(x, k[:, h].t()) * s["scale"]).masked_fill_(hidden, -math.inf)
                w = torch.exp(score - score.amax(-1, keepdim=True))
                o = torch.matmul(w, v[:, h]) / w.sum(-1, keepdim=True)
                out[at + r:at + r + m, h] = o.view(m, group, D).to(out.dtype)
        at += n


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of `run` in 64 bits, from the definitions: a stream, a head
    or a block at a time."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "copy":
        pools = s["k_pool"].double(), s["v_pool"].double()
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            for pool in pools:
                pool[j] = pool[i]
        return pools
    if op == "fork":
        pools, table, ctx = (s["k_pool"].double(), s["v_pool"].double()), s["table"].tolist(), s["ctx"].tolist()
        for p, c, fresh in zip(s["parent"].tolist(), s["child"].tolist(), s["new_block"].tolist()):
            ctx[c] = ctx[p]
            shared = ctx[p] // BLOCK
            table[c][:shared] = table[p][:shared]
            if ctx[p] > shared * BLOCK:
                table[c][shared] = fresh
                for pool in pools:
                    pool[fresh] = pool[table[p][shared]]
        return pools + (torch.tensor(table, dtype=torch.int32, device="cuda"), torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    if op == "compact":
        pools, to = (s["k_pool"].double(), s["v_pool"].double()), s["map"].tolist()
        for i, j in enumerate(to):
            if i != j:
                for pool in pools:
                    pool[j] = pool[i]
        table = [[to[i] if i >= 0 else i for i in row] for row in s["table"].tolist()]
        return pools + (torch.tensor(table, dtype=torch.int32, device="cuda"),)
    if op == "append":
        pools, D = (s["k_pool"].double(), s["v_pool"].double()), _dim(case)
        out = s["q"].double()
        turn = torch.tensor([ROPE_BASE ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
            pos = torch.arange(p, p + n, device="cuda")
            k, q = s["k_new"][at:at + n].double(), out[at:at + n]
            if case["rope"]:
                unit = torch.polar(torch.ones(n, D // 2, dtype=torch.float64, device="cuda"), pos.double()[:, None] * turn)
                turned = [torch.complex(x[..., :D // 2], x[..., D // 2:]) * unit[:, None] for x in (k, q)]
                k, q = (torch.cat((x.real, x.imag), 2) for x in turned)
            out[at:at + n] = q
            for pool, x in zip(pools, (k, s["v_new"][at:at + n].double())):
                for h in range(case["Hkv"]):
                    pool[s["table"][b].long()[pos // BLOCK], h, pos % BLOCK] = x[:, h]
            at += n
        return pools + ((out,) if case["rope"] else ())
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    group, window, sinks = case["Hq"] // case["Hkv"], case["window"] or 1 << 40, case["sinks"]
    causal = op == "prompt" or case["causal"]
    pools = _values(s["k_pool"], torch.float64) if case["dtype"] == "fp8" else (s["k_pool"], s["v_pool"])
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
        last = torch.arange(p, p + n, device="cuda") if causal else torch.full((n,), n + p - 1, device="cuda")
        t = torch.arange(n + p, device="cuda")
        t = t[(t < sinks) | (t > int(last[0]) - window)]
        bias = torch.zeros(n, len(t), dtype=torch.float64, device="cuda")
        back = last[:, None] - t
        bias[(back < 0) | ((back >= window) & (t >= sinks))] = -math.inf
        blocks = s["table"][b].long()[t // BLOCK]
        for g in range(case["Hkv"]):
            key, val = (pool[blocks, g, t % BLOCK].double() for pool in pools)
            for h in range(g * group, (g + 1) * group):
                a = s["q"][at:at + n, h].double() @ key.t()
                out[at:at + n, h] = torch.softmax(a.mul_(s["scale"]).add_(bias), 1) @ val
        at += n
    return out
