"""The operators of the latent KV cache, as cases to measure.

A latent cache keeps one row a token, shared by every head: a latent vector c
(latent_dim values) and one rotated key part kr (64 values).  With per-head
weights w_uk [Hq][nope_dim][latent_dim] and w_uv [Hq][v_dim][latent_dim], head
h's key for a token is (w_uk[h] c, kr) and its value w_uv[h] c.  Operators:

  append   this step's latents and rotated key parts go to their slots of the
           paged pool; the queries' rotary parts are rotated at the same
           positions.
  decode   a few query rows a stream attend over the paged latents directly
           (the absorbed form: the queries are multiplied by w_uk first, the
           attended latent by w_uv last).
  prefill  the rows of whole prompts, packed ragged, attend over their
           streams' tokens (the expanded form: keys and values per head).

`run` computes them with elementary torch operations in 32 bits, or, with
`own` set, by the library's calls.  `exact` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16        # tokens a block of the paged pool
ROPE_DIM = 64     # rotated values of a query or key
ROPE_BASE = 10000.0


# -------------------------------------------------------------------- cases

def _append(name, B, new, prefix, Hq=16, latent=512, ragged=False, lens=1):
    return {"name": name, "op": "append", "B": B, "new_lo": new[0], "new_hi": new[1], "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "Hq": Hq, "latent": latent, "ragged": ragged, "lens": lens}


def _decode(name, B, ctx, q_len=1, Hq=16, latent=512, nope=128, v=128, causal=False, log=False, lens=1):
    return {"name": name, "op": "decode", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "q_len": q_len, "Hq": Hq,
            "latent": latent, "nope": nope, "v": v, "causal": causal, "log": log, "lens": lens}


def _prefill(name, B, new, prefix=(0, 0), Hq=16, latent=512, nope=128, v=128, lens=1):
    return {"name": name, "op": "prefill", "B": B, "new_lo": new[0], "new_hi": new[1], "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "Hq": Hq, "latent": latent, "nope": nope, "v": v, "lens": lens}


def listed():
    """The cases.  Batches, heads and context ranges are the decode step's own
    workloads (semantic, acoustic, sampled, speculative verify)."""
    return [
        # one token of each of 64 acoustic streams joins the cache
        _append("append-step-b64", 64, (1, 1), (49, 1499)),
        # a speculative step's five tokens a stream
        _append("append-verify-b64", 64, (5, 5), (251, 2043)),
        # voice prompts and text of 12 new streams, written in one call
        _append("append-prompts-b12", 12, (37, 1500), (0, 0), ragged=True),
        # a stream's first steps: one short, odd context, latency only
        _decode("decode-first-b1", 1, (17, 17)),
        # semantic stage: 16 streams of text, prompt and 12.5 Hz frames
        _decode("decode-semantic-b16", 16, (200, 600)),
        # acoustic stage: 64 ragged streams
        _decode("decode-acoustic-b64", 64, (50, 1500)),
        # the largest step batch, contexts of 32 to 4096 tokens
        _decode("decode-sampled-b256", 256, (32, 4096), log=True),
        # speculative verify: five causal rows a stream, 80 rows with its heads
        _decode("decode-verify-b64", 64, (256, 2048), q_len=5, causal=True),
        # one stream that keeps hours of dialogue: the work is split over the context
        _decode("decode-long-b1", 1, (65533, 65533)),
        # one new stream's text and voice prompt: time to the first token
        _prefill("prefill-one", 1, (333, 333)),
        # a burst of 16 new streams of different lengths, smaller heads and latents
        _prefill("prefill-burst-b16", 16, (61, 700), Hq=8, latent=256, nope=64, v=64),
        # a long script read in whole: 8,191 rows, after 700 cached tokens of the voice
        _prefill("prefill-script", 1, (8191, 8191), prefix=(700, 700)),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["append", "decode", "decode", "prefill"])
    Hq = rng.choice([2, 4, 8, 12, 16, 16, 20, 32])
    latent = rng.choice([128, 256, 384, 512, 512])
    nope, v = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    lens = rng.randrange(1, 1 << 20)
    if op == "append":
        if rng.random() < 0.5:
            n = _log_int(rng, 1, 8)
            c = _append("", _log_int(rng, 1, 256), (n, n), (0, _log_int(rng, 16, 4000)), Hq, latent, False, lens)
        else:
            B = _log_int(rng, 1, 32)
            c = _append("", B, (1, _log_int(rng, 2, 16000 // B)), (0, rng.choice([0, 100, 1000])), Hq, latent, True, lens)
    elif op == "decode":
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, min(65536, 400000 // B))
        q_len = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        while q_len > 1 and B * hi * q_len * Hq > 64 * 2048 * 80:
            q_len -= 1
        lo = max(q_len, _log_int(rng, 1, hi))
        c = _decode("", B, (lo, max(lo, hi)), q_len, Hq, latent, nope, v, rng.random() < 0.5, rng.random() < 0.3, lens)
    else:
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 16, min(8191, 12000 // B))
        prefix = rng.choice([0, 0, 55, 500])
        c = _prefill("", B, (_log_int(rng, 1, hi), hi), (0, prefix), min(Hq, 16), latent, nope, v, lens)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens cached before them) of each stream, from the case alone."""
    rng = random.Random(case["lens"])
    B = case["B"]
    if case["op"] == "decode":
        q = case["q_len"]
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        ctx = [_log_int(rng, lo, hi) if case["log"] else rng.randint(lo, hi) for _ in range(B)]
        return [q] * B, [max(c, q) - q for c in ctx]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    return new, [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(B)]


def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once; the products of the form the operator takes."""
    new, before = _lengths(case)
    L, Hq, T = case["latent"], case["Hq"], sum(new)
    row = 2 * (L + ROPE_DIM)
    if case["op"] == "append":
        return {"bytes": T * (2 * row + 4 * Hq * ROPE_DIM) + 8 * case["B"], "flops": 3 * T * ROPE_DIM * (Hq + 1)}
    nope, v = case["nope"], case["v"]
    ctx = [n + p for n, p in zip(new, before)]
    io = 2 * T * Hq * (nope + ROPE_DIM + v) + 2 * Hq * L * (nope + v) + row * sum(ctx)
    if case["op"] == "decode":
        pairs = sum(n * c for n, c in zip(new, ctx))
        return {"bytes": io, "flops": 2 * Hq * (pairs * (2 * L + ROPE_DIM) + T * L * (nope + v))}
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, before))
    return {"bytes": io, "flops": 2 * Hq * (pairs * (nope + ROPE_DIM + v) + sum(ctx) * L * (nope + v))}


# ------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Tensors of one case, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, before = _lengths(case)
    B, T, L, Hq = case["B"], sum(new), case["latent"], case["Hq"]
    ctx = [n + p for n, p in zip(new, before)]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    need = [-(-c // BLOCK) for c in ctx]
    num_blocks = sum(need) + 7
    # blocks of the pool in random order; entries past a stream's blocks are -1
    perm = torch.randperm(num_blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"case": case, "new": new, "before_list": before, "table": table, "before": ints(before), "ctx": ints(ctx),
         "row_start": ints(start), "max_ctx": max(ctx), "T": T,
         # latents come normalised: entries of size one; slots without a token hold what an earlier stream left
         "pool": normal(num_blocks, BLOCK, L + ROPE_DIM)}
    if case["op"] == "append":
        s["c_new"], s["kr_new"] = normal(T, L), normal(T, ROPE_DIM)
        s["q_rope"] = normal(T, Hq, ROPE_DIM)
        s["q_out"] = torch.empty_like(s["q_rope"])
        return s
    nope, v = case["nope"], case["v"]
    s["q_nope"], s["q_rope"] = normal(T, Hq, nope), normal(T, Hq, ROPE_DIM)
    s["w_uk"] = normal(Hq, nope, L, std=L ** -0.5)
    s["w_uv"] = normal(Hq, v, L, std=L ** -0.5)
    s["out"] = torch.empty(T, Hq, v, dtype=torch.bfloat16, device=dev)
    s["scale"] = (nope + ROPE_DIM) ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from decode_step_gb300 import binding as bd
        B, Hq, L = case["B"], case["Hq"], case["latent"]
        s["cache"] = bd.LatentCache(s["pool"], L)
        if case["op"] == "decode":
            n = bd.tts_latent_decode_attn_workspace_size(B, case["q_len"], Hq, L, case["nope"], case["v"], s["max_ctx"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        elif case["op"] == "prefill":
            s["total_ctx"] = sum(s["new"]) + sum(s["before_list"])
            n = bd.tts_latent_prefill_attn_workspace_size(B, s["T"], Hq, L, case["nope"], case["v"], s["total_ctx"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------- run

def run(s):
    """One pass through the case's operator."""
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from decode_step_gb300 import binding as bd
    c = s["case"]
    B, Hq = c["B"], c["Hq"]
    if c["op"] == "append":
        bd.tts_latent_append(s["cache"], s["table"], s["before"], s["c_new"], s["kr_new"], s["q_rope"], s["q_out"],
                             ROPE_BASE, row_start=s["row_start"] if c["ragged"] else None)
        return s["pool"], s["q_out"]
    if c["op"] == "decode":
        q = c["q_len"]
        bd.tts_latent_decode_attn(s["cache"], s["table"], s["ctx"], s["max_ctx"], s["q_nope"].view(B, q, Hq, -1),
                                  s["q_rope"].view(B, q, Hq, -1), s["w_uk"], s["w_uv"], s["out"].view(B, q, Hq, -1),
                                  s["ws"], s["scale"], causal=c["causal"])
        return s["out"]
    bd.tts_latent_prefill_attn(s["cache"], s["table"], s["ctx"], s["total_ctx"], s["row_start"], s["q_nope"],
                               s["q_rope"], s["w_uk"], s["w_uv"], s["out"], s["ws"], s["scale"])
    return s["out"]


def _rotate(x, angle):
    """Rotate-half of the last 64 values by `angle` (64-bit, 32 values a row)."""
    cos, sin = angle.cos().float(), angle.sin().float()
    x1, x2 = x[..., :ROPE_DIM // 2].float(), x[..., ROPE_DIM // 2:].float()
    return torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "append":
        rows = torch.arange(s["T"], device="cuda")
        stream = (rows[:, None] >= s["row_start"][None, 1:]).sum(1)
        pos = s["before"][stream] + rows - s["row_start"][stream]
        theta = ROPE_BASE ** (-torch.arange(ROPE_DIM // 2, dtype=torch.float64, device="cuda") * 2 / ROPE_DIM)
        angle = pos.double()[:, None] * theta
        kr = _rotate(s["kr_new"], angle).to(torch.bfloat16)
        s["pool"][s["table"][stream, pos // BLOCK].long(), pos % BLOCK] = torch.cat((s["c_new"], kr), -1)
        s["q_out"].copy_(_rotate(s["q_rope"], angle[:, None]))
        return s["pool"], s["q_out"]
    if c["op"] == "decode":
        # absorbed: scores and sums over the latents themselves
        B, q, Hq, L = c["B"], c["q_len"], c["Hq"], c["latent"]
        kv = s["pool"][s["table"].clamp(min=0).long()].reshape(B, -1, L + ROPE_DIM)[:, :s["max_ctx"]].float()
        q_lat = torch.matmul(s["q_nope"].float().transpose(0, 1), s["w_uk"].float()).transpose(0, 1)
        qk = torch.cat((q_lat, s["q_rope"].float()), -1).reshape(B, q * Hq, L + ROPE_DIM)
        score = torch.matmul(qk, kv.transpose(1, 2)).view(B, q, Hq, -1) * s["scale"]
        limit = s["ctx"].view(B, 1, 1, 1)
        if c["causal"]:
            limit = limit - q + 1 + torch.arange(q, device="cuda").view(1, q, 1, 1)
        seen = torch.arange(s["max_ctx"], device="cuda") < limit
        score = score.masked_fill(~seen, -math.inf)
        p = torch.exp(score - score.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        lat = torch.matmul(p.view(B, q * Hq, -1), kv[..., :L]).view(B * q, Hq, L)
        o = torch.matmul(lat.transpose(0, 1), s["w_uv"].float().transpose(1, 2)).transpose(0, 1)
        s["out"].copy_(o)
        return s["out"]
    # prefill, expanded: a stream at a time, four heads at a time
    Hq, L, v = c["Hq"], c["latent"], c["v"]
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
        ctx = n + p
        kv = s["pool"][s["table"][b, :-(-ctx // BLOCK)].long()].reshape(-1, L + ROPE_DIM)[:ctx].float()
        rows = slice(at, at + n)
        hidden = torch.arange(ctx, device="cuda") > torch.arange(p, ctx, device="cuda")[:, None]
        for h in range(0, Hq, 4):
            hs = slice(h, min(h + 4, Hq))
            key = torch.matmul(kv[:, :L], s["w_uk"][hs].float().transpose(1, 2))
            val = torch.matmul(kv[:, :L], s["w_uv"][hs].float().transpose(1, 2))
            score = torch.matmul(s["q_nope"][rows, hs].float().transpose(0, 1), key.transpose(1, 2))
            score += torch.matmul(s["q_rope"][rows, hs].float().transpose(0, 1), kv[:, L:].t())
            score = (score * s["scale"]).masked_fill_(hidden, -math.inf)
            w = torch.exp(score - score.amax(-1, keepdim=True))
            o = torch.matmul(w, val) / w.sum(-1, keepdim=True)
            s["out"][rows, hs] = o.transpose(0, 1).to(torch.bfloat16)
        at += n
    return s["out"]


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of `run` in 64 bits, from the definition: one stream and one
    head at a time, keys and values multiplied out."""
    s = _inputs(case, seed)
    L, Hq = case["latent"], case["Hq"]
    half = ROPE_DIM // 2
    if case["op"] == "append":
        pool, q_out = s["pool"].double(), torch.empty_like(s["q_rope"], dtype=torch.float64)
        turn = torch.tensor([ROPE_BASE ** (-2.0 * i / ROPE_DIM) for i in range(half)], dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
            pos = torch.arange(p, p + n, device="cuda")
            unit = torch.polar(torch.ones(n, half, dtype=torch.float64, device="cuda"), pos.double()[:, None] * turn)
            k, q = s["kr_new"][at:at + n].double(), s["q_rope"][at:at + n].double()
            k, q = torch.complex(k[:, :half], k[:, half:]) * unit, torch.complex(q[..., :half], q[..., half:]) * unit[:, None]
            slots = s["table"][b].long()[pos // BLOCK], pos % BLOCK
            pool[slots] = torch.cat((s["c_new"][at:at + n].double(), k.real, k.imag), 1)
            q_out[at:at + n] = torch.cat((q.real, q.imag), 2)
            at += n
        return pool, q_out
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    causal = case.get("causal", True)
    w_uk, w_uv = s["w_uk"].double(), s["w_uv"].double()
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["before_list"])):
        blocks = s["table"][b, :-(-(n + p) // BLOCK)].long()
        kv = s["pool"][blocks].flatten(0, 1)[:n + p].double()
        c, kr = kv[:, :L], kv[:, L:]
        key, val = torch.einsum("tl,hdl->htd", c, w_uk), torch.einsum("tl,hdl->htd", c, w_uv)
        for h in range(Hq):
            a = s["q_nope"][at:at + n, h].double() @ key[h].t() + s["q_rope"][at:at + n, h].double() @ kr.t()
            a *= s["scale"]
            if causal:
                a += torch.full_like(a, -math.inf).triu_(p + 1)
            out[at:at + n, h] = torch.softmax(a, 1) @ val[h]
        at += n
    return out
