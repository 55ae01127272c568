"""Inputs, the 64-bit reference and derived tolerances of the tests of packed
prompts, sliding windows and page moves over the paged KV cache.

Tolerances.  The kernels round the softmax weights (times the value's scale in
an FP8 cache) to the matrix product's type before they meet the values, and the
output.  A rounding is off by at most u of the value (bf16 2^-8, f16 2^-11),
taken as independent with variance at most u^2 / 3 of the value's square.  An
element passes when it is within
  u_out |out| + 8 sqrt(sum_t (w_t v_t)^2 u_p^2 / 3) + 2^-16 (|out| + sum_t w_t |v_t|)
of the reference: the output's own rounding, eight standard deviations of the
weights' (a single term's full half step is 1.7), and fp32 arithmetic (sums of a
few thousand terms, hardware exponentials, scores of size up to some tens).  u_p
is 2^-8 for bf16 caches, 2^-11 for FP8 ones (whose codes are exact in f16) and
0 for fp32 ones, whose output is off by 2^-24.
"""
from __future__ import annotations

import math

import torch

U_OUT = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -8, "f32": 2.0 ** -24}
U_P = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -11, "f32": 0.0}


def dim(dtype):
    return 64 if dtype == "f32" else 128


def quantise(x):
    """(codes as uint8, fp32 scales) of rows x [..., 128]: one block a row."""
    scale = x.float().abs().amax(-1) / 448.0
    codes = torch.where(scale[..., None] > 0, x.float() / scale[..., None], torch.zeros_like(x, dtype=torch.float32))
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), scale


def records(k_codes, k_scale, v_codes, v_scale):
    """FP8 records [nb][Hkv][4224] of codes [nb][Hkv][16][128] and scales [nb][Hkv][16]."""
    nb, H = k_codes.shape[:2]
    out = torch.zeros(nb, H, 4224, dtype=torch.uint8)
    for s in range(16):
        for c in range(8):
            at = 128 * s + 16 * (c ^ (s % 8))
            out[:, :, at:at + 16] = k_codes[:, :, s, 16 * c:16 * c + 16]
        out[:, :, 2048 + 4 * (s % 8 // 2) + s % 2 + 2 * (s // 8):4096:16] = v_codes[:, :, s]
    out[:, :, 4096:4160] = k_scale.contiguous().view(torch.uint8)
    out[:, :, 4160:4224] = v_scale.contiguous().view(torch.uint8)
    return out


def row_limits(s, b):
    """Tokens below which each of stream b's rows sees."""
    n, ctx = s["new"][b], s["ctx"][b]
    return [ctx - n + j + 1 if s["causal"] else ctx for j in range(n)]


def visible(s, b):
    """[n][ctx]: which tokens each of stream b's rows sees."""
    t = torch.arange(s["ctx"][b])
    rows = []
    for limit in row_limits(s, b):
        m = t < limit
        if s["window"]:
            m &= (t >= limit - s["window"]) | (t < s["sinks"])
        rows.append(m)
    return torch.stack(rows) if rows else torch.zeros(0, s["ctx"][b], dtype=torch.bool)


def make(new, before, Hq, Hkv, dtype="bf16", window=0, sinks=0, causal=True, seed=0, garbage=float("nan"), spare=3,
         max_blocks=None, q_gain=1.0, hide=True):
    """CPU tensors of streams with the given new and cached tokens; slots and
    tokens that no row sees hold `garbage`, and with `hide` the table entries of
    blocks without a visible token are -1."""
    g = torch.Generator().manual_seed(seed)
    D = dim(dtype)
    elem = torch.float32 if dtype == "f32" else torch.bfloat16
    ctx = [n + p for n, p in zip(new, before)]
    s = dict(new=list(new), before=list(before), ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, window=window, sinks=sinks,
             causal=causal, scale=1.0 / math.sqrt(D))
    need = [-(-c // 16) for c in ctx]
    nb = sum(need) + spare
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    s["table"] = torch.full((len(ctx), max_blocks or max([1] + need)), -1, dtype=torch.int32)
    k = torch.full((nb, Hkv, 16, D), garbage, dtype=elem)
    v = k.clone()
    s["k"], s["v"] = [], []       # the streams' tokens [ctx][Hkv][D], as the cache's type holds them
    at = 0
    for b, n in enumerate(need):
        ids = perm[at:at + n].long()
        at += n
        seen = visible(s, b).any(0)
        shown = torch.zeros(n * 16, dtype=torch.bool)
        shown[:ctx[b]] = seen
        if hide:
            ids_shown = torch.where(shown.view(n, 16).any(1), ids, torch.full_like(ids, -1))
        else:
            ids_shown = ids
        s["table"][b, :n] = ids_shown.to(torch.int32)
        for pool in (k, v):
            x = torch.full((n * 16, Hkv, D), garbage, dtype=elem)
            x[shown] = torch.randn(int(seen.sum()), Hkv, D, generator=g).to(elem)
            pool[ids] = x.view(n, 16, Hkv, D).transpose(1, 2)
    T = sum(new)
    s["q"] = (torch.randn(T, Hq, D, generator=g) * q_gain).to(elem)
    s["T"] = T
    s["row_start"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32)
    s["ctx_before"] = torch.tensor(list(before), dtype=torch.int32)
    s["k_pool"], s["v_pool"] = k, v
    finish(s)
    return s


def finish(s):
    """The device form of the pools and, for FP8, the values that their codes stand for."""
    k, v = s["k_pool"], s["v_pool"]
    if s["dtype"] == "fp8":
        (kc, ks), (vc, vs) = quantise(k), quantise(v)
        # rows of garbage: NaN codes and scales
        kc[torch.isnan(ks)], vc[torch.isnan(vs)] = 0x7F, 0x7F
        s["k_val"] = kc.view(torch.float8_e4m3fn).double() * ks.double()[..., None]
        s["v_val"] = vc.view(torch.float8_e4m3fn).double() * vs.double()[..., None]
        s["pools"] = (records(kc, ks, vc, vs), None)
    else:
        s["k_val"], s["v_val"] = k.double(), v.double()
        s["pools"] = (k, v)


def cached(s, b, g):
    """(keys, values, valid) of stream b's tokens and KV head g, float64."""
    nb = s["k_val"].shape[0]
    n = -(-s["ctx"][b] // 16)
    ids = s["table"][b, :n].long()
    ok = (ids >= 0) & (ids < nb)
    at = ids.clamp(0, nb - 1)
    k = s["k_val"][at, g].reshape(n * 16, -1)[:s["ctx"][b]]
    v = s["v_val"][at, g].reshape(n * 16, -1)[:s["ctx"][b]]
    return k, v, ok.repeat_interleave(16)[:s["ctx"][b]]


def attend(s, b):
    """(out, tolerance) of stream b's rows, float64 [n][Hq][D]; rows without a
    token are zero."""
    n, Hq, Hkv = s["new"][b], s["Hq"], s["Hkv"]
    at = int(s["row_start"][b])
    out = torch.zeros(n, Hq, s["D"], dtype=torch.float64)
    tol = torch.zeros_like(out)
    see = visible(s, b)
    for g in range(Hkv):
        k, v, ok = cached(s, b, g)
        m = see & ok[None]
        for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
            sc = s["scale"] * (s["q"][at:at + n, h].double() @ k.t())
            sc = torch.where(m, sc, torch.full_like(sc, -math.inf))
            top = sc.amax(1, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            w = torch.exp(sc - top)
            tot = w.sum(1, keepdim=True)
            w = torch.where(tot == 0, torch.zeros_like(w), w / torch.where(tot == 0, torch.ones_like(tot), tot))
            # a token that a row does not see has no part in it, whatever it holds
            if torch.isfinite(v).all():
                o, size, sq = w @ v, w @ v.abs(), (w * w) @ (v * v)
            else:
                zero = torch.zeros((), dtype=torch.float64)
                terms = torch.where(m[:, :, None], w[:, :, None] * v[None], zero)
                o, size, sq = terms.sum(1), terms.abs().sum(1), (terms * terms).sum(1)
            out[:, h] = o
            tol[:, h] = U_OUT[s["dtype"]] * o.abs() + 8 * (sq / 3).sqrt() * U_P[s["dtype"]] + 2.0 ** -16 * (o.abs() + size)
    return out, tol


def attend_all(s, skip=()):
    """attend() for every stream, packed like the rows; streams in `skip` are zero."""
    out = torch.zeros(s["T"], s["Hq"], s["D"], dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, n in enumerate(s["new"]):
        if n and b not in skip:
            at = int(s["row_start"][b])
            out[at:at + n], tol[at:at + n] = attend(s, b)
    return out, tol


def check(got, ref, tol, label=""):
    """Every element within its tolerance; not finite where the reference is not."""
    got = got.double().cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{label}: NaN at other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{label}: infinities differ"
    err = (got - ref).abs()[fin]
    bad = ~(err <= tol[fin])
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} elements, worst {float((err / tol[fin].clamp(min=1e-30)).max()):.3g} tolerances"


def rotate(x, pos, base):
    """Rotate-half of rows x [..., D] at integer positions (float64)."""
    D = x.shape[-1]
    th = base ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    a = pos.double()[..., None] * th
    x = x.double()
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat((x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()), -1)
