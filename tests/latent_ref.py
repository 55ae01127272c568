"""Inputs, the 64-bit reference and derived tolerances of the latent-cache tests.

Tolerances.  A rounding to bf16 is off by at most u = 2^-8 of the value, and is
taken as independent with variance at most u^2 / 3 of the value's square.  To
first order an error ds_t of token t's score moves out by w_t ds_t (v_t - out),
w the softmax weights.  The forms round:
  absorbed: q~_l:   ds_t = scale dq~_l c_tl for every t, so out moves by
                    dq~_l g_l, g_l = scale sum_t w_t c_tl (v_t - out)
            p_t:    w_t v_t          (weights enter the matrix product in bf16)
            o~_l:   w_uv_l o~_l
  expanded: k_td:   w_t scale q_d (v_t - out)
            p_t:    w_t v_t;   v_t: w_t v_t
each times the rounded value's relative error.  With S the sum of the squares
of those terms, an element passes when it is within
  u |out| + 8 sqrt(S u^2 / 3) + 2^-16 (|out| + sum_t w_t |v_t|)
of the reference: the output's own rounding, eight standard deviations (a
single term's full half step is 1.7), and fp32 arithmetic (sums of a few
thousand terms, hardware exponentials, scores of size up to some tens).
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -8
ROPE = 64


def make(lens_new, lens_before, Hq, L, nope, v, seed, garbage=float("nan"), spare=3, max_blocks=None, q_gain=1.0):
    """Bf16 inputs (CPU tensors) for streams with the given new and cached
    token counts; pool slots without a token hold `garbage`."""
    g = torch.Generator().manual_seed(seed)
    ctx = [n + p for n, p in zip(lens_new, lens_before)]
    need = [-(-c // 16) for c in ctx]
    nb = sum(need) + spare
    T = sum(lens_new)
    width = L + ROPE

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)

    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max_blocks or max([1] + need)), -1, dtype=torch.int32)
    pool = torch.full((nb, 16, width), garbage, dtype=torch.bfloat16)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        rows = torch.full((n * 16, width), garbage, dtype=torch.bfloat16)
        rows[:ctx[b]] = normal(ctx[b], width)
        pool[table[b, :n].long()] = rows.view(n, 16, width)
    start = np.concatenate([[0], np.cumsum(lens_new)]).astype(np.int32)
    return dict(new=list(lens_new), before=list(lens_before), ctx=ctx, table=table, pool=pool, L=L, Hq=Hq, nope=nope, v=v,
                T=T, ctx_lens=torch.tensor(ctx, dtype=torch.int32), row_start=torch.from_numpy(start),
                ctx_before=torch.tensor(list(lens_before), dtype=torch.int32),
                q_nope=normal(T, Hq, nope, std=q_gain), q_rope=normal(T, Hq, ROPE, std=q_gain),
                w_uk=normal(Hq, nope, L, std=L ** -0.5), w_uv=normal(Hq, v, L, std=L ** -0.5),
                c_new=normal(T, L), kr_new=normal(T, ROPE), scale=1.0 / math.sqrt(nope + ROPE))


def cached_rows(s, b):
    """(rows of stream b's tokens in float64, mask of those in valid blocks)."""
    nb = s["pool"].shape[0]
    n = -(-s["ctx"][b] // 16)
    ids = s["table"][b, :n].long()
    ok = (ids >= 0) & (ids < nb)
    rows = s["pool"][ids.clamp(0, nb - 1)].reshape(n * 16, -1)[:s["ctx"][b]].double()
    ok = ok.repeat_interleave(16)[:s["ctx"][b]]
    return torch.where(ok[:, None], rows, torch.zeros_like(rows)), ok


def attend(s, b, causal, absorbed):
    """(out, tolerance) of stream b's rows, float64 [n][Hq][v]."""
    n, L, Hq = s["new"][b], s["L"], s["Hq"]
    at = int(s["row_start"][b])
    rows, ok = cached_rows(s, b)
    c, kr = rows[:, :L], rows[:, L:]
    ctx = s["ctx"][b]
    hidden = torch.zeros(n, ctx, dtype=torch.bool)
    if causal:
        hidden = torch.arange(ctx)[None, :] > torch.arange(ctx - n, ctx)[:, None]
    hidden = hidden | ~ok[None, :]
    out = torch.zeros(n, Hq, s["v"], dtype=torch.float64)
    tol = torch.zeros_like(out)
    for h in range(Hq):
        wuk, wuv = s["w_uk"][h].double(), s["w_uv"][h].double()
        k, val = c @ wuk.t(), c @ wuv.t()
        qn, qr = s["q_nope"][at:at + n, h].double(), s["q_rope"][at:at + n, h].double()
        sc = s["scale"] * (qn @ k.t() + qr @ kr.t())
        sc = sc.masked_fill(hidden, -math.inf)
        m = sc.amax(1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        w = torch.exp(sc - m)
        tot = w.sum(1, keepdim=True)
        w = torch.where(tot > 0, w / tot.clamp(min=1e-300), torch.zeros_like(w))
        o = w @ val
        wv2 = (w * w) @ (val * val)
        if absorbed:
            qt = qn @ wuk
            # g_l = scale (sum_t w_t c_tl v_t - out sum_t w_t c_tl), per row and output dim
            lat = w @ c
            S = wv2 + (lat * lat) @ (wuv * wuv).t()
            for r in range(n):
                gl = s["scale"] * ((w[r][:, None] * c).t() @ val - lat[r][:, None] * o[r][None, :])
                S[r] += (qt[r] ** 2) @ (gl * gl)
        else:
            S = 2 * wv2
            var = s["scale"] ** 2 * ((qn * qn) @ (k * k).t()) * (w * w)
            # sum_t var_t (v_t - out)^2
            S = S + var @ (val * val) - 2 * o * (var @ val) + o * o * var.sum(1, keepdim=True)
        out[:, h] = o
        tol[:, h] = U * o.abs() + 8 * (S.clamp(min=0) / 3).sqrt() * U + 2.0 ** -16 * (o.abs() + w @ val.abs())
    return out, tol


def attend_all(s, causal, absorbed, skip=()):
    """attend() for every stream, packed like the rows; streams in `skip` are zero."""
    out = torch.zeros(s["T"], s["Hq"], s["v"], dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, n in enumerate(s["new"]):
        if n and b not in skip:
            at = int(s["row_start"][b])
            out[at:at + n], tol[at:at + n] = attend(s, b, causal, absorbed)
    return out, tol


def rotate(x, pos, base):
    """Rotate-half of rows x [..., 64] at integer positions (float64)."""
    th = base ** (-torch.arange(ROPE // 2, dtype=torch.float64) * 2 / ROPE)
    a = pos.double()[..., None] * th
    x = x.double()
    x1, x2 = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat((x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()), -1)
