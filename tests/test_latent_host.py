"""Latent-cache entry points on the host: bad arguments are refused before
anything is launched, workspace queries, the descriptor's layout (CPU only)."""
import ctypes
import shutil
import subprocess

import pytest
import torch

import decode_step_gb300 as pkg
from decode_step_gb300 import _lib
from decode_step_gb300.build import build

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    build()
    return pkg.lib()


def _cache(num_blocks=8, block=16, latent=512, rope=64, dtype=1, pool=FAKE):
    return _lib.LatentCacheDesc(num_blocks, block, latent, rope, dtype, pool)


BAD_CACHES = [(dict(pool=None), INVALID), (dict(num_blocks=0), INVALID), (dict(block=32), UNSUPPORTED),
              (dict(latent=100), UNSUPPORTED), (dict(latent=576), UNSUPPORTED), (dict(latent=0), UNSUPPORTED),
              (dict(rope=32), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
              (dict(pool=ODD), INVALID), (dict(num_blocks=1 << 28), UNSUPPORTED)]


def _append(L, c=None, **k):
    c = _cache() if c is None else c
    return L.tts_latent_append(k.get("cache", ctypes.byref(c)), k.get("table", FAKE), k.get("maxb", 4),
                               k.get("before", FAKE), k.get("B", 2), k.get("start", None), k.get("T", 4),
                               k.get("Hq", 16), k.get("base", 10000.0), k.get("c_new", FAKE), k.get("kr", FAKE),
                               k.get("q", FAKE), k.get("qo", FAKE), None, None)


def _decode(L, c=None, **k):
    c = _cache() if c is None else c
    return L.tts_latent_decode_attn(k.get("cache", ctypes.byref(c)), k.get("table", FAKE), k.get("maxb", 4),
                                    k.get("ctx", FAKE), k.get("maxctx", 64), k.get("B", 2), k.get("q_len", 1),
                                    k.get("Hq", 16), k.get("nope", 128), k.get("v", 128), k.get("scale", 0.07),
                                    0, k.get("qn", FAKE), k.get("qr", FAKE), k.get("uk", FAKE), k.get("uv", FAKE),
                                    k.get("out", FAKE), k.get("ws", FAKE), k.get("wsb", 0), None, None)


def _prefill(L, c=None, **k):
    c = _cache() if c is None else c
    return L.tts_latent_prefill_attn(k.get("cache", ctypes.byref(c)), k.get("table", FAKE), k.get("maxb", 4),
                                     k.get("ctx", FAKE), k.get("total", 64), k.get("B", 2), k.get("start", FAKE),
                                     k.get("T", 8), k.get("Hq", 16), k.get("nope", 128), k.get("v", 128),
                                     k.get("scale", 0.07), k.get("qn", FAKE), k.get("qr", FAKE), k.get("uk", FAKE),
                                     k.get("uv", FAKE), k.get("out", FAKE), k.get("ws", FAKE), k.get("wsb", 0),
                                     None, None)


@pytest.mark.parametrize("call", [_append, _decode, _prefill])
def test_cache_checks(L, call):
    assert call(L, cache=None) == INVALID
    assert call(L, table=None) == INVALID
    assert call(L, maxb=0) == INVALID and call(L, maxb=(1 << 20) + 1) == INVALID
    for kw, code in BAD_CACHES:
        assert call(L, _cache(**kw)) == code, kw


def test_append_checks(L):
    assert _append(L, before=None) == INVALID
    assert _append(L, c_new=None) == INVALID and _append(L, kr=None) == INVALID
    assert _append(L, q=None) == INVALID and _append(L, qo=None) == INVALID
    assert _append(L, q=ODD) == INVALID and _append(L, qo=ODD) == INVALID
    assert _append(L, c_new=ODD) == INVALID and _append(L, kr=ODD) == INVALID
    assert _append(L, B=-1) == INVALID and _append(L, T=-1) == INVALID
    assert _append(L, T=5) == INVALID                       # 5 rows of 2 streams, no row_start
    assert _append(L, B=0, T=4) == INVALID
    assert _append(L, base=1.0) == INVALID and _append(L, base=0.0) == INVALID
    assert _append(L, base=float("inf")) == INVALID and _append(L, base=float("nan")) == INVALID
    assert _append(L, Hq=-1) == INVALID and _append(L, Hq=1025) == INVALID
    assert _append(L, T=0) == 0 and _append(L, B=0, T=0) == 0
    assert _append(L, B=0, T=4, start=FAKE) == 0            # rows of no stream


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_checks(L, call):
    for name in ("ctx", "qn", "qr", "uk", "uv", "out"):
        assert call(L, **{name: None}) == INVALID, name
    for name in ("qn", "qr", "uk", "uv", "out"):
        assert call(L, **{name: ODD}) == INVALID, name
    assert call(L, B=-1) == INVALID and call(L, Hq=0) == INVALID
    assert call(L, nope=0) == INVALID and call(L, v=-3) == INVALID
    assert call(L, nope=96) == UNSUPPORTED and call(L, v=192) == UNSUPPORTED
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(L, scale=scale) == INVALID
    assert call(L, wsb=0) == WORKSPACE and call(L, ws=None, wsb=1 << 30) == WORKSPACE
    assert call(L, ws=ODD, wsb=1 << 30) == WORKSPACE
    assert call(L, B=0) == 0


def test_decode_checks(L):
    assert _decode(L, q_len=0) == INVALID and _decode(L, maxctx=0) == INVALID
    assert _decode(L, q_len=65) == UNSUPPORTED               # 1040 query rows
    ws = L.tts_latent_decode_attn_workspace_size
    assert ws(64, 1, 16, 512, 128, 128, 1500) > 0
    assert ws(64, 5, 16, 512, 128, 128, 2048) >= ws(64, 1, 16, 512, 128, 128, 2048)
    for bad in [(-1, 1, 16, 512, 128, 128, 10), (1, 0, 16, 512, 128, 128, 10), (1, 1, 0, 512, 128, 128, 10),
                (1, 1, 16, 500, 128, 128, 10), (1, 1, 16, 512, 96, 128, 10), (1, 1, 16, 512, 128, 32, 10),
                (1, 1, 16, 512, 128, 128, 0), (1, 3, 512, 512, 128, 128, 10)]:
        assert ws(*bad) == 0, bad


def test_prefill_checks(L):
    assert _prefill(L, start=None) == INVALID
    assert _prefill(L, T=-1) == INVALID and _prefill(L, total=-1) == INVALID
    assert _prefill(L, Hq=1025) == UNSUPPORTED
    assert _prefill(L, T=0) == 0
    ws = L.tts_latent_prefill_attn_workspace_size
    assert ws(4, 1000, 16, 512, 128, 128, 1000) > 0
    for bad in [(-1, 8, 16, 512, 128, 128, 10), (1, -8, 16, 512, 128, 128, 10), (1, 8, 0, 512, 128, 128, 10),
                (1, 8, 16, 60, 128, 128, 10), (1, 8, 16, 512, 256, 128, 10), (1, 8, 16, 512, 128, 128, -1)]:
        assert ws(*bad) == 0, bad


def test_latent_cache_layout_matches_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    D = _lib.LatentCacheDesc
    fields = [f for f, _ in D._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "tts_decode.h"', "int main(void) {",
           'printf("%zu\\n", sizeof(tts_latent_cache));']
    src += [f'printf("%zu\\n", offsetof(tts_latent_cache, {f}));' for f in fields] + ["return 0; }"]
    (tmp_path / "lay.c").write_text("\n".join(src) + "\n")
    subprocess.run([cc, "-I", str(_lib.HEADER.parent), "-o", str(tmp_path / "lay"), str(tmp_path / "lay.c")], check=True)
    out = subprocess.run([str(tmp_path / "lay")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(D)] + [getattr(D, f).offset for f in fields]


def test_binding_refuses_host_tensors_and_bad_pools():
    from decode_step_gb300 import binding as bd
    with pytest.raises(ValueError, match="latent pool"):
        bd.LatentCache(torch.zeros(4, 8, 576, dtype=torch.bfloat16), 512)
    with pytest.raises(ValueError, match="latent pool"):
        bd.LatentCache(torch.zeros(4, 16, 576), 512)
    with pytest.raises(ValueError, match="latent_dim"):
        bd.LatentCache(torch.zeros(4, 16, 576, dtype=torch.bfloat16), 576)
    with pytest.raises(ValueError, match="CUDA"):
        bd.LatentCache(torch.zeros(4, 16, 576, dtype=torch.bfloat16), 512)
