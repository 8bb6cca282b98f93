"""Refusals of the 8-bit cache and log-probability calls, before any CUDA call
(CPU only)."""
import ctypes
import gc
import weakref

import pytest
import torch

import greedy_speculative_verify_b200 as vgv
from greedy_speculative_verify_b200 import build as vbuild

A = 1 << 40  # fake, aligned, never dereferenced: validation fails first
G = 1 << 30


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vgv.load()


def cache(**kw):
    f = dict(format=0, B=2, L_max=256, n_kv=10, dim=128, block=64, k=A, v=A + G, k_amax=A + 2 * G, v_amax=A + 3 * G)
    return ctypes.byref(vgv.vg_kv8(*{**f, **kw}.values()))


BAD_CACHES = [(dict(B=-1), 1), (dict(L_max=0), 1), (dict(n_kv=0), 1), (dict(L_max=200), 1), (dict(k=None), 1),
              (dict(v_amax=None), 1), (dict(v=A + G + 8), 1), (dict(k_amax=A + 2), 1), (dict(format=2), 2), (dict(dim=96), 2),
              (dict(block=8), 2), (dict(block=48), 2), (dict(L_max=1 << 21), 2), (dict(n_kv=1025), 2)]


def append(lib, c, rows=4, k=A + 4 * G, ks=1280, v=A + 5 * G, vs=1280, pos=A + 6 * G, n=None):
    return lib.vg_kv8_append(c, rows, k, ks, v, vs, pos, n, None)


def read(lib, c, rows=4, pos=A + 6 * G, n=None, kind=0, k=A + 4 * G, ks=1280, v=A + 5 * G, vs=1280):
    return lib.vg_kv8_read(c, rows, pos, n, kind, k, ks, v, vs, None)


def attn(lib, c, rows=4, heads=10, q=A + 4 * G, qs=1280, lens=A + 6 * G, first=None, n=None, scale=0.1, o=A + 5 * G, os=1280,
         ws=A + 7 * G, bytes=1 << 29):
    return lib.vg_kv8_attn(c, rows, heads, q, qs, lens, first, n, scale, o, os, ws, bytes, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):
    for f in (append, read, attn):
        assert f(lib, cache(**kw)) == status
    assert lib.vg_kv8_attn_workspace_bytes(cache(**kw), 4, 10) == 0
    assert append(lib, None) == 1 and read(lib, None) == 1 and attn(lib, None) == 1


def test_append(lib):
    assert append(lib, cache(B=0)) == 0 and append(lib, cache(), rows=0) == 0
    for kw in (dict(rows=-1), dict(k=None), dict(v=None), dict(pos=None), dict(k=A + 4 * G + 8), dict(pos=A + 2), dict(n=A + 1),
               dict(ks=1279), dict(vs=1284), dict(ks=1 << 25), dict(k=A + 64), dict(v=A + 2 * G)):
        assert append(lib, cache(), **kw) == 1, kw
    assert append(lib, cache(), rows=(1 << 20) + 1) == 2
    assert append(lib, cache(B=1 << 20, n_kv=1024, block=16, L_max=16), ks=1 << 17, vs=1 << 17) == 2  # more blocks than a launch holds


def test_read(lib):
    assert read(lib, cache(B=0)) == 0 and read(lib, cache(), rows=0) == 0 and read(lib, cache(), k=None, v=None) == 0
    for kw in (dict(rows=-1), dict(kind=2), dict(pos=None), dict(k=A + 4 * G + 8), dict(vs=1272), dict(ks=1282), dict(v=A + 4 * G),
               dict(v=A + 4 * G + 2560 * 2), dict(k=A + G), dict(n=A + 2), dict(ks=2560, vs=2568, v=A + 4 * G + 2560),
               dict(ks=2560, vs=2560, v=A + 4 * G + 2544)):
        assert read(lib, cache(), **kw) == 1, kw


def test_attention(lib):
    need = lib.vg_kv8_attn_workspace_bytes(cache(), 4, 10)
    assert need > 0
    assert attn(lib, cache(B=0)) == 0
    for kw in (dict(rows=0), dict(heads=0), dict(heads=15), dict(q=None), dict(lens=None), dict(o=None), dict(q=A + 4 * G + 2),
               dict(qs=1272), dict(os=1281), dict(o=A + 4 * G), dict(o=A), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(first=A + 2), dict(n=A + 3)):
        assert attn(lib, cache(), **kw) == 1, kw
    assert attn(lib, cache(), rows=9) == 2 and attn(lib, cache(n_kv=1), heads=17, qs=2176, os=2176) == 2
    assert attn(lib, cache(), bytes=need - 1) == 3 and attn(lib, cache(), ws=None) == 3 and attn(lib, cache(), ws=A + 7 * G + 8) == 3


def test_layer(lib):
    f = lib.vg_attn_verify_kv8
    need = lib.vg_attn_verify_kv8_workspace_bytes(cache(), 3)

    def call(c=None, K=3, x=A + 4 * G, wq=A + 5 * G, wo=A + 6 * G, lens=A + 7 * G, out=A + 8 * G, o=None, ws=A + 9 * G, n=need):
        return f(c or cache(), K, x, wq, wo, lens, out, o, ws, n, None)

    assert need > 0 and call(cache(B=0)) == 0
    for kw in (dict(K=-1), dict(K=8), dict(x=None), dict(wq=None), dict(lens=None), dict(out=None), dict(wo=A + 8), dict(out=A + 4 * G + 64),
               dict(out=A + 64), dict(o=A + 8 * G), dict(o=A + 4 * G), dict(o=A + G)):
        assert call(**kw) == 1, kw
    assert call(cache(n_kv=5)) == 2 and call(cache(dim=64)) == 2 and call(cache(L_max=65536)) == 2
    assert call(n=need - 1) == 3 and call(ws=A + 9 * G + 8) == 3
    assert lib.vg_attn_verify_kv8_workspace_bytes(cache(n_kv=5), 3) == 0 and lib.vg_attn_verify_kv8_workspace_bytes(cache(), 8) == 0


def test_logprobs(lib):
    f = lib.vg_token_logprobs
    need = lib.vg_token_logprobs_workspace_bytes(4, 1280, 129280, 5)

    def call(R=4, H=1280, V=129280, h=A, lm=A + G, tok=A + 2 * G, n=5, lp=A + 3 * G, en=A + 4 * G, ids=A + 5 * G, tl=A + 6 * G,
             ws=A + 7 * G, bytes=need):
        return f(R, H, V, h, lm, tok, n, lp, en, ids, tl, ws, bytes, None)

    assert need > 0 and call(R=0) == 0
    for kw in (dict(R=-1), dict(V=0), dict(H=0), dict(n=-1), dict(V=4), dict(h=None), dict(lm=None), dict(tok=None), dict(ids=None),
               dict(tl=None), dict(h=A + 8), dict(lm=A + G + 4), dict(tok=A + 1), dict(en=A + 2)):
        assert call(**kw) == 1, kw
    assert call(H=1288) == 2 and call(H=8256) == 2 and call(n=21) == 2 and call(R=1 << 24) == 2
    assert call(bytes=need - 1) == 3 and call(ws=None) == 3 and call(ws=A + 7 * G + 8) == 3
    for bad in ((-1, 1280, 100, 5), (4, 1000, 100, 5), (4, 1280, 100, 21), (4, 1280, 3, 5)):
        assert lib.vg_token_logprobs_workspace_bytes(*bad) == 0


def test_binding_refuses_wrong_tensors():
    """Shapes, types, density and devices, before any library call."""
    k = torch.zeros(2, 3, 64, 64, dtype=torch.int8)
    a = torch.zeros(2, 3, 4)
    c = vgv.make_kv8(k, k.clone(), a, a.clone())
    assert (c.format, c.B, c.n_kv, c.L_max, c.dim, c.block) == (vgv.VG_KV8_INT8, 2, 3, 64, 64, 16)
    assert vgv.make_kv8(k.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), a, a).format == vgv.VG_KV8_E4M3
    for bad in ((k.float(), k, a, a), (k, k.view(torch.float8_e4m3fn), a, a), (k.transpose(1, 2), k, a, a), (k, k[:1], a, a),
                (k, k, a.double(), a), (k, k, a, a[:, :2]), (k, k, torch.zeros(2, 3, 5), a), (k[0], k[0], a, a),
                (k, k.to("meta"), a, a)):
        with pytest.raises(ValueError):
            vgv.make_kv8(*bad)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    for f in (lambda: vgv.vg_kv8_append(c, 4, bf(8, 191), bf(8, 192), i), lambda: vgv.vg_kv8_append(c, 4, bf(7, 192), bf(8, 192), i),
              lambda: vgv.vg_kv8_append(c, 4, bf(8, 192).float(), bf(8, 192), i), lambda: vgv.vg_kv8_append(c, 4, bf(192, 8).T, bf(8, 192), i),
              lambda: vgv.vg_kv8_append(c, 4, bf(8, 192), bf(8, 192), i.long()), lambda: vgv.vg_kv8_append(c, 4, bf(8, 192), bf(8, 192), i[:1]),
              lambda: vgv.vg_kv8_append(c, 4, bf(8, 192).to("meta"), bf(8, 192), i),
              lambda: vgv.vg_kv8_read(c, 4, i, bf(8, 192), bf(8, 192).float()),
              lambda: vgv.vg_kv8_attn(c, 4, 6, bf(8, 192), i, 1.0, bf(8, 384), ws),
              lambda: vgv.vg_attn_verify_kv8(c, 3, bf(8, 192), bf(576, 192), bf(192, 192), i, bf(8, 191), ws),
              lambda: vgv.vg_token_logprobs(bf(4, 64), bf(9, 128), i, None, None, None, None, ws),
              lambda: vgv.vg_token_logprobs(bf(2, 64), bf(9, 64), i, a[0, 0, :2].double(), None, None, None, ws),
              lambda: vgv.vg_token_logprobs(bf(2, 64).T.contiguous().T, bf(9, 64), i, None, None, None, None, ws)):
        with pytest.raises(ValueError):
            f()


def test_binding_refuses_host_tensors():
    """Tensors that lie in host memory: a kernel would take their addresses as they are."""
    k, a = torch.zeros(2, 3, 64, 64, dtype=torch.int8), torch.zeros(2, 3, 4)
    c = vgv.make_kv8(k, k.clone(), a, a.clone())
    x, i, ws = torch.zeros(8, 192, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    h, f = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2)
    for call in (lambda: vgv.vg_kv8_append(c, 4, x, x.clone(), i), lambda: vgv.vg_kv8_read(c, 4, i, x, None),
                 lambda: vgv.vg_kv8_attn(c, 4, 3, x, i, 0.1, x.clone(), ws),
                 lambda: vgv.vg_token_logprobs(h, h.clone(), i, f, None, None, None, ws)):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call()


def test_handle_lets_its_tensors_go():
    """Without its handle and the caller's names a cache's memory is free at once,
    not when a collector next runs; a call with the handle changes nothing in that."""
    k, a = torch.zeros(2, 3, 64, 64, dtype=torch.int8), torch.zeros(2, 3, 4)
    v, b = k.clone(), a.clone()
    c = vgv.make_kv8(k, v, a, b)
    assert vgv.vg_kv8_attn_workspace_bytes(c, 4, 3) > 0 and c.k == k.data_ptr()
    held = [weakref.ref(t) for t in (k, v, a, b)]
    gc.disable()
    try:
        del k, v, a, b
        assert all(r() is not None for r in held)  # the handle keeps them
        del c
        assert all(r() is None for r in held)
    finally:
        gc.enable()


def test_writes_refuse_a_cache_whose_parts_share_memory(lib):
    """Keys and values in one tensor, one magnitude tensor for both, magnitudes
    inside the codes: what is written for one would lie over the other."""
    codes, am = 2 * 10 * 256 * 128, 2 * 10 * 4 * 4
    need = lib.vg_attn_verify_kv8_workspace_bytes(cache(), 3)
    layer = lambda c: lib.vg_attn_verify_kv8(c, 3, A + 4 * G, A + 5 * G, A + 6 * G, A + 7 * G, A + 8 * G, None, A + 9 * G, need, None)
    for kw in (dict(v=A), dict(v=A + codes - 16), dict(v=A - codes + 16), dict(v_amax=A + 2 * G), dict(v_amax=A + 2 * G + am - 4),
               dict(k_amax=A), dict(k_amax=A + G + codes - 4), dict(v_amax=A + codes - 4), dict(v_amax=A + G)):
        assert append(lib, cache(**kw)) == 1, kw
        assert layer(cache(**kw)) == 1, kw


def test_row_stride_of_a_single_row():
    """A single row may come from a matrix of any width: no row lies behind it."""
    bf16 = torch.bfloat16
    for wide in (192, 195, 200, 1 << 25):
        one = torch.empty(1, wide, dtype=bf16, device="meta")[:, :192]
        assert vgv._rows("k", one, 1, 192, (bf16,)) == 192
    assert vgv._rows("k", torch.empty(2, 200, dtype=bf16)[:, :192], 2, 192, (bf16,)) == 200
