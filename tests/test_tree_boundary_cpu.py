"""The entry points of drafted trees refuse bad arguments on the host, before any
CUDA call."""
import math

import pytest
import torch

from transformer_head_scaled_gb300 import binding
from transformer_head_scaled_gb300.build import build

INV, UNS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED
A = 0x10000  # a fake, never dereferenced, 16-byte aligned device address


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def test_decode_tree_arguments_rejected_on_host(lib):
    def call(q=A, kt=A, vt=A, k=A, v=A, ks=A, vs=A, parents=A, o=A, lse=None, B=1, h=2, hk=1, n=4,
             L=64, d=64, strides=None, fmt=binding.CACHE_E4M3, T=64, scale=0.125, cap=0.0,
             slopes=None, lens=None, window=-1, ws=None, ws_bytes=0):
        return binding.attn_decode_tree_raw(q, kt, vt, k, v, ks, vs, parents, o, lse, B, h, hk, n,
                                            L, d, strides, fmt, T, scale, cap, slopes, lens,
                                            window, ws, ws_bytes, None)
    for name in ("q", "kt", "vt", "k", "v", "ks", "vs", "parents", "o"):
        assert call(**{name: None}) == INV, name
    for name in ("q", "kt", "vt", "k", "v", "o"):
        assert call(**{name: A + 8}) == INV, name
    for name in ("parents", "ks", "vs", "lse", "slopes", "lens"):
        assert call(**{name: A + 2}) == INV, name
    for name in ("B", "h", "hk", "n", "L", "d"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    assert call(h=3, hk=2) == INV
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=scale) == INV
    for cap in (-1.0, math.nan, math.inf, 2.0 ** 65):
        assert call(cap=cap) == INV
    assert call(window=-2) == INV
    for fmt in (3, -1):
        assert call(fmt=fmt) == INV
    for T in (0, 8, 24, 48, 256):
        assert call(T=T) == INV
    good = [64, 64, 64] * 6
    for at in range(18):
        for bad in (0, -64, 8 if 9 <= at < 15 else 4):
            s = list(good)
            s[at] = bad
            assert call(strides=s) == INV, (at, bad)
    assert call(n=129) == UNS
    assert call(d=48) == UNS and call(d=256) == UNS
    assert call(L=(1 << 30) + 1) == UNS
    assert call(B=1 << 20, h=8, n=4) == UNS


def test_tree_verify_arguments_rejected_on_host(lib):
    def call(p=A, q=A, tokens=A, parents=A, u=A, path=A, lens=A, out=A, B=1, n=4, V=100,
             strides=None, kind=binding.PROB_F32):
        return binding.attn_tree_verify_raw(p, q, tokens, parents, u, path, lens, out, B, n, V,
                                            strides, kind, None)
    for name in ("p", "tokens", "parents", "u", "path", "lens", "out"):
        assert call(**{name: None}) == INV, name
        assert call(**{name: A + 2}) == INV, name
    assert call(q=A + 2) == INV
    assert call(p=A + 1, kind=binding.PROB_BF16) == INV
    assert call(q=A + 1, kind=binding.PROB_BF16) == INV
    for name in ("B", "n", "V"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    for kind in (-1, 2):
        assert call(kind=kind) == INV
    for at in range(4):
        for bad in (-1, 1 << 40):
            s = [400, 100, 400, 100]
            s[at] = bad
            assert call(strides=s) == INV, (at, bad)
    assert call(n=129) == UNS and call(V=(1 << 24) + 1) == UNS and call(B=(1 << 24) + 1) == UNS


def test_append_tree_arguments_rejected_on_host(lib):
    def call(kt=A, vt=A, path=A, pl=A, k=A, v=A, ks=A, vs=A, layers=1, B=1, h=1, n=4, L=64, d=64,
             strides=None, fmt=binding.CACHE_E4M3, T=64, lens=A):
        return binding.attn_cache_append_tree_raw(kt, vt, path, pl, k, v, ks, vs, layers, B, h, n,
                                                  L, d, strides, fmt, T, lens, None)
    for name in ("kt", "vt", "path", "pl", "k", "v", "ks", "vs"):
        assert call(**{name: None}) == INV, name
    for name in ("kt", "vt", "k", "v"):
        assert call(**{name: A + 8}) == INV, name
    for name in ("path", "pl", "ks", "vs", "lens"):
        assert call(**{name: A + 2}) == INV, name
    for name in ("layers", "B", "h", "n", "L", "d"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    for fmt in (3, -1):
        assert call(fmt=fmt) == INV
    for T in (0, 8, 24, 48, 256):
        assert call(T=T) == INV
    good = [64, 64, 64, 64] * 4
    for at in range(16):
        for bad in (0, -64, 8 if at >= 8 else 4):
            s = list(good)
            s[at] = bad
            assert call(strides=s) == INV, (at, bad)
    assert call(n=129) == UNS and call(d=48) == UNS and call(L=(1 << 30) + 1) == UNS
    assert call(layers=1 << 10, B=1 << 11, h=1 << 10) == UNS  # grid


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    ids = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.attn_decode_tree(x, x, x, ids, x, x)
    with pytest.raises(ValueError):
        binding.attn_tree_verify(torch.zeros((1, 4, 10)), ids, ids, torch.zeros((1, 4)))
    with pytest.raises(ValueError):
        binding.attn_cache_append_tree(x, x, ids, ids[:, 0], x, x, None)
