"""The entry points of the 8-bit cache and of attention with changed scores
refuse bad arguments on the host, before any CUDA call."""
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


def test_append_arguments_rejected_on_host(lib):
    def call(kn=A, vn=A, k=A, v=A, ks=A, vs=A, B=1, h=1, n_new=1, L=64, d=64, strides=None,
             fmt=binding.CACHE_E4M3, T=64, lens=A, new=None):
        return binding.attn_cache_append_raw(kn, vn, k, v, ks, vs, B, h, n_new, L, d, strides, fmt,
                                             T, lens, new, None)
    for name in ("kn", "vn", "k", "v", "ks", "vs"):
        assert call(**{name: None}) == INV, name
    for name in ("kn", "vn", "k", "v"):
        assert call(**{name: A + 8}) == INV, name
    for name in ("ks", "vs", "lens", "new"):
        assert call(**{name: A + 2}) == INV, name
    for name in ("B", "h", "n_new", "L", "d"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    for fmt in (binding.CACHE_BF16, 3, -1):
        assert call(fmt=fmt) == INV
    for T in (0, 8, 24, 48, 256):
        assert call(T=T) == INV
    good = [64, 64, 64] * 4
    for at in range(12):
        for bad in (0, -64, 8):
            s = list(good)
            s[at] = bad
            if bad == 8 and at < 6:
                continue  # eight bf16 elements are 16 bytes
            assert call(strides=s) == INV, (at, bad)
    assert call(B=1 << 20, h=1 << 12) == INV
    assert call(d=48) == UNS and call(d=256) == UNS
    assert call(B=1 << 15, h=1 << 10, n_new=4096, L=4096) == UNS  # grid


def test_decode_scored_arguments_rejected_on_host(lib):
    def call(q=A, k=A, v=A, ks=A, vs=A, o=A, lse=None, B=1, h=2, hk=1, n_q=1, L=64, d=64,
             strides=None, fmt=binding.CACHE_E4M3, T=64, scale=0.125, cap=0.0, slopes=None,
             lens=None, window=-1, ws=None, ws_bytes=0):
        return binding.attn_decode_scored_raw(q, k, v, ks, vs, o, lse, B, h, hk, n_q, L, d, strides,
                                              fmt, T, scale, cap, slopes, lens, window, ws,
                                              ws_bytes, None)
    for name in ("q", "k", "v", "ks", "vs", "o"):
        assert call(**{name: None}) == INV, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: A + 8}) == INV, name
    for name in ("ks", "vs", "lse", "slopes", "lens"):
        assert call(**{name: A + 2}) == INV, name
    for name in ("B", "h", "hk", "n_q", "L", "d"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    assert call(h=3, hk=2) == INV
    assert call(fmt=3) == INV and call(fmt=-1) == INV
    assert call(T=24) == INV
    assert call(window=-2) == INV
    for bad in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=bad) == INV
    for bad in (-1.0, math.nan, math.inf, 1e-40):
        assert call(cap=bad) == INV
    for at in range(12):
        s = [64] * 12
        s[at] = 4
        assert call(strides=s) == INV, at
    assert call(n_q=9) == UNS and call(d=48) == UNS and call(d=256) == UNS
    assert call(B=1 << 13, h=1 << 12, hk=1) == UNS
    assert call(L=(1 << 30) + 1) == UNS
    assert lib.attn_decode_scored_workspace_bytes(1, 2, 1, 9, 64, 64, 1, -1) == 0
    assert lib.attn_decode_scored_workspace_bytes(1, 3, 2, 1, 64, 64, 1, -1) == 0


def test_mask_plan_arguments_rejected_on_host(lib):
    def call(B=1, n_q=64, n_k=64, left=-1, right=0, lens=None, docs=None, prefix=None, plan=A,
             size=1 << 20):
        return binding.attn_mask_plan_raw(B, n_q, n_k, left, right, lens, docs, prefix, plan, size,
                                          None)
    for name in ("B", "n_q", "n_k"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    assert call(left=-2) == INV and call(right=-2) == INV
    for name in ("lens", "docs", "prefix"):
        assert call(**{name: A + 2}) == INV, name
    assert call(plan=None) == INV and call(plan=A + 8) == INV
    assert call(size=lib.attn_mask_plan_bytes(1, 64, 64) - 1) == INV
    assert call(docs=A, n_k=65) == INV            # documents need n_q == n_k
    assert call(prefix=A, left=3) == INV          # two runs of keys
    assert call(n_q=(1 << 30) + 1) == UNS
    assert call(B=1 << 20, n_q=1 << 20, n_k=1 << 20) == UNS
    assert lib.attn_mask_plan_bytes(0, 1, 1) == 0
    assert lib.attn_mask_plan_bytes(1, (1 << 30) + 1, 1) == 0


def _scored_refusals(call, tensors, strides):
    for name in tensors:
        assert call(**{name: None}) == INV, name
        assert call(**{name: A + 8}) == INV, name
    for name in ("B", "h", "hk", "n_q", "n_k", "d"):
        assert call(**{name: 0}) == INV and call(**{name: -1}) == INV, name
    assert call(h=3, hk=2) == INV
    assert call(slopes=A + 2) == INV and call(lse=A + 2) == INV
    for bad in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=bad) == INV
    for bad in (-1.0, math.nan, math.inf, 1e-40):
        assert call(cap=bad) == INV
    assert call(plan=A + 8) == INV
    assert call(plan=A, plan_bytes=100) == INV    # too small for these sizes
    for at in range(strides):
        for bad in (0, -8, 4):
            s = [64] * strides
            s[at] = bad
            assert call(strides=s) == INV, (at, bad)
    assert call(d=48) == UNS and call(d=256) == UNS
    assert call(n_q=(1 << 30) + 1, d=16) == UNS


def test_fwd_scored_arguments_rejected_on_host(lib):
    def call(q=A, k=A, v=A, o=A, lse=None, B=1, h=2, hk=1, n_q=8, n_k=8, d=64, strides=None,
             scale=0.125, cap=0.0, slopes=None, plan=None, plan_bytes=0):
        return binding.attn_fwd_scored_raw(q, k, v, o, lse, B, h, hk, n_q, n_k, d, strides, scale,
                                           cap, slopes, plan, plan_bytes, None)
    _scored_refusals(call, ("q", "k", "v", "o"), 12)


def test_bwd_scored_arguments_rejected_on_host(lib):
    def call(q=A, k=A, v=A, o=A, dout=A, lse=A, dq=A, dk=A, dv=A, B=1, h=2, hk=1, n_q=8, n_k=8,
             d=64, strides=None, scale=0.125, cap=0.0, slopes=None, plan=None, plan_bytes=0, ws=A,
             ws_bytes=1 << 40):
        return binding.attn_bwd_scored_raw(q, k, v, o, dout, lse, dq, dk, dv, B, h, hk, n_q, n_k, d,
                                           strides, scale, cap, slopes, plan, plan_bytes, ws,
                                           ws_bytes, None)
    _scored_refusals(call, ("q", "k", "v", "o", "dout", "dq", "dk", "dv", "ws"), 24)
    assert call(lse=None) == INV
    assert call(ws_bytes=lib.attn_bwd_scored_workspace_bytes(1, 2, 1, 8, 8, 64) - 1) == INV
    assert call(d=128) == UNS
    assert lib.attn_bwd_scored_workspace_bytes(1, 2, 1, 8, 8, 128) == 0
    assert lib.attn_bwd_scored_workspace_bytes(1, 3, 2, 8, 8, 64) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 1, 64, 64, dtype=torch.int8)
    s = torch.zeros(1, 1, 1)
    with pytest.raises(ValueError):
        binding.attn_cache_append(x, x, c, c, s, s, None)
    with pytest.raises(ValueError):
        binding.attn_decode_scored(x, c, c, k_scale=s, v_scale=s)
    with pytest.raises(ValueError):
        binding.attn_mask_plan(1, 4, 4, device="cpu")
    with pytest.raises(ValueError):
        binding.attn_fwd_scored(x, x, x)
    with pytest.raises(ValueError):
        binding.attn_bwd_scored(x, x, x, x, s, x)
