"""The decoding step against 8-bit caches whose blocks have scales far apart: what
one block's values are must not cost the others precision, whether or not that
block has any weight.

Tolerances as in test_cache_gpu: half a step of bf16 of O, a rounding of every
probability to f16 (2^-11 of sum_j p_j |v_j|) and twice the scores' error of the
same sum.
"""
import math

import numpy as np
import pytest
import torch

from oracle import scored
from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu

SCORE_TOL = 3e-4
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from transformer_head_scaled_gb300.build import build
    build()
    return binding.load()


def _random(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def _quantised(x, dtype, block):
    """Codes, scales and float64 values of x [B, h, L, d], L a multiple of block."""
    top = 127.0 if dtype == INT8 else 448.0
    B, h, L, d = x.shape
    s = x.reshape(B, h, L // block, block * d).abs().amax(-1) / top
    y = x / s.repeat_interleave(block, 2)[..., None]
    c = y.round().clamp(-127, 127).to(INT8) if dtype == INT8 else y.clamp(-448, 448).to(E4M3)
    wide = c.float().cpu().double().numpy() * np.repeat(s.cpu().double().numpy(), block, 2)[..., None]
    return c, s, wide


def _check(got, q, k, v, lens, **kw):
    o, lse = (t.float().cpu().double().numpy() for t in got)
    qd = q.double().cpu().numpy()
    scale = 1 / math.sqrt(q.shape[-1])
    ro, rl = scored.decode(qd, k, v, lens, scale, **kw)
    weight, _ = scored.decode(qd, k, np.abs(v), lens, scale, **kw)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * SCORE_TOL) * weight + 1e-6
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= tol).all(), (np.abs(o - ro) / tol).max()
    assert (np.abs(lse - rl) <= SCORE_TOL).all(), np.abs(lse - rl).max()


# one sequence split over warps, and many short ones that a warp takes whole
SIZES = {"split": (1, 2, 4096), "whole": (128, 10, 160)}


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("log_ratio", [10, 18, 30])
@pytest.mark.parametrize("against", [0.0, 0.4, 1.0])
def test_one_block_of_large_values(dtype, size, place, log_ratio, against):
    """A block whose values are 2^10 to 2^30 times the others', with keys of
    ordinary scores (against = 0) or against the query: scores of -13 or -32."""
    B, h, L = SIZES[size]
    d, block = 64, 16
    q = _random((B, h, 1, d), 1, 2.0).to(BF16)
    kx, vx = _random((B, h, L, d), 2), _random((B, h, L, d), 3)
    rows = slice(0, block) if place == "first" else slice(L - block, L)
    if against:
        kx[:, :, rows] = -against * q.float()
    vx[:, :, rows] *= 2.0 ** log_ratio
    kc, ks, k = _quantised(kx, dtype, block)
    vc, vs, v = _quantised(vx, dtype, block)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block)
    binding.check()
    _check(got, q, k, v, [L] * B)


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("h,n_q,d", [(4, 1, 64), (4, 3, 128), (8, 4, 32), (16, 2, 16)])
@pytest.mark.parametrize("log_ratio", [18, 60])
def test_rows_of_one_tile_weigh_different_blocks(dtype, h, n_q, d, log_ratio):
    """Query heads that share a key head: a block of large values that the first
    query does not look at and the others do, another the other way round."""
    L, block = 2048, 32
    q = _random((1, h, n_q, d), 1, 2.0).to(BF16)
    kx, vx = _random((1, 1, L, d), 2), _random((1, 1, L, d), 3)
    away = 32 * math.sqrt(d) / q[0, 0, 0].float().square().sum()   # a score of -32
    kx[:, :, 1024:1024 + block] = -away * q[0, 0, 0].float()
    kx[:, :, 64:64 + block] = -away * q[0, -1, -1].float() * (
        q[0, 0, 0].float().square().sum() / q[0, -1, -1].float().square().sum())
    vx[:, :, 1024:1024 + block] *= 2.0 ** log_ratio
    vx[:, :, 64:64 + block] *= 2.0 ** (log_ratio // 2)
    kc, ks, k = _quantised(kx, dtype, block)
    vc, vs, v = _quantised(vx, dtype, block)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block)
    binding.check()
    _check(got, q, k, v, [L])


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
def test_scales_from_the_least_to_the_largest(dtype):
    """Blocks of 2^-100 up to values of 2^100, each looked at by a query of its own."""
    h, L, d, block = 8, 256, 64, 32
    q = _random((1, h, 1, d), 1, 2.0).to(BF16)
    kx, vx = 0.05 * _random((1, 1, L, d), 2), _random((1, 1, L, d), 3)
    vx = vx / vx.abs().amax(-1, keepdim=True)
    for i in range(h):
        at = slice(i * block, (i + 1) * block)
        kx[0, 0, at] = 150 * 8 * q[0, i, 0].float() / q[0, i, 0].float().square().sum()
        vx[0, 0, at] *= 2.0 ** (-90 + 190 * i / (h - 1))
    kc, ks, k = _quantised(kx, dtype, block)
    vc, vs, v = _quantised(vx, dtype, block)
    o, lse = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block)
    binding.check()
    ro, rl = scored.decode(q.double().cpu().numpy(), k, v, [L], 0.125)
    weight, _ = scored.decode(q.double().cpu().numpy(), k, np.abs(v), [L], 0.125)
    # scores of 150 here: five times the sums of products behind SCORE_TOL
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 10 * SCORE_TOL) * weight
    o = o.double().cpu().numpy()
    assert np.isfinite(o).all() and (np.abs(o - ro) <= tol).all(), (np.abs(o - ro) / tol).max()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= 5 * SCORE_TOL).all()


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
def test_a_key_without_values_takes_nearly_all_the_weight(dtype):
    """A first token of zero value and a score 17 above the rest: the others, each of
    weight 2^-24, make up the output."""
    h, L, d, block = 2, 4096, 64, 64
    q = _random((1, h, 1, d), 1, 0.5).to(BF16)
    kx, vx = 0.2 * _random((1, h, L, d), 2), 1024 * _random((1, h, L, d), 3)
    kx[:, :, :1] = 17 * 8 * q.float() / q.float().square().sum(-1, keepdim=True)
    vx[:, :, :1] = 0
    kc, ks, k = _quantised(kx, dtype, block)
    vc, vs, v = _quantised(vx, dtype, block)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block)
    binding.check()
    _check(got, q, k, v, [L])


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (E4M3, 128), (INT8, 64)])
@pytest.mark.parametrize("rows", [1, 16, 32])
def test_the_parts_of_a_split_cache_are_those_of_resident_warps(dtype, d, rows):
    """Two parts of d values and four more floats a row, at most, for each warp that
    228 KB of shared memory an SM have room for: two or more stages of 4 KB of keys and
    values, or three of 2 KB, a warp, and 3 KB a CTA of four."""
    fmt = {BF16: binding.CACHE_BF16, E4M3: binding.CACHE_E4M3, INT8: binding.CACHE_INT8}[dtype]
    row_bytes = d * (2 if dtype == BF16 else 1)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    need = binding.decode_scored_workspace_bytes(1, 8 * rows, 8, 1, 1 << 20, d, fmt)
    tile = 16 * row_bytes if row_bytes >= 128 else 2048   # the least
    ring = 3 * 2 * max(tile, 2048)
    fit = 228 * 1024 // (4 * ring + 3 * 1024)
    warps = sms * 4 * fit
    row_tile = 8 if rows <= 8 else (16 if rows <= 16 else 32)
    assert 0 < need <= 4 * (4 + warps * 2 * row_tile * (d + 4))
