"""NaN and infinities that nodes of a drafted tree see (attn_decode_tree): a NaN
among what a node sees is in its output and its LSE, whichever kernel takes the call
and however the keys are split, and in nobody else's; a score of -inf weighs
nothing.  Every 8-bit code enters both products exactly.

Tolerances: O half a step of bf16 (2^-8 |O|), each probability rounded to bf16 once
(2^-8 of that share of sum p |v|), scores to 3e-4 as in test_tree_gpu; where a test
says so outputs have the same bits.
"""
import math

import numpy as np
import pytest
import torch

from oracle import tree
from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu

SCORE_TOL = 3e-4
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16

# B, h, h_kv, n, L_max, d.  Few query rows of a key head (up to 16, or 32), and many:
# up to 64 (twice in a tile), up to 128, up to 256; keys whole and in parts.
SHAPES = pytest.mark.parametrize("B,h,hk,n,L,d", [
    (2, 2, 1, 5, 60, 64), (1, 2, 1, 6, 9000, 64), (48, 8, 8, 4, 1000, 16), (1, 2, 1, 16, 3000, 64),
    (160, 4, 4, 3, 200, 32), (2, 1, 1, 40, 200, 64), (1, 1, 1, 40, 5000, 64),
    (2, 2, 1, 40, 200, 128), (1, 2, 1, 40, 5000, 32), (1, 2, 1, 100, 200, 128),
    (1, 2, 1, 100, 5000, 64)])


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


def _case(B, h, hk, n, L, d, seed=1):
    q = _random((B, h, n, d), seed).to(BF16)
    own = [_random((B, hk, n, d), seed + i).to(BF16) for i in (1, 2)]
    cache = [_random((B, hk, L, d), seed + i).to(BF16) for i in (3, 4)]
    rng = np.random.default_rng(seed)
    parents = np.array([[-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]
                        for _ in range(B)], dtype=np.int32).reshape(B, n)
    return q, own, cache, parents


def _run(q, own, cache, parents, lens=None, **kw):
    got = binding.attn_decode_tree(q, *own, torch.tensor(parents, device="cuda"), *cache, lens, **kw)
    binding.check()
    return got


def _same(a, b, at):
    """The rows (and columns) `at` of two results are the same bits."""
    return torch.equal(a[at].contiguous().view(torch.int16 if a.dtype == BF16 else torch.int32),
                       b[at].contiguous().view(torch.int16 if b.dtype == BF16 else torch.int32))


def _against_reference(got, q, own, cache, parents, lens, softcap=0.0):
    f = [t.double().cpu().numpy() for t in (q, *own, *cache)]
    with np.errstate(invalid="ignore"):
        ro, rl = tree.attention(*f, parents, lens, 1 / math.sqrt(q.shape[3]), softcap)
        f[2], f[4] = np.abs(f[2]), np.abs(f[4])
        weight, _ = tree.attention(*f, parents, lens, 1 / math.sqrt(q.shape[3]), softcap)
    o, lse = (t.double().cpu().numpy() for t in got)
    assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * SCORE_TOL) * weight + 1e-6).all()
    none = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), none) and (lse[none] < 0).all()
    assert (np.abs(lse[~none] - rl[~none]) <= SCORE_TOL).all()


@SHAPES
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_nan_in_a_cached_key_is_seen(B, h, hk, n, L, d, cap):
    q, own, (k, v), parents = _case(B, h, hk, n, L, d)
    clean = _run(q, own, (k, v), parents, softcap=cap)
    group = h // hk
    for at in (0, L // 2, L - 1, slice(0, L)):
        bad = k.clone()
        bad[0, 0, at, 3] = math.nan
        o, lse = _run(q, own, (bad, v), parents, softcap=cap)
        assert torch.isnan(o[0, :group]).all() and torch.isnan(lse[0, :group]).all(), at
        o[0, :group], lse[0, :group] = clean[0][0, :group], clean[1][0, :group]
        assert _same(o, clean[0], slice(None)) and _same(lse, clean[1], slice(None)), at


@SHAPES
def test_nan_in_a_cached_value_is_seen(B, h, hk, n, L, d):
    q, own, (k, v), parents = _case(B, h, hk, n, L, d)
    clean = _run(q, own, (k, v), parents)
    for at in (0, L - 1):
        bad = v.clone()
        bad[0, 0, at, 5] = math.nan
        o, lse = _run(q, own, (k, bad), parents)
        assert torch.isnan(o[0, :h // hk, :, 5]).all() and _same(lse, clean[1], slice(None))
        o[0, :h // hk, :, 5] = clean[0][0, :h // hk, :, 5]
        assert _same(o, clean[0], slice(None))


@SHAPES
@pytest.mark.parametrize("slopes", [False, True])
def test_nan_in_a_nodes_key_is_its_descendants(B, h, hk, n, L, d, slopes):
    q, (kt, vt), cache, parents = _case(B, h, hk, n, L, d)
    kw = dict(slopes=torch.full((h,), 0.125, device="cuda") if slopes else None)
    clean = _run(q, (kt, vt), cache, parents, **kw)
    lines = tree.lineages(parents[0])
    for node in (0, n // 2, n - 1):
        bad = kt.clone()
        bad[0, 0, node, 1] = math.nan
        o, lse = _run(q, (bad, vt), cache, parents, **kw)
        sees = torch.tensor([node in line for line in lines], device="cuda")
        assert torch.isnan(o[0, :h // hk, sees]).all() and torch.isnan(lse[0, :h // hk, sees]).all()
        o[0, :h // hk, sees] = clean[0][0, :h // hk, sees]
        lse[0, :h // hk, sees] = clean[1][0, :h // hk, sees]
        assert _same(o, clean[0], slice(None)) and _same(lse, clean[1], slice(None)), node


@SHAPES
def test_nan_in_a_query_is_its_own(B, h, hk, n, L, d):
    q, own, cache, parents = _case(B, h, hk, n, L, d)
    clean = _run(q, own, cache, parents)
    bad = q.clone()
    bad[0, 0, n - 1, 2] = math.nan
    o, lse = _run(bad, own, cache, parents)
    assert torch.isnan(o[0, 0, n - 1]).all() and torch.isnan(lse[0, 0, n - 1])
    o[0, 0, n - 1], lse[0, 0, n - 1] = clean[0][0, 0, n - 1], clean[1][0, 0, n - 1]
    assert _same(o, clean[0], slice(None)) and _same(lse, clean[1], slice(None))


@SHAPES
def test_infinite_scores(B, h, hk, n, L, d):
    """+inf has no softmax (NaN) but under a cap; -inf weighs nothing."""
    if B > 2:
        B = 2
    q, (kt, vt), (k, v), parents = _case(B, h, hk, n, L, d)
    q[..., 0] = 1.0
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    up, down = k.clone(), k.clone()
    up[0, 0, L // 3, 0], down[0, 0, L // 3, 0] = math.inf, -math.inf
    o, lse = _run(q, (kt, vt), (up, v), parents, lens)
    assert torch.isnan(o[0, :h // hk]).all() and torch.isnan(lse[0, :h // hk]).all()
    got = _run(q, (kt, vt), (up, v), parents, lens, softcap=20.0)
    _against_reference(got, q, (kt, vt), (up, v), parents, [L] * B, 20.0)
    got = _run(q, (kt, vt), (down, v), parents, lens)
    _against_reference(got, q, (kt, vt), (down, v), parents, [L] * B)
    # a node's own key, with a cache and without: all that a root sees then
    kt[0, 0, 0, 0] = kt[0, 0, n // 2, 0] = -math.inf
    for m in (L, 1, 0):
        lens.fill_(m)
        got = _run(q, (kt, vt), (k, v), parents, lens)
        _against_reference(got, q, (kt, vt), (k, v), parents, [m] * B)
    assert (got[0][0, 0, 0] == 0).all() and got[1][0, 0, 0] == -math.inf


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [16, 40, 128], ids=["few", "many", "most"])
def test_every_code_enters_exactly(dtype, d, n):
    """One cached token a sequence, with scale 1, and nodes' own keys that weigh nothing: O
    is the token's value codes, exactly, and node i, whose query is the unit vector
    i mod d, has its i-th key code for LSE: four fp32 roundings of it (2^-22), and what
    the exponential of a number near 0 and the logarithm of one near 1 are off by, 2^-22
    and 2^-21.4 in steps of log2 (2^-21 together)."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(dtype)
    value = codes.float()
    finite = torch.isfinite(value)
    order = torch.cat([torch.nonzero(finite)[:, 0], torch.nonzero(~finite)[:, 0]])
    rows = -(-int(finite.sum()) // d)
    use = torch.zeros((rows + 1) * d, dtype=torch.long, device="cuda")  # (code 0: the number 0)
    use[:int(finite.sum())] = order[:int(finite.sum())]
    if int(finite.sum()) < 256:  # codes of NaN in a sequence of their own
        use[rows * d:rows * d + 2] = order[int(finite.sum()):]
    B = rows + 1
    grid = codes.view(torch.uint8)[use].view(dtype).view(B, 1, 1, d)
    cache = torch.zeros((B, 1, 100, d), dtype=torch.uint8, device="cuda").view(dtype)
    cache.view(torch.uint8).fill_(0x7f)  # behind the token: NaN, or 127
    cache[:, :, :1] = grid
    ones = torch.ones((B, 1, 7), device="cuda")
    q = torch.eye(d, device="cuda").repeat(-(-n // d), 1)[:n].expand(B, 1, n, d).to(BF16).contiguous()
    kt = torch.full((B, 1, n, d), -4096.0, device="cuda", dtype=BF16)
    vt = torch.ones((B, 1, n, d), device="cuda", dtype=BF16)
    parents = np.full((B, n), -1, dtype=np.int32)
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    plain = torch.zeros_like(cache)
    plain[:, :, :1] = torch.ones((), device="cuda").to(dtype)
    kw = dict(k_scale=ones, v_scale=ones, block_tokens=16, scale=1.0)
    o, _ = _run(q, (kt, vt), (plain, cache), parents, lens, **kw)
    want = grid.float().expand(B, 1, n, d)
    gone = torch.isnan(want)
    assert torch.equal(torch.isnan(o), gone)
    assert torch.equal(o.float()[~gone], want[~gone])
    _, lse = _run(q, (kt, vt), (cache, plain), parents, lens, **kw)
    want = grid.float().view(B, 1, d).repeat(1, 1, -(-n // d))[:, :, :n]
    gone = torch.isnan(want).any(-1, keepdim=True).expand_as(want)  # (NaN times 0 too)
    assert torch.equal(torch.isnan(lse), gone)
    assert ((lse - want).abs()[~gone] <= 2.0 ** -22 * want.abs()[~gone] + 2.0 ** -21).all()
