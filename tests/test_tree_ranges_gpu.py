"""Attention over drafted trees (attn_decode_tree) where its arguments end, for few and
for many query rows of a key head: scores in the thousands, value scales over many
powers of two, caps from tiny to idle, hidden keys with anything in them, more units
of work than SMs, the largest groups of query heads.

Tolerances count roundings as in test_tree_gpu: O half a step of bf16 and each
probability rounded once to bf16, 2^-8 each; scores (and LSE) to SCORE_TOL, with the
general form of the tanh 3e-7 of the cap more, and sums of d products whose terms add
up to `size` to (d + 8) 2^-24 size.
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
TYPES = pytest.mark.parametrize("dtype", [BF16, E4M3, INT8], ids=["bf16", "e4m3", "int8"])
# query heads of one key head, nodes: 6 and 24 query rows, 70, 200
ROWS = pytest.mark.parametrize("h,n", [(1, 6), (2, 12), (1, 70), (2, 100)],
                               ids=["6", "24", "70", "200"])


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


def _cache(x, dtype, block, top=4.0):
    """Rows x (about `top` at most) as a cache: rows or codes, scales, float64 values."""
    if dtype == BF16:
        c = x.to(BF16)
        return c, None, c.double()
    most = 127.0 if dtype == INT8 else 448.0
    c = (x * (most / top)).clamp(-most, most)
    c = c.round().to(INT8) if dtype == INT8 else c.to(E4M3)
    s = torch.full((*x.shape[:2], -(-x.shape[2] // block)), top / most, device="cuda")
    return c, s, c.float().double() * s.double().repeat_interleave(block, 2)[:, :, :x.shape[2], None]


def _parents(B, n, seed=0, holes=False):
    rng = np.random.default_rng(seed)
    p = np.array([[-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]
                  for _ in range(B)], dtype=np.int32).reshape(B, n)
    if holes:
        p[:, 2::7] = -2
    return p


def _reference(q, kt, vt, k, v, parents, lens, scale, softcap=0.0, slopes=None, window=None):
    """O, LSE and sum p |v| in 64 bits, all sequences at once; NaN is not allowed."""
    B, h, n, d = q.shape
    hk, L = k.shape[1:3]
    see = torch.zeros((B, n, L + n), dtype=torch.bool)
    far = torch.zeros((B, n, L + n), dtype=torch.float64)
    for b in range(B):
        for i, line in enumerate(tree.lineages(parents[b])):
            if line:
                see[b, i, :lens[b]] = True
                far[b, i, :L] = lens[b] + len(line) - 1 - torch.arange(L)
                at = L + torch.tensor(line)
                see[b, i, at] = True
                far[b, i, at] = torch.arange(len(line) - 1, -1, -1, dtype=torch.float64)
    see, far = see.cuda()[:, None, None], far.cuda()[:, None, None]
    if window is not None:
        see = see & (far <= window)
    keys, values = (torch.cat([a, b], 2).double()[:, :, None] for a, b in ((k, kt), (v, vt)))
    x = torch.matmul(q.double().view(B, hk, h // hk, n, d), keys.transpose(-1, -2)) * scale
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
    if slopes is not None:
        x = x - slopes.double().view(1, hk, h // hk, 1, 1) * far
    x = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.where(see, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)), 0.0)
    return (torch.matmul(p, values).view(B, h, n, d), lse.view(B, h, n),
            torch.matmul(p, values.abs()).view(B, h, n, d))


def _check(got, want, tol=SCORE_TOL, extra=0.0):
    (o, lse), (ro, rl, weight) = got, want
    assert torch.isfinite(o).all()
    off = (o.double() - ro).abs()
    most = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * tol) * weight + 1e-6 + extra
    assert (off <= most).all(), (off / most).max()
    none = rl == -math.inf
    assert torch.equal(lse == -math.inf, none)
    assert ((lse.double() - rl).abs()[~none] <= tol).all(), (lse.double() - rl).abs()[~none].max()


def _run(q, kt, vt, parents, kc, vc, lens, **kw):
    got = binding.attn_decode_tree(q, kt, vt, torch.tensor(parents, device="cuda"), kc, vc,
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), **kw)
    binding.check()
    return got


def _inputs(h, n, L, d, dtype, block, std=2.0, B=1, hk=1, seed=1):
    q = _random((B, h, n, d), seed, std).to(BF16)
    own = [_random((B, hk, n, d), seed + i).to(BF16) for i in (1, 2)]
    kc, ks, k = _cache(_random((B, hk, L, d), seed + 3), dtype, block)
    vc, vs, v = _cache(_random((B, hk, L, d), seed + 4), dtype, block)
    return q, own, (kc, vc), (ks, vs), (k, v)


def _slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


@TYPES
@ROWS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [200, 6000])
def test_large_scores_and_scales_of_many_powers(dtype, h, n, d, L):
    """Scores in the thousands (a softmax of one key, whose place changes from tile to
    tile), value scales from 2^-30 to 2^30.  Probabilities times value scales in f16 (few
    rows) are off by half a step of its subnormal numbers at least, 2^-25 where a row's
    largest is 2^7 or more: `extra`."""
    block = 16
    q, own, caches, (ks, vs), (k, v) = _inputs(h, n, L, d, dtype, block, 400.0)
    if ks is not None:
        power = 5.0 * (torch.arange(vs.shape[2], device="cuda") % 13 - 6)
        vs *= torch.exp2(power)
        v *= torch.exp2(power).double().repeat_interleave(block)[:L, None]
    parents, scale = _parents(1, n), 2.0 ** -6
    got = _run(q, *own, parents, *caches, [L], k_scale=ks, v_scale=vs, block_tokens=block,
               scale=scale)
    keys = torch.cat([k, own[0].double()], 2)
    size = scale * torch.matmul(q.double().abs(), keys.abs().transpose(-1, -2)).max().item()
    tol = SCORE_TOL + (d + 8) * 2.0 ** -24 * size
    want, extra = _reference(q, *own, k, v, parents, [L], scale), 0.0
    if ks is not None:
        s = torch.matmul(q.double(), k.transpose(-1, -2)) * scale
        p = torch.exp(s - want[1][..., None].clamp(min=-1e300))
        most = (p * vs.double().repeat_interleave(block, 2)[:, :, None, :L]).amax(-1, keepdim=True)
        extra = 2.0 ** -32 * most * caches[1].float().double().abs().sum(2, keepdim=True)
    _check(got, want, math.expm1(2 * tol) / 2, extra)


@TYPES
@ROWS
@pytest.mark.parametrize("alibi", [False, True], ids=["plain", "alibi"])
@pytest.mark.parametrize("cap", [1e-6, 0.01, 1.0, 300.0, 1e9, 2.0 ** 64])
def test_caps_from_tiny_to_idle(dtype, h, n, cap, alibi):
    d, L, block = 64, 330, 64
    q, own, caches, (ks, vs), (k, v) = _inputs(h, n, L, d, dtype, block)
    slopes, parents = _slopes(h) if alibi else None, _parents(1, n, 2, holes=True)
    got = _run(q, *own, parents, *caches, [L - 9], k_scale=ks, v_scale=vs, block_tokens=block,
               softcap=cap, slopes=slopes)
    _check(got, _reference(q, *own, k, v, parents, [L - 9], 0.125, cap, slopes))


@TYPES
@ROWS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("alibi", [False, True], ids=["plain", "alibi"])
@pytest.mark.parametrize("sign", [1.0, -1.0], ids=["above", "below"])
def test_scores_past_the_polynomials(dtype, h, n, d, alibi, sign):
    """Under a wide cap one cached key, and one node's, of 0.6 caps among ordinary ones."""
    L, block, cap = 330, 16, 300.0
    q = (_random((1, h, n, d), 1) * 0.05 + 2.0).to(BF16)
    kt, vt = (_random((1, 1, n, d), i).to(BF16) for i in (2, 3))
    x = _random((1, 1, L, d), 4)
    x[:, :, 130] = sign * 0.3 * cap / math.sqrt(d)
    kt[:, :, n // 3] = sign * 0.3 * cap / math.sqrt(d)
    kc, ks, k = _cache(x, dtype, block, 0.3 * cap / math.sqrt(d))
    vc, vs, v = _cache(_random((1, 1, L, d), 5), dtype, block)
    slopes, parents = _slopes(h) if alibi else None, _parents(1, n, 2)
    scale = 1 / math.sqrt(d)
    s = torch.matmul(q.double(), k.transpose(-1, -2)) * scale
    assert (s[..., 130].abs() > 0.3 * cap).all() and (s[..., 131:].abs() < 0.3 * cap).all()
    got = _run(q, kt, vt, parents, kc, vc, [L], k_scale=ks, v_scale=vs, block_tokens=block,
               softcap=cap, slopes=slopes)
    tol = SCORE_TOL + 3e-7 * cap + (d + 8) * 2.0 ** -24 * cap
    _check(got, _reference(q, kt, vt, k, v, parents, [L], scale, cap, slopes), tol)


@TYPES
@ROWS
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("window", [None, 150])
def test_what_nobody_sees_changes_no_bit_under_a_cap(dtype, h, n, d, window):
    """Cache rows behind the last token and before every window, keys, values and queries
    of places that are no node: zeros, or large."""
    L, block, lens, cap = 700, 16, [500, 3], 100.0
    q, own, caches, (ks, vs), _ = _inputs(h, n, L, d, dtype, block, B=2)
    parents = _parents(2, n, 2, holes=True)
    gone = torch.tensor([[not x for x in tree.lineages(parents[b])] for b in range(2)], device="cuda")
    hidden = torch.zeros((2, L), dtype=torch.bool, device="cuda")
    for b, m in enumerate(lens):
        hidden[b, m:] = True
        if window is not None:
            hidden[b, :max(0, m - window)] = True
    res = []
    for large in (0.0, 1.0, 0.0):
        kc, vc, kt, vt, qq = (t.clone() for t in (*caches, *own, q))
        for b in range(2):
            for t, fill in ((kc, 3e4), (vc, 3e4)):
                if dtype == BF16:
                    t[b, :, hidden[b]] = fill * large
                else:  # 96 and 112, the same byte of a code as for e4m3 numbers
                    t.view(torch.uint8)[b, :, hidden[b]] = 0x70 if large else 0
            for t in (kt, vt, qq):
                t[b, :, gone[b]] = 3e4 * large
        if large:  # what an earlier call left in shared memory
            _run(qq, kt, vt, parents, torch.full_like(kc, 100.0) if dtype != E4M3 else kc, vc,
                 [L, L], k_scale=ks, v_scale=vs, block_tokens=block, softcap=cap)
        res.append(_run(qq, kt, vt, parents, kc, vc, lens, k_scale=ks, v_scale=vs,
                        block_tokens=block, softcap=cap, window=window))
    for other in res[1:]:
        assert torch.equal(res[0][0], other[0]) and torch.equal(res[0][1], other[1])


UNITS = [
    # B, h, h_kv, n, L_max, d, window, lens.  Sequences x key heads (x blocks of 256 query
    # rows) past 152 and 304.
    (40, 8, 8, 40, 300, 64, None, (0, 300)),       # 320 units of 40 rows, whole
    (40, 16, 8, 50, 300, 128, None, (0, 300)),     # of 100
    (20, 32, 8, 50, 300, 64, None, (0, 300)),      # of 200
    (40, 12, 4, 100, 260, 128, None, (0, 260)),    # 300 rows: blocks of 256 and of 44 in turn
    (40, 12, 4, 100, 500, 32, None, (0, 500)),
    (64, 8, 8, 40, 3000, 64, None, (0, 200)),      # runs of many short units
    (64, 16, 8, 50, 3000, 128, None, (0, 500)),
    (48, 12, 4, 100, 3000, 128, None, (0, 300)),
    (24, 32, 4, 41, 3000, 128, None, (0, 3000)),   # 328 rows, short and long ones
    (24, 32, 8, 40, 3000, 64, 300, (0, 3000)),
    (24, 32, 8, 40, 3000, 16, None, (0, 3000)),
    (100, 8, 8, 4, 3000, 64, None, (0, 600)),      # few rows
    (100, 16, 8, 4, 400, 128, 100, (0, 400)),
]


@TYPES
@pytest.mark.parametrize("B,h,hk,n,L,d,window,lens", UNITS)
@pytest.mark.parametrize("changed", [False, True], ids=["plain", "cap+alibi"])
def test_more_units_than_sms(dtype, B, h, hk, n, L, d, window, lens, changed):
    block = 32
    q, own, caches, (ks, vs), (k, v) = _inputs(h, n, L, d, dtype, block, B=B, hk=hk)
    rng = np.random.default_rng(B + n)
    lens = [int(x) for x in rng.integers(lens[0], lens[1] + 1, B)]
    lens[3], lens[-1] = 0, 1
    parents = _parents(B, n, 7, holes=True)
    kw = dict(softcap=20.0, slopes=_slopes(h)) if changed else {}
    got = _run(q, *own, parents, *caches, lens, k_scale=ks, v_scale=vs, block_tokens=block,
               window=window, **kw)
    for b0 in range(0, B, 10):  # (a few at a time: 64-bit scores are large)
        at = slice(b0, b0 + 10)
        want = _reference(q[at], own[0][at], own[1][at], k[at], v[at], parents[at], lens[at],
                          1 / math.sqrt(d), window=window, **kw)
        _check((got[0][at], got[1][at]), want)
    again = _run(q, *own, parents, *caches, lens, k_scale=ks, v_scale=vs, block_tokens=block,
                 window=window, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("h,n", [(69798, 63), (131072, 127), (131072, 128), (4200000, 3)])
def test_the_largest_groups_of_query_heads(h, n):
    """Millions of query rows of one key head, packed as projections are, so that a row of
    another head or node is another address: against 256 heads at a time (whole blocks of
    256 rows, so that rows have the same bits)."""
    L, d = 20, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, n, h + 2, d), generator=g, device="cuda", dtype=BF16)
    q, kt, vt = (t.transpose(1, 2) for t in x.split([h, 1, 1], 2))
    kc, vc = (torch.randn((1, 1, L, d), generator=g, device="cuda", dtype=BF16) for _ in "kv")
    parents = _parents(1, n, 4, holes=True)
    o, lse = _run(q, kt, vt, parents, kc, vc, [L])
    for at in (0, h // 2, 4 * h // 5, h - 256):
        part = q[:, at:at + 256].contiguous()
        want = _run(part, kt, vt, parents, kc, vc, [L])
        assert torch.equal(o[:, at:at + 256], want[0]) and torch.equal(lse[:, at:at + 256], want[1])
    last = slice(h - 3, h)
    _check((o[:, last], lse[:, last]), _reference(q[:, last], kt, vt, kc, vc, parents, [L], 0.25))
