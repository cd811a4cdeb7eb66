"""GPU parity of attention over a tree of drafted tokens (attn_decode_tree) with
the float64 reference.

Tolerances count the roundings, as for the decoding step with changed scores:
 * O: half a step of bf16 (2^-8 |O|); each probability (times the value scale of
   an 8-bit cache) rounded once to bf16, 2^-8 of that share of sum_j p_j |v_j|; and
   the scores' error below, worth as much again of the same sum;
 * scores (and LSE): fp32 products of d terms, at most (d + 8) 2^-24 of
   scale * sum |q k| <= 32 here, the cap's and the bias's own fp32 rounding
   (2^-22 of 50 and of slope * distance <= 256): together below 3e-4.
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


def _cache(B, hk, L, d, dtype, block, seed):
    """A filled cache: rows or codes, scales, and its float64 values."""
    x = _random((B, hk, L, d), seed)
    if dtype == BF16:
        c = x.to(BF16)
        return c, None, c.double().cpu().numpy()
    top = 127.0 if dtype == INT8 else 448.0
    x = (x * (top / 4)).clamp(-top, top)
    c = x.round().to(INT8) if dtype == INT8 else x.to(E4M3)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = torch.rand((B, hk, -(-L // block)), generator=g, device="cuda") * 0.02 + 0.005
    wide = c.float().cpu().double().numpy()
    return c, s, wide * np.repeat(s.cpu().double().numpy(), block, 2)[:, :, :L, None]


def _spoil(c, s, b, rows, block):
    """NaN in rows of a cache that nobody may use, and in the scales of whole blocks of them."""
    c[b, :, rows] = (float("nan") if c.dtype == BF16 else
                     torch.full((), 0x7f, dtype=torch.uint8, device="cuda").view(c.dtype))
    if s is not None:
        at = range(*rows.indices(c.shape[2]))
        if len(at):
            s[b, :, -(-at[0] // block):(at[-1] + 1) // block if at[-1] + 1 < c.shape[2] else None] \
                = float("nan")


def _parents(B, n, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "chain":
        p = np.tile(np.arange(-1, n - 1), (B, 1))
    elif kind == "star":
        p = np.tile(np.where(np.arange(n) == 0, -1, 0), (B, 1))
    elif kind == "roots":
        p = np.full((B, n), -1)
    else:
        p = np.array([[-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]
                      for _ in range(B)])
    if kind == "holes":  # places that are no node, and what hangs below them
        p[:, 1::4] = [-2, n, 7 - n, 1 << 30][seed % 4]
    return p.astype(np.int32)


def _slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def _check(got, q, kt, vt, k, v, parents, lens, scale, softcap, slopes, window):
    o, lse = (t.float().cpu().double().numpy() for t in got)
    qd, kt, vt = (t.double().cpu().numpy() for t in (q, kt, vt))
    sl = None if slopes is None else slopes.double().cpu().numpy()
    ro, rl = tree.attention(qd, kt, vt, k, v, parents, lens, scale, softcap, sl, window)
    weight, _ = tree.attention(qd, kt, np.abs(vt), k, np.abs(v), parents, lens, scale, softcap, sl,
                               window)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * SCORE_TOL) * weight + 1e-6
    assert np.isfinite(o).all()
    off = np.abs(o - ro)
    assert (off <= tol).all(), (off.max(), np.argwhere(off > tol)[:5])
    none = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), none) and (lse[none] < 0).all()
    assert (np.abs(lse[~none] - rl[~none]) <= SCORE_TOL).all(), np.abs(lse[~none] - rl[~none]).max()


CASES = [
    # B, h, h_kv, n, L_max, d, block, cap, alibi, window, tree, lens
    (1, 1, 1, 1, 1, 64, 16, 0.0, False, None, "chain", [1]),
    (3, 2, 2, 5, 77, 64, 16, 0.0, False, None, "random", [77, 0, 1]),
    (2, 4, 2, 16, 300, 64, 64, 30.0, True, None, "random", [300, 129]),
    (2, 8, 1, 7, 513, 128, 128, 50.0, False, 50, "random", [513, 17]),
    (2, 4, 2, 61, 257, 128, 32, 0.0, True, None, "holes", [257, 64]),
    (1, 4, 1, 33, 900, 32, 64, 30.0, True, 333, "chain", [899]),
    (2, 4, 1, 40, 130, 16, 16, 0.0, False, 0, "random", [130, 3]),
    (1, 6, 2, 128, 200, 64, 128, 0.0, False, None, "star", [199]),
    (1, 2, 1, 127, 70, 128, 64, 50.0, True, 20, "chain", [70]),
    (1, 8, 1, 100, 140, 32, 16, 0.0, True, 3, "random", [129]),  # many tiles of query rows
    (2, 2, 2, 65, 128, 128, 128, 0.0, False, None, "roots", [128, 127]),
    (1, 2, 1, 9, 9000, 64, 128, 0.0, True, None, "random", [8999]),  # the cache is split
    (1, 2, 2, 12, 5000, 128, 16, 30.0, False, 2100, "random", [4996]),
    (2, 2, 1, 70, 3, 64, 16, 0.0, True, 5, "chain", [3, 0]),  # a window wider than the cache
    (1, 4, 1, 16, 700, 64, 32, 0.0, True, 200, "holes", [650]),  # 64 query rows
    (2, 1, 1, 33, 400, 128, 64, 20.0, False, None, "random", [400, 260]),
    (1, 3, 1, 10, 9000, 32, 128, 0.0, False, None, "star", [8991]),
    (2, 2, 2, 32, 260, 16, 16, 0.0, True, 64, "chain", [260, 30]),
    (5, 2, 1, 3, 640, 16, 64, 0.0, False, None, "holes", [640, 1, 0, 333, 64]),
    # many query rows, biased: the cached tiles from the newest on, in runs, with windows
    (2, 8, 2, 33, 1500, 64, 32, 0.0, True, 700, "random", [1500, 901]),
    (1, 16, 2, 70, 2100, 128, 128, 30.0, True, None, "random", [2100]),
    (3, 8, 2, 20, 700, 32, 16, 20.0, True, 130, "holes", [700, 3, 0]),
    (2, 6, 2, 13, 5000, 16, 64, 0.0, True, None, "random", [5000, 2049]),
    # query rows of a key head on both sides of where the kernel changes
    (17, 4, 2, 8, 130, 128, 64, 0.0, False, None, "random", list(range(114, 131))),    # 16 rows
    (17, 2, 2, 17, 130, 128, 64, 0.0, False, None, "random", list(range(114, 131))),   # 17 of 34
    (16, 2, 2, 32, 130, 128, 64, 20.0, False, None, "random", list(range(115, 131))),  # 32 of 32
    (2, 3, 3, 33, 130, 128, 64, 0.0, False, 40, "random", [130, 128]),
    (2, 4, 2, 16, 200, 64, 32, 0.0, True, None, "holes", [200, 191]),
    (2, 3, 1, 11, 200, 64, 32, 0.0, True, None, "holes", [200, 191]),
    (2, 2, 1, 16, 200, 32, 32, 0.0, False, None, "chain", [200, 192]),
    (2, 3, 1, 11, 200, 32, 32, 0.0, False, None, "chain", [200, 192]),
    (1, 1, 1, 32, 200, 64, 32, 0.0, True, 20, "chain", [200]),
]


@TYPES
@pytest.mark.parametrize("B,h,hk,n,L,d,block,cap,alibi,window,kind,lens", CASES)
def test_decode_tree_matches_reference(dtype, B, h, hk, n, L, d, block, cap, alibi, window, kind,
                                       lens):
    q = _random((B, h, n, d), 1, 2.0).to(BF16)
    kt, vt = _random((B, hk, n, d), 8).to(BF16), _random((B, hk, n, d), 9).to(BF16)
    kc, ks, k = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, hk, L, d, dtype, block, 4)
    parents = _parents(B, n, kind)
    slopes = _slopes(h) if alibi else None
    # what nobody sees is never used: rows behind the last token, rows before every
    # window, keys and values of places that are no node
    for b, m in enumerate(lens):
        for c, s in ((kc, ks), (vc, vs)):
            _spoil(c, s, b, slice(m, L), block)
            if window is not None and m - window > 0:
                _spoil(c, s, b, slice(0, m - window), block)
        gone = torch.tensor([not x for x in tree.lineages(parents[b])], device="cuda")
        kt[b][:, gone] = vt[b][:, gone] = float("nan")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = (q, kt, vt, torch.tensor(parents, device="cuda"), kc, vc, lens_t)
    kw = dict(k_scale=ks, v_scale=vs, block_tokens=block, softcap=cap, slopes=slopes, window=window)
    got = binding.attn_decode_tree(*args, **kw)
    binding.check()
    _check(got, q, kt, vt, k, v, parents, lens, 1 / math.sqrt(d), cap, slopes, window)
    again = binding.attn_decode_tree(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # no order that changes results


@TYPES
def test_a_chain_is_the_decoding_step(dtype):
    """Over a cache that holds the nodes, attn_decode_scored gives the same answers
    to within the roundings of both (the tree's own keys are not in 8 bits, so the
    nodes' rows are values that 8 bits hold)."""
    B, h, hk, n, L, d, block = 2, 8, 2, 4, 300, 64, 64
    q = _random((B, h, n, d), 1).to(BF16)
    kc, ks, _ = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, _ = _cache(B, hk, L, d, dtype, block, 4)
    if ks is not None:
        ks[:], vs[:] = 2.0 ** -7, 2.0 ** -6
    lens = torch.tensor([300, 71], dtype=torch.int32, device="cuda")
    own = []
    for c, s in ((kc, ks), (vc, vs)):
        at = (lens[:, None] - n + torch.arange(n, device="cuda")).long()
        rows = c.float().gather(2, at[:, None, :, None].expand(B, hk, n, d))
        own.append((rows if s is None else rows * s[0, 0, 0]).to(BF16))
    parents = torch.tensor(_parents(B, n, "chain"), device="cuda")
    o, lse = binding.attn_decode_tree(q, *own, parents, kc, vc, lens - n, ks, vs, block, softcap=20.,
                                      slopes=_slopes(h), window=100)
    o2, lse2 = binding.attn_decode_scored(q, kc, vc, lens, ks, vs, block, softcap=20.,
                                          slopes=_slopes(h), window=100)
    binding.check()
    assert (lse - lse2).abs().max() <= 2 * SCORE_TOL
    # two outputs off by 2^-8 each, and two roundings of P, of values up to 5 or so
    assert (o.float() - o2.float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -8 + 2 * SCORE_TOL) * 5


@TYPES
def test_strided_views(dtype):
    """Projections packed as [B, n, heads, d], a cache kept as [B, L, h_kv, d]."""
    B, h, hk, n, L, d, block = 2, 6, 2, 21, 150, 64, 32
    x = _random((B, n, h + 2 * hk, d), 1).to(BF16)
    q, kt, vt = (t.transpose(1, 2) for t in x.split([h, hk, hk], 2))
    kc, ks, k = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, hk, L, d, dtype, block, 4)
    kc, vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc))
    parents = _parents(B, n, "random", 3)
    lens = [150, 40]
    out = torch.full((B, n, h, d), 7.0, device="cuda", dtype=BF16).transpose(1, 2)
    got = binding.attn_decode_tree(q, kt, vt, torch.tensor(parents, device="cuda"), kc, vc,
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), ks, vs,
                                   block, out=out)
    binding.check()
    assert got[0] is out
    _check(got, q, kt, vt, k, v, parents, lens, 1 / math.sqrt(d), 0.0, None, None)


@TYPES
def test_large_and_small_scores_and_scales(dtype):
    """Scores in the thousands (a softmax of one key), value scales over many powers
    of two, codes at the ends of their range."""
    B, h, n, L, d, block = 1, 2, 6, 200, 64, 16
    q = _random((B, h, n, d), 1, 400.0).to(BF16)
    kt, vt = _random((B, h, n, d), 8).to(BF16), _random((B, h, n, d), 9).to(BF16)
    kc, ks, k = _cache(B, h, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, h, L, d, dtype, block, 4)
    if ks is not None:
        power = torch.arange(ks.shape[2], device="cuda") - 6
        vs *= torch.exp2(5.0 * power)
        v = vc.float().cpu().double().numpy() * np.repeat(vs.cpu().double().numpy(), block,
                                                          2)[:, :, :L, None]
    parents = _parents(B, n, "random", 5)
    # (scores up to 400 * 64 * 4 / 8 and their fp32 sums: |s| (d + 8) 2^-24 is 0.06 of
    # a score here, so the score tolerance of the other tests does not hold)
    got = binding.attn_decode_tree(q, kt, vt, torch.tensor(parents, device="cuda"), kc, vc,
                                   k_scale=ks, v_scale=vs, block_tokens=block, scale=2.0 ** -6)
    binding.check()
    qd = q.double().cpu().numpy()
    ktd, vtd = kt.double().cpu().numpy(), vt.double().cpu().numpy()
    size = np.abs(qd).max() * 2 ** -6 * d * max(np.abs(k).max(), np.abs(ktd).max())
    slack = size * (d + 8) * 2.0 ** -24
    ro, rl = tree.attention(qd, ktd, vtd, k, v, parents, [L], 2.0 ** -6)
    weight, _ = tree.attention(qd, ktd, np.abs(vtd), k, np.abs(v), parents, [L], 2.0 ** -6)
    o, lse = (t.float().cpu().double().numpy() for t in got)
    assert (np.abs(lse - rl) <= slack + 1e-6).all()
    # (a score off by slack changes a probability by exp(2 slack) - 1 of itself)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + np.expm1(2 * slack)) * weight + 1e-6
    assert (np.abs(o - ro) <= tol).all()


def test_no_cache_lens_and_own_buffers():
    B, h, n, L, d = 2, 4, 10, 100, 64
    q, kt, vt = (_random((B, h, n, d), i).to(BF16) for i in range(3))
    kc, vc = (_random((B, h, L, d), i).to(BF16) for i in (5, 6))
    parents = torch.tensor(_parents(B, n, "random"), device="cuda")
    full = torch.full((B,), L, dtype=torch.int32, device="cuda")
    a = binding.attn_decode_tree(q, kt, vt, parents, kc, vc)
    need = max(binding.decode_tree_workspace_bytes(B, h, h, n, L, d), 16)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((B, h, n), device="cuda")
    over = full + 1000  # clamped to L
    b = binding.attn_decode_tree(q, kt, vt, parents, kc, vc, over, out=out, lse=lse, workspace=ws)
    binding.check()
    assert b[0] is out and b[1] is lse
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    under = binding.attn_decode_tree(q, kt, vt, parents, kc, vc, -full)
    none = binding.attn_decode_tree(q, kt, vt, parents, kc, vc, full * 0)
    assert all(torch.equal(x, y) for x, y in zip(under, none))


def test_rows_of_other_tensors_are_left_alone():
    """out and lse inside larger buffers: what lies around them is not written."""
    B, h, n, L, d = 2, 3, 11, 70, 64
    q, kt, vt = (_random((B, h, n, d), i).to(BF16) for i in range(3))
    kc, vc = (_random((B, h, L, d), i).to(BF16) for i in (5, 6))
    parents = torch.tensor(_parents(B, n, "random"), device="cuda")
    wide = torch.full((B, h, n + 5, d + 64), 3.0, device="cuda", dtype=BF16)
    flat = torch.full((B * h * n + 64,), 3.0, device="cuda")
    out, lse = wide[:, :, 2:2 + n, :d], flat[32:32 + B * h * n].view(B, h, n)
    binding.attn_decode_tree(q, kt, vt, parents, kc, vc, out=out, lse=lse)
    want = binding.attn_decode_tree(q, kt, vt, parents, kc, vc)
    binding.check()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out.fill_(3.0)
    lse.fill_(3.0)
    assert (wide == 3).all() and (flat == 3).all()


@TYPES
@pytest.mark.parametrize("n", [30, 4], ids=["many", "few"])
def test_captured_step_and_two_streams(dtype, n):
    """A captured call replayed on new inputs; calls of two streams at once, each
    with a workspace of its own."""
    B, h, hk, L, d, block = 2, 8, 2, 3000, 64, 64
    q = _random((B, h, n, d), 1).to(BF16)
    kt, vt = _random((B, hk, n, d), 8).to(BF16), _random((B, hk, n, d), 9).to(BF16)
    kc, ks, _ = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, _ = _cache(B, hk, L, d, dtype, block, 4)
    parents = torch.tensor(_parents(B, n, "random"), device="cuda")
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    args, kw = (kt, vt, parents, kc, vc, lens), dict(k_scale=ks, v_scale=vs, block_tokens=block)
    new = (_random((B, h, n, d), 33).to(BF16), torch.tensor([17, 2999], dtype=torch.int32,
                                                            device="cuda"))
    want = binding.attn_decode_tree(q, *args, **kw)
    want_new = binding.attn_decode_tree(new[0], kt, vt, parents, kc, vc, new[1], **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    q2, lens2 = q.clone(), lens.clone()
    with torch.cuda.stream(side):
        binding.attn_decode_tree(q2, kt, vt, parents, kc, vc, lens2, **kw)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = binding.attn_decode_tree(q2, kt, vt, parents, kc, vc, lens2, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q2.copy_(new[0])
    lens2.copy_(new[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want_new))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(8):
        res.append((binding.attn_decode_tree(q, *args, stream=a, **kw), want))
        res.append((binding.attn_decode_tree(new[0], kt, vt, parents, kc, vc, new[1], stream=b,
                                             **kw), want_new))
    torch.cuda.synchronize()
    for x, y in res:
        assert all(torch.equal(i, j) for i, j in zip(x, y))
    binding.check()


def test_refusals():
    q = torch.zeros((1, 2, 4, 64), dtype=BF16, device="cuda")
    c = torch.zeros((1, 1, 32, 64), dtype=BF16, device="cuda")
    t = torch.zeros((1, 1, 4, 64), dtype=BF16, device="cuda")
    ids = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    ok = dict(q=q, k_tree=t, v_tree=t, parents=ids, k_cache=c, v_cache=c)
    binding.attn_decode_tree(**ok)
    eight = torch.zeros((1, 1, 32, 64), dtype=INT8, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[0]), dict(k_tree=t[:, :, :3]), dict(v_tree=t.expand(1, 2, 4, 64)),
           dict(parents=ids.long()), dict(parents=ids[:, :3]), dict(parents=None),
           dict(k_cache=c.half()), dict(k_cache=c[..., :32]), dict(v_cache=c[:, :, :16]),
           dict(k_cache=eight, v_cache=eight), dict(cache_lens=ids[0]),
           dict(slopes=torch.zeros(3, device="cuda")), dict(window=-1),
           dict(out=q[:, :1]), dict(out=q.float()), dict(lse=torch.zeros(3, device="cuda")),
           dict(q=q.transpose(2, 3)), dict(parents=ids.cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            binding.attn_decode_tree(**{**ok, **change})
    many = torch.zeros((1, 2, 129, 64), dtype=BF16, device="cuda")
    few = torch.zeros((1, 2, 4, 48), dtype=BF16, device="cuda")
    for x, cc in ((many, c), (few, c[..., :48])):
        with pytest.raises(binding.AttnError) as e:
            n = x.shape[2]
            binding.attn_decode_tree(x, x[:, :1], x[:, :1],
                                     torch.zeros((1, n), dtype=torch.int32, device="cuda"), cc, cc)
        assert e.value.status == binding.ATTN_ERR_UNSUPPORTED
    odd = torch.zeros((1, 2, 4, 68), dtype=BF16, device="cuda")[..., :64]  # rows off 16 bytes
    with pytest.raises(binding.AttnError):
        binding.attn_decode_tree(**{**ok, "q": odd})
