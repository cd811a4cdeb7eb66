"""GPU parity of the verification of drafted trees (attn_tree_verify) and of the
append of the accepted path (attn_cache_append_tree), and a run of the whole step.

Whole numbers have to be equal, but next to a border: a remaining probability is
rounded to fp32 once (2^-24 of itself), so sums and borders between next tokens
are known to 2^-23 of the total, tests of a node to 2^-22 of what is compared.
"""
import math

import numpy as np
import pytest
import torch

from oracle import tree
from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu

E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from transformer_head_scaled_gb300.build import build
    build()
    return binding.load()


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _case(B, n, V, dtype, with_draft, seed, sharp=3.0, noise=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((B, n, V), generator=g, device="cuda") * sharp
    p = torch.softmax(z, -1).to(dtype)
    q = torch.softmax(z + noise * torch.randn((B, n, V), generator=g, device="cuda"), -1).to(dtype)
    parents = np.array([[-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
                        for _ in range(B)], dtype=np.int32)
    rows = q.float()[torch.arange(B)[:, None], torch.tensor(parents).clamp(min=0)].view(B * n, V)
    tokens = torch.multinomial(rows, 1, generator=g).view(B, n).to(torch.int32)
    u = torch.rand((B, n), generator=g, device="cuda")
    return p, q if with_draft else None, tokens, parents, u


def _check(got, p, q, tokens, parents, u):
    path, lens, token = (t.cpu().numpy() for t in got)
    n, far = p.shape[1], 0
    for b in range(p.shape[0]):
        want, r, margin = tree.verify(p[b].double().cpu().numpy(), tokens[b].cpu().numpy(),
                                      parents[b], u[b].cpu().numpy(),
                                      None if q is None else q[b].double().cpu().numpy())
        if margin < 2.0 ** -22:
            continue  # too near to a border to say
        far += 1
        assert lens[b] == len(want), b
        assert path[b].tolist() == want + [-1] * (n - len(want)), b
        assert int(token[b]) in tree.next_tokens(r, float(u[b, 0]), 2.0 ** -23), b
    assert far >= p.shape[0] - 1


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "none"])
@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (3, 2, 2), (40, 6, 5), (2, 17, 1000), (9, 33, 513),
                                   (2, 128, 777), (1, 5, 50001), (1, 9, 140000), (30, 12, 16384),
                                   (400, 4, 100)])
def test_verify_matches_reference(B, n, V, dtype, with_draft):
    p, q, tokens, parents, u = _case(B, n, V, dtype, with_draft, 7)
    got = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=q)
    _check(got, p, q, tokens, parents, u)
    again = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=q)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("noise", [0.0, 0.05, 3.0])
def test_drafts_near_and_far_from_the_target(noise):
    """A draft equal to the target (everything stands), one near it (little is left
    after a rejection), one far from it (many rejections at a node)."""
    p, q, tokens, _, u = _case(60, 24, 400, torch.float32, True, 11, noise=noise)
    parents = np.tile(np.where(np.arange(24) == 0, -1, (np.arange(24) - 1) // 8), (60, 1))
    rows = q[torch.arange(60)[:, None], torch.tensor(parents).clamp(min=0)].view(-1, 400)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.multinomial(rows, 1, generator=g).view(60, 24).to(torch.int32)
    got = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=q)
    _check(got, p, q, tokens, parents, u)
    if noise == 0.0:
        assert (got[0][:, 1] == 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(5, 30001), (2, 131072), (1, 300007), (1, 500000), (1, 4500000)])
def test_many_rejections_over_large_rows(B, V, dtype):
    """Rows that shared memory holds, holds in part, and segments of several blocks."""
    p, q, _, _, u = _case(B, 2, V, dtype, True, 5, noise=4.0)
    n = 9
    p, q = (x[:, [0, 1] + [1] * (n - 2)].contiguous() for x in (p, q))
    g = torch.Generator(device="cuda").manual_seed(4)
    cum = q[:, 0].double().cumsum(-1)  # (multinomial takes 2^24 values at most)
    tokens = torch.searchsorted(cum, torch.rand((B, n), generator=g, device="cuda",
                                                dtype=torch.float64) * cum[:, -1:])
    tokens = tokens.clamp(max=V - 1).to(torch.int32)
    u = torch.rand((B, n), generator=g, device="cuda") * 0.5 + 0.5
    parents = np.tile(np.where(np.arange(n) == 0, -1, 0), (B, 1))
    got = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=q)
    _check(got, p, q, tokens, parents, u)
    got = binding.attn_tree_verify(p, tokens, _int(parents), u)
    _check(got, p, None, tokens, parents, u)


def _one(p, tokens, parents, u, q=None):
    """A single sequence of exactly held numbers."""
    p = torch.tensor([p], device="cuda", dtype=torch.float32)
    q = None if q is None else torch.tensor([q], device="cuda", dtype=torch.float32)
    got = binding.attn_tree_verify(p, _int([tokens]), _int([parents]),
                                   torch.tensor([u], device="cuda"), draft=q)
    path, lens, token = (t.cpu().tolist() for t in got)
    return path[0], lens[0], token[0]


def test_borders():
    p, q = [0.25, 0.5, 0.25, 0.0], [0.5, 0.25, 0.25, 0.0]
    for u1, stands in ((0.5, False), (0.49999997, True), (0.0, True)):  # u q < p, not <=
        path, lens, _ = _one([p, p], [0, 0], [-1, 0], [0.0, u1], [q, q])
        assert lens == (2 if stands else 1) and path == [0, 1 if stands else -1]
    # what is left after a rejection of token 0 is token 1 alone
    for u0 in (0.0, 0.5, 0.99999994):
        assert _one([p, p], [0, 0], [-1, 0], [u0, 0.9], [q, q])[2] == 1
    # the next token: the lowest whose running sum exceeds u
    for u0, want in ((0.0, 0), (0.25, 1), (0.24999999, 0), (0.75, 2), (0.74999994, 1),
                     (0.99999994, 2), (1.0, 2), (-1.0, 0), (math.nan, 0), (1e-40, 0)):
        assert _one([p], [0], [-1], [u0])[2] == want, u0
    # a token of no probability never stands, one outside the vocabulary neither
    for x in (3, -1, 4, 1 << 30):
        assert _one([p, p], [0, x], [-1, 0], [0.0, 0.0])[:2] == ([0, -1], 1)
        assert _one([p, p], [0, x], [-1, 0], [0.0, 0.0], [q, q])[:2] == ([0, -1], 1)
    # without a draft: the second child is tested against what the first has left
    assert _one([p] * 3, [0, 1, 0], [-1, 0, 0], [0.0, 0.5, 0.4999])[:2] == ([0, 2, -1], 2)
    assert _one([p] * 3, [0, 1, 0], [-1, 0, 0], [0.0, 0.5, 0.5])[:2] == ([0, -1, -1], 1)
    # the same token again has nothing left, and is taken off once
    assert _one([p] * 4, [0, 1, 1, 1], [-1, 0, 0, 0], [0.5, 0.9, 0.0, 0.0]) == ([0, -1, -1, -1], 1, 2)


def test_nothing_left():
    zero, p = [0.0] * 4, [0.5, 0.5, 0.0, 0.0]
    assert _one([zero], [0], [-1], [0.5])[2] == -1
    assert _one([[math.nan] * 4], [0], [-1], [0.5])[2] == -1
    assert _one([[math.nan, 0.5, 0.5, 0.0]], [0], [-1], [0.6])[2] == 2
    # the draft's row covers the target's: the next token comes from the target's own
    big = [0.75, 0.5, 0.0, 0.0]
    assert _one([p, p], [0, 0], [-1, 0], [0.7, 0.9], [big, big])[2] == 1
    # the only token was rejected: from the target's own again
    only = [0.0, 0.5, 0.0, 0.0]
    assert _one([only, only], [0, 1], [-1, 0], [0.7, 0.9]) == ([0, -1], 1, 1)


def test_places_that_are_no_node():
    p = [1.0, 0.0]
    for bad in (-1, -2, 1, 2, 99, -(1 << 31)):
        assert _one([p] * 3, [0, 0, 0], [-1, bad, 1], [0.0, 0.0, 0.0])[:2] == ([0, -1, -1], 1)
    assert _one([p] * 3, [0, 0, 0], [77, 0, 1], [0.0, 0.0, 0.0])[:2] == ([0, 1, 2], 3)


@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
def test_strides(dtype):
    """Rows inside a wider, padded vocabulary and a shared draft (stride 0), off 16 bytes too."""
    p, q, tokens, parents, u = _case(5, 7, 1021, dtype, True, 3)
    want = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=q)
    for pad in (1, 3, 1027):
        wide = torch.full((5, 9, 1021 + pad), 1.0, device="cuda", dtype=dtype)
        wide[:, 1:8, :1021] = p
        wq = torch.full((5, 7, 2048), 1.0, device="cuda", dtype=dtype)
        wq[:, :, 5:1026] = q
        got = binding.attn_tree_verify(wide[:, 1:8, :1021], tokens, _int(parents), u,
                                       draft=wq[:, :, 5:1026])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), pad
    same = q[:1].expand(5, 7, 1021)
    a = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=same)
    b = binding.attn_tree_verify(p, tokens, _int(parents), u, draft=same.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_kept_tokens_are_distributed_as_the_target():
    """200000 sequences over 5 tokens: the first token behind the root has the
    target's probabilities to five standard deviations of its count."""
    B, n, V = 200000, 4, 5
    p = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05], device="cuda")
    q = torch.tensor([0.1, 0.15, 0.2, 0.25, 0.3], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.multinomial(q.expand(B, V), n, replacement=True, generator=g).to(torch.int32)
    parents = _int([-1, 0, 0, 0]).expand(B, n).contiguous()
    u = torch.rand((B, n), generator=g, device="cuda")
    for draft in (q.expand(B, n, V), None):
        if draft is None:
            tokens = _int([0, 4, 1, 2]).expand(B, n).contiguous()
        path, lens, token = binding.attn_tree_verify(p.expand(B, n, V), tokens, parents, u,
                                                     draft=draft)
        kept = tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0]
        first = torch.where(lens > 1, kept, token)
        count = torch.bincount(first.long(), minlength=V).double().cpu()
        pd = p.double().cpu()
        assert ((count - B * pd).abs() <= 5 * (B * pd * (1 - pd)).sqrt()).all(), count / B


def test_verify_captured():
    p, q, tokens, parents, u = _case(6, 9, 3000, torch.float32, True, 5)
    p2, q2, tokens2, parents2, u2 = _case(6, 9, 3000, torch.float32, True, 6)
    want = binding.attn_tree_verify(p2, tokens2, _int(parents2), u2, draft=q2)
    ids = _int(parents)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = binding.attn_tree_verify(p, tokens, ids, u, draft=q)
    for a, b in ((p, p2), (q, q2), (tokens, tokens2), (ids, _int(parents2)), (u, u2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_verify_on_two_streams():
    """Calls of two streams at once, of clusters of 16 CTAs and of one."""
    cases = [_case(1, 9, 140000, torch.float32, True, 2), _case(300, 9, 900, BF16, False, 3)]
    calls = [(p, tokens, _int(parents), u, q) for p, q, tokens, parents, u in cases]
    want = [binding.attn_tree_verify(*c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [(i, binding.attn_tree_verify(*calls[i], stream=streams[i])) for _ in range(8)
           for i in (0, 1)]
    torch.cuda.synchronize()
    for i, res in got:
        assert all(torch.equal(a, b) for a, b in zip(res, want[i]))


def test_verify_refusals():
    p = torch.full((2, 3, 8), 0.125, device="cuda")
    ids, u = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.zeros((2, 3), device="cuda")
    ok = dict(target=p, tokens=ids, parents=ids, uniforms=u, draft=p)
    binding.attn_tree_verify(**ok)
    for change in (dict(target=p.double()), dict(target=p[0]), dict(draft=p.to(BF16)),
                   dict(draft=p[:, :2]), dict(draft=p.cpu()), dict(tokens=ids.long()),
                   dict(tokens=ids[:1]), dict(parents=None), dict(uniforms=u.to(BF16)),
                   dict(path=ids[:, :2]), dict(path_lens=u[:, 0]), dict(next_tokens=ids),
                   dict(target=p.transpose(1, 2), draft=None)):
        with pytest.raises(ValueError):
            binding.attn_tree_verify(**{**ok, **change})
    wide = torch.zeros((1, 129, 8), device="cuda")
    ids, u = (torch.zeros((1, 129), dtype=t, device="cuda") for t in (torch.int32, torch.float32))
    with pytest.raises(binding.AttnError) as e:
        binding.attn_tree_verify(wide, ids, ids, u)
    assert e.value.status == binding.ATTN_ERR_UNSUPPORTED


# ---------------------------------------------------------------- the accepted path

def _tree_rows(layers, B, h, n, d, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((layers, B, h, n, d), generator=g, device="cuda") * std).to(BF16)


def _cache(layers, B, h, L, d, dtype, block, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((layers, B, h, L, d), generator=g, device="cuda")
    if dtype == BF16:
        return x.to(BF16), None
    top = 127.0 if dtype == INT8 else 448.0
    x = (x * (top / 4)).clamp(-top, top)
    c = x.round().to(INT8) if dtype == INT8 else x.to(E4M3)
    s = torch.rand((layers, B, h, -(-L // block)), generator=g, device="cuda") * 0.02 + 0.005
    return c, s


def _paths(B, n, seed):
    rng = np.random.default_rng(seed)
    path = np.full((B, n), -1, dtype=np.int32)
    lens = np.zeros(B, dtype=np.int32)
    for b in range(B):
        nodes = [0] + [i for i in range(1, n) if rng.random() < 0.4]
        path[b, :len(nodes)] = nodes
        lens[b] = rng.integers(1, len(nodes) + 1)
    return path, lens


def _same(cache, scale, want, want_scale):
    assert np.array_equal(cache.float().cpu().double().numpy(), want)
    if scale is not None:
        assert np.array_equal(scale.cpu().numpy(), want_scale)


APPENDS = [
    # layers, B, h, n, L, d, block, lens
    (1, 1, 1, 1, 1, 64, 16, [0]),
    (2, 3, 2, 7, 64, 64, 16, [0, 15, 60]),       # the last one does not fit whole
    (3, 2, 5, 13, 100, 32, 32, [31, 97]),
    (1, 2, 4, 40, 300, 128, 64, [250, 63]),
    (2, 4, 1, 128, 200, 16, 128, [0, 72, 199, 200]),
    (5, 2, 3, 33, 129, 128, 16, [-4, 300]),      # lengths are clamped
]


@pytest.mark.parametrize("dtype", [BF16, E4M3, INT8], ids=["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("layers,B,h,n,L,d,block,lens", APPENDS)
def test_append_path_matches_reference(dtype, layers, B, h, n, L, d, block, lens):
    kt, vt = _tree_rows(layers, B, h, n, d, 1), _tree_rows(layers, B, h, n, d, 2, 9.0)
    kc, ks = _cache(layers, B, h, L, d, dtype, block, 3)
    vc, vs = _cache(layers, B, h, L, d, dtype, block, 4)
    path, path_lens = _paths(B, n, 5)
    want = []
    for c, s, t in ((kc, ks, kt), (vc, vs, vt)):
        w = c.float().cpu().double().numpy()
        ws = None if s is None else s.cpu().numpy().copy()
        tree.append_path(w, ws, t.double().cpu().numpy(), path, path_lens, lens, block,
                         dtype == INT8)
        want.append((w, ws))
    binding.attn_cache_append_tree(kt, vt, _int(path), _int(path_lens), kc, vc, _int(lens), ks, vs,
                                   block)
    binding.check()
    _same(kc, ks, *want[0])
    _same(vc, vs, *want[1])


@pytest.mark.parametrize("dtype", [BF16, E4M3, INT8], ids=["bf16", "e4m3", "int8"])
def test_append_bad_paths_and_strides(dtype):
    """Entries outside the tree end a path, lengths are clamped, a node may stand on
    a path twice; the tree's rows from a packed projection, the caches as
    [B, layers, L, h, d]."""
    layers, B, h, n, L, d, block = 2, 5, 3, 40, 96, 64, 32
    x = _tree_rows(layers, B, n, 2 * h, d, 1)  # [layers, B, n, 2h, d]
    kt, vt = (t.transpose(2, 3) for t in x.split(h, 3))
    caches = []
    for seed in (3, 4):
        c, s = _cache(layers, B, h, L, d, dtype, block, seed)
        c = c.permute(1, 0, 3, 2, 4).contiguous().permute(1, 0, 3, 2, 4)
        caches.append((c, s))
    path = np.tile(np.arange(n), (B, 1))
    path[0, 35] = n          # too large, past the first 32
    path[1, 2] = -1
    path[2, 0] = 1 << 30
    path[3, 1] = 0           # twice the same
    path_lens = [n, 5, 3, 4, 1000]
    lens = [3, 10, 0, 31, 50]
    want = []
    for (c, s), t in zip(caches, (kt, vt)):
        w = c.float().cpu().double().numpy()
        ws = None if s is None else s.cpu().numpy().copy()
        tree.append_path(w, ws, t.double().cpu().numpy(), path, path_lens, lens, block,
                         dtype == INT8)
        want.append((w, ws))
    (kc, ks), (vc, vs) = caches
    binding.attn_cache_append_tree(kt, vt, _int(path), _int(path_lens), kc, vc, _int(lens), ks, vs,
                                   block)
    binding.check()
    _same(kc, ks, *want[0])
    _same(vc, vs, *want[1])
    # one layer without its dimension; empty caches
    kc0, ks0 = kc[0].clone(), None if ks is None else ks[0].clone()
    vc0, vs0 = vc[0].clone(), None if vs is None else vs[0].clone()
    binding.attn_cache_append_tree(kt[0], vt[0], _int(path), _int(path_lens), kc0, vc0, None, ks0,
                                   vs0, block)
    w, ws = kc[0].float().cpu().double().numpy(), None if ks is None else ks[0].cpu().numpy()
    tree.append_path(w[None], None if ws is None else ws[None], kt[:1].double().cpu().numpy(), path,
                     path_lens, [0] * B, block, dtype == INT8)
    _same(kc0, ks0, w, ws)


def test_append_refusals():
    t = torch.zeros((2, 1, 2, 4, 64), dtype=BF16, device="cuda")
    c = torch.zeros((2, 1, 2, 32, 64), dtype=BF16, device="cuda")
    e = torch.zeros((2, 1, 2, 32, 64), dtype=INT8, device="cuda")
    s = torch.ones((2, 1, 2, 2), device="cuda")
    ids = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    ok = dict(k_tree=t, v_tree=t, path=ids, path_lens=ids[:, 0].contiguous(), k_cache=c, v_cache=c.clone(),
              cache_lens=None)
    binding.attn_cache_append_tree(**ok)
    binding.attn_cache_append_tree(**{**ok, "k_cache": e, "v_cache": e.clone(), "k_scale": s,
                                      "v_scale": s.clone(), "block_tokens": 16})
    for change in (dict(k_tree=t.float()), dict(v_tree=t[:, :, :1]), dict(path=ids[:, :3]),
                   dict(path=None), dict(path_lens=None), dict(path_lens=ids[0]),
                   dict(k_cache=c.half()), dict(v_cache=c[:1]), dict(cache_lens=ids[0]),
                   dict(k_cache=e, v_cache=e), dict(k_cache=e, v_cache=e, k_scale=s, v_scale=s),
                   dict(k_cache=e, v_cache=e, k_scale=s, v_scale=s, block_tokens=24),
                   dict(k_tree=t.transpose(3, 4))):
        with pytest.raises(ValueError):
            binding.attn_cache_append_tree(**{**ok, **change})


# ---------------------------------------------------------------- the whole step

@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_a_step_over_drafted_tokens(dtype):
    """Two steps of a two-layer decoder's attention: the tree's nodes over the
    cache, the walk over (given) probabilities, the path into the cache; then the
    next step's root sees the cache that plain appends of the kept tokens give."""
    layers, B, h, hk, n, L, d, V, block = 2, 3, 4, 2, 12, 128, 64, 50, 32
    p, q, tokens, parents, u = _case(B, n, V, torch.float32, True, 21)
    lens = _int([5, 30, 61])
    kc, ks = _cache(layers, B, hk, L, d, dtype, block, 3)
    vc, vs = _cache(layers, B, hk, L, d, dtype, block, 4)
    kept = [x if x is None else x.clone() for x in (kc, vc, ks, vs)]
    kt, vt = _tree_rows(layers, B, hk, n, d, 1), _tree_rows(layers, B, hk, n, d, 2)
    ids = _int(parents)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # everything on a stream of its own, no host in between
        path, path_lens, token = binding.attn_tree_verify(p, tokens, ids, u, draft=q)
        binding.attn_cache_append_tree(kt, vt, path, path_lens, kc, vc, lens, ks, vs, block)
        new_lens = lens + path_lens
        outs = []
        for layer in range(layers):
            qn = _tree_rows(1, B, h, n, d, 50 + layer)[0]
            outs.append(binding.attn_decode_tree(
                qn, kt[layer], vt[layer], ids, kc[layer], vc[layer], new_lens,
                None if ks is None else ks[layer], None if vs is None else vs[layer], block))
    torch.cuda.current_stream().wait_stream(side)
    binding.check()
    assert (path_lens > 1).any() and ((0 <= token) & (token < V)).all()
    # the same tokens, appended one sequence at a time by plain copies
    kc2, vc2, ks2, vs2 = kept
    for layer in range(layers):
        for b in range(B):
            rows = path[b, :int(path_lens[b])].long()
            if dtype == BF16:
                at = slice(int(lens[b]), int(lens[b]) + len(rows))
                kc2[layer, b, :, at], vc2[layer, b, :, at] = kt[layer, b][:, rows], vt[layer, b][:, rows]
            else:
                binding.attn_cache_append(kt[layer, b:b + 1][:, :, rows].contiguous(),
                                          vt[layer, b:b + 1][:, :, rows].contiguous(),
                                          kc2[layer, b:b + 1], vc2[layer, b:b + 1],
                                          ks2[layer, b:b + 1], vs2[layer, b:b + 1], lens[b:b + 1],
                                          block)
        qn = _tree_rows(1, B, h, n, d, 50 + layer)[0]
        want = binding.attn_decode_tree(qn, kt[layer], vt[layer], ids, kc2[layer], vc2[layer],
                                        new_lens, None if ks is None else ks2[layer],
                                        None if vs is None else vs2[layer], block)
        assert all(torch.equal(a, b) for a, b in zip(outs[layer], want))
    raw = [x.view(torch.uint8) for x in (kc, vc, kc2, vc2)]
    assert torch.equal(raw[0], raw[2]) and torch.equal(raw[1], raw[3])
    if ks is not None:
        assert torch.equal(ks, ks2) and torch.equal(vs, vs2)
