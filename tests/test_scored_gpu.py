"""GPU parity of attention with changed scores (attn_mask_plan, attn_fwd_scored,
attn_bwd_scored) with the float64 reference.

Tolerances, from the roundings:
 * scores and LSE: fp32 products of d <= 128 terms, at most (d + 8) 2^-24 of
   scale * sum |q k| <= 32; the cap's and the bias's own fp32 rounding (2^-22 of
   50, of slope * distance <= 512): together below 5e-4;
 * O: half a step of bf16 (2^-8 |O|), every P rounded once to bf16 (2^-8 of
   sum_j p_j |v_j|), and twice the scores' error of the same sum;
 * gradients: three independent bf16 roundings reach each (P or dS, the O inside
   D, the output), each off by at most 2^-8 of its value and by 1.7e-3 of it in
   the mean square (uniform inside half a step, over the mantissa): 2.9e-3
   together.  5e-3 in the 2-norm, and 1.5e-2 (four times 2^-8) of the largest
   entry, as for attn_bwd.
"""
import math

import numpy as np
import pytest
import torch

from oracle import scored
from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu

SCORE_TOL = 5e-4
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from transformer_head_scaled_gb300.build import build
    build()
    return binding.load()


def _random(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def _ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _f64(t):
    return t.double().cpu().numpy()


def _docs(n, *lens):
    """Ids of documents of the given lengths, the rest of the row padding."""
    ids = []
    for i, length in enumerate(lens):
        ids += [i % 3] * length   # neighbours differ, ids come again
    return (ids + [-1] * n)[:n]


# name: per batch entry masks
MASKS = {
    "none": dict(),
    "causal": dict(right=0),
    "window": dict(left=20, right=0),
    "band": dict(left=7, right=130),
    "left": dict(left=40),
    "lens": dict(key_len="lens"),
    "causal_lens": dict(right=0, key_len="lens"),
    "prefix": dict(right=0, prefix="prefix"),
    "docs": dict(docs=True),
    "docs_causal": dict(right=0, docs=True),
    "docs_prefix": dict(right=0, docs=True, prefix="prefix"),
    "docs_window_lens": dict(left=30, right=0, docs=True, key_len="lens"),
}


def _mask(name, B, n_q, n_k):
    """The plan and the reference's truth values."""
    m = MASKS[name]
    lens = [n_k, 0, n_k // 2, 1][:B] if m.get("key_len") else None
    prefix = [n_k // 3, 0, n_k + 5, 1][:B] if m.get("prefix") else None
    docs = None
    if m.get("docs"):
        cuts = [(1, 3, 126, 2, n_q), (n_q // 2,), (n_q,), (130, 1, 1, 40)][:B]
        docs = [_docs(n_q, *c) for c in cuts]
    plan = binding.attn_mask_plan(B, n_q, n_k, left=m.get("left"), right=m.get("right"),
                                  key_lens=_ints(lens), doc_ids=_ints(docs),
                                  prefix_lens=_ints(prefix), device="cuda")
    see = [scored.visible(n_q, n_k, m.get("left"), m.get("right"),
                          None if lens is None else lens[b],
                          None if docs is None else np.array(docs[b]),
                          None if prefix is None else prefix[b]) for b in range(B)]
    return plan, see


@pytest.mark.parametrize("n_q,n_k", [(1, 1), (128, 128), (300, 300), (129, 257), (257, 100)])
@pytest.mark.parametrize("name", list(MASKS))
def test_plan_is_the_mask(name, n_q, n_k):
    """The plan's intervals and tile bounds against the mask's definition."""
    if n_q != n_k and MASKS[name].get("docs"):
        pytest.skip("documents need n_q == n_k")
    B = 4
    plan, see = _mask(name, B, n_q, n_k)
    raw = plan.cpu().numpy()
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    qb, kt = -(-n_q // 256), -(-n_k // 128)
    at, parts = 256, []
    for count, width in ((B * n_q, 2), (B * n_k, 2), (B * qb, 8), (B * kt, 4)):
        parts.append(raw[at:at + count * width * 4].view(np.int32).reshape(count, width))
        at += up(count * width * 4)
    rows, keys, q_items, k_items = parts
    assert list(raw[:12].view(np.int32)) == [n_q, n_k, B]
    for b in range(B):
        for got, want in ((rows[b * n_q:(b + 1) * n_q], see[b]),
                          (keys[b * n_k:(b + 1) * n_k], see[b].T)):
            n = want.shape[1]
            made = (np.arange(n) >= got[:, :1]) & (np.arange(n) < got[:, 1:])
            assert np.array_equal(made, want)

    def span(part):
        seen = np.flatnonzero(part.any(0))
        return (seen[0], seen[-1] + 1) if seen.size else (0, 0)
    assert sorted(map(tuple, q_items[:, :2])) == [(b, x) for b in range(B) for x in range(qb)]
    for b, block, first, end0, end1, work, *_ in q_items:
        halves = [span(see[b][256 * block + 128 * i:256 * block + 128 * i + 128]) for i in (0, 1)]
        assert (end0, end1) == (halves[0][1], halves[1][1])
        assert first == min((lo for lo, hi in halves if hi), default=0)
        assert work == sum(-(-hi // 128) - first // 128 for _, hi in halves if hi)
    assert sorted(map(tuple, k_items[:, :2])) == [(b, x) for b in range(B) for x in range(kt)]
    for b, tile, first, count in k_items:
        lo, hi = span(see[b].T[128 * tile:128 * tile + 128])
        assert (first, count) == ((lo // 128, -(-hi // 128) - lo // 128) if hi else (0, 0))
    if MASKS[name].get("docs"):   # by falling work, ties in index order
        for work, index in ((q_items[:, 5], q_items[:, 0] * qb + q_items[:, 1]),
                            (k_items[:, 3], k_items[:, 0] * kt + k_items[:, 1])):
            place = list(zip(-work, index))
            assert place == sorted(place)


def _check_fwd(got, q, k, v, see, scale, cap, slopes):
    o, lse = _f64(got[0].float()), _f64(got[1])
    q, k, v = _f64(q), _f64(k), _f64(v)
    sl = None if slopes is None else _f64(slopes)
    ro, rl = scored.attention(q, k, v, see, scale, cap, sl)
    weight, _ = scored.attention(q, k, np.abs(v), see, scale, cap, sl)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * SCORE_TOL) * weight + 1e-6
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= tol).all(), np.abs(o - ro).max()
    none = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), none) and (lse[none] < 0).all()
    assert (np.abs(lse[~none] - rl[~none]) <= SCORE_TOL).all()
    return ro, rl


def _check_grads(got, want):
    for name, a, b in zip(("dq", "dk", "dv")[-len(got):], got, want):
        a = _f64(a.float())
        assert np.isfinite(a).all(), name
        big = np.abs(b).max()
        if big < 1e-9:   # every query sees one key at most: exact zeros, but for fp32 rounding
            assert np.abs(a).max() <= 1e-4, name
            continue
        rel, worst = np.linalg.norm(a - b) / np.linalg.norm(b), np.abs(a - b).max() / big
        assert rel <= 5e-3 and worst <= 1.5e-2, (name, rel, worst)


CASES = [
    # h, h_kv, n_q, n_k, d, cap, alibi
    (2, 2, 1, 1, 64, 0.0, False),
    (4, 2, 128, 128, 64, 30.0, False),
    (4, 1, 300, 300, 32, 0.0, True),
    (2, 1, 333, 333, 16, 20.0, True),
    (3, 3, 520, 520, 64, 0.0, True),
    (2, 2, 129, 257, 64, 30.0, True),
    (4, 2, 257, 100, 128, 50.0, True),
    (6, 2, 260, 260, 128, 0.0, False),
]


@pytest.mark.parametrize("h,hk,n_q,n_k,d,cap,alibi", CASES)
@pytest.mark.parametrize("name", list(MASKS))
def test_forward_and_backward_match_reference(name, h, hk, n_q, n_k, d, cap, alibi):
    if n_q != n_k and MASKS[name].get("docs"):
        pytest.skip("documents need n_q == n_k")
    B, scale = 4, 1 / math.sqrt(d)
    plan, see = _mask(name, B, n_q, n_k)
    q, k, v = _random((B, h, n_q, d), 1, 2.0), _random((B, hk, n_k, d), 2), _random((B, hk, n_k, d), 3)
    slopes = _slopes(h) if alibi else None
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=cap, slopes=slopes)
    binding.check()
    _check_fwd((o, lse), q, k, v, see, scale, cap, slopes)
    if d == 128:
        return
    dout = _random((B, h, n_q, d), 4)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=cap, slopes=slopes)
    binding.check()
    want = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, scale, cap,
                            None if slopes is None else _f64(slopes))
    _check_grads(got, want)


@pytest.mark.parametrize("n", [17, 24, 48])
@pytest.mark.parametrize("docs", [2, 5, 9])
def test_gradients_of_short_documents(n, docs):
    """Queries with few keys: dP - D cancels, so that D must not come from the
    rounded O."""
    B, h, d, scale = 2, 2, 16, 0.25
    r = np.random.default_rng(docs)
    cuts = [np.sort(r.integers(1, n, docs - 1)) for _ in range(B)]
    ids = [[int((i >= c).sum()) for i in range(n)] for c in cuts]
    plan = binding.attn_mask_plan(B, n, n, right=0, doc_ids=_ints(ids))
    see = [scored.visible(n, n, right=0, doc_ids=np.array(x)) for x in ids]
    q, k, v, dout = (_random((B, h, n, d), s, 2.0 if s == 1 else 1.0) for s in (1, 2, 3, 4))
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan)
    binding.check()
    want = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, scale)
    _check_grads(got, want)


@pytest.mark.parametrize("B,h,hk,n_q,n_k,d", [(2, 2, 1, 40, 2, 64), (2, 2, 2, 300, 7, 32),
                                              (1, 4, 2, 5, 16, 16), (2, 2, 1, 40, 17, 64),
                                              (80, 16, 4, 20, 20, 16), (90, 7, 7, 9, 9, 64)])
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_of_queries_with_few_keys(B, h, hk, n_q, n_k, d, masked):
    """Without a plan and with one, few heads and many, capped and biased."""
    plan = binding.attn_mask_plan(B, n_q, n_k, right=0, device="cuda") if masked else None
    see = [scored.visible(n_q, n_k, right=0 if masked else None)] * B
    q, dout = _random((B, h, n_q, d), 1, 2.0), _random((B, h, n_q, d), 4)
    k, v = _random((B, hk, n_k, d), 2), _random((B, hk, n_k, d), 3)
    kw = dict(softcap=20.0, slopes=_slopes(h), plan=plan)
    o, lse = binding.attn_fwd_scored(q, k, v, **kw)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, **kw)
    binding.check()
    want = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, 1 / math.sqrt(d), 20.0,
                            _f64(_slopes(h)))
    _check_grads(got, want)


def test_gradients_are_those_of_finite_differences():
    """Along random directions, in float64, of the reference's forward."""
    B, h, hk, n, d, cap = 1, 4, 2, 40, 16, 5.0
    plan, see = _mask("docs_causal", B, n, n)
    q, k, v = _random((B, h, n, d), 1), _random((B, hk, n, d), 2), _random((B, hk, n, d), 3)
    dout, slopes = _random((B, h, n, d), 4), _slopes(h)
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=cap, slopes=slopes)
    grads = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=cap, slopes=slopes)
    binding.check()
    base = [_f64(t) for t in (q, k, v)]

    def loss(t):
        return (scored.attention(*t, see, 0.25, cap, _f64(slopes))[0] * _f64(dout)).sum()
    r = np.random.default_rng(0)
    for which in range(3):
        for _ in range(3):
            direction = r.normal(size=base[which].shape)
            up, down = [[x.copy() for x in base] for _ in range(2)]
            up[which] += 1e-5 * direction
            down[which] -= 1e-5 * direction
            want = (loss(up) - loss(down)) / 2e-5
            g = _f64(grads[which].float())
            # 5e-3 of the gradient's norm, times the direction's (unit normal) length along it
            assert abs((g * direction).sum() - want) <= 4 * 5e-3 * np.linalg.norm(g)


def test_strided_views_and_packed_gradients():
    """Q, K, V from one projection [B, n, h + 2 h_kv, d], O into [B, n, h, d], the
    gradients into one packed buffer."""
    B, h, hk, n, d = 2, 4, 2, 200, 64
    x = _random((B, n, h + 2 * hk, d), 1)
    q, k, v = (t.transpose(1, 2) for t in x.split([h, hk, hk], 2))
    plan, see = _mask("docs_causal", B, n, n)
    out = torch.zeros((B, n, h, d), dtype=BF16, device="cuda").transpose(1, 2)
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=20.0, out=out)
    binding.check()
    assert o is out
    _check_fwd((o, lse), q, k, v, see, 0.125, 20.0, None)
    dout = _random((B, n, h, d), 5).transpose(1, 2)
    packed = torch.full((B, n, h + 2 * hk + 1, d), 3.0, dtype=BF16, device="cuda")
    views = [t.transpose(1, 2) for t in packed[:, :, 1:].split([h, hk, hk], 2)]
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=20.0, dq=views[0],
                                  dk=views[1], dv=views[2])
    binding.check()
    want = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, 0.125, 20.0)
    _check_grads(got, want)
    assert (packed[:, :, 0] == 3.0).all()


def test_unchanged_scores_equal_the_plain_forward():
    """No cap, no bias, no plan (and a causal plan): the same arithmetic as attn_fwd."""
    q, k, v = (_random((2, 3, 300, 64), s) for s in (1, 2, 3))
    for mask, kw in ((binding.MASK_NONE, None), (binding.MASK_CAUSAL, dict(right=0))):
        plan = None if kw is None else binding.attn_mask_plan(2, 300, 300, device="cuda", **kw)
        want = binding.attn_fwd(q, k, v, mask=mask)
        got = binding.attn_fwd_scored(q, k, v, plan=plan)
        binding.check()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cap", [1e-6, 0.01, 1.0, 300.0, 1e6])
def test_caps_from_tiny_to_idle(cap):
    """Arguments of the tanh from saturated to all but linear, zero scores among
    them, in forward and gradients."""
    B, h, n, d = 1, 2, 150, 64
    q, k, v, dout = (_random((B, h, n, d), s) for s in (1, 2, 3, 4))
    q[:, :, :20] = 0
    see = [scored.visible(n, n, right=0)]
    plan = binding.attn_mask_plan(B, n, n, right=0, device="cuda")
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=cap)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=cap)
    binding.check()
    _check_fwd((o, lse), q, k, v, see, 0.125, cap, None)
    want = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, 0.125, cap)
    assert all(torch.isfinite(t.float()).all() for t in got)
    if cap >= 1.0:   # (below, scores are flat but in the first rows: dq and dk are next to nothing)
        _check_grads(got, want)
    else:
        _check_grads(got[2:], want[2:])


def test_long_packed_row_by_parts():
    """A row of 20,000 tokens in documents, every document against itself alone."""
    h, hk, d, lens = 2, 1, 64, [7000, 1, 129, 4870, 6000, 2000]
    n = sum(lens)
    ids = sum(([i] * x for i, x in enumerate(lens)), [])
    q, k, v, dout = (_random((1, x, n, d), s) for x, s in ((h, 1), (hk, 2), (hk, 3), (h, 4)))
    slopes = _slopes(h)
    plan = binding.attn_mask_plan(1, n, n, right=0, doc_ids=_ints([ids]))
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=30.0, slopes=slopes)
    grads = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=30.0, slopes=slopes)
    binding.check()
    at = 0
    for x in lens:
        part = [t[:, :, at:at + x].contiguous() for t in (q, k, v)]
        own = binding.attn_mask_plan(1, x, x, right=0, device="cuda")
        po, pl = binding.attn_fwd_scored(*part, plan=own, softcap=30.0, slopes=slopes)
        pg = binding.attn_bwd_scored(*part, po, pl, dout[:, :, at:at + x], plan=own, softcap=30.0,
                                     slopes=slopes)
        binding.check()
        # each is within half a step of bf16 and of P's rounding of the other
        assert (o[:, :, at:at + x].float() - po.float()).abs().max() <= 3e-2
        assert (lse[:, :, at:at + x] - pl).abs().max() <= 2 * SCORE_TOL
        for a, b in zip(grads, pg):
            a, b = a[:, :, at:at + x].float(), b.float()
            assert (a - b).norm() <= 1e-2 * b.norm() + 1e-4 * math.sqrt(b.numel())
        at += x


@pytest.mark.parametrize("B,h,hk", [(1, 32, 2), (2, 32, 16)])
def test_documents_dealt_out_by_load(B, h, hk):
    """Few, uneven key tiles with enough rows to be dealt out by load, the query
    heads of a key head in parts and in one; every document against itself alone."""
    n, d = 4096 if B == 1 else 2048, 64
    lens = [[n // 2 + 1, 1, 300, n // 2 - 302], [5, n - 700, 695]][:B]
    ids = [sum(([i] * x for i, x in enumerate(row)), []) for row in lens]
    q, k, v, dout = (_random((B, x, n, d), s) for x, s in ((h, 1), (hk, 2), (hk, 3), (h, 4)))
    plan = binding.attn_mask_plan(B, n, n, right=0, doc_ids=_ints(ids))
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=30.0)
    grads = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=30.0)
    again = binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, softcap=30.0)
    binding.check()
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])
    for b, row in enumerate(lens):
        at = 0
        for x in row:
            part = [t[b:b + 1, :, at:at + x].contiguous() for t in (q, k, v)]
            own = binding.attn_mask_plan(1, x, x, right=0, device="cuda")
            po, pl = binding.attn_fwd_scored(*part, plan=own, softcap=30.0)
            pg = binding.attn_bwd_scored(*part, po, pl, dout[b:b + 1, :, at:at + x], plan=own,
                                         softcap=30.0)
            binding.check()
            for g, w in zip(grads, pg):
                g, w = g[b:b + 1, :, at:at + x].float(), w.float()
                # (as above: each within half a step of bf16 and the roundings of P and dS)
                assert (g - w).norm() <= 1e-2 * w.norm() + 1e-4 * math.sqrt(w.numel())
            at += x


@pytest.mark.parametrize("n", [5, 300])
def test_sides_longer_than_the_sequence_bound_nothing(n):
    whole = binding.attn_mask_plan(2, n, n, device="cuda").clone()
    for far in (n - 1, n, 2 * n, 2 ** 31 - 1, 2 ** 32, 2 ** 40):
        assert scored.visible(n, n, left=far, right=far).all()
        plan = binding.attn_mask_plan(2, n, n, left=far, right=far, device="cuda")
        q, k, v = (_random((2, 2, n, 16), s) for s in (1, 2, 3))
        for a, b in zip(binding.attn_fwd_scored(q, k, v, plan=plan),
                        binding.attn_fwd_scored(q, k, v, plan=whole)):
            assert torch.equal(a, b), far
    binding.check()


def test_training_step_as_a_captured_graph():
    """Plan, two layers forward and backward captured once and replayed on new
    inputs and documents; dK, dV and O are the eager calls' bit for bit."""
    B, h, hk, n, d = 2, 4, 2, 260, 32
    q, dout = (torch.empty((B, h, n, d), dtype=BF16, device="cuda") for _ in range(2))
    k, v = (torch.empty((B, hk, n, d), dtype=BF16, device="cuda") for _ in range(2))
    ids = torch.zeros((B, n), dtype=torch.int32, device="cuda")

    def step():
        plan = binding.attn_mask_plan(B, n, n, right=0, doc_ids=ids)
        o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, softcap=30.0)
        o2, lse2 = binding.attn_fwd_scored(o, k, v, plan=plan, softcap=30.0)
        d2 = binding.attn_bwd_scored(o, k, v, o2, lse2, dout, plan=plan, softcap=30.0)
        d1 = binding.attn_bwd_scored(q, k, v, o, lse, d2[0], plan=plan, softcap=30.0)
        return o, o2, d2[1], d2[2], d1[0]
    for t, s in ((q, 1), (k, 2), (v, 3), (dout, 4)):
        t.copy_(_random(t.shape, s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        for t, s in ((q, 1), (k, 2), (v, 3), (dout, 4)):
            t.copy_(_random(t.shape, 10 * i + s))
        ids.copy_(_ints([_docs(n, 50 + i, 100), _docs(n, n - 7 * i)]))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        binding.check()
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)
        # dq adds key tiles in the order in which they finish
        assert (got[4].float() - want[4].float()).norm() <= 4e-3 * want[4].float().norm()


def test_calls_on_two_streams():
    B, h, n, d = 1, 4, 700, 64
    sets = [[_random((B, h, n, d), 10 * i + s) for s in range(4)] for i in range(2)]
    plan = binding.attn_mask_plan(B, n, n, right=0, device="cuda")
    want = []
    for q, k, v, g in sets:
        o, lse = binding.attn_fwd_scored(q, k, v, plan=plan)
        want.append((o, lse, *binding.attn_bwd_scored(q, k, v, o, lse, g, plan=plan)[1:]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (st, (q, k, v, g)) in enumerate(zip(streams, sets)):
            o, lse = binding.attn_fwd_scored(q, k, v, plan=plan, stream=st)
            got[i].append((o, lse, *binding.attn_bwd_scored(q, k, v, o, lse, g, plan=plan,
                                                            stream=st)[1:]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_a_plan_of_other_sizes_is_reported():
    q, k, v = (_random((1, 2, 100, 64), s) for s in (1, 2, 3))
    other = binding.attn_mask_plan(1, 101, 101, right=0, device="cuda")
    o, lse = binding.attn_fwd_scored(q, k, v, plan=other)
    with pytest.raises(binding.AttnError) as e:
        binding.check()
    assert e.value.status == binding.ATTN_ERR_WRONG_PLAN
    binding.attn_bwd_scored(q, k, v, o, lse, q, plan=other)
    with pytest.raises(binding.AttnError) as e:
        binding.check()
    assert e.value.status == binding.ATTN_ERR_WRONG_PLAN
    binding.check()   # reported once
