"""Attention with changed scores where its arguments end: caps from wide to idle,
scores past the polynomials' range in some tiles and not in others, plans of other
sizes, workspaces with anything in them, the default stream by its number.

Tolerances as in test_scored_gpu, and with the general form of the tanh 3e-7 of the
cap more for scores and LSE.
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


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _check_fwd(got, want, weight, tol=SCORE_TOL):
    o, lse = _f64(got[0]), _f64(got[1])
    ro, rl = want
    assert np.isfinite(o).all()
    err = np.abs(o - ro) / (2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * tol) * weight + 1e-6)
    assert (err <= 1).all(), err.max()
    none = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), none) and (lse[none] < 0).all()
    assert (np.abs(lse[~none] - rl[~none]) <= tol).all(), np.abs(lse[~none] - rl[~none]).max()


def _check_grads(got, want):
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        a = _f64(a)
        assert np.isfinite(a).all(), name
        rel, worst = np.linalg.norm(a - b) / np.linalg.norm(b), np.abs(a - b).max() / np.abs(b).max()
        assert rel <= 5e-3 and worst <= 1.5e-2, (name, rel, worst)


def _both_ways(h, hk, n, d, mask, cap, slopes, q, k, v, tol=SCORE_TOL, gradients=True,
               scale=None):
    """Forward, and gradients where d has them, of one batch entry against the reference."""
    see = [scored.visible(n, n, **mask)]
    plan = binding.attn_mask_plan(1, n, n, device="cuda", **mask)
    scale = 1 / math.sqrt(d) if scale is None else scale
    kw = dict(plan=plan, softcap=cap, slopes=slopes, scale=scale)
    o, lse = binding.attn_fwd_scored(q, k, v, **kw)
    binding.check()
    ref = (_f64(q), _f64(k), _f64(v))
    want = scored.attention(*ref, see, scale, cap, _f64(slopes))
    weight, _ = scored.attention(*ref[:2], np.abs(ref[2]), see, scale, cap, _f64(slopes))
    _check_fwd((o, lse), want, weight, tol)
    if d == 128 or not gradients:
        return
    dout = _random(q.shape, 4)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, **kw)
    binding.check()
    _check_grads(got, scored.gradients(*ref, _f64(dout), see, scale, cap, _f64(slopes)))


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("mask", [dict(), dict(right=0), dict(left=40, right=0)],
                         ids=["none", "causal", "window"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("cap", [300.0, 1e6, 1e9, 1e12, 2.0 ** 64])
def test_wide_and_idle_caps(cap, d, mask, alibi):
    """A cap far above every score changes nothing."""
    h, hk, n = 2, 1, 300
    q, k, v = _random((1, h, n, d), 1, 2.0), _random((1, hk, n, d), 2), _random((1, hk, n, d), 3)
    _both_ways(h, hk, n, d, mask, cap, _slopes(h) if alibi else None, q, k, v)


@pytest.mark.parametrize("mask", [dict(), dict(right=0)], ids=["none", "causal"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("cap", [1e8, 1e9, 1e10, 1e12])
def test_large_scores_under_an_idle_cap(cap, d, mask):
    """Scores of up to 150, where the running maximum must not carry the general
    form's error of 3e-7 of the cap (forward)."""
    h, hk, n = 2, 1, 300
    q, k, v = _random((1, h, n, d), 1, 40.0), _random((1, hk, n, d), 2), _random((1, hk, n, d), 3)
    sums = (np.abs(_f64(q)) @ np.abs(_f64(k)).swapaxes(2, 3)).max() / math.sqrt(d)
    _both_ways(h, hk, n, d, mask, cap, None, q, k, v, SCORE_TOL + (d + 8) * 2.0 ** -24 * sums,
               gradients=False)


@pytest.mark.parametrize("dtype", [BF16, torch.int8, torch.float8_e4m3fn],
                         ids=["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", [300.0, 1e9, 1e12, 2.0 ** 64])
def test_decode_under_wide_and_idle_caps(cap, alibi, dtype):
    h, L, d = 2, 400, 64
    q = _random((1, h, 1, d), 1, 2.0)
    k, v = (_random((1, h, L, d), s, 1.0 if dtype == BF16 else 40.0).to(dtype) for s in (2, 3))
    ks = None if dtype == BF16 else torch.full((1, h, 25), 1 / 40, device="cuda")
    unit = 1.0 if ks is None else float(ks[0, 0, 0])
    slopes = _slopes(h) if alibi else None
    o, lse = binding.attn_decode_scored(q, k, v, k_scale=ks, v_scale=ks, block_tokens=16,
                                        softcap=cap, slopes=slopes)
    binding.check()
    kw = dict(lens=[L], scale=0.125, softcap=cap, slopes=_f64(slopes))
    kd, vd = _f64(k.float()) * unit, _f64(v.float()) * unit
    want = scored.decode(_f64(q), kd, vd, **kw)
    _check_fwd((o, lse), want, scored.decode(_f64(q), kd, np.abs(vd), **kw)[0])


@pytest.mark.parametrize("sign", [-1, 1], ids=["against", "toward"])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("cap", [300.0, 1000.0])
def test_scores_past_the_polynomials_in_some_tiles(cap, d, alibi, sign):
    """Under a wide cap, key tiles whose scores stay within 0.3 caps and others that
    hold one of 0.6 caps, against every query (its tile's other keys keep their
    weights) or toward it (forward alone: it takes all the weight)."""
    h, hk, n = 2, 1, 420
    q, k, v = _random((1, h, n, d), 1), _random((1, hk, n, d), 2), _random((1, hk, n, d), 3)
    q = (q.float() + 2).to(BF16)   # q . (1, 1, ..) is 2 d, give or take sqrt(d)
    k[0, 0, 130] = sign * 0.3 * cap / math.sqrt(d)
    s = _f64(q[0]) @ _f64(k[0, 0]).T / math.sqrt(d)
    assert (np.abs(s[:, :, 130]) > 0.3 * cap).all()
    assert np.abs(np.delete(s, 130, 2)).max() < 0.3 * cap
    tol = SCORE_TOL + 3e-7 * cap
    if sign > 0:   # sums of products as large as the cap have the weight
        tol += (d + 8) * 2.0 ** -24 * cap
    _both_ways(h, hk, n, d, dict(right=0), cap, _slopes(h) if alibi else None, q, k, v, tol,
               gradients=sign < 0)


@pytest.mark.parametrize("dtype", [BF16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("sign", [-1, 1], ids=["against", "toward"])
@pytest.mark.parametrize("cap", [300.0, 1000.0])
def test_decode_scores_past_the_polynomials(cap, sign, dtype):
    """The same in the decoding step: one key of 0.6 caps among ordinary ones."""
    h, L, d = 2, 300, 64
    q = (_random((1, h, 1, d), 1).float() + 2).to(BF16)
    x = _random((1, h, L, d), 2).float().clamp(-3.5, 3.5)
    x[:, :, 130] = sign * 0.3 * cap / math.sqrt(d)
    v = _random((1, h, L, d), 3).float().clamp(-3.5, 3.5)
    if dtype == BF16:
        codes, scales = [x.to(BF16), v.to(BF16)], [None, None]
        unit = [1.0, 1.0]
    else:   # a block of 16 tokens holds the large key: its scale is its own
        scales = [t.reshape(1, h, 20, 16 * d).abs().amax(-1) / 448 for t in (
            torch.cat([t, t[:, :, :20]], 2) for t in (x, v))]
        wide = [s.repeat_interleave(16, 2)[:, :, :L, None] for s in scales]
        codes = [(t / s).to(dtype) for t, s in zip((x, v), wide)]
        scales = [s[:, :, :19].contiguous() for s in scales]
        unit = [_f64(s) for s in wide]
    o, lse = binding.attn_decode_scored(q, *codes, k_scale=scales[0], v_scale=scales[1],
                                        block_tokens=16, softcap=cap)
    binding.check()
    k, v = (_f64(c.float()) * u for c, u in zip(codes, unit))
    kw = dict(lens=[L], scale=0.125, softcap=cap)
    tol = SCORE_TOL + 3e-7 * cap + ((d + 8) * 2.0 ** -24 * cap if sign > 0 else 0.0)
    _check_fwd((o, lse), scored.decode(_f64(q), k, v, **kw),
               scored.decode(_f64(q), k, np.abs(v), **kw)[0], tol)


@pytest.mark.parametrize("mask", [dict(), dict(right=0), dict(left=70, right=0), dict(right=60)],
                         ids=["none", "causal", "window", "ahead"])
@pytest.mark.parametrize("cap,alibi", [(50.0, False), (2.0, False), (0.0, True)])
@pytest.mark.parametrize("h,hk,n", [(2, 1, 200), (3, 3, 513)])
def test_heads_of_128_with_a_cap_or_a_bias_alone(h, hk, n, cap, alibi, mask):
    d = 128
    q, k, v = _random((1, h, n, d), 1, 2.0), _random((1, hk, n, d), 2), _random((1, hk, n, d), 3)
    _both_ways(h, hk, n, d, mask, cap, _slopes(h) if alibi else None, q, k, v)


@pytest.mark.parametrize("h,hk", [(2, 2), (4, 1)])
def test_a_plan_of_other_sizes_writes_nothing(h, hk):
    """Outputs and gradients keep what they held, those of key heads whose query heads
    are worked on in parts too."""
    q, k, v = (_random((1, x, 100, 64), s) for x, s in ((h, 1), (hk, 2), (hk, 3)))
    other = binding.attn_mask_plan(1, 101, 101, right=0, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full((1, h, 100), 5.0, device="cuda")
    grads = [torch.full_like(t, 5.0) for t in (q, k, v)]
    binding.attn_fwd_scored(q, k, v, plan=other, out=out, lse=lse)
    binding.attn_bwd_scored(q, k, v, q, torch.zeros_like(lse), q, plan=other, dq=grads[0],
                            dk=grads[1], dv=grads[2])
    with pytest.raises(binding.AttnError) as e:
        binding.check()
    assert e.value.status == binding.ATTN_ERR_WRONG_PLAN
    for t in (out, lse, *grads):
        assert (t == 5.0).all()


@pytest.mark.parametrize("lost", [False, True])
def test_gradients_do_not_depend_on_what_the_workspace_held(lost):
    """Queries with few keys among them; and (lost) with an LSE of -inf for one that
    sees keys, as scores of -inf leave it."""
    h, n, d = 2, 140, 64
    q, k, v, dout = (_random((1, h, n, d), s) for s in (1, 2, 3, 4))
    plan = binding.attn_mask_plan(1, n, n, left=5, right=0, device="cuda")
    o, lse = binding.attn_fwd_scored(q, k, v, plan=plan)
    if lost:
        lse[:, :, 7] = -math.inf
        o[:, :, 7] = 0
    need = binding.bwd_scored_workspace_bytes(1, h, h, n, n, d)
    got = []
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append(binding.attn_bwd_scored(q, k, v, o, lse, dout, plan=plan, workspace=ws))
    binding.check()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.isfinite(b.float()).all()
            assert (a.float() - b.float()).abs().max() <= 1e-2 * a.float().abs().max()


def test_the_default_stream_by_its_number():
    """stream=0 is the default stream: the call waits for what was put there before."""
    q, k, v = (_random((1, 2, 100, 64), s) for s in (1, 2, 3))
    cache = [t.contiguous() for t in (k, v)]
    want = [*binding.attn_fwd_scored(q, k, v), *binding.attn_decode_scored(q[:, :, :1], *cache)]
    late = torch.zeros_like(q)
    torch.cuda.Stream()   # (making a process's first one waits for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.default_stream()):
        torch.cuda._sleep(200_000_000)   # a tenth of a second
        late.copy_(q)
    got = [*binding.attn_fwd_scored(late, k, v, stream=0),
           *binding.attn_decode_scored(late[:, :, :1], *cache, stream=0)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -20])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_the_least_scales(d, alibi, scale):
    """What is divided by the scale (the bias, LSE) keeps its precision."""
    h, hk, n = 2, 1, 300
    q, k, v = _random((1, h, n, d), 1, 2.0), _random((1, hk, n, d), 2), _random((1, hk, n, d), 3)
    _both_ways(h, hk, n, d, dict(right=0), 0.0, _slopes(h) if alibi else None, q, k, v, scale=scale)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("cap", [0.0, 50.0, 3000.0])
@pytest.mark.parametrize("d", [16, 64])
def test_gradients_of_two_keys_of_which_one_has_all_but_the_weight(d, cap, masked):
    """Weights of 1 - p and p, p about e^-9: dP - D is p of dP, so that an error of the
    LSE of 4e-6 (a score of 20 by the cap's polynomial) must not reach D: it would be
    3 % of p.  What does reach it is fp32 rounding, 2^-23 / p = 1e-3, beside the three
    of bf16."""
    B, h, n = 2, 2, 60
    k, v = _random((B, h, 2, d), 2), _random((B, h, 2, d), 3)
    a, z = k[:, :, :1].float(), k[:, :, 1:].float()
    unit = (a - z) / (a - z).square().sum(-1, keepdim=True)
    side = (a + z) - ((a + z) * unit).sum(-1, keepdim=True) * (a - z)
    side = side / (side * (a + z)).sum(-1, keepdim=True)
    g = torch.Generator(device="cuda").manual_seed(7)
    gap = 8.5 + torch.rand((B, h, n, 1), generator=g, device="cuda")
    q = (math.sqrt(d) * (gap * unit + 30 * side)).to(BF16)   # scores of 15 + gap / 2, 15 - gap / 2
    dout = _random((B, h, n, d), 4)
    plan = binding.attn_mask_plan(B, n, 2, device="cuda") if masked else None
    kw = dict(plan=plan, softcap=cap)
    o, lse = binding.attn_fwd_scored(q, k, v, **kw)
    got = binding.attn_bwd_scored(q, k, v, o, lse, dout, **kw)
    binding.check()
    see = [np.ones((n, 2), bool)] * B
    ref = scored.gradients(_f64(q), _f64(k), _f64(v), _f64(dout), see, 1 / math.sqrt(d), cap)
    _check_grads(got, ref)
