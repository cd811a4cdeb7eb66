"""The float64 reference of attention with changed scores and of the 8-bit
cache, pinned on the CPU: to the plain oracle where nothing is changed, to
finite differences, and to the number formats' own definitions."""
import numpy as np
import pytest
import torch

import oracle
from oracle import scored

MASKS = [
    dict(),
    dict(right=0),
    dict(left=3, right=0),
    dict(left=2, right=4),
    dict(key_len=0),
    dict(right=0, key_len=5),
    dict(right=0, prefix=4),
    dict(doc_ids=[0, 0, 0, 7, 7, 2, 2, 2, 2, -1, -1, 0]),
    dict(right=0, doc_ids=[5, 5, 3, 3, 3, 3, 3, 3, 5, 5, 5, 5]),
]


def _qkv(n=12, d=16, h=4, hk=2, B=1, seed=0):
    r = np.random.default_rng(seed)
    return r.normal(size=(B, h, n, d)), r.normal(size=(B, hk, n, d)), r.normal(size=(B, hk, n, d))


def test_unchanged_scores_are_the_plain_oracle():
    oracle.build()
    q, k, v = (torch.randn(1, 2, 12, 16, generator=torch.Generator().manual_seed(s)) for s in (0, 1, 2))
    for mask, kw in ((0, dict()), (1, dict(right=0))):
        want = oracle.attn_fwd(q, k, v, 0.25, mask, None)
        see = [scored.visible(12, 12, **kw)]
        got = scored.attention(*(t.double().numpy() for t in (q, k, v)), see, 0.25)
        for a, b in zip(got, want):
            assert np.abs(a - b).max() <= 1e-12


@pytest.mark.parametrize("kw", MASKS)
def test_each_query_and_each_key_sees_one_run(kw):
    see = scored.visible(12, 12, **kw)
    for m in (see, see.T):
        for row in m:
            at = np.flatnonzero(row)
            assert at.size == 0 or at[-1] - at[0] + 1 == at.size


@pytest.mark.parametrize("kw", MASKS)
@pytest.mark.parametrize("softcap", [0.0, 1.5])
def test_gradients_are_those_of_finite_differences(kw, softcap):
    q, k, v = _qkv()
    slopes = np.array([0.5, 0.25, 0.125, 0.0625])
    see = [scored.visible(12, 12, **kw)]
    dout = np.random.default_rng(9).normal(size=q.shape)

    def loss(*t):
        return (scored.attention(*t, see, 0.25, softcap, slopes)[0] * dout).sum()
    grads = scored.gradients(q, k, v, dout, see, 0.25, softcap, slopes)
    r = np.random.default_rng(3)
    for which in range(3):
        for _ in range(4):
            at = tuple(r.integers(0, s) for s in (q, k, v)[which].shape)
            step = []
            for e in (1e-5, -1e-5):
                t = [x.copy() for x in (q, k, v)]
                t[which][at] += e
                step.append(loss(*t))
            # central differences: error e^2 |f'''| / 6 + rounding 1e-16 |f| / e
            assert abs((step[0] - step[1]) / 2e-5 - grads[which][at]) <= 1e-7


def test_large_cap_and_zero_slope_change_nothing():
    q, k, v = _qkv(seed=4)
    see = [scored.visible(12, 12, right=0)]
    a = scored.attention(q, k, v, see, 0.25)
    b = scored.attention(q, k, v, see, 0.25, 1e9, np.zeros(4))
    assert np.abs(a[0] - b[0]).max() <= 1e-12


def test_decode_is_the_last_rows_of_causal_attention():
    q, k, v = _qkv(n=20, B=2, seed=5)
    slopes = np.array([0.5, 0.25, 0.125, 0.0625])
    for n_q, window in ((1, None), (3, None), (4, 5)):
        see = [scored.visible(20, 20, left=window, right=0)] * 2
        o, lse = scored.attention(q, k, v, see, 0.25, 2.0, slopes)
        o2, lse2 = scored.decode(q[:, :, -n_q:], k, v, [20, 20], 0.25, 2.0, slopes, window)
        assert np.abs(o[:, :, -n_q:] - o2).max() <= 1e-13
        assert np.abs(lse[:, :, -n_q:] - lse2).max() <= 1e-13


def test_e4m3_numbers_and_rounding_are_the_types():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(scored.e4m3_values(), codes.double().numpy())
    x = torch.cat([torch.linspace(-500, 500, 4001), torch.logspace(-4, 2.7, 2000)])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(scored.nearest_e4m3(x.double().numpy()), want)


@pytest.mark.parametrize("int8", [False, True])
def test_append_keeps_values_within_half_a_step(int8):
    """Written once: half a step of the type.  Rescaled: another half step of
    the new scale for each time the scale grew."""
    r = np.random.default_rng(0)
    cache, scale = np.zeros((1, 1, 64, 16)), np.zeros((1, 1, 4), np.float32)
    x = r.normal(size=(1, 1, 40, 16)).astype(np.float32)
    n = 0
    while n < 40:  # one to five tokens at a time
        m = min(int(r.integers(1, 6)), 40 - n)
        scored.append(cache, scale, x[:, :, n:n + m], [n], [m], 16, int8)
        n += m
    got = cache[0, 0, :40] * np.repeat(scale[0, 0], 16)[:40, None]
    top = np.repeat(scale[0, 0], 16)[:40, None] * (1.0 if int8 else 448 / 16)
    assert (np.abs(got - x[0, 0]) <= 16 * 0.5 * top).all()
    assert not cache[0, 0, 40:].any()
