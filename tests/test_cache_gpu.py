"""GPU parity of the 8-bit cache (attn_cache_append) and of the decoding step
with changed scores (attn_decode_scored) with the float64 reference.

Codes and scales are defined in float32 with one rounding each, so they must
be equal.  For the decoding step the tolerances count the roundings:
 * O: half a step of bf16 (2^-8 |O|); each probability rounded once to f16
   (2^-11, 8-bit caches) or bf16 (2^-8), worth that share of sum_j p_j |v_j|;
   and the scores' error below, worth as much again of the same sum;
 * scores (and LSE): fp32 products of d terms, at most (d + 8) 2^-24 of
   scale * sum |q k| <= 32 here, the cap's and the bias's own fp32 rounding
   (2^-22 of 50 and of slope * distance <= 256), q to f16 at 2^-25 of its
   largest entry: together below 3e-4.
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


def _values(codes):
    """float64 NumPy code values of a cache."""
    return codes.float().cpu().double().numpy()


def _random(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def _cache(B, hk, L, d, dtype, block, seed):
    """A filled cache: codes and scales, and its float64 values."""
    x = _random((B, hk, L, d), seed)
    if dtype == BF16:
        c = x.to(BF16)
        return c, None, c.double().cpu().numpy()
    top = 127.0 if dtype == INT8 else 448.0
    x = (x * (top / 4)).clamp(-top, top)
    c = x.round().to(INT8) if dtype == INT8 else x.to(E4M3)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = torch.rand((B, hk, -(-L // block)), generator=g, device="cuda") * 0.02 + 0.005
    wide = _values(c) * np.repeat(s.cpu().double().numpy(), block, 2)[:, :, :L, None]
    return c, s, wide


def _check(got, q, k, v, lens, scale, softcap, slopes, window, dtype):
    o, lse = (t.float().cpu().double().numpy() for t in got)
    qd = q.double().cpu().numpy()
    sl = None if slopes is None else slopes.double().cpu().numpy()
    ro, rl = scored.decode(qd, k, v, lens, scale, softcap, sl, window)
    weight, _ = scored.decode(qd, k, np.abs(v), lens, scale, softcap, sl, window)
    p_step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(ro) + (p_step + 2 * SCORE_TOL) * weight + 1e-6
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= tol).all(), np.abs(o - ro).max()
    none = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), none) and (lse[none] < 0).all()
    assert (np.abs(lse[~none] - rl[~none]) <= SCORE_TOL).all(), np.abs(lse[~none] - rl[~none]).max()


def _slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


CASES = [
    # B, h, h_kv, n_q, L_max, d, block, cap, alibi, window, lens
    (1, 1, 1, 1, 1, 64, 16, 0.0, False, None, [1]),
    (3, 4, 4, 1, 77, 64, 16, 0.0, False, None, [77, 0, 1]),
    (2, 4, 2, 1, 513, 64, 64, 30.0, True, None, [513, 200]),
    (2, 8, 1, 1, 300, 128, 128, 50.0, False, 50, [300, 17]),
    (2, 6, 2, 3, 257, 128, 32, 0.0, True, None, [257, 2]),
    (1, 16, 2, 2, 900, 32, 64, 30.0, True, 333, [899]),
    (2, 8, 1, 4, 130, 16, 16, 0.0, False, 0, [130, 3]),
    (1, 16, 1, 4, 700, 64, 128, 50.0, True, None, [655]),
    (1, 24, 1, 8, 200, 128, 64, 0.0, True, 1000, [200]),  # several tiles of query rows
    (1, 2, 1, 1, 9000, 64, 128, 0.0, True, None, [8999]),  # the cache is split
    (1, 2, 2, 8, 5000, 128, 16, 30.0, False, 2100, [4996]),
]


@pytest.mark.parametrize("dtype", [E4M3, INT8, BF16], ids=["e4m3", "int8", "bf16"])
@pytest.mark.parametrize("B,h,hk,n_q,L,d,block,cap,alibi,window,lens", CASES)
def test_decode_scored_matches_reference(dtype, B, h, hk, n_q, L, d, block, cap, alibi, window,
                                         lens):
    q = _random((B, h, n_q, d), 1, 2.0).to(BF16)
    kc, ks, k = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, hk, L, d, dtype, block, 4)
    slopes = _slopes(h) if alibi else None
    # what lies behind the last token is never used: NaN codes and scales
    for b, n in enumerate(lens):
        for c, s in ((kc, ks), (vc, vs)):
            if dtype == BF16:
                c[b, :, n:] = float("nan")
            else:
                c[b, :, n:] = torch.full((), 0x7f, dtype=torch.uint8, device="cuda").view(dtype)
                s[b, :, -(-n // block):] = float("nan")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(d)
    got = binding.attn_decode_scored(q, kc, vc, lens_t, k_scale=ks, v_scale=vs, block_tokens=block,
                                     softcap=cap, slopes=slopes, window=window)
    binding.check()
    _check(got, q, k, v, lens, scale, cap, slopes, window, dtype)
    again = binding.attn_decode_scored(q, kc, vc, lens_t, k_scale=ks, v_scale=vs,
                                       block_tokens=block, softcap=cap, slopes=slopes,
                                       window=window)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # no order that changes results


@pytest.mark.parametrize("dtype", [E4M3, INT8, BF16], ids=["e4m3", "int8", "bf16"])
def test_decode_scored_ignores_what_lies_before_the_window(dtype):
    B, h, L, d, block, window = 1, 2, 400, 64, 16, 37
    q = _random((B, h, 1, d), 1).to(BF16)
    kc, ks, k = _cache(B, h, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, h, L, d, dtype, block, 4)
    first = L - 1 - window
    if ks is not None:   # nor the scales of the blocks before it
        ks[:, :, :first // block] = float("inf")
        vs[:, :, :first // block] = float("nan")
    for c in (kc, vc):
        c[:, :, :first] = float("nan") if dtype == BF16 else torch.full(
            (), 0x7f, dtype=torch.uint8, device="cuda").view(dtype)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block,
                                     window=window)
    binding.check()
    _check(got, q, k, v, [L], 0.125, 0.0, None, window, dtype)


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_decode_scored_on_strided_views(dtype):
    """A cache kept [B, L, h, d], queries and outputs inside packed buffers."""
    B, h, hk, n_q, L, d, block = 2, 4, 2, 2, 190, 64, 32
    x = _random((B, n_q, h + 3, d), 1).to(BF16)
    q = x[:, :, 1:h + 1].transpose(1, 2)
    kc, ks, k = _cache(B, hk, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, hk, L, d, dtype, block, 4)
    kt, vt = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc))
    out = torch.full((B, n_q, h + 2, d), 7.0, dtype=BF16, device="cuda")
    o, lse = binding.attn_decode_scored(q, kt, vt, k_scale=ks, v_scale=vs, block_tokens=block,
                                        softcap=20.0, out=out[:, :, 2:].transpose(1, 2))
    binding.check()
    _check((o, lse), q, k, v, [L, L], 0.125, 20.0, None, None, dtype)
    assert (out[:, :, :2] == 7.0).all()


def test_decode_scored_tiny_values_and_equal_scales_of_zero():
    """Scales down to the least, zero scales (their tokens still count in the
    softmax) and zero queries."""
    B, h, L, d, block = 1, 1, 64, 64, 16
    q = _random((B, h, 1, d), 1).to(BF16)
    kc, ks, k = _cache(B, h, L, d, INT8, block, 2)
    vc, vs, v = _cache(B, h, L, d, INT8, block, 4)
    factor = torch.tensor([0.0, 1.0, 2.0 ** -60, 0.0], device="cuda")
    vs = vs * factor
    v = v * np.repeat(factor.cpu().double().numpy(), block)[None, None, :, None]
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block)
    _check(got, q, k, v, [L], 0.125, 0.0, None, None, INT8)
    got = binding.attn_decode_scored(torch.zeros_like(q), kc, vc, k_scale=ks, v_scale=vs,
                                     block_tokens=block)
    _check(got, torch.zeros_like(q), k, v, [L], 0.125, 0.0, None, None, INT8)


@pytest.mark.parametrize("cap", [1e-6, 0.01, 1.0, 300.0, 1e6])
@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_decode_scored_caps_from_tiny_to_idle(dtype, cap):
    B, h, L, d, block = 2, 2, 200, 64, 32
    q = _random((B, h, 1, d), 1, 2.0).to(BF16)
    kc, ks, k = _cache(B, h, L, d, dtype, block, 2)
    vc, vs, v = _cache(B, h, L, d, dtype, block, 4)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, block_tokens=block,
                                     softcap=cap)
    binding.check()
    _check(got, q, k, v, [L] * B, 0.125, cap, None, None, dtype)


def test_decode_scored_reads_past_32_bit_offsets():
    """The second head starts 2^31 + 2^17 bytes into the cache."""
    L, d, block, window = (1 << 24) + 1024, 128, 128, 700
    kc = torch.zeros((1, 2, L, d), dtype=INT8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.full((1, 2, L // block), 0.01, device="cuda")
    tail = 1024
    kt, _, _ = _cache(1, 2, tail, d, INT8, block, 2)
    vt, _, _ = _cache(1, 2, tail, d, INT8, block, 4)
    kc[:, :, L - tail:], vc[:, :, L - tail:] = kt, vt
    q = _random((1, 2, 1, d), 1).to(BF16)
    got = binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=ks, block_tokens=block,
                                     window=window)
    binding.check()
    _check(got, q, _values(kt) * np.float64(np.float32(0.01)),
           _values(vt) * np.float64(np.float32(0.01)), [tail], 1 / math.sqrt(d), 0.0, None, window,
           INT8)


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("B,h,n_new,L,d,block,lens,new", [
    (1, 1, 1, 1, 16, 16, [0], None),
    (2, 3, 1, 100, 64, 64, [63, 64], None),
    (3, 2, 5, 100, 32, 16, [0, 14, 97], None),        # the last tokens do not fit
    (2, 2, 40, 200, 128, 32, [31, 100], [40, 0]),     # a padded batch, one entry empty
    (1, 2, 300, 517, 64, 128, [100], [299]),
    (2, 1, 130, 131, 128, 128, [1, 0], [130, 129]),
    (1, 1, 700, 640, 64, 64, [0], None),              # a prompt longer than the cache
])
def test_append_equals_reference(dtype, B, h, n_new, L, d, block, lens, new):
    kc, ks, _ = _cache(B, h, L, d, dtype, block, 2)
    vc, vs, _ = _cache(B, h, L, d, dtype, block, 4)
    x = _random((B, n_new, 2, h, d), 6).to(BF16)
    x[:, :, 1] *= 3
    kn, vn = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
    wants = []
    for c, s, n in ((kc, ks, kn), (vc, vs, vn)):
        wc, ws = _values(c), s.cpu().numpy().copy()
        scored.append(wc, ws, n.float().cpu().numpy(), lens, new or [n_new] * B, block,
                      dtype == INT8)
        wants += [wc, ws]
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    binding.attn_cache_append(kn, vn, kc, vc, ks, vs, lens_t, block_tokens=block, new_lens=new_t)
    binding.check()
    for got, want in zip((_values(kc), ks.cpu().numpy(), _values(vc), vs.cpu().numpy()), wants):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
def test_append_of_zeros_and_tiny_values(dtype):
    """The least scale is 2^-100: zeros stay zero and nothing becomes NaN."""
    kc, ks, _ = _cache(1, 1, 32, 16, dtype, 16, 2)
    vc, vs, _ = _cache(1, 1, 32, 16, dtype, 16, 4)
    kn = torch.zeros((1, 1, 16, 16), dtype=BF16, device="cuda")
    vn = torch.full((1, 1, 16, 16), 1e-38, dtype=BF16, device="cuda")
    binding.attn_cache_append(kn, vn, kc, vc, ks, vs, None, block_tokens=16)
    binding.check()
    assert not _values(kc)[:, :, :16].any() and not _values(vc)[:, :, :16].any()
    assert ks[0, 0, 0] == 2.0 ** -100 and vs[0, 0, 0] == 2.0 ** -100


def test_append_into_a_token_major_cache_leaves_the_rest():
    """[B, L, h, d] caches: only the new rows change."""
    B, h, L, d, block = 2, 2, 64, 64, 16
    k = torch.full((B, L, h, d), 5, dtype=INT8, device="cuda")
    v = torch.full((B, L, h, d), 6, dtype=INT8, device="cuda")
    ks, vs = (torch.full((B, h, L // block), 9.0, device="cuda") for _ in "kv")
    x = _random((B, h, 3, d), 1).to(BF16)
    lens = torch.tensor([16, 32], dtype=torch.int32, device="cuda")
    binding.attn_cache_append(x, x, k.transpose(1, 2), v.transpose(1, 2), ks, vs, lens,
                              block_tokens=block)
    binding.check()
    for c, fill, s in ((k, 5, ks), (v, 6, vs)):
        for b, n in enumerate((16, 32)):
            new = torch.zeros(L, dtype=torch.bool)
            new[n:n + 3] = True
            assert (c[b][~new.cuda()] == fill).all() and (c[b][new.cuda()] != fill).any()
            rest = [i for i in range(L // block) if i != n // block]
            assert (s[b][:, rest] == 9.0).all() and (s[b][:, n // block] != 9.0).all()


@pytest.mark.parametrize("dtype", [E4M3, INT8], ids=["e4m3", "int8"])
def test_prompt_then_steps_as_a_captured_graph(dtype):
    """A ragged prompt into an empty cache, then decoding steps (append one
    token, attend) replayed from one captured graph, against the reference run
    token by token."""
    B, h, hk, L, d, block, steps = 2, 4, 2, 160, 64, 16, 5
    ks, vs = (torch.zeros((B, hk, L // block), device="cuda") for _ in "kv")
    kc, vc = (torch.zeros((B, hk, L, d), dtype=dtype, device="cuda") for _ in "kv")
    slopes = _slopes(h)
    prompt = [_random((B, hk, 60, d), s).to(BF16) for s in (1, 2)]
    new = torch.tensor([60, 31], dtype=torch.int32, device="cuda")
    binding.attn_cache_append(*prompt, kc, vc, ks, vs, None, block_tokens=block, new_lens=new)
    ref = [[np.zeros((B, hk, L, d)), np.zeros((B, hk, L // block), np.float32)] for _ in "kv"]
    for r, x in zip(ref, prompt):
        scored.append(*r, x.float().cpu().numpy(), [0, 0], [60, 31], block, dtype == INT8)
    lens = new.clone()
    x = [torch.empty((B, n, 1, d), dtype=BF16, device="cuda") for n in (h, hk, hk)]
    out = torch.empty((B, h, 1, d), dtype=BF16, device="cuda")
    lse = torch.empty((B, h, 1), device="cuda")

    def step():
        binding.attn_cache_append(x[1], x[2], kc, vc, ks, vs, lens, block_tokens=block)
        lens.add_(1)
        binding.attn_decode_scored(x[0], kc, vc, lens, k_scale=ks, v_scale=vs,
                                   block_tokens=block, softcap=30.0, slopes=slopes, out=out,
                                   lse=lse)
    saved = [t.clone() for t in (kc, vc, ks, vs, lens)]
    for t in x:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # outside the capture once
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((kc, vc, ks, vs, lens), saved):
        t.copy_(s)
    at = [60, 31]
    for i in range(steps):
        for n, t in enumerate(x):
            t.copy_(_random(t.shape, 100 + 10 * i + n))
        graph.replay()
        torch.cuda.synchronize()
        for r, t in zip(ref, x[1:]):
            scored.append(*r, t.float().cpu().numpy(), at, [1] * B, block, dtype == INT8)
        at = [n + 1 for n in at]
        assert lens.tolist() == at
        k, v = (c * np.repeat(s.astype(np.float64), block, 2)[..., None] for c, s in ref)
        _check((out, lse), x[0], k, v, at, 0.125, 30.0, slopes, None, dtype)
    for got, (c, s) in zip(((kc, ks), (vc, vs)), ref):
        np.testing.assert_array_equal(_values(got[0]), c)
        np.testing.assert_array_equal(got[1].cpu().numpy(), s)


def test_two_steps_at_once_on_two_streams():
    """Calls on two streams with their own workspaces do not disturb one another."""
    B, h, L, d, block = 1, 2, 20000, 64, 64
    kc, ks, _ = _cache(B, h, L, d, E4M3, block, 2)
    vc, vs, _ = _cache(B, h, L, d, E4M3, block, 4)
    qs = [_random((B, h, 1, d), s).to(BF16) for s in (7, 8)]
    want = [binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, (q, st) in enumerate(zip(qs, streams)):
            got[i].append(binding.attn_decode_scored(q, kc, vc, k_scale=ks, v_scale=vs, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("window", [63, 64, 2 ** 31 - 1, 2 ** 32, 2 ** 40])
def test_decode_scored_window_longer_than_the_cache(window):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g).to(torch.bfloat16).cuda()
               for s in ((2, 4, 2, 64), (2, 2, 64, 64), (2, 2, 64, 64)))
    for a, b in zip(binding.attn_decode_scored(q, k, v, window=window),
                    binding.attn_decode_scored(q, k, v)):
        assert torch.equal(a, b)
    binding.check()
