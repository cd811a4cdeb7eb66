"""Attention with changed scores, and the 8-bit key/value cache: what is measured.

Four operators of the library, each in its plain form (elementary torch
operations in 32 bits) and, where ``own`` is set, as the call a user makes:

  fwd     attention whose scores are capped by a tanh and biased by distance,
          under masks that leave each query one run of keys (causal, window,
          key padding, documents packed in one row, a prefix all may see),
          with query heads that share key heads;
  bwd     its gradients;
  append  new keys and values into a cache held in 8 bits with one scale for
          each block of tokens and head;
  decode  a few new queries against such a cache (or a bf16 one), with the
          same capped and biased scores.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
INT8_MAX = 127.0
SCALE_MIN = 2.0 ** -100  # the least scale of a block: its reciprocal is finite
# A mean cache or document length below stands for lengths drawn evenly, so
# work() counts the expected number of visible pairs.
ATTN = dict(op="fwd", B=1, h=8, group=1, n=64, d=64, mask="causal", left=0, docs=0, cap=0.0,
            alibi=False, gain=1.0, packed=False)
CACHE = dict(op="append", B=1, h=8, group=1, L=512, d=64, n_new=1, fmt="e4m3", T=64)
DECODE = dict(op="decode", B=1, h=8, group=1, L=512, d=64, n_new=1, fmt="e4m3", T=64, cap=0.0,
              alibi=False, gain=1.0, window=-1, lo=0.125)


def listed():
    return [
        # the forward of one short sequence, where the launch counts
        dict(ATTN, name="fwd_alibi_short", alibi=True),
        # a batch of sentences with a prefix that every position may see, odd length
        dict(ATTN, name="fwd_prefix_base", B=64, n=501, mask="prefix"),
        # training on long rows packed with documents, capped scores, shared key heads
        dict(ATTN, name="fwd_docs_cap_d128", B=4, h=16, group=4, n=4096, d=128,
             mask="docs_causal", docs=6, cap=50.0, gain=2.0, packed=True),
        # the big model's long causal sequences with the distance bias
        dict(ATTN, name="fwd_alibi_big", B=8, h=16, n=4096, mask="causal", alibi=True),
        # gradients of small packed documents, odd length, shared key heads
        dict(ATTN, name="bwd_docs_cap_odd", op="bwd", B=2, h=8, group=4, n=333, d=32,
             mask="docs_causal", docs=4, cap=30.0, gain=2.0),
        # gradients of long packed rows, capped scores, shared key heads
        dict(ATTN, name="bwd_docs_cap_long", op="bwd", B=4, h=16, group=4, n=4096,
             mask="docs_causal", docs=6, cap=50.0, gain=2.0, packed=True),
        # gradients of the big model's long causal sequences with the distance bias
        dict(ATTN, name="bwd_alibi_big", op="bwd", B=8, h=16, n=4096, mask="causal", alibi=True),
        # one new token for each of many sequences (a decoding step's write)
        dict(CACHE, name="append_token_int8", B=256, fmt="int8"),
        # prompts of ragged lengths written to the cache
        dict(CACHE, name="append_prompt_e4m3", B=32, h=16, L=4096, n_new=2048, T=128),
        # a decoding step over beams, base model
        dict(DECODE, name="decode_beam_int8", B=256, fmt="int8"),
        # a decoding step over long caches, capped scores, big model
        dict(DECODE, name="decode_long_cap_e4m3", B=32, h=16, L=4096, cap=50.0, gain=2.0, lo=0.5,
             T=128),
        # one of very long contexts with shared key heads and the distance bias
        dict(DECODE, name="decode_context_gqa", B=4, h=32, group=4, L=131072, d=128, alibi=True,
             lo=0.5, T=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "append", "decode", "decode"])
    if op in ("fwd", "bwd"):
        d = rng.choice([16, 32, 64, 128] if op == "fwd" else [16, 32, 64])
        group = rng.choice([1, 1, 2, 4])
        h = group * rng.choice([1, 2, 4, 8])
        B, n = _log(rng, 1, 64), _log(rng, 17, 4096)
        mask = rng.choice(["none", "causal", "window", "padding", "docs", "docs_causal", "prefix"])
        # no more pairs than the largest listed case has
        while B * h * n * n > 8 * 16 * 4096 * 4096:
            B = max(1, B // 2)
        return dict(ATTN, op=op, B=B, h=h, group=group, n=n, d=d, mask=mask,
                    left=_log(rng, 8, 1024) if mask == "window" else 0,
                    docs=rng.randint(2, 9) if mask.startswith("docs") else 0,
                    cap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                    gain=rng.choice([1.0, 2.0]), packed=rng.random() < 0.5)
    T = rng.choice([16, 32, 64, 128])
    d = rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 256)
    if op == "append":
        h, n_new = rng.choice([1, 2, 4, 8, 16]), _log(rng, 1, 2048)
        L = T * max(1, _log(rng, 512, 8192) // T, -(-n_new // T))
        while B * h * L * d > 32 * 16 * 4096 * 64:
            B = max(1, B // 2)
            h = max(1, h // 2) if B == 1 else h
        return dict(CACHE, B=B, h=h, L=L, d=d, n_new=n_new, T=T,
                    fmt=rng.choice(["e4m3", "int8"]))
    group = rng.choice([1, 2, 4, 8])
    h = group * rng.choice([1, 2, 4, 8])
    L = T * max(1, _log(rng, 256, 131072) // T)
    while B * (h // group) * L * d > 4 * 8 * 131072 * 128 // 4:
        B, L = max(1, B // 2), (L if B > 1 else T * max(1, L // T // 2))
    return dict(DECODE, B=B, h=h, group=group, L=L, d=d, T=T,
                n_new=rng.choice([1, 1, 1, 2, 4, 5, 8]), fmt=rng.choice(["e4m3", "int8", "bf16"]),
                cap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                gain=rng.choice([1.0, 2.0]), lo=rng.choice([0.125, 0.5]),
                window=rng.choice([-1, -1, _log(rng, 64, 4096)]))


def _slopes(h, device):
    """The geometric slopes of the linear distance bias: 2^(-8 (i + 1) / h)."""
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c = dict(case)
    B, h, d = c["B"], c["h"], c["d"]
    hk = h // c["group"]
    scale = 1.0 / math.sqrt(d)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev)

    s = dict(c, scale=scale, slopes=_slopes(h, dev) if c.get("alibi") else None)
    if c["op"] in ("fwd", "bwd"):
        n = c["n"]
        if c["packed"]:  # one projection's output, [B, n, heads of q, k and v, d]
            x = normal(B, n, h + 2 * hk, d)
            x[:, :, :h] *= c["gain"]
            x = x.to(torch.bfloat16)
            s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in x.split([h, hk, hk], 2))
        else:
            s["q"] = (normal(B, h, n, d) * c["gain"]).to(torch.bfloat16)
            s["k"] = normal(B, hk, n, d).to(torch.bfloat16)
            s["v"] = normal(B, hk, n, d).to(torch.bfloat16)
        s["doc_ids"] = s["prefix_lens"] = s["key_lens"] = None
        if c["docs"]:  # rows cut into documents at random places
            cuts = ints(0, n, B, c["docs"] - 1)
            at = torch.arange(n, device=dev)
            s["doc_ids"] = (at[None, :, None] >= cuts[:, None, :]).sum(-1).to(torch.int32)
        if c["mask"] == "prefix":
            s["prefix_lens"] = ints(1, max(2, n // 2), B).to(torch.int32)
        if c["mask"] == "padding":
            s["key_lens"] = ints(max(1, n // 2), n + 1, B).to(torch.int32)
        if c["op"] == "bwd":
            s["dout"] = normal(B, h, n, d).to(torch.bfloat16)
            s["o"], s["lse"] = _attention(s)
        return s
    L, T, n_new, fmt = c["L"], c["T"], c["n_new"], c["fmt"]
    nblk = L // T
    if c["op"] == "append":
        x = normal(B, n_new, 2, h, d).to(torch.bfloat16)  # one projection's keys and values
        s["k_new"], s["v_new"] = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
        s["lens"] = ints(0, L - n_new + 1, B).to(torch.int32)
        s["new_lens"] = ints(max(1, n_new // 2), n_new + 1, B).to(torch.int32)
    else:
        s["q"] = (normal(B, h, n_new, d) * c["gain"]).to(torch.bfloat16)
        s["lens"] = ints(max(1, int(L * c["lo"])), L + 1, B).to(torch.int32)
    for name in ("k", "v"):
        if fmt == "bf16":
            s[name + "_cache"] = normal(B, hk, L, d).to(torch.bfloat16)
            s[name + "_scale"] = None
            continue
        # a block's largest value is about 4.3 standard deviations
        top = INT8_MAX if fmt == "int8" else E4M3_MAX
        codes = torch.empty((B, hk, L, d), device=dev,
                            dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
        for b in range(B):
            x = (normal(hk, L, d) * (top / 4.3)).clamp(-top, top)
            codes[b] = (x.round() if fmt == "int8" else x).to(codes.dtype)
        s[name + "_cache"] = codes
        s[name + "_scale"] = (4.3 / top) * (1 + 0.2 * torch.rand((B, hk, nblk), generator=g,
                                                                 device=dev))
    return s


# ----------------------------------------------------------------- plain forms

def _visible(s, device):
    """Which keys a query sees: [B or 1, n, n]."""
    n = s["n"]
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(n, device=device)[None, :]
    see = torch.ones((1, n, n), dtype=torch.bool, device=device)
    if s["mask"] in ("causal", "docs_causal"):
        see = see & (j <= i)
    if s["mask"] == "window":
        see = see & (j <= i) & (j >= i - s["left"])
    if s["prefix_lens"] is not None:
        see = see & ((j <= i) | (j < s["prefix_lens"][:, None, None]))
    if s["key_lens"] is not None:
        see = see & (j < s["key_lens"][:, None, None])
    if s["doc_ids"] is not None:
        see = see & (s["doc_ids"][:, :, None] == s["doc_ids"][:, None, :])
    return see


def _scores(s, q, k, tanh=None):
    """Capped and biased scores [B, hk, group, n, n], masked; and tanh(score / cap)."""
    x = torch.matmul(q, k.transpose(-1, -2)[:, :, None]).mul_(s["scale"])
    t = None
    if s["cap"] > 0:
        t = torch.tanh(x / s["cap"])
        x = t * s["cap"]
    if s["slopes"] is not None:
        at = torch.arange(s["n"], device=q.device)
        far = (at[:, None] - at[None, :]).abs().float()
        x -= s["slopes"].view(-1, s["group"], 1, 1) * far
    see = _visible(s, q.device)[:, None, None]
    return x.masked_fill_(~see, -math.inf), t


def _grouped(s, x):
    B, h, n, d = x.shape
    return x.float().view(B, h // s["group"], s["group"], n, d)


def _attention(s):
    q, k, v = _grouped(s, s["q"].contiguous()), s["k"].float(), s["v"].float()
    x, _ = _scores(s, q, k)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp_(x.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, :, None]) / torch.where(l > 0, l, 1.0)
    shape = s["q"].shape
    return o.view(shape).to(torch.bfloat16), (m + torch.log(l)).view(shape[:3])


def _gradients(s):
    q, k, v = _grouped(s, s["q"].contiguous()), s["k"].float(), s["v"].float()
    dout = _grouped(s, s["dout"])
    x, t = _scores(s, q, k)
    lse = s["lse"].view(x.shape[:-1]).unsqueeze(-1)
    p = torch.exp_(x.sub_(torch.where(lse == -math.inf, 0.0, lse)))
    dv = torch.matmul(p.transpose(-1, -2), dout).sum(2)
    dp = torch.matmul(dout, v.transpose(-1, -2)[:, :, None])
    dp -= (p * dp).sum(-1, keepdim=True)
    ds = dp.mul_(p)
    if t is not None:
        ds *= 1 - t * t
    dq = torch.matmul(ds, k[:, :, None]) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * s["scale"]
    return (dq.view(s["q"].shape).to(torch.bfloat16), dk.to(torch.bfloat16),
            dv.to(torch.bfloat16))


def _encode(x, fmt):
    """8-bit codes of x (already over its scale), nearest, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _append(s, new, cache, scale):
    """Writes new [B, h, n_new, d] behind the first lens[b] tokens.  A block's
    scale never shrinks while it fills: the codes it holds are rescaled."""
    B, h, L, d = cache.shape
    T, n_new, fmt = s["T"], s["n_new"], s["fmt"]
    nblk = L // T
    nb = min(nblk, (n_new + T - 1) // T + 1)  # blocks that one sequence's tokens can touch
    dev = cache.device
    lens, new_lens = s["lens"].long(), s["new_lens"].long()
    blk = (lens // T).clamp(max=nblk - nb)[:, None] + torch.arange(nb, device=dev)  # [B, nb]
    pos = blk[..., None] * T + torch.arange(T, device=dev)                          # [B, nb, T]
    at = pos - lens[:, None, None]
    fresh = (at >= 0) & (at < new_lens[:, None, None])
    held = (at < 0) & fresh.any(-1, keepdim=True)
    b = torch.arange(B, device=dev)
    x = new.transpose(1, 2)[b[:, None, None], at.clamp(0, n_new - 1)]  # [B, nb, T, h, d]
    x = x.permute(0, 3, 1, 2, 4).float()
    fresh, held = fresh[:, None, :, :, None], held[:, None, :, :, None]
    x = torch.where(fresh, x, 0.0)
    top = torch.full((), INT8_MAX if fmt == "int8" else E4M3_MAX, device=dev)
    blocks = cache.view(B, h, nblk, T, d)
    i = (b[:, None, None], torch.arange(h, device=dev)[None, :, None], blk[:, None, :])
    was = scale[i]                                                     # [B, h, nb]
    kept = torch.where(held.any(3)[..., 0], was, 0.0)
    now = torch.maximum(kept, x.abs().amax((-1, -2)) / top).clamp(min=SCALE_MIN)
    inv = torch.reciprocal(now)[..., None, None]
    codes = blocks[i]
    old = codes.float() * (kept[..., None, None] * inv)
    raw = codes.view(torch.int8)
    out = torch.where(held, _encode(old, fmt).view(torch.int8), raw)
    out = torch.where(fresh, _encode(x * inv, fmt).view(torch.int8), out)
    blocks.view(torch.int8)[i] = out
    scale[i] = torch.where(fresh.any(3)[..., 0], now, was)


def _widen(s, name):
    x = s[name + "_cache"].float()
    if s[name + "_scale"] is None:
        return x
    B, hk, L, d = x.shape
    return (x.view(B, hk, L // s["T"], s["T"], d) * s[name + "_scale"][..., None, None]).view(x.shape)


def _decode(s):
    """Query i of n_new stands at position lens[b] - n_new + i and sees the
    keys up to there (with a window: that key and the `window` ones before)."""
    q, k, v = _grouped(s, s["q"]), _widen(s, "k"), _widen(s, "v")
    x = torch.matmul(q, k.transpose(-1, -2)[:, :, None]) * s["scale"]  # [B, hk, g, n_new, L]
    if s["cap"] > 0:
        x = torch.tanh(x / s["cap"]) * s["cap"]
    n_new = s["n_new"]
    at = s["lens"].long()[:, None] - n_new + torch.arange(n_new, device=q.device)  # [B, n_new]
    back = at[..., None] - torch.arange(s["L"], device=q.device)                  # [B, n_new, L]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(-1, s["group"], 1, 1) * back[:, None, None].float()
    see = back >= 0
    if s["window"] >= 0:
        see = see & (back <= s["window"])
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, :, None]) / torch.where(l > 0, l, 1.0)
    shape = s["q"].shape
    return o.view(shape).to(torch.bfloat16), (m + torch.log(l)).view(shape[:3])


# ------------------------------------------------------------------------- run

def _own(s):
    from transformer_head_scaled_gb300 import binding
    if s["op"] in ("fwd", "bwd"):
        causal = s["mask"] in ("causal", "docs_causal", "window", "prefix")
        plan = binding.attn_mask_plan(
            s["B"], s["n"], s["n"], left=s["left"] if s["mask"] == "window" else None,
            right=0 if causal else None, key_lens=s["key_lens"], doc_ids=s["doc_ids"],
            prefix_lens=s["prefix_lens"], device=s["q"].device)
        if s["op"] == "fwd":
            return binding.attn_fwd_scored(s["q"], s["k"], s["v"], plan=plan, scale=s["scale"],
                                           softcap=s["cap"], slopes=s["slopes"])
        return binding.attn_bwd_scored(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"],
                                       plan=plan, scale=s["scale"], softcap=s["cap"],
                                       slopes=s["slopes"])
    if s["op"] == "append":
        binding.attn_cache_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                  s["k_scale"], s["v_scale"], s["lens"], block_tokens=s["T"],
                                  new_lens=s["new_lens"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return binding.attn_decode_scored(
        s["q"], s["k_cache"], s["v_cache"], s["lens"], k_scale=s["k_scale"],
        v_scale=s["v_scale"], block_tokens=s["T"], scale=s["scale"], softcap=s["cap"],
        slopes=s["slopes"], window=s["window"] if s["window"] >= 0 else None)


def run(state):
    """One call.  append returns the codes as the cache holds them (their
    rounding is part of what the operator is, so they have to be equal; e4m3
    codes are numbers of their own type) with the scales beside them."""
    if own:
        return _own(state)
    if state["op"] == "fwd":
        return _attention(state)
    if state["op"] == "bwd":
        return _gradients(state)
    if state["op"] == "append":
        _append(state, state["k_new"], state["k_cache"], state["k_scale"])
        _append(state, state["v_new"], state["v_cache"], state["v_scale"])
        return state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"]
    return _decode(state)


# ------------------------------------------------------------------------ work

def _pairs(c):
    """Expected visible (query, key) pairs of one row of the batch."""
    n = c["n"]
    if c["mask"] == "causal":
        return n * (n + 1) / 2
    if c["mask"] == "window":
        w = min(c["left"] + 1, n)
        return n * w - w * (w - 1) / 2
    if c["mask"] == "padding":
        return n * (0.75 * n)
    if c["mask"] == "prefix":  # the prefix (a quarter on average) sees itself whole
        return n * (n + 1) / 2 + (n / 2) ** 2 / 6
    if c["docs"]:  # mean of the squared lengths of pieces cut at even random places
        full = 2 * n * n / (c["docs"] + 1)
        return (full + n) / 2 if c["mask"] == "docs_causal" else full
    return n * n


def work(case):
    c = dict(case)
    B, h, d = c["B"], c["h"], c["d"]
    hk = h // c["group"]
    if c["op"] in ("fwd", "bwd"):
        n = c["n"]
        qo, kv, lse = 2 * B * h * n * d, 2 * B * hk * n * d, 4 * B * h * n
        if c["op"] == "fwd":
            return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4.0 * B * h * _pairs(c) * d}
        return {"bytes": 4 * qo + 4 * kv + lse, "flops": 10.0 * B * h * _pairs(c) * d}
    each = 2 if c["fmt"] == "bf16" else 1
    if c["op"] == "append":  # k and v: bf16 in, codes and scales out; lengths
        new = c["n_new"] if c["n_new"] == 1 else 0.75 * c["n_new"]
        return {"bytes": 2 * B * h * (new * d * (2 + each) + 4 * max(1, new / c["T"])) + 8 * B,
                "flops": 4.0 * B * h * new * d}
    seen = (1 + c["lo"]) / 2 * c["L"]
    if c["window"] >= 0:
        seen = min(seen, c["window"] + c["n_new"])
    scales = 0 if c["fmt"] == "bf16" else 2 * B * hk * 4 * seen / c["T"]
    return {"bytes": 2 * B * hk * seen * d * each + scales + 4 * B * h * c["n_new"] * (d + 1) + 4 * B,
            "flops": 4.0 * B * h * c["n_new"] * seen * d}


# ----------------------------------------------------------------------- exact

def _exact_head(s, b, hh, see, far):
    """One head in 64 bits: probabilities, the log-sum-exp, the cap's derivative."""
    q, k = s["q"][b, hh].double(), s["k"][b, hh // s["group"]].double()
    y = q @ k.T * s["scale"]
    slope = torch.ones_like(y) if s["cap"] > 0 and s["op"] == "bwd" else None
    if s["cap"] > 0:
        y = s["cap"] * torch.tanh(y / s["cap"])
        if slope is not None:
            slope = 1 - (y / s["cap"]) ** 2
    if s["slopes"] is not None:
        y = y - s["slopes"][hh].double() * far
    y = torch.where(see, y, -math.inf)
    lse = torch.logsumexp(y, -1)
    p = torch.exp(y - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return p, lse, slope


def _exact_attention(s):
    B, h, n, d = s["q"].shape
    dev, hk = s["q"].device, s["k"].shape[1]
    at = torch.arange(n, device=dev)
    far = (at[:, None] - at[None, :]).abs().double()
    o = torch.zeros((B, h, n, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, h, n), dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros((B, hk, n, d), dtype=torch.float64, device=dev)
                                        for _ in "kv")
    for b in range(B):
        # first and last key of each query, from the mask's definition
        lo, hi = torch.zeros_like(at), torch.full_like(at, n - 1)
        if s["doc_ids"] is not None:
            ids = s["doc_ids"][b].long()
            count = torch.bincount(ids, minlength=s["docs"])
            end = torch.cumsum(count, 0)[ids]
            lo, hi = end - count[ids], end - 1
        if s["mask"] in ("causal", "docs_causal", "window"):
            hi = torch.minimum(hi, at)
        if s["mask"] == "window":
            lo = torch.maximum(lo, at - s["left"])
        if s["prefix_lens"] is not None:
            hi = torch.maximum(at, s["prefix_lens"][b].long() - 1)
        if s["key_lens"] is not None:
            hi = torch.minimum(hi, s["key_lens"][b].long() - 1)
        see = (at[None, :] >= lo[:, None]) & (at[None, :] <= hi[:, None])
        for hh in range(h):
            g = hh // s["group"]
            p, lse[b, hh], slope = _exact_head(s, b, hh, see, far)
            v = s["v"][b, g].double()
            o[b, hh] = p @ v
            if s["op"] == "bwd":
                dout = s["dout"][b, hh].double()
                ds = p * (dout @ v.T - (dout * o[b, hh]).sum(-1, keepdim=True))
                if slope is not None:
                    ds = ds * slope
                dq[b, hh] = ds @ s["k"][b, g].double() * s["scale"]
                dk[b, g] += ds.T @ s["q"][b, hh].double() * s["scale"]
                dv[b, g] += p.T @ dout
    return (o, lse) if s["op"] == "fwd" else (dq, dk, dv)


def _exact_cache(s, name):
    """The codes before their rounding, and the scales, in 64 bits."""
    cache, scale, new = s[name + "_cache"].double(), s[name + "_scale"].double(), s[name + "_new"]
    T, top = s["T"], INT8_MAX if s["fmt"] == "int8" else E4M3_MAX
    lens, new_lens = s["lens"].tolist(), s["new_lens"].tolist()
    for b in range(s["B"]):
        end = lens[b] + new_lens[b]
        for blk in range(lens[b] // T, (end - 1) // T + 1):
            a, z = max(lens[b], blk * T), min(end, (blk + 1) * T)
            x = new[b, :, a - lens[b]:z - lens[b]].double()
            to = (x.abs().amax((-1, -2)) / top).clamp(min=SCALE_MIN)
            if a > blk * T:
                to = torch.maximum(to, scale[b, :, blk])
                cache[b, :, blk * T:a] *= (scale[b, :, blk] / to)[:, None, None]
            scale[b, :, blk] = to
            cache[b, :, a:z] = x / to[:, None, None]
    return (cache if s["fmt"] == "e4m3" else None), scale


def _exact_decode(s):
    B, h, n_new, d = s["q"].shape
    dev = s["q"].device
    o = torch.zeros((B, h, n_new, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, h, n_new), dtype=torch.float64, device=dev)
    lens = s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        wide = []
        for name in ("k", "v"):
            x = s[name + "_cache"][b, :, :n].double()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"][b].double().repeat_interleave(s["T"], 1)[:, :n, None]
            wide.append(x.repeat_interleave(s["group"], 0))
        y = torch.einsum("hid,hjd->hij", s["q"][b].double(), wide[0]) * s["scale"]
        if s["cap"] > 0:
            y = s["cap"] * torch.tanh(y / s["cap"])
        back = (n - n_new + torch.arange(n_new, device=dev))[:, None] - torch.arange(n, device=dev)
        if s["slopes"] is not None:
            y = y - s["slopes"].double()[:, None, None] * back
        see = (back >= 0) & (back <= (s["window"] if s["window"] >= 0 else n))
        y = torch.where(see, y, -math.inf)
        lse[b] = torch.logsumexp(y, -1)
        p = torch.exp(y - torch.where(torch.isinf(lse[b]), 0.0, lse[b])[..., None])
        o[b] = torch.einsum("hij,hjd->hid", p, wide[1])
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("fwd", "bwd"):
        return _exact_attention(s)
    if s["op"] == "append":
        (k, ks), (v, vs) = _exact_cache(s, "k"), _exact_cache(s, "v")
        return k, v, ks, vs
    return _exact_decode(s)
