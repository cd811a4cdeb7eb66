"""A decoding step over drafted tokens: what is measured.

Three operators of the library, each in its plain form (elementary torch
operations) and, where ``own`` is set, as the call a user makes:

  tree    attention of a tree of drafted tokens over a key/value cache: each
          node sees the cached tokens and its own ancestors;
  verify  which of the drafted tokens stand, given the target's (and the
          draft's) probabilities and random numbers, and the token after them;
  append  the keys and values of the accepted path into the cache, for all
          layers at once.

A tree of n nodes is an array of n parents: parents[0] = -1 is the root (the
newest token that stands already), every other node comes after its parent,
and a parent of -2 marks a place that holds no node (a batch of trees of
different sizes).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
INT8_MAX = 127.0
SCALE_MIN = 2.0 ** -100  # the least scale of a block: its reciprocal is finite
# A mean cache length below stands for lengths drawn evenly, so work() counts
# the expected number of visible keys.
TREE = dict(op="tree", B=1, h=8, group=1, n=8, L=512, d=64, fmt="bf16", T=64, shape="random",
            ragged=False, packed=False, cap=0.0, alibi=False, gain=1.0, window=-1, lo=0.5)
VERIFY = dict(op="verify", B=1, n=8, V=32000, dtype="f32", draft=True, shape="random",
              sharp=4.0, noise=1.0)
APPEND = dict(op="append", layers=1, B=1, h=8, n=8, L=512, d=64, fmt="bf16", T=64, packed=False)


def listed():
    return [
        # one sequence with a short draft, where the launches count
        dict(TREE, name="tree_chain_short", n=5, shape="chain"),
        # small trees for many sequences, 8-bit cache
        dict(TREE, name="tree_batch_int8", B=64, n=16, fmt="int8", lo=0.125),
        # long caches, capped scores, trees of different sizes, odd widths
        dict(TREE, name="tree_long_cap_e4m3", B=32, h=16, n=25, L=4096, fmt="e4m3", T=128,
             ragged=True, cap=50.0, gain=2.0),
        # big trees with shared key heads, a window and the distance bias
        dict(TREE, name="tree_window_alibi", B=8, h=32, group=8, n=61, L=16384, d=128, fmt="e4m3",
             alibi=True, window=2047, packed=True),
        # very long contexts with shared key heads
        dict(TREE, name="tree_context_gqa", B=4, h=32, group=4, n=64, L=131072, d=128,
             packed=True),
        # one sequence's short draft, where the launch counts
        dict(VERIFY, name="verify_chain_small", n=6, shape="chain"),
        # trees over a vocabulary of odd size
        dict(VERIFY, name="verify_tree_odd", B=32, n=24, V=50001),
        # trees of the draft's likeliest tokens (no chance in the draft), bf16
        dict(VERIFY, name="verify_top_bf16", B=64, n=64, V=131072, dtype="bf16", draft=False),
        # a large batch over a large vocabulary
        dict(VERIFY, name="verify_tree_batch", B=128, n=32, V=131072),
        # one layer's accepted tokens into a bf16 cache
        dict(APPEND, name="append_layer", B=8),
        # 8-bit codes, odd sizes
        dict(APPEND, name="append_int8_odd", layers=4, B=3, h=5, n=13, d=32, fmt="int8", T=16),
        # all layers' accepted tokens of a batch, 8-bit codes
        dict(APPEND, name="append_layers_e4m3", layers=24, B=32, n=32, d=128, fmt="e4m3",
             packed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "append"])
    shape = rng.choice(["random", "random", "chain"])
    T = rng.choice([16, 32, 64, 128])
    d = rng.choice([16, 32, 64, 128])
    if op == "tree":
        group = rng.choice([1, 2, 4, 8])
        h = group * rng.choice([1, 2, 4, 8])
        B, n = _log(rng, 1, 128), _log(rng, 1, 128)
        L = T * max(1, _log(rng, 128, 131072) // T)
        # no more cache and no more scores than the largest listed case has
        while (B * (h // group) * L * d > 4 * 8 * 131072 * 128 // 4
               or B * h * n * L > 4 * 32 * 64 * 131072 // 2):
            B, L = max(1, B // 2), (L if B > 1 else T * max(1, L // T // 2))
        return dict(TREE, B=B, h=h, group=group, n=n, L=L, d=d, T=T, shape=shape,
                    fmt=rng.choice(["bf16", "e4m3", "int8"]), ragged=rng.random() < 0.3,
                    packed=rng.random() < 0.5, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    alibi=rng.random() < 0.3, gain=rng.choice([1.0, 2.0]),
                    lo=rng.choice([0.125, 0.5]), window=rng.choice([-1, -1, _log(rng, 64, 4096)]))
    if op == "verify":
        B, n, V = _log(rng, 1, 128), _log(rng, 2, 64), _log(rng, 1000, 160000)
        while B * n * V > 128 * 32 * 131072 // 2:
            B = max(1, B // 2)
        return dict(VERIFY, B=B, n=n, V=V, dtype=rng.choice(["f32", "f32", "bf16"]),
                    draft=rng.random() < 0.7, shape=shape, sharp=rng.choice([2.0, 4.0]),
                    noise=rng.choice([0.3, 1.0]))
    layers, B, h = _log(rng, 1, 32), _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
    n = _log(rng, 1, 128)
    L = T * max(1, _log(rng, 256, 2048) // T, -(-n // T))
    while layers * B * h * L * d > 24 * 32 * 8 * 512 * 128 or layers * B * h * n > 24 * 32 * 8 * 32:
        layers, B = (max(1, layers // 2), B) if layers > B else (layers, max(1, B // 2))
    return dict(APPEND, layers=layers, B=B, h=h, n=n, L=L, d=d, T=T,
                fmt=rng.choice(["bf16", "e4m3", "int8"]), packed=rng.random() < 0.5)


def _slopes(h, device):
    """The geometric slopes of the linear distance bias: 2^(-8 (i + 1) / h)."""
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=device)


def _parents(c, g, dev):
    """[B, n] parents: a chain, or each node below an earlier one at random (most
    below one of the last few, as drafts that follow their best guess are)."""
    B, n = c["B"], c["n"]
    at = torch.arange(n, device=dev)
    if c["shape"] == "chain":
        parents = (at - 1).expand(B, n).clone()
    else:
        back = torch.rand((B, n), generator=g, device=dev) ** 2 * at  # nearer ones likelier
        parents = at - 1 - back.long().clamp(max=n)
        parents = torch.maximum(parents, torch.where(at > 0, 0, -1))
    if c.get("ragged"):
        size = torch.randint(max(1, n // 4), n + 1, (B, 1), generator=g, device=dev)
        parents = torch.where(at < size, parents, -2)
    return parents.to(torch.int32)


def _codes(c, name, s, shape, normal, g, dev):
    """A cache's rows (and scales) of the given format: [..., h, L, d]."""
    fmt, top = c["fmt"], INT8_MAX if c["fmt"] == "int8" else E4M3_MAX
    types = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
    codes = torch.empty(shape, device=dev, dtype=types[fmt])
    for part in codes.view(-1, *shape[-3:]).split(max(1, (1 << 27) // math.prod(shape[-3:]))):
        x = normal(*part.shape)
        if fmt != "bf16":  # a block's largest value is about 4.3 standard deviations
            x = (x * (top / 4.3)).clamp(-top, top)
        part.copy_((x.round() if fmt == "int8" else x).to(codes.dtype))
    s[name + "_cache"], s[name + "_scale"] = codes, None
    if fmt != "bf16":
        blocks = (*shape[:-2], shape[-2] // c["T"])
        s[name + "_scale"] = (4.3 / top) * (1 + 0.2 * torch.rand(blocks, generator=g, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c = dict(case)
    B, n = c["B"], c["n"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev)

    s = dict(c)
    if c["op"] == "tree":
        h, d, L = c["h"], c["d"], c["L"]
        hk = h // c["group"]
        s["scale"] = 1.0 / math.sqrt(d)
        s["slopes"] = _slopes(h, dev) if c["alibi"] else None
        s["parents"] = _parents(c, g, dev)
        if c["packed"]:  # one projection's output, [B, n, heads of q, k and v, d]
            x = normal(B, n, h + 2 * hk, d)
            x[:, :, :h] *= c["gain"]
            x = x.to(torch.bfloat16)
            s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in x.split([h, hk, hk], 2))
        else:
            s["q"] = (normal(B, h, n, d) * c["gain"]).to(torch.bfloat16)
            s["k"] = normal(B, hk, n, d).to(torch.bfloat16)
            s["v"] = normal(B, hk, n, d).to(torch.bfloat16)
        s["lens"] = ints(max(1, int(L * c["lo"])), L + 1, B).to(torch.int32)
        for name in ("k", "v"):
            _codes(c, name, s, (B, hk, L, d), normal, g, dev)
        return s
    if c["op"] == "verify":
        V, dtype = c["V"], torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        s["parents"] = _parents(c, g, dev)
        logits = normal(B, n, V).mul_(c["sharp"])
        s["target"] = torch.softmax(logits, -1).to(dtype)
        logits.add_(normal(B, n, V), alpha=c["noise"])  # the draft is about as the target is
        above = s["parents"].long().clamp(min=0)
        if c["draft"]:
            s["draft"] = torch.softmax(logits, -1).to(dtype)
            rows = s["draft"].float().view(B * n, V)
            rows = rows[(above + n * torch.arange(B, device=dev)[:, None]).view(-1)]
            s["tokens"] = torch.multinomial(rows, 1, generator=g).view(B, n).to(torch.int32)
        else:  # a node's children are the draft's likeliest tokens there, in order
            s["draft"] = None
            best = logits.topk(n, -1).indices
            earlier = torch.arange(n, device=dev)[:, None] > torch.arange(n, device=dev)
            rank = ((above[:, :, None] == above[:, None, :]) & earlier).sum(-1)
            b = torch.arange(B, device=dev)[:, None]
            s["tokens"] = best[b, above, rank].to(torch.int32)
        s["uniforms"] = torch.rand((B, n), generator=g, device=dev)
        return s
    layers, h, d, L = c["layers"], c["h"], c["d"], c["L"]
    x = normal(layers, B, n, 2, h, d).to(torch.bfloat16)  # one projection's keys and values
    s["k"], s["v"] = x[:, :, :, 0].transpose(2, 3), x[:, :, :, 1].transpose(2, 3)
    if not c["packed"]:
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    path = torch.cumsum(torch.cat([ints(0, 1, B, 1), ints(1, 4, B, n - 1)], 1), 1)
    most = (path < n).sum(-1)
    s["path_lens"] = (1 + (torch.rand(B, generator=g, device=dev) * most).long()).to(torch.int32)
    kept = torch.arange(n, device=dev) < s["path_lens"][:, None]
    s["path"] = torch.where(kept, path, -1).to(torch.int32)
    s["lens"] = ints(0, L - n + 1, B).to(torch.int32)
    for name in ("k", "v"):
        _codes(c, name, s, (layers, B, h, L, d), normal, g, dev)
    return s


# ----------------------------------------------------------------- plain forms

def _lineage(parents):
    """[B, n, n] whether node i has node j among its ancestors (or is it), and
    [B, n] its depth below the root; nothing of places without a node."""
    B, n = parents.shape
    at = torch.arange(n, device=parents.device)
    up = (parents[:, :, None] == at).float() + torch.eye(n, device=parents.device)
    for _ in range(max(1, (n - 1).bit_length())):  # paths of 1, 2, 4, ... steps
        up = (torch.matmul(up, up) > 0).float()
    see = (up > 0) & (parents[:, :, None] >= -1)
    return see, see.sum(-1) - 1


def _widen(s, name):
    x = s[name + "_cache"].float()
    if s[name + "_scale"] is None:
        return x
    shape = x.shape
    x = x.view(*shape[:-2], shape[-2] // s["T"], s["T"], shape[-1])
    return (x * s[name + "_scale"][..., None, None]).view(shape)


def _tree(s):
    """Node i stands at position lens[b] + depth_i and sees the cached keys (with
    a window: the `window` ones before its position) and its ancestors."""
    B, h, n, d = s["q"].shape
    g, L, dev = s["group"], s["L"], s["q"].device
    hk = h // g
    see_tree, depth = _lineage(s["parents"])
    node = s["parents"] >= -1
    at = s["lens"][:, None].long() + depth                                     # [B, n]
    back = at[:, :, None] - torch.arange(L, device=dev)                        # [B, n, L]
    see = node[:, :, None] & (torch.arange(L, device=dev) < s["lens"][:, None, None])
    back_tree = (depth[:, :, None] - depth[:, None, :])                        # [B, n, n]
    if s["window"] >= 0:
        see, see_tree = see & (back <= s["window"]), see_tree & (back_tree <= s["window"])
    q = s["q"].float().reshape(B, hk, g, n, d)

    def scores(k, see, back):
        x = torch.matmul(q, k.transpose(-1, -2)[:, :, None]).mul_(s["scale"])
        if s["cap"] > 0:
            x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
        if s["slopes"] is not None:
            x -= s["slopes"].view(-1, g, 1, 1) * back[:, None, None].float()
        return x.masked_fill_(~see[:, None, None], -math.inf)

    x = torch.cat([scores(_widen(s, "k"), see, back), scores(s["k"].float(), see_tree, back_tree)],
                  -1)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp_(x.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., :L], _widen(s, "v")[:, :, None])
    o += torch.matmul(p[..., L:], s["v"].float()[:, :, None])
    o /= torch.where(total > 0, total, 1.0)
    return (o.view(B, h, n, d).to(torch.bfloat16), (m + torch.log(total)).view(B, h, n))


def _verify(s):
    """From the root on, a node's children are tried in order: child c of token x
    stands if u_c * Z * q(x) < r(x).  At first r = p (the target's probabilities
    at the node) and Z = 1; after k children that did not stand r = max(p - C q, 0),
    Z = sum r, C the sum of the earlier Z: what is left of the target's
    probability.  Without the draft's probabilities q(x) = 1, and r is p without
    those children's tokens.  The next token is drawn from the r of the node
    where the walk ends.  (64 bits: every test is next to a border.)"""
    target, parents, tokens = s["target"], s["parents"], s["tokens"].long()
    B, n, V = target.shape
    dev = target.device
    b = torch.arange(B, device=dev)
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    length = torch.ones_like(cur)
    path = torch.full((B, n), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0
    taken = torch.zeros(B, dtype=torch.float64, device=dev)  # C
    left = torch.ones(B, dtype=torch.float64, device=dev)    # Z
    out = torch.zeros((B, V), dtype=torch.bool, device=dev)  # tokens that did not stand

    def rest():
        r = target[b, cur].double()
        if s["draft"] is None:
            return torch.where(out, 0.0, r)
        return (r - taken[:, None] * s["draft"][b, cur].double()).clamp(min=0)

    for c in range(1, n):  # children come after their parents, siblings in order
        here = parents[:, c] == cur
        x, u = tokens[:, c], s["uniforms"][:, c].double()
        p = target[b, cur, x].double()
        if s["draft"] is None:
            q = 1.0
            p = torch.where(out[b, x], 0.0, p)
        else:
            q = s["draft"][b, cur, x].double()
            p = (p - taken * q).clamp(min=0)
        stands = here & (u * left * q < p)
        fails = here & ~stands
        taken = torch.where(stands, 0.0, torch.where(fails, taken + left, taken))
        out[b, x] |= fails
        out &= ~stands[:, None]
        cur = torch.where(stands, c, cur)
        if s["draft"] is None:
            left = torch.where(stands, 1.0, torch.where(fails, left - p, left))
        else:
            left = torch.where(stands, 1.0, torch.where(fails, rest().sum(-1), left))
        path[b, length.clamp(max=n - 1)] = torch.where(stands, c, path[b, length.clamp(max=n - 1)])
        length = length + stands
    r = rest()
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, target[b, cur].double())
    upto = torch.cumsum(r, -1)
    token = (upto <= s["uniforms"][:, :1].double() * upto[:, -1:]).sum(-1)
    token = token.clamp(max=V - 1)
    return path.to(torch.int32), length.to(torch.int32), token.to(torch.int32)


def _encode(x, fmt):
    """8-bit codes of x (already over its scale), nearest, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _append(s, name):
    """Row i of the path goes behind the first lens[b] + i tokens.  A block's scale
    never shrinks while it fills: the codes it holds are rescaled."""
    tree, cache, scale = s[name], s[name + "_cache"], s[name + "_scale"]
    layers, B, h, L, d = cache.shape
    n, fmt, dev = s["n"], s["fmt"], cache.device
    lens, more = s["lens"].long(), s["path_lens"].long()
    b = torch.arange(B, device=dev)
    new = tree.permute(1, 3, 0, 2, 4)[b[:, None], s["path"].long().clamp(min=0)]
    # new [B, n, layers, h, d], cache as [B, L, layers, h, d]
    if fmt == "bf16":
        rows = lens[:, None] + torch.arange(n, device=dev)
        keep = (torch.arange(n, device=dev) < more[:, None])[..., None, None, None]
        view = cache.permute(1, 3, 0, 2, 4)
        view[b[:, None], rows] = torch.where(keep, new, view[b[:, None], rows])
        return
    T = s["T"]
    nblk = L // T
    nb = min(nblk, (n + T - 1) // T + 1)  # blocks that one sequence's tokens can touch
    blk = (lens // T).clamp(max=nblk - nb)[:, None] + torch.arange(nb, device=dev)  # [B, nb]
    at = blk[..., None] * T + torch.arange(T, device=dev) - lens[:, None, None]     # [B, nb, T]
    fresh = (at >= 0) & (at < more[:, None, None])
    held = (at < 0) & fresh.any(-1, keepdim=True)
    x = new[b[:, None, None], at.clamp(0, n - 1)].float()  # [B, nb, T, layers, h, d]
    fresh, held = fresh[..., None, None, None], held[..., None, None, None]
    x = torch.where(fresh, x, 0.0)
    top = torch.full((), INT8_MAX if fmt == "int8" else E4M3_MAX, device=dev)
    blocks = cache.view(layers, B, h, nblk, T, d).permute(1, 3, 4, 0, 2, 5)
    scales = scale.view(layers, B, h, nblk).permute(1, 3, 0, 2)
    i = (b[:, None], blk)
    was = scales[i]                                                 # [B, nb, layers, h]
    kept = torch.where(held.any(2)[..., 0], was, 0.0)
    now = torch.maximum(kept, x.abs().amax((2, 5)) / top).clamp(min=SCALE_MIN)
    inv = torch.reciprocal(now)[:, :, None, :, :, None]
    codes = blocks[i]                                               # [B, nb, T, layers, h, d]
    old = codes.float() * (kept[:, :, None, :, :, None] * inv)
    raw = codes.view(torch.int8)
    res = torch.where(held, _encode(old, fmt).view(torch.int8), raw)
    res = torch.where(fresh, _encode(x * inv, fmt).view(torch.int8), res)
    blocks.view(torch.int8)[i] = res
    scales[i] = torch.where(fresh.any(2)[..., 0], now, was)


# ------------------------------------------------------------------------- run

def _own(s):
    from transformer_head_scaled_gb300 import binding
    if s["op"] == "tree":
        return binding.attn_decode_tree(
            s["q"], s["k"], s["v"], s["parents"], s["k_cache"], s["v_cache"], s["lens"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], block_tokens=s["T"], scale=s["scale"],
            softcap=s["cap"], slopes=s["slopes"],
            window=s["window"] if s["window"] >= 0 else None)
    if s["op"] == "verify":
        return binding.attn_tree_verify(s["target"], s["tokens"], s["parents"], s["uniforms"],
                                        draft=s["draft"])
    binding.attn_cache_append_tree(s["k"], s["v"], s["path"], s["path_lens"], s["k_cache"],
                                   s["v_cache"], s["lens"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"], block_tokens=s["T"])
    return _caches(s)


def _caches(s):
    return [s[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale")
            if s[name] is not None]


def run(state):
    """One call.  append returns the codes as the cache holds them (their
    rounding is part of what the operator is, so they have to be equal; e4m3
    codes are numbers of their own type) with the scales beside them."""
    if own:
        return _own(state)
    if state["op"] == "tree":
        return _tree(state)
    if state["op"] == "verify":
        return _verify(state)
    _append(state, "k")
    _append(state, "v")
    return _caches(state)


# ------------------------------------------------------------------------ work

def work(case):
    c = dict(case)
    B, n = c["B"], c["n"]
    if c["op"] == "verify":
        # the target's and the draft's row where the walk ends, and each node's numbers
        rows, each = 2 if c["draft"] else 1, 4 if c["dtype"] == "f32" else 2
        return {"bytes": B * (rows * c["V"] * each + n * (12 + rows * each) + 4 * n + 8),
                "flops": 3.0 * B * c["V"]}
    each, h, d = 2 if c["fmt"] == "bf16" else 1, c["h"], c["d"]
    if c["op"] == "append":  # half of a path of at most about n / 2 nodes on average
        new = max(1.0, n / 4)
        scales = 0 if each == 2 else 8 * max(1, new / c["T"])
        return {"bytes": c["layers"] * 2 * B * h * (new * d * (2 + each) + scales) + 4 * B * (n + 2),
                "flops": 4.0 * c["layers"] * B * h * new * d}
    hk = h // c["group"]
    nodes = 0.625 * n if c["ragged"] else n
    seen = (1 + c["lo"]) / 2 * c["L"]
    if c["window"] >= 0:
        seen = min(seen, c["window"])
    scales = 0 if each == 2 else 2 * B * hk * 4 * seen / c["T"]
    return {"bytes": 2 * B * hk * (seen * d * each + 2 * n * d) + scales
            + 4 * B * h * n * (d + 1) + 4 * B * (n + 1),
            "flops": 4.0 * B * h * nodes * seen * d}


# ----------------------------------------------------------------------- exact

def _exact_tree(s):
    B, h, n, d = s["q"].shape
    dev, g = s["q"].device, s["group"]
    hk = h // g
    o = torch.zeros((B, h, n, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, h, n), -math.inf, dtype=torch.float64, device=dev)
    lens, parents = s["lens"].tolist(), s["parents"].tolist()
    for b in range(B):
        size = lens[b]
        line = [[] for _ in range(n)]  # each node's ancestors and itself, root first
        for i, p in enumerate(parents[b]):
            if p >= -1:
                line[i] = (line[p] if p >= 0 else []) + [i]
        wide = []
        for name in ("k", "v"):
            x = s[name + "_cache"][b, :, :size].double()
            if s[name + "_scale"] is not None:
                x *= s[name + "_scale"][b].double().repeat_interleave(s["T"], 1)[:, :size, None]
            wide.append(torch.cat([x, s[name][b].double()], 1))
        y = (s["q"][b].double().reshape(hk, g * n, d) @ wide[0].mT).view(h, n, -1) * s["scale"]
        if s["cap"] > 0:
            y = s["cap"] * torch.tanh(y / s["cap"])
        place = [size + len(a) - 1 for a in line]  # of the nodes
        keys = torch.tensor(list(range(size)) + place, device=dev)
        see = torch.zeros((n, size + n), dtype=torch.bool)
        for i, a in enumerate(line):
            if a:
                w = s["window"] + 1 if s["window"] >= 0 else size + n  # itself among them
                see[i, max(0, place[i] + 1 - w):size] = True
                see[i, [size + j for j in a[-w:]]] = True
        if s["slopes"] is not None:
            far = torch.tensor(place, device=dev)[:, None] - keys
            y -= s["slopes"].double()[:, None, None] * far
        y.masked_fill_(~see.to(dev), -math.inf)
        lse[b] = torch.logsumexp(y, -1)
        y -= torch.where(torch.isinf(lse[b]), 0.0, lse[b])[..., None]
        o[b] = (y.exp_().view(hk, g * n, -1) @ wide[1]).view(h, n, d)
    return o, lse


def _exact_verify(s):
    """One sequence at a time, from the definition of drawing with rejections."""
    B, n, V = s["target"].shape
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    chance = s["uniforms"].double().tolist()
    path = torch.full((B, n), -1, dtype=torch.int32)
    count = torch.zeros(B, dtype=torch.int32)
    token = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        walk = [0]
        while True:
            node, went = walk[-1], False
            weight = s["target"][b, node].double()  # what is left to draw from
            total = 1.0
            for c in [i for i in range(1, n) if parents[b][i] == node]:
                x = tokens[b][c]
                if s["draft"] is None:
                    went = chance[b][c] * total < float(weight[x])
                    if not went:
                        total -= float(weight[x])
                        weight = weight.clone()
                        weight[x] = 0.0
                else:
                    q = s["draft"][b, node].double()
                    went = chance[b][c] * total * float(q[x]) < float(weight[x])
                    if not went:
                        weight = torch.relu(weight - total * q)
                        total = float(weight.sum())
                if went:
                    walk.append(c)
                    break
            if not went:
                break
        if not bool((weight > 0).any()):
            weight = s["target"][b, node].double()
        upto = weight.cumsum(0)
        token[b] = torch.searchsorted(upto, upto[-1:] * chance[b][0], right=True)[0]
        path[b, :len(walk)] = torch.tensor(walk, dtype=torch.int32)
        count[b] = len(walk)
    return path, count, token


def _exact_append(s, name):
    """The cache (8-bit: the codes before their rounding) and the scales in 64 bits."""
    new, T = s[name], s["T"]
    cache = s[name + "_cache"].double() if s["fmt"] != "int8" else None
    scale = s[name + "_scale"]
    scale = None if scale is None else scale.double().view(s["layers"], s["B"], s["h"], -1)
    top = INT8_MAX if s["fmt"] == "int8" else E4M3_MAX
    lens, path = s["lens"].tolist(), s["path"].tolist()
    for b, more in enumerate(s["path_lens"].tolist()):
        x = new[:, b][:, :, path[b][:more]].double()  # [layers, h, more, d]
        start, end = lens[b], lens[b] + more
        if scale is None:
            cache[:, b, :, start:end] = x
            continue
        for blk in range(start // T, (end - 1) // T + 1):
            a, z = max(start, blk * T), min(end, (blk + 1) * T)
            part = x[:, :, a - start:z - start]
            to = (part.abs().amax((-1, -2)) / top).clamp(min=SCALE_MIN)
            if a > blk * T:
                was = scale[:, b, :, blk]
                to = torch.maximum(to, was)
                if cache is not None:
                    cache[:, b, :, blk * T:a] *= (was / to)[..., None, None]
            scale[:, b, :, blk] = to
            if cache is not None:
                cache[:, b, :, a:z] = part / to[..., None, None]
    return cache, scale


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tree":
        return _exact_tree(s)
    if s["op"] == "verify":
        return _exact_verify(s)
    (k, ks), (v, vs) = _exact_append(s, "k"), _exact_append(s, "v")
    return [k, v] if ks is None else [k, v, ks, vs]
