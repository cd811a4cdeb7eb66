"""Verification of drafted trees (attn_tree_verify) on rows that hold NaN: it counts as 0
in the target's rows and in the draft's."""
import math

import pytest
import torch

from oracle import tree
from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from transformer_head_scaled_gb300.build import build
    build()
    return binding.load()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(40, 12), (6, 1001), (3, 4096), (1, 140000)])
def test_nan_counts_as_zero(B, V, dtype):
    """Every third value of the draft's rows and every fifth of the target's.  Children
    that the draft likes far better than the target does, so that most are rejected, and a
    last one, in every second sequence, whose draft's value is NaN.  Zeros in the same
    places give the same answers."""
    n = min(9, V // 2)
    g = torch.Generator(device="cuda").manual_seed(B)
    p, q = (torch.softmax(2 * torch.randn((B, n, V), generator=g, device="cuda"), -1).to(dtype)
            for _ in range(2))
    parents = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    liked = (q[:, 0].float() - 4 * p[:, 0].float())
    liked[:, 1::3] = -1.0
    tokens = liked.topk(n, -1).indices.to(torch.int32)
    tokens[1::2, -1] = 1
    u = torch.rand((B, n), generator=g, device="cuda") * 0.25 + 0.75
    rows = {}
    for fill in (0.0, math.nan):
        a, b = p.clone(), q.clone()
        a[:, :, 2::5], b[:, :, 1::3] = fill, fill
        rows[fill] = binding.attn_tree_verify(a, tokens, parents, u, draft=b)
        alone = binding.attn_tree_verify(a, tokens, parents, u)
        rows[fill] = (*rows[fill], *alone)
        binding.check()
    assert all(torch.equal(x, y) for x, y in zip(*rows.values()))
    assert (rows[0.0][1] == 1).any()  # (walks that end at the root, after rejections)


def test_a_token_of_the_drafts_nan_may_follow():
    """p = (1/4, 1/2, 1/4), q = (1, 0, NaN): what is left after a rejection of token 0 is
    tokens 1 and 2, two thirds and one."""
    p = torch.tensor([[[0.25, 0.5, 0.25]] * 2], device="cuda")
    q = torch.tensor([[[1.0, 0.0, math.nan]] * 2], device="cuda")
    tokens = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for u0, want in ((0.0, 1), (0.66, 1), (0.67, 2), (0.99, 2)):
        u = torch.tensor([[u0, 0.5]], device="cuda")
        path, lens, token = binding.attn_tree_verify(p, tokens, tokens, u, draft=q)
        want_path, r, _ = tree.verify(p[0].double().cpu().numpy(), [0, 0], [-1, 0],
                                      u[0].cpu().numpy(), q[0].double().cpu().numpy())
        assert want_path == [0] and tree.next_tokens(r, u0, 1e-9) == {want}
        assert lens.tolist() == [1] and path.tolist() == [[0, -1]] and token.tolist() == [want]


def test_buffers_side_by_side():
    """Inputs and outputs as neighbours in one buffer are no overlap; in place is refused."""
    B, n, V = 2, 3, 50
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn((B, n, V), generator=g, device="cuda"), -1)
    parents = torch.tensor([[-1, 0, 1], [-1, 0, 0]], dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand((B, n), generator=g, device="cuda") * 0.02
    want = binding.attn_tree_verify(p, tokens, parents, u)
    flat = torch.zeros(3 * B * n + 2 * B, dtype=torch.int32, device="cuda")
    parts = flat.split([B * n, B * n, B, B, B * n])
    tok, path, lens, token, par = (parts[0].view(B, n), parts[1].view(B, n), parts[2], parts[3],
                                   parts[4].view(B, n))
    tok.copy_(tokens)
    par.copy_(parents)
    got = binding.attn_tree_verify(p, tok, par, u, path=path, path_lens=lens, next_tokens=token)
    binding.check()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(par, parents)
    for kw in (dict(path=tok), dict(path=par), dict(path=lens.new_empty(1), path_lens=lens),
               dict(path_lens=token, next_tokens=token), dict(path_lens=tok.view(-1)[:B])):
        with pytest.raises((binding.AttnError, ValueError)):
            binding.attn_tree_verify(p, tok, par, u, **kw)
