"""A bf16 cache has no blocks of scales: attn_decode_tree and attn_cache_append_tree take it
with any block_tokens, as attn_decode_scored does."""
import pytest
import torch

from transformer_head_scaled_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from transformer_head_scaled_gb300.build import build
    build()
    return binding.load()


@pytest.mark.parametrize("n", [4, 40])
def test_block_tokens_of_a_bf16_cache(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    q, kt, vt = (torch.randn((2, 1, n, 64), generator=g, device="cuda").bfloat16() for _ in range(3))
    kc, vc = (torch.randn((2, 1, 90, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    lens = torch.tensor([40, 3], dtype=torch.int32, device="cuda")
    path = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    kept = torch.tensor([n, 2], dtype=torch.int32, device="cuda")
    res = []
    for block in (64, 0, 7):
        caches = kc.clone(), vc.clone()
        out = binding.attn_decode_tree(q, kt, vt, parents, *caches, lens, block_tokens=block)
        binding.attn_decode_scored(q[:, :, :4], *caches, lens, block_tokens=block)
        binding.attn_cache_append_tree(kt, vt, path, kept, *caches, lens, block_tokens=block)
        res.append((*out, *caches))
    binding.check()
    for other in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], other))


@pytest.mark.parametrize("block", [0, 7, 256])
def test_block_tokens_of_an_8_bit_cache(block):
    x = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((1, 1, 32, 64), dtype=torch.int8, device="cuda")
    s = torch.ones(1, device="cuda")
    ids = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        binding.attn_decode_tree(x, x, x, ids, c, c, None, s, s, block)
    with pytest.raises(ValueError):
        binding.attn_cache_append_tree(x, x, ids, ids[0, :1], c, c, None, s, s, block)
