"""attn_tree_verify refuses outputs that overlap its inputs or one another on the host,
before any CUDA call: the CTAs of a sequence read its tree each for itself."""
import pytest

from transformer_head_scaled_gb300 import binding
from transformer_head_scaled_gb300.build import build

INV, UNS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED
B, n, V = 3, 4, 100
# fake addresses, never dereferenced, far from one another
AT = {name: 0x100000 * (i + 1) for i, name in enumerate(
    ("target", "draft", "tokens", "parents", "uniforms", "path", "path_lens", "next_tokens"))}


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def _call(n=n, strides=None, kind=binding.PROB_F32, **at):
    return binding.attn_tree_verify_raw(*{**AT, **at}.values(), B, n, V, strides, kind, None)


@pytest.mark.parametrize("out", ["path", "path_lens", "next_tokens"])
def test_outputs_over_inputs_are_refused(lib, out):
    small = {name: 4 * B * n for name in ("tokens", "parents", "uniforms")}
    rows = {name: 4 * B * n * V for name in ("target", "draft")}
    for name, size in {**small, **rows}.items():
        for off in (0, 4, size - 4):
            assert _call(**{out: AT[name] + off}) == INV, (name, off)
    size = 4 * B * (n if out == "path" else 1)
    for name in small:  # the output's last entry over the input's first
        assert _call(**{out: AT[name] - size + 4}) == INV, name


def test_outputs_over_one_another_are_refused(lib):
    for off in (0, 4, 4 * B * n - 4):
        assert _call(path_lens=AT["path"] + off) == INV
        assert _call(next_tokens=AT["path"] + off) == INV
    for off in (-4 * (B - 1), 0, 4 * (B - 1)):
        assert _call(next_tokens=AT["path_lens"] + off) == INV


def test_strides_and_types_count(lib):
    wide = [1000, 200, 1000, 200]
    last = 4 * ((B - 1) * 1000 + (n - 1) * 200 + V) - 4
    assert _call(strides=wide, path=AT["target"] + last) == INV
    assert _call(strides=wide, path=AT["draft"] + last) == INV
    assert _call(strides=[0, 0, 0, 0], path=AT["target"] + 4 * (V - 1)) == INV
    assert _call(kind=binding.PROB_BF16, path=AT["target"] + 2 * B * n * V - 4) == INV
    assert _call(n=129, path=AT["tokens"]) == UNS  # sizes first
