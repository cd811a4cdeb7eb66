"""What the entry points of the 8-bit cache and of attention with changed scores refuse
before any CUDA call, beside test_scored_boundary_cpu: other devices' streams and
sizes whose arithmetic would leave int."""
import pytest
import torch

from transformer_head_scaled_gb300 import binding
from transformer_head_scaled_gb300.build import build

A = 0x10000  # a fake, never dereferenced, 16-byte aligned device address


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def test_a_stream_of_another_device_is_refused():
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
            self.cuda_stream = A
    with pytest.raises(ValueError, match="stream"):
        binding._call_on(torch.device("cuda", 0), Stream(1))
    with pytest.raises(ValueError, match="stream"):
        binding._call_on(torch.device("cuda", 1), Stream(0))


def test_append_to_caches_past_the_index_arithmetic_is_refused(lib):
    def call(L, n_new=1):
        return binding.attn_cache_append_raw(A, A, A, A, A, A, 2, 1, n_new, L, 16, None,
                                             binding.CACHE_E4M3, 16, A, None, None)
    for L in ((1 << 30) + 1, 2 ** 31 - 1):
        assert call(L) == binding.ATTN_ERR_UNSUPPORTED, L
        assert call(L, n_new=L) == binding.ATTN_ERR_UNSUPPORTED, L


@pytest.mark.parametrize("cap,ok", [(2.0 ** 64, True), (2.0 ** 64 * (1 + 2.0 ** -23), False),
                                    (1e30, False), (3e38, False)])
def test_caps_above_2_to_the_64_are_refused(lib, cap, ok):
    """(2^64 itself gets past this check, to that of the head size or the queries.)"""
    got = (binding.attn_fwd_scored_raw(A, A, A, A, None, 1, 2, 1, 8, 8, 48, None, 0.125, cap, None,
                                       None, 0, None),
           binding.attn_bwd_scored_raw(A, A, A, A, A, A, A, A, A, 1, 2, 1, 8, 8, 48, None, 0.125, cap,
                                       None, None, 0, A, 1 << 40, None),
           binding.attn_decode_scored_raw(A, A, A, A, A, A, None, 1, 2, 1, 9, 64, 64, None,
                                          binding.CACHE_E4M3, 64, 0.125, cap, None, None, -1, None,
                                          0, None))
    want = binding.ATTN_ERR_UNSUPPORTED if ok else binding.ATTN_ERR_INVALID_ARG
    assert all(rc == want for rc in got), got


def test_scales_that_something_is_divided_by_are_refused_below_2_to_the_minus_64(lib):
    def fwd(scale, slopes):
        return binding.attn_fwd_scored_raw(A, A, A, A, None, 1, 2, 1, 8, 8, 48, None, scale, 0.0,
                                           slopes, None, 0, None)

    def bwd(scale):
        return binding.attn_bwd_scored_raw(A, A, A, A, A, A, A, A, A, 1, 2, 1, 8, 8, 48, None, scale,
                                           0.0, None, None, 0, A, 1 << 40, None)
    assert fwd(2.0 ** -65, A) == bwd(2.0 ** -65) == binding.ATTN_ERR_INVALID_ARG
    assert fwd(2.0 ** -64, A) == bwd(2.0 ** -64) == binding.ATTN_ERR_UNSUPPORTED
    assert fwd(2.0 ** -65, None) == binding.ATTN_ERR_UNSUPPORTED
