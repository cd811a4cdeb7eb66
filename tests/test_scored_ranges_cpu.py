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
