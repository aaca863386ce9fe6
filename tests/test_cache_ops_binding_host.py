"""What the Python binding of the cache-side operators refuses by itself (no GPU)."""
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 5, sys.maxsize, -1])
def test_token_counts_past_32_bits_are_refused(tsa, n):
    """2^32 + 5 is not 5: the library takes 32 bits, which ctypes would cut to."""
    cu = torch.tensor([0, 3, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="max_new"):
        tsa._offsets(cu, 5, n, 2, "max_new")
    with pytest.raises(ValueError, match="max_q"):
        tsa.window_attn_prefill_workspace(2, 8, 2, n, 1024, 4, 64, device="cpu")
    assert tsa._offsets(cu, 5, (1 << 31) - 1, 2, "max_new") == (1 << 31) - 1


def test_a_cache_of_two_shapes_or_devices_is_refused(tsa):
    """The kernels read v and the page table by k's shape on k's device."""
    k = torch.zeros((4, 2, 32, 128), dtype=torch.bfloat16)
    pt = torch.zeros((1, 4), dtype=torch.int32)
    for v in (k[:3].contiguous(), k[:, :1].contiguous(), k.view(4, 1, 64, 128)):
        with pytest.raises(ValueError, match="shape"):
            tsa.kv_contiguous(k, v)
        with pytest.raises(ValueError, match="shape"):
            tsa.kv_paged(k, v, pt)
    with pytest.raises(ValueError, match="v is on meta"):
        tsa.kv_contiguous(k, torch.zeros(k.shape, dtype=k.dtype, device="meta"))
    with pytest.raises(ValueError, match="page_table is on meta"):
        tsa.kv_paged(k, k, pt.to("meta"))
    assert tsa.kv_paged(k, k, pt).l_cap == 128
