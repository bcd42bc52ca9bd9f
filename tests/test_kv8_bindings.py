"""CPU checks of the bindings' own argument checks."""
import pytest
import torch


def test_request_strides():
    """Strides as the library takes them; requests that share or overlap storage are refused (their
    stride of 0 would mean contiguous requests: rows far past the tensor's end)."""
    from sparse_dense_kv_b200._lib import _request_stride as stride
    block = torch.zeros(4, 7, 2, 64, dtype=torch.bfloat16)
    assert stride(block, 7 * 128, "k_new") == 7 * 128
    assert stride(block[:, 3:4], 128, "k_new") == 7 * 128
    assert stride(block[:1, :2], 2 * 128, "k_new") == 2 * 128            # one request: its rows
    assert stride(block[:1].expand(1, 7, 2, 64), 7 * 128, "k_new") == 7 * 128
    assert stride(block[:, :0], 0, "k_new") == 7 * 128                   # no rows
    for bad, least in ((block[:1].expand(4, 7, 2, 64), 7 * 128), (block[0, :1].expand(3, 2, 64), 128),
                       (block.view(-1)[:10 * 128].as_strided((4, 2, 2, 64), (128, 128, 64, 1)), 2 * 128)):
        with pytest.raises(ValueError):
            stride(bad, least, "k_new")
