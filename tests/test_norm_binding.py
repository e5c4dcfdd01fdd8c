"""Layer norm: what the binding says of calls that the library refuses (no GPU
needed: these helpers only look at shapes, types, strides and addresses)."""
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F


@pytest.mark.parametrize("dtype,code", [(torch.float32, F.F32), (torch.bfloat16, F.BF16)])
def test_rows_that_start_inside_16_bytes_are_named(dtype, code):
    """x[1:] of a contiguous tensor of odd width starts inside a 16-byte line:
    the error says so and names the tensor."""
    norm = F.make_norm(5, 1001, dtype=code)
    x = torch.zeros(6, 1001, dtype=dtype)
    assert x.data_ptr() % 16 == 0 and x[1:].data_ptr() % 16
    assert F._rows(x[:5], norm, 0, "x") == x.data_ptr()
    with pytest.raises(ValueError, match="dy: .*16-byte"):
        F._rows(x[1:], norm, 0, "dy")
    none = F.make_norm(0, 1001, dtype=code)                     # no rows: no address
    F._rows(x[6:], none, 0, "x")
