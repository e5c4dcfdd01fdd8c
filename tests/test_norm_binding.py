"""Layer norm: what the binding takes and what it says of calls that the library
refuses.  Without a GPU: helpers that only look at shapes, types, strides and
addresses."""
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


def test_a_single_groups_affine_may_have_one_dimension():
    one, two = F.make_norm(4, 64), F.make_norm(4, 64, groups=2)
    w = torch.ones(64)
    assert F._affine(w, one, "weight") == w.data_ptr() and F._affine(None, one, "weight") is None
    assert F._affine(w.view(1, 64), one, "weight") == w.data_ptr()
    for norm, bad in ((two, w), (two, torch.ones(128)), (one, torch.ones(32)), (one, w.double()),
                      (one, torch.ones(128)[::2]), (one, torch.ones(64, 1))):
        with pytest.raises(ValueError, match="bias: expected"):
            F._affine(bad, norm, "bias")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(torch.float32, F.F32), (torch.bfloat16, F.BF16)])
def test_one_dimensional_weights(dtype, code):
    """The weight and bias of a torch layer norm as they are, and gradients of
    their shape: the bits of the [1, channels] call."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, dy = (torch.randn(7, 5, 96, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w, b = (torch.randn(96, generator=gen, device="cuda") for _ in range(2))
    norm = F.make_norm(35, 96, dtype=code)
    ws = F.norm_workspace(norm)
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    dx, dw, db = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w)
    assert dw.shape == db.shape == w.shape
    y2, _, _ = F.layer_norm_fwd(norm, x, weight=w[None], bias=b[None])
    dx2, dw2, db2 = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w[None])
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2[0]) and torch.equal(db, db2[0])
    out = (None, torch.empty_like(w), torch.empty_like(w))
    assert torch.equal(F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w, grads=out)[1], dw2[0])
