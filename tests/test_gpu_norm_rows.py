"""GPU parity of the layer norm on rows that are hard on its arithmetic:
one element far from the others, against the bounds of the other norm tests
(every rounding is one of the row's mean |x|, wherever the far element is)."""
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from tests.test_gpu_norm import DT, check_bwd, check_fwd, make, plain, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("far", [1e2, 1e4])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("rows,C", [(3, 64), (700, 64), (5, 1000), (2000, 1001), (4, 1024), (3, 5120), (600, 5120),
                                    (6, 8192), (700, 8192), (3, 10000)])
def test_one_far_element(rows, C, where, far, dtype):
    x, w, b, dy = make(rows, C, 1, dtype, 7)
    x = (x.float().clamp(-1, 1) + 1).to(DT[dtype][0])
    x[:, {"first": 0, "middle": C // 2, "last": C - 1}[where]] = far
    norm = F.make_norm(rows, C, 1, dtype=DT[dtype][1])
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    r = plain(x, w, b, dy, 1, 1e-6, False)
    check_fwd(y, mean, rstd, r, x, DT[dtype][2])
    check_bwd(*F.layer_norm_bwd(norm, x, dy, mean, rstd, F.norm_workspace(norm), weight=w), r, DT[dtype][2])


def test_the_mean_of_rows_with_an_infinity():
    """An infinite element makes the row's mean infinite and its y NaN; a NaN
    makes both NaN; the other rows stay as they are."""
    for rows, C in ((4, 64), (4, 3000), (900, 3000)):
        x = torch.randn(rows, C, generator=torch.Generator("cuda").manual_seed(0), device="cuda")
        norm = F.make_norm(rows, C, dtype=F.F32)
        y0, mean0, rstd0 = F.layer_norm_fwd(norm, x)
        x[1, C - 1], x[2, 0], x[3, C // 2] = float("inf"), -float("inf"), float("nan")
        y, mean, rstd = F.layer_norm_fwd(norm, x)
        assert mean[1] == float("inf") and mean[2] == -float("inf") and mean[3].isnan()
        assert y[1:4].isnan().all() and rstd[1:4].isnan().all()
        for i in (0, *range(4, rows, 100)):
            assert torch.equal(y[i], y0[i]) and mean[i] == mean0[i] and rstd[i] == rstd0[i]


def by_the_saved_statistics(x, dy, gain, mean, rstd, groups):
    """(dx, dw, their error scales) of the backward's formula in 64 bits, for the statistics it is given."""
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    gain = gain.double().repeat_interleave(x.shape[0] // groups, 0)
    xh, gy = (x - mean) * rstd, dy * gain
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    size = rstd * (gy.abs() + gy.abs().mean(1, keepdim=True) + xh.abs() * (gy * xh).abs().mean(1, keepdim=True))
    cols = lambda t: t.reshape(groups, -1, t.shape[1]).sum(1)  # noqa: E731
    return dx, cols(dy * xh), size, cols((dy * xh).abs())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C,groups", [(40, 64, 2), (300, 1001, 3), (150, 1536, 1), (60, 5120, 4), (8, 9000, 2)])
def test_backward_with_a_mean_far_above_the_deviation(rows, C, groups, dtype):
    """mean / std of 600 (three of 64 elements a step above the others:
    2^7 / sqrt(3/64 61/64)) to 12,000: x - mean is off by 2^-24 of itself, so dx and
    dweight keep the bounds of ordinary rows, 2^-18 and 2^-17 of their terms'
    magnitudes, for the statistics they are given."""
    gen = torch.Generator("cuda").manual_seed(12)
    if dtype == "f32":
        x = torch.randn(rows, C, generator=gen, device="cuda") + 4096.0
    else:                            # a few elements one bf16 step above the others
        x = torch.where(torch.rand(rows, C, generator=gen, device="cuda") < 2.0 ** -10, 1 + 2.0 ** -7, 1.0)
        x[:, 5] = 1 + 2.0 ** -7
        x = x.to(torch.bfloat16)
    dy = torch.randn(rows, C, generator=gen, device="cuda").to(DT[dtype][0])
    w = torch.randn(groups, C, generator=gen, device="cuda")
    norm = F.make_norm(rows, C, groups, dtype=DT[dtype][1], eps=0.0)
    _, mean, rstd = F.layer_norm_fwd(norm, x, weight=w)
    assert float((mean.abs() * rstd).min()) > 600
    dx, dw, db = F.layer_norm_bwd(norm, x, dy, mean, rstd, F.norm_workspace(norm), weight=w)
    want_dx, want_dw, size, aw = by_the_saved_statistics(x, dy, w, mean, rstd, groups)
    within(dx, want_dx, DT[dtype][2] * want_dx.abs() + 2.0 ** -18 * size, "dx")
    within(dw, want_dw, 2.0 ** -17 * aw, "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", [(3, 256), (2000, 256), (3, 1024), (900, 1024), (900, 8192), (3, 16384)])
def test_a_variance_of_three_smallest_steps(rows, C, dtype):
    """eps = 0 and three of eight elements +-2^-73, the others 0: every sum is
    exact, the variance is 3 x 2^-149, and rstd and y are it to 2^-21 (the
    root's 2^-22, a product's 2^-24; bf16: half a step of y)."""
    a = 2.0 ** -73
    x = torch.tensor([a, -a, a, -a, a, -a] + [0.0] * 10, device="cuda").repeat(rows, C // 16).to(DT[dtype][0])
    y, mean, rstd = F.layer_norm_fwd(F.make_norm(rows, C, dtype=DT[dtype][1], eps=0.0), x)
    want = (3 * 2.0 ** -149) ** -0.5
    assert (mean == 0).all()
    assert ((rstd.double() - want).abs() <= 2.0 ** -21 * want).all()
    within(y, x.double() * want, (DT[dtype][2] + 2.0 ** -21) * (x.double() * want).abs(), "y")
