"""GPU parity of the layer norm's forward and backward against a plain 64-bit
implementation.

Tolerances, from the arithmetic (u = half a step of the stored type relative
to the value: 2^-8 bf16, 2^-24 fp32).  fp32 sums of C values in a tree of
depth <= 32 steps keep 2^-19 of the sum of the magnitudes:
  mean      2^-19 mean|x| (the sum's bound over C), rstd relative 2^-19 (1 + mean^2 rstd^2 2^-4);
  forward   |y - exact| <= u |y| + 2^-19 (|xhat gain| + |bias| + mean|x| rstd |gain|): the mean's own
            bound carried through (x - mean) rstd gain, so it is mean|x| that counts and not |mean|,
            which can be 0 where the sum's rounding is not;
  backward  |dx - exact| <= u |dx| + 2^-18 rstd (|gy| + mean|gy| + |xhat| mean|gy xhat|)
                            + the saved statistics' rounding, 2^-22 (1 + |mean| rstd) of the same scale,
  dw, db    2^-17 sum |terms|: rows are added one after another, then blocks (at most
            rows / blocks + blocks + 8 < 2^7 additions here, each 2^-24 of the sum)."""
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, F.BF16, 2.0 ** -8), "f32": (torch.float32, F.F32, 2.0 ** -24)}

# rows, channels, groups
SHAPES = [(1, 1, 1), (3, 2, 1), (5, 7, 1), (7, 64, 7), (33, 130, 3), (64, 512, 2), (300, 513, 4), (1000, 129, 5),
          (513, 1001, 3), (40, 1536, 1), (130, 5120, 13), (700, 5120, 2), (9, 8192, 3), (5, 8193, 1), (12, 10000, 4),
          (3, 65536, 1), (2000, 48, 1), (4096, 256, 1024)]


def make(rows, C, groups, dtype, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = (rnd(rows, C) * (0.2 + rnd(rows, 1).abs()) + rnd(rows, 1)).to(DT[dtype][0])
    return x, rnd(groups, C) * 0.5, rnd(groups, C), rnd(rows, C).to(DT[dtype][0])


def plain(x, w, b, dy, groups, eps, gain_one):
    x, dy = x.double(), dy.double()
    rows, C = x.shape
    rep = rows // groups
    one = torch.ones(groups, C, dtype=torch.float64, device="cuda")
    gain = one if w is None else w.double() + (1 if gain_one else 0)
    gain = gain.repeat_interleave(rep, 0)
    bias = torch.zeros_like(gain) if b is None else b.double().repeat_interleave(rep, 0)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).pow(2).mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    gy = dy * gain
    r = {"mean": mean, "rstd": rstd, "xh": xh, "gain": gain, "bias": bias, "gy": gy, "y": xh * gain + bias}
    r["dx"] = rstd * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    r["dw"] = (dy * xh).reshape(groups, rep, C).sum(1)
    r["db"] = dy.reshape(groups, rep, C).sum(1)
    r["aw"] = (dy * xh).abs().reshape(groups, rep, C).sum(1)
    r["ab"] = dy.abs().reshape(groups, rep, C).sum(1)
    return r


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (what, float((err - tol).max()), float(err.max()))


def check_fwd(y, mean, rstd, r, x, u):
    shift = r["mean"].abs() * r["rstd"]
    size = x.double().abs().mean(1, keepdim=True) * r["rstd"]
    within(y, r["y"], u * r["y"].abs() + 2.0 ** -19 * ((r["xh"] * r["gain"]).abs() + r["bias"].abs()
                                                      + size * r["gain"].abs()), "y")
    within(mean, r["mean"][:, 0], 2.0 ** -19 * x.double().abs().mean(1) + 1e-30, "mean")
    within(rstd, r["rstd"][:, 0], 2.0 ** -19 * (r["rstd"] * (1 + shift ** 2 / 16))[:, 0], "rstd")


def check_bwd(dx, dw, db, r, u):
    shift = r["mean"].abs() * r["rstd"]
    size = r["rstd"] * (r["gy"].abs() + r["gy"].abs().mean(1, keepdim=True)
                        + r["xh"].abs() * (r["gy"] * r["xh"]).abs().mean(1, keepdim=True))
    if dx is not None:
        within(dx, r["dx"], u * r["dx"].abs() + (2.0 ** -18 + 2.0 ** -22 * shift) * size, "dx")
    per_row = 2.0 ** -17 + 2.0 ** -22 * float(shift.max())
    if dw is not None:
        within(dw, r["dw"], per_row * (r["aw"] + r["ab"]), "dweight")
    if db is not None:
        within(db, r["db"], 2.0 ** -17 * r["ab"], "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("affine", ["both", "gain_one", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(shape, affine, dtype):
    rows, C, groups = shape
    x, w, b, dy = make(rows, C, groups, dtype)
    if affine == "none":
        w = b = None
    norm = F.make_norm(rows, C, groups, dtype=DT[dtype][1], eps=1e-5, gain_one=affine == "gain_one")
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    r = plain(x, w, b, dy, groups, 1e-5, affine == "gain_one")
    check_fwd(y, mean, rstd, r, x, DT[dtype][2])
    ws = F.norm_workspace(norm)
    dx, dw, db = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w)
    check_bwd(dx, dw, db, r, DT[dtype][2])
    again = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,xs,ys", [(512, 520, 512), (256, 259, 258), (33, 40, 37), (5120, 5120, 6000)])
def test_strided_rows(C, xs, ys, dtype):
    rows, groups = 60, 3
    x0, w, b, dy0 = make(rows, C, groups, dtype, 1)
    def strided(t, s):
        buf = torch.full((rows * s,), 9.0, dtype=t.dtype, device="cuda").as_strided((rows, C), (s, 1))
        return buf.copy_(t)
    x, dy = strided(x0, xs), strided(dy0, ys)
    norm = F.make_norm(rows, C, groups, dtype=DT[dtype][1], x_stride=xs, y_stride=ys)
    y = strided(torch.zeros_like(x0), ys)
    whole = y.as_strided((rows * ys,), (1,))
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b, y=y)
    if ys > C:
        assert (whole.view(rows, ys)[:, C:] == 9).all()
    r = plain(x0, w, b, dy0, groups, 1e-6, False)
    check_fwd(y, mean, rstd, r, x0, DT[dtype][2])
    check_bwd(*F.layer_norm_bwd(norm, x, dy, mean, rstd, F.norm_workspace(norm), weight=w), r, DT[dtype][2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 512, 5120])
def test_gain_and_bias_at_a_floats_alignment(C, dtype):
    """weight and bias that start 4 bytes into a 16-byte line (a slice of a
    larger buffer), and per-row statistics likewise."""
    rows, groups = 21, 3
    x, w0, b0, dy = make(rows, C, groups, dtype, 6)
    buf = torch.empty(2, groups * C + 1, device="cuda")
    w, b = (buf[i, 1:].view(groups, C) for i in range(2))
    w.copy_(w0), b.copy_(b0)
    assert w.data_ptr() % 16 == 4
    norm = F.make_norm(rows, C, groups, dtype=DT[dtype][1])
    stat = torch.empty(2, rows + 1, device="cuda")
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b, mean=stat[0, 1:], rstd=stat[1, 1:])
    r = plain(x, w0, b0, dy, groups, 1e-6, False)
    check_fwd(y, mean, rstd, r, x, DT[dtype][2])
    check_bwd(*F.layer_norm_bwd(norm, x, dy, mean, rstd, F.norm_workspace(norm), weight=w), r, DT[dtype][2])


@pytest.mark.parametrize("C", [96, 1536, 10000])
def test_in_place_and_single_gradients(C):
    rows, groups = 50, 2
    x, w, b, dy = make(rows, C, groups, "f32", 2)
    norm = F.make_norm(rows, C, groups, dtype=F.F32)
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    ws = F.norm_workspace(norm)
    full = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w)
    buf = x.clone()
    F.layer_norm_fwd(norm, buf, weight=w, bias=b, y=buf)
    assert torch.equal(buf, y)
    for into in ("x", "dy"):
        xi, di = x.clone(), dy.clone()
        tgt = xi if into == "x" else di
        got = F.layer_norm_bwd(norm, xi, di, mean, rstd, ws, weight=w,
                               grads=(tgt, torch.empty_like(full[1]), torch.empty_like(full[2])))
        assert all(torch.equal(p, q) for p, q in zip(got, full))
    for keep in range(3):
        grads = [torch.full_like(t, 3.0) if i == keep else None for i, t in enumerate(full)]
        got = F.layer_norm_bwd(norm, x, dy, mean, rstd, ws, weight=w, grads=grads)
        assert torch.equal(got[keep], full[keep])


def test_no_rows_and_constant_rows_and_nan():
    norm = F.make_norm(0, 64, 2, dtype=F.F32)
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(2, 64, device="cuda")
    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=w)
    assert y.shape == (0, 64)
    dx, dw, db = F.layer_norm_bwd(norm, x, x, mean, rstd, F.norm_workspace(norm), weight=w)
    assert (dw == 0).all() and (db == 0).all()
    # a constant row has variance 0 however large it is: y is exactly the bias
    norm = F.make_norm(4, 1000, dtype=F.F32)
    x = torch.tensor([0.1, 1e4, -3e7, 0.0], device="cuda")[:, None].expand(4, 1000).contiguous()
    y, mean, rstd = F.layer_norm_fwd(norm, x)
    assert (y.abs() <= 2.0 ** -24 * x.abs() * rstd[:, None]).all()
    # a NaN or an infinity stays in its own row
    x = torch.randn(4, 1000, device="cuda")
    x[1, 17], x[3, 5] = float("nan"), float("inf")
    y, _, _ = F.layer_norm_fwd(norm, x)
    assert y[1].isnan().all() and y[3].isnan().all() and y[0].isfinite().all() and y[2].isfinite().all()


def test_a_large_mean_keeps_the_variance():
    """mean / std = 2^12: the variance comes from the differences, not from
    the sum of squares."""
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(64, 1536, generator=gen, device="cuda") + 4096.0
    norm = F.make_norm(64, 1536, dtype=F.F32, eps=0.0)
    y, mean, rstd = F.layer_norm_fwd(norm, x)
    xd = x.double()
    m = xd.mean(1, keepdim=True)
    sd = (xd - m).pow(2).mean(1, keepdim=True).sqrt()
    within(y, (xd - m) / sd, 2.0 ** -18 * (1 + ((xd - m) / sd).abs()), "y")


def test_gradient_against_differences():
    """dx, dw, db against central differences of the forward in 64 bits."""
    x, w, b, dy = make(3, 40, 1, "f32", 4)
    norm = F.make_norm(3, 40, 1, dtype=F.F32)
    _, mean, rstd = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    dx, dw, db = F.layer_norm_bwd(norm, x, dy, mean, rstd, F.norm_workspace(norm), weight=w)
    f = lambda x, w, b: (plain(x, w, b, dy, 1, 1e-6, False)["y"] * dy.double()).sum()  # noqa: E731
    base = [t.double() for t in (x, w, b)]
    h = 1e-5
    for which, grad in enumerate((dx, dw, db)):
        for pos in range(0, base[which].numel(), 7):
            args = [[t.clone() for t in base] for _ in range(2)]
            args[0][which].view(-1)[pos] += h
            args[1][which].view(-1)[pos] -= h
            diff = (f(*args[0]) - f(*args[1])) / (2 * h)
            assert abs(float(diff) - float(grad.reshape(-1)[pos])) <= 1e-4 * (1 + abs(float(diff)))


def test_side_stream_and_graph():
    x, w, b, dy = make(128, 1536, 4, "bf16", 5)
    norm = F.make_norm(128, 1536, 4)
    want = F.layer_norm_fwd(norm, x, weight=w, bias=b)
    ws = F.norm_workspace(norm)
    gwant = F.layer_norm_bwd(norm, x, dy, want[1], want[2], ws, weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.layer_norm_fwd(norm, x, weight=w, bias=b, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    xs = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y, mean, rstd = F.layer_norm_fwd(norm, xs, weight=w, bias=b)
        grads = F.layer_norm_bwd(norm, xs, dy, mean, rstd, ws, weight=w)
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and all(torch.equal(p, q) for p, q in zip(grads, gwant))
