"""The operators run together as a streaming video model's attention block
uses them, forward and backward, through the public entry points:

  frames x [B, N, C] --layer norm with one scale / shift per frame-->
  --projection + RoPE at the frames' offset--> q, k, v
  --attention over a window of frames and the first frame--> out
  and back: dq, dk, dv, (the projection's input gradient in plain torch,)
  the norm's dx and its per-frame scale / shift gradients;

and frame by frame against a growing cache, which has to give what the whole
clip gives.  Compared with the same block in 64 bits whose intermediate
tensors are rounded to bf16 where the block stores them."""
import numpy as np
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from oracle import fvattn_oracle as O
from tests.window_util import plain_bwd, plain_fwd

pytestmark = pytest.mark.gpu
GRID, H, D, C, WINDOW, SINKS = (8, 8, 8), 2, 128, 256, 3, 1
FRAME, N = 64, 512


def setup():
    gen = torch.Generator("cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = rnd(1, N, C).to(torch.bfloat16)
    w = (rnd(3 * H * D, C) / C ** 0.5).to(torch.bfloat16)
    return x, rnd(8, C) * 0.2, rnd(8, C) * 0.2, w, rnd(1, H, N, D).to(torch.bfloat16)


def test_block_forward_and_backward():
    x, scale, shift, w, dout = setup()
    norm = F.make_norm(N, C, groups=8, gain_one=True)
    shape = F.make_shape(1, H, D, GRID)
    rope = F.make_rope()
    pws = torch.empty(F.workspace_size_qkv(shape, rope), dtype=torch.uint8, device="cuda")
    win = F.make_window(1, H, D, N, N, WINDOW, sinks=SINKS, unit=FRAME)
    ws, nws = F.window_workspace(win, backward=True), F.norm_workspace(norm)

    y, mean, rstd = F.layer_norm_fwd(norm, x, weight=scale, bias=shift)
    q, k, v = F.qkv_rope(shape, y, w, pws, rope=rope, t_offset=0)
    out, lse = F.window_fwd(win, q, k, v, ws)
    dq, dk, dv = F.window_bwd(win, q, k, v, out, dout, lse, ws)
    assert F.device_status(pws) == 0 and F.device_status(ws) == 0

    # forward: each stage against 64 bits on the stage's own inputs
    xd = x[0].double()
    mu = xd.mean(1, keepdim=True)
    rs = 1 / torch.sqrt((xd - mu).pow(2).mean(1, keepdim=True) + 1e-6)
    gain = (1 + scale.double()).repeat_interleave(FRAME, 0)
    xh = (xd - mu) * rs
    want = xh * gain + shift.double().repeat_interleave(FRAME, 0)
    assert ((y[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * (1 + xh.abs() * gain.abs())).all()
    raw = O.qkv_rope(y.double().cpu().numpy(), w.double().cpu().numpy(), None, GRID, H, D,
                     dict(dims=(44, 42, 42), base=10000.0))
    for got, r in zip((q, k, v), raw):
        assert np.abs(got.double().cpu().numpy() - r).max() <= 2.0 ** -7 * max(1.0, np.abs(r).max())
    ref, rl, spread = plain_fwd(q, k, v, FRAME, WINDOW, SINKS)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * spread).all()

    # backward of the attention, then through the projection (without the
    # rotation: v's part only needs none) and the norm
    exact, err = plain_bwd(q, k, v, dout, FRAME, WINDOW, SINKS)
    for name, g, e, s in zip(("dq", "dk", "dv"), (dq, dk, dv), exact, err):
        frac = 2.0 ** -8 + 2.0 ** -12 if name == "dv" else 2.0 ** -6
        assert ((g.double() - e).abs() <= 2.0 ** -8 * e.abs() + frac * s).all(), name
    dy = (dv[0].permute(1, 0, 2).reshape(N, H * D).double() @ w[2 * H * D:].double()).to(torch.bfloat16)
    dx, dscale, dshift = F.layer_norm_bwd(norm, x, dy[None], mean, rstd, nws, weight=scale)
    g = dy.double()
    gy = g * gain
    c1, c2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    wx = rs * (gy - c1 - xh * c2)
    size = rs * (gy.abs() + gy.abs().mean(1, keepdim=True) + xh.abs() * (gy * xh).abs().mean(1, keepdim=True))
    assert ((dx[0].double() - wx).abs() <= 2.0 ** -8 * wx.abs() + 2.0 ** -18 * size).all()
    for got, terms in ((dscale, g * xh), (dshift, g)):
        t = terms.reshape(8, FRAME, C)
        bound = 2.0 ** -17 * (t.abs().sum(1) + g.abs().reshape(8, FRAME, C).sum(1))
        assert ((got.double() - t.sum(1)).abs() <= bound).all()


def test_frame_by_frame_equals_the_clip():
    """Frame f's queries against the cache of the frames so far, in a buffer
    whose rows behind them hold NaN, give the clip's rows."""
    x, scale, shift, w, _ = setup()
    norm = F.make_norm(N, C, groups=8, gain_one=True)
    shape, rope = F.make_shape(1, H, D, GRID), F.make_rope()
    pws = torch.empty(F.workspace_size_qkv(shape, rope), dtype=torch.uint8, device="cuda")
    y, _, _ = F.layer_norm_fwd(norm, x, weight=scale, bias=shift)
    q, k, v = F.qkv_rope(shape, y, w, pws, rope=rope)
    clip = F.make_window(1, H, D, N, N, WINDOW, sinks=SINKS, unit=FRAME)
    ref, rl, spread = plain_fwd(q, k, v, FRAME, WINDOW, SINKS)
    whole, wl = F.window_fwd(clip, q, k, v, F.window_workspace(clip))
    kc, vc = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    step = F.make_window(1, H, D, FRAME, N, WINDOW, sinks=SINKS, unit=FRAME)
    ws = F.window_workspace(step)
    for f in range(8):
        a, b = f * FRAME, (f + 1) * FRAME
        kc[:, :, a:b], vc[:, :, a:b] = k[:, :, a:b], v[:, :, a:b]
        lens = torch.tensor([b], dtype=torch.int32, device="cuda")
        out, lse = F.window_fwd(step, q[:, :, a:b], kc, vc, ws, kv_lens=lens)
        assert F.device_status(ws) == 0
        tol = 2.0 ** -8 * ref[:, :, a:b].abs() + (2.0 ** -8 + 2.0 ** -12) * spread[:, :, a:b]
        assert ((out.double() - ref[:, :, a:b]).abs() <= tol).all(), f
        assert ((out.double() - whole[:, :, a:b].double()).abs() <= 2 * tol).all(), f
        assert ((lse.double() - rl[:, :, a:b]).abs() <= 2.0 ** -12).all()


def test_workspaces_of_two_graphs():
    """Two captured calls with a workspace of their own, replayed at the same
    time on two streams."""
    gen = torch.Generator("cuda").manual_seed(5)
    calls = []
    for n in (1, 300):
        q = torch.randn(2, 4, n, 64, generator=gen, device="cuda").to(torch.bfloat16)
        k, v = (torch.randn(2, 2, 1500, 64, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        win = F.make_window(2, 4, 64, n, 1500, 700, sinks=4, kv_heads=2)
        ws = F.window_workspace(win)
        want = F.window_fwd(win, q, k, v, ws)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            F.window_fwd(win, q, k, v, ws, out=out, lse=lse)
        calls.append((graph, torch.cuda.Stream(), out, lse, want, (q, k, v, ws)))
    for _ in range(20):
        for graph, stream, *_ in calls:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, lse, want, keep in calls:
        assert F.device_status(keep[3]) == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals_on_the_device():
    win = F.make_window(1, 2, 64, 4, 4, 2)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = F.window_workspace(win)
    with pytest.raises(ValueError, match="CUDA"):
        F.window_fwd(win, q, q, q.cpu(), ws)
    with pytest.raises(ValueError, match="k: expected"):
        F.window_fwd(win, q, q[:, :1], q, ws)
    with pytest.raises(ValueError, match="q_lens"):
        F.window_fwd(win, q, q, q, ws, q_lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(F.FvattnError, match="workspace"):
        F.window_fwd(win, q, q, q, torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(F.FvattnError, match="invalid argument"):
        F.window_fwd(win, q, q.expand(1, 2, 4, 64), q[:, :1].expand(1, 2, 4, 64), ws)
