"""GPU parity of the sliding-window attention's backward against a plain
64-bit implementation, and against differences of the plain forward.

The GPU's own forward gives out and lse.  Tolerance, from the arithmetic: P
and dS are rounded to bf16 (2^-8 relative each), rowsum(dout * out) carries
the forward's error (|out - exact| <= 2^-7 sum_j p_j |v_j|, see
test_gpu_window.py), every gradient is rounded once (2^-8 of it).  With
a = scale p (|dp| + sum_c |dout_c| sum_j p_j |v_jc|) the error of scale dS is
at most 2^-8 a (rounding) + 2^-7 a (rowsum) < 2^-6 a, so
  dq, dk: |gpu - exact| <= 2^-8 |exact| + 2^-6 (a |k| or a^T |q|),
  dv:     |gpu - exact| <= 2^-8 |exact| + (2^-8 + 2^-12) p^T |dout|."""
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from tests.window_util import heads, plain_bwd, plain_fwd

pytestmark = pytest.mark.gpu


def run(win, q, k, v, dout, grads=None, **kw):
    ws = F.window_workspace(win, backward=True)
    out, lse = F.window_fwd(win, q, k, v, ws, **kw)
    got = F.window_bwd(win, q, k, v, out, dout, lse, ws, grads=grads, **kw)
    assert F.device_status(ws) == 0
    return got


def check(got, ref, q_lens=None, kv_lens=None):
    exact, scale = ref
    for name, g, e, s, lens in zip(("dq", "dk", "dv"), got, exact, scale, (q_lens, kv_lens, kv_lens)):
        frac = 2.0 ** -8 + 2.0 ** -12 if name == "dv" else 2.0 ** -6
        tol = 2.0 ** -8 * e.abs() + frac * s
        err = (g.double() - e).abs()
        for b in range(g.shape[0]):
            n = g.shape[2] if lens is None else lens[b]
            assert (err[b, :, :n] <= tol[b, :, :n]).all(), (name, b, float((err - tol)[b, :, :n].max()))


# B, H, Hk, D, q_len, kv_len, unit, window, sinks
CASES = [
    (1, 1, 1, 128, 1, 1, 1, 0, 0),
    (1, 2, 1, 64, 1, 300, 1, 100, 4),
    (2, 4, 2, 128, 64, 64, 1, 0, 0),
    (1, 3, 1, 64, 65, 65, 1, 7, 1),
    (1, 2, 2, 128, 128, 128, 1, 128, 0),
    (2, 6, 2, 128, 129, 129, 1, 40, 3),
    (1, 2, 1, 64, 300, 300, 1, 1, 0),
    (1, 14, 2, 64, 331, 331, 1, 100, 7),
    (1, 2, 2, 128, 515, 515, 1, 77, 140),
    (1, 3, 3, 128, 640, 640, 64, 2, 1),
    (2, 2, 1, 128, 300, 700, 48, 3, 2),
    (1, 2, 2, 64, 257, 1025, 100, 1, 0),
    (1, 2, 2, 128, 40, 20, 1, 8, 2),          # more queries than keys
    (1, 2, 2, 128, 300, 130, 16, 2, 1),
    (1, 2, 1, 128, 9, 0, 1, 8, 2),            # no key
    (1, 2, 1, 128, 0, 9, 1, 8, 2),            # no query
    (30, 6, 3, 64, 130, 130, 1, 50, 2),       # more items than SMs
]


@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "slice"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, layout):
    B, H, Hk, D, Nq, Nk, unit, window, sinks = case
    gen = torch.Generator("cuda").manual_seed(1)
    q, dout = heads(gen, B, H, Nq, D, layout, 2.0), heads(gen, B, H, Nq, D, layout)
    k, v = heads(gen, B, Hk, Nk, D, layout), heads(gen, B, Hk, Nk, D, layout)
    win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks, unit=unit, kv_heads=Hk)
    got = run(win, q, k, v, dout)
    check(got, plain_bwd(q, k, v, dout, unit, window, sinks))
    assert all(torch.equal(a, b) for a, b in zip(got, run(win, q, k, v, dout)))


@pytest.mark.parametrize("D", [64, 128])
def test_padded_batch(D):
    """Sequences of their own lengths: rows behind them are not read into
    anything (they hold NaN) and not written; keys out of every window may
    hold NaN too."""
    B, H, Hk, N = 5, 4, 2, 300
    gen = torch.Generator("cuda").manual_seed(2)
    q, dout = heads(gen, B, H, N, D, mul=2.0), heads(gen, B, H, N, D)
    k, v = heads(gen, B, Hk, N, D), heads(gen, B, Hk, N, D)
    ql, kl = [300, 131, 0, 64, 20], [300, 131, 129, 0, 255]
    window, sinks = 90, 5
    for b in range(B):
        for t in (k, v):
            t[b, :, kl[b]:] = float("nan")
        for t in (q, dout):
            t[b, :, ql[b]:] = float("nan")
        first = max(0, kl[b] - ql[b] - window + 1)
        if first > sinks and ql[b]:
            k[b, :, sinks:first] = float("inf")
            v[b, :, sinks:first] = float("nan")
    win = F.make_window(B, H, D, N, N, window, sinks=sinks, kv_heads=Hk)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = F.window_workspace(win, backward=True)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((B, H, N), float("nan"), device="cuda")
    kw = dict(q_lens=t(ql), kv_lens=t(kl))
    F.window_fwd(win, q, k, v, ws, out=out, lse=lse, **kw)
    grads = tuple(torch.full_like(x, 7.0) for x in (q, k, v))
    F.window_bwd(win, q, k, v, out, dout, lse, ws, grads=grads, **kw)
    assert F.device_status(ws) == 0
    check(grads, plain_bwd(q, k, v, dout, 1, window, sinks, q_lens=ql, kv_lens=kl), ql, kl)
    for g, lens in zip(grads, (ql, kl, kl)):
        for b in range(B):
            assert (g[b, :, lens[b]:] == 7).all()


@pytest.mark.parametrize("unit,window,sinks", [(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (3, 1, 2 ** 31 - 1), (2 ** 31 - 1, 1, 0)])
def test_extreme_parameters(unit, window, sinks):
    B, H, D, Nq, Nk = 1, 2, 64, 150, 200
    gen = torch.Generator("cuda").manual_seed(9)
    q, dout, k, v = (heads(gen, B, H, n, D) for n in (Nq, Nq, Nk, Nk))
    win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks, unit=unit)
    cut = [min(x, 10 ** 6) for x in (unit, window, sinks)]
    check(run(win, q, k, v, dout), plain_bwd(q, k, v, dout, *cut))


def test_gradient_against_differences():
    """Central differences of the plain 64-bit forward along random
    directions: the bf16 gradients have to give the same slopes."""
    B, H, Hk, D, N, unit, window, sinks = 1, 4, 2, 64, 150, 10, 3, 1
    gen = torch.Generator("cuda").manual_seed(3)
    q, dout = heads(gen, B, H, N, D), heads(gen, B, H, N, D)
    k, v = heads(gen, B, Hk, N, D), heads(gen, B, Hk, N, D)
    win = F.make_window(B, H, D, N, N, window, sinks=sinks, unit=unit, kv_heads=Hk)
    got = run(win, q, k, v, dout)
    ref, scale = plain_bwd(q, k, v, dout, unit, window, sinks)
    base = [t.double() for t in (q, k, v)]
    h = 1e-4
    for i in range(3):
        d = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = [(plain_fwd(*[t + s * h * d if j == i else t for j, t in enumerate(base)], unit, window, sinks)[0]
              * dout.double()).sum() for s in (1, -1)]
        slope = float(f[0] - f[1]) / (2 * h)
        tol = float(((2.0 ** -8 * ref[i].abs() + 2.0 ** -6 * scale[i]) * d.abs()).sum())
        assert abs(slope - float((got[i].double() * d).sum())) <= tol + 1e-5 * abs(slope)
        # and the plain gradient, far closer
        assert abs(slope - float((ref[i] * d).sum())) <= 1e-5 * (1 + float((ref[i] * d).abs().sum()))


def test_side_stream_and_graph():
    """Forward and backward captured together and replayed on new inputs."""
    B, H, Hk, D, N = 1, 4, 2, 128, 257
    gen = torch.Generator("cuda").manual_seed(4)
    ts = [heads(gen, B, n, N, D) for n in (H, Hk, Hk, H)]
    q, k, v, dout = ts
    win = F.make_window(B, H, D, N, N, 100, sinks=4, kv_heads=Hk)
    ws = F.window_workspace(win, backward=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = F.window_fwd(win, q, k, v, ws, stream=side)
    got = F.window_bwd(win, q, k, v, out, dout, lse, ws, stream=side)
    side.synchronize()
    check(got, plain_bwd(q, k, v, dout, 1, 100, 4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = F.window_fwd(win, q, k, v, ws)
        got = F.window_bwd(win, q, k, v, out, dout, lse, ws)
    for seed in (5, 6):
        gen = torch.Generator("cuda").manual_seed(seed)
        for t in ts:
            t.copy_(heads(gen, B, t.shape[1], N, D))
        graph.replay()
        torch.cuda.synchronize()
        assert F.device_status(ws) == 0
        check(got, plain_bwd(q, k, v, dout, 1, 100, 4))


def test_calls_one_behind_another():
    """The kernels of a call overlap; calls that share a workspace and reads
    of the gradients behind each must not: the bits of a run alone."""
    cases = []
    for seed, (H, Hk, D, N, window) in enumerate([(4, 2, 128, 700, 150), (14, 2, 64, 515, 90), (2, 2, 128, 70, 0)]):
        gen = torch.Generator("cuda").manual_seed(seed)
        q, k, v, dout = (heads(gen, 1, n, N, D) for n in (H, Hk, Hk, H))
        win = F.make_window(1, H, D, N, N, window, sinks=5 if window else 0, kv_heads=Hk)
        own = F.window_workspace(win, backward=True)
        out, lse = F.window_fwd(win, q, k, v, own)
        args = (q, k, v, out, dout, lse)
        alone = F.window_bwd(win, *args, own)
        torch.cuda.synchronize()
        cases.append((win, args, alone))
    ws = max((F.window_workspace(c[0], backward=True) for c in cases), key=lambda t: t.numel())
    grads = [tuple(torch.empty_like(t) for t in c[2]) for c in cases]
    for profiled in (False, True):      # events between the kernels keep them apart
        F.profile_enable(profiled)
        try:
            seen = []
            for _ in range(6):
                for (win, args, _), g in zip(cases, grads):
                    F.window_bwd(win, *args, ws, grads=g)
                    seen.append([t.clone() for t in g])
                    F.window_fwd(win, *args[:3], ws)
                    for t in g:
                        t.zero_()
            torch.cuda.synchronize()
        finally:
            F.profile_enable(False)
            F.profile_read()
        assert F.device_status(ws) == 0
        for n, got in enumerate(seen):
            for a, b in zip(got, cases[n % len(cases)][2]):
                assert torch.equal(a, b)
