"""GPU parity of the sliding-window attention's forward against a plain
64-bit implementation.

Tolerance, from the arithmetic: the kernel rounds the probabilities to bf16
(relative 2^-8 at most each) and the output once (2^-8 of it); its exponential
is within 2^-13 and the fp32 sums far below that:
  |out - exact| <= 2^-8 |exact| + (2^-8 + 2^-12) sum_j p_j |v_j|,
  |lse - exact| <= 2^-13 + 2^-20 (1 + |lse| + max |s|)."""
import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from tests.window_util import heads, plain_fwd

pytestmark = pytest.mark.gpu


def run(win, q, k, v, **kw):
    ws = F.window_workspace(win)
    out, lse = F.window_fwd(win, q, k, v, ws, **kw)
    assert F.device_status(ws) == 0
    return out, lse


def check(out, lse, ref):
    want, wl, spread = ref
    rows = ~want[..., 0].isnan()
    err = (out.double() - want).abs()[rows]
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread)[rows]
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    empty = wl.isinf() & rows
    assert (out[empty] == 0).all() and (lse[empty] == -float("inf")).all()
    some = rows & ~empty
    if some.any():
        d = (lse.double() - wl).abs()[some]
        assert (d <= 2.0 ** -13 + 2.0 ** -20 * (64 + wl.abs()[some])).all(), float(d.max())


# B, H, Hk, D, q_len, kv_len, unit, window, sinks
CASES = [
    (1, 1, 1, 128, 1, 1, 1, 1, 0),
    (1, 2, 1, 64, 1, 1, 1, 0, 0),
    (2, 4, 2, 128, 1, 777, 1, 100, 4),
    (3, 8, 2, 64, 1, 129, 1, 0, 0),
    (1, 7, 1, 128, 5, 1000, 1, 300, 129),
    (1, 14, 2, 64, 37, 300, 1, 64, 1),
    (2, 3, 3, 128, 127, 127, 1, 40, 3),
    (1, 2, 2, 128, 128, 128, 1, 0, 0),
    (1, 2, 1, 128, 129, 257, 1, 1, 0),
    (1, 2, 2, 128, 300, 300, 1, 128, 128),
    (2, 2, 1, 64, 515, 515, 1, 77, 5),
    (1, 3, 3, 128, 640, 640, 64, 2, 1),
    (1, 2, 2, 128, 600, 700, 48, 3, 2),
    (1, 2, 2, 64, 257, 1025, 100, 1, 0),
    (1, 1, 1, 128, 2049, 2049, 1, 500, 260),
    (1, 2, 2, 128, 40, 20, 1, 8, 2),          # more queries than keys: the first see none
    (1, 2, 2, 128, 300, 130, 16, 2, 1),
    (1, 2, 1, 128, 9, 0, 1, 8, 2),            # no key at all
    (1, 200, 1, 128, 3, 400, 1, 50, 4),       # more heads a KV head than a tile has rows
    (1, 128, 1, 64, 2, 260, 1, 0, 0),
    (1, 1, 1, 128, 64, 9000, 1, 0, 0),        # split over many CTAs
    (1, 1, 1, 128, 200, 9000, 1, 5000, 4),
    (150, 1, 1, 64, 2, 200, 1, 90, 3),        # more items than SMs
]


@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "slice"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, layout):
    B, H, Hk, D, Nq, Nk, unit, window, sinks = case
    gen = torch.Generator("cuda").manual_seed(1)
    q = heads(gen, B, H, Nq, D, layout, 2.0)
    k, v = heads(gen, B, Hk, Nk, D, layout), heads(gen, B, Hk, Nk, D, layout)
    win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks, unit=unit, kv_heads=Hk)
    out, lse = run(win, q, k, v)
    check(out, lse, plain_fwd(q, k, v, unit, window, sinks))
    again = run(win, q, k, v)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [1, 6, 131, 300])
def test_lengths(D, Nq):
    """Per-sequence lengths; rows behind them stay as they were, and keys
    behind them or out of every window may hold NaN."""
    B, H, Hk, Nk = 5, 4, 2, 700
    gen = torch.Generator("cuda").manual_seed(2)
    q, k, v = heads(gen, B, H, Nq, D, mul=2.0), heads(gen, B, Hk, Nk, D), heads(gen, B, Hk, Nk, D)
    ql = [Nq, max(0, Nq - 1), 0, min(3, Nq), Nq]
    kl = [700, 333, 129, 0, 512]
    unit, window, sinks = 1, 90, 5
    for b in range(B):
        k[b, :, kl[b]:] = float("nan")
        v[b, :, kl[b]:] = float("nan")
        first = max(0, kl[b] - ql[b] - window + 1)       # first key of the first query's window
        if first > sinks and ql[b]:
            k[b, :, sinks:first] = float("inf")
            v[b, :, sinks:first] = float("nan")
        q[b, :, ql[b]:] = float("nan")
    win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks, unit=unit, kv_heads=Hk)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((B, H, Nq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, Nq), 7.0, device="cuda")
    run(win, q, k, v, q_lens=t(ql), kv_lens=t(kl), out=out, lse=lse)
    ref = plain_fwd(q, k, v, unit, window, sinks, q_lens=ql, kv_lens=kl)
    check(out, lse, ref)
    behind = ref[0][..., 0].isnan()
    assert (out[behind] == 7).all() and (lse[behind] == 7).all()
    # lengths outside the tensors are cut to them
    far = [x if x < m else 10 ** 6 for x, m in zip(ql, [Nq] * B)], [x if x else -5 for x in kl]
    out2, lse2 = run(win, q, k, v, q_lens=t(far[0]), kv_lens=t(far[1]))
    assert torch.equal(out2[~behind], out[~behind])


@pytest.mark.parametrize("Nq", [4, 256])
def test_large_logits_move_the_reference(Nq):
    """Logits that grow along the keys, so a row's running reference has to
    move several times, and rows whose last key takes all the mass."""
    B, H, D, Nk = 1, 2, 128, 1024
    gen = torch.Generator("cuda").manual_seed(3)
    q = torch.ones(B, H, Nq, D, dtype=torch.bfloat16, device="cuda")
    k = heads(gen, B, H, Nk, D, mul=0.05) + (torch.arange(Nk, device="cuda") // 128 * 16.0)[:, None].to(torch.bfloat16)
    v = heads(gen, B, H, Nk, D)
    win = F.make_window(B, H, D, Nq, Nk, 0)
    out, lse = run(win, q, k, v)
    check(out, lse, plain_fwd(q, k, v, 1, 0, 0))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [3, 40, 100, 130, 260])
def test_reference_moves_inside_a_tile(Nq, D):
    """Logits that jump by more than 2^64 every 32 keys, up and down again, in
    every form: rows held four times, twice and once, and two query tiles."""
    B, H, Nk = 1, 1, 600
    gen = torch.Generator("cuda").manual_seed(8)
    q = torch.ones(B, H, Nq, D, dtype=torch.bfloat16, device="cuda")
    steps = torch.arange(Nk, device="cuda") // 32
    ramp = torch.where(steps < 12, steps, 24 - steps) * (128.0 / D)
    k = heads(gen, B, H, Nk, D, mul=0.02) + (ramp * 8.0)[:, None].to(torch.bfloat16)
    v = heads(gen, B, H, Nk, D)
    for window, sinks in ((0, 0), (200, 40)):
        win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks)
        out, lse = run(win, q, k, v)
        check_far(out, lse, plain_fwd(q, k, v, 1, window, sinks))


def check_far(out, lse, ref):
    """check() for logits of size s: one fp32 rounding of s, relative 2^-24,
    is |s| 2^-24 of a logit, which the probabilities and lse carry as
    ln 2 times as much; here |s| < 2^12, so 2^-11 of both covers it."""
    want, wl, spread = ref
    err = (out.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * spread).all(), float(err.max())
    assert ((lse.double() - wl).abs() <= 2.0 ** -11 * (1 + wl.abs() * 2.0 ** -9)).all()


@pytest.mark.parametrize("unit,window,sinks", [(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1, 0), (3, 1, 2 ** 31 - 1),
                                               (2 ** 31 - 1, 1, 0), (7, 2, 50)])
def test_extreme_parameters(unit, window, sinks):
    B, H, D, Nq, Nk = 1, 2, 64, 150, 200
    gen = torch.Generator("cuda").manual_seed(9)
    q, k, v = (heads(gen, B, H, n, D) for n in (Nq, Nk, Nk))
    win = F.make_window(B, H, D, Nq, Nk, window, sinks=sinks, unit=unit)
    out, lse = run(win, q, k, v)
    # what does not fit the plain form's sizes is more than there is: the same as 10^6
    cut = [min(x, 10 ** 6) for x in (unit, window, sinks)]
    check(out, lse, plain_fwd(q, k, v, *cut))


def test_scale_and_stream_and_graph():
    """A given scale, a side stream, and a captured call that is replayed on
    new inputs, a split one (few queries) among them."""
    B, H, D = 2, 4, 64
    for Nq, Nk in ((1, 2000), (200, 200)):
        gen = torch.Generator("cuda").manual_seed(4)
        q, k, v = (heads(gen, B, H, n, D) for n in (Nq, Nk, Nk))
        win = F.make_window(B, H, D, Nq, Nk, 150, sinks=4, scale=0.3)
        ws = F.window_workspace(win)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out, lse = F.window_fwd(win, q, k, v, ws, stream=side)
        side.synchronize()
        check(out, lse, plain_fwd(q, k, v, 1, 150, 4, scale=0.3))
        graph = torch.cuda.CUDAGraph()
        out, lse = torch.empty_like(out), torch.empty_like(lse)
        with torch.cuda.graph(graph):
            F.window_fwd(win, q, k, v, ws, out=out, lse=lse)
        for seed in (5, 6):
            gen = torch.Generator("cuda").manual_seed(seed)
            for t, n in ((q, Nq), (k, Nk), (v, Nk)):
                t.copy_(heads(gen, B, H, n, D))
            graph.replay()
            torch.cuda.synchronize()
            assert F.device_status(ws) == 0
            check(out, lse, plain_fwd(q, k, v, 1, 150, 4, scale=0.3))


def test_cache_past_32_bit_offsets():
    """A cache whose elements' offsets pass 2^31 and 2^32 (bytes)."""
    B, H, D, Nk = 3, 8, 128, 720896
    k = torch.zeros(B, H, Nk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(B, H, Nk, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(7)
    q = heads(gen, B, H, 1, D, mul=2.0)
    for t in (k, v):
        t[:, :, -700:] = heads(gen, B, H, 700, D)
        t[:, :, :8] = heads(gen, B, H, 8, D)
    win = F.make_window(B, H, D, 1, Nk, 700, sinks=8)
    out, lse = run(win, q, k, v)
    ks, vs = (torch.cat([t[:, :, :8], t[:, :, -700:]], 2) for t in (k, v))
    check(out, lse, plain_fwd(q, ks, vs, 1, 0, 0))
