"""GPU parity of the sliding-window attention where a row's running reference
moves more than once inside a step and what it leaves behind still counts:
probabilities stored earlier in the step and the output of earlier steps are
read back from tensor memory, scaled and stored again.  A tile's keys are
worked on 32 at a time, so the logits (in units of log 2, exact in bf16) rise
from one 32 keys to the next by just less, or just more, than what moves it."""
import math

import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from tests.test_gpu_window import check_far, run
from tests.window_util import plain_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [4, 40, 100, 200])
@pytest.mark.parametrize("rise", [18, 58])
@pytest.mark.parametrize("twice", [False, True])
def test_moves_that_leave_weight_behind(twice, rise, Nq, D):
    """Tiles at 0, then at `rise` (32 keys sum to 2^(rise + 5): no move past a
    bound of 2^(rise + 6)), then tiles whose 32 keys stand at `rise`,
    rise + 2 (one move: the keys before, and the tiles before, keep a quarter
    of its weight each) or at rise + 2, 2 (rise + 2) (two moves: the tiles
    before must be scaled by both).  One item a (batch, head), 150 of them, so
    that no item's keys are split."""
    B, H, tiles = 150, 1, 6
    up = rise + 2
    chunks = torch.zeros(tiles + 2, 4)
    chunks[2:4] = rise
    chunks[4:6] = torch.tensor([up, 2 * up, up, 2 * up] if twice else [rise, up, rise, up]).float()
    Nk = 128 * tiles + Nq
    level = chunks.reshape(-1).repeat_interleave(32)[:Nk].cuda()
    gen = torch.Generator("cuda").manual_seed(11)
    q = torch.zeros(B, H, Nq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    q[..., 1:] = torch.randn(B, H, Nq, D - 1, generator=gen, device="cuda").to(torch.bfloat16) * 0.25
    k = torch.randn(B, H, Nk, D, generator=gen, device="cuda").to(torch.bfloat16) * 0.125
    k[..., 0] = level.to(torch.bfloat16)
    v = torch.randn(B, H, Nk, D, generator=gen, device="cuda").to(torch.bfloat16)
    win = F.make_window(B, H, D, Nq, Nk, 0, scale=math.log(2.0))
    out, lse = run(win, q, k, v)
    check_far(out, lse, plain_fwd(q, k, v, 1, 0, 0, scale=math.log(2.0)))
    again = run(win, q, k, v)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,B", [(1, 1), (4, 150), (40, 150), (100, 150), (200, 40)])
def test_large_and_small_values_under_a_reference_that_lags(Nq, B, D):
    """|v| up to 2^80 and down to 2^-80 with most keys' logits far above the
    first tile's, or at its level: the output is a mean of v, and no sum on the
    way to it leaves fp32."""
    H, Nk = 1, 2000
    gen = torch.Generator("cuda").manual_seed(13)
    q = torch.zeros(B, H, Nq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    k = torch.randn(B, H, Nk, D, generator=gen, device="cuda").to(torch.bfloat16)
    for rise, size in ((15, 79), (18, 79), (50, 79), (56, 79), (0, 79), (0, -80), (56, -80)):
        k[..., 0] = (torch.arange(Nk, device="cuda") >= 140).to(torch.bfloat16) * rise
        v = (torch.rand(B, H, Nk, D, generator=gen, device="cuda") + 1).to(torch.bfloat16) * 2.0 ** size
        win = F.make_window(B, H, D, Nq, Nk, 0, scale=math.log(2.0))
        out, lse = run(win, q, k, v)
        assert out.isfinite().all()
        check_far(out, lse, plain_fwd(q, k, v, 1, 0, 0, scale=math.log(2.0)))
