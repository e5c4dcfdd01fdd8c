"""Layer norm and sliding-window attention: struct layouts, workspace sizes and
refusals of the C ABI and of the binding, all before any device work (no GPU
needed), and the plain implementation the GPU tests compare against."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from block_sparse_spatiotemporal_b200 import fvattn as F
from tests.window_util import plain_bwd, plain_fwd, visible

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -8
AL = 0x100000                                   # an aligned address that no call may touch


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(F.library_path()):
        from block_sparse_spatiotemporal_b200 import build
        build.build()
    return F.lib()


def test_struct_layouts_match_the_c_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"fvattn_norm": F.Norm, "fvattn_window": F.Window, "fvattn_view": F.View}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fvattn.h"', "int main(void){"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += ['printf("stages %d\\n", FVATTN_STAGE_COUNT);', "return 0;}"]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
    assert int(got["stages"]) == len(F.STAGES)


def norm_fwd(lib, norm, x=AL, w=AL, b=AL, y=AL, mean=AL, rstd=AL):
    return lib.fvattn_layer_norm_fwd(ctypes.byref(norm), x, w, b, y, mean, rstd, None)


def norm_bwd(lib, norm, x=AL, dy=AL, w=AL, mean=AL, rstd=AL, dx=AL, dw=AL, db=AL, ws=AL, n=1 << 40):
    return lib.fvattn_layer_norm_bwd(ctypes.byref(norm), x, dy, w, mean, rstd, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(channels=0), SHAPE), (dict(channels=65537), SHAPE),
    (dict(groups=0), SHAPE), (dict(rows=10, groups=3), SHAPE), (dict(dtype=2), DTYPE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x_stride=63), INVALID),
    (dict(y_stride=-64), INVALID)])
def test_norm_struct_refusals(lib, kw, code):
    norm = F.make_norm(**{**dict(rows=12, channels=64), **kw})
    assert norm_fwd(lib, norm) == code and norm_bwd(lib, norm) == code
    n = ctypes.c_size_t()
    assert lib.fvattn_workspace_size_norm(ctypes.byref(norm), ctypes.byref(n)) == code


def test_norm_pointer_refusals(lib):
    norm = F.make_norm(12, 64)
    for bad in (dict(x=None), dict(y=None), dict(x=AL + 8), dict(y=AL + 2), dict(w=AL + 2), dict(b=AL + 1),
                dict(mean=AL + 2), dict(rstd=AL + 2)):
        assert norm_fwd(lib, norm, **bad) == INVALID, bad
    for bad in (dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(dx=AL + 8), dict(ws=None),
                dict(ws=AL + 16), dict(dw=AL + 2), dict(db=AL + 2), dict(dx=None, dw=None, db=None)):
        assert norm_bwd(lib, norm, **bad) == INVALID, bad
    assert norm_bwd(lib, norm, n=16) == WORKSPACE
    assert lib.fvattn_layer_norm_fwd(None, AL, AL, AL, AL, AL, AL, None) == INVALID
    assert lib.fvattn_workspace_size_norm(ctypes.byref(norm), None) == INVALID


def test_norm_workspace_grows_with_groups_and_width(lib):
    def size(*a, **kw):
        n = ctypes.c_size_t()
        assert lib.fvattn_workspace_size_norm(ctypes.byref(F.make_norm(*a, **kw)), ctypes.byref(n)) == 0
        return n.value
    assert 0 < size(0, 64) < size(1000, 64) < size(1000, 64, groups=10) < size(1000, 640, groups=10)


def view(data=AL, batch=1 << 20, head=1 << 14, token=128):
    return F.View(data, batch, head, token)


def win_fwd(lib, win, q=None, k=None, v=None, out=None, lse=AL, q_lens=None, kv_lens=None, ws=AL, n=1 << 40):
    r = lambda t: ctypes.byref(t if t is not None else view())  # noqa: E731
    return lib.fvattn_window_fwd(ctypes.byref(win), r(q), r(k), r(v), q_lens, kv_lens, r(out), lse, ws, n, None)


def win_bwd(lib, win, bad=None, lse=AL, q_lens=None, kv_lens=None, ws=AL, n=1 << 40):
    t = {i: view() for i in range(8)}
    t.update(bad or {})
    b = [ctypes.byref(t[i]) for i in range(8)]
    return lib.fvattn_window_bwd(ctypes.byref(win), *b[:5], lse, q_lens, kv_lens, *b[5:], ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(heads=6, kv_heads=4), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(q_len=-1), SHAPE), (dict(kv_len=-1), SHAPE), (dict(q_len=(1 << 28) + 1), SHAPE),
    (dict(batch=1 << 11, heads=1 << 10, kv_heads=1), SHAPE), (dict(batch=1 << 10, heads=1 << 10, kv_len=1 << 28), SHAPE),
    (dict(dtype=F.F32), DTYPE), (dict(unit=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID)])
def test_window_struct_refusals(lib, kw, code):
    win = F.make_window(**{**dict(batch=2, heads=4, head_dim=128, q_len=64, kv_len=64, window=8), **kw})
    assert win_fwd(lib, win) == code and win_bwd(lib, win) == code
    n = ctypes.c_size_t()
    assert lib.fvattn_workspace_size_window(ctypes.byref(win), ctypes.byref(n)) == code
    assert lib.fvattn_workspace_size_window_bwd(ctypes.byref(win), ctypes.byref(n)) == code


def test_window_pointer_and_stride_refusals(lib):
    win = F.make_window(2, 4, 128, 64, 64, 8)
    bad_views = [view(data=None), view(data=AL + 8), view(token=124), view(token=0), view(head=0), view(batch=-8),
                 view(head=(1 << 39))]
    for t in bad_views:
        for name in ("q", "k", "v", "out"):
            assert win_fwd(lib, win, **{name: t}) == INVALID, (name, t.data, t.token, t.head, t.batch)
        for i in range(8):
            assert win_bwd(lib, win, {i: t}) == INVALID, i
    overlapping = view(token=64)                # rows of 128 values 64 apart: an input may, an output may not
    assert win_fwd(lib, win, out=overlapping) == INVALID
    for i in (5, 6, 7):
        assert win_bwd(lib, win, {i: overlapping}) == INVALID
    assert win_fwd(lib, win, out=view(head=128, token=128)) == INVALID      # heads on top of each other's rows
    for kw in (dict(lse=None), dict(lse=AL + 2), dict(q_lens=AL + 2), dict(kv_lens=AL + 1), dict(ws=None), dict(ws=AL + 16)):
        assert win_fwd(lib, win, **kw) == INVALID and win_bwd(lib, win, **kw) == INVALID, kw
    assert win_fwd(lib, win, n=8) == WORKSPACE and win_bwd(lib, win, n=8) == WORKSPACE
    assert lib.fvattn_window_fwd(None, *[None] * 8, 0, None) == INVALID


def test_binding_refusals_without_a_gpu():
    """Tensors that are not on a GPU, and streams of no use, are refused
    before the library is called."""
    norm = F.make_norm(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.layer_norm_fwd(norm, x)
    with pytest.raises(ValueError, match="CUDA"):
        F.layer_norm_bwd(norm, x, x, torch.zeros(4), torch.zeros(4), torch.zeros(1 << 20, dtype=torch.uint8))
    win = F.make_window(1, 2, 64, 4, 4, 2)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        F.window_fwd(win, q, q, q, ws)
    with pytest.raises(ValueError, match="CUDA"):
        F.window_bwd(win, q, q, q, q, q, torch.zeros(1, 2, 4), ws)
    # helpers that only look at shapes, types and strides
    with pytest.raises(ValueError, match="q: expected"):
        F._view(q.float(), 1, 2, 4, 64, "q")
    with pytest.raises(ValueError, match="q: expected"):
        F._view(q.transpose(2, 3), 1, 2, 64, 4, "q")
    with pytest.raises(ValueError, match="row stride"):
        F._rows(x[:, :32], F.make_norm(4, 32), 0, "x")
    with pytest.raises(ValueError, match="rows of 64"):
        F._rows(x.float(), norm, 0, "x")
    with pytest.raises(ValueError, match="weight"):
        F._typed(torch.zeros(64), torch.float32, (1, 64), "weight")
    assert F._rows(x[:, :32], F.make_norm(4, 32, x_stride=64), 64, "x") == x.data_ptr()


def test_workspace_for_both_directions(lib):
    win = F.make_window(1, 14, 64, 1531, 1531, 300, sinks=7, kv_heads=2)
    a = F.window_workspace(win, device="cpu").numel()
    b = F.window_workspace(win, backward=True, device="cpu").numel()
    n = ctypes.c_size_t()
    assert lib.fvattn_workspace_size_window_bwd(ctypes.byref(win), ctypes.byref(n)) == 0
    assert b == max(a, n.value)


# ------------------------------------------------- the plain implementation
def test_visibility_by_hand():
    # tokens: window 2, one sink
    assert visible(4, 4, 1, 2, 1).int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 1, 1, 0], [1, 0, 1, 1]]
    # frames of two tokens: a frame sees itself whole, and with window 1 and no sink nothing else
    assert visible(4, 4, 2, 1, 0).int().tolist() == [[1, 1, 0, 0], [1, 1, 0, 0], [0, 0, 1, 1], [0, 0, 1, 1]]
    # the last query stands at the last key
    assert visible(1, 5, 1, 2, 1).int().tolist() == [[1, 0, 0, 1, 1]]
    # more queries than keys: the first stand before the first key
    assert visible(3, 1, 1, 0, 0).int().tolist() == [[0], [0], [1]]
    # a partial last frame is visible as far as it goes
    assert visible(3, 3, 2, 1, 0).int().tolist() == [[1, 1, 0], [1, 1, 0], [0, 0, 1]]


def test_plain_forms_against_softmax_and_autograd():
    gen = torch.Generator().manual_seed(0)
    q, dout = (torch.randn(2, 4, 9, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(2, 2, 11, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(2, 1) for t in leaves[1:])
    vis = visible(9, 11, 2, 2, 1)
    s = (leaves[0] @ kk.transpose(2, 3) / math.sqrt(8)).masked_fill(~vis, -math.inf)
    out = torch.softmax(s, -1) @ vv
    grads = torch.autograd.grad(out, leaves, dout)
    o, lse, _ = plain_fwd(q, k, v, 2, 2, 1)
    assert torch.allclose(o, out, atol=1e-12) and torch.allclose(lse, torch.logsumexp(s, -1), atol=1e-12)
    got, _ = plain_bwd(q, k, v, dout, 2, 2, 1)
    for a, b in zip(got, grads):
        assert torch.allclose(a, b, atol=1e-12)
