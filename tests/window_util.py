"""Plain 64-bit implementation of the sliding-window attention and its
gradients for the tests, with the error scales its tolerances use."""
import math

import torch


def visible(q_len, kv_len, unit, window, sinks):
    """[q_len, kv_len] truth values of one sequence of these lengths."""
    p = torch.arange(q_len)[:, None] + (kv_len - q_len)
    j = torch.arange(kv_len)[None, :]
    up, uj = torch.div(p, unit, rounding_mode="floor"), torch.div(j, unit, rounding_mode="floor")
    vis = (uj <= up) & (p >= 0)
    if window > 0:
        vis = vis & ((up - uj < window) | (uj < sinks))
    return vis


def plain_fwd(q, k, v, unit, window, sinks, scale=None, q_lens=None, kv_lens=None):
    """(out, lse, p |v|) in float64 for [B, H, N, d] tensors; rows behind
    q_lens are NaN."""
    B, H, Nq, D = q.shape
    G = H // k.shape[1]
    scale = scale or 1.0 / math.sqrt(D)
    out = torch.full((B, H, Nq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse, spread = out[..., 0].clone(), out.clone()
    for b in range(B):
        ql = Nq if q_lens is None else int(q_lens[b])
        kl = k.shape[2] if kv_lens is None else int(kv_lens[b])
        vis = visible(ql, kl, unit, window, sinks).to(q.device)
        seen = vis.any(0)
        qs = q[b, :, :ql].double()
        ks, vs = (t[b, :, :kl].double().repeat_interleave(G, 0) for t in (k, v))
        ks, vs = (torch.where(seen[None, :, None], t, 0.0) for t in (ks, vs))
        s = (qs @ ks.transpose(1, 2) * scale).masked_fill(~vis, -math.inf)
        l = torch.logsumexp(s, -1) if kl else torch.full((H, ql), -math.inf, dtype=torch.float64, device=q.device)
        p = torch.where(vis, torch.exp(s - torch.where(l.isinf(), 0.0, l)[..., None]), 0.0)
        out[b, :, :ql], lse[b, :, :ql], spread[b, :, :ql] = p @ vs, l, p @ vs.abs()
    return out, lse, spread


def plain_bwd(q, k, v, dout, unit, window, sinks, scale=None, q_lens=None, kv_lens=None):
    """(dq, dk, dv) in float64 and the error scales (a |k|, a^T |q|, p^T |dout|)
    with a = scale p (|dp| + sum |dout| p|v|); rows behind the lengths are 0."""
    B, H, Nq, D = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    G = H // Hk
    scale = scale or 1.0 / math.sqrt(D)
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=t.device)  # noqa: E731
    g, e = [z(q), z(k), z(v)], [z(q), z(k), z(v)]
    for b in range(B):
        ql = Nq if q_lens is None else int(q_lens[b])
        kl = Nk if kv_lens is None else int(kv_lens[b])
        if ql == 0 or kl == 0:
            continue
        vis = visible(ql, kl, unit, window, sinks).to(q.device)
        seen = vis.any(0)
        qs, do = q[b, :, :ql].double(), dout[b, :, :ql].double()
        ks, vs = (t[b, :, :kl].double().repeat_interleave(G, 0) for t in (k, v))
        ks, vs = (torch.where(seen[None, :, None], t, 0.0) for t in (ks, vs))
        s = (qs @ ks.transpose(1, 2) * scale).masked_fill(~vis, -math.inf)
        l = torch.logsumexp(s, -1)
        p = torch.where(vis, torch.exp(s - torch.where(l.isinf(), 0.0, l)[..., None]), 0.0)
        o = p @ vs
        dp = do @ vs.transpose(1, 2)
        ds = p * (dp - (do * o).sum(-1, keepdim=True))
        a = scale * p * (dp.abs() + (do.abs() * (p @ vs.abs())).sum(-1, keepdim=True))
        heads = lambda t: t.reshape(Hk, G, kl, D).sum(1)  # noqa: E731
        g[0][b, :, :ql], e[0][b, :, :ql] = scale * ds @ ks, a @ ks.abs()
        g[1][b, :, :kl], e[1][b, :, :kl] = heads(scale * ds.transpose(1, 2) @ qs), heads(a.transpose(1, 2) @ qs.abs())
        g[2][b, :, :kl], e[2][b, :, :kl] = heads(p.transpose(1, 2) @ do), heads(p.transpose(1, 2) @ do.abs())
    return g, e


def heads(gen, B, H, N, D, layout="bhnd", mul=1.0, device="cuda"):
    """A random bf16 [B, H, N, D] tensor: head-major, token-major, or a
    slice of a larger buffer."""
    def rnd(*shape):
        return (torch.randn(*shape, generator=gen, device=device) * mul).to(torch.bfloat16)
    if layout == "bhnd":
        return rnd(B, H, N, D)
    if layout == "bnhd":
        return rnd(B, N, H, D).transpose(1, 2)
    return rnd(B, H + 1, N + 3, D + 8)[:, 1:, 2:N + 2, 8:]
