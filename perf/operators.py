"""Performance cases of the layer norm and of the sliding-window attention.

Each case is one call as a program makes it: the layer norm in front of the
QKV projection (forward and backward) and causal attention with a sliding
window and sinks (forward over whole sequences, over a chunk or a single
token against a cache, and backward).  ``run`` computes a case in plain torch
operations or, when ``own`` is true, through the package's entry points;
``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, op, rows, channels, groups, dtype, gain_one):
    return {"name": name, "op": op, "rows": rows, "channels": channels, "groups": groups, "dtype": dtype,
            "gain_one": gain_one}


def _win(name, op, batch, heads, kv_heads, head_dim, q_len, kv_len, unit, window, sinks, ragged=False,
         token_major=False):
    return {"name": name, "op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "q_len": q_len, "kv_len": kv_len, "unit": unit, "window": window, "sinks": sinks, "ragged": ragged,
            "token_major": token_major}


def listed():
    return [
        # the norm before the projection of a 20 x 32 x 52 latent at 40 heads of 128, one scale / shift per frame
        _norm("norm_fwd_480p", "norm_fwd", 33280, 5120, 20, "bf16", True),
        # one frame of a streaming step, one affine for all rows, 12 heads of 128
        _norm("norm_fwd_frame", "norm_fwd", 1024, 1536, 1, "bf16", False),
        # fp32 activations of an odd width
        _norm("norm_fwd_f32_odd", "norm_fwd", 4099, 1001, 1, "f32", False),
        # training: the norm's backward at the same latent, modulation gradients per frame
        _norm("norm_bwd_480p", "norm_bwd", 33280, 5120, 20, "bf16", True),
        # training in fp32, one affine for every row, a width that no vector load divides
        _norm("norm_bwd_f32_odd", "norm_bwd", 4099, 1001, 1, "f32", False),
        # streaming video over a whole clip: frames of 32 x 52 tokens, three frames of window, the first stays visible
        _win("win_fwd_480p", "win_fwd", 1, 40, 40, 128, 33280, 33280, 1664, 3, 1),
        # token-causal sequences with grouped heads, an odd length, four sink tokens, token-major tensors
        _win("win_fwd_tokens", "win_fwd", 2, 32, 8, 128, 4099, 4099, 1, 1024, 4, token_major=True),
        # one new frame against the cache of the frames before it
        _win("win_fwd_chunk", "win_fwd", 1, 12, 12, 128, 1024, 7168, 1024, 6, 1),
        # single tokens of 32 sequences of different lengths against a long cache
        _win("win_decode_batch", "win_fwd", 32, 32, 8, 128, 1, 32768, 1, 8192, 4, ragged=True),
        # the smallest call: one token of one sequence
        _win("win_decode_one", "win_fwd", 1, 16, 4, 64, 1, 1000, 1, 512, 4),
        # training at a 16 x 32 x 32 latent, 12 heads
        _win("win_bwd_16k", "win_bwd", 1, 12, 12, 128, 16384, 16384, 1024, 3, 1),
        # training on tokens, grouped heads, an odd length and the smaller head
        _win("win_bwd_tokens", "win_bwd", 2, 14, 2, 64, 1531, 1531, 1, 300, 7, token_major=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "win_fwd", "win_fwd", "win_decode", "win_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        channels = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            channels = max(64, channels // 64 * 64)
        groups = rng.choice([1, 1, 1, 2, 5, 20])
        rows = min(_log(rng, 1, 33280), 33280 * 5120 // channels)
        if rng.random() < 0.5:                          # narrow rows come in larger numbers
            rows = min(33280 * 5120 // channels, rows * 4)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        rows = max(groups, rows // groups * groups)
        return {"op": op, "rows": rows, "channels": channels, "groups": groups, "dtype": dtype,
                "gain_one": rng.random() < 0.5}
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 7])
    sinks = rng.choice([0, 1, 4, 64])
    if op == "win_decode":
        batch = _log(rng, 1, 32)
        kv_len = _log(rng, 1, 32768)
        q_len = min(kv_len, rng.choice([1, 1, 1, 2, 5, 8]))
        return {"op": "win_fwd", "batch": batch, "heads": heads, "kv_heads": kv_heads, "head_dim": d, "q_len": q_len,
                "kv_len": kv_len, "unit": 1, "window": _log(rng, 16, 8192), "sinks": sinks,
                "ragged": rng.random() < 0.7, "token_major": rng.random() < 0.3}
    batch = rng.choice([1, 1, 2, 3])
    unit = rng.choice([1, 1, _log(rng, 16, 1664)])
    q_len = _log(rng, 16, 8192)
    kv_len = q_len
    if op == "win_fwd" and rng.random() < 0.4:          # a chunk after a cache
        kv_len = q_len + _log(rng, 1, 8192)
    if unit == 1:
        window = rng.choice([0, _log(rng, 16, 4096), _log(rng, 16, 4096)])
    else:
        window, sinks = rng.choice([0, 1, 2, 3, 6]), rng.choice([0, 1, 2])
    while batch * heads * q_len * kv_len * d > 40 * 33280 * 6000 * 64:
        heads //= 2
        kv_heads = 1
        heads = max(1, heads)
        batch = 1
        if heads == 1:
            break
    return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "head_dim": d, "q_len": q_len,
            "kv_len": kv_len, "unit": unit, "window": window, "sinks": sinks,
            "ragged": kv_len > q_len and rng.random() < 0.5, "token_major": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _heads(g, batch, heads, tokens, d, token_major, mul):
    if token_major:
        x = torch.randn(batch, tokens, heads, d, device="cuda", generator=g)
        return (x * mul).to(torch.bfloat16).transpose(1, 2)
    x = torch.randn(batch, heads, tokens, d, device="cuda", generator=g)
    return (x * mul).to(torch.bfloat16)


def _inputs(case, seed):
    g = _gen(seed)
    st = {}
    if case["op"].startswith("norm"):
        R, C, G = case["rows"], case["channels"], case["groups"]
        dt = _DT[case["dtype"]]
        row = torch.randn(R, 1, device="cuda", generator=g)
        st["x"] = (torch.randn(R, C, device="cuda", generator=g) * (0.5 + row.abs()) + 0.5 * row).to(dt)
        st["w"] = torch.randn(G, C, device="cuda", generator=g) * 0.2 + (0.0 if case["gain_one"] else 1.0)
        st["b"] = torch.randn(G, C, device="cuda", generator=g) * 0.2
        if case["op"] == "norm_bwd":
            st["dy"] = torch.randn(R, C, device="cuda", generator=g).to(dt)
        return st
    B, H, Hk, D = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    tm = case["token_major"]
    # logits of unit spread times 2: rows from nearly uniform to a few dominant keys
    st["q"] = _heads(g, B, H, case["q_len"], D, tm, 2.0)
    st["k"] = _heads(g, B, Hk, case["kv_len"], D, tm, 1.0)
    st["v"] = _heads(g, B, Hk, case["kv_len"], D, tm, 1.0)
    st["kv_lens"] = None
    if case["ragged"]:
        lo = max(case["q_len"], case["kv_len"] // 4)
        st["kv_lens"] = torch.randint(lo, case["kv_len"] + 1, (B,), device="cuda", generator=g).to(torch.int32)
    if case["op"] == "win_bwd":
        st["dout"] = _heads(g, B, H, case["q_len"], D, tm, 1.0)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    eps = 1e-6
    if st.get("kv_lens") is not None:                   # a program knows its sequences' lengths on the host too
        st["lens_host"] = st["kv_lens"].tolist()
    if case["op"] == "norm_bwd":                        # the forward's saved statistics
        x = st["x"].double()
        mean = x.mean(1)
        var = (x - mean[:, None]).pow(2).mean(1)
        st["mean"], st["rstd"] = mean.float(), (1.0 / (var + eps).sqrt()).float()
    if case["op"] == "win_bwd":                         # the forward's outputs
        st["out"], st["lse"] = _plain_win_fwd(st)
        if case["token_major"]:
            st["out"] = st["out"].transpose(1, 2).contiguous().transpose(1, 2)
    if own:
        from block_sparse_spatiotemporal_b200 import fvattn as F
        if case["op"].startswith("norm"):
            st["plan"] = F.make_norm(case["rows"], case["channels"], groups=case["groups"],
                                     dtype=F.BF16 if case["dtype"] == "bf16" else F.F32, eps=eps,
                                     gain_one=case["gain_one"])
            if case["op"] == "norm_bwd":
                st["ws"] = F.norm_workspace(st["plan"])
        else:
            st["plan"] = F.make_window(case["batch"], case["heads"], case["head_dim"], case["q_len"], case["kv_len"],
                                       case["window"], sinks=case["sinks"], unit=case["unit"],
                                       kv_heads=case["kv_heads"])
            st["ws"] = F.window_workspace(st["plan"], backward=case["op"] == "win_bwd")
    return st


# ------------------------------------------------------------ plain forms
def _affine(st, R):
    w = st["w"] + 1.0 if st["case"]["gain_one"] else st["w"]
    rep = R // st["case"]["groups"]
    return w.repeat_interleave(rep, 0), st["b"].repeat_interleave(rep, 0)


def _plain_norm_fwd(st):
    x = st["x"].float()
    w, b = _affine(st, x.shape[0])
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / (xc.pow(2).mean(1) + 1e-6).sqrt()
    y = xc * rstd[:, None] * w + b
    return y.to(st["x"].dtype), mean, rstd


def _plain_norm_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    G = st["case"]["groups"]
    w, _ = _affine(st, x.shape[0])
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    gy = dy * w
    dx = st["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    dw = (dy * xh).reshape(G, -1, x.shape[1]).sum(1)
    db = dy.reshape(G, -1, x.shape[1]).sum(1)
    return dx.to(st["x"].dtype), dw, db


def _visible(case, kv_len, i0, i1, j0, j1):
    """Visibility of keys j0..j1-1 for queries i0..i1-1 of a sequence with kv_len keys."""
    unit = case["unit"]
    p = torch.arange(i0, i1, device="cuda") + (kv_len - case["q_len"])
    up = torch.div(p, unit, rounding_mode="floor")[:, None]
    j = torch.arange(j0, j1, device="cuda")
    uj = torch.div(j, unit, rounding_mode="floor")[None, :]
    vis = (uj <= up) & (p >= 0)[:, None] & (j < kv_len)[None, :]
    if case["window"] > 0:
        vis &= (up - uj < case["window"]) | (uj < case["sinks"])
    return vis


def _spans(case, kv_len, i0, i1):
    """Key ranges that queries i0..i1-1 can see: the sinks' and the window's."""
    unit = case["unit"]
    p0, p1 = max(0, i0 + kv_len - case["q_len"]), i1 - 1 + kv_len - case["q_len"]
    hi = min(kv_len, (p1 // unit + 1) * unit)
    lo = 0 if case["window"] == 0 else max(0, p0 // unit - case["window"] + 1) * unit
    sk = min(case["sinks"] * unit, hi)
    return [(0, hi)] if sk >= lo else [(0, sk), (lo, hi)]


def _cat(t, spans):
    return torch.cat([t[..., a:b, :] for a, b in spans], dim=-2)


def _chunks(case, st):
    """(batch, query rows, key spans, visibility) pieces of bounded size."""
    per = max(16, int(2 ** 29 // (4 * case["heads"] * max(1, min(case["kv_len"], 16384)))))
    for b in range(case["batch"]):
        n = case["kv_len"] if st["kv_lens"] is None else st["lens_host"][b]
        for i0 in range(0, case["q_len"], per):
            i1 = min(case["q_len"], i0 + per)
            spans = _spans(case, n, i0, i1)
            vis = torch.cat([_visible(case, n, i0, i1, a, c) for a, c in spans], dim=1)
            yield b, i0, i1, spans, vis


def _plain_win_fwd(st):
    case = st["case"]
    rep = case["heads"] // case["kv_heads"]
    scale = 1.0 / math.sqrt(case["head_dim"])
    out = torch.empty(case["batch"], case["heads"], case["q_len"], case["head_dim"], dtype=torch.bfloat16,
                      device="cuda")
    lse = torch.empty(out.shape[:-1], device="cuda")
    for b, i0, i1, spans, vis in _chunks(case, st):
        k, v = _cat(st["k"][b], spans).float(), _cat(st["v"][b], spans).float()
        q = st["q"][b, :, i0:i1].float().reshape(case["kv_heads"], -1, case["head_dim"])
        s = (q @ k.transpose(-1, -2) * scale).reshape(case["heads"], i1 - i0, -1)
        s.masked_fill_(~vis, float("-inf"))
        m = s.amax(-1, keepdim=True)
        s.sub_(m).exp_()
        tot = s.sum(-1, keepdim=True)
        o = (s.reshape(case["kv_heads"], rep * (i1 - i0), -1) @ v).reshape(case["heads"], i1 - i0, -1) / tot
        out[b, :, i0:i1] = o.to(torch.bfloat16)
        lse[b, :, i0:i1] = (m + tot.log())[..., 0]
    return out, lse


def _plain_win_bwd(st):
    case = st["case"]
    Hk, D, N = case["kv_heads"], case["head_dim"], case["q_len"]
    scale = 1.0 / math.sqrt(D)
    dq = torch.zeros(case["batch"], case["heads"], N, D, device="cuda")
    dk = torch.zeros(case["batch"], Hk, case["kv_len"], D, device="cuda")
    dv = torch.zeros_like(dk)
    for b, i0, i1, spans, vis in _chunks(case, st):
        n = i1 - i0
        k, v = _cat(st["k"][b], spans).float(), _cat(st["v"][b], spans).float()
        q = st["q"][b, :, i0:i1].float().reshape(Hk, -1, D)
        g = st["dout"][b, :, i0:i1].float().reshape(Hk, -1, D)
        o = st["out"][b, :, i0:i1].float().reshape(Hk, -1, D)
        p = (q @ k.transpose(-1, -2) * scale).reshape(case["heads"], n, -1)
        p = (p - st["lse"][b, :, i0:i1, None]).exp_().masked_fill_(~vis, 0.0).reshape(Hk, -1, vis.shape[1])
        gv = p.transpose(-1, -2) @ g
        ds = p * (g @ v.transpose(-1, -2) - (g * o).sum(-1, keepdim=True))
        gk = ds.transpose(-1, -2) @ q * scale
        dq[b, :, i0:i1] = (ds @ k * scale).reshape(case["heads"], n, D)
        at = 0
        for a, c in spans:
            dk[b, :, a:c] += gk[:, at:at + c - a]
            dv[b, :, a:c] += gv[:, at:at + c - a]
            at += c - a
    return tuple(t.to(torch.bfloat16) for t in (dq, dk, dv))


def run(state):
    op = state["case"]["op"]
    if own:
        from block_sparse_spatiotemporal_b200 import fvattn as F
        if op == "norm_fwd":
            return F.layer_norm_fwd(state["plan"], state["x"], weight=state["w"], bias=state["b"])
        if op == "norm_bwd":
            return F.layer_norm_bwd(state["plan"], state["x"], state["dy"], state["mean"], state["rstd"], state["ws"],
                                    weight=state["w"])
        if op == "win_fwd":
            return F.window_fwd(state["plan"], state["q"], state["k"], state["v"], state["ws"],
                                kv_lens=state["kv_lens"])
        return F.window_bwd(state["plan"], state["q"], state["k"], state["v"], state["out"], state["dout"],
                            state["lse"], state["ws"], kv_lens=state["kv_lens"])
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "win_fwd": _plain_win_fwd,
            "win_bwd": _plain_win_bwd}[op](state)


# ------------------------------------------------------------------- work
def _count(case, n):
    """Visible (query, key) pairs and keys that any query sees, of one head of a sequence with n keys."""
    unit, w, q = case["unit"], case["window"], case["q_len"]
    pairs = 0
    i = 0
    while i < q:                                        # the queries of one unit see the same keys
        u = (i + n - q) // unit
        i1 = min(q, (u + 1) * unit - (n - q))
        hi = min(n, (u + 1) * unit)
        lo = 0 if w == 0 else max(0, u - w + 1) * unit
        pairs += (i1 - i) * (hi - lo + min(case["sinks"] * unit, lo))
        i = i1
    lo = 0 if w == 0 else max(0, (n - q) // unit - w + 1) * unit
    return pairs, n - lo + min(case["sinks"] * unit, lo)


def work(case):
    if case["op"].startswith("norm"):
        size = 2 if case["dtype"] == "bf16" else 4
        n, gc = case["rows"] * case["channels"], case["groups"] * case["channels"]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * size * n + 8 * gc + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * size * n + 12 * gc + 8 * case["rows"], "flops": 14 * n}
    lens = [case["kv_len"]] * case["batch"]
    if case["ragged"]:                                  # the mean of the lengths drawn
        lens = [(max(case["q_len"], case["kv_len"] // 4) + case["kv_len"]) // 2] * case["batch"]
    pairs = keys = 0
    for n in lens:
        a, b = _count(case, n)
        pairs += a
        keys += b
    D = case["head_dim"]
    qo = case["batch"] * case["heads"] * case["q_len"] * D * 2
    kv = keys * case["kv_heads"] * D * 2 * 2
    lse = case["batch"] * case["heads"] * case["q_len"] * 4
    if case["op"] == "win_fwd":
        return {"bytes": 2 * qo + kv + lse, "flops": 4 * D * pairs * case["heads"]}
    return {"bytes": 4 * qo + 2 * kv + lse, "flops": 10 * D * pairs * case["heads"]}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"].startswith("norm"):
        x = st["x"].double().requires_grad_(case["op"] == "norm_bwd")
        w = st["w"].double().requires_grad_(case["op"] == "norm_bwd")
        b = st["b"].double().requires_grad_(case["op"] == "norm_bwd")
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + 1e-6)
        xg = ((x - mean.unsqueeze(1)) * rstd.unsqueeze(1)).view(case["groups"], -1, case["channels"])
        y = torch.addcmul(b.unsqueeze(1), xg, (w + 1 if case["gain_one"] else w).unsqueeze(1)).view_as(x)
        if case["op"] == "norm_fwd":
            return y, mean, rstd
        return torch.autograd.grad(y, (x, w, b), st["dy"].double())
    q, k, v = (st[n].double() for n in "qkv")
    back = case["op"] == "win_bwd"
    B, H, Nq, D = q.shape
    rep = H // case["kv_heads"]
    out, lse = torch.empty_like(q), q.new_empty(B, H, Nq)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = max(1, int(2 ** 27 // max(1, case["kv_len"])))
    unit = case["unit"]
    for b in range(B):
        n = case["kv_len"] if st["kv_lens"] is None else int(st["kv_lens"][b])
        key_unit = torch.arange(n, device="cuda") // unit
        for i0 in range(0, Nq, rows):
            pos = torch.arange(i0, min(Nq, i0 + rows), device="cuda") + n - Nq
            age = (pos // unit)[:, None] - key_unit[None, :]
            hide = age < 0
            if case["window"] > 0:
                hide |= (age >= case["window"]) & (key_unit >= case["sinks"])[None, :]
            for h in range(H):
                qs, ks, vs = (t.detach().requires_grad_(back)
                              for t in (q[b, h, i0:i0 + rows], k[b, h // rep, :n], v[b, h // rep, :n]))
                logits = torch.where(hide, -math.inf, torch.einsum("id,jd->ij", qs, ks) / math.sqrt(D))
                o = torch.softmax(logits, dim=1) @ vs
                if back:
                    gq, gk, gv = torch.autograd.grad(o, (qs, ks, vs), st["dout"][b, h, i0:i0 + rows].double())
                    dq[b, h, i0:i0 + rows] = gq
                    dk[b, h // rep, :n] += gk
                    dv[b, h // rep, :n] += gv
                else:
                    out[b, h, i0:i0 + rows] = o
                    lse[b, h, i0:i0 + rows] = torch.logsumexp(logits, dim=1)
    return (dq, dk, dv) if back else (out, lse)
