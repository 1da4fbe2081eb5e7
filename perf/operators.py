"""Cases of the hybrid block's operators beside the gated delta rule: windowed
attention with sinks, the gated linear recurrence, and the block norm.

``own`` false: ``run`` computes an operator in elementary torch operations, in
fp32, rounded once at the end.  ``own`` true: ``run`` makes the calls a user of
gated_delta_rule_118_b200 makes.  Both take the state of ``prepare`` and return
the same outputs; ``exact`` computes them from the definitions in fp64.

Windowed attention (token i at position past + i, scale 1 / sqrt(d)):
    key j is visible to query position p  iff  j <= p and (p - j < window or j < sinks)
    o_i = sum_j softmax_j(scale q_i . k_j) v_j,   lse_i = log sum_j exp(scale q_i . k_j)
Gated linear recurrence, per channel:
    h_t = exp(log_alpha_t) h_{t-1} + w_t x_t,   y_t = h_t
Block norm, per row of D channels:
    r' = r + res_scale * sigmoid(g) * RMSNorm(y) * w_post,   x' = RMSNorm(r') * w_pre
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # prefill of one attention layer: 16 heads of 128, 4K context, 2K window, four sinks
        {"name": "swa layer", "op": "swa", "grad": False, "B": 1, "T": 4096, "past": 0, "Hq": 16, "Hk": 16, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16", "ragged": False},
        # a training batch of sequences of unequal length, grouped key/value heads, forward and backward
        {"name": "swa training", "op": "swa", "grad": True, "B": 4, "T": 4096, "past": 0, "Hq": 16, "Hk": 4, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16", "ragged": True},
        # long-context prefill
        {"name": "swa long", "op": "swa", "grad": False, "B": 1, "T": 65536, "past": 0, "Hq": 16, "Hk": 16, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16", "ragged": False},
        # small fp32 training step at odd sizes (gradient checks, small models)
        {"name": "swa odd f32", "op": "swa", "grad": True, "B": 3, "T": 333, "past": 0, "Hq": 6, "Hk": 2, "d": 64,
         "window": 100, "sinks": 3, "dtype": "f32", "ragged": True},
        # decoding 256 sequences against a full ring of 2K window tokens and the sinks
        {"name": "swa decode batch", "op": "decode", "B": 256, "slots": 2052, "Hq": 16, "Hk": 4, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16", "pos_lo": 2000, "pos_hi": 9000},
        # decoding one sequence (latency)
        {"name": "swa decode one", "op": "decode", "B": 1, "slots": 2052, "Hq": 16, "Hk": 16, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16", "pos_lo": 3000, "pos_hi": 3001},
        # recurrence over a long context, 16 heads x 128 channels
        {"name": "scan long", "op": "scan", "grad": False, "B": 1, "T": 65536, "C": 2048, "dtype": "bf16"},
        # training batch of the recurrence, forward and backward
        {"name": "scan training", "op": "scan", "grad": True, "B": 8, "T": 4096, "C": 2048, "dtype": "bf16"},
        # one decoded token of 256 sequences
        {"name": "scan step", "op": "step", "B": 256, "C": 2048, "dtype": "bf16"},
        # block norm over a training batch (8 x 4096 tokens), forward and backward
        {"name": "norm training", "op": "norm", "grad": True, "N": 32768, "D": 2048, "gate": True, "dtype": "bf16"},
        # block norm of a prefill at an odd row length, fp32, no gate
        {"name": "norm odd f32", "op": "norm", "grad": True, "N": 1111, "D": 1001, "gate": False, "dtype": "f32"},
        # block norm of one decode batch
        {"name": "norm decode", "op": "norm", "grad": False, "N": 256, "D": 2048, "gate": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["swa", "swa", "swa", "decode", "decode", "scan", "scan", "step", "norm", "norm"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("swa", "decode"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        G = rng.choice([1, 1, 2, 4, 5, 8])
        while Hk * G > 32:
            G = rng.choice([1, 2])
        d = rng.choice([64, 128])
        W = _log(rng, 4, 4096)
        S = rng.choice([0, 0, 1, 4, 16, _log(rng, 1, 200)])
        if op == "decode":
            B = _log(rng, 1, 256)
            slots = S + W + rng.choice([0, 0, rng.randrange(0, 500)])
            while B * slots * Hk * d > (1 if dt == "bf16" else 0.5) * 256 * 2052 * 4 * 128:
                B = max(1, B // 2)
                if B == 1:
                    Hk, G = 1, 4
            lo = rng.choice([0, slots, 3 * slots])
            return {"op": "decode", "B": B, "slots": slots, "Hq": Hk * G, "Hk": Hk, "d": d, "window": W, "sinks": S,
                    "dtype": dt, "pos_lo": lo, "pos_hi": lo + slots}
        grad = rng.random() < 0.6
        T = _log(rng, 8 if grad else 1, 8192)  # one token that sees itself alone has no gradient to compare
        B = _log(rng, 1, 8)
        past = rng.choice([0, 0, 0, rng.randrange(1, 1000)])
        while B * T * Hk * G * min(W + S, T + past) > (1 if dt == "bf16" else 0.1) * 4 * 4096 * 16 * 2048:
            if B > 1:
                B //= 2
            else:
                T //= 2
        return {"op": "swa", "grad": grad, "B": B, "T": T, "past": past, "Hq": Hk * G, "Hk": Hk, "d": d,
                "window": W, "sinks": min(S, T + past), "dtype": dt, "ragged": rng.random() < 0.4}
    if op == "scan":
        B, C = _log(rng, 1, 16), _log(rng, 1, 4096)
        T = _log(rng, 1, 65536)
        while B * T * C > 8 * 4096 * 2048:
            if B > 1:
                B //= 2
            else:
                T //= 2
        return {"op": "scan", "grad": rng.random() < 0.6, "B": B, "T": T, "C": C, "dtype": dt}
    if op == "step":
        return {"op": "step", "B": _log(rng, 1, 1024), "C": _log(rng, 1, 8192), "dtype": dt}
    D = rng.choice([_log(rng, 16, 16384), 8 * _log(rng, 4, 1024)])
    N = max(1, min(_log(rng, 1, 65536), 32768 * 2048 // D))
    return {"op": "norm", "grad": rng.random() < 0.6, "N": N, "D": D, "gate": rng.random() < 0.6, "dtype": dt}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def randn(*shape, dtype=dt, scale=1.0, mean=0.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, scale, generator=gen)
        return t.to(dtype)

    def uniform(*shape, lo, hi):
        return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=gen)

    s = {"case": case}
    op = case["op"]
    if op == "swa":
        B, T, Tk, Hq, Hk, d = (case["B"], case["T"], case["T"] + case["past"], case["Hq"], case["Hk"], case["d"])
        s["q"], s["k"], s["v"] = randn(B, T, Hq, d, scale=1.5), randn(B, Tk, Hk, d), randn(B, Tk, Hk, d)
        s["dO"] = randn(B, T, Hq, d) if case["grad"] else None
        s["lens"] = None
        if case["ragged"]:  # sequences padded to the longest of the batch
            s["lens"] = torch.randint(max(1, T // 2), T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    elif op == "decode":
        B, n, Hq, Hk, d = case["B"], case["slots"], case["Hq"], case["Hk"], case["d"]
        s["q"], s["k"], s["v"] = randn(B, Hq, d, scale=1.5), randn(B, Hk, d), randn(B, Hk, d)
        s["kc"], s["vc"] = randn(B, n, Hk, d), randn(B, n, Hk, d)
        s["pos"] = torch.randint(case["pos_lo"], case["pos_hi"], (B,), generator=gen, device="cuda", dtype=torch.int32)
    elif op in ("scan", "step"):
        shape = (case["B"], case["T"], case["C"]) if op == "scan" else (case["B"], case["C"])
        s["x"] = randn(*shape)
        s["w"] = torch.sigmoid(randn(*shape, dtype=torch.float32)).to(dt)
        s["la"] = -torch.exp(uniform(*shape, lo=-5.0, hi=-1.0))
        s["h"] = randn(case["B"], case["C"], dtype=torch.float32, scale=0.5)
        if op == "scan" and case["grad"]:
            s["dy"] = randn(*shape)
            s["dh"] = randn(case["B"], case["C"], dtype=torch.float32)
    else:
        N, D = case["N"], case["D"]
        s["r"], s["y"] = randn(N, D, scale=2.0), randn(N, D, scale=0.7)
        s["g"] = randn(N, D) if case["gate"] else None
        s["w_post"], s["w_pre"] = (randn(D, dtype=torch.float32, scale=0.1, mean=1.0) for _ in range(2))
        s["res"] = randn(D, dtype=torch.float32, scale=0.1, mean=0.5)
        if case["grad"]:
            s["dr"], s["dx"] = randn(N, D), randn(N, D)
    return s


# ---------------------------------------------------------------- plain forms
def _band(case):
    """Queries in blocks of L; each block sees the keys of its band (L + window - 1 of them) and the sinks."""
    T, past, S = case["T"], case["past"], case["sinks"]
    W = min(case["window"], T + past)
    L = min(T, max(W, 64))
    nb = -(-T // L)
    first = past + torch.arange(nb, device="cuda") * L
    pos = first[:, None] + torch.arange(L, device="cuda")  # [nb, L]
    key = first[:, None] - (W - 1) + torch.arange(L + W - 1, device="cuda")  # [nb, M]
    dist = pos[:, :, None] - key[:, None, :]
    near = (key[:, None, :] >= 0) & (dist >= 0) & (dist < W)
    far = pos[:, :, None] - torch.arange(S, device="cuda") >= W  # a sink behind the window
    return L, nb, torch.cat([far, near], -1), key.clamp(0, T + past - 1)


def _rows(case, lens, L, nb):
    """[B or 1, nb * L]: the rows that hold a token."""
    t = torch.arange(nb * L, device="cuda")
    return ((t < case["T"])[None] if lens is None else t[None] < lens[:, None].clamp(0, case["T"]))


def _blocks(t, L, nb, Hk):
    """[B, T, H, d] -> fp32 [B, Hk, nb, G * L, d], padded with zero rows."""
    B, T, H, d = t.shape
    t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, nb * L - T))
    return t.view(B, nb, L, Hk, H // Hk, d).permute(0, 3, 1, 4, 2, 5).reshape(B, Hk, nb, -1, d)


def _unblocks(t, case, L, nb):
    B, T, Hk, G, d = case["B"], case["T"], case["Hk"], case["Hq"] // case["Hk"], t.shape[-1]
    return t.view(B, Hk, nb, G, L, d).permute(0, 2, 4, 1, 3, 5).reshape(B, nb * L, Hk * G, d)[:, :T]


def _keys(t, case, key, nb):
    """[B, Tk, Hk, d] -> fp32 [B, Hk, nb, sinks + M, d]: the sinks, then each block's band."""
    S = case["sinks"]
    sink = t[:, None, :S].expand(-1, nb, -1, -1, -1)
    return torch.cat([sink, t[:, key]], 2).permute(0, 3, 1, 2, 4).float()


def _swa_plain(s):
    case = s["case"]
    B, T, Hk, G, d, S = case["B"], case["T"], case["Hk"], case["Hq"] // case["Hk"], case["d"], case["sinks"]
    scale = d ** -0.5
    L, nb, vis, key = _band(case)
    rows = _rows(case, s["lens"], L, nb)
    vis = vis[None] & rows.view(-1, nb, L, 1)
    q, k, v = _blocks(s["q"], L, nb, Hk), _keys(s["k"], case, key, nb), _keys(s["v"], case, key, nb)
    p = q @ k.transpose(-1, -2)  # [B, Hk, nb, G * L, S + M]
    p = p.view(B, Hk, nb, G, L, -1).mul_(scale).masked_fill_(~vis[:, None, :, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = p.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l == 0, torch.ones_like(l), l)).view(B, Hk, nb, G * L, -1)
    o = p @ v
    dt = s["q"].dtype
    out = {"o": _unblocks(o, case, L, nb).to(dt)}
    if not case["grad"]:
        return out
    lse = _unblocks((m0 + l.log()).reshape(B, Hk, nb, G * L, 1), case, L, nb)
    out["lse"] = lse[..., 0].transpose(1, 2).contiguous()
    live = rows[:, :T, None, None]
    dO = _blocks(torch.where(live, s["dO"], torch.zeros_like(s["dO"])), L, nb, Hk)
    dv = p.transpose(-1, -2) @ dO
    ds = dO @ v.transpose(-1, -2)
    ds = ds.sub_((dO * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    del p
    out["dq"] = _unblocks(ds @ k, case, L, nb).to(dt)
    dk = ds.transpose(-1, -2) @ q
    for name, g in (("dk", dk), ("dv", dv)):
        g = g.permute(0, 2, 3, 1, 4)  # [B, nb, S + M, Hk, d]
        full = torch.zeros(s["k"].shape, dtype=torch.float32, device="cuda")
        full.index_add_(1, key.reshape(-1), g[:, :, S:].reshape(B, -1, Hk, d))
        full[:, :S] += g[:, :, :S].sum(1)
        out[name] = full.to(dt)
    return out


def _slot_positions(case, pos):
    """Position held by every slot [B, slots] once the token at `pos` is in the cache, and whether it is visible."""
    S, n, W = case["sinks"], case["slots"], case["window"]
    slot = torch.arange(n, device="cuda")
    pos = pos.long()[:, None]
    ring = pos - torch.remainder(pos - slot, n - S)  # the latest position that maps to the slot
    at = torch.where(slot < S, slot, ring)
    ok = (at <= pos) & torch.where(slot < S, at >= 0, at >= S) & ((at < S) | (pos - at < W))
    return ok


def _decode_plain(s):
    case = s["case"]
    B, n, Hk, G, d, S = case["B"], case["slots"], case["Hk"], case["Hq"] // case["Hk"], case["d"], case["sinks"]
    pos = s["pos"].long()
    new = torch.where(pos < S, pos, S + torch.remainder(pos - S, n - S))
    rows = torch.arange(B, device="cuda")
    s["kc"][rows, new] = s["k"]
    s["vc"][rows, new] = s["v"]
    ok = _slot_positions(case, s["pos"])
    q = s["q"].float().view(B, Hk, G, d)
    k, v = s["kc"].permute(0, 2, 1, 3).float(), s["vc"].permute(0, 2, 1, 3).float()
    p = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~ok[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True)
    return {"o": o.view(B, Hk * G, d).to(s["q"].dtype), "k_cache": s["kc"], "v_cache": s["vc"]}


def _doubling(a, u):
    """u_t <- sum_s (prod_{r in (s, t]} a_r) u_s along dim 1, by doubling the span of every sum."""
    span = 1
    while span < u.shape[1]:
        u = torch.cat([u[:, :span], u[:, span:] + a[:, span:] * u[:, :-span]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return u


def _scan_plain(s):
    case, dt = s["case"], s["x"].dtype
    a, x, w = s["la"].exp(), s["x"].float(), s["w"].float()
    u = x * w
    u[:, 0] += a[:, 0] * s["h"]
    h = _doubling(a, u)
    out = {"y": h.to(dt), "h_T": h[:, -1].clone()}
    if not case["grad"]:
        return out
    g = s["dy"].float()  # g_t = dy_t + a_{t+1} g_{t+1}
    g[:, -1] += s["dh"]
    ar = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    g = _doubling(ar, g.flip(1)).flip(1)
    out["dx"], out["dw"] = (g * w).to(dt), (g * x).to(dt)
    out["dlog_alpha"] = g * a * torch.cat([s["h"][:, None], h[:, :-1]], 1)
    out["dh0"] = g[:, 0] * a[:, 0]
    return out


def _step_plain(s):
    s["h"].mul_(s["la"].exp()).add_(s["w"].float() * s["x"].float())
    return {"y": s["h"].to(s["x"].dtype), "h": s["h"]}


def _norm_plain(s):
    case, dt = s["case"], s["r"].dtype
    r, y = s["r"].float(), s["y"].float()
    inv_y = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    yh = y * inv_y
    gate = torch.sigmoid(s["g"].float()) if s["g"] is not None else torch.ones_like(y)
    t = s["res"] * s["w_post"]
    r1 = r + t * gate * yh
    inv_r = torch.rsqrt(r1.square().mean(-1, keepdim=True) + EPS)
    xh = r1 * inv_r
    out = {"r_out": r1.to(dt), "x_out": (xh * s["w_pre"]).to(dt)}
    if not case["grad"]:
        return out
    dx, dr = s["dx"].float(), s["dr"].float()
    out["dw_pre"] = (dx * xh).sum(0)
    dxh = dx * s["w_pre"]
    dr = dr + inv_r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    out["dr"] = dr.to(dt)
    b = dr * gate * yh
    bs = b.sum(0)
    out["dw_post"], out["dres_scale"] = bs * s["res"], bs * s["w_post"]
    if s["g"] is not None:
        out["dg_logit"] = (b * t * (1 - gate)).to(dt)
    dyh = dr * t * gate
    out["dy"] = (inv_y * (dyh - yh * (dyh * yh).mean(-1, keepdim=True))).to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls
def _own_calls(s):
    import gated_delta_rule_118_b200 as g
    case = s["case"]
    op = case["op"]
    if op == "swa":
        kw = dict(window=case["window"], sinks=case["sinks"])
        o, lse = g.gdn2_swa_fwd(s["q"], s["k"], s["v"], s["lens"], want_lse=case["grad"], **kw)
        if not case["grad"]:
            return {"o": o}
        return {"o": o, "lse": lse, **g.gdn2_swa_bwd(s["q"], s["k"], s["v"], o, lse, s["dO"], s["lens"], **kw)}
    if op == "decode":
        o = g.gdn2_swa_decode(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], window=case["window"],
                              sinks=case["sinks"])
        return {"o": o, "k_cache": s["kc"], "v_cache": s["vc"]}
    if op == "scan":
        if not case["grad"]:
            y, h_T = g.gdn2_scan_fwd(s["x"], s["w"], s["la"], s["h"])
            return {"y": y, "h_T": h_T}
        y, h_T, ckpt = g.gdn2_scan_fwd(s["x"], s["w"], s["la"], s["h"], want_ckpt=True)
        return {"y": y, "h_T": h_T, **g.gdn2_scan_bwd(s["x"], s["w"], s["la"], ckpt, s["dy"], s["dh"])}
    if op == "step":
        y = g.gdn2_scan_step(s["x"], s["w"], s["la"], s["h"])  # the state advances in place
        return {"y": y, "h": s["h"]}
    r_out, x_out = g.gdn2_block_norm_fwd(s["r"], s["y"], s["g"], s["w_post"], s["res"], s["w_pre"], EPS)
    out = {"r_out": r_out, "x_out": x_out}
    if case["grad"]:
        out.update(g.gdn2_block_norm_bwd(s["r"], s["y"], s["g"], s["w_post"], s["res"], s["w_pre"], s["dr"], s["dx"],
                                         EPS))
    return out


def run(state):
    if own:
        return {k: v for k, v in _own_calls(state).items() if v is not None}
    return {"swa": _swa_plain, "decode": _decode_plain, "scan": _scan_plain, "step": _step_plain,
            "norm": _norm_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def _pairs(case):
    """Visible (query, key) pairs of one head over a whole sequence."""
    T, past, W, S = case["T"], case["past"], case["window"], case["sinks"]
    total = 0
    for p in range(past, past + T):
        total += min(W, p + 1) + max(0, min(S, p - W + 1))
    return total


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "swa":
        q, kv = case["B"] * case["T"] * case["Hq"] * case["d"], case["B"] * (case["T"] + case["past"]) * case["Hk"] * case["d"]
        pairs = _pairs(case) * case["B"] * case["Hq"] * (0.75 if case["ragged"] else 1.0)
        if not case["grad"]:
            return {"bytes": e * (2 * q + 2 * kv), "flops": 4 * case["d"] * pairs}
        return {"bytes": e * (4 * q + 4 * kv) + 4 * case["B"] * case["T"] * case["Hq"], "flops": 14 * case["d"] * pairs}
    if op == "decode":
        seen = min(case["window"] + case["sinks"], (case["pos_lo"] + case["pos_hi"]) // 2 + 1)
        kv = case["B"] * case["Hk"] * case["d"]
        return {"bytes": e * (2 * case["B"] * case["Hq"] * case["d"] + kv * 2 * (seen + 1)),
                "flops": 4 * case["B"] * case["Hq"] * case["d"] * seen}
    if op == "scan":
        n, st = case["B"] * case["T"] * case["C"], 4 * case["B"] * case["C"]
        if not case["grad"]:
            return {"bytes": n * (3 * e + 4) + 2 * st, "flops": 4 * n}
        return {"bytes": n * (6 * e + 8) + 4 * st, "flops": 14 * n}
    if op == "step":
        n = case["B"] * case["C"]
        return {"bytes": n * (3 * e + 12), "flops": 4 * n}
    n, gate = case["N"] * case["D"], int(case["gate"])
    if not case["grad"]:
        return {"bytes": n * e * (4 + gate) + 12 * case["D"], "flops": 14 * n}
    return {"bytes": n * e * (8 + 2 * gate) + 24 * case["D"], "flops": 45 * n}


# ---------------------------------------------------------------- fp64
def _exact_swa(s):
    case = s["case"]
    B, T, past, Hq, Hk, d = case["B"], case["T"], case["past"], case["Hq"], case["Hk"], case["d"]
    W, S = case["window"], case["sinks"]
    G, step = Hq // Hk, 1024
    q, k, v = (s[n].double().transpose(1, 2) for n in ("q", "k", "v"))  # [B, H, T, d]
    o, lse = torch.zeros_like(q), torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    grad = case["grad"]
    dO = s["dO"].double().transpose(1, 2) if grad else None
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        n = T if s["lens"] is None else int(s["lens"][b])
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            pos = past + torch.arange(i0, i1, device="cuda")
            lo = max(0, past + i0 - W + 1)
            js = torch.cat([torch.arange(0, min(S, lo), device="cuda"), torch.arange(lo, past + i1, device="cuda")])
            see = (js[None] <= pos[:, None]) & ((pos[:, None] - js[None] < W) | (js[None] < S))
            for h in range(Hq):
                kk, vv = k[b, h // G, js], v[b, h // G, js]
                z = (q[b, h, i0:i1] @ kk.T) / math.sqrt(d)
                z[~see] = -math.inf
                lz = torch.logsumexp(z, -1)
                p = torch.exp(z - lz[:, None])
                o[b, h, i0:i1], lse[b, h, i0:i1] = p @ vv, lz
                if grad:
                    g = dO[b, h, i0:i1]
                    dp = g @ vv.T
                    dz = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, i0:i1] = dz @ kk
                    dk[b, h // G].index_add_(0, js, dz.T @ q[b, h, i0:i1])
                    dv[b, h // G].index_add_(0, js, p.T @ g)
    out = {"o": o.transpose(1, 2)}
    if grad:
        out.update(lse=lse, dq=dq.transpose(1, 2), dk=dk.transpose(1, 2), dv=dv.transpose(1, 2))
    return out


def _exact_decode(s):
    case = s["case"]
    B, n, Hk, d, S, W = case["B"], case["slots"], case["Hk"], case["d"], case["sinks"], case["window"]
    G, R = case["Hq"] // Hk, n - S
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        P = int(s["pos"][b])
        slot_of = lambda p: p if p < S else S + (p - S) % R  # noqa: E731
        seen = list(range(0, min(S, P + 1))) + list(range(max(S, P - W + 1), P + 1))
        seen = sorted(set(seen))
        at = torch.tensor([slot_of(p) for p in seen], device="cuda")
        s["kc"][b, slot_of(P)], s["vc"][b, slot_of(P)] = s["k"][b], s["v"][b]
        k, v = s["kc"][b, at].double(), s["vc"][b, at].double()  # [n, Hk, d]
        q = s["q"][b].double().view(Hk, G, d)
        z = torch.einsum("kgd,nkd->kgn", q, k) / math.sqrt(d)
        o[b] = torch.einsum("kgn,nkd->kgd", torch.softmax(z, -1), v).reshape(Hk * G, d)
    return {"o": o, "k_cache": s["kc"].double(), "v_cache": s["vc"].double()}


def _exact_scan(s):
    T, grad = s["x"].shape[1], s["case"]["grad"]
    h = s["h"].double()
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    for t in range(T):
        h = torch.exp(s["la"][:, t].double()) * h + s["w"][:, t].double() * s["x"][:, t].double()
        y[:, t] = h
    out = {"y": y, "h_T": h}
    if not grad:
        return out
    out.update({n: torch.empty_like(y) for n in ("dx", "dw", "dlog_alpha")})
    g = s["dh"].double()  # gradient of h_t, from later tokens
    for t in range(T - 1, -1, -1):
        g = g + s["dy"][:, t].double()
        out["dx"][:, t], out["dw"][:, t] = g * s["w"][:, t].double(), g * s["x"][:, t].double()
        g = g * torch.exp(s["la"][:, t].double())
        out["dlog_alpha"][:, t] = g * (y[:, t - 1] if t else s["h"].double())
    out["dh0"] = g
    return out


def _exact_norm(s):
    case = s["case"]
    names = ["r", "y", "w_post", "res", "w_pre"] + (["g"] if s["g"] is not None else [])
    z = {n: s[n].double().requires_grad_(case["grad"]) for n in names}

    def rms(t):
        return t / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + EPS)

    gate = 1 / (1 + torch.exp(-z["g"])) if "g" in z else 1.0
    r1 = z["r"] + z["res"] * gate * rms(z["y"]) * z["w_post"]
    x1 = rms(r1) * z["w_pre"]
    out = {"r_out": r1.detach(), "x_out": x1.detach()}
    if case["grad"]:
        got = torch.autograd.grad((r1 * s["dr"].double()).sum() + (x1 * s["dx"].double()).sum(), [z[n] for n in names])
        keys = {"r": "dr", "y": "dy", "w_post": "dw_post", "res": "dres_scale", "w_pre": "dw_pre", "g": "dg_logit"}
        out.update({keys[n]: t for n, t in zip(names, got)})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        h = torch.exp(s["la"].double()) * s["h"].double() + s["w"].double() * s["x"].double()
        return {"y": h, "h": h}
    return {"swa": _exact_swa, "decode": _exact_decode, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
