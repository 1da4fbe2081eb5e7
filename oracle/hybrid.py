"""fp64 definitions of the hybrid block's other operators, and elementwise error
bounds for the tests: windowed attention with sinks, the gated linear recurrence
and the block norm.  Plain torch in float64 on whatever device the inputs have.
"""
import math

import torch


def visible(T, Tk, window, sinks, device):
    """[T, Tk]: key j is visible to query i (position p = Tk - T + i)."""
    p = torch.arange(Tk - T, Tk, device=device)[:, None]
    j = torch.arange(Tk, device=device)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def swa(q, k, v, lens=None, dO=None, *, window, sinks, scale, u=2.0 ** -8):
    """Outputs, gradients and bounds as dicts.  ``u``: half a step of the type that
    probabilities, score gradients and outputs are rounded to.

    Bounds: every rounding to the type contributes u times the magnitude of what is
    rounded, carried through the sums; fp32 arithmetic contributes c = 2^-24 (4 d + n +
    64) times the sum of magnitudes (a dot of d terms, a sum of n, and the exponential
    with an argument of up to a few dozen).
    """
    B, T, Hq, d = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk
    Q, K, V = (t.double().transpose(1, 2) for t in (q, k, v))
    K, V = (t.repeat_interleave(G, 1) for t in (K, V))
    see = visible(T, Tk, window, sinks, q.device)[None, None].expand(B, 1, T, Tk)
    if lens is not None:
        row = torch.arange(T, device=q.device)[None] < lens.long()[:, None]
        see = see & row[:, None, :, None]
    c = 2.0 ** -24 * (4 * d + Tk + 64)
    s = (Q @ K.transpose(-1, -2)) * scale
    s_abs = (Q.abs() @ K.abs().transpose(-1, -2)) * scale
    cs = c + 2.0 ** -24 * d * torch.where(see, s_abs, torch.zeros_like(s_abs)).amax(-1, keepdim=True)
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(see, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    o = p @ V
    out = {"o": o.transpose(1, 2), "lse": lse}
    tol = {"o": (u * o.abs() + (u + cs) * (p @ V.abs())).transpose(1, 2),
           "lse": cs[..., 0] * (1 + lse.abs().nan_to_num(0, 0, 0))}
    if dO is None:
        return out, tol
    g = dO.double().transpose(1, 2)
    if lens is not None:
        g = torch.where(row[:, None, :, None], g, 0.0)
    dP, dP_abs = g @ V.transpose(-1, -2), g.abs() @ V.abs().transpose(-1, -2)
    D, D_abs = (g * o).sum(-1, keepdim=True), (g * o).abs().sum(-1, keepdim=True)
    dS = p * (dP - D)
    dS_err = u * dS.abs() + p * (cs * (dP_abs + D_abs) + u * D_abs)
    # the forward's o carries the rounding of its probabilities into D as well
    dS_err = dS_err + p * u * (g.abs() * (p @ V.abs())).sum(-1, keepdim=True)
    grp = lambda t: t.view(B, Hk, G, Tk, d).sum(2)  # noqa: E731
    dq, dk, dv = dS @ K * scale, grp(dS.transpose(-1, -2) @ Q) * scale, grp(p.transpose(-1, -2) @ g)
    out.update(dq=dq.transpose(1, 2), dk=dk.transpose(1, 2), dv=dv.transpose(1, 2))
    cc = c * G
    tol.update(dq=(u * dq.abs() + scale * (dS_err + cc * dS.abs()) @ K.abs()).transpose(1, 2),
               dk=(u * dk.abs() + scale * grp((dS_err + cc * dS.abs()).transpose(-1, -2) @ Q.abs())).transpose(1, 2),
               dv=(u * dv.abs() + grp((p * (u + cs + cc)).transpose(-1, -2) @ g.abs())).transpose(1, 2))
    return out, tol


def swa_decode(q, k, v, k_cache, v_cache, pos, *, window, sinks, scale, u=2.0 ** -8):
    """o, the updated caches and the bound of o, one sequence at a time over the positions it sees."""
    B, Hq, d = q.shape
    slots, Hk = k_cache.shape[1:3]
    kc, vc = k_cache.clone(), v_cache.clone()
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    slot = lambda p: p if p < sinks else sinks + (p - sinks) % (slots - sinks)  # noqa: E731
    for b in range(B):
        P = int(pos[b])
        if P < 0:
            continue
        kc[b, slot(P)], vc[b, slot(P)] = k[b], v[b]
        seen = [p for p in range(P + 1) if p < sinks or P - p < window] if P < 20000 else (
            list(range(sinks)) + list(range(P - window + 1, P + 1)))
        at = torch.tensor([slot(p) for p in seen], device=q.device)
        K, V = (t[b, at].double().repeat_interleave(Hq // Hk, 1) for t in (kc, vc))  # [n, Hq, d]
        Q = q[b].double()
        s = torch.einsum("hd,nhd->hn", Q, K) * scale
        cs = 2.0 ** -24 * (4 * d + len(seen) + 64
                           + d * scale * torch.einsum("hd,nhd->hn", Q.abs(), K.abs()).amax(-1, keepdim=True))
        pr = torch.softmax(s, -1)
        o[b] = torch.einsum("hn,nhd->hd", pr, V)
        tol[b] = u * o[b].abs() + (u + cs) * torch.einsum("hn,nhd->hd", pr, V.abs())
    return o, kc, vc, tol


def scan(x, w, log_alpha, h0=None, dy=None, dh_T=None, *, u=2.0 ** -8):
    """Outputs, gradients and bounds of the recurrence, token by token.

    Every fp32 step rounds the decay, the product and the sum (4 half steps of 2^-24 of
    the magnitudes in all, log_alpha's own exponential up to 3 of them); the magnitudes
    obey the same recurrence, and so do the errors.
    """
    B, T, C = x.shape
    X, W, A = x.double(), w.double(), log_alpha.double().exp()
    e = 8 * 2.0 ** -24
    h = torch.zeros(B, C, dtype=torch.float64, device=x.device) if h0 is None else h0.double()
    h_first, err = h, torch.zeros_like(h)
    ys, es = [], []
    for t in range(T):
        h_new = A[:, t] * h + W[:, t] * X[:, t]
        err = A[:, t] * err + e * (A[:, t] * h.abs() + (W[:, t] * X[:, t]).abs())
        h = h_new
        ys.append(h)
        es.append(err)
    y = torch.stack(ys, 1) if T else torch.zeros_like(X)
    ye = torch.stack(es, 1) if T else torch.zeros_like(X)
    out, tol = {"y": y, "h_T": h}, {"y": u * y.abs() + ye * (1 + u), "h_T": err + 2.0 ** -24 * h.abs()}
    if dy is None:
        return out, tol
    g = torch.zeros_like(h) if dh_T is None else dh_T.double()
    ge = torch.zeros_like(g)
    names = ("dx", "dw", "dlog_alpha")
    out.update({n: torch.zeros_like(X) for n in names})
    tol.update({n: torch.zeros_like(X) for n in names})
    for t in range(T - 1, -1, -1):
        ge = ge + 2.0 ** -23 * (g.abs() + dy[:, t].double().abs())
        g = g + dy[:, t].double()
        hp = y[:, t - 1] if t else h_first
        hpe = ye[:, t - 1] if t else torch.zeros_like(h_first)
        for n, f in (("dx", W[:, t]), ("dw", X[:, t])):
            out[n][:, t] = g * f
            tol[n][:, t] = (u + e) * (g * f).abs() + ge * f.abs()
        ge = A[:, t] * ge + e * (A[:, t] * g).abs()
        g = A[:, t] * g
        out["dlog_alpha"][:, t] = g * hp
        tol["dlog_alpha"][:, t] = e * (g * hp).abs() + ge * hp.abs() + g.abs() * hpe
    out["dh0"], tol["dh0"] = g, ge + 2.0 ** -24 * g.abs()
    return out, tol


def block_norm(r, y, g_logit, w_post, res_scale, w_pre, eps, dr_out=None, dx_out=None, *, u=2.0 ** -8):
    """Outputs, gradients and bounds of the block norm, gradients by autograd in fp64.

    Bounds: u of what is rounded to the type, and fp32 arithmetic of c = 2^-24 (D + 32)
    (a sum of D squares, a handful of products) of the magnitudes that are added.
    """
    D = r.shape[-1]
    c = 2.0 ** -24 * (D + 32)
    with_gate = g_logit is not None
    z = [t.double().detach().requires_grad_() for t in (r, y, w_post, res_scale, w_pre)]
    R, Y, wp, rs, wq = z
    gl = g_logit.double().detach().requires_grad_() if with_gate else None
    gate = torch.sigmoid(gl) if with_gate else torch.ones_like(R)
    rms = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + eps)  # noqa: E731
    add = rs * gate * rms(Y) * wp
    r1 = R + add
    x1 = rms(r1) * wq
    inv = torch.rsqrt((r1 * r1).mean(-1, keepdim=True) + eps)
    mag = (R.abs() + add.abs()).detach()  # r1 before any cancellation
    out = {"r_out": r1.detach(), "x_out": x1.detach()}
    tol = {"r_out": u * r1.abs() + c * mag,
           "x_out": u * x1.abs() + 2 * c * (mag + r1.abs() * (mag * mag).mean(-1, keepdim=True).sqrt() * inv) * inv * wq.abs()}
    tol = {n: t.detach() for n, t in tol.items()}
    if dr_out is None:
        return out, tol
    dro, dxo = dr_out.double(), dx_out.double()
    leaves = z + ([gl] if with_gate else [])
    grads = torch.autograd.grad((r1 * dro).sum() + (x1 * dxo).sum(), leaves)
    out.update(dict(zip(("dr", "dy", "dw_post", "dres_scale", "dw_pre", "dg_logit"), grads)))
    with torch.no_grad():
        N = max(1, r.numel() // D)
        xh = r1 * inv
        relx = 2 * c * (mag * mag).mean(-1, keepdim=True).sqrt() * inv  # relative error of inv, and of r1 in the mean
        dxh = dxo * wq
        m_abs = (dxh * xh).abs().mean(-1, keepdim=True)
        dr_mag = dro.abs() + inv * (dxh.abs() + xh.abs() * m_abs)
        dr_err = (2 * c + 4 * relx) * dr_mag + 4 * c * inv * inv * mag * m_abs
        tol["dr"] = u * out["dr"].abs() + dr_err
        iy = torch.rsqrt((Y * Y).mean(-1, keepdim=True) + eps)
        yh = Y * iy
        t = (rs * wp * gate).abs()
        dyh_err = t * (dr_err + 4 * c * dr_mag)
        mean_abs = (t * dr_mag * yh.abs()).mean(-1, keepdim=True)
        mean_err = (dyh_err * yh.abs()).mean(-1, keepdim=True) + 4 * c * mean_abs
        tol["dy"] = u * out["dy"].abs() + iy * (dyh_err + yh.abs() * mean_err + 4 * c * (t * dr_mag + yh.abs() * mean_abs))
        b_err = (gate * yh).abs() * (dr_err + 4 * c * dr_mag)
        cn = 2.0 ** -24 * (N + 16)
        b_abs = (out["dr"] * gate * yh).abs()
        lead = tuple(range(r.dim() - 1))
        b_sum = b_err.sum(lead) + cn * b_abs.sum(lead)
        tol["dw_post"], tol["dres_scale"] = b_sum * rs.abs(), b_sum * wp.abs()
        xh_err = (relx + 2 * c) * xh.abs() + 2 * c * inv * mag
        tol["dw_pre"] = (dxo.abs() * xh_err).sum(lead) + cn * (dxo * xh).abs().sum(lead)
        if with_gate:
            tol["dg_logit"] = u * out["dg_logit"].abs() + (rs * wp).abs() * (1 - gate) * (b_err + 4 * c * b_abs)
    return out, tol
