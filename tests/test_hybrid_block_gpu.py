"""The hybrid block's operators used together: block norms around a gated delta
rule layer, a window-attention layer and a gated linear recurrence; prefill then
decode, and a training step whose gradients are checked against autograd in fp64."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import gated_delta_rule_118_b200 as g
from oracle import hybrid

pytestmark = pytest.mark.gpu
EPS = 1e-6


def weights(H, d, gen):
    D = H * d
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    lin = lambda o: f(D, o) * D ** -0.5  # noqa: E731
    return {"gdn": {n: lin(D) for n in ("q", "k", "v", "b", "w", "la")}, "swa": {n: lin(D) for n in ("q", "k", "v")},
            "scan": {n: lin(D) for n in ("x", "w", "la")},
            "norm": [[1 + 0.1 * f(D), 0.5 + 0.1 * f(D), 1 + 0.1 * f(D)] for _ in range(3)]}


def test_prefill_and_decode_agree():
    """A three-layer stack over T + n tokens at once equals a prefill of T tokens and n single steps."""
    B, T, n, H, d, W, S = 2, 130, 9, 2, 128, 40, 2
    gen = torch.Generator("cuda").manual_seed(1)
    P = weights(H, d, gen)
    x = torch.randn(B, T + n, H * d, generator=gen, device="cuda")
    heads = lambda t: t.view(*t.shape[:-1], H, d)  # noqa: E731

    def gdn_in(h):
        p = {k: heads(h @ w) for k, w in P["gdn"].items()}
        unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
        return [t.contiguous() for t in (unit(p["q"]), unit(p["k"]), p["v"], p["b"].sigmoid(), p["w"].sigmoid(),
                                         torch.nn.functional.logsigmoid(p["la"] + 3))]

    def scan_in(h):
        return h @ P["scan"]["x"], torch.sigmoid(h @ P["scan"]["w"]), torch.nn.functional.logsigmoid(h @ P["scan"]["la"] + 2)

    def stack(x, mixers):
        r, h = x, x
        for mix, (wp, rs, wq) in zip(mixers, P["norm"]):
            r, h = g.gdn2_block_norm_fwd(r, mix(h).reshape(h.shape).contiguous(), None, wp, rs, wq, EPS)
        return h

    slots = S + W
    cache = [torch.zeros(B, slots, H, d, device="cuda") for _ in range(2)]
    state = {}

    def gdn_fwd(h):
        o, state["S"] = g.gdn2_fwd_chunked(*gdn_in(h))
        return o

    def swa_fwd(h):
        q, k, v = (heads(h @ P["swa"][m]) for m in "qkv")
        for c, t in zip(cache, (k, v)):
            for p in range(t.shape[1]):
                c[:, p if p < S else S + (p - S) % W] = t[:, p]
        return g.gdn2_swa_fwd(q, k, v, window=W, sinks=S)[0]

    def scan_fwd(h):
        y, state["h"] = g.gdn2_scan_fwd(*scan_in(h))
        return y

    whole = stack(x, (gdn_fwd, swa_fwd, scan_fwd))
    first = stack(x[:, :T].contiguous(), (gdn_fwd, swa_fwd, scan_fwd))
    tol = 2e-3  # fp32 sums in another order, through three layers and their norms
    assert ((first - whole[:, :T]).abs() <= tol).all()
    for t in range(T, T + n):
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        mixers = (lambda h: g.gdn2_decode_step(*gdn_in(h), state["S"]),
                  lambda h: g.gdn2_swa_decode(*(heads(h @ P["swa"][m]) for m in "qkv"), *cache, pos, window=W, sinks=S),
                  lambda h: g.gdn2_scan_step(*scan_in(h), state["h"]))
        h = stack(x[:, t].contiguous(), mixers)
        assert ((h - whole[:, t]).abs() <= tol).all(), t
    assert g.gdn2_check_device_error() == g.GDN2_OK


def test_training_step_gradients():
    """norm(attention) -> norm(recurrence): the operators' backward calls, chained by hand, against autograd."""
    B, T, H, d, W, S = 2, 150, 2, 64, 30, 2
    gen = torch.Generator("cuda").manual_seed(2)
    P = weights(H, d, gen)
    D = H * d
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    r0, q, k, v, gl = f(B, T, D), f(B, T, H, d), f(B, T, 1, d), f(B, T, 1, d), f(B, T, D)
    w, la, dr2, dx2 = torch.sigmoid(f(B, T, D)), -torch.exp(f(B, T, D) - 2), f(B, T, D), f(B, T, D)
    n1, n2 = P["norm"][:2]
    kw = dict(window=W, sinks=S)
    # forward
    o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
    y1 = o.view(B, T, D)
    r1, x1 = g.gdn2_block_norm_fwd(r0, y1, gl, *n1, EPS)
    h, _, ckpt = g.gdn2_scan_fwd(x1, w, la, want_ckpt=True)
    # backward of the second norm, the recurrence, the first norm, the attention
    b2 = g.gdn2_block_norm_bwd(r1, h, None, *n2, dr2, dx2, EPS)
    bs = g.gdn2_scan_bwd(x1, w, la, ckpt, b2["dy"])
    b1 = g.gdn2_block_norm_bwd(r0, y1, gl, *n1, b2["dr"], bs["dx"], EPS)
    ba = g.gdn2_swa_bwd(q, k, v, o, lse, b1["dy"].view(B, T, H, d), **kw)
    # the same in fp64 under autograd
    leaves = {n: t.double().requires_grad_() for n, t in dict(r0=r0, q=q, k=k, v=v, gl=gl, w=w, la=la).items()}
    L = leaves
    see = hybrid.visible(T, T, W, S, "cuda")
    sc = torch.einsum("bihd,bjd->bhij", L["q"], L["k"][:, :, 0]) * d ** -0.5
    att = torch.einsum("bhij,bjd->bihd", torch.softmax(sc.masked_fill(~see, -float("inf")), -1), L["v"][:, :, 0])

    def norm(r, y, gate, wts):
        wp, rs, wq = (t.double() for t in wts)
        rms = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)  # noqa: E731
        r = r + rs * gate * rms(y) * wp
        return r, rms(r) * wq

    r1d, x1d = norm(L["r0"], att.reshape(B, T, D), torch.sigmoid(L["gl"]), n1)
    hs, hd = [], torch.zeros(B, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        hd = torch.exp(L["la"][:, t]) * hd + L["w"][:, t] * x1d[:, t]
        hs.append(hd)
    r2d, x2d = norm(r1d, torch.stack(hs, 1), 1.0, n2)
    ref = torch.autograd.grad((r2d * dr2.double()).sum() + (x2d * dx2.double()).sum(), list(leaves.values()))
    got = [b1["dr"], ba["dq"], ba["dk"], ba["dv"], b1["dg_logit"], bs["dw"], bs["dlog_alpha"]]
    for name, a, b in zip(leaves, got, ref):
        assert (a.double() - b).norm() <= 2e-5 * b.norm(), (name, (a.double() - b).norm() / b.norm())


FIRST_CALL = """
import torch
import gated_delta_rule_118_b200 as g
x = torch.randn(2, 300, 128, device="cuda")
v = torch.ones(128, device="cuda")
q = torch.randn(1, 300, 2, 128, device="cuda").bfloat16()
t, cache = q[0, :4], q[0, :280].view(4, 70, 2, 128).clone()
pos = torch.tensor([5, 69, 70, -1], dtype=torch.int32, device="cuda")
calls = dict(swa_fwd=lambda: g.gdn2_swa_fwd(q, q, q, window=64, sinks=2)[0],
             swa_bwd=lambda: g.gdn2_swa_bwd(q, q, q, q, torch.zeros(1, 2, 300, device="cuda"), q, window=64)["dq"],
             decode=lambda: g.gdn2_swa_decode(t, t, t, cache, cache + 1, pos, window=64, sinks=2),
             scan=lambda: g.gdn2_scan_fwd(x, x, -x.abs())[0],
             norm_bwd=lambda: g.gdn2_block_norm_bwd(x, x, x, v, v, v, x, x)["dr"])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls["%s"]()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, calls["%s"]())
"""


@pytest.mark.parametrize("call", ["swa_fwd", "swa_bwd", "decode", "scan", "norm_bwd"])
def test_the_first_call_of_a_process_can_be_captured(call):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % (call, call)], cwd=Path(__file__).resolve().parents[1],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_graphs_with_workspaces_replayed_on_two_streams():
    """Graphs of calls that take workspaces, replayed at the same time, do not share them."""
    gen = torch.Generator("cuda").manual_seed(3)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    sets = []
    for _ in range(2):
        q, k, v, dO = (f(1, 900, 4, 64).bfloat16() for _ in range(4))
        o, lse = g.gdn2_swa_fwd(q, k, v, window=100, sinks=3)
        args = (f(400, 256), f(400, 256), f(400, 256), f(256), f(256), f(256), f(400, 256), f(400, 256))
        both = lambda q=q, k=k, v=v, o=o, lse=lse, dO=dO, args=args: (  # noqa: E731
            *g.gdn2_swa_bwd(q, k, v, o, lse, dO, window=100, sinks=3).values(), *g.gdn2_block_norm_bwd(*args).values())
        ref = both()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
        sets.append((graph, got, ref, both))  # (the inputs stay alive with their graph)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (graph, *_) in zip(streams, sets):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, ref, _ in sets:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_calls_from_two_threads():
    import threading
    gen = torch.Generator("cuda").manual_seed(4)
    q, k, v, dO = (torch.randn(1, 700, 4, 128, generator=gen, device="cuda").bfloat16() for _ in range(4))
    kw = dict(window=90, sinks=2)
    o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
    ref = [o, *g.gdn2_swa_bwd(q, k, v, o, lse, dO, **kw).values()]
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
                got = [o, *g.gdn2_swa_bwd(q, k, v, o, lse, dO, **kw).values()]
                torch.cuda.current_stream().synchronize()
                bad.extend(i for i, (a, b) in enumerate(zip(got, ref)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
