"""gdn2_scan_fwd, gdn2_scan_bwd and gdn2_scan_step against the fp64 recurrence
(oracle/hybrid.py), element by element within derived bounds."""
import pytest
import torch

import gated_delta_rule_118_b200 as g
from oracle import hybrid
from test_swa_gpu import BF, F32, U, close

pytestmark = pytest.mark.gpu


def make(B, T, C, dtype, seed, strong=False):
    gen = torch.Generator("cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, w = f(B, T, C).to(dtype), torch.sigmoid(f(B, T, C)).to(dtype)
    lo, hi = (-2.0, 3.0) if strong else (-7.0, -1.0)
    la = -torch.exp(lo + (hi - lo) * torch.rand(B, T, C, generator=gen, device="cuda"))
    return x, w, la, f(B, C), f(B, T, C).to(dtype), f(B, C)


def check(x, w, la, h0, dy, dh):
    y, h_T, ckpt = g.gdn2_scan_fwd(x, w, la, h0, want_ckpt=True)
    got = {"y": y, "h_T": h_T, **g.gdn2_scan_bwd(x, w, la, ckpt, dy, dh)}
    ref, tol = hybrid.scan(x, w, la, h0, dy, dh, u=U[x.dtype])
    for n in got:
        close(got[n], ref[n], tol[n], n)
    assert g.gdn2_check_device_error() == g.GDN2_OK
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (2, 15, 3), (1, 16, 8), (3, 17, 130), (1, 64, 64), (2, 129, 66),
                                   (1, 1000, 31), (5, 333, 256), (1, 2049, 512), (2, 700, 1001), (1, 5000, 7),
                                   (40, 70, 96), (1, 4096, 64), (300, 3, 5)])
def test_shapes(B, T, C, dtype):
    check(*make(B, T, C, dtype, seed=T + C))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [1024, 1030, 1001])
@pytest.mark.parametrize("T", [337, 64])
def test_a_cta_walks_over_several_spans_by_itself(T, C, dtype):
    """As many channel tiles as SMs and more: no clusters, and more spans than tiles are fetched ahead."""
    check(*make(10, T, C, dtype, seed=T + C))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_decay_resets_and_no_state(dtype):
    x, w, la, h0, dy, dh = make(2, 300, 68, dtype, seed=1, strong=True)
    la[:, 100] = -float("inf")   # a new document: nothing before it remains
    la[:, 200:210] = 0.0         # no decay
    got = check(x, w, la, None, dy, None)
    alone = g.gdn2_scan_fwd(x[:, 100:].contiguous(), w[:, 100:].contiguous(), la[:, 100:].contiguous())[0]
    assert ((got["y"][:, 100:] - alone).abs() <= 4 * U[dtype] * alone.abs() + 1e-6).all()
    assert (got["dlog_alpha"][:, 100] == 0).all()


def test_non_finite_values_stay_in_their_channel_and_after_their_token():
    x, w, la, h0, dy, dh = make(1, 200, 40, F32, seed=2)
    base = check(x, w, la, h0, dy, dh)
    x[0, 90, 7] = float("nan")
    x[0, 50, 8] = float("inf")
    y, h_T, ckpt = g.gdn2_scan_fwd(x, w, la, h0, want_ckpt=True)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0, 90:, 7] = keep[0, 50:, 8] = False
    assert torch.equal(y[keep], base["y"][keep]) and not y[~keep].isfinite().any()
    got = g.gdn2_scan_bwd(x, w, la, ckpt, dy, dh)
    assert torch.equal(got["dx"], base["dx"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pieces_equal_the_whole_and_steps_continue(dtype):
    x, w, la, h0, _, _ = make(2, 150, 72, dtype, seed=3)
    y, h_T = g.gdn2_scan_fwd(x, w, la, h0)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    h = h0.clone()
    parts = []
    for a, b in ((0, 40), (40, 41), (41, 140)):
        part, h2 = g.gdn2_scan_fwd(cut(x, a, b), cut(w, a, b), cut(la, a, b), h, h_T=h)  # state in place
        assert h2.data_ptr() == h.data_ptr()
        parts.append(part)
    for t in range(140, 150):
        parts.append(g.gdn2_scan_step(x[:, t].contiguous(), w[:, t].contiguous(), la[:, t].contiguous(), h)[:, None])
    ref, tol = hybrid.scan(x, w, la, h0, u=U[dtype])
    close(torch.cat(parts, 1), ref["y"], tol["y"], "y")
    close(h, ref["h_T"], tol["h_T"], "h")


@pytest.mark.parametrize("C", [64, 130, 65])
def test_state_in_place_where_ctas_share_a_sequence(C):
    """Every CTA of a cluster starts from h0, which one of them overwrites with h_T."""
    x, w, la, h0, dy, dh = make(1, 700, C, F32, seed=6)
    la.mul_(1e-3)  # (h0 is still there at the end)
    y, h_T = g.gdn2_scan_fwd(x, w, la, h0)
    for _ in range(50):
        h = h0.clone()
        again, _ = g.gdn2_scan_fwd(x, w, la, h, h_T=h)
        assert torch.equal(h, h_T) and torch.equal(again, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 5), (256, 2048), (7, 1001)])
def test_step(B, C, dtype):
    x, w, la, h0, _, _ = make(B, 1, C, dtype, seed=B + C)
    ref, tol = hybrid.scan(x, w, la, h0, u=U[dtype])
    h = h0.clone()
    y = g.gdn2_scan_step(x[:, 0], w[:, 0], la[:, 0], h)
    close(y, ref["y"][:, 0], tol["y"][:, 0], "y")
    close(h, ref["h_T"], tol["h_T"], "h")


def test_empty_sequence_copies_the_state():
    x = torch.zeros(2, 0, 8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    y, h_T, ckpt = g.gdn2_scan_fwd(x, x, x, h0, want_ckpt=True)
    assert torch.equal(h_T, h0)
    assert torch.equal(g.gdn2_scan_bwd(x, x, x, ckpt, x, h0)["dh0"], h0)
    assert (g.gdn2_scan_fwd(x, x, x)[1] == 0).all()


def test_gradient_against_differences():
    x, w, la, h0, dy, dh = make(1, 60, 12, F32, seed=4)
    got = check(x, w, la, h0, dy, dh)
    names = ("dx", "dw", "dlog_alpha", "dh0")
    for i, n in enumerate(names):
        gen = torch.Generator("cuda").manual_seed(i)
        dirn = torch.randn(got[n].shape, generator=gen, device="cuda").double()
        side = []
        for sgn in (1, -1):
            args = [t.double() for t in (x, w, la, h0)]
            args[i] = args[i] + sgn * 1e-4 * dirn
            out, _ = hybrid.scan(*args)
            side.append((out["y"] * dy.double()).sum() + (out["h_T"] * dh.double()).sum())
        num, ana = (side[0] - side[1]) / 2e-4, (got[n].double() * dirn).sum()
        assert abs(num - ana) <= 1e-4 * (got[n].double() * dirn).norm(), n


def test_repeated_calls_streams_and_graphs_give_identical_bits():
    x, w, la, h0, dy, dh = make(2, 600, 200, BF, seed=5)

    def both(**kw):
        y, h_T, ckpt = g.gdn2_scan_fwd(x, w, la, h0, want_ckpt=True, **kw)
        return [y, h_T, ckpt, *g.gdn2_scan_bwd(x, w, la, ckpt, dy, dh, **kw).values()]

    ref = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(), got))


def test_long_offsets_pass_32_bits():
    """More than 2^31 elements: the end of the sequence is right."""
    T, C = 530_000, 4096
    la = torch.full((1, T, C), -1.0, device="cuda")
    x = torch.ones(1, T, C, dtype=BF, device="cuda")
    y, h_T = g.gdn2_scan_fwd(x, x, la)
    want = 1 / (1 - torch.exp(torch.tensor(-1.0, dtype=torch.float64)))
    assert ((h_T.double().cpu() - want).abs() <= 1e-5).all()
    assert ((y[0, -1000:].double().cpu() - want).abs() <= 2.0 ** -8 * want).all()
