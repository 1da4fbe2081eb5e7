"""gdn2_swa_fwd, gdn2_swa_bwd and gdn2_swa_decode against the fp64 definitions
(oracle/hybrid.py), element by element within derived bounds."""
import math

import pytest
import torch

import gated_delta_rule_118_b200 as g
from oracle import hybrid

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def make(B, T, Tk, Hq, Hk, d, dtype, seed, scale=1.5):
    gen = torch.Generator("cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, dO = f(B, T, Hq, d) * scale, f(B, Tk, Hk, d), f(B, Tk, Hk, d), f(B, T, Hq, d)
    return tuple(t.to(dtype) for t in (q, k, v, dO))


def close(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~same & ~((got - ref).abs() <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], tol.expand_as(got)[bad][:4])


def check(q, k, v, dO, lens, window, sinks, scale=None, bwd=True):
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    o, lse = g.gdn2_swa_fwd(q, k, v, lens, window=window, sinks=sinks, scale=scale)
    got = {"o": o, "lse": lse}
    if bwd:
        got.update(g.gdn2_swa_bwd(q, k, v, o, lse, dO, lens, window=window, sinks=sinks, scale=scale))
    assert g.gdn2_check_device_error() == g.GDN2_OK
    ref, tol = hybrid.swa(q, k, v, lens, dO if bwd else None, window=window, sinks=sinks, scale=sc, u=U[q.dtype])
    for n in got:
        close(got[n], ref[n], tol[n], n)
    return got


SHAPES = [  # B, T, Tk, Hq, Hk, d, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0),
    (2, 1, 200, 4, 2, 128, 50, 3),       # one query against earlier keys
    (1, 127, 127, 2, 2, 128, 1000, 0),   # window longer than the sequence: plain causal
    (1, 128, 128, 3, 1, 64, 128, 128),
    (2, 129, 129, 4, 4, 128, 1, 0),      # each row sees itself only
    (1, 257, 257, 2, 1, 128, 1, 5),      # itself and the sinks
    (1, 300, 300, 5, 1, 64, 64, 200),    # sinks over several key tiles
    (3, 333, 333, 6, 2, 64, 100, 3),
    (1, 640, 640, 8, 1, 128, 130, 4),    # window ends inside a tile
    (2, 511, 700, 4, 2, 128, 256, 129),  # queries continue a sequence
    (1, 65, 1000, 2, 2, 64, 77, 1),
    (1, 1100, 1100, 2, 2, 128, 512, 0),
    (1, 2000, 2000, 2, 1, 128, 300, 260),  # many rows behind the sinks' window
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Tk,Hq,Hk,d,W,S", SHAPES)
def test_shapes(B, T, Tk, Hq, Hk, d, W, S, dtype):
    check(*make(B, T, Tk, Hq, Hk, d, dtype, seed=T + W), None, W, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_lengths_with_garbage_in_the_padding(dtype, d):
    q, k, v, dO = make(5, 300, 300, 4, 2, d, dtype, seed=5)
    lens = torch.tensor([300, 0, 1, 129, 256], dtype=torch.int32, device="cuda")
    clean = check(q, k, v, dO, lens, 90, 3)
    for b in range(5):
        for t in (q, k, v, dO):
            t[b, lens[b]:] = float("nan") if b % 2 else float("inf")
    o, lse = g.gdn2_swa_fwd(q, k, v, lens, window=90, sinks=3)
    got = {"o": o, "lse": lse, **g.gdn2_swa_bwd(q, k, v, o, lse, dO, lens, window=90, sinks=3)}
    for n in clean:  # the padding's rows are zero (lse -infinity), the others as before
        # rows whose products met the garbage are formed again in another order: at most a few roundings away
        a, b = got[n].double(), clean[n].double()
        assert a[~b.isinf()].isfinite().all(), n
        scale = b[~b.isinf()].abs().max()
        assert ((a - b)[~b.isinf()].abs() <= (0.03 if dtype == BF else 1e-5) * scale).all(), n
        assert (a[b.isinf()] == -math.inf).all()
    for b in range(5):
        assert (o[b, lens[b]:] == 0).all() and (lse[b, :, lens[b]:] == -math.inf).all()
        for n in ("dq", "dk", "dv"):
            assert (got[n][b, lens[b]:] == 0).all(), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Tk,Hq,Hk,d,W,S", [(5, 700, 700, 16, 4, 128, 200, 3), (5, 700, 700, 16, 4, 64, 1000, 0),
                                                (4, 300, 500, 12, 2, 128, 64, 130), (3, 130, 130, 2, 1, 64, 5, 2)])
def test_padding_that_is_not_finite_changes_no_bit(B, T, Tk, Hq, Hk, d, W, S, dtype):
    """No row of a sequence is formed again, or by another rounding, for what its padding holds."""
    q, k, v, dO = make(B, T, Tk, Hq, Hk, d, dtype, seed=B + d)
    n = [T, T // 2 + 1, 1, 0, T - 2][:B]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    runs = []
    for fill in (0.0, float("nan"), float("inf"), torch.finfo(dtype).max):
        for b in range(B):
            for t in (q, k, v, dO):
                t[b, t.shape[1] - T + n[b]:] = fill
        o, lse = g.gdn2_swa_fwd(q, k, v, lens, window=W, sinks=S)
        runs.append(dict(o=o, lse=lse, **g.gdn2_swa_bwd(q, k, v, o, lse, dO, lens, window=W, sinks=S)))
    assert g.gdn2_check_device_error() == g.GDN2_OK
    ref, tol = hybrid.swa(q, k, v, lens, None, window=W, sinks=S, scale=d ** -0.5, u=U[dtype])
    close(runs[0]["o"], ref["o"].nan_to_num(0), tol["o"].nan_to_num(0), "o")
    for got in runs[1:]:
        for name in got:
            assert torch.equal(got[name], runs[0][name]), name


def test_lengths_outside_the_range_are_cut():
    q, k, v, dO = make(2, 70, 70, 2, 2, 64, BF, seed=6)
    lens = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    o, lse = g.gdn2_swa_fwd(q, k, v, lens, window=16)
    full, _ = g.gdn2_swa_fwd(q, k, v, window=16)
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(o[1], full[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_non_finite_values_stay_where_they_are_seen(dtype, what):
    """A key and value that only rows [150, 250) see reach those rows only, in every output."""
    T, W, j = 400, 100, 150
    q, k, v, dO = make(1, T, T, 2, 1, 128, dtype, seed=7)
    base = check(q, k, v, dO, None, W, 2)
    v2 = v.clone()
    v2[0, j] = float(what)
    o, lse = g.gdn2_swa_fwd(q, k, v2, window=W, sinks=2)
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[j:j + W] = True
    assert not o[0, hit].isfinite().any() and o[0, ~hit].isfinite().all()
    assert torch.allclose(o[0, ~hit].float(), base["o"][0, ~hit].float(), rtol=2e-2 if dtype == BF else 1e-4, atol=1e-2 if dtype == BF else 1e-5)
    # a query and output gradient that is not finite: keys no such row sees keep their gradients
    dO2 = dO.clone()
    dO2[0, j] = float("nan")
    got = g.gdn2_swa_bwd(q, k, v, base["o"], base["lse"], dO2, window=W, sinks=2)
    seen = hybrid.visible(T, T, W, 2, "cuda")[j]
    for n in ("dk", "dv"):
        assert got[n][0, seen].isnan().any(-1).all() and got[n][0, ~seen].isfinite().all(), n
        a, b = got[n][0, ~seen].float(), base[n][0, ~seen].float()
        assert ((a - b).abs() <= (0.03 if dtype == BF else 1e-5) * b.abs().max()).all(), n
    row = torch.arange(T, device="cuda") == j
    assert got["dq"][0, ~row].isfinite().all() and got["dq"][0, row].isnan().any()
    # a key that is not finite: dq of the rows that do not see it
    k2 = k.clone()
    k2[0, j] = float("nan")
    got = g.gdn2_swa_bwd(q, k2, v, base["o"], base["lse"], dO, window=W, sinks=2)
    assert got["dq"][0, ~hit].isfinite().all() and got["dq"][0, hit].isnan().all()


def test_rows_whose_scores_are_all_minus_infinity():
    q, k, v, dO = make(1, 140, 140, 1, 1, 64, F32, seed=8)
    q[0, :, 0, 0] = 1.0
    k[0, :, 0, 0] = -math.inf
    for dtype in (F32, BF):
        o, lse = g.gdn2_swa_fwd(q.to(dtype), k.to(dtype), v.to(dtype), window=20, sinks=1)
        assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores_and_lowest_values(dtype):
    """Scores in the thousands (one key takes all the weight), and keys at the type's lowest value."""
    q, k, v, dO = make(1, 200, 200, 2, 2, 64, dtype, seed=9, scale=60.0)
    o, lse = g.gdn2_swa_fwd(q, k, v, window=64, sinks=1, scale=1.0)
    ref, tol = hybrid.swa(q, k, v, window=64, sinks=1, scale=1.0, u=U[dtype])
    close(o, ref["o"], tol["o"] + 1e-4, "o")
    close(lse, ref["lse"], tol["lse"], "lse")
    k[0, 50] = torch.finfo(dtype).min
    q[0, :, :, :] = q.abs()[0] / 60.0
    o, _ = g.gdn2_swa_fwd(q, k, v, window=64, sinks=1)
    assert o.isfinite().all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_views_of_one_projection(dtype):
    B, T, Hq, Hk, d = 2, 150, 4, 2, 64
    gen = torch.Generator("cuda").manual_seed(10)
    x = torch.randn(B, T, Hq + 2 * Hk, d, generator=gen, device="cuda").to(dtype)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    dO = torch.randn(B, T, Hq, d, generator=gen, device="cuda").to(dtype)
    got = check(q, k, v, dO, None, 40, 2)
    dense = check(q.contiguous(), k.contiguous(), v.contiguous(), dO, None, 40, 2)
    for n in got:
        assert torch.equal(got[n], dense[n]), n
    # heads outermost
    qt, kt, vt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    again = check(qt, kt, vt, dO, None, 40, 2)
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", ["sequences", "heads"])
def test_views_whose_rows_share_memory(order, dtype):
    """Windows that slide over one buffer, by a token a sequence or by a token a head: every row of the view
    counts as its own, in the outputs and in the gradients."""
    B, T, H, d = 3, 140, 4, 64
    gen = torch.Generator("cuda").manual_seed(16)
    n = (T + B + H) * H * d
    q, k, v = (torch.randn(n, generator=gen, device="cuda").to(dtype).as_strided(
        (B, T, H, d), (H * d, H * d, d, 1) if order == "sequences" else (T * d, d, d, 1)) for _ in range(3))
    dO = torch.randn(B, T, H, d, generator=gen, device="cuda").to(dtype)
    got = check(q, k, v, dO, None, 40, 2)
    dense = check(q.contiguous(), k.contiguous(), v.contiguous(), dO, None, 40, 2)
    for name in got:
        assert torch.equal(got[name], dense[name]), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_calls_give_identical_bits(dtype):
    q, k, v, dO = make(2, 500, 500, 8, 2, 128, dtype, seed=11)
    runs = []
    for _ in range(3):
        o, lse = g.gdn2_swa_fwd(q, k, v, window=100, sinks=4)
        runs.append((o, lse, *g.gdn2_swa_bwd(q, k, v, o, lse, dO, window=100, sinks=4).values()))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Tk,W,S", [(200, 200, 6, 3), (130, 140, 1, 4), (150, 150, 12, 0), (24, 24, 100, 0), (3, 20, 100, 2)])
def test_few_visible_keys_in_bf16(T, Tk, W, S, d):
    """Rows that see up to a dozen keys: score gradients carry no rounding of o, and the gradients
    little but their own (a relative rounding of at most 2^-8, evenly spread: 2^-8 / sqrt(3) in the
    mean square; operands of 16 bits and fp32 sums stay below 2^-12)."""
    q, k, v, dO = make(3, T, Tk, 6, 2, d, BF, seed=T + W)
    lens = torch.tensor([T, T // 2, 0], dtype=torch.int32, device="cuda")
    got = check(q, k, v, dO, lens, W, S)
    ref, tol = hybrid.swa(q, k, v, lens, dO, window=W, sinks=S, scale=d ** -0.5)
    if W + S <= 12 or Tk <= 24:
        for n in ("dq", "dk"):
            assert (got[n].double() - ref[n]).norm() <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12) * ref[n].norm(), n
    for t in (q, dO):
        t[1, T // 2:] = float("nan")
    o, lse = g.gdn2_swa_fwd(q, k, v, lens, window=W, sinks=S)
    # (within the bounds, not bit by bit: a row whose tile holds a NaN is formed again in fp32)
    again = g.gdn2_swa_bwd(q, k, v, o, lse, dO, lens, window=W, sinks=S)
    for n in again:
        close(again[n], ref[n], tol[n], n)


def test_gradient_against_differences():
    """Directional derivatives of sum(o * dO), fp32, against central differences of the fp64 forward."""
    q, k, v, dO = make(1, 90, 90, 4, 2, 64, F32, seed=12)
    kw = dict(window=33, sinks=2, scale=0.125)
    o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
    got = g.gdn2_swa_bwd(q, k, v, o, lse, dO, **kw)
    h = 1e-4
    for n, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        gen = torch.Generator("cuda").manual_seed(13 + i)
        dirn = torch.randn(got[n].shape, generator=gen, device="cuda").double()
        side = []
        for sgn in (1, -1):
            args = [t.double() for t in (q, k, v)]
            args[i] = args[i] + sgn * h * dirn
            side.append((hybrid.swa(*args, **kw)[0]["o"] * dO.double()).sum())
        num, ana = (side[0] - side[1]) / (2 * h), (got[n].double() * dirn).sum()
        mag = (got[n].double() * dirn).norm()
        assert abs(num - ana) <= 1e-4 * mag, (n, num, ana)


def test_long_offsets_pass_32_bits():
    """More than 2^31 elements in the keys: the last positions are addressed right."""
    Tk, H, d, T = 140_000, 128, 128, 130
    k = torch.zeros(1, Tk, H, d, dtype=BF, device="cuda")
    v = torch.zeros(1, Tk, H, d, dtype=BF, device="cuda")
    gen = torch.Generator("cuda").manual_seed(14)
    n = 400
    k[:, -n:] = torch.randn(1, n, H, d, generator=gen, device="cuda").to(BF)
    v[:, -n:] = torch.randn(1, n, H, d, generator=gen, device="cuda").to(BF)
    q = torch.randn(1, T, H, d, generator=gen, device="cuda").to(BF)
    o, _ = g.gdn2_swa_fwd(q, k, v, window=100)
    ref, tol = hybrid.swa(q, k[:, -n:], v[:, -n:], window=100, sinks=0, scale=d ** -0.5)
    close(o, ref["o"], tol["o"], "o")


def test_empty_calls():
    q = torch.zeros(2, 0, 4, 64, dtype=BF, device="cuda")
    k = torch.randn(2, 10, 2, 64, device="cuda").to(BF)
    o, lse = g.gdn2_swa_fwd(q, k, k, window=4)
    assert o.shape == q.shape
    got = g.gdn2_swa_bwd(q, k, k, o, lse, q, window=4)
    assert (got["dk"] == 0).all() and (got["dv"] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_stream_and_captured_graph(dtype):
    q, k, v, dO = make(2, 300, 300, 4, 2, 128, dtype, seed=15)
    kw = dict(window=64, sinks=2)
    o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
    ref = g.gdn2_swa_bwd(q, k, v, o, lse, dO, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = g.gdn2_swa_fwd(q, k, v, stream=side, **kw)
    got = g.gdn2_swa_bwd(q, k, v, o2, lse2, dO, stream=side, **kw)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(ref[n], got[n]) for n in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = g.gdn2_swa_fwd(q, k, v, **kw)
        got = g.gdn2_swa_bwd(q, k, v, o3, lse3, dO, **kw)
    q.copy_(torch.randn(q.shape, device="cuda"))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o, lse = g.gdn2_swa_fwd(q, k, v, **kw)
    ref = g.gdn2_swa_bwd(q, k, v, o, lse, dO, **kw)
    assert torch.equal(o, o3) and all(torch.equal(ref[n], got[n]) for n in ref)


@pytest.mark.parametrize("Hk,d,W,S", [(8, 64, 300, 3), (32, 128, 1000, 0)])
def test_more_blocks_than_the_device_holds_at_once(Hk, d, W, S):
    """480 blocks of 256 rows, full ones, short ones and padding: a CTA of the forward takes several, and
    carries its rings, score buffers and phases from one to the next."""
    B, T, Hq = 5, 700, 32
    q, k, v, dO = make(B, T, T, Hq, Hk, d, BF, seed=d)
    lens = torch.tensor([700, 300, 0, 257, 513], dtype=torch.int32, device="cuda")
    check(q, k, v, dO, lens, W, S)
    o, lse = g.gdn2_swa_fwd(q, k, v, window=W, sinks=S)
    for b in (1, 3):  # rows do not depend on what else the batch holds
        one, lse1 = g.gdn2_swa_fwd(q[b:b + 1], k[b:b + 1], v[b:b + 1], window=W, sinks=S)
        assert torch.equal(o[b:b + 1], one) and torch.equal(lse[b:b + 1], lse1)


@pytest.mark.parametrize("B,T,Tk,Hq,Hk,d,W,S,ragged", [(1, 2300, 2300, 2, 1, 64, 200, 4, False), (2, 2300, 2300, 2, 2, 128, 300, 260, True),
                                                       (1, 4500, 4500, 2, 1, 64, 500, 4, False), (1, 4500, 4700, 2, 1, 128, 128, 260, True)])
def test_query_segments_of_the_sinks(B, T, Tk, Hq, Hk, d, W, S, ragged):
    """More than 16 query tiles and sinks: the sinks' queries are split into segments, whose partial sums
    another kernel adds; and its rows that are not finite are formed again."""
    q, k, v, dO = make(B, T, Tk, Hq, Hk, d, BF, seed=T + S)
    lens = torch.tensor([T - 150, T // 3][:B], dtype=torch.int32, device="cuda") if ragged else None
    base = check(q, k, v, dO, lens, W, S)
    again = g.gdn2_swa_bwd(q, k, v, base["o"], base["lse"], dO, lens, window=W, sinks=S)
    assert all(torch.equal(base[n], again[n]) for n in again)
    row = T // 3 - 7
    dO[0, row] = float("nan")
    got = g.gdn2_swa_bwd(q, k, v, base["o"], base["lse"], dO, lens, window=W, sinks=S)
    seen = hybrid.visible(T, Tk, W, S, "cuda")[row]
    assert seen[:S].all() and not seen[S:128].any()  # (the sinks' tile holds keys of both kinds)
    for n in ("dk", "dv"):
        assert got[n][0, seen].isnan().any(-1).all() and got[n][0, ~seen].isfinite().all(), n
        a, b = got[n][0, ~seen].float(), base[n][0, ~seen].float()
        assert ((a - b).abs() <= 0.03 * b.abs().max()).all(), n


def test_long_segments_of_the_sinks():
    """So many query tiles that segments are longer than 16 of them: the sinks' dk and dv against fp64 sums
    over all rows, with the probabilities formed from the forward's lse."""
    T, d, W, S = 40_000, 64, 128, 4
    q, k, v, dO = make(1, T, T, 1, 1, d, BF, seed=31)
    o, lse = g.gdn2_swa_fwd(q, k, v, window=W, sinks=S)
    got = g.gdn2_swa_bwd(q, k, v, o, lse, dO, window=W, sinks=S)
    Q, K, V, G, O = (t[0, :, 0].double() for t in (q, k, v, dO, o))
    see = torch.arange(T, device="cuda")[:, None] >= torch.arange(S, device="cuda")[None]
    p = torch.where(see, torch.exp(Q @ K[:S].T * d ** -0.5 - lse[0, 0].double()[:, None]), 0.0)
    dS = p * (G @ V[:S].T - (G * O).sum(-1, keepdim=True))
    # P is rounded by at most 2^-8 of itself for dv, independently row by row, and so the sum's error is at
    # most 2^-8 of the sum in the mean square; the output's rounding is another 2^-8
    for n, ref in (("dv", p.T @ G), ("dk", dS.T @ Q * d ** -0.5)):
        assert (got[n][0, :S, 0].double() - ref).norm() <= 2.0 ** -7 * ref.norm(), n


@pytest.mark.parametrize("d", [64, 128])
def test_later_keys_that_outgrow_the_first_tiles_by_far(d):
    """Scores that jump by 2^90 and by more than fp32 holds between blocks all of whose keys are visible:
    those blocks are taken again with a new reference."""
    T = 900
    q, k, v, dO = make(1, T, T, 2, 1, d, BF, seed=32, scale=0.3)
    q[..., 0] = 8.0
    for j, level in ((0, 0.0), (130, 8.0), (330, 12.0), (520, 40.0), (700, 3.0)):  # scores of 0, 64, 96, 320, 24
        k[:, j:, :, 0] = level
    for lens in (None, torch.tensor([610], dtype=torch.int32, device="cuda")):
        check(q, k, v, dO, lens, T, 0, scale=1.0)
        check(q, k, v, dO, lens, 512, 70, scale=1.0)


# ---------------------------------------------------------------- decode
def decode_case(B, slots, Hq, Hk, d, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    return f(B, Hq, d), f(B, Hk, d), f(B, Hk, d), f(B, slots, Hk, d), f(B, slots, Hk, d)


def check_decode(q, k, v, kc, vc, pos, window, sinks):
    ref, kr, vr, tol = hybrid.swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks, scale=q.shape[-1] ** -0.5,
                                         u=U[q.dtype])
    o = g.gdn2_swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks)
    assert torch.equal(kc, kr) and torch.equal(vc, vr)
    close(o, ref, tol, "o")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,d", [(1, 1, 64), (4, 4, 128), (4, 2, 64), (5, 1, 128), (6, 2, 128), (16, 2, 64),
                                     (16, 1, 128), (20, 1, 64), (33, 1, 128)])
@pytest.mark.parametrize("window,sinks,extra", [(1, 0, 0), (50, 3, 0), (64, 0, 17), (700, 130, 5)])
def test_decode(Hq, Hk, d, window, sinks, extra, dtype):
    slots = window + sinks + extra
    pos = torch.tensor([0, 1, sinks, slots - 1, slots, 2 * slots + 3, -1, 1_000_003], dtype=torch.int32, device="cuda")
    q, k, v, kc, vc = decode_case(len(pos), slots, Hq, Hk, d, dtype, seed=Hq + window)
    check_decode(q, k, v, kc, vc, pos, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 5, 8, 12])
@pytest.mark.parametrize("B,Hk,window,sinks", [(64, 4, 300, 3), (64, 8, 50, 2)])
def test_decode_of_a_batch(B, Hk, window, sinks, G, d, dtype):
    """Batches that fill the device: few CTAs a row, and (the second) one, which needs no cluster."""
    slots = window + sinks + 3
    q, k, v, kc, vc = decode_case(B, slots, G * Hk, Hk, d, dtype, seed=G + d)
    pos = torch.arange(B, dtype=torch.int32, device="cuda") * 37 % 800 - 1
    check_decode(q, k, v, kc, vc, pos, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_leaves_rows_without_a_sequence_alone_and_ignores_unseen_slots(dtype):
    window, sinks, slots = 40, 2, 60
    pos = torch.tensor([-1, 30, 500], dtype=torch.int32, device="cuda")
    q, k, v, kc, vc = decode_case(3, slots, 4, 2, 128, dtype, seed=3)
    kc[1, 31:], vc[1, 31:] = float("nan"), float("inf")  # not written yet
    ring = slots - sinks
    for p in range(500 - ring + 1, 500 - window + 1):    # behind the window
        kc[2, sinks + (p - sinks) % ring] = float("inf")
        vc[2, sinks + (p - sinks) % ring] = float("nan")
    before = kc[0].clone()
    ref, _, _, tol = hybrid.swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks, scale=128 ** -0.5, u=U[dtype])
    o = g.gdn2_swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks)
    close(o, ref, tol, "o")
    assert (o[0] == 0).all() and torch.equal(kc[0], before)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [2, 80])
def test_decode_of_an_infinite_value_that_is_seen(B, d, dtype):
    """An infinity in a visible value row reaches its channel as an infinity, also where that row
    is the last of a run of positions (whose length is seldom a multiple of a step)."""
    window, sinks = 45, 2
    slots = window + sinks
    for P in (0, 6, 17, 40, 46, 100):
        seen = [p for p in range(P + 1) if p < sinks or P - p < window]
        for at in {seen[0], seen[len(seen) // 2], seen[-2] if P else 0, seen[-1]}:
            q, k, v, kc, vc = decode_case(B, slots, 12, 4, d, dtype, seed=P)
            pos = torch.full((B,), P, dtype=torch.int32, device="cuda")
            row = v if at == P else vc[:, at if at < sinks else sinks + (at - sinks) % window]
            row[:, :, 5], row[:, :, 9] = math.inf, -math.inf
            ref = hybrid.swa_decode(q[:2], k[:2], v[:2], kc[:2], vc[:2], pos[:2], window=window, sinks=sinks, scale=d ** -0.5)[0]
            o = g.gdn2_swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks)
            assert (o[..., 5] == math.inf).all() and (o[..., 9] == -math.inf).all(), (P, at)
            rest = [c for c in range(d) if c not in (5, 9)]
            # roundings of the probabilities and of o, and fp32 sums: as the bounds elsewhere, of values up to 6
            assert ((o[:2].double() - ref)[..., rest].abs() <= 2 * U[dtype] * 6 + 1e-4).all(), (P, at)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_strided_graph_and_large_cache(dtype):
    """Views of a packed projection, inside a captured graph whose position advances on the device,
    with a cache of more than 2^31 bytes."""
    B, Hq, Hk, d, window, sinks = 3, 4, 2, 128, 64, 4
    slots = 1_500_000 if dtype == BF else 800_000
    kc, vc = (torch.zeros(B, slots, Hk, d, dtype=dtype, device="cuda") for _ in range(2))
    x = torch.empty(B, Hq + 2 * Hk, d, dtype=dtype, device="cuda")
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    pos = torch.tensor([slots - 2, 0, 5], dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(4)
    for t in (kc, vc):
        t[:, -200:] = torch.randn(B, 200, Hk, d, generator=gen, device="cuda").to(dtype)
        t[:, :20] = torch.randn(B, 20, Hk, d, generator=gen, device="cuda").to(dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = g.gdn2_swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks)
        pos += 1
    for step in range(4):  # runs over the end of the ring
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        ref, kr, vr, tol = hybrid.swa_decode(q, k, v, kc, vc, pos, window=window, sinks=sinks, scale=d ** -0.5, u=U[dtype])
        graph.replay()
        torch.cuda.synchronize()
        close(o, ref, tol, f"o at step {step}")
        assert torch.equal(kc, kr) and torch.equal(vc, vr)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_continues_a_prefill(dtype):
    """Prefill, then token by token through the ring: the same rows as one long prefill."""
    B, T, n, Hq, Hk, d, W, S = 2, 90, 25, 4, 2, 64, 32, 3
    q, k, v, _ = make(B, T + n, T + n, Hq, Hk, d, dtype, seed=21)
    full, _ = g.gdn2_swa_fwd(q, k, v, window=W, sinks=S)
    slots = S + W
    kc, vc = (torch.zeros(B, slots, Hk, d, dtype=dtype, device="cuda") for _ in range(2))
    for p in range(T):
        s = p if p < S else S + (p - S) % W
        kc[:, s], vc[:, s] = k[:, p], v[:, p]
    for p in range(T, T + n):
        pos = torch.full((B,), p, dtype=torch.int32, device="cuda")
        o = g.gdn2_swa_decode(q[:, p], k[:, p], v[:, p], kc, vc, pos, window=W, sinks=S)
        tol = 2.0 ** -6 if dtype == BF else 1e-5
        assert ((o - full[:, p]).abs() <= tol * v.abs().max()).all()
