"""gdn2_block_norm_fwd and gdn2_block_norm_bwd against the fp64 definition
(oracle/hybrid.py), element by element within derived bounds."""
import pytest
import torch

import gated_delta_rule_118_b200 as g
from oracle import hybrid
from test_swa_gpu import BF, F32, U, close

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(shape, dtype, gate, seed, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    D = shape[-1]
    r, y, gl, dr, dx = ((f(*shape) * scale).to(dtype) for _ in range(5))
    return [r, y, gl if gate else None, 1 + 0.1 * f(D), 0.5 + 0.1 * f(D), 1 + 0.1 * f(D)], dr, dx


def check(args, dr, dx, eps=EPS):
    r_out, x_out = g.gdn2_block_norm_fwd(*args, eps)
    got = {"r_out": r_out, "x_out": x_out, **g.gdn2_block_norm_bwd(*args, dr, dx, eps)}
    ref, tol = hybrid.block_norm(*args, eps, dr, dx, u=U[args[0].dtype])
    for n in got:
        if got[n] is None:
            assert args[2] is None and n == "dg_logit"
            continue
        close(got[n], ref[n], tol[n], n)
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (2, 7), (5, 64), (1, 128), (2, 3, 256), (37, 1000), (9, 1001),
                                   (700, 2048), (3, 4096), (5, 4100), (2, 8192), (300, 8200), (3, 10007), (4, 16384),
                                   (2, 16383), (5000, 96)])
def test_shapes(shape, gate, dtype):
    check(*make(shape, dtype, gate, seed=sum(shape)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape", [(5000, 96), (700, 2048), (2500, 1001), (900, 5120), (300, 8200), (60, 16384)])
def test_errors_in_the_mean_square(shape, gate, dtype):
    """Beside the bounds of each element, which grow with the length of a row and the number of rows: sums
    whose terms have no common sign, in trees and chains of at most about 100 fp32 roundings, stay within
    100 * 2^-24 = 6e-6 in the mean square; what is written in the type has its own rounding besides."""
    args, dr, dx = make(shape, dtype, gate, seed=sum(shape) + 1)
    r_out, x_out = g.gdn2_block_norm_fwd(*args, EPS)
    got = {"r_out": r_out, "x_out": x_out, **g.gdn2_block_norm_bwd(*args, dr, dx, EPS)}
    ref, _ = hybrid.block_norm(*args, EPS, dr, dx, u=U[dtype])
    for n, t in got.items():
        if t is None:
            continue
        own = U[dtype] / 3 ** 0.5 if t.dtype == BF else 0.0
        err = (t.double() - ref[n]).norm() / ref[n].norm()
        assert err <= own * 1.01 + 1e-5, (n, err)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tiny_rows_large_rows_and_strong_gates(dtype):
    args, dr, dx = make((6, 512), dtype, True, seed=1)
    args[0][0] = args[1][0] = 0          # a row of zeros: eps alone
    args[1][1] *= 1e-4
    args[0][2] *= 1e4
    args[2][3] = -60.0                   # a closed gate
    args[2][4] = 60.0                    # an open one
    got = check(args, dr, dx)
    assert all(t.isfinite().all() for t in got.values())
    assert (got["dg_logit"][3].abs() < 1e-20).all()


@pytest.mark.parametrize("D", [512, 1001, 8200])
def test_non_finite_rows_stay_alone(D):
    args, dr, dx = make((10, D), F32, True, seed=2)
    base = check(args, dr, dx)
    args[1][4, 5] = float("nan")
    args[0][7, 1] = float("inf")
    r_out, x_out = g.gdn2_block_norm_fwd(*args, EPS)
    keep = torch.ones(10, dtype=torch.bool)
    keep[[4, 7]] = False
    assert torch.equal(r_out[keep], base["r_out"][keep]) and torch.equal(x_out[keep], base["x_out"][keep])
    got = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
    for n in ("dr", "dy", "dg_logit"):
        assert torch.equal(got[n][keep], base[n][keep]), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [256, 999, 12000])
def test_in_place_and_repeated(D, dtype):
    args, dr, dx = make((150, D), dtype, True, seed=3)
    r_ref, x_ref = g.gdn2_block_norm_fwd(*args, EPS)
    ref = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
    again = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
    assert all(torch.equal(ref[n], again[n]) for n in ref)
    args[0] = args[0].clone()
    r_out, x_out = g.gdn2_block_norm_fwd(*args, EPS, r_out=args[0])
    assert r_out.data_ptr() == args[0].data_ptr()
    assert torch.equal(r_out, r_ref) and torch.equal(x_out, x_ref)


def test_streams_and_graphs():
    args, dr, dx = make((300, 640), BF, True, seed=4)
    both = lambda **kw: [*g.gdn2_block_norm_fwd(*args, EPS, **kw),  # noqa: E731
                         *g.gdn2_block_norm_bwd(*args, dr, dx, EPS, **kw).values()]
    ref = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    args[1].mul_(0.3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(), got))


def test_empty():
    args, dr, dx = make((0, 64), F32, False, seed=5)
    r_out, x_out = g.gdn2_block_norm_fwd(*args, EPS)
    assert r_out.shape == (0, 64) and x_out.shape == (0, 64)
    got = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
    assert all((got[n] == 0).all() for n in ("dw_post", "dres_scale", "dw_pre"))


def test_gradient_against_differences():
    args, dr, dx = make((7, 48), F32, True, seed=6)
    got = check(args, dr, dx)
    for i, n in enumerate(("dr", "dy", "dg_logit", "dw_post", "dres_scale", "dw_pre")):
        gen = torch.Generator("cuda").manual_seed(i)
        dirn = torch.randn(got[n].shape, generator=gen, device="cuda").double()
        side = []
        for sgn in (1, -1):
            a = [t.double() for t in args]
            a[i] = a[i] + sgn * 1e-5 * dirn
            out, _ = hybrid.block_norm(*a, EPS)
            side.append((out["r_out"] * dr.double()).sum() + (out["x_out"] * dx.double()).sum())
        num, ana = (side[0] - side[1]) / 2e-5, (got[n].double() * dirn).sum()
        assert abs(num - ana) <= 1e-4 * (got[n].double() * dirn).norm(), n


def test_more_than_2_31_elements():
    N, D = 1_050_000, 2056
    gen = torch.Generator("cuda").manual_seed(7)
    vec = [1 + 0.1 * torch.randn(D, generator=gen, device="cuda") for _ in range(3)]
    r, y = (torch.empty(N, D, dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    r_out, x_out = g.gdn2_block_norm_fwd(r, y, None, *vec, EPS)
    ref, tol = hybrid.block_norm(r[-5:], y[-5:], None, *vec, EPS)
    close(r_out[-5:], ref["r_out"], tol["r_out"], "r_out")
    close(x_out[-5:], ref["x_out"], tol["x_out"], "x_out")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 1001, 4096, 8200])
def test_logit_gradients_of_gates_between_closed_and_open(D, dtype):
    """dg_logit is proportional to gate * (1 - gate): both keep their relative accuracy, so the
    gradient of a gate at 1 - 1e-7 is right and not the rounding of the gate."""
    args, dr, dx = make((6, D), dtype, True, seed=8)
    args[2] = torch.linspace(-20, 20, 6 * D, device="cuda").view(6, D).to(dtype)
    got = check(args, dr, dx)
    ref, _ = hybrid.block_norm(*args, EPS, dr, dx, u=U[dtype])
    open_ = args[2] > 10
    err = (got["dg_logit"].double() - ref["dg_logit"])[open_].norm() / ref["dg_logit"][open_].norm()
    # its own rounding (evenly spread, U / sqrt(3)); e^-20 is formed within 20 * 2^-24, sums within a few 2^-24
    assert err <= U[dtype] / 3 ** 0.5 + 2.0 ** -18, err
    for far in (-120.0, 120.0, float("-inf"), float("inf")):
        args[2] = torch.full_like(args[2], far)
        got = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
        assert (got["dg_logit"] == 0).all() and all(got[n].isfinite().all() for n in got)
    args[2] = torch.zeros_like(args[2])
    args[2][2, 3] = float("nan")
    got = g.gdn2_block_norm_bwd(*args, dr, dx, EPS)
    assert got["dg_logit"][2, 3].isnan() and got["dg_logit"][[0, 1, 3, 4, 5]].isfinite().all()
