"""Refusals of the hybrid block's entry points: the C ABI's argument checks (no
GPU is touched) and the Python binding's."""
import ctypes

import pytest
import torch

import gated_delta_rule_118_b200 as g
from gated_delta_rule_118_b200 import build

P = ctypes.c_void_p(0x10000)    # never dereferenced: every call is refused first
MIS = ctypes.c_void_p(0x10008)
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return g.lib()


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


def swa_fwd(lib, *, q=P, k=P, lens=None, o=P, lse=P, B=1, T=8, Tk=8, Hq=4, Hk=2, d=64, window=4, sinks=0, scale=1.0,
            st=None, dtype=1):
    return lib.gdn2_swa_fwd(q, k, P, lens, o, lse, B, T, Tk, Hq, Hk, d, window, sinks, scale, st, dtype, None)


def swa_bwd(lib, *, q=P, dO=P, dq=P, dk=P, lse=P, B=1, T=8, Tk=8, Hq=4, Hk=2, d=64, window=4, sinks=0, scale=1.0,
            st=None, dtype=1):
    return lib.gdn2_swa_bwd(q, P, P, P, lse, dO, None, dq, dk, P, B, T, Tk, Hq, Hk, d, window, sinks, scale, st, dtype,
                            None)


SWA_BAD = [
    (dict(dtype=2), g.GDN2_ERR_DTYPE), (dict(B=0), g.GDN2_ERR_SHAPE), (dict(Hq=0), g.GDN2_ERR_SHAPE),
    (dict(Hk=-1), g.GDN2_ERR_SHAPE), (dict(Hq=3), g.GDN2_ERR_SHAPE), (dict(T=-1), g.GDN2_ERR_SHAPE),
    (dict(Tk=7), g.GDN2_ERR_SHAPE), (dict(window=0), g.GDN2_ERR_SHAPE), (dict(sinks=-1), g.GDN2_ERR_SHAPE),
    (dict(scale=0.0), g.GDN2_ERR_SHAPE), (dict(scale=-1.0), g.GDN2_ERR_SHAPE),
    (dict(scale=float("nan")), g.GDN2_ERR_SHAPE), (dict(scale=float("inf")), g.GDN2_ERR_SHAPE),
    (dict(d=96), g.GDN2_ERR_UNSUPPORTED), (dict(d=256), g.GDN2_ERR_UNSUPPORTED), (dict(d=0), g.GDN2_ERR_SHAPE),
    (dict(B=70000), g.GDN2_ERR_UNSUPPORTED), (dict(q=None), g.GDN2_ERR_NULL), (dict(q=MIS), g.GDN2_ERR_ALIGN),
    (dict(lse=MIS), g.GDN2_ERR_ALIGN),
    # strides {batch, token, head} of q, k, v: below d, negative, not a multiple of 16 bytes
    (dict(st=strides(999, 256, 63, 1, 128, 64, 1, 128, 64)), g.GDN2_ERR_SHAPE),
    (dict(st=strides(999, -256, 64, 1, 128, 64, 1, 128, 64)), g.GDN2_ERR_SHAPE),
    (dict(st=strides(999, 0, 64, 1, 128, 64, 1, 128, 64)), g.GDN2_ERR_SHAPE),
    (dict(st=strides(999, 256, 64, 1, 132, 64, 1, 128, 64)), g.GDN2_ERR_ALIGN),
    (dict(st=strides(999, 256, 64, 1, 128, 64, 1, 128, 68)), g.GDN2_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", SWA_BAD + [(dict(o=None), g.GDN2_ERR_NULL), (dict(k=None), g.GDN2_ERR_NULL),
                                               (dict(lens=MIS), g.GDN2_ERR_ALIGN)])
def test_swa_fwd_refuses(lib, kw, code):
    assert swa_fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SWA_BAD + [(dict(dO=None), g.GDN2_ERR_NULL), (dict(lse=None), g.GDN2_ERR_NULL),
                                               (dict(dq=None), g.GDN2_ERR_NULL), (dict(dk=None), g.GDN2_ERR_NULL),
                                               (dict(dO=MIS), g.GDN2_ERR_ALIGN)])
def test_swa_bwd_refuses(lib, kw, code):
    assert swa_bwd(lib, **kw) == code


def decode(lib, *, q=P, kc=P, pos=P, B=2, slots=10, Hq=4, Hk=2, d=64, window=8, sinks=2, scale=1.0, st=None, dtype=1):
    return lib.gdn2_swa_decode(q, P, P, kc, P, pos, P, B, slots, Hq, Hk, d, window, sinks, scale, st, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), g.GDN2_ERR_DTYPE), (dict(B=0), g.GDN2_ERR_SHAPE), (dict(Hq=5), g.GDN2_ERR_SHAPE),
    (dict(slots=9), g.GDN2_ERR_SHAPE), (dict(slots=0), g.GDN2_ERR_SHAPE), (dict(window=0), g.GDN2_ERR_SHAPE),
    (dict(window=BIG, sinks=BIG, slots=BIG), g.GDN2_ERR_SHAPE), (dict(sinks=-2), g.GDN2_ERR_SHAPE),
    (dict(scale=0.0), g.GDN2_ERR_SHAPE), (dict(d=32), g.GDN2_ERR_UNSUPPORTED), (dict(pos=None), g.GDN2_ERR_NULL),
    (dict(kc=None), g.GDN2_ERR_NULL), (dict(kc=MIS), g.GDN2_ERR_ALIGN), (dict(pos=MIS), g.GDN2_ERR_ALIGN),
    (dict(st=strides(256, 60, 128, 64, 128, 64)), g.GDN2_ERR_SHAPE),
    (dict(st=strides(260, 64, 128, 64, 128, 64)), g.GDN2_ERR_ALIGN),
])
def test_swa_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), g.GDN2_ERR_DTYPE), (dict(B=0), g.GDN2_ERR_SHAPE), (dict(C=0), g.GDN2_ERR_SHAPE),
    (dict(T=-1), g.GDN2_ERR_SHAPE), (dict(B=70000), g.GDN2_ERR_UNSUPPORTED), (dict(p=None), g.GDN2_ERR_NULL),
    (dict(p=MIS), g.GDN2_ERR_ALIGN),
])
def test_scan_refuses(lib, kw, code):
    a = dict(p=P, B=1, T=4, C=8, dtype=1)
    a.update(kw)
    n = a["B"], a["T"], a["C"], a["dtype"], None
    assert lib.gdn2_scan_fwd(a["p"], P, P, None, P, P, None, *n) == code
    assert lib.gdn2_scan_fwd(P, P, P, None, a["p"], P, None, *n) == code
    assert lib.gdn2_scan_bwd(a["p"], P, P, P, P, None, P, P, P, None, *n) == code
    assert lib.gdn2_scan_bwd(P, P, P, a["p"], P, None, P, P, P, None, *n) == code
    if a["T"] > 0:
        assert lib.gdn2_scan_step(P, P, P, a["p"], P, a["B"], a["C"], a["dtype"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), g.GDN2_ERR_DTYPE), (dict(N=-1), g.GDN2_ERR_SHAPE), (dict(D=0), g.GDN2_ERR_SHAPE),
    (dict(eps=-1.0), g.GDN2_ERR_SHAPE), (dict(eps=float("nan")), g.GDN2_ERR_SHAPE),
    (dict(D=16385), g.GDN2_ERR_UNSUPPORTED), (dict(p=None), g.GDN2_ERR_NULL), (dict(p=MIS), g.GDN2_ERR_ALIGN),
])
def test_block_norm_refuses(lib, kw, code):
    a = dict(p=P, N=4, D=64, eps=1e-6, dtype=0)
    a.update(kw)
    n = a["N"], a["D"], a["dtype"], None
    assert lib.gdn2_block_norm_fwd(a["p"], P, P, P, P, P, a["eps"], P, P, *n) == code
    assert lib.gdn2_block_norm_fwd(P, P, P, P, P, P, a["eps"], P, a["p"], *n) == code
    assert lib.gdn2_block_norm_bwd(P, P, P, P, P, P, a["eps"], P, P, a["p"], P, P, P, P, P, *n) == code
    assert lib.gdn2_block_norm_bwd(P, P, P, P, P, P, a["eps"], P, P, P, P, P, P, P, a["p"], *n) == code


def test_block_norm_gate_gradient_goes_with_the_gate(lib):
    args = lambda gl, dgl: (P, P, gl, P, P, P, 1e-6, P, P, P, P, dgl, P, P, P, 4, 64, 0, None)  # noqa: E731
    assert lib.gdn2_block_norm_bwd(*args(None, P)) == g.GDN2_ERR_NULL
    assert lib.gdn2_block_norm_bwd(*args(P, None)) == g.GDN2_ERR_NULL


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4, 4, 64)
    for call in (lambda: g.gdn2_swa_fwd(x, x, x, window=4), lambda: g.gdn2_scan_fwd(x[0], x[0], x[0]),
                 lambda: g.gdn2_block_norm_fwd(x, x, None, x[0, 0, 0], x[0, 0, 0], x[0, 0, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_types_and_layouts():
    q = torch.zeros(2, 8, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(2, 8, 2, 64, device="cuda", dtype=torch.bfloat16)
    bad = [
        (ValueError, lambda: g.gdn2_swa_fwd(q, k[:1], k, window=4)),
        (ValueError, lambda: g.gdn2_swa_fwd(q, k, k[:, :4], window=4)),
        (TypeError, lambda: g.gdn2_swa_fwd(q, k.float(), k, window=4)),
        (TypeError, lambda: g.gdn2_swa_fwd(q.half(), k.half(), k.half(), window=4)),
        (ValueError, lambda: g.gdn2_swa_fwd(q, k.cpu(), k, window=4)),
        (ValueError, lambda: g.gdn2_swa_fwd(q[..., ::2], k[..., ::2], k[..., ::2], window=4)),
        (TypeError, lambda: g.gdn2_swa_fwd(q, k, k, torch.zeros(2, device="cuda"), window=4)),
        (ValueError, lambda: g.gdn2_swa_fwd(q, k, k, torch.zeros(3, device="cuda", dtype=torch.int32), window=4)),
        (g.Gdn2Error, lambda: g.gdn2_swa_fwd(q, k, k, window=0)),
        (g.Gdn2Error, lambda: g.gdn2_swa_fwd(q, k[:, :4], k[:, :4], window=4)),          # fewer keys than queries
        (g.Gdn2Error, lambda: g.gdn2_swa_fwd(q, k[:1].expand(2, -1, -1, -1), k, window=4)),  # broadcast axis
        (ValueError, lambda: g.gdn2_swa_fwd(q, k, k, o=q[:, :4], window=4)),
        (ValueError, lambda: g.gdn2_swa_fwd(q, k, k, o=q.transpose(0, 1).contiguous().transpose(0, 1), window=4)),
    ]
    x = torch.zeros(2, 8, 16, device="cuda")
    bad += [
        (ValueError, lambda: g.gdn2_scan_fwd(x, x[:, :4], x)),
        (TypeError, lambda: g.gdn2_scan_fwd(x.bfloat16(), x.bfloat16(), x.bfloat16())),
        (ValueError, lambda: g.gdn2_scan_fwd(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2))),
        (ValueError, lambda: g.gdn2_scan_bwd(x, x, x, x[:, :3], x)),
        (ValueError, lambda: g.gdn2_scan_step(x[0], x[0], x[0], x[0, :4])),
        (ValueError, lambda: g.gdn2_block_norm_fwd(x, x, x[:1], x[0, 0], x[0, 0], x[0, 0])),
        (ValueError, lambda: g.gdn2_block_norm_fwd(x, x, None, x[0, 0, :4], x[0, 0], x[0, 0])),
        (TypeError, lambda: g.gdn2_block_norm_fwd(x, x, None, x[0, 0].double(), x[0, 0], x[0, 0])),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {i} was accepted")
