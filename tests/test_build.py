"""The build's two products: the library, and the module that calls it from Python."""
import sysconfig

import pytest

import gated_delta_rule_118_b200 as g
from gated_delta_rule_118_b200 import build

P, MIS = 0x10000, 0x10008  # never dereferenced: every call is refused first


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_library()


def test_the_library_is_built_where_the_calling_module_cannot_be(monkeypatch, tmp_path):
    """Without a host compiler (or Python's headers) the library is in place and up to date all the same."""
    monkeypatch.setattr(build, "CALLER", tmp_path / build.CALLER.name)
    for cc in ("/bin/false", str(tmp_path / "missing")):
        monkeypatch.setenv("CC", cc)
        with pytest.warns(UserWarning, match="ctypes"):
            assert build.build_library() == build.LIBRARY
        with pytest.raises(RuntimeError):
            build.build_caller()
        assert build.LIBRARY.exists() and not build.is_stale() and not build.CALLER.exists()


def test_the_calling_module_is_the_interpreters_own():
    assert build.CALLER.name == "_call" + sysconfig.get_config_var("EXT_SUFFIX")


CALLS = {  # arguments, and where the first pointer, a size, the type, a float and the strides stand
    "swa_fwd": ((P, P, P, None, P, P, 1, 8, 8, 4, 2, 64, 4, 0, 1.0, (999, 256, 64, 1, 128, 64, 1, 128, 64), 1, 0), 6, 16, 14, 15),
    "swa_bwd": ((P, P, P, P, P, P, None, P, P, P, 1, 8, 8, 4, 2, 64, 4, 0, 1.0, (999, 256, 64, 1, 128, 64, 1, 128, 64), 1, 0),
                10, 20, 18, 19),
    "swa_decode": ((P, P, P, P, P, P, P, 2, 10, 4, 2, 64, 8, 2, 1.0, (256, 64, 128, 64, 128, 64), 1, 0), 7, 16, 14, 15),
    "scan_fwd": ((P, P, P, None, P, P, None, 1, 4, 8, 1, 0), 7, 10, None, None),
    "scan_bwd": ((P, P, P, P, P, None, P, P, P, None, 1, 4, 8, 1, 0), 10, 13, None, None),
    "scan_step": ((P, P, P, P, P, 1, 8, 1, 0), 5, 7, None, None),
    "block_norm_fwd": ((P, P, None, P, P, P, 1e-6, P, P, 4, 64, 0, 0), 10, 11, 6, None),
    "block_norm_bwd": ((P, P, None, P, P, P, 1e-6, P, P, P, P, None, P, P, P, 4, 64, 0, 0), 16, 17, 6, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_both_ways_of_calling_answer_alike(name):
    """The module and ctypes: every call here is refused by the library's first checks, or by the way itself."""
    args, size, dtype, real, strides = CALLS[name]
    wrong = [(0, None, g.GDN2_ERR_NULL), (0, MIS, g.GDN2_ERR_ALIGN), (size, -1, g.GDN2_ERR_SHAPE), (dtype, 9, g.GDN2_ERR_DTYPE),
             (size, 2 ** 31, OverflowError), (size, -2 ** 31 - 1, OverflowError)]
    if real is not None:
        wrong += [(real, -1.0, g.GDN2_ERR_SHAPE), (real, float("nan"), g.GDN2_ERR_SHAPE)]
    if strides is not None:
        wrong += [(strides, (*args[strides][:-1], 63), g.GDN2_ERR_SHAPE), (strides, (*args[strides][:-1], 68), g.GDN2_ERR_ALIGN)]
    for at, value, expected in wrong:
        for calls in (g._native(), g._Ctypes(g.lib())):
            a = (*args[:at], value, *args[at + 1:])
            if isinstance(expected, int):
                assert getattr(calls, name)(*a) == expected, (at, value)
            else:
                with pytest.raises(expected):
                    getattr(calls, name)(*a)


@pytest.mark.gpu
def test_calls_through_ctypes_give_the_same_results(monkeypatch):
    import torch
    gen = torch.Generator("cuda").manual_seed(1)
    f = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = f(2, 100, 8, 64).bfloat16()
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    t, w, vec = f(2, 100, 64), f(2, 100, 64), f(64).abs()
    kc, vc = f(2, 40, 2, 64).bfloat16(), f(2, 40, 2, 64).bfloat16()
    pos = torch.tensor([7, 90], dtype=torch.int32, device="cuda")

    def calls():
        o, lse = g.gdn2_swa_fwd(q, k, v, window=30, sinks=2)
        y, h, ckpt = g.gdn2_scan_fwd(t, w, -t.abs(), want_ckpt=True)
        state = h.clone()
        return [o, lse, *g.gdn2_swa_bwd(q, k, v, o, lse, o, window=30, sinks=2).values(), y, h, ckpt,
                g.gdn2_swa_decode(q[:, 0], k[:, 0], v[:, 0], kc, vc, pos, window=30, sinks=2), kc.clone(),
                *g.gdn2_scan_bwd(t, w, -t.abs(), ckpt, y, h).values(), g.gdn2_scan_step(t[:, 0].contiguous(), h, -h.abs(), state), state,
                *g.gdn2_block_norm_fwd(t, w, None, vec, vec, vec), *(n for n in g.gdn2_block_norm_bwd(t, w, w, vec, vec, vec, t, w).values())]

    ref = calls()
    assert not isinstance(g._native(), g._Ctypes)
    monkeypatch.setattr(g, "_caller", g._Ctypes(g.lib()))
    assert all(torch.equal(a, b) for a, b in zip(ref, calls(), strict=True))
