"""Host-side refusals of the layer's entry points: fake (never dereferenced) addresses, so only without a GPU."""
import ctypes

import pytest
import torch

import gated_delta_rule_125_b200 as kda
from gated_delta_rule_125_b200 import build as kbuild

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer calls only without a GPU")
A = 0x10000
INVALID, UNSUPPORTED, MISALIGNED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


SSM = dict(x=A, dt=A, B=A, C=A, z=None, ch=64, n=16, g=1, A=A, D=None, bias=None, N=1, dtype=1, flags=kda.KDA_FLAG_SOFTPLUS)
SSM_BAD = [
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(B=None), INVALID), (dict(C=None), INVALID),
    (dict(A=None), INVALID), (dict(y=None), INVALID), (dict(dtype=2), INVALID), (dict(flags=0x10), INVALID),
    (dict(flags=kda.KDA_FLAG_EXACT), INVALID), (dict(ch=0), INVALID), (dict(g=0), INVALID), (dict(n=0), INVALID),
    (dict(ch=60), UNSUPPORTED), (dict(ch=64, g=3), UNSUPPORTED), (dict(ch=48, g=4), UNSUPPORTED),
    (dict(n=12), UNSUPPORTED), (dict(n=256), UNSUPPORTED),
    (dict(x=A + 8), MISALIGNED), (dict(B=A + 4), MISALIGNED), (dict(z=A + 2), MISALIGNED), (dict(A=A + 4), MISALIGNED),
    (dict(D=A + 2), MISALIGNED), (dict(bias=A + 1), MISALIGNED), (dict(y=A + 8), MISALIGNED),
]


def ssm_struct(a):
    return ctypes.byref(kda.Ssm(a["ch"], a["n"], a["g"], a["A"], a["D"], a["bias"]))


def ssm_prefill(lib, **over):
    a = dict(SSM, S0=None, cu=None, T=4096, y=A, S_T=A, tiles=None, ws=A, wsb=1 << 40)
    a.update(over)
    return lib.kda_ssm_prefill(a["x"], a["dt"], a["B"], a["C"], a["z"], ssm_struct(a), a["S0"], a["cu"], a["N"], a["T"],
                               a["dtype"], a["flags"], a["y"], a["S_T"], a["tiles"], a["ws"], a["wsb"], None)


def ssm_step(lib, **over):
    a = dict(SSM, S=A, y=A)
    a.update(over)
    return lib.kda_ssm_step(a["x"], a["dt"], a["B"], a["C"], a["z"], ssm_struct(a), a["S"], a["N"], a["dtype"],
                            a["flags"], a["y"], None)


@no_gpu
@pytest.mark.parametrize("over,code", SSM_BAD + [
    (dict(N=0), INVALID), (dict(N=3), INVALID), (dict(N=65536, cu=A), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, A=None), INVALID), (dict(S0=A + 4), MISALIGNED), (dict(S_T=A + 8), MISALIGNED),
    (dict(cu=A + 4, N=2), MISALIGNED), (dict(tiles=A + 4), MISALIGNED),
    (dict(ws=None), kda.KDA_ERR_WORKSPACE), (dict(wsb=64), kda.KDA_ERR_WORKSPACE), (dict(ws=A + 8), MISALIGNED)])
def test_ssm_prefill_rejects(lib, over, code):
    assert ssm_prefill(lib, **over) == code


@no_gpu
@pytest.mark.parametrize("over,code", SSM_BAD + [(dict(N=0), INVALID), (dict(S=None), INVALID), (dict(S=A + 8), MISALIGNED)])
def test_ssm_step_rejects(lib, over, code):
    assert ssm_step(lib, **over) == code


def test_ssm_tile_states_size(lib):
    f = lib.kda_ssm_tile_states_size
    assert f(1, 0, 64, 16) == f(1, 127, 64, 16) == 64 * 16 * 4 and f(1, 128, 64, 16) == 2 * 64 * 16 * 4 == f(2, 1, 64, 16)
    assert f(1, 1 << 20, 8192, 128) == ((1 << 13) + 1) * 8192 * 128 * 4
    assert f(0, 1, 64, 16) == 0 and f(1, -1, 64, 16) == 0 and f(1, 5, 0, 16) == 0


def test_ssm_binding_checks():
    """The binding refuses what the C ABI cannot see: devices, dtypes, shapes."""
    x = torch.zeros(4, 16)
    B, a = torch.zeros(4, 1, 8), torch.zeros(16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_prefill(x, x, B, B, a)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_step(x, x, B, B, a, torch.zeros(4, 16, 8))


def ssm_backward(lib, **over):
    a = dict(SSM, S0=None, cu=None, T=256, tiles=A, dy=A, dS=None, dx=A, ddt=A, dB=A, dC=A, dz=None, dA=A, dD=None,
             ddt_bias=None, dS0=None, ws=A, wsb=1 << 40)
    a.update(over)
    g = kda.SsmGrads(*(a[n] for n, _ in kda.SsmGrads._fields_))
    return lib.kda_ssm_backward(a["x"], a["dt"], a["B"], a["C"], a["z"], ssm_struct(a), a["S0"], a["cu"], a["N"], a["T"],
                                a["dtype"], a["flags"], a["tiles"], a["dy"], a["dS"], ctypes.byref(g), a["ws"], a["wsb"], None)


@no_gpu
@pytest.mark.parametrize("over,code", [(o, c) for o, c in SSM_BAD if "y" not in o and o != dict(z=A + 2)] + [
    (dict(z=A + 2, dz=A), MISALIGNED), (dict(z=A), INVALID), (dict(dz=A), INVALID), (dict(tiles=None), INVALID),
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dC=None), INVALID), (dict(dA=None), INVALID),
    (dict(N=2), INVALID), (dict(T=-1), INVALID), (dict(dS=A + 4), MISALIGNED), (dict(dS0=A + 8), MISALIGNED),
    (dict(dD=A + 2), MISALIGNED), (dict(tiles=A + 4), MISALIGNED), (dict(ws=None), kda.KDA_ERR_WORKSPACE),
    (dict(wsb=1024), kda.KDA_ERR_WORKSPACE), (dict(ws=A + 8), MISALIGNED)])
def test_ssm_backward_rejects(lib, over, code):
    assert ssm_backward(lib, **over) == code


@no_gpu
def test_ssm_null_structs(lib):
    assert lib.kda_ssm_step(A, A, A, A, None, None, A, 1, 1, 0, A, None) == INVALID
    assert lib.kda_ssm_backward(A, A, A, A, None, ssm_struct(SSM), None, None, 1, 1, 1, 0, A, A, None, None, A, 1 << 40, None) == INVALID


def test_ssm_queries(lib):
    w, n = lib.kda_ssm_prefill_workspace_size, lib.kda_ssm_prefill_launches
    assert n(1, 128, 4096, 16, 1) == 1 and w(1, 128, 4096, 16, 1) == 0
    assert n(1, 8192, 512, 16, 1) == 3 and w(1, 8192, 512, 16, 1) > 0
    assert n(1, 8192, 4096, 16, 1) == 1 and w(1, 8192, 4096, 16, 1) == 0  # enough channels: uncut
    assert n(0, 128, 4096, 16, 1) == -1 and n(1, 128, 4096, 12, 1) == -1 and n(1, 128, 12, 16, 1) == -1
    b = lib.kda_ssm_backward_workspace_size
    assert 0 < b(1, 128, 64, 16, 1) < b(1, 256, 64, 16, 1) < b(1, 256, 128, 16, 1)
    assert b(1, 0, 64, 16, 1) == 64 * 18 * 4 and b(1, -1, 64, 16, 1) == 0


CONV = dict(x=A, y=A + (1 << 24), width=4, w=A, sin=None, sout=None, bias=None, cu=None, N=1, T=64, C=256, dtype=1)
CONV_BAD = [(dict(width=0), UNSUPPORTED), (dict(width=9), UNSUPPORTED), (dict(C=12), INVALID), (dict(C=0), INVALID),
            (dict(dtype=3), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID), (dict(x=A + 8), MISALIGNED),
            (dict(w=A + 2), MISALIGNED), (dict(bias=A + 2), MISALIGNED), (dict(C=(1 << 20) + 8), UNSUPPORTED)]


def conv_struct(a):
    return ctypes.byref(kda.ShortConv(a["width"], a["w"], a["sin"], a["sout"]))


@no_gpu
@pytest.mark.parametrize("over,code", CONV_BAD + [(dict(y=A + 512), INVALID), (dict(N=2), INVALID), (dict(T=-1), INVALID),
                                                  (dict(sin=A + 4), MISALIGNED), (dict(y=None), INVALID)])
def test_conv_ex_rejects(lib, over, code):
    a = dict(CONV, **over)
    assert lib.kda_short_conv_swish_ex(a["x"], a["y"], conv_struct(a), a["bias"], a["cu"], a["N"], a["T"], a["C"],
                                       a["dtype"], None) == code


@no_gpu
@pytest.mark.parametrize("over,code", CONV_BAD + [(dict(T=0), INVALID), (dict(sout=None), INVALID), (dict(sout=A + 8), MISALIGNED),
                                                  (dict(y=A + 64), INVALID)])
def test_conv_step_rejects(lib, over, code):
    a = dict(CONV, sout=A)
    a.update(over)
    assert lib.kda_short_conv_step(a["x"], a["y"], conv_struct(a), a["bias"], a["T"], a["C"], a["dtype"], None) == code


@no_gpu
@pytest.mark.parametrize("over,code", CONV_BAD + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dyt=7), INVALID),
    (dict(dtype=0, dyt=1), UNSUPPORTED), (dict(N=2), INVALID), (dict(ws=None), kda.KDA_ERR_WORKSPACE),
    (dict(wsb=64), kda.KDA_ERR_WORKSPACE), (dict(ws=A + 4), MISALIGNED), (dict(ds=A + 4), MISALIGNED), (dict(dy=A + 8), MISALIGNED)])
def test_conv_backward_rejects(lib, over, code):
    a = dict(CONV, dy=A, dyt=0, dx=A, dw=A, db=None, ds=None, ws=A, wsb=1 << 30)
    a.update(over)
    assert lib.kda_short_conv_backward(a["x"], conv_struct(a), a["bias"], a["cu"], a["N"], a["T"], a["C"], a["dtype"], a["dy"],
                                       a["dyt"], a["dx"], a["dw"], a["db"], a["ds"], a["ws"], a["wsb"], None) == code


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(x=A + 4096), dict(dy=A + 65536 - 16, x=A + (1 << 24)),
                                  dict(dx=A + 32768 - 16, dy=A + (1 << 24)), dict(dyt=0, dx=A + 65536 - 16, x=A + (1 << 24))])
def test_conv_backward_rejects_overlaps(lib, over):
    """dx (65536 bytes here) in the place of x (32768) or dy (32768, fp32: 65536): the rows around a run are read from there."""
    a = dict(x=A, dy=A, dyt=1, dx=A, w=A)
    a.update(over)
    c = ctypes.byref(kda.ShortConv(4, A, None, None))
    assert lib.kda_short_conv_backward(a["x"], c, None, None, 1, 64, 256, 1, a["dy"], a["dyt"], a["dx"], A, None, None, A, 1 << 30,
                                       None) == INVALID


@no_gpu
@pytest.mark.parametrize("x,y,state", [(A, A + 32768, A + 32768 - 16), (A, A + 32768, A + 65536 - 16), (A + 98304 - 16, A + (1 << 24), A)])
def test_conv_step_rejects_overlaps(lib, x, y, state):
    """x and y of 32768 bytes, the state of 98304."""
    c = ctypes.byref(kda.ShortConv(4, A, None, state))
    assert lib.kda_short_conv_step(x, y, c, None, 64, 256, 1, None) == INVALID


NORM = dict(y=A, r=A, gate=A, w_post=A, scale=A, w_pre=A, res_scale=1.0, eps=1e-6, rows=4, D=64, dtype=1, res_dtype=0)
NORM_BAD = [(dict(y=None), INVALID), (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(D=12), INVALID), (dict(eps=0.0), INVALID),
            (dict(eps=float("nan")), INVALID), (dict(dtype=4), INVALID), (dict(res_dtype=4), INVALID), (dict(D=8200), UNSUPPORTED),
            (dict(dtype=0, res_dtype=1), UNSUPPORTED), (dict(y=A + 8), MISALIGNED), (dict(gate=A + 2), MISALIGNED),
            (dict(w_pre=A + 4), MISALIGNED), (dict(scale=A + 4), MISALIGNED)]


def norm_struct(a):
    return ctypes.byref(kda.ResidualNorm(*(a[n] for n, _ in kda.ResidualNorm._fields_)))


@no_gpu
@pytest.mark.parametrize("over,code", NORM_BAD + [(dict(x=None), INVALID), (dict(w_pre=None), INVALID), (dict(out=None), INVALID),
                                                  (dict(out=A + 8), MISALIGNED)])
def test_residual_norm_rejects(lib, over, code):
    a = dict(NORM, x=A, out=A)
    a.update(over)
    assert lib.kda_residual_norm(norm_struct(a), a["x"], a["out"], None) == code


@no_gpu
@pytest.mark.parametrize("over,code", NORM_BAD + [
    (dict(dx=None), INVALID), (dict(w_pre=None), INVALID), (dict(dy=None), INVALID), (dict(dgate=None), INVALID),
    (dict(gate=None), INVALID), (dict(w_post=None), INVALID), (dict(scale=None), INVALID), (dict(dr=A + 4), MISALIGNED),
    (dict(dw=A + 4), MISALIGNED), (dict(ws=None), kda.KDA_ERR_WORKSPACE), (dict(wsb=64), kda.KDA_ERR_WORKSPACE)])
def test_residual_norm_backward_rejects(lib, over, code):
    a = dict(NORM, dx=A, dr_out=A, dy=A, dr=A, dgate=A, dw=A, ws=A, wsb=1 << 30)
    a.update(over)
    assert lib.kda_residual_norm_backward(norm_struct(a), a["dx"], a["dr_out"], a["dy"], a["dr"], a["dgate"], a["dw"], a["dw"],
                                          a["dw"], a["ws"], a["wsb"], None) == code


def test_norm_queries(lib):
    f = lib.kda_residual_norm_backward_workspace_size
    assert f(1, 64) == 3 * 64 * 4 and f(0, 64) > 0 and f(1, 8200) == 0 and f(-1, 64) == 0 and f(10, 4096) == 10 * 3 * 4096 * 4
    c = lib.kda_short_conv_backward_workspace_size
    assert c(0, 64, 4) == 0 and c(1, 64, 4) == 5 * 64 * 4 and c(10, 12, 4) == 0 and c(10, 64, 9) == 0
