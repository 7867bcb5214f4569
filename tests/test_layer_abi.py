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
    (dict(T=1 << 31), UNSUPPORTED), (dict(S0=A + 4), MISALIGNED), (dict(S_T=A + 8), MISALIGNED),
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
    assert f(0, 64, 16) == 0 and f(1, 64, 16) == f(128, 64, 16) == 64 * 16 * 4 and f(129, 64, 16) == 2 * f(1, 64, 16)
    assert f(1 << 20, 8192, 128) == (1 << 13) * 8192 * 128 * 4 and f(-1, 64, 16) == 0 and f(5, 0, 16) == 0


def test_ssm_binding_checks():
    """The binding refuses what the C ABI cannot see: devices, dtypes, shapes."""
    x = torch.zeros(4, 16)
    B, a = torch.zeros(4, 1, 8), torch.zeros(16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_prefill(x, x, B, B, a)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_step(x, x, B, B, a, torch.zeros(4, 16, 8))
