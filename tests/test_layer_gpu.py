"""GPU tests of the layer around the recurrences (selective scan, short convolution with a bias and its
backward, residual norms) against the fp64 oracle on the exact bits the GPU consumed.

Tolerances. A bf16 output is within half a step of the fp32 value (eps / 2 = 2^-8 relative). The fp32
value of a sum is held to its magnitude M, the same sum over absolute values: a chain of L recurrence
steps multiplies at most L decays, each an exponential good to 2^-22 of an argument good to 2^-23
(products delta * A, A log2 e: their relative error counts times the argument, at most 1 / e of the
decay itself), and rounds each product and sum to 2^-24; so a contribution that went through L steps is
within L (2^-22 + 2^-23 + 2^-23) = L 2^-21 of itself, and the 64 operations before and after the chain
(softplus, gates, read-out sums over at most 128 states) add at most 64 2^-21. Gradients run through two
such chains and one more sum over tokens or channels (fp32, relative error at most its depth, 2^-24 a
step, less than the chain's).
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_125_b200 as kda
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    kda.load_library()


def host(v):
    return None if v is None else v.detach().to("cpu", torch.float64).numpy()


def cu_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


def within(got, ref, mag, chain, what=""):
    """got (a tensor) within the rounding of its type and chain * 2^-21 of the magnitude."""
    g = host(got)
    assert np.isfinite(g).all(), what
    half = torch.finfo(got.dtype).eps / 2
    bound = half * np.abs(ref) + (1 + half) * chain * 2.0 ** -21 * mag + 1e-30
    over = np.abs(g - ref) / bound
    assert g.size == 0 or over.max() <= 1, "%s: %.3g times the bound" % (what, over.max())


def randn(*shape, seed=0, std=1.0, mean=0.0, dtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1009 + sum(shape) + 31 * len(shape))
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


# ------------------------------------------------------------- selective scan ----

def ssm_case(lengths, ch, n, groups=1, dtype=F32, gate=True, start=True, skip=True, bias=True, soft=True, seed=0,
             cu=True):
    T, N = sum(lengths), len(lengths)
    # steps of about 0.02 to 1, decay rates 0.3 to 3
    return dict(x=randn(T, ch, seed=seed + 1, dtype=dtype),
                dt=randn(T, ch, seed=seed + 2, mean=-1.5 if soft else 0.0, dtype=dtype) if soft
                else randn(T, ch, seed=seed + 2, dtype=dtype).abs() * 0.3,
                B=randn(T, groups, n, seed=seed + 3, dtype=dtype), C=randn(T, groups, n, seed=seed + 4, dtype=dtype),
                A=-torch.exp(randn(ch, n, seed=seed + 5, std=0.5)), S0=randn(N, ch, n, seed=seed + 6) if start else None,
                cu=cu_of(lengths) if cu else None, D=randn(ch, seed=seed + 7) if skip else None,
                dt_bias=randn(ch, seed=seed + 8, std=0.3) if bias else None,
                z=randn(T, ch, seed=seed + 9, dtype=dtype) if gate else None, soft=soft)


def ssm_run(k, **kw):
    return kda.kda_ssm_prefill(k["x"], k["dt"], k["B"], k["C"], k["A"], k["S0"], k["cu"], D=k["D"],
                               dt_bias=k["dt_bias"], z=k["z"], softplus=k["soft"], **kw)


def ssm_host(k):
    return {n: (v if n == "soft" else v.cpu().numpy() if n == "cu" and v is not None else host(v)) for n, v in k.items()}


def ssm_magnitude(h):
    """The scan over absolute values: what its rounding errors are measured by. (Without softplus a step may be
    negative: the sign goes into x, so that delta x is positive.)"""
    a = {n: (np.abs(v) if n in ("x", "B", "C", "S0", "D", "z") and v is not None else v) for n, v in h.items()}
    raw = h["dt"] + (0 if h["dt_bias"] is None else h["dt_bias"])
    sign = 1.0 if h["soft"] else np.sign(raw)
    y, S = L.ssm(**{**a, "x": a["x"] * sign, "D": None, "z": None})
    if h["D"] is not None:
        y = y + a["D"] * a["x"]
    if h["z"] is not None:
        y = y * np.abs(h["z"] * L.sigmoid(h["z"]))
    return y, S


def ssm_check(k, y, S_T, lengths, what=""):
    h = ssm_host(k)
    y_ref, S_ref = L.ssm(**h)
    y_mag, S_mag = ssm_magnitude(h)
    chain = max(lengths + [0]) + 64
    # negative steps (no softplus) grow a state without bound: channels that come near fp32's largest value are left out
    ok = (y_mag.max(0, initial=0) < 2.0 ** 100) & (S_mag.max((0, 2)) < 2.0 ** 100)
    assert ok.any()
    pick = torch.from_numpy(np.flatnonzero(ok)).to(DEV)
    within(y[:, pick], y_ref[:, ok], y_mag[:, ok], chain, what + " y")
    within(S_T[:, pick], S_ref[:, ok], S_mag[:, ok], chain, what + " S_T")


def nan_like(t):
    return torch.full_like(t, float("nan"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[1], [127], [128], [129], [300], [0, 5, 1, 0, 130, 128, 127, 0], [2] * 70 + [3, 0, 1]])
def test_ssm_prefill_lengths(lengths, dtype):
    k = ssm_case(lengths, 40, 16, dtype=dtype, seed=len(lengths))
    y, S_T = ssm_run(k, y=nan_like(k["x"]), S_T=torch.full((len(lengths), 40, 16), float("nan"), device=DEV))
    ssm_check(k, y, S_T, lengths)
    for s, m in enumerate(lengths):
        if m == 0:
            assert torch.equal(S_T[s], k["S0"][s])


@pytest.mark.parametrize("ch,n,groups", [(8, 8, 1), (16, 32, 2), (24, 64, 1), (48, 128, 2), (8 * 5 * 3, 16, 5), (4096, 16, 1),
                                         (2400, 8, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_prefill_shapes(ch, n, groups, dtype):
    lengths = [70, 3, 66]
    k = ssm_case(lengths, ch, n, groups, dtype, seed=n)
    y, S_T = ssm_run(k)
    ssm_check(k, y, S_T, lengths)


@pytest.mark.parametrize("gate,start,skip,bias,soft", [(0, 0, 0, 0, 0), (1, 0, 1, 0, 1), (0, 1, 0, 1, 0), (1, 1, 1, 1, 0)])
def test_ssm_prefill_options(gate, start, skip, bias, soft):
    lengths = [200, 57]
    k = ssm_case(lengths, 32, 16, 2, BF16, bool(gate), bool(start), bool(skip), bool(bias), bool(soft), seed=3)
    y, S_T = ssm_run(k)
    ssm_check(k, y, S_T, lengths)


def test_ssm_prefill_one_sequence_without_offsets():
    k = ssm_case([333], 64, 16, dtype=BF16, seed=5)
    a = ssm_run(k)
    b = ssm_run(dict(k, cu=None))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_ssm_prefill_state_in_place_and_continuation():
    """S_T may be S0; a prompt cut anywhere and continued from its state equals the whole."""
    k = ssm_case([300], 64, 16, dtype=F32, seed=6)
    y, S_T = ssm_run(k)
    for cut in (1, 128, 200):
        S = k["S0"].clone()
        parts = []
        for a, b in ((0, cut), (cut, 300)):
            p = dict(k, S0=S, cu=None, **{m: k[m][a:b].clone() for m in ("x", "dt", "B", "C", "z")})
            parts.append(ssm_run(p, S_T=S)[0])
        ssm_check(k, torch.cat(parts), S, [300], "cut at %d" % cut)


def test_ssm_prefill_leaves_rows_behind_the_last_sequence():
    k = ssm_case([100, 50], 32, 16, dtype=BF16, seed=8)
    pad = {m: torch.cat([k[m], torch.full_like(k[m][:90], float("nan"))]) for m in ("x", "dt", "B", "C", "z")}
    y = torch.full_like(pad["x"], 7.0)
    out, S_T = ssm_run(dict(k, **pad), y=y)
    assert (y[150:] == 7.0).all()
    ssm_check(k, out[:150], S_T, [100, 50])


def test_ssm_prefill_extreme_decays_and_gates():
    """Steps so large that every decay is 0, steps of 0, gates that saturate: finite and right."""
    k = ssm_case([64], 16, 16, dtype=F32, soft=False, bias=False, seed=9)
    k["dt"][::3] = 200.0
    k["dt"][1::3] = 0.0
    k["z"][::2] = 80.0
    k["z"][1::4] = -120.0
    y, S_T = ssm_run(k)
    ssm_check(k, y, S_T, [64])


def test_ssm_prefill_stream_and_graph():
    k = ssm_case([200, 33], 64, 16, dtype=BF16, seed=10)
    y, S_T = ssm_run(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, S2 = ssm_run(k, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3, S3 = ssm_run(k)
    for seed in (11, 12):
        new = ssm_case([200, 33], 64, 16, dtype=BF16, seed=seed)
        for m in ("x", "dt", "B", "C", "z", "S0"):
            k[m].copy_(new[m])
        g.replay()
        y4, S4 = ssm_run(k)
        assert torch.equal(y3, y4) and torch.equal(S3, S4)


def test_ssm_tile_states():
    lengths = [300, 0, 84, 129]
    k = ssm_case(lengths, 24, 16, dtype=F32, seed=13)
    _, _, tiles = ssm_run(k, save_states=True)
    h = ssm_host(k)
    ref = L.ssm_states(**h)[::128]
    mag = L.ssm_states(**{n: (np.abs(v) if n in ("x", "B", "S0") else v) for n, v in h.items()})[::128]
    starts = [i for i, t in enumerate(range(0, sum(lengths), 128)) if t in set(h["cu"][:-1])]
    assert starts == [0, 3]  # token 384 is a sequence's first: its entry is unspecified
    keep = [i for i in range(len(ref)) if i not in starts]
    within(tiles[keep], ref[keep], mag[keep], 364)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,ch,n,groups", [(1, 8, 8, 1), (3, 40, 16, 1), (5, 48, 32, 2), (2, 24, 64, 3), (4, 8, 128, 1),
                                           (70, 4096, 16, 1), (600, 72, 8, 1)])
def test_ssm_step(N, ch, n, groups, dtype):
    k = ssm_case([1] * N, ch, n, groups, dtype, seed=N)
    S = k["S0"].clone()
    y = kda.kda_ssm_step(k["x"], k["dt"], k["B"], k["C"], k["A"], S, D=k["D"], dt_bias=k["dt_bias"], z=k["z"],
                         y=nan_like(k["x"]))
    ssm_check(k, y, S, [1])
    # without the optional inputs
    S = k["S0"].clone()
    y = kda.kda_ssm_step(k["x"], k["dt"].abs(), k["B"], k["C"], k["A"], S, softplus=False)
    k2 = dict(k, dt=k["dt"].abs(), D=None, dt_bias=None, z=None, soft=False)
    ssm_check(k2, y, S, [1])


def test_ssm_steps_continue_a_prompt():
    k = ssm_case([60], 64, 16, dtype=F32, seed=14)
    y, S_T = ssm_run(k)
    part = dict(k, cu=None, **{m: k[m][:50].clone() for m in ("x", "dt", "B", "C", "z")})
    ys, S = ssm_run(part)
    out = [ys]
    for t in range(50, 60):
        one = {m: k[m][t:t + 1].clone() for m in ("x", "dt", "B", "C", "z")}
        out.append(kda.kda_ssm_step(one["x"], one["dt"], one["B"], one["C"], k["A"], S, D=k["D"], dt_bias=k["dt_bias"],
                                    z=one["z"]))
    ssm_check(k, torch.cat(out), S, [60])


@pytest.mark.parametrize("lengths,ch,n,groups,dtype", [
    ([2100], 40, 16, 1, BF16),           # nine segments of 256 tokens, the last one short
    ([700, 0, 1300, 256, 3], 24, 8, 1, F32), ([513], 48, 32, 2, F32), ([1030, 600], 16, 64, 1, BF16), ([800], 8, 128, 1, F32),
    ([2048, 1, 512], 1024, 16, 2, BF16),  # two lanes to a channel
])
def test_ssm_prefill_segments(lengths, ch, n, groups, dtype):
    """Long sequences cut into segments: outputs, final states and tile states."""
    assert kda.load_library().kda_ssm_prefill_launches(len(lengths), sum(lengths), ch, n, groups) > 1
    k = ssm_case(lengths, ch, n, groups, dtype, seed=n + 1)
    nbytes = kda.load_library().kda_ssm_prefill_workspace_size(len(lengths), sum(lengths), ch, n, groups)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN where nothing is written
    y, S_T, tiles = ssm_run(k, save_states=True, workspace=ws)
    ssm_check(k, y, S_T, lengths)
    h = ssm_host(k)
    ref = L.ssm_states(**h)[::128]
    mag = L.ssm_states(**{m: (np.abs(v) if m in ("x", "B", "S0") else v) for m, v in h.items()})[::128]
    keep = [i for i, t in enumerate(range(0, sum(lengths), 128)) if t not in set(h["cu"][:-1])]
    within(tiles[keep], ref[keep], mag[keep], max(lengths) + 64)
    again = ssm_run(k, workspace=ws)
    assert torch.equal(y, again[0]) and torch.equal(S_T, again[1])


# ------------------------------------------------ selective scan, gradients ----

def ssm_grad_run(k, dy, dS_T, **kw):
    y, S_T, tiles = ssm_run(k, save_states=True)
    g = kda.kda_ssm_backward(k["x"], k["dt"], k["B"], k["C"], k["A"], dy, tiles, dS_T, k["S0"], k["cu"], D=k["D"],
                             dt_bias=k["dt_bias"], z=k["z"], softplus=k["soft"], **kw)
    return g


def ssm_grad_check(k, dy, dS_T, g, lengths, what=""):
    """Each gradient against the formula's, by the magnitude of the terms it is a sum of: the backward over
    absolute values (steps and decay rates keep their signs, their parts of a sum counted positive)."""
    h = ssm_host(k)
    ref = L.ssm_backward(dy=host(dy), dS_T=host(dS_T), **h)
    mag = ssm_grad_magnitude(h, host(dy), host(dS_T))
    chain = 2 * max(lengths + [0]) + 128
    for n in ("dx", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "dS0"):
        got = getattr(g, n)
        if got is not None:
            within(got, ref[n], mag[n], chain, what + " " + n)


def ssm_grad_magnitude(h, dy, dS_T):
    """The sums of L.ssm_backward with every term taken positive."""
    a = {n: np.abs(v) if v is not None and n not in ("cu", "soft", "dt", "dt_bias", "A") else v for n, v in h.items()}
    groups, per = h["B"].shape[1], h["x"].shape[1] // h["B"].shape[1]
    raw = h["dt"] + (0 if h["dt_bias"] is None else h["dt_bias"])
    delta = L.softplus(raw) if h["soft"] else np.abs(raw)
    T, ch, n = h["x"].shape + (h["A"].shape[1],)
    cu = [0, T] if h["cu"] is None else h["cu"]
    Bd, Cd = np.repeat(a["B"], per, 1), np.repeat(a["C"], per, 1)
    D = np.zeros(ch) if a["D"] is None else a["D"]
    gate = np.ones((T, ch)) if h["z"] is None else np.abs(h["z"] * L.sigmoid(h["z"]))
    m = {k: np.zeros(s) for k, s in dict(dx=(T, ch), ddt=(T, ch), dz=(T, ch), dA=(ch, n), dD=ch, ddt_bias=ch,
                                         dS0=(len(cu) - 1, ch, n), dB=(T, ch, n), dC=(T, ch, n)).items()}
    sig = L.sigmoid(raw) if h["soft"] else np.ones_like(raw)
    for s in range(len(cu) - 1):
        hs = [np.zeros((ch, n)) if a["S0"] is None else a["S0"][s]]
        sign = 1.0 if h["soft"] else np.sign(raw)
        for t in range(cu[s], cu[s + 1]):
            hs.append(np.exp((delta[t] * (sign if np.isscalar(sign) else sign[t]))[:, None] * h["A"]) * hs[-1]
                      + (delta[t] * a["x"][t])[:, None] * Bd[t])
        G = np.zeros((ch, n)) if dS_T is None else np.abs(dS_T[s])
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            st, before = hs[t - cu[s] + 1], hs[t - cu[s]]
            e = np.abs(dy[t]) * gate[t]
            if h["z"] is not None:
                m["dz"][t] = np.abs(dy[t]) * ((Cd[t] * st).sum(-1) + D * a["x"][t]) * (1 + a["z"][t])
            G = G + Cd[t] * e[:, None]
            dec = np.exp((delta[t] * (sign if np.isscalar(sign) else sign[t]))[:, None] * h["A"])
            m["dC"][t], m["dB"][t] = st * e[:, None], G * (delta[t] * a["x"][t])[:, None]
            gb, ga = (G * Bd[t]).sum(-1), G * before * dec
            m["dx"][t] = delta[t] * gb + D * e
            m["dD"] += e * a["x"][t]
            m["dA"] += ga * delta[t][:, None]
            m["ddt"][t] = ((ga * np.abs(h["A"])).sum(-1) + gb * a["x"][t]) * sig[t]
            G = G * dec
        m["dS0"][s] = G
    m["ddt_bias"] = m["ddt"].sum(0)
    m["dB"], m["dC"] = (m[k].reshape(T, groups, per, n).sum(2) for k in ("dB", "dC"))
    return m


def ssm_grad_case(lengths, ch, n, groups=1, dtype=F32, seed=0, dS=True, **kw):
    k = ssm_case(lengths, ch, n, groups, dtype, seed=seed, **kw)
    return k, randn(sum(lengths), ch, seed=seed + 20, dtype=dtype), randn(len(lengths), ch, n, seed=seed + 21) if dS else None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[1], [7], [8], [127], [128], [129], [300], [0, 5, 1, 0, 130, 128, 127, 0], [2] * 30 + [3, 0, 1]])
def test_ssm_backward_lengths(lengths, dtype):
    k, dy, dS = ssm_grad_case(lengths, 24, 16, dtype=dtype, seed=len(lengths))
    ssm_grad_check(k, dy, dS, ssm_grad_run(k, dy, dS), lengths)


@pytest.mark.parametrize("ch,n,groups", [(8, 8, 1), (96, 8, 3), (16, 32, 2), (40, 32, 1), (24, 64, 1), (48, 128, 2), (8 * 5 * 3, 16, 5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_backward_shapes(ch, n, groups, dtype):
    lengths = [70, 3, 66]
    k, dy, dS = ssm_grad_case(lengths, ch, n, groups, dtype, seed=n)
    ssm_grad_check(k, dy, dS, ssm_grad_run(k, dy, dS), lengths)


@pytest.mark.parametrize("gate,start,skip,bias,soft,dS", [(0, 0, 0, 0, 1, 0), (1, 0, 1, 0, 1, 1), (0, 1, 0, 1, 1, 0), (1, 1, 1, 0, 0, 1)])
def test_ssm_backward_options(gate, start, skip, bias, soft, dS):
    lengths = [200, 57]
    k, dy, d = ssm_grad_case(lengths, 32, 16, 2, BF16, seed=3, dS=bool(dS), gate=bool(gate), start=bool(start),
                             skip=bool(skip), bias=bool(bias), soft=bool(soft))
    g = ssm_grad_run(k, dy, d)
    assert (g.dz is None, g.dS0 is None, g.dD is None, g.ddt_bias is None) == (not gate, not start, not skip, not bias)
    ssm_grad_check(k, dy, d, g, lengths)


def test_ssm_backward_long_sequences():
    """Tile states of a forward that cut its sequences into segments."""
    lengths = [1100, 0, 900]
    k, dy, dS = ssm_grad_case(lengths, 16, 16, dtype=F32, seed=40)
    assert kda.load_library().kda_ssm_prefill_launches(3, 2000, 16, 16, 1) > 1
    ssm_grad_check(k, dy, dS, ssm_grad_run(k, dy, dS), lengths)


def test_ssm_backward_same_bits_and_rows_behind():
    lengths = [150, 90]
    k, dy, dS = ssm_grad_case(lengths, 64, 16, dtype=BF16, seed=41)
    a, b = ssm_grad_run(k, dy, dS), ssm_grad_run(k, dy, dS)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    nan = float("nan")
    pad = {m: torch.cat([k[m], torch.full_like(k[m][:70], nan)]) for m in ("x", "dt", "B", "C", "z")}
    c = ssm_grad_run(dict(k, **pad), torch.cat([dy, torch.full_like(dy[:70], nan)]), dS)
    for n, u, v in zip(a._fields, a, c):
        assert torch.equal(u, v[:240] if n in ("dx", "ddt", "dz", "dB", "dC") else v), n


def test_ssm_backward_differences():
    """The gradient of a step along a direction against the difference of two forward runs."""
    k, dy, dS = ssm_grad_case([90, 40], 16, 16, dtype=F32, seed=42)
    g = ssm_grad_run(k, dy, dS)

    def loss(c):
        y, S = ssm_run(c)
        return float((y.double() * dy).sum() + (S.double() * dS).sum())

    for n, name in (("x", "dx"), ("dt", "ddt"), ("B", "dB"), ("C", "dC"), ("z", "dz"), ("A", "dA"), ("D", "dD"), ("dt_bias", "ddt_bias"), ("S0", "dS0")):
        v = randn(*k[n].shape, seed=50)
        h = 2.0 ** -8
        up, down = loss(dict(k, **{n: k[n] + h * v})), loss(dict(k, **{n: k[n] - h * v}))
        want = float((getattr(g, name).double() * v).sum())
        # truncation h^2 (third derivatives of O(1) per unit direction, grown by the direction's length), rounding of
        # the forward outputs 2^-20 of their size over 2 h
        scale = float(getattr(g, name).double().norm() * v.double().norm()) + 1.0
        assert abs((up - down) / (2 * h) - want) <= 3e-2 * scale, n


def test_ssm_backward_graph():
    """Captured together with its forward and replayed on other inputs."""
    k, dy, dS = ssm_grad_case([200, 33], 64, 16, dtype=BF16, seed=43)
    ssm_grad_run(k, dy, dS)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = ssm_grad_run(k, dy, dS)
    new, dy2, dS2 = ssm_grad_case([200, 33], 64, 16, dtype=BF16, seed=44)
    for m in ("x", "dt", "B", "C", "z", "S0"):
        k[m].copy_(new[m])
    dy.copy_(dy2)
    gr.replay()
    ref = ssm_grad_run(k, dy, dS)
    for u, v in zip(out, ref):
        assert torch.equal(u, v)
