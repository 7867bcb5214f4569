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


def tile_states_check(k, tiles, lengths):
    """The state before each 128 tokens of every sequence."""
    h = ssm_host(k)
    ref = L.ssm_states(**h)
    mag = L.ssm_states(**{n: (np.abs(v) if n in ("x", "B", "S0") else v) for n, v in h.items()})
    at = [(h["cu"][s] // 128 + s + j, h["cu"][s] + 128 * j) for s, m in enumerate(lengths) for j in range(-(-m // 128))]
    assert len(set(i for i, _ in at)) == len(at) and max(i for i, _ in at) < tiles.shape[0] == sum(lengths) // 128 + len(lengths)
    i, t = [list(v) for v in zip(*at)]
    within(tiles[i], ref[t], mag[t], max(lengths) + 64, "tile states")


def test_ssm_tile_states():
    lengths = [300, 0, 84, 129, 128, 1]
    k = ssm_case(lengths, 24, 16, dtype=F32, seed=13)
    _, _, tiles = ssm_run(k, save_states=True)
    tile_states_check(k, tiles, lengths)


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


def test_ssm_no_tokens():
    """Only empty sequences: S_T = S0 (or zeros), gradients of the states pass through, the others are 0."""
    k = ssm_case([0, 0, 0], 16, 8, dtype=BF16, seed=15)
    y, S_T, tiles = ssm_run(k, save_states=True)
    assert y.shape == (0, 16) and torch.equal(S_T, k["S0"])
    assert (ssm_run(dict(k, S0=None))[1] == 0).all()
    dS = randn(3, 16, 8, seed=16)
    g = kda.kda_ssm_backward(k["x"], k["dt"], k["B"], k["C"], k["A"], k["x"], tiles, dS, k["S0"], k["cu"], D=k["D"],
                             dt_bias=k["dt_bias"], z=k["z"])
    assert torch.equal(g.dS0, dS) and all((v == 0).all() for v in (g.dA, g.dD, g.ddt_bias))
    c = conv_case([0, 0], 16, 4, BF16, seed=17)
    last = torch.empty_like(c["state"])
    kda.kda_short_conv_swish(c["x"], c["w"], c["cu"], state_in=c["state"], state_out=last, bias=c["bias"])
    assert torch.equal(last, c["state"])
    d = kda.kda_short_conv_backward(c["x"], c["w"], c["x"].float(), c["cu"], bias=c["bias"], state_in=c["state"], want_dstate=True)
    assert all((v == 0).all() for v in d[1:])


def test_ssm_two_calls_at_once():
    """Two prompts on two streams, each with its own workspace, and a third one behind them."""
    a, b = ssm_case([3000], 64, 16, dtype=BF16, seed=18), ssm_case([2500, 700], 64, 16, dtype=BF16, seed=19)
    assert kda.load_library().kda_ssm_prefill_launches(1, 3000, 64, 16, 1) > 1
    ref = ssm_run(a), ssm_run(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = ssm_run(a, stream=streams[0]), ssm_run(b, stream=streams[1])
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for u, v in zip(ref, got):
            assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])


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
    ([2048, 1, 512], 256, 16, 2, BF16),
])
def test_ssm_prefill_segments(lengths, ch, n, groups, dtype):
    """Long sequences cut into segments: outputs, final states and tile states."""
    assert kda.load_library().kda_ssm_prefill_launches(len(lengths), sum(lengths), ch, n, groups) > 1
    k = ssm_case(lengths, ch, n, groups, dtype, seed=n + 1)
    nbytes = kda.load_library().kda_ssm_prefill_workspace_size(len(lengths), sum(lengths), ch, n, groups)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN where nothing is written
    y, S_T, tiles = ssm_run(k, save_states=True, workspace=ws)
    ssm_check(k, y, S_T, lengths)
    tile_states_check(k, tiles, lengths)
    # the final states over the initial ones, which the first segments read while the last ones write
    S = k["S0"].clone()
    again = ssm_run(dict(k, S0=S), S_T=S, workspace=ws)
    assert torch.equal(y, again[0]) and torch.equal(S_T, again[1])


def ssm_slow_case(lengths, ch, n, groups=1, dtype=F32, seed=0):
    """Steps so small that a state lasts for segments of 256 tokens (rate times steps of a segment: about 0.1 to 4), larger
    in some segments than in their neighbours, and initial states that stand out."""
    k = ssm_case(lengths, ch, n, groups, dtype, seed=seed)
    t = torch.arange(sum(lengths), device=DEV, dtype=F32).unsqueeze(1)
    k["dt"] = (randn(sum(lengths), ch, seed=seed + 2, std=0.5, mean=-6.0) + 0.7 * torch.sin(t * (2 * np.pi / 600))).to(dtype)
    k["S0"] = 8 * k["S0"]
    return k


def ssm_with_join(h, seg, decays):
    """The scan by segments of `seg` tokens whose join takes decays(steps of the segment, of the one before, A): y, S_T and
    the segments' first states with their first tokens."""
    delta = L.softplus(h["dt"] + h["dt_bias"])
    cuts, seqs = [], []
    for s, (b, e) in enumerate(zip(h["cu"][:-1], h["cu"][1:])):
        mine = list(range(b, e, seg)) or [b]
        cuts += mine
        seqs += [s] * len(mine)
    cuts.append(h["cu"][-1])
    first = [i == 0 or seqs[i - 1] != s for i, s in enumerate(seqs)]
    start = np.stack([h["S0"][s] if f else np.zeros_like(h["A"]) for s, f in zip(seqs, first)])
    ends = L.ssm(**{**h, "S0": start, "cu": np.array(cuts)})[1]
    for i in range(1, len(seqs)):
        if not first[i]:
            start[i] = ends[i - 1]
            if not first[i - 1]:
                steps = [delta[cuts[j]:cuts[j + 1]].sum(0)[:, None] for j in (i - 1, i - 2)]
                start[i] += decays(*steps, h["A"]) * start[i - 1]
    y, S_T = L.ssm(**{**h, "S0": start, "cu": np.array(cuts)})
    return y, S_T[[i for i in range(len(seqs)) if i + 1 == len(seqs) or first[i + 1]]], start, cuts


@pytest.mark.parametrize("lengths,ch,n,groups,dtype", [
    ([2100], 40, 16, 1, BF16), ([1300, 0, 1030, 3], 24, 8, 1, F32), ([1100], 48, 32, 2, F32), ([1030, 1026], 16, 64, 1, BF16),
    ([1280], 8, 128, 1, F32)])
def test_ssm_prefill_segments_carry_their_states(lengths, ch, n, groups, dtype):
    """States that last for several segments: outputs, final states, tile states, all of which would be far off if a segment's
    state were not carried on, or carried by another segment's decay."""
    assert kda.load_library().kda_ssm_prefill_launches(len(lengths), sum(lengths), ch, n, groups) == 3
    k = ssm_slow_case(lengths, ch, n, groups, dtype, seed=n + 1)
    y, S_T, tiles = ssm_run(k, save_states=True)
    ssm_check(k, y, S_T, lengths)
    tile_states_check(k, tiles, lengths)
    h = ssm_host(k)
    (y_ref, S_ref), (y_mag, S_mag), half = L.ssm(**h), ssm_magnitude(h), torch.finfo(dtype).eps / 2
    long, chain = [m > 512 for m in lengths], (max(lengths) + 64) * 2.0 ** -21
    bounds = half * np.abs(y_ref) + chain * y_mag, chain * S_mag
    right = ssm_with_join(h, 256, lambda own, before, A: np.exp(own * A))
    assert np.allclose(right[0], y_ref, rtol=1e-9, atol=1e-9) and np.allclose(right[1], S_ref, rtol=1e-9, atol=1e-9)
    for wrong in (lambda own, before, A: 0.0, lambda own, before, A: np.exp(before * A)):
        y_bad, S_bad = ssm_with_join(h, 256, wrong)[:2]
        assert (np.abs(y_bad - y_ref) / bounds[0]).max() > 50
        assert all(o.max() > 20 for o in (np.abs(S_bad - S_ref) / bounds[1])[long])


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


def test_ssm_backward_segments_carry_their_states():
    """Gradients over the tile states of such a forward, whose reverse chains last as long."""
    lengths = [1300, 0, 1030, 3]
    k = ssm_slow_case(lengths, 24, 8, seed=45)
    assert kda.load_library().kda_ssm_prefill_launches(4, 2333, 24, 8, 1) == 3
    dy, dS = randn(2333, 24, seed=46), 32 * randn(4, 24, 8, seed=47)
    ssm_grad_check(k, dy, dS, ssm_grad_run(k, dy, dS), lengths)
    # dS_T reaches the first tokens: without it dS0 would be far off
    h = ssm_host(k)
    ref, cut = (L.ssm_backward(dy=host(dy), dS_T=d, **h)["dS0"] for d in (host(dS), None))
    mag = ssm_grad_magnitude(h, host(dy), host(dS))["dS0"]
    assert all((np.abs(ref - cut) / (2 * 1300 + 128) / 2.0 ** -21 / mag)[s].max() > 20 for s in (0, 2))


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


def test_ssm_backward_not_a_number_stays_in_sight():
    """A NaN reaches the gradients that it reaches in the formulas, those of the tokens before it among them, and no
    other sequence."""
    k = ssm_case([200, 90], 24, 16, seed=31)
    dy, dS = randn(290, 24, seed=32), randn(2, 24, 16, seed=33)
    k["dt"][150, 5] = float("nan")
    g = ssm_grad_run(k, dy, dS)
    ref = L.ssm_backward(dy=host(dy), dS_T=host(dS), **ssm_host(k))
    for name in g._fields:
        np.testing.assert_array_equal(np.isnan(host(getattr(g, name))), np.isnan(ref[name]), err_msg=name)
    assert np.isnan(ref["ddt"][:200, 5]).all() and np.isnan(ref["dB"][:151]).all() and not np.isnan(ref["dB"][200:]).any()


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


@pytest.mark.parametrize("lengths,ch,n,groups,soft", [([90, 40], 16, 16, 1, True), ([65, 1, 0, 30], 16, 8, 2, False)])
def test_ssm_backward_differences_along_the_gradient(lengths, ch, n, groups, soft):
    """Each gradient g against the difference of two forward runs along g / |g|, where the slope is |g| itself: another sign,
    half or twice the size, or a part that points elsewhere shows.

    The difference is off by its truncation (twice the change from half the step, with the formulas in 64 bits: its error
    falls with the step's square, so that change is three quarters of it) and by the rounding of both runs' outputs (their
    bounds, added up, over the step). The slope of the kernel's g is off by the bound of g, added up along the direction."""
    k, dy, dS = ssm_grad_case(lengths, ch, n, groups, seed=42, soft=soft, bias=soft)
    g, h = ssm_grad_run(k, dy, dS), ssm_host(k)
    grad_mag, chain, step = ssm_grad_magnitude(h, host(dy), host(dS)), max(lengths) + 64, 0.25
    hy, hS = host(dy), host(dS)

    def loss(c):
        y, S = ssm_run(c)
        return (host(y) * hy).sum() + (host(S) * hS).sum()

    def exact(c):
        y, S = L.ssm(**ssm_host(c))
        return (y * hy).sum() + (S * hS).sum()

    y_mag, S_mag = ssm_magnitude(h)
    for name, of in (("x", "dx"), ("dt", "ddt"), ("B", "dB"), ("C", "dC"), ("z", "dz"), ("A", "dA"), ("D", "dD"),
                     ("dt_bias", "ddt_bias"), ("S0", "dS0")):
        if k[name] is None:
            continue
        grad = getattr(g, of)
        size = float(grad.double().norm())
        move = lambda s: (dict(k, **{name: k[name] + (f * s / size * grad)}) for f in (1, -1))
        up, down = move(step)
        along = (host(up[name]) - host(down[name])) / (2 * step)  # as the inputs' rounding leaves it
        want, got = (host(grad) * along).sum(), (loss(up) - loss(down)) / (2 * step)
        a, b = [(exact(u) - exact(d)) / (2 * s) for s in (step, step / 2) for u, d in [move(s)]]
        y_up, S_up = ssm_magnitude(ssm_host(up))
        outputs = [(np.maximum(u, v) * np.abs(w)).sum() for u, v, w in ((y_up, y_mag, hy), (S_up, S_mag, hS))]
        tol = 2 * abs(a - b) + 2 * chain * 2.0 ** -21 * sum(outputs) / step \
            + 2 * chain * 2.0 ** -21 * (grad_mag[of] * np.abs(along)).sum()
        assert tol < size / 4, "%s: the test cannot tell: %.3g of %.3g" % (name, tol, size)
        assert abs(got - want) <= tol, "%s: %.6g, by differences %.6g, tolerance %.3g" % (name, want, got, tol)


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


def ssm_in_fp32(h, dy, dS_T):
    """S_T, dS0 and dA of one sequence (one group) as the formulas give them token by token with every operation rounded to
    fp32, but for the exponentials of the states' chain: those err as the hardware's do.

    The hardware's 2^x was measured against fp64 at a million points of each [-2^e, -2^(e-1)], e = -15 .. 1: off by at most
    2^-22.7 of itself, and too small on average: by at most 8e-9 above -2^-8, 2.7e-8 down to -1/4, 5.1e-8 below. So here,
    with a uniform part of up to 2^-22.7."""
    rng, f = np.random.default_rng(0), np.float32
    x, dt, B, C, A, z, bias = (h[n].astype(f) for n in ("x", "dt", "B", "C", "A", "z", "dt_bias"))
    delta, e = L.softplus(dt + bias), dy.astype(f) * z * L.sigmoid(z)
    S, G, dA, block, before, a = h["S0"][0].astype(f), dS_T[0].astype(f), np.zeros_like(A), np.zeros_like(A), [], []
    for t in range(len(x)):
        before.append(S)
        a.append(np.exp(delta[t][:, None] * A))
        v = np.float64(delta[t][:, None] * A)
        low = np.where(v > -2.0 ** -8 * np.log(2), 8e-9, np.where(v > -0.25 * np.log(2), 2.7e-8, 5.1e-8))
        S = ((1 - low + 2.0 ** -22.7 * rng.uniform(-1, 1, A.shape)) * np.exp(v) * S + (delta[t] * x[t])[:, None] * B[t]).astype(f)
    for t in range(len(x) - 1, -1, -1):
        G = a[t] * (G + C[t] * e[t][:, None])
        block = block + G * before[t] * delta[t][:, None]
        if t % 128 == 0:
            dA, block = dA + block, np.zeros_like(block)
    assert all(v.dtype == f for v in (S, G, dA))
    return S, G, dA


@pytest.mark.parametrize("T,n,mean", [(500, 16, -6.0), (1422, 8, -4.0), (1422, 16, -6.0)])
def test_ssm_long_chains_keep_their_bits(T, n, mean):
    """Slow decays over one long sequence in fp32, by norm: S_T, dS0 and dA are off by at most twice what rounding each
    operation to fp32 leaves, with the hardware's exponentials in the states' chain and exact ones in the gradients' own.

    S_T comes through the states' chain alone and dS0 through the gradients' alone (the hardware's exponentials there would
    leave 3 to 5 times as much). dA = sum_t delta_t G_t a_t h_(t-1) takes one factor from each: a relative error of h_(t-1)
    is one of the term, and one that leans to one side, a step's worth for every step that a part of h_(t-1) has come
    through, does not average out over the tokens. So the states' exponentials count in dA as they do in S_T."""
    ch = 64
    k = ssm_case([T], ch, n, seed=76)
    k["dt"] = randn(T, ch, seed=79, std=0.5, mean=mean)
    dy, dS = randn(T, ch, seed=80), randn(1, ch, n, seed=81)
    g, S_T, h = ssm_grad_run(k, dy, dS), ssm_run(k)[1], ssm_host(k)
    ref, S_ref = L.ssm_backward(dy=host(dy), dS_T=host(dS), **h), L.ssm(**h)[1]
    error = lambda got, want: np.linalg.norm(got - want) / np.linalg.norm(want)
    model = ssm_in_fp32(h, host(dy), host(dS))
    for name, got, want, m in (("S_T", S_T[0], S_ref[0], model[0]), ("dS0", g.dS0[0], ref["dS0"][0], model[1]),
                               ("dA", g.dA, ref["dA"], model[2])):
        have, allow = error(host(got), want), 2 * error(m, want)
        print("%s: %.2e of its norm, allowed %.2e" % (name, have, allow))
        assert have <= allow, "%s: %.3g of its norm, allowed %.3g" % (name, have, allow)


# ----------------------------------------------------------- short convolution ----
# A sum of W products and a bias: (W + 1) 2^-24 of its terms' magnitude, through a Swish whose slope is at
# most 1.1, its exponential and reciprocal good to 2^-22 each: chain 4 W + 16 steps of 2^-21 covers it. dw
# and dbias add T terms (at most T 2^-24, 64 in a row and then the runs).

def conv_case(lengths, C, W, dtype, bias=True, state=True, seed=0):
    T, N = sum(lengths), len(lengths)
    return dict(x=randn(T, C, seed=seed + 1, dtype=dtype), w=randn(C, W, seed=seed + 2, std=W ** -0.5), cu=cu_of(lengths),
                bias=randn(C, seed=seed + 3) if bias else None,
                state=randn(N, W - 1, C, seed=seed + 4, dtype=dtype) if state else None)


def conv_check(k, y, last, lengths):
    h = {n: (None if v is None else v.cpu().numpy() if n == "cu" else host(v)) for n, v in k.items()}
    ref, last_ref = L.conv(h["x"], h["w"], h["cu"], h["state"], h["bias"])
    a = {n: None if v is None or n == "cu" else np.abs(v) for n, v in h.items()}
    rows = np.zeros_like(ref)
    W = h["w"].shape[1]
    for s, b, e, r in L._windows(a["x"], W, h["cu"], a["state"]):
        rows[b:e] = sum(a["w"][:, j] * r[j:j + e - b] for j in range(W)) + (0 if a["bias"] is None else a["bias"])
    within(y, ref, 1.1 * rows, 4 * W + 16, "y")
    if last is not None:
        np.testing.assert_array_equal(host(last), last_ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,C,W", [([1], 8, 4), ([100], 72, 4), ([0, 5, 1, 0, 17, 16, 2, 0], 24, 4), ([33, 20], 16, 1),
                                         ([1] * 40, 16, 8), ([50, 3], 8, 8), ([40, 9], 40, 5), ([16, 33], 16, 2), ([31], 8, 3)])
def test_conv_bias(lengths, C, W, dtype):
    k = conv_case(lengths, C, W, dtype, seed=W)
    last = torch.empty_like(k["state"])
    y = kda.kda_short_conv_swish(k["x"], k["w"], k["cu"], state_in=k["state"], state_out=last, bias=k["bias"], y=nan_like(k["x"]))
    conv_check(k, y, last, lengths)
    y = kda.kda_short_conv_swish(k["x"], k["w"], k["cu"], bias=k["bias"])
    conv_check(dict(k, state=None), y, None, lengths)
    # the state in place
    st = k["state"].clone()
    kda.kda_short_conv_swish(k["x"], k["w"], k["cu"], state_in=st, state_out=st, bias=k["bias"])
    assert torch.equal(st, last)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,C,W", [(1, 8, 4), (5, 4096, 4), (300, 40, 4), (3, 16, 1), (4, 24, 8), (2, 8, 2)])
def test_conv_step(N, C, W, dtype):
    k = conv_case([1] * N, C, W, dtype, seed=N)
    st = k["state"].clone()
    y = kda.kda_short_conv_step(k["x"], k["w"], st if W > 1 else None, bias=k["bias"])
    conv_check(k, y, st, [1] * N)
    st = k["state"].clone()
    conv_check(dict(k, bias=None), kda.kda_short_conv_step(k["x"], k["w"], st), st, [1] * N)


def test_conv_steps_continue_a_prompt():
    k = conv_case([20], 64, 4, BF16, seed=5)
    last = torch.empty_like(k["state"])
    y = kda.kda_short_conv_swish(k["x"], k["w"], state_in=k["state"], state_out=last, bias=k["bias"])
    st = torch.empty_like(last)
    out = [kda.kda_short_conv_swish(k["x"][:15].clone(), k["w"], state_in=k["state"], state_out=st, bias=k["bias"])]
    out += [kda.kda_short_conv_step(k["x"][t:t + 1].clone(), k["w"], st, bias=k["bias"]) for t in range(15, 20)]
    assert torch.equal(torch.cat(out), y) and torch.equal(st, last)


@pytest.mark.parametrize("dtype,dy_dtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("lengths,C,W", [([1], 8, 4), ([64], 16, 4), ([65], 16, 4), ([0, 5, 1, 0, 64, 2, 63, 130, 0], 24, 4), ([70, 3], 8, 1),
                                         ([1] * 70, 16, 8), ([62, 4, 200], 8, 8), ([67], 8, 5), ([66, 66], 72, 2), ([63, 1, 3], 8, 3)])
def test_conv_backward(lengths, C, W, dtype, dy_dtype):
    k = conv_case(lengths, C, W, dtype, seed=W + 1)
    T = sum(lengths)
    dy = randn(T, C, seed=9, dtype=dy_dtype)
    h = {n: (v.cpu().numpy() if n == "cu" else host(v)) for n, v in k.items()}
    for state in (True, False):
        got = kda.kda_short_conv_backward(k["x"], k["w"], dy, k["cu"], bias=k["bias"], state_in=k["state"] if state else None,
                                          want_dstate=True)
        st = h["state"] if state else None
        ref = L.conv_backward(h["x"], h["w"], host(dy), h["cu"], st, h["bias"])
        # magnitudes: every product of the gradient of v (at most 1.1 |dy| and its own error, that of v, 4 W + 16 steps
        # of its terms) with a tap or a row
        v = np.abs(L.conv(np.abs(h["x"]), np.abs(h["w"]), h["cu"], None if st is None else np.abs(st), np.abs(h["bias"]))[0]) + 1
        g = 1.1 * np.abs(host(dy)) * (2 + 2 * v)
        mdx, mdw, mdb, mds = np.zeros_like(h["x"]), np.zeros_like(h["w"]), g.sum(0), np.zeros((len(lengths), W - 1, C))
        for s, b, e, rows in L._windows(np.abs(h["x"]), W, h["cu"], None if st is None else np.abs(st)):
            d = np.zeros_like(rows)
            for j in range(W):
                d[j:j + e - b] += g[b:e] * np.abs(h["w"][:, j])
                mdw[:, j] += (g[b:e] * rows[j:j + e - b]).sum(0)
            mdx[b:e], mds[s] = d[W - 1:], d[:W - 1]
        chain = 4 * W + 16
        for n, a, r, m in zip(("dx", "dw", "dbias", "dstate"), got, ref, (mdx, mdw, mdb, mds)):
            within(a, r, m, chain + (T / 8 if n in ("dw", "dbias") else 0), n)
    # without the optional outputs the rest keeps its bits
    again = kda.kda_short_conv_backward(k["x"], k["w"], dy, k["cu"], bias=k["bias"])
    assert all(torch.equal(a, b) for a, b in zip(again[:3], got[:3])) and again[3] is None
    again = kda.kda_short_conv_backward(k["x"], k["w"], dy, k["cu"])
    assert again[2] is None
    within(again[0], L.conv_backward(h["x"], h["w"], host(dy), h["cu"])[0], mdx, chain, "dx without bias")


def test_conv_backward_long_runs():
    """Wide calls take longer runs of tokens than narrow ones: the same dx and dstate to the bit, and column sums that
    differ by the order of their additions alone (at most 128 in a run and 30 over the runs here, 32 and 46 there)."""
    lengths, C, W = [3000, 2, 0, 5190, 1408], 4096, 4
    T = sum(lengths)
    k = conv_case(lengths, C, W, BF16, seed=12)
    dy = randn(T, C, seed=13, dtype=BF16)
    wide = kda.kda_short_conv_backward(k["x"], k["w"], dy, k["cu"], bias=k["bias"], state_in=k["state"], want_dstate=True)
    for c in (slice(0, 16), slice(2040, 2056), slice(C - 16, C)):
        part = {n: k[n][..., c].contiguous() for n in ("x", "state", "bias")}
        part["w"] = k["w"][c].contiguous()
        dyc = dy[:, c].contiguous()
        dx, dw, db, ds = kda.kda_short_conv_backward(part["x"], part["w"], dyc, k["cu"], bias=part["bias"], state_in=part["state"],
                                                     want_dstate=True)
        assert torch.equal(wide[0][:, c], dx) and torch.equal(wide[3][..., c], ds)
        g, mag = 1.1 * np.abs(host(dyc)), np.zeros((16, W))
        for s, b, e, rows in L._windows(np.abs(host(part["x"])), W, k["cu"].cpu().numpy(), np.abs(host(part["state"]))):
            for j in range(W):
                mag[:, j] += (g[b:e] * rows[j:j + e - b]).sum(0)
        assert (np.abs(host(wide[1][c]) - host(dw)) <= 236 * 2.0 ** -24 * mag).all()
        assert (np.abs(host(wide[2][c]) - host(db)) <= 236 * 2.0 ** -24 * g.sum(0)).all()


def test_conv_rows_behind_the_last_sequence():
    k = conv_case([50, 20], 16, 4, F32, seed=6)
    x = torch.cat([k["x"], torch.full((130, 16), float("nan"), device=DEV)])
    dy = torch.cat([randn(70, 16, seed=7), torch.full((130, 16), float("nan"), device=DEV)])
    y = torch.full_like(x, 7.0)
    kda.kda_short_conv_swish(x, k["w"], k["cu"], bias=k["bias"], y=y)
    assert (y[70:] == 7.0).all() and torch.equal(y[:70], kda.kda_short_conv_swish(k["x"], k["w"], k["cu"], bias=k["bias"]))
    a = kda.kda_short_conv_backward(x, k["w"], dy, k["cu"], bias=k["bias"])
    b = kda.kda_short_conv_backward(k["x"], k["w"], dy[:70].clone(), k["cu"], bias=k["bias"])
    assert torch.equal(a[0][:70], b[0])
    for u, v in zip(a[1:3], b[1:3]):
        assert torch.equal(u, v)


# -------------------------------------------------------------- residual norms ----
# Row sums of D terms by a tree of at most 8 + log2(512) + 9 additions; everything else a few operations on the
# element: chain 64 covers it. Column sums add rows (at most rows / 8 + 8 in a row).

def norm_case(rows, D, dtype, res, post=True, gate=True, scale=True, pre=True, stream=True, seed=0):
    pick = lambda has, *a, **k: randn(*a, **k) if has else None
    return dict(y=randn(rows, D, seed=seed + 1, dtype=dtype), r=pick(stream, rows, D, seed=seed + 2, std=2.0, dtype=res),
                w_pre=pick(pre, D, seed=seed + 3, mean=1.0, std=0.3), w_post=pick(post, D, seed=seed + 4, mean=1.0, std=0.3),
                gate=pick(gate, rows, D, seed=seed + 5, dtype=dtype), scale=pick(scale, D, seed=seed + 6))


def norm_call(k, **kw):
    return kda.kda_residual_norm(k["y"], k["r"], k["w_pre"], w_post=k["w_post"], gate=k["gate"], scale=k["scale"],
                                 res_scale=0.75, eps=1e-5, **kw)


NORM_OPTIONS = [(1, 1, 1, 1, 1), (0, 0, 0, 1, 1), (1, 0, 0, 0, 1), (0, 1, 1, 1, 0), (0, 0, 0, 0, 1), (1, 1, 0, 1, 1)]


def norm_mags(h):
    """|terms| of r' and of x: x divides by the row's rms, whose own relative error is that of a sum of squares."""
    u = np.abs(L.norm(h["y"], None, None, h["w_post"], h["gate"], h["scale"], 0.75, 1e-5)[1])
    out = u + (0 if h["r"] is None else 0.75 * np.abs(h["r"]))
    return out


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,D", [(1, 8), (3, 264), (5, 4096), (700, 128), (4, 8192), (9, 5000), (2, 4104), (1, 1024)])
def test_residual_norm(rows, D, dtype, res):
    for opt in NORM_OPTIONS:
        post, gate, scale, pre, stream = opt
        k = norm_case(rows, D, dtype, res if stream else dtype, post, gate, scale, pre, stream, seed=D)
        x, r = norm_call(k)
        h = {n: host(v) for n, v in k.items()}
        x_ref, r_ref = L.norm(**h, res_scale=0.75, eps=1e-5)
        mag = norm_mags(h)
        within(r, r_ref, mag, 64, "r' %s" % (opt,))
        if pre:
            rms = np.sqrt((r_ref ** 2).mean(-1, keepdims=True) + 1e-5)
            within(x, x_ref, mag / rms * np.abs(h["w_pre"]) * (1 + (mag * np.abs(r_ref)).mean(-1, keepdims=True) / rms ** 2), 64, "x %s" % (opt,))
        else:
            assert x is None
        if stream:  # the stream in place
            keep = k["r"].clone()
            norm_call(k, r_out=k["r"])
            assert torch.equal(k["r"], r)
            k["r"] = keep


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,D", [(1, 8), (3, 264), (300, 4096), (1500, 128), (4, 8192), (9, 5000), (2, 4104)])
def test_residual_norm_backward(rows, D, dtype, res):
    for opt in NORM_OPTIONS:
        post, gate, scale, pre, stream = opt
        k = norm_case(rows, D, dtype, res if stream else dtype, post, gate, scale, pre, stream, seed=D + 1)
        dx = randn(rows, D, seed=31, dtype=dtype) if pre else None
        for dr in (randn(rows, D, seed=32), None):
            if dr is None and not pre:
                continue
            g = kda.kda_residual_norm_backward(k["y"], k["r"], k["w_pre"], dx, dr, w_post=k["w_post"], gate=k["gate"],
                                               scale=k["scale"], res_scale=0.75, eps=1e-5)
            h = {n: host(v) for n, v in k.items()}
            ref = L.norm_backward(dx=host(dx), dr=host(dr), **h, res_scale=0.75, eps=1e-5)
            mag = norm_grad_mags(h, host(dx), host(dr))
            for n in ("dy", "dr", "dgate", "dw_post", "dscale", "dw_pre"):
                got = getattr(g, n)
                if got is None:
                    assert (k if n != "dy" else h)[n[1:]] is None
                    continue
                within(got, ref[n], mag[n], 64 + (rows / 8 if n in ("dw_post", "dscale", "dw_pre") else 0), "%s %s" % (n, opt))


def norm_grad_mags(h, dx, dr):
    """norm_backward with every term taken positive, its row factors as they are; a row's 1 / rms enters each
    twice, with the relative error of its sum."""
    out = L.norm(**h, res_scale=0.75, eps=1e-5)[1]
    om = norm_mags(h)
    d = np.zeros_like(out) if dr is None else np.abs(dr)
    m = {}
    amp = 1.0
    if h["w_pre"] is not None:
        rs = 1 / np.sqrt((out ** 2).mean(-1, keepdims=True) + 1e-5)
        amp = 2 + 2 * (om * np.abs(out)).mean(-1, keepdims=True) * rs ** 2
        m["dw_pre"] = (np.abs(dx) * om * rs * amp).sum(0)
        dh = np.abs(dx * h["w_pre"])
        d = d + rs * amp * (dh + om * rs * (dh * om * rs).mean(-1, keepdims=True))
    m["dr"] = 0.75 * d
    rs = None if h["w_post"] is None else 1 / np.sqrt((h["y"] ** 2).mean(-1, keepdims=True) + 1e-5)
    u = np.abs(h["y"] if rs is None else h["y"] * rs * h["w_post"])
    s = 1.0 if h["gate"] is None else L.sigmoid(h["gate"])
    m["dscale"] = 2 * (d * s * u).sum(0)
    d = d if h["scale"] is None else d * np.abs(h["scale"])
    if h["gate"] is not None:
        m["dgate"] = 4 * d * u * s
        d = d * s
    if rs is not None:
        hat = np.abs(h["y"] * rs)
        m["dw_post"] = 2 * (d * hat).sum(0)
        dh = d * np.abs(h["w_post"])
        d = 2 * rs * (dh + hat * (dh * hat).mean(-1, keepdims=True))
    m["dy"] = d
    return m


def test_residual_norm_many_rows_same_bits():
    """More rows than CTAs; the column sums give the same bits each time; zero rows."""
    k = norm_case(5000, 512, BF16, F32, seed=3)
    dx, dr = randn(5000, 512, seed=4, dtype=BF16), randn(5000, 512, seed=5)
    run = lambda kk, a, b: kda.kda_residual_norm_backward(kk["y"], kk["r"], kk["w_pre"], a, b, w_post=kk["w_post"], gate=kk["gate"],
                                                          scale=kk["scale"], res_scale=0.75, eps=1e-5)
    a, b = run(k, dx, dr), run(k, dx, dr)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    h = {n: host(v) for n, v in k.items()}
    ref = L.norm_backward(dx=host(dx), dr=host(dr), **h, res_scale=0.75, eps=1e-5)
    mag = norm_grad_mags(h, host(dx), host(dr))
    for n in ("dw_post", "dscale", "dw_pre"):
        within(getattr(a, n), ref[n], mag[n], 64 + 5000 / 8, n)
    none = {n: (v[:0] if v is not None and v.dim() == 2 else v) for n, v in k.items()}
    assert norm_call(none)[0].shape == (0, 512)
    g = run(none, dx[:0], dr[:0])
    assert (g.dw_pre == 0).all() and (g.dscale == 0).all()


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,D", [(3, 264), (300, 4096), (5, 8192)])
def test_residual_norm_backward_without_w_pre_does_not_depend_on_the_stream(rows, D, dtype, res):
    """Without a norm before the next block r' = a r + s u enters no gradient: infinities and NaN in r change no bit."""
    for post, gate, scale in ((1, 1, 1), (0, 0, 0), (1, 0, 1)):
        k = norm_case(rows, D, dtype, res, post, gate, scale, pre=False, seed=D + 2)
        dr = randn(rows, D, seed=33)
        run = lambda r: kda.kda_residual_norm_backward(k["y"], r, None, None, dr, w_post=k["w_post"], gate=k["gate"],
                                                       scale=k["scale"], res_scale=0.75, eps=1e-5)
        odd = k["r"].clone()
        odd[0, 5], odd[1, D - 1], odd[rows - 1, 0] = float("inf"), float("-inf"), float("nan")
        h = {n: host(v) for n, v in k.items()}
        ref, mag = L.norm_backward(dx=None, dr=host(dr), **h, res_scale=0.75, eps=1e-5), norm_grad_mags(h, None, host(dr))
        for n, want, got in zip(("dy", "dr", "dgate", "dw_post", "dscale", "dw_pre"), run(k["r"]), run(odd)):
            assert (want is None) == (got is None) and (got is None or torch.equal(want, got)), n
            if got is not None:
                within(got, ref[n], mag[n], 64 + (rows / 8 if n in ("dw_post", "dscale") else 0), n)


def test_layer_together():
    """A block as it is used: norm before, convolution, scan, norm after with gate and residual, forwards and
    backwards, every call's outputs the next one's inputs; on a side stream and in a graph the same bits."""
    lengths, C, n = [150, 60, 1], 64, 16
    T, cu = sum(lengths), cu_of(lengths)
    ssm = ssm_case(lengths, C, n, 1, BF16, seed=60)
    conv = conv_case(lengths, C, 4, BF16, seed=61)
    nk = norm_case(T, C, BF16, F32, seed=62)
    y0, dx_out = randn(T, C, seed=63, dtype=BF16), randn(T, C, seed=64, dtype=BF16)

    def block():
        p = dict(w_post=nk["w_post"], gate=nk["gate"], scale=nk["scale"], res_scale=0.75, eps=1e-5)
        x, r = kda.kda_residual_norm(y0, nk["r"], nk["w_pre"], **p)
        u = kda.kda_short_conv_swish(x, conv["w"], cu, state_in=conv["state"], bias=conv["bias"])
        sp = dict(D=ssm["D"], dt_bias=ssm["dt_bias"], z=ssm["z"])
        y, S, tiles = kda.kda_ssm_prefill(u, ssm["dt"], ssm["B"], ssm["C"], ssm["A"], ssm["S0"], cu, save_states=True, **sp)
        x2, r2 = kda.kda_residual_norm(y, r, nk["w_pre"], **p)
        g2 = kda.kda_residual_norm_backward(y, r, nk["w_pre"], dx_out, None, **p)
        gs = kda.kda_ssm_backward(u, ssm["dt"], ssm["B"], ssm["C"], ssm["A"], g2.dy.to(BF16), tiles, None, ssm["S0"], cu, **sp)
        gc = kda.kda_short_conv_backward(x, conv["w"], gs.dx, cu, state_in=conv["state"], bias=conv["bias"])
        g1 = kda.kda_residual_norm_backward(y0, nk["r"], nk["w_pre"], gc[0].to(BF16), g2.dr, **p)
        return [x2, r2, S, *g1, *gc[:3], gs.dA]

    out = block()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = block()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = block()
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(out, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)

    # against the oracle: each call's inputs are the last one's rounded outputs, so the chain is compared piece by piece
    h = lambda v: None if v is None else host(v)
    x_ref, r_ref = L.norm(h(y0), h(nk["r"]), h(nk["w_pre"]), h(nk["w_post"]), h(nk["gate"]), h(nk["scale"]), 0.75, 1e-5)
    u_ref = L.conv(x_ref, h(conv["w"]), cu.cpu().numpy(), h(conv["state"]), h(conv["bias"]))[0]
    y_ref, S_ref = L.ssm(u_ref, h(ssm["dt"]), h(ssm["B"]), h(ssm["C"]), h(ssm["A"]), h(ssm["S0"]), cu.cpu().numpy(), h(ssm["D"]),
                         h(ssm["dt_bias"]), h(ssm["z"]))
    x2_ref, r2_ref = L.norm(y_ref, r_ref, h(nk["w_pre"]), h(nk["w_post"]), h(nk["gate"]), h(nk["scale"]), 0.75, 1e-5)
    # bf16 rounds x, u and y by 2^-8 each on the way (relative to rows of unit size): a few times that by norm
    for got, ref in ((out[0], x2_ref), (out[1], r2_ref), (out[2], S_ref)):
        assert np.linalg.norm(h(got) - ref) <= 4 * 2.0 ** -8 * np.linalg.norm(ref)


def test_layer_other_device_is_refused_and_current_device_kept():
    k = norm_case(2, 64, BF16, F32)
    with pytest.raises(ValueError):
        kda.kda_residual_norm(k["y"], k["r"].cpu(), k["w_pre"])
    with pytest.raises(TypeError):
        kda.kda_residual_norm(k["y"], k["r"], k["w_pre"].to(BF16))
    with pytest.raises(ValueError):
        kda.kda_residual_norm(k["y"].t(), None, None)
    with pytest.raises(kda.KDAError):
        kda.kda_residual_norm(randn(2, 12), None, randn(12))
    assert torch.cuda.current_device() == 0
