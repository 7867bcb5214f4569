"""The layer operators around the gated recurrences, as they are measured: their cases, inputs,
plain forms and definitions in 64 bits.

The operators (packed token axis T, sequences by ``cu_seqlens``; "io" is bf16 or fp32):

* the selective state space scan, per channel d and state n, with G groups of channels sharing B and C,

      delta = softplus(dt + dt_bias),  h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
      y_t = (sum_n C_t h_t + D x_t) * silu(z_t),

  over prompts (``scan_prompt``), for one token of each sequence (``scan_step``) and forward and
  backward (``scan_train``);
* the causal short convolution with a bias and Swish, forward and backward (``conv_train``) and for
  one token of each sequence (``conv_step``);
* the norms after a block and before the next one with the residual stream between them,

      r' = a r + s * sigmoid(g) * RMSNorm(y) w_post,   x = RMSNorm(r') w_pre,

  forward (``norm``) and forward and backward (``norm_train``).

``run`` computes them in plain torch, or with ``own`` by the calls a user makes of the package.
"""
import random

import torch

own = False

EPS = 1e-6
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a 256-token prompt of a small model in fp32: launch latency
        dict(name="scan_prompt_tiny", op="scan_prompt", io="f32", tokens=256, seqs=1, channels=128, states=16,
             groups=1, gate=False, start=False),
        # one 8192-token prompt at the width of 32 heads of 128 channels
        dict(name="scan_prompt_8k", op="scan_prompt", io="bf16", tokens=8192, seqs=1, channels=4096, states=16,
             groups=1, gate=True, start=True),
        # a packed batch of 16 prompts of uneven lengths, wider states, B and C in two groups
        dict(name="scan_prompt_ragged", op="scan_prompt", io="bf16", tokens=6151, seqs=16, channels=1024, states=64,
             groups=2, gate=True, start=True),
        # the next token of one sequence: latency
        dict(name="scan_step_1", op="scan_step", io="bf16", seqs=1, channels=4096, states=16, groups=1, gate=True),
        # the next token of 256 sequences: the state's traffic
        dict(name="scan_step_256", op="scan_step", io="bf16", seqs=256, channels=4096, states=16, groups=1, gate=True),
        # a training step on short rows in fp32, an odd length
        dict(name="scan_train_f32", op="scan_train", io="f32", tokens=509, seqs=3, channels=256, states=16,
             groups=1, gate=False, start=True),
        # a training step on a packed row of four documents
        dict(name="scan_train_4k", op="scan_train", io="bf16", tokens=4096, seqs=4, channels=4096, states=16,
             groups=1, gate=True, start=False),
        # the convolution of one projection of 32 heads of 128 channels in training, four documents
        dict(name="conv_train_8k", op="conv_train", io="bf16", tokens=8192, seqs=4, channels=4096, width=4),
        # the convolution of the next token of 256 sequences
        dict(name="conv_step_256", op="conv_step", io="bf16", seqs=256, channels=4096, width=4),
        # between two blocks while decoding one sequence: latency
        dict(name="norm_1", op="norm", io="bf16", res="f32", tokens=1, channels=4096, post=True, gate=True, scale=True),
        # between two blocks over a prompt
        dict(name="norm_8k", op="norm", io="bf16", res="bf16", tokens=8192, channels=4096, post=True, gate=True,
             scale=True),
        # the same in training, an odd number of rows, the residual stream in fp32
        dict(name="norm_train_8k", op="norm_train", io="bf16", res="f32", tokens=8191, channels=4096, post=True,
             gate=True, scale=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["scan_prompt", "scan_prompt", "scan_step", "scan_step", "scan_train", "scan_train",
                     "conv_train", "conv_step", "norm", "norm_train"])
    io = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, io=io)
    if op.startswith("scan"):
        g = rng.choice([1, 1, 2, 4])
        n = rng.choice([8, 16, 16, 32, 64, 128])
        d = 8 * g * _log(rng, 1, 512 // g)
        c.update(channels=d, states=n, groups=g, gate=rng.random() < 0.6)
        if op == "scan_step":
            c.update(seqs=_log(rng, 1, max(1, min(256, (1 << 24) // (d * n)))))
        else:
            most = (1 << 29 if op == "scan_prompt" else 1 << 28) // (d * n)
            t = _log(rng, 1, min(8192 if op == "scan_prompt" else 4096, most))
            c.update(tokens=t, seqs=_log(rng, 1, 64), start=rng.random() < 0.5)
    elif op == "conv_train":
        c.update(tokens=_log(rng, 1, 8192), seqs=_log(rng, 1, 64), channels=8 * _log(rng, 1, 512),
                 width=rng.randint(2, 8))
    elif op == "conv_step":
        c.update(seqs=_log(rng, 1, 256), channels=8 * _log(rng, 1, 512), width=rng.randint(2, 8))
    else:
        c.update(res=rng.choice(["f32", io]), tokens=_log(rng, 1, 8191), channels=8 * _log(rng, 4, 512),
                 post=rng.random() < 0.7, gate=rng.random() < 0.6, scale=rng.random() < 0.6)
    return c


def _lengths(case):
    """Lengths of the packed sequences: uneven, some of them one token or empty where there are many."""
    t, n = case["tokens"], case["seqs"]
    rng = random.Random(1000003 * t + n)
    cuts = sorted(rng.randint(0, t) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


def work(case):
    """Each input read once, each output written once; a multiply and an add count two operations."""
    op, e = case["op"], SIZE[case["io"]]
    if op.startswith("scan"):
        d, n, g = case["channels"], case["states"], case["groups"]
        z = 1 if case["gate"] else 0
        t = case["seqs"] if op == "scan_step" else case["tokens"]
        rows = t * (d * (3 + z) + 2 * g * n) * e  # x, dt, y (, z), B, C
        par = 4 * d * (n + 2)
        states = case["seqs"] * d * n * 4
        if op == "scan_step":
            return {"bytes": rows + par + 2 * states, "flops": 7 * t * d * n}
        fwd = rows + par + states * (2 if case["start"] else 1)
        if op == "scan_prompt":
            return {"bytes": fwd, "flops": 7 * t * d * n}
        grads = t * (d * (2 + z) + 2 * g * n) * 4 + par  # dx, ddt (, dz), dB, dC and the parameters'
        bwd = t * (d * (3 + z) + 2 * g * n) * e + par + grads + states * (3 if case["start"] else 1)
        return {"bytes": fwd + bwd, "flops": 25 * t * d * n}
    if op.startswith("conv"):
        d, w = case["channels"], case["width"]
        par = 4 * d * (w + 1)
        states = case["seqs"] * (w - 1) * d * e
        if op == "conv_step":
            return {"bytes": 2 * case["seqs"] * d * e + par + 2 * states, "flops": case["seqs"] * d * (2 * w + 6)}
        td = case["tokens"] * d
        return {"bytes": td * (2 * e) + par + 2 * states + td * (e + 4 + 4) + 2 * par + states * 3,
                "flops": td * (8 * w + 16)}
    t, d, r = case["tokens"], case["channels"], SIZE[case["res"]]
    gate = 1 if case["gate"] else 0
    fwd = t * d * (e * (2 + gate) + 2 * r) + 12 * d
    if op == "norm":
        return {"bytes": fwd, "flops": 14 * t * d}
    bwd = t * d * (e * (2 + gate) + r + 4 + 4 * (2 + gate)) + 24 * d  # y, dx (, gate), r, dr'; dy, dr (, dgate)
    return {"bytes": fwd + bwd, "flops": 50 * t * d}


# ----------------------------------------------------------------- inputs ----

def _inputs(case, seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    io = IO[case["io"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=device) * std + mean).to(dtype)

    op, s = case["op"], {"case": case}
    d = case["channels"]
    if op in ("scan_prompt", "scan_train", "conv_train"):
        lengths = _lengths(case)
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        s.update(lengths=lengths, cu=torch.tensor(cu, dtype=torch.int32, device=device))
        # positions of the first and last token of each sequence that has any
        some = [i for i, n in enumerate(lengths) if n]
        s.update(some=torch.tensor(some, device=device), first=torch.tensor([cu[i] for i in some], device=device),
                 last=torch.tensor([cu[i + 1] - 1 for i in some], device=device))
    if op.startswith("scan"):
        n, grp = case["states"], case["groups"]
        t = case["seqs"] if op == "scan_step" else case["tokens"]
        # steps of 0.001 to 0.1 and decay rates about 1 .. n, as such layers are initialised
        step = torch.exp(torch.rand(d, generator=g, device=device) * 4.605 - 6.908)
        s.update(x=normal(t, d, dtype=io), dt=normal(t, d, std=0.5, dtype=io), B=normal(t, grp, n, dtype=io),
                 C=normal(t, grp, n, dtype=io), A=-torch.arange(1, n + 1, device=device) * torch.exp(normal(d, n, std=0.1)),
                 D=normal(d, std=0.1, mean=1.0), dt_bias=torch.log(torch.expm1(step)),
                 z=normal(t, d, dtype=io) if case["gate"] else None)
        if op == "scan_step":
            s.update(S=normal(case["seqs"], d, n, std=0.1))
        else:
            s.update(S0=normal(case["seqs"], d, n, std=0.1) if case["start"] else None)
        if op == "scan_train":
            s.update(dy=normal(t, d, dtype=io), dS_T=normal(case["seqs"], d, n, std=0.1) if case["start"] else None)
    elif op.startswith("conv"):
        w = case["width"]
        t = case["seqs"] if op == "conv_step" else case["tokens"]
        s.update(x=normal(t, d, dtype=io), w=normal(d, w, std=w ** -0.5), bias=normal(d, std=0.1),
                 state=normal(case["seqs"], w - 1, d, dtype=io))
        if op == "conv_train":
            s.update(dy=normal(t, d))  # the gradients that come back from the recurrences are fp32
    else:
        t = case["tokens"]
        s.update(y=normal(t, d, dtype=io), r=normal(t, d, std=2.0, dtype=IO[case["res"]]),
                 w_pre=normal(d, std=0.1, mean=1.0), w_post=normal(d, std=0.1, mean=1.0) if case["post"] else None,
                 gate=normal(t, d, dtype=io) if case["gate"] else None,
                 scale=normal(d, std=0.1, mean=0.5) if case["scale"] else None, a=0.9)
        if op == "norm_train":
            s.update(dx=normal(t, d, dtype=io), dr=normal(t, d))
    return s


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    if "S" in s:
        s["S_now"] = s["S"].clone()
    if case["op"] == "conv_step":
        s["state_now"] = s["state"].clone()
    return s


# ------------------------------------------------------------ plain forms ----

def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling (both arguments are overwritten)."""
    k = 1
    while k < a.shape[0]:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _scan_forward(s):
    """delta, the true decays, the states and their predecessors, y before the gate; [T, G, D/G (, n)]."""
    case = s["case"]
    t, grp, n = s["x"].shape[0], case["groups"], case["states"]
    sh = (t, grp, -1)
    x, v = s["x"].float().view(sh), s["dt"].float() + s["dt_bias"]
    delta, A = _softplus(v).view(sh), s["A"].view(grp, -1, n)
    B, C = s["B"].float().unsqueeze(2), s["C"].float().unsqueeze(2)
    decay = torch.exp(delta.unsqueeze(-1) * A)
    b = (delta * x).unsqueeze(-1) * B
    a = decay.clone()
    if s["S0"] is not None:
        S0 = s["S0"].view(-1, grp, a.shape[2], n)
        b[s["first"]] += a[s["first"]] * S0[s["some"]]
    a[s["first"]] = 0
    h = _linear_scan(a, b)
    y = (h * C).sum(-1) + s["D"].view(grp, -1) * x
    return x, v.view(sh), delta, A, B, C, decay, h, y


def _final_states(s, h):
    n = len(s["lengths"])
    S_T = s["S0"].clone() if s["S0"] is not None else h.new_zeros(n, s["A"].shape[0], s["A"].shape[1])
    S_T[s["some"]] = h[s["last"]].reshape(-1, *S_T.shape[1:])
    return S_T


def _plain_scan_prompt(s):
    h, y = _scan_forward(s)[-2:]
    out = y.reshape(s["x"].shape)
    if s["z"] is not None:
        z = s["z"].float()
        out = out * z * _sigmoid(z)
    return {"y": out.to(s["x"].dtype), "S_T": _final_states(s, h)}


def _plain_scan_train(s):
    x, v, delta, A, B, C, decay, h, y = _scan_forward(s)
    t = x.shape[0]
    dy = s["dy"].float().view(x.shape)
    r = {}
    out = y
    if s["z"] is not None:
        z = s["z"].float().view(x.shape)
        sg = _sigmoid(z)
        out = y * z * sg
        r["dz"] = (dy * y * sg * (1 + z * (1 - sg))).view(t, -1)
        dy = dy * z * sg
    r.update(y=out.reshape(t, -1).to(s["x"].dtype), S_T=_final_states(s, h))
    # the gradient of each state: G_t = C_t dy_t + decay_{t+1} G_{t+1}, and dS_T at a sequence's last token
    src = (dy.unsqueeze(-1) * C)
    if s["dS_T"] is not None:
        src[s["last"]] += s["dS_T"].view(-1, *h.shape[1:])[s["some"]]
    back = torch.zeros_like(decay)
    back[:-1] = decay[1:]
    back[s["last"]] = 0
    G = _linear_scan(back.flip(0), src.flip(0)).flip(0)
    del back, src
    r["dC"] = (dy.unsqueeze(-1) * h).sum(2)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[s["first"]] = 0 if s["S0"] is None else s["S0"].view(-1, *h.shape[1:])[s["some"]]
    if s["S0"] is not None:
        dS0 = torch.zeros_like(s["S0"]) if s["dS_T"] is None else s["dS_T"].clone()
        dS0[s["some"]] = (decay[s["first"]] * G[s["first"]]).reshape(-1, *dS0.shape[1:])
        r["dS0"] = dS0
    gh = before.mul_(decay).mul_(G)  # G decay h_{t-1}
    r["dA"] = (gh * delta.unsqueeze(-1)).sum(0).view(-1, A.shape[-1])
    gb = (G * B).sum(-1)
    ddelta = (gh * A).sum(-1) + gb * x
    ddt = ddelta * _sigmoid(v)
    r.update(dx=(gb * delta + s["D"].view(A.shape[:2]) * dy).view(t, -1), ddt=ddt.view(t, -1),
             dB=(G * (delta * x).unsqueeze(-1)).sum(2), dD=(dy * x).sum(0).view(-1), ddt_bias=ddt.sum(0).view(-1))
    return r


def _plain_scan_step(s):
    case, S = s["case"], s["S_now"]
    grp = case["groups"]
    x, delta = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    per = s["A"].shape[0] // grp
    B = s["B"].float().unsqueeze(2).expand(-1, -1, per, -1).reshape(S.shape)
    C = s["C"].float().unsqueeze(2).expand(-1, -1, per, -1).reshape(S.shape)
    S.mul_(torch.exp(delta.unsqueeze(-1) * s["A"])).add_((delta * x).unsqueeze(-1) * B)
    y = (S * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return {"y": y.to(s["x"].dtype), "S": S}


def _history(s):
    """[T, W, C]: each token's window of raw inputs, oldest first, and whether it lies in the initial state."""
    x, w, dev = s["x"].float(), s["w"].shape[1], s["x"].device
    t = torch.arange(x.shape[0], device=dev)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    pos = t - s["cu"][seq].long()
    back = torch.arange(1 - w, 1, device=dev)
    at = pos.unsqueeze(1) + back
    win = torch.where((at >= 0).unsqueeze(-1), x[(t.unsqueeze(1) + back).clamp(min=0)],
                      s["state"].float()[seq.unsqueeze(1), (at + w - 1).clamp(0, w - 2)])
    return win, seq, at


def _plain_conv_train(s):
    win, seq, at = _history(s)
    w, n = s["w"].shape[1], s["state"].shape[0]
    v = (win * s["w"].t()).sum(1) + s["bias"]
    sg = _sigmoid(v)
    y = v * sg
    # the last W - 1 raw inputs of each sequence
    lengths = (s["cu"][1:] - s["cu"][:-1]).long()
    k = torch.arange(1 - w, 0, device=v.device) + lengths.unsqueeze(1)
    state = torch.where((k >= 0).unsqueeze(-1), s["x"][(s["cu"][:-1].long().unsqueeze(1) + k).clamp(0, max(0, v.shape[0] - 1))],
                        torch.gather(s["state"], 1, (k + w - 1).clamp(0, w - 2).unsqueeze(-1).expand(-1, -1, v.shape[1])))
    g = s["dy"] * sg * (1 + v * (1 - sg))
    each = g.unsqueeze(1) * s["w"].t()  # [T, W, C]: what each window's place gets
    rows = torch.arange(v.shape[0], device=v.device).unsqueeze(1) + torch.arange(1 - w, 1, device=v.device)
    inside = (at >= 0)
    dx = torch.zeros_like(v).index_add_(0, rows[inside], each[inside])
    dstate = v.new_zeros(n * (w - 1), v.shape[1])
    slot = seq.unsqueeze(1) * (w - 1) + at + w - 1
    dstate.index_add_(0, slot[~inside], each[~inside])
    return {"y": y.to(s["x"].dtype), "state": state, "dx": dx, "dw": (g.unsqueeze(1) * win).sum(0).t(),
            "dbias": g.sum(0), "dstate": dstate.view(n, w - 1, -1)}


def _plain_conv_step(s):
    state, x = s["state_now"], s["x"]
    win = torch.cat([state, x.unsqueeze(1)], 1)
    v = (win.float() * s["w"].t()).sum(1) + s["bias"]
    state.copy_(win[:, 1:])
    return {"y": (v * _sigmoid(v)).to(x.dtype), "state": state}


def _norm_parts(s):
    y, r = s["y"].float(), s["r"].float()
    rs1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if s["w_post"] is not None else None
    u = y if rs1 is None else y * rs1 * s["w_post"]
    m = _sigmoid(s["gate"].float()) if s["gate"] is not None else None
    f = u if m is None else u * m
    f = f if s["scale"] is None else f * s["scale"]
    out = s["a"] * r + f
    rs2 = torch.rsqrt((out * out).mean(-1, keepdim=True) + EPS)
    return y, rs1, u, m, out, rs2


def _plain_norm(s):
    out, rs2 = _norm_parts(s)[-2:]
    return {"x": (out * rs2 * s["w_pre"]).to(s["y"].dtype), "r": out.to(s["r"].dtype)}


def _plain_norm_train(s):
    y, rs1, u, m, out, rs2 = _norm_parts(s)
    res = {"x": (out * rs2 * s["w_pre"]).to(s["y"].dtype), "r": out.to(s["r"].dtype)}
    dx = s["dx"].float()
    hat = out * rs2
    dh = dx * s["w_pre"]
    d = s["dr"] + rs2 * (dh - hat * (dh * hat).mean(-1, keepdim=True))
    res.update(dw_pre=(dx * hat).sum(0), dr=s["a"] * d)
    if s["scale"] is not None:
        res["dscale"] = (d * (u if m is None else u * m)).sum(0)
        d = d * s["scale"]
    if m is not None:
        res["dgate"] = d * u * m * (1 - m)
        d = d * m
    if rs1 is not None:
        yh = y * rs1
        res["dw_post"] = (d * yh).sum(0)
        dh = d * s["w_post"]
        d = rs1 * (dh - yh * (dh * yh).mean(-1, keepdim=True))
    res["dy"] = d
    return res


# ------------------------------------------------- the package's own calls ----

def _own_scan_prompt(s):
    import gated_delta_rule_125_b200 as kda
    y, S_T = kda.kda_ssm_prefill(s["x"], s["dt"], s["B"], s["C"], s["A"], s["S0"], s["cu"], D=s["D"],
                                 dt_bias=s["dt_bias"], z=s["z"])
    return {"y": y, "S_T": S_T}


def _own_scan_train(s):
    import gated_delta_rule_125_b200 as kda
    p = dict(D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
    x, dt, B, C, A, S0, cu = (s[k] for k in ("x", "dt", "B", "C", "A", "S0", "cu"))
    y, S_T, tiles = kda.kda_ssm_prefill(x, dt, B, C, A, S0, cu, save_states=True, **p)
    g = kda.kda_ssm_backward(x, dt, B, C, A, s["dy"], tiles, s["dS_T"], S0, cu, **p)
    r = {"y": y, "S_T": S_T, "dx": g.dx, "ddt": g.ddt, "dB": g.dB, "dC": g.dC, "dA": g.dA, "dD": g.dD,
         "ddt_bias": g.ddt_bias}
    if s["z"] is not None:
        r["dz"] = g.dz
    if S0 is not None:
        r["dS0"] = g.dS0
    return r


def _own_scan_step(s):
    import gated_delta_rule_125_b200 as kda
    y = kda.kda_ssm_step(s["x"], s["dt"], s["B"], s["C"], s["A"], s["S_now"], D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
    return {"y": y, "S": s["S_now"]}


def _own_conv_train(s):
    import gated_delta_rule_125_b200 as kda
    state = torch.empty_like(s["state"])
    y = kda.kda_short_conv_swish(s["x"], s["w"], s["cu"], state_in=s["state"], state_out=state, bias=s["bias"])
    dx, dw, dbias, dstate = kda.kda_short_conv_backward(s["x"], s["w"], s["dy"], s["cu"], state_in=s["state"],
                                                        bias=s["bias"], want_dstate=True)
    return {"y": y, "state": state, "dx": dx, "dw": dw, "dbias": dbias, "dstate": dstate}


def _own_conv_step(s):
    import gated_delta_rule_125_b200 as kda
    y = kda.kda_short_conv_step(s["x"], s["w"], s["state_now"], bias=s["bias"])
    return {"y": y, "state": s["state_now"]}


def _norm_arguments(s):
    return dict(w_post=s["w_post"], gate=s["gate"], scale=s["scale"], res_scale=s["a"], eps=EPS)


def _own_norm(s):
    import gated_delta_rule_125_b200 as kda
    x, r = kda.kda_residual_norm(s["y"], s["r"], s["w_pre"], **_norm_arguments(s))
    return {"x": x, "r": r}


def _own_norm_train(s):
    import gated_delta_rule_125_b200 as kda
    x, r = kda.kda_residual_norm(s["y"], s["r"], s["w_pre"], **_norm_arguments(s))
    g = kda.kda_residual_norm_backward(s["y"], s["r"], s["w_pre"], s["dx"], s["dr"], **_norm_arguments(s))
    res = {"x": x, "r": r, "dy": g.dy, "dr": g.dr, "dw_pre": g.dw_pre}
    res.update({k: getattr(g, k) for k, has in (("dw_post", s["w_post"]), ("dgate", s["gate"]), ("dscale", s["scale"]))
                if has is not None})
    return res


PLAIN = {"scan_prompt": _plain_scan_prompt, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step,
         "conv_train": _plain_conv_train, "conv_step": _plain_conv_step, "norm": _plain_norm,
         "norm_train": _plain_norm_train}


def run(state):
    if own:
        calls = {"scan_prompt": _own_scan_prompt, "scan_train": _own_scan_train, "scan_step": _own_scan_step,
                 "conv_train": _own_conv_train, "conv_step": _own_conv_step, "norm": _own_norm,
                 "norm_train": _own_norm_train}
        return calls[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------ definitions, 64 bits ----

def exact(case, seed):
    """The definitions token by token in 64 bits; gradients by automatic differentiation."""
    s = _inputs(case, seed, "cuda")
    grad = case["op"].endswith("train")
    leaf = {k: v.double().requires_grad_(grad) for k, v in s.items()
            if torch.is_tensor(v) and v.is_floating_point() and k not in ("dy", "dS_T", "dx", "dr")}
    get = lambda k: leaf.get(k)
    with torch.set_grad_enabled(grad):
        out, pairs = _EXACT[case["op"]](s, leaf, get)
    out = {k: v.detach() for k, v in out.items()}
    if grad:
        names = [k for k in _GRADS[case["op"]] if k in leaf]
        total = sum((v * g.double()).sum() for v, g in pairs)
        for k, g in zip(names, torch.autograd.grad(total, [leaf[k] for k in names], allow_unused=True)):
            out[_GRADS[case["op"]][k]] = torch.zeros_like(leaf[k]) if g is None else g
    return out


_GRADS = {"scan_train": dict(x="dx", dt="ddt", B="dB", C="dC", z="dz", A="dA", D="dD", dt_bias="ddt_bias", S0="dS0"),
          "conv_train": dict(x="dx", w="dw", bias="dbias", state="dstate"),
          "norm_train": dict(y="dy", r="dr", gate="dgate", scale="dscale", w_pre="dw_pre", w_post="dw_post")}


def _exact_tokens(s, leaf, get, lengths, start):
    case = s["case"]
    grp = case["groups"]
    A, per = leaf["A"], leaf["A"].shape[0] // grp
    delta = torch.nn.functional.softplus(leaf["dt"] + leaf["dt_bias"], threshold=60)
    u = delta * leaf["x"]
    rows, finals, t = [], [], 0
    deltas, us, Bs, Cs = delta.unbind(0), u.unbind(0), leaf["B"].unbind(0), leaf["C"].unbind(0)
    for i, length in enumerate(lengths):
        h = (start[i] if start is not None else torch.zeros_like(A)).view(grp, per, -1)
        for _ in range(length):
            h = torch.exp(deltas[t].unsqueeze(-1) * A).view(h.shape) * h + us[t].view(grp, per, 1) * Bs[t].unsqueeze(1)
            rows.append(torch.matmul(h, Cs[t].unsqueeze(-1)).reshape(-1))
            t += 1
        finals.append(h.reshape(A.shape))
    y = torch.stack(rows) + leaf["D"] * leaf["x"]
    if get("z") is not None:
        y = y * torch.nn.functional.silu(leaf["z"])
    return y, torch.stack(finals)


def _exact_scan(s, leaf, get):
    y, S_T = _exact_tokens(s, leaf, get, s["lengths"], get("S0"))
    pairs = []
    if "dy" in s:
        pairs = [(y, s["dy"])] + ([(S_T, s["dS_T"])] if s["dS_T"] is not None else [])
    return {"y": y, "S_T": S_T}, pairs


def _exact_step(s, leaf, get):
    y, S = _exact_tokens(s, leaf, get, [1] * s["case"]["seqs"], leaf["S"])
    return {"y": y, "S": S}, []


def _exact_conv(s, leaf, get):
    w, n = leaf["w"].shape[1], s["case"]["seqs"]
    lengths = s.get("lengths", [1] * n)
    ys, states, t = [], [], 0
    for i, length in enumerate(lengths):
        row = torch.cat([leaf["state"][i], leaf["x"][t:t + length]])
        states.append(row[row.shape[0] - (w - 1):])
        if length:
            ys.append(torch.nn.functional.conv1d(row.t().unsqueeze(0), leaf["w"].unsqueeze(1), leaf["bias"],
                                                 groups=row.shape[1])[0].t())
        t += length
    y = torch.nn.functional.silu(torch.cat(ys))
    return {"y": y, "state": torch.stack(states)}, [(y, s["dy"])] if "dy" in s else []


def _exact_norm(s, leaf, get):
    def rms(v, w):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS) * w
    u = leaf["y"] if get("w_post") is None else rms(leaf["y"], leaf["w_post"])
    for k, f in (("gate", torch.sigmoid), ("scale", lambda v: v)):
        if get(k) is not None:
            u = u * f(leaf[k])
    r = s["a"] * leaf["r"] + u
    x = rms(r, leaf["w_pre"])
    return {"x": x, "r": r}, [(x, s["dx"]), (r, s["dr"])] if "dx" in s else []


_EXACT = {"scan_prompt": _exact_scan, "scan_train": _exact_scan, "scan_step": _exact_step, "conv_train": _exact_conv,
          "conv_step": _exact_conv, "norm": _exact_norm, "norm_train": _exact_norm}
