"""Cases and plain forms of the gated linear recurrence (its scan over prompts, the backward pass, single
tokens) and of the group norm with an activation, channels last.

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or calls the
framework (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DECAY = 8.0  # the recurrence's exponent scale
EPS = 1e-5
BLOCK = 32   # a forward pass leaves the state before every 32nd token to the backward pass


# ---- cases -------------------------------------------------------------------------------


def listed():
    return [
        # A long prompt of one sequence, carried on from a cached state, with the output gate.
        dict(name="scan_fwd_16384", op="scan_fwd", dtype="bf16", seqs=1, lo=16384, hi=16384, C=4096, gate=True, state=True, packed=True),
        # Ragged packed prompts in 32 bits, rows that are no whole 16-byte pieces.
        dict(name="scan_fwd_ragged_f32", op="scan_fwd", dtype="f32", seqs=7, lo=1, hi=700, C=1530, gate=True, state=True, packed=True),
        # A training step's backward pass, a batch of two sequences, what the forward pass kept in hand.
        dict(name="scan_bwd_2x2048", op="scan_bwd", dtype="bf16", seqs=2, lo=2048, hi=2048, C=4096, gate=True, state=False, packed=False,
             kept=True),
        # Packed documents of many lengths, with gradients of the states and nothing kept.
        dict(name="scan_bwd_packed", op="scan_bwd", dtype="bf16", seqs=16, lo=1, hi=700, C=4096, gate=False, state=True, packed=True,
             kept=False),
        # One sequence's decode step: latency.
        dict(name="scan_step_1", op="scan_step", dtype="bf16", N=1, C=4096, gate=True, pool=8),
        # A full serving batch.
        dict(name="scan_step_512", op="scan_step", dtype="bf16", N=512, C=8192, gate=True, pool=600),
        # The 96 heads of 128 channels of every token, with SiLU.
        dict(name="norm_token_4096", op="norm_fwd", over="token", dtype="bf16", seqs=1, lo=4096, hi=4096, C=12288, G=96, act=1, affine=True),
        # The same layer's backward pass.
        dict(name="norm_token_bwd_4096", op="norm_bwd", over="token", dtype="bf16", seqs=1, lo=4096, hi=4096, C=12288, G=96, act=1,
             affine=True),
        # One token in decode: latency.
        dict(name="norm_token_1", op="norm_fwd", over="token", dtype="bf16", seqs=1, lo=1, hi=1, C=4096, G=32, act=1, affine=True),
        # Eight long sequences of a convolutional front end, 16 channels a group.
        dict(name="norm_seq_8x4096", op="norm_fwd", over="sequence", dtype="bf16", seqs=8, lo=4096, hi=4096, C=512, G=32, act=1,
             affine=True, packed=False),
        # Ragged packed sequences in 32 bits, groups of 51 channels.
        dict(name="norm_seq_ragged_f32", op="norm_fwd", over="sequence", dtype="f32", seqs=7, lo=1, hi=700, C=1530, G=30, act=0,
             affine=True, packed=True),
        # A training step's backward pass over two sequences, the statistics in hand.
        dict(name="norm_seq_bwd_2x2048", op="norm_bwd", over="sequence", dtype="bf16", seqs=2, lo=2048, hi=2048, C=4096, G=32, act=1,
             affine=True, packed=False, kept=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, most):
    """Sequences of up to 16384 tokens, at most `most` in all: (seqs, lo, hi)."""
    hi = _log_int(rng, 1, max(2, min(16384, most)))
    seqs = min(_log_int(rng, 1, 64), max(1, most // hi))
    return seqs, max(1, hi // rng.choice([1, 8, 1000])), hi


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = 1 if dtype == "bf16" else 2
    if op == "scan_step":
        N, C = _log_int(rng, 1, 1024), _log_int(rng, 64, 8192)
        return dict(op=op, dtype=dtype, N=N, C=C, gate=rng.random() < 0.7, pool=N + _log_int(rng, 1, 64))
    if op in ("scan_fwd", "scan_bwd"):
        C = _log_int(rng, 64, 8192)
        most = (16384 * 4096 if op == "scan_fwd" else 8192 * 4096) // wide
        seqs, lo, hi = _lens(rng, most // C)
        packed = lo != hi or rng.random() < 0.5
        case = dict(op=op, dtype=dtype, seqs=seqs, lo=lo, hi=hi, C=C, gate=rng.random() < 0.7, state=rng.random() < 0.5, packed=packed)
        if op == "scan_bwd":
            case["kept"] = rng.random() < 0.7
        return case
    over = rng.choice(["token", "sequence"])
    G = rng.choice([1, 2, 5, 8, 16, 30, 32, 96])
    C = G * _log_int(rng, max(1, 64 // G), 12288 // G)
    seqs, lo, hi = _lens(rng, 8192 * 12288 // wide // C)
    case = dict(op=op, over=over, dtype=dtype, seqs=seqs, lo=lo, hi=hi, C=C, G=G, act=rng.choice([0, 1, 1]), affine=rng.random() < 0.8)
    if over == "sequence":
        case["packed"] = lo != hi or rng.random() < 0.5
        if op == "norm_bwd":
            case["kept"] = rng.random() < 0.7
    return case


def _lengths(case):
    """Lengths of the case's sequences, spread evenly over [lo, hi] in a fixed scrambled order."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((i * 7 + 3) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


# ---- inputs ------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    dev = "cuda"
    op, C = case["op"], case["C"]

    def rn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    s = {"case": case}
    if op == "scan_step":
        N = case["N"]
        lead = (N,)
        s["slots"] = torch.randperm(case["pool"], generator=g, device=dev)[:N].to(torch.int32)
        s["state"] = rn(case["pool"], C)
    else:
        lens = _lengths(case)
        N, T = len(lens), sum(lens)
        lead = (1, T) if case.get("packed", True) else (N, T // N)
        s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], device=dev)
        s["cu"] = s["offsets"].to(torch.int32) if case.get("packed") else None
    if op.startswith("scan"):
        # the usual initialisation of such layers: decays of an open gate spread evenly over 0.9..0.999
        a = 0.9 + 0.099 * torch.rand(C, generator=g, device=dev)
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / DECAY))
        s["x"], s["r"], s["i"] = (rn(*lead, C).to(dt) for _ in range(3))
        s["z"] = rn(*lead, C).to(dt) if case["gate"] else None
        if op == "scan_step":
            return s
        s["state"] = rn(N, C) if case["state"] else None
        if op == "scan_bwd":
            s["dy"] = rn(*lead, C).to(dt)
            s["dfinal"] = rn(N, C) if case["state"] else None
            s["states"] = _kept_states(s) if case["kept"] else None
        return s
    # activations with a mean of their own a channel
    s["x"] = (rn(*lead, C) * (1.0 + 0.2 * rn(C)) + 0.5 * rn(C)).to(dt)
    s["w"] = 1.0 + rn(C, std=0.2) if case["affine"] else None
    s["b"] = rn(C, std=0.2) if case["affine"] else None
    if op == "norm_bwd":
        s["dy"] = rn(*lead, C).to(dt)
        s["stats"] = torch.stack(_seq_stats(s, case), dim=-1) if case.get("kept") else None
    return s


# ---- one pass ----------------------------------------------------------------------------


def run(s):
    case = s["case"]
    return _RUN[case["op"]][1 if own else 0](s, case)


def _kda():
    import kimi_delta_attention_chunk_gb300 as kda
    return kda


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _dsilu(x):
    e = _sigmoid(x)
    return e * (1.0 + x * (1.0 - e))


# the gated recurrence


def _affine_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, in log2(T) doublings."""
    step = 1
    while step < b.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _gates(s):
    """Flat rows in 32 bits: x, the gates, c softplus(lam), the exponent, the decay and the input's weight."""
    C = s["lam"].numel()
    x, sr, si = s["x"].reshape(-1, C).float(), _sigmoid(s["r"].reshape(-1, C).float()), _sigmoid(s["i"].reshape(-1, C).float())
    rate = DECAY * (s["lam"].clamp(min=0.0) + torch.log1p(torch.exp(-s["lam"].abs())))
    e = rate * sr
    return x, sr, si, rate, torch.exp(-e), torch.sqrt(-torch.expm1(-2.0 * e))


def _marks(s, at):
    return torch.zeros(s["x"].numel() // s["lam"].numel(), dtype=torch.bool, device=at.device).index_fill_(0, at, True)


def _states(s, a, u):
    """States after every token."""
    first = s["offsets"][:-1]
    if s["state"] is not None:
        u = u.index_add(0, first, a[first] * s["state"])
    return _affine_scan(a.masked_fill(_marks(s, first)[:, None], 0.0), u)


def _kept_states(s):
    """The state before every BLOCK-th token of a row, zeros where a sequence begins."""
    x, _, si, _, a, m = _gates(s)
    h = _states(s, a, m * si * x)
    before = torch.cat([h[:1], h[:-1]]).masked_fill(_marks(s, s["offsets"][:-1])[:, None], 0.0)
    return before.view(s["x"].shape)[:, ::BLOCK].contiguous()


def _scan_fwd_plain(s, case):
    x, _, si, _, a, m = _gates(s)
    h = _states(s, a, m * si * x)
    y = h
    if s["z"] is not None:
        z = s["z"].reshape(h.shape).float()
        y = h * z * _sigmoid(z)
    return {"y": y.to(s["x"].dtype).view(s["x"].shape), "state": h[s["offsets"][1:] - 1]}


def _scan_fwd_own(s, case):
    y, state = _kda().gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], z=s["z"], decay=DECAY, initial_state=s["state"],
                                     cu_seqlens=s["cu"])
    return {"y": y, "state": state}


def _scan_bwd_plain(s, case):
    x, sr, si, rate, a, m = _gates(s)
    h = _states(s, a, m * si * x)
    first, last = s["offsets"][:-1], s["offsets"][1:] - 1
    like = lambda v: v.to(s["dy"].dtype).view(s["dy"].shape)  # noqa: E731
    g = s["dy"].reshape(x.shape).float()
    out = {}
    if s["z"] is not None:
        z = s["z"].reshape(x.shape).float()
        out["dz"] = like(g * h * _dsilu(z))
        g = g * z * _sigmoid(z)
    if s["dfinal"] is not None:
        g = g.index_add(0, last, s["dfinal"])
    onward = torch.cat([a[1:], a[:1]]).masked_fill(_marks(s, last)[:, None], 0.0)
    dh = _affine_scan(onward.flip(0), g.flip(0)).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = 0.0 if s["state"] is None else s["state"]
    ds = dh * (si * x * a * a / m - a * before)
    out["dx"], out["di"] = like(dh * m * si), like(dh * m * x * si * (1.0 - si))
    out["dr"] = like(ds * rate * sr * (1.0 - sr))
    out["dlam"] = DECAY * _sigmoid(s["lam"]) * (ds * sr).double().sum(0).float()
    if s["state"] is not None:
        out["dinitial_state"] = (a * dh)[first]
    return out


def _scan_bwd_own(s, case):
    r = _kda().gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], z=s["z"], decay=DECAY, initial_state=s["state"],
                              cu_seqlens=s["cu"], dfinal_state=s["dfinal"], states=s["states"])
    return {k: v for k, v in r.items() if v is not None}


def _scan_step_plain(s, case):
    slots = s["slots"].long()
    x, _, si, _, a, m = _gates(s)
    h = a * s["state"][slots] + m * si * x
    s["state"][slots] = h
    if s["z"] is not None:
        z = s["z"].float()
        h = h * z * _sigmoid(z)
    return {"y": h.to(s["x"].dtype), "state": s["state"]}


def _scan_step_own(s, case):
    y = _kda().gated_step(s["x"], s["r"], s["i"], s["lam"], s["state"], z=s["z"], decay=DECAY, slots=s["slots"])
    return {"y": y, "state": s["state"]}


# the group norm


def _seq_means(s, v):
    """Means over a group's channels and a sequence's tokens of v [T, G, channels]: [N, G]."""
    n, cg = s["offsets"].diff(), v.shape[2]
    belongs = _seq_of(s) == torch.arange(n.numel(), device=v.device)[:, None]
    return (belongs.double() @ v.sum(2).double() / (n[:, None] * cg)).float()


def _seq_of(s):
    return torch.repeat_interleave(torch.arange(s["offsets"].numel() - 1, device=s["x"].device), s["offsets"].diff())


def _seq_stats(s, case):
    x = s["x"].reshape(-1, case["G"], case["C"] // case["G"]).float()
    mean = _seq_means(s, x)
    var = _seq_means(s, (x - mean[_seq_of(s)][:, :, None]).square())
    return mean, 1.0 / torch.sqrt(var + EPS)


def _normed(s, case):
    """(xhat, rstd) of the flat rows [T, G, channels] in 32 bits."""
    x = s["x"].reshape(-1, case["G"], case["C"] // case["G"]).float()
    if case["over"] == "token":
        x = x - x.mean(2, keepdim=True)
        rstd = 1.0 / torch.sqrt(x.square().mean(2, keepdim=True) + EPS)
        return x * rstd, rstd
    mean, rstd = _seq_stats(s, case)
    seq = _seq_of(s)
    rstd = rstd[seq][:, :, None]
    return (x - mean[seq][:, :, None]) * rstd, rstd


def _affine(s, case, xhat):
    return xhat if s["w"] is None else xhat * s["w"].view(case["G"], -1) + s["b"].view(case["G"], -1)


def _norm_fwd_plain(s, case):
    p = _affine(s, case, _normed(s, case)[0])
    if case["act"]:
        p = p * _sigmoid(p)
    return {"y": p.to(s["x"].dtype).view(s["x"].shape)}


def _norm_kw(s, case):
    kw = dict(weight=s["w"], bias=s["b"], eps=EPS, act=case["act"], over=case["over"])
    if case["over"] == "sequence":
        kw["cu_seqlens"] = s["cu"]
    return kw


def _norm_fwd_own(s, case):
    return {"y": _kda().group_norm_fwd(s["x"], case["G"], **_norm_kw(s, case))}


def _norm_bwd_plain(s, case):
    xhat, rstd = _normed(s, case)
    dp = s["dy"].reshape(xhat.shape).float()
    if case["act"]:
        dp = dp * _dsilu(_affine(s, case, xhat))
    out = {}
    q = dp
    if s["w"] is not None:
        out["dweight"] = (dp * xhat).double().sum(0).float().view(-1)
        out["dbias"] = dp.double().sum(0).float().view(-1)
        q = dp * s["w"].view(case["G"], -1)
    if case["over"] == "token":
        mq, mqx = q.mean(2, keepdim=True), (q * xhat).mean(2, keepdim=True)
    else:
        seq = _seq_of(s)
        mq, mqx = _seq_means(s, q)[seq][:, :, None], _seq_means(s, q * xhat)[seq][:, :, None]
    out["dx"] = (rstd * (q - mq - xhat * mqx)).to(s["dy"].dtype).view(s["x"].shape)
    return out


def _norm_bwd_own(s, case):
    kw = _norm_kw(s, case)
    if case["over"] == "sequence":
        kw["stats"] = s["stats"]
    r = _kda().group_norm_bwd(s["x"], case["G"], s["dy"], **kw)
    return {k: v for k, v in r.items() if v is not None}


_RUN = {"scan_fwd": (_scan_fwd_plain, _scan_fwd_own), "scan_bwd": (_scan_bwd_plain, _scan_bwd_own),
        "scan_step": (_scan_step_plain, _scan_step_own), "norm_fwd": (_norm_fwd_plain, _norm_fwd_own),
        "norm_bwd": (_norm_bwd_plain, _norm_bwd_own)}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    op, es, C = case["op"], DTYPES[case["dtype"]].itemsize, case["C"]
    N = case["N"] if op == "scan_step" else case["seqs"]
    T = N if op == "scan_step" else sum(_lengths(case))
    rows = es * T * C
    if op.startswith("scan"):
        z, state = 1 if case["gate"] else 0, 4 * N * C
        if op == "scan_step":
            return {"bytes": (4 + z) * rows + 2 * state + 4 * C, "flops": T * C * (20 + 5 * z)}
        if op == "scan_fwd":
            return {"bytes": (4 + z) * rows + (2 if case["state"] else 1) * state + 4 * C, "flops": T * C * (20 + 5 * z)}
        kept = 4 * C * (-(-T // BLOCK)) if case["kept"] else 0
        return {"bytes": (7 + 2 * z) * rows + (3 if case["state"] else 0) * state + kept + 8 * C, "flops": T * C * (45 + 10 * z)}
    affine, act = 1 if case["affine"] else 0, 5 * case["act"]
    if op == "norm_fwd":
        return {"bytes": 2 * rows + 8 * C * affine, "flops": T * C * (7 + 2 * affine + act)}
    stats = 8 * N * case["G"] if case.get("kept") else 0
    return {"bytes": 3 * rows + 16 * C * affine + stats, "flops": T * C * (16 + 6 * affine + 2 * act)}


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    if case["op"] == "scan_step":
        return _exact_step(s)
    return _exact_scan(s, case) if case["op"].startswith("scan") else _exact_norm(s, case)


def _coefficients(s):
    """Exponent, decay, the input gate and the input's weight, in 64 bits."""
    e = DECAY * torch.logaddexp(s["lam"], torch.zeros_like(s["lam"])) * torch.sigmoid(s["r"])
    return e, torch.exp(-e), torch.sigmoid(s["i"]), (-torch.expm1(-2 * e)).sqrt()


def _exact_step(s):
    _, a, gi, m = _coefficients(s)
    h = s["state"].clone()
    at = s["slots"].long()
    h[at] = a * h[at] + m * gi * s["x"]
    y = h[at]
    return {"y": y if s["z"] is None else torch.nn.functional.silu(s["z"]) * y, "state": h}


def _exact_scan(s, case):
    """Token by token, all sequences of a case one after another."""
    C = case["C"]
    lead = s["x"].shape
    t = dict(s, **{k: s[k].reshape(-1, C) for k in ("x", "r", "i", "z", "dy") if s.get(k) is not None})
    offsets = s["offsets"].tolist()
    e, a, gi, m = _coefficients(t)
    u = m * gi * t["x"]
    h, finals, zero = torch.empty_like(u), [], u.new_zeros(C)
    for n, (b, end) in enumerate(zip(offsets, offsets[1:])):
        at = s["state"][n] if s["state"] is not None else zero
        for k in range(b, end):
            at = torch.addcmul(u[k], a[k], at, out=h[k])
        finals.append(at.clone())
    sz = None if s["z"] is None else torch.sigmoid(t["z"])
    if case["op"] == "scan_fwd":
        return {"y": (h if sz is None else h * t["z"] * sz).view(lead), "state": torch.stack(finals)}
    out = {}
    dh = t["dy"].clone()
    if sz is not None:
        out["dz"] = (dh * h * (sz + t["z"] * sz * (1 - sz))).view(lead)
        dh *= t["z"] * sz
    d0 = []
    before = torch.empty_like(h)
    for n, (b, end) in enumerate(zip(offsets, offsets[1:])):
        carry = s["dfinal"][n] if s["dfinal"] is not None else zero
        for k in range(end - 1, b - 1, -1):
            dh[k] += carry
            carry = a[k] * dh[k]
        d0.append(carry)
        before[b] = s["state"][n] if s["state"] is not None else 0.0
        before[b + 1:end] = h[b:end - 1]
    # d m / d e = e^-2e / m
    de = dh * gi * t["x"] * torch.exp(-2 * e) / m - dh * a * before
    sr = torch.sigmoid(t["r"])
    out["dx"], out["di"] = (dh * m * gi).view(lead), (dh * u * (1 - gi)).view(lead)
    out["dr"] = (de * e * (1 - sr)).view(lead)
    out["dlam"] = (de * DECAY * sr).sum(0) * torch.sigmoid(s["lam"])
    if s["state"] is not None:
        out["dinitial_state"] = torch.stack(d0)
    return out


def _exact_norm(s, case):
    """Sequence by sequence, or token by token (as rows of one view)."""
    G, C = case["G"], case["C"]
    flat = s["x"].reshape(-1, G, C // G)
    dy = s["dy"].reshape(flat.shape) if case["op"] == "norm_bwd" else None
    offsets, out = s["offsets"].tolist(), torch.empty_like(flat)
    dw, db = flat.new_zeros(G, C // G), flat.new_zeros(G, C // G)
    # pieces of whole statistics: a sequence, or a thousand tokens
    step = 1024
    spans = list(zip(offsets, offsets[1:])) if case["over"] == "sequence" else [(b, min(b + step, len(flat))) for b in range(0, len(flat), step)]
    dims = (0, 2) if case["over"] == "sequence" else (2,)
    for b, e in spans:
        x = flat[b:e]
        var, mean = torch.var_mean(x, dim=dims, correction=0, keepdim=True)
        xhat = (x - mean) / (var + EPS).sqrt()
        p = xhat if s["w"] is None else xhat * s["w"].view(G, -1) + s["b"].view(G, -1)
        sg = torch.sigmoid(p)
        if dy is None:
            out[b:e] = p * sg if case["act"] else p
            continue
        dp = dy[b:e] * (sg * (1 + p * (1 - sg))) if case["act"] else dy[b:e]
        dw += (dp * xhat).sum(0)
        db += dp.sum(0)
        q = dp if s["w"] is None else dp * s["w"].view(G, -1)
        out[b:e] = (q - q.mean(dims, keepdim=True) - xhat * (q * xhat).mean(dims, keepdim=True)) / (var + EPS).sqrt()
    if dy is None:
        return {"y": out.view(s["x"].shape)}
    res = {"dx": out.view(s["x"].shape)}
    if s["w"] is not None:
        res = {"dweight": dw.view(-1), "dbias": db.view(-1), **res}
    return res
