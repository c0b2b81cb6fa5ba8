"""Cases and plain forms of the recurrent layer's serving and training operators: the short
convolution, the selective state space scan, the decode steps on a pool of states, and the
pages of a cache.

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or calls the
framework (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NEVER_FULL = 1 << 30  # tokens of a page that holds a sequence's whole state


# ---- cases -------------------------------------------------------------------------------


def listed():
    return [
        # The short convolution of q, k or v of the 96 x 128 layer over a packed batch of prompts that carry on
        # from cached histories, its input a slice of the fused projection's rows.
        dict(name="conv_fwd_packed", op="conv_fwd", dtype="bf16", seqs=16, lo=512, hi=8192, C=12288, W=4, act=1, bias=False,
             history=True, wide=2),
        # The same layer's training step on one sequence.
        dict(name="conv_bwd_4096", op="conv_bwd", dtype="bf16", seqs=1, lo=4096, hi=4096, C=12288, W=4, act=1, bias=True,
             history=False, wide=1),
        # Decode: one token of 256 sequences, histories in a pool read by slot.
        dict(name="conv_step_256", op="conv_step", dtype="bf16", N=256, C=12288, W=4, act=1, bias=False, pool=300),
        # A long prompt of one sequence: few channels' worth of parallelism, so the time axis has to be split.
        dict(name="scan_fwd_long", op="scan_fwd", dtype="bf16", seqs=1, lo=16384, hi=16384, C=4096, S=16, G=1, gate=True,
             state=True),
        # Ragged packed prompts in 32 bits, odd channel count, two groups, a wider state.
        dict(name="scan_fwd_ragged_f32", op="scan_fwd", dtype="f32", seqs=7, lo=1, hi=700, C=1530, S=64, G=2, gate=True,
             state=True),
        # A training step: the gradients of everything, a batch of two sequences.
        dict(name="scan_bwd_2x2048", op="scan_bwd", dtype="bf16", seqs=2, lo=2048, hi=2048, C=4096, S=16, G=1, gate=True,
             state=False),
        # A single sequence's decode step: latency.
        dict(name="scan_step_1", op="scan_step", dtype="bf16", N=1, C=4096, S=16, G=1, gate=True, pool=8),
        # A full serving batch.
        dict(name="scan_step_512", op="scan_step", dtype="bf16", N=512, C=8192, S=16, G=1, gate=True, pool=600),
        # KDA decode of 256 sequences of the 96-head layer, states in a pool read by slot.
        dict(name="kda_step_256", op="kda_step", dtype="bf16", N=256, H=96, K=128, V=128, pool=288),
        # KDA decode of a few sequences of a small layer, in 32 bits.
        dict(name="kda_step_5_f32", op="kda_step", dtype="f32", N=5, H=6, K=64, V=64, pool=9),
        # One prompt's token pages forked into samples: full pages shared, the last one copied.
        dict(name="fork_samples", op="fork", dtype="bf16", parents=8, children=64, width=128, page_tokens=64, elems=65536,
             free=128),
        # Sequences end, the pool of 96-head layer states is closed up, and others are let in.
        dict(name="churn_states", op="churn", dtype="f32", rows=96, width=1, sets=4, elems=96 * 128 * 128, spare=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "kda_step",
                     "fork", "churn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv_fwd", "conv_bwd"):
        hi = _log_int(rng, 1, 8192)
        seqs = min(_log_int(rng, 1, 64), max(1, (65536 if dtype == "bf16" else 32768) // hi))
        return dict(op=op, dtype=dtype, seqs=seqs, lo=max(1, hi // 8), hi=hi, C=_log_int(rng, 64, 12288), W=rng.choice([2, 3, 4, 4]),
                    act=rng.choice([0, 1]), bias=rng.random() < 0.5, history=rng.random() < 0.5, wide=rng.choice([1, 2]))
    if op == "conv_step":
        N = _log_int(rng, 1, 1024)
        return dict(op=op, dtype=dtype, N=N, C=_log_int(rng, 64, 12288), W=rng.choice([2, 3, 4, 4]), act=rng.choice([0, 1]),
                    bias=rng.random() < 0.5, pool=N + _log_int(rng, 1, 64))
    if op in ("scan_fwd", "scan_bwd"):
        most = 16384 * 4096 * 16 if op == "scan_fwd" else 4096 * 4096 * 16
        S, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        C = G * _log_int(rng, 16, 8192 // G)
        hi = _log_int(rng, 1, max(2, min(8192, most // (C * S))))
        seqs = min(_log_int(rng, 1, 32), max(1, most // (C * S * hi)))
        return dict(op=op, dtype=dtype, seqs=seqs, lo=max(1, hi // 8), hi=hi, C=C, S=S, G=G, gate=rng.random() < 0.7,
                    state=rng.random() < 0.5)
    if op == "scan_step":
        N, S, G = _log_int(rng, 1, 1024), rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2])
        C = G * _log_int(rng, 32, 8192 // G)
        N = max(1, min(N, 512 * 8192 * 16 // (C * S)))
        return dict(op=op, dtype=dtype, N=N, C=C, S=S, G=G, gate=rng.random() < 0.7, pool=N + _log_int(rng, 1, 64))
    if op == "kda_step":
        K, V, H = rng.choice([64, 128]), rng.choice([64, 128]), _log_int(rng, 1, 96)
        N = _log_int(rng, 1, 256)
        return dict(op=op, dtype=dtype, N=N, H=H, K=K, V=V, pool=N + _log_int(rng, 1, 32))
    if op == "fork":
        parents, width = _log_int(rng, 1, 16), _log_int(rng, 1, 256)
        children = _log_int(rng, 1, 128)
        return dict(op=op, dtype=dtype, parents=parents, children=children, width=width, page_tokens=rng.choice([16, 64, 128, NEVER_FULL]),
                    elems=8 * _log_int(rng, 16, 16384), free=children + rng.randrange(32))
    sets, width = rng.choice([2, 3, 4, 8]), _log_int(rng, 1, 16)
    rows = sets * _log_int(rng, 1, 32)
    return dict(op="churn", dtype=dtype, rows=rows, width=width, sets=sets, elems=8 * _log_int(rng, 16, 16384),
                spare=_log_int(rng, 1, 64))


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
    op = case["op"]

    def rn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def pick(n, most):
        return torch.randperm(most, generator=g, device=dev)[:n].to(torch.int32)

    s = {"case": case}
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        s["w"] = rn(C, W, std=0.5)
        s["bias"] = rn(C, std=0.1) if case["bias"] else None
        if op == "conv_step":
            s["x"] = rn(case["N"], C).to(dt)
            s["hist"] = rn(case["pool"], W - 1, C).to(dt)
            s["slots"] = pick(case["N"], case["pool"])
            return s
        lens = _lengths(case)
        T, N = sum(lens), len(lens)
        s["x"] = rn(1, T, case["wide"] * C).to(dt)[:, :, :C]
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device=dev)
        s["hist"] = rn(N, W - 1, C).to(dt) if case["history"] else None
        if op == "conv_bwd":
            s["dy"] = rn(1, T, C).to(dt)
            s["dfinal"] = rn(N, W - 1, C).to(dt) if case["history"] else None
        return s
    if op.startswith("scan"):
        C, S, G = case["C"], case["S"], case["G"]
        # the usual initialisation of such layers: decay rates 1..S, step sizes spread over 0.001..0.1 by a bias
        s["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32).repeat(C, 1) * torch.exp(rn(C, S, std=0.1))
        step = torch.exp(torch.rand(C, generator=g, device=dev) * math.log(100.0) + math.log(0.001))
        s["bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1.0 + rn(C, std=0.1)
        if op == "scan_step":
            N = case["N"]
            lead = (N,)
            s["state"] = rn(case["pool"], C, S, std=0.2)
            s["slots"] = pick(N, case["pool"])
        else:
            lens = _lengths(case)
            T, N = sum(lens), len(lens)
            lead = (1, T)
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device=dev)
            s["state"] = rn(N, C, S, std=0.2) if case["state"] else None
        s["u"] = rn(*lead, C).to(dt)
        s["delta"] = rn(*lead, C, std=0.5).to(dt)
        # the input and output vectors lie side by side in one projection's rows
        bc = rn(*lead, 2, G, S).to(dt)
        s["B"], s["C"] = bc[..., 0, :, :], bc[..., 1, :, :]
        s["z"] = rn(*lead, C).to(dt) if case["gate"] else None
        if op == "scan_bwd":
            s["dy"] = rn(*lead, C).to(dt)
            s["dfinal"] = rn(N, C, S) if case["state"] else None
        return s
    if op == "kda_step":
        N, H, K, V = case["N"], case["H"], case["K"], case["V"]
        unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
        s["q"], s["k"], s["v"] = unit(rn(N, H, K)).to(dt), unit(rn(N, H, K)).to(dt), rn(N, H, V).to(dt)
        s["g"] = (-torch.log1p(torch.exp(rn(N, H, K)))).clamp(min=-5.0).to(dt)
        s["beta"] = torch.sigmoid(rn(N, H)).to(dt)
        s["state"] = rn(case["pool"], H, K, V, std=0.02)
        s["slots"] = pick(N, case["pool"])
        return s
    if op == "fork":
        n, m, width = case["parents"], case["children"], case["width"]
        pages = n * width + case["free"]
        s["tables"] = torch.full((n + m, width), -1, dtype=torch.int32, device=dev)
        s["tables"][:n] = pick(n * width, pages).view(n, width)
        most = min(width * case["page_tokens"], (1 << 31) - 1)
        if case["page_tokens"] == NEVER_FULL:
            most = NEVER_FULL - 1
        s["lens"] = torch.zeros(n + m, dtype=torch.int32, device=dev)
        s["lens"][:n] = torch.randint(max(1, most // 2), most + 1, (n,), generator=g, device=dev).to(torch.int32)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["refs"][s["tables"][:n].reshape(-1).long()] = 1
        s["from"] = torch.randint(0, n, (m,), generator=g, device=dev).to(torch.int32)
        s["to"] = (n + torch.randperm(m, generator=g, device=dev)).to(torch.int32)
        s["pool"] = rn(pages, case["elems"]).to(dt)
        return s
    rows, width = case["rows"], case["width"]
    pages = rows * width + case["spare"]
    s["tables"] = pick(rows * width, pages).view(rows, width)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
    s["refs"][s["tables"].reshape(-1).long()] = 1
    s["sets"] = torch.randperm(rows, generator=g, device=dev).view(case["sets"], -1)
    s["pool"] = rn(pages, case["elems"]).to(dt)
    s["turn"] = 0
    return s


# ---- one pass ----------------------------------------------------------------------------


def run(s):
    case = s["case"]
    return _RUN[case["op"]][1 if own else 0](s, case)


def _kda():
    import kimi_delta_attention_chunk_gb300 as kda
    return kda


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _dsilu(x):
    e = 1.0 / (1.0 + torch.exp(-x))
    return e * (1.0 + x * (1.0 - e))


# the short convolution: every sequence's history laid before its tokens in one stream


def _conv_stream(s, case, x):
    W, C = case["W"], case["C"]
    cu = s["cu"].long()
    N, T = cu.numel() - 1, x.shape[0]
    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    at = t + (seq + 1) * (W - 1)
    before = (cu[:-1] + torch.arange(N, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    e = torch.zeros(T + N * (W - 1), C, device=x.device)
    e[at] = x
    if s["hist"] is not None:
        e[before] = s["hist"].float()
    after = (cu[1:] + torch.arange(1, N + 1, device=x.device) * (W - 1))[:, None] + torch.arange(-(W - 1), 0, device=x.device)
    return e, at, before, after


def _conv_pre(s, case, e, at):
    W, w = case["W"], s["w"]
    p = sum(e[at - (W - 1) + j] * w[:, j] for j in range(W))
    return p if s["bias"] is None else p + s["bias"]


def _conv_fwd_plain(s, case):
    dt = DTYPES[case["dtype"]]
    e, at, _, after = _conv_stream(s, case, s["x"][0].float())
    p = _conv_pre(s, case, e, at)
    y = _silu(p) if case["act"] else p
    return {"y": y.to(dt)[None], "final": e[after].to(dt)}


def _conv_fwd_own(s, case):
    y, final = _kda().short_conv_fwd(s["x"], s["w"], bias=s["bias"], conv_act=case["act"], initial=s["hist"], cu_seqlens=s["cu"])
    return {"y": y, "final": final}


def _conv_bwd_plain(s, case):
    dt, W = DTYPES[case["dtype"]], case["W"]
    e, at, before, after = _conv_stream(s, case, s["x"][0].float())
    dp = s["dy"][0].float()
    if case["act"]:
        dp = dp * _dsilu(_conv_pre(s, case, e, at))
    de = torch.zeros_like(e)
    if s["dfinal"] is not None:
        de[after] = s["dfinal"].float()
    de = sum((de.index_add(0, at - (W - 1) + j, dp * s["w"][:, j]) if j == 0 else
              torch.zeros_like(e).index_add_(0, at - (W - 1) + j, dp * s["w"][:, j])) for j in range(W))
    dw = torch.stack([(dp * e[at - (W - 1) + j]).sum(0) for j in range(W)], dim=1)
    out = {"dx": de[at].to(dt)[None], "dweight": dw}
    if s["bias"] is not None:
        out["dbias"] = dp.sum(0)
    if s["hist"] is not None:
        out["dinitial"] = de[before].to(dt)
    return out


def _conv_bwd_own(s, case):
    r = _kda().short_conv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], conv_act=case["act"], initial=s["hist"], cu_seqlens=s["cu"],
                              dfinal=s["dfinal"])
    return {k: r[k] for k in ("dx", "dweight", "dbias", "dinitial") if r[k] is not None}


def _conv_step_plain(s, case):
    dt, slots = DTYPES[case["dtype"]], s["slots"].long()
    e = torch.cat([s["hist"][slots], s["x"][:, None]], dim=1)
    p = (e.float() * s["w"].t()).sum(1)
    p = p if s["bias"] is None else p + s["bias"]
    s["hist"][slots] = e[:, 1:]
    return {"y": (_silu(p) if case["act"] else p).to(dt), "history": s["hist"]}


def _conv_step_own(s, case):
    y = _kda().short_conv_step(s["x"], s["hist"], s["w"], bias=s["bias"], conv_act=case["act"], slots=s["slots"])
    return {"y": y, "history": s["hist"]}


# the selective scan


def _scan_inputs(s, case):
    """Step sizes, inputs and the group vectors spread over the channels, in 32 bits, one flat stream."""
    C, S, G = case["C"], case["S"], case["G"]
    raw = s["delta"].reshape(-1, C).float() + s["bias"]
    d = raw.clamp(min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    u = s["u"].reshape(-1, C).float()
    spread = lambda x: x.reshape(-1, G, S).float().repeat_interleave(C // G, dim=1)  # noqa: E731
    return d, u, spread(s["B"]), spread(s["C"])


def _affine_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, in log2(T) doublings."""
    step = 1
    while step < b.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _scan_states(s, d, u, Bx):
    """Decays and states after every token, and the state before every sequence's first token."""
    cu = s["cu"].long()
    a = torch.exp(d[:, :, None] * s["A"])
    b = (d * u)[:, :, None] * Bx
    first = torch.zeros(a.shape[0], dtype=torch.bool, device=a.device).index_fill_(0, cu[:-1], True)
    if s["state"] is not None:
        b.index_add_(0, cu[:-1], a[cu[:-1]] * s["state"])
    h = _affine_scan(a.masked_fill(first[:, None, None], 0.0), b)
    return a, h, first


def _scan_fwd_plain(s, case):
    d, u, Bx, Cx = _scan_inputs(s, case)
    _, h, _ = _scan_states(s, d, u, Bx)
    y = (h * Cx).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"][0].float())
    return {"y": y.to(DTYPES[case["dtype"]])[None], "state": h[s["cu"].long()[1:] - 1]}


def _scan_fwd_own(s, case):
    y, state = _kda().ssm_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], delta_bias=s["bias"],
                                   softplus=True, initial_state=s["state"], cu_seqlens=s["cu"])
    return {"y": y, "state": state}


def _scan_bwd_plain(s, case):
    dt, C, S, G = DTYPES[case["dtype"]], case["C"], case["S"], case["G"]
    cu = s["cu"].long()
    d, u, Bx, Cx = _scan_inputs(s, case)
    a, h, first = _scan_states(s, d, u, Bx)
    dout = s["dy"][0].float()
    out = {}
    if s["z"] is not None:
        z = s["z"][0].float()
        y = (h * Cx).sum(-1) + s["D"] * u
        out["dz"] = (dout * y * _dsilu(z)).to(dt)[None]
        dout = dout * _silu(z)
    g = dout[:, :, None] * Cx
    if s["dfinal"] is not None:
        g[cu[1:] - 1] += s["dfinal"]
    last = torch.zeros_like(first).index_fill_(0, cu[1:] - 1, True)
    onward = torch.cat([a[1:], a[:1]]).masked_fill(last[:, None, None], 0.0)
    dh = _affine_scan(onward.flip(0), g.flip(0)).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[cu[:-1]] = 0.0 if s["state"] is None else s["state"]
    ah = dh * a * before
    q1, q2 = (dh * Bx).sum(-1), (ah * s["A"]).sum(-1)
    raw = s["delta"][0].float() + s["bias"]
    ddelta = (q2 + u * q1) / (1.0 + torch.exp(-raw))
    out["du"] = (d * q1 + s["D"] * dout).to(dt)[None]
    out["ddelta"] = ddelta.to(dt)[None]
    out["dA"] = (ah * d[:, :, None]).sum(0)
    out["dB"] = (dh * (d * u)[:, :, None]).view(-1, G, C // G, S).sum(2).to(dt)[None]
    out["dC"] = (h * dout[:, :, None]).view(-1, G, C // G, S).sum(2).to(dt)[None]
    out["dD"] = (dout * u).sum(0)
    out["ddelta_bias"] = ddelta.sum(0)
    if s["state"] is not None:
        out["dinitial_state"] = (a * dh)[cu[:-1]]
    return out


def _scan_bwd_own(s, case):
    r = _kda().ssm_scan_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dy"], D=s["D"], z=s["z"], delta_bias=s["bias"],
                            softplus=True, initial_state=s["state"], cu_seqlens=s["cu"], dfinal_state=s["dfinal"])
    return {k: v for k, v in r.items() if v is not None}


def _scan_step_plain(s, case):
    slots = s["slots"].long()
    d, u, Bx, Cx = _scan_inputs(s, case)
    h = torch.exp(d[:, :, None] * s["A"]) * s["state"][slots] + (d * u)[:, :, None] * Bx
    s["state"][slots] = h
    y = (h * Cx).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(DTYPES[case["dtype"]]), "state": s["state"]}


def _scan_step_own(s, case):
    y = _kda().ssm_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"], delta_bias=s["bias"],
                        softplus=True, slots=s["slots"])
    return {"y": y, "state": s["state"]}


# KDA decode on the pool


def _kda_step_plain(s, case):
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    slots = s["slots"].long()
    S = s["state"][slots] * torch.exp(g)[..., None]
    delta = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * delta[..., None, :]
    s["state"][slots] = S
    return {"o": case["K"] ** -0.5 * (S * q[..., None]).sum(-2), "state": s["state"]}


def _kda_step_own(s, case):
    o = _kda().recurrent_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
    return {"o": o, "state": s["state"]}


# pages: a page with no references is free, and the lowest free pages are given out first


def _free_plain(refs, pages):
    pages = pages.reshape(-1).long()
    refs.index_add_(0, pages.clamp(min=0), -(pages >= 0).to(torch.int32))
    refs.clamp_(min=0)


def _free_pages(refs, n):
    """The n lowest free pages, -1 where there are none left."""
    order = torch.argsort((refs != 0).to(torch.uint8), stable=True)[:n]
    return torch.where(refs[order] == 0, order, -1)


def _copy_plain(pool, src, dst):
    at = dst >= 0
    pool[dst[at].long()] = pool[src[at].long()]


def _fork_plain(s, case):
    tables, lens, refs, tokens = s["tables"], s["lens"], s["refs"], case["page_tokens"]
    frm, to = s["from"].long(), s["to"].long()
    _free_plain(refs, tables[to])
    size = lens[frm]
    full, part = size // tokens, size % tokens != 0
    col = torch.arange(case["width"], device=refs.device)
    rows = torch.where(col < full[:, None], tables[frm], -1)
    got = _free_pages(refs, frm.numel()).to(torch.int32)
    rank = part.long().cumsum(0) - 1
    new = torch.where(part, got[rank.clamp(min=0)], -1).to(torch.int32)
    old = torch.where(part, tables[frm].gather(1, full.long().clamp(max=case["width"] - 1)[:, None])[:, 0], -1)
    rows = torch.where((col == full[:, None]) & part[:, None], new[:, None], rows)
    refs.index_add_(0, rows.reshape(-1).long().clamp(min=0), (rows >= 0).reshape(-1).to(torch.int32))
    tables[to] = rows
    lens[to] = size
    _copy_plain(s["pool"], old, new)
    return {"src": old, "dst": new, "tables": tables, "lens": lens, "refs": refs, "pool": s["pool"]}


def _fork_own(s, case):
    kda = _kda()
    kda.pages_free(s["refs"], s["tables"][s["to"].long()])
    src, dst = kda.pages_fork(s["tables"], s["lens"], s["refs"], s["from"], s["to"], case["page_tokens"])
    kda.pages_copy(s["pool"], src, dst)
    return {"src": src, "dst": dst, "tables": s["tables"], "lens": s["lens"], "refs": s["refs"], "pool": s["pool"]}


def _churn_plain(s, case):
    tables, refs = s["tables"], s["refs"]
    gone = s["sets"][s["turn"] % case["sets"]]
    s["turn"] += 1
    _free_plain(refs, tables[gone])
    tables[gone] = -1
    # closing up: the used pages behind the number of used pages move into the holes before it, both in order
    P = refs.numel()
    at, used = torch.arange(P, device=refs.device), refs != 0
    live = used.sum()
    hole, tail = ~used & (at < live), used & (at >= live)
    src = torch.argsort((~tail).to(torch.uint8), stable=True)[: P // 2]
    dst = torch.argsort((~hole).to(torch.uint8), stable=True)[: P // 2]
    move = torch.arange(P // 2, device=refs.device) < hole.sum()
    src, dst = torch.where(move, src, -1).to(torch.int32), torch.where(move, dst, -1).to(torch.int32)
    place = torch.cat([at, at[:1]]).index_copy_(0, torch.where(move, src, P).long(), dst.long())
    tables.copy_(torch.where(tables >= 0, place[tables.long().clamp(min=0)], -1))
    count = torch.cat([refs, refs[:1]])
    count = count.index_copy(0, torch.where(move, dst, P).long(), count[src.long()]).index_fill(0, torch.where(move, src, P).long(), 0)
    refs.copy_(count[:P])
    _copy_plain(s["pool"], src, dst)
    new = _free_pages(refs, gone.numel() * case["width"])
    refs[new] = 1
    tables[gone] = new.to(torch.int32).view(-1, case["width"])
    return {"src": src, "dst": dst, "tables": tables, "refs": refs, "pool": s["pool"]}


def _churn_own(s, case):
    kda = _kda()
    gone = s["sets"][s["turn"] % case["sets"]]
    s["turn"] += 1
    kda.pages_free(s["refs"], s["tables"][gone])
    s["tables"][gone] = -1
    src, dst = kda.pages_compact(s["refs"], s["tables"])
    kda.pages_copy(s["pool"], src, dst)
    s["tables"][gone] = kda.pages_alloc(s["refs"], gone.numel() * case["width"]).view(-1, case["width"])
    return {"src": src, "dst": dst, "tables": s["tables"], "refs": s["refs"], "pool": s["pool"]}


_RUN = {"conv_fwd": (_conv_fwd_plain, _conv_fwd_own), "conv_bwd": (_conv_bwd_plain, _conv_bwd_own),
        "conv_step": (_conv_step_plain, _conv_step_own), "scan_fwd": (_scan_fwd_plain, _scan_fwd_own),
        "scan_bwd": (_scan_bwd_plain, _scan_bwd_own), "scan_step": (_scan_step_plain, _scan_step_own),
        "kda_step": (_kda_step_plain, _kda_step_own), "fork": (_fork_plain, _fork_own), "churn": (_churn_plain, _churn_own)}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    op, es = case["op"], DTYPES[case["dtype"]].itemsize
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        N = case["N"] if op == "conv_step" else case["seqs"]
        T = N if op == "conv_step" else sum(_lengths(case))
        small = 4 * C * (W + (1 if case["bias"] else 0))
        hist = es * N * (W - 1) * C
        if op == "conv_fwd":
            return {"bytes": 2 * es * T * C + small + hist * (2 if case["history"] else 1), "flops": T * C * (2 * W + 4)}
        if op == "conv_step":
            return {"bytes": 2 * es * T * C + small + 2 * hist, "flops": T * C * (2 * W + 4)}
        return {"bytes": 3 * es * T * C + 2 * small + hist * (3 if case["history"] else 0), "flops": T * C * (6 * W + 10)}
    if op.startswith("scan"):
        C, S, G = case["C"], case["S"], case["G"]
        N = case["N"] if op == "scan_step" else case["seqs"]
        T = N if op == "scan_step" else sum(_lengths(case))
        rows, vec, z = es * T * C, es * T * G * S, 1 if case["gate"] else 0
        small, state = 4 * C * (S + 2), 4 * N * C * S
        if op == "scan_bwd":
            return {"bytes": (5 + 2 * z) * rows + 4 * vec + 2 * small + (3 * state if case["state"] else 0),
                    "flops": T * C * (22 * S + 20)}
        kept = 2 if op == "scan_step" or case["state"] else 1
        return {"bytes": (3 + z) * rows + 2 * vec + small + kept * state, "flops": T * C * (7 * S + 14)}
    if op == "kda_step":
        N, H, K, V = case["N"], case["H"], case["K"], case["V"]
        return {"bytes": N * H * (8 * K * V + es * (3 * K + V + 1) + 4 * V), "flops": N * H * (7 * K * V + 4 * V)}
    page = es * case["elems"]
    if op == "fork":
        n, m, width = case["parents"], case["children"], case["width"]
        pages = n * width + case["free"]
        return {"bytes": 2 * m * page + 8 * pages + 4 * width * (min(n, m) + 2 * m) + 28 * m, "flops": pages}
    gone = case["rows"] // case["sets"] * case["width"]
    pages = case["rows"] * case["width"] + case["spare"]
    # in the steady turn the leaving pages' holes are filled from the tail
    return {"bytes": 2 * gone * page + 8 * pages + 8 * case["rows"] * case["width"] + 8 * (pages // 2) + 8 * gone, "flops": pages}


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "churn"):  # copies and whole numbers: nothing is computed
        return None
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    return {"conv_fwd": _exact_conv, "conv_bwd": _exact_conv, "conv_step": _exact_conv_step, "scan_fwd": _exact_scan,
            "scan_bwd": _exact_scan, "scan_step": _exact_scan_step, "kda_step": _exact_kda_step}[op](s, case)


def _exact_conv(s, case):
    """Sequence by sequence."""
    W, C, cu = case["W"], case["C"], s["cu"].tolist()
    x = s["x"][0]
    if x.numel() > 1 << 28:  # in pieces of the channels, for the memory
        half = C // 2
        parts = []
        for a, b in ((0, half), (half, C)):
            t = dict(s, x=s["x"][:, :, a:b], w=s["w"][a:b], bias=None if s["bias"] is None else s["bias"][a:b])
            for n in ("hist", "dfinal", "dy"):
                if s.get(n) is not None:
                    t[n] = s[n][..., a:b]
            parts.append(_exact_conv(t, dict(case, C=b - a)))
        cat = {"dweight": 0, "dbias": 0}
        return {k: torch.cat([p[k] for p in parts], dim=cat.get(k, -1)) for k in parts[0]}
    bwd = case["op"] == "conv_bwd"
    y, final, dx, dinit = torch.empty_like(x), [], torch.empty_like(x), []
    dw, db = torch.zeros_like(s["w"]), x.new_zeros(C)
    for n, (b, e) in enumerate(zip(cu, cu[1:])):
        L = e - b
        past = s["hist"][n] if s["hist"] is not None else x.new_zeros(W - 1, C)
        line = torch.cat([past, x[b:e]])
        p = x.new_zeros(L, C) if s["bias"] is None else s["bias"].expand(L, C).clone()
        for j in range(W):
            p += line[j:j + L] * s["w"][:, j]
        if not bwd:
            y[b:e] = p * torch.sigmoid(p) if case["act"] else p
            final.append(line[L:])
            continue
        dp = s["dy"][0, b:e]
        if case["act"]:
            sg = torch.sigmoid(p)
            dp = dp * (sg + p * sg * (1 - sg))
        dline = torch.zeros_like(line)
        if s["dfinal"] is not None:
            dline[L:] += s["dfinal"][n]
        for j in range(W):
            dline[j:j + L] += dp * s["w"][:, j]
            dw[:, j] += (dp * line[j:j + L]).sum(0)
        db += dp.sum(0)
        dx[b:e] = dline[W - 1:]
        dinit.append(dline[:W - 1])
    if not bwd:
        return {"y": y[None], "final": torch.stack(final)}
    out = {"dx": dx[None], "dweight": dw}
    if s["bias"] is not None:
        out["dbias"] = db
    if s["hist"] is not None:
        out["dinitial"] = torch.stack(dinit)
    return out


def _exact_conv_step(s, case):
    slots = s["slots"].tolist()
    hist, ys = s["hist"], []
    for i, n in enumerate(slots):
        p = s["x"][i] * s["w"][:, -1] + (hist[n] * s["w"][:, :-1].t()).sum(0)
        p = p if s["bias"] is None else p + s["bias"]
        ys.append(p * torch.sigmoid(p) if case["act"] else p)
        hist[n] = torch.cat([hist[n][1:], s["x"][i:i + 1]])
    return {"y": torch.stack(ys), "history": hist}


def _exact_scan(s, case):
    """Token by token."""
    C, S, G = case["C"], case["S"], case["G"]
    bwd = case["op"] == "scan_bwd"
    cu = s["cu"].tolist()
    T = cu[-1]
    if (T + 1) * C * S * 8 > 60e9 and bwd:
        return None
    d = torch.nn.functional.softplus(s["delta"][0] + s["bias"], threshold=200.0)
    u, A = s["u"][0], s["A"]
    group = torch.arange(C, device=u.device) // (C // G)
    Bs, Cs = s["B"][0], s["C"][0]
    y = torch.empty_like(u)
    states = u.new_empty(T, C, S) if bwd else None
    finals, zero = [], u.new_zeros(C, S)
    for n, (b, e) in enumerate(zip(cu, cu[1:])):
        h = s["state"][n] if s["state"] is not None else zero
        for t in range(b, e):
            h = torch.exp(d[t, :, None] * A) * h + (d[t] * u[t])[:, None] * Bs[t][group]
            y[t] = (h * Cs[t][group]).sum(-1)
            if bwd:
                states[t] = h
        finals.append(h)
    y += s["D"] * u
    sz = torch.sigmoid(s["z"][0]) if s["z"] is not None else None
    if not bwd:
        return {"y": (y if sz is None else y * s["z"][0] * sz)[None], "state": torch.stack(finals)}
    dout = s["dy"][0]
    out = {}
    if sz is not None:
        out["dz"] = (dout * y * (sz + s["z"][0] * sz * (1 - sz)))[None]
        dout = dout * s["z"][0] * sz
    du, dd, dA = s["D"] * dout, torch.empty_like(u), torch.zeros_like(A)
    dB, dC, d0 = torch.zeros_like(Bs), torch.zeros_like(Cs), []
    for n, (b, e) in enumerate(zip(cu, cu[1:])):
        carry = s["dfinal"][n] if s["dfinal"] is not None else zero
        for t in range(e - 1, b - 1, -1):
            before = states[t - 1] if t > b else s["state"][n] if s["state"] is not None else zero
            dh = carry + Cs[t][group] * dout[t, :, None]
            a = torch.exp(d[t, :, None] * A)
            through = dh * a * before
            q = (dh * Bs[t][group]).sum(-1)
            du[t] += d[t] * q
            dd[t] = (through * A).sum(-1) + u[t] * q
            dA += through * d[t, :, None]
            dB[t] = (dh * (d[t] * u[t])[:, None]).view(G, C // G, S).sum(1)
            dC[t] = (states[t] * dout[t, :, None]).view(G, C // G, S).sum(1)
            carry = a * dh
        d0.append(carry)
    ddelta = dd * torch.sigmoid(s["delta"][0] + s["bias"])
    out.update(du=du[None], ddelta=ddelta[None], dA=dA, dB=dB[None], dC=dC[None], dD=(dout * u).sum(0), ddelta_bias=ddelta.sum(0))
    if s["state"] is not None:
        out["dinitial_state"] = torch.stack(d0)
    return out


def _exact_scan_step(s, case):
    C, G = case["C"], case["G"]
    group = torch.arange(C, device=s["u"].device) // (C // G)
    ys = []
    for i, n in enumerate(s["slots"].tolist()):
        d = torch.nn.functional.softplus(s["delta"][i] + s["bias"], threshold=200.0)
        h = torch.exp(d[:, None] * s["A"]) * s["state"][n] + (d * s["u"][i])[:, None] * s["B"][i][group]
        s["state"][n] = h
        y = (h * s["C"][i][group]).sum(-1) + s["D"] * s["u"][i]
        ys.append(y if s["z"] is None else y * s["z"][i] * torch.sigmoid(s["z"][i]))
    return {"y": torch.stack(ys), "state": s["state"]}


def _exact_kda_step(s, case):
    os = []
    for i, n in enumerate(s["slots"].tolist()):
        S = torch.exp(s["g"][i])[..., None] * s["state"][n]
        kS = torch.einsum("hk,hkv->hv", s["k"][i], S)
        S = S - torch.einsum("h,hk,hv->hkv", s["beta"][i], s["k"][i], kS - s["v"][i])
        s["state"][n] = S
        os.append(case["K"] ** -0.5 * torch.einsum("hk,hkv->hv", s["q"][i], S))
    return {"o": torch.stack(os), "state": s["state"]}
