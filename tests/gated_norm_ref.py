"""Plain 64-bit forms of the gated linear recurrence and the group norm (numpy, written from the formulas), each value with
the error that its 32-bit kernel may have.

Gated recurrence.  e^-v by the special-function unit is off by 2^-22 relative and |v| 2^-23 for its rounded exponent, a reciprocal by
2^-23: a sigmoid by 2^-20 + |v| 2^-22.  rate = decay softplus(lam) comes from the accurate functions: 2^-21.  So s = rate sigmoid(r) is
off by ds = 2^-19 + |r| 2^-22, a = e^-s by da = 2^-21 + s ds.  m = sqrt(1 - a^2): below s = 1/4 a product of s, a and a series, above it a
difference of which a^2 / m^2 <= 1.6 times a's error stays: dm = ds + 2 da + 2^-20 covers either.  Errors follow the recurrences: a state adds
|a h| da, |u| du and 2^-22 |h| for its roundings (one a token, and fewer than one a token for the folded maps).

Group norm.  A mean over a token's group is a sum of at most 16 values a lane and 10 levels: k = 32 roundings of 2^-24 of the mean
magnitude.  Over a sequence the joins of a thread's rows count too (a run's tokens / 32), and the last sum's terms a thread: k as given.  The
variance is summed around that mean: off by k 2^-22 relative, and the mean's error squared."""
import numpy as np

from tests.layer_ref import dsilu, f64, half_step, silu, softplus  # noqa: F401


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def soft(v):
    """Relative error of a sigmoid at v."""
    return 2.0 ** -20 + np.abs(v) * 2.0 ** -22


def gated(x, r, i, lam, decay, z, initial, cu, dy=None, dfinal=None):
    """x, r, i, z [T, C]; lam [C].  A dict: y, state, before (the state before every token, zeros at a sequence's first), and with
    dy the gradients; each with name + "_err"."""
    T, C = x.shape
    N = len(cu) - 1
    rate, sr, si = decay * softplus(lam), sigmoid(r), sigmoid(i)
    s = rate * sr
    a, m = np.exp(-s), np.sqrt(-np.expm1(-2 * s))
    u = m * si * x
    ds = 2.0 ** -19 + np.abs(r) * 2.0 ** -22
    da = 2.0 ** -21 + s * ds
    dm = ds + 2 * da + 2.0 ** -20
    du = dm + soft(i) + 2.0 ** -22
    sz = np.ones_like(x) if z is None else silu(z)
    dsz = 0 if z is None else soft(z)
    h, eh, hp, ehp = (np.zeros((T, C)) for _ in range(4))
    out = {"state": np.zeros((N, C)), "state_err": np.zeros((N, C)), "before": np.zeros((T, C)), "before_err": np.zeros((T, C))}
    for n in range(N):
        v = np.zeros(C) if initial is None else initial[n]
        e = np.zeros(C)
        for t in range(cu[n], cu[n + 1]):
            hp[t], ehp[t] = v, e
            if t > cu[n]:
                out["before"][t], out["before_err"][t] = v, e
            e = a[t] * e + np.abs(a[t] * v) * da[t] + np.abs(u[t]) * du[t]
            v = a[t] * v + u[t]
            e = e + 2.0 ** -22 * np.abs(v)
            h[t], eh[t] = v, e
        out["state"][n], out["state_err"][n] = v, e
    out["y"], out["y_err"] = h * sz, eh * np.abs(sz) + np.abs(h * sz) * (dsz + 2.0 ** -23)
    if dy is None:
        return out
    g, eg = np.zeros((T, C)), np.zeros((T, C))
    out["dinitial_state"], out["dinitial_state_err"] = np.zeros((N, C)), np.zeros((N, C))
    yb = dy * sz
    eyb = np.abs(yb) * (dsz + 2.0 ** -22)
    for n in range(N):
        v = np.zeros(C) if dfinal is None else dfinal[n]
        e = np.zeros(C)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            g[t] = yb[t] + v
            eg[t] = eyb[t] + e + 2.0 ** -22 * (np.abs(g[t]) + np.abs(v))
            v, e = a[t] * g[t], a[t] * eg[t] + np.abs(a[t] * g[t]) * da[t]
        out["dinitial_state"][n], out["dinitial_state_err"][n] = v, e + 2.0 ** -23 * np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        wm = np.where(m > 0, si * x * a * a / m, 0.0)
    dwm = soft(i) + 2 * da + dm + 2.0 ** -20
    de = g * (wm - a * hp)
    ede = eg * np.abs(wm - a * hp) + np.abs(g) * (np.abs(wm) * dwm + a * (ehp + np.abs(hp) * da) + 2.0 ** -22 * (np.abs(wm) + np.abs(a * hp)))
    out["dx"], out["dx_err"] = g * m * si, eg * m * si + np.abs(g * m * si) * (dm + soft(i) + 2.0 ** -22)
    ci = 1 - si
    out["di"] = g * u * ci
    out["di_err"] = eg * np.abs(u) * ci + np.abs(g * u) * (si * soft(i) + 2.0 ** -23) + np.abs(out["di"]) * (du + 2.0 ** -22)
    out["dr"] = de * s * (1 - sr)
    out["dr_err"] = ede * s * (1 - sr) + np.abs(de) * s * (sr * soft(r) + 2.0 ** -23) + np.abs(out["dr"]) * (soft(r) + 2.0 ** -20)
    slope = decay * sigmoid(lam)
    part, epart = de * sr, ede * sr + np.abs(de * sr) * (soft(r) + T * 2.0 ** -24)
    inside = np.zeros(T, bool)
    inside[cu[0]:cu[-1]] = True
    out["dlam"] = slope * part[inside].sum(0)
    out["dlam_err"] = slope * epart[inside].sum(0) + np.abs(out["dlam"]) * 2.0 ** -20
    if z is not None:
        sg = sigmoid(z)
        out["dz"] = dy * h * dsilu(z)
        size = sg + np.abs(z) * sg * (1 - sg)
        out["dz_err"] = np.abs(dy) * (eh * np.abs(dsilu(z)) + np.abs(h) * (size * (2 * soft(z) + 2.0 ** -21) + np.abs(z) * sg * sg * soft(z)))
    return out


def norm(x, G, w, b, eps, act, spans, over, k, dy=None):
    """x [T, C]; spans: (first, one behind the last) token of every sequence; over: "token" or "sequence"; k: roundings of a sum.  A dict: y, or
    with dy dx, dweight, dbias; stats over sequences; each with name + "_err"."""
    T, C = x.shape
    cg = C // G
    out = {"y": np.zeros((T, G, cg)), "y_err": np.zeros((T, G, cg)), "dx": np.zeros((T, G, cg)), "dx_err": np.zeros((T, G, cg)), "stats": []}
    sums = {n: np.zeros((G, cg)) for n in ("dweight", "dweight_err", "dbias", "dbias_err", "n")}
    w1 = np.ones(C) if w is None else w
    w1, b1 = w1.reshape(G, cg), (np.zeros(C) if b is None else b).reshape(G, cg)
    dims = (2,) if over == "token" else (0, 2)
    for first, last in spans:
        if first == last:
            out["stats"].append(np.stack([np.zeros(G), np.full(G, eps ** -0.5)], -1))
            continue
        v = x[first:last].reshape(-1, G, cg)
        mean = v.mean(dims, keepdims=True)
        em = k * 2.0 ** -23 * np.abs(v).mean(dims, keepdims=True) + 2.0 ** -23 * np.abs(mean)
        var = ((v - mean) ** 2).mean(dims, keepdims=True)
        rstd = 1 / np.sqrt(var + eps)
        dr = (k * 2.0 ** -22 * var + em ** 2 + (2.0 ** -22 * np.abs(v) * np.abs(v - mean)).mean(dims, keepdims=True)) * rstd ** 2 / 2 + 2.0 ** -21
        if over == "sequence":
            out["stats"].append(np.stack([mean.reshape(G), rstd.reshape(G)], -1))
        xh = (v - mean) * rstd
        exh = (em + 2.0 ** -23 * np.abs(v - mean)) * rstd + np.abs(xh) * dr
        p = xh * w1 + b1
        ep = np.abs(w1) * exh + 2.0 ** -22 * (np.abs(xh * w1) + np.abs(b1))
        at = slice(first, last)
        if dy is None:
            out["y"][at] = silu(p) if act else p
            out["y_err"][at] = (1.1 * ep + np.abs(silu(p)) * (soft(p) + 2.0 ** -23)) if act else ep
            continue
        d = dy[at].reshape(-1, G, cg)
        dp, edp = d, np.zeros_like(d)
        if act:
            sg = sigmoid(p)
            dp = d * dsilu(p)
            edp = np.abs(d) * (0.5 * ep + (sg + np.abs(p) * sg * (1 - sg)) * (2 * soft(p) + 2.0 ** -21) + np.abs(p) * sg * sg * soft(p))
        q, eq = dp * w1, np.abs(w1) * edp + 2.0 ** -24 * np.abs(dp * w1)
        mq, emq = q.mean(dims, keepdims=True), (eq + k * 2.0 ** -23 * np.abs(q)).mean(dims, keepdims=True)
        mx = (q * xh).mean(dims, keepdims=True)
        emx = (eq * np.abs(xh) + np.abs(q) * exh + k * 2.0 ** -23 * np.abs(q * xh)).mean(dims, keepdims=True)
        out["dx"][at] = rstd * (q - mq - xh * mx)
        out["dx_err"][at] = rstd * (eq + emq + exh * np.abs(mx) + np.abs(xh) * emx + 2.0 ** -22 * (np.abs(q) + np.abs(mq) + np.abs(xh * mx))) + \
            np.abs(out["dx"][at]) * (dr + 2.0 ** -22)
        n = T * 2.0 ** -24
        sums["dweight"] += (dp * xh).sum(0)
        sums["dweight_err"] += (edp * np.abs(xh) + np.abs(dp) * exh + n * np.abs(dp * xh)).sum(0)
        sums["dbias"] += dp.sum(0)
        sums["dbias_err"] += (edp + n * np.abs(dp)).sum(0)
    for name in ("y", "y_err", "dx", "dx_err"):
        out[name] = out[name].reshape(T, C)
    for name in ("dweight", "dweight_err", "dbias", "dbias_err"):
        out[name] = sums[name].reshape(C)
    out["stats"] = np.stack(out["stats"]) if out["stats"] else None
    return out


def within(got, ref, err, dtype, name=""):
    got = f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    off = np.abs(got - ref) - (half_step(dtype) * np.abs(ref) + err * (1 + half_step(dtype)) + 1e-30)
    assert (off <= 0).all(), f"{name}: off by up to {off.max():.3e} more than allowed, {int((off > 0).sum())} of {off.size} values"
