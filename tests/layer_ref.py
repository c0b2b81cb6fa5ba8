"""Plain 64-bit forms of the recurrent layer's operators (numpy, written from the formulas),
and the books of the pages of a cache as Python lists."""
import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def silu(p):
    with np.errstate(over="ignore"):
        return p / (1 + np.exp(-p))


def dsilu(p):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-p))
    return s * (1 + p * (1 - s))


def softplus(x):
    return np.logaddexp(x, 0.0)


def conv(x, w, bias, act, initial, cu, dy=None, dfinal=None):
    """x [T, C], w [C, W], initial [N, W-1, C] or None.  Without dy: (y, final, M) with M the sum of
    the magnitudes in p; with dy: a dict of gradients and of their magnitude sums."""
    T, C = x.shape
    W, N = w.shape[1], len(cu) - 1
    y, M = np.zeros_like(x), np.zeros_like(x)
    final = np.zeros((N, W - 1, C))
    g = {"dx": np.zeros_like(x), "dx_mag": np.zeros_like(x), "dweight": np.zeros_like(w), "dw_mag": np.zeros_like(w),
         "dbias": np.zeros(C), "db_mag": np.zeros(C), "dinitial": np.zeros_like(final), "di_mag": np.zeros_like(final)}
    for n in range(N):
        b, e = cu[n], cu[n + 1]
        line = np.concatenate([np.zeros((W - 1, C)) if initial is None else initial[n], x[b:e]])
        L = e - b
        p = np.zeros((L, C)) + (0 if bias is None else bias)
        m = np.zeros((L, C)) + (0 if bias is None else np.abs(bias))
        for j in range(W):
            p += line[j:j + L] * w[:, j]
            m += np.abs(line[j:j + L] * w[:, j])
        y[b:e], M[b:e] = silu(p) if act else p, m
        final[n] = line[L:]
        if dy is None:
            continue
        dp = dy[b:e] * (dsilu(p) if act else 1.0)
        dpm = np.abs(dy[b:e]) * (1 + (m if act else 0))
        dl, dlm = np.zeros_like(line), np.zeros_like(line)
        if dfinal is not None:
            dl[L:] += dfinal[n]
            dlm[L:] += np.abs(dfinal[n])
        for j in range(W):
            dl[j:j + L] += dp * w[:, j]
            dlm[j:j + L] += dpm * np.abs(w[:, j])
            g["dweight"][:, j] += (dp * line[j:j + L]).sum(0)
            g["dw_mag"][:, j] += (dpm * np.abs(line[j:j + L])).sum(0)
        g["dbias"] += dp.sum(0)
        g["db_mag"] += dpm.sum(0)
        g["dx"][b:e], g["dx_mag"][b:e] = dl[W - 1:], dlm[W - 1:]
        g["dinitial"][n], g["di_mag"][n] = dl[:W - 1], dlm[:W - 1]
    return (y, final, M) if dy is None else g


def scan(u, delta, A, B, C, D, z, bias, sp, initial, cu, dy=None, dfinal=None):
    """u, delta, z [T, c]; A [c, S]; B, C [T, G, S].  A dict: y, state, and with dy the gradients; every
    value x with x + "_err", the sum of magnitudes that a relative error of the parts is taken of: of the
    terms, states and decays, a decay counting (1 + |d A|) times for its exponent's error, which the
    states behind it inherit."""
    T, c = u.shape
    S, G, N = A.shape[1], B.shape[1], len(cu) - 1
    grp = np.arange(c) // (c // G)
    raw = delta + (0 if bias is None else bias)
    d = softplus(raw) if sp else raw
    D0 = np.zeros(c) if D is None else D
    sz = np.ones_like(u) if z is None else silu(z)
    h, eh = np.zeros((T, c, S)), np.zeros((T, c, S))
    out = {"y": np.zeros_like(u), "y_err": np.zeros_like(u), "state": np.zeros((N, c, S)), "state_err": np.zeros((N, c, S))}
    lin, elin = np.zeros_like(u), np.zeros_like(u)
    befores, ebefores, decays = np.zeros((T, c, S)), np.zeros((T, c, S)), np.zeros((T, c, S))
    for n in range(N):
        s = np.zeros((c, S)) if initial is None else initial[n]
        e = np.zeros((c, S))
        for t in range(cu[n], cu[n + 1]):
            befores[t], ebefores[t] = s, e
            a = decays[t] = np.exp(d[t][:, None] * A)
            b = (d[t] * u[t])[:, None] * B[t][grp]
            e = a * e + a * np.abs(s) * (1 + np.abs(d[t][:, None] * A)) + np.abs(b)
            s = a * s + b
            h[t], eh[t] = s, e
            lin[t] = (C[t][grp] * s).sum(-1) + D0 * u[t]
            elin[t] = (np.abs(C[t][grp]) * (e + np.abs(s))).sum(-1) + np.abs(D0 * u[t])
        out["state"][n], out["state_err"][n] = s, e + np.abs(s)
    out["y"], out["y_err"] = lin * sz, elin * np.abs(sz) + np.abs(lin * sz) * (1 + (0 if z is None else np.abs(z)))
    if dy is None:
        return out
    yb = dy * sz
    eyb = np.abs(yb) * (2 + (0 if z is None else np.abs(z)))
    for k, shape in (("du", u.shape), ("ddelta", u.shape), ("dA", A.shape), ("dB", B.shape), ("dC", B.shape), ("dinitial_state", (N, c, S))):
        out[k], out[k + "_err"] = np.zeros(shape), np.zeros(shape)
    slope = 1 / (1 + np.exp(-raw)) if sp else np.ones_like(raw)
    for n in range(N):
        g = np.zeros((c, S)) if dfinal is None else dfinal[n]
        eg = np.zeros((c, S))
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            Bt, Ct, dt, ut = B[t][grp], C[t][grp], d[t][:, None], u[t]
            dh = g + Ct * yb[t][:, None]
            edh = eg + np.abs(g) + np.abs(Ct) * eyb[t][:, None]
            a = decays[t]
            ex = 1 + np.abs(dt * A)
            through = dh * a * befores[t]
            ethrough = edh * a * np.abs(befores[t]) + np.abs(dh) * a * (ebefores[t] + np.abs(befores[t]) * ex)
            q1, eq1 = (dh * Bt).sum(-1), ((edh + np.abs(dh)) * np.abs(Bt)).sum(-1)
            out["du"][t], out["du_err"][t] = d[t] * q1 + D0 * yb[t], np.abs(d[t]) * (eq1 + np.abs(q1)) + np.abs(D0) * eyb[t]
            out["ddelta"][t] = ((through * A).sum(-1) + ut * q1) * slope[t]
            out["ddelta_err"][t] = (((ethrough + np.abs(through)) * np.abs(A)).sum(-1) + np.abs(ut) * (eq1 + np.abs(q1))) * slope[t] * \
                (2 + np.abs(raw[t]))
            out["dA"] += through * dt
            out["dA_err"] += (ethrough + 2 * np.abs(through)) * np.abs(dt)
            x = (d[t] * ut)[:, None]
            for i, (v, ev) in (("dB", (dh * x, (edh + 2 * np.abs(dh)) * np.abs(x))),
                               ("dC", (h[t] * yb[t][:, None], (eh[t] + np.abs(h[t])) * np.abs(yb[t])[:, None] + np.abs(h[t]) * eyb[t][:, None]))):
                out[i][t], out[i + "_err"][t] = v.reshape(G, c // G, S).sum(1), ev.reshape(G, c // G, S).sum(1)
            g, eg = a * dh, a * edh + np.abs(a * dh) * ex
        out["dinitial_state"][n], out["dinitial_state_err"][n] = g, eg + np.abs(g)
    out["dD"], out["dD_err"] = (yb * u).sum(0), (eyb * np.abs(u)).sum(0)
    out["ddelta_bias"], out["ddelta_bias_err"] = out["ddelta"].sum(0), out["ddelta_err"].sum(0)
    if z is not None:
        out["dz"] = dy * lin * dsilu(z)
        out["dz_err"] = np.abs(dy) * (elin + np.abs(lin) * (2 + np.abs(z))) * 1.2
    return out


class Books:
    """refs, tables and lens as lists; every operation returns what it gives out and whether a
    request was refused."""

    def __init__(self, refs, tables=None, lens=None):
        self.refs = [int(r) for r in refs]
        self.tables = None if tables is None else [[int(e) for e in row] for row in tables]
        self.lens = None if lens is None else [int(v) for v in lens]

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def alloc(self, n):
        got = self.free_pages()[:n]
        for p in got:
            self.refs[p] = 1
        return got + [-1] * (n - len(got)), len(got) < n

    def free(self, pages):
        bad = False
        for p in pages:
            if p == -1:
                continue
            if 0 <= p < len(self.refs) and self.refs[p] > 0:
                self.refs[p] -= 1
            else:
                bad = True
        return bad

    def fork(self, parents, children, tokens):
        S, width, P = len(self.tables), len(self.tables[0]), len(self.refs)
        live = [p != -1 and c != -1 for p, c in zip(parents, children)]
        stands, refused = [], False
        for k, (p, c) in enumerate(zip(parents, children)):
            if not live[k]:
                stands.append(False)
                continue
            ok = 0 <= p < S and 0 <= c < S and 0 <= self.lens[p] <= width * tokens
            for j in range(len(parents)):
                if live[j] and (parents[j] == c or (j != k and children[j] == c)):
                    ok = False
            if ok:
                held = -(-self.lens[p] // tokens)
                ok = all(0 <= e < P and self.refs[e] > 0 for e in self.tables[p][:held])
            stands.append(ok)
            refused |= not ok
        free = self.free_pages()
        src, dst = [-1] * len(parents), [-1] * len(parents)
        grants, taken = [], 0
        for k in range(len(parents)):
            part = stands[k] and self.lens[parents[k]] % tokens != 0
            page = None
            if part:
                if taken < len(free):
                    page = free[taken]
                else:
                    stands[k], refused = False, True
                taken += 1
            grants.append(page)
        for k, (p, c) in enumerate(zip(parents, children)):
            if not stands[k]:
                continue
            full = self.lens[p] // tokens
            row = self.tables[p][:full] + [-1] * (width - full)
            for e in row[:full]:
                self.refs[e] += 1
            if grants[k] is not None:
                row[full] = dst[k] = grants[k]
                src[k] = self.tables[p][full]
                self.refs[grants[k]] = 1
            self.tables[c], self.lens[c] = row, self.lens[p]
        return src, dst, refused

    def compact(self):
        P = len(self.refs)
        used = sum(r != 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] == 0]
        tails = [p for p in range(used, P) if self.refs[p] != 0]
        place = dict(zip(tails, holes))
        refused = False
        for row in self.tables or []:
            for j, e in enumerate(row):
                if e in place:
                    row[j] = place[e]
                elif e != -1 and not 0 <= e < used:
                    refused = True
        for s, d in place.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        pad = [-1] * (P // 2 - len(holes))
        return tails + pad, holes + pad, refused


def copy_pages(pool, src, dst):
    """pool: a numpy array [P, ...]; returns whether a pair was refused."""
    P = len(pool)
    live = [(i, s, d) for i, (s, d) in enumerate(zip(src, dst)) if s != -1 and d != -1]
    ok = [(i, s, d) for i, s, d in live if 0 <= s < P and 0 <= d < P]
    bad = len(ok) < len(live)
    ok = [t for t in ok if t[1] != t[2]]
    read = {s for _, s, _ in ok}
    last = {d: i for i, _, d in ok}
    before = pool.copy()
    for i, s, d in ok:
        if last[d] == i and d not in read:
            pool[d] = before[s]
        else:
            bad = True
    return bad
