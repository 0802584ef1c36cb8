"""Plain 64-bit forms (CPU torch) of the operators around the routed experts, each with a bound of
the error that 32-bit arithmetic and one final rounding may leave: the sum of the terms' magnitudes
times the roundings a term goes through, plus half a step of the output's type."""
import math

import torch

F32 = 2.0 ** -24  # half a step of f32, relative


def half_step(ref, dtype):
    """The final rounding: half a step of `dtype` at |ref| (and at its smallest normal number)."""
    fi = torch.finfo(dtype)
    return fi.eps / 2 * ref.abs().clamp(min=fi.smallest_normal)


def assert_within(got, ref, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what
    fine = torch.isfinite(ref)
    over = ((got - ref).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (
        f"{what}: {int((over > 0).sum())} of {over.numel()} past the bound, worst by "
        f"{float(over.max()):.3e}")


# ------------------------------------------------------------------------------------- linear
def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "relu2":
        return z.clamp(min=0) ** 2
    return z


def linear64(x, w, bias, act, residual, out_dtype):
    """(reference, bound).  The sum: K/16 + 16 f32 additions, each off by at most one step (the
    tensor cores may truncate) of what has been summed.  The activations have slopes of at most
    1.2 (silu, gelu) and 2|z| (relu2), and their own f32 evaluation is good to 2^-20."""
    K = x.shape[1]
    x, w = x.cpu().double(), w.cpu().double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.cpu().double(), mag + bias.cpu().double().abs()
    off = (K / 16 + 16) * 2 * F32 * mag
    a = act64(z, act)
    slope = {"none": 1.0, "silu": 1.2, "gelu_tanh": 1.2}.get(act)
    err = off * (2 * (z.abs() + off) if slope is None else slope)
    if act != "none":
        # z may cross the steep part of e^-z by `off` only; the value itself is good to 2^-20
        err = err + 2.0 ** -20 * a.abs()
    if residual is not None:
        r = residual.cpu().double()
        a, err = a + r, err + 2 * F32 * (a.abs() + r.abs())
    return a, err + half_step(a, out_dtype) * (1 + 2.0 ** -7)


# ----------------------------------------------------------------------------------- the norm
_NORM = 64 * F32  # roundings of a term: products, the mean's tree, rsqrt


def _rstd(v, eps):
    return 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)


def _w(w, o):
    return 1.0 if w is None else o + w


def norm64(branch, residual, gate, wq, wp, post, pre, a, o, eps):
    """(stream, normed or None) of 64-bit inputs; gate broadcast already."""
    u = branch
    if post:
        u = u * _rstd(u, eps) * _w(wq, o)
    r = gate * u
    if residual is not None:
        r = r + a * residual
    return r, (r * _rstd(r, eps) * _w(wp, o) if pre else None)


def norm_bounds(branch, residual, gate, wq, wp, post, pre, a, o, eps, dtype):
    r, h = norm64(branch, residual, gate, wq, wp, post, pre, a, o, eps)
    u = r - (0 if residual is None else a * residual)
    e = _NORM * (u.abs() + (0 if residual is None else (a * residual).abs()))
    out = [e + half_step(r, dtype) * (1 + 2.0 ** -7)]
    if h is not None:
        w = _w(wp, o)
        rr = _rstd(r, eps)
        # an error of the row moves its mean square too
        rel = (2 * (e * r.abs()).mean(dim=1, keepdim=True)) * rr * rr
        out.append(e * rr * (w.abs() if wp is not None else 1.0) + (rel + _NORM) * h.abs()
                   + half_step(h, dtype) * (1 + 2.0 ** -7))
    else:
        out.append(None)
    return out


def norm_bwd64(dr, dh, branch, residual, gate, wq, wp, post, pre, a, o, eps):
    """The gradients by the formulas, and the sums of their terms' magnitudes: two dicts over
    branch, residual, gate (per element), post and pre (per element: the caller sums)."""
    y, zero = branch, torch.zeros_like(branch)
    ry = _rstd(y, eps) if post else torch.ones_like(y[:, :1])
    q = _w(wq, o) if post else 1.0
    yh = y * ry
    u = yh * q
    x = zero if residual is None else residual
    r = a * x + gate * u
    rm = (a * x).abs() + (gate * u).abs()  # magnitude behind r
    D = zero if dr is None else dr
    Dm = D.abs()
    grads, mags = {}, {}
    if pre:
        rr = _rstd(r, eps)
        rh, rhm = r * rr, rm * rr
        dn = dh * _w(wp, o)
        grads["pre"], mags["pre"] = dh * rh, dh.abs() * rhm
        m = (dn * rh).mean(dim=1, keepdim=True)
        mm = (dn.abs() * rhm).mean(dim=1, keepdim=True)
        D = D + rr * (dn - rh * m)
        # the statistics carry the row's own cancellation
        loss = 1 + (rhm * rhm).mean(dim=1, keepdim=True)
        Dm = Dm + rr * (dn.abs() + rhm * mm) * loss
    grads["residual"], mags["residual"] = a * D, abs(a) * Dm
    grads["gate"], mags["gate"] = D * u, Dm * u.abs()
    g = gate if torch.is_tensor(gate) else torch.full_like(y, gate)
    du, dum = D * g, Dm * g.abs()
    grads["post"], mags["post"] = du * yh, dum * yh.abs()
    if post:
        dn, dnm = du * q, dum * (q.abs() if torch.is_tensor(q) else abs(q))
        du = ry * (dn - yh * (dn * yh).mean(dim=1, keepdim=True))
        dum = ry * (dnm + yh.abs() * (dnm * yh.abs()).mean(dim=1, keepdim=True))
    grads["branch"], mags["branch"] = du, dum
    return grads, mags


def grad_bound(ref, mag, dtype, terms=1):
    """Half a step of the type, and 2^-17 of the terms' magnitudes (128 f32 roundings: the norm's
    own 64, twice); a sum over `terms` tokens adds their count of roundings."""
    return (2 * _NORM + terms * F32) * mag + half_step(ref, dtype) * (1 + 2.0 ** -7)


# --------------------------------------------------------------------------------- the router
def probs64(x, scoring):
    """p of each row; a row of -inf alone gives zeros."""
    dead = torch.isneginf(x).all(dim=1, keepdim=True)
    if scoring == "softmax":
        p = torch.softmax(torch.where(dead, torch.zeros_like(x), x), dim=1)
    else:
        # log sigmoid, normalised: exact where every sigmoid underflows
        ls = torch.nn.functional.logsigmoid(torch.where(dead, torch.zeros_like(x), x))
        p = torch.softmax(ls, dim=1)
    return torch.where(dead, torch.zeros_like(p), p)


def balance64(x, ids, coeff, scoring, offsets):
    """(loss, counts, live, prob_sum, coef), sequence by sequence."""
    T, E = x.shape
    k = ids.shape[1]
    off = [0, T] if offsets is None else [int(v) for v in offsets]
    n = len(off) - 1
    p = probs64(x, scoring)
    counts = torch.zeros(n, E, dtype=torch.int32)
    live = torch.zeros(n, dtype=torch.int32)
    sums = torch.zeros(n, E, dtype=torch.float64)
    for s in range(n):
        for t in range(off[s], off[s + 1]):
            mine = [int(i) for i in ids[t] if 0 <= int(i) < E]
            if mine:
                live[s] += 1
                sums[s] = sums[s] + p[t]
                for i in mine:
                    counts[s, i] += 1
    n_live = max(1, int((live > 0).sum()))
    T_s = live.clamp(min=1).double()[:, None]
    coef = coeff * E * counts.double() / (n_live * k * T_s * T_s)
    return (coef * sums).sum(), counts, live, sums, coef


def router_loss64(x, ids, dw, coef, offsets, scoring, renorm, factor, d_loss):
    """The scalar whose gradient moe_router_bwd returns: d_loss * sum coef p + sum dw w."""
    T, E = x.shape
    p = probs64(x, scoring)
    seq = torch.full((T,), -1) if offsets is not None else torch.zeros(T, dtype=torch.long)
    if offsets is not None:
        for s in range(len(offsets) - 1):
            seq[int(offsets[s]):int(offsets[s + 1])] = s
    total = torch.zeros((), dtype=torch.float64)
    for t in range(T):
        mine = [(j, int(i)) for j, i in enumerate(ids[t]) if 0 <= int(i) < E]
        if not mine:
            continue
        if coef is not None and seq[t] >= 0:
            total = total + d_loss * (coef[seq[t]] * p[t]).sum()
        if dw is not None:
            sel = torch.tensor([i for _, i in mine])
            g = dw[t][[j for j, _ in mine]]
            if renorm:
                score = x[t][sel] if scoring == "softmax" else (
                    torch.nn.functional.logsigmoid(x[t][sel]))
                w = torch.softmax(score, dim=0)
            else:
                w = p[t][sel] if scoring == "softmax" else torch.sigmoid(x[t][sel])
            total = total + factor * (g * w).sum()
    return total
