"""Plain 64-bit forms of the sequence operators, from their definitions, with
a bound on the error each kernel may make: u = 2^-24 is half a step of f32, and
an output in t is rounded once, by at most eps(t) / 2 of its value."""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(v, dtype):
    """Largest error of rounding v to dtype (half the smallest subnormal near 0)."""
    f = torch.finfo(dtype)
    return v.abs() * half_step(dtype) + f.smallest_normal * f.eps / 2


def assert_close(got, want, tol, what):
    """|got - want| <= tol elementwise; the same places not finite."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    fin = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), what + ": NaN in other places"
    assert torch.equal(g[~fin & ~torch.isnan(w)], w[~fin & ~torch.isnan(w)]), what
    over = ((g - w).abs() - tol.double().cpu())[fin]
    if over.numel() and over.max() > 0:
        k = int(over.argmax())
        raise AssertionError("%s: %d of %d values too far off; the worst: got %r, want %r, allowed %r" % (
            what, int((over > 0).sum()), g.numel(), float(g[fin][k]), float(w[fin][k]),
            float(tol.double().cpu().expand_as(w)[fin][k])))


# ------------------------------------------------------------ 8-bit row store

def quantise(src, fmt, group):
    """(codes, scales) of rows, exactly as defined (numpy f32, one rounding per
    operation; the conversion to 8 bits to nearest even)."""
    x = src.detach().cpu().float().numpy()
    n, d = x.shape
    g = group or d
    ng = -(-d // g)
    top = np.float32(TOP[fmt])
    codes = np.zeros((n, d), np.float32)
    scales = np.zeros((n, ng), np.float32)
    with np.errstate(all="ignore"):
        for k in range(ng):
            part = x[:, k * g:(k + 1) * g]
            a = np.where(np.isfinite(part), np.abs(part), np.float32(0)).max(1)
            a = np.maximum(a, np.float32(2.0 ** -100))
            s = (a * (np.float32(1) / top)).astype(np.float32)
            inv = (np.float32(1) / s).astype(np.float32)
            q = (part * inv[:, None]).astype(np.float32)
            q = np.where(q > top, top, np.where(q < -top, -top, q))
            if fmt == torch.int8:
                q = np.rint(np.where(np.isnan(q), np.float32(0), q))
            codes[:, k * g:(k + 1) * g] = q
            scales[:, k] = s
    return torch.from_numpy(codes).to(fmt), torch.from_numpy(scales)


def dequantise(codes, scales, group, dtype):
    d = codes.shape[1]
    g = group or d
    col = torch.arange(d) // g
    return (codes.cpu().float() * scales.cpu()[:, col]).to(dtype)


# ----------------------------------------------------- gated linear recurrence

def scan(x, g, reset=None, length=None, h0=None, dy=None, dh_last=None, dtype=torch.float32):
    """Forward and, given dy, backward in f64; every value with the error an f32
    computation may have made.  A gate is off by delta = (1.5 |g| + 8) u of
    itself (the exponent's rounding, the exponential, the reciprocal); a state
    gathers delta of its summands and the roundings of the step; twice that for
    the different order in which the tiles are joined."""
    x, g = x.detach().cpu().double(), g.detach().cpu().double()
    B, T, D = x.shape
    f, i = torch.sigmoid(g), torch.sigmoid(-g)
    delta = (1.5 * g.abs() + 8) * U
    n = torch.full((B,), T) if length is None else length.cpu().clamp(0, T)
    rs = torch.zeros(B, T, dtype=torch.bool) if reset is None else reset.cpu().bool()
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.detach().cpu().double().clone()
    e = torch.zeros_like(h)
    hp, he = torch.zeros_like(x), torch.zeros_like(x)
    y, ye = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        on = (t < n)[:, None]
        p = torch.where(rs[:, t, None], torch.zeros_like(h), h)
        pe = torch.where(rs[:, t, None], torch.zeros_like(h), e)
        xt = torch.where(on, x[:, t], torch.zeros_like(h))
        ft, it, dt = (torch.where(on, v[:, t], torch.zeros_like(h)) for v in (f, i, delta))
        new = ft * p + it * xt
        err = ft * pe + (dt + 2 * U) * ((ft * p).abs() + (it * xt).abs()) + U * new.abs()
        hp[:, t], he[:, t] = p, pe
        h, e = torch.where(on, new, h), torch.where(on, err, e)
        y[:, t], ye[:, t] = torch.where(on, new, torch.zeros_like(h)), torch.where(on, err, torch.zeros_like(h))
    out = {"y": (y, 2 * ye + rounding(y, dtype)), "h": (h, 2 * e + U * h.abs())}
    if dy is None:
        return out
    dy = dy.detach().cpu().double()
    E = torch.zeros(B, D, dtype=torch.float64) if dh_last is None else dh_last.detach().cpu().double().clone()
    Ee = torch.zeros_like(E)
    dx, dxe, dg, dge = (torch.zeros_like(x) for _ in range(4))
    zero = torch.zeros_like(E)
    for t in reversed(range(T)):
        on = (t < n)[:, None]
        full = E + torch.where(on, dy[:, t], zero)
        fe = Ee + U * full.abs()
        xt, ft, it, dt = (torch.where(on, v[:, t], zero) for v in (x, f, i, delta))
        dx[:, t] = full * it
        dxe[:, t] = fe * it + (dt + 2 * U) * (full * it).abs()
        diff = hp[:, t] - xt
        dg[:, t] = full * diff * ft * it
        dge[:, t] = ((fe * diff.abs() + full.abs() * (2 * he[:, t] + U * diff.abs())) * ft * it
                     + (2 * dt + 4 * U) * dg[:, t].abs())
        back = torch.where(rs[:, t, None], zero, full * ft)
        berr = torch.where(rs[:, t, None], zero, fe * ft + (dt + 2 * U) * back.abs())
        E, Ee = torch.where(on, back, E), torch.where(on, berr, Ee)
    out["dx"] = (dx, 2 * dxe + rounding(dx, dtype))
    out["dg"] = (dg, 2 * dge + rounding(dg, dtype))
    out["dh0"] = (E, 2 * Ee + U * E.abs())
    return out


# ----------------------------------------------------------------- distillation

def distill(z, tidx, t, tlse=None, tau=1.0, weight=None, dtype=torch.float32):
    """Loss and gradient in f64, each with its allowed error.  One exponential
    is off by (3 |z - m| / tau + 4) u of itself; a sum over the row also by 200 u
    (no thread adds more than 17 chunks of 8, and 16 waves are joined)."""
    z, t = z.detach().cpu().double(), t.detach().cpu().double()
    N, V = z.shape
    loss, loss_tol = torch.zeros(N, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    grad, tol = torch.zeros(N, V, dtype=torch.float64), torch.zeros(N, V, dtype=torch.float64)
    w = torch.ones(N, dtype=torch.float64) if weight is None else weight.detach().cpu().double()
    for n in range(N):
        if w[n] == 0:
            continue
        ids = tidx[n].cpu().long()
        ok = (ids >= 0) & (ids < V)
        ids, tk = ids[ok], t[n][ok] / tau
        if tlse is None:
            if ids.numel() == 0 or torch.all(tk == -math.inf):
                continue
            d = tk - tk.max()  # 64 bits lose log K next to logits at the type's lowest value
            logp = d - torch.logsumexp(d, 0)
        else:
            logp = tk - float(tlse[n])
        p = logp.exp()
        zn = z[n]
        m = zn.max()
        if m == -math.inf:
            continue
        e = ((zn - m) / tau).exp()
        ee = (3 * ((zn - m) / tau).abs().clamp(max=1e6) + 4) * U  # relative, by token
        ee = torch.where(e == 0, torch.zeros_like(ee), ee)
        S = e.sum()
        eS = float((e * ee).sum() / S) + 200 * U
        q = e / S
        pv = p > 0
        terms = p[pv] * (logp[pv] - (zn[ids[pv]] - m) / tau + S.log())
        L = terms.sum() if pv.any() else torch.zeros((), dtype=torch.float64)
        # the sum over the entries takes p in f32
        Le = p.sum() * eS + U * (p[pv] * ((zn[ids[pv]] - m) / tau).abs().clamp(max=1e30)).sum()
        P = torch.zeros(V, dtype=torch.float64).index_add_(0, ids, p)
        g = q - P
        ge = q * (ee + eS + 4 * U) + P * 4 * U + U * g.abs()
        if tlse is not None:
            rest = float((1 - p.sum()).clamp(min=0))
            out = torch.ones(V, dtype=torch.bool)
            out[ids] = False
            Sr = e[out].sum()
            if Sr > 0:
                eR = float((e[out] * ee[out]).sum() / Sr) + 200 * U
                if rest > 0:
                    L = L + rest * (math.log(rest) - Sr.log() + S.log())
                    Le = Le + rest * (eS + eR)
                share = rest * e / Sr
                g = torch.where(out, q - share, g)
                ge = torch.where(out, (q + share) * (ee + eS + eR + 6 * U) + U * g.abs(), ge)
        loss[n] = tau * tau * L
        loss_tol[n] = tau * tau * Le + (loss[n].abs() * U if torch.isfinite(loss[n]) else 0.0)
        grad[n] = w[n] * tau * g
        tol[n] = w[n].abs() * tau * ge + 2 * U * grad[n].abs()
    return {"loss": (loss, loss_tol + 2.0 ** -149), "grad": (grad, tol + rounding(grad, dtype))}
