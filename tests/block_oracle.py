"""Plain 64-bit forms of the operators of include/per_block.h, from their
definitions, with a bound on the error each kernel may make: u = 2^-24 is half a step
of f32, a sum of n terms in f32 is off by at most n u times the sum of their sizes,
and an output in t is rounded once."""
from __future__ import annotations

import torch

from train_oracle import U, rounding

CHUNK = 64


# ------------------------------------------------------------------ embedding

def embed(tokens, table, scale, dtype):
    t = tokens.cpu().long()
    V = table.shape[0]
    ok = (t >= 0) & (t < V)
    want = table.detach().cpu().double()[t.clamp(0, V - 1)] * scale
    want[~ok] = 0
    return want, U * want.abs() * 2 + rounding(want, dtype)


def embed_grad(tokens, dout, V, scale, dtype=torch.float32, old=None):
    """A token's rows are added up to 64 at a time, then the parts in four runs: the
    longest chain has 64 + parts / 4 + 4 additions, and parts hold 8 rows at least."""
    t = tokens.cpu().long()
    ok = (t >= 0) & (t < V)
    d = dout.detach().cpu().double()[ok]
    want = torch.zeros(V, d.shape[1], dtype=torch.float64).index_add_(0, t[ok], d) * scale
    size = torch.zeros_like(want).index_add_(0, t[ok], d.abs()) * abs(scale)
    count = torch.bincount(t[ok], minlength=V).double()[:, None]
    tol = (count.clamp(max=64) + count / 32 + 8) * U * size
    if old is not None:
        o = old.detach().cpu().double()
        want, size = want + o, size + o.abs()
    tol = tol + 2 * U * size
    return want, tol + rounding(want, dtype)


# ----------------------------------------------------------------- layer norm

def norm(x, weight=None, bias=None, eps=1e-5, dy=None):
    """Forward and, given dy, backward, each with its allowed error.  A sum over the row
    is off by n u of its terms' sizes, n = 64 + D / 1024 (a thread adds up to 32 values,
    or D / 1024 in long rows; then lanes and waves); one over N rows by N / 256 + 64."""
    dt = x.dtype
    x = x.detach().cpu().double()
    N, D = x.shape
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.detach().cpu().double()
    b = torch.zeros(D, dtype=torch.float64) if bias is None else bias.detach().cpu().double()
    n = 64 + D / 1024
    m = x.mean(1, keepdim=True)
    d = x - m
    var = d.square().mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    h = d * r
    # the distances are corrected by their own mean: what is left of the mean's error is
    # that of summing the distances; the deviation has half the error of its square
    eh = r * (3 * U * d.abs() + n * U * d.abs().mean(1, keepdim=True)) + h.abs() * (n + 8) * U
    y = h * w + b
    out = {"y": (y, eh * w.abs() + 3 * U * ((h * w).abs() + b.abs()) + rounding(y, dt)),
           "mean": (m[:, 0], (n * U * d.abs().mean(1) + 2 * U * m[:, 0].abs())),
           "rstd": (r[:, 0], r[:, 0] * (n + 8) * U)}
    if dy is None:
        return out
    dy = dy.detach().cpu().double()
    eh = eh + r * U * 2 * m.abs()  # the mean is saved in f32
    e = dy * w
    s1, s2 = e.mean(1, keepdim=True), (e * h).mean(1, keepdim=True)
    es1 = (n + 2) * U * e.abs().mean(1, keepdim=True)
    es2 = (n + 4) * U * (e * h).abs().mean(1, keepdim=True) + (e.abs() * eh).mean(1, keepdim=True)
    dx = r * (e - s1 - h * s2)
    edx = (r * (4 * U * (e.abs() + s1.abs() + (h * s2).abs()) + es1 + eh * s2.abs() + h.abs() * es2)
           + dx.abs() * (n + 8) * U)
    k = N / 256 + 64
    out["dx"] = (dx, edx + rounding(dx, dt))
    out["dweight"] = ((dy * h).sum(0), (dy.abs() * eh).sum(0) + k * U * (dy * h).abs().sum(0))
    out["dbias"] = (dy.sum(0), k * U * dy.abs().sum(0))
    return out


# ----------------------------------------------------------- gated delta rule

def delta(q, k, v, g, b, reset=None, length=None, s0=None, scale=1.0):
    """The rule step by step in f64, for autograd: (o, s_last)."""
    B, T, H = v.shape[:3]
    sh = H // q.shape[2]
    q, k = (x.double().repeat_interleave(sh, 2) for x in (q, k))
    # by their logarithms: the gradient of sigmoid is taken as f (1 - f), which is 0 in f64
    # from g = 37 on, where it is exp(-g)
    v, f, w = v.double(), *(torch.nn.functional.logsigmoid(x.double()).exp() for x in (g, b))
    s = torch.zeros(B, H, q.shape[3], v.shape[3], dtype=torch.float64) if s0 is None else s0.double()
    n = torch.full((B,), T) if length is None else length.cpu().clamp(0, T)
    outs = []
    for t in range(T):
        on = (t < n)[:, None, None]
        clear = torch.zeros(B, dtype=torch.bool) if reset is None else reset[:, t].cpu().bool()
        qt, kt, vt = (torch.where(on, x[:, t], 0.0) for x in (q, k, v))
        ft, wt = (torch.where(on[..., 0], x[:, t], 0.5) for x in (f, w))
        p = torch.where(clear[:, None, None, None], 0.0, s) * ft[..., None, None]
        u = wt[..., None] * (vt - (p * kt[..., None]).sum(2))
        new = p + kt[..., None] * u[:, :, None]
        s = torch.where(on[..., None], new, s)
        outs.append(torch.where(on, scale * (new * qt[..., None]).sum(2), 0.0))
    o = torch.stack(outs, 1) if T else torch.zeros(v.shape, dtype=torch.float64)
    return o, s


def delta_all(q, k, v, g, b, reset=None, length=None, s0=None, scale=1.0, do=None, ds_last=None):
    """Values and, given do, gradients by every input, from the steps."""
    ins = [x.detach().cpu().double().requires_grad_() for x in (q, k, v, g, b)]
    B, T, H, DV = v.shape
    z = torch.zeros(B, H, q.shape[3], DV, dtype=torch.float64) if s0 is None else s0.detach().cpu().double().clone()
    ins.append(z.requires_grad_())
    with torch.enable_grad():
        o, s = delta(*ins[:5], reset, length, ins[5], scale)
        out = {"o": o.detach(), "s": s.detach()}
        if do is not None:
            total = (o * do.detach().cpu().double()).sum() if T else 0.0
            total = total + ((s * ds_last.detach().cpu().double()).sum() if ds_last is not None else 0.0 * s.sum())
            grads = torch.autograd.grad(total, ins, allow_unused=True)
            for name, x, d in zip(("dq", "dk", "dv", "dg", "db", "ds0"), ins, grads):
                out[name] = torch.zeros_like(x) if d is None else d
    return out


def delta_size(q, k, v, g, b, reset=None, length=None, s0=None, scale=1.0, do=None, ds_last=None):
    """How large the terms are that a chunked evaluation adds up for each result: its
    error is at most that times the error of one product and sum.

    Inside a chunk: products of the factors' absolute values; the inverse X of I + A is
    off by the error of one product and sum times |X| |A| |X|.  From chunk to chunk: an
    error of the state goes through the gates and the maps I - w k k^T, which do not
    stretch it (w |k|^2 <= 2), so per column its 2-norm shrinks by the gates alone."""
    B, T, H, DV = v.shape
    HK, DK = q.shape[2:]
    sh = H // HK
    n = [T] * B if length is None else length.cpu().clamp(0, T).tolist()
    z = {"o": torch.zeros(B, T, H, DV), "s": torch.zeros(B, H, DK, DV), "dq": torch.zeros(B, T, HK, DK),
         "dk": torch.zeros(B, T, HK, DK), "dv": torch.zeros(B, T, H, DV), "dg": torch.zeros(B, T, H),
         "db": torch.zeros(B, T, H), "ds0": torch.zeros(B, H, DK, DV)}
    z = {x: y.double() for x, y in z.items()}
    q, k, v, g, b = (x.detach().cpu().double() for x in (q, k, v, g, b))
    for bi in range(B):
        for h in range(H):
            s = torch.zeros(DK, DV, dtype=torch.float64) if s0 is None else s0[bi, h].detach().cpu().double()
            se = torch.zeros(DV, dtype=torch.float64)  # of the state's error, by column
            saved = []
            for t0 in range(0, n[bi], CHUNK):
                r = slice(t0, min(n[bi], t0 + CHUNK))
                Q, K, V = q[bi, r, h // sh], k[bi, r, h // sh], v[bi, r, h]
                w, lf = torch.sigmoid(b[bi, r, h]), torch.nn.functional.logsigmoid(g[bi, r, h]).clamp(min=-200)
                seen = torch.zeros(len(Q), dtype=torch.long) if reset is None else reset[bi, r].cpu().long().cumsum(0)
                c = lf.cumsum(0)
                low = torch.ones(len(Q), len(Q), dtype=torch.bool).tril()
                D = torch.where((seen[:, None] == seen) & low, (c[:, None] - c).exp(), 0.0)
                first = torch.where(seen == 0, c.exp(), 0.0)
                last = torch.where(seen == seen[-1], (c[-1] - c).exp(), 0.0)
                A = (w[:, None] * D * (K @ K.t())).tril(-1)
                Ab = (w[:, None] * D * (K.abs() @ K.abs().t())).tril(-1)
                X = torch.linalg.inv(torch.eye(len(Q), dtype=torch.float64) + A)
                S = torch.where(torch.isfinite(s), s, 0.0)
                R = w[:, None] * (V - first[:, None] * (K @ S))
                Rb = w[:, None] * (V.abs() + first[:, None] * (K.abs() @ S.abs() + K.norm(dim=1)[:, None] * se))
                U_, Xa = X @ R, X.abs()
                Ub = Xa @ Rb + Xa @ (Ab @ (Xa @ Rb))
                P, Pb = (Q @ K.t()) * D, (Q.abs() @ K.abs().t()) * D
                z["o"][bi, r, h] = abs(scale) * (first[:, None] * (Q.abs() @ S.abs() + Q.norm(dim=1)[:, None] * se) + Pb @ Ub)
                saved.append((r, Q, K, V, w, D, first, last, X, Ab, S, se, U_, Ub, P, Pb, lf, g[bi, r, h], seen))
                s = first[-1] * S + (K * last[:, None]).t() @ U_
                se = first[-1] * (se + S.norm(dim=0)) + ((K.abs() * last[:, None]).t() @ Ub).norm(dim=0)
            z["s"][bi, h] = se + s.norm(dim=0)
            if do is None:
                continue
            d = torch.zeros(DK, DV, dtype=torch.float64) if ds_last is None else ds_last[bi, h].detach().cpu().double()
            de = torch.zeros(DV, dtype=torch.float64)
            for (r, Q, K, V, w, D, first, last, X, Ab, S, se, U_, Ub, P, Pb, lf, gr, seen) in reversed(saved):
                O = scale * do[bi, r, h].detach().cpu().double()
                Oa, Xt = O.abs(), X.abs().t()
                kn, qn = K.norm(dim=1)[:, None], Q.norm(dim=1)[:, None]
                y = Pb.t() @ Oa + last[:, None] * (K.abs() @ d.abs() + kn * de)
                E = X.t() @ (P.t() @ O + last[:, None] * (K @ d))
                Eb = Xt @ y + Xt @ (Ab.t() @ (Xt @ y))
                G, Gb = w[:, None] * E, w[:, None] * Eb
                z["dv"][bi, r, h] = Gb
                Sa = S.abs() + se / DK ** 0.5  # an error of a column, spread over its rows
                da = d.abs() + de / DK ** 0.5
                dP = (Oa @ Ub.t()) * D
                M = ((Gb @ Ub.t()) * D).tril(-1)
                dq = first[:, None] * (Oa @ Sa.t()) + dP @ K.abs()
                dk = last[:, None] * (Ub @ da.t()) + dP.t() @ Q.abs() + first[:, None] * (Gb @ Sa.t()) + (M + M.t()) @ K.abs()
                z["dq"][bi, r, h // sh] += dq
                z["dk"][bi, r, h // sh] += dk
                z["db"][bi, r, h] = (Eb * Ub).sum(1) * (1 - w)
                end = first[-1] * (S.abs() * d.abs()).sum() + first[-1] * (se * d.norm(dim=0) + de * S.norm(dim=0)).sum() \
                    + ((K.abs() * last[:, None]) * (Ub @ da.t())).sum()
                each = (Q.abs() * dq).sum(1) + (Gb * V.abs()).sum(1)
                z["dg"][bi, r, h] = (each.flip(0).cumsum(0).flip(0) + end) * torch.sigmoid(-gr)
                nd = first[-1] * d + (Q * first[:, None]).t() @ O - (K * first[:, None]).t() @ G
                de = first[-1] * (de + d.norm(dim=0)) + ((Q.abs() * first[:, None]).t() @ Oa + (K.abs() * first[:, None]).t() @ Gb).norm(dim=0)
                d = nd
            z["ds0"][bi, h] = de + d.norm(dim=0)
    return z


def delta_tolerance(size, values, dtype):
    """The longest chain of nested sums has DK + 4 * 64 <= 384 terms, at u each, and a
    decay's exponent (up to 200, in f32) and exponential a few hundred u at worst where it
    is e^-200; states are held to that.  Outputs in 16 bits come from products of factors
    held to 16 bits, off by 3 * 2^-16, and are rounded."""
    out = {}
    for name, want in values.items():
        state = name in ("s", "ds0")
        t = torch.float32 if state else dtype
        rel = 400 * U + (0 if t == torch.float32 else 3 * 2.0 ** -16)
        out[name] = rel * size[name] + rounding(want, t)
    return out
