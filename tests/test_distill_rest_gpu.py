"""Distillation with a rest where the student's mass on the rest is far below
the row's largest logit: every path of the three calls against the definition in
64 bits, the rest's log-sum-exp taken by itself."""
import math

import pytest
import torch

from train_oracle import TYPES, U, assert_close, rounding

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def reference(z, tidx, t, tlse, tau, w, dtype):
    """(loss, grad) with their allowed errors.  An exponential of u is off by (3 |u|
    + 4) u of itself, u being taken from the rest's largest logit, or from the
    row's while the rest is within 45 tau of it; sums by 200 u as well.  The distance
    between the two maxima enters in 64 bits."""
    z, t = z.double(), t.double() / tau
    N, V = z.shape
    loss, loss_tol = torch.zeros(N, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    grad, tol = torch.zeros(N, V, dtype=torch.float64), torch.zeros(N, V, dtype=torch.float64)
    for n in range(N):
        ids = tidx[n].long()
        p = (t[n] - float(tlse[n])).exp()
        rest = max(0.0, float(1 - p.sum()))
        u = z[n] / tau
        m = u.max()
        logS = torch.logsumexp(u - m, 0)  # differences first: logits at the type's lowest value cancel
        logq = u - m - logS
        q = logq.exp()
        out = torch.ones(V, dtype=torch.bool)
        out[ids] = False
        far = (m - u).clamp(max=1e6)
        eq = torch.where(q > 0, (3 * far + 4) * U, torch.zeros_like(q))
        eS = float((q * eq).sum()) + 200 * U
        seen = p > 0
        L = (p[seen] * (t[n][seen] - float(tlse[n]) - logq[ids[seen]])).sum()
        Le = float(p.sum()) * eS
        target = torch.zeros(V, dtype=torch.float64).index_add_(0, ids, p)
        ge = (q + target) * (eq + eS + 6 * U)
        if rest > 0 and bool((u[out] > -math.inf).any()):
            mr = u[out].max()
            logR = torch.logsumexp(u[out] - mr, 0)
            share = torch.where(out, (u - mr - logR).exp(), torch.zeros_like(u))
            er = (3 * ((mr - u).clamp(min=0, max=1e6) + min(float(m - mr), 45.0)) + 4) * U
            er = torch.where(share > 0, er, torch.zeros_like(er))
            eR = float((share * er).sum()) + 200 * U
            L = L + rest * (math.log(rest) - (mr - m + logR - logS))
            Le = Le + rest * (eS + eR)
            target = target + rest * share
            ge = ge + rest * share * (er + eR + 6 * U)
        loss[n] = tau * tau * L
        loss_tol[n] = tau * tau * Le + (2 * U * loss[n].abs() if torch.isfinite(loss[n]) else 0.0)
        grad[n] = float(w[n]) * tau * (q - target)
        tol[n] = float(w[n]) * tau * ge + 2 * U * grad[n].abs()
    return (loss, loss_tol + 2.0 ** -149), (grad, tol + rounding(grad, dtype))


def rows(N, V, K, dtype, gap, tau, seed):
    """Logits of spread tau, the top's about gap * tau above the rest's."""
    g = gen(seed)
    z = tau * torch.randn(N, V, generator=g)
    tidx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    z.scatter_add_(1, tidx, torch.full((N, K), gap * tau))
    t = (tau * torch.randn(N, K, generator=g)).to(dtype)
    share = 0.3 + 0.69 * torch.rand(N, generator=g, dtype=torch.float64)
    tlse = (torch.logsumexp(t.double() / tau, 1) - share.log()).float()
    w = torch.rand(N, generator=g)
    w[0] = 65536.0 if dtype != torch.float16 else 64.0
    return z.to(dtype), tidx.to(torch.int32), t, tlse, w


def check(z, tidx, t, tlse, w, tau, copies=1):
    """All three calls on `copies` times the rows, in which the first are checked."""
    import sum_tree_sampling_amd as p
    N = z.shape[0]
    loss_want, grad_want = reference(z, tidx, t, tlse, tau, w, z.dtype)
    gz, gi, gt, gl, gw = (a.repeat(copies, *(1,) * (a.dim() - 1)).cuda() for a in (z, tidx, t, tlse, w))
    loss, grad = p.per_distill(gz, gi, gt, tlse=gl, temperature=tau, weight=gw)
    l2, saved = p.per_distill_forward(gz, gi, gt, tlse=gl, temperature=tau)
    g2 = p.per_distill_backward(gz, gi, gt, saved, gw, tlse=gl, temperature=tau)
    for lo in (0, (copies - 1) * N):
        k = slice(lo, lo + N)
        assert_close(loss[k], *loss_want, "loss")
        assert_close(l2[k], *loss_want, "forward loss")
        assert_close(grad[k], *grad_want, "grad")
        assert_close(g2[k], *grad_want, "backward grad")
    a = gz.clone()
    p.per_distill_backward(a, gi, gt, saved, gw, tlse=gl, temperature=tau, grad=a)
    assert torch.equal(a.view(torch.uint8), g2.view(torch.uint8))


GAPS = [0, 40, 50, 80, 87, 110, 500]


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("tau,dtype", [(0.01, "f32"), (0.1, "bf16"), (1.0, "f16"), (1.0, "f32"), (2.0, "bf16")])
@pytest.mark.parametrize("V,copies", [(300, 1), (1000, 1), (3001, 400)])
def test_rest_by_waves(V, copies, dtype, tau, gap):
    """Rows held by one wave each, alone and among many."""
    print("rest", V, copies, dtype, tau, gap, flush=True)
    check(*rows(4, V, 9, TYPES[dtype], gap, tau, V + gap), tau, copies)


@pytest.mark.parametrize("gap", [50, 87, 110, 500])
@pytest.mark.parametrize("tau,dtype", [(0.01, "f32"), (0.02, "bf16"), (1.0, "f16"), (2.0, "bf16")])
@pytest.mark.parametrize("V,copies", [(9001, 1), (11000, 200), (20000, 40), (30000, 200), (40001, 50), (66000, 60)])
def test_rest_by_workgroups(V, copies, dtype, tau, gap):
    """Rows held by one workgroup, by two hundred and more; the two calls apart take
    the long ones in parts."""
    print("rest", V, copies, dtype, tau, gap, flush=True)
    check(*rows(3, V, 70, TYPES[dtype], gap, tau, V + gap), tau, copies)


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("tau,dtype", [(0.01, "f32"), (1.0, "f32"), (0.1, "bf16"), (2.0, "f16")])
@pytest.mark.parametrize("V", [131071, 300001])
def test_rest_in_parts(V, dtype, tau, gap):
    print("rest", V, dtype, tau, gap, flush=True)
    check(*rows(2, V, 30, TYPES[dtype], gap, tau, V + gap), tau)


@pytest.mark.parametrize("V", [200, 9001, 150001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rest_masked(V, dtype):
    """The rest at the type's lowest value, one token of it left, none left, and a
    row whose top is ruled out."""
    z, tidx, t, tlse, w = rows(6, V, 5, TYPES[dtype], 3, 1.0, V)
    w[0] = 0.5
    top = torch.zeros(6, V, dtype=torch.bool).scatter_(1, tidx.long(), True)
    z[0] = torch.where(top[0], z[0], torch.tensor(torch.finfo(z.dtype).min, dtype=z.dtype))
    z[1] = torch.where(top[1], z[1], torch.tensor(-math.inf, dtype=z.dtype))
    z[1, int((~top[1]).nonzero()[V // 2])] = -200.0
    z[2] = torch.where(top[2], z[2], torch.tensor(-math.inf, dtype=z.dtype))
    z[3] = torch.where(top[3], torch.tensor(-300.0, dtype=z.dtype), z[3])
    z[4] = torch.where(top[4], z[4], torch.tensor(-math.inf, dtype=z.dtype))
    z[4, ~top[4]] = torch.where(torch.arange(V - 5) % 3 == 0, torch.tensor(-150.0, dtype=z.dtype), z[4, ~top[4]])
    check(z, tidx, t, tlse, w, 1.0)


@pytest.mark.parametrize("V", [200, 9001, 150001])
def test_rest_not_finite(V):
    """NaN and +Inf, in the rest or in the top, make the whole row NaN, also where
    the rest is far below the top."""
    import sum_tree_sampling_amd as p
    z, tidx, t, tlse, w = rows(5, V, 5, torch.float32, 120, 1.0, V)
    other = int((~torch.zeros(V, dtype=torch.bool).scatter_(0, tidx[0].long(), True)).nonzero()[V // 3])
    z[0, other] = math.nan
    other = int((~torch.zeros(V, dtype=torch.bool).scatter_(0, tidx[1].long(), True)).nonzero()[V // 3])
    z[1, other] = math.inf
    z[2, tidx[2, 1].long()] = math.nan
    z[3, tidx[3, 1].long()] = math.inf
    args = [a.cuda() for a in (z, tidx, t)]
    loss, grad = p.per_distill(*args, tlse=tlse.cuda())
    l2, saved = p.per_distill_forward(*args, tlse=tlse.cuda())
    g2 = p.per_distill_backward(*args, saved, torch.ones(5).cuda(), tlse=tlse.cuda())
    for v in (loss, l2):
        assert torch.isnan(v[:4]).all() and torch.isfinite(v[4])
    for v in (grad, g2):
        assert torch.isnan(v[:4]).all() and torch.isfinite(v[4]).all()


def test_rest_differences():
    """The rest's gradient against differences of the loss, 100 tau below the top."""
    import sum_tree_sampling_amd as p
    z, tidx, t, tlse, _ = rows(3, 500, 6, torch.float32, 100, 1.0, 5)
    gz, gi, gt, gl = (a.cuda() for a in (z, tidx, t, tlse))
    _, grad = p.per_distill(gz, gi, gt, tlse=gl)
    r = torch.randn(z.shape, generator=gen(1)).cuda()
    eps = 2.0 ** -6

    def f(v):
        return p.per_distill_forward(v, gi, gt, tlse=gl)[0].double()

    num = (f(gz + eps * r) - f(gz - eps * r)) / (2 * eps)
    ana = (grad.double() * r.double()).sum(1)
    # third derivative by one direction: at most about 8; the loss, below 100, is rounded to f32, and z + eps r to
    # steps of 2^-17 of logits near 100
    assert ((num - ana).abs() <= eps ** 2 * 8 + 64 * U * 128 / eps).all(), (num, ana)


@pytest.mark.parametrize("tau", [8.0, 20.0, 32.0, 64.0])
@pytest.mark.parametrize("V,K,N", [(4001, 30, 1100), (9001, 64, 64), (30000, 64, 200), (120000, 50, 16)])
def test_loss_at_large_temperatures(V, K, N, tau):
    """A student near its teacher, whose loss is far below tau^2.  An exponential is
    off by at most 4 u and they are independent, so the mean of V of them is off by
    less than 4 * 4 u / sqrt(V) (four standard deviations), S and S_r alike."""
    import sum_tree_sampling_amd as p
    teacher = torch.randn(N, V, generator=gen(V))
    z = teacher + 0.06 * torch.randn(N, V, generator=gen(1))
    t, at = teacher.topk(K, 1)
    tlse = torch.logsumexp(teacher.double() / tau, 1).float()
    logp = t.double() / tau - tlse.double()[:, None]
    logq = torch.log_softmax(z.double() / tau, 1)
    rest = 1 - logp.exp().sum(1)
    log_rest = torch.logsumexp(logq.scatter(1, at, -math.inf), 1)
    want = tau * tau * ((logp.exp() * (logp - logq.gather(1, at))).sum(1) + rest * (rest.log() - log_rest))
    args = (z.cuda(), at.to(torch.int32).cuda(), t.cuda())
    fused, _ = p.per_distill(*args, tlse=tlse.cuda(), temperature=tau)
    apart, _ = p.per_distill_forward(*args, tlse=tlse.cuda(), temperature=tau)
    tol = tau * tau * 32 * U / math.sqrt(V) + 2 * U * want.abs()
    assert_close(fused, want, tol, "loss")
    assert_close(apart, want, tol, "forward loss")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V", [("f32", 262140), ("bf16", 200003), ("f32", 131073)])
def test_long_rows_in_one_part(dtype, V, tail):
    """From 641 rows on a row of up to 2^18 tokens is one workgroup's, whose threads
    add up to 1024 exponentials each: 8 or 16 at a time, so that no sum is longer than 128
    + 16 roundings.  One of the rows has nearly equal logits."""
    import sum_tree_sampling_amd as p
    from train_oracle import distill
    N, K, tau = 1300, 40, 1.2
    g = gen(V)
    z = 3 * torch.randn(3, V, generator=g)
    z[1] = 1e-3 * torch.randn(V, generator=g)
    z = z.to(TYPES[dtype])
    tidx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(3)]).to(torch.int32)
    t, w = (3 * torch.randn(3, K, generator=g)).to(TYPES[dtype]), torch.rand(3, generator=g)
    tlse = (torch.logsumexp(t.double() / tau, 1) + 0.5).float() if tail else None
    want = distill(z, tidx, t, tlse, tau, w, z.dtype)
    plain = distill(z, tidx, t, tlse, tau, None, z.dtype)["loss"]
    at = torch.arange(N) % 3
    gz, gi, gt, gw = (a.cuda()[at.cuda()] for a in (z, tidx, t, w))
    gl = None if tlse is None else tlse[at].cuda()
    loss, saved = p.per_distill_forward(gz, gi, gt, tlse=gl, temperature=tau)
    grad = p.per_distill_backward(gz, gi, gt, saved, gw, tlse=gl, temperature=tau)
    for lo in (0, N // 3 * 3 - 3):
        assert_close(loss[lo:lo + 3], *plain, "loss")
        assert_close(grad[lo:lo + 3], *want["grad"], "grad")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,N", [(300, 5), (4000, 1100), (11000, 520), (40000, 130), (150001, 3)])
def test_rows_of_weight_0(V, N, tail):
    """Loss 0 and gradient 0, whatever the row's logits, entries and normaliser hold."""
    import sum_tree_sampling_amd as p
    K = 5
    z = torch.randn(N, V, device="cuda")
    tidx = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t, w = torch.randn(N, K, device="cuda"), torch.rand(N, device="cuda") + 0.1
    tlse = torch.logsumexp(t, 1) + 0.5 if tail else None
    clean = p.per_distill(z, tidx, t, tlse=tlse, weight=w)
    off = torch.arange(N, device="cuda") % 3 == 1
    w[off] = 0.0
    z[off] = math.nan
    t[off] = math.inf
    tidx[off] = -7
    if tail:
        tlse[off] = math.nan
    loss, grad = p.per_distill(z, tidx, t, tlse=tlse, weight=w)
    _, saved = p.per_distill_forward(z, tidx, t, tlse=tlse)
    g2 = p.per_distill_backward(z, tidx, t, saved, w, tlse=tlse)
    assert not loss[off].any() and not grad[off].any() and not g2[off].any()
    assert torch.equal(loss[~off], clean[0][~off]) and torch.equal(grad[~off], clean[1][~off])
