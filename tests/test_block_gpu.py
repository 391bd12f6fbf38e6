"""The operators of include/per_block.h on the GPU against their 64-bit forms, within
the error bounds that the oracle carries along with each value."""
import math

import pytest
import torch

import block_oracle as O
from train_oracle import TYPES, assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


def per():
    import sum_tree_sampling_amd as p
    return p


def gen(seed):
    return torch.Generator().manual_seed(seed)


def say(*a):
    print(*a, flush=True)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ embedding

def tokens_of(n, v, index, seed, hot=0.3, padding=0.1):
    g = gen(seed)
    t = torch.randint(0, v, (n,), generator=g)
    t = torch.where(torch.rand(n, generator=g) < hot, v // 2, t)
    r = torch.rand(n, generator=g)
    far = -(1 << 31) if index == torch.int32 else -(1 << 40)
    t = torch.where(r < padding, torch.where(r < padding / 2, -1, torch.where(r < 0.75 * padding, v, far)), t)
    return t.to(index)


@pytest.mark.parametrize("n,v,d", [(0, 5, 8), (1, 1, 1), (1, 1000, 333), (63, 7, 9), (512, 50000, 256), (1000, 501, 2049),
                                   (5, 3, 5000)])
@pytest.mark.parametrize("table", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_embed_forward(n, v, d, table, out):
    p = per()
    g = gen(n + d)
    big = torch.randn(v, d + 3, generator=g).to(TYPES[table]).cuda()
    tab = big[:, 1:d + 1]  # rows apart, not aligned
    t = tokens_of(n, v, torch.int32 if n % 2 else torch.int64, d)
    want, tol = O.embed(t, tab, math.sqrt(d), TYPES[out])
    got = p.per_embed_forward(t.cuda(), tab, scale=math.sqrt(d), dtype=TYPES[out])
    assert_close(got, want, tol, "out")
    room = torch.full((n, d + 2), 7.0, dtype=TYPES[out], device=DEV)
    p.per_embed_forward(t.cuda(), tab, scale=math.sqrt(d), out=room[:, 1:d + 1])
    assert same(room[:, 1:d + 1], got) and (room[:, 0] == 7).all() and (room[:, -1] == 7).all()


@pytest.mark.parametrize("n,v,d", [(0, 5, 8), (1, 1, 1), (7, 1, 33), (64, 100000, 3), (65, 3, 520), (1000, 501, 2049), (1024, 70000, 16),
                                   (1025, 511, 64), (8192, 512, 100), (8193, 513, 65), (20001, 501, 333), (70001, 200003, 24),
                                   (300000, 1000, 8)])
@pytest.mark.parametrize("dout,grad", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_embed_backward(n, v, d, dout, grad):
    p = per()
    say("embed backward", n, v, d, dout, grad)
    g = gen(n + v + d)
    rows = torch.randn(n, d + 1, generator=g).to(TYPES[dout]).cuda()[:, :d]
    t = tokens_of(n, v, torch.int32 if n % 2 else torch.int64, v)
    want, tol = O.embed_grad(t, rows, v, 0.5, TYPES[grad])
    room = torch.full((v, d + 2), 7.0, dtype=TYPES[grad], device=DEV)
    got = p.per_embed_backward(t.cuda(), rows, v, scale=0.5, grad=room[:, 1:d + 1])
    assert_close(got, want, tol, "grad")
    assert (room[:, 0] == 7).all() and (room[:, -1] == 7).all()
    again = p.per_embed_backward(t.cuda(), rows, v, scale=0.5, grad=torch.empty_like(got))
    assert same(again, got)
    old = torch.randn(v, d, generator=g).to(TYPES[grad]).cuda()
    want, tol = O.embed_grad(t, rows, v, 0.5, TYPES[grad], old)
    into = old.clone()
    p.per_embed_backward(t.cuda(), rows, v, scale=0.5, grad=into, accumulate=True)
    assert_close(into, want, tol, "accumulated")
    absent = torch.ones(v, dtype=torch.bool)
    k = t.long()
    absent[k[(k >= 0) & (k < v)]] = False
    assert same(into.cpu()[absent], old.cpu()[absent])


@pytest.mark.parametrize("n", [300, 9000, 40000])
@pytest.mark.parametrize("kind", ["one", "absent", "rising", "runs"])
def test_embed_backward_orders(n, kind):
    """One token for all rows; none at all; each its own; runs that end on chunk borders."""
    p = per()
    v, d = 1 << 16, 40
    k = torch.arange(n)
    t = {"one": torch.full((n,), v - 1), "absent": torch.full((n,), v), "rising": k, "runs": k // 64 * 3}[kind]
    rows = torch.randn(n, d, generator=gen(n)).cuda()
    want, tol = O.embed_grad(t, rows, v, 1.0)
    assert_close(p.per_embed_backward(t.cuda(), rows, v), want, tol, kind)


def test_embed_values_stay_in_their_rows():
    """Infinities and NaN in the rows of absent tokens, and of other tokens."""
    p = per()
    t = torch.tensor([3, -1, 5, 3, 99, 5])
    rows = torch.ones(6, 20)
    rows[1] = math.nan
    rows[4] = math.inf
    rows[2] = math.nan
    got = p.per_embed_backward(t.cuda(), rows.cuda(), 50).cpu()
    assert torch.isnan(got[5]).all() and (got[3] == 2).all()
    got[5] = 0
    got[3] = 0
    assert not got.any()
    table = torch.randn(50, 20)
    table[7] = math.inf
    got = p.per_embed_forward(torch.tensor([-1, 7, 50, 8]).cuda(), table.cuda(), scale=2.0).cpu()
    assert not got[0].any() and not got[2].any() and torch.isinf(got[1]).all() and same(got[3], 2 * table[8])


# ----------------------------------------------------------------- layer norm

NORM = [(1, 1), (3, 2), (5, 7), (33, 64), (70, 128), (9, 129), (513, 300), (4095, 1001), (100, 1024), (70, 2048), (7, 4095),
        (6, 8192), (3, 16000), (2, 33000), (2, 70001)]


@pytest.mark.parametrize("n,d", NORM)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["f32", "own", "none", "weight"])
def test_norm(n, d, dtype, kind):
    p = per()
    dt = TYPES[dtype]
    say("norm", n, d, dtype, kind)
    g = gen(n + d)
    x = (torch.randn(n, d + 5, generator=g) + 3 * torch.randn(n, 1, generator=g)).to(dt).cuda()[:, 2:d + 2]
    dy = torch.randn(n, d + 1, generator=g).to(dt).cuda()[:, :d]
    at = torch.float32 if kind != "own" else dt
    w = None if kind == "none" else (1 + torch.randn(d, generator=g)).to(at).cuda()
    b = None if kind in ("none", "weight") else torch.randn(d, generator=g).to(at).cuda()
    want = O.norm(x, w, b, 1e-5, dy)
    y, stats = p.per_norm_forward(x, w, b, eps=1e-5)
    assert_close(y, *want["y"], "y")
    assert_close(stats[:, 0], *want["mean"], "mean")
    assert_close(stats[:, 1], *want["rstd"], "rstd")
    dx, dw, db = p.per_norm_backward(x, stats, dy, w)
    assert_close(dx, *want["dx"], "dx")
    assert_close(dw, *want["dweight"], "dweight")
    assert_close(db, *want["dbias"], "dbias")
    only, none, none2 = p.per_norm_backward(x, stats, dy, w, sums=False)
    assert same(only, dx) and none is None and none2 is None
    inplace = dy.clone()
    p.per_norm_backward(x, stats, inplace, w, dx=inplace)
    assert same(inplace, dx)
    inplace = x.clone()
    p.per_norm_forward(inplace, w, b, eps=1e-5, y=inplace)
    assert same(inplace, y)
    again = p.per_norm_backward(x, stats, dy, w)
    assert all(same(i, j) for i, j in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("n", [0, 1, 2047, 2049, 20000])
def test_norm_row_counts(n):
    p = per()
    x, dy = (torch.randn(n, 24, generator=gen(n + i)).cuda() for i in range(2))
    want = O.norm(x, None, None, 1e-3, dy)
    y, stats = p.per_norm_forward(x, eps=1e-3)
    out = p.per_norm_backward(x, stats, dy)
    assert_close(y, *want["y"], "y")
    for got, name in zip(out, ("dx", "dweight", "dbias")):
        assert_close(got, *want[name], name)


def test_norm_odd_rows():
    """Equal values; a mean far from its deviation; values that are not finite; a row past f32's squares."""
    p = per()
    g = gen(4)
    x = torch.randn(8, 300, generator=g)
    x[0] = 2.5
    x[1] += 1e4
    x[2, 7] = math.nan
    x[3, 9] = math.inf
    x[4] *= 1e-20
    w = torch.randn(300, generator=g)
    y, stats = (t.cpu() for t in p.per_norm_forward(x.cuda(), w.cuda()))
    assert (y[0] == 0).all() and stats[0, 0] == 2.5
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    ok = torch.tensor([1, 4, 5, 6, 7])
    want = O.norm(x[ok], w)
    assert_close(y[ok], *want["y"], "y")
    zero = p.per_norm_forward(torch.zeros(2, 300, device=DEV), eps=0.0)[1].cpu()
    assert torch.isinf(zero[:, 1]).all()


# ----------------------------------------------------------- gated delta rule

def delta_case(B, T, H, HK, DK, DV, dtype, seed, ragged=False, resets=0.02, wide=True):
    """Inputs as views with gaps between rows; what lies past a sequence's end is NaN."""
    g = gen(seed)
    dt = TYPES[dtype]

    def r(*s):
        return torch.randn(*s, generator=g)
    q, k = r(B, T, HK, DK), r(B, T, HK, DK) + 0.5 * r(B, 1, HK, DK)
    q, k = (torch.nn.functional.normalize(x, dim=-1).to(dt) for x in (q, k))
    gate, write = (r(B, T, H) * 2 + 2).to(dt), r(B, T, H).to(dt)
    a = dict(q=q, k=k, v=r(B, T, H, DV).to(dt), g=gate, b=write, do=r(B, T, H, DV).to(dt))
    a["length"] = torch.randint(0, T + 1, (B,), generator=g) if ragged else None
    if ragged:
        past = torch.arange(T) >= a["length"][:, None]
        for x in ("q", "k", "v", "g", "b", "do"):
            a[x][past] = math.nan
    a["reset"] = torch.rand(B, T, generator=g) < resets
    a["s0"], a["ds_last"] = r(B, H, DK, DV), r(B, H, DK, DV)
    a["scale"] = DK ** -0.5
    dev = {}
    for x, y in a.items():
        if torch.is_tensor(y):
            if wide and x in ("q", "k", "v", "do"):  # heads' rows apart, at odd places
                room = torch.full((*y.shape[:-1], y.shape[-1] + 3), math.nan, dtype=y.dtype)
                room[..., 1:y.shape[-1] + 1] = y
                dev[x] = room.cuda()[..., 1:y.shape[-1] + 1]
            else:
                dev[x] = y.cuda()
        else:
            dev[x] = y
    return a, dev


def clean(a):
    """The oracle's inputs: nothing past the end."""
    b = dict(a)
    if a["length"] is not None:
        past = torch.arange(a["q"].shape[1]) >= a["length"][:, None]
        for x in ("q", "k", "v", "g", "b", "do"):
            b[x] = a[x].clone()
            b[x][past] = 0
    return b


def run(p, d, save=True, **kw):
    o, s, c = p.per_delta_forward(*(d[x] for x in "qkvgb"), reset=d["reset"], length=d["length"], s0=d["s0"],
                                  scale=d["scale"], save=save, **kw)
    return o, s, c


def back(p, d, c, **kw):
    return p.per_delta_backward(*(d[x] for x in "qkvgb"), c, d["do"], reset=d["reset"], length=d["length"],
                                ds_last=d["ds_last"], scale=d["scale"], **kw)


GRADS = ("dq", "dk", "dv", "dg", "db", "ds0")


def check_delta(dev, host, dtype):
    p = per()
    a = clean(host)
    want = O.delta_all(**a)
    size = O.delta_size(**a)
    tol = O.delta_tolerance(size, want, TYPES[dtype])
    o, s, c = run(p, dev)
    assert_close(o, want["o"], tol["o"], "o")
    assert_close(s, want["s"], tol["s"], "s")
    grads = back(p, dev, c)
    for name, got in zip(GRADS, grads):
        assert_close(got, want[name], tol[name], name)
    return o, s, c, grads


@pytest.mark.parametrize("B,T,H,HK,DK,DV", [
    (1, 1, 1, 1, 1, 1), (2, 3, 2, 1, 8, 5), (1, 63, 1, 1, 16, 16), (2, 64, 2, 2, 32, 64), (1, 65, 2, 1, 33, 65),
    (2, 130, 4, 2, 48, 33), (1, 200, 2, 2, 64, 64), (1, 257, 1, 1, 65, 129), (2, 100, 3, 1, 100, 40), (1, 192, 2, 1, 128, 128),
    (1, 128, 1, 1, 127, 256), (1, 70, 8, 1, 24, 200)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ragged", [False, True])
def test_delta(B, T, H, HK, DK, DV, dtype, ragged):
    say("delta", B, T, H, HK, DK, DV, dtype, ragged)
    host, dev = delta_case(B, T, H, HK, DK, DV, dtype, T + DK, ragged, resets=0.05)
    check_delta(dev, host, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_long(dtype):
    host, dev = delta_case(1, 1500, 1, 1, 16, 16, dtype, 5, wide=False)
    check_delta(dev, host, dtype)


@pytest.mark.parametrize("B,T,H,HK,DK,DV,resets", [(2, 1300, 2, 1, 33, 40, 0.0), (1, 1024, 1, 1, 128, 70, 0.002),
                                                   (3, 1000, 1, 1, 8, 8, 0.01)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_delta_cut(B, T, H, HK, DK, DV, resets, dtype):
    """Few long sequences, whose time axis is cut, some of them ending early."""
    host, dev = delta_case(B, T, H, HK, DK, DV, dtype, T, ragged=B > 1, resets=resets)
    if B > 1:
        host["length"][0] = T - 3
        dev["length"] = host["length"].cuda()
        host, dev = delta_recut(host, dev)
    check_delta(dev, host, dtype)


def delta_recut(host, dev):
    """NaN past the (changed) ends, and finite values before them."""
    past = torch.arange(host["q"].shape[1]) >= host["length"][:, None]
    for x in ("q", "k", "v", "g", "b", "do"):
        host[x] = torch.where(torch.isnan(host[x]), torch.full_like(host[x], 0.125), host[x])
        host[x][past] = math.nan
        dev[x].copy_(host[x])
    return host, dev


def test_delta_cut_masked_states():
    """A state that is not finite does not pass a reset where the time axis is cut."""
    p = per()
    host, dev = delta_case(2, 1100, 1, 1, 32, 48, "f32", 8, resets=0.0)
    dev["reset"][0, 0] = True
    dev["reset"][1, 300] = True
    good = run(p, dev)
    gg = back(p, dev, good[2])
    s0 = dev["s0"].clone()
    s0[0] = math.nan
    s0[1, 0, 3, 5] = math.inf
    bad = run(p, dict(dev, s0=s0))
    assert same(bad[0][0], good[0][0]) and same(bad[1], good[1]) and same(bad[0][1, 300:], good[0][1, 300:])
    gb = back(p, dict(dev, s0=s0), bad[2])
    assert all(same(x[0], y[0]) and same(x[1, 300:], y[1, 300:]) for x, y in zip(gb[:5], gg[:5])) and same(gb[5], gg[5])
    d = dev["ds_last"].clone()
    d[1] = math.nan
    gb = back(p, dict(dev, ds_last=d), good[2])
    assert all(same(x[1, :300], y[1, :300]) for x, y in zip(gb[:5], gg[:5])) and same(gb[5], gg[5])


def test_delta_gates_and_strengths():
    """Gates shut and open, strengths of 0 and 1, keys that repeat, a reset at every step."""
    B, T = 4, 150
    host, dev = delta_case(B, T, 2, 2, 32, 32, "f32", 9, resets=0.0, wide=False)
    host["g"][0, ::3] = -60
    host["g"][0, 1::3] = 60
    host["g"][1] = 40
    host["b"][1, ::2] = -120
    host["b"][1, 1::2] = 120
    host["k"][2] = host["k"][2, :1]
    host["reset"][3] = True
    dev.update({x: y.cuda() for x, y in host.items() if torch.is_tensor(y)})
    check_delta(dev, host, "f32")
    assert not back(per(), dev, run(per(), dev)[2])[5][3].any()  # nothing gets past a reset
    host["g"][0, 5] = -math.inf
    host["g"][0, 70] = math.inf
    dev["g"] = host["g"].cuda()
    o, s, c = run(per(), dev)
    assert torch.isfinite(o).all() and torch.isfinite(s).all()
    assert all(torch.isfinite(x).all() for x in back(per(), dev, c))
    o2, s2, _ = run(per(), dict(dev, s0=dev["s0"] + 1))  # nor past a gate that is 0
    assert same(o2[0, 5:], o[0, 5:]) and same(s2[0], s[0])


def test_delta_without_states_and_masks():
    host, dev = delta_case(2, 90, 2, 1, 24, 24, "f32", 3, resets=0.0)
    for a in (host, dev):
        a["reset"] = a["s0"] = a["ds_last"] = None
    check_delta(dev, host, "f32")


@pytest.mark.parametrize("T", [0, 5, 100])
def test_delta_empty(T):
    """No steps, by T or by length: the state stays, gradients of the steps are 0."""
    p = per()
    host, dev = delta_case(3, T, 2, 2, 24, 40, "bf16", 1)
    dev["length"] = torch.tensor([0, -4, 0]).cuda()
    o, s, c = run(p, dev)
    assert not o.any() and same(s, dev["s0"])
    g = back(p, dev, c)
    assert not any(x.any() for x in g[:5]) and same(g[5], dev["ds_last"])
    none = {x: (y[:0] if torch.is_tensor(y) else y) for x, y in dev.items()}
    o, s, c = run(p, none)
    assert o.shape == (0, T, 2, 40) and [x.shape[0] for x in back(p, none, c)] == [0] * 6


def test_delta_lengths_past_the_end_are_clamped():
    p = per()
    host, dev = delta_case(2, 70, 1, 1, 16, 16, "f32", 1)
    o, s, c = run(p, dev)
    dev["length"] = torch.tensor([70, 1 << 40]).cuda()
    o2, s2, c2 = run(p, dev)
    assert same(o, o2) and same(s, s2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_masked_states(dtype):
    """A state that is not finite does not pass a reset; other sequences and heads are not touched."""
    p = per()
    host, dev = delta_case(3, 200, 2, 2, 32, 48, dtype, 8, resets=0.0)
    dev["reset"][0, 0] = True
    dev["reset"][1, 100] = True
    good = run(p, dev)
    gg = back(p, dev, good[2])
    s0 = dev["s0"].clone()
    s0[0] = math.nan
    s0[1, 0, 3, 5] = math.inf
    bad = run(p, dict(dev, s0=s0))
    assert same(bad[0][0], good[0][0]) and same(bad[1], good[1])
    assert same(bad[0][1, :, 1], good[0][1, :, 1]) and same(bad[0][2], good[0][2])
    assert same(bad[0][1, 100:], good[0][1, 100:])
    gb = back(p, dict(dev, s0=s0), bad[2])
    for x, y in zip(gb[:5], gg[:5]):
        assert same(x[0], y[0]) and same(x[2], y[2]) and same(x[1, 100:], y[1, 100:])
    assert same(gb[5], gg[5])  # the gradient by a state does not use it
    d = dev["ds_last"].clone()
    d[1, 0] = math.nan
    gb = back(p, dict(dev, ds_last=d), good[2])
    assert same(gb[5], gg[5])
    for x, y in zip(gb[:5], gg[:5]):
        assert same(x[0], y[0]) and same(x[2], y[2]) and same(x[1, :100], y[1, :100])


def test_delta_is_the_same_in_pieces():
    """Two calls that hand the state on, against one."""
    p = per()
    host, dev = delta_case(2, 192, 2, 1, 32, 32, "f32", 2, resets=0.02, wide=False)
    o, s, c = run(p, dev)
    half = 128
    one = {x: (y[:, :half] if x in ("q", "k", "v", "g", "b") else y) for x, y in dev.items()}
    two = {x: (y[:, half:] if x in ("q", "k", "v", "g", "b") else y) for x, y in dev.items()}
    one["reset"], two["reset"] = dev["reset"][:, :half].contiguous(), dev["reset"][:, half:].contiguous()
    o1, s1, _ = run(p, one, save=False)
    two["s0"] = s1
    o2, s2, _ = run(p, two, save=False, s_last=s1)  # in place
    assert same(torch.cat([o1, o2], 1), o) and same(s2, s)


def test_delta_views():
    """Slices of one projection in, slices of one gradient out, heads before steps."""
    p = per()
    B, T, H, D = 2, 100, 3, 32
    host, dev = delta_case(B, T, H, H, D, D, "bf16", 4, wide=False)
    o, s, c = run(p, dev)
    want = back(p, dev, c)
    one = torch.cat([dev["q"], dev["k"], dev["v"], dev["g"][..., None], dev["b"][..., None]], -1)
    one = one.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    grad = torch.full_like(one, 7)
    parts = torch.split(one, [D, D, D, 1, 1], -1)
    outs = torch.split(grad, [D, D, D, 1, 1], -1)
    view = dict(dev, q=parts[0], k=parts[1], v=parts[2], g=parts[3][..., 0], b=parts[4][..., 0])
    o2, s2, c2 = run(p, view)
    assert same(o, o2) and same(s, s2) and same(c, c2)
    got = back(p, view, c2, dq=outs[0], dk=outs[1], dv=outs[2], dg=outs[3][..., 0], db=outs[4][..., 0])
    assert all(same(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_expanded_inputs(dtype):
    """Steps, heads and sequences that share their rows."""
    p = per()
    host, dev = delta_case(2, 90, 2, 2, 32, 40, dtype, 7, wide=False)
    for a in (host, dev):
        a["length"] = torch.tensor([70, 90]).to(a["q"].device)
        a["q"] = a["q"][:, :1].expand(-1, 90, -1, -1)
        a["k"] = a["k"][:, :, :1].expand(-1, -1, 2, -1)
        a["v"] = a["v"][:, :1].expand(-1, 90, -1, -1)
        a["do"] = a["do"][:1, :1].expand(2, 90, -1, -1)
        a["g"] = a["g"][:, :1].expand(-1, 90, -1)
    check_delta(dev, {k: v.contiguous() if torch.is_tensor(v) else v for k, v in host.items()}, dtype)


@pytest.mark.parametrize("B,H,HK,DK,DV", [(1, 1, 1, 1, 1), (3, 2, 1, 64, 64), (5, 4, 2, 33, 65), (2, 2, 2, 128, 128),
                                          (2, 1, 1, 100, 256), (70, 3, 3, 17, 129)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_delta_step(B, H, HK, DK, DV, dtype):
    p = per()
    host, dev = delta_case(B, 1, H, HK, DK, DV, dtype, DK, resets=0.3)
    want = O.delta_all(*(host[x] for x in "qkvgb"), reset=host["reset"], s0=host["s0"], scale=host["scale"])
    tol = O.delta_tolerance(O.delta_size(*(host[x] for x in "qkvgb"), reset=host["reset"], s0=host["s0"],
                                         scale=host["scale"]), want, TYPES[dtype])
    one = [dev[x][:, 0] for x in "qkvgb"]
    reset = dev["reset"][:, 0].contiguous()
    s_out = torch.empty_like(dev["s0"])
    o, s = p.per_delta_step(*one, dev["s0"], reset=reset, scale=host["scale"], s_out=s_out)
    assert s.data_ptr() == s_out.data_ptr()
    assert_close(o, want["o"][:, 0], tol["o"][:, 0], "o")
    assert_close(s, want["s"], tol["s"], "s")
    state = dev["s0"].clone()
    o2, s2 = p.per_delta_step(*one, state, reset=reset, scale=host["scale"])
    assert s2.data_ptr() == state.data_ptr() and same(o2, o) and same(s2, s)
    state = torch.full_like(state, math.nan)
    o3, s3 = p.per_delta_step(*one, state, reset=torch.ones_like(reset), scale=host["scale"])
    assert torch.isfinite(o3.float()).all() and torch.isfinite(s3).all()


def test_delta_step_fills_the_chip():
    """Every store of a state waits behind many others."""
    p = per()
    B, H, D = 256, 16, 128
    host, dev = delta_case(1, 1, H, H, D, D, "f32", 12)
    want = O.delta_all(*(host[x] for x in "qkvgb"), s0=host["s0"], scale=host["scale"])
    tol = O.delta_tolerance(O.delta_size(*(host[x] for x in "qkvgb"), s0=host["s0"], scale=host["scale"]), want,
                            torch.float32)
    one = [dev[x][:, 0].expand(B, *dev[x].shape[2:]) for x in "qkvgb"]
    s0 = dev["s0"].repeat(B, 1, 1, 1)
    for _ in range(3):
        o, s = p.per_delta_step(*one, s0, scale=dev["scale"], s_out=torch.empty_like(s0))
        assert same(s, s[:1].expand_as(s)) and same(o, o[:1].expand_as(o))
        assert_close(s[0], want["s"][0], tol["s"][0], "s")


def test_delta_steps_follow_the_sequence():
    p = per()
    B, T, H, D = 2, 70, 2, 32
    host, dev = delta_case(B, T, H, 1, D, D, "f32", 6, resets=0.05)
    o, s, _ = run(p, dev, save=False)
    state = dev["s0"].clone()
    size = O.delta_size(*(host[x] for x in "qkvgb"), reset=host["reset"], s0=host["s0"], scale=host["scale"])
    tol = O.delta_tolerance(size, {"o": o.cpu().double(), "s": s.cpu().double()}, torch.float32)
    for t in range(T):
        ot, _ = p.per_delta_step(*(dev[x][:, t] for x in "qkvgb"), state, reset=dev["reset"][:, t].contiguous(),
                                 scale=dev["scale"])
        assert_close(ot, o[:, t], 2 * tol["o"][:, t], "o")
    assert_close(state, s, 2 * tol["s"], "s")


# ---------------------------------------------------- streams, graphs, the whole

def block(p, d):
    """Every operator after the others, as a student runs them: (loss, gradients)."""
    B, T, H, D = d["shape"]
    dim = H * D
    x = p.per_embed_forward(d["tokens"], d["table"], scale=4.0, dtype=d["dtype"])
    y, st = p.per_norm_forward(x, d["w"], d["b"])
    proj = (y @ d["p"]).view(B, T, H, 3 * D + 2)
    parts = [proj[..., :D], proj[..., D:2 * D], proj[..., 2 * D:3 * D], proj[..., 3 * D], proj[..., 3 * D + 1]]
    n = [p.per_norm_forward(parts[i].reshape(-1, D), eps=1e-6) for i in range(2)]
    qk = [(z[0] * D ** -0.5).view(B, T, H, D) for z in n]
    o, s, c = p.per_delta_forward(*qk, *parts[2:], reset=d["reset"], s0=d["s0"])
    z, zs = p.per_norm_forward(o.view(-1, dim), d["w"], d["b"])
    logits = z @ d["table"].to(d["dtype"]).t()
    loss, dl = p.per_distill(logits, d["tidx"], d["tlogit"])
    dz = dl @ d["table"].to(d["dtype"])
    do, dw, db = p.per_norm_backward(o.view(-1, dim), zs, dz, d["w"])
    g = p.per_delta_backward(*qk, *parts[2:], c, do.view_as(o), reset=d["reset"])
    dproj = torch.empty_like(proj)
    for i in range(2):
        dn, _, _ = p.per_norm_backward(parts[i].reshape(-1, D), n[i][1], (g[i] * D ** -0.5).reshape(-1, D), sums=False)
        dproj[..., i * D:(i + 1) * D] = dn.view(B, T, H, D)
    dproj[..., 2 * D:3 * D], dproj[..., 3 * D], dproj[..., 3 * D + 1] = g[2], g[3], g[4]
    flat = dproj.view(B * T, -1)
    dy, dp = flat @ d["p"].t(), y.t() @ flat
    dx, dw2, db2 = p.per_norm_backward(x, st, dy, d["w"])
    dt = p.per_embed_backward(d["tokens"], dx, d["table"].shape[0], scale=4.0)
    return [loss, dp, dw, db, dw2, db2, dt, g[5]]


def block_inputs(dtype, seed=0):
    B, T, H, D, V, K = 3, 70, 2, 32, 97, 5
    g = gen(seed)

    def r(*s):
        return torch.randn(*s, generator=g)
    return dict(shape=(B, T, H, D), dtype=TYPES[dtype], tokens=torch.randint(-1, V, (B * T,), generator=g).cuda(),
                table=(0.3 * r(V, H * D)).cuda(), w=(1 + 0.1 * r(H * D)).cuda(), b=(0.1 * r(H * D)).cuda(),
                p=(r(H * D, H * (3 * D + 2)) * (H * D) ** -0.5).to(TYPES[dtype]).cuda(),
                reset=(torch.rand(B, T, generator=g) < 0.02).cuda(), s0=(0.1 * r(B, H, D, D)).cuda(),
                tidx=torch.randint(0, V, (B * T, K), generator=g).to(torch.int32).cuda(), tlogit=r(B * T, K).cuda())


def block_plain(d):
    """The same student in f64 on the CPU, its gradients by autograd: gradients of the
    first projection, both norms' weights, the embedding's use of the table and s0."""
    B, T, H, D = d["shape"]
    c = {k: (v.cpu().double() if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in d.items()}
    leaf = {k: c[k].clone().requires_grad_() for k in ("p", "s0")}
    w1, b1, w2, b2 = (c[k].clone().requires_grad_() for k in ("w", "b", "w", "b"))
    table = c["table"].clone().requires_grad_()
    tok = d["tokens"].cpu()
    x = torch.where((tok >= 0)[:, None], 4.0 * table[tok.clamp(min=0)], 0.0)

    def norm(x, w=None, b=None, eps=1e-5):
        return torch.nn.functional.layer_norm(x, x.shape[-1:], w, b, eps)
    y = norm(x, w1, b1)
    proj = (y @ leaf["p"]).view(B, T, H, 3 * D + 2)
    q, k = (norm(proj[..., i * D:(i + 1) * D], eps=1e-6) * D ** -0.5 for i in range(2))
    o, _ = O.delta(q, k, proj[..., 2 * D:3 * D], proj[..., 3 * D], proj[..., 3 * D + 1], reset=d["reset"].cpu(), s0=leaf["s0"])
    z = norm(o.reshape(-1, H * D), w2, b2)
    logq = torch.log_softmax(z @ c["table"].t(), 1)
    lp = torch.log_softmax(c["tlogit"], 1)
    loss = (lp.exp() * (lp - logq.gather(1, d["tidx"].cpu().long()))).sum(1)
    loss.sum().backward()
    return [loss.detach(), leaf["p"].grad, w2.grad, b2.grad, w1.grad, b1.grad, table.grad, leaf["s0"].grad]


def test_the_whole_student():
    """All of them in a row against f64 and autograd.  In f32 each of some ten operators
    in turn is off by some tens of u of its terms; 1e-3 of each gradient's own norm leaves
    that (10 * 64 * u = 4e-5) room to grow through the products between them."""
    p = per()
    d = block_inputs("f32")
    got, want = block(p, d), block_plain(d)
    for i, (x, y) in enumerate(zip(got, want)):
        assert (x.cpu().double() - y).norm() <= 1e-3 * y.norm(), i


def test_two_streams_at_once():
    p = per()
    a, b = block_inputs("bf16", 1), block_inputs("bf16", 2)
    wa, wb = block(p, a), block(p, b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            ga = block(p, a)
        with torch.cuda.stream(t):
            gb = block(p, b)
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(ga, wa)) and all(same(x, y) for x, y in zip(gb, wb))


def test_stream_argument():
    p = per()
    host, dev = delta_case(2, 100, 2, 1, 32, 32, "bf16", 4)
    o, s, c = run(p, dev)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, s2, c2 = run(p, dev, stream=st)
    g2 = back(p, dev, c2, stream=st.cuda_stream)
    st.synchronize()
    assert same(o, o2) and same(s, s2)
    assert all(same(x, y) for x, y in zip(back(p, dev, c), g2))


@pytest.mark.parametrize("n", [700, 9000])
def test_graph_replays(n):
    """The new operators captured, replayed on changing inputs, against eager calls."""
    p = per()
    host, dev = delta_case(2, 130, 2, 1, 32, 48, "bf16", 4, wide=False)
    t = tokens_of(n, 300, torch.int64, 5).cuda()
    rows = torch.randn(n, 40, device=DEV)
    w = torch.randn(40, device=DEV)

    def once():
        o, s, c = run(p, dev)
        g = back(p, dev, c)
        e = p.per_embed_forward(t, w[None].expand(300, 40).contiguous())
        dt = p.per_embed_backward(t, rows, 300)
        y, st = p.per_norm_forward(rows, w)
        return [o, s, *g, e, dt, y, *p.per_norm_backward(rows, st, rows, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    for k in range(4):
        dev["v"].copy_(torch.randn(dev["v"].shape, generator=gen(k)))
        rows.copy_(torch.randn(n, 40, generator=gen(k)))
        t.copy_(tokens_of(n, 300, torch.int64, 5 + k))
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = once()
        assert all(same(x, y) for x, y in zip(out, want)), k


def test_autograd_function():
    """Inside an autograd.Function the explicit calls give the gradients of the rule."""
    p = per()

    class Delta(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, b):
            o, s, c = p.per_delta_forward(q, k, v, g, b)
            ctx.save_for_backward(q, k, v, g, b, c)
            return o

        @staticmethod
        def backward(ctx, do):
            return p.per_delta_backward(*ctx.saved_tensors, do.contiguous())[:5]
    host, dev = delta_case(1, 70, 2, 1, 16, 16, "f32", 2, wide=False)
    ins = [dev[x].clone().requires_grad_() for x in "qkvgb"]
    o = Delta.apply(*ins)
    (o * dev["do"]).sum().backward()
    a = dict(host, reset=None, s0=None, ds_last=None, length=None, scale=1.0)
    want = O.delta_all(**a)
    tol = O.delta_tolerance(O.delta_size(**a), want, torch.float32)
    for x, name in zip(ins, GRADS):
        assert_close(x.grad, want[name], tol[name], name)
