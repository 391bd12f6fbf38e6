"""The sequence operators on the GPU against their 64-bit forms: rows in 8 bits
exactly, the recurrence and the distillation within the error bounds that the
oracle carries along with each value."""
import math

import pytest
import torch

from train_oracle import (TYPES, U, assert_close, dequantise, distill, quantise, rounding, scan)

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def per():
    import sum_tree_sampling_amd as p
    return p


def say(*a):
    print(*a, flush=True)


def bits(t):
    return t.cpu().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------ 8-bit row store

def make_rows(n, d, dtype, seed):
    g = gen(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(2 * torch.randn(d, generator=g))
    return x.to(dtype)


@pytest.mark.parametrize("dim", [1, 7, 8, 33, 64, 333, 512, 1001, 2048, 2049, 5000, 9001, 33000])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_rows_round_trip(dim, group, fmt):
    p = per()
    n, cap = 37, 64
    dtype = TYPES[["f32", "bf16", "f16"][(dim + group) % 3]]
    say("rows", dim, group, fmt, dtype)
    src = make_rows(n, dim, dtype, dim + group)
    if dtype == torch.float16:
        src = src.clamp(-60000, 60000)
    codes, scales = p.rows_alloc(cap, dim, FORMATS[fmt], group)
    raw_before = codes.untyped_storage()
    first = 50  # wraps
    p.per_rows_write(codes, scales, src.cuda(), first, group=group)
    want_c, want_s = quantise(src, FORMATS[fmt], group)
    at = (torch.arange(n) + first) % cap
    assert torch.equal(bits(codes)[at], bits(want_c)), "codes"
    assert torch.equal(bits(scales.contiguous())[at], bits(want_s)), "scales"
    rest = torch.ones(cap, dtype=torch.bool)
    rest[at] = False
    assert not bits(codes)[rest].any() and not scales.cpu()[rest].any()
    # the bytes between codes and scales, and behind them, are not touched
    ng = scales.shape[1]
    whole = torch.tensor([], dtype=torch.uint8, device=DEV).set_(raw_before).view(cap, -1).cpu().clone()
    whole[:, :dim] = 0
    s0 = -(-dim // 4) * 4
    whole[:, s0:s0 + 4 * ng] = 0
    assert not whole.any()
    for out_type in (torch.float32, torch.bfloat16, torch.float16):
        for window in (1, 3):
            idx = torch.tensor([50, 63, 0, 13, -1, 64, 1 << 40, 22, 50])
            got = p.per_rows_read(codes, scales, idx.cuda(), window=window, group=group, dtype=out_type)
            slot = idx[:, None] + torch.arange(window)
            ok = (idx >= 0) & (idx < cap)
            slot = torch.where(ok[:, None], slot % cap, torch.zeros_like(slot))
            full_c, full_s = codes.cpu(), scales.cpu()
            flat = slot.reshape(-1)
            fc = full_c.view(torch.uint8)[flat].view(FORMATS[fmt])
            want = dequantise(fc, full_s[flat], group, out_type).view(len(idx), window, dim)
            want = torch.where(ok[:, None, None], want, torch.zeros_like(want))
            assert torch.equal(got.cpu().float(), want.float())


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dim,group", [(100, 32), (100, 0), (3000, 0), (700, 128)])
def test_rows_odd_values(fmt, dim, group):
    """Zeros, subnormals, infinities, NaN and the type's largest values."""
    p = per()
    src = make_rows(16, dim, torch.float32, 3)
    src[0] = 0
    src[1] = 1e-42
    src[2, 5] = math.inf
    src[3, 6] = -math.inf
    src[4, 7] = math.nan
    src[5] = math.nan
    src[6] = torch.finfo(torch.float32).max
    src[7, :3] = torch.finfo(torch.float32).min
    src[8] = -0.0
    src[9] = math.inf
    src[10] = 2.0 ** -101
    codes, scales = p.rows_alloc(16, dim, FORMATS[fmt], group)
    p.per_rows_write(codes, scales, src.cuda(), 0, group=group)
    wc, ws = quantise(src, FORMATS[fmt], group)
    got = codes.cpu()
    assert torch.equal(bits(scales.contiguous()), bits(ws))
    nan = torch.isnan(wc.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(torch.where(nan, 0.0, got.float()), torch.where(nan, 0.0, wc.float()))


@pytest.mark.parametrize("dim,group,count", [(40, 32, 1), (1001, 64, 700), (5000, 0, 300), (5000, 128, 300), (33000, 0, 200), (8, 0, 3000), (300, 0, 257)])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_rows_write_at_last_position_wins(dim, group, count, fmt):
    p = per()
    cap = 128
    g = gen(count)
    src = make_rows(count, dim, torch.bfloat16, count)
    slots = torch.randint(-3, cap + 3, (count,), generator=g)
    codes, scales = p.rows_alloc(cap, dim, FORMATS[fmt], group)
    claims = torch.zeros(cap, dtype=torch.int32, device=DEV)
    order = {}
    for k, s in enumerate(slots.tolist()):
        if 0 <= s < cap:
            order[s] = k
    wc, ws = quantise(src, FORMATS[fmt], group)
    for _ in range(3):
        codes.view(torch.uint8).zero_()
        scales.zero_()
        p.per_rows_write_at(codes, scales, src.cuda(), slots.cuda(), claims, group=group)
        ec, es = torch.zeros(cap, dim, dtype=torch.uint8), torch.zeros(cap, scales.shape[1])
        for s, k in order.items():
            ec[s], es[s] = bits(wc)[k], ws[k]
        assert torch.equal(bits(codes), ec) and torch.equal(scales.cpu(), es)
        assert not claims.any()


def test_rows_strides_and_far_offsets():
    """Source, output and store with padded rows, beyond 2^32 bytes of store."""
    p = per()
    cap, dim = 1 << 23, 500
    codes = torch.zeros(cap, 520, dtype=torch.uint8, device=DEV)[:, 3:3 + dim].view(torch.int8)
    scales = torch.zeros(cap, 5, device=DEV)[:, :4]
    src = make_rows(64, dim + 9, torch.float32, 1).cuda()[:, 1:1 + dim]
    first = cap - 40
    p.per_rows_write(codes, scales, src, first, group=128)
    wc, ws = quantise(src.cpu(), torch.int8, 128)
    at = (torch.arange(64) + first) % cap
    assert torch.equal(codes[at.cuda()].cpu(), wc) and torch.equal(scales[at.cuda()].cpu(), ws)
    got = p.per_rows_read(codes, scales, torch.tensor([first], device=DEV), window=64, group=128)
    assert torch.equal(got[0].cpu(), dequantise(wc, ws, 128, torch.float32))


# ----------------------------------------------------- gated linear recurrence

def seq_inputs(B, T, D, dtype, seed, resets, ragged):
    g = gen(seed)
    x = torch.randn(B, T, D, generator=g).to(dtype)
    gt = (torch.randn(B, T, D, generator=g) * 3 + 1).to(dtype)
    dy = torch.randn(B, T, D, generator=g).to(dtype)
    h0, dl = torch.randn(B, D, generator=g), torch.randn(B, D, generator=g)
    rs = torch.rand(B, T, generator=g) < resets if resets else None
    ln = torch.randint(-1, T + 2, (B,), generator=g) if ragged else None
    return x, gt, dy, h0, dl, rs, ln


def cu(t):
    return None if t is None else t.cuda()


def check_scan(x, g, dy, h0, dl, rs, ln, views=False):
    p = per()
    dtype = x.dtype
    want = scan(x, g, rs, ln, h0, dy, dl, dtype)
    B, T, D = x.shape
    if views:  # x and g as halves of one projection with sequences inside, gradients the same way
        both = torch.empty(T, B, 2 * D, dtype=dtype, device=DEV).transpose(0, 1)
        gx, gg = both[..., :D], both[..., D:]
        gx.copy_(x)
        gg.copy_(g)
        db = torch.full((B, T, 2 * D + 3), 7.0, dtype=dtype, device=DEV)
        outs = dict(dx=db[..., 1:1 + D], dg=db[..., D + 2:2 * D + 2])
    else:
        gx, gg, outs = x.cuda(), g.cuda(), {}
    y, h, carries = p.per_scan_forward(gx, gg, reset=cu(rs), length=cu(ln), h0=cu(h0))
    dx, dg, dh0 = p.per_scan_backward(gx, gg, carries, dy.cuda(), reset=cu(rs), length=cu(ln), dh_last=cu(dl), **outs)
    torch.cuda.synchronize()
    for name, got in (("y", y), ("h", h), ("dx", dx), ("dg", dg), ("dh0", dh0)):
        assert_close(got, *want[name], name)
    if views:
        assert (db[..., 0] == 7).all() and (db[..., D + 1] == 7).all() and (db[..., 2 * D + 2] == 7).all()
    return y, h, dx, dg, dh0


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 81, 127, 128, 129, 300, 1500])
@pytest.mark.parametrize("D", [1, 8, 15, 32, 63, 64, 65, 130, 333])
def test_scan_sizes(T, D):
    dtype = TYPES[["f32", "bf16", "f16"][(T + D) % 3]]
    say("scan", T, D, dtype)
    a = seq_inputs(3, T, D, dtype, T * 1000 + D, 0.05 if T % 2 else 0, D % 2 == 0)
    check_scan(*a, views=T % 3 == 0)


@pytest.mark.parametrize("T", [40, 200, 600])
@pytest.mark.parametrize("D", [127, 129, 131, 255, 257, 333])
def test_scan_odd_rows_in_pairs(T, D):
    """Rows of odd length in a batch that fills the chip: the last lane's pair starts
    a channel early.  h_last may be h0 there too."""
    dtype = TYPES[["f32", "bf16", "f16"][(T // 40 + D) % 3]]
    say("scan odd", T, D, dtype)
    a = seq_inputs(200, T, D, dtype, T + D, 0.03, True)
    y, h, *_ = check_scan(*a, views=D % 4 == 1)
    x, g, _, h0, _, rs, ln = a
    st = h0.cuda()
    y2, _, _ = per().per_scan_forward(x.cuda(), g.cuda(), reset=rs.cuda(), length=ln.cuda(), h0=st, h_last=st)
    assert torch.equal(st, h) and torch.equal(y2, y)


@pytest.mark.parametrize("shape", [(1, 186, 164), (2, 511, 26), (2, 512, 66), (2, 513, 66), (9, 400, 250)])
def test_scan_few_sequences(shape):
    """Few sequences of up to 512 steps, by workgroups of 16 waves, and of one more."""
    for dtype in TYPES.values():
        check_scan(*seq_inputs(*shape, dtype, shape[1], 0.01, False))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scan_long_time_split(dtype):
    """Few channels and a long axis: segments, with resets in some of them."""
    x, g, dy, h0, dl, rs, ln = seq_inputs(2, 9000, 66, TYPES[dtype], 5, 0.0004, False)
    check_scan(x, g, dy, h0, dl, rs, torch.tensor([9000, 4321]))
    check_scan(x[:1], g[:1] + 6, dy[:1], h0[:1], dl[:1], None, None)


@pytest.mark.parametrize("D", [5, 32, 100])
def test_scan_flags_of_bytes(D):
    """Resets as bytes of any value but 0, on odd rows of them, in sequences that
    share a wave and in others."""
    p = per()
    B, T = 23, 211
    x, g, dy, h0, dl, _, ln = seq_inputs(B, T, D, torch.float32, D, 0, True)
    rs = torch.randint(0, 40, (B, T), generator=gen(D))
    rs = torch.where(rs == 0, torch.randint(1, 256, (B, T), generator=gen(D + 1)), 0).to(torch.uint8)
    want = scan(x, g, rs != 0, ln, h0, dy, dl)
    y, h, c = p.per_scan_forward(x.cuda(), g.cuda(), reset=rs.cuda(), length=cu(ln), h0=cu(h0))
    dx, dg, dh0 = p.per_scan_backward(x.cuda(), g.cuda(), c, dy.cuda(), reset=rs.cuda(), length=cu(ln), dh_last=cu(dl))
    for n, t in (("y", y), ("h", h), ("dx", dx), ("dg", dg), ("dh0", dh0)):
        assert_close(t, *want[n], n)


def test_recorded_inputs_are_refused():
    """A call that would cut an autograd graph says so; inside a Function, and
    under no_grad, it runs."""
    p = per()
    x, g = torch.randn(2, 8, 16, device=DEV, requires_grad=True), torch.randn(2, 8, 16, device=DEV)
    h = torch.zeros(2, 16, device=DEV, requires_grad=True)
    z = torch.randn(2, 16, device=DEV, requires_grad=True)
    ti, t = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.zeros(2, 1, device=DEV)
    for f in (lambda: p.per_scan_forward(x, g), lambda: p.per_scan_forward(g, x), lambda: p.per_scan_forward(g, g, h0=h),
              lambda: p.per_scan_step(g[:, 0], g[:, 0], h), lambda: p.per_distill(z, ti, t),
              lambda: p.per_distill_forward(z, ti, t)):
        with pytest.raises(ValueError, match="requires grad"):
            f()
        with torch.no_grad():
            f()

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b):
            y, _, c = p.per_scan_forward(a, b)
            ctx.save_for_backward(a, b, c)
            return y

        @staticmethod
        def backward(ctx, dy):
            a, b, c = ctx.saved_tensors
            return p.per_scan_backward(a, b, c, dy.contiguous())[:2]

    Scan.apply(x, g).square().sum().backward()
    want = scan(x, g)["y"][0]
    full = scan(x, g, dy=2 * want)
    # dy = 2 y is itself off by y's error, at most 1e-5 of values below 4
    assert_close(x.grad, full["dx"][0], full["dx"][1] + 1e-4, "dx")


def test_scan_filled_chip():
    """Enough sequences that the time axis is not split, over several tiles."""
    check_scan(*seq_inputs(256, 200, 8, torch.float32, 9, 0.02, True))


def test_scan_defaults_and_empty():
    p = per()
    x, g, dy, *_ = seq_inputs(2, 20, 10, torch.float32, 1, 0, False)
    want = scan(x, g, dy=dy)
    y, h, c = p.per_scan_forward(x.cuda(), g.cuda())
    dx, dg, dh0 = p.per_scan_backward(x.cuda(), g.cuda(), c, dy.cuda())
    for n, t in (("y", y), ("h", h), ("dx", dx), ("dg", dg), ("dh0", dh0)):
        assert_close(t, *want[n], n)
    e = torch.empty(2, 0, 10, device=DEV)
    h0 = torch.randn(2, 10, device=DEV)
    y, h, c = p.per_scan_forward(e, e, h0=h0)
    assert y.shape == (2, 0, 10) and torch.equal(h, h0) and c.shape == (2, 0, 10)
    dx, dg, dh0 = p.per_scan_backward(e, e, c, e, dh_last=h0)
    assert torch.equal(dh0, h0)
    e = torch.empty(0, 5, 10, device=DEV)
    y, h, c = p.per_scan_forward(e, e)
    assert y.shape == (0, 5, 10)


@pytest.mark.parametrize("T", [100, 3000])
def test_scan_reset_stops_nan_and_inf(T):
    """What lies before an episode's begin, or past a sequence's end, does not
    reach the other side, forwards or backwards, whatever its value."""
    p = per()
    D, cut, end = 70, T // 3, T - 30
    x, g, dy, h0, dl, _, _ = seq_inputs(1, T, D, torch.float32, 2, 0, False)
    rs = torch.zeros(1, T, dtype=torch.bool)
    rs[0, cut] = True
    ln = torch.tensor([end])
    bx, bg, bdy, bh = x.clone(), g.clone(), dy.clone(), h0.clone()
    bh[:, ::3] = math.nan
    bx[:, :cut, 1::3] = math.inf
    bx[:, end:] = math.nan
    bg[:, end:] = math.nan
    bdy[:, end:] = math.nan
    want = scan(x, g, rs, ln, h0, dy, dl)
    y, h, c = p.per_scan_forward(bx.cuda(), bg.cuda(), reset=cu(rs), length=cu(ln), h0=cu(bh))
    dx, dg, dh0 = p.per_scan_backward(bx.cuda(), bg.cuda(), c, bdy.cuda(), reset=cu(rs), length=cu(ln), dh_last=cu(dl))
    s = slice(cut, None)
    for n, t in (("y", y), ("dx", dx), ("dg", dg)):
        assert_close(t[:, s], want[n][0][:, s], want[n][1][:, s], n)
    assert_close(h, *want["h"], "h")
    assert not y[:, end:].any() and not dx[:, end:].any() and not dg[:, end:].any()
    # backwards: NaN gradients after the cut stay there
    bdy = dy.clone()
    bdy[:, cut + 5] = math.nan
    y, h, c = p.per_scan_forward(x.cuda(), g.cuda(), reset=cu(rs), length=cu(ln), h0=cu(h0))
    dx, dg, dh0 = p.per_scan_backward(x.cuda(), g.cuda(), c, bdy.cuda(), reset=cu(rs), length=cu(ln), dh_last=cu(dl))
    for n, t in (("dx", dx), ("dg", dg)):
        assert_close(t[:, :cut], want[n][0][:, :cut], want[n][1][:, :cut], n)
    assert_close(dh0, *want["dh0"], "dh0")


def test_scan_differences():
    """The gradient against differences of the kernel's own forward pass."""
    p = per()
    x, g, dy, h0, dl, rs, _ = seq_inputs(2, 40, 6, torch.float32, 4, 0.1, False)
    gx, gg, gdy, gh, gdl, grs = (cu(t) for t in (x, g, dy, h0, dl, rs))

    def f(a, b, c):
        y, h, _ = p.per_scan_forward(a, b, reset=grs, h0=c)
        return float((y.double() * gdy.double()).sum() + (h.double() * gdl.double()).sum())

    _, _, car = p.per_scan_forward(gx, gg, reset=grs, h0=gh)
    dx, dg, dh0 = p.per_scan_backward(gx, gg, car, gdy, reset=grs, dh_last=gdl)
    r = [torch.randn(t.shape, generator=gen(7)).cuda() for t in (x, g, h0)]
    eps = 2.0 ** -7
    num = (f(gx + eps * r[0], gg + eps * r[1], gh + eps * r[2])
           - f(gx - eps * r[0], gg - eps * r[1], gh - eps * r[2])) / (2 * eps)
    ana = sum(float((a.double() * b.double()).sum()) for a, b in zip((dx, dg, dh0), r))
    # third derivatives: eps^2 / 6 times a sum of about 500 terms of size 10; rounding: 500 values u / eps
    assert abs(num - ana) < eps ** 2 / 6 * 500 * 10 + 500 * 10 * U / eps, (num, ana)


def test_scan_in_place_state_and_repeat():
    """h_last may be h0, also where the axis is split; the same bits every time."""
    p = per()
    for T in (50, 5000):
        x, g, dy, h0, dl, rs, _ = seq_inputs(2, T, 100, torch.bfloat16, T, 0.001, False)
        gx, gg = x.cuda(), g.cuda()
        y0, h_last, c0 = p.per_scan_forward(gx, gg, reset=cu(rs), h0=cu(h0))
        for _ in range(5):
            st = h0.cuda()
            y, h, c = p.per_scan_forward(gx, gg, reset=cu(rs), h0=st, h_last=st)
            assert h is st and torch.equal(h, h_last) and torch.equal(y, y0) and torch.equal(c, c0)


def test_scan_chunks_continue():
    """A sequence in two calls, the state handed over, is the sequence in one."""
    p = per()
    x, g, dy, h0, dl, rs, _ = seq_inputs(2, 300, 40, torch.float32, 8, 0.02, False)
    want = scan(x, g, rs, None, h0)
    gx, gg, grs = x.cuda(), g.cuda(), rs.cuda()
    y1, h1, _ = p.per_scan_forward(gx[:, :111], gg[:, :111], reset=grs[:, :111].contiguous(), h0=cu(h0))
    y2, h2, _ = p.per_scan_forward(gx[:, 111:], gg[:, 111:], reset=grs[:, 111:].contiguous(), h0=h1)
    assert_close(torch.cat([y1, y2], 1), *want["y"], "y")
    assert_close(h2, *want["h"], "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,D", [(1, 1), (5, 7), (300, 64), (7, 1000), (70000, 12), (3, 5001)])
def test_scan_step(dtype, B, D):
    p = per()
    say("step", dtype, B, D)
    x, g, _, h, _, rs, _ = seq_inputs(B, 1, D, TYPES[dtype], B + D, 0.2, False)
    want = scan(x, g, rs, None, h, dtype=TYPES[dtype])
    both = torch.cat([x[:, 0], g[:, 0]], 1).cuda()
    state = h.cuda()
    y, ho = p.per_scan_step(both[:, :D], both[:, D:], state, reset=rs[:, 0].contiguous().cuda(),
                            h_out=torch.empty_like(state))
    assert_close(y, want["y"][0][:, 0], want["y"][1][:, 0], "y")
    assert_close(ho, *want["h"], "h")
    assert torch.equal(state.cpu(), h)
    y2, ho2 = p.per_scan_step(both[:, :D], both[:, D:], state, reset=rs[:, 0].contiguous().cuda())
    assert ho2 is state and torch.equal(state, ho) and torch.equal(y2, y)


def test_scan_far_offsets():
    """More than 2^31 elements: the last sequences and channels."""
    p = per()
    B, T, D = 17, 1 << 14, 8192
    x1 = torch.randn(1, T, 64, generator=gen(1)).to(torch.bfloat16)
    g1 = (torch.randn(1, T, 64, generator=gen(2)) + 2).to(torch.bfloat16)
    x = x1.cuda().repeat(1, 1, D // 64).expand(B, T, D)
    g = g1.cuda().repeat(1, 1, D // 64).expand(B, T, D)
    y, h, c = p.per_scan_forward(x, g)
    want = scan(x1, g1, dtype=torch.bfloat16)
    for b, d in ((0, 0), (B - 1, D - 64), (B // 2, 4096)):
        assert_close(y[b:b + 1, :, d:d + 64], *want["y"], "y")
        assert_close(h[b:b + 1, d:d + 64], *want["h"], "h")


# ----------------------------------------------------------------- distillation

def top_inputs(N, V, K, dtype, seed, tail, distinct=True):
    g = gen(seed)
    z = (3 * torch.randn(N, V, generator=g)).to(dtype)
    if distinct:
        tidx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32)
    else:
        tidx = torch.randint(0, V, (N, K), generator=g).to(torch.int32)
    t = (3 * torch.randn(N, K, generator=g) + 3).to(dtype)
    w = torch.rand(N, generator=g)
    return z, tidx, t, w


def with_rest(t, tau, seed):
    share = 0.3 + 0.69 * torch.rand(t.shape[0], generator=gen(seed), dtype=torch.float64)
    return (torch.logsumexp(t.double() / tau, 1) - share.log()).float()


def check_distill(z, tidx, t, w, tlse, tau, in_place=True):
    p = per()
    want = distill(z, tidx, t, tlse, tau, w, z.dtype)
    gz, gi, gt, gw, gl = z.cuda(), tidx.cuda(), t.cuda(), w.cuda(), cu(tlse)
    loss, grad = p.per_distill(gz, gi, gt, tlse=gl, temperature=tau, weight=gw)
    assert_close(loss, *want["loss"], "loss")
    assert_close(grad, *want["grad"], "grad")
    all_loss = distill(z, tidx, t, tlse, tau, None, z.dtype)["loss"]
    l2, saved = p.per_distill_forward(gz, gi, gt, tlse=gl, temperature=tau)
    g2 = p.per_distill_backward(gz, gi, gt, saved, gw, tlse=gl, temperature=tau)
    assert_close(l2, *all_loss, "forward loss")
    assert_close(g2, *want["grad"], "backward grad")
    if in_place:
        a = gz.clone()
        p.per_distill_backward(a, gi, gt, saved, gw, tlse=gl, temperature=tau, grad=a)
        assert torch.equal(a.view(torch.uint8), g2.view(torch.uint8))
        a = gz.clone()
        p.per_distill(a, gi, gt, tlse=gl, temperature=tau, weight=gw, grad=a)
        assert torch.equal(a.view(torch.uint8), grad.view(torch.uint8))
    return loss, grad


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (9, 3), (250, 8), (600, 130), (1000, 64), (1000, 20), (2053, 65), (5000, 200), (9001, 1)])
def test_distill_sizes(V, K, dtype, tail):
    say("distill", V, K, dtype, tail)
    tau = [1.0, 2.0, 0.7][(V + K) % 3]
    z, tidx, t, w = top_inputs(5, V, K, TYPES[dtype], V + K, tail)
    check_distill(z, tidx, t, w, with_rest(t, tau, V) if tail else None, tau)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("chunks", [300, 512, 700, 769, 1100, 1537, 2048, 2300, 3584, 4000])
def test_distill_many_rows(chunks, dtype, tail):
    """Rows by one wave each, by workgroups of each size, and the two calls apart in
    one part: every row of many is the row of a small batch."""
    p = per()
    V, K, tau = chunks * (4 if dtype == "f32" else 8) - 11, 70, 1.3
    z, tidx, t, w = top_inputs(4, V, K, TYPES[dtype], chunks, tail)
    tl = with_rest(t, tau, V) if tail else None
    want = distill(z, tidx, t, tl, tau, w, z.dtype)
    for N in (257, 1029) if chunks <= 2048 else (257, 517):
        say("distill rows", N, V, dtype, tail)
        at = torch.arange(N) % 4
        gz, gi, gt, gw, gl = z[at].cuda(), tidx[at].cuda(), t[at].cuda(), w[at].cuda(), cu(None if tl is None else tl[at])
        loss, grad = p.per_distill(gz, gi, gt, tlse=gl, temperature=tau, weight=gw)
        l2, saved = p.per_distill_forward(gz, gi, gt, tlse=gl, temperature=tau)
        g2 = p.per_distill_backward(gz, gi, gt, saved, gw, tlse=gl, temperature=tau)
        assert_close(loss[:4], *want["loss"], "loss")
        assert_close(grad[:4], *want["grad"], "grad")
        assert_close(g2[:4], *want["grad"], "backward grad")
        assert_close(l2[:4], *distill(z, tidx, t, tl, tau, None, z.dtype)["loss"], "forward loss")
        # rows are aligned to 16 bytes in different ways, so sums are in four orders
        for q in range(4, 24):
            k = q % 4
            assert_close(loss[q], *(b[k] for b in want["loss"]), "loss")
            assert_close(grad[q], *(b[k] for b in want["grad"]), "grad")
            assert_close(g2[q], *(b[k] for b in want["grad"]), "backward grad")
        span = 16  # 16 rows of any length begin alike again
        for got in (loss, grad, l2, saved, g2):
            head = got[:span]
            for q in range(span, N, span):
                m = min(span, N - q)
                assert torch.equal(got[q:q + m], head[:m])


@pytest.mark.parametrize("chunks", [4000, 8192])
def test_distill_logits_past_the_caches(chunks):
    """Batches of 128 MB and more give the bits of smaller ones."""
    p = per()
    V, K, part = chunks * 8, 64, 520
    N = (1 << 27) // (V * 2) + 9
    g = torch.Generator(device=DEV).manual_seed(chunks)
    z = torch.randn(N, V, generator=g, device=DEV).to(torch.bfloat16) * 3
    tidx = torch.randint(0, V, (N, K), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randn(N, K, generator=g, device=DEV)
    loss, grad = p.per_distill(z, tidx, t)
    for q in range(0, N, part):
        m = min(part, N - q)
        if m < part:
            q, m = N - part, part
        l2, g2 = p.per_distill(z[q:q + m], tidx[q:q + m], t[q:q + m])
        assert torch.equal(loss[q:q + m], l2) and torch.equal(grad[q:q + m], g2)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V", [(130, 20000), (130, 40001), (129, 66000), (3, 131071), (2, 300001)])
def test_distill_large_rows(N, V, dtype, tail):
    """Rows in one workgroup's registers, in parts, and past both."""
    say("distill large", N, V, dtype, tail)
    z, tidx, t, w = top_inputs(4, V, 50, TYPES[dtype], V, tail)
    k = -(-N // 4)
    z, tidx, t = (a.repeat(k, 1)[:N] for a in (z, tidx, t))
    w = w.repeat(k)[:N]
    tlse = with_rest(t[:4], 2.0, V).repeat(k)[:N] if tail else None
    p = per()
    want = distill(z[:4], tidx[:4], t[:4], None if tlse is None else tlse[:4], 2.0, w[:4], z.dtype)
    args = (z.cuda(), tidx.cuda(), t.cuda())
    loss, grad = p.per_distill(*args, tlse=cu(tlse), temperature=2.0, weight=w.cuda())
    n = min(4, N)
    assert_close(loss[:n], want["loss"][0][:n], want["loss"][1][:n], "loss")
    assert_close(grad[:n], want["grad"][0][:n], want["grad"][1][:n], "grad")
    l2, saved = p.per_distill_forward(*args, tlse=cu(tlse), temperature=2.0)
    g2 = p.per_distill_backward(*args, saved, w.cuda(), tlse=cu(tlse), temperature=2.0)
    assert_close(l2[:n], want["loss"][0][:n], want["loss"][1][:n], "forward loss")
    assert_close(g2[:n], want["grad"][0][:n], want["grad"][1][:n], "backward grad")
    if V % 8 == 0 and N > 4:  # the same row at the same alignment gives the same bits
        for r in range(4, N):
            assert torch.equal(grad[r], grad[r % 4]) and torch.equal(loss[r], loss[r % 4])


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [500, 30011])
def test_distill_odd_entries(V, tail):
    """Repeated, absent and masked entries; rows without any; rows of weight 0."""
    N, K = 12, 20
    z, tidx, t, w = top_inputs(N, V, K, torch.float32, 6, tail, distinct=False)
    tidx[0, 5:] = tidx[0, 0]                 # one token many times
    tidx[1, ::2] = -1
    tidx[2, 3] = V
    tidx[2, 4] = 2 ** 31 - 1
    tidx[3] = -1                             # no entry present
    t[4, 1:] = -math.inf                     # one entry left
    w[5] = 0
    t[6] = torch.finfo(torch.float32).min    # all at the type's lowest value
    z[7] = -math.inf                         # nothing left of the student
    z[8, 10:] = torch.finfo(torch.float32).min
    z[8, :10] = 0
    z[9, :] = torch.finfo(torch.float32).min
    tlse = None
    if tail:
        tlse = with_rest(t.clamp(min=-50), 1.0, 3)
        tlse[0] = 12.0
        tlse[6] = 0.0
    for r in (8, 9):                         # the teacher within what the student allows
        tidx[r] = torch.arange(K) % 10
    if tail:
        tlse[8] += 3.0
    keep = [0, 1, 2, 3, 4, 5, 7, 10, 11] + ([] if tail else [6, 8, 9])
    s = torch.tensor(keep)
    loss, grad = check_distill(z[s], tidx[s], t[s], w[s], None if tlse is None else tlse[s], 1.0)
    for r in (3, 5, 7):
        if r != 3 or not tail:
            assert not grad[keep.index(r)].any() and loss[keep.index(r)] == 0


def test_distill_every_logit_masked_by_entries():
    """A student that rules out a teacher's token has an infinite loss and a
    finite gradient; NaN and +Inf logits give NaN."""
    p = per()
    z, tidx, t, w = top_inputs(4, 300, 6, torch.float32, 3, False)
    z[0, tidx[0, 2].long()] = -math.inf
    z[1, 17] = math.nan
    z[2, 18] = math.inf
    loss, grad = p.per_distill(z.cuda(), tidx.cuda(), t.cuda())
    want = distill(z[:1], tidx[:1], t[:1])
    assert loss[0] == math.inf
    assert_close(grad[:1], *want["grad"], "grad")
    assert torch.isnan(loss[1]) and torch.isnan(grad[1]).all()
    assert torch.isnan(loss[2]) and torch.isnan(grad[2]).all()
    assert torch.isfinite(loss[3]) and torch.isfinite(grad[3]).all()


def test_distill_tail_covers_everything():
    """All tokens named: the rest has no student mass and adds nothing."""
    z, tidx, t, w = top_inputs(3, 16, 16, torch.float32, 3, True)
    tlse = torch.logsumexp(t.double(), 1).float()
    check_distill(z, tidx, t, w, tlse, 1.0)


def test_distill_strides_and_types():
    p = per()
    z, tidx, t, w = top_inputs(6, 700, 12, torch.bfloat16, 9, True)
    tlse = with_rest(t, 1.5, 2)
    want = distill(z, tidx, t, tlse, 1.5, w, torch.bfloat16)
    wide = torch.randn(6, 1001).to(torch.bfloat16).cuda()
    zv = wide[:, 5:705]
    zv.copy_(z)
    gw = torch.full((6, 800), 3.0, dtype=torch.bfloat16, device=DEV)
    for tt in (torch.bfloat16, torch.float32):  # the same logits in another type
        loss, grad = p.per_distill(zv, tidx.cuda(), t.to(tt).cuda(), tlse=tlse.cuda(), temperature=1.5,
                                   weight=w.cuda(), grad=gw[:, 50:750])
        assert_close(loss, *want["loss"], "loss")
        assert_close(grad, *want["grad"], "grad")
        assert (gw[:, :50] == 3).all() and (gw[:, 750:] == 3).all()


@pytest.mark.parametrize("tail", [False, True])
def test_distill_differences(tail):
    p = per()
    z, tidx, t, _ = top_inputs(3, 400, 10, torch.float32, 21, tail)
    tau = 2.0
    gl = with_rest(t, tau, 1).cuda() if tail else None
    gz, gi, gt = z.cuda(), tidx.cuda(), t.cuda()
    loss, grad = p.per_distill(gz, gi, gt, tlse=gl, temperature=tau)
    r = torch.randn(z.shape, generator=gen(1)).cuda()
    eps = 2.0 ** -6

    def f(v):
        return p.per_distill_forward(v, gi, gt, tlse=gl, temperature=tau)[0].double()

    num = (f(gz + eps * r) - f(gz - eps * r)) / (2 * eps)
    ana = (grad.double() * r.double()).sum(1)
    # third derivative by one direction: at most tau^2 (E|r/tau|^3) about 4; roundings of the loss and of z
    assert ((num - ana).abs() <= eps ** 2 * 4 + 64 * U * (loss.double().abs() + 16) / eps).all(), (num, ana)


def test_distill_far_offsets():
    """More than 2^31 logits: the last rows, in place."""
    p = per()
    N, V = 16500, 131072
    z1, tidx, t, w = top_inputs(2, V, 9, torch.bfloat16, 2, False)
    z = torch.zeros(N, V, dtype=torch.bfloat16, device=DEV)
    z[-2:] = z1.cuda()
    wt = torch.zeros(N)
    wt[-2:] = w
    gi, gt = tidx.cuda().repeat(N // 2, 1), t.cuda().repeat(N // 2, 1)
    loss, grad = p.per_distill(z, gi, gt, weight=wt.cuda(), grad=z)
    want = distill(z1, tidx, t, None, 1.0, w, torch.bfloat16)
    assert_close(loss[-2:], *want["loss"], "loss")
    assert_close(grad[-2:], *want["grad"], "grad")
    assert not grad[0].any() and not grad[N // 2].any() and not loss[:-2].any()


# ------------------------------------------------------------ streams and graphs

def everything(p, s, stream=None):
    """All operators once, in caller-owned outputs."""
    p.per_rows_write(s["codes"], s["scales"], s["src"], 5, group=64, stream=stream)
    p.per_rows_write_at(s["codes"], s["scales"], s["src2"], s["slots"], s["claims"], group=64, stream=stream)
    p.per_rows_read(s["codes"], s["scales"], s["idx"], window=200, group=64, out=s["rows"], stream=stream)
    x, g = s["rows"][..., :96], s["rows"][..., 96:]
    y, h, c = p.per_scan_forward(x, g, h0=s["h0"], y=s["y"], h_last=s["h"], carries=s["c"], stream=stream)
    p.per_scan_step(x[:, 3], g[:, 3], s["h"], h_out=s["h2"], y=s["y2"], stream=stream)
    z = s["y"].view(-1, 96)
    p.per_distill(z, s["tidx"], s["t"], tlse=s["tlse"], weight=s["w"], loss=s["loss"], grad=s["dy"].view(-1, 96),
                  stream=stream)
    _, saved = p.per_distill_forward(z, s["tidx"], s["t"], tlse=s["tlse"], loss=s["loss2"], saved=s["saved"],
                                     stream=stream)
    p.per_distill_backward(z, s["tidx"], s["t"], saved, s["w"], tlse=s["tlse"], grad=s["dz"], stream=stream)
    p.per_scan_backward(x, g, c, s["dy"], dx=s["dx"], dg=s["dg"], dh0=s["dh0"], stream=stream)
    return [s[k] for k in ("rows", "y", "h", "h2", "y2", "loss", "loss2", "dy", "dz", "dx", "dg", "dh0")]


def state(p):
    s = {}
    s["codes"], s["scales"] = p.rows_alloc(512, 192, group=64)
    s["src"], s["src2"] = make_rows(400, 192, torch.float32, 1).cuda(), make_rows(60, 192, torch.float32, 2).cuda()
    s["slots"] = torch.randint(0, 512, (60,), generator=gen(1)).cuda()
    s["claims"] = torch.zeros(512, dtype=torch.int32, device=DEV)
    s["idx"] = torch.randint(0, 512, (4,), generator=gen(2)).cuda()
    s["rows"] = torch.empty(4, 200, 192, device=DEV)
    for k in ("y", "dy", "dx", "dg"):
        s[k] = torch.empty(4, 200, 96, device=DEV)
    for k in ("h0", "h", "h2", "y2", "dh0"):
        s[k] = torch.zeros(4, 96, device=DEV)
    s["c"] = torch.empty(4, -(-200 // p.train.PER_SCAN_CHUNK), 96, device=DEV)
    s["dz"] = torch.empty(800, 96, device=DEV)
    s["tidx"] = torch.stack([torch.randperm(96, generator=gen(k))[:7] for k in range(800)]).to(torch.int32).cuda()
    t = torch.randn(800, 7, generator=gen(3))
    s["t"], s["tlse"] = t.cuda(), with_rest(t, 1.0, 4).cuda()
    s["w"] = torch.rand(800, generator=gen(5)).cuda()
    s["saved"] = torch.empty(800, 4 + 7, device=DEV)
    s["loss"], s["loss2"] = torch.empty(800, device=DEV), torch.empty(800, device=DEV)
    return s


def test_other_stream():
    p = per()
    s = state(p)
    want = [t.clone() for t in everything(p, s)]
    torch.cuda.synchronize()
    for st in (torch.cuda.Stream(), ):
        for t in (s["rows"], s["y"], s["dx"], s["loss"]):
            t.zero_()
        torch.cuda.synchronize()
        got = everything(p, s, stream=st)
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        got = everything(p, s, stream=st.cuda_stream)
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_graph_replays():
    """One captured pass of everything, replayed with other inputs, each replay
    against the eager pass on the same inputs."""
    p = per()
    s = state(p)
    everything(p, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything(p, s)
    for k in range(4):
        s["src"].copy_(make_rows(400, 192, torch.float32, 10 + k))
        s["idx"].copy_(torch.randint(0, 512, (4,), generator=gen(10 + k)))
        s["slots"].copy_(torch.randint(0, 512, (60,), generator=gen(20 + k)))
        graph.replay()
        torch.cuda.synchronize()
        got = [s[n].clone() for n in ("rows", "y", "h", "h2", "y2", "loss", "loss2", "dy", "dz", "dx", "dg", "dh0")]
        want = everything(p, s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


def test_distill_parts_graph():
    """The calls that need a workspace, captured: rows in parts, a split time axis."""
    p = per()
    z, tidx, t, w = top_inputs(3, 90001, 9, torch.bfloat16, 1, False)
    gz, gi, gt, gw = (a.cuda() for a in (z, tidx, t, w))
    x, g, dy, h0, dl, rs, _ = seq_inputs(1, 4000, 64, torch.bfloat16, 1, 0.001, False)
    gx, gg, gdy = x.cuda(), g.cuda(), dy.cuda()

    def run():
        a = p.per_distill(gz, gi, gt, weight=gw)
        b = p.per_scan_forward(gx, gg)
        c = p.per_scan_backward(gx, gg, b[2], gdy)
        return [*a, *b, *c]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        gx.copy_(torch.randn(x.shape, generator=gen(k)))
        gz.copy_(torch.randn(z.shape, generator=gen(k)) * 3)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_next_call_can_be_timed():
    """per_time_next brackets these calls too."""
    p = per()
    codes, scales = p.rows_alloc(64, 64)
    src = torch.randn(64, 64, device=DEV)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    b.record()
    torch.cuda.synchronize()
    p.per_time_next(a, b)
    p.per_rows_write(codes, scales, src, 0)
    torch.cuda.synchronize()
    assert 0 < a.elapsed_time(b) < 1000


def test_rounding_bound_itself():
    """What the tolerances count: a rounding is off by at most half a step."""
    v = torch.randn(10000, dtype=torch.float64, generator=gen(1))
    for t in TYPES.values():
        assert ((v.to(t).double() - v).abs() <= rounding(v, t)).all()


def test_example_learns():
    """The example runs every operator together, and its student learns."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "replay_distill.py")
    spec = importlib.util.spec_from_file_location("replay_distill", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.main(steps=120, say=None)
    assert torch.isfinite(losses).all()
    assert losses[-10:].mean() < 0.7 * losses[:5].mean(), losses
