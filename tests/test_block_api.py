"""The block operators' ABI (include/per_block.h): every declared function is exported
and bound, and bad arguments are refused on the host before anything is enqueued (no GPU
is needed: the pointers below are never used)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch
import torch.autograd.forward_ad as fwd

import sum_tree_sampling_amd as p

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "per_block.h")
P = 0x100000  # an aligned address
EINVAL, ENOSPC = -1, -2

_i64, _i32, _f64, _vp, _sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_void_p,
                              ctypes.c_size_t)


class Seq(ctypes.Structure):
    _fields_ = [("p", _vp), ("sb", _i64), ("st", _i64), ("sh", _i64)]


_DELTA = [_i64] * 6 + [_i32] + [Seq] * 5 + [_vp, _vp]
SIG = {
    "per_embed_forward": [_i64] * 3 + [_vp, _i32, _vp, _i32, _i64, _f64, _vp, _i32, _i64, _vp],
    "per_embed_workspace_bytes": [_i64] * 3 + [ctypes.POINTER(_sz)],
    "per_embed_backward": [_i64] * 3 + [_vp, _i32, _vp, _i32, _i64, _f64, _i32, _vp, _i32, _i64, _vp, _sz, _vp],
    "per_norm_forward": [_i64, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _f64, _vp, _i64, _vp, _vp],
    "per_norm_workspace_bytes": [_i64, _i64, _i32, ctypes.POINTER(_sz)],
    "per_norm_backward": [_i64, _i64, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _vp, _vp, _sz, _vp],
    "per_delta_workspace_bytes": [_i64] * 6 + [_i32, _i32, ctypes.POINTER(_sz)],
    "per_delta_forward": _DELTA + [_vp, _f64, Seq, _vp, _vp, _vp, _sz, _vp],
    "per_delta_backward": _DELTA + [_vp, Seq, _vp, _f64] + [Seq] * 5 + [_vp, _vp, _sz, _vp],
    "per_delta_step": [_i64] * 5 + [_i32] + [Seq] * 5 + [_vp, _vp, _f64, _vp, Seq, _vp],
}


@pytest.fixture(scope="module")
def call():
    from sum_tree_sampling_amd import build, per
    if not os.path.exists(per.LIB_PATH) or not os.path.exists(build.MARSHAL_LIB):
        build.build()
    lib = ctypes.CDLL(per.LIB_PATH)
    per.load()
    for name, args in SIG.items():
        getattr(lib, name).argtypes = args

    def f(name, *args):
        rc = getattr(lib, name)(*args)
        if rc:
            assert per.per_last_error()
        return rc
    return f


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(per_[a-z_]+)\s*\(", text)))


def test_declared_exported_bound(call):
    from sum_tree_sampling_amd import per, train
    out = subprocess.run(["nm", "-D", "--defined-only", per.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (per_\w+)$", out, flags=re.M))
    names = declared()
    assert names == sorted(SIG) and set(names) == set(train.BLOCK_NAMES)
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for n in names:
        assert n in exported and callable(getattr(p, n)), n
        args = re.search(r"\b%s\s*\((.*?)\)" % n, text, flags=re.S).group(1)
        assert len(args.split(",")) == len(SIG[n]), n


EF = dict(N=8, V=100, D=16, tokens=P, token_bytes=8, table=P, table_type=0, table_stride=16, scale=1.0, out=P, out_type=1,
          out_stride=16, stream=None)
EB = dict(N=8, V=100, D=16, tokens=P, token_bytes=4, dout=P, dout_type=1, dout_stride=16, scale=1.0, accumulate=0, grad=P,
          grad_type=0, grad_stride=16, ws=P, ws_bytes=1 << 30, stream=None)
TOKENS = [dict(N=-1), dict(N=(1 << 28) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(D=0), dict(D=(1 << 20) + 1),
          dict(tokens=None), dict(tokens=P + 2), dict(token_bytes=2), dict(token_bytes=0), dict(scale=float("nan")),
          dict(scale=float("inf")), dict(scale=1e300)]


@pytest.mark.parametrize("kw", TOKENS + [
    dict(table=None), dict(table=P + 2), dict(table_type=3), dict(table_stride=15), dict(table_stride=-16), dict(out=None),
    dict(out=P + 1), dict(out_type=-1), dict(out_stride=15), dict(out_stride=1 << 41), dict(tokens=P + 4),
    dict(N=1 << 28, D=1 << 20, table_stride=1 << 20, out_stride=1 << 20)])
def test_embed_forward_refuses(call, kw):
    assert call("per_embed_forward", *{**EF, **kw}.values()) == EINVAL


@pytest.mark.parametrize("kw", TOKENS + [
    dict(dout=None), dict(dout=P + 1), dict(dout_type=3), dict(dout_stride=15), dict(grad=None), dict(grad=P + 2),
    dict(grad_type=9), dict(grad_stride=-1), dict(ws=None), dict(ws=P + 8)])
def test_embed_backward_refuses(call, kw):
    assert call("per_embed_backward", *{**EB, **kw}.values()) == EINVAL


def test_embed_workspace(call):
    need = p.per_embed_workspace_bytes
    assert need(0, 100, 16) == 0 and need(8, 100, 16) > 0
    a = {**EB, "N": 20000, "ws_bytes": need(20000, 100, 16) - 1}
    assert call("per_embed_backward", *a.values()) == ENOSPC
    for bad in ((-1, 5, 5), (1, 0, 5), (1, 5, 0), (1, 5, 1 << 21)):
        with pytest.raises(RuntimeError):
            need(*bad)


NF = dict(N=8, D=16, type=1, x=P, xs=16, w=P, b=P, at=0, eps=1e-5, y=2 * P, ys=16, stats=P, stream=None)
NB = dict(N=8, D=16, type=1, x=P, xs=16, stats=P, dy=P, dys=16, w=P, at=1, dx=2 * P, dxs=16, dw=P, db=P, ws=P, ws_bytes=1 << 30,
          stream=None)
ROWS = [dict(N=-1), dict(N=1 << 31), dict(D=0), dict(D=(1 << 20) + 1), dict(type=3), dict(type=-1), dict(x=None),
        dict(x=P + 1), dict(xs=15), dict(xs=1 << 41), dict(w=P + 1), dict(at=2), dict(at=7)]


@pytest.mark.parametrize("kw", ROWS + [
    dict(b=P + 2), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e300), dict(y=None),
    dict(y=P + 1), dict(ys=15), dict(y=P, ys=24), dict(stats=P + 2),
    dict(N=1 << 28, D=4096, xs=4096, ys=4096)])
def test_norm_forward_refuses(call, kw):
    assert call("per_norm_forward", *{**NF, **kw}.values()) == EINVAL


@pytest.mark.parametrize("kw", ROWS + [
    dict(stats=None), dict(stats=P + 2), dict(dy=None), dict(dy=P + 1), dict(dys=15), dict(dx=None), dict(dx=P + 1),
    dict(dxs=15), dict(dx=P, dxs=24), dict(dw=P + 2), dict(db=P + 1), dict(ws=None), dict(ws=P + 4)])
def test_norm_backward_refuses(call, kw):
    assert call("per_norm_backward", *{**NB, **kw}.values()) == EINVAL


def test_norm_workspace(call):
    need = p.per_norm_workspace_bytes
    assert need(0, 64, 0) == 0 and need(1000, 64, 0) > 0
    assert call("per_norm_backward", *{**NB, "ws_bytes": need(8, 16, 1) - 1}.values()) == ENOSPC
    for bad in ((-1, 5, 0), (1, 0, 0), (1, 5, 3)):
        with pytest.raises(RuntimeError):
            need(*bad)


def seqs(B, T, H, D):
    return Seq(P, T * H * D, H * D, D)


SIZE = dict(B=2, T=100, H=4, HK=2, DK=16, DV=32, type=1)
IN = dict(q=seqs(2, 100, 2, 16), k=seqs(2, 100, 2, 16), v=seqs(2, 100, 4, 32), g=seqs(2, 100, 4, 1), b=seqs(2, 100, 4, 1))
DF = {**SIZE, **IN, "reset": None, "length": None, "s0": None, "scale": 1.0, "o": seqs(2, 100, 4, 32), "s_last": None,
      "carries": None, "ws": P, "ws_bytes": 1 << 40, "stream": None}
DB = {**SIZE, **IN, "reset": None, "length": None, "carries": P, "do": seqs(2, 100, 4, 32), "ds": None, "scale": 1.0,
      "dq": seqs(2, 100, 2, 16), "dk": seqs(2, 100, 2, 16), "dv": seqs(2, 100, 4, 32), "dg": seqs(2, 100, 4, 1),
      "db": seqs(2, 100, 4, 1), "ds0": None, "ws": P, "ws_bytes": 1 << 40, "stream": None}
SHAPES = [dict(B=-1), dict(T=-1), dict(B=1 << 31), dict(T=1 << 31), dict(H=0), dict(H=1 << 16, HK=1), dict(HK=0), dict(HK=3),
          dict(HK=8), dict(DK=0), dict(DK=129), dict(DV=0), dict(DV=257), dict(type=3), dict(type=-1),
          dict(B=1 << 20, T=1 << 20), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e300)]
VIEWS = [dict(q=Seq(None, 0, 0, 0)), dict(k=Seq(P + 1, 16, 16, 16)), dict(v=Seq(P, -1, 16, 16)), dict(g=Seq(P, 1, -1, 1)),
         dict(b=Seq(P, 1, 1, 1 << 41)), dict(length=P + 4)]


def out_views(name, D, H):
    """An output whose rows overlap, is missing, or steps back."""
    return [{name: s} for s in (Seq(None, 0, 0, 0), Seq(P + 1, 100 * H * D, H * D, D), Seq(P, 100 * H * D, H * D, -D),
                                Seq(P, 100 * H * D - 1, H * D, D), Seq(P, 100 * H * D, H * D - 1, D), Seq(P, 0, H * D, D),
                                Seq(P, 100 * H * D, H * D, 0), Seq(P, 1 << 41, H * D, D))]


@pytest.mark.parametrize("kw", SHAPES + VIEWS + out_views("o", 32, 4) + [
    dict(s0=P + 2), dict(s_last=P + 1), dict(carries=P + 2), dict(ws=None), dict(ws=P + 8)])
def test_delta_forward_refuses(call, kw):
    assert call("per_delta_forward", *{**DF, **kw}.values()) == EINVAL


@pytest.mark.parametrize("kw", SHAPES + VIEWS + out_views("dq", 16, 2) + out_views("dv", 32, 4) + [
    dict(do=Seq(None, 0, 0, 0)), dict(dk=Seq(P, 0, 0, 0)), dict(dg=Seq(P, 0, 4, 1)), dict(db=Seq(P, 400, 4, 0)),
    dict(carries=None), dict(carries=P + 2), dict(ds=P + 2), dict(ds0=P + 1), dict(ws=None), dict(ws=P + 8)])
def test_delta_backward_refuses(call, kw):
    assert call("per_delta_backward", *{**DB, **kw}.values()) == EINVAL


def test_delta_workspace(call):
    need = p.per_delta_workspace_bytes
    size = tuple(SIZE.values())
    assert need(0, *size[1:]) == 0 and 0 < need(*size) < need(*size, True)
    assert call("per_delta_forward", *{**DF, "ws_bytes": need(*size) - 1}.values()) == ENOSPC
    assert call("per_delta_backward", *{**DB, "ws_bytes": need(*size, True) - 1}.values()) == ENOSPC
    for bad in ((-1, 1, 1, 1, 1, 1, 0), (1, 1, 2, 3, 1, 1, 0), (1, 1, 1, 1, 129, 1, 0), (1, 1, 1, 1, 1, 1, 5)):
        with pytest.raises(RuntimeError):
            need(*bad)


def test_delta_calls_that_no_launch_holds(call):
    """2^32 work-items are refused before the first launch."""
    kw = dict(B=1 << 20, T=64, H=32, HK=32)
    assert call("per_delta_forward", *{**DF, **kw, "o": Seq(P, 64 * 32 * 32, 32 * 32, 32), "ws_bytes": 1 << 62}.values()) == EINVAL


@pytest.mark.parametrize("kw", [k for k in SHAPES if "T" not in k] + VIEWS[:5] + [
    dict(s=None), dict(s=P + 2), dict(s_out=None), dict(s_out=P + 1), dict(o=Seq(None, 0, 0, 0)), dict(o=Seq(P, 127, 0, 32)),
    dict(o=Seq(P, 128, 0, 31))])
def test_delta_step_refuses(call, kw):
    a = {k: v for k, v in SIZE.items() if k != "T"}
    a = {**a, **IN, "reset": None, "s": P, "scale": 1.0, "s_out": P, "o": Seq(P, 128, 0, 32), "stream": None}
    assert call("per_delta_step", *{**a, **kw}.values()) == EINVAL


def test_empty_calls_enqueue_nothing(call):
    none = Seq(None, 0, 0, 0)
    assert call("per_embed_forward", *{**EF, "N": 0, "tokens": None, "table": None, "out": None}.values()) == 0
    assert call("per_norm_forward", *{**NF, "N": 0, "x": None, "y": None}.values()) == 0
    views = {k: none for k in ("q", "k", "v", "g", "b", "o", "do", "dq", "dk", "dv", "dg", "db")}
    assert call("per_delta_forward", *{**DF, **{k: none for k in views if k in DF}, "B": 0, "ws": None}.values()) == 0
    assert call("per_delta_backward", *{**DB, **{k: none for k in views if k in DB}, "B": 0, "carries": None}.values()) == 0


def arguments(device):
    """Each call with all of its tensors by name, and those it writes."""
    def f(*shape):
        return torch.randn(*shape, device=device)
    B, T, H, HK, DK, DV, N, V, D = 2, 70, 4, 2, 16, 24, 5, 30, 40
    tokens = torch.zeros(N, dtype=torch.int64, device=device)
    seq = dict(q=f(B, T, HK, DK), k=f(B, T, HK, DK), v=f(B, T, H, DV), g=f(B, T, H), b=f(B, T, H))
    masks = dict(reset=torch.zeros(B, T, dtype=torch.bool, device=device), length=torch.full((B,), T, device=device))
    one = {k: v[:, 0].contiguous() for k, v in seq.items()}
    carries = f(B, 2, H, DK + 64, DV)
    return {
        "per_embed_forward": (dict(tokens=tokens, table=f(V, D), out=f(N, D)), {"out"}),
        "per_embed_backward": (dict(tokens=tokens, dout=f(N, D), vocab=V, grad=f(V, D)), {"grad"}),
        "per_norm_forward": (dict(x=f(N, D), weight=f(D), bias=f(D), y=f(N, D), stats=f(N, 2)), {"y", "stats"}),
        "per_norm_backward": (dict(x=f(N, D), stats=f(N, 2), dy=f(N, D), weight=f(D), dx=f(N, D), dweight=f(D), dbias=f(D)),
                              {"dx", "dweight", "dbias"}),
        "per_delta_forward": (dict(seq, **masks, s0=f(B, H, DK, DV), out=f(B, T, H, DV), s_last=f(B, H, DK, DV),
                                   carries=carries), {"out", "s_last", "carries"}),
        "per_delta_backward": (dict(seq, carries=carries, do=f(B, T, H, DV), **masks, ds_last=f(B, H, DK, DV),
                                    **{"d" + k: torch.empty_like(v) for k, v in seq.items()}, ds0=f(B, H, DK, DV)),
                               {"dq", "dk", "dv", "dg", "db", "ds0"}),
        "per_delta_step": (dict(one, s=f(B, H, DK, DV), reset=torch.zeros(B, dtype=torch.bool, device=device),
                                s_out=f(B, H, DK, DV), out=f(B, H, DV)), {"s_out", "out"}),
    }


CALLS = sorted(arguments("cpu"))


def floats(args):
    return [k for k, v in args.items() if torch.is_tensor(v) and v.is_floating_point()]


@pytest.mark.parametrize("name", CALLS)
def test_arguments_that_require_grad_are_refused(name):
    args, _ = arguments("cpu")[name]
    for k in floats(args):
        given = dict(args, **{k: args[k].clone().requires_grad_()})
        with pytest.raises(ValueError, match=k + " requires grad"):
            getattr(p, name)(**given)
        with torch.no_grad(), pytest.raises(ValueError, match="current device"):
            getattr(p, name)(**given)


@pytest.mark.parametrize("name", CALLS)
def test_arguments_with_tangents_are_refused(name):
    args, _ = arguments("cpu")[name]
    with fwd.dual_level():
        for k in floats(args):
            given = dict(args, **{k: fwd.make_dual(args[k], torch.ones_like(args[k]))})
            with pytest.raises(ValueError, match=k + " carries a forward-mode tangent"):
                getattr(p, name)(**given)


@pytest.mark.parametrize("name", CALLS)
def test_missing_and_unknown_arguments_are_refused(name):
    args, _ = arguments("cpu")[name]
    with pytest.raises(ValueError):
        getattr(p, name)()
    with pytest.raises(ValueError):
        getattr(p, name)(**args, nothing=1)
    with pytest.raises(ValueError):
        getattr(p, name)(3, *list(args.values())[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_change_version(name):
    args, written = arguments("cuda")[name]
    before = {k: v._version for k, v in args.items() if torch.is_tensor(v)}
    getattr(p, name)(**args)
    for k, v in before.items():
        assert (args[k]._version > v) == (k in written), k
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_binding_refuses():
    """Shapes, types, strides and devices that do not fit each other."""
    def f(*s, dtype=torch.float32):
        return torch.zeros(*s, dtype=dtype, device="cuda")
    t, table = f(4, dtype=torch.int64), f(9, 6)
    seq = arguments("cuda")["per_delta_forward"][0]
    five = [seq[k] for k in "qkvgb"]
    bad = [
        (p.per_embed_forward, (t.float(), table), {}), (p.per_embed_forward, (t[None], table), {}),
        (p.per_embed_forward, (t.cpu(), table), {}), (p.per_embed_forward, (t, table[0]), {}),
        (p.per_embed_forward, (t, table.t()), {}), (p.per_embed_forward, (t, table.double()), {}),
        (p.per_embed_forward, (f(8, dtype=torch.int64)[::2], table), {}), (p.per_embed_forward, (t, table), dict(out=f(4, 5))),
        (p.per_embed_forward, (t, table), dict(dtype=torch.int32)), (p.per_embed_forward, (t, table), dict(dtype=3)),
        (p.per_embed_forward, (t, table), dict(out=f(4, 6), dtype=torch.float16)), (p.per_embed_forward, (t, table), dict(scale="x")),
        (p.per_embed_backward, (t, f(5, 6), 9), {}), (p.per_embed_backward, (t, f(4, 6), 9), dict(accumulate=True)),
        (p.per_embed_backward, (t, f(4, 6), 9), dict(grad=f(8, 6))), (p.per_embed_backward, (t, f(4, 6), 2.5), {}),
        (p.per_norm_forward, (table[0],), {}), (p.per_norm_forward, (table, f(5)), {}), (p.per_norm_forward, (table, f(6).half()), {}),
        (p.per_norm_forward, (table.half(), f(6), f(6).half()), {}), (p.per_norm_forward, (table,), dict(y=f(9, 6).half())),
        (p.per_norm_forward, (table,), dict(stats=f(9))), (p.per_norm_backward, (table, f(9, 2), f(9, 5)), {}),
        (p.per_norm_backward, (table, f(9, 3), table), {}), (p.per_norm_backward, (table, f(9, 2), table), dict(sums=False, dbias=f(6))),
        (p.per_delta_forward, five[:4] + [seq["b"][:, 1:]], {}), (p.per_delta_forward, five[:1] + [seq["k"].half()] + five[2:], {}),
        (p.per_delta_forward, [seq["q"][..., :8]] + five[1:], {}), (p.per_delta_forward, five, dict(reset=f(2, 70))),
        (p.per_delta_forward, five, dict(length=f(2, dtype=torch.int32))), (p.per_delta_forward, five, dict(s0=f(2, 4, 16, 23))),
        (p.per_delta_forward, five, dict(save=False, carries=seq["carries"])), (p.per_delta_forward, five, dict(carries=f(2, 4))),
        (p.per_delta_forward, [x.transpose(-1, -2) for x in five], {}),
        (p.per_delta_step, [x[:, 0] for x in five] + [f(2, 4, 16, 20)], {}), (p.per_delta_step, five + [f(2, 4, 16, 24)], {}),
    ]
    for i, (fn, args, kw) in enumerate(bad):
        with pytest.raises(ValueError):
            fn(*args, **kw)
            raise AssertionError("call %d (%s) was taken" % (i, fn))
    for fn, args, kw in [(p.per_embed_backward, (t, f(4, 6), 0), {}), (p.per_norm_forward, (table,), dict(eps=-1.0)),
                         (p.per_delta_forward, (f(1, 2, 1, 129), f(1, 2, 1, 129), *(x[:1, :2, :1] for x in five[2:])), {}),
                         (p.per_delta_forward, five, dict(scale=float("nan"))),
                         (p.per_delta_forward, five, dict(out=seq["v"][:1].expand(2, -1, -1, -1)))]:
        with pytest.raises(p.PerError):
            fn(*args, **kw)
