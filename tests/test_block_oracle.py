"""The 64-bit forms the block operators are held to: gradients against differences,
and the chunked sizes above every result."""
import torch

import block_oracle as O


def _inputs(B=2, T=70, H=4, HK=2, DK=5, DV=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    def r(*s): return torch.randn(*s, generator=g, dtype=torch.float64)
    q, k = (torch.nn.functional.normalize(r(B, T, HK, DK), dim=-1) for _ in range(2))
    reset = torch.rand(B, T, generator=g) < 0.05
    return dict(q=q, k=k, v=r(B, T, H, DV), g=r(B, T, H) + 2, b=r(B, T, H), reset=reset,
                length=torch.tensor([T, T - 9]), s0=r(B, H, DK, DV), scale=0.4), r(B, T, H, DV), r(B, H, DK, DV)


def test_delta_gradients_against_differences():
    a, do, ds = _inputs()
    got = O.delta_all(**a, do=do, ds_last=ds)
    n = a["length"]
    go = (torch.arange(do.shape[1]) < n[:, None])[..., None, None]

    def f(**kw):
        o, s = O.delta(**{**a, **kw})
        return float((o * do * go).sum() + (s * ds).sum())
    g = torch.Generator().manual_seed(5)
    for name in ("q", "k", "v", "g", "b", "s0"):
        d = torch.randn(a[name].shape, generator=g, dtype=torch.float64)
        e = 1e-5
        diff = (f(**{name: a[name] + e * d}) - f(**{name: a[name] - e * d})) / (2 * e)
        want = float((got["d" + name] * d).sum())
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name


def test_delta_sizes_are_above_the_values():
    a, do, ds = _inputs(T=150, seed=3)
    a["length"] = torch.tensor([150, 101])
    got = O.delta_all(**a, do=do, ds_last=ds)
    size = O.delta_size(**a, do=do, ds_last=ds)
    for name, want in got.items():
        assert torch.isfinite(size[name]).all()
        assert (want.abs() <= size[name] * (1 + 1e-9) + 1e-12).all(), name


def test_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(4, 9, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(9, generator=g, dtype=torch.float64) for _ in range(2))
    out = O.norm(x, w, b, 1e-3, dy)
    for name, at in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        d = torch.randn(([x, w, b][at]).shape, generator=g, dtype=torch.float64)
        def f(e):
            a = [x, w, b]
            a[at] = a[at] + e * d
            return float((O.norm(*a, 1e-3)["y"][0] * dy).sum())
        diff = (f(1e-5) - f(-1e-5)) / 2e-5
        want = float((out[name][0] * d).sum())
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name
