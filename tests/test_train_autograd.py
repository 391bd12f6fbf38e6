"""The binding of the sequence operators next to autograd: every argument whose
gradient or tangent a call would drop is refused, and every tensor it writes counts
as changed in place."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import sum_tree_sampling_amd as p


def arguments(device):
    """Each call with all of its tensors by name."""
    def f(*shape):
        return torch.randn(*shape, device=device)

    def i(*shape, dtype=torch.int64):
        return torch.zeros(*shape, dtype=dtype, device=device)

    codes, scales = p.rows_alloc(16, 40, dtype=torch.int8, device=device)
    B, T, D, N, V, K = 2, 8, 16, 3, 30, 4
    rows = dict(codes=codes, scales=scales)
    seq = dict(x=f(B, T, D), g=f(B, T, D), reset=torch.zeros(B, T, dtype=torch.bool, device=device),
               length=torch.full((B,), T, device=device))
    top = dict(logits=f(N, V), tidx=i(N, K, dtype=torch.int32) + torch.arange(K, device=device, dtype=torch.int32),
               tlogit=f(N, K), tlse=f(N) + 3)
    return {
        "per_rows_write": (dict(rows, src=f(5, 40)), {"codes", "scales"}),
        "per_rows_write_at": (dict(rows, src=f(5, 40), slots=i(5), claims=i(16, dtype=torch.int32)),
                              {"codes", "scales", "claims"}),
        "per_rows_read": (dict(rows, idx=i(4), out=f(4, 1, 40)), {"out"}),
        "per_scan_forward": (dict(seq, h0=f(B, D), y=f(B, T, D), h_last=f(B, D), carries=f(B, 1, D)),
                             {"y", "h_last", "carries"}),
        "per_scan_backward": (dict(seq, carries=f(B, 1, D), dy=f(B, T, D), dh_last=f(B, D), dx=f(B, T, D),
                                   dg=f(B, T, D), dh0=f(B, D)), {"dx", "dg", "dh0"}),
        "per_scan_step": (dict(x=f(B, D), g=f(B, D), h=f(B, D), h_out=f(B, D), y=f(B, D)), {"h_out", "y"}),
        "per_distill": (dict(top, weight=f(N), loss=f(N), grad=f(N, V)), {"loss", "grad"}),
        "per_distill_forward": (dict(top, loss=f(N), saved=f(N, 4 + K)), {"loss", "saved"}),
        "per_distill_backward": (dict(top, saved=f(N, 4 + K), gloss=f(N), grad=f(N, V)), {"grad"}),
    }


CALLS = sorted(arguments("cpu"))


def floats(args):
    return [k for k, v in args.items() if v.is_floating_point()]


@pytest.mark.parametrize("name", CALLS)
def test_arguments_that_require_grad_are_refused(name):
    args, _ = arguments("cpu")[name]
    assert floats(args)
    for k in floats(args):
        given = dict(args, **{k: args[k].clone().requires_grad_()})
        if name.startswith("per_rows") and k == "scales":
            given["scales"] = args["scales"].detach().requires_grad_()
        with pytest.raises(ValueError, match=k + " requires grad"):
            getattr(p, name)(**given)
        with torch.no_grad(), pytest.raises(ValueError, match="current device"):
            getattr(p, name)(**given)  # goes on to the next check


@pytest.mark.parametrize("name", CALLS)
def test_arguments_with_tangents_are_refused(name):
    args, _ = arguments("cpu")[name]
    with fwd.dual_level():
        for k in floats(args):
            given = dict(args, **{k: fwd.make_dual(args[k], torch.ones_like(args[k]))})
            with pytest.raises(ValueError, match=k + " carries a forward-mode tangent"):
                getattr(p, name)(**given)
            with fwd._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="current device"):
                getattr(p, name)(**given)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_written_tensors_change_version(name):
    args, written = arguments("cuda")[name]
    before = {k: v._version for k, v in args.items()}
    getattr(p, name)(**args)
    for k, v in args.items():
        assert (v._version > before[k]) == (k in written or (k in ("codes", "scales") and "codes" in written)), k
    with torch.inference_mode():
        getattr(p, name)(**args)
        inference = {k: v.clone() for k, v in args.items()}
        if name.startswith("per_rows"):
            inference.update(codes=args["codes"], scales=args["scales"])
    getattr(p, name)(**inference)  # tensors without a version are written all the same
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_overwritten_saved_tensors_are_noticed():
    """A state that a graph has saved, stepped in place."""
    x, g = torch.randn(2, 16, device="cuda"), torch.randn(2, 16, device="cuda")
    h = torch.randn(2, 16, device="cuda")
    w = torch.randn(2, 16, device="cuda", requires_grad=True)
    loss = (w * h).sum()
    version = h._version
    with torch.no_grad():
        p.per_scan_step(x, g, h)
    assert h._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    z = torch.randn(3, 30, device="cuda")
    loss = (torch.randn(3, 30, device="cuda", requires_grad=True) * z).sum()
    with torch.no_grad():
        p.per_distill(z, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, 1, device="cuda"), grad=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
