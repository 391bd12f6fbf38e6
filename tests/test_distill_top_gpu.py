"""Distillation from up to 1024 teacher entries, distinct and repeated."""
import pytest
import torch

from train_oracle import TYPES, assert_close, distill

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def inputs(N, V, K, dtype, seed, repeats):
    g = gen(seed)
    z = (3 * torch.randn(N, V, generator=g)).to(dtype)
    if repeats == "none":
        tidx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    else:  # each token a few times, the copies far apart; one token in a hundred entries
        few = torch.stack([torch.randperm(V, generator=g)[:-(-K // 3)] for _ in range(N)])
        tidx = few.repeat(1, 3)[:, :K].contiguous()
        tidx[0, 5:105] = tidx[0, 0]
    tidx[-1, ::7] = -1
    t = (3 * torch.randn(N, K, generator=g)).to(dtype)
    return z, tidx.to(torch.int32), t, torch.rand(N, generator=g)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("repeats", ["none", "some"])
@pytest.mark.parametrize("K", [257, 512, 1024])
@pytest.mark.parametrize("N,V,dtype", [(5, 1100, "f32"), (1100, 4000, "bf16"), (3, 11000, "f16"), (520, 11000, "bf16"),
                                       (130, 40000, "bf16"), (130, 66000, "f32"), (3, 200001, "bf16")])
def test_many_entries(N, V, dtype, K, repeats, tail):
    """Rows by waves, by workgroups and in parts."""
    import sum_tree_sampling_amd as p
    print("top", N, V, dtype, K, repeats, tail, flush=True)
    some = min(N, 3)
    z, tidx, t, w = inputs(some, V, K, TYPES[dtype], V + K, repeats)
    tau = 1.5
    tlse = None
    if tail:
        live = torch.where(tidx >= 0, t.double() / tau, torch.tensor(-1e9, dtype=torch.float64))
        tlse = (torch.logsumexp(live, 1) + 0.4).float()
    want = distill(z, tidx, t, tlse, tau, w, z.dtype)
    plain = distill(z, tidx, t, tlse, tau, None, z.dtype)["loss"]
    at = torch.arange(N) % some
    gz, gi, gt, gw = (a[at].cuda() for a in (z, tidx, t, w))
    gl = None if tlse is None else tlse[at].cuda()
    loss, grad = p.per_distill(gz, gi, gt, tlse=gl, temperature=tau, weight=gw)
    l2, saved = p.per_distill_forward(gz, gi, gt, tlse=gl, temperature=tau)
    g2 = p.per_distill_backward(gz, gi, gt, saved, gw, tlse=gl, temperature=tau)
    for lo in (0, (N - some) // some * some):
        k = slice(lo, lo + some)
        assert_close(loss[k], *want["loss"], "loss")
        assert_close(grad[k], *want["grad"], "grad")
        assert_close(l2[k], *plain, "forward loss")
        assert_close(g2[k], *want["grad"], "backward grad")


def test_tokens_far_apart_cost_no_second_look():
    """1024 distinct tokens take as long whichever they are: two of them 2^17 apart
    (they met in the table that finds repeated ones) do not send every entry over
    all the others."""
    import sum_tree_sampling_amd as p
    N, V, K = 1024, 139000, 1024
    z = torch.randn(N, V, device="cuda").to(torch.bfloat16)
    t = torch.randn(N, K, device="cuda")
    near = torch.arange(K, dtype=torch.int32, device="cuda").repeat(N, 1)
    far = near.clone()
    far[:, 1] = 2 ** 17
    grad = torch.empty_like(z)
    times = {}
    for _ in range(4):
        for name, tidx in (("near", near), ("far", far)):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            p.per_distill(z, tidx, t, grad=grad)
            a.record()
            for _ in range(3):
                p.per_distill(z, tidx, t, grad=grad)
            b.record()
            torch.cuda.synchronize()
            times.setdefault(name, []).append(a.elapsed_time(b))
    assert min(times["far"]) < 1.3 * min(times["near"]), times
