"""The recurrence where a state or a gradient is infinite and nothing resets it: it
stays infinite through gates of any size, as f * Inf does."""
import math

import pytest
import torch

from train_oracle import TYPES, assert_close, scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [-12.0, -3.0, 2.0])
@pytest.mark.parametrize("B,T,D", [(2, 40, 70), (2, 200, 70), (3, 300, 8), (200, 300, 130), (2, 3000, 66)])
def test_infinite_states_and_gradients(B, T, D, gate, dtype):
    import sum_tree_sampling_amd as p
    print("inf", B, T, D, gate, dtype, flush=True)
    g = torch.Generator().manual_seed(T)
    x, dy = (torch.randn(B, T, D, generator=g).to(TYPES[dtype]) for _ in range(2))
    gt = (gate + 0.1 * torch.randn(B, T, D, generator=g)).to(TYPES[dtype])
    h0, dl = torch.randn(B, D, generator=g), torch.randn(B, D, generator=g)
    h0[:, 0::4] = math.inf
    h0[:, 1::4] = -math.inf
    x[:, T // 2, 2::4] = math.inf
    want = scan(x, gt, None, None, h0, dtype=x.dtype)
    y, h, _ = p.per_scan_forward(x.cuda(), gt.cuda(), h0=h0.cuda())
    assert torch.isinf(want["y"][0][:, :, 0::4]).all() and torch.isinf(want["h"][0][:, 2::4]).all()
    assert_close(y, *want["y"], "y")
    assert_close(h, *want["h"], "h")
    # gradients: infinite ones flow back to dx and dh0
    x[:, T // 2, 2::4] = 1.0
    h0 = torch.randn(B, D, generator=g)
    dl[:, 0::4] = math.inf
    dy[:, T - 3, 1::4] = -math.inf
    want = scan(x, gt, None, None, h0, dy, dl, x.dtype)
    y, h, c = p.per_scan_forward(x.cuda(), gt.cuda(), h0=h0.cuda())
    dx, _, dh0 = p.per_scan_backward(x.cuda(), gt.cuda(), c, dy.cuda(), dh_last=dl.cuda())
    assert torch.isinf(want["dx"][0][:, :, 0::4]).all() and torch.isinf(want["dh0"][0][:, 1::4]).all()
    assert_close(dx, *want["dx"], "dx")
    assert_close(dh0, *want["dh0"], "dh0")
