"""Ranges of the sequence operators (include/per_train.h) that are refused on the
host, before anything is enqueued: the pointers below are never followed."""
import ctypes

import pytest

from test_train_api import EINVAL, P, TOP, call  # noqa: F401  (call is a fixture)


@pytest.mark.parametrize("tau", [64.001, 100.0, 1024.0, 2.0 ** 20])
@pytest.mark.parametrize("name,kw", [
    ("per_distill", dict(weight=None, loss=P, grad=2 * P, gs=100, ws=None, ws_bytes=0)),
    ("per_distill_forward", dict(loss=P, saved=P, ws=None, ws_bytes=0)),
    ("per_distill_backward", dict(saved=P, gloss=P, grad=2 * P, gs=100))])
def test_temperatures_past_the_loss_s_precision(call, name, kw, tau):  # noqa: F811
    assert call(name, *{**TOP, **kw, "tau": tau}.values(), None) == EINVAL


BIG = 1 << 30


@pytest.mark.parametrize("count,dim,group", [(1 << 26, 512, 32), (1 << 26, 505, 0), (1 << 26, 100000, 128),
                                             (1 << 24, 2049, 0), (1 << 22, 8200, 0), ((1 << 31) - 1, 17, 0)])
def test_rows_that_no_launch_holds(call, count, dim, group):  # noqa: F811
    """2^32 work-items and more are refused before the claims are taken: they would
    stay in d_claims, and later calls would skip those slots."""
    rows = [BIG, dim, 0, group, P, 1 << 20, P, 1 << 20]
    assert call("per_rows_write_at", *rows, count, P, P, P, 1, dim, None) == EINVAL
    if count <= BIG:
        assert call("per_rows_write", *rows, count, 0, P, 1, dim, None) == EINVAL


@pytest.mark.parametrize("B,window,dim", [(1 << 26, 1, 512), (1 << 16, 1 << 10, 500), ((1 << 31) - 1, 1, 9)])
def test_reads_that_no_launch_holds(call, B, window, dim):  # noqa: F811
    assert call("per_rows_read", BIG, dim, 1, 0, P, 1 << 20, P, 1 << 20, B, P, window, P, 1, dim, None) == EINVAL


@pytest.mark.parametrize("B,T,D,views", [(1 << 26, 1, 64, 1), (1 << 24, 200, 64, 1), ((1 << 31) - 1, 200, 128, 1)])
def test_sequences_that_no_launch_holds(call, B, T, D, views):  # noqa: F811
    v = [P, T * D, D]
    assert call("per_scan_forward", B, T, D, 1, *v, *v, None, None, None, *v, None, None, P, 1 << 62, None) == EINVAL
    assert call("per_scan_backward", B, T, D, 1, *v, *v, None, None, P, *v, None, *v, *v, None, P, 1 << 62,
                None) == EINVAL


@pytest.mark.parametrize("B,D", [(1 << 24, 1024), (1 << 28, 64), ((1 << 31) - 1, 8)])
def test_steps_that_no_launch_holds(call, B, D):  # noqa: F811
    assert call("per_scan_step", B, D, 1, P, D, P, D, None, P, P, P, D, None) == EINVAL


@pytest.mark.parametrize("N,V", [(1 << 26, 500), (1 << 24, 11000), (1 << 26, 100)])
def test_logits_that_no_launch_holds(call, N, V):  # noqa: F811
    top = {**TOP, "N": N, "V": V, "stride": V, "K": 64}
    ws = dict(ws=P, ws_bytes=1 << 62)
    assert call("per_distill", *top.values(), None, P, 2 * P, V, *ws.values(), None) == EINVAL
    assert call("per_distill_forward", *top.values(), P, P, *ws.values(), None) == EINVAL
    assert call("per_distill_backward", *top.values(), P, P, 2 * P, V, None) == EINVAL
