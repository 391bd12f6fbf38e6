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
