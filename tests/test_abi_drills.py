"""Refusals of the failure-detection drills of the tensor-core kernels: host
side, before any launch.  No GPU."""
import pytest

import mx_scale_reusing_gb300 as mx

F = 1 << 40  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from mx_scale_reusing_gb300 import _build
    _build.build()
    return mx.lib()


BAD_DRILLS = [dict(load=2), dict(load=-1), dict(stage=-1), dict(ns=999_999), dict(ns=1_000_000_001), dict(T=0)]


@pytest.mark.parametrize("bad", BAD_DRILLS + [dict(T=-1), dict(K=100), dict(N=63), dict(layout=2), dict(out=None)])
def test_wgrad_drill_refusals(L, bad):
    a = dict(c=F, s=F, layout=0, inv=F, do=F, T=8, K=128, N=64, out=F, ws=None, wsb=0, load=0, stage=0, ns=2_000_000) | bad
    assert L.mxnorm_linear_wgrad_wait_drill(*a.values(), None) == 1
    assert L.mxnorm_last_error()


def test_wgrad_drill_needs_the_workspace_of_the_call(L):
    n = L.mxnorm_linear_wgrad_workspace_bytes(100000, 128, 64)
    assert n > 0
    f = L.mxnorm_linear_wgrad_wait_drill
    assert f(F, F, 0, F, F, 100000, 128, 64, F, F, n - 1, 0, 0, 2_000_000, None) == 1
    assert f(F, F, 0, F, F, 100000, 128, 64, F, F + 8, n, 0, 0, 2_000_000, None) == 3


@pytest.mark.parametrize("bad", [dict(stage=-1), dict(ns=999_999), dict(ns=1_000_000_001), dict(T=0), dict(T=-1), dict(K=64),
                                 dict(N=0), dict(fmt=9), dict(out=None), dict(xg=F)])
def test_product_drill_refusals(L, bad):
    a = dict(x=F, xs=F, inv=F, w=F, ws=F, T=8, K=128, N=64, fmt=1, xg=None, wg=None, out=F, stage=0, ns=2_000_000) | bad
    assert L.mxnorm_linear_fp4_wait_drill(*a.values(), None) == 1
    assert L.mxnorm_last_error()
