"""The checkpoint gradients where they are easiest to get wrong: the pair's
hand-over between its CTAs under load, the whole rounding error of dW, rows
without a single value, and the gradients of a rotated layer."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import mx_scale_reusing_gb300 as mx
from mx_scale_reusing_gb300 import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mx_scale_reusing_gb300 import _build
    _build.build()
    mx.lib()


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T,K,N", [(700, 96, 24), (6000, 512, 520), (3000, 1152, 136), (2050, 2304, 2568), (4096, 1024, 1024)])
def test_dw_hand_over_between_the_ctas_of_a_pair(T, K, N):
    """Half of every stage's h is written by the CTA that does not issue the MMAs.  Many calls on two streams at once,
    so that the CTAs of a pair drift apart: every one gives the same bits, and no column block of either CTA is off."""
    x, dout = dev(synth.make_random_rows(T, K, 1, 2.0)), dev(synth.make_random_rows(T, N, 2, 0.1))
    c, s, inv = mx.quant_fwd(x)
    h = (mx.mx_dequant(c, s).float() * inv[:, None]).to(torch.bfloat16).double()
    g = dout.double()
    want, size = g.t() @ h, g.abs().t() @ h.abs()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(mx.linear_wgrad_ckpt(c, s, inv, dout, "row_major"))
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    # products exact in fp32, T + 8 additions off by at most one ulp of a partial sum, one rounding to bf16
    bound = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * 2 * (T + 8) * U * size + 1e-38
    assert ((outs[0].double() - want).abs() <= bound).all()
    assert mx.device_errors() == 0
