"""The FP4 cast and product where they are easiest to get wrong: tensor scales
that underflow, rows without a single value."""
import numpy as np
import pytest
import torch

import mx_scale_reusing_gb300 as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mx_scale_reusing_gb300 import _build
    _build.build()
    mx.lib()


# w 2^-133 j (bf16 subnormals) times a gain of 2^-e: the largest product over 2688 = 21 2^7 lies below, at and above half
# of 2^-149, the smallest fp32
@pytest.mark.parametrize("N,K", [(8, 64), (4096, 512)])   # one launch, and the wide form
@pytest.mark.parametrize("j,e,want", [(1, 10, 1.0), (21, 10, 1.0), (22, 10, 2.0 ** -149), (21, 9, 2.0 ** -149),
                                      (42, 9, 2.0 ** -148), (21, 6, 2.0 ** -146)])
def test_derived_scale_of_a_tiny_weight_is_positive(N, K, j, e, want):
    bits = torch.zeros((N, K), dtype=torch.int16, device="cuda")
    bits[N // 2, K // 3] = j
    w = bits.view(torch.bfloat16)
    gamma = torch.full((K,), 2.0 ** -e, device="cuda")
    g = mx.nvfp4_tensor_scale_gain(w, gamma)
    assert np.float32(g.item()) == np.float32(want) and g.item() > 0
    codes, scales, ts = mx.mx_cast_fp4(w, "nvfp4", gamma)
    torch.cuda.synchronize()
    assert ts.item() == g.item() and mx.device_errors() == 0
    if want == 1.0:   # the values themselves round to 0 in bf16
        assert (mx.mx_dequant(codes, scales, "nvfp4", "mma", ts) == 0).all()


def test_no_value_but_zero_has_scale_one():
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    assert mx.nvfp4_tensor_scale_gain(w, torch.full((64,), 0.5, device="cuda")).item() == 1.0
    assert mx.nvfp4_tensor_scale(w).item() == 1.0


@pytest.mark.parametrize("rows", [63, 65, 128])
def test_inv_rms_of_other_rows_is_refused(rows):
    """One factor a row: an inv_rms of a padded batch or of another one does not pass by its length."""
    x = torch.randn((64, 256), device="cuda").to(torch.bfloat16)
    w = torch.randn((136, 256), device="cuda").to(torch.bfloat16)
    xc, xs, inv = mx.quant_fwd_mma(x, fmt="mxfp4")
    wc, ws, _ = mx.mx_cast_fp4(w)
    c, s, r = mx.quant_fwd(x)
    other = torch.ones(rows, device="cuda")
    dout = torch.randn((64, 136), device="cuda").to(torch.bfloat16)
    for fn in (lambda f: mx.linear_fwd_fp4(xc, xs, f, wc, ws), lambda f: mx.linear_wgrad_ckpt(c, s, f, dout, "row_major"),
               lambda f: mx.bwd_ste_ckpt(c, s, x, f)):
        with pytest.raises(ValueError, match="inv_rms"):
            fn(other)
        fn(r)
    with pytest.raises(ValueError, match="inv_rms"):
        mx.bwd_ste_ckpt(c, s, x, None)
