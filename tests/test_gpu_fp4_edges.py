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


@pytest.mark.parametrize("T", [5, 70, 333, 700])
@pytest.mark.parametrize("p", [1, 2])
def test_rows_without_a_value_stay_zero_through_a_layer(T, p):
    """Padding rows, and rows whose every block scale is lost beside the tensor's largest value, get inv_rms = +Inf from
    the NVFP4 pass.  Forward and both gradients treat them as zeros and every other row as if they were not there."""
    K, N = 512, 264
    torch.manual_seed(T)
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    dead = torch.zeros(T, dtype=torch.bool, device="cuda")
    dead[[0, T // 2, T - 1]] = True
    x[0] = 0
    x[T - 1] = 0
    x[T // 2] *= 2.0 ** -30
    w = (torch.randn((N, K), device="cuda") * 0.05).to(torch.bfloat16)
    dout, dh = torch.randn((T, N), device="cuda").to(torch.bfloat16), torch.randn((T, K), device="cuda").to(torch.bfloat16)
    xc, xs, inv, xg = mx.quant_fwd_nvfp4_mma(x, p)
    assert torch.equal(torch.isinf(inv), dead)
    wc, ws, wg = mx.mx_cast_fp4(w, "nvfp4")
    kc, ks = mx.mx_cast(x, "mma")
    got = (mx.linear_fwd_fp4(xc, xs, inv, wc, ws, "nvfp4", xg, wg), mx.bwd_ste_ckpt(kc, ks, dh, inv, "mma"),
           mx.linear_wgrad_ckpt(kc, ks, inv, dout))
    zeroed = torch.where(dead, torch.zeros_like(inv), inv)
    want = (mx.linear_fwd_fp4(xc, xs, zeroed, wc, ws, "nvfp4", xg, wg), mx.bwd_ste_ckpt(kc, ks, dh, zeroed, "mma"),
            mx.linear_wgrad_ckpt(kc, ks, zeroed, dout))
    for a, b in zip(got, want):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert (got[0][dead] == 0).all() and (got[1][dead] == 0).all()
    # dW against its formula over the rows that are there: the bound of a sum of T products in fp32, rounded once
    live = ~dead
    h = (mx.mx_dequant(kc, ks, layout="mma").float()[live] * inv[live][:, None]).to(torch.bfloat16).double()
    g = dout[live].double()
    ref, size = g.t() @ h, g.abs().t() @ h.abs()
    assert ((got[2].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * (T + 8) * 2.0 ** -24 * size * 1.01 + 1e-38).all()


@pytest.mark.parametrize("T", [1, 333])
def test_nan_rows_are_not_taken_for_empty_ones(T):
    x = torch.randn((T, 256), device="cuda").to(torch.bfloat16)
    x[T - 1, 7] = float("nan")
    w = torch.randn((64, 256), device="cuda").to(torch.bfloat16)
    xc, xs, inv, xg = mx.quant_fwd_nvfp4_mma(x)
    wc, ws, wg = mx.mx_cast_fp4(w, "nvfp4")
    kc, ks = mx.mx_cast(x, "mma")
    assert mx.linear_fwd_fp4(xc, xs, inv, wc, ws, "nvfp4", xg, wg)[T - 1].isnan().all()
    assert mx.bwd_ste_ckpt(kc, ks, x, inv, "mma")[T - 1].isnan().all()
    assert mx.linear_wgrad_ckpt(kc, ks, inv, w.new_ones((T, 64))).isnan().all()
