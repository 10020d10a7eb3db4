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


def hadamard_matrix(n):
    """Orthonormal, Sylvester order: entry (i, j) has the sign of the parity of i & j."""
    i = torch.arange(n)
    bits = (i[:, None] & i[None, :])
    parity = sum((bits >> k) & 1 for k in range(5)) % 2
    return ((1 - 2 * parity).double() / n ** 0.5).cuda()


@pytest.mark.parametrize("fmt,n", [("mxfp4_h16", 16), ("mxfp4_h32", 32)])
def test_training_step_of_a_rotated_layer(fmt, n):
    """The weight that a rotated product used reads back rotated.  dh of the layer's (unrotated) normalised input is
    dout @ w_used rotated once more: against central differences in 64 bits of sum(dout * (h H) w_used^T), which is
    linear in h.  It then goes into dx beside unrotated codes."""
    T, K, N = 70, 256, 136
    x, w = dev(synth.make_random_rows(T, K, 1, 2.0)), dev(synth.make_random_rows(N, K, 2, 0.05))
    gb = synth.make_random_rows(T, N, 3, 0.1)
    dout = dev(gb)
    xc, xs, inv = mx.quant_fwd_mma(x, fmt=fmt)
    wc, ws, _ = mx.mx_cast_fp4(w, fmt)
    out = mx.linear_fwd_fp4(xc, xs, inv, wc, ws, fmt)
    w_used, Hn = mx.mx_dequant(wc, ws, fmt, "mma"), hadamard_matrix(n)

    def rotated(v):
        return (v.unflatten(1, (-1, n)) @ Hn).flatten(1)

    # the forward multiplied these: rotated rows by rotated rows
    xr = mx.mx_dequant(xc, xs, fmt, "mma").double()
    want = inv.double()[:, None] * (xr @ w_used.double().t())
    size = inv.double()[:, None] * (xr.abs() @ w_used.double().abs().t())
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2 * K * U * size + 3 * U * want.abs()) * 1.01).all()
    # rotating twice is nothing, and the rotated cast of x approximates x rotated
    assert torch.allclose(rotated(rotated(x.double())), x.double(), rtol=0, atol=1e-9)
    assert torch.nn.functional.cosine_similarity(rotated(xr).flatten(), x.double().flatten(), dim=0) > 0.95
    dh = rotated(dout.double() @ w_used.double())
    h0, g = torch.randn((T, K), dtype=torch.float64, device="cuda"), dout.double()
    for j in range(0, K, 37):
        e = torch.zeros_like(h0)
        e[:, j] = 0.5
        up, down = ((g * (rotated(h0 + s * e) @ w_used.double().t())).sum(1) for s in (1, -1))
        assert torch.allclose(up - down, dh[:, j], rtol=1e-9, atol=1e-9)
    kc, ks, r = mx.quant_fwd_mma(x)   # the checkpoint: unrotated codes, with their own inverse RMS
    dhb = dh.to(torch.bfloat16)
    dx = mx.bwd_ste_ckpt(kc, ks, dhb, r, "mma").double()
    xv, d, rr = mx.mx_dequant(kc, ks, layout="mma").double(), dhb.double(), r.double()[:, None]
    exact = rr * d - rr ** 3 * xv * (d * xv).mean(1, keepdim=True)
    size = rr * d.abs() + rr ** 3 * xv.abs() * (d * xv).abs().mean(1, keepdim=True)
    # bf16 output; fp32 steps, each within u of its term: a dozen for the sum's tree, six around it
    assert ((dx - exact).abs() <= 2.0 ** -8 * exact.abs() + 20 * U * size).all()


@pytest.mark.parametrize("T,K,N,layout", [(1, 32, 8, "row_major"), (100, 416, 264, "row_major"), (700, 256, 136, "mma"),
                                          (2043, 768, 768, "mma"), (20000, 64, 72, "row_major")])
def test_dw_whole_rounding_error(T, K, N, layout):
    """dW against dout^T (r x^) in 64 bits, with nothing rounded before the sum.  The operand h = r x^ rounds to bf16 (half
    a step: 2^-8 of each term, after two fp32 roundings), products and sums as in fp32, the result 2^-8:
      |dw - exact| <= 2^-8 |exact| + (1 + 2^-8) (2^-8 + 3 u + 2 (T + 8) u (1 + 2^-8)) S,  S = sum |dout r x^|.
    The roundings of h are as good as independent, so that over the matrix they add in squares: the 2-norm of the error is
    within 2^-8 of ||exact|| + ||sqrt(sum (dout r x^)^2)||, the accumulation's share aside."""
    x, dout = dev(synth.make_random_rows(T, K, T, 2.0)), dev(synth.make_random_rows(T, N, T + 1, 0.05))
    c, s, inv = mx.quant_fwd(x) if layout == "row_major" else mx.quant_fwd_mma(x)
    dw = mx.linear_wgrad_ckpt(c, s, inv, dout, layout).double()
    h, g = mx.mx_dequant(c, s, layout=layout).double() * inv.double()[:, None], dout.double()
    exact, size = g.t() @ h, g.abs().t() @ h.abs()
    err = (dw - exact).abs()
    r = 2.0 ** -8
    assert (err <= r * exact.abs() + (1 + r) * (r + 3 * U + 2 * (T + 8) * U * (1 + r)) * size + 1e-38).all()
    squares = ((g * g).t() @ (h * h)).sum().sqrt()
    assert err.norm() <= r * (exact.norm() + squares) + 2 * (T + 8) * U * size.norm()


@pytest.mark.parametrize("T,H,layout", [(70, 32, "row_major"), (70, 128, "mma"), (71, 224, "row_major"), (70, 512, "mma"), (2000, 1024, "mma"),
                                        (70, 1024, "mma"), (5000, 2048, "mma"), (70, 4096, "mma"), (5000, 4096, "row_major"),
                                        (9, 8192, "mma"), (5, 16384, "mma"), (5, 16416, "row_major")])
def test_dx_of_rows_without_a_value(T, H, layout):
    """inv_rms = +Inf gives dx = 0 in every form of the kernel (several rows a warp, a warp, a CTA a row, rows read twice),
    NaN stays NaN, and the other rows keep the bits that they have without such neighbours."""
    x, dy = dev(synth.make_random_rows(T, H, 1, 2.0)), dev(synth.make_random_rows(T, H, 2))
    c, s, inv = mx.quant_fwd(x) if layout == "row_major" else mx.quant_fwd_mma(x)
    want = mx.bwd_ste_ckpt(c, s, dy, inv, layout)
    empty, bad = torch.zeros(T, dtype=torch.bool, device="cuda"), torch.zeros(T, dtype=torch.bool, device="cuda")
    empty[0::3] = True
    bad[1::7] = True
    bad &= ~empty
    r = inv.clone()
    r[empty], r[bad] = float("inf"), float("nan")
    got = mx.bwd_ste_ckpt(c, s, dy, r, layout)
    assert (got[empty] == 0).all() and got[bad].isnan().all()
    rest = ~(empty | bad)
    assert torch.equal(got[rest], want[rest])
