"""Failure detection in the tensor-core kernels' pipelines without a GPU
fault: a drill withholds one load of a stage and shortens the limit of the
bounded waits.  The waits behind the load must run out and be reported in the
kernel's bit of the device error word, the call must return within a few
limits with its copies landed and its tensor memory freed, nothing outside
the output may change, and the next normal calls must be exact and clean."""
import time

import pytest
import torch

import mx_scale_reusing_gb300 as mx
from mx_scale_reusing_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mx_scale_reusing_gb300 import _build
    _build.build()
    mx.lib()


def dev(b):
    return torch.from_numpy(b.view("int16")).view(torch.bfloat16).cuda()


def drilled(call, rows, cols):
    """Run call(out) on a guarded output; (error word, seconds)."""
    buf = torch.full((rows * cols + 64,), 7.5, dtype=torch.bfloat16, device="cuda")
    mx.device_errors(clear=True)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call(buf[:rows * cols].view(rows, cols))
    torch.cuda.synchronize()
    seconds = time.perf_counter() - t0
    assert (buf[rows * cols:] == 7.5).all()
    return mx.device_errors(clear=True), seconds


# one accumulator narrow and wide, two accumulators narrow and wide, rows whole and split, several tiles a pair
WGRAD = [(700, 96, 24), (1725, 32, 4952), (6000, 512, 520), (20000, 64, 72), (200, 768, 768), (1025, 1024, 1000),
         (2050, 2304, 2568), (5375, 3648, 272)]


@pytest.mark.parametrize("T,K,N", WGRAD)
@pytest.mark.parametrize("load", [0, 1])
def test_wgrad_waits_expire_and_are_reported(T, K, N, load):
    x, dout = dev(synth.make_random_rows(T, K, 1, 2.0)), dev(synth.make_random_rows(T, N, 2, 0.1))
    c, s, inv = mx.quant_fwd(x)
    want = mx.linear_wgrad_ckpt(c, s, inv, dout, "row_major")
    for stage in (0, 1, 9):
        err, seconds = drilled(lambda o: mx.linear_wgrad_wait_drill(c, s, inv, dout, "row_major", load, stage, out=o), N, K)
        # a pair whose share has no such stage loses nothing; the first stage is every pair's
        assert err in (0, 16) and (err == 16 or stage > 0)
        assert seconds < 0.5, f"the drill took {seconds:.3f} s"
        assert torch.equal(want, mx.linear_wgrad_ckpt(c, s, inv, dout, "row_major"))
        assert mx.device_errors() == 0
    err, _ = drilled(lambda o: mx.linear_wgrad_wait_drill(c, s, inv, dout, "row_major", load, 1 << 40, out=o), N, K)
    assert err == 0


def test_wgrad_drill_without_a_withheld_load_is_the_call():
    x, dout = dev(synth.make_random_rows(300, 256, 1, 2.0)), dev(synth.make_random_rows(300, 136, 2, 0.1))
    c, s, inv = mx.quant_fwd(x)
    assert torch.equal(mx.linear_wgrad_ckpt(c, s, inv, dout, "row_major"),
                       mx.linear_wgrad_wait_drill(c, s, inv, dout, "row_major", 1, 1 << 40))
    assert mx.device_errors() == 0


# few rows: K whole, split over two, four and eight CTAs, one and two CTAs an SM; many rows: one tile and several a
# pair, halved tiles, rows of every alignment
PRODUCT = [(3, 640, 1300), (1, 4096, 2048), (33, 4096, 2050), (65, 4096, 6144), (1, 1024, 28672), (128, 4096, 28672),
           (300, 768, 1000), (700, 2304, 768), (2125, 4096, 2057), (2200, 384, 904)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,K,N", PRODUCT)
def test_product_waits_expire_and_are_reported(T, K, N, fmt):
    x, w = dev(synth.make_random_rows(T, K, 3, 2.0)), dev(synth.make_random_rows(64, K, 4, 0.05)).repeat(-(-N // 64), 1)[:N]
    if fmt == "nvfp4":
        xc, xs, inv, xg = mx.quant_fwd_nvfp4_mma(x)
    else:
        (xc, xs, inv), xg = mx.quant_fwd_mma(x, fmt=fmt), None
    wc, ws, wg = mx.mx_cast_fp4(w.contiguous(), fmt)
    args = (xc, xs, inv, wc, ws, fmt, xg, wg)
    want = mx.linear_fwd_fp4(*args)
    for stage in (0, 1, 7):
        err, seconds = drilled(lambda o: mx.linear_fp4_wait_drill(*args, stage, out=o), T, N)
        # work that has no such stage loses nothing; the first stage is everyone's
        assert err in (0, 8) and (err == 8 or stage > 0)
        assert seconds < 0.5, f"the drill took {seconds:.3f} s"
        assert torch.equal(want, mx.linear_fwd_fp4(*args))
        assert mx.device_errors() == 0
    out = mx.linear_fp4_wait_drill(*args, 1 << 40)
    assert torch.equal(want, out) and mx.device_errors() == 0
