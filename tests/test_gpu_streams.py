"""The `stream` argument: what a call allocates is neither handed to the
current stream while the argument's stream still uses it, nor to the
argument's stream while the current one still reads it.  The streams are held
back by a timed spin, so that every reuse that the allocator allows happens."""
import pytest
import torch

import mx_scale_reusing_gb300 as mx

pytestmark = pytest.mark.gpu
SPIN = 20_000_000   # clocks: some 10 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mx_scale_reusing_gb300 import _build
    _build.build()
    mx.lib()


T, H, N = 512, 1024, 256


@pytest.fixture(scope="module")
def d():
    torch.manual_seed(0)
    bf = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
    v = {"x": bf(T, H), "y": bf(T, H), "w": bf(N, H), "dout": bf(T, N), "gamma": torch.ones(H, device="cuda")}
    v["c"], v["s"], v["inv"] = mx.quant_fwd(v["x"])
    v["xc"], v["xs"], v["r"] = mx.quant_fwd_mma(v["x"])
    v["wc"], v["ws"] = mx.mx_cast_gain(v["w"], v["gamma"])
    v["x4"], v["x4s"], v["r4"] = mx.quant_fwd_mma(v["x"], fmt="mxfp4")
    v["w4"], v["w4s"], _ = mx.mx_cast_fp4(v["w"])
    v["g"] = torch.tensor([0.004], device="cuda")
    return v


CALLS = {
    "quant_fwd": lambda d, s: mx.quant_fwd(d["x"], stream=s),
    "rmsnorm": lambda d, s: mx.rmsnorm_mxfp8_ref_fwd(d["x"], stream=s),
    "quant_fwd_nvfp4": lambda d, s: mx.quant_fwd_nvfp4(d["x"], 2, d["g"], stream=s),
    "quant_fwd_mma": lambda d, s: mx.quant_fwd_mma(d["x"], stream=s),
    "mx_cast": lambda d, s: mx.mx_cast(d["x"], stream=s),
    "mx_cast_gain": lambda d, s: mx.mx_cast_gain(d["w"], d["gamma"], stream=s),
    "linear_fwd": lambda d, s: [mx.linear_fwd(d["xc"], d["xs"], d["r"], d["wc"], d["ws"], stream=s)],
    "bwd_ste": lambda d, s: [mx.bwd_ste(d["x"], d["y"], d["inv"], stream=s)],
    "quant_fwd_nvfp4_mma": lambda d, s: mx.quant_fwd_nvfp4_mma(d["x"], 2, d["g"], stream=s)[:3],
    "mx_cast_fp4": lambda d, s: mx.mx_cast_fp4(d["w"], stream=s)[:2],
    "mx_dequant": lambda d, s: [mx.mx_dequant(d["c"], d["s"], stream=s)],
    "linear_fwd_fp4": lambda d, s: [mx.linear_fwd_fp4(d["x4"], d["x4s"], d["r4"], d["w4"], d["w4s"], stream=s)],
    "bwd_ste_ckpt": lambda d, s: [mx.bwd_ste_ckpt(d["c"], d["s"], d["y"], d["inv"], stream=s)],
    "linear_wgrad_ckpt": lambda d, s: [mx.linear_wgrad_ckpt(d["c"], d["s"], d["inv"], d["dout"], "row_major", stream=s)],
}


@pytest.mark.parametrize("name", CALLS)
def test_dropped_outputs_are_not_reused_before_they_are_written(name, d):
    """The call waits behind the spin on its stream, its outputs are dropped, and the current stream fills memory of the
    same sizes: nothing of the late call may appear there."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    outs = CALLS[name](d, side)
    shapes = [(o.shape, o.dtype) for o in outs]
    del outs
    fill = [torch.full(s, 3, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    assert all((f == 3).all() for f in fill)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_being_read_are_not_written_again(name, d):
    """The current stream reads the outputs late, behind a spin, and drops them; another call on the same stream takes
    outputs of the same sizes meanwhile, on inputs of its own."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = CALLS[name](d, side)
    side.synchronize()
    want = [o.cpu() for o in outs]
    torch.cuda._sleep(SPIN)
    late = [o.clone() for o in outs]
    shapes = [(o.shape, o.dtype) for o in outs]
    del outs
    with torch.cuda.stream(side):
        fill = [torch.full(s, 3, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8)) for a, b in zip(want, late))
    del fill


def test_a_stream_that_only_names_its_handle(d):
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = mx.quant_fwd(d["x"], stream=Handle(side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (d["c"], d["s"], d["inv"])))


def test_stream_argument_in_a_capture(d):
    """A fork of the captured stream: the calls' memory is the graph's, whichever stream they name."""
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = mx.linear_wgrad_ckpt(*mx.quant_fwd(d["x"]), d["dout"], "row_major")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        side.wait_stream(current)
        for _ in range(3):   # outputs dropped and taken again within the capture
            got = mx.linear_wgrad_ckpt(*mx.quant_fwd(d["x"], stream=side), d["dout"], "row_major", stream=side)
        current.wait_stream(side)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
