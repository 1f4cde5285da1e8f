"""The helpers of the 4-bit streams and the expert routing on a stream of the
caller's: inputs that the caller lets go of as soon as a call returns."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def calls(wc, device):
    """name -> (function of (stream, inputs...), inputs); each returns its results."""
    g = torch.Generator(device="cpu").manual_seed(5)
    w = torch.randn((64, 256), generator=g).to(device, torch.bfloat16)
    m = wc.quantize_q4(w, 64, zeros=True)
    x = torch.randn((24, 256), generator=g).to(device, torch.bfloat16)
    codes = torch.randint(0, 16, (64, 256), generator=g).to(device, torch.uint8)
    scales = torch.rand((64, 4), generator=g).to(device, torch.bfloat16)
    zeros = torch.randint(0, 16, (64, 4), generator=g).to(device, torch.uint8)
    ids = torch.randint(0, 4, (12, 2), generator=g).to(device, torch.int32)
    plan = wc.moe_sort(ids, 4)
    weights = torch.rand((12, 2), generator=g).to(device)

    def q4(b):
        return wc.Q4Matrix(b, 64, 256, 64, True, torch.bfloat16)

    def inverse(t):
        return wc.MoePlan(plan.offsets, None, t)
    return {
        "quantize": (lambda s, a: wc.quantize_q4(a, 64, zeros=True, stream=s).buffer, [w]),
        "pack": (lambda s, a, b, c: wc.pack_q4(a, b, c, group=64, stream=s).buffer, [codes, scales, zeros]),
        "dequantize": (lambda s, a: wc.dequantize_q4(q4(a), stream=s), [m.buffer]),
        "product": (lambda s, a, b: wc.gemm_q4(q4(a), b, stream=s), [m.buffer, x]),
        "few rows": (lambda s, a, b: wc.gemm_q4(q4(a), b, stream=s), [m.buffer, x[:3].clone()]),
        "experts": (lambda s, a, b, c: wc.gemm_q4_experts(q4(a), b, c, stream=s),
                    [m.buffer.expand(4, -1).contiguous(), x, plan.offsets]),
        "sort": (lambda s, a: [t for t in vars(wc.moe_sort(a, 4, stream=s)).values()], [ids]),
        "gather": (lambda s, a, b: wc.moe_gather(a, inverse(b), stream=s), [x[:12].clone(), plan.inverse]),
        "combine": (lambda s, a, b, c: wc.moe_combine(a, inverse(b), c, stream=s), [x, plan.inverse, weights]),
        "gather's gradient": (lambda s, a, b: wc.moe_gather_backward(a, inverse(b), stream=s), [x, plan.inverse]),
        "combine's gradients": (lambda s, a, b, c, d: list(wc.moe_combine_backward(a, b, inverse(c), d, stream=s)),
                                [x[:12].clone(), x, plan.inverse, weights]),
    }


NAMES = ["quantize", "pack", "dequantize", "product", "few rows", "experts", "sort", "gather", "combine",
         "gather's gradient", "combine's gradients"]


@pytest.mark.parametrize("name", NAMES)
def test_inputs_let_go_of_after_a_call_on_another_stream(wclib, cuda, name):
    """The caller's last reference to each input goes with the call, and its
    memory is asked for again and overwritten on the caller's stream while the
    call still waits behind other work on its own."""
    f, inputs = calls(wclib, cuda)[name]
    want = f(None, *inputs)
    want = [t.clone() for t in (want if isinstance(want, list) else [want])]
    side = torch.cuda.Stream()
    f(side, *inputs)
    torch.cuda.synchronize()
    own = [t.clone() for t in inputs]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = f(side, *[own.pop(0) for _ in inputs])
    noise = [torch.zeros_like(t) for t in inputs for _ in range(4)]
    torch.cuda.synchronize()
    got = got if isinstance(got, list) else [got]
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 0).all() for t in noise)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_that_joins_a_capture(wclib, cuda, name):
    """A call on a second stream of a capture, its inputs made and let go of
    within the capture; replayed on new inputs."""
    f, inputs = calls(wclib, cuda)[name]
    held = [t.clone() for t in inputs]
    side = torch.cuda.Stream()
    f(side, *inputs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        made = [t + 0 for t in held]
        side.wait_stream(main)
        got = f(side, *[made.pop(0) for _ in inputs])
        noise = [torch.zeros_like(t) for t in inputs]
        main.wait_stream(side)
    got = got if isinstance(got, list) else [got]
    for _ in range(2):
        want = f(None, *held)
        want = want if isinstance(want, list) else [want]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if name not in ("dequantize", "product", "few rows", "experts"):  # (their first input is a stream)
            held[0].copy_(held[0].flip(0))
    assert all((t == 0).all() for t in noise)
