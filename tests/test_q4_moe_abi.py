"""Host side of the 4-bit streams and the expert routing: sizes, headers and
the refusal of unusable arguments. No call here reaches the GPU."""
import numpy as np
import pytest
import torch

import q4_plain

A = 1 << 20  # an aligned stand-in for a device address; every call returns before using it


def test_sizes_match_the_plain_streams(wclib):
    rng = np.random.default_rng(0)
    for rows, cols, group, zeros in [(1, 1, 32, True), (16, 128, 128, False), (17, 129, 64, True),
                                     (130, 300, 32, False), (257, 64, 128, True)]:
        q, s, z = q4_plain.make(rng, rows, cols, group, zeros, False)
        assert wclib.wc_q4_bytes(rows, cols, group, int(zeros)) == \
            q4_plain.stream(q, s, z, group, False).size
    assert wclib.wc_q4_bytes(0, 5, 32, 0) == 128  # a bare header
    for bad in [(4, 0, 32, 0), (4, 4, 16, 0), (4, 4, 256, 0), (4, 4, 32, 4), (2**22 + 1, 4, 32, 0),
                (4, 2**20 + 1, 32, 0)]:
        assert wclib.wc_q4_bytes(*bad) == 0, bad


def test_stream_info_reads_4bit_headers(wclib):
    rng = np.random.default_rng(1)
    q, s, z = q4_plain.make(rng, 33, 200, 64, True, True)
    b = q4_plain.stream(q, s, z, 64, True)
    assert wclib.wc_stream_info(b[:128].tobytes()) == (0, 33 * 200, 64, b.size)
    for off in (0, 4, 8, 12, 13, 16, 24, 32, 40, 64, 72, 80, 88, 92, 100):
        bad = bytearray(b[:128].tobytes())
        bad[off] ^= 1
        assert wclib.wc_stream_info(bytes(bad))[0] == wclib.WC_ERR_CORRUPT_STREAM, off


def test_q4_arguments(wclib):
    c, INV = wclib, wclib.WC_ERR_INVALID_ARG
    size = c.wc_q4_bytes(32, 256, 128, 0)
    assert c.wc_q4_quantize(A, 256, 32, 256, 100, 0, A, size, None) == INV       # group
    assert c.wc_q4_quantize(A, 255, 32, 256, 128, 0, A, size, None) == INV       # ld < cols
    assert c.wc_q4_quantize(A + 1, 256, 32, 256, 128, 0, A, size, None) == INV   # odd address
    assert c.wc_q4_quantize(A, 256, 32, 256, 128, 0, A + 8, size, None) == INV   # stream alignment
    assert c.wc_q4_quantize(None, 256, 32, 256, 128, 0, A, size, None) == INV
    assert c.wc_q4_quantize(A, 256, 32, 256, 128, 4, A, size, None) == INV       # a product's flag
    assert c.wc_q4_quantize(A, 256, 32, 256, 128, 0, A, size - 1, None) == c.WC_ERR_BUFFER_TOO_SMALL
    assert c.wc_q4_pack(A, A, None, 32, 256, 128, 1, A, 2 * size, None) == INV   # no zero points
    assert c.wc_q4_pack(A, A, A, 32, 256, 128, 0, A, 2 * size, None) == INV      # unasked ones
    assert c.wc_q4_pack(A, A, None, 32, 256, 128, 0, A, size - 1, None) == c.WC_ERR_BUFFER_TOO_SMALL
    assert c.wc_q4_dequantize(A, size - 1, 32, 256, 128, 0, A, 256, 0, None, None) == \
        c.WC_ERR_CORRUPT_STREAM
    assert c.wc_q4_dequantize(A, size, 32, 256, 128, 0, A, 256, 3, None, None) == INV  # dtype
    assert c.wc_q4_dequantize(A, size, 32, 256, 128, 0, A + 2, 256, 2, None, None) == INV
    assert c.wc_q4_dequantize(A, size, 32, 256, 128, 0, A, 100, 0, None, None) == INV
    g = dict(flags=0, x=A, ldx=256, tokens=4, y=A, ldy=32, size=size)

    def gemm(**kw):
        a = dict(g, **kw)
        return c.wc_q4_gemm(A, a["size"], 32, 256, 128, a["flags"], a["x"], a["ldx"], a["tokens"],
                            a["y"], a["ldy"], None, None)
    assert gemm(size=size - 1) == c.WC_ERR_CORRUPT_STREAM
    for bad in (dict(flags=16), dict(x=None), dict(y=None), dict(x=A + 1), dict(y=A + 2),
                dict(y=A + 1, flags=8), dict(ldx=255), dict(ldy=31), dict(tokens=2**24 + 1)):
        assert gemm(**bad) == INV, bad

    def experts(stride=size, experts=2, offsets=A, streams=A):
        return c.wc_q4_gemm_experts(streams, stride, experts, 32, 256, 128, 0, A, 256, 4, offsets,
                                    A, 32, None, None)
    assert experts(stride=size - 16) == c.WC_ERR_CORRUPT_STREAM
    for bad in (dict(stride=size + 8), dict(experts=0), dict(experts=1025), dict(offsets=None),
                dict(offsets=A + 2), dict(streams=None)):
        assert experts(**bad) == INV, bad


def test_moe_arguments(wclib):
    c, INV = wclib, wclib.WC_ERR_INVALID_ARG
    for bad in [(A, 8, 0, A, None, A), (A, 8, 1025, A, None, A), (None, 8, 4, A, None, A),
                (A, 8, 4, None, None, A), (A, 8, 4, A, None, None), (A + 2, 8, 4, A, None, A),
                (A, 2**31, 4, A, None, A)]:
        assert c.wc_moe_sort(*bad, None) == INV, bad

    def gather(x=A, ldx=8, tokens=4, top=2, cols=8, dtype=0, inv=A, rows=A, ldr=8, n=8):
        return c.wc_moe_gather(x, ldx, tokens, top, cols, dtype, inv, rows, ldr, n, None)

    def combine(rows=A, ldr=8, n=8, tokens=4, top=2, cols=8, dtype=0, inv=A, w=A, out=A, ldo=8):
        return c.wc_moe_combine(rows, ldr, n, tokens, top, cols, dtype, inv, w, out, ldo, None)

    def backward(d=A, ldd=8, rows=A, ldr=8, n=8, tokens=4, top=2, cols=8, dtype=0, inv=A, w=A,
                 dr=A, lddr=8, dw=A):
        return c.wc_moe_combine_backward(d, ldd, rows, ldr, n, tokens, top, cols, dtype, inv, w, dr,
                                         lddr, dw, None)
    for f in (gather, combine, backward):
        for bad in (dict(dtype=3), dict(inv=None), dict(inv=A + 1), dict(ldr=7), dict(rows=None),
                    dict(rows=A + 1), dict(tokens=2**31, top=1), dict(tokens=2**20, top=2**12),
                    dict(cols=2**24 + 1, ldr=2**25)):
            assert f(**bad) == INV, (f, bad)
    assert gather(x=None) == INV and gather(ldx=7) == INV
    assert combine(out=None) == INV and combine(ldo=7) == INV and combine(w=A + 2) == INV
    assert backward(d=None) == INV and backward(dr=None) == INV and backward(lddr=7) == INV
    assert backward(dw=A + 1) == INV and backward(w=A + 2) == INV
    # nothing to do
    assert gather(tokens=0) == 0 and combine(tokens=0) == 0 and backward(tokens=0) == 0
    assert gather(cols=0) == 0 and combine(cols=0) == 0


def test_helpers_refuse_host_tensors_and_wrong_shapes(wclib):
    w = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        wclib.quantize_q4(w)
    with pytest.raises(TypeError):
        wclib.quantize_q4(w.float())
    with pytest.raises(wclib.WcodecError):
        wclib.quantize_q4(w, 48)
    with pytest.raises(ValueError, match="dense rows"):
        wclib.quantize_q4(w.T)
    m = wclib.Q4Matrix(torch.zeros(128 + 1056, dtype=torch.uint8), 4, 8, 128, False, torch.bfloat16)
    with pytest.raises(ValueError, match="8 columns"):
        wclib.gemm_q4(m, torch.zeros((1, 9), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="FP32 or has x's type"):
        wclib.gemm_q4(m, w, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="BF16 or FP16"):
        wclib.gemm_q4(m, w.float())
    with pytest.raises(ValueError, match="2 dimension"):
        wclib.gemm_q4_experts(m, w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows"):
        wclib.gemm_q4(m, w, y=torch.zeros((3, 4)))
    with pytest.raises(ValueError, match="CUDA"):
        wclib.gemm_q4(m, w)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="experts"):
        wclib.moe_sort(ids, 1025)
    with pytest.raises(ValueError, match="int32"):
        wclib.moe_sort(ids.long(), 8)
    with pytest.raises(ValueError, match="CUDA"):
        wclib.moe_sort(ids, 8)
    plan = wclib.MoePlan(torch.zeros(9, dtype=torch.int32), None, ids)
    with pytest.raises(ValueError, match="4 rows"):
        wclib.moe_gather(w[:3], plan)
    with pytest.raises(TypeError):
        wclib.moe_combine(ids.double().expand(4, 2), plan, None)
    with pytest.raises(ValueError, match="weights"):
        wclib.moe_combine(w, plan, torch.zeros((4, 3)))
    with pytest.raises(ValueError, match="dense rows"):
        wclib.moe_combine_backward(torch.zeros((1, 8), dtype=torch.bfloat16).expand(4, 8), w, plan,
                                   None)


def test_experts_streams_shorter_than_their_stride(wclib):
    """Views of a stack whose rows are too short for a stream, however far apart
    they lie, are refused as a short stream of one matrix is; views that hold
    their streams pass (and are then refused for lying on the host)."""
    size = wclib.wc_q4_bytes(32, 256, 128, 0)
    big = torch.zeros((4, size + 64), dtype=torch.uint8)
    x, off = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)

    def call(b):
        return wclib.gemm_q4_experts(wclib.Q4Matrix(b, 32, 256, 128, False, torch.bfloat16), x,
                                     off[:b.shape[0] + 1])
    for short in (big[:, 80:], big[:, :size - 1], big[:, :0], big[:1, :size - 1], big[2:, 65:]):
        with pytest.raises(wclib.WcodecError) as e:
            call(short)
        assert e.value.status == wclib.WC_ERR_CORRUPT_STREAM
    for whole in (big, big[:, 64:], big[:, :size], big[:1, :size + 8]):
        with pytest.raises(ValueError, match="CUDA"):
            call(whole)


def test_a_stream_of_another_device_is_refused(wclib):
    """(Not taken silently for the current stream of the tensors' device.)"""
    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        with wclib._there(torch.device("cuda", 0), Stream()):
            pass


def test_tensors_that_autograd_follows_are_refused(wclib):
    """Results have no graph, so inputs and outputs that need one are refused,
    unless gradients are off; what is left is the refusal of host tensors."""
    m = wclib.Q4Matrix(torch.zeros(128 + 1056, dtype=torch.uint8), 4, 8, 128, False, torch.bfloat16)
    stack = wclib.Q4Matrix(m.buffer[None], 4, 8, 128, False, torch.bfloat16)
    plan = wclib.MoePlan(torch.zeros(3, dtype=torch.int32), None, torch.zeros((4, 2), dtype=torch.int32))
    off = torch.tensor([0, 4], dtype=torch.int32)
    w = torch.zeros((4, 8), dtype=torch.bfloat16)
    g = w.clone().requires_grad_()
    rows, grows = torch.zeros((8, 8), dtype=torch.bfloat16), torch.zeros((8, 8), dtype=torch.bfloat16, requires_grad=True)
    gw = torch.ones((4, 2), requires_grad=True)
    y = torch.zeros((4, 4), requires_grad=True)
    calls = [lambda: wclib.gemm_q4(m, g), lambda: wclib.gemm_q4(m, w, y=y), lambda: wclib.gemm_q4_experts(stack, g, off),
             lambda: wclib.dequantize_q4(m, out=g), lambda: wclib.moe_gather(g, plan),
             lambda: wclib.moe_gather(w, plan, out=grows), lambda: wclib.moe_combine(grows, plan, None),
             lambda: wclib.moe_combine(rows, plan, gw), lambda: wclib.moe_combine(rows, plan, None, out=g),
             lambda: wclib.moe_gather_backward(grows, plan), lambda: wclib.moe_combine_backward(g, rows, plan, None),
             lambda: wclib.moe_combine_backward(w, grows, plan, None),
             lambda: wclib.moe_combine_backward(w, rows, plan, gw),
             lambda: wclib.moe_combine_backward(w, rows, plan, None, drows=grows)]
    for call in calls:
        with pytest.raises(ValueError, match="autograd graph"):
            call()
        with pytest.raises(ValueError, match="CUDA"), torch.no_grad():
            call()
    with pytest.raises(ValueError, match="CUDA"):  # bytes need no graph
        wclib.quantize_q4(g)
