"""4-bit streams and their products on the GPU against plain 64-bit forms.

Streams: byte for byte. Products: with G = group and K groups a row, a group's
FP32 sum of G exact products is off by at most G 2^-22 of its sum of magnitudes
(the tensor cores' accumulation rounds in an unspecified way; 2^-22 covers
truncation with a guard bit, as for the other fused products), and scaling and
adding the K groups and the at most 64 partial sums of warps and thread blocks
by at most (K + 64) 2^-24 more. So every FP32 output is within
(G + K + 64) 2^-22 sum |w x| of the exact sum, a 16-bit one half a step further.
"""
import numpy as np
import pytest
import torch

import q4_plain

pytestmark = pytest.mark.gpu

DT = {False: torch.bfloat16, True: torch.float16}


def dev(a, device):
    return torch.from_numpy(np.array(a)).to(device)


def half_words(bits, half, device):
    return dev(bits.view(np.int16), device).view(DT[half])


def matrix(wc, rng, rows, cols, group, zeros, half, device):
    q, s, z = q4_plain.make(rng, rows, cols, group, zeros, half)
    b = dev(q4_plain.stream(q, s, z, group, half), device)
    return wc.Q4Matrix(b, rows, cols, group, zeros, DT[half]), q4_plain.weights(q, s, z, group, half)


def acts(rng, tokens, cols, half, device):
    x = dev(rng.standard_normal((tokens, cols)).astype(np.float32), device).to(DT[half])
    return x, x.double().cpu().numpy()


def check(y, W, x, group, cols):
    ref, absum = x @ W.T, np.abs(x) @ np.abs(W).T
    tol = (group + -(-cols // group) + 64) * 2.0 ** -22 * absum + 1e-30
    if y.dtype != torch.float32:
        f = torch.finfo(y.dtype)  # below the smallest normal value steps stay smallest_normal * eps
        tol = tol + f.eps / 2 * (np.abs(ref) + tol + f.smallest_normal)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("rows,cols,group,zeros,half", [
    (1, 1, 32, False, False), (5, 130, 32, True, True), (16, 128, 64, False, True),
    (129, 300, 128, True, False), (300, 1000, 64, True, False), (64, 257, 128, False, False)])
def test_pack_and_dequantize(wclib, cuda, rows, cols, group, zeros, half):
    rng = np.random.default_rng(rows + cols)
    q, s, z = q4_plain.make(rng, rows, cols, group, zeros, half)
    m = wclib.pack_q4(dev(q, cuda), half_words(s, half, cuda), None if z is None else dev(z, cuda),
                      group=group)
    assert np.array_equal(m.buffer.cpu().numpy(), q4_plain.stream(q, s, z, group, half))
    W = torch.from_numpy(q4_plain.weights(q, s, z, group, half))
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        out = wclib.dequantize_q4(m, dt, status=status).cpu()
        assert status.item() == 0
        # FP32 holds s (q - z) exactly, so the 16-bit values are rounded once
        assert torch.equal(out, W.float().to(dt))
    wide = torch.full((rows, cols + 3), 7.0, device=cuda)
    wclib.dequantize_q4(m, out=wide[:, 1:cols + 1])
    assert torch.equal(wide[:, 1:cols + 1].cpu(), W.float())
    assert (wide[:, 0] == 7).all() and (wide[:, cols + 1:] == 7).all()


def plain_quantize(w, group, zeros, dtype):
    """Scale bits, zero points and codes in 64 bits (w float64)."""
    rows, cols = w.shape
    g = q4_plain.groups_of(cols, group)
    S, Z, Q = np.zeros((rows, g)), np.zeros((rows, g)), np.zeros((rows, cols))
    for k in range(g):
        p = w[:, k * group:(k + 1) * group]
        if zeros:
            lo, hi = np.minimum(p.min(1), 0), np.maximum(p.max(1), 0)
            s = torch.from_numpy((hi - lo) / 15).to(dtype).double().numpy()
        else:
            s = torch.from_numpy(np.abs(p).max(1) / 7).to(dtype).double().numpy()
        d = np.where(s > 0, s, 1)
        z = np.clip(np.rint(-lo / d), 0, 15) if zeros else np.full(rows, 8.0)
        S[:, k], Z[:, k] = s, z
        Q[:, k * group:(k + 1) * group] = np.clip(np.rint(p / d[:, None]) + z[:, None], 0, 15)
    bits = torch.from_numpy(S).to(dtype).view(torch.int16).numpy().view(np.uint16)
    return Q.astype(np.uint8), bits, Z.astype(np.uint8) if zeros else None


@pytest.mark.parametrize("rows,cols,group,zeros,half", [
    (1, 1, 128, True, False), (33, 100, 32, False, True), (130, 384, 64, True, True),
    (257, 1030, 128, False, False), (128, 256, 32, True, False)])
def test_quantize_matches_64_bits(wclib, cuda, rows, cols, group, zeros, half):
    rng = np.random.default_rng(rows * 7 + cols)
    w = torch.from_numpy(rng.standard_normal((rows, cols)) * rng.uniform(0.001, 3, (rows, 1)))
    w[rows // 2] = 0.0                      # a row of zeros: scale 0, codes that stand for zero
    w[0, :] = w[0, 0].abs()                 # a row of one value
    if rows > 4:
        w[3] = w[3].abs()                   # one sign only
        w[4, ::2] = torch.finfo(DT[half]).tiny / 4  # subnormal values
    w = w.to(DT[half])
    m = wclib.quantize_q4(w.to(cuda), group, zeros=zeros)
    q, s, z = plain_quantize(w.double().numpy(), group, zeros, DT[half])
    assert np.array_equal(m.buffer.cpu().numpy(), q4_plain.stream(q, s, z, group, half))
    # rows apart and off 16-byte boundaries: the same stream
    wide = torch.zeros((rows, cols + 5), dtype=DT[half], device=cuda)
    wide[:, 1:cols + 1] = w.to(cuda)
    assert torch.equal(wclib.quantize_q4(wide[:, 1:cols + 1], group, zeros=zeros).buffer, m.buffer)


def test_quantize_carries_nan_and_infinity(wclib, cuda):
    for zeros in (False, True):
        w = torch.randn((16, 256), device=cuda).to(torch.bfloat16)
        w[1, 3], w[2, 200], w[5, 0] = float("nan"), float("inf"), float("-inf")
        d = wclib.dequantize_q4(wclib.quantize_q4(w, 128, zeros=zeros), torch.float32)
        assert d[1, :128].isnan().all() and d[1, 128:].isfinite().all()
        assert not d[2, 128:].isfinite().any() and not d[5, :128].isfinite().any()
        keep = [r for r in range(16) if r not in (1, 2, 5)]
        assert d[keep].isfinite().all()


SHAPES = [(1, 1, 32, True), (16, 128, 128, False), (7, 1024, 64, False), (130, 384, 32, True),
          (257, 4096, 128, True), (300, 1290, 64, True), (2053, 520, 128, False), (64, 14336, 32, False)]


@pytest.mark.parametrize("rows,cols,group,zeros", SHAPES)
@pytest.mark.parametrize("tokens", [1, 2, 8, 9, 16, 17, 33, 64, 128, 129, 300])
def test_product(wclib, cuda, rows, cols, group, zeros, tokens):
    rng = np.random.default_rng(rows * 131 + cols + tokens)
    half = bool((rows + tokens) % 2)
    m, W = matrix(wclib, rng, rows, cols, group, zeros, not half, cuda)
    x, xd = acts(rng, tokens, cols, half, cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    y = wclib.gemm_q4(m, x, status=status)
    assert status.item() == 0 and y.dtype == torch.float32
    check(y, W, xd, group, cols)
    assert torch.equal(y, wclib.gemm_q4(m, x))  # the same bits
    check(wclib.gemm_q4(m, x, out_dtype=x.dtype), W, xd, group, cols)


@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("rows,cols,group,zeros", SHAPES[3:6])
def test_product_of_strided_and_unaligned_rows(wclib, cuda, rows, cols, group, zeros, tokens):
    rng = np.random.default_rng(rows + tokens)
    m, W = matrix(wclib, rng, rows, cols, group, zeros, False, cuda)
    x, xd = acts(rng, tokens, cols, False, cuda)
    for pad, at in ((8, 0), (8, 8), (3, 1), (2, 2)):
        xs = torch.full((tokens, cols + pad), float("nan"), dtype=x.dtype, device=cuda)
        xs[:, at:at + cols] = x[:, :xs.shape[1] - at] if at + cols <= xs.shape[1] else x
        ys = torch.full((tokens, rows + 5), 7.0, device=cuda)
        wclib.gemm_q4(m, xs[:, at:at + cols], y=ys[:, 2:rows + 2])
        check(ys[:, 2:rows + 2], W, xd, group, cols)
        assert (ys[:, :2] == 7).all() and (ys[:, rows + 2:] == 7).all()


@pytest.mark.parametrize("tokens_at_once", [8, 64])
@pytest.mark.parametrize("half", [False, True])
def test_unit_vectors_give_every_weight_exactly(wclib, cuda, half, tokens_at_once):
    """x = unit vectors: each output is one weight, whatever the order of the sum."""
    for rows, cols, group, zeros in [(130, 384, 32, True), (48, 256, 64, False), (33, 200, 128, True)]:
        rng = np.random.default_rng(rows)
        m, W = matrix(wclib, rng, rows, cols, group, zeros, half, cuda)
        eye = torch.eye(cols, dtype=DT[half], device=cuda)
        y = torch.cat([wclib.gemm_q4(m, eye[k:k + tokens_at_once])
                       for k in range(0, cols, tokens_at_once)])
        assert np.array_equal(y.double().cpu().numpy(), W.T)


@pytest.mark.parametrize("tokens", [4, 48])
def test_infinities_and_nan(wclib, cuda, tokens):
    rng = np.random.default_rng(tokens)
    m, W = matrix(wclib, rng, 64, 512, 64, False, False, cuda)
    x, xd = acts(rng, tokens, 512, False, cuda)
    x[1, 7], x[2, 300] = float("inf"), float("nan")
    y = wclib.gemm_q4(m, x)
    keep = [t for t in range(tokens) if t not in (1, 2)]
    check(y[keep], W, xd[keep], 64, 512)
    assert y[2].isnan().all()
    w7 = torch.from_numpy(W[:, 7])
    assert torch.equal(y[1].isnan().cpu(), w7 == 0)
    assert torch.equal(y[1].cpu()[w7 != 0] > 0, w7[w7 != 0] > 0) and y[1].isinf().cpu()[w7 != 0].all()


def experts_case(wclib, cuda, E, rows, cols, group, zeros, half, seed):
    rng = np.random.default_rng(seed)
    ms = [matrix(wclib, rng, rows, cols, group, zeros, half, cuda) for _ in range(E)]
    size = (ms[0][0].buffer.numel() + 15) // 16 * 16 + 48  # a stride beyond the size
    buf = torch.zeros((E, size), dtype=torch.uint8, device=cuda)
    for e, (m, _) in enumerate(ms):
        buf[e, :m.buffer.numel()] = m.buffer
    return rng, wclib.Q4Matrix(buf, rows, cols, group, zeros, DT[half]), [w for _, w in ms]


COUNTS = [[0, 1, 0, 5], [0, 0, 0, 0], [3], [1, 1, 1, 1, 1, 1, 1, 1], [130, 0, 17, 1, 64],
          [0, 300, 2], [8, 9, 16, 33]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("rows,cols,group,zeros,half", [(200, 384, 32, True, False),
                                                        (48, 520, 128, False, True)])
def test_experts(wclib, cuda, counts, rows, cols, group, zeros, half):
    E, total = len(counts), sum(counts)
    rng, m, Ws = experts_case(wclib, cuda, E, rows, cols, group, zeros, half, E + total)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xd = acts(rng, total + 5, cols, half, cuda)
    x[total:] = float("nan")  # rows behind the last expert's
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    for dt in (torch.float32, DT[half]):
        y = torch.full((total + 5, rows), 7.0, dtype=dt, device=cuda)
        wclib.gemm_q4_experts(m, x, dev(offsets, cuda), y=y, status=status)
        assert status.item() == 0
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            if b > a:
                check(y[a:b], Ws[e], xd[a:b], group, cols)
        assert (y[total:] == 7).all()
        y2 = torch.full_like(y, 7.0)
        wclib.gemm_q4_experts(m, x, dev(offsets, cuda), y=y2)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("rows,cols", [(200, 2056), (1000, 130)])
@pytest.mark.parametrize("crowd", [5, 40, 90])
def test_one_crowded_expert_among_many(wclib, cuda, rows, cols, crowd):
    """Few rows an expert on average, many at one: several tiles of rows of x
    against the same matrix, in the product of few rows (up to 6 an expert) and
    in the other; the first and last experts empty."""
    E = 16
    rng, m, Ws = experts_case(wclib, cuda, E, rows, cols, 64, True, False, rows + crowd)
    counts = [0, 0, 1, crowd] + [0] * 10 + [2, 0]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xd = acts(rng, sum(counts), cols, False, cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    y = wclib.gemm_q4_experts(m, x, dev(offsets, cuda), status=status)
    assert status.item() == 0
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            check(y[a:b], Ws[e], xd[a:b], 64, cols)
    assert torch.equal(y, wclib.gemm_q4_experts(m, x, dev(offsets, cuda)))


def test_every_alignment_of_rows_of_x(wclib, cuda):
    """Rows of x at every multiple of 2 bytes from a 16-byte boundary, dense and
    odd lengths, few rows and many: the same bits as from an aligned copy."""
    rng = np.random.default_rng(77)
    m, W = matrix(wclib, rng, 150, 333, 32, True, True, cuda)
    for tokens in (5, 70):
        x, xd = acts(rng, tokens, 333, True, cuda)
        wide = torch.zeros((tokens, 336), dtype=x.dtype, device=cuda)
        wide[:, :333] = x
        ref = wclib.gemm_q4(m, wide[:, :333])
        check(ref, W, xd, 32, 333)
        for at in range(8):
            for pad in (334, 336, 340, 341):
                buf = torch.full((tokens * pad + 16,), float("nan"), dtype=x.dtype, device=cuda)
                v = buf[at:at + tokens * pad].view(tokens, pad)[:, :333]
                v.copy_(x)
                assert torch.equal(wclib.gemm_q4(m, v), ref), (tokens, at, pad)


@pytest.mark.parametrize("cols", [1, 2, 3, 8, 16, 31, 64, 127])
def test_narrow_matrices(wclib, cuda, cols):
    """Matrices of less than a slice, in one row of x and many, aligned and not."""
    rng = np.random.default_rng(cols)
    for rows in (1, 17, 129):
        m, W = matrix(wclib, rng, rows, cols, 32, bool(rows % 2), False, cuda)
        for tokens in (1, 9, 20, 130):
            x, xd = acts(rng, tokens, cols, False, cuda)
            check(wclib.gemm_q4(m, x), W, xd, 32, cols)


def test_no_expert_has_rows(wclib, cuda):
    """Offsets all equal, with few rows of x and with many: nothing is written."""
    rng, m, _ = experts_case(wclib, cuda, 4, 64, 256, 64, False, False, 6)
    for tokens in (3, 100):
        x, _ = acts(rng, tokens, 256, False, cuda)
        for at in (0, 2, tokens):
            y = torch.full((tokens, 64), 7.0, device=cuda)
            off = torch.full((5,), at, dtype=torch.int32, device=cuda)
            wclib.gemm_q4_experts(m, x, off, y=y)
            assert (y == 7).all()


def test_many_experts_of_both_products(wclib, cuda):
    """1024 experts (the most), some empty, in the product of few rows and the other."""
    rng = np.random.default_rng(12)
    q, s, z = q4_plain.make(rng, 16, 128, 128, False, False)
    one = dev(q4_plain.stream(q, s, z, 128, False), cuda)
    W = q4_plain.weights(q, s, z, 128, False)
    m = wclib.Q4Matrix(one.repeat(1024, 1).contiguous(), 16, 128, 128, False, torch.bfloat16)
    for most in (3, 20):
        counts = rng.integers(0, most, 1024)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        x, xd = acts(rng, int(offsets[-1]), 128, False, cuda)
        check(wclib.gemm_q4_experts(m, x, dev(offsets, cuda)), W, xd, 128, 128)


def test_offsets_past_32_bits(wclib, cuda):
    """A matrix of more than 2^32 elements: its last rows are those of a matrix of
    their own, quantized, expanded and multiplied (few rows of x and many)."""
    rows, cols, tail = 524288 + 256, 8192, 256
    w = torch.empty((rows, cols), dtype=torch.bfloat16, device=cuda)
    for k in range(0, rows, 65536):
        w[k:k + 65536].normal_()
    m = wclib.quantize_q4(w, 128)
    last = wclib.quantize_q4(w[-tail:], 128)
    assert torch.equal(m.buffer[128 - last.buffer.numel():], last.buffer[128:])
    w.zero_()
    wclib.dequantize_q4(m, out=w)
    assert torch.equal(w[-tail:], wclib.dequantize_q4(last))
    del w
    for tokens in (2, 40):
        x = torch.randn((tokens, cols), device=cuda).to(torch.bfloat16)
        y = wclib.gemm_q4(m, x)[:, -tail:].double()
        W = wclib.dequantize_q4(last, torch.float32).double()
        tol = (128 + 64 + 64) * 2.0 ** -22 * (x.double().abs() @ W.abs().T)
        assert ((y - x.double() @ W.T).abs() <= tol).all()
    torch.cuda.empty_cache()


def test_calls_from_two_threads(wclib, cuda):
    """Two host threads, each on its own stream, many calls at once."""
    import threading
    rng = np.random.default_rng(78)
    m, W = matrix(wclib, rng, 300, 640, 64, False, False, cuda)
    xs = [acts(rng, t, 640, False, cuda)[0] for t in (3, 40)]
    want = [wclib.gemm_q4(m, x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        s = torch.cuda.Stream()
        for _ in range(50):
            y = wclib.gemm_q4(m, xs[k], stream=s)
            s.synchronize()
            if not torch.equal(y, want[k]):
                bad.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_experts_with_wild_offsets_stay_inside(wclib, cuda):
    """Offsets outside the matrices are clamped: no row outside x and y is touched."""
    rng, m, Ws = experts_case(wclib, cuda, 3, 64, 256, 64, False, False, 5)
    big = torch.full((64, 64), 7.0, device=cuda)
    x, xd = acts(rng, 20, 256, False, cuda)
    for off in ([-5, 4, 10, 1000], [0, 2**31 - 1, 3, 7], [9, 3, -2**31, 12]):
        big.fill_(7.0)
        y = big[20:40]
        wclib.gemm_q4_experts(m, x, dev(np.array(off, np.int32), cuda), y=y)
        assert (big[:20] == 7).all() and (big[40:] == 7).all()
        torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [2, 40])
def test_corrupt_headers_are_reported(wclib, cuda, tokens):
    rng = np.random.default_rng(9)
    m, _ = matrix(wclib, rng, 40, 256, 64, True, False, cuda)
    x, _ = acts(rng, tokens, 256, False, cuda)
    for at in (0, 8, 12, 16, 72, 88, 100):
        bad = m.buffer.clone()
        bad[at] ^= 1
        b = wclib.Q4Matrix(bad, 40, 256, 64, True, torch.bfloat16)
        for f in (lambda s: wclib.gemm_q4(b, x, status=s), lambda s: wclib.dequantize_q4(b, status=s),
                  lambda s: wclib.gemm_q4_experts(
                      wclib.Q4Matrix(bad[None], 40, 256, 64, True, torch.bfloat16), x,
                      torch.tensor([0, tokens], dtype=torch.int32, device=cuda), status=s)):
            s = torch.zeros(1, dtype=torch.int32, device=cuda)
            f(s)
            assert s.item() == wclib.WC_ERR_CORRUPT_STREAM, at
    short = wclib.Q4Matrix(m.buffer[:-16], 40, 256, 64, True, torch.bfloat16)
    with pytest.raises(wclib.WcodecError):
        wclib.gemm_q4(short, x)
    # random bytes as records: any result, nothing outside the buffers, the device usable
    noise = m.buffer.clone()
    noise[128:] = torch.randint(0, 256, (noise.numel() - 128,), device=cuda, dtype=torch.uint8)
    wclib.gemm_q4(wclib.Q4Matrix(noise, 40, 256, 64, True, torch.bfloat16), x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [1, 24, 200])
def test_products_in_a_graph_and_on_streams(wclib, cuda, tokens):
    """Captured and replayed on new inputs; two calls at once on two streams."""
    rng = np.random.default_rng(tokens)
    m, W = matrix(wclib, rng, 512, 1024, 128, False, False, cuda)
    x, _ = acts(rng, tokens, 1024, False, cuda)
    y = torch.empty((tokens, 512), device=cuda)
    side = torch.cuda.Stream()
    wclib.gemm_q4(m, x, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wclib.gemm_q4(m, x, y=y)
    for k in range(3):
        xn, xd = acts(rng, tokens, 1024, False, cuda)
        x.copy_(xn)
        graph.replay()
        x2, xd2 = acts(rng, tokens, 1024, False, cuda)
        side.wait_stream(torch.cuda.current_stream())
        y2 = wclib.gemm_q4(m, x2, stream=side)
        torch.cuda.synchronize()
        check(y, W, xd, 128, 1024)
        check(y2, W, xd2, 128, 1024)


def test_empty_products(wclib, cuda):
    rng = np.random.default_rng(3)
    m, _ = matrix(wclib, rng, 20, 64, 32, False, False, cuda)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device=cuda)
    assert wclib.gemm_q4(m, x).shape == (0, 20)
    e = wclib.quantize_q4(torch.zeros((0, 64), dtype=torch.bfloat16, device=cuda), 64)
    assert e.buffer.numel() == 128 and wclib.dequantize_q4(e).shape == (0, 64)
    assert wclib.wc_stream_info(bytes(e.buffer.cpu().numpy()))[0] == 0
    assert wclib.gemm_q4(e, torch.zeros((3, 64), dtype=torch.bfloat16, device=cuda)).shape == (3, 0)


def test_quantized_layer_matches_its_dequantized_weights(wclib, cuda):
    """Quantize, expand and multiply together on a full projection: the product
    is that of the expanded weights."""
    from lossless_weight_compression_b200 import synth
    w = synth.gaussian_bf16((4096, 4096), 0.02, 3, cuda)
    for group, zeros in ((128, False), (32, True)):
        m = wclib.quantize_q4(w, group, zeros=zeros)
        W = wclib.dequantize_q4(m, torch.float32).double()
        step = (w.double().view(4096, -1, group).abs().amax(2) / (7.5 if zeros else 7)).repeat_interleave(group, 1)
        # half a step, and what rounding the scale to BF16 (2^-8) moves the 8 or 15 codes by
        assert ((w.double() - W).abs() <= step * (0.5 + 16 * 2.0 ** -8) + 1e-12).all()
        for tokens in (1, 64):
            x = torch.randn((tokens, 4096), device=cuda).to(torch.bfloat16)
            ref, absum = x.double() @ W.T, x.double().abs() @ W.abs().T
            y = wclib.gemm_q4(m, x)
            assert ((y.double() - ref).abs() <= (group + 4096 // group + 64) * 2.0 ** -22 * absum).all()


def plain_quantize_fp32_ranges(w, group, zeros, dtype):
    """plain_quantize with a group's range and the range's quotient in FP32, as
    the definition has them (w float64 of finite values): a range of both signs
    may be rounded there, or be infinite."""
    rows, cols = w.shape
    g = q4_plain.groups_of(cols, group)
    S, Z, Q = np.zeros((rows, g)), np.zeros((rows, g)), np.zeros((rows, cols))
    for k in range(g):
        p = w[:, k * group:(k + 1) * group]
        lo, hi = np.minimum(p.min(1), 0), np.maximum(p.max(1), 0)
        with np.errstate(over="ignore"):
            span = hi.astype(np.float32) - lo.astype(np.float32) if zeros else np.maximum(hi, -lo).astype(np.float32)
            s = torch.from_numpy(span / np.float32(15 if zeros else 7)).to(dtype).double().numpy()
        d = np.where(s > 0, s, 1)
        z = np.clip(np.rint(-lo / d), 0, 15) if zeros else np.full(rows, 8.0)
        z = np.where(s > 0, z, 0.0 if zeros else 8.0)
        q = np.clip(np.rint(p / d[:, None]) + z[:, None], 0, 15)
        S[:, k], Z[:, k] = s, z
        Q[:, k * group:(k + 1) * group] = np.where(s[:, None] > 0, q, z[:, None])
    bits = torch.from_numpy(S).to(dtype).view(torch.int16).numpy().view(np.uint16)
    return Q.astype(np.uint8), bits, Z.astype(np.uint8) if zeros else None


# Largest magnitudes of a row's groups: the largest finite values, scales on both sides of 1e30 and
# 1e-30 (where the kernel changes its way to a quotient), subnormal scales, scales that round to 0.
MAGNITUDES = {
    False: [3.39e38, 3.2e38, 3.0e38, 2.99e38, 1e37, 1.6e31, 7.1e30, 6.9e30, 1e30, 7.1e-30, 6.9e-30, 1e-32, 8e-38,
            1e-38, 1e-39, 9e-41, 3e-40],
    True: [65504.0, 65000.0, 30.0, 1e-4, 6e-5, 4e-5, 3e-6, 5e-7, 2e-7, 6e-8],
}


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("group", [32, 128])
def test_quantize_over_the_whole_range_of_the_type(wclib, cuda, group, half, zeros):
    """Groups whose scale is among the type's largest or smallest, of both signs
    and of one, byte for byte; half steps among the values (ties to even)."""
    rng = np.random.default_rng(group + half)
    cols = 300
    rows = []
    for mag in MAGNITUDES[half]:
        for kind in range(4):
            u = rng.uniform(-1, 1, cols)
            if kind == 1:
                u = np.abs(u)
            elif kind == 2:
                u = -np.abs(u)
            elif kind == 3:  # halves of a fourteenth (of a thirtieth) of the range
                u = rng.integers(-14, 15, cols) / (30 if zeros else 14)
            u[::group] = -1.0 if kind == 2 else 1.0  # each group's largest magnitude
            if kind == 0:
                u[1::group] = -0.5
            rows.append(u * mag)
    w = torch.from_numpy(np.stack(rows)).float().to(DT[half])
    assert w.isfinite().all()
    q, s, z = plain_quantize_fp32_ranges(w.double().numpy(), group, zeros, DT[half])
    got = wclib.quantize_q4(w.to(cuda), group, zeros=zeros).buffer.cpu().numpy()
    assert np.array_equal(got, q4_plain.stream(q, s, z, group, half))


def test_quantize_finite_weights_whose_range_is_infinite(wclib, cuda):
    """With zero points a range of both signs can pass FP32: the scale is then
    infinite, as the definition's FP32 range is. Without them it cannot."""
    w = torch.full((16, 128), 3e38, dtype=torch.bfloat16)
    w[:, ::2] = -3e38
    for zeros in (False, True):
        q, s, z = plain_quantize_fp32_ranges(w.double().numpy(), 128, zeros, torch.bfloat16)
        got = wclib.quantize_q4(w.to(cuda), 128, zeros=zeros).buffer.cpu().numpy()
        assert np.array_equal(got, q4_plain.stream(q, s, z, 128, False))
        assert np.isinf(q4_plain.scale_values(s, False)).all() == zeros


def test_streams_of_experts_in_a_wider_buffer(wclib, cuda):
    """Streams that lie apart in a buffer of more columns, and one expert's with
    a few bytes behind it: the same bits as from a stack of their own."""
    rng, m, Ws = experts_case(wclib, cuda, 3, 64, 256, 64, False, False, 8)
    size = wclib.wc_q4_bytes(64, 256, 64, 0)
    own = m.buffer[:, :size].contiguous()
    wide = torch.zeros((3, size + 96), dtype=torch.uint8, device=cuda)
    wide[:, 32:32 + size] = own
    off = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device=cuda)
    x, xd = acts(rng, 12, 256, False, cuda)

    def call(b, o):
        return wclib.gemm_q4_experts(wclib.Q4Matrix(b, 64, 256, 64, False, torch.bfloat16), x[:int(o[-1])], o)
    y = call(own, off)
    check(y[:5], Ws[0], xd[:5], 64, 256)
    check(y[5:], Ws[2], xd[5:], 64, 256)
    assert torch.equal(call(wide[:, 32:32 + size], off), y)
    assert torch.equal(call(wide[:, 32:], off), y)
    assert torch.equal(call(wide[:1, 32:32 + size + 8], off[:2]), y[:5])


@pytest.mark.parametrize("tokens", [12, 20])
def test_ranges_of_wild_offsets(wclib, cuda, tokens):
    """Offsets outside the matrices and out of order, in the product of few rows
    (12 of 3 experts) and in the other (20): the clamped ranges hold their
    expert's product, every other row of y stays as it was."""
    rng, m, Ws = experts_case(wclib, cuda, 3, 64, 256, 64, False, False, 5)
    x, xd = acts(rng, tokens, 256, False, cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    for off in ([-5, 4, 10, 1000], [9, 3, -2**31, 7], [2**31 - 1, 0, 3, -4], [3, 5, 5, 2**31 - 1],
                [-2**31, -1, 0, 1], [tokens, tokens + 1, 2, 9]):
        y = torch.full((tokens + 8, 64), 7.0, device=cuda)
        wclib.gemm_q4_experts(m, x, dev(np.array(off, np.int32), cuda), y=y[4:tokens + 4], status=status)
        left = torch.ones(tokens + 8, dtype=torch.bool, device=cuda)
        for e in range(3):
            a = min(max(off[e], 0), tokens)
            b = min(max(off[e + 1], a), tokens)
            if b > a:
                check(y[4 + a:4 + b], Ws[e], xd[a:b], 64, 256)
                left[4 + a:4 + b] = False
        assert (y[left] == 7).all()
    assert status.item() == 0
