"""Rows sorted by expert and back, and the gradients, on the GPU against plain
64-bit forms.

Plans and copies: exactly. Sums of k products in FP32, one FMA each, are off by
at most k 2^-24 of the sum of magnitudes, and the result's rounding by half a
step of its type; a gradient weight[t, j] * dout[t] by an FP32 rounding and half
a step of its type.
"""
import numpy as np
import pytest
import torch

import q4_plain

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half a step below the smallest normal value, where steps no longer shrink
    with the value: they all are smallest_normal * eps (FP16: 2^-14 2^-10), so a
    rounding is off by half of that however small the value is."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def route(rng, tokens, top, experts, drop):
    ids = np.stack([rng.choice(experts, top, replace=top > experts) for _ in range(tokens)]) if tokens \
        else np.zeros((0, top))
    ids = ids.astype(np.int32).reshape(tokens, top)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def plan_of(wc, ids, experts, device):
    return wc.moe_sort(torch.from_numpy(ids).to(device), experts)


@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 1), (0, 2, 4), (33, 2, 8), (700, 8, 64),
                                                (3, 5, 1024), (5000, 3, 257), (20000, 6, 60),
                                                (4096, 1, 2), (4097, 1, 3)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_sort(wclib, cuda, tokens, top, experts, drop):
    rng = np.random.default_rng(tokens + experts)
    ids = rng.integers(0, experts, (tokens, top)).astype(np.int32)
    ids[rng.random(ids.shape) < drop / 2] = -1
    ids[rng.random(ids.shape) < drop / 2] = experts
    if drop == 1.0:
        ids[:] = np.where(ids % 2 == 0, -2**31, 2**31 - 1)
    plan = plan_of(wclib, ids, experts, cuda)
    offsets, order, inverse = q4_plain.sort(ids, experts)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.inverse.cpu().numpy(), inverse)
    assert np.array_equal(plan.order.cpu().numpy(), order)


def test_sort_of_one_expert_and_many_slots(wclib, cuda):
    """Every slot to one expert (the longest chain of ranks), and 2^20 slots."""
    ids = torch.full((3000, 4), 7, dtype=torch.int32, device=cuda)
    plan = wclib.moe_sort(ids, 9)
    assert plan.offsets.tolist() == [0] * 8 + [12000] * 2
    assert torch.equal(plan.inverse.view(-1), torch.arange(12000, dtype=torch.int32, device=cuda))
    ids = torch.randint(-1, 200, (2**17, 8), device=cuda).to(torch.int32)
    plan = wclib.moe_sort(ids, 200)
    key = torch.where(ids.view(-1) < 0, 200, ids.view(-1))
    want = torch.argsort(key, stable=True)
    n = int((ids >= 0).sum())
    assert int(plan.offsets[-1]) == n
    assert torch.equal(plan.order[:n].long(), want[:n]) and (plan.order[n:] == -1).all()
    assert torch.equal(plan.inverse.view(-1)[want[:n]].long(), torch.arange(n, device=cuda))
    assert torch.equal(plan.offsets[:-1].long(), torch.searchsorted(key[want], torch.arange(200, device=cuda)))


CASES = [(1, 1, 1, 1, 0.0), (0, 2, 4, 8, 0.0), (33, 2, 8, 2050, 0.2), (70, 8, 64, 4096, 0.1),
         (500, 6, 16, 129, 0.5), (9, 3, 5, 96, 1.0), (40, 20, 32, 515, 0.1), (300, 1, 3, 7168, 0.0)]


def both_ways(wc, rng, device, tokens, top, experts, cols, drop, dt):
    ids = route(rng, tokens, top, experts, drop)
    plan = plan_of(wc, ids, experts, device)
    x = torch.from_numpy(rng.standard_normal((tokens, cols))).to(dt)
    return ids, plan, x


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,top,experts,cols,drop", CASES)
def test_gather_and_its_gradient(wclib, cuda, tokens, top, experts, cols, drop, dt):
    rng = np.random.default_rng(tokens * 3 + cols)
    ids, plan, x = both_ways(wclib, rng, cuda, tokens, top, experts, cols, drop, dt)
    offsets, order, inverse = q4_plain.sort(ids, experts)
    n = offsets[-1]
    out = torch.full((tokens * top + 2, cols), 7.0, dtype=dt, device=cuda)
    wclib.moe_gather(x.to(cuda), plan, out=out)
    assert torch.equal(out[:n].cpu(), x[order[:n] // top])
    assert (out[n:] == 7).all()  # rows behind the last expert's stay
    drows = torch.from_numpy(rng.standard_normal((tokens * top, cols))).to(dt)
    drows[n:] = float("nan")
    dx = wclib.moe_gather_backward(drows.to(cuda), plan).double().cpu()
    ref, mag = torch.zeros((tokens, cols), dtype=torch.float64), torch.zeros((tokens, cols), dtype=torch.float64)
    ref.index_add_(0, torch.from_numpy(order[:n] // top).long(), drows[:n].double())
    mag.index_add_(0, torch.from_numpy(order[:n] // top).long(), drows[:n].double().abs())
    assert ((dx - ref).abs() <= top * 2.0 ** -24 * mag * 2 + half_step(dt) * ref.abs() + tiny(dt)).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,top,experts,cols,drop", CASES)
def test_combine_and_its_gradients(wclib, cuda, tokens, top, experts, cols, drop, dt):
    rng = np.random.default_rng(tokens * 5 + cols)
    ids, plan, dout = both_ways(wclib, rng, cuda, tokens, top, experts, cols, drop, dt)
    _, order, inverse = q4_plain.sort(ids, experts)
    n = int((inverse >= 0).sum())
    rows = torch.from_numpy(rng.standard_normal((tokens * top, cols))).to(dt)
    rows[n:] = float("nan")
    w = torch.from_numpy(rng.random((tokens, top))).float()
    out = wclib.moe_combine(rows.to(cuda), plan, w.to(cuda)).double().cpu()
    kept = torch.from_numpy(inverse >= 0)
    at = torch.from_numpy(inverse).long().clamp(min=0)
    picked = torch.where(kept[..., None], rows.double()[at] if tokens else torch.zeros((0, top, cols)).double(),
                         torch.zeros((), dtype=torch.float64))
    term = picked * w.double()[..., None]
    ref, mag = term.sum(1), term.abs().sum(1)
    assert ((out - ref).abs() <= top * 2.0 ** -23 * mag + half_step(dt) * ref.abs() + tiny(dt)).all()
    drows = torch.full((tokens * top, cols), 7.0, dtype=dt, device=cuda)
    d2, dw = wclib.moe_combine_backward(dout.to(cuda), rows.to(cuda), plan, w.to(cuda), drows=drows)
    assert d2 is drows and (drows[n:] == 7).all()
    slot = torch.from_numpy(order[:n]).long()
    want = w.view(-1).double()[slot][:, None] * dout.double()[slot // top]
    got = drows[:n].double().cpu()
    assert ((got - want).abs() <= (half_step(dt) + 2.0 ** -23) * want.abs() + tiny(dt)).all()
    prod = picked * dout.double()[:, None, :]
    dref, dmag = prod.sum(2), prod.abs().sum(2)
    dw = dw.double().cpu()
    assert ((dw - dref).abs() <= (cols + 16) * 2.0 ** -24 * dmag).all()
    assert (dw[~kept] == 0).all()
    again, dw2 = wclib.moe_combine_backward(dout.to(cuda), rows.to(cuda), plan, w.to(cuda))
    assert torch.equal(dw2.double().cpu(), dw) and torch.equal(again[:n], drows[:n])


def test_gradients_against_differences(wclib, cuda):
    """combine and gather are linear in each input: the difference of two calls
    is the gradient's product with the step, up to the FP32 sums' roundings."""
    rng = np.random.default_rng(11)
    tokens, top, experts, cols = 40, 3, 6, 200
    ids, plan, dout = both_ways(wclib, rng, cuda, tokens, top, experts, cols, 0.1, torch.float32)
    dout = dout.to(cuda)
    n = int(plan.offsets[-1])

    def rnd(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).float().to(cuda)
    rows, w, step, wstep = rnd(tokens * top, cols), rnd(tokens, top), rnd(tokens * top, cols), rnd(tokens, top)
    drows, dw = wclib.moe_combine_backward(dout, rows, plan, w, drows=torch.zeros_like(rows))

    def loss(r, ww):
        return (wclib.moe_combine(r, plan, ww).double() * dout.double()).sum()
    size = tokens * cols * top * 2.0 ** -24 * 64  # terms of size up to about 64
    for r2, w2, slope in ((rows + step, w, (drows.double() * (rows + step).double().sub(rows.double())).sum()),
                          (rows, w + wstep, (dw.double() * (w + wstep).double().sub(w.double())).sum())):
        assert abs(float(loss(r2, w2) - loss(rows, w) - slope)) <= size
    x, xs = rnd(tokens, cols), rnd(tokens, cols)
    g = rnd(tokens * top, cols)
    dx = wclib.moe_gather_backward(g, plan)

    def lg(v):
        return (wclib.moe_gather(v, plan).double()[:n] * g.double()[:n]).sum()
    slope = (dx.double() * (x + xs).double().sub(x.double())).sum()
    assert abs(float(lg(x + xs) - lg(x) - slope)) <= size


def test_strided_rows_and_null_weights(wclib, cuda):
    rng = np.random.default_rng(12)
    tokens, top, experts, cols = 50, 2, 4, 136
    ids, plan, x = both_ways(wclib, rng, cuda, tokens, top, experts, cols, 0.0, torch.bfloat16)
    x = x.to(cuda)
    for pad, at in ((8, 0), (24, 8), (5, 1), (2, 2)):
        xs = torch.zeros((tokens, cols + pad), dtype=x.dtype, device=cuda)
        xs[:, at:at + cols] = x
        big = torch.full((tokens * top, cols + pad), 7.0, dtype=x.dtype, device=cuda)
        rows = big[:, at:at + cols]
        wclib.moe_gather(xs[:, at:at + cols], plan, out=rows)
        assert torch.equal(rows, x[(plan.order // top).long()])
        assert (big[:, :at] == 7).all() and (big[:, at + cols:] == 7).all()
        ob = torch.full((tokens, cols + pad), 7.0, dtype=x.dtype, device=cuda)
        wclib.moe_combine(rows, plan, None, out=ob[:, at:at + cols])
        assert torch.equal(ob[:, at:at + cols], x * 2)
        db = torch.full_like(big, 7.0)
        _, dw = wclib.moe_combine_backward(xs[:, at:at + cols], rows, plan, None, drows=db[:, at:at + cols])
        assert torch.equal(db[:, at:at + cols], rows)
        assert (db[:, :at] == 7).all() and (db[:, at + cols:] == 7).all()
        ref = x.double().square().sum(1, keepdim=True).expand(tokens, top)
        assert ((dw.double() - ref).abs() <= (cols + 16) * 2.0 ** -24 * ref).all()


def test_wild_inverse_names_no_row(wclib, cuda):
    """Values outside the sorted rows mean that a slot has none."""
    inv = torch.tensor([[0, 99], [-7, 2**31 - 1]], dtype=torch.int32, device=cuda)
    plan = wclib.MoePlan(torch.tensor([0, 1], dtype=torch.int32, device=cuda), None, inv)
    x = torch.ones((2, 64), device=cuda)
    out = wclib.moe_gather(x, plan, out=torch.zeros((4, 64), device=cuda))
    assert out[0].eq(1).all() and out[1:].eq(0).all()
    y = wclib.moe_combine(out + 1, plan, torch.full((2, 2), 3.0, device=cuda))
    assert y[0].eq(6).all() and y[1].eq(0).all()
    _, dw = wclib.moe_combine_backward(x, out + 1, plan, None)
    assert dw.tolist() == [[128.0, 0.0], [0.0, 0.0]]


def test_rows_past_32_bits(wclib, cuda):
    """Sorted rows of more than 2^32 elements: copied, summed and their gradients."""
    tokens, top, cols = 140000, 4, 8192
    ids = torch.randint(0, 64, (tokens, top), device=cuda).to(torch.int32)
    plan = wclib.moe_sort(ids, 64)
    x = torch.randn((tokens, cols), device=cuda, dtype=torch.bfloat16)
    rows = wclib.moe_gather(x, plan)
    for a in (0, tokens * top - 500):
        assert torch.equal(rows[a:a + 500], x[(plan.order[a:a + 500] // top).long()])
    out = wclib.moe_combine(rows, plan, None)
    assert torch.equal(out, x * 4)  # four equal terms: exact
    del out
    w = torch.full((tokens, top), 2.0, device=cuda)
    drows, dw = wclib.moe_combine_backward(x, rows, plan, w)
    assert torch.equal(drows[-500:], rows[-500:] * 2) and torch.equal(drows[:500], rows[:500] * 2)
    ref = x[-50:].double().square().sum(1, keepdim=True).expand(50, top)
    assert ((dw[-50:].double() - ref).abs() <= (cols + 16) * 2.0 ** -24 * ref).all()
    del rows, drows
    torch.cuda.empty_cache()


def quantized_experts(wc, E, rows, cols, group, device, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    ms = [wc.quantize_q4((torch.randn((rows, cols), generator=g) * 0.05).to(device, torch.bfloat16), group)
          for _ in range(E)]
    stack = wc.Q4Matrix(torch.stack([m.buffer for m in ms]), rows, cols, group, False, torch.bfloat16)
    return stack, torch.stack([wc.dequantize_q4(m, torch.float32) for m in ms]).double()


@pytest.mark.parametrize("tokens,top,E", [(1, 2, 8), (9, 3, 16), (200, 2, 4)])
def test_a_layer_of_experts(wclib, cuda, tokens, top, E):
    """Sort, gather, up and down products and combine, as a layer runs them;
    every step checked against 64 bits on the step's own inputs, then the whole
    captured in a graph and replayed on new tokens."""
    d, f, group = 256, 384, 64
    up, Wu = quantized_experts(wclib, E, f, d, group, cuda, 1)
    down, Wd = quantized_experts(wclib, E, d, f, group, cuda, 2)
    x = torch.empty((tokens, d), dtype=torch.bfloat16, device=cuda)
    ids = torch.empty((tokens, top), dtype=torch.int32, device=cuda)
    w = torch.empty((tokens, top), device=cuda)

    def draw(seed):
        g = torch.Generator(device="cpu").manual_seed(seed)
        x.copy_(torch.randn((tokens, d), generator=g))
        score = torch.randn((tokens, E), generator=g)
        ids.copy_(score.topk(top, 1).indices)
        ids[0, 0] = -1  # dropped
        w.copy_(torch.rand((tokens, top), generator=g))

    def layer():
        plan = wclib.moe_sort(ids, E)
        rows = wclib.moe_gather(x, plan, out=torch.zeros((tokens * top, d), dtype=x.dtype, device=cuda))
        h = wclib.gemm_q4_experts(up, rows, plan.offsets, out_dtype=x.dtype)
        a = torch.relu(h)
        o = wclib.gemm_q4_experts(down, a, plan.offsets, out_dtype=x.dtype)
        return plan, rows, h, a, o, wclib.moe_combine(o, plan, w)

    def check(plan, rows, h, a, o, y):
        n = int(plan.offsets[-1])
        e = torch.bucketize(torch.arange(n, device=cuda), plan.offsets[1:].long(), right=True)
        assert torch.equal(rows[:n], x[(plan.order[:n] // top).long()])
        assert torch.equal(ids.view(-1)[plan.order[:n].long()].long(), e)
        for xin, yout, W in ((rows, h, Wu), (a, o, Wd)):
            k = W.shape[2]
            for q in range(E):
                m = (e == q).nonzero()[:, 0]
                if not len(m):
                    continue
                ref = xin[m].double() @ W[q].T
                mag = xin[m].double().abs() @ W[q].abs().T
                tol = (group + k // group + 64) * 2.0 ** -22 * mag
                assert ((yout[m].double() - ref).abs() <= tol + half_step(x.dtype) * (ref.abs() + tol)).all()
        kept = plan.inverse >= 0
        term = torch.where(kept[..., None], o.double()[plan.inverse.clamp(min=0).long()], 0) * w.double()[..., None]
        ref = term.sum(1)
        assert ((y.double() - ref).abs() <= top * 2.0 ** -23 * term.abs().sum(1) + half_step(x.dtype) * ref.abs()).all()

    draw(0)
    check(*layer())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = layer()
    for seed in (1, 2):
        draw(seed)
        graph.replay()
        torch.cuda.synchronize()
        check(*res)


def test_sorted_rows_feed_the_products_of_streams(wclib, orc, cuda):
    """The sorted rows of each expert through wc_gemm on that expert's BF16
    stream (plain and escape-coded weights read losslessly), and back."""
    from lossless_weight_compression_b200 import synth
    tokens, top, E, d, f, B = 60, 2, 4, 256, 130, 256
    rng = np.random.default_rng(21)
    ids = route(rng, tokens, top, E, 0.1)
    plan = plan_of(wclib, ids, E, cuda)
    x = torch.from_numpy(rng.standard_normal((tokens, d))).to(cuda, torch.bfloat16)
    rows = wclib.moe_gather(x, plan)
    Ws = [synth.gaussian_bf16((f, d), 0.02, 40 + e, cuda) for e in range(E)]
    y = torch.zeros((tokens * top, f), device=cuda)
    off = plan.offsets.tolist()
    for e in range(E):
        if off[e + 1] > off[e]:
            wclib.gemm(wclib.compress(Ws[e], B).buffer, f, d, B, rows[off[e]:off[e + 1]],
                       y=y[off[e]:off[e + 1]])
    w = torch.from_numpy(rng.random((tokens, top))).float().to(cuda)
    out = wclib.moe_combine(y, plan, w).double()
    ref, mag = torch.zeros_like(out), torch.zeros_like(out)
    for t in range(tokens):
        for j in range(top):
            if ids[t, j] >= 0:
                W = Ws[ids[t, j]].double()
                ref[t] += float(w[t, j]) * (W @ x[t].double())
                mag[t] += float(w[t, j]) * (W.abs() @ x[t].double().abs())
    assert ((out - ref).abs() <= (d * 2.0 ** -22 + top * 2.0 ** -23 + 2.0 ** -24) * mag).all()


def test_gradients_through_a_layer_whose_products_have_gradients(wclib, cuda):
    """Gather and combine with their gradients inside autograd functions of the
    caller's, around torch products of each expert's rows: the layer's gradients
    against those of the same layer in 64 bits. All values are small integers
    and quarters, so that every sum is exact in FP32 and the results are equal."""
    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, plan):
            ctx.plan = plan
            return wclib.moe_gather(x, plan, out=x.new_zeros((plan.inverse.numel(), x.shape[1])))

        @staticmethod
        def backward(ctx, drows):
            return wclib.moe_gather_backward(drows, ctx.plan), None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, w, plan):
            ctx.plan = plan
            ctx.save_for_backward(rows, w)
            return wclib.moe_combine(rows, plan, w)

        @staticmethod
        def backward(ctx, dout):
            rows, w = ctx.saved_tensors
            return (*wclib.moe_combine_backward(dout, rows, ctx.plan, w, drows=torch.zeros_like(rows)), None)

    rng = np.random.default_rng(31)
    tokens, top, E, d, f = 45, 3, 5, 40, 24
    ids = route(rng, tokens, top, E, 0.2)
    plan = plan_of(wclib, ids, E, cuda)
    off = plan.offsets.tolist()

    def ints(*shape):
        return torch.from_numpy(rng.integers(-3, 4, shape)).float().to(cuda)
    x, W, w, dout = ints(tokens, d), ints(E, f, d), ints(tokens, top) / 4, ints(tokens, f)
    a = [t.clone().requires_grad_() for t in (x, W, w)]
    rows = Gather.apply(a[0], plan)
    prod = torch.cat([rows[off[e]:off[e + 1]] @ a[1][e].T for e in range(E)] + [rows.new_zeros((len(rows) - off[-1], f))])
    out = Combine.apply(prod, a[2], plan)
    out.backward(dout)
    b = [t.double().requires_grad_() for t in (x, W, w)]
    kept = torch.from_numpy(ids >= 0).to(cuda)
    every = torch.einsum("td,efd->tef", b[0], b[1])
    picked = every[torch.arange(tokens, device=cuda)[:, None], torch.from_numpy(ids).to(cuda).clamp(min=0).long()]
    ref = (picked * (b[2] * kept)[..., None]).sum(1)
    ref.backward(dout.double())
    assert torch.equal(out.double(), ref)
    for got, want in zip(a, b):
        assert torch.equal(got.grad.double(), want.grad)
