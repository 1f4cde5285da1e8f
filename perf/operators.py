"""The 4-bit products and the expert routing operators: what is measured, and their plain forms.

Operators (each case's "op"):
  product   y = x W^T with W held as a 4-bit stream with group scales
  experts   the same for rows sorted by expert, each range with its expert's matrix
  dispatch  tokens sorted by expert: the plan and the gathered rows ("train": and the gradient of the rows)
  combine   rows brought back to their tokens with weights applied ("train": and both gradients)
  quantize  a 16-bit matrix to a 4-bit stream and the stream back to 16-bit values

A 4-bit stream is 128 header bytes and records of 16 rows x 128 columns (rows and columns padded).
A record: 1024 bytes of codes, [t 0..3][row 0..15][i 0..3] 32-bit words, word (t, i) holding columns
32 i + 8 t + (0..7), element e at nibble (e >> 1) + 4 (e & 1); then the scales [128 / group][16 rows] as
16-bit values; then, with zero points, [128 / group][16 rows] bytes, padded to 32. Records are ordered
[128-row block][128-column slice][16-row block within the 128 rows].
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token through an attention projection: the latency of single-stream decoding
        dict(name="product-1x4096x4096", op="product", tokens=1, rows=4096, cols=4096, group=128, zeros=False, x="bf16",
             scales="bf16", y="same"),
        # a small batch on a ragged matrix: rows and columns that fill no tile, rows of x off 16-byte boundaries
        dict(name="product-13x1027x4100", op="product", tokens=13, rows=1027, cols=4100, group=32, zeros=True, x="fp16",
             scales="fp16", y="fp32"),
        # a decoding batch through an up projection
        dict(name="product-64x14336x4096", op="product", tokens=64, rows=14336, cols=4096, group=128, zeros=False, x="bf16",
             scales="bf16", y="same"),
        # a prefill chunk through a down projection
        dict(name="product-512x4096x14336", op="product", tokens=512, rows=4096, cols=14336, group=64, zeros=True, x="bf16",
             scales="fp16", y="same"),
        # a few decoding tokens over many small experts: most experts have no row or one
        dict(name="experts-48of64", op="experts", tokens=8, top=6, experts=64, rows=2048, cols=1024, group=64, zeros=False,
             x="bf16", scales="bf16", y="same"),
        # a prefill chunk over few large experts, unevenly loaded
        dict(name="experts-2000of8", op="experts", tokens=1000, top=2, experts=8, rows=14336, cols=4096, group=128, zeros=True,
             x="bf16", scales="bf16", y="same"),
        # a decoding batch to few experts
        dict(name="dispatch-32", op="dispatch", tokens=32, top=2, experts=8, cols=4096, dtype="bf16", train=False, drop=0.0),
        # a training batch to many experts, some slots over capacity
        dict(name="dispatch-16384-train", op="dispatch", tokens=16384, top=6, experts=64, cols=2048, dtype="bf16", train=True,
             drop=0.05),
        # a decoding batch back from many experts, an odd row length
        dict(name="combine-33", op="combine", tokens=33, top=8, experts=64, cols=2050, dtype="fp16", train=False, drop=0.1),
        # a training batch back from few experts
        dict(name="combine-8192-train", op="combine", tokens=8192, top=2, experts=8, cols=4096, dtype="bf16", train=True,
             drop=0.0),
        # a ragged matrix with zero points
        dict(name="quantize-1000x4100", op="quantize", rows=1000, cols=4100, group=32, zeros=True, dtype="fp16"),
        # an up projection
        dict(name="quantize-14336x4096", op="quantize", rows=14336, cols=4096, group=128, zeros=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "experts", "dispatch", "combine", "quantize"])
    group, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "product":
        while True:
            c = dict(op=op, tokens=_spread(rng, 1, 512), rows=_spread(rng, 16, 16384), cols=_spread(rng, 64, 16384), group=group,
                     zeros=zeros, x=rng.choice(["bf16", "fp16"]), scales=rng.choice(["bf16", "fp16"]), y=rng.choice(["same", "fp32"]))
            if 2**19 <= c["rows"] * c["cols"] <= 14336 * 4096:
                return c
    if op == "experts":
        while True:
            experts = _spread(rng, 2, 128)
            c = dict(op=op, tokens=_spread(rng, 1, 2048), top=rng.randint(1, min(8, experts)), experts=experts,
                     rows=_spread(rng, 64, 14336), cols=_spread(rng, 128, 4096), group=group, zeros=zeros,
                     x=rng.choice(["bf16", "fp16"]), scales=rng.choice(["bf16", "fp16"]), y=rng.choice(["same", "fp32"]))
            size = c["rows"] * c["cols"]
            if 2**20 <= experts * size <= 8 * 14336 * 4096 and c["tokens"] * c["top"] * size <= 2000 * 14336 * 4096:
                return c
    if op in ("dispatch", "combine"):
        while True:
            experts = _spread(rng, 2, 256)
            c = dict(op=op, tokens=_spread(rng, 1, 16384), top=rng.randint(1, min(8, experts)), experts=experts,
                     cols=_spread(rng, 64, 8192), dtype=rng.choice(["bf16", "fp16", "fp32"]), train=rng.random() < 0.5,
                     drop=rng.choice([0.0, 0.1]))
            if c["tokens"] * c["top"] * c["cols"] <= 16384 * 6 * 2048:
                return c
    while True:
        c = dict(op=op, rows=_spread(rng, 16, 16384), cols=_spread(rng, 64, 16384), group=group, zeros=zeros,
                 dtype=rng.choice(["bf16", "fp16"]))
        if 2**16 <= c["rows"] * c["cols"] <= 14336 * 4096:
            return c


def _stream_bytes(c):
    """What a stream cannot do without: codes, scales and zero points."""
    groups = -(-c["cols"] // c["group"])
    return c["rows"] * (-(-c["cols"] // 2) + groups * (3 if c["zeros"] else 2))


def work(c):
    op = c["op"]
    if op == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * (2 * n + _stream_bytes(c)), "flops": 0}
    if op in ("product", "experts"):
        n = c["tokens"] * c.get("top", 1)
        used = min(c.get("experts", 1), n)
        ysize = 4 if c["y"] == "fp32" else 2
        return {"bytes": used * _stream_bytes(c) + n * (2 * c["cols"] + ysize * c["rows"]), "flops": 2 * n * c["rows"] * c["cols"]}
    t, s, size = c["tokens"], c["tokens"] * c["top"], 4 if c["dtype"] == "fp32" else 2
    row = c["cols"] * size
    kept = int(s * (1 - c["drop"]))
    if op == "dispatch":
        b = 4 * s + (t + kept) * row + 8 * s + 4 * (c["experts"] + 1)
        return {"bytes": b + ((kept + t) * row + 4 * s if c["train"] else 0), "flops": kept * c["cols"] if c["train"] else 0}
    b = 8 * s + (t + kept) * row
    f = 2 * kept * c["cols"]
    # backward: dout and y are read, dy and dw written
    return {"bytes": b + ((t + 2 * kept) * row + 12 * s if c["train"] else 0), "flops": f + (3 * kept * c["cols"] if c["train"] else 0)}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _codes(c, seed, experts=1):
    """Codes (bell-shaped), group scales and zero points of `experts` matrices."""
    g = _gen(seed)
    groups = -(-c["cols"] // c["group"])
    shape = (experts, c["rows"], c["cols"])
    q = torch.randint(0, 6, shape, generator=g, device="cuda", dtype=torch.uint8)
    for _ in range(2):
        q += torch.randint(0, 6, shape, generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand((experts, c["rows"], groups), generator=g, device="cuda").add_(0.5).mul_(0.007).to(DT[c["scales"]])
    z = torch.randint(4, 12, (experts, c["rows"], groups), generator=g, device="cuda", dtype=torch.uint8) if c["zeros"] else None
    return q, s, z


def _pack(q, s, z, group):
    """Streams (experts, bytes) of codes (experts, rows, cols), scales and zero points (experts, rows, groups)."""
    E, rows, cols = q.shape
    R, S, per = -(-rows // 16), -(-cols // 128), 128 // group
    groups = s.shape[2]
    if z is None:
        full = torch.full((E, R * 16, S * 128), 8, dtype=torch.uint8, device=q.device)
    else:  # padding holds the code that stands for zero
        zf = torch.zeros((E, R * 16, S * per), dtype=torch.uint8, device=q.device)
        zf[:, :rows, :groups] = z
        full = zf.repeat_interleave(group, dim=2)
    full[:, :rows, :cols] = q
    sf = torch.zeros((E, R * 16, S * per), dtype=s.dtype, device=q.device)
    sf[:, :rows, :groups] = s
    # (E, R, row, S, i, t, k, half) -> (E, R, S, t, row, i, half, k): nibble 4 half + k holds element 2 k + half
    w = full.view(E, R, 16, S, 4, 4, 4, 2).permute(0, 1, 3, 5, 2, 4, 7, 6).reshape(E, R, S, 1024, 2)
    parts = [w[..., 0] | (w[..., 1] << 4)]
    parts.append(sf.view(E, R, 16, S, per).permute(0, 1, 3, 4, 2).contiguous().view(torch.uint8).view(E, R, S, 32 * per))
    if z is not None:
        zz = zf.view(E, R, 16, S, per).permute(0, 1, 3, 4, 2).reshape(E, R, S, 16 * per)
        parts.append(torch.nn.functional.pad(zz, (0, -(16 * per) % 32)))
    rec = torch.cat(parts, dim=3)
    nf = R // 8 * 8
    body = [rec[:, :nf].reshape(E, nf // 8, 8, S, -1).transpose(2, 3).reshape(E, -1)]
    if R > nf:
        body.append(rec[:, nf:].transpose(1, 2).reshape(E, -1))
    body = torch.cat(body, dim=1)
    n, total = rows * cols, 128 + body.shape[1]
    flags = 8 | (16 if z is not None else 0) | (32 if s.dtype == torch.float16 else 0)
    head = torch.zeros(128, dtype=torch.uint8)
    for at, size, v in ((0, 4, 0x31424357), (4, 2, 1), (6, 2, 128), (8, 4, group), (12, 4, flags), (16, 8, n), (24, 8, rows * groups),
                        (32, 8, 128), (64, 8, total - 128), (72, 8, total), (88, 4, rows), (92, 4, cols)):
        head[at:at + size] = torch.tensor(list(v.to_bytes(size, "little")), dtype=torch.uint8)
    return torch.cat([head.to(q.device).expand(E, 128), body], dim=1).contiguous()


def _route(c, seed):
    """Expert ids (uneven, some dropped as -1) and router weights of each token's slots."""
    g = _gen(seed + 1)
    score = torch.rand((c["tokens"], c["experts"]), generator=g, device="cuda").log_().neg_().log_().neg_()
    score += torch.linspace(1.0, -1.0, c["experts"], device="cuda")
    ids = score.topk(c["top"], dim=1).indices.to(torch.int32)
    if c.get("drop"):
        ids[torch.rand(ids.shape, generator=g, device="cuda") < c["drop"]] = -1
    weights = torch.rand(ids.shape, generator=g, device="cuda") + 0.1
    return ids, weights / weights.sum(1, keepdim=True)


def _plan(ids, experts):
    """The plan by a running count for each expert: offsets, order, inverse."""
    flat = ids.reshape(-1)
    hot = flat[:, None] == torch.arange(experts, device=flat.device, dtype=torch.int32)
    count = hot.cumsum(0, dtype=torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = count[-1].cumsum(0)
    valid = (flat >= 0) & (flat < experts)
    e = flat.clamp(0, experts - 1).long()
    pos = offsets[e] + count.gather(1, e[:, None])[:, 0] - 1
    inverse = torch.where(valid, pos, torch.full_like(pos, -1)).to(torch.int32)
    order = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device=flat.device)
    order[torch.where(valid, pos, torch.full_like(pos, flat.numel())).long()] = torch.arange(flat.numel(), dtype=torch.int32,
                                                                                             device=flat.device)
    return offsets, order[:-1].contiguous(), inverse.view(ids.shape)


def prepare(case, seed):
    c = dict(case)
    op, g = c["op"], _gen(seed + 2)
    if op == "product":
        q, s, z = _codes(c, seed)
        return dict(c, stream=_pack(q, s, z, c["group"])[0], data=_normal(g, (c["tokens"], c["cols"]), DT[c["x"]]))
    if op == "experts":
        q, s, z = _codes(c, seed, c["experts"])
        ids, _ = _route(c, seed)
        offsets, _, _ = _plan(ids, c["experts"])
        counts = offsets.diff()
        return dict(c, stream=_pack(q, s, z, c["group"]), offsets=offsets, most=int(counts.max()),
                    data=_normal(g, (ids.numel(), c["cols"]), DT[c["x"]]))
    if op == "quantize":
        std = torch.exp(torch.empty((c["rows"], 1), device="cuda").uniform_(-1.0, 1.0, generator=g)) * 0.02
        return dict(c, data=(torch.randn((c["rows"], c["cols"]), generator=g, device="cuda") * std).to(DT[c["dtype"]]))
    ids, weights = _route(c, seed)
    offsets, order, inverse = _plan(ids, c["experts"])
    dt, slots = DT[c["dtype"]], ids.numel()
    kept = (torch.arange(slots, device="cuda") < offsets[-1])[:, None]
    if op == "dispatch":  # rows behind the last expert's stay as they are
        return dict(c, ids=ids, data=_normal(g, (c["tokens"], c["cols"]), dt),
                    rows_out=torch.zeros((slots, c["cols"]), dtype=dt, device="cuda"),
                    drows=_normal(g, (slots, c["cols"]), dt) if c["train"] else None)
    return dict(c, weights=weights, offsets=offsets, order=order, inverse=inverse, data=_normal(g, (slots, c["cols"]), dt) * kept,
                dout=_normal(g, (c["tokens"], c["cols"]), dt) if c["train"] else None,
                drows_out=torch.zeros((slots, c["cols"]), dtype=dt, device="cuda") if c["train"] else None)


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _unpack(streams, c):
    """FP32 weights (experts, rows, cols) of streams (experts, bytes)."""
    E, rows, cols, group = streams.shape[0], c["rows"], c["cols"], c["group"]
    R, S, per = -(-rows // 16), -(-cols // 128), 128 // group
    size = 1024 + 32 * per + ((16 * per + 31) // 32 * 32 if c["zeros"] else 0)
    nf = R // 8 * 8
    cut = 128 + nf * S * size
    rec = streams[:, 128:cut].reshape(E, nf // 8, S, 8, size).transpose(2, 3).reshape(E, nf, S, size)
    if R > nf:
        rec = torch.cat([rec, streams[:, cut:cut + (R - nf) * S * size].reshape(E, S, R - nf, size).transpose(1, 2)], dim=1)
    codes = rec[..., :1024]
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).view(E, R, S, 4, 16, 4, 2, 4)
    q = nib.permute(0, 1, 4, 2, 5, 3, 7, 6).reshape(E, R * 16, S * 128)
    s = rec[..., 1024:1024 + 32 * per].contiguous().view(DT[c["scales"]]).view(E, R, S, per, 16).permute(0, 1, 4, 2, 3)
    s = s.reshape(E, R * 16, S * per, 1).float()
    if c["zeros"]:
        z = rec[..., 1024 + 32 * per:1024 + 48 * per].reshape(E, R, S, per, 16).permute(0, 1, 4, 2, 3).reshape(E, R * 16, S * per, 1)
        z = z.float()
    else:
        z = 8.0
    w = (q.view(E, R * 16, S * per, group).float() - z) * s
    return w.view(E, R * 16, S * 128)[:, :rows, :cols]


def _plain(st):
    op = st["op"]
    if op == "product":
        y = st["data"].float() @ _unpack(st["stream"][None], st)[0].T
        return y if st["y"] == "fp32" else y.to(DT[st["x"]])
    if op == "experts":  # each expert's rows in a padded batch
        x, off, E, most = st["data"], st["offsets"], st["experts"], st["most"]
        p = torch.arange(x.shape[0], device="cuda", dtype=torch.int32)
        e = (p[:, None] >= off[None, 1:]).sum(1)
        at = p.long() - off[e].long()
        xs = torch.zeros((E, most, st["cols"]), device="cuda")
        xs[e, at] = x.float()
        y = (xs @ _unpack(st["stream"], st).transpose(1, 2))[e, at]
        return y if st["y"] == "fp32" else y.to(x.dtype)
    if op == "quantize":
        w, G = st["data"].float(), st["group"]
        rows, cols = w.shape
        w = torch.nn.functional.pad(w, (0, -cols % G)).view(rows, -1, G)
        if st["zeros"]:
            lo, hi = w.amin(2, keepdim=True).clamp(max=0), w.amax(2, keepdim=True).clamp(min=0)
            s = ((hi - lo) / 15).to(DT[st["dtype"]]).float()
            d = torch.where(s > 0, s, torch.ones_like(s))
            z = torch.round(-lo / d).clamp(0, 15)
            q = (torch.round(w / d) + z).clamp(0, 15) - z
        else:
            s = (w.abs().amax(2, keepdim=True) / 7).to(DT[st["dtype"]]).float()
            q = torch.round(w / torch.where(s > 0, s, torch.ones_like(s))).clamp(-8, 7)
        return (q * s).view(rows, -1)[:, :cols].to(DT[st["dtype"]])
    if op == "dispatch":
        x, (offsets, order, inverse) = st["data"], _plan(st["ids"], st["experts"])
        kept = (torch.arange(order.numel(), device="cuda") < offsets[-1])[:, None]
        token = (order.clamp(min=0) // st["top"]).long()
        rows = torch.where(kept, x[token], st["rows_out"])
        out = dict(rows=rows, offsets=offsets, inverse=inverse)
        if st["train"]:
            d = st["drows"].float()[inverse.clamp(min=0).long()] * (inverse >= 0)[..., None]
            out["dx"] = d.sum(1).to(x.dtype)
        return out
    y, inverse, weights = st["data"], st["inverse"], st["weights"]
    at, kept = inverse.clamp(min=0).long(), inverse >= 0
    picked = y.float()[at] * kept[..., None]
    out = dict(out=(picked * weights[..., None]).sum(1).to(y.dtype))
    if st["train"]:
        d = st["dout"].float()[:, None, :]
        out["dweights"] = (picked * d).sum(2)
        order, n = st["order"], st["offsets"][-1]
        slot = order.clamp(min=0).long()
        dy = weights.reshape(-1)[slot][:, None] * st["dout"].float()[slot // st["top"]]
        out["drows"] = torch.where((torch.arange(order.numel(), device="cuda") < n)[:, None], dy.to(y.dtype), st["drows_out"])
    return out


# ------------------------------------------------------------------------------------------------
# the framework's calls
# ------------------------------------------------------------------------------------------------
def _own(st):
    from lossless_weight_compression_b200 import wcodec

    op = st["op"]
    if op in ("product", "experts"):
        m = wcodec.Q4Matrix(st["stream"], st["rows"], st["cols"], st["group"], st["zeros"], DT[st["scales"]])
        out = torch.float32 if st["y"] == "fp32" else DT[st["x"]]
        if op == "product":
            return wcodec.gemm_q4(m, st["data"], out_dtype=out)
        return wcodec.gemm_q4_experts(m, st["data"], st["offsets"], out_dtype=out)
    if op == "quantize":
        return wcodec.dequantize_q4(wcodec.quantize_q4(st["data"], st["group"], zeros=st["zeros"]), st["data"].dtype)
    if op == "dispatch":
        plan = wcodec.moe_sort(st["ids"], st["experts"])
        out = dict(rows=wcodec.moe_gather(st["data"], plan, out=st["rows_out"]), offsets=plan.offsets, inverse=plan.inverse)
        if st["train"]:
            out["dx"] = wcodec.moe_gather_backward(st["drows"], plan)
        return out
    plan = wcodec.MoePlan(st["offsets"], st["order"], st["inverse"])
    out = dict(out=wcodec.moe_combine(st["data"], plan, st["weights"]))
    if st["train"]:
        out["drows"], out["dweights"] = wcodec.moe_combine_backward(st["dout"], st["data"], plan, st["weights"], drows=st["drows_out"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    op, g = c["op"], _gen(seed + 2)
    if op in ("product", "experts"):
        E = c.get("experts", 1)
        q, s, z = _codes(c, seed, E)
        col = torch.arange(c["cols"], device="cuda") // c["group"]
        if op == "product":
            x, bounds = _normal(g, (c["tokens"], c["cols"]), DT[c["x"]]), [0, c["tokens"]]
        else:
            ids, _ = _route(c, seed)
            x = _normal(g, (ids.numel(), c["cols"]), DT[c["x"]])
            bounds = [0] + torch.bincount(ids.reshape(-1).long(), minlength=E).cumsum(0).tolist()
        y = torch.empty((x.shape[0], c["rows"]), dtype=torch.float64, device="cuda")
        for e in range(E):
            if bounds[e + 1] > bounds[e]:
                w = q[e].double() - (z[e].double()[:, col] if z is not None else 8.0)
                w *= s[e].double()[:, col]
                y[bounds[e]:bounds[e + 1]] = x[bounds[e]:bounds[e + 1]].double() @ w.T
        return y
    if op == "quantize":
        std = torch.exp(torch.empty((c["rows"], 1), device="cuda").uniform_(-1.0, 1.0, generator=g)) * 0.02
        w = (torch.randn((c["rows"], c["cols"]), generator=g, device="cuda") * std).to(DT[c["dtype"]]).double()
        out = torch.empty_like(w)
        for at in range(0, c["cols"], c["group"]):
            part = w[:, at:at + c["group"]]
            if c["zeros"]:
                lo = torch.minimum(part.min(1, keepdim=True).values, torch.zeros((), device="cuda", dtype=torch.float64))
                hi = torch.maximum(part.max(1, keepdim=True).values, torch.zeros((), device="cuda", dtype=torch.float64))
                s = ((hi - lo) / 15).to(DT[c["dtype"]]).double()
                z = (-lo / s).nan_to_num(0.0).round().clamp(0, 15)
                v = (part / s).nan_to_num(0.0).round() + z
                out[:, at:at + c["group"]] = s * (v.clamp(0, 15) - z)
            else:
                s = (part.abs().max(1, keepdim=True).values / 7).to(DT[c["dtype"]]).double()
                out[:, at:at + c["group"]] = s * (part / s).nan_to_num(0.0).round().clamp(-8, 7)
        return out
    ids, weights = _route(c, seed)
    dt, slots, T, k = DT[c["dtype"]], ids.numel(), c["tokens"], c["top"]
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, c["experts"]), flat)
    ranked = torch.argsort(key, stable=True)
    n = int((flat >= 0).sum())
    ranked = ranked[:n]
    if op == "dispatch":
        x = _normal(g, (T, c["cols"]), dt).double()
        rows = torch.zeros((slots, c["cols"]), dtype=torch.float64, device="cuda")
        rows[:n] = x[ranked // k]
        out = dict(rows=rows, offsets=None, inverse=None)
        if c["train"]:
            d = _normal(g, (slots, c["cols"]), dt).double()
            out["dx"] = torch.zeros((T, c["cols"]), dtype=torch.float64, device="cuda").index_add_(0, ranked // k, d[:n])
        return out
    y = _normal(g, (slots, c["cols"]), dt).double()[:n]
    w = weights.reshape(-1).double()[ranked][:, None]
    out = dict(out=torch.zeros((T, c["cols"]), dtype=torch.float64, device="cuda").index_add_(0, ranked // k, w * y))
    if c["train"]:
        d = _normal(g, (T, c["cols"]), dt).double()[ranked // k]
        dw = torch.zeros(slots, dtype=torch.float64, device="cuda")
        dw[ranked] = (d * y).sum(1)
        drows = torch.zeros((slots, c["cols"]), dtype=torch.float64, device="cuda")
        drows[:n] = w * d
        out["dweights"], out["drows"] = dw.view(T, k), drows
    return out
