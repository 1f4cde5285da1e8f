"""Plain numpy forms (64 bits) of the 4-bit streams, their products and the
expert routing, written from the definitions in include/wcodec.h."""
import numpy as np

MAGIC = 0x31424357


def groups_of(cols, group):
    return -(-cols // group)


def make(rng, rows, cols, group, zeros, half):
    """Random codes, scales (as float64 values of the 16-bit type) and zero points."""
    g = groups_of(cols, group)
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    s = (rng.uniform(0.5, 1.5, (rows, g)) * 0.01).astype(np.float32)
    if half:
        bits = s.astype(np.float16).view(np.uint16)
    else:
        bits = (s.view(np.uint32) >> 16).astype(np.uint16)
    z = rng.integers(0, 16, (rows, g)).astype(np.uint8) if zeros else None
    return q, bits, z


def scale_values(bits, half):
    if half:
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def weights(q, bits, z, group, half):
    rows, cols = q.shape
    col = np.arange(cols) // group
    zz = z.astype(np.float64)[:, col] if z is not None else 8.0
    return scale_values(bits, half)[:, col] * (q.astype(np.float64) - zz)


def stream(q, bits, z, group, half):
    """The stream's bytes, record by record."""
    rows, cols = q.shape
    g, per = groups_of(cols, group), 128 // group
    blocks, slices = -(-rows // 16), -(-cols // 128)
    out = []
    for first in range(0, blocks, 8):
        for s in range(slices):
            for b in range(first, min(first + 8, blocks)):
                words = np.zeros((4, 16, 4), np.uint32)
                sc, zp = np.zeros((per, 16), np.uint16), np.zeros((per, 16), np.uint8)
                for r in range(16):
                    row = 16 * b + r
                    for k in range(per):
                        gg = s * per + k
                        if row < rows and gg < g:
                            sc[k, r] = bits[row, gg]
                            if z is not None:
                                zp[k, r] = z[row, gg]
                    for c in range(128):
                        col = 128 * s + c
                        code = (zp[c // group, r] if z is not None else 8)
                        if row < rows and col < cols:
                            code = q[row, col]
                        i, t, e = c // 32, c % 32 // 8, c % 8
                        words[t, r, i] |= np.uint32(int(code) << (4 * ((e >> 1) + 4 * (e & 1))))
                rec = words.tobytes() + sc.tobytes()
                if z is not None:
                    rec += zp.tobytes() + b"\0" * (-(16 * per) % 32)
                out.append(rec)
    body = b"".join(out)
    flags = 8 | (16 if z is not None else 0) | (32 if half else 0)
    head = bytearray(128)
    for at, size, v in ((0, 4, MAGIC), (4, 2, 1), (6, 2, 128), (8, 4, group), (12, 4, flags),
                        (16, 8, rows * cols), (24, 8, rows * g), (32, 8, 128), (64, 8, len(body)),
                        (72, 8, 128 + len(body)), (88, 4, rows), (92, 4, cols)):
        head[at:at + size] = int(v).to_bytes(size, "little")
    return np.frombuffer(bytes(head) + body, np.uint8)


def sort(ids, experts):
    """offsets, order, inverse of (tokens, top) ids."""
    flat = ids.reshape(-1)
    order, offsets = [], [0]
    for e in range(experts):
        order += list(np.nonzero(flat == e)[0])
        offsets.append(len(order))
    inverse = np.full(flat.size, -1, np.int32)
    inverse[order] = np.arange(len(order))
    order = np.array(order + [-1] * (flat.size - len(order)), np.int32)
    return np.array(offsets, np.int32), order, inverse.reshape(ids.shape)
