"""MXFP4 and routing in 64 bits with numpy, from their definitions (test infrastructure)."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """float64 [M,K] -> (element codes uint8 [M,K], scale codes uint8 [M,K/32])."""
    m, k = x.shape
    v = x.reshape(m, k // 32, 32)
    finite = np.isfinite(v).all(axis=2)
    mag = np.abs(np.where(finite[:, :, None], v, 0.0))
    top = mag.max(axis=2)
    _, e = np.frexp(top)                                   # top = f * 2^e, f in [0.5, 1)
    exponent = np.where(top > 0, np.maximum(e - 3, -127), -127)
    a = np.ldexp(mag, -exponent[:, :, None])
    q = np.zeros(a.shape, dtype=np.uint8)
    for c in range(7):                                     # midpoints: ties go to the even code
        mid = (VALUES[c] + VALUES[c + 1]) / 2
        q += (a > mid) if c % 2 == 0 else (a >= mid)
    q += (8 * np.signbit(v)).astype(np.uint8)
    q[~finite] = 0
    code = np.where(finite, exponent + 127, 255).astype(np.uint8)
    return q.reshape(m, k), code


def pack(q, code):
    """Codes and scales in the library's storage."""
    m, blocks = code.shape
    kb = (blocks + 7) // 8
    s = np.zeros((kb, m, 8), dtype=np.uint8)
    for b in range(blocks):
        s[b // 8, :, b % 8] = code[:, b]
    return q[:, 0::2] | (q[:, 1::2] << 4), s


def unpack(codes, scales):
    """Storage -> (element codes, scale codes)."""
    m, half = codes.shape
    q = np.empty((m, 2 * half), dtype=np.uint8)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    blocks = 2 * half // 32
    code = np.stack([scales[b // 8, :, b % 8] for b in range(blocks)], axis=1)
    return q, code


def values(q, code):
    """The numbers that codes stand for, float64 [M,K]."""
    m, k = q.shape
    v = VALUES[q & 7] * np.where(q & 8, -1.0, 1.0)
    scale = np.where(code == 255, np.nan, np.ldexp(1.0, code.astype(np.int64) - 127))
    return (v.reshape(m, k // 32, 32) * scale[:, :, None]).reshape(m, k)


def sort(ids, experts):
    """(offsets, slot_pos, row_token) of expert ids [T,top]."""
    T, top = ids.shape
    flat = ids.reshape(-1)
    groups = [np.flatnonzero(flat == e) for e in range(experts)]
    dropped = np.flatnonzero((flat < 0) | (flat >= experts))
    order = np.concatenate(groups + [dropped]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(g) for g in groups])]).astype(np.int32)
    row = np.empty(T * top, dtype=np.int64)
    row[order] = np.arange(T * top)
    slot_pos = row.copy()
    slot_pos[dropped] = ~row[dropped]
    row_token = order // top
    row_token[offsets[-1]:] = -1
    return offsets, slot_pos.reshape(T, top).astype(np.int32), row_token.astype(np.int32)


def gather(x, slot_pos):
    T, top = slot_pos.shape
    rows = np.zeros((T * top, x.shape[1]))
    for t in range(T):
        for p in slot_pos[t]:
            if p >= 0:
                rows[p] = x[t]
    return rows


def combine(rows, slot_pos, weights=None):
    """(sums, sums of the magnitudes) per token."""
    T, top = slot_pos.shape
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j, p in enumerate(slot_pos[t]):
            if p >= 0:
                v = rows[p] * (1.0 if weights is None else weights[t, j])
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def combine_backward(d_out, rows, slot_pos, weights):
    """(d_rows, d_weights, sums of the magnitudes in d_weights)."""
    T, top = slot_pos.shape
    d_rows = np.zeros(rows.shape)
    d_w, mag = np.zeros((T, top)), np.zeros((T, top))
    for t in range(T):
        for j, p in enumerate(slot_pos[t]):
            if p >= 0:
                d_rows[p] = weights[t, j] * d_out[t]
                d_w[t, j] = (d_out[t] * rows[p]).sum()
                mag[t, j] = np.abs(d_out[t] * rows[p]).sum()
    return d_rows, d_w, mag


def swiglu(gu):
    gate, up = gu[:, 0::2], gu[:, 1::2]
    with np.errstate(over="ignore"):                        # exp(-gate) = inf: the quotient is -0
        return gate / (1.0 + np.exp(-gate)) * up
