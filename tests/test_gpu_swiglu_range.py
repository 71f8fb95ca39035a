"""SwiGLU where the sigmoid leaves fp32's normal range: gates far below zero, ups far above one."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from quantized_gemm_quantize_amd import binding as b
from test_gpu_mxfp4 import DEV

pytestmark = pytest.mark.gpu


def gate_row(value, k):
    """Elements 6, ..., 6, the rest, 0.5 whose sum is `value` (a multiple of 0.5): k signed codes."""
    row, left, codes = np.zeros(k, dtype=np.uint8), abs(value), [(6.0, 7), (4.0, 6), (3.0, 5), (2.0, 4), (1.0, 2), (0.5, 1)]
    i = 0
    for step, code in codes:
        while left >= step:
            row[i], left, i = code, left - step, i + 1
    assert left == 0
    return row | (8 if value < 0 else 0)


def check_within(hq, hs, h, slack):
    """MXFP4 rows of values known within `slack`, which may be as large as they are: every block's scale
    lies between those of the least and the largest top, every element is the rounding of a value within
    the slack. Blocks with a value past fp32's range are NaN."""
    q, code = ref.unpack(hq.cpu().numpy(), hs.cpu().numpy())
    m, f = h.shape
    over = (np.abs(h).reshape(m, f // 32, 32) > np.finfo(np.float32).max).any(axis=2)
    assert np.array_equal(code == 255, over)
    each = np.repeat(over, 32, axis=1)
    q, code, h = np.where(each, 0, q), np.where(over, 0, code), np.where(each, 0.0, h)
    top, wide = (v.reshape(m, f // 32, 32).max(axis=2) for v in (np.abs(h), slack))
    low, high = (ref.quantize(np.repeat(t, 32, axis=1))[1] for t in (np.maximum(top - wide, 0), top + wide))
    assert ((code >= low) & (code <= high)).all()
    scale = np.ldexp(1.0, np.repeat(code.astype(np.int64), 32, axis=1) - 127)
    idx = q & 7
    lo = np.where(idx == 0, -1.0, (ref.VALUES[idx] + ref.VALUES[np.maximum(idx, 1) - 1]) / 2)
    hi = np.where(idx == 7, 1e30, (ref.VALUES[idx] + ref.VALUES[np.minimum(idx + 1, 7)]) / 2)
    a, s = np.abs(h) / scale, slack / scale
    assert ((a >= lo - s) & (a <= hi + s)).all()
    sign = np.where(q & 8, -1, 1)
    assert (np.sign(h) * sign >= 0)[(idx > 0) & (np.abs(h) > slack)].all()


@pytest.mark.parametrize("rows,lift", [(3, 100), (40, 100), (300, 100), (3, 0), (3, 120)])
def test_gates_far_below_zero(rows, lift):
    """gate / (1 + exp(-gate)) * up for gates of -80 to -104 and 80 to 104 and ups of 2^lift times 0.5 to
    6, one block of 32 units per gate. The sigmoid is held in fp32: below 2^-126 to half a step of
    2^-149; the exponential's argument rounds to 2^-24 of at most 150 (2^-16.7 of its value), the other
    steps to 2^-21 together."""
    gates = np.concatenate([-np.arange(80.0, 104.5, 0.5), np.arange(80.0, 104.5, 8.0)])
    F, K = 32 * len(gates), 64
    q, code = np.zeros((2 * F, K), dtype=np.uint8), np.full((2 * F, 2), 127, dtype=np.uint8)
    q[0::2] = np.repeat(np.stack([gate_row(g, K) for g in gates]), 32, axis=0)
    q[1::2, 0] = np.tile(np.array([1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 12, 13, 14, 15, 2, 4], dtype=np.uint8), F // 16)
    code[1::2] = 127 + lift
    w = ref.pack(q, code)
    x = ref.pack(np.full((rows, K), 2, dtype=np.uint8), np.full((rows, 2), 127, dtype=np.uint8))
    hq, hs = b.mxfp4_expert_swiglu(*[torch.from_numpy(t).to(DEV) for t in x],
                                   torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                                   torch.from_numpy(w[0][None]).to(DEV), torch.from_numpy(w[1][None]).to(DEV))
    gu = np.ones((rows, K)) @ ref.values(q, code).T
    h = ref.swiglu(gu)
    slack = np.abs(h) * 2.0 ** -16 + np.abs(gu[:, 0::2]) * 2.0 ** -150 * np.abs(gu[:, 1::2]) + 2.0 ** -149
    check_within(hq, hs, h, slack)
